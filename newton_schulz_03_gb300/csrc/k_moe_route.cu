// k_moe_route.cu -- routing of tokens to experts, forward and backward.
//
// Forward, per token with logits x: scores s = sigmoid(x) or softmax(x); the
// choice value of expert e is c_e = s_e + bias_e (softmax without a bias: x_e,
// which orders the experts the same way without rounding); with groups only
// the experts of the best groups stay; the k largest c are taken, ties to the
// lowest index; w_j = scale s_j, divided by the chosen scores' sum where
// asked.  The bias chooses, it does not weigh.
// Backward: with g the gradient of w and w the weights over `scale`,
//   sigmoid          dx_j = scale g_j s_j (1 - s_j)
//   sigmoid, renorm  dx_j = scale w_j (g_j - sum_i g_i w_i) (1 - s_j)
//   softmax          dx_e = s_e (scale g_e - sum_i scale g_i s_i), every open e
//   softmax, renorm  dx_j = scale w_j (g_j - sum_i g_i w_i)
// Scores are recomputed from the logits: they cost a few instructions, storing
// them would cost a write and a read of tokens x experts.
//
// One warp holds one token's logits in registers.  The logits are read once and
// their gradient written once.  Measured: 16384 x 512 FP32 softmax 12 us forward,
// 13 us backward (floors 5 and 10); 65531 x 512 BF16 sigmoid with 16 groups 77 and
// 21 us (floors 10 and 11); one token 2.7 us.  What holds them: forward, the
// instructions of a warp per token (620 softmax, 1200 with groups: a look at every
// value, then the few candidates) and their latencies, issue slots 67% and 81%
// busy; backward, one chain of dependent loads per token (ids, logits, score,
// store), slots 60% busy, most stalls on those loads; one token, latency.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <cstdint>

#include "kernels.h"
#include "launch.cuh"
#include "moe.h"

namespace muon {
namespace {

constexpr int kWarps = 4;                 // tokens per block
constexpr uint32_t kAll = 0xffffffffu;

template <typename T>
struct Elem;
template <>
struct Elem<float> {
  static __device__ __forceinline__ float load(const float* p) { return *p; }
  static __device__ __forceinline__ void load4(const float* p, float (&v)[4]) {
    const float4 u = *reinterpret_cast<const float4*>(p);
    v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
  }
  static __device__ __forceinline__ void store(float* p, float v) { *p = v; }
  static __device__ __forceinline__ void store4(float* p, const float (&v)[4]) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  }
};
template <>
struct Elem<__nv_bfloat16> {
  static __device__ __forceinline__ float load(const __nv_bfloat16* p) { return __bfloat162float(*p); }
  static __device__ __forceinline__ void load4(const __nv_bfloat16* p, float (&v)[4]) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    v[0] = __uint_as_float(u.x << 16); v[1] = __uint_as_float(u.x & 0xffff0000u);
    v[2] = __uint_as_float(u.y << 16); v[3] = __uint_as_float(u.y & 0xffff0000u);
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
  static __device__ __forceinline__ void store4(__nv_bfloat16* p, const float (&v)[4]) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
    uint2 u;
    u.x = *reinterpret_cast<const uint32_t*>(&a);
    u.y = *reinterpret_cast<const uint32_t*>(&b);
    *reinterpret_cast<uint2*>(p) = u;
  }
};

// Largest of the warp's values (a NaN does not take part).
__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

// 1 / (1 + exp(-x)), each operation rounded to FP32.
__device__ __forceinline__ float sigmoid(float x) { return __frcp_rn(1.0f + expf(-x)); }

// The same within 4e-7, in four instructions: for telling which experts cannot
// be among the chosen.  (The exponential's argument is rounded once, |x| 6e-8 of
// it, which the sigmoid's slope s (1 - s) takes below 2e-8; the two approximate
// instructions and the sum are within 2^-22 each.)
__device__ __forceinline__ float sigmoid_near(float x) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * -1.442695041f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return r;
}

__device__ __forceinline__ bool is_open(float x) { return fabsf(x) <= FLT_MAX; }

// Expert of register r of a lane: V neighbours per lane and vector.
template <int V>
__device__ __forceinline__ int expert_of(int r, int lane) {
  return ((r / V) * 32 + lane) * V + (r % V);
}

// Logits of one token; experts past the end read as closed.
template <typename T, int V, int R>
__device__ __forceinline__ void load_row(const T* row, int experts, int lane, float (&x)[R]) {
#pragma unroll
  for (int r = 0; r < R; r += V) {
    const int e = expert_of<V>(r, lane);
    if (V == 4) {
      float v[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
      if (e < experts) Elem<T>::load4(row + e, v);
#pragma unroll
      for (int q = 0; q < 4; ++q) x[(r + q) % R] = v[q];
    } else {
      x[r] = e < experts ? Elem<T>::load(row + e) : -INFINITY;
    }
  }
}

// Lane of the warp's largest value, the first of equal ones; -1 when all are
// -inf.  `top` receives the value.
__device__ __forceinline__ int warp_best_lane(float v, float& top) {
  top = warp_max(v);
  if (!(top > -INFINITY)) return -1;
  return __ffs(__ballot_sync(kAll, v == top)) - 1;
}

// Value of a group from its best two choice values (-inf: closed).
__device__ __forceinline__ float group_value(float first, float second, int group_top) {
  return group_top == 2 && second > -INFINITY ? first + second : first;
}

// Groups of `lanes` = 1, 2, 4 .. 32 neighbouring lanes of a vector of 128
// experts: the best two by a butterfly, then every group's value to its lane.
template <int R>
__device__ __forceinline__ float group_values_by_lanes(const float (&c)[R], int lanes, int groups,
                                                       int group_top, int lane) {
  const int per_vector = 32 / lanes;              // groups in one vector
  float mine = -INFINITY;
#pragma unroll
  for (int i = 0; i < R / 4; ++i) {
    if (i * per_vector >= groups) break;
    const float hi0 = fmaxf(c[4 * i], c[4 * i + 1]), lo0 = fminf(c[4 * i], c[4 * i + 1]);
    const float hi1 = fmaxf(c[4 * i + 2], c[4 * i + 3]), lo1 = fminf(c[4 * i + 2], c[4 * i + 3]);
    float first = fmaxf(hi0, hi1);
    float second = fmaxf(fminf(hi0, hi1), hi0 > hi1 ? lo0 : lo1);
    for (int o = 1; o < lanes; o <<= 1) {
      const float f = __shfl_xor_sync(kAll, first, o), q = __shfl_xor_sync(kAll, second, o);
      second = fmaxf(fminf(first, f), fmaxf(second, q));
      first = fmaxf(first, f);
    }
    const float g = __shfl_sync(kAll, group_value(first, second, group_top), (lane % per_vector) * lanes);
    if (lane / per_vector == i) mine = g;
  }
  return lane < groups ? mine : -INFINITY;
}

// Any group size: lane g walks group g in shared memory, each lane starting
// elsewhere (distinct banks).
__device__ __forceinline__ float group_values_by_walk(const float* values, int size, int groups,
                                                      int group_top, int lane) {
  if (lane >= groups) return -INFINITY;
  float first = -INFINITY, second = -INFINITY;
  int j = lane % size;
  for (int i = 0; i < size; ++i) {
    const float v = values[lane * size + j];
    second = fmaxf(second, fminf(first, v));
    first = fmaxf(first, v);
    if (++j == size) j = 0;
  }
  return group_value(first, second, group_top);
}

// A token's routing state that does not depend on the expert.
struct Row {
  const void* logits;
  const float* bias;
  float top, denom;      // softmax
  bool by_logit;
};

// Choice value of one expert from its logit, in FP32 as written.
template <bool SOFTMAX>
__device__ __forceinline__ float choice_value(const Row& w, float x, int e) {
  if (w.by_logit) return x;
  const float s = SOFTMAX ? expf(x - w.top) / w.denom : sigmoid(x);
  return w.bias != nullptr ? s + w.bias[e] : s;
}

struct Choice {
  int id;                // -1: none
  float x;               // its logit
};

// A candidate's choice value and expert as one ordered number: the larger
// value, of equal ones the lower expert.  0 is below every one.
using Candidate = unsigned long long;
__device__ __forceinline__ Candidate candidate(float c, int e) {
  const uint32_t u = __float_as_uint(c + 0.0f);   // -0 ties with +0
  const uint32_t ordered = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
  return (static_cast<unsigned long long>(ordered) << 32) | static_cast<uint32_t>(~e);
}

// The k best of the lanes' values, ties to the lowest expert: the j-th one in
// lane j.  near: the values are within the tolerance of the choice values only.
// The k-th largest of the lanes' maxima bounds the k-th largest value from
// below, so only the few values that reach it (less the tolerance, twice) can be
// chosen; they are gathered one per lane, valued exactly and ranked by counting.
// false: more than 32 reach it.
template <typename T, int R, bool SOFTMAX, typename ExpertOf>
__device__ __forceinline__ bool choose(const Row& w, const float (&c)[R], ExpertOf expert, bool near,
                                       int k, int lane, Candidate* list, Choice& out) {
  float most = c[0];
#pragma unroll
  for (int r = 1; r < R; ++r) most = fmaxf(most, c[r]);
  float bound = -FLT_MAX, left = most;
  for (int got = 0; got < k;) {
    const float top = warp_max(left);
    if (!(top > -INFINITY)) {
      bound = -FLT_MAX;
      break;
    }
    bound = top;
    const bool is_top = left == top;
    got += __popc(__ballot_sync(kAll, is_top));
    if (is_top) left = -INFINITY;
  }
  if (near && bound > -FLT_MAX) {
    bound -= 2e-6f + 1e-6f * fabsf(bound);
    if (!(bound > -FLT_MAX)) return false;        // biases beyond any sense
  }
  uint32_t reach = 0u;
#pragma unroll
  for (int r = 0; r < R; ++r) reach |= c[r] >= bound ? 1u << r : 0u;
  int end = __popc(reach);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(kAll, end, o);
    if (lane >= o) end += v;
  }
  const int total = __shfl_sync(kAll, end, 31);
  if (total > 32) return false;
  int* experts = reinterpret_cast<int*>(list);
  for (int at = end - __popc(reach); reach != 0u; reach &= reach - 1u, ++at)
    experts[at] = expert(__ffs(reach) - 1);
  __syncwarp();
  int e = 0;
  float x = 0.f;
  Candidate own = 0ull;
  if (lane < total) {
    e = experts[lane];
    x = Elem<T>::load(static_cast<const T*>(w.logits) + e);
    own = candidate(choice_value<SOFTMAX>(w, x, e), e);
  }
  __syncwarp();
  list[lane] = own;
  __syncwarp();
  int rank = 0;
  for (int j = 0; j < total; j += 4) {            // past the end: zeros
    const ulonglong2 p = *reinterpret_cast<const ulonglong2*>(list + j);
    const ulonglong2 q = *reinterpret_cast<const ulonglong2*>(list + j + 2);
    rank += (p.x > own ? 1 : 0) + (p.y > own ? 1 : 0) + (q.x > own ? 1 : 0) + (q.y > own ? 1 : 0);
  }
  __syncwarp();
  float2* place = reinterpret_cast<float2*>(list);
  if (lane < total) place[rank] = make_float2(x, __int_as_float(e));   // ranks are distinct
  __syncwarp();
  out.id = -1;
  if (lane < min(k, total)) {
    const float2 v = place[lane];
    out.x = v.x;
    out.id = __float_as_int(v.y);
  }
  return true;
}

// The same by k rounds of the warp's best, for rows with many equal values;
// c holds the exact choice values.
template <typename T, int R, typename ExpertOf>
__device__ __forceinline__ void choose_by_rounds(const Row& w, float (&c)[R], ExpertOf expert, int k,
                                                 int lane, Choice& out) {
  out.id = -1;
  for (int j = 0; j < k; ++j) {
    float best = -INFINITY;
    int e = INT32_MAX;
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (c[r] > best) {                          // a lane's experts are in order
        best = c[r];
        e = expert(r);
      }
    const float top = warp_max(best);
    if (!(top > -INFINITY)) break;
    e = __reduce_min_sync(kAll, best == top ? e : INT32_MAX);
    if (lane == j) out.id = e;
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (expert(r) == e) c[r] = -INFINITY;
  }
  if (out.id >= 0) out.x = Elem<T>::load(static_cast<const T*>(w.logits) + out.id);
}

// Either way; false: not certain from near values.
template <typename T, int R, bool SOFTMAX, typename ExpertOf>
__device__ __forceinline__ bool choose_any(const Row& w, float (&c)[R], ExpertOf expert, bool near,
                                           int k, int lane, Candidate* list, Choice& out) {
  if (choose<T, R, SOFTMAX>(w, c, expert, near, k, lane, list, out)) return true;
  if (near) return false;
  choose_by_rounds<T, R>(w, c, expert, k, lane, out);
  return true;
}

// Among the n experts of the listed groups (n <= 32 R), in order over the lanes.
template <typename T, int R, bool SOFTMAX>
__device__ __forceinline__ bool choose_of(const Row& w, const float* values, const int* groups,
                                          int size, uint32_t per_group, int n, bool near, int k,
                                          int lane, Candidate* list, Choice& out) {
  float c[R];
  const auto expert = [&](int r) {
    const int i = r * 32 + lane;
    const int g = per_group == 0u ? i : static_cast<int>(__umulhi(i, per_group));
    return i < n ? groups[g] * size + (i - g * size) : INT32_MAX;
  };
#pragma unroll
  for (int r = 0; r < R; ++r) {
    c[r] = -INFINITY;
    if (r * 32 + lane < n) c[r] = values[expert(r)];
  }
  return choose_any<T, R, SOFTMAX>(w, c, expert, near, k, lane, list, out);
}

// Shared memory of one warp's token.
struct Scratch {
  Candidate* list;       // [32]
  int* groups;           // [kMoeMaxGroups]
  float* values;         // [experts], with groups
};

// One token's choice.  NEAR: from near sigmoids (false: they do not settle it).
template <typename T, int V, int R, bool SOFTMAX, bool GROUPS, bool NEAR>
__device__ __forceinline__ bool route_row(const RouteArgs& a, Row& w, int lane, const Scratch& sc,
                                          Choice& mine) {
  float c[R];
  load_row<T, V, R>(static_cast<const T*>(w.logits), a.experts, lane, c);
  // Whether every logit (and bias) is finite: v * 0 is NaN otherwise.
  const bool whole = a.experts == 32 * R;
  float z = 0.f;
#pragma unroll
  for (int r = 0; r < R; ++r)
    if (whole || expert_of<V>(r, lane) < a.experts) z = fmaf(c[r], 0.f, z);
  uint32_t closed = 0u;                           // registers of closed experts
  if (!__all_sync(kAll, z == 0.f) || !whole) {
    bool bad = false;
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (!is_open(c[r])) {
        bad = bad || !(c[r] < 0.f);               // NaN or +inf: closed, and reported
        c[r] = -INFINITY;
        closed |= 1u << r;
      }
    if (bad) atomicOr(a.err, kDevErrInput);
  }
  if (SOFTMAX) {
    // Statistics over the open experts: a closed one's exp is 0.
    w.top = -FLT_MAX;
    w.denom = 0.f;
    if (!(w.by_logit && a.renorm)) {
#pragma unroll
      for (int r = 0; r < R; ++r) w.top = fmaxf(w.top, c[r]);
      w.top = warp_max(w.top);
#pragma unroll
      for (int r = 0; r < R; ++r) w.denom += expf(c[r] - w.top);
      w.denom = warp_sum(w.denom);
    }
    if (!w.by_logit) {
#pragma unroll
      for (int r = 0; r < R; ++r) c[r] = expf(c[r] - w.top) / w.denom;
    }
  } else {
#pragma unroll
    for (int r = 0; r < R; ++r) c[r] = NEAR ? sigmoid_near(c[r]) : sigmoid(c[r]);
  }
  if (a.bias != nullptr) {
    float b[R];
    load_row<float, V, R>(a.bias, a.experts, lane, b);
    z = 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (whole || expert_of<V>(r, lane) < a.experts) z = fmaf(b[r], 0.f, z);
      c[r] += b[r];
    }
    if (!__all_sync(kAll, z == 0.f)) {            // a NaN bias closes
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (c[r] != c[r]) closed |= 1u << r;
    }
  }
  if (__any_sync(kAll, closed != 0u)) {
#pragma unroll
    for (int r = 0; r < R; ++r)
      if ((closed >> r) & 1u) c[r] = -INFINITY;
  }

  if constexpr (!GROUPS) {
    const auto expert = [&](int r) { return expert_of<V>(r, lane); };
    return choose_any<T, R, SOFTMAX>(w, c, expert, NEAR, a.k, lane, sc.list, mine);
  } else {
#pragma unroll
    for (int r = 0; r < R; r += V) {
      const int e = expert_of<V>(r, lane);
      if (e >= a.experts) continue;
      if (V == 4)
        *reinterpret_cast<float4*>(sc.values + e) =
            make_float4(c[r], c[(r + 1) % R], c[(r + 2) % R], c[(r + 3) % R]);
      else
        sc.values[e] = c[r];
    }
    __syncwarp();
    const int size = a.group_size;
    const int lanes = size / 4;                     // of a group within a vector
    float gv;
    if (V == 4 && size % 4 == 0 && lanes <= 32 && (lanes & (lanes - 1)) == 0)
      gv = group_values_by_lanes<R>(c, lanes, a.groups, a.group_top, lane);
    else
      gv = group_values_by_walk(sc.values, size, a.groups, a.group_top, lane);
    uint32_t stay = 0u;
    float last = INFINITY;
    for (int i = 0; i < a.top_groups; ++i) {
      float v;
      const int g = warp_best_lane(gv, v);
      if (g < 0) break;
      last = v;
      stay |= 1u << g;
      if (lane == g) gv = -INFINITY;
    }
    // Near values settle the groups when the next one is well below: two values
    // of each are off by the tolerance.
    if (NEAR) {
      const float next = warp_max(gv);
      if (next > -INFINITY && !(last - next > 8e-6f + 4e-6f * fabsf(last))) return false;
    }
    if ((stay >> lane) & 1u) sc.groups[__popc(stay & ((1u << lane) - 1u))] = lane;
    __syncwarp();
    const int n = __popc(stay) * size;
    if (n <= 8 * R)
      return choose_of<T, R / 4, SOFTMAX>(w, sc.values, sc.groups, size, a.per_group, n, NEAR, a.k,
                                          lane, sc.list, mine);
    return choose_of<T, R, SOFTMAX>(w, sc.values, sc.groups, size, a.per_group, n, NEAR, a.k, lane,
                                    sc.list, mine);
  }
}

// The exact second look at a token, rarely taken: out of line.
template <typename T, int V, int R, bool GROUPS>
__device__ __noinline__ Choice route_row_again(const RouteArgs& a, Row w, int lane, Scratch sc) {
  Choice mine;
  __syncwarp();
  route_row<T, V, R, false, GROUPS, false>(a, w, lane, sc, mine);
  return mine;
}

template <typename T, int V, int R, bool SOFTMAX, bool GROUPS>
__global__ void __launch_bounds__(kWarps * 32, R <= 16 ? 8 : 4)
    route_kernel(const __grid_constant__ RouteArgs a) {
  extern __shared__ float smem_values[];
  __shared__ __align__(16) Candidate lists[kWarps][32];
  __shared__ int group_list[kWarps][kMoeMaxGroups];
  grid_dep_wait();
  grid_dep_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  if (t >= a.tokens) return;
  int32_t* ids = a.ids + t * a.k;
  float* weights = a.weights + t * a.k;
  if (a.mask != nullptr && a.mask[t] == 0) {
    if (lane < a.k) {
      ids[lane] = -1;
      weights[lane] = 0.f;
    }
    return;
  }
  Row w;
  w.logits = static_cast<const T*>(a.logits) + t * a.experts;
  w.bias = a.bias;
  w.by_logit = SOFTMAX && a.bias == nullptr && a.group_top == 1;
  const Scratch sc{lists[warp], group_list[warp], smem_values + (GROUPS ? warp * a.experts : 0)};
  // Sigmoids are first taken near: hundreds of them written out in FP32 cost
  // more than all the rest, and only the chosen ones' last bits matter.
  Choice mine;
  if (!route_row<T, V, R, SOFTMAX, GROUPS, !SOFTMAX>(a, w, lane, sc, mine))
    mine = route_row_again<T, V, R, GROUPS>(a, w, lane, sc);
  const int my_id = mine.id;
  const float top = w.top, denom = w.denom;

  // Lane j holds the j-th choice.
  float s = 0.f;
  const float xj = my_id >= 0 ? mine.x : -INFINITY;
  if (SOFTMAX && a.renorm) {
    float m = xj;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
    s = my_id >= 0 ? expf(xj - m) : 0.f;
  } else if (my_id >= 0) {
    s = SOFTMAX ? expf(xj - top) / denom : sigmoid(xj);
  }
  float share = s;
  if (a.renorm) {
    const float sum = warp_sum(s);
    share = sum > 0.f ? s / sum : 0.f;   // every chosen score underflowed: no weight
  }
  if (lane < a.k) {
    ids[lane] = my_id;
    weights[lane] = share * a.scale;
  }
}

template <typename T, int V, int R>
__global__ void __launch_bounds__(kWarps * 32) route_backward_kernel(const RouteArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  if (t >= a.tokens) return;
  const T* row = static_cast<const T*>(a.logits) + t * a.experts;
  T* out = static_cast<T*>(a.grad_logits) + t * a.experts;

  int id = -1;
  float g = 0.f, xj = -INFINITY;
  if (lane < a.k) {
    id = a.ids[t * a.k + lane];
    if (id >= a.experts || id < -1) {
      atomicOr(a.err, kDevErrIndex);
      id = -1;
    }
    if (id >= 0) {
      g = a.grad[t * a.k + lane] * a.scale;
      xj = Elem<T>::load(row + id);
      if (!is_open(xj)) id = -1;         // a closed expert has no gradient
    }
    if (id < 0) g = 0.f;
  }

  float dx = 0.f;                        // gradient at this lane's choice
  if (a.softmax && !a.renorm) {
    float x[R];
    load_row<T, V, R>(row, a.experts, lane, x);
    float top = -INFINITY, denom = 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (!is_open(x[r])) x[r] = -INFINITY;
      top = fmaxf(top, x[r]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
#pragma unroll
    for (int r = 0; r < R; ++r) {
      x[r] = x[r] > -INFINITY ? expf(x[r] - top) : 0.f;
      denom += x[r];
    }
    denom = warp_sum(denom);
    const float pj = id >= 0 ? expf(xj - top) / denom : 0.f;
    const float dot = warp_sum(id >= 0 ? g * pj : 0.f);
    const float c = denom > 0.f && dot != 0.f ? -dot / denom : 0.f;
#pragma unroll
    for (int r = 0; r < R; r += V) {
      const int e = expert_of<V>(r, lane);
      if (e >= a.experts) continue;
      if (V == 4) {
        float v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = x[(r + q) % R] * c;
        Elem<T>::store4(out + e, v);
      } else {
        Elem<T>::store(out + e, x[r] * c);
      }
    }
    dx = pj * (g - dot);
  } else {
#pragma unroll
    for (int r = 0; r < R; r += V) {
      const int e = expert_of<V>(r, lane);
      if (e >= a.experts) continue;
      if (V == 4) {
        const float v[4] = {0.f, 0.f, 0.f, 0.f};
        Elem<T>::store4(out + e, v);
      } else {
        Elem<T>::store(out + e, 0.f);
      }
    }
    if (a.softmax) {
      float m = id >= 0 ? xj : -INFINITY;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
      float w = id >= 0 ? expf(xj - m) : 0.f;
      const float sum = warp_sum(w);
      w = sum > 0.f ? w / sum : 0.f;
      const float dot = warp_sum(id >= 0 ? g * w : 0.f);
      dx = w * (g - dot);
    } else {
      // 1 - s as sigmoid(-x): no cancellation for large x.
      const float s = id >= 0 ? sigmoid(xj) : 0.f;
      const float rest = id >= 0 ? sigmoid(-xj) : 0.f;
      if (a.renorm) {
        // Through the weights: a single choice's is exactly 1, and its
        // gradient exactly 0.  They are at most 1 where the scores' sum is
        // next to nothing: no quotient by it, which could overflow.
        const float sum = warp_sum(s);
        const float share = sum > 0.f ? s / sum : 0.f;
        const float dot = warp_sum(id >= 0 ? g * share : 0.f);
        dx = share * (g - dot) * rest;
      } else {
        dx = g * (s * rest);
      }
    }
  }
  // The row's other values are written above by other lanes of this warp:
  // the choices' follow them.
  __syncwarp();
  if (id >= 0) Elem<T>::store(out + id, dx);
}

template <typename T, int V, int R>
cudaError_t launch_rv(const RouteArgs& a, bool backward, cudaStream_t s) {
  const int64_t blocks = (a.tokens + kWarps - 1) / kWarps;
  const dim3 grid(static_cast<unsigned>(blocks)), block(kWarps * 32);
  if (backward) return launch_pdl(route_backward_kernel<T, V, R>, grid, block, 0, s, a);
  if (a.groups > 1) {
    const size_t smem = size_t(kWarps) * a.experts * 4;
    return launch_pdl(a.softmax ? route_kernel<T, V, R, true, true> : route_kernel<T, V, R, false, true>,
                      grid, block, smem, s, a);
  }
  return launch_pdl(a.softmax ? route_kernel<T, V, R, true, false> : route_kernel<T, V, R, false, false>,
                    grid, block, 0, s, a);
}

// Registers per lane: 4, 16 or 32, the least that holds the row.  Rows of a
// multiple of four experts are read four at a time.
template <typename T>
cudaError_t launch_t(const RouteArgs& a, bool backward, cudaStream_t s) {
  const int per = (a.experts + 31) / 32;
  if (a.experts % 4 == 0) {
    if (per <= 4) return launch_rv<T, 4, 4>(a, backward, s);
    if (per <= 16) return launch_rv<T, 4, 16>(a, backward, s);
    return launch_rv<T, 4, 32>(a, backward, s);
  }
  if (per <= 4) return launch_rv<T, 1, 4>(a, backward, s);
  return launch_rv<T, 1, 32>(a, backward, s);
}

}  // namespace

cudaError_t launch_moe_route(const RouteArgs& a, bool bf16, cudaStream_t s) {
  return bf16 ? launch_t<__nv_bfloat16>(a, false, s) : launch_t<float>(a, false, s);
}

cudaError_t launch_moe_route_backward(const RouteArgs& a, bool bf16, cudaStream_t s) {
  return bf16 ? launch_t<__nv_bfloat16>(a, true, s) : launch_t<float>(a, true, s);
}

}  // namespace muon
