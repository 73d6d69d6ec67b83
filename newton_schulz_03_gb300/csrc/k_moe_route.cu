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
//   sigmoid, renorm  dx_j = scale (g_j - sum_i g_i w_i) / S  s_j (1 - s_j)
//   softmax          dx_e = s_e (scale g_e - sum_i scale g_i s_i), every open e
//   softmax, renorm  dx_j = scale w_j (g_j - sum_i g_i w_i)
// Scores are recomputed from the logits: they cost a few instructions, storing
// them would cost a write and a read of tokens x experts.
//
// One warp holds one token's logits in registers.  Bound: the logits are read
// once (and their gradient written once), against k rounds of a warp-wide
// maximum, so memory for large batches and latency for one token.
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

// A number that orders as the float does; 0 (below every finite one) stands
// for a closed expert.  -0 is made +0 first, so that the two tie.
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

// 1 / (1 + exp(-x)), each operation rounded to FP32.
__device__ __forceinline__ float sigmoid(float x) { return __frcp_rn(1.0f + expf(-x)); }

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

// The warp's best (key, expert) given each lane's best; ties: lowest expert.
__device__ __forceinline__ void warp_best(uint32_t& key, int& e) {
  const uint32_t top = __reduce_max_sync(kAll, key);
  e = __reduce_min_sync(kAll, key == top ? e : INT32_MAX);
  key = top;
}

// Values of the groups, group g's in lane g: the ordered sum of its best
// group_top open experts' choice values, 0 where none is open.
__device__ __forceinline__ uint32_t group_key(uint32_t first, uint32_t second, int group_top) {
  if (first == 0u) return 0u;
  const float f = unordered(first);
  return ordered(group_top == 2 && second != 0u ? f + unordered(second) : f);
}

// Groups of `lanes` = 1, 2, 4 .. 32 neighbouring lanes of a vector: the best
// two by a butterfly, then every group's key to its lane.
template <int R>
__device__ __forceinline__ uint32_t group_keys_by_lanes(const uint32_t (&key)[R], int lanes,
                                                        int groups, int group_top, int lane) {
  const int per_vector = 32 / lanes;              // groups in one vector of 128 experts
  uint32_t mine = 0u;
#pragma unroll
  for (int i = 0; i < R / 4; ++i) {
    if (i * per_vector >= groups) break;
    const uint32_t a = key[4 * i], b = key[4 * i + 1], c = key[4 * i + 2], d = key[4 * i + 3];
    const uint32_t hi0 = max(a, b), lo0 = min(a, b), hi1 = max(c, d), lo1 = min(c, d);
    uint32_t first = max(hi0, hi1);
    uint32_t second = max(min(hi0, hi1), hi0 > hi1 ? lo0 : lo1);
    for (int o = 1; o < lanes; o <<= 1) {
      const uint32_t f = __shfl_xor_sync(kAll, first, o), q = __shfl_xor_sync(kAll, second, o);
      second = max(min(first, f), max(second, q));
      first = max(first, f);
    }
    const uint32_t g = __shfl_sync(kAll, group_key(first, second, group_top),
                                   (lane % per_vector) * lanes);
    if (lane / per_vector == i) mine = g;
  }
  return lane < groups ? mine : 0u;
}

// Any group size: lane g walks group g in shared memory, each lane starting
// elsewhere (distinct banks).
__device__ __forceinline__ uint32_t group_keys_by_walk(const uint32_t* keys, int size, int groups,
                                                       int group_top, int lane) {
  if (lane >= groups) return 0u;
  uint32_t first = 0u, second = 0u;
  int j = lane % size;
  for (int i = 0; i < size; ++i) {
    const uint32_t v = keys[lane * size + j];
    second = max(second, min(first, v));
    first = max(first, v);
    if (++j == size) j = 0;
  }
  return group_key(first, second, group_top);
}

// The k largest of the lanes' keys over the warp, ties to the lowest expert;
// returns the j-th one's expert in lane j (-1: fewer than k are open).  A
// lane's keys lie in order of expert.  The k-th largest of the lanes' maxima is
// a lower bound of the k-th largest key: only the few keys that reach it are
// gathered, one per lane, and ranked by counting.
template <int R>
__device__ __forceinline__ int choose(uint32_t (&key)[R], const int (&expert)[R], int k, int lane,
                                      uint2* list) {
  uint32_t most = 0u;
#pragma unroll
  for (int r = 0; r < R; ++r) most = max(most, key[r]);
  uint32_t bound = 1u, left = most;               // no closed expert reaches 1
  for (int got = 0; got < k;) {
    const uint32_t top = __reduce_max_sync(kAll, left);
    if (top == 0u) {
      bound = 1u;
      break;
    }
    bound = top;
    const bool is_top = left == top;
    got += __popc(__ballot_sync(kAll, is_top));
    if (is_top) left = 0u;
  }
  // Places of this lane's candidates.
  int mine = 0;
#pragma unroll
  for (int r = 0; r < R; ++r)
    mine += key[r] >= bound ? 1 : 0;
  int end = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(kAll, end, o);
    if (lane >= o) end += v;
  }
  const int total = __shfl_sync(kAll, end, 31);
  if (total <= 32) {
    int at = end - mine;
    if (mine > 0) {
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (key[r] >= bound) list[at++] = make_uint2(key[r], static_cast<uint32_t>(expert[r]));
    }
    __syncwarp();
    uint2 own = make_uint2(0u, 0u);
    if (lane < total) own = list[lane];
    int rank = 0;
    for (int j = 0; j < total; ++j) {
      const uint2 other = list[j];
      rank += other.x > own.x || (other.x == own.x && other.y < own.y) ? 1 : 0;
    }
    __syncwarp();
    if (lane < total) list[rank].y = own.y;       // ranks are distinct
    __syncwarp();
    return lane < min(k, total) ? static_cast<int>(list[lane].y) : -1;
  }
  // Many equal keys: k rounds of the warp's best one.
  int id = -1;
  for (int j = 0; j < k; ++j) {
    uint32_t best = 0u;
    int e = INT32_MAX;
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (key[r] > best) {
        best = key[r];
        e = expert[r];
      }
    warp_best(best, e);
    if (best == 0u) break;
    if (lane == j) id = e;
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (expert[r] == e) key[r] = 0u;
  }
  return id;
}

// choose() among the n experts of the listed groups (n <= 32 R).
template <int R>
__device__ __forceinline__ int choose_of(const uint32_t* keys, const int* groups, int size, int n,
                                         int k, int lane, uint2* list) {
  uint32_t key[R];
  int expert[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int c = r * 32 + lane;
    key[r] = 0u;
    expert[r] = INT32_MAX;
    if (c < n) {
      const int g = c / size;
      expert[r] = groups[g] * size + (c - g * size);
      key[r] = keys[expert[r]];
    }
  }
  return choose<R>(key, expert, k, lane, list);
}

template <typename T, int V, int R>
__global__ void __launch_bounds__(kWarps * 32) route_kernel(const RouteArgs a) {
  extern __shared__ uint32_t smem_keys[];
  __shared__ uint2 lists[kWarps][32];
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
  float x[R];
  load_row<T, V, R>(static_cast<const T*>(a.logits) + t * a.experts, a.experts, lane, x);

  // Whether every logit is finite: x * 0 is NaN otherwise.
  const bool whole = a.experts == 32 * R;
  float z = 0.f;
#pragma unroll
  for (int r = 0; r < R; ++r)
    if (whole || expert_of<V>(r, lane) < a.experts) z = fmaf(x[r], 0.f, z);
  const bool finite = __all_sync(kAll, z == 0.f);
  if (!finite) {
    bool bad = false;
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (!is_open(x[r])) {
        bad = bad || !(x[r] < 0.f);   // NaN or +inf: closed, and reported
        x[r] = -INFINITY;
      }
    if (bad) atomicOr(a.err, kDevErrInput);
  }
  // Softmax statistics; a closed expert's exp is 0.
  float top = -FLT_MAX, denom = 0.f;
  const bool by_logit = a.softmax && a.bias == nullptr && a.group_top == 1;
  if (a.softmax && !(by_logit && a.renorm)) {
#pragma unroll
    for (int r = 0; r < R; ++r) top = fmaxf(top, x[r]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
#pragma unroll
    for (int r = 0; r < R; ++r) denom += expf(x[r] - top);
    denom = warp_sum(denom);
  }

  // Choice values as ordered numbers.
  uint32_t key[R];
  int expert[R];
#pragma unroll
  for (int r = 0; r < R; ++r) expert[r] = expert_of<V>(r, lane);
  float c[R];
  if (by_logit) {
#pragma unroll
    for (int r = 0; r < R; ++r) c[r] = x[r];
  } else if (a.softmax) {
#pragma unroll
    for (int r = 0; r < R; ++r) c[r] = expf(x[r] - top) / denom;
  } else {
#pragma unroll
    for (int r = 0; r < R; ++r) c[r] = sigmoid(x[r]);
  }
  if (a.bias != nullptr) {
    float b[R];
    load_row<float, V, R>(a.bias, a.experts, lane, b);
#pragma unroll
    for (int r = 0; r < R; ++r) c[r] += b[r];
  }
#pragma unroll
  for (int r = 0; r < R; ++r) key[r] = ordered(c[r]);
  if (!(finite && whole)) {
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (!(x[r] > -INFINITY) || c[r] != c[r]) key[r] = 0u;
  }
  int my_id = -1;

  if (a.groups > 1) {
    uint32_t* keys = smem_keys + warp * a.experts;
#pragma unroll
    for (int r = 0; r < R; r += V) {
      const int e = expert_of<V>(r, lane);
      if (e >= a.experts) continue;
      if (V == 4)
        *reinterpret_cast<uint4*>(keys + e) =
            make_uint4(key[r], key[(r + 1) % R], key[(r + 2) % R], key[(r + 3) % R]);
      else
        keys[e] = key[r];
    }
    __syncwarp();
    const int size = a.experts / a.groups;
    const int lanes = size / 4;                   // of a group within a vector
    uint32_t gkey;
    if (V == 4 && size % 4 == 0 && lanes <= 32 && (lanes & (lanes - 1)) == 0)
      gkey = group_keys_by_lanes<R>(key, lanes, a.groups, a.group_top, lane);
    else
      gkey = group_keys_by_walk(keys, size, a.groups, a.group_top, lane);
    uint32_t stay = 0u;
    for (int i = 0; i < a.top_groups; ++i) {
      uint32_t best = gkey;
      int g = lane;
      warp_best(best, g);
      if (best == 0u) break;
      stay |= 1u << g;
      if (lane == g) gkey = 0u;
    }
    // The groups' experts, in order, spread over the lanes anew.
    if ((stay >> lane) & 1u) group_list[warp][__popc(stay & ((1u << lane) - 1u))] = lane;
    __syncwarp();
    const int n = __popc(stay) * size;
    if (n <= 8 * R) {
      my_id = choose_of<R / 4>(keys, group_list[warp], size, n, a.k, lane, lists[warp]);
    } else {
      my_id = choose_of<R>(keys, group_list[warp], size, n, a.k, lane, lists[warp]);
    }
  } else {
    my_id = choose<R>(key, expert, a.k, lane, lists[warp]);
  }

  // Lane j holds the j-th choice; its logit is in L1.
  float s = 0.f;
  const float xj = my_id >= 0 ? Elem<T>::load(static_cast<const T*>(a.logits) + t * a.experts + my_id)
                              : -INFINITY;
  if (a.softmax && a.renorm) {
    float m = xj;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
    s = my_id >= 0 ? expf(xj - m) : 0.f;
  } else if (my_id >= 0) {
    s = a.softmax ? expf(xj - top) / denom : sigmoid(xj);
  }
  float w = s;
  if (a.renorm) {
    const float sum = warp_sum(s);
    w = sum > 0.f ? s / sum : 0.f;     // every chosen score underflowed: no weight
  }
  if (lane < a.k) {
    ids[lane] = my_id;
    weights[lane] = w * a.scale;
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
      const float ds = id >= 0 ? s * sigmoid(-xj) : 0.f;
      if (a.renorm) {
        const float sum = warp_sum(s);
        const float dot = warp_sum(id >= 0 ? g * s : 0.f);
        dx = sum > 0.f ? (g - dot / sum) / sum * ds : 0.f;
      } else {
        dx = g * ds;
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
  const size_t smem = a.groups > 1 ? size_t(kWarps) * a.experts * 4 : 0;
  return launch_pdl(route_kernel<T, V, R>, grid, block, smem, s, a);
}

// Registers per lane: the least power of two that holds the row.  Rows of a
// multiple of four experts are read four at a time.
template <typename T>
cudaError_t launch_t(const RouteArgs& a, bool backward, cudaStream_t s) {
  const int per = (a.experts + 31) / 32;
  if (a.experts % 4 == 0) {
    if (per <= 4) return launch_rv<T, 4, 4>(a, backward, s);
    if (per <= 8) return launch_rv<T, 4, 8>(a, backward, s);
    if (per <= 16) return launch_rv<T, 4, 16>(a, backward, s);
    return launch_rv<T, 4, 32>(a, backward, s);
  }
  if (per <= 4) return launch_rv<T, 1, 4>(a, backward, s);
  if (per <= 16) return launch_rv<T, 1, 16>(a, backward, s);
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
