// k_loss.cu -- losses on logits, with the logits' gradient: distillation from a
// teacher's top logits, and the clipped policy loss with a KL term.
//
// Of one token's logits z, with q = softmax(z / T) and L = log sum exp(z / T):
//   distillation  p = softmax(t / T) over the teacher's given logits;
//                 loss = scale sum_j p_j (log p_j - log q_{i_j})
//                 dz_v = g scale / T (q_v - sum of the p_j with i_j = v)
//   policy        lp = z_a / T - L, r = exp(lp - old), d = ref - lp;
//                 loss = -min(r A, clip(r) A) + kl (exp(d) - d - 1)
//                 dz_v = g slope / T ([v = a] - q_v),
//                 slope = d loss / d lp = -r A (0 where the clip binds) + kl (1 - exp(d))
// Both gradients are A q_v with a few sparse terms, written over the dense value:
// the policy's by the thread that wrote that, the distillation's one thread per
// target, behind a barrier (loss_kernel) or in the warp that wrote it.
//
// Both read a row once for its statistics (maximum and sum in one pass) and, with the
// gradient, write it once: HBM bounds them, 2 V or 4 V bytes of a BF16 token.  A row is
// not kept for the gradient unless it stays on the chip, so two kernels:
//
// loss_kernel: few rows, the loss alone, the gradient from an lse.  One block takes a row
// (a cluster of up to 8 where rows are few), piece by piece: kVecs vectors of
// 16 bytes per thread.  Each warp sums exp((z - m) / T)
// against its own maximum m so far; the pairs (m, sum) go to every
// block of the cluster, one barrier, and every warp joins them in the same order.
// The gradient needs the row again.  As much of it as there is room for stays on
// the chip, where the thread that read it finds it without a barrier: the first
// pieces in shared memory, the last one in registers.  The pieces between are
// read again from L2, the latest first.  Measured: the loss of 8191 x 131072 BF16 290 us
// (7.4 TB/s, reads alone), of one row 3.4 us in a graph (8 blocks; latencies of the
// launch, the loads, the cluster's barrier); loss and gradient of 4096 x 131072 FP32
// 697 us (6.2 TB/s).
//
// loss_stream_kernel: loss and gradient of many rows.  In the kernel above reading and
// writing take turns within a block, and at these sizes only one or two fit an SM
// (8192 x 131072 BF16, 64 targets, a tenth of the tokens left out: 782 us).  Here a warp
// of its own loads the next row while this one is computed and written (638 us: 6.4 TB/s
// of what has to move; where all count 667, the policy loss 652; its 16384 x 50257 520).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "kernels.h"
#include "launch.cuh"
#include "loss.h"
#include "pair_math.cuh"
#include "sm103_ptx.cuh"

namespace muon {
namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr int kThreads = 1024;          // at most
constexpr int kVecs = 4;                // 16-byte vectors per thread and piece
constexpr int kMaxCluster = 8;
constexpr int kMaxWarps = kThreads / 32;
constexpr float kLn2 = 0.6931471805599453f;

enum Kind { kDistill, kPolicy };
enum Mode { kLossOnly, kBoth, kBackward };

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

template <typename T>
struct Elem;
template <>
struct Elem<float> {
  static constexpr int N = 4;
  static constexpr uint32_t kClosed = 0xff800000u;                     // -inf
  static __device__ __forceinline__ float value(float x) { return x; }
  static __device__ __forceinline__ float make(float x) { return x; }
  template <int V>
  static __device__ __forceinline__ float max_of(const uint4 (&d)[V]) {
    float m = -INFINITY;
#pragma unroll
    for (int r = 0; r < V; ++r)
      m = fmaxf(m, fmaxf(fmaxf(__uint_as_float(d[r].x), __uint_as_float(d[r].y)),
                         fmaxf(__uint_as_float(d[r].z), __uint_as_float(d[r].w))));
    return m;
  }
  static __device__ __forceinline__ void unpack(const uint4& u, Pair (&v)[2]) {
    v[0] = pair_of(__uint_as_float(u.x), __uint_as_float(u.y));
    v[1] = pair_of(__uint_as_float(u.z), __uint_as_float(u.w));
  }
  static __device__ __forceinline__ uint4 pack(const Pair (&v)[2]) {
    float a, b, c, d;
    split(v[0], a, b);
    split(v[1], c, d);
    return make_uint4(__float_as_uint(a), __float_as_uint(b), __float_as_uint(c), __float_as_uint(d));
  }
};
template <>
struct Elem<__nv_bfloat16> {
  static constexpr int N = 8;
  static constexpr uint32_t kClosed = 0xff80ff80u;
  static __device__ __forceinline__ float value(__nv_bfloat16 x) { return __bfloat162float(x); }
  static __device__ __forceinline__ __nv_bfloat16 make(float x) { return __float2bfloat16_rn(x); }
  static __device__ __forceinline__ __nv_bfloat162 pair(uint32_t w) {
    return *reinterpret_cast<const __nv_bfloat162*>(&w);
  }
  template <int V>
  static __device__ __forceinline__ float max_of(const uint4 (&d)[V]) {
    __nv_bfloat162 m = pair(kClosed);
#pragma unroll
    for (int r = 0; r < V; ++r)
      m = __hmax2(m, __hmax2(__hmax2(pair(d[r].x), pair(d[r].y)), __hmax2(pair(d[r].z), pair(d[r].w))));
    return fmaxf(__low2float(m), __high2float(m));
  }
  static __device__ __forceinline__ void unpack(const uint4& u, Pair (&v)[4]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = pair_of(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
  static __device__ __forceinline__ uint4 pack(const Pair (&v)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a, b;
      split(v[i], a, b);
      const __nv_bfloat162 t = __floats2bfloat162_rn(a, b);
      w[i] = *reinterpret_cast<const uint32_t*>(&t);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// How a row is divided: `head` elements to the first 16-byte boundary, `full`
// vectors, the rest.  The elements beside the vectors (at most 2 (N - 1)) are
// one each of the last block's first threads.
struct Row {
  int head, full, edges;
  int per;                 // vectors per block of the cluster
  int lo, hi;              // this block's

  template <int N>
  __device__ __forceinline__ int edge(int j) const {
    return j < head ? j : j + full * N;
  }
  // The block that has element e.
  template <int N>
  __device__ __forceinline__ int owner(int e, int blocks) const {
    const int v = e - head;
    return v < 0 || v >= full * N ? blocks - 1 : v / N / per;
  }
  // The thread that reads and writes element e, in the block that has it (nthr: a
  // power of two).
  template <int N>
  __device__ __forceinline__ int thread(int e, int nthr) const {
    const int v = e - head;
    return v < 0 ? e : v >= full * N ? e - full * N : (v / N - lo) & (nthr - 1);
  }
  template <int N>
  __device__ __forceinline__ bool has(int e, int rank, int blocks, int tid, int nthr) const {
    return owner<N>(e, blocks) == rank && thread<N>(e, nthr) == tid;
  }
};

template <typename T>
__device__ __forceinline__ Row divide(const T* row, int vocab, int rank, int blocks) {
  constexpr int N = Elem<T>::N;
  Row r;
  const int past = static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
  r.head = min((N - past) % N, vocab);
  r.full = (vocab - r.head) / N;
  r.edges = vocab - r.full * N;
  r.per = max(1, (r.full + blocks - 1) / blocks);
  r.lo = min(rank * r.per, r.full);
  r.hi = min(r.lo + r.per, r.full);
  return r;
}

// Sums against a maximum: sum of exp((z - ref) / T); -inf and 0 for nothing.
struct alignas(8) Stat {                    // (goes to other blocks in one store)
  float ref, sum;
};

// exp((z - ref) / T) as exp2(c z - c ref), c = log2(e) / T, the difference in one
// fused operation.  (c ref is rounded; all that is divided by the sum shares that, and
// a logarithm of the sum takes it off again.)
// Past |c ref| = 2^31 what it is rounded by would leave FP32's exponents.  Any two values
// there are equal or 128 and more apart (times c), so a power of two in place of c, whose
// product is exact, gives the same weights, 1 and 0; and 1/4 past |ref| = 2^100, the
// masks of a type's lowest values, where c z would overflow.
__device__ __forceinline__ float factor_at(float ref, float c) {
  if (fabsf(ref) > 0x1p100f) return 0.25f;
  return fabsf(ref * c) > 0x1p31f ? __uint_as_float(__float_as_uint(c) & 0x7f800000u) : c;
}

struct Scale {
  float c, minus;

  __device__ __forceinline__ Scale(float c_, float ref) {
    c = factor_at(ref, c_);
    minus = ref > -INFINITY ? -__fmul_rn(ref, c) : ref == ref ? 0.0f : ref;
  }
  __device__ __forceinline__ float of(float z) const { return exp2_near(fmaf(z, c, minus)); }
  // Two at a time.
  __device__ __forceinline__ Pair of(Pair z) const {
    float a, b;
    split(fma2(z, pair_of(c, c), pair_of(minus, minus)), a, b);
    return pair_of(exp2_near(a), exp2_near(b));
  }
};

// What takes sums against `ref` to sums against `to` >= ref.
__device__ __forceinline__ float rescale(float ref, float to, float c) {
  if (!(ref > -INFINITY)) return 0.0f;
  if (factor_at(to, c) != c || factor_at(ref, c) != c) return exp2_near((ref - to) * c);
  // (both products rounded, as in the weights)
  return exp2_near(__fmul_rn(ref, c) - __fmul_rn(to, c));
}

// ln of the sum against `ref`: the whole powers of two apart from the rest, since
// log2f of the sum itself is off by half a step of a number like 17; and without what
// c ref was rounded by, which every weight in the sum carries.
__device__ __forceinline__ float ln_sum(const Stat& s, float c_) {
  const Scale at(c_, s.ref);
  const bool ordinary = s.sum >= 1.0f && s.sum < INFINITY;
  const uint32_t b = __float_as_uint(s.sum);
  const float whole = ordinary ? static_cast<float>(static_cast<int>(b >> 23) - 127) : 0.0f;
  const float rest = log2f(ordinary ? __uint_as_float((b & 0x007fffffu) | 0x3f800000u) : s.sum) -
                     fmaf(s.ref, at.c, at.minus);
  return fmaf(whole, kLn2, rest * kLn2);
}

// A teacher's weight against the largest logit.  Few values: the exact functions.
struct Teacher {
  float ref, temperature;
  __device__ __forceinline__ float of(float t) const { return expf((t - ref) / temperature); }
};

// T (log p_j - log q_j) of one target, from small numbers: t_j - z_j and all the rest in
// one (of the sums, the teacher's, of weights from 1 to the number of targets, has a
// logarithm near 0); or, where the two sides' references are apart, from differences
// with these.
struct LogRatio {
  float t0, z0, shift;

  __device__ __forceinline__ LogRatio(const Stat& all, float ln_all, const Stat& teacher, float temperature) {
    const float apart = all.ref - teacher.ref;
    const bool near = fabsf(apart) <= 16.0f;
    t0 = near ? 0.0f : teacher.ref;
    z0 = near ? 0.0f : all.ref;
    shift = fmaf(temperature, ln_all - logf(teacher.sum), near ? apart : 0.0f);
  }
  __device__ __forceinline__ float of(float t, float z) const { return ((t - t0) - (z - z0)) + shift; }
};

// Joins n pairs, the same way in every warp.
__device__ __forceinline__ Stat join_all(const Stat* part, int n, int lane, float c) {
  float top = -INFINITY, sum = 0.0f;
  for (int i = lane; i < n; i += 32) top = fmaxf(top, part[i].ref);
  top = warp_max(top);
  for (int i = lane; i < n; i += 32) sum = fmaf(part[i].sum, rescale(part[i].ref, top, c), sum);
  return {top, warp_sum(sum)};
}

// A row's targets in shared memory: as many as a multiple of 4, those past the
// last one left out (id -1).
__host__ __device__ constexpr int padded(int targets) { return (targets + 3) / 4 * 4; }

// Whether target j is the first of its id, and the weights of all of that id, in
// their order.
__device__ __forceinline__ bool first_of(const int32_t* ids, const float* teach, int targets, int j,
                                         const Teacher& at, float& sum) {
  const int id = ids[j];
  bool first = true;
  sum = 0.0f;
#pragma unroll 4
  for (int i = 0; i < targets; i += 4) {
    const int4 q = *reinterpret_cast<const int4*>(ids + i);
    if (q.x == id || q.y == id || q.z == id || q.w == id) {
      const int four[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (four[u] == id) {
          first = first && i + u >= j;
          sum += at.of(teach[i + u]);
        }
    }
  }
  return first;
}

// The policy loss of a token and its slope by the log probability.
struct PolicyTerms {
  float adv, old, ref;
  bool has_old, has_ref;

  __device__ __forceinline__ void load(const LossArgs& a, int64_t tok) {
    adv = a.advantages[tok];
    has_old = a.old_logp != nullptr;
    has_ref = a.ref_logp != nullptr;
    old = has_old ? a.old_logp[tok] : 0.0f;
    ref = has_ref ? a.ref_logp[tok] : 0.0f;
  }
  __device__ __forceinline__ float slope(const LossArgs& a, float lp, float* loss_out) const {
    const float ratio = has_old ? expf(lp - old) : 1.0f;
    const bool high = adv > 0.0f && ratio > a.ratio_high, low = adv < 0.0f && ratio < a.ratio_low;
    float loss = adv == 0.0f ? 0.0f : -adv * (high ? a.ratio_high : low ? a.ratio_low : ratio);
    float s = high || low || adv == 0.0f ? 0.0f : -adv * ratio;
    if (has_ref) {
      const float dist = ref - lp, e = expm1f(dist);
      loss = fmaf(a.kl_coef, e - dist, loss);
      s = fmaf(-a.kl_coef, e, s);
    }
    *loss_out = loss;
    return s;
  }
};

template <typename T, int KIND, int MODE>
__global__ void __launch_bounds__(MODE == kBoth ? kThreads : kThreads / 2, MODE == kBoth ? 1 : 3) loss_kernel(const LossArgs a, const int blocks, const int kept) {
  using E = Elem<T>;
  constexpr int N = E::N;
  // kept pieces (loss with gradient), then the targets: ids (-1: left out), the
  // teacher's logits, the student's.
  extern __shared__ __align__(128) uint8_t dyn[];
  __shared__ Stat part[kMaxCluster * kMaxWarps];
  __shared__ Stat teacher_part[KIND == kDistill ? kMaxWarps : 1];
  const int tid = threadIdx.x, nthr = blockDim.x;
  const int warp = tid >> 5, lane = tid & 31, warps = nthr >> 5;
  const int rank = static_cast<int>(blockIdx.x) % blocks;
  const int64_t tok = static_cast<int64_t>(blockIdx.x) / blocks;
  const bool cluster = MODE != kBackward && blocks > 1;
  if (cluster) cluster_arrive();                    // every block of the cluster runs
  grid_dep_wait();
  grid_dep_launch();

  const int span = kVecs * nthr;                    // vectors per piece
  uint4* keep = reinterpret_cast<uint4*>(dyn) + tid;
  int32_t* ids = reinterpret_cast<int32_t*>(dyn + static_cast<size_t>(kept) * span * 16);
  float* teach = reinterpret_cast<float*>(ids + padded(a.targets));
  float* zs = teach + padded(a.targets);
  const T* x = static_cast<const T*>(a.logits) + tok * a.ld;
  T* out = MODE == kLossOnly ? nullptr : static_cast<T*>(a.grad_logits) + tok * a.grad_ld;
  const Row row = divide<T>(x, a.vocab, rank, blocks);
  const T* xv = x + row.head;
  const int edge = rank == blocks - 1 && tid < row.edges ? row.edge<N>(tid) : -1;
  // The gradient's rows start at the same place within 16 bytes as the logits':
  // vectors can be stored.
  const bool same = MODE != kLossOnly && ((reinterpret_cast<uintptr_t>(out) ^ reinterpret_cast<uintptr_t>(x)) & 15) == 0;

  int action = 0;
  bool live = a.mask == nullptr || a.mask[tok] != 0;
  if (KIND == kPolicy && live) {
    action = a.actions[tok];
    if (action < -1 || action >= a.vocab) {
      if (rank == 0 && tid == 0) atomicOr(a.err, kDevErrIndex);
      action = -1;
    }
    live = action >= 0;
  }

  // ------------------------------------------------------------ loads
  const int pieces = max(1, (row.hi - row.lo + span - 1) / span);
  uint4 d[kVecs];
  float xe = -INFINITY;
  // Pieces 0 .. whole - 1 have a vector for every thread and place.
  const int whole = (row.hi - row.lo) / span;
  const uint4* first = reinterpret_cast<const uint4*>(xv) + row.lo + tid;
  const auto load = [&](int k, bool last_time) {
    const uint4* at = first + k * span;
    if (k < whole) {
      // (what comes again stays in L2, the rest passes through)
      if (last_time) {
#pragma unroll
        for (int r = 0; r < kVecs; ++r) d[r] = __ldcs(at + r * nthr);
      } else {
#pragma unroll
        for (int r = 0; r < kVecs; ++r) d[r] = at[r * nthr];
      }
    } else {
#pragma unroll
      for (int r = 0; r < kVecs; ++r) {
        d[r] = make_uint4(E::kClosed, E::kClosed, E::kClosed, E::kClosed);
        if (row.lo + k * span + tid + r * nthr < row.hi) d[r] = __ldcs(at + r * nthr);
      }
    }
  };
  const bool again = MODE == kBoth && kept < pieces - 1;
  float weight_of_loss = 0.0f, lse_in = 0.0f;
  PolicyTerms terms{};
  if (live) {
    load(0, !(again && kept == 0));
    if (edge >= 0) xe = E::value(x[edge]);
    if (KIND == kPolicy) terms.load(a, tok);
    if (MODE != kLossOnly) weight_of_loss = a.grad_loss[tok];
    if (MODE == kBackward) lse_in = a.lse[tok];
  }
  const float c = a.log2e_over_t;

  // Zeros, whatever the logits hold.
  const auto leave_out = [&] {
    if (MODE != kBackward && rank == 0 && tid == 0) {
      a.loss[tok] = 0.0f;
      a.lse[tok] = 0.0f;
      if (KIND == kPolicy) a.logp[tok] = 0.0f;
    }
    if (MODE != kLossOnly) {
      const T zero = E::make(0.0f);
      for (int i = row.lo + tid; i < row.hi; i += nthr) {
        T* to = out + row.head + static_cast<int64_t>(i) * N;
        if (same) {
          __stcs(reinterpret_cast<uint4*>(to), make_uint4(0u, 0u, 0u, 0u));
        } else {
#pragma unroll
          for (int q = 0; q < N; ++q) to[q] = zero;
        }
      }
      if (edge >= 0) out[edge] = zero;
    }
  };

  // ------------------------------------------------------------ targets
  // (Nothing here waits for the targets' logits, nor for the other warps, before the
  // row's own loads are used: the loss of 37 x 131072 BF16 with 20 targets each
  // 5.6 us in a graph, 5.8 with a barrier here.)
  Stat teacher = {-INFINITY, 0.0f};
  float z_action = 0.0f, z_target = 0.0f;           // z_target: of target tid
  const auto join_teacher = [&] {
    float most = -INFINITY;
    for (int w = lane; w < warps; w += 32) most = fmaxf(most, teacher_part[w].ref);
    teacher.ref = warp_max(most);
    const Teacher at_most{teacher.ref, a.temperature};
    float sum = 0.0f;
    for (int w = lane; w < warps; w += 32)
      if (teacher_part[w].ref > -INFINITY) sum = fmaf(teacher_part[w].sum, at_most.of(teacher_part[w].ref), sum);
    teacher.sum = warp_sum(sum);
    return teacher.ref > -INFINITY;                 // a target at least
  };
  if constexpr (KIND == kDistill) {
    if (live) {
      float top = -INFINITY;
      if (tid < padded(a.targets) - a.targets) ids[a.targets + tid] = -1;
      for (int j = tid; j < a.targets; j += nthr) {
        const int64_t at = tok * a.targets + j;
        int id = a.ids[at];
        const float t = a.teacher_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.teacher)[at])
                                       : static_cast<const float*>(a.teacher)[at];
        if (id < -1 || id >= a.vocab) {
          if (rank == 0) atomicOr(a.err, kDevErrIndex);
          id = -1;
        }
        if (t == -INFINITY) id = -1;
        ids[j] = id;
        teach[j] = t;
        if (id >= 0) top = t == t ? fmaxf(top, t) : INFINITY;   // a NaN makes the sums NaN
        // The first block has the loss to sum, each block its own targets' gradient.
        if (id >= 0 && ((MODE != kBackward && rank == 0) || row.owner<N>(id, blocks) == rank)) {
          if (j == tid)
            z_target = E::value(x[id]);
          else
            zs[j] = E::value(x[id]);
        }
      }
      top = warp_max(top);
      float sum = 0.0f;
      const Teacher at_top{top, a.temperature};
      for (int j = tid; j < a.targets; j += nthr)
        if (ids[j] >= 0) sum += at_top.of(teach[j]);
      sum = warp_sum(sum);
      if (lane == 0) teacher_part[warp] = {top, sum};
      if (MODE == kBackward) {
        __syncthreads();
        live = join_teacher();
      }
    }
  } else if (live && (MODE != kBackward || row.has<N>(action, rank, blocks, tid, nthr))) {
    // (read before it may be overwritten: by this very thread, or after a barrier)
    z_action = E::value(x[action]);
  }

  if (!live) {                                      // the same for every block of the row
    if (cluster) cluster_wait();
    leave_out();
    return;
  }

  // ------------------------------------------------------------ statistics
  Stat all;
  if (MODE == kBackward) {
    all = {__fmul_rn(lse_in, a.temperature), 1.0f};
  } else {
    // The warp's sum against a reference: the first piece's maximum, and another
    // only where a value passes it by more than 2^32 times in weight.
    Stat mine = {-INFINITY, 0.0f};
    Scale scale(c, -INFINITY);
    const auto take = [&](bool with_edge) {
      const float top = fmaxf(with_edge ? xe : -INFINITY, E::max_of(d));
      if (__any_sync(kAll, fmaf(top, scale.c, scale.minus) > 32.0f || !(mine.ref > -INFINITY))) {
        const float ref = fmaxf(mine.ref, warp_max(top));
        mine = {ref, mine.sum * rescale(mine.ref, ref, c)};
        scale = Scale(c, ref);
      }
      Pair s0 = pair_of(with_edge ? scale.of(xe) : 0.0f, 0.0f), s1 = 0;
#pragma unroll
      for (int r = 0; r < kVecs; ++r) {
        Pair v[N / 2];
        E::unpack(d[r], v);
#pragma unroll
        for (int q = 0; q < N / 2; q += 2) {
          s0 = add2(s0, scale.of(v[q]));
          s1 = add2(s1, scale.of(v[q + 1]));
        }
      }
      float a0, a1;
      split(add2(s0, s1), a0, a1);
      mine.sum += a0 + a1;
    };
    for (int k = 0;;) {
      take(k == 0);
      if (k == pieces - 1) break;
      if (MODE == kBoth && k < kept) {
#pragma unroll
        for (int r = 0; r < kVecs; ++r) keep[(k * kVecs + r) * nthr] = d[r];
      }
      ++k;
      load(k, !(again && k >= kept && k < pieces - 1));
    }
    mine.sum = warp_sum(mine.sum);
    if (KIND == kDistill && tid < a.targets) zs[tid] = z_target;
    if (!cluster) {
      if (lane == 0) part[warp] = mine;
      __syncthreads();
    } else {
      cluster_wait();
      if (lane < blocks) {
        const uint32_t to = ptx::mapa_shared(ptx::smem_addr(&part[rank * warps + warp]),
                                             static_cast<uint32_t>(lane));
        asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(to), "f"(mine.ref), "f"(mine.sum)
                     : "memory");
      }
      ptx::cluster_sync();
    }
    all = join_all(part, blocks * warps, lane, c);
    if (KIND == kDistill && !join_teacher()) {
      leave_out();
      return;
    }
  }

  // ------------------------------------------------------------ the loss
  float coef = 0.0f;                                // gradient: coef q_v beside the targets
  if constexpr (KIND == kDistill) {
    if (MODE != kBackward && rank == 0 && warp == 0) {
      const Teacher at_teacher{teacher.ref, a.temperature};
      const float ln_all = ln_sum(all, c);
      const LogRatio ratio(all, ln_all, teacher, a.temperature);
      float sum = 0.0f;
      for (int j = lane; j < a.targets; j += 32) {
        if (ids[j] < 0) continue;
        const float w = at_teacher.of(teach[j]);
        if (w != 0.0f) sum = fmaf(w, ratio.of(teach[j], zs[j]), sum);
      }
      sum = warp_sum(sum);
      if (lane == 0) {
        const float loss = a.scale * (sum / (teacher.sum * a.temperature));
        const float lse = all.ref / a.temperature + ln_all;
        a.loss[tok] = loss;
        a.lse[tok] = lse;
        if (!isfinite(loss) || !isfinite(lse)) atomicOr(a.err, kDevErrInput);
      }
    }
    if (MODE != kLossOnly) coef = weight_of_loss * (a.scale * a.inv_temperature);
  } else {
    const float ln_all = ln_sum(all, c);
    const float lp = MODE == kBackward ? a.logp[tok] : (z_action - all.ref) / a.temperature - ln_all;
    float loss;
    const float slope = terms.slope(a, lp, &loss);
    if (MODE != kBackward && rank == 0 && tid == 0) {
      const float lse = all.ref / a.temperature + ln_all;
      a.loss[tok] = loss;
      a.lse[tok] = lse;
      a.logp[tok] = lp;
      if (!isfinite(loss) || !isfinite(lse)) atomicOr(a.err, kDevErrInput);
    }
    if (MODE != kLossOnly) coef = -weight_of_loss * slope * a.inv_temperature;
  }
  if (MODE == kLossOnly) return;

  // ------------------------------------------------------------ the gradient
  float f = coef / all.sum;
  const Scale at(c, all.ref);
  if (MODE == kBackward && at.c == c) {
    // What was rounded off lse T, and off its product with c: steps of numbers like 17,
    // which every value of the row would carry.
    const float off = fmaf(lse_in, a.temperature, -all.ref) * c + fmaf(all.ref, c, at.minus);
    f *= exp2_near(-off);
  }
  const auto graded = [&](const uint4& u, Pair (&v)[N / 2]) {
    E::unpack(u, v);
#pragma unroll
    for (int q = 0; q < N / 2; ++q) v[q] = mul2(at.of(v[q]), pair_of(f, f));
  };
  T* const out_first = out + row.head + static_cast<int64_t>(row.lo + tid) * N;
  const auto put = [&](int k) {
    if (k < whole && same) {
      uint4* to = reinterpret_cast<uint4*>(out_first) + k * span;
#pragma unroll
      for (int r = 0; r < kVecs; ++r) {
        Pair v[N / 2];
        graded(d[r], v);
        __stcs(to + r * nthr, E::pack(v));
      }
    } else {
#pragma unroll
      for (int r = 0; r < kVecs; ++r) {
        if (row.lo + k * span + tid + r * nthr < row.hi) {
          Pair v[N / 2];
          graded(d[r], v);
          T* to = out_first + static_cast<int64_t>(k * span + r * nthr) * N;
          if (same) {
            __stcs(reinterpret_cast<uint4*>(to), E::pack(v));
          } else {
#pragma unroll
            for (int q = 0; q < N / 2; ++q) {
              float a0, a1;
              split(v[q], a0, a1);
              to[2 * q] = E::make(a0);
              to[2 * q + 1] = E::make(a1);
            }
          }
        }
      }
    }
  };
  if (MODE == kBackward) {
    for (int k = 0;;) {
      put(k);
      if (++k >= pieces) break;
      load(k, true);
    }
  } else {
    put(pieces - 1);
    for (int k = pieces - 2; k >= kept; --k) {
      load(k, true);
      put(k);
    }
    for (int k = min(kept, pieces - 1) - 1; k >= 0; --k) {
#pragma unroll
      for (int r = 0; r < kVecs; ++r) d[r] = keep[(k * kVecs + r) * nthr];
      put(k);
    }
  }
  if (edge >= 0) out[edge] = E::make(f * at.of(xe));
  if constexpr (KIND == kDistill) {
    __syncthreads();                                // dense values before the targets'
    const float inv = 1.0f / teacher.sum;
    const Teacher at_teacher{teacher.ref, a.temperature};
    for (int j = tid; j < a.targets; j += nthr) {
      const int id = ids[j];
      if (id < 0 || row.owner<N>(id, blocks) != rank) continue;
      // Targets of the same id: the first writes for all.
      float p = 0.0f;
      if (first_of(ids, teach, a.targets, j, at_teacher, p))
        out[id] = E::make(fmaf(f, at.of(j == tid ? z_target : zs[j]), -coef * (p * inv)));
    }
  } else {
    if (row.has<N>(action, rank, blocks, tid, nthr)) {
      out[action] = E::make(fmaf(f, at.of(z_action), -coef));
    }
  }
}

constexpr int kMinThreads = 64;
constexpr int64_t kRoom = int64_t(227) << 10;         // shared memory of an SM

// Dynamic shared memory of one of `threads` threads' blocks, as many as the
// registers hold on an SM.
int64_t room_of(int threads) {
  return kRoom / (kThreads / threads) - 1024 -
         static_cast<int64_t>(sizeof(Stat)) * (kMaxCluster + 1) * kMaxWarps;
}

// ---------------------------------------------------------------- many rows
// Loss and gradient of many rows: persistent blocks that take whole rows, with
// two warps beside those that compute.  One streams chunks (PT vectors per
// thread) through a ring in shared memory, row after row without a pause: a row's
// chunks for the statistics, then those before the last `kept` again, from L2, for
// the gradient.  The last `kept` stay where they are in between.  The other warp
// brings what else a row needs, one row ahead.
//
// Tokens left out cost a write alone.  Where rows are long (`listed`), every block
// ranks the tokens first, so that each gets its share of both sorts; short rows go
// round by number.
constexpr int kMaxSlots = 32;
constexpr int kBuckets = 256;           // of the targets, by id
constexpr int64_t kMaxListed = 65536;   // tokens
constexpr int kStreamWarps = 16;        // computing warps, at most
constexpr int kStreamBound = 640;       // threads that the registers would be enough for
constexpr int kStreamRegs = 65536 / kStreamBound / 8 * 8;

template <int KIND>
struct StreamShared {
  uint64_t full[kMaxSlots], empty[kMaxSlots];
  uint64_t meta_full[2], meta_empty[2];
  int abort;
  int late[2];                            // a computing warp's wait has run out
  int ranks[kStreamBound / 32];            // counts of the warps
  struct {
    int live, action;
    float z_action, weight;
    PolicyTerms terms;
    Stat teacher;
    float edge[16];
    int start[kStreamWarps + 1];           // of each warp's targets in their order
  } meta[2];
  int count[kStreamWarps];
  Stat part[2][kStreamWarps];
  float loss[2][KIND == kDistill ? kStreamWarps : 1];
};

__device__ __forceinline__ void bulk_load(void* to, const void* from, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          ptx::smem_addr(to)),
      "l"(from), "r"(bytes), "r"(ptx::smem_addr(bar))
      : "memory");
}

template <typename T, int KIND, int PT>
__global__ void __launch_bounds__(kStreamBound, 1)
    loss_stream_kernel(const LossArgs a, const int slots, const int keep, const int listed) {
  using E = Elem<T>;
  constexpr int N = E::N;
  extern __shared__ __align__(128) uint8_t dyn[];
  __shared__ StreamShared<KIND> sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int warps = (blockDim.x >> 5) - 2, nthr = warps * 32;
  const int span = PT * nthr;               // vectors per chunk
  // Targets of two rows in turn: ids (-1: left out), the teacher's logits, the
  // student's, the weights of the id (below 0: of a target before this one), the
  // targets' order by the warp that writes their element, and their own weights.
  int32_t* all_ids = reinterpret_cast<int32_t*>(dyn + static_cast<size_t>(slots) * span * 16);
  const float c = a.log2e_over_t;
  const int32_t tokens = static_cast<int32_t>(a.tokens), step = static_cast<int32_t>(gridDim.x);
  // listed: this block's tokens that count, then those left out.
  int32_t* bucket = all_ids + 12 * padded(a.targets);      // of the targets being brought
  int32_t* link = bucket + kBuckets;
  int32_t* list = all_ids + (KIND == kDistill ? 13 * padded(a.targets) + kBuckets : 0);
  int32_t* rest = list + tokens / step + 1;
  if (tid == 0) {
    for (int i = 0; i < slots; ++i) {
      ptx::mbar_init(&sh.full[i], 1);
      ptx::mbar_init(&sh.empty[i], static_cast<uint32_t>(warps));
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&sh.meta_full[i], 1);
      ptx::mbar_init(&sh.meta_empty[i], static_cast<uint32_t>(warps));
    }
    sh.abort = sh.late[0] = sh.late[1] = 0;
    ptx::fence_barrier_init();
  }
  __syncthreads();
  grid_dep_wait();
  grid_dep_launch();
  const volatile int* abort = &sh.abort;
  const auto give_up = [&] {
    sh.abort = 1;
    atomicOr(a.err, kDevErrTimeout);
  };
  const auto row_of = [&](int64_t tok) { return static_cast<const T*>(a.logits) + tok * a.ld; };
  // A token's mask and action, loaded without a branch, ahead of their use.
  struct Look {
    int mask, action;
  };
  const auto look = [&](int tok) {
    const int at = min(tok, tokens - 1);
    return Look{a.mask != nullptr ? static_cast<int>(a.mask[at]) : 1, KIND == kPolicy ? a.actions[at] : 0};
  };
  const auto counts = [&](const Look& l) {
    return l.mask != 0 && l.action >= 0 && l.action < a.vocab;
  };
  int n_rows = (tokens - static_cast<int>(blockIdx.x) + step - 1) / step, n_rest = 0;
  if (listed) {
    // Each warp a range of tokens, 32 to a word (kept in the ring, still unused).
    uint32_t* words = reinterpret_cast<uint32_t*>(dyn);
    const int groups = (tokens + 31) / 32, all_warps = static_cast<int>(blockDim.x >> 5);
    const int lo = groups * warp / all_warps, hi = groups * (warp + 1) / all_warps;
    int live = 0;
    for (int g = lo; g < hi; g += 8) {
      Look l[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) l[q] = look((g + q) * 32 + lane);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const uint32_t on = __ballot_sync(kAll, (g + q) * 32 + lane < tokens && counts(l[q]));
        if (g + q < hi) {
          live += __popc(on);
          if (lane == 0) words[g + q] = on;
        }
      }
    }
    if (lane == 0) sh.ranks[warp] = live;
    __syncthreads();
    int before = 0, total = 0;
    for (int w = 0; w < all_warps; ++w) {
      if (w < warp) before += sh.ranks[w];
      total += sh.ranks[w];
    }
    const int me = static_cast<int>(blockIdx.x);
    for (int g = lo; g < hi; ++g) {
      const uint32_t on = words[g];
      const int t = g * 32 + lane, under = __popc(on & ((1u << lane) - 1u));
      const bool mine = (on >> lane & 1u) != 0;
      const int rank = mine ? before + under : t - before - under;
      if (t < tokens && rank % step == me) (mine ? list : rest)[rank / step] = t;
      before += __popc(on);
    }
    n_rows = (total - me + step - 1) / step;
    n_rest = (tokens - total - me + step - 1) / step;
    ptx::fence_proxy_async_smem();            // (the words' place is loaded into next)
    __syncthreads();
  }
  const auto nth = [&](int i) {
    if (listed) return i < n_rows ? list[i] : tokens;
    return static_cast<int>(blockIdx.x) + i * step;
  };

  if (warp == warps) {
    // ------------------------------------------------------------ chunks
    if (lane == 0) {
      if (a.stall == kLossStallLogits) n_rows = min(n_rows, 1);     // (self-test of the waits)
      int slot = 0;
      uint32_t phase = 0;
      int64_t issued = 0;
      bool ok = true;
      Look here = look(nth(0)), next = look(nth(1));
      for (int i = 0; ok && i < n_rows; ++i) {
        const int tok = nth(i);
        const Look after = look(nth(i + 2));
        if (counts(here)) {
          const T* x = row_of(tok);
          const Row row = divide<T>(x, a.vocab, 0, 1);
          const int chunks = (row.full + span - 1) / span;
          const int again = max(chunks - keep, 0);
          for (int j = 0; j < chunks + again; ++j) {
            const int k = j < chunks ? j : again - 1 - (j - chunks);
            if (!ptx::mbar_wait(&sh.empty[slot], phase ^ 1u, abort)) {
              ok = false;
              break;
            }
            const uint32_t bytes = static_cast<uint32_t>(min(span, row.full - k * span)) * 16u;
            ptx::mbar_arrive_expect_tx(&sh.full[slot], bytes);
            bulk_load(dyn + static_cast<size_t>(slot) * span * 16,
                      x + row.head + static_cast<int64_t>(k) * span * N, bytes, &sh.full[slot]);
            ++issued;
            if (++slot == slots) {
              slot = 0;
              phase ^= 1u;
            }
          }
        }
        here = next;
        next = after;
      }
      if (!ok) give_up();
      // Copies in flight end before the block does, whoever gave up.
      for (int i = 0; i < slots && i < issued; ++i) {
        if (slot == 0) {
          slot = slots;
          phase ^= 1u;
        }
        --slot;
        ptx::mbar_wait(&sh.full[slot], phase, nullptr);
      }
    }
  } else if (warp == warps + 1) {
    // ------------------------------------------------------------ the rest of a row
    if (a.stall == kLossStallTargets) n_rows = min(n_rows, 1);
    int turn = 0;
    uint32_t phase = 0;
    Look here = look(nth(0)), next = look(nth(1));
    for (int i = 0; i < n_rows; ++i) {
      const int tok = nth(i), action = here.action;
      const Look after = look(nth(i + 2));
      const bool live = counts(here);
      const T* x = row_of(tok);
      const Row row = divide<T>(x, a.vocab, 0, 1);
      float edge = -INFINITY, z_action = 0.0f, weight = 0.0f;
      PolicyTerms terms{};
      if (live) {
        if (lane < row.edges) edge = E::value(x[row.edge<N>(lane)]);
        weight = a.grad_loss[tok];
        if (KIND == kPolicy) {
          z_action = E::value(x[action]);
          terms.load(a, tok);
        }
      } else if (here.mask != 0 && action != -1 && lane == 0) {
        atomicOr(a.err, kDevErrIndex);
      }
      if (!__all_sync(kAll, ptx::mbar_wait(&sh.meta_empty[turn], phase ^ 1u, abort))) {
        if (lane == 0) give_up();
        break;
      }
      auto& m = sh.meta[turn];
      Stat teacher = {0.0f, 1.0f};
      if constexpr (KIND == kDistill) {
        int32_t* ids = all_ids + turn * 6 * padded(a.targets);
        float* teach = reinterpret_cast<float*>(ids + padded(a.targets));
        float* zs = teach + padded(a.targets);
        float top = -INFINITY;
        if (live) {
          if (lane < padded(a.targets) - a.targets) ids[a.targets + lane] = -1;
          // (Four loads of either in flight: one by one they would take longer than a row
          // of 50257 from some 100 targets on.)
          for (int j0 = lane; j0 - lane < a.targets; j0 += 128) {
            const int64_t row0 = static_cast<int64_t>(tok) * a.targets;
            int id4[4];
            float t4[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) id4[u] = a.ids[row0 + min(j0 + u * 32, a.targets - 1)];
            if (a.teacher_bf16) {
#pragma unroll
              for (int u = 0; u < 4; ++u)
                t4[u] = __bfloat162float(
                    static_cast<const __nv_bfloat16*>(a.teacher)[row0 + min(j0 + u * 32, a.targets - 1)]);
            } else {
#pragma unroll
              for (int u = 0; u < 4; ++u)
                t4[u] = static_cast<const float*>(a.teacher)[row0 + min(j0 + u * 32, a.targets - 1)];
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const int j = j0 + u * 32;
              if (j >= a.targets) continue;
              int id = id4[u];
              const float t = t4[u];
              if (id < -1 || id >= a.vocab) {
                atomicOr(a.err, kDevErrIndex);
                id = -1;
              }
              if (t == -INFINITY) id = -1;
              ids[j] = id;
              teach[j] = t;
              if (id >= 0) top = t == t ? fmaxf(top, t) : INFINITY;   // a NaN makes the sums NaN
            }
          }
          top = warp_max(top);
          const Teacher at_top{top, a.temperature};
          float sum = 0.0f;
          __syncwarp();
          float* total = zs + padded(a.targets);
          int32_t* order = reinterpret_cast<int32_t*>(total + padded(a.targets));
          float* own = total + 2 * padded(a.targets);
#pragma unroll 4
          for (int j = lane; j < a.targets; j += 32)
            if (ids[j] >= 0) {
              own[j] = at_top.of(teach[j]);
              sum += own[j];
            }
          teacher = {top, warp_sum(sum)};
          // The weights of equal ids together, in their order, with the first of each: 32
          // targets at a time, the lowest of an id looks for one before them in its bucket's
          // chain, which has the first of each id alone, and adds up its equals' weights.
          // (4093 rows of 50257 FP32 with 1000 targets of 5 ids 1.1 ms, of as many ids 1.2;
          // 92 and 1.5 where each target walked a chain of all.)
          for (int b = lane; b < kBuckets; b += 32) bucket[b] = -1;
          __syncwarp();
          const auto id_at = [&](int j) { return j < a.targets ? ids[j] : -1; };
          const auto head_of = [&](int id) { return bucket + (static_cast<uint32_t>(id) * 0x9e3779b1u >> 24); };
          int id = id_at(lane);
          for (int j = lane; j - lane < a.targets; j += 32) {
            const int after = id_at(j + 32);
            int at = *head_of(id);
            float p = id >= 0 ? own[j] : 0.0f;
            const uint32_t equal = __match_any_sync(kAll, id);
            const bool lowest = id >= 0 && (equal & ((1u << lane) - 1u)) == 0;
            if (lowest) {
              while (at >= 0 && ids[at] != id) at = link[at];
              if (at >= 0) p += total[at];
              for (uint32_t rest = equal & (equal - 1u); rest != 0; rest &= rest - 1)
                p += own[j - lane + __ffs(rest) - 1];
              total[at >= 0 ? at : j] = p;
            }
            if (id >= 0 && (!lowest || at >= 0)) total[j] = -1.0f;
            __syncwarp();                           // (chains change when none is looked through)
            if (lowest && at < 0) link[j] = atomicExch(head_of(id), j);
            __syncwarp();
            id = after;
          }
          // Each target to the warp that writes its element.
          if (lane < kStreamWarps) sh.count[lane] = 0;
          __syncwarp();
          const auto warp_of = [&](int j) {
            return j < a.targets && ids[j] >= 0 ? row.thread<N>(ids[j], nthr) / 32 : kStreamWarps;
          };
          for (int j = lane; j < a.targets; j += 32) {
            const int w = warp_of(j);
            if (w < kStreamWarps) atomicAdd(&sh.count[w], 1);
          }
          __syncwarp();
          const int n = lane < kStreamWarps ? sh.count[lane] : 0;
          int before = n;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(kAll, before, o);
            if (lane >= o) before += v;
          }
          before -= n;
          if (lane <= kStreamWarps) m.start[lane] = before;
          __syncwarp();
          if (lane < kStreamWarps) sh.count[lane] = before;
          __syncwarp();
          for (int j0 = 0; j0 < a.targets; j0 += 32) {
            const int w = warp_of(j0 + lane);
            const uint32_t same_warp = __match_any_sync(kAll, w);
            const int rank = __popc(same_warp & ((1u << lane) - 1u));
            const int at = w < kStreamWarps ? sh.count[w] + rank : 0;
            __syncwarp();
            if (w < kStreamWarps) {
              order[at] = j0 + lane;
              if (rank == 0) sh.count[w] += __popc(same_warp);
            }
            __syncwarp();
          }
        }
      }
      if (lane < 16) m.edge[lane] = edge;
      if (lane == 0) {
        m.live = live;
        m.action = action;
        m.z_action = z_action;
        m.weight = weight;
        m.terms = terms;
        m.teacher = teacher;
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&sh.meta_full[turn]);
      turn ^= 1;
      if (turn == 0) phase ^= 1u;
      here = next;
      next = after;
    }
  } else {
    // ------------------------------------------------------------ the rows
    // A wait that runs out is reported, and ends the rows for all warps together.  They
    // meet once per row that counts and at the end; a warp whose targets have not come
    // does not know whether its row counts: it reads nothing of it, goes to the next
    // meeting at once and leaves.  late[meeting] is written before that meeting and read
    // after it, and its place used again two meetings later.
    int meeting = 0;
    bool left = false;
    const auto miss = [&] {
      give_up();
      sh.late[meeting] = 1;
    };
    const auto expect = [&](uint64_t* bar, uint32_t phase) {
      if (!ptx::mbar_wait(bar, phase, abort)) miss();
    };
    const auto meet_rows = [&] {                    // whether a wait has run out
      asm volatile("barrier.cta.sync.aligned 1, %0;" ::"r"(nthr) : "memory");
      const int late = *const_cast<const volatile int*>(&sh.late[meeting]);
      meeting ^= 1;
      return late != 0;
    };
    // Hands shared memory back: the warp's reads of it come before what is written there
    // next.  (A relaxed arrival, which leaves that to every value having been used, takes
    // no less: 8192 x 131072 BF16 with 64 targets, a tenth left out, 638 us either way,
    // policy 8191 x 131072 555 and 556.)
    const auto release = [&](uint64_t* bar) {
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar);
    };
    int turn = 0, swap = 0, slot = 0;
    uint32_t meta_phase = 0, phase = 0;
    int pending = -1;
    float over = 1.0f;                              // what the parts' sum is divided by
    const auto advance = [&] {
      if (++slot == slots) {
        slot = 0;
        phase ^= 1u;
      }
    };
    // Zeros, whatever the logits hold.
    const auto leave_out = [&](int tok) {
      T* out = static_cast<T*>(a.grad_logits) + static_cast<int64_t>(tok) * a.grad_ld;
      const Row row = divide<T>(out, a.vocab, 0, 1);      // (its own vectors)
      for (int i = tid; i < row.full; i += nthr)
        __stcs(reinterpret_cast<uint4*>(out + row.head) + i, make_uint4(0u, 0u, 0u, 0u));
      if (tid < row.edges) out[row.edge<N>(tid)] = E::make(0.0f);
      if (tid == 0) {
        a.loss[tok] = 0.0f;
        a.lse[tok] = 0.0f;
        if (KIND == kPolicy) a.logp[tok] = 0.0f;
      }
    };
    // Distillation: the loss of the row before, whose parts have been met for.
    const auto finish = [&](int from) {
      if (KIND != kDistill || pending < 0 || warp != 0) return;
      const float loss = a.scale * (warp_sum(lane < warps ? sh.loss[from][lane] : 0.0f) / over);
      if (lane == 0) {
        a.loss[pending] = loss;
        if (!isfinite(loss)) atomicOr(a.err, kDevErrInput);
      }
    };
    for (int i = 0; i < n_rows; ++i) {
      const int tok = nth(i);
      // (one outcome in all of a warp: it stays converged)
      if (!__all_sync(kAll, ptx::mbar_wait(&sh.meta_full[turn], meta_phase, abort))) {
        miss();
        meet_rows();
        left = true;
        break;
      }
      const auto& m = sh.meta[turn];
      const T* x = row_of(tok);
      T* out = static_cast<T*>(a.grad_logits) + static_cast<int64_t>(tok) * a.grad_ld;
      const Row row = divide<T>(x, a.vocab, 0, 1);
      const bool same = ((reinterpret_cast<uintptr_t>(out) ^ reinterpret_cast<uintptr_t>(x)) & 15) == 0;
      const int chunks = (row.full + span - 1) / span;
      const int again = max(chunks - keep, 0);
      const int edge = tid < row.edges ? row.edge<N>(tid) : -1;
      const bool live = m.live != 0;
      const Stat teacher = m.teacher;
      const bool counted = live && (KIND == kPolicy || teacher.ref > -INFINITY);
      uint4 d[PT];
      const auto take_chunk = [&](int slot_, int k) {
        const uint4* from = reinterpret_cast<const uint4*>(dyn) + slot_ * span + tid;
        if ((k + 1) * span <= row.full) {
#pragma unroll
          for (int r = 0; r < PT; ++r) d[r] = from[r * nthr];
        } else {
#pragma unroll
          for (int r = 0; r < PT; ++r) {
            d[r] = make_uint4(E::kClosed, E::kClosed, E::kClosed, E::kClosed);
            if (k * span + tid + r * nthr < row.full) d[r] = from[r * nthr];
          }
        }
      };
      const int slot0 = slot;
      const float xe = edge >= 0 ? m.edge[tid] : -INFINITY;
      Stat mine = {-INFINITY, 0.0f};
      if (live) {
        Scale scale(c, -INFINITY);
        const auto refer = [&](float top) {
          if (__any_sync(kAll, fmaf(top, scale.c, scale.minus) > 32.0f || !(mine.ref > -INFINITY))) {
            const float ref = fmaxf(mine.ref, warp_max(top));
            mine = {ref, mine.sum * rescale(mine.ref, ref, c)};
            scale = Scale(c, ref);
          }
        };
        for (int k = 0; k < chunks; ++k) {
          expect(&sh.full[slot], phase);
          take_chunk(slot, k);
          refer(E::max_of(d));
          if (k < again) release(&sh.empty[slot]);
          Pair s0 = 0, s1 = 0;
#pragma unroll
          for (int r = 0; r < PT; ++r) {
            Pair v[N / 2];
            E::unpack(d[r], v);
#pragma unroll
            for (int q = 0; q < N / 2; q += 2) {
              s0 = add2(s0, scale.of(v[q]));
              s1 = add2(s1, scale.of(v[q + 1]));
            }
          }
          float a0, a1;
          split(add2(s0, s1), a0, a1);
          mine.sum += a0 + a1;
          advance();
        }
        if (row.edges > 0) {
          refer(xe);
          mine.sum += scale.of(xe);
        }
      }
      // The targets' logits, from L2 where the row now is (ahead of the row they would
      // be reads of their own from HBM: 42 us of 717 for 8192 rows of 131072 BF16, a
      // tenth left out, with 64 targets each; left pending behind the gradient's stores
      // 18 us).  Each warp those whose elements it writes itself, so that no barrier is
      // needed between the dense values and the targets' terms (with one, and the first
      // warps taking all targets, the same rows 682 us instead of 656).
      T z_target = E::make(0.0f);
      int target = -1;
      if constexpr (KIND == kDistill) {
        int32_t* ids = all_ids + turn * 6 * padded(a.targets);
        float* zs = reinterpret_cast<float*>(ids) + 2 * padded(a.targets);
        const int32_t* order = ids + 4 * padded(a.targets);
        if (counted) {
          const int end = m.start[warp + 1];
          int i = m.start[warp] + lane;
          if (i < end) {
            target = order[i];
            z_target = x[ids[target]];
          }
          for (i += 32; i < end; i += 32) zs[order[i]] = E::value(x[ids[order[i]]]);
        }
      }
      Stat all = {0.0f, 1.0f};
      float f = 0.0f, coef = 0.0f, ln_all = 0.0f;
      if (counted) {
        mine.sum = warp_sum(mine.sum);
        if (lane == 0) sh.part[swap][warp] = mine;
        // (looked at behind the parts: 65536 x 4096 BF16 262 us, at once 264)
        const bool late = meet_rows();
        all = join_all(sh.part[swap], warps, lane, c);
        if (late) {
          left = true;
          break;
        }
        finish(swap ^ 1);
        ln_all = ln_sum(all, c);
        const float lse = all.ref / a.temperature + ln_all;
        if constexpr (KIND == kDistill) {
          if (tid == 0) {
            a.lse[tok] = lse;
            if (!isfinite(lse)) atomicOr(a.err, kDevErrInput);
          }
          coef = m.weight * (a.scale * a.inv_temperature);
        } else {
          const float lp = (m.z_action - all.ref) / a.temperature - ln_all;
          float loss;
          const float slope = m.terms.slope(a, lp, &loss);
          if (tid == 0) {
            a.loss[tok] = loss;
            a.lse[tok] = lse;
            a.logp[tok] = lp;
            if (!isfinite(loss) || !isfinite(lse)) atomicOr(a.err, kDevErrInput);
          }
          coef = -m.weight * slope * a.inv_temperature;
        }
        f = coef / all.sum;
      }

      // ------------------------------------------------------------ the gradient
      const Scale at(c, all.ref);
      T* const out_first = out + row.head + static_cast<int64_t>(tid) * N;
      const auto put_chunk = [&](int k) {
        if ((k + 1) * span <= row.full && same) {
          uint4* to = reinterpret_cast<uint4*>(out_first) + k * span;
#pragma unroll
          for (int r = 0; r < PT; ++r) {
            Pair v[N / 2];
            E::unpack(d[r], v);
#pragma unroll
            for (int q = 0; q < N / 2; ++q) v[q] = mul2(at.of(v[q]), pair_of(f, f));
            __stcs(to + r * nthr, E::pack(v));
          }
        } else {
#pragma unroll
          for (int r = 0; r < PT; ++r) {
            if (k * span + tid + r * nthr < row.full) {
              Pair v[N / 2];
              E::unpack(d[r], v);
#pragma unroll
              for (int q = 0; q < N / 2; ++q) v[q] = mul2(at.of(v[q]), pair_of(f, f));
              T* to = out_first + static_cast<int64_t>(k * span + r * nthr) * N;
              if (same) {
                __stcs(reinterpret_cast<uint4*>(to), E::pack(v));
              } else {
#pragma unroll
                for (int q = 0; q < N / 2; ++q) {
                  float a0, a1;
                  split(v[q], a0, a1);
                  to[2 * q] = E::make(a0);
                  to[2 * q + 1] = E::make(a1);
                }
              }
            }
          }
        }
      };
      if (!counted) leave_out(tok);
      if (live) {
        // (a row without any target has been streamed too)
        for (int k = chunks - 1; k >= again; --k) {
          int at_slot = slot0 + k;                  // modulo the ring
          at_slot %= slots;
          if (counted) {
            take_chunk(at_slot, k);
            put_chunk(k);
          }
          release(&sh.empty[at_slot]);
        }
        for (int k = again - 1; k >= 0; --k) {
          expect(&sh.full[slot], phase);
          take_chunk(slot, k);
          if (counted) put_chunk(k);
          release(&sh.empty[slot]);
          advance();
        }
        if (counted && edge >= 0) out[edge] = E::make(f * at.of(xe));
      }
      if (counted) {
        if constexpr (KIND == kDistill) {
          const int32_t* ids = all_ids + turn * 6 * padded(a.targets);
          const float* teach = reinterpret_cast<const float*>(ids + padded(a.targets));
          const float* zs = teach + padded(a.targets);
          const int32_t* order = ids + 4 * padded(a.targets);
          // The targets' parts of the loss, and their terms.
          __syncwarp();                             // dense values before the targets'
          const float* own = zs + 3 * padded(a.targets);
          const LogRatio ratio(all, ln_all, teacher, a.temperature);
          const float inv = 1.0f / teacher.sum;
          const int end = m.start[warp + 1];
          float sum = 0.0f;
          for (int i = m.start[warp] + lane; i < end; i += 32) {
            const int j = i < m.start[warp] + 32 ? target : order[i];
            const float w = own[j], z = j == target ? E::value(z_target) : zs[j];
            if (w != 0.0f) sum = fmaf(w, ratio.of(teach[j], z), sum);
            // Targets of the same id: the first writes for all.
            const float p = zs[padded(a.targets) + j];
            if (!(p < 0.0f)) out[ids[j]] = E::make(fmaf(f, at.of(z), -coef * (p * inv)));
          }
          sum = warp_sum(sum);
          if (lane == 0) sh.loss[swap][warp] = sum;
          pending = tok;
          over = teacher.sum * a.temperature;
        } else {
          if (row.has<N>(m.action, 0, 1, tid, nthr))
            out[m.action] = E::make(fmaf(f, at.of(m.z_action), -coef));
        }
        swap ^= 1;
      }
      release(&sh.meta_empty[turn]);
      turn ^= 1;
      if (turn == 0) meta_phase ^= 1u;
    }
    if (!left) meet_rows();                         // (with a warp that leaves, or all at the end)
    finish(swap ^ 1);
    for (int i = 0; i < n_rest; ++i) {
      const int tok = rest[i];
      leave_out(tok);
      if (KIND == kPolicy && tid == 0) {
        const Look l = look(tok);
        if (l.mask != 0 && l.action != -1) atomicOr(a.err, kDevErrIndex);
      }
    }
  }
}

template <typename T, int KIND, int PT>
cudaError_t start_stream(const LossArgs& a, int warps, int blocks, int64_t slots, int64_t keep,
                         bool listed, size_t smem, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(static_cast<unsigned>((warps + 2) * 32));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, loss_stream_kernel<T, KIND, PT>, a, static_cast<int>(slots),
                            static_cast<int>(keep), listed ? 1 : 0);
}

// Whether the call has rows enough for persistent blocks, and their launch.  By
// bytes of a row (304 of the longer ones do not stay in L2), measured with loss and
// gradient (us, distillation with 64 targets / policy):
//                             one block per SM   two
//   98 KB   16384 x 25001 FP32    586 / 542    526 / 552
//   98 KB   16384 x 50257 BF16    647 / 595    537 / 519
//   109 KB  16384 x 28001 FP32    599 / 564    596 / 614
//   125 KB  16384 x 32000 FP32    643 / 634    697 / 706
//   125 KB  16384 x 64000 BF16    709 / 665    685 / 711
//   195 KB  16384 x 100003 BF16  1057 / 1035  1247 / 1256
//   196 KB  8192 x 50257 FP32     509 / 504    618 / 622
//                             one block per SM   a block per row, part of it on the chip
//   312 KB  4096 x 80003 FP32     463 / 466    599 / 464
//   351 KB  4096 x 90001 FP32     539 / 540    646 / 524
//   378 KB  4096 x 97001 FP32     592 / 595    676 / 545
//   390 KB  6144 x 200003 BF16    914 / 918   1119 / 918
//   429 KB  4096 x 110003 FP32    688 / 689    727 / 615
//   468 KB  4096 x 120001 FP32    765 / 767    801 / 682
//   512 KB  4096 x 131072 FP32    834 / 832    798 / 697
// (Streaming is worth more to the distillation, whose targets it brings ahead: its
// rows cross between 468 and 512 KB, the policy's at 312.)
constexpr int64_t kTwoRows = 112 << 10, kLongRow = 384 << 10;

template <typename T, int KIND>
bool stream_rows(const LossArgs& a, int num_sms, cudaStream_t s, cudaError_t* e) {
  const int64_t row = (static_cast<int64_t>(a.vocab) + Elem<T>::N - 1) / Elem<T>::N * 16;
  const int64_t targets = KIND == kDistill ? int64_t(52) * padded(a.targets) + 4 * kBuckets : 0;
  for (int warps = 2; warps <= kStreamWarps; warps *= 2) {
    const int pt = warps == kStreamWarps ? 2 : 4;
    const int per_sm = 65536 / (kStreamRegs * (warps + 2) * 32);
    const int blocks = per_sm * num_sms;
    const int64_t chunk = int64_t(warps) * 32 * pt * 16, chunks = (row + chunk - 1) / chunk;
    const bool listed = (a.mask != nullptr || KIND == kPolicy) && warps >= 8 && a.tokens <= kMaxListed;
    const int64_t lists = listed ? (a.tokens / blocks + 1) * 8 : 0;
    int64_t slots = (kRoom / per_sm - 1024 - static_cast<int64_t>(sizeof(StreamShared<KIND>)) - targets - lists) / chunk;
    if (slots > kMaxSlots) slots = kMaxSlots;
    // The fewest warps whose ring holds a row and half of the next one; or, with two
    // blocks per SM, most of a row.
    if (warps < kStreamWarps && 2 * slots < 3 * chunks && !(warps == 8 && row <= kTwoRows)) continue;
    if (slots < 2 || row > kLongRow || a.tokens < 2 * blocks || a.tokens > INT32_MAX / 2) return false;
    const int64_t keep = 2 * slots >= 3 * chunks ? chunks : slots * 3 / 4;
    const size_t smem = static_cast<size_t>(slots * chunk + targets + lists);
    *e = pt == 2 ? start_stream<T, KIND, 2>(a, warps, blocks, slots, keep, listed, smem, s)
                 : start_stream<T, KIND, 4>(a, warps, blocks, slots, keep, listed, smem, s);
    return true;
  }
  return false;
}

template <typename T, int KIND, int MODE>
cudaError_t start_mode(const LossArgs& a, int num_sms, cudaStream_t s) {
  if (MODE == kBoth) {
    cudaError_t e;
    if (stream_rows<T, KIND>(a, num_sms, s, &e)) return e;
  }
  const int64_t vecs = (static_cast<int64_t>(a.vocab) + Elem<T>::N - 1) / Elem<T>::N;
  // Few rows: several blocks for each.
  int blocks = 1;
  while (blocks < kMaxCluster && a.tokens * blocks < 2 * num_sms && vecs > blocks * int64_t(kThreads / 2))
    blocks *= 2;
  const int64_t per = (vecs + blocks - 1) / blocks;
  const int64_t targets = KIND == kDistill ? int64_t(12) * padded(a.targets) : 0;
  int threads = kMinThreads;
  if (MODE == kBoth) {
    // The fewest threads that hold the row on the chip: more rows at one time.
    const auto holds = [&](int t) {
      const int64_t piece = int64_t(t) * kVecs;
      return per <= piece * (1 + (room_of(t) - targets) / (piece * 16));
    };
    while (threads < kThreads && (room_of(threads) < targets || !holds(threads))) threads *= 2;
  } else {
    // A piece each, as far as that goes.
    while (threads < (MODE == kLossOnly ? kThreads / 4 : kThreads / 2) && per > int64_t(threads) * kVecs) threads *= 2;
    // More rows than run at one time: narrower blocks, whose waits overlap with more
    // others'.  Measured at 512 MB of BF16 logits (FP32 takes up to a tenth less, in the same
    // order), by threads, us: loss of the distillation with 8 targets / of the policy,
    // and their gradients from the lse:
    //   vectors        64       128       256       64       128       256       512
    //   300       451/296   407/284   606/497  568/312   520/281   666/471  1335/911
    //   512       277/179   238/165   359/294  349/221   302/190   401/291   791/555
    //   1024      182/133   154/110   180/145  250/202   219/167   236/172   428/306
    //   1400      169/134   134/103   167/138  241/207   206/165   218/166   332/235
    //   2048      139/116   111/90    118/97   216/195   180/160   178/156   252/173
    //   3000      134/118   102/89    101/89   216/202   178/165   170/160   221/168
    //   4096      118/107    93/84     92/83   201/192   171/163   165/160   187/157
    //   6000      121/113    92/85     90/82   205/196   174/166   169/163   173/159
    //   8000      122/116    92/86     87/82   201/197   174/168   169/166   168/161
    if (a.tokens * blocks > num_sms * int64_t(3 * kThreads / 2 / threads)) {
      const int64_t most = MODE == kLossOnly ? 2048 : 1024, wide = KIND == kDistill ? 4096 : 2048;
      if (per > int64_t(kMinThreads) * kVecs && per <= most) threads = 128;
      else if (MODE == kBackward && per > most && per <= wide) threads = 256;
    }
  }
  const int64_t piece = int64_t(threads) * kVecs, pieces = (per + piece - 1) / piece;
  int64_t kept = MODE == kBoth ? (room_of(threads) - targets) / (piece * 16) : 0;
  if (kept > pieces - 1) kept = pieces - 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.tokens * blocks));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(kept * piece * 16) + targets;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(blocks);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, loss_kernel<T, KIND, MODE>, a, blocks, static_cast<int>(kept));
}

template <int KIND>
cudaError_t launch(const LossArgs& a, bool bf16, bool grad, bool backward, int num_sms, cudaStream_t s) {
  using B = __nv_bfloat16;
  if (backward)
    return bf16 ? start_mode<B, KIND, kBackward>(a, num_sms, s) : start_mode<float, KIND, kBackward>(a, num_sms, s);
  if (grad) return bf16 ? start_mode<B, KIND, kBoth>(a, num_sms, s) : start_mode<float, KIND, kBoth>(a, num_sms, s);
  return bf16 ? start_mode<B, KIND, kLossOnly>(a, num_sms, s) : start_mode<float, KIND, kLossOnly>(a, num_sms, s);
}

}  // namespace

cudaError_t loss_init() {
  constexpr cudaFuncAttribute what = cudaFuncAttributeMaxDynamicSharedMemorySize;
  const int most = static_cast<int>(room_of(kThreads));
  cudaError_t e = cudaFuncSetAttribute(loss_kernel<float, kDistill, kBoth>, what, most);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(loss_kernel<float, kPolicy, kBoth>, what, most);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(loss_kernel<__nv_bfloat16, kDistill, kBoth>, what, most);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(loss_kernel<__nv_bfloat16, kPolicy, kBoth>, what, most);
  const auto allow = [&](auto kernel, int64_t fixed) {
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, what, static_cast<int>(kRoom - 1024 - fixed));
  };
  constexpr int64_t distill = sizeof(StreamShared<kDistill>), policy = sizeof(StreamShared<kPolicy>);
  allow(loss_stream_kernel<float, kDistill, 2>, distill);
  allow(loss_stream_kernel<float, kDistill, 4>, distill);
  allow(loss_stream_kernel<__nv_bfloat16, kDistill, 2>, distill);
  allow(loss_stream_kernel<__nv_bfloat16, kDistill, 4>, distill);
  allow(loss_stream_kernel<float, kPolicy, 2>, policy);
  allow(loss_stream_kernel<float, kPolicy, 4>, policy);
  allow(loss_stream_kernel<__nv_bfloat16, kPolicy, 2>, policy);
  allow(loss_stream_kernel<__nv_bfloat16, kPolicy, 4>, policy);
  return e;
}

cudaError_t launch_distill_loss(const LossArgs& a, bool bf16, bool grad, bool backward, int num_sms,
                                cudaStream_t s) {
  return launch<kDistill>(a, bf16, grad, backward, num_sms, s);
}

cudaError_t launch_policy_loss(const LossArgs& a, bool bf16, bool grad, bool backward, int num_sms,
                               cudaStream_t s) {
  return launch<kPolicy>(a, bf16, grad, backward, num_sms, s);
}

}  // namespace muon
