// Token log probabilities, forward and backward, the clipped policy loss with its gradient
// and the preference loss over pairs of packed sequences (definitions in include/moe_lora.h).
//
// Rows of logits are long (a vocabulary) and pass through memory once: HBM is the bound.
// A row is cut into slices, one per block of a cluster; a block copies its slice into
// shared memory, 64 KB at most where that is enough, so that three blocks of an SM are at
// different points of their rows: some copy while others write.  A thread reads only what
// it copied itself, so its copies need no barrier.  It keeps a running maximum and sum over
// its own elements; the threads' pairs meet once, in distributed shared memory, and where a
// gradient is wanted it is formed from the slice in shared memory: one read and one write.
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "element.cuh"
#include "launch.h"
#include "prof.h"
#include "sm100_ptx.cuh"

namespace moelora {

namespace {

constexpr int kGroup = 4;            // vectors of a thread that are waited for together
constexpr int kRowThreads = 256;     // of a block that works on a slice of a row
constexpr int kShortThreads = 128;   // of a block whose warps have a row each
constexpr int kMaxCluster = 16;
constexpr int kMaxVocab = 1 << 19;
constexpr int kCountParts = 16;      // partial counts of an adapter's live tokens
constexpr int kTerms = 5;            // a loss and four statistics
constexpr int kSumThreads = 1024, kSumCluster = 8;
constexpr float kLog2e = 1.4426950408889634f;

struct Ranges {  // of adapters: tokens, or pairs
  int n;
  int64_t off[kMaxAdapters + 1];
};
// The range of index i: ranges end before the next begins, empty ones hold nothing.
__device__ __forceinline__ int range_of(const Ranges& r, int64_t i) {
  int a = 0;
  for (int j = 1; j < r.n; ++j) a += r.off[j] <= i;
  return a;
}

struct RowArgs {
  const void* x;
  int64_t ld, rows;
  int n;
  float inv_temp;
  const int32_t* targets;
  float *logp, *lse, *entropy;
  int* err;
};
struct PolicyArgs {
  const float *adv, *old, *ref, *weight, *dloss;
  float low, high, kl;  // borders of the ratio, weight of the KL term
  const int* count;     // [A][kCountParts] live tokens, where there are no weights
  float* terms;         // [kTerms][rows]
};
struct GradArgs {
  void* dx;
  int64_t ldd;
};

// 2^x, to 2 units in the last place; results below 2^-126 become 0.
__device__ __forceinline__ float ex2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Where a slice of a row lies: vectors of 16 aligned bytes, and single elements ahead of
// the row's first vector (first slice) and behind its last (last slice).
template <class T>
struct Slice {
  static constexpr int VL = 16 / sizeof(T);
  const T* p;      // the row
  int lead, count; // elements ahead of the first vector; vectors of this slice
  int first;       // column of the slice's first vector
  int edge;        // this thread's single element, -1 = none
  __device__ __forceinline__ Slice(const T* row, int n, int rank, int slices, int tid) : p(row) {
    const int off = (int)(reinterpret_cast<uintptr_t>(row) & 15) / (int)sizeof(T);
    lead = min(n, off ? VL - off : 0);
    const int all = (n - lead) / VL, per = (all + slices - 1) / slices;
    const int v0 = min(all, rank * per);
    count = min(per, all - v0);
    first = lead + v0 * VL;
    const int end = lead + all * VL;
    edge = rank == 0 && tid < lead                                          ? tid
           : rank == slices - 1 && tid >= VL && tid < VL + n - end ? end + tid - VL
                                                                            : -1;
  }
};

// Stores a vector at column c of a gradient row, whose alignment may differ from the logits'.
template <class T>
__device__ __forceinline__ void store_vec(T* row, int c, bool aligned, const Vec<T, 16 / sizeof(T)>& v) {
  if (aligned) {
    v.store(row + c, 0);
    return;
  }
  constexpr int kP = Vec<T, 16 / sizeof(T)>::kPairs;
#pragma unroll
  for (int i = 0; i < kP; ++i) {
    const float2 f = v.get(i);  // widened and narrowed again: exact
    row[c + 2 * i] = from_f32<T>(f.x);
    row[c + 2 * i + 1] = from_f32<T>(f.y);
  }
}
template <class T>
__device__ __forceinline__ bool same_phase(const T* a, const T* b) {
  return ((reinterpret_cast<uintptr_t>(a) ^ reinterpret_cast<uintptr_t>(b)) & 15) == 0;
}

// A target outside [0, n) other than -1 is noted and counts as -1.
__device__ __forceinline__ int checked_target(int y, int n, int* err, bool note) {
  if ((unsigned)y < (unsigned)n) return y;
  if (y != -1 && err && note) atomicOr(err, MOE_LORA_DEV_BAD_ID);
  return -1;
}

// Gradient row of zeros.
template <class T, int kTeam>
__device__ __forceinline__ void zero_slice(const Slice<T>& sl, T* out, bool aligned, int tid) {
  Vec<T, 16 / sizeof(T)> z;
  z.clear();
  for (int v = tid; v < sl.count; v += kTeam) store_vec<T>(out, sl.first + v * sl.VL, aligned, z);
  if (sl.edge >= 0) out[sl.edge] = from_f32<T>(0.f);
}

// d = q * e (+ coef at the target) for the eight (four) elements from column c on.
template <class T>
__device__ __forceinline__ Vec<T, 16 / sizeof(T)> grad_vec(const float2 (&e)[8 / sizeof(T)], float q, float coef, int c,
                                                           int y) {
  constexpr int VL = 16 / sizeof(T);
  float2 d[VL / 2];
#pragma unroll
  for (int i = 0; i < VL / 2; ++i) d[i] = mul2(e[i], both(q));
  if ((unsigned)(y - c) < (unsigned)VL) {
#pragma unroll
    for (int i = 0; i < VL / 2; ++i) {
      if (y - c == 2 * i) d[i].x += coef;
      if (y - c == 2 * i + 1) d[i].y += coef;
    }
  }
  Vec<T, VL> v;
#pragma unroll
  for (int i = 0; i < VL / 2; ++i) v.put(i, d[i]);
  return v;
}

// Log probabilities (kPolicy false), or the policy loss's terms and, with kGrad, its
// gradient.  kTeam threads work on a slice: a block's 256, or a warp whose slice is the row.
//
// Both reductions (the maximum, then the sums relative to it) are symmetric, so that every
// thread of the cluster has the same bits.
template <class T, int kTeam, int kGroups, bool kEntropy, bool kPolicy, bool kGrad>
__global__ void __launch_bounds__(kTeam == 32 ? kShortThreads : kTeam)
    token_row_kernel(const __grid_constant__ RowArgs g, const __grid_constant__ PolicyArgs pg,
                     const __grid_constant__ GradArgs dg, const __grid_constant__ Ranges ad, int slices) {
  constexpr int VL = 16 / sizeof(T), kP = VL / 2, kWarps = kTeam / 32;
  extern __shared__ __align__(16) uint8_t row_smem[];
  __shared__ float3 part[kMaxCluster * kWarps];
  __shared__ float at_target;
  const Ring<1, kGroups * kGroup> ring(row_smem);
  const int tid = threadIdx.x % kTeam, lane = threadIdx.x & 31, rank = kTeam == 32 ? 0 : blockIdx.x % slices;
  const int64_t t = kTeam == 32 ? (int64_t)blockIdx.x * (kShortThreads / 32) + (threadIdx.x >> 5) : blockIdx.x / slices;
  if (kPolicy) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (t >= g.rows) return;  // (a warp's own row)
  const T* row = static_cast<const T*>(g.x) + t * g.ld;
  const int y = checked_target(g.targets[t], g.n, g.err, rank == 0 && tid == 0);
  const Slice<T> sl(row, g.n, rank, slices, tid);
  T* out = kGrad ? static_cast<T*>(dg.dx) + t * dg.ldd : nullptr;
  const bool aligned = kGrad && same_phase(row, out);
  if (y < 0) {  // the same for the whole cluster, which has not met yet
    if (rank == 0 && tid == 0) {
      if (g.logp) g.logp[t] = 0.f;
      if (g.lse) g.lse[t] = 0.f;
      if (g.entropy) g.entropy[t] = 0.f;
      if (kPolicy)
#pragma unroll
        for (int i = 0; i < kTerms; ++i) pg.terms[i * g.rows + t] = 0.f;
    }
    if (kGrad) zero_slice<T, kTeam>(sl, out, aligned, tid);
    if (kPolicy) asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  // a thread's vectors: tid, tid + kTeam, ... of the slice
#pragma unroll
  for (int i = 0; i < kGroups * kGroup; ++i) {
    const int v = tid + i * kTeam;
    if (v < sl.count) async_copy16(ring.slot(0, i), row + sl.first + v * VL);
    if (i % kGroup == kGroup - 1) async_commit();
  }
  if (kTeam > 32 && slices > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  const float xe = sl.edge >= 0 ? to_f32(row[sl.edge]) : -INFINITY;
  // The target's logit is read before the block meets: a gradient may take its place afterwards.
  float xy = 0.f;
  if (kTeam == 32 || tid == 0) xy = to_f32(row[y]);
  if (kTeam > 32 && tid == 0) at_target = xy;
  float adv = 0.f, old = 0.f, ref = 0.f, wt = 1.f, up = 1.f;
  int a = 0;
  if (kPolicy) {
    a = range_of(ad, t);
    adv = pg.adv[t];
    old = pg.old[t];
    if (pg.ref) ref = pg.ref[t];
    if (pg.weight) wt = pg.weight[t];
    if (pg.dloss) up = pg.dloss[a];
  }

  const float c = g.inv_temp * kLog2e;
  // An empty place reads as -inf.
  const uint32_t none = sizeof(T) == 4 ? 0xFF800000u : std::is_same<T, __half>::value ? 0xFC00FC00u : 0xFF80FF80u;
  float m = -INFINITY;
  float2 s2 = both(0.f), w2 = both(0.f);
  const auto shift = [&](float top) {  // sums relative to the maximum so far, or 0 while there is none
    const float from = m, to = fmaxf(m, top), ref0 = to == -INFINITY ? 0.f : to;
    const float d = fmaxf((from - ref0) * c, -127.f), f = ex2_fast(d);
    if (kEntropy) w2 = mul2(fma2(s2, both(d), w2), both(f));
    s2 = mul2(s2, both(f));
    m = to;
    return ref0;
  };
#pragma unroll
  for (int gr = 0; gr < kGroups; ++gr) {
    if (gr * kGroup * kTeam >= sl.count) break;
    // groups behind this one may still be under way
    if (gr == kGroups - 1)
      async_wait<0>();
    else if (gr == kGroups - 2)
      async_wait<1>();
    else if (gr == kGroups - 3)
      async_wait<2>();
    else if (gr == kGroups - 4)
      async_wait<3>();
    else
      async_wait<4>();
    Vec<T, VL> u[kGroup];
    float top = -INFINITY;
#pragma unroll
    for (int j = 0; j < kGroup; ++j) {
      const int i = gr * kGroup + j;
      if (tid + i * kTeam < sl.count)
        u[j].from_smem(ring.slot(0, i));
      else
        u[j].w[0] = u[j].w[1] = u[j].w[2] = u[j].w[3] = none;
#pragma unroll
      for (int p = 0; p < kP; ++p) {
        const float2 f = u[j].get(p);
        top = fmaxf(top, fmaxf(f.x, f.y));
      }
    }
    const float r = shift(top);
#pragma unroll
    for (int j = 0; j < kGroup; ++j)
#pragma unroll
      for (int p = 0; p < kP; ++p) {
        float2 x = mul2(add2(u[j].get(p), both(-r)), both(c));
        const float2 e = make_float2(ex2_fast(x.x), ex2_fast(x.y));
        s2 = add2(s2, e);
        // 0 * -inf is 0 here, and a NaN stays one in e
        if (kEntropy) w2 = fma2(e, make_float2(fmaxf(x.x, -127.f), fmaxf(x.y, -127.f)), w2);
      }
  }
  async_wait<0>();
  if (sl.edge >= 0) {
    const float r = shift(xe);
    const float x = (xe - r) * c, e = ex2_fast(x);
    s2.x += e;
    if (kEntropy) w2.x += e * fmaxf(x, -127.f);
  }
  // the warp's, then the cluster's maximum and sums
  float s = s2.x + s2.y, w = w2.x + w2.y;
  const auto meet = [&](float top, float mine, float& sum, float& wsum) {  // sum relative to `mine` -> to `top`
    const float d = fmaxf((mine - (top == -INFINITY ? 0.f : top)) * c, -127.f), f = ex2_fast(d);
    if (kEntropy) wsum = f * (wsum + sum * d);
    sum *= f;
  };
  float top = m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  meet(top, m, s, w);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s += __shfl_xor_sync(0xffffffffu, s, o);
    if (kEntropy) w += __shfl_xor_sync(0xffffffffu, w, o);
  }
  m = top;
  if (kTeam > 32) {
    const int warp = threadIdx.x >> 5;
    if (slices > 1) {
      asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // all blocks have started
      if (lane < slices) {
        const uint32_t at = mapa_shared(smem_u32(&part[rank * kWarps + warp]), lane);
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(m) : "memory");
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at + 4), "f"(s) : "memory");
        if (kEntropy) asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at + 8), "f"(w) : "memory");
      }
      cluster_sync_all();
    } else {
      if (lane == 0) part[warp] = make_float3(m, s, w);
      __syncthreads();
    }
    xy = at_target;
    const int all = slices * kWarps;
    constexpr int kParts = (kMaxCluster * kWarps + 31) / 32;
    float mi[kParts];
    top = -INFINITY;
#pragma unroll
    for (int i = 0; i < kParts; ++i) {
      mi[i] = lane + 32 * i < all ? part[lane + 32 * i].x : -INFINITY;
      top = fmaxf(top, mi[i]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    s = w = 0.f;
#pragma unroll
    for (int i = 0; i < kParts; ++i)
      if (lane + 32 * i < all) {
        float si = part[lane + 32 * i].y, wi = kEntropy ? part[lane + 32 * i].z : 0.f;
        meet(top, mi[i], si, wi);
        s += si;
        w += wi;
      }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      s += __shfl_xor_sync(0xffffffffu, s, o);
      if (kEntropy) w += __shfl_xor_sync(0xffffffffu, w, o);
    }
    m = top;
  }
  const float r = m == -INFINITY ? 0.f : m, ls = logf(s);
  // target minus maximum first: their difference is what counts, not their size
  const float logp = (xy - m) * g.inv_temp - ls;
  const float inv_s = 1.0f / s, entropy = kEntropy ? ls - w * inv_s * 0.6931471805599453f : 0.f;
  const bool scribe = rank == 0 && tid == 0;
  if (kPolicy && !pg.weight) {
    // the counts, and with them every launch that the sums behind this one rely on
    asm volatile("griddepcontrol.wait;" ::: "memory");
    int k = 0;
    if (kGrad)
#pragma unroll
      for (int i = 0; i < kCountParts; ++i) k += pg.count[a * kCountParts + i];
    up /= (float)max(k, 1);
  }
  if (scribe) {
    if (g.logp) g.logp[t] = logp;
    if (g.lse) g.lse[t] = m * g.inv_temp + ls;
    if (g.entropy) g.entropy[t] = entropy;
  }
  if (!kPolicy) return;
  const float rho = expf(logp - old), clip = fminf(fmaxf(rho, pg.low), pg.high);
  const bool cut = (adv > 0.f && rho > pg.high) || (adv < 0.f && rho < pg.low);
  float loss = -(cut ? clip : rho) * adv, kl = 0.f, dl = cut ? 0.f : -rho * adv;
  if (pg.ref) {
    const float d = ref - logp, em = expm1f(d);
    kl = em - d;
    loss += pg.kl * kl;
    dl -= pg.kl * em;
  }
  if (scribe) {  // a token of weight 0 has no part in the loss, whatever its values
    float* to = pg.terms + t;
    to[0] = wt == 0.f ? 0.f : wt * loss;
    to[g.rows] = wt == 0.f ? 0.f : wt * kl;
    to[2 * g.rows] = cut ? wt : 0.f;
    to[3 * g.rows] = wt == 0.f ? 0.f : wt * rho;
    to[4 * g.rows] = wt == 0.f ? 0.f : wt * entropy;
  }
  if (!kGrad) return;
  if (wt == 0.f) {
    zero_slice<T, kTeam>(sl, out, aligned, tid);
    return;
  }
  const float coef = up * wt * dl * g.inv_temp, q = -coef * inv_s;
#pragma unroll
  for (int i = 0; i < kGroups * kGroup; ++i) {
    const int v = tid + i * kTeam;
    if (v >= sl.count) break;
    Vec<T, VL> u;
    u.from_smem(ring.slot(0, i));
    float2 e[kP];
#pragma unroll
    for (int p = 0; p < kP; ++p) {
      const float2 x = mul2(add2(u.get(p), both(-r)), both(c));
      e[p] = make_float2(ex2_fast(x.x), ex2_fast(x.y));
    }
    store_vec<T>(out, sl.first + v * VL, aligned, grad_vec<T>(e, q, coef, sl.first + v * VL, y));
  }
  if (sl.edge >= 0) out[sl.edge] = from_f32<T>(q * ex2_fast((xe - r) * c) + (sl.edge == y ? coef : 0.f));
}

// dlogits from a saved lse: no reduction, every element on its own.  A block takes up to
// kBwdVecs vectors a thread of one row, all their loads under way together.
constexpr int kBwdThreads = 256, kBwdVecs = 4;
template <class T, int kTeam>
__global__ void __launch_bounds__(kBwdThreads)
    token_bwd_kernel(const __grid_constant__ RowArgs g, const __grid_constant__ GradArgs dg, const float* dlogp, int slices) {
  constexpr int VL = 16 / sizeof(T), kP = VL / 2;
  const int tid = threadIdx.x % kTeam;
  const int rank = kTeam == 32 ? 0 : blockIdx.x % slices;
  const int64_t t = kTeam == 32 ? (int64_t)blockIdx.x * (kBwdThreads / 32) + threadIdx.x / 32 : blockIdx.x / slices;
  if (t >= g.rows) return;
  const T* row = static_cast<const T*>(g.x) + t * g.ld;
  T* out = static_cast<T*>(dg.dx) + t * dg.ldd;
  const int y = checked_target(g.targets[t], g.n, g.err, rank == 0 && tid == 0);
  const Slice<T> sl(row, g.n, rank, slices, tid);
  const bool aligned = same_phase(row, out);
  const float up = y < 0 ? 0.f : dlogp[t];
  if (up == 0.f) {
    zero_slice<T, kTeam>(sl, out, aligned, tid);
    return;
  }
  const float coef = up * g.inv_temp, lse = g.lse[t];
  const float xe = sl.edge >= 0 ? to_f32(row[sl.edge]) : 0.f;
  for (int v0 = tid; v0 < sl.count; v0 += kBwdVecs * kTeam) {
    Vec<T, VL> u[kBwdVecs];
#pragma unroll
    for (int j = 0; j < kBwdVecs; ++j)
      if (v0 + j * kTeam < sl.count) u[j].load(row + sl.first + (v0 + j * kTeam) * VL, 0);
#pragma unroll
    for (int j = 0; j < kBwdVecs; ++j) {
      const int v = v0 + j * kTeam;
      if (v >= sl.count) break;
      float2 e[kP];
#pragma unroll
      for (int p = 0; p < kP; ++p) {
        // the difference first: its rounding is relative to itself, not to the logits' size
        const float2 x = mul2(fma2(u[j].get(p), both(g.inv_temp), both(-lse)), both(kLog2e));
        e[p] = make_float2(ex2_fast(x.x), ex2_fast(x.y));
      }
      store_vec<T>(out, sl.first + v * VL, aligned, grad_vec<T>(e, -coef, coef, sl.first + v * VL, y));
    }
  }
  if (sl.edge >= 0) out[sl.edge] = from_f32<T>(-coef * ex2_fast(fmaf(xe, g.inv_temp, -lse) * kLog2e) + (sl.edge == y ? coef : 0.f));
}

// Live tokens of each adapter in kCountParts parts.
__global__ void __launch_bounds__(256) token_count_kernel(const int32_t* targets, int n, const __grid_constant__ Ranges ad, int* count) {
  __shared__ int sum;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int a = blockIdx.x / kCountParts, part = blockIdx.x % kCountParts;
  if (threadIdx.x == 0) sum = 0;
  __syncthreads();
  int c = 0;
#pragma unroll 8
  for (int64_t t = ad.off[a] + part * 256 + threadIdx.x; t < ad.off[a + 1]; t += kCountParts * 256)
    c += (unsigned)targets[t] < (unsigned)n;
  c = __reduce_add_sync(0xffffffffu, c);
  if ((threadIdx.x & 31) == 0 && c) atomicAdd(&sum, c);
  __syncthreads();
  if (threadIdx.x == 0) count[blockIdx.x] = sum;
}

// Sums of an adapter's terms, a cluster per adapter: thread i of the cluster adds its
// elements i, i + 8192, ... in order, then warps, block and cluster.  Where every adapter
// has at most 1024 elements the first block alone has any, and runs alone: the same sums.
struct SumArgs {
  const float* terms;  // [kTerms][stride]
  int64_t stride;
  const int* count;    // live tokens (NULL: see by_range)
  bool by_range;       // divide by the range's length
  float *loss, *stats;
};
template <int kC>
__global__ void __launch_bounds__(kSumThreads) term_sum_kernel(const __grid_constant__ SumArgs g, const __grid_constant__ Ranges ad) {
  __shared__ float warp_sum[kSumThreads / 32][kTerms], block_sum[kTerms];
  const int a = blockIdx.x / kC, rank = kC > 1 ? (int)cluster_rank() : 0;
  const int64_t lo = ad.off[a], hi = ad.off[a + 1];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float s[kTerms] = {};
#pragma unroll 2
  for (int64_t i = lo + rank * kSumThreads + threadIdx.x; i < hi; i += kSumCluster * kSumThreads)
#pragma unroll
    for (int k = 0; k < kTerms; ++k) s[k] += g.terms[k * g.stride + i];
#pragma unroll
  for (int k = 0; k < kTerms; ++k) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s[k] += __shfl_xor_sync(0xffffffffu, s[k], o);
    if ((threadIdx.x & 31) == 0) warp_sum[threadIdx.x >> 5][k] = s[k];
  }
  __syncthreads();
  const int k = threadIdx.x >> 5, lane = threadIdx.x & 31;  // a warp per term
  if (k < kTerms) {
    float v = warp_sum[lane][k];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (lane == 0) block_sum[k] = v;
  }
  if (kC > 1)
    cluster_sync_all();
  else
    __syncthreads();
  if (rank == 0 && k < kTerms) {
    float v = 0.f;
    if (lane < kC) {
      if (kC > 1)
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(mapa_shared(smem_u32(&block_sum[k]), lane)) : "memory");
      else
        v = block_sum[k];
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (lane == 0) {
      float by = 1.f;
      if (g.count) {
        int n = 0;
        for (int i = 0; i < kCountParts; ++i) n += g.count[a * kCountParts + i];
        by = 1.0f / (float)max(n, 1);
      } else if (g.by_range) {
        by = 1.0f / (float)max(hi - lo, (int64_t)1);
      }
      if (k == 0)
        g.loss[a] = v * by;
      else
        g.stats[a * (kTerms - 1) + k - 1] = v * by;
    }
  }
  if (kC > 1) cluster_sync_all();  // nobody leaves while its sums are read
}

// ------------------------------------------------------------------ preference loss
struct PrefArgs {
  const float* logp;
  const int32_t* targets;
  int64_t T;
  const int64_t* seq;
  const float* ref;
  float beta, margin, smooth;
  int kind, average;
  const float* dloss;
  float *seq_logp, *dlogp;
  float* terms;  // [kTerms][pairs]
  int64_t pairs;
  int* err;
};
// A block per pair: sums of both sequences (64 bits from the threads' own sums on, since
// the loss lives on the difference of two large sums), the pair's terms, then the gradient.
template <int kThreads>
__global__ void __launch_bounds__(kThreads) pref_kernel(const __grid_constant__ PrefArgs g, const __grid_constant__ Ranges ad) {
  __shared__ double sums[2][kThreads / 32];
  __shared__ int counts[2][kThreads / 32];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t i = blockIdx.x;
  int64_t off[3];
  bool bad = false;
  for (int j = 0; j < 3; ++j) {  // offsets that go back or past the end are noted; what is left of them is inside
    const int64_t o = g.seq[2 * i + j], at = max(j ? off[j - 1] : (int64_t)0, min(o, g.T));
    bad |= at != o;
    off[j] = at;
  }
  if (bad && g.err && threadIdx.x == 0) atomicOr(g.err, MOE_LORA_DEV_BAD_ID);
  // everything below is of the sequence whose half of the block this is
  constexpr int kHalf = kThreads / 2;
  const int j = threadIdx.x / kHalf, tid = threadIdx.x % kHalf, lane = threadIdx.x & 31, warp = tid >> 5;
  float s = 0.f;
  int n = 0;
#pragma unroll 4
  for (int64_t t = off[j] + tid; t < off[j + 1]; t += kHalf) {
    const bool live = g.targets[t] >= 0;
    s += live ? g.logp[t] : 0.f;
    n += live;
  }
  double d = s;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
  n = __reduce_add_sync(0xffffffffu, n);
  if (lane == 0) {
    sums[j][warp] = d;
    counts[j][warp] = n;
  }
  __syncthreads();
  double tot[2];
  int cnt[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    tot[q] = 0;
    cnt[q] = 0;
    for (int w = 0; w < kHalf / 32; ++w) {
      tot[q] += sums[q][w];
      cnt[q] += counts[q][w];
    }
    if (g.average) tot[q] /= max(cnt[q], 1);
  }
  const double rc = tot[0] - (g.ref ? (double)g.ref[2 * i] : 0.0), rr = tot[1] - (g.ref ? (double)g.ref[2 * i + 1] : 0.0);
  const double hd = rc - rr;
  const float h = (float)hd, x = (float)(g.beta * hd - g.margin);
  float loss, dh;
  if (g.kind == MOE_LORA_PREF_SIGMOID) {
    const float e = expf(-fabsf(x)), soft = log1pf(e), near = e / (1.f + e);  // 1 - sigmoid(|x|)
    loss = (1.f - g.smooth) * (soft + fmaxf(-x, 0.f)) + g.smooth * (soft + fmaxf(x, 0.f));
    // sigmoid(x) - (1 - smooth) without the difference of two numbers near 1
    dh = g.beta * (x >= 0.f ? g.smooth - near : near - (1.f - g.smooth));
  } else if (g.kind == MOE_LORA_PREF_SQUARED) {
    const float o = (float)(hd - 0.5 / (double)g.beta);
    loss = o * o;
    dh = 2.f * o;
  } else {
    loss = fmaxf(1.f - x, 0.f);
    dh = x < 1.f ? -g.beta : 0.f;
    if (isnan(x)) loss = dh = x;
  }
  const int a = range_of(ad, i);
  if (threadIdx.x == 0) {
    float* to = g.terms + i;
    to[0] = loss;
    to[g.pairs] = x > 0.f ? 1.f : 0.f;
    to[2 * g.pairs] = (float)(g.beta * rc);
    to[3 * g.pairs] = (float)(g.beta * rr);
    to[4 * g.pairs] = h;
    if (g.seq_logp) {
      g.seq_logp[2 * i] = (float)tot[0];
      g.seq_logp[2 * i + 1] = (float)tot[1];
    }
  }
  if (!g.dlogp) return;
  const float up = (g.dloss ? g.dloss[a] : 1.f) / (float)(ad.off[a + 1] - ad.off[a]);
  const float v = up * dh * (j ? -1.f : 1.f) / (g.average ? (float)max(cnt[j], 1) : 1.f);
#pragma unroll 4
  for (int64_t t = off[j] + tid; t < off[j + 1]; t += kHalf) g.dlogp[t] = g.targets[t] >= 0 ? v : 0.f;
}

// ------------------------------------------------------------------ host
struct RowLaunch {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[2];
  RowLaunch(int64_t grid, int threads, size_t smem, int cluster, bool overlap, cudaStream_t s) {
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = at;
    if (overlap) {
      at[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
      at[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (cluster > 1) {
      at[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
      at[cfg.numAttrs].val.clusterDim.x = cluster;
      at[cfg.numAttrs].val.clusterDim.y = at[cfg.numAttrs].val.clusterDim.z = 1;
      ++cfg.numAttrs;
    }
  }
};

int check_rows(const moe_lora_rows* r) {
  if (!r) return MOE_LORA_ERR_NULL;
  if (!dtype_ok(r->dtype)) return MOE_LORA_ERR_UNSUPPORTED;
  if (r->rows < 0 || r->rows > (int64_t)1 << 26 || r->n < 1) return MOE_LORA_ERR_DIMS;
  if (r->n > kMaxVocab) return MOE_LORA_ERR_UNSUPPORTED;
  if ((r->ld && r->ld < r->n) || (r->ldd && r->ldd < r->n) || r->ld > (int64_t)1 << 32 || r->ldd > (int64_t)1 << 32)
    return MOE_LORA_ERR_DIMS;
  // the base-2 scale has to be a normal number
  if (!(r->inv_temp >= 1e-30f) || !(r->inv_temp <= 1e30f)) return MOE_LORA_ERR_DIMS;
  return MOE_LORA_OK;
}
RowArgs row_args(const moe_lora_rows* r, const void* x, const int32_t* targets, float* logp, float* lse, float* entropy, int32_t* err) {
  return RowArgs{x, r->ld ? r->ld : r->n, r->rows, r->n, r->inv_temp, targets, logp, lse, entropy, err};
}

template <class T, int kTeam, int kGroups, bool kEntropy, bool kPolicy, bool kGrad>
int launch_rows(const RowArgs& g, const PolicyArgs& pg, const GradArgs& dg, const Ranges& ad, int slices, bool overlap, cudaStream_t s) {
  const int64_t grid = kTeam == 32 ? (g.rows + kShortThreads / 32 - 1) / (kShortThreads / 32) : g.rows * slices;
  const int threads = kTeam == 32 ? kShortThreads : kTeam;
  const RowLaunch l(grid, threads, ring_bytes<1, kGroups * kGroup>(threads), slices, overlap, s);
  const int slot = kPolicy ? K_POLICY : K_TOKEN_FWD;
  prof_begin(slot, s);
  const cudaError_t e = launch_allowed(l.cfg, slices > 8, token_row_kernel<T, kTeam, kGroups, kEntropy, kPolicy, kGrad>, g, pg, dg, ad, slices);
  prof_end(slot, s);
  return e == cudaSuccess ? MOE_LORA_OK : MOE_LORA_ERR_CUDA;
}

// Slices of a row and what a block holds of it.  Rows of a few thousand elements belong to
// a warp.  Longer ones to the fewest blocks that hold 64 KB each (128 KB beyond eight), and
// to more, up to eight, where there are too few rows to give every SM a block.
template <class T, bool kEntropy, bool kPolicy, bool kGrad>
int pick_rows(const RowArgs& g, const PolicyArgs& pg, const GradArgs& dg, const Ranges& ad, int sms, bool overlap, cudaStream_t s) {
  constexpr int VL = 16 / sizeof(T);
  const int vecs = g.n / VL;
  if (vecs <= 32 * kGroup) return launch_rows<T, 32, 1, kEntropy, kPolicy, kGrad>(g, pg, dg, ad, 1, overlap, s);
  if (vecs <= 32 * 4 * kGroup && g.rows >= sms) return launch_rows<T, 32, 4, kEntropy, kPolicy, kGrad>(g, pg, dg, ad, 1, overlap, s);
  constexpr int one = kRowThreads * kGroup;  // vectors of a group of a block
  const auto need = [&](int per) { return (vecs + per - 1) / per; };
  int slices = need(4 * one);
  if (slices > 8) slices = std::max(8, need(8 * one));
  while (slices < 8 && g.rows * (slices + 1) <= sms && vecs / (slices + 1) >= kRowThreads) ++slices;
  const int per = (vecs + slices - 1) / slices;
  return per <= one       ? launch_rows<T, kRowThreads, 1, kEntropy, kPolicy, kGrad>(g, pg, dg, ad, slices, overlap, s)
         : per <= 2 * one ? launch_rows<T, kRowThreads, 2, kEntropy, kPolicy, kGrad>(g, pg, dg, ad, slices, overlap, s)
         : per <= 4 * one ? launch_rows<T, kRowThreads, 4, kEntropy, kPolicy, kGrad>(g, pg, dg, ad, slices, overlap, s)
                          : launch_rows<T, kRowThreads, 8, kEntropy, kPolicy, kGrad>(g, pg, dg, ad, slices, overlap, s);
}
template <class T>
int run_logp(const RowArgs& g, int sms, cudaStream_t s) {
  return g.entropy ? pick_rows<T, true, false, false>(g, {}, {}, {}, sms, false, s)
                   : pick_rows<T, false, false, false>(g, {}, {}, {}, sms, false, s);
}
template <class T>
int run_policy(const RowArgs& g, const PolicyArgs& pg, const GradArgs& dg, const Ranges& ad, int sms, bool overlap, cudaStream_t s) {
  return dg.dx ? pick_rows<T, true, true, true>(g, pg, dg, ad, sms, overlap, s)
               : pick_rows<T, true, true, false>(g, pg, dg, ad, sms, overlap, s);
}
template <class T>
int run_bwd(const RowArgs& g, const GradArgs& dg, const float* dlogp, cudaStream_t s) {
  constexpr int VL = 16 / sizeof(T);
  const int vecs = g.n / VL, slices = std::max(1, (vecs + kBwdThreads * kBwdVecs - 1) / (kBwdThreads * kBwdVecs));
  prof_begin(K_TOKEN_BWD, s);
  if (vecs <= 32 * kBwdVecs)
    token_bwd_kernel<T, 32><<<(unsigned)((g.rows + kBwdThreads / 32 - 1) / (kBwdThreads / 32)), kBwdThreads, 0, s>>>(g, dg, dlogp, 1);
  else
    token_bwd_kernel<T, kBwdThreads><<<(unsigned)(g.rows * slices), kBwdThreads, 0, s>>>(g, dg, dlogp, slices);
  prof_end(K_TOKEN_BWD, s);
  return cudaGetLastError() == cudaSuccess ? MOE_LORA_OK : MOE_LORA_ERR_CUDA;
}

// Adapters' ranges of n items from the caller's offsets [A + 1] on the host (NULL allowed for one).
int make_ranges(int A, const int64_t* off, int64_t n, Ranges* r) {
  if (A < 1 || A > kMaxAdapters) return MOE_LORA_ERR_DIMS;
  if (A > 1 && !off) return MOE_LORA_ERR_NULL;
  r->n = A;
  for (int a = 0; a <= A; ++a) {
    r->off[a] = off ? off[a] : a ? n : 0;
    if (r->off[a] < (a ? r->off[a - 1] : 0) || r->off[a] > n) return MOE_LORA_ERR_DIMS;
  }
  return r->off[0] != 0 || r->off[A] != n ? MOE_LORA_ERR_DIMS : MOE_LORA_OK;
}

int launch_sums(const SumArgs& g, const Ranges& ad, cudaStream_t s) {
  int64_t most = 0;
  for (int a = 0; a < ad.n; ++a) most = std::max(most, ad.off[a + 1] - ad.off[a]);
  const bool one = most <= kSumThreads;
  const RowLaunch l((int64_t)ad.n * (one ? 1 : kSumCluster), kSumThreads, 0, one ? 1 : kSumCluster, true, s);
  prof_begin(K_TERM_SUM, s);
  const cudaError_t e = one ? cudaLaunchKernelEx(&l.cfg, term_sum_kernel<1>, g, ad) : cudaLaunchKernelEx(&l.cfg, term_sum_kernel<kSumCluster>, g, ad);
  prof_end(K_TERM_SUM, s);
  return e == cudaSuccess ? MOE_LORA_OK : MOE_LORA_ERR_CUDA;
}

// Scratch of the losses: the items' terms, then the adapters' partial counts.
size_t terms_bytes(int64_t items) { return align_up(sizeof(float) * kTerms * (size_t)std::max<int64_t>(items, 1), 256); }

}  // namespace

}  // namespace moelora

using namespace moelora;

extern "C" int moe_lora_token_logp_forward(const moe_lora_rows* r, const void* logits, const int32_t* targets, float* logp,
                                           float* lse, float* entropy, int32_t* err, void* stream) {
  int rc = check_rows(r);
  if (rc) return rc;
  if (reinterpret_cast<uintptr_t>(err) & 3u) return MOE_LORA_ERR_ALIGN;
  if ((rc = check_opt(logp)) || (rc = check_opt(lse)) || (rc = check_opt(entropy))) return rc;
  if (r->rows == 0) return MOE_LORA_OK;
  if (!logp && !lse && !entropy) return MOE_LORA_ERR_NULL;
  if ((rc = check_ptr(logits)) || (rc = check_ptr(targets))) return rc;
  int sms;
  if ((rc = device_sms(&sms))) return rc;
  const RowArgs g = row_args(r, logits, targets, logp, lse, entropy, err);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return r->dtype == MOE_LORA_F32    ? run_logp<float>(g, sms, s)
         : r->dtype == MOE_LORA_BF16 ? run_logp<__nv_bfloat16>(g, sms, s)
                                     : run_logp<__half>(g, sms, s);
}

extern "C" int moe_lora_token_logp_backward(const moe_lora_rows* r, const void* logits, const int32_t* targets,
                                            const float* lse, const float* dlogp, void* dlogits, int32_t* err, void* stream) {
  int rc = check_rows(r);
  if (rc) return rc;
  if (reinterpret_cast<uintptr_t>(err) & 3u) return MOE_LORA_ERR_ALIGN;
  if (r->rows == 0) return MOE_LORA_OK;
  if ((rc = check_ptr(logits)) || (rc = check_ptr(targets)) || (rc = check_ptr(lse)) || (rc = check_ptr(dlogp)) ||
      (rc = check_ptr(dlogits)))
    return rc;
  const GradArgs dg{dlogits, r->ldd ? r->ldd : r->n};
  const RowArgs g = row_args(r, logits, targets, nullptr, const_cast<float*>(lse), nullptr, err);
  if (logits == dlogits && dg.ldd != g.ld) return MOE_LORA_ERR_DIMS;
  int sms;
  if ((rc = device_sms(&sms))) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return r->dtype == MOE_LORA_F32    ? run_bwd<float>(g, dg, dlogp, s)
         : r->dtype == MOE_LORA_BF16 ? run_bwd<__nv_bfloat16>(g, dg, dlogp, s)
                                     : run_bwd<__half>(g, dg, dlogp, s);
}

extern "C" size_t moe_lora_policy_scratch_bytes(int64_t rows, int32_t adapters) {
  if (rows < 0 || rows > (int64_t)1 << 26 || adapters < 1 || adapters > kMaxAdapters) return 0;
  return terms_bytes(rows) + align_up(sizeof(int) * kCountParts * adapters, 256);
}

extern "C" int moe_lora_policy_loss(const moe_lora_rows* r, const moe_lora_policy* o, const void* logits, const int32_t* targets,
                                    const float* advantages, const float* old_logp, const float* ref_logp, const float* weight,
                                    const int64_t* adapter_offsets, const float* dloss, float* loss, float* stats, float* logp,
                                    void* dlogits, int32_t* err, void* scratch, size_t scratch_bytes, void* stream) {
  int rc = check_rows(r);
  if (rc) return rc;
  if (!o) return MOE_LORA_ERR_NULL;
  if (!(o->clip_low >= 0.f && o->clip_low <= 1.f) || !(o->clip_high >= 0.f) || !isfinite(o->clip_high) || !isfinite(o->kl_coef))
    return MOE_LORA_ERR_DIMS;
  Ranges ad;
  if ((rc = make_ranges(o->adapters, adapter_offsets, r->rows, &ad))) return rc;
  if (reinterpret_cast<uintptr_t>(err) & 3u) return MOE_LORA_ERR_ALIGN;
  if ((rc = check_ptr(loss)) || (rc = check_ptr(stats)) || (rc = check_ptr(scratch)) || (rc = check_opt(ref_logp)) ||
      (rc = check_opt(weight)) || (rc = check_opt(dloss)) || (rc = check_opt(logp)) || (rc = check_opt(dlogits)))
    return rc;
  if (scratch_bytes < moe_lora_policy_scratch_bytes(r->rows, o->adapters)) return MOE_LORA_ERR_WORKSPACE;
  if (r->rows > 0 && ((rc = check_ptr(logits)) || (rc = check_ptr(targets)) || (rc = check_ptr(advantages)) || (rc = check_ptr(old_logp))))
    return rc;
  const GradArgs dg{dlogits, r->ldd ? r->ldd : r->n};
  const RowArgs g = row_args(r, logits, targets, logp, nullptr, nullptr, err);
  if (dlogits && logits == dlogits && dg.ldd != g.ld) return MOE_LORA_ERR_DIMS;
  int sms;
  if ((rc = device_sms(&sms))) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int* count = reinterpret_cast<int*>(static_cast<char*>(scratch) + terms_bytes(r->rows));
  PolicyArgs pg{advantages, old_logp, ref_logp, weight, dloss, 1.f - o->clip_low, 1.f + o->clip_high, o->kl_coef, count,
                static_cast<float*>(scratch)};
  if (!weight) {
    prof_begin(K_TOKEN_COUNT, s);
    token_count_kernel<<<ad.n * kCountParts, 256, 0, s>>>(targets, r->n, ad, count);
    prof_end(K_TOKEN_COUNT, s);
    if (cudaGetLastError() != cudaSuccess) return MOE_LORA_ERR_CUDA;
  }
  if (r->rows > 0) {
    rc = r->dtype == MOE_LORA_F32    ? run_policy<float>(g, pg, dg, ad, sms, !weight, s)
         : r->dtype == MOE_LORA_BF16 ? run_policy<__nv_bfloat16>(g, pg, dg, ad, sms, !weight, s)
                                     : run_policy<__half>(g, pg, dg, ad, sms, !weight, s);
    if (rc) return rc;
  }
  return launch_sums(SumArgs{static_cast<float*>(scratch), r->rows, weight ? nullptr : count, false, loss, stats}, ad, s);
}

extern "C" size_t moe_lora_preference_scratch_bytes(int64_t pairs) {
  return pairs < 0 || pairs > (int64_t)1 << 26 ? 0 : terms_bytes(pairs);
}

extern "C" int moe_lora_preference_loss(const moe_lora_preference* o, const float* logp, const int32_t* targets,
                                        const int64_t* seq_offsets, const float* ref, const int64_t* pair_offsets,
                                        const float* dloss, float* loss, float* stats, float* seq_logp, float* dlogp,
                                        int32_t* err, void* scratch, size_t scratch_bytes, void* stream) {
  if (!o) return MOE_LORA_ERR_NULL;
  if (o->kind < 0 || o->kind > MOE_LORA_PREF_HINGE) return MOE_LORA_ERR_UNSUPPORTED;
  if (o->tokens < 0 || o->tokens > (int64_t)1 << 40 || o->pairs < 0 || o->pairs > (int64_t)1 << 26) return MOE_LORA_ERR_DIMS;
  if (!(o->beta > 0.f) || !isfinite(o->beta) || !isfinite(o->margin) || !(o->label_smoothing >= 0.f && o->label_smoothing <= 0.5f))
    return MOE_LORA_ERR_DIMS;
  Ranges ad;
  int rc = make_ranges(o->adapters, pair_offsets, o->pairs, &ad);
  if (rc) return rc;
  if (reinterpret_cast<uintptr_t>(err) & 3u) return MOE_LORA_ERR_ALIGN;
  if ((rc = check_ptr(loss)) || (rc = check_ptr(stats)) || (rc = check_ptr(scratch)) || (rc = check_opt(ref)) || (rc = check_opt(dloss)) ||
      (rc = check_opt(seq_logp)) || (rc = check_opt(dlogp)))
    return rc;
  if (scratch_bytes < moe_lora_preference_scratch_bytes(o->pairs)) return MOE_LORA_ERR_WORKSPACE;
  if (o->pairs > 0 && (rc = check_ptr(seq_offsets))) return rc;
  if (o->pairs > 0 && o->tokens > 0 && ((rc = check_ptr(logp)) || (rc = check_ptr(targets)))) return rc;
  int sms;
  if ((rc = device_sms(&sms))) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  float* terms = static_cast<float*>(scratch);
  if (o->pairs > 0) {
    const PrefArgs g{logp, targets, o->tokens, seq_offsets, ref, o->beta, o->margin, o->label_smoothing, o->kind, o->average,
                     dloss, seq_logp, dlogp, terms, o->pairs, err};
    // sequences of a thousand tokens and more get a large block
    const bool wide = o->tokens / (2 * o->pairs) >= 1024;
    prof_begin(K_PREF, s);
    if (wide)
      pref_kernel<1024><<<(unsigned)o->pairs, 1024, 0, s>>>(g, ad);
    else
      pref_kernel<256><<<(unsigned)o->pairs, 256, 0, s>>>(g, ad);
    prof_end(K_PREF, s);
    if (cudaGetLastError() != cudaSuccess) return MOE_LORA_ERR_CUDA;
  }
  return launch_sums(SumArgs{terms, o->pairs, nullptr, true, loss, stats}, ad, s);
}
