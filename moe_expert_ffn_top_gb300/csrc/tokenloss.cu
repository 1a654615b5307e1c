// Token log probabilities, forward and backward, the clipped policy loss with its gradient
// and the preference loss over pairs of packed sequences (definitions in include/moe_lora.h).
//
// Rows of logits are long (a vocabulary) and pass through memory once: HBM is the bound.
// A row is cut into slices, one per block of a cluster; a block copies its slice into
// shared memory, 32 KB at most where that is enough, so that six blocks of an SM are at
// different points of their rows: some copy while others write.  A thread reads only what
// it copied itself, so its copies need no barrier.  It keeps a running maximum and sum over
// its own elements; the threads' pairs meet once, in distributed shared memory, and where a
// gradient is wanted it is formed from the slice in shared memory: one read and one write.
//
// Measured on one GB300 (GPU time): the policy loss with its gradient over 8,192 x 151,936 bf16, 30% of the rows
// without a target, 680 us (6.2 TB/s, 92% of the measured copy bandwidth); log probabilities with
// entropies of 16,384 x 65,536 bf16 341 us (5.7 TB/s, 83%), their backward 639 us (94%); the preference
// loss of 1,024 pairs of 1,400 tokens 14 us.
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
constexpr int kRowThreads = 128;     // of a block that works on a slice of a row
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
  float inv_temp, c, up, floor;  // see Temper
  const int32_t* targets;
  float *logp, *lse, *entropy;
  int* err;
};
struct PolicyArgs {
  const float *adv, *old, *ref, *weight, *dloss;
  float low, high, kl;  // borders of the ratio, weight of the KL term
  const int* count;     // [A][kCountParts] live tokens, where there are no weights
  float* terms;         // [kTerms][rows]
  bool few;             // so few rows that the last one done adds the terms
  unsigned* ticket;     // of those
  float *loss, *stats;
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
  // `per` vectors to a slice; enough for the row
  __device__ __forceinline__ Slice(const T* row, int n, int rank, int slices, int per, int tid) : p(row) {
    const int off = (int)(reinterpret_cast<uintptr_t>(row) & 15) / (int)sizeof(T);
    lead = min(n, off ? VL - off : 0);
    const int all = (n - lead) / VL;
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

// The largest value of a warp's lanes (NaN is passed over).
__device__ __forceinline__ float warp_top(float v) {
  float r;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
// A reference M, the sum of 2^(x c - M) and of that times x c - M.  M is the maximum of x c rounded
// up to a whole number, so that x c - M is rounded once and moving to another M scales exactly;
// -inf where there is no element.
struct Softmax {
  float m, s, w;
  // the same sums relative to another reference
  template <bool kEntropy>
  __device__ __forceinline__ void move(float to) {
    const float d = m - (to == -INFINITY ? 0.f : to), f = ex2_fast(d);
    if (kEntropy) w = f > 0.f ? f * (w + s * d) : 0.f;
    s *= f;
    m = to;
  }
  // of all lanes: the maximum first, then symmetric sums, so that every lane has the same bits
  template <bool kEntropy>
  __device__ __forceinline__ void over_warp() {
    move<kEntropy>(warp_top(m));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      s += __shfl_xor_sync(0xffffffffu, s, o);
      if (kEntropy) w += __shfl_xor_sync(0xffffffffu, w, o);
    }
  }
};

// z in base 2 is x c.  Logits below `floor`, whose x up is about -2^126, count as `floor`: -inf, and the types'
// lowest numbers where they pass that.  Next to any other logit their probability is 0, and 0 times their
// distance is 0, not NaN.  floor is a bf16 number.
//
// M misses x c by 64 at most below 2^31, for which exponents have room.  From there on two different logits'
// x c are more than 128 apart, so that next to the largest all others' probabilities are 0; with `up`, the power
// of two from c on, in the place of c that stays so, x up is exact, and the largest logit's exponent is 0.
constexpr float kFar = 0x1p31f;
struct Temper {
  float c, up, floor;
  __device__ __forceinline__ float factor(float m) const { return fabsf(m) >= kFar ? up : c; }  // of a row with that reference
  __device__ __forceinline__ float lift(float x) const {  // NaN kept
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(x), "f"(floor));
    return d;
  }
  // The same of a vector's words, two elements at a time, where the type reaches that far;
  template <class T>
  __device__ __forceinline__ void lift_words(uint32_t (&w)[4]) const {
    if constexpr (std::is_same<T, __nv_bfloat16>::value) {
      const uint32_t both_floors = __float_as_uint(floor) | __float_as_uint(floor) >> 16;
#pragma unroll
      for (int k = 0; k < 4; ++k) asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(w[k]) : "r"(both_floors));
    }
  }
  // elsewhere in fp32, as pairs are taken.
  template <class T>
  __device__ __forceinline__ float2 lifted(const Vec<T, 16 / sizeof(T)>& u, int p) const {
    const float2 f = u.get(p);
    return std::is_same<T, __nv_bfloat16>::value ? f : make_float2(lift(f.x), lift(f.y));
  }
  __device__ __forceinline__ float reference(float x) const { return ceilf(x * factor(x * c)); }
  // 2^(x f - m) of a pair, f the factor that goes with m, and the exponents
  static __device__ __forceinline__ float2 exp(float2 x, float f, float m, float2& t) {
    t = fma2(x, both(f), both(-m));
    return make_float2(ex2_fast(t.x), ex2_fast(t.y));
  }
};
// The largest of a vector's elements (NaN is passed over) and `top`, in words.
template <class T>
__device__ __forceinline__ uint32_t top_word(uint32_t a, uint32_t b) {
  uint32_t d;
  if constexpr (sizeof(T) == 4)
    d = __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  else if constexpr (std::is_same<T, __half>::value)
    asm("max.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  else
    asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// A thread's maximum and sums over its own elements, so far.
template <class T, bool kEntropy>
struct Running {
  static constexpr int VL = 16 / sizeof(T), kP = VL / 2;
  // an empty place reads as -inf
  static constexpr uint32_t kNone = sizeof(T) == 4 ? 0xFF800000u : std::is_same<T, __half>::value ? 0xFC00FC00u : 0xFF80FF80u;
  Temper z;
  float m, f;  // reference, and its factor
  float2 s2, w2;
  __device__ __forceinline__ explicit Running(const Temper& z_) : z(z_), m(-INFINITY), f(z_.c), s2(both(0.f)), w2(both(0.f)) {}
  __device__ __forceinline__ Softmax sums() const { return Softmax{m, s2.x + s2.y, w2.x + w2.y}; }
  // sums relative to a reference that `top` does not pass
  __device__ __forceinline__ void shift(float top) {
    const float x = fmaxf(top, z.floor);
    float to = fmaxf(m, ceilf(x * z.c));
    f = z.c;
    if (fabsf(to) >= kFar) {  // rare; what is below a far maximum may take either factor
      to = fmaxf(m, x * z.up);
      f = z.up;
    }
    const float d = m - to, by = ex2_fast(d);
    if (kEntropy) w2 = by > 0.f ? mul2(fma2(s2, both(d), w2), both(by)) : both(0.f);
    s2 = mul2(s2, both(by));
    m = to;
  }
  // up to kGroup vectors, v, v + kTeam, ... of `count`, from a row of the ring
  template <int kTeam, class R>
  __device__ __forceinline__ void add(const R& ring, int stage, int first, int v, int count) {
    Vec<T, VL> u[kGroup];
    uint32_t tw = kNone;
#pragma unroll
    for (int j = 0; j < kGroup; ++j)
      if (v + j * kTeam < count) {
        u[j].from_smem(ring.slot(stage, first + j));
#pragma unroll
        for (int k = 0; k < 4; ++k) tw = top_word<T>(tw, u[j].w[k]);
      }
    if (v >= count) return;
    if constexpr (sizeof(T) == 4) {
      shift(__uint_as_float(tw));
    } else {
      const float2 t2 = Two<T>::get(&tw);
      shift(fmaxf(t2.x, t2.y));
    }
#pragma unroll
    for (int j = 0; j < kGroup; ++j)
      if (v + j * kTeam < count) {
        z.template lift_words<T>(u[j].w);
#pragma unroll
        for (int p = 0; p < kP; ++p) {
          float2 t;
          const float2 e = z.exp(z.template lifted<T>(u[j], p), f, m, t);
          s2 = add2(s2, e);
          if (kEntropy) w2 = fma2(e, t, w2);
        }
      }
  }
  __device__ __forceinline__ void add_one(float x) {
    shift(x);
    const float t = fmaf(z.lift(x), f, -m), e = ex2_fast(t);
    s2.x += e;
    if (kEntropy) w2.x += e * t;
  }
};
// What a row's sums say of the element with logit x.
struct Outcome {
  float logp, lse, entropy, inv_s;
  __device__ __forceinline__ Outcome(const Softmax& sm, float x, const Temper& z) {
    constexpr float kLn2 = 0.6931471805599453f;
    const float ls = log2f(sm.s), y = x == -INFINITY ? x : z.lift(x);
    // element minus reference first: their difference is what counts, not their size
    if (fabsf(sm.m) < kFar) {
      logp = kLn2 * (fmaf(y, z.c, -sm.m) - ls);
      lse = kLn2 * (sm.m + ls);
    } else {
      const float top = sm.m / z.up;  // the largest logit
      logp = kLn2 * ((y - top) * z.c - ls);
      lse = kLn2 * (top * z.c + ls);
    }
    inv_s = 1.0f / sm.s;
    entropy = kLn2 * (ls - sm.w * inv_s);
    // Both numbers of a difference are up to 1 where the result is near 0: rounding may carry it past that.
    asm("min.NaN.f32 %0, %0, 0f00000000;" : "+f"(logp));
    asm("max.NaN.f32 %0, %0, 0f00000000;" : "+f"(entropy));
  }
};
// The gradient of a vector whose first element is column `col`: q 2^(x f - m), and coef more at the target.
template <class T>
__device__ __forceinline__ Vec<T, 16 / sizeof(T)> grad_of(Vec<T, 16 / sizeof(T)> u, const Temper& z, float f, float m, float q, float coef, int col, int y) {
  constexpr int kP = 8 / sizeof(T);
  float2 e[kP], t;
  z.template lift_words<T>(u.w);
#pragma unroll
  for (int p = 0; p < kP; ++p) e[p] = z.exp(z.template lifted<T>(u, p), f, m, t);
  return grad_vec<T>(e, q, coef, col, y);
}

// A sum as an fp32 number and what its rounding left: a preference loss lives on the difference of two
// large sums, a policy loss on terms of either sign, and fp64 additions are slow here.  Once a sum is infinite what is left is NaN and does not count.
struct Long {
  float hi, lo;
  __device__ __forceinline__ void add(float v) {  // exactly
    const float t = hi + v, b = t - hi;
    lo += (hi - (t - b)) + (v - b);
    hi = t;
  }
  __device__ __forceinline__ void add(const Long& v) {
    add(v.hi);
    lo += v.lo;
  }
  __device__ __forceinline__ float value() const { return isinf(hi) ? hi : hi + lo; }
  __device__ __forceinline__ Long over(float n) const {
    const float q = hi / n;
    return Long{q, (fmaf(-q, n, hi) + lo) / n};
  }
};
__device__ __forceinline__ Long long_over_warp(Long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v.add(Long{__shfl_xor_sync(0xffffffffu, v.hi, o), __shfl_xor_sync(0xffffffffu, v.lo, o)});
  return v;
}

// A warp's sums of kTerms numbers: lanes halve what they hold of eight (five of them anything) while they halve
// themselves, nine additions instead of twenty-five.  Lane 4 j ends with the sum of term j (lane 16 of term 4).
__device__ __forceinline__ Long terms_over_warp(const Long (&v)[kTerms]) {
  static_assert(kTerms <= 8, "three halvings");
  const int lane = threadIdx.x & 31;
  Long h[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) h[k] = k < kTerms ? v[k < kTerms ? k : 0] : Long{0.f, 0.f};
#pragma unroll
  for (int n = 4, o = 16; n > 0; n /= 2, o /= 2)
#pragma unroll
    for (int k = 0; k < n; ++k) {
      const bool up = lane & o;
      const Long keep = up ? h[k + n] : h[k], give = up ? h[k] : h[k + n];
      h[k] = keep;
      h[k].add(Long{__shfl_xor_sync(0xffffffffu, give.hi, o), __shfl_xor_sync(0xffffffffu, give.lo, o)});
    }
#pragma unroll
  for (int o = 2; o > 0; o >>= 1) h[0].add(Long{__shfl_xor_sync(0xffffffffu, h[0].hi, o), __shfl_xor_sync(0xffffffffu, h[0].lo, o)});
  return h[0];
}
// The sums of few rows (pairs) by the warp that came last, an adapter after the other: lanes add
// their elements in order, then a butterfly.
template <class F>
__device__ __forceinline__ void sum_terms_here(const float* terms, int64_t stride, const Ranges& ad, F by, float* loss, float* stats) {
  const int lane = threadIdx.x & 31;
  for (int a = 0; a < ad.n; ++a) {
    Long v[kTerms] = {};
#pragma unroll 4
    for (int64_t i = ad.off[a] + lane; i < ad.off[a + 1]; i += 32)
#pragma unroll
      for (int k = 0; k < kTerms; ++k) v[k].add(__ldcg(terms + k * stride + i));
    const float f = by(a);
    const float t = terms_over_warp(v).value() * f;
    const int k = lane / 4;
    if (lane % 4 == 0 && k < kTerms) (k ? stats[a * (kTerms - 1) + k - 1] : loss[a]) = t;
  }
}
// Notes that this warp's terms are written (by its first lane); true for all lanes of the warp that
// came last of `all`.
__device__ __forceinline__ bool came_last(unsigned* ticket, unsigned all) {
  unsigned at = 0;
  if ((threadIdx.x & 31) == 0)  // back to 0 after the last
    asm volatile("atom.acq_rel.gpu.global.inc.u32 %0, [%1], %2;" : "=r"(at) : "l"(ticket), "r"(all - 1) : "memory");
  const bool last = __shfl_sync(0xffffffffu, at, 0) == all - 1;
  __syncwarp();  // what the first lane has seen, all have
  return last;
}
__device__ __forceinline__ int live_in(const int32_t* targets, int n, int64_t lo, int64_t hi) {
  int c = 0;
#pragma unroll 4
  for (int64_t t = lo + (threadIdx.x & 31); t < hi; t += 32) c += (unsigned)targets[t] < (unsigned)n;
  return __reduce_add_sync(0xffffffffu, c);
}

// 1 / (live tokens of adapter a), from the counts of a launch before.
__device__ __forceinline__ float count_factor(const PolicyArgs& pg, int a) {
  const int lane = threadIdx.x & 31;
  const int k = __reduce_add_sync(0xffffffffu, lane < kCountParts ? pg.count[a * kCountParts + lane] : 0);
  return 1.0f / (float)max(k, 1);
}
// What a token's own values make of the softmax of its row.
struct Token {
  float adv, old, ref, wt, up;
  int a;  // adapter
  __device__ __forceinline__ Token() {}
  __device__ __forceinline__ Token(const PolicyArgs& pg, const Ranges& ad, int64_t t) : ref(0.f), wt(1.f), up(1.f) {
    a = range_of(ad, t);
    adv = pg.adv[t];
    old = pg.old[t];
    if (pg.ref) ref = pg.ref[t];
    if (pg.weight) wt = pg.weight[t];
    if (pg.dloss) up = pg.dloss[a];
  }
  // The loss's terms (stored where `writes`), and the factor of the gradient to the log probability.
  __device__ __forceinline__ float terms(const PolicyArgs& pg, int64_t rows, int64_t t, float logp, float entropy, bool writes) const {
    const float rho = expf(logp - old), clip = fminf(fmaxf(rho, pg.low), pg.high);
    const bool cut = (adv > 0.f && rho > pg.high) || (adv < 0.f && rho < pg.low);
    // a ratio past fp32's range is a number all the same: none of it is left times an advantage of 0
    const float gain = adv == 0.f && rho == INFINITY ? 0.f : rho * adv;
    float loss = cut ? -clip * adv : -gain, kl = 0.f, dl = cut ? 0.f : -gain;
    if (pg.ref) {
      const float d = ref - logp, em = expm1f(d);
      kl = d == INFINITY ? d : em - d;
      if (pg.kl != 0.f) {  // else it is reported alone, and may be infinite
        loss += pg.kl * kl;
        dl -= pg.kl * em;
      }
    }
    if (writes) {  // a token of weight 0 has no part in the loss, whatever its values
      float* to = pg.terms + t;
      to[0] = wt == 0.f ? 0.f : wt * loss;
      to[rows] = wt == 0.f ? 0.f : wt * kl;
      to[2 * rows] = cut ? wt : 0.f;
      to[3 * rows] = wt == 0.f ? 0.f : wt * rho;
      to[4 * rows] = wt == 0.f ? 0.f : wt * entropy;
    }
    return wt == 0.f ? 0.f : up * wt * dl;
  }
};

// Log probabilities (kPolicy false), or the policy loss's terms and, with kGrad, its
// gradient.  kTeam threads work on a slice: a block's, or a warp whose slice is the row.
// What happens once per row is left to one warp: a lane has 16 vectors of a slice of 32 KB, and a
// few hundred instructions around them cost as much as the vectors.
template <class T, int kTeam, int kGroups, bool kEntropy, bool kPolicy, bool kGrad>
__global__ void __launch_bounds__(kTeam == 32 ? kShortThreads : kTeam, 1)
    token_row_kernel(const __grid_constant__ RowArgs g, const __grid_constant__ PolicyArgs pg,
                     const __grid_constant__ GradArgs dg, const __grid_constant__ Ranges ad, int slices, int per) {
  constexpr int VL = 16 / sizeof(T), kWarps = kTeam / 32;
  extern __shared__ __align__(16) uint8_t row_smem[];
  __shared__ Softmax part[kMaxCluster + kWarps];
  __shared__ float3 result;  // the reference, the factor of all exponentials and of the target's one
  __shared__ float at_target;
  const Ring<1, kGroups * kGroup> ring(row_smem);
  const int tid = threadIdx.x % kTeam, lane = threadIdx.x & 31, warp = tid >> 5;
  const int rank = kTeam > 32 && slices > 1 ? (int)cluster_rank() : 0;
  int64_t t = blockIdx.x;
  if (kTeam == 32)
    t = t * (kShortThreads / 32) + (threadIdx.x >> 5);
  else if (slices > 1)
    asm("{ .reg .u32 c; mov.u32 c, %%clusterid.x; cvt.u64.u32 %0, c; }" : "=l"(t));
  if (kPolicy) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (t >= g.rows) return;  // (a warp's own row)
  const T* row = static_cast<const T*>(g.x) + t * g.ld;
  const int y = checked_target(g.targets[t], g.n, g.err, rank == 0 && tid == 0);
  const Slice<T> sl(row, g.n, rank, slices, per, tid);
  T* out = kGrad ? static_cast<T*>(dg.dx) + t * dg.ldd : nullptr;
  const bool aligned = kGrad && same_phase(row, out);
  const bool clerk = rank == 0 && warp == 0;  // the warp that works for the row
  const auto finish = [&] {  // few rows: the last one adds them all
    if (kPolicy && pg.few && clerk && came_last(pg.ticket, (unsigned)g.rows))
      sum_terms_here(pg.terms, g.rows, ad, [&](int a) {
        return pg.weight ? 1.f : 1.f / (float)max(live_in(g.targets, g.n, ad.off[a], ad.off[a + 1]), 1);
      }, pg.loss, pg.stats);
  };
  if (y < 0) {  // the same for the whole cluster, which has not met yet
    if (clerk && lane == 0) {
      if (g.logp) g.logp[t] = 0.f;
      if (g.lse) g.lse[t] = 0.f;
      if (g.entropy) g.entropy[t] = 0.f;
      if (kPolicy)
#pragma unroll
        for (int i = 0; i < kTerms; ++i) pg.terms[i * g.rows + t] = 0.f;
    }
    if (kGrad) zero_slice<T, kTeam>(sl, out, aligned, tid);
    if (kPolicy) asm volatile("griddepcontrol.wait;" ::: "memory");
    finish();
    return;
  }
  // a thread's vectors: tid, tid + kTeam, ... of the slice
  {
    const T* src = row + sl.first + tid * VL;
#pragma unroll
    for (int i = 0; i < kGroups * kGroup; ++i) {
      if (tid + i * kTeam < sl.count) async_copy16(ring.slot(0, i), src + i * kTeam * VL);
      if (i % kGroup == kGroup - 1) async_commit();
    }
  }
  if (kTeam > 32 && slices > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  const float xe = sl.edge >= 0 ? to_f32(row[sl.edge]) : -INFINITY;
  // The target's logit is read before the block meets: a gradient may take its place afterwards.
  float xy = 0.f;
  if (kTeam == 32 || tid == 0) xy = to_f32(row[y]);
  if (kTeam > 32 && tid == 0) at_target = xy;
  Token tok = kPolicy && warp == 0 ? Token(pg, ad, t) : Token();
  if (kPolicy && kGrad && warp == 0 && pg.few && !pg.weight)
    tok.up /= (float)max(live_in(g.targets, g.n, ad.off[tok.a], ad.off[tok.a + 1]), 1);

  const Temper z{g.c, g.up, g.floor};
  Running<T, kEntropy> run(z);
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
    run.template add<kTeam>(ring, 0, gr * kGroup, tid + gr * kGroup * kTeam, sl.count);
  }
  async_wait<0>();
  if (sl.edge >= 0) run.add_one(xe);
  Softmax sm = run.sums();
  sm.over_warp<kEntropy>();
  float q = 0.f, coef = 0.f;
  if (kTeam > 32) {
    if (lane == 0) part[kMaxCluster + warp] = sm;
    __syncthreads();
    if (warp == 0) {  // the block's sums
      sm = lane < kWarps ? part[kMaxCluster + lane] : Softmax{-INFINITY, 0.f, 0.f};
      sm.over_warp<kEntropy>();
    }
    if (slices > 1) {  // and the cluster's
      asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // all blocks have started
      if (warp == 0 && lane < slices) {
        const uint32_t at = mapa_shared(smem_u32(&part[rank]), lane);
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(sm.m) : "memory");
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at + 4), "f"(sm.s) : "memory");
        if (kEntropy) asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at + 8), "f"(sm.w) : "memory");
      }
      cluster_sync_all();
      if (warp == 0) {
        sm = lane < slices ? part[lane] : Softmax{-INFINITY, 0.f, 0.f};
        sm.over_warp<kEntropy>();
      }
    }
    xy = at_target;
  }
  if (warp == 0 && (kPolicy || rank == 0)) {
    const Outcome o(sm, xy, z);
    if (clerk && lane == 0) {
      if (g.logp) g.logp[t] = o.logp;
      if (g.lse) g.lse[t] = o.lse;
      if (g.entropy) g.entropy[t] = o.entropy;
    }
    if (kPolicy) {
      if (!pg.weight && !pg.few) {
        // the counts, and with them every launch that the sums behind this one rely on
        asm volatile("griddepcontrol.wait;" ::: "memory");
        tok.up *= count_factor(pg, tok.a);
      }
      coef = tok.terms(pg, g.rows, t, o.logp, o.entropy, clerk && lane == 0) * g.inv_temp;
      q = -coef * o.inv_s;
      if (kTeam > 32 && kGrad && lane == 0) result = make_float3(sm.m, q, coef);
    }
  }
  if (!kGrad) {
    finish();
    return;
  }
  if (kTeam > 32) {
    __syncthreads();
    sm.m = result.x;
    q = result.y;
    coef = result.z;
  }
  if (coef == 0.f) {  // clipped, without a KL term
    zero_slice<T, kTeam>(sl, out, aligned, tid);
    finish();
    return;
  }
  const float f = z.factor(sm.m);
  // all sixteen at once fill the instruction cache: 700 us instead of 679 for 8,192 x 151,936
#pragma unroll 4
  for (int i = 0; i < kGroups * kGroup; ++i) {
    const int v = tid + i * kTeam;
    if (v >= sl.count) break;
    Vec<T, VL> u;
    u.from_smem(ring.slot(0, i));
    store_vec<T>(out, sl.first + v * VL, aligned, grad_of<T>(u, z, f, sm.m, q, coef, sl.first + v * VL, y));
  }
  if (sl.edge >= 0) out[sl.edge] = from_f32<T>(q * ex2_fast(fmaf(z.lift(xe), f, -sm.m)) + (sl.edge == y ? coef : 0.f));
  finish();
}

// dlogits where fp32 holds a row's lse coarsely, to 2^-14 and more, which is then a probability's relative
// error.  The row's sum is formed anew from its logits, by a warp or a block, in three sweeps: 2.5 ms for
// 16,384 x 65,536 bf16, 0.64 with logits near 0.
constexpr float kCoarse = 1024.f;
template <class T, int kTeam>
__device__ __noinline__ void row_anew(const RowArgs& g, const GradArgs& dg, int64_t t, float coef, int y) {
  constexpr int kWarps = kTeam / 32;
  const T* row = static_cast<const T*>(g.x) + t * g.ld;
  T* out = static_cast<T*>(dg.dx) + t * dg.ldd;
  const int n = g.n;
  const Temper z{g.c, g.up, g.floor};
  __shared__ float tops[kWarps];
  __shared__ Long sums[kWarps];
  const int tid = threadIdx.x % kTeam, lane = tid & 31, warp = tid >> 5;
  float x = z.floor;
#pragma unroll 8
  for (int i = tid; i < n; i += kTeam) x = fmaxf(x, to_f32(row[i]));
  x = warp_top(x);
  if (kTeam > 32) {
    if (lane == 0) tops[warp] = x;
    __syncthreads();
    x = warp_top(lane < kWarps ? tops[lane] : z.floor);
  }
  const float m = z.reference(x), f = z.factor(m);
  Long s{0.f, 0.f};
#pragma unroll 8
  for (int i = tid; i < n; i += kTeam) s.add(ex2_fast(fmaf(z.lift(to_f32(row[i])), f, -m)));
  s = long_over_warp(s);
  if (kTeam > 32) {
    if (lane == 0) sums[warp] = s;
    __syncthreads();  // and all have read the row, whose place the gradient may take
    s = long_over_warp(lane < kWarps ? sums[lane] : Long{0.f, 0.f});
  }
  const float q = -coef / s.value();
#pragma unroll 8
  for (int i = tid; i < n; i += kTeam)
    out[i] = from_f32<T>(q * ex2_fast(fmaf(z.lift(to_f32(row[i])), f, -m)) + (i == y ? coef : 0.f));
}

// dlogits from a saved lse: no reduction, every element on its own.  A block takes up to
// kBwdVecs vectors a thread of one row, all their loads under way together.
constexpr int kBwdThreads = 256, kBwdVecs = 4, kBwdWarpVecs = 1024;
template <class T, int kTeam>
__global__ void __launch_bounds__(kBwdThreads)
    token_bwd_kernel(const __grid_constant__ RowArgs g, const __grid_constant__ GradArgs dg, const float* dlogp, int slices, int per) {
  constexpr int VL = 16 / sizeof(T), kP = VL / 2;
  const int tid = threadIdx.x % kTeam;
  const int rank = kTeam == 32 ? 0 : blockIdx.x % slices;
  const int64_t t = kTeam == 32 ? (int64_t)blockIdx.x * (kBwdThreads / 32) + threadIdx.x / 32 : blockIdx.x / slices;
  if (t >= g.rows) return;
  const T* row = static_cast<const T*>(g.x) + t * g.ld;
  T* out = static_cast<T*>(dg.dx) + t * dg.ldd;
  const int y = checked_target(g.targets[t], g.n, g.err, rank == 0 && tid == 0);
  const Slice<T> sl(row, g.n, rank, slices, per, tid);
  const bool aligned = same_phase(row, out);
  const float up = y < 0 ? 0.f : dlogp[t];
  if (up == 0.f) {
    zero_slice<T, kTeam>(sl, out, aligned, tid);
    return;
  }
  const float coef = up * g.inv_temp, lse = g.lse[t];
  if (!(fabsf(lse) < kCoarse)) {
    if (rank == 0) row_anew<T, kTeam>(g, dg, t, coef, y);
    return;
  }
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
  Long target;   // squared: 1 / (2 beta)
  bool few;      // so few pairs that the last one done adds the terms
  unsigned* ticket;
  unsigned* again;  // set where the offsets go back: see pairs_again
  float *loss, *stats;
};
// What a warp makes of a pair's sums and counts: its terms, and the gradient of each sequence's tokens.
__device__ __forceinline__ float2 pair_terms(const PrefArgs& g, const Ranges& ad, int64_t i, int a, Long (&r)[2], const int (&count)[2],
                                             const float (&ref)[2], float up) {
  const bool writes = (threadIdx.x & 31) == 0;
  float cnt[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    cnt[q] = g.average ? (float)max(count[q], 1) : 1.f;
    if (g.average) r[q] = r[q].over(cnt[q]);
    if (g.seq_logp && writes) g.seq_logp[2 * i + q] = r[q].value();
    if (g.ref) r[q].add(-ref[q]);
  }
  Long d = r[0];
  d.add(Long{-r[1].hi, -r[1].lo});
  const float h = d.value(), x = g.beta * h - g.margin;
  float loss, dh;
  if (g.kind == MOE_LORA_PREF_SIGMOID) {
    const float e = expf(-fabsf(x)), soft = log1pf(e), near = e / (1.f + e);  // 1 - sigmoid(|x|)
    loss = (1.f - g.smooth) * (soft + fmaxf(-x, 0.f));
    if (g.smooth > 0.f) loss += g.smooth * (soft + fmaxf(x, 0.f));  // (x may be infinite)
    // sigmoid(x) - (1 - smooth) without the difference of two numbers near 1
    dh = g.beta * (x >= 0.f ? g.smooth - near : near - (1.f - g.smooth));
  } else if (g.kind == MOE_LORA_PREF_SQUARED) {
    d.add(-g.target.hi);
    d.lo -= g.target.lo;
    const float o = d.value();
    loss = o * o;
    dh = 2.f * o;
  } else {
    loss = fmaxf(1.f - x, 0.f);
    dh = x < 1.f ? -g.beta : 0.f;
  }
  if (isnan(x)) loss = dh = x;
  if (writes) {
    float* to = g.terms + i;
    to[0] = loss;
    to[g.pairs] = x > 0.f ? 1.f : 0.f;
    to[2 * g.pairs] = g.beta * r[0].value();
    to[3 * g.pairs] = g.beta * r[1].value();
    to[4 * g.pairs] = h;
  }
  const float each = up / (float)(ad.off[a + 1] - ad.off[a]);
  return make_float2(each * dh / cnt[0], -each * dh / cnt[1]);
}
// Pairs [lo, hi) once more, by a warp, where the list of offsets goes back or past the tokens.  Each
// offset counts as the largest so far, which depends on the whole list, and a pair's block sees its own
// three: every fault of a list is one of some pair's own three, which share one with the next pair's; its
// block sets *again, and what adds the terms, which runs after all blocks, comes here first.  Blocks write
// nothing ahead of the first offset, so all that they have written lies in sequences as they count, and is
// written anew.  (Looking through the offsets ahead in every block: 1,000 pairs of 100 tokens 9.9 us
// instead of 8.6.)
__device__ __noinline__ void pairs_again(const PrefArgs& g, const Ranges& ad, int64_t lo, int64_t hi) {
  if (lo >= hi) return;
  const int lane = threadIdx.x & 31;
  int64_t top = 0;
  for (int64_t j = lane; j < 2 * lo; j += 32) top = max(top, g.seq[j]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = max(top, (int64_t)__shfl_xor_sync(0xffffffffu, (long long)top, o));
  for (int64_t i = lo; i < hi; ++i) {
    int64_t off[3];
    for (int j = 0; j < 3; ++j) off[j] = min(top = max(top, g.seq[2 * i + j]), g.T);
    Long r[2] = {};
    int n[2] = {0, 0};
    for (int q = 0; q < 2; ++q) {
#pragma unroll 8
      for (int64_t t = off[q] + lane; t < off[q + 1]; t += 32) {  // both loaded, so that many are on their way
        const bool live = g.targets[t] >= 0;
        const float f = g.logp[t];
        r[q].add(live ? f : 0.f);
        n[q] += live;
      }
      r[q] = long_over_warp(r[q]);
      n[q] = __reduce_add_sync(0xffffffffu, n[q]);
    }
    const int a = range_of(ad, i);
    const float ref[2] = {g.ref ? g.ref[2 * i] : 0.f, g.ref ? g.ref[2 * i + 1] : 0.f};
    const float2 each = pair_terms(g, ad, i, a, r, n, ref, g.dloss ? g.dloss[a] : 1.f);
    if (g.dlogp)
#pragma unroll 8
      for (int64_t t = off[0] + lane; t < off[2]; t += 32) g.dlogp[t] = g.targets[t] < 0 ? 0.f : t < off[1] ? each.x : each.y;
  }
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
template <int kC, bool kPairs>
__global__ void __launch_bounds__(kSumThreads)
    term_sum_kernel(const __grid_constant__ SumArgs g, const __grid_constant__ Ranges ad, const __grid_constant__ PrefArgs pref) {
  __shared__ Long warp_sum[kSumThreads / 32][kTerms], block_sum[kTerms];
  const int a = blockIdx.x / kC, rank = kC > 1 ? (int)cluster_rank() : 0;
  const int64_t lo = ad.off[a], hi = ad.off[a + 1];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (kPairs && __ldcg(pref.again)) {  // the same for all blocks, the last of which clears it
    const int64_t warps = kC * (kSumThreads / 32), each = (hi - lo + warps - 1) / warps;
    const int64_t first = min(hi, lo + (rank * (kSumThreads / 32) + (threadIdx.x >> 5)) * each);
    pairs_again(pref, ad, first, min(hi, first + each));
    __syncthreads();
    if (threadIdx.x < 32 && came_last(pref.ticket, gridDim.x) && threadIdx.x == 0) *pref.again = 0;
    if (kC > 1) cluster_sync_all();
  }
  Long s[kTerms] = {};
#pragma unroll 2
  for (int64_t i = lo + rank * kSumThreads + threadIdx.x; i < hi; i += kSumCluster * kSumThreads)
#pragma unroll
    for (int k = 0; k < kTerms; ++k) s[k].add(__ldcg(g.terms + k * g.stride + i));
  const int k = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Long mine = terms_over_warp(s);
  if (lane % 4 == 0 && lane / 4 < kTerms) warp_sum[k][lane / 4] = mine;
  __syncthreads();  // a warp per term from here on
  if (k < kTerms) {
    const Long v = long_over_warp(warp_sum[lane][k]);
    if (lane == 0) block_sum[k] = v;
  }
  if (kC > 1)
    cluster_sync_all();
  else
    __syncthreads();
  if (rank == 0 && k < kTerms) {
    Long sum{0.f, 0.f};
    if (lane < kC) {
      if (kC > 1) {
        const uint32_t at = mapa_shared(smem_u32(&block_sum[k]), lane);
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(sum.hi) : "r"(at) : "memory");
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(sum.lo) : "r"(at + 4) : "memory");
      } else {
        sum = block_sum[k];
      }
    }
#pragma unroll
    for (int o = kSumCluster / 2; o > 0; o >>= 1)
      sum.add(Long{__shfl_xor_sync(0xffffffffu, sum.hi, o), __shfl_xor_sync(0xffffffffu, sum.lo, o)});
    const float v = sum.value();
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

// A block per pair, whose two sequences lie one behind the other: their sums, the pair's
// terms, then the gradient.  Latency bounds it: a thread has four vectors of four tokens
// under way, and what it learnt of the first four (which tokens are live) stays with it.
constexpr int kPrefAhead = 4;
template <int kThreads>
__global__ void __launch_bounds__(kThreads) pref_kernel(const __grid_constant__ PrefArgs g, const __grid_constant__ Ranges ad) {
  __shared__ Long sums[2][kThreads / 32];
  __shared__ int counts[2][kThreads / 32];
  __shared__ float per_token[2];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t i = blockIdx.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t off[3];
  bool bad = false;
#pragma unroll
  for (int j = 0; j < 3; ++j) off[j] = g.seq[2 * i + j];
  const int64_t start = g.seq[0];
#pragma unroll
  for (int j = 0; j < 3; ++j) {  // offsets that go back or past the end are noted; what is left of them is inside
    const int64_t at = min(max(j ? off[j - 1] : max(start, (int64_t)0), off[j]), g.T);
    bad |= at != off[j];
    off[j] = at;
  }
  if (bad && threadIdx.x == 0) {
    *g.again = 1;
    if (g.err) atomicOr(g.err, MOE_LORA_DEV_BAD_ID);
  }
  // asked for early, used late
  const int a = range_of(ad, i);
  const float ref[2] = {g.ref ? g.ref[2 * i] : 0.f, g.ref ? g.ref[2 * i + 1] : 0.f}, up = g.dloss ? g.dloss[a] : 1.f;
  const int64_t base = off[0] & ~(int64_t)3;
  const int64_t vecs = (off[2] - base + 3) / 4;  // of four tokens, on 16 bytes; the first and last may be partly outside
  const auto load_mask = [&](int64_t v, float (&x)[4]) {  // live tokens of a vector that belong to the pair, and their values
    const int64_t t = base + 4 * v;
    int y[4];
    if (t + 4 <= g.T) {
      const int4 u = *reinterpret_cast<const int4*>(g.targets + t);
      const float4 f = *reinterpret_cast<const float4*>(g.logp + t);
      y[0] = u.x, y[1] = u.y, y[2] = u.z, y[3] = u.w;
      x[0] = f.x, x[1] = f.y, x[2] = f.z, x[3] = f.w;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        y[e] = t + e < g.T ? g.targets[t + e] : -1;
        x[e] = t + e < g.T ? g.logp[t + e] : 0.f;
      }
    }
    uint32_t live = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) live |= (y[e] >= 0 && t + e >= off[0] && t + e < off[2]) << e;
    return live;
  };
  Long s[2] = {};
  int n[2] = {0, 0};
  uint32_t known = 0;  // live tokens of this thread's first vectors
  for (int64_t v0 = threadIdx.x; v0 < vecs; v0 += kPrefAhead * kThreads) {
    float x[kPrefAhead][4];
    uint32_t live[kPrefAhead];
#pragma unroll
    for (int j = 0; j < kPrefAhead; ++j) live[j] = v0 + j * kThreads < vecs ? load_mask(v0 + j * kThreads, x[j]) : 0;
#pragma unroll
    for (int j = 0; j < kPrefAhead; ++j) {
      if (v0 < kThreads) known |= live[j] << (4 * j);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (live[j] >> e & 1) {
          const int q = base + 4 * (v0 + j * kThreads) + e >= off[1];
          const float f = x[j][e];
          s[0].add(q ? 0.f : f);
          s[1].add(q ? f : 0.f);
          n[q] += 1;
        }
    }
  }
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    s[q] = long_over_warp(s[q]);
    n[q] = __reduce_add_sync(0xffffffffu, n[q]);
    if (lane == 0) {
      sums[q][warp] = s[q];
      counts[q][warp] = n[q];
    }
  }
  __syncthreads();
  if (warp == 0) {
    Long r[2];
    int count[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      r[q] = long_over_warp(lane < kThreads / 32 ? sums[q][lane] : Long{0.f, 0.f});
      count[q] = __reduce_add_sync(0xffffffffu, lane < kThreads / 32 ? counts[q][lane] : 0);
    }
    const float2 each = pair_terms(g, ad, i, a, r, count, ref, up);
    if (lane == 0) {
      per_token[0] = each.x;
      per_token[1] = each.y;
    }
  }
  if (g.dlogp) {
    __syncthreads();
    const float p0 = per_token[0], p1 = per_token[1];
    for (int64_t v = threadIdx.x, j = 0; v < vecs; v += kThreads, ++j) {
      const int64_t t = base + 4 * v;
      uint32_t live;
      if (j < kPrefAhead) {
        live = known >> (4 * (int)j) & 15;
      } else {
        float unused[4];
        live = load_mask(v, unused);
      }
      float o[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = live >> e & 1 ? (t + e < off[1] ? p0 : p1) : 0.f;
      if (t >= off[0] && t + 4 <= off[2]) {
        *reinterpret_cast<float4*>(g.dlogp + t) = make_float4(o[0], o[1], o[2], o[3]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (t + e >= off[0] && t + e < off[2]) g.dlogp[t + e] = o[e];
      }
    }
  }
  if (!g.few) return;
  if (g.dlogp) __syncthreads();  // the block's gradients are written before it counts as done
  if (warp == 0 && came_last(g.ticket, (unsigned)g.pairs)) {
    const bool again = __ldcg(g.again);  // on its way while the terms are
    const auto sum = [&] {
      sum_terms_here(g.terms, g.pairs, ad, [&](int a) { return 1.f / (float)max(ad.off[a + 1] - ad.off[a], (int64_t)1); }, g.loss, g.stats);
    };
    sum();
    if (again) {
      pairs_again(g, ad, 0, g.pairs);
      __syncwarp();
      sum();
      if (lane == 0) *g.again = 0;
    }
  }
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
  if (!(r->inv_temp >= 1e-6f) || !(r->inv_temp <= 1e6f)) return MOE_LORA_ERR_DIMS;
  return MOE_LORA_OK;
}
RowArgs row_args(const moe_lora_rows* r, const void* x, const int32_t* targets, float* logp, float* lse, float* entropy, int32_t* err) {
  const float c = r->inv_temp * kLog2e;
  int e;
  const float up = frexpf(c, &e) == 0.5f ? c : ldexpf(1.f, e);
  constexpr float kLowest = -0x1.FEp127f;  // of bf16
  const float floor = up <= 0.25f ? kLowest : -0x1p126f / up;
  return RowArgs{x, r->ld ? r->ld : r->n, r->rows, r->n, r->inv_temp, c, up, floor, targets, logp, lse, entropy, err};
}

template <class T, int kTeam, int kGroups, bool kEntropy, bool kPolicy, bool kGrad>
int launch_rows(const RowArgs& g, const PolicyArgs& pg, const GradArgs& dg, const Ranges& ad, int slices, bool overlap, cudaStream_t s) {
  const int vecs = g.n / (int)(16 / sizeof(T)), per = (vecs + slices - 1) / slices;
  const int64_t grid = kTeam == 32 ? (g.rows + kShortThreads / 32 - 1) / (kShortThreads / 32) : g.rows * slices;
  const int threads = kTeam == 32 ? kShortThreads : kTeam;
  const RowLaunch l(grid, threads, ring_bytes<1, kGroups * kGroup>(threads), slices, overlap, s);
  const int slot = kPolicy ? K_POLICY : K_TOKEN_FWD;
  prof_begin(slot, s);
  const cudaError_t e = launch_allowed(l.cfg, slices > 8, token_row_kernel<T, kTeam, kGroups, kEntropy, kPolicy, kGrad>, g, pg, dg, ad, slices, per);
  prof_end(slot, s);
  return e == cudaSuccess ? MOE_LORA_OK : MOE_LORA_ERR_CUDA;
}

// Slices of a row and what a block holds of it.  Up to 128 vectors (1,024 elements of 16 bits) belong to
// a warp (20,000 x 1,000 log probabilities 8.2 us, as blocks 11.8; 200 x 1,000 2.1 and 2.3), up to 512
// where there are enough rows for every SM's warps (20,000 x 4,000 27.8 and 33.1 us, the policy's gradient 64
// and 117; 2,000 x 4,096 11.7 and 15.4, but 600 x 4,000 8.8 and 6.8).  Longer rows belong to the fewest
// blocks of 128 threads that hold 32 KB each, up to sixteen, which then hold up to 128 KB.  Log
// probabilities of 16,384 x 65,536 took 348 us so, with 16 KB 418, with 64 KB 393, with 256 threads
// and 64 KB 417, with 64 threads 414; of 8,192 x 151,936 467 us in clusters of ten, 589 in five of
// 64 KB.  The policy loss over 8,192 x 151,936 707 us, with 256 threads and 64 KB 757, 32 KB 812;
// 2,048 x 50,257 73 and 72 (each with the gradient's loop unrolled by sixteen).  Where there are too few rows to give every SM a block, a row is shared by
// more, up to eight (one row of 32,000: 2.9 us instead of 4.4).
template <class T, bool kEntropy, bool kPolicy, bool kGrad>
int pick_rows(const RowArgs& g, const PolicyArgs& pg, const GradArgs& dg, const Ranges& ad, int sms, bool overlap, cudaStream_t s) {
  constexpr int VL = 16 / sizeof(T);
  const int vecs = g.n / VL;
  if (vecs <= 32 * kGroup) return launch_rows<T, 32, 1, kEntropy, kPolicy, kGrad>(g, pg, dg, ad, 1, overlap, s);
  if (vecs <= 32 * 4 * kGroup && g.rows >= 8 * sms) return launch_rows<T, 32, 4, kEntropy, kPolicy, kGrad>(g, pg, dg, ad, 1, overlap, s);
  constexpr int one = kRowThreads * kGroup;  // vectors of a group of a block
  int slices = std::min((vecs + 4 * one - 1) / (4 * one), kMaxCluster);
  while (slices < 8 && g.rows * (slices + 1) <= sms && vecs / (slices + 1) >= 2 * kRowThreads) ++slices;
  const int per = (vecs + slices - 1) / slices;
  const auto run = [&](auto groups) {
    return launch_rows<T, kRowThreads, decltype(groups)::value, kEntropy, kPolicy, kGrad>(g, pg, dg, ad, slices, overlap, s);
  };
  return per <= one       ? run(std::integral_constant<int, 1>{})
         : per <= 2 * one ? run(std::integral_constant<int, 2>{})
         : per <= 4 * one ? run(std::integral_constant<int, 4>{})
         : per <= 8 * one ? run(std::integral_constant<int, 8>{})
                          : run(std::integral_constant<int, 16>{});
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
int run_bwd(const RowArgs& g, const GradArgs& dg, const float* dlogp, int sms, cudaStream_t s) {
  constexpr int VL = 16 / sizeof(T);
  const int vecs = g.n / VL, slices = std::max(1, (vecs + kBwdThreads * kBwdVecs - 1) / (kBwdThreads * kBwdVecs));
  prof_begin(K_TOKEN_BWD, s);
  // a warp per row: 20,000 x 1,000 9.9 us, as blocks 32; 20,000 x 4,000 53 and 74; 20,000 x 8,000 102 and
  // 106; but 1,300 x 8,000 9.3 and 6.2
  if (vecs <= 32 * kBwdVecs || (vecs <= kBwdWarpVecs && g.rows >= 16 * sms))
    token_bwd_kernel<T, 32><<<(unsigned)((g.rows + kBwdThreads / 32 - 1) / (kBwdThreads / 32)), kBwdThreads, 0, s>>>(g, dg, dlogp, 1, vecs);
  else
    token_bwd_kernel<T, kBwdThreads><<<(unsigned)(g.rows * slices), kBwdThreads, 0, s>>>(g, dg, dlogp, slices, (vecs + slices - 1) / slices);
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

template <bool kPairs>
int launch_sums(const SumArgs& g, const Ranges& ad, const PrefArgs& pref, cudaStream_t s) {
  int64_t most = 0;
  for (int a = 0; a < ad.n; ++a) most = std::max(most, ad.off[a + 1] - ad.off[a]);
  const bool one = most <= kSumThreads;
  const RowLaunch l((int64_t)ad.n * (one ? 1 : kSumCluster), kSumThreads, 0, one ? 1 : kSumCluster, true, s);
  prof_begin(K_TERM_SUM, s);
  const cudaError_t e = one ? cudaLaunchKernelEx(&l.cfg, term_sum_kernel<1, kPairs>, g, ad, pref)
                            : cudaLaunchKernelEx(&l.cfg, term_sum_kernel<kSumCluster, kPairs>, g, ad, pref);
  prof_end(K_TERM_SUM, s);
  return e == cudaSuccess ? MOE_LORA_OK : MOE_LORA_ERR_CUDA;
}

// Scratch of the losses: a ticket, the items' terms, then the adapters' partial counts.
constexpr size_t kTicketBytes = 256;
size_t terms_bytes(int64_t items) { return align_up(sizeof(float) * kTerms * (size_t)std::max<int64_t>(items, 1), 256); }
// Few items: counted, and their terms added, where the items are worked on, in one launch.  64 rows of
// 4,096: 8.5 us in one launch or three on the GPU, 12 and 16 us of the host's time; 128 rows 6.4 and
// 5.8 us, 200 rows 7.8 and 5.4.  64 pairs 6.0 us either way, 256 pairs 8.2 and 8.6, 1,024 pairs 22 and 12.
constexpr int kFewRows = 64, kFewPairs = 256;

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
  return r->dtype == MOE_LORA_F32    ? run_bwd<float>(g, dg, dlogp, sms, s)
         : r->dtype == MOE_LORA_BF16 ? run_bwd<__nv_bfloat16>(g, dg, dlogp, sms, s)
                                     : run_bwd<__half>(g, dg, dlogp, sms, s);
}

extern "C" size_t moe_lora_policy_scratch_bytes(int64_t rows, int32_t adapters) {
  if (rows < 0 || rows > (int64_t)1 << 26 || adapters < 1 || adapters > kMaxAdapters) return 0;
  return kTicketBytes + terms_bytes(rows) + align_up(sizeof(int) * kCountParts * adapters, 256);
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
  char* at = static_cast<char*>(scratch);
  float* terms = reinterpret_cast<float*>(at + kTicketBytes);
  int* count = reinterpret_cast<int*>(at + kTicketBytes + terms_bytes(r->rows));
  const bool few = r->rows > 0 && r->rows <= kFewRows;
  const PolicyArgs pg{advantages, old_logp, ref_logp, weight, dloss, 1.f - o->clip_low, 1.f + o->clip_high, o->kl_coef, count, terms,
                      few, reinterpret_cast<unsigned*>(at), loss, stats};
  if (!weight && !few) {
    prof_begin(K_TOKEN_COUNT, s);
    token_count_kernel<<<ad.n * kCountParts, 256, 0, s>>>(targets, r->n, ad, count);
    prof_end(K_TOKEN_COUNT, s);
    if (cudaGetLastError() != cudaSuccess) return MOE_LORA_ERR_CUDA;
  }
  if (r->rows > 0) {
    rc = r->dtype == MOE_LORA_F32    ? run_policy<float>(g, pg, dg, ad, sms, !weight && !few, s)
         : r->dtype == MOE_LORA_BF16 ? run_policy<__nv_bfloat16>(g, pg, dg, ad, sms, !weight && !few, s)
                                     : run_policy<__half>(g, pg, dg, ad, sms, !weight && !few, s);
    if (rc || few) return rc;
  }
  return launch_sums<false>(SumArgs{terms, r->rows, weight ? nullptr : count, false, loss, stats}, ad, {}, s);
}

extern "C" size_t moe_lora_preference_scratch_bytes(int64_t pairs) {
  return pairs < 0 || pairs > (int64_t)1 << 26 ? 0 : kTicketBytes + terms_bytes(pairs);
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
  float* terms = reinterpret_cast<float*>(static_cast<char*>(scratch) + kTicketBytes);
  unsigned* ticket = static_cast<unsigned*>(scratch);
  const bool few = o->pairs <= kFewPairs;
  const double target = 0.5 / (double)o->beta;
  const PrefArgs g{logp, targets, o->tokens, seq_offsets, ref, o->beta, o->margin, o->label_smoothing, o->kind, o->average,
                   dloss, seq_logp, dlogp, terms, o->pairs, err, Long{(float)target, (float)(target - (float)target)},
                   few, ticket, ticket + 1, loss, stats};
  if (o->pairs > 0) {
    // few pairs of more tokens than a small block has under way get large blocks: 16 of 40,000 tokens
    // 21 us instead of 39, 64 of 8,000 8.5 and 9.7; but 512 of 6,000 22 and 15
    const bool wide = o->pairs <= sms && o->tokens / o->pairs >= 256 * 4 * kPrefAhead;
    prof_begin(K_PREF, s);
    if (wide)
      pref_kernel<1024><<<(unsigned)o->pairs, 1024, 0, s>>>(g, ad);
    else
      pref_kernel<256><<<(unsigned)o->pairs, 256, 0, s>>>(g, ad);
    prof_end(K_PREF, s);
    if (cudaGetLastError() != cudaSuccess) return MOE_LORA_ERR_CUDA;
    if (few) return MOE_LORA_OK;
  }
  return launch_sums<true>(SumArgs{terms, o->pairs, nullptr, true, loss, stats}, ad, g, s);
}
