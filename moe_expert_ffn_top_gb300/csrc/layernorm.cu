// Layer norm over rows of [rows, n], forward and backward (definitions in
// include/moe_lora.h).
//
// Forward: mean, then the sum of squared deviations from it, both from the row in
// registers (one pass over memory; a one-pass variance would cancel where the mean is
// large).  Backward: with h = (x - mean) rstd and u = dy gamma, dx needs avg u and
// avg(u h); dgamma = sum dy h and dbeta = sum dy run down the columns.  HBM is the bound:
// 2 x 8 KB per 4,096-column bf16 row forward, 4 x 8 KB backward with the residual's
// gradient.  Measured on one GB300 (copy bandwidth 6.78 TB/s): 65,536 x 4,096 bf16 forward
// 161 us (6.7 TB/s, 98%), backward with dres and both weight gradients 327 us (6.6 TB/s,
// 97%); one row of 4,096 2.7 us; 347 x 577 fp32 backward 7.0 us (two launches).
//
// Which kernel: rows that stream (norm_*_stream_kernel) when there are enough of them, or
// always backward; norm_fwd_kernel for few rows, where a row spread over many threads is
// faster than a ring that never fills (one row of 4,096 2.7 us; 1,024 rows 6.7 us); the
// staged backward (norm_bwd_odd_kernel) where the tensors' strides differ modulo 16 bytes;
// norm_fwd_long_kernel for forward rows beyond 8,192 vectors of a block's registers.
#include <algorithm>

#include "element.cuh"
#include "launch.h"
#include "prof.h"
#include "sm100_ptx.cuh"

namespace moelora {

namespace {

// A row is handled by a group of `tpr` threads (8, 16, or whole warps); a block holds
// `groups` groups, each with rows of its own.  Thread i of a group holds slots i,
// i + tpr, ... of the row, NV of them, in registers as loaded: a slot is 16 bytes, or
// (VL = 1) two single elements tpr columns apart.
constexpr int kFwdThreads = 512;
constexpr int kNormParts = 152;   // most partial rows of the weight gradients: one per block

struct RowShape {
  int tpr, groups, threads;
  int64_t steps;  // rows / groups
};
// Row `st * groups + group`; a group past the last row repeats it (and stores nothing).
struct RowAt {
  int64_t r;
  bool on;
  __device__ __forceinline__ RowAt(const RowShape& rs, int64_t rows, int64_t st, int group) {
    r = st * rs.groups + group;
    on = r < rows;
    if (!on) r = rows - 1;
  }
};
// Sums over a row's threads, the same in all of them: lanes of a warp, or up to 16 whole
// warps (32 in a block of one row) that meet at barrier `bar`.  Alternating buffers make
// one barrier per sum enough.
struct RowSum {
  int tpr, bar;
  float* red;  // this group's 2 x kRedWords floats
  int buf = 0;
  static constexpr int kRedWords = 64;
  template <int N>
  __device__ __forceinline__ void operator()(float (&v)[N]) {
    if (tpr >= 32) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
      if (tpr > 32) across(v);
    } else {
      for (int o = tpr >> 1; o > 0; o >>= 1)
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    }
  }
  template <int N>
  __device__ __forceinline__ void across(float (&v)[N]) {
    float* r = red + buf * kRedWords;
    buf ^= 1;
    const int gw = tpr >> 5;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
      for (int k = 0; k < N; ++k) r[(threadIdx.x % tpr >> 5) * N + k] = v[k];
    meet();
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = 0.f;
    int w = 0;
    for (; w + 4 / N <= gw; w += 4 / N) {  // 16 bytes at a time
      const float4 u = *reinterpret_cast<const float4*>(r + w * N);
      if (N == 1) {
        v[0] += (u.x + u.y) + (u.z + u.w);
      } else {
        v[0] += u.x + u.z;
        v[N - 1] += u.y + u.w;
      }
    }
    for (; w < gw; ++w)
#pragma unroll
      for (int k = 0; k < N; ++k) v[k] += r[w * N + k];
  }
  // all threads of the row
  __device__ __forceinline__ void meet() const {
    if (tpr <= 32)
      __syncwarp();
    else if (bar < 0)
      __syncthreads();
    else
      asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(tpr) : "memory");
  }
  __device__ __forceinline__ float operator()(float x) {
    float v[1] = {x};
    (*this)(v);
    return v[0];
  }
  __device__ __forceinline__ float2 operator()(float2 x) {
    float v[2] = {x.x, x.y};
    (*this)(v);
    return make_float2(v[0], v[1]);
  }
};
constexpr int kMaxTeams = 15;  // of several warps: one named barrier each

// gamma or beta: NULL, or n elements of a type that is known at run time only (a uniform
// branch per load of a row's slots, against three times the kernels).
struct Weight {
  const void* p;
  int dtype;
  // The elements of N slots, `none` where there are no weights; place(i): slot i.  One
  // branch and no condition inside: all loads are under way together (with a branch per
  // slot their latencies add up, 10 us ahead of the first row).
  template <class W, int VL, int N, int kP, class Place>
  __device__ __forceinline__ void load_as(float2 (&f)[N][kP], const Place& place) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const SlotAt<VL> at = place(i);
      ld_pairs<W, VL>(static_cast<const W*>(p) + (at.in ? at.c : 0), at.in ? at.hop : 0, f[i]);
    }
  }
  template <int VL, int N, int kP, class Place>
  __device__ __forceinline__ void load(float2 (&f)[N][kP], float none, const Place& place) const {
    if (!p) {
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < kP; ++j) f[i][j] = both(none);
    } else if (dtype == MOE_LORA_F32) {
      load_as<float, VL>(f, place);
    } else if (dtype == MOE_LORA_BF16) {
      load_as<__nv_bfloat16, VL>(f, place);
    } else {
      load_as<__half, VL>(f, place);
    }
  }
  // N vectors of 2 kP elements from any column, element by element; columns outside [0, n)
  // give some weight.
  template <class W, int N, int kP, class Col>
  __device__ __forceinline__ void load_any_as(float2 (&f)[N][kP], int first, int n, const Col& col) const {
    const W* w = static_cast<const W*>(p) + first;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < kP; ++j) {
        const int c = col(i) + 2 * j;
        f[i][j] = make_float2(to_f32(w[min(max(c, 0), n - 1)]), to_f32(w[min(max(c + 1, 0), n - 1)]));
      }
  }
  template <int N, int kP, class Col>
  __device__ __forceinline__ void load_any(float2 (&f)[N][kP], float none, int first, int n, const Col& col) const {
    if (!p) {
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < kP; ++j) f[i][j] = both(none);
    } else if (dtype == MOE_LORA_F32) {
      load_any_as<float>(f, first, n, col);
    } else if (dtype == MOE_LORA_BF16) {
      load_any_as<__nv_bfloat16>(f, first, n, col);
    } else {
      load_any_as<__half>(f, first, n, col);
    }
  }
  __device__ __forceinline__ float at(int64_t c, float none) const {
    return !p                        ? none
           : dtype == MOE_LORA_F32  ? static_cast<const float*>(p)[c]
           : dtype == MOE_LORA_BF16 ? to_f32(static_cast<const __nv_bfloat16*>(p)[c])
                                    : to_f32(static_cast<const __half*>(p)[c]);
  }
};

// Few rows, or rows that 16-byte vectors do not fit.  The weights are asked for together
// with the row, so that their latency passes with its.  Groups of more than one warp
// have the block for themselves (groups = 1).
template <class T, int VL, int NV>
__global__ void __launch_bounds__(kFwdThreads) norm_fwd_kernel(moe_lora_norm nm, RowShape rs, const T* x,
                                                               Weight gamma, Weight beta, T* y, float* mean,
                                                               float* rstd) {
  __shared__ __align__(16) float red[kMaxTeams * 2 * RowSum::kRedWords];
  constexpr int kP = Vec<T, VL>::kPairs;
  const int n = nm.n;
  const int lane = threadIdx.x % rs.tpr, group = threadIdx.x / rs.tpr;
  RowSum sum{rs.tpr, -1, red};
  const float rn = 1.0f / n;
  constexpr int kAhead = VL == 1 ? 8 : 2;  // slots whose weights fit in registers beside the row
  for (int64_t st = blockIdx.x; st < rs.steps; st += gridDim.x) {
    const RowAt row(rs, nm.rows, st, group);
    const T* xr = x + row.r * nm.ldx;
    Vec<T, VL> v[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const SlotAt<VL> at(lane, i, rs.tpr, n);
      if (at.in)
        v[i].load(xr + at.c, at.hop);
      else
        v[i].clear();
    }
    constexpr int kW = NV < kAhead ? NV : kAhead;
    float2 g[kW][kP], b[kW][kP];
    const auto weights = [&](int i0) {
      const auto place = [&](int i) { return SlotAt<VL>(lane, i0 + i, rs.tpr, n); };
      gamma.load<VL>(g, 1.f, place);
      beta.load<VL>(b, 0.f, place);
    };
    if (NV <= kAhead) weights(0);
    float2 s = both(0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < kP; ++j) s = add2(s, v[i].get(j));
    const float mu = sum(s.x + s.y) * rn;
    float2 q = both(0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const SlotAt<VL> at(lane, i, rs.tpr, n);
      if (at.in)
#pragma unroll
        for (int j = 0; j < kP; ++j) {
          const float2 d = add2(v[i].get(j), at.pair(-mu));
          q = fma2(d, d, q);
        }
    }
    const float rt = rsqrtf(sum(q.x + q.y) * rn + nm.eps);
    T* yr = y + row.r * nm.ldy;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const SlotAt<VL> at(lane, i, rs.tpr, n);
      if (NV > kAhead && i % kW == 0) weights(i);
      if (at.in && row.on) {
        const auto &gi = g[i % kW], &bi = b[i % kW];
        Vec<T, VL> o;
#pragma unroll
        for (int j = 0; j < kP; ++j) o.put(j, fma2(mul2(add2(v[i].get(j), both(-mu)), both(rt)), gi[j], bi[j]));
        o.store(yr + at.c, at.hop);
      }
    }
    if (mean && row.on && lane == 0) {
      mean[row.r] = mu;
      rstd[row.r] = rt;
    }
  }
}

// Rows of whole 16-byte vectors stream through shared memory: one resident block per SM,
// its teams (the threads of a row: 8, 16 or 32 lanes, or several warps) take rows in
// turn.  Every thread copies its own slots kStages - 1 rows ahead with asynchronous
// copies and reads only those, so rows in flight cost neither registers nor barriers; a
// thread has the same columns in every row, so its weights stay in its registers.
// Forward: 64 columns a thread, 255 registers: what a warp does once per row (sums,
// addresses, waits) is half of the instructions at 32 columns (65,536 x 4,096 bf16: 163
// us against 179 us, and 253 us at 16).  Backward: 16 columns and their two sums (32
// columns in 256 threads: 351 us against 328 us).
constexpr int kFwdStreamThreads = 256, kFwdColumns = 64;
constexpr int kBwdStreamThreads = 512, kBwdColumns = 16;
constexpr int kOddThreads = 512;
// From here on shifted rows stream forward.  In registers and streamed, us: 130 columns 2.6
// and 3.4 at 256 rows, 2.9 and 3.4 at 1,029, 4.5 and 3.5 at 2,048; 577 columns 3.1 and 4.5,
// 5.1 and 4.5, 6.9 and 4.7; 1,027 bf16 3.4 and 5.5 at 256 rows, 5.5 and 5.5 at 512; 2,049
// fp16 3.6 and 5.9 at 150, 5.5 and 5.8 at 256, 7.6 and 6.0 at 384; 4,097 bf16 4.9 and 5.7 at
// 150, 7.7 and 5.6 at 192, 17.4 and 11.0 at 1,029; 8,191 bf16 5.2 and 5.1 up to 150, 8.8 and
// 6.8 at 256.  One number of rows for all widths: narrow rows would stay in registers for
// longer (by 1 us), rows of 4,096 and more could stream from 160 rows on (2 us).
constexpr int kShiftRows = 256;
struct StreamShape {
  int tpr, teams;
};

// How rows lie on the 16-byte grid: as whole vectors that fill every slot of every thread
// (kFull, no bounds checks: 65,536 x 4,096 bf16 forward 161 us against 176 us), as whole
// vectors, or (kShift) they begin and end anywhere.  A shifted row
// is taken in the aligned vectors that cover it, so that its first column is `shift`
// elements into the first vector (what lies before it belongs to the row before: the
// tensor itself starts aligned).  shift = r * ld mod VL depends on the row; the grid is
// such that all rows of a team have the same, which keeps a thread's columns, its weights
// and its sums in place.
enum RowFit { kFull, kAligned, kShift };
// What a thread knows of its columns: slot i starts at column c0 + i * dc, `nv` slots lie
// (in part) inside the row.  NV is the number that the row needs, or one more: all but
// the last two slots are inside for every thread, and only the first and the last three
// can hold an end of the row, so that the others carry no checks.
// (kExact false: the row may be any shorter, as the last slice of a wide one.)
template <RowFit kFit, int NV, bool kExact = true>
struct Columns {
  int c0, dc, nv, n;
  __device__ __forceinline__ Columns(int lane, int tpr, int n, int vl, int shift) : n(n) {
    c0 = lane * vl - (kFit == kShift ? shift : 0);
    dc = tpr * vl;
    nv = c0 < n ? (n - c0 + dc - 1) / dc : 0;
  }
  __device__ __forceinline__ bool in(int i) const { return kFit == kFull || (kExact && i < NV - 2) || i < nv; }
  __device__ __forceinline__ int col(int i) const { return c0 + i * dc; }
  template <int kP>
  __device__ __forceinline__ bool edge(int i) const {
    return kFit == kShift && (((!kExact || i == 0) && col(i) < 0) || ((!kExact || i >= NV - 3) && col(i) + 2 * kP > n));
  }
  // 0 for what is not the row's
  template <int kP>
  __device__ __forceinline__ void clip(int i, float2 (&v)[kP]) const {
    if constexpr (kFit == kShift) {
      if (!edge<kP>(i)) return;
#pragma unroll
      for (int j = 0; j < kP; ++j) {
        if ((unsigned)(col(i) + 2 * j) >= (unsigned)n) v[j].x = 0.f;
        if ((unsigned)(col(i) + 2 * j + 1) >= (unsigned)n) v[j].y = 0.f;
      }
    }
  }
  template <class T>
  __device__ __forceinline__ void copy(uint4* slot, const T* row, int i) const {
    if (kFit == kShift && (!kExact || i >= NV - 3))
      async_copy16_part(slot, row + col(i), min(16, (n - col(i)) * (int)sizeof(T)));
    else
      async_copy16(slot, row + col(i));
  }
  // a slot's results; `fits`: the output's rows lie on the grid as the input's do
  template <class T, int VL, int kP>
  __device__ __forceinline__ void store(T* row, int i, const float2 (&v)[kP], bool fits) const {
    if (kFit != kShift || (fits && !edge<kP>(i))) {
      Vec<T, VL> o;
#pragma unroll
      for (int j = 0; j < kP; ++j) o.put(j, v[j]);
      o.store(row + col(i), 0);
    } else {
#pragma unroll
      for (int j = 0; j < kP; ++j) {
        const int c = col(i) + 2 * j;
        if ((unsigned)c < (unsigned)n) row[c] = from_f32<T>(v[j].x);
        if ((unsigned)(c + 1) < (unsigned)n) row[c + 1] = from_f32<T>(v[j].y);
      }
    }
  }
};

template <class T, int NV, int kStages, RowFit kFit>
__global__ void __launch_bounds__(kFwdStreamThreads, 1)
    norm_fwd_stream_kernel(moe_lora_norm nm, StreamShape ss, const T* x, Weight gamma, Weight beta, T* y, float* mean,
                           float* rstd) {
  constexpr int VL = 16 / sizeof(T), kP = VL / 2;
  extern __shared__ __align__(16) uint8_t ring_sm[];
  __shared__ __align__(16) float red[kMaxTeams * 2 * RowSum::kRedWords];
  const int n = nm.n;
  const Ring<kStages, NV> ring(ring_sm);
  const int lane = threadIdx.x % ss.tpr, team = threadIdx.x / ss.tpr;
  RowSum sum{ss.tpr, team + 1, red + (ss.tpr > 32 ? team * 2 * RowSum::kRedWords : 0)};
  const float rn = 1.0f / n;
  const int64_t step = (int64_t)gridDim.x * ss.teams, first = blockIdx.x * (int64_t)ss.teams + team;
  const Columns<kFit, NV> cl(lane, ss.tpr, n, VL, (int)(first * nm.ldx & (VL - 1)));
  const bool y_fits = ((nm.ldx ^ nm.ldy) & (VL - 1)) == 0;
  const auto copy_row = [&](int64_t r, int s) {
    if (r < nm.rows) {
      const T* xr = x + r * nm.ldx;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (cl.in(i)) cl.copy(ring.slot(s, i), xr, i);
    }
    async_commit();
  };
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) copy_row(first + s * step, s);
  float2 g[NV][kP], b[NV][kP];
  if (kFit == kShift) {
    const auto col = [&](int i) { return cl.col(i); };
    gamma.load_any(g, 1.f, 0, n, col);
    beta.load_any(b, 0.f, 0, n, col);
  } else {
    const auto place = [&](int i) { return SlotAt<VL>(lane, i, ss.tpr, n); };
    gamma.load<VL>(g, 1.f, place);
    beta.load<VL>(b, 0.f, place);
  }
  int s = 0;
  // all teams of the block leave together: one without a row works on what its slots hold
  for (int64_t r = first; r - team < nm.rows; r += step) {
    copy_row(r + (kStages - 1) * step, s == 0 ? kStages - 1 : s - 1);
    async_wait<kStages - 1>();
    float2 v[NV][kP];
    float2 t[2] = {both(0.f), both(0.f)};
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (cl.in(i)) {
        Vec<T, VL> w;
        w.from_smem(ring.slot(s, i));
#pragma unroll
        for (int j = 0; j < kP; ++j) v[i][j] = w.get(j);
        cl.clip(i, v[i]);
#pragma unroll
        for (int j = 0; j < kP; ++j) t[j & 1] = add2(t[j & 1], v[i][j]);
      }
    t[0] = add2(t[0], t[1]);
    const float mu = sum(t[0].x + t[0].y) * rn;
    t[0] = t[1] = both(0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (cl.in(i)) {
#pragma unroll
        for (int j = 0; j < kP; ++j) v[i][j] = add2(v[i][j], both(-mu));
        cl.clip(i, v[i]);
#pragma unroll
        for (int j = 0; j < kP; ++j) t[j & 1] = fma2(v[i][j], v[i][j], t[j & 1]);
      }
    t[0] = add2(t[0], t[1]);
    const float rt = rsqrtf(sum(t[0].x + t[0].y) * rn + nm.eps);
    if (r < nm.rows) {
      T* yr = y + r * nm.ldy;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (cl.in(i)) {
          float2 o[kP];
#pragma unroll
          for (int j = 0; j < kP; ++j) o[j] = fma2(mul2(v[i][j], both(rt)), g[i][j], b[i][j]);
          cl.template store<T, VL>(yr, i, o, y_fits);
        }
      if (mean && lane == 0) {
        mean[r] = mu;
        rstd[r] = rt;
      }
    }
    s = s == kStages - 1 ? 0 : s + 1;
  }
}

// dx, and per block the sums of the weight gradients over its rows: dgamma / dbeta at
// block * part_ld (the partial rows, or the outputs themselves when one block has all
// rows).  Same streaming; dx needs one sum (of two values) per row, the weight gradients
// stay in registers until the block's rows are done.
//
// Rows wider than kBwdSlice are worked on in slices (blockIdx.y).  Up to eight slices are
// a cluster (kCluster): its blocks exchange a row's sums through distributed shared
// memory.  More take two launches: kSums leaves every slice's part of a row's sums in
// `sums` [rows][slices], kApply adds them and reads x and dy again (4,096 x 16,384 bf16:
// 2.5 TB/s in two launches, 3.4 TB/s as clusters; fp32 3.5 and 5.4 TB/s).
enum BwdMode { kWhole, kCluster, kSums, kApply };
constexpr int kBwdSlice = kBwdStreamThreads * kBwdColumns;
constexpr int kBwdCluster = 8;
// Slice blockIdx.y, `width` columns, of a row of n (of one slice, kWhole).
template <BwdMode kMode>
struct Slice {
  int first, n;
  __device__ __forceinline__ Slice(int all, int width)
      : first(kMode == kWhole ? 0 : blockIdx.y * width), n(kMode == kWhole ? all : min(width, all - first)) {}
};
// The slices' parts of the rows that a cluster's teams work on, in two buffers: a block
// writes the second time into one only after all have read it (they meet in between).
struct SliceSums {
  float2 v[2][kMaxTeams][kBwdCluster];
};
// A row's two sums over all slices, from this slice's; false: the row is done (kSums).
template <BwdMode kMode, class Sum>
__device__ __forceinline__ bool row_sums(Sum& sum, float2 mine, float2& all, float2* sums, int64_t r, bool on,
                                         int lane, SliceSums* sm = nullptr, int team = 0, int buf = 0) {
  if (kMode == kApply) {
    all = both(0.f);
    if (on)
      for (int i = 0; i < (int)gridDim.y; ++i) all = add2(all, sums[r * gridDim.y + i]);
    return true;
  }
  all = sum(mine);
  if (kMode == kWhole) return true;
  if (kMode == kCluster) {
    const int slices = gridDim.y;
    if (lane < slices) {
      const uint32_t to = mapa_shared(smem_u32(&sm->v[buf][team][blockIdx.y]), lane);
      asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(to), "f"(all.x), "f"(all.y) : "memory");
    }
    cluster_sync_all();
    all = both(0.f);
    for (int i = 0; i < slices; ++i) all = add2(all, sm->v[buf][team][i]);
    return true;
  }
  if (on && lane == 0) sums[r * gridDim.y + blockIdx.y] = all;
  return false;
}
// A block's sums of the weight gradients from its teams' [teams][2][n] in shared memory
// (`acc`, 16 columns of either per thread), teams in order: to dgamma / dbeta, or, where
// all blocks are one cluster (`together`), first added over the blocks in order.
__device__ __forceinline__ void store_wgrad(float* acc, int teams, int n, float* dgamma, float* dbeta, bool together) {
  const auto store = [&](int i, float v) {
    if (i < n) {
      if (dgamma) dgamma[i] = v;
    } else if (dbeta) {
      dbeta[i - n] = v;
    }
  };
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * n; i += blockDim.x) {
    float v = acc[i];
    for (int k = 1; k < teams; ++k) v += acc[(int64_t)k * 2 * n + i];
    if (together)
      acc[i] = v;
    else
      store(i, v);
  }
  if (!together) return;
  cluster_sync_all();
  const int ranks = gridDim.x, per = (2 * n + ranks - 1) / ranks, end = min(2 * n, (int)(blockIdx.x + 1) * per);
  for (int i = blockIdx.x * per + threadIdx.x; i < end; i += blockDim.x) {
    float v = 0.f;
    for (int k = 0; k < ranks; ++k) {
      float u;
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(u) : "r"(mapa_shared(smem_u32(acc + i), k)) : "memory");
      v += u;
    }
    store(i, v);
  }
  cluster_sync_all();  // nobody leaves while its sums are read
}

template <class T, int NV, int kStages, BwdMode kMode, RowFit kFit>
__global__ void __launch_bounds__(kBwdStreamThreads, 1)
    norm_bwd_stream_kernel(moe_lora_norm nm, StreamShape ss, const T* x, Weight gamma, const float* mean,
                           const float* rstd, const T* dy, const T* dres, T* dx, float* dgamma, float* dbeta,
                           int64_t part_ld, float2* sums, int slice) {
  constexpr int VL = 16 / sizeof(T), kP = VL / 2;
  extern __shared__ __align__(16) uint8_t ring_sm[];  // afterwards: the teams' sums [teams][2][n]
  __shared__ __align__(16) float red[kMaxTeams * 2 * RowSum::kRedWords];
  const Slice<kMode> sl(nm.n, slice);
  const int n = sl.n;
  if (kMode != kWhole) {
    x += sl.first;
    dy += sl.first;
    dres += dres ? sl.first : 0;
    dx += sl.first;
  }
  __shared__ SliceSums slice_sm;
  const Ring<kStages, 3 * NV> ring(ring_sm);
  const int lane = threadIdx.x % ss.tpr, team = threadIdx.x / ss.tpr;
  RowSum sum{ss.tpr, team + 1, red + (ss.tpr > 32 ? team * 2 * RowSum::kRedWords : 0)};
  const float rn = 1.0f / nm.n;
  const int64_t step = (int64_t)gridDim.x * ss.teams, first = blockIdx.x * (int64_t)ss.teams + team;
  const Columns<kFit, NV, kMode == kWhole> cl(lane, ss.tpr, n, VL, (int)(first * nm.ldx & (VL - 1)));
  const auto copy_row = [&](int64_t r, int s) {
    if (r < nm.rows) {
      const T *xr = x + r * nm.ldx, *gr = dy + r * nm.ldy, *er = dres + r * nm.lddres;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (cl.in(i)) {
          cl.copy(ring.slot(s, i), xr, i);
          cl.copy(ring.slot(s, NV + i), gr, i);
          if (kMode != kSums && dres) cl.copy(ring.slot(s, 2 * NV + i), er, i);
        }
    }
    async_commit();
  };
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) copy_row(first + s * step, s);
  float2 g[NV][kP], dg[NV][kP], db[NV][kP];
  if (kFit == kShift)
    gamma.load_any(g, 1.f, sl.first, n, [&](int i) { return cl.col(i); });
  else
    gamma.load<VL>(g, 1.f, [&](int i) { return SlotAt<VL>(lane, i, ss.tpr, n).shifted(sl.first); });
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < kP; ++j) dg[i][j] = db[i][j] = both(0.f);
  const auto stat = [&](const float* p, int64_t r) { return r < nm.rows ? p[r] : 0.f; };
  float mu = stat(mean, first), rt = stat(rstd, first);
  int s = 0, buf = 0;
  if (kMode == kCluster) cluster_sync_all();  // all of the cluster run before one writes into another
  for (int64_t r = first; r - team < nm.rows; r += step) {
    copy_row(r + (kStages - 1) * step, s == 0 ? kStages - 1 : s - 1);
    const float mu1 = stat(mean, r + step), rt1 = stat(rstd, r + step);
    async_wait<kStages - 1>();
    const bool on = r < nm.rows;
    float2 h[NV][kP], u[NV][kP];
    float2 su = both(0.f), sh = both(0.f);
    if (on)
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (cl.in(i)) {
          Vec<T, VL> xv, gv;
          xv.from_smem(ring.slot(s, i));
          gv.from_smem(ring.slot(s, NV + i));
          float2 d[kP];
#pragma unroll
          for (int j = 0; j < kP; ++j) {
            d[j] = gv.get(j);
            h[i][j] = mul2(add2(xv.get(j), both(-mu)), both(rt));
          }
          cl.clip(i, d);
          cl.clip(i, h[i]);
#pragma unroll
          for (int j = 0; j < kP; ++j) {
            u[i][j] = mul2(d[j], g[i][j]);
            su = add2(su, u[i][j]);
            sh = fma2(u[i][j], h[i][j], sh);
            dg[i][j] = fma2(d[j], h[i][j], dg[i][j]);
            db[i][j] = add2(db[i][j], d[j]);
          }
        }
    float2 t;
    const bool more =
        row_sums<kMode>(sum, make_float2(su.x + su.y, sh.x + sh.y), t, sums, r, on, lane, &slice_sm, team, buf);
    buf ^= 1;
    const float2 na = both(-t.x * rn), nb = both(-t.y * rn);
    if (on && more) {
      T* dr = dx + r * nm.lddx;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (cl.in(i)) {
          Vec<T, VL> ev;
          float2 o[kP];
          if (dres) ev.from_smem(ring.slot(s, 2 * NV + i));
#pragma unroll
          for (int j = 0; j < kP; ++j) {
            const float2 w = fma2(h[i][j], nb, add2(u[i][j], na));
            o[j] = dres ? fma2(w, both(rt), ev.get(j)) : mul2(w, both(rt));
          }
          cl.template store<T, VL>(dr, i, o, true);
        }
    }
    mu = mu1;
    rt = rt1;
    s = s == kStages - 1 ? 0 : s + 1;
  }
  if (kMode == kSums || (!dgamma && !dbeta)) return;
  async_wait<0>();
  __syncthreads();
  float* acc = reinterpret_cast<float*>(ring_sm);
  float *ag = acc + team * 2 * n, *ab = ag + n;
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (cl.in(i))
#pragma unroll
      for (int j = 0; j < kP; j += 2) {
        const int e = cl.col(i) + 2 * j;
        if (kFit == kShift) {  // the columns of the row, one by one
          const float vg[4] = {dg[i][j].x, dg[i][j].y, dg[i][j + 1].x, dg[i][j + 1].y};
          const float vb[4] = {db[i][j].x, db[i][j].y, db[i][j + 1].x, db[i][j + 1].y};
#pragma unroll
          for (int l = 0; l < 4; ++l)
            if ((unsigned)(e + l) < (unsigned)n) {
              ag[e + l] = vg[l];
              ab[e + l] = vb[l];
            }
          continue;
        }
        *reinterpret_cast<float4*>(ag + e) = make_float4(dg[i][j].x, dg[i][j].y, dg[i][j + 1].x, dg[i][j + 1].y);
        *reinterpret_cast<float4*>(ab + e) = make_float4(db[i][j].x, db[i][j].y, db[i][j + 1].x, db[i][j + 1].y);
      }
  const int64_t at = blockIdx.x * part_ld + sl.first;
  store_wgrad(acc, ss.teams, n, dgamma ? dgamma + at : nullptr, dbeta ? dbeta + at : nullptr,
              kMode == kWhole && part_ld == 0);
}

// The backward where the tensors' rows lie on the 16-byte grid in different ways, so that
// no vector of one matches a vector of the others.  A team copies the aligned 16-byte
// pieces that cover a row, what lies before its start in the first piece included (never
// before the tensor's: that start is aligned), nothing past its end; then every thread
// reads its elements, tpr columns apart.  Pieces are read by other threads than copied
// them, so a team meets when a row has come, and a stage is refilled only after the sums
// of the next row, which all of the team have to reach.  2.4-3.5 TB/s at 1,024 to 4,096
// columns bf16, bound by instructions.
template <class T>
struct OddStage {
  char* base;  // of this team; stages of `tensors` pieces of `cap` bytes
  int cap, tensors;
  // asynchronous copy of n elements from p
  __device__ __forceinline__ void copy(int stage, int k, const T* p, int n, int lane, int tpr) const {
    const int o = (int)(reinterpret_cast<uintptr_t>(p) & 15), bytes = o + n * (int)sizeof(T);
    const char* src = reinterpret_cast<const char*>(p) - o;
    char* dst = base + (stage * tensors + k) * cap;
    for (int c = lane * 16; c < bytes; c += tpr * 16) async_copy16_part(dst + c, src + c, min(16, bytes - c));
  }
  __device__ __forceinline__ const T* row(int stage, int k, const T* p) const {
    return reinterpret_cast<const T*>(base + (stage * tensors + k) * cap + (reinterpret_cast<uintptr_t>(p) & 15));
  }
};
inline int odd_cap(int n, int size) { return (n * size + 15 + 15) / 16 * 16; }
__device__ __forceinline__ int odd_cap_device(int n, int size) { return (n * size + 15 + 15) / 16 * 16; }
// The two elements of slot `at` of a staged row.
template <class T>
__device__ __forceinline__ float2 odd_pair(const T* row, const SlotAt<1>& at) {
  return make_float2(to_f32(row[at.c]), at.hop ? to_f32(row[at.c + at.hop]) : 0.f);
}

template <class T, int NP, int kStages, BwdMode kMode>
__global__ void __launch_bounds__(kOddThreads, 1)
    norm_bwd_odd_kernel(moe_lora_norm nm, StreamShape ss, const T* x, Weight gamma, const float* mean,
                        const float* rstd, const T* dy, const T* dres, T* dx, float* dgamma, float* dbeta,
                        int64_t part_ld, float2* sums, int slice) {
  extern __shared__ __align__(16) char stage_sm[];  // afterwards: the teams' sums [teams][2][n]
  __shared__ __align__(16) float red[kMaxTeams * 2 * RowSum::kRedWords];
  const Slice<kMode> sl(nm.n, slice);
  const int n = sl.n, lane = threadIdx.x % ss.tpr, team = threadIdx.x / ss.tpr;
  const int tensors = kMode != kSums && dres ? 3 : 2;
  if (kMode != kWhole) {
    x += sl.first;
    dy += sl.first;
    dres += dres ? sl.first : 0;
    dx += sl.first;
  }
  const int cap = odd_cap_device(n, sizeof(T));
  const OddStage<T> st{stage_sm + (size_t)team * kStages * tensors * cap, cap, tensors};
  RowSum sum{ss.tpr, team + 1, red + (ss.tpr > 32 ? team * 2 * RowSum::kRedWords : 0)};
  const float rn = 1.0f / nm.n;
  const int64_t step = (int64_t)gridDim.x * ss.teams, first = blockIdx.x * (int64_t)ss.teams + team;
  const auto copy_row = [&](int64_t r, int s) {
    if (r < nm.rows) {
      st.copy(s, 0, x + r * nm.ldx, n, lane, ss.tpr);
      st.copy(s, 1, dy + r * nm.ldy, n, lane, ss.tpr);
      if (tensors == 3) st.copy(s, 2, dres + r * nm.lddres, n, lane, ss.tpr);
    }
    async_commit();
  };
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) copy_row(first + s * step, s);
  float2 g[NP][1], dg[NP], db[NP];
  gamma.load<1>(g, 1.f, [&](int i) { return SlotAt<1>(lane, i, ss.tpr, n).shifted(sl.first); });
#pragma unroll
  for (int i = 0; i < NP; ++i) dg[i] = db[i] = both(0.f);
  const auto stat = [&](const float* p, int64_t r) { return r < nm.rows ? p[r] : 0.f; };
  float mu = stat(mean, first), rt = stat(rstd, first);
  int s = 0;
  for (int64_t r = first; r - team < nm.rows; r += step) {
    const float mu1 = stat(mean, r + step), rt1 = stat(rstd, r + step);
    async_wait<kStages - 2>();
    sum.meet();
    const bool on = r < nm.rows;
    const int64_t ra = on ? r : 0;
    const T *xr = st.row(s, 0, x + ra * nm.ldx), *gr = st.row(s, 1, dy + ra * nm.ldy);
    float2 h[NP], u[NP], su = both(0.f), sh = both(0.f);
    if (on)
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const SlotAt<1> at(lane, i, ss.tpr, n);
        if (at.in) {
          const float2 d = odd_pair(gr, at);
          h[i] = mul2(add2(odd_pair(xr, at), at.pair(-mu)), both(rt));
          u[i] = mul2(d, g[i][0]);
          su = add2(su, u[i]);
          sh = fma2(u[i], h[i], sh);
          dg[i] = fma2(d, h[i], dg[i]);
          db[i] = add2(db[i], d);
        }
      }
    float2 t;
    const bool more = row_sums<kMode>(sum, make_float2(su.x + su.y, sh.x + sh.y), t, sums, r, on, lane);
    if (kMode == kApply) sum.meet();  // no sum to meet at: the stage before this one is read by nobody any more
    copy_row(r + (kStages - 1) * step, s == 0 ? kStages - 1 : s - 1);
    const float2 na = both(-t.x * rn), nb = both(-t.y * rn);
    if (on && more) {
      T* dr = dx + r * nm.lddx;
      const T* er = tensors == 3 ? st.row(s, 2, dres + r * nm.lddres) : nullptr;
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const SlotAt<1> at(lane, i, ss.tpr, n);
        if (at.in) {
          const float2 w = fma2(h[i], nb, add2(u[i], na));
          const float2 o = er ? fma2(w, both(rt), odd_pair(er, at)) : mul2(w, both(rt));
          dr[at.c] = from_f32<T>(o.x);
          if (at.hop) dr[at.c + at.hop] = from_f32<T>(o.y);
        }
      }
    }
    mu = mu1;
    rt = rt1;
    s = s == kStages - 1 ? 0 : s + 1;
  }
  if (kMode == kSums || (!dgamma && !dbeta)) return;
  async_wait<0>();
  __syncthreads();
  float* acc = reinterpret_cast<float*>(stage_sm);
  float *ag = acc + team * 2 * n, *ab = ag + n;
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const SlotAt<1> at(lane, i, ss.tpr, n);
    if (at.in) {
      ag[at.c] = dg[i].x;
      ab[at.c] = db[i].x;
    }
    if (at.hop) {
      ag[at.c + at.hop] = dg[i].y;
      ab[at.c + at.hop] = db[i].y;
    }
  }
  const int64_t at0 = blockIdx.x * part_ld + sl.first;
  store_wgrad(acc, ss.teams, n, dgamma ? dgamma + at0 : nullptr, dbeta ? dbeta + at0 : nullptr,
              kMode == kWhole && part_ld == 0);
}

// dgamma and dbeta (blockIdx.y) from the blocks' partial rows: 32 columns per block,
// warp w adds every 8th partial, then the warps' sums are added in order.
__global__ void __launch_bounds__(256) norm_wgrad_kernel(int n, int parts, const float* part, float* dgamma,
                                                         float* dbeta) {
  __shared__ float sm[8][33];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  float* out = blockIdx.y ? dbeta : dgamma;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!out) return;
  float s = 0.f;
  if (c < n)
#pragma unroll 4
    for (int p = w; p < parts; p += 8) s += part[((int64_t)p * 2 + blockIdx.y) * n + c];
  sm[w][lane] = s;
  __syncthreads();
  if (w == 0 && c < n) {
#pragma unroll
    for (int i = 1; i < 8; ++i) s += sm[i][lane];
    out[c] = s;
  }
}

// Rows longer than a block's registers hold: the row is read again for every pass.
constexpr int kLongThreads = 512;
__device__ __forceinline__ float block_sum(float v, float* sm) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.f;
  for (int w = 0; w < kLongThreads / 32; ++w) s += sm[w];
  return s;
}
template <class T>
__global__ void __launch_bounds__(kLongThreads) norm_fwd_long_kernel(moe_lora_norm nm, const T* x, Weight gamma,
                                                                     Weight beta, T* y, float* mean, float* rstd) {
  __shared__ float sm[32];
  const int n = nm.n;
  for (int64_t r = blockIdx.x; r < nm.rows; r += gridDim.x) {
    const T* xr = x + r * nm.ldx;
    float s = 0.f;
    for (int c = threadIdx.x; c < n; c += blockDim.x) s += to_f32(xr[c]);
    const float mu = block_sum(s, sm) / n;
    float q = 0.f;
    for (int c = threadIdx.x; c < n; c += blockDim.x) {
      const float d = to_f32(xr[c]) - mu;
      q += d * d;
    }
    const float rs = 1.0f / sqrtf(block_sum(q, sm) / n + nm.eps);
    T* yr = y + r * nm.ldy;
    for (int c = threadIdx.x; c < n; c += blockDim.x) {
      const float h = (to_f32(xr[c]) - mu) * rs;
      yr[c] = from_f32<T>(h * gamma.at(c, 1.f) + beta.at(c, 0.f));
    }
    if (mean && threadIdx.x == 0) {
      mean[r] = mu;
      rstd[r] = rs;
    }
  }
}
// Scratch of the backward: partial rows of the weight gradients, then the slices' row
// sums (wide rows).
size_t part_bytes(const moe_lora_norm& nm) { return (size_t)kNormParts * 2 * nm.n * sizeof(float); }
size_t sums_bytes(const moe_lora_norm& nm) {
  return nm.n > kBwdSlice ? sizeof(float2) * (size_t)nm.rows * ((nm.n + kBwdSlice - 9) / (kBwdSlice - 8)) : 0;
}

int check_ld(int64_t* ld, int n) {
  if (*ld == 0) *ld = n;
  return *ld < n || *ld > ((int64_t)1 << 40) ? MOE_LORA_ERR_DIMS : MOE_LORA_OK;
}

// Sizes and types of `in`, its strides completed in `out`.
int check_norm(const moe_lora_norm* in, moe_lora_norm* out) {
  if (!in) return MOE_LORA_ERR_NULL;
  *out = *in;
  if (!dtype_ok(in->dtype) || !dtype_ok(in->wdtype)) return MOE_LORA_ERR_UNSUPPORTED;
  if (in->rows < 0 || in->rows > ((int64_t)1 << 40) || in->n < 1 || in->n > 1 << 24) return MOE_LORA_ERR_DIMS;
  int rc;
  if ((rc = check_ld(&out->ldx, in->n)) || (rc = check_ld(&out->ldy, in->n)) || (rc = check_ld(&out->lddx, in->n)) ||
      (rc = check_ld(&out->lddres, in->n)))
    return rc;
  return MOE_LORA_OK;
}

// 16-byte vectors need every row of every tensor to start on a 16-byte boundary (the
// bases do) and to end on one.
bool rows_aligned(const moe_lora_norm& nm, bool bwd, bool dres) {
  int64_t a = nm.n | nm.ldx | nm.ldy;
  if (bwd) a |= nm.lddx;
  if (dres) a |= nm.lddres;
  return a % (16 / dtype_bytes(nm.dtype)) == 0;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Threads for rows of `slots` slots, nv at most per thread: the fewest that hold a row
// (8, 16 or whole warps).
int row_threads(int slots, int nv) {
  const int need = (int)ceil_div(slots, nv);
  return need <= 8 ? 8 : need <= 16 ? 16 : (int)ceil_div(need, 32) * 32;
}
RowShape row_shape(int64_t rows, int tpr, int groups) {
  return RowShape{tpr, groups, tpr * groups, ceil_div(rows, groups)};
}

struct FwdArgs {
  const moe_lora_norm& nm;
  const void* x;
  Weight gamma, beta;
  void* y;
  float *mean, *rstd;
  int sms;
  cudaStream_t s;
};

template <class T, int VL, int NV>
int launch_fwd(const FwdArgs& a, const RowShape& rs) {
  const int64_t grid = std::min<int64_t>(rs.steps, 0x7fffffff);
  prof_begin(K_NORM_FWD, a.s);
  norm_fwd_kernel<T, VL, NV>
      <<<(unsigned)grid, rs.threads, 0, a.s>>>(a.nm, rs, (const T*)a.x, a.gamma, a.beta, (T*)a.y, a.mean, a.rstd);
  prof_end(K_NORM_FWD, a.s);
  return cudaGetLastError() == cudaSuccess ? MOE_LORA_OK : MOE_LORA_ERR_CUDA;
}

constexpr size_t kMaxSmem = 216 * 1024;  // dynamic, beside the kernels' static 9.6 KB at most (227 KB in all)

// Stages of the rings: 64 to 128 KB of copies under way per SM at full width, where an SM
// needs about 45 KB to hide the memory's latency (65,536 x 4,096 bf16 backward: three
// stages 328 us, four 331 us; forward: two 173 us, three 164-168 us, four 161 us).
template <class T>
constexpr int fwd_stages() { return sizeof(T) == 2 ? 4 : 3; }
template <class T>
constexpr int bwd_stages() { return sizeof(T) == 2 ? 3 : 2; }

// Threads of a row of `slots` slots and, in *nv, slots per thread (`most` at most, even
// beyond 4 for fp32's many).  What a warp does once per row costs about three slots.
StreamShape stream_shape(int slots, int most, int threads, int* nv) {
  StreamShape best = {0, 0};
  float cost = 0.f;
  for (int tpr = 8; tpr <= threads; tpr = tpr < 32 ? 2 * tpr : tpr + 32) {
    int v = (int)ceil_div(slots, tpr);
    if (v > most) continue;
    if (most > 8 && v > 4) v += v & 1;
    const float c = (3.f + v) / (threads / tpr);
    if (!best.tpr || c < cost) {
      best = StreamShape{tpr, threads / tpr};
      cost = c;
      *nv = v;
    }
  }
  return best;
}

// Blocks of a streamed kernel: rows whose vectors are shifted need teams that step by a
// multiple of VL rows, unless no team has a second row.
int stream_grid(int64_t rows, int teams, int most, bool shift) {
  int64_t grid = ceil_div(rows, teams);
  if (grid <= most) return (int)grid;
  return shift ? std::max(8, most / 8 * 8) : most;
}

template <class T, int NV>
int launch_fwd_stream(const FwdArgs& a, const StreamShape& ss, bool shift) {
  constexpr int kS = fwd_stages<T>();
  const bool full = !shift && a.nm.n == ss.tpr * NV * 16 / (int)sizeof(T);
  const auto kernel = full    ? norm_fwd_stream_kernel<T, NV, kS, kFull>
                      : shift ? norm_fwd_stream_kernel<T, NV, kS, kShift>
                              : norm_fwd_stream_kernel<T, NV, kS, kAligned>;
  const int threads = ss.tpr * ss.teams;
  const size_t smem = ring_bytes<fwd_stages<T>(), NV>(threads);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(stream_grid(a.nm.rows, ss.teams, a.sms, shift));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = a.s;
  prof_begin(K_NORM_FWD, a.s);
  const cudaError_t e = launch_allowed(cfg, false, kernel, a.nm, ss, static_cast<const T*>(a.x), a.gamma, a.beta,
                                       static_cast<T*>(a.y), a.mean, a.rstd);
  prof_end(K_NORM_FWD, a.s);
  return e == cudaSuccess ? MOE_LORA_OK : MOE_LORA_ERR_CUDA;
}

// Shared memory of the staged kernels: as many teams as fit.
template <class T>
size_t odd_shape(StreamShape* ss, int n, int columns, int stages, int tensors) {
  ss->tpr = row_threads((n + 1) / 2, columns / 2);
  const size_t team = (size_t)stages * tensors * odd_cap(n, sizeof(T));
  const int fit = (int)(kMaxSmem / team), unit = ss->tpr < 32 ? 32 / ss->tpr : 1;
  ss->teams = std::max(unit, std::min(kOddThreads / ss->tpr, fit) / unit * unit);
  return team * ss->teams;
}

// The streamed forward, where a row fits a block and the rows are enough; false: not.
template <class T>
bool stream_fwd(const FwdArgs& a, bool shift, int* rc) {
  constexpr int VL = 16 / sizeof(T);
  // a shifted row may touch one vector more than its length has
  const int slots = (int)ceil_div(a.nm.n + (shift ? VL - 1 : 0), VL);
  int nv = 0;
  const StreamShape ss = stream_shape(slots, kFwdColumns / VL, kFwdStreamThreads, &nv);
  if (!ss.tpr || (shift && a.sms < 8)) return false;
  if (a.nm.rows < (shift ? kShiftRows : 4LL * ss.teams * a.sms)) return false;
  switch (nv) {
    case 1: *rc = launch_fwd_stream<T, 1>(a, ss, shift); break;
    case 2: *rc = launch_fwd_stream<T, 2>(a, ss, shift); break;
    case 3: *rc = launch_fwd_stream<T, 3>(a, ss, shift); break;
    case 4: *rc = launch_fwd_stream<T, 4>(a, ss, shift); break;
    case 6: *rc = launch_fwd_stream<T, 6>(a, ss, shift); break;
    case 8: *rc = launch_fwd_stream<T, 8>(a, ss, shift); break;
    default:
      if constexpr (sizeof(T) == 2)
        *rc = nv == 5 ? launch_fwd_stream<T, 5>(a, ss, shift) : launch_fwd_stream<T, 7>(a, ss, shift);
      else
        *rc = nv == 10   ? launch_fwd_stream<T, 10>(a, ss, shift)
              : nv == 12 ? launch_fwd_stream<T, 12>(a, ss, shift)
              : nv == 14 ? launch_fwd_stream<T, 14>(a, ss, shift)
                         : launch_fwd_stream<T, 16>(a, ss, shift);
  }
  return true;
}

template <class T, int VL>
int pick_fwd(const FwdArgs& a) {
  const int slots = (int)ceil_div(a.nm.n, VL == 1 ? 2 : VL);
  if (slots > kFwdThreads * 16) {
    const int grid = (int)std::min<int64_t>(a.nm.rows, 4LL * a.sms);
    prof_begin(K_NORM_FWD, a.s);
    norm_fwd_long_kernel<T><<<grid, kLongThreads, 0, a.s>>>(a.nm, (const T*)a.x, a.gamma, a.beta, (T*)a.y, a.mean,
                                                           a.rstd);
    prof_end(K_NORM_FWD, a.s);
    return cudaGetLastError() == cudaSuccess ? MOE_LORA_OK : MOE_LORA_ERR_CUDA;
  }
  int rc = 0;
  if (stream_fwd<T>(a, VL == 1, &rc)) return rc;
  // few rows want many threads
  int nv = 16;
  while (nv > 1 && (slots <= 8 * (nv / 2) || (a.nm.rows * ceil_div(slots, nv) < 512LL * a.sms &&
                                               ceil_div(slots, nv / 2) <= kFwdThreads)))
    nv /= 2;
  const int tpr = row_threads(slots, nv);
  const RowShape rs = row_shape(a.nm.rows, tpr, tpr > 32 ? 1 : a.nm.rows > 32LL * a.sms ? 128 / tpr : 32 / tpr);
  switch (nv) {
    case 1: return launch_fwd<T, VL, 1>(a, rs);
    case 2: return launch_fwd<T, VL, 2>(a, rs);
    case 4: return launch_fwd<T, VL, 4>(a, rs);
    case 8: return launch_fwd<T, VL, 8>(a, rs);
    default: return launch_fwd<T, VL, 16>(a, rs);
  }
}

template <class T>
int run_fwd(const FwdArgs& a) {
  return rows_aligned(a.nm, false, false) ? pick_fwd<T, 16 / sizeof(T)>(a) : pick_fwd<T, 1>(a);
}

// The partial rows' sum.  Its launch is prepared while the kernel before it runs; its blocks
// start when that kernel's have exited.  (Let in at that kernel's start, to wait on the SMs,
// they save 0.1 us at 128 x 577 fp32, but 256 x 4,096 bf16 takes 10.4 us instead of 8.7 and
// 1,024 x 4,096 15.1 instead of 13.6.)
int launch_wgrad(int n, int parts, const float* part, float* dgamma, float* dbeta, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)ceil_div(n, 32), 2);
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  prof_begin(K_NORM_WGRAD, s);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, norm_wgrad_kernel, n, parts, part, dgamma, dbeta);
  prof_end(K_NORM_WGRAD, s);
  return e == cudaSuccess ? MOE_LORA_OK : MOE_LORA_ERR_CUDA;
}

struct BwdArgs {
  const moe_lora_norm& nm;
  const void* x;
  Weight gamma;
  const float *mean, *rstd;
  const void *dy, *dres;
  void* dx;
  float *dgamma, *dbeta, *part;
  float2* sums;
  int sms;
  cudaStream_t s;
};

// One kernel over all rows (of one slice, or of every slice).
template <class T, BwdMode kMode, class Kernel>
int launch_bwd(const BwdArgs& a, Kernel kernel, const StreamShape& ss, int slice, size_t smem, bool shift,
               bool* parts, int* blocks) {
  const int slices = (int)ceil_div(a.nm.n, slice);
  const bool wgrad = kMode != kSums && (a.dgamma || a.dbeta);
  smem = std::max(smem, wgrad ? 2 * sizeof(float) * ss.teams * std::min(a.nm.n, slice) : 0);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[1];
  cfg.gridDim = dim3(1, slices);
  cfg.blockDim = dim3(ss.tpr * ss.teams);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = a.s;
  int most = std::max(1, std::min(a.sms, kNormParts) / slices);
  if (kMode == kCluster) {
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = at[0].val.clusterDim.z = 1;
    at[0].val.clusterDim.y = slices;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    // as many clusters as run together (fewer than blocks would: a cluster stays inside one
    // processing cluster); one more is a second wave as long as the first
    int fit = 0;
    const auto ask = [&](bool again) {
      const cudaError_t e = allow_options(reinterpret_cast<const void*>(kernel), again);
      return e == cudaSuccess ? cudaOccupancyMaxActiveClusters(&fit, kernel, &cfg) : e;
    };
    if (ask(false) != cudaSuccess) {
      (void)cudaGetLastError();
      if (ask(true) != cudaSuccess) return MOE_LORA_ERR_CUDA;
    }
    most = std::max(1, std::min(most, fit));
  }
  int grid = stream_grid(a.nm.rows, ss.teams, most, shift);
  // Few rows, one a team at most: up to sixteen blocks, a cluster, add the weight gradients
  // themselves.  The GPU takes as long as with a second launch (128 x 577 fp32 6.2 and 6.5
  // us, 32 x 4,096 bf16 7.8 and 7.7, 1,024 x 64 bf16 4.1 and 4.7), a call 2 us less of the
  // host's time (8.5 and 10.4).  With a second and third row a team the cluster is behind:
  // 192 x 577 fp32 7.7 us on the GPU against 6.8, 347 x 577 9.1 against 7.0, 96 x 4,096 bf16
  // 10.3 against 8.2.  (Calls of 347 x 577 in a row, where host and GPU are about level: 11.2
  // to 11.5 us as a cluster, 10.5 to 13.1 in two launches.)
  bool together = false;
  if (kMode == kWhole && wgrad && grid > 1) {
    int cluster = 2;
    while (cluster < 16 && cluster < grid) cluster *= 2;
    together = a.nm.rows <= (int64_t)ss.teams * cluster;
    if (together) {
      grid = cluster;
      at[0].id = cudaLaunchAttributeClusterDimension;
      at[0].val.clusterDim.x = cluster;
      at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
      cfg.attrs = at;
      cfg.numAttrs = 1;
    }
  }
  cfg.gridDim.x = grid;
  *parts = wgrad && grid > 1 && !together;
  *blocks = grid;
  float* dg = !wgrad ? nullptr : *parts ? a.part : a.dgamma;
  float* db = !wgrad ? nullptr : *parts ? a.part + a.nm.n : a.dbeta;
  prof_begin(K_NORM_BWD, a.s);
  const cudaError_t e = launch_allowed(
      cfg, together && grid > 8, kernel, a.nm, ss, static_cast<const T*>(a.x), a.gamma, a.mean, a.rstd,
      static_cast<const T*>(a.dy), static_cast<const T*>(a.dres), static_cast<T*>(a.dx), dg, db,
      *parts ? (int64_t)2 * a.nm.n : 0, a.sums, slice);
  prof_end(K_NORM_BWD, a.s);
  return e == cudaSuccess ? MOE_LORA_OK : MOE_LORA_ERR_CUDA;
}

template <class T, int NV, RowFit kFit>
int launch_bwd_stream(const BwdArgs& a, const StreamShape& ss, int slice, bool* parts, int* blocks) {
  constexpr int kS = bwd_stages<T>();
  const size_t smem = ring_bytes<kS, 3 * NV>(ss.tpr * ss.teams);
  const int64_t slices = ceil_div(a.nm.n, slice);
#define RUN(MODE)                                                                                              \
  launch_bwd<T, MODE>(a, norm_bwd_stream_kernel<T, NV, kS, MODE, kFit>, ss, slice, smem, kFit == kShift, parts, blocks)
  if (slices == 1) return RUN(kWhole);
  if (slices <= kBwdCluster) return RUN(kCluster);
  const int rc = RUN(kSums);
  return rc ? rc : RUN(kApply);
#undef RUN
}

template <class T, int kS>
int launch_bwd_odd(const BwdArgs& a, bool* parts, int* blocks) {
  constexpr int kNP = kBwdColumns / 2;
  StreamShape ss;
  const size_t smem = odd_shape<T>(&ss, std::min(a.nm.n, kBwdSlice), kBwdColumns, kS, a.dres ? 3 : 2);
#define RUN(MODE) \
  launch_bwd<T, MODE>(a, norm_bwd_odd_kernel<T, kNP, kS, MODE>, ss, kBwdSlice, smem, false, parts, blocks)
  if (a.nm.n <= kBwdSlice) return RUN(kWhole);
  const int rc = RUN(kSums);
  return rc ? rc : RUN(kApply);
#undef RUN
}

template <class T, RowFit kFit>
int pick_bwd_stream(const BwdArgs& a, bool* parts, int* blocks) {
  constexpr int VL = 16 / sizeof(T), kNV = kBwdColumns / VL;
  // equal slices of whole vectors; a shifted one may touch one vector more than it has
  const int64_t room = kBwdSlice - (kFit == kShift ? VL : 0), slices = ceil_div(a.nm.n, room);
  const int slice = (int)ceil_div(ceil_div(a.nm.n, slices), VL) * VL;
  const int slots = (int)ceil_div(std::min(slice, a.nm.n) + (kFit == kShift ? VL - 1 : 0), VL);
  int nv = 0;
  const StreamShape ss = stream_shape(slots, kNV, kBwdStreamThreads, &nv);
  if (nv == 1) return launch_bwd_stream<T, 1, kFit>(a, ss, slice, parts, blocks);
  if constexpr (kNV == 4) {
    if (nv == 3) return launch_bwd_stream<T, 3, kFit>(a, ss, slice, parts, blocks);
    if (nv == 4) return launch_bwd_stream<T, 4, kFit>(a, ss, slice, parts, blocks);
  }
  return launch_bwd_stream<T, 2, kFit>(a, ss, slice, parts, blocks);
}

// The teams of shifted rows step by whole multiples of eight blocks, which there must be
// (of clusters, where the rows are wide).
bool shifted_rows_fit(const BwdArgs& a) {
  return std::min(a.sms, kNormParts) / ceil_div(a.nm.n, kBwdSlice - 8) >= 8;
}

template <class T>
int run_bwd(const BwdArgs& a) {
  const int n = a.nm.n;
  constexpr int64_t kMask = 16 / sizeof(T) - 1;
  bool parts = false;
  int blocks = 0, rc;
  // all rows shifted alike (an output shifted otherwise, stored by single elements, makes this
  // slower than the staged kernel: 1.7 against 2.8 TB/s at 16,384 x 2,049 bf16)
  const int64_t differ = (a.nm.ldx ^ a.nm.ldy) | (a.nm.ldx ^ a.nm.lddx) | (a.dres ? a.nm.ldx ^ a.nm.lddres : 0);
  const bool alike = (differ & kMask) == 0;
  if (rows_aligned(a.nm, true, a.dres != nullptr))
    rc = pick_bwd_stream<T, kAligned>(a, &parts, &blocks);
  else if (alike && shifted_rows_fit(a))
    rc = pick_bwd_stream<T, kShift>(a, &parts, &blocks);
  else  // three stages of the widest slice of fp32 rows are more than shared memory holds
    rc = sizeof(T) == 4 && n > 4096 ? launch_bwd_odd<T, 2>(a, &parts, &blocks)
                                    : launch_bwd_odd<T, 3>(a, &parts, &blocks);
  return rc || !parts ? rc : launch_wgrad(n, blocks, a.part, a.dgamma, a.dbeta, a.s);
}

// CALL<T>(args) for the element type of nm.
#define NORM_DISPATCH(CALL, ...)                                  \
  (nm.dtype == MOE_LORA_F32    ? CALL<float>(__VA_ARGS__)         \
   : nm.dtype == MOE_LORA_BF16 ? CALL<__nv_bfloat16>(__VA_ARGS__) \
                               : CALL<__half>(__VA_ARGS__))

}  // namespace

}  // namespace moelora

using namespace moelora;

extern "C" {

int moe_lora_layernorm_forward(const moe_lora_norm* in, const void* x, const void* gamma, const void* beta, void* y,
                               float* mean, float* rstd, void* stream) {
  moe_lora_norm nm;
  int rc = check_norm(in, &nm);
  if (rc) return rc;
  if (!(nm.eps > 0.0f)) return MOE_LORA_ERR_DIMS;
  if ((rc = check_opt(gamma)) || (rc = check_opt(beta)) || (rc = check_opt(mean)) || (rc = check_opt(rstd))) return rc;
  if (!mean != !rstd) return MOE_LORA_ERR_NULL;
  if (nm.rows == 0) return MOE_LORA_OK;
  if ((rc = check_ptr(x)) || (rc = check_ptr(y))) return rc;
  int sms;
  if ((rc = device_sms(&sms))) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const FwdArgs a{nm, x, {gamma, nm.wdtype}, {beta, nm.wdtype}, y, mean, rstd, sms, s};
  return NORM_DISPATCH(run_fwd, a);
}

size_t moe_lora_layernorm_scratch_bytes(const moe_lora_norm* in) {
  moe_lora_norm nm;
  return check_norm(in, &nm) ? 0 : part_bytes(nm) + sums_bytes(nm);
}

int moe_lora_layernorm_backward(const moe_lora_norm* in, const void* x, const void* gamma, const float* mean,
                                const float* rstd, const void* dy, const void* dres, void* dx, float* dgamma,
                                float* dbeta, void* scratch, size_t scratch_bytes, void* stream) {
  moe_lora_norm nm;
  int rc = check_norm(in, &nm);
  if (rc) return rc;
  if ((rc = check_opt(gamma)) || (rc = check_opt(dres)) || (rc = check_opt(dgamma)) || (rc = check_opt(dbeta)))
    return rc;
  const bool wgrad = dgamma || dbeta;
  if (wgrad || (nm.n > kBwdSlice && nm.rows > 0)) {
    if ((rc = check_ptr(scratch))) return rc;
    if (scratch_bytes < moe_lora_layernorm_scratch_bytes(in)) return MOE_LORA_ERR_WORKSPACE;
  }
  int sms;
  if (nm.rows == 0) {
    if (!wgrad) return MOE_LORA_OK;
    if ((rc = device_sms(&sms))) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    for (float* p : {dgamma, dbeta})
      if (p && cudaMemsetAsync(p, 0, sizeof(float) * nm.n, s) != cudaSuccess) return MOE_LORA_ERR_CUDA;
    return MOE_LORA_OK;
  }
  if ((rc = check_ptr(x)) || (rc = check_ptr(mean)) || (rc = check_ptr(rstd)) || (rc = check_ptr(dy)) ||
      (rc = check_ptr(dx)))
    return rc;
  if ((rc = device_sms(&sms))) return rc;
  const BwdArgs a{nm,     x,     {gamma, nm.wdtype}, mean, rstd, dy, dres, dx, dgamma, dbeta,
                  static_cast<float*>(scratch), reinterpret_cast<float2*>(static_cast<char*>(scratch) + part_bytes(nm)),
                  sms,    static_cast<cudaStream_t>(stream)};
  return NORM_DISPATCH(run_bwd, a);
}

}  // extern "C"
