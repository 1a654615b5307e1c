// Muon: momentum, an update orthogonalised by Newton-Schulz products, and the weights
// (definitions in include/moe_lora.h).
//
// Every matrix has a short side s <= 128 and a long side L.  The steps X <- Q(X X^T) X, with
// Q(G) = a + b G + c G^2, need X itself only where G = X X^T is formed: G and the steps'
// polynomials are s x s.  A few steps therefore run on the s x s matrices alone,
//     T = G G,  Q = a + b G + c T,  P <- Q P,  G <- Q (Q G),
// and X is multiplied by P once.  What limits their number is that G holds squares: rounding
// G to fp32 relative to its largest value leaves an error that the steps amplify by a^2 each
// in the directions that start small.  Five steps on one G lose those (measured on the host:
// 6e-3 of the update where most singular values are 1e-3 of the largest); two, then a fresh G
// from the X of that point, then three stay within 5e-5, close to what fp32 products through
// all five steps give (1e-5).  Hence five launches:
//   gram    m <- momentum; partial G of the tensor (products of the update with itself)
//   poly    the first steps on G; P
//   apply   X <- P X, kept in the scratch; partial G of that
//   poly    the other steps; P
//   update  O = P X; the weights
//
// All products run on the tensor cores (tcgen05) with operands in parts whose sum is the
// fp32 value to 2^-22 or better.  gram: three bf16 parts h + m + l, since the update's size is
// not known yet and bf16 has fp32's range; G = hh + mm + h(m + l) + (m + l)h, the last term
// being the transpose of the third.  Afterwards sizes are known (singular values below 1.5)
// and two fp16 parts of scaled values do with three products.
//
// A tile is 128 rows of the short sides: 128 / s matrices of a tensor, one below the other,
// whose products with each other are set to 0 wherever a tile of G is read.  A chunk is 64
// places of the long side.  Blocks share all chunks evenly; what a block has of one tile is a
// stretch, and leaves one partial G.
//
// Measured on one GB300, 203 M elements of rank 128 (bf16 weights, fp32 masters and gradients): 1,722 us,
// of which gram 455 (12 bytes an element, 5.3 TB/s), apply 540 (12 bytes, 4.5), update 475 (14 bytes,
// 6.0) and the two polys 248 together.  The three that stream are bound by the chain of a chunk (loads,
// operand stores, a barrier, products; in apply twice), which two blocks an SM cover in part: registers
// and tensor memory take no third.  38.6 M elements of rank 8 in bf16: 308 us.
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

constexpr int kTile = 128, kChunk = 64, kThreads = 256;
constexpr int kQuads = kTile * kChunk / 4 / kThreads;  // four neighbouring elements, of a thread's share of a chunk
constexpr int kMaxTensors = 128;                       // of a launch; their table travels in its parameters
constexpr int kMaxSteps = 5, kFirstSteps = 2;
constexpr int kPart = kTile * kChunk * 2;              // bytes of a part of a chunk
constexpr int kTileBytes = kTile * kTile * 2;          // of a part of a square tile
constexpr int kImage = 2 * kPart;                      // X of a chunk in the scratch: both parts as they lie in shared memory
constexpr int kPoly = 2 * kTileBytes;                  // P of a tile, the same
// A matrix's norm from its square.  One of at most 2^-60 counts as 0: the parts of its squares run out of
// fp32's range, and so does (1 / norm)^2 kGScale.
__device__ __forceinline__ float counted_norm(float n2) {
  const float norm = sqrtf(n2);
  return norm > 0x1p-60f ? norm : 0.f;
}
// Powers of two that bring values into the middle of fp16's range.
constexpr float kXScale = 1024.f, kGScale = 256.f, kQScale = 64.f;
// X's where the norm is far below eps and with it X = u / (norm + eps): 2^k kXScale, k for singular values
// of at most 1 / 4, so that the first steps (a factor of 64 at most) stay in the range; kXScale from about
// 1 / 8 on.  `factor` is the matrix's (see MuonTable): 2^9 to 2^10 of it make the norm of X.
__device__ __forceinline__ int x_shift(float factor) {
  return factor > 0.f ? max(0, 127 - 13 - (int)(__float_as_uint(factor) >> 23)) : 0;
}
__device__ __forceinline__ float two_to(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }
__device__ __forceinline__ float x_scale(float factor) { return kXScale * two_to(x_shift(factor)); }
__device__ __forceinline__ float x_unit(float factor) { return 1.f / kXScale * two_to(-x_shift(factor)); }

struct MuonTensor {
  void* p;
  float* master;
  const void* g;
  float* m;
  int64_t batch;                 // matrices
  int32_t tile0, chunk0;         // first tile and chunk of the launch
  int32_t s, L, tall;            // tall: [L, s] in memory
  int32_t per, chunks;           // matrices, and chunks, of a tile
  int32_t p_dtype, g_dtype;
  float decay, step;             // 1 - lr * weight_decay, lr * scale
};
struct MuonTable {
  int n, blocks, chunks;         // tensors; blocks, which share the chunks evenly
  float mu, nu, eps, a, b, c;    // nu = 1 - mu
  int nesterov;
  const float* gs;
  int* err;
  float *gram, *norm;            // [tiles + blocks][128][128], [tiles][2][128]: scale and factor of a row's matrix
  uint8_t *poly, *x;             // [tiles][kPoly], [chunks][kImage]: X times x_scale
  MuonTensor t[kMaxTensors];
};
static_assert(sizeof(MuonTable) <= 32764, "kernel parameter limit");

// Block b's chunks begin at b * chunks / blocks: all blocks have the same number, give or take
// one, wherever tiles begin.
__device__ __forceinline__ int first_chunk(const MuonTable& tab, int b) { return (int)((int64_t)b * tab.chunks / tab.blocks); }
// Where the sums of a stretch of a tile that begins at chunk x lie: stretches begin with tiles and
// with blocks, so that the tile and the blocks begun by then number them without gaps within a tile.
__device__ __forceinline__ int64_t stretch_slot(const MuonTable& tab, int tile, int x) {
  return tile + ((int64_t)(x + 1) * tab.blocks - 1) / tab.chunks;
}
struct Place {  // a stretch of one tile's chunks
  const MuonTensor* t;
  int tile, x;          // of the launch; its first chunk, whose image in the scratch has that place
  int64_t first;        // first matrix
  int rows;             // short sides in use
  int c0, c1;           // chunks of the tile
};
// The stretch from chunk x on that ends with its tile or at chunk `end`.
__device__ __forceinline__ Place place_of(const MuonTable& tab, int x, int end) {
  int lo = 0, hi = tab.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (x >= tab.t[mid].chunk0)
      lo = mid;
    else
      hi = mid - 1;
  }
  const MuonTensor& t = tab.t[lo];
  const int tile = (x - t.chunk0) / t.chunks;
  Place p;
  p.t = &t;
  p.tile = t.tile0 + tile;
  p.x = x;
  p.first = (int64_t)tile * t.per;
  p.rows = (int)min((int64_t)t.per, t.batch - p.first) * t.s;
  p.c0 = x - t.chunk0 - tile * t.chunks;
  p.c1 = min(t.chunks, p.c0 + (end - x));
  return p;
}

// ------------------------------------------------------------------ a thread's share of a chunk
// A thread's quads of a chunk, four neighbouring elements in memory each.  Of [s, L]: along the
// long side, 16 to a row.  Of tall matrices [L, s]: along the short side; a warp's 32 are one run of
// memory where s is a power of two from 8 on (128 / s long places of one matrix), and otherwise a long
// place of all matrices of the tile.  (That for s = 8 too, in runs of 16 or 32 bytes: 38.6 M elements
// 488 us instead of 437.)  Divisions are done once: quad i is i % 4 short and i / 4 long steps from quad 0.
struct Walk {
  int64_t at, hop, hop4, chunk;  // element of quad 0 in chunk 0 of the tile; the steps, and to the next chunk
  int row, col;                  // of quad 0: short side within the tile, long side within the chunk
  int hop_row, hop_col, hop_row4, hop_col4;
  uint32_t place, hop_place;     // bytes in a part of an operand tile, where all steps are the same
  uint32_t whole;                // quads of a whole chunk that lie inside, a bit each
  int rows, L;
  // Operand tiles have rows of 128 bytes whose 16-byte units are exchanged by row (unit ^ row % 8).
  // A chunk of [s, L]: 128 rows of 64 long places.  Of [L, s]: two halves of 64 short places, a
  // row per long place.  No step changes row % 8 or the unit.
  __device__ __forceinline__ Walk(const MuonTensor& t, int64_t first, int rows_) : rows(rows_), L(t.L) {
    constexpr int kWarps = kThreads / 32;
    const int64_t base = first * t.s * t.L;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    hop_row = hop_col = hop_row4 = 0;
    int line, k;
    if (!t.tall) {
      row = threadIdx.x >> 4;
      col = (threadIdx.x & 15) * 4;
      hop_row = kThreads / 16;
      hop_row4 = 4 * hop_row;
      hop_col4 = 0;
      hop_place = hop_row * 128;
      at = base + (int64_t)row * L + col;
      line = row, k = col;
    } else {
      int j, r;  // matrix, and place on its short side
      if (t.s >= 8 && (t.s & (t.s - 1)) == 0) {
        const int places = kTile / t.s, mats = min(places, kWarps);  // of a run; matrices that the warps take side by side
        r = lane * 4 % t.s;
        j = warp % mats;
        col = lane * 4 / t.s + warp / mats * places;
        hop_col = kWarps / mats * places;
      } else {
        j = lane * 4 / t.s;
        r = lane * 4 - j * t.s;
        col = warp;
        hop_col = kWarps;
      }
      hop_col4 = 4 * hop_col;
      if (hop_col4 == kChunk) {  // s = 8: four steps go through the chunk, the other four take the other half
        hop_col4 = 0;
        hop_row4 = kTile / 2;
      }
      hop_place = hop_col * 128;
      row = j * t.s + r;
      at = base + ((int64_t)j * L + col) * t.s + r;
      line = col, k = row % 64;
    }
    place = line * 128 + ((((k >> 3) ^ (line & 7)) << 4) | ((k & 4) << 1)) + (t.tall ? row / 64 * (kPart / 2) : 0);
    hop = (int64_t)hop_row * L + (int64_t)hop_col * t.s;
    hop4 = (int64_t)hop_row4 * L + (int64_t)hop_col4 * t.s;
    chunk = t.tall ? (int64_t)kChunk * t.s : kChunk;
    whole = 0;
#pragma unroll
    for (int i = 0; i < kQuads; ++i) whole |= (uint32_t)(row_of(i) < rows) << i;
  }
  __device__ __forceinline__ int64_t element(int i) const { return (i & 3) * hop + (i >> 2) * hop4; }  // from quad 0
  __device__ __forceinline__ int row_of(int i) const { return row + (i & 3) * hop_row + (i >> 2) * hop_row4; }
  __device__ __forceinline__ int col_of(int i) const { return col + (i & 3) * hop_col + (i >> 2) * hop_col4; }
  __device__ __forceinline__ uint32_t operand(int i) const { return place + i * hop_place; }
  // The same of chunk c, where quads lie inside or outside as a whole.
  __device__ __forceinline__ uint32_t inside(int c) const {
    const int l = L - c * kChunk;
    if (l >= kChunk) return whole;
    uint32_t in = 0;
#pragma unroll 1
    for (int i = 0; i < kQuads; ++i) in |= (uint32_t)(col_of(i) < l) << i;
    return in & whole;
  }
};
// Whether quads lie inside one matrix's run of memory, and on 16 bytes (8 of 16-bit types).
__device__ __forceinline__ bool quads_aligned(const MuonTensor& t) { return t.tall ? t.s % 4 == 0 : t.L % 4 == 0; }
// Element e of quad i elsewhere: its offset, or -1 outside.
__device__ __forceinline__ int64_t element_at(const MuonTensor& t, const Walk& w, int64_t first, int c, int i, int e) {
  const int row = w.row_of(i) + (t.tall ? e : 0), l = c * kChunk + w.col_of(i) + (t.tall ? 0 : e);
  if (row >= w.rows || l >= t.L) return -1;
  const int j = row / t.s, r = row - j * t.s;
  return (first + j) * t.s * t.L + (t.tall ? (int64_t)l * t.s + r : (int64_t)r * t.L + l);
}

struct Four {
  float2 a, b;
};
template <int kType>
__device__ __forceinline__ uint4 ld_quad(const void* p, int64_t i) {
  if (kType == MOE_LORA_F32) return *reinterpret_cast<const uint4*>(static_cast<const float*>(p) + i);
  const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i);
  return make_uint4(u.x, u.y, 0, 0);
}
template <int kType>
__device__ __forceinline__ Four widen(const uint4& u) {
  if constexpr (kType == MOE_LORA_F32) return Four{Two<float>::get(&u.x), Two<float>::get(&u.z)};
  using E = typename std::conditional<kType == MOE_LORA_F16, __half, __nv_bfloat16>::type;
  return Four{Two<E>::get(&u.x), Two<E>::get(&u.y)};
}
template <int kType>
__device__ __forceinline__ void st_quad(void* p, int64_t i, const Four& v) {
  if constexpr (kType == MOE_LORA_F32) {
    *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = make_float4(v.a.x, v.a.y, v.b.x, v.b.y);
  } else {
    using E = typename std::conditional<kType == MOE_LORA_F16, __half, __nv_bfloat16>::type;
    uint2 u;
    Two<E>::put(&u.x, v.a);
    Two<E>::put(&u.y, v.b);
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + i) = u;
  }
}
template <int kType>
__device__ __forceinline__ float ld_one(const void* p, int64_t i) {
  using E = typename std::conditional<kType == MOE_LORA_F32, float, typename std::conditional<kType == MOE_LORA_F16, __half, __nv_bfloat16>::type>::type;
  return to_f32(static_cast<const E*>(p)[i]);
}
template <int kType>
__device__ __forceinline__ void st_one(void* p, int64_t i, float v) {
  using E = typename std::conditional<kType == MOE_LORA_F32, float, typename std::conditional<kType == MOE_LORA_F16, __half, __nv_bfloat16>::type>::type;
  static_cast<E*>(p)[i] = from_f32<E>(v);
}

// A pointer in registers: the table's own lie in the constant bank, and reading one again for every
// quad held the warps up.
template <class P>
__device__ __forceinline__ P* in_register(P* p) {
  asm volatile("" : "+l"(p));
  return p;
}
// The gradient and momentum of a thread's quads of a chunk, on their way: the next chunk's take a
// quad's place as soon as it is used.
template <int kType>
struct Loads {
  const void* gp;
  const float* mp;
  uint4 g[kQuads], m[kQuads];
  __device__ __forceinline__ explicit Loads(const MuonTensor& t) : gp(in_register(t.g)), mp(in_register(t.m)) {}
  __device__ __forceinline__ void quad(int64_t at, int i, bool in, bool with_g) {
    g[i] = m[i] = make_uint4(0, 0, 0, 0);
    if (in) {
      if (with_g) g[i] = ld_quad<kType>(gp, at);
      m[i] = ld_quad<MOE_LORA_F32>(mp, at);
    }
  }
  __device__ __forceinline__ void chunk(const Walk& w, int c, bool with_g) {
    const uint32_t in = w.inside(c);
    const int64_t at = w.at + c * w.chunk;
#pragma unroll
    for (int i = 0; i < kQuads; ++i) quad(at + w.element(i), i, in >> i & 1, with_g);
  }
};
// Four elements of a quad that does not lie on 16 bytes or within one matrix.
template <int kType>
__device__ __forceinline__ Four ld_loose(const void* p, const MuonTensor& t, const Walk& w, int64_t first, int c, int i) {
  float f[4] = {};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int64_t at = element_at(t, w, first, c, i, e);
    if (at >= 0) f[e] = ld_one<kType>(p, at);
  }
  return Four{make_float2(f[0], f[1]), make_float2(f[2], f[3])};
}
template <int kType>
__device__ __forceinline__ void st_loose(void* p, const MuonTensor& t, const Walk& w, int64_t first, int c, int i, const Four& v) {
  const float f[4] = {v.a.x, v.a.y, v.b.x, v.b.y};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int64_t at = element_at(t, w, first, c, i, e);
    if (at >= 0) st_one<kType>(p, at, f[e]);
  }
}
// mu m + nu g
__device__ __forceinline__ Four mix(float mu, const Four& m, float nu, const Four& g) {
  return Four{fma2(both(mu), m.a, mul2(both(nu), g.a)), fma2(both(mu), m.b, mul2(both(nu), g.b))};
}

// ------------------------------------------------------------------ operands in shared memory
__device__ __forceinline__ uint32_t hf2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return reinterpret_cast<const uint32_t&>(h);
}
// Two values to a bf16 pair; `v` keeps what the rounding left.
__device__ __forceinline__ uint32_t take_bf16(float2& v) {
  const uint32_t h = pack_bf16x2(v.x, v.y);
  v = fma2(make_float2(bf16_lo(h), bf16_hi(h)), both(-1.f), v);
  return h;
}
// ... to their two fp16 parts.
__device__ __forceinline__ void fp16_parts(float2 v, uint32_t& hi, uint32_t& lo) {
  hi = hf2(v.x, v.y);
  v = fma2(__half22float2(reinterpret_cast<const __half2&>(hi)), both(-1.f), v);
  lo = hf2(v.x, v.y);
}

// Instruction descriptor of kind::f16 with fp32 accumulation: fp16 operands (type code 0)
// instead of bf16 ones (1).
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, bool a_mn, bool b_mn) {
  return idesc_bf16_f32(M, N, a_mn, b_mn) & ~((1u << 7) | (1u << 10));
}

__device__ __forceinline__ void bulk_store(void* dst, const void* src_smem, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(src_smem)), "r"(bytes) : "memory");
}

__device__ __forceinline__ uint8_t* aligned_smem(uint8_t* p) { return p + ((1024 - (smem_u32(p) & 1023)) & 1023); }
// Tensor memory of a block, opened and closed by all its threads.
__device__ __forceinline__ uint32_t tmem_open(uint32_t* slot, int columns) {
  if (threadIdx.x < 32) {
    tmem_alloc(slot, columns);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  return *slot;
}
__device__ __forceinline__ void tmem_close(uint32_t base, int columns) {
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (threadIdx.x < 32) tmem_dealloc(base, columns);
}
// Every thread's wait for products; one that did not end in time is noted, and the thread's later
// waits are left out, so that the block ends with its barriers in step.
struct Waits {
  int* err;
  bool late = false;
  __device__ __forceinline__ void operator()(uint64_t* bar, uint32_t parity) {
    if (!late) late = !mbar_wait(bar, parity, err);
    tc_fence_after();
  }
};
// This thread's 32 columns from `col` on of its row: warp w has rows 32 (w % 4) + lane.
__device__ __forceinline__ void tmem_row32(uint32_t base, int col, float (&v)[32]) {
  const uint32_t lanes = ((threadIdx.x >> 5) & 3) * 32;
  tmem_ld32(base + (lanes << 16) + col, v);
}
__device__ __forceinline__ int my_row() { return ((threadIdx.x >> 5) & 3) * 32 + (threadIdx.x & 31); }
__device__ __forceinline__ int my_part() { return threadIdx.x >> 7; }  // of the columns

// Each launch starts while the one before it runs out, and waits for it before it touches what
// that one, or any before, has written.
__device__ __forceinline__ void launch_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_last() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// f(integral constant of the tensor's type, constant of whether its quads are aligned): a loop of its
// own for each, small enough for the instruction caches
template <class F>
__device__ __forceinline__ void with_kind(int dtype, bool aligned, F f) {
  const auto typed = [&](auto type) {
    if (aligned)
      f(type, std::true_type{});
    else
      f(type, std::false_type{});
  };
  if (dtype == MOE_LORA_F32)
    typed(std::integral_constant<int, MOE_LORA_F32>{});
  else if (dtype == MOE_LORA_BF16)
    typed(std::integral_constant<int, MOE_LORA_BF16>{});
  else
    typed(std::integral_constant<int, MOE_LORA_F16>{});
}

// ------------------------------------------------------------------ gram
constexpr int kGramStages = 2, kGramSmem = kGramStages * 3 * kPart + 1024;
constexpr int kGramCols = 256;

__global__ void __launch_bounds__(kThreads, 2) muon_gram_kernel(const __grid_constant__ MuonTable tab) {
  extern __shared__ uint8_t muon_smem[];
  __shared__ uint64_t done[kGramStages];
  __shared__ uint32_t slot;
  uint8_t* sm = aligned_smem(muon_smem);
  launch_next();
  if (threadIdx.x == 0) {
    for (int i = 0; i < kGramStages; ++i) mbar_init(&done[i], 1);
    fence_mbar_init();
  }
  const uint32_t acc = tmem_open(&slot, kGramCols);
  Waits wait{tab.err};
  int used = 0;  // chunks so far
  const float nu = tab.nu * (tab.gs ? *tab.gs : 1.f);
  const int end = first_chunk(tab, blockIdx.x + 1);
  for (int x = first_chunk(tab, blockIdx.x); x < end;) {
    const Place pl = place_of(tab, x, end);
    const MuonTensor& t = *pl.t;
    const bool tall = t.tall;
    const Walk w(t, pl.first, pl.rows);
    with_kind(t.g_dtype, quads_aligned(t), [&](auto type, auto quads) {
      constexpr int kType = decltype(type)::value;
      constexpr bool kAligned = decltype(quads)::value;
      Loads<kType> ld(t);
      float* const mp = in_register(t.m);
      if (kAligned) ld.chunk(w, pl.c0, true);
      for (int c = pl.c0; c < pl.c1; ++c, ++used) {
        const int st = used % kGramStages;
        uint8_t* part = sm + st * 3 * kPart;
        if (used >= kGramStages) wait(&done[st], (used / kGramStages - 1) & 1);
        const auto put = [&](int i, const Four& g, const Four& m) {
          Four u = tab.nesterov ? mix(tab.mu, m, nu, g) : m;
          uint8_t* to = part + w.operand(i);
#pragma unroll
          for (int q = 0; q < 3; ++q) {
            const uint32_t a = take_bf16(u.a), b = take_bf16(u.b);
            *reinterpret_cast<uint2*>(to + q * kPart) = make_uint2(a, b);
          }
        };
        if constexpr (kAligned) {
          const uint32_t in = w.inside(c), next = c + 1 < pl.c1 ? w.inside(c + 1) : 0;
          const int64_t at = w.at + c * w.chunk;
#pragma unroll
          for (int i = 0; i < kQuads; ++i) {
            const Four g = widen<kType>(ld.g[i]), m = mix(tab.mu, widen<MOE_LORA_F32>(ld.m[i]), nu, g);
            ld.quad(at + w.chunk + w.element(i), i, next >> i & 1, true);
            if (in >> i & 1) st_quad<MOE_LORA_F32>(mp, at + w.element(i), m);
            put(i, g, m);
          }
        } else {
#pragma unroll 1
          for (int i = 0; i < kQuads; ++i) {
            const Four g = ld_loose<kType>(ld.gp, t, w, pl.first, c, i), m = mix(tab.mu, ld_loose<MOE_LORA_F32>(mp, t, w, pl.first, c, i), nu, g);
            st_loose<MOE_LORA_F32>(mp, t, w, pl.first, c, i, m);
            put(i, g, m);
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncthreads();
        if (threadIdx.x == 0) {
          tc_fence_after();
          const uint32_t h = smem_u32(part), m = h + kPart, l = m + kPart;
          const uint32_t id = idesc_bf16_f32(kTile, kTile, tall, tall);
          const uint32_t step = tall ? 2048 : 32, lbo = tall ? kPart / 2 : 16;
#pragma unroll
          for (int kk = 0; kk < kChunk / 16; ++kk) {
            const uint64_t dh = sw128_desc(h + kk * step, lbo, 1024), dm = sw128_desc(m + kk * step, lbo, 1024),
                           dl = sw128_desc(l + kk * step, lbo, 1024);
            const uint32_t more = c > pl.c0 || kk > 0;
            mma_bf16(acc, dh, dh, id, more);
            mma_bf16(acc, dm, dm, id, 1);
            mma_bf16(acc + kTile, dh, dm, id, more);
            mma_bf16(acc + kTile, dh, dl, id, 1);
          }
          mma_commit(&done[st]);
        }
      }
    });
    wait(&done[(used - 1) % kGramStages], ((used - 1) / kGramStages) & 1);
    // (hh + mm) / 2 + h(m + l): this and its transpose are added where it is read, so that its rows may
    // be stored as columns, a warp's side by side
    float* out = tab.gram + stretch_slot(tab, pl.tile, x) * kTile * kTile + my_row();
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int col = my_part() * 64 + b * 32;
      float v[32], y[32];
      tmem_row32(acc, col, v);
      tmem_row32(acc + kTile, col, y);
#pragma unroll
      for (int i = 0; i < 32; ++i) out[(col + i) * kTile] = 0.5f * v[i] + y[i];
    }
    x += pl.c1 - pl.c0;
  }
  tmem_close(acc, kGramCols);
}

// ------------------------------------------------------------------ poly
// A block per tile, a thread per row and quarter of the columns.  The square matrices pass
// through shared memory as operands (fp16 parts of scaled values, zero outside the matrices'
// own blocks); G stays in tensor memory beside the products.  A product is a chain of
// latencies (operands written, 24 instructions on the tensor cores, 32 columns read back), of
// which five or eight follow each other.
constexpr int kPolyThreads = 512, kPolySmem = 3 * kPoly + 1024, kPolyCols = 512;

// Writes this thread's 32 columns as fp16 parts of a square tile: two halves of 64 columns, then the
// lower parts.
__device__ __forceinline__ void put_row32(uint8_t* tile, const float (&v)[32]) {
  const int r = my_row(), q = my_part();
  uint8_t* at = tile + (q >> 1) * kPart + r * 128;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) fp16_parts(make_float2(v[8 * u + 2 * i], v[8 * u + 2 * i + 1]), hi[i], lo[i]);
    const int sw = (((q & 1) * 4 + u) ^ (r & 7)) << 4;
    *reinterpret_cast<uint4*>(at + sw) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(at + kTileBytes + sw) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
}
// D = A B^T of square tiles (both fp16 parts; the product of the lower parts is below fp32's
// rounding).  The tiles are zero outside blocks of `width` (16, 32, 64 or 128) rows and columns: a step
// along 16 columns of both has to fill its own block's columns of D alone, and nobody reads the others.
__device__ __forceinline__ void square_product(uint32_t d, uint32_t a, uint32_t b, int width) {
  const uint32_t id = idesc_f16_f32(kTile, width, false, false);
#pragma unroll 1
  for (int p = 0; p < 3; ++p) {
    const uint32_t pa = a + (p == 2 ? kTileBytes : 0), pb = b + (p == 1 ? kTileBytes : 0);
#pragma unroll
    for (int kk = 0; kk < kTile / 16; ++kk) {
      const uint32_t at = kk / 4 * kPart + kk % 4 * 32;
      const int n0 = kk * 16 & ~(width - 1);  // the block's first row of B, column of D
      mma_bf16(d + n0, sw128_desc(pa + at, 16, 1024), sw128_desc(pb + at + n0 * 128, 16, 1024), id, p > 0 || kk * 16 > n0);
    }
  }
}
__device__ __forceinline__ void tmem_put_row32(uint32_t base, int col, const float (&v)[32]) {
  const uint32_t at = base + ((((threadIdx.x >> 5) & 3) * 32) << 16) + col;
#pragma unroll
  for (int i = 0; i < 32; i += 4)
    tmem_st4(at + i, __float_as_uint(v[i]), __float_as_uint(v[i + 1]), __float_as_uint(v[i + 2]), __float_as_uint(v[i + 3]));
  tmem_wait_st();
}

// `first`: G is of the update itself, whose norm is taken here.  Otherwise G is of X in the
// scratch, times x_scale^2.  Blocks work through tiles one after the other; the sums of the next are on
// their way while the last product of one runs.  Where all matrices of a tile have s = 64 or less, most of
// a square tile is 0: only warps whose rows and columns meet a matrix work on it.
__global__ void __launch_bounds__(kPolyThreads, 1) muon_poly_kernel(const __grid_constant__ MuonTable tab, int tiles, int steps, bool first) {
  constexpr int kEach = kTile * kTile / kPolyThreads;
  extern __shared__ uint8_t muon_smem[];
  __shared__ uint64_t done[2];
  __shared__ uint32_t slot;
  __shared__ float diag[kTile];
  uint8_t* sm = aligned_smem(muon_smem);
  uint8_t *qt = sm, *gt = sm + kPoly, *pt = sm + 2 * kPoly;
  const int row = my_row(), col = my_part() * 32;
  if (threadIdx.x == 0) {
    mbar_init(&done[0], 1);
    mbar_init(&done[1], 1);
    fence_mbar_init();
  }
  launch_next();
  const uint32_t tmem = tmem_open(&slot, kPolyCols);
  const uint32_t g_at = tmem, x_at = tmem + kTile, p_at = tmem + 2 * kTile;  // G, another product, P
  Waits wait{tab.err};
  uint32_t phase[2] = {0, 0};
  const uint32_t qa = smem_u32(qt), ga = smem_u32(gt), pa = smem_u32(pt);
  const float ka = tab.a * kQScale, kb = tab.b * (kQScale / kGScale), kc = tab.c * (kQScale / (kGScale * kGScale));
  const auto tensor_of = [&](int tile) {
    int ti = 0;
    while (ti + 1 < tab.n && tile >= tab.t[ti + 1].tile0) ++ti;
    return ti;
  };
  // This thread's share of the sums of a tile's stretches, in order, and the factor of its row's matrix.
  float sum[kEach], factor = 0.f;
  const auto load_sums = [&](int tile) {
    const MuonTensor& t = tab.t[tensor_of(tile)];
    const int x = t.chunk0 + (tile - t.tile0) * t.chunks;
    const int64_t s0 = stretch_slot(tab, tile, x);
    const int stretches = (int)(stretch_slot(tab, tile, x + t.chunks - 1) - s0) + 1;
    const float* in = tab.gram + s0 * kTile * kTile + threadIdx.x;
    if (!first) factor = tab.norm[(int64_t)tile * 2 * kTile + kTile + row];
#pragma unroll
    for (int i = 0; i < kEach; ++i) sum[i] = in[i * kPolyThreads];
    for (int p = 1; p < stretches; ++p)
#pragma unroll
      for (int i = 0; i < kEach; ++i) sum[i] += in[p * kTile * kTile + i * kPolyThreads];
  };
  wait_for_last();
  load_sums(blockIdx.x);
  for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const MuonTensor& t = tab.t[tensor_of(tile)];
    const int rows = (int)min((int64_t)t.per, t.batch - (int64_t)(tile - t.tile0) * t.per) * t.s;
    // the columns [lo, hi) of this thread's 32 that belong to its row's matrix
    const int block = row < rows ? row / t.s * t.s : kTile;
    const int lo = block - col, hi = min(block + t.s, rows) - col;
    const bool whole = t.s == kTile;
    const bool even = (t.s & (t.s - 1)) == 0;  // matrices that fill blocks of 16, 32, 64 or 128
    const int width = even ? max(t.s, 16) : kTile;
    // whether any of this warp's rows meets any of its columns
    const int r0 = row & ~31;
    const bool busy = width == kTile || (col < (r0 & ~(width - 1)) + max(width, 32) && col + 32 > (r0 & ~(width - 1)));
    const auto scaled = [&](float (&v)[32], float f) {  // times f, and 0 outside the matrix
#pragma unroll
      for (int i = 0; i < 32; i += 2) {
        const float2 x = mul2(make_float2(v[i], v[i + 1]), both(f));
        v[i] = x.x;
        v[i + 1] = x.y;
      }
      if (!whole)
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = i >= lo && i < hi ? v[i] : 0.f;
    };
    // Runs products issued by one thread; operands are in shared memory.  begin and end apart: the second
    // of two is under way while the first one's result is used.
    const auto begin = [&] {
      fence_proxy_async_smem();
      tc_fence_before();
      __syncthreads();
      if (threadIdx.x == 0) tc_fence_after();
    };
    const auto product = [&](int bar, uint32_t d, uint32_t a, uint32_t b) {
      if (threadIdx.x == 0) {
        square_product(d, a, b, width);
        mma_commit(&done[bar]);
      }
    };
    const auto end = [&](int bar) {
      wait(&done[bar], phase[bar]);
      phase[bar] ^= 1;
    };
    // G: the sums and their transpose meet in shared memory
    float v[32];
    {
      float* e = reinterpret_cast<float*>(qt);
      float* to = e + threadIdx.x / kTile * (kTile + 1) + threadIdx.x % kTile;
#pragma unroll
      for (int i = 0; i < kEach; ++i) to[i * (kPolyThreads / kTile) * (kTile + 1)] = sum[i];
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = e[row * (kTile + 1) + col + i] + e[(col + i) * (kTile + 1) + row];
    }
    float unit = 1.f;
    bool fine = true;
    if (!first) {  // X in the scratch is scaled
      unit = x_unit(factor) * x_unit(factor);
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (col + i == row) diag[row] = v[i];
      __syncthreads();
      float n2 = 0.f;
      if (whole) {
        for (int i = threadIdx.x & 31; i < kTile; i += 32) n2 += diag[i];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) n2 += __shfl_xor_sync(0xffffffffu, n2, o);
      } else {
#pragma unroll 8
        for (int i = lo; i < hi; ++i) n2 += diag[col + i];
      }
      // a norm whose square fp32 does not hold counts as 0, or is not finite, which is passed on as NaN
      fine = n2 < INFINITY;
      const float norm = fine ? counted_norm(n2) : 0.f, inv = 1.f / (norm + tab.eps);
      // X = u / (norm + eps) = (u * up) * down, up a power of two that makes the matrix's norm 2^9 to 2^10
      const float up = norm > 0.f ? ldexpf(1.f, 9 - ilogbf(norm)) : 0.f;
      unit = norm > 0.f ? inv * inv : 0.f;
      if (my_part() == 0) {
        tab.norm[(int64_t)tile * 2 * kTile + row] = up;
        tab.norm[(int64_t)tile * 2 * kTile + kTile + row] = !fine ? NAN : norm > 0.f ? inv / up : 0.f;
      }
    }
    if (!fine)
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = 0.f;
    // all matrices are held times their scales from here on
    scaled(v, unit * kGScale);
    if (threadIdx.x == 0) bulk_wait_group_read<0>();  // the last tile's P
    __syncthreads();                                   // and all have read the sums
    if (busy) tmem_put_row32(g_at, col, v);
    put_row32(gt, v);
    if (!busy) {  // what stays 0 is written once
      put_row32(qt, v);
      put_row32(pt, v);
    }
    if (steps == 0) {
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = col + i == row ? kQScale : 0.f;
      scaled(v, 1.f);
      put_row32(pt, v);
    }
#pragma unroll 1
    for (int k = 0; k < steps; ++k) {
      const bool last = k == steps - 1;
      begin();
      product(0, x_at, ga, ga);
      if (last && tile + gridDim.x < tiles) load_sums(tile + gridDim.x);
      end(0);
      if (busy) {
        float g[32];
        tmem_row32(g_at, col, g);
        tmem_row32(x_at, col, v);
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
          const float2 x = fma2(both(kc), make_float2(v[i], v[i + 1]), mul2(both(kb), make_float2(g[i], g[i + 1])));
          v[i] = x.x + (col + i == row ? ka : 0.f);
          v[i + 1] = x.y + (col + i + 1 == row ? ka : 0.f);
        }
        if (!whole) scaled(v, 1.f);
        put_row32(qt, v);
        if (k == 0) put_row32(pt, v);
      }
      if (last && k == 0) break;
      begin();
      if (!last) product(0, x_at, qa, ga);
      if (k > 0) product(1, p_at, qa, pa);
      if (!last) {
        end(0);
        if (busy) {
          tmem_row32(x_at, col, v);
          scaled(v, 1.f / kQScale);
          put_row32(gt, v);
        }
      }
      if (k > 0) {
        end(1);
        if (busy) {
          tmem_row32(p_at, col, v);
          scaled(v, 1.f / kQScale);
          put_row32(pt, v);
        }
      }
      if (last) break;
      begin();
      product(0, x_at, qa, ga);
      end(0);
      if (busy) {
        tmem_row32(x_at, col, v);
        scaled(v, 1.f / kQScale);
        tmem_put_row32(g_at, col, v);
        put_row32(gt, v);
      }
    }
    if (steps == 0 && tile + gridDim.x < tiles) load_sums(tile + gridDim.x);
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (threadIdx.x == 0) {
      bulk_store(tab.poly + (int64_t)tile * kPoly, pt, kPoly);
      bulk_commit_group();
    }
  }
  if (threadIdx.x == 0) bulk_wait_group<0>();
  tmem_close(tmem, kPolyCols);
}

// The same where all short sides are 32 or less: a warp per matrix, in fp32 without tensor cores, whose
// 24 instructions for a product take as long for 16 columns as for 128 (smallest training configuration:
// a step 51 us instead of 74, 38.6 M elements of rank 8 312 instead of 396).  A lane has a column; matrices lie in shared memory, symmetric, so that a row of
// the left factor, read by all lanes at once, stands for its column.  Only the matrices' own blocks of the
// sums are read.
constexpr int kSmall = 32, kSmallThreads = 512;
constexpr int kSmallBytes = 8 * 3 * kSmall * kSmall * 4;  // three matrices for each of eight warps, or more smaller ones
constexpr int kSmallSmem = kPoly + kSmallBytes + 1024;

// S: 8, 16 or 32, at least s; the tile has at most 128 / (S / 2 + 1) matrices beyond S = 8, which has two a warp or more.
template <int S>
__device__ __forceinline__ void small_polys(const MuonTable& tab, const MuonTensor& t, int tile, int mats, int steps, bool first, uint8_t* pt) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, s = t.s;
  constexpr int kWarps = S == 32 ? 8 : kSmallThreads / 32;
  static_assert(kWarps * 3 * S * S * 4 <= kSmallBytes, "shared memory");
  if (warp >= kWarps) return;
  float* const gm = reinterpret_cast<float*>(pt + kPoly) + warp * 3 * S * S;
  float *const qm = gm + S * S, *const pm = qm + S * S;
  const int x = t.chunk0 + (tile - t.tile0) * t.chunks;
  const int64_t s0 = stretch_slot(tab, tile, x);
  const int stretches = (int)(stretch_slot(tab, tile, x + t.chunks - 1) - s0) + 1;
  const float* sums = tab.gram + s0 * kTile * kTile;
  float* norms = tab.norm + (int64_t)tile * 2 * kTile;
  const bool in = lane < s;
  const auto put = [&](float* to, const float (&v)[S]) {
    __syncwarp();
    if (lane < S)
#pragma unroll
      for (int i = 0; i < S; ++i) to[i * S + lane] = v[i];
    __syncwarp();
  };
  const auto times = [&](const float* left, const float* right, float (&acc)[S]) {
#pragma unroll
    for (int i = 0; i < S; ++i) acc[i] = 0.f;
#pragma unroll 4
    for (int k = 0; k < S; ++k) {
      const float v = right[k * S + lane % S];
#pragma unroll
      for (int i = 0; i < S; i += 4) {
        const float4 u = *reinterpret_cast<const float4*>(left + k * S + i);
        acc[i] = fmaf(u.x, v, acc[i]);
        acc[i + 1] = fmaf(u.y, v, acc[i + 1]);
        acc[i + 2] = fmaf(u.z, v, acc[i + 2]);
        acc[i + 3] = fmaf(u.w, v, acc[i + 3]);
      }
    }
  };
#pragma unroll 1
  for (int mat = warp; mat < mats; mat += kWarps) {
    const int at = mat * s;  // first row and column
    float g[S], v[S];
#pragma unroll
    for (int i = 0; i < S; ++i) g[i] = 0.f;
#pragma unroll 1
    for (int k = 0; k < stretches; ++k) {
      const float* e = sums + (int64_t)k * kTile * kTile;
#pragma unroll
      for (int i = 0; i < S; ++i)
        if (in && i < s) g[i] += e[(at + i) * kTile + at + lane] + e[(at + lane) * kTile + at + i];
    }
    float unit = 1.f;
    if (!first) {
      const float factor = norms[kTile + at];
      unit = x_unit(factor) * x_unit(factor);
    } else {  // as in the kernel above
      float n2 = 0.f;
#pragma unroll
      for (int i = 0; i < S; ++i) n2 += i == lane ? g[i] : 0.f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) n2 += __shfl_xor_sync(0xffffffffu, n2, o);
      const bool fine = n2 < INFINITY;
      const float norm = fine ? counted_norm(n2) : 0.f, inv = 1.f / (norm + tab.eps);
      const float up = norm > 0.f ? ldexpf(1.f, 9 - ilogbf(norm)) : 0.f;
      unit = norm > 0.f ? inv * inv : 0.f;
      if (in) {
        norms[at + lane] = up;
        norms[kTile + at + lane] = !fine ? NAN : norm > 0.f ? inv / up : 0.f;
      }
      if (!fine)
#pragma unroll
        for (int i = 0; i < S; ++i) g[i] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < S; ++i) {
      g[i] *= unit;
      v[i] = i == lane ? 1.f : 0.f;
    }
    put(gm, g);
    if (steps == 0) put(pm, v);
#pragma unroll 1
    for (int k = 0; k < steps; ++k) {
      times(gm, gm, v);
#pragma unroll
      for (int i = 0; i < S; ++i) v[i] = fmaf(tab.c, v[i], fmaf(tab.b, g[i], i == lane && in ? tab.a : 0.f));
      put(qm, v);
      if (k > 0) times(qm, pm, v);
      put(pm, v);
      if (k < steps - 1) {
        times(qm, gm, g);
        put(gm, g);
        times(qm, gm, g);
        put(gm, g);
      }
    }
    if (in)
#pragma unroll 4
      for (int i = 0; i < s; ++i) {
        const float f = pm[i * S + lane] * kQScale;
        const __half hi = __float2half_rn(f), lo = __float2half_rn(f - __half2float(hi));
        const int r = at + i, c = at + lane;
        uint8_t* to = pt + (c >> 6) * kPart + r * 128 + ((((c & 63) >> 3) ^ (r & 7)) << 4) + (c & 7) * 2;
        *reinterpret_cast<__half*>(to) = hi;
        *reinterpret_cast<__half*>(to + kTileBytes) = lo;
      }
  }
}
__global__ void __launch_bounds__(kSmallThreads, 1) muon_small_kernel(const __grid_constant__ MuonTable tab, int steps, bool first) {
  extern __shared__ uint8_t muon_smem[];
  uint8_t* pt = aligned_smem(muon_smem);
  const int tile = blockIdx.x;
  launch_next();
  int ti = 0;
  while (ti + 1 < tab.n && tile >= tab.t[ti + 1].tile0) ++ti;
  const MuonTensor& t = tab.t[ti];
  const int mats = (int)min((int64_t)t.per, t.batch - (int64_t)(tile - t.tile0) * t.per), row = threadIdx.x;
#pragma unroll
  for (int i = 0; i < kPoly / 16 / kSmallThreads; ++i) reinterpret_cast<uint4*>(pt)[threadIdx.x + i * kSmallThreads] = make_uint4(0, 0, 0, 0);
  __syncthreads();
  wait_for_last();
  if (first && row < kTile && row >= mats * t.s)  // rows of no matrix
    tab.norm[(int64_t)tile * 2 * kTile + row] = tab.norm[(int64_t)tile * 2 * kTile + kTile + row] = 0.f;
  if (t.s <= 8)
    small_polys<8>(tab, t, tile, mats, steps, first, pt);
  else if (t.s <= 16)
    small_polys<16>(tab, t, tile, mats, steps, first, pt);
  else
    small_polys<32>(tab, t, tile, mats, steps, first, pt);
  fence_proxy_async_smem();
  __syncthreads();
  if (threadIdx.x == 0) {
    bulk_store(tab.poly + (int64_t)tile * kPoly, pt, kPoly);
    bulk_commit_group();
    bulk_wait_group<0>();
  }
}

// ------------------------------------------------------------------ apply and update
// D [128 x 64] = P X of a chunk.  X as two fp16 parts: rows of 64 long places (a short side
// each), or two halves of 64 short places (a row per long place).
__device__ __forceinline__ void poly_product(uint32_t d, uint32_t p, uint32_t x, bool tall) {
  const uint32_t id = idesc_f16_f32(kTile, kChunk, false, !tall);
  const uint32_t lbo = tall ? 16 : 8192;
#pragma unroll 1
  for (int q = 0; q < 3; ++q) {
    const uint32_t a = p + (q == 2 ? kTileBytes : 0), b = x + (q == 1 ? kPart : 0);
#pragma unroll
    for (int kk = 0; kk < kTile / 16; ++kk) {
      const uint32_t at = tall ? kk / 4 * (kPart / 2) + kk % 4 * 32 : kk * 2048;
      mma_bf16(d, sw128_desc(a + kk / 4 * kPart + kk % 4 * 32, 16, 1024), sw128_desc(b + at, lbo, 1024), id, q > 0 || kk > 0);
    }
  }
}
template <int kBytes>
__device__ __forceinline__ void copy_async(uint8_t* dst, const uint8_t* src) {
#pragma unroll
  for (int i = 0; i < kBytes / 16 / kThreads; ++i) async_copy16(dst + (threadIdx.x + i * kThreads) * 16, src + (threadIdx.x + i * kThreads) * 16);
  async_commit();
}

constexpr int kApplySmem = kPoly + kImage + 1024, kApplyCols = 256;

// X <- P X in fp16 parts (kept), and the partial G of it.
__global__ void __launch_bounds__(kThreads, 2) muon_apply_kernel(const __grid_constant__ MuonTable tab) {
  extern __shared__ uint8_t muon_smem[];
  __shared__ uint64_t done[2];
  __shared__ uint32_t slot;
  __shared__ float row_up[kTile];
  uint8_t* sm = aligned_smem(muon_smem);
  uint8_t *pt = sm, *xt = sm + kPoly;
  if (threadIdx.x == 0) {
    mbar_init(&done[0], 1);
    mbar_init(&done[1], 1);
    fence_mbar_init();
  }
  launch_next();
  const uint32_t acc = tmem_open(&slot, kApplyCols), gram = acc + 64;
  wait_for_last();
  Waits wait{tab.err};
  int used = 0;  // chunks so far
  const int r = my_row();
  const bool with_g = tab.nesterov;
  const float nu = tab.nu * (tab.gs ? *tab.gs : 1.f);
  const int end = first_chunk(tab, blockIdx.x + 1);
  for (int x = first_chunk(tab, blockIdx.x); x < end;) {
    const Place pl = place_of(tab, x, end);
    const MuonTensor& t = *pl.t;
    const bool tall = t.tall;
    const Walk w(t, pl.first, pl.rows);
    copy_async<kPoly>(pt, tab.poly + (int64_t)pl.tile * kPoly);  // no product is under way here
    const float* norm = tab.norm + (int64_t)pl.tile * 2 * kTile;
    __syncthreads();  // the last stretch's scales have been read
    if (threadIdx.x < kTile) row_up[threadIdx.x] = norm[threadIdx.x];
    // P's scale, and the factor that makes the products X
    const float factor = norm[kTile + r], down = factor == factor ? factor * (x_scale(factor) * (1.f / kQScale)) : 0.f;
    with_kind(t.g_dtype, quads_aligned(t), [&](auto type, auto quads) {
      constexpr int kType = decltype(type)::value;
      constexpr bool kAligned = decltype(quads)::value;
      Loads<kType> ld(t);
      if (kAligned) ld.chunk(w, pl.c0, with_g);
      async_wait<0>();
      __syncthreads();
      for (int c = pl.c0; c < pl.c1; ++c, ++used) {
        if (used > 0) {  // the products and the copy that read the tile
          wait(&done[1], (used - 1) & 1);
          if (threadIdx.x == 0) bulk_wait_group_read<0>();
          __syncthreads();
        }
        const auto put = [&](int i, Four u, const Four& g) {
          if (with_g) u = mix(tab.mu, u, nu, g);
          const float* f = row_up + w.row_of(i);
          const float2 fa = tall ? make_float2(f[0], f[1]) : both(f[0]), fb = tall ? make_float2(f[2], f[3]) : both(f[0]);
          u = Four{mul2(u.a, fa), mul2(u.b, fb)};
          // matrices without a norm (0, or not finite) take no part
          u.a = make_float2(fa.x > 0.f ? u.a.x : 0.f, fa.y > 0.f ? u.a.y : 0.f);
          u.b = make_float2(fb.x > 0.f ? u.b.x : 0.f, fb.y > 0.f ? u.b.y : 0.f);
          uint2 hi, lo;
          fp16_parts(u.a, hi.x, lo.x);
          fp16_parts(u.b, hi.y, lo.y);
          uint8_t* to = xt + w.operand(i);
          *reinterpret_cast<uint2*>(to) = hi;
          *reinterpret_cast<uint2*>(to + kPart) = lo;
        };
        if constexpr (kAligned) {
#pragma unroll
          for (int i = 0; i < kQuads; ++i) put(i, widen<MOE_LORA_F32>(ld.m[i]), widen<kType>(ld.g[i]));
        } else {
#pragma unroll 1
          for (int i = 0; i < kQuads; ++i)
            put(i, ld_loose<MOE_LORA_F32>(ld.mp, t, w, pl.first, c, i),
                with_g ? ld_loose<kType>(ld.gp, t, w, pl.first, c, i) : Four{both(0.f), both(0.f)});
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncthreads();
        if (threadIdx.x == 0) {
          tc_fence_after();
          poly_product(acc, smem_u32(pt), smem_u32(xt), tall);
          mma_commit(&done[0]);
        }
        // not before: the products wait for the operands' stores, which the loads would hold up (734 us
        // instead of 606 for 203 M elements, all else equal)
        if (kAligned && c + 1 < pl.c1) ld.chunk(w, c + 1, with_g);
        wait(&done[0], used & 1);
        // rows of 64 long places from here on: half a row each
        {
          float v[32];
          tmem_row32(acc, my_part() * 32, v);
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) fp16_parts(mul2(make_float2(v[8 * u + 2 * i], v[8 * u + 2 * i + 1]), both(down)), hi[i], lo[i]);
            const int at = r * 128 + (((my_part() * 4 + u) ^ (r & 7)) << 4);
            *reinterpret_cast<uint4*>(xt + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4*>(xt + kPart + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncthreads();
        if (threadIdx.x == 0) {
          tc_fence_after();
          const uint32_t h = smem_u32(xt), l = h + kPart, id = idesc_f16_f32(kTile, kTile, false, false);
#pragma unroll
          for (int kk = 0; kk < kChunk / 16; ++kk) {
            const uint64_t dh = sw128_desc(h + kk * 32, 16, 1024), dl = sw128_desc(l + kk * 32, 16, 1024);
            mma_bf16(gram, dh, dh, id, c > pl.c0 || kk > 0);
            mma_bf16(gram, dh, dl, id, 1);
            mma_bf16(gram, dl, dh, id, 1);
          }
          mma_commit(&done[1]);
          // the tile as it lies, 32 KB in one copy (16-byte stores by the threads that formed it: 789 us
          // instead of 539 for 203 M elements)
          bulk_store(tab.x + (x + c - pl.c0) * (int64_t)kImage, xt, kImage);
          bulk_commit_group();
        }
      }
    });
    wait(&done[1], (used - 1) & 1);
    float* out = tab.gram + stretch_slot(tab, pl.tile, x) * kTile * kTile + r;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int col = my_part() * 64 + b * 32;
      float v[32];
      tmem_row32(gram, col, v);
#pragma unroll
      for (int i = 0; i < 32; ++i) out[(col + i) * kTile] = 0.5f * v[i];
    }
    x += pl.c1 - pl.c0;
  }
  if (threadIdx.x == 0) bulk_wait_group<0>();
  tmem_close(acc, kApplyCols);
}

// The products change threads through shared memory, where X was, so that quads can be read:
// rows of the short side, or of long places where the weights are tall.
constexpr int kPitch = 68, kTallPitch = 132;
constexpr int kOutBytes = kTile * kPitch * 4;
static_assert(kOutBytes >= kImage && kOutBytes >= kChunk * kTallPitch * 4, "one place for both");
constexpr int kUpdateSmem = kPoly + kOutBytes + 1024, kUpdateCols = 64;

// O = P X and the weights of the tensors of one kind (kW: type of the weights that are read, master
// or p; kP: of p).  A launch for each kind that there is; its blocks pass over the others' stretches.
template <int kW, int kP>
__global__ void __launch_bounds__(kThreads, 2) muon_update_kernel(const __grid_constant__ MuonTable tab) {
  constexpr bool kMaster = kW != kP;
  extern __shared__ uint8_t muon_smem[];
  __shared__ uint64_t done;
  __shared__ uint32_t slot;
  uint8_t* sm = aligned_smem(muon_smem);
  uint8_t *pt = sm, *xt = sm + kPoly;
  if (threadIdx.x == 0) {
    mbar_init(&done, 1);
    fence_mbar_init();
  }
  launch_next();
  const uint32_t acc = tmem_open(&slot, kUpdateCols);
  wait_for_last();
  Waits wait{tab.err};
  uint32_t used = 0;  // chunks so far
  const int end = first_chunk(tab, blockIdx.x + 1);
  for (int x = first_chunk(tab, blockIdx.x); x < end;) {
    const Place pl = place_of(tab, x, end);
    const MuonTensor& t = *pl.t;
    const uint8_t* image = tab.x + x * (int64_t)kImage;
    x += pl.c1 - pl.c0;
    if ((t.master != nullptr) != kMaster || t.p_dtype != kP) continue;
    copy_async<kPoly>(pt, tab.poly + (int64_t)pl.tile * kPoly);  // no product is under way, and all have read the last ones
    copy_async<kImage>(xt, image);
    const float factor = tab.norm[(int64_t)pl.tile * 2 * kTile + kTile + my_row()];
    // NaN for a matrix whose norm is not finite
    const float f = (factor == factor ? 1.f : factor) * (x_unit(factor) * (1.f / kQScale));
    const bool aligned = quads_aligned(t), tall = t.tall;
    const void* const wp = in_register(kMaster ? static_cast<void*>(t.master) : t.p);
    void* const pp = in_register(t.p);
    const float decay = t.decay, step = t.step;
    const Walk w(t, pl.first, pl.rows);
    float* o = reinterpret_cast<float*>(xt);
    // a thread's quads among the products
    const float* mine = tall ? o + w.col * kTallPitch + w.row : o + w.row * kPitch + w.col;
    const int hop = tall ? w.hop_col * kTallPitch : w.hop_row * kPitch, hop4 = tall ? w.hop_col4 * kTallPitch + w.hop_row4 : 4 * hop;
    for (int c = pl.c0; c < pl.c1; ++c, ++used) {
      const uint32_t in = w.inside(c);
      const int64_t at = w.at + c * w.chunk;
      async_wait<0>();
      fence_proxy_async_smem();
      tc_fence_before();
      __syncthreads();
      if (threadIdx.x == 0) {
        tc_fence_after();
        poly_product(acc, smem_u32(pt), smem_u32(xt), false);
        mma_commit(&done);
      }
      uint4 old[kQuads];
      if (aligned)
#pragma unroll
        for (int i = 0; i < kQuads; ++i) old[i] = in >> i & 1 ? ld_quad<kW>(wp, at + w.element(i)) : make_uint4(0, 0, 0, 0);
      wait(&done, used & 1);
      {
        float v[32];
        tmem_row32(acc, my_part() * 32, v);
        if (tall) {
          float* to = o + my_part() * 32 * kTallPitch + my_row();
#pragma unroll
          for (int i = 0; i < 32; ++i) to[i * kTallPitch] = v[i] * f;
        } else {
          float* to = o + my_row() * kPitch + my_part() * 32;
#pragma unroll
          for (int i = 0; i < 32; i += 4) *reinterpret_cast<float4*>(to + i) = make_float4(v[i] * f, v[i + 1] * f, v[i + 2] * f, v[i + 3] * f);
        }
      }
      __syncthreads();
      const auto stepped = [&](const Four& u, const float4& y) {
        return Four{fma2(both(-step), make_float2(y.x, y.y), mul2(u.a, both(decay))),
                    fma2(both(-step), make_float2(y.z, y.w), mul2(u.b, both(decay)))};
      };
      Four y[kQuads];  // the weights
      if (aligned) {
#pragma unroll
        for (int i = 0; i < kQuads; ++i) y[i] = stepped(widen<kW>(old[i]), *reinterpret_cast<const float4*>(mine + (i & 3) * hop + (i >> 2) * hop4));
      } else {
#pragma unroll 1
        for (int i = 0; i < kQuads; ++i) {
          const Four u = stepped(ld_loose<kW>(wp, t, w, pl.first, c, i), *reinterpret_cast<const float4*>(mine + (i & 3) * hop + (i >> 2) * hop4));
          if (kMaster) st_loose<MOE_LORA_F32>(const_cast<void*>(wp), t, w, pl.first, c, i, u);
          st_loose<kP>(pp, t, w, pl.first, c, i, u);
        }
      }
      __syncthreads();
      image += kImage;
      if (c + 1 < pl.c1) copy_async<kImage>(xt, image);
      if (aligned) {
#pragma unroll
        for (int i = 0; i < kQuads; ++i)
          if (in >> i & 1) {
            const Four& u = y[i];
            if (kMaster) st_quad<MOE_LORA_F32>(const_cast<void*>(wp), at + w.element(i), u);
            st_quad<kP>(pp, at + w.element(i), u);
          }
      }
    }
  }
  tmem_close(acc, kUpdateCols);
}

// ------------------------------------------------------------------ host
int check_shape(const moe_lora_muon_tensor& t) {
  if (t.batch < 0 || t.rows < 1 || t.cols < 1) return MOE_LORA_ERR_DIMS;
  if (std::min(t.rows, t.cols) > kTile) return MOE_LORA_ERR_UNSUPPORTED;
  if (t.batch > (int64_t)1 << 32 || t.batch * t.rows > ((int64_t)1 << 40) / t.cols) return MOE_LORA_ERR_DIMS;
  return MOE_LORA_OK;
}
int check_muon(const moe_lora_muon_tensor& t) {
  int rc = check_shape(t);
  if (rc) return rc;
  if (!dtype_ok(t.p_dtype) || !dtype_ok(t.g_dtype)) return MOE_LORA_ERR_UNSUPPORTED;
  if (t.master && t.p_dtype == MOE_LORA_F32) return MOE_LORA_ERR_UNSUPPORTED;
  if (!isfinite(t.lr) || !isfinite(t.weight_decay) || !isfinite(t.scale)) return MOE_LORA_ERR_DIMS;
  if (t.batch == 0) return MOE_LORA_OK;
  if ((rc = check_ptr(t.p)) || (rc = check_ptr(t.g)) || (rc = check_ptr(t.m))) return rc;
  return check_opt(t.master);
}
struct Shape {
  int s, L, per;
  int64_t tiles, chunks;
};
Shape shape_of(const moe_lora_muon_tensor& t) {
  Shape h;
  h.s = std::min(t.rows, t.cols);
  h.L = std::max(t.rows, t.cols);
  h.per = kTile / h.s;
  h.tiles = (t.batch + h.per - 1) / h.per;
  h.chunks = (h.L + kChunk - 1) / kChunk;
  return h;
}
// Two blocks on each of 152 SMs share the chunks of a launch; where that would be more than 128 chunks a
// block, twice, three times, ... as many do (a stretch adds up in one accumulator of the tensor cores,
// whose additions are cut off rather than rounded).
constexpr int kBlocks = 304, kMaxStretch = 128;
struct Layout {
  size_t err, norm, poly, gram, x, total;
  int blocks;
  int64_t tiles, chunks;
};
Layout layout_of(const moe_lora_muon_tensor* t, int n) {
  Layout l = {};
  for (int i = 0; i < n; ++i) {
    const Shape h = shape_of(t[i]);
    l.tiles += h.tiles;
    l.chunks += h.tiles * h.chunks;
  }
  l.blocks = (int)std::min<int64_t>(l.chunks, kBlocks * std::max<int64_t>(1, (l.chunks + kBlocks * kMaxStretch - 1) / (kBlocks * kMaxStretch)));
  size_t o = 0;
  const auto take = [&](size_t bytes) { const size_t at = o; o = align_up(o + bytes, 256); return at; };
  l.err = take(16);
  l.norm = take(sizeof(float) * 2 * kTile * l.tiles);
  l.poly = take((size_t)kPoly * l.tiles);
  l.gram = take(sizeof(float) * kTile * kTile * (l.tiles + l.blocks));
  l.x = take((size_t)kImage * l.chunks);
  l.total = o;
  return l;
}

template <class K, class... A>
int launch_muon(int slot, K kernel, int64_t grid, int threads, size_t smem, bool overlap, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at;
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = overlap ? 1 : 0;
  prof_begin(slot, s);
  const cudaError_t e = launch_allowed(cfg, false, kernel, args...);
  prof_end(slot, s);
  return e == cudaSuccess ? MOE_LORA_OK : MOE_LORA_ERR_CUDA;
}

// The five launches over up to kMaxTensors tensors.
int run_muon(const moe_lora_muon* o, const moe_lora_muon_tensor* in, int n, uint8_t* ws, int sms, cudaStream_t s) {
  const Layout l = layout_of(in, n);
  if (l.tiles == 0) return MOE_LORA_OK;
  MuonTable tab;
  tab.n = 0;
  tab.blocks = l.blocks;
  tab.chunks = (int)l.chunks;
  tab.mu = (float)o->momentum;
  tab.nu = (float)(1 - o->momentum);
  tab.eps = (float)o->eps;
  tab.a = (float)o->a;
  tab.b = (float)o->b;
  tab.c = (float)o->c;
  tab.nesterov = o->nesterov != 0;
  tab.gs = o->grad_scale;
  tab.err = reinterpret_cast<int*>(ws + l.err);
  tab.norm = reinterpret_cast<float*>(ws + l.norm);
  tab.poly = ws + l.poly;
  tab.gram = reinterpret_cast<float*>(ws + l.gram);
  tab.x = ws + l.x;
  int64_t tile = 0, chunk = 0;
  for (int i = 0; i < n; ++i) {
    const Shape h = shape_of(in[i]);
    if (h.tiles == 0) continue;
    MuonTensor& t = tab.t[tab.n++];
    t = MuonTensor{in[i].p, in[i].master, in[i].g, in[i].m, in[i].batch, (int)tile, (int)chunk, h.s, h.L, in[i].rows > in[i].cols, h.per,
                   (int)h.chunks, in[i].p_dtype, in[i].g_dtype,
                   (float)(1 - in[i].lr * in[i].weight_decay), (float)(in[i].lr * in[i].scale)};
    tile += h.tiles;
    chunk += h.tiles * h.chunks;
  }
  const int first = std::min(kFirstSteps, o->steps > 3 ? 2 : 1);
  int rc;
  bool small = true;
  for (int i = 0; i < tab.n; ++i) small = small && tab.t[i].s <= kSmall;
  const auto poly = [&](int steps, bool is_first) {
    return small ? launch_muon(K_MUON_POLY, muon_small_kernel, l.tiles, kSmallThreads, kSmallSmem, true, s, tab, steps, is_first)
                 : launch_muon(K_MUON_POLY, muon_poly_kernel, std::min<int64_t>(l.tiles, sms), kPolyThreads, kPolySmem, true, s, tab,
                               (int)l.tiles, steps, is_first);
  };
  if ((rc = launch_muon(K_MUON_GRAM, muon_gram_kernel, l.blocks, kThreads, kGramSmem, false, s, tab)) || (rc = poly(first, true)) ||
      (rc = launch_muon(K_MUON_APPLY, muon_apply_kernel, l.blocks, kThreads, kApplySmem, true, s, tab)) ||
      (rc = poly(o->steps - first, false)))
    return rc;
  bool overlap = true;  // the first kind's launch with what is before it; the others follow it as any launch does
  const auto update = [&](auto kernel, int dtype, bool master) {
    for (int i = 0; i < tab.n; ++i)
      if (tab.t[i].p_dtype == dtype && (tab.t[i].master != nullptr) == master) {
        const int e = launch_muon(K_MUON_UPDATE, kernel, l.blocks, kThreads, kUpdateSmem, overlap, s, tab);
        overlap = false;
        return e;
      }
    return MOE_LORA_OK;
  };
  if ((rc = update(muon_update_kernel<MOE_LORA_F32, MOE_LORA_BF16>, MOE_LORA_BF16, true)) ||
      (rc = update(muon_update_kernel<MOE_LORA_F32, MOE_LORA_F16>, MOE_LORA_F16, true)) ||
      (rc = update(muon_update_kernel<MOE_LORA_F32, MOE_LORA_F32>, MOE_LORA_F32, false)) ||
      (rc = update(muon_update_kernel<MOE_LORA_BF16, MOE_LORA_BF16>, MOE_LORA_BF16, false)) ||
      (rc = update(muon_update_kernel<MOE_LORA_F16, MOE_LORA_F16>, MOE_LORA_F16, false)))
    return rc;
  return MOE_LORA_OK;
}

}  // namespace

}  // namespace moelora

using namespace moelora;

extern "C" size_t moe_lora_muon_scratch_bytes(const moe_lora_muon_tensor* tensors, int32_t n) {
  if (n < 0 || (n > 0 && !tensors)) return 0;
  size_t most = 256;
  for (int i = 0; i < n; ++i)
    if (check_shape(tensors[i])) return 0;
  for (int i = 0; i < n; i += kMaxTensors) most = std::max(most, layout_of(tensors + i, std::min(kMaxTensors, n - i)).total);
  return most;
}

extern "C" int moe_lora_muon_step(const moe_lora_muon* o, const moe_lora_muon_tensor* tensors, int32_t n, void* scratch,
                                  size_t scratch_bytes, void* stream) {
  if (!o || (n > 0 && !tensors)) return MOE_LORA_ERR_NULL;
  if (n < 0) return MOE_LORA_ERR_DIMS;
  if (o->steps < 1 || o->steps > kMaxSteps) return MOE_LORA_ERR_UNSUPPORTED;
  if (!(o->momentum >= 0 && o->momentum < 1) || !(o->eps >= 1e-30) || !(o->eps <= 1)) return MOE_LORA_ERR_DIMS;
  if (!(fabs(o->a) <= 8) || !(fabs(o->b) <= 16) || !(fabs(o->c) <= 16)) return MOE_LORA_ERR_DIMS;
  int rc;
  if (reinterpret_cast<uintptr_t>(o->grad_scale) & 3u) return MOE_LORA_ERR_ALIGN;
  for (int i = 0; i < n; ++i)
    if ((rc = check_muon(tensors[i]))) return rc;
  if ((rc = check_ptr(scratch))) return rc;
  if (scratch_bytes < moe_lora_muon_scratch_bytes(tensors, n)) return MOE_LORA_ERR_WORKSPACE;
  for (int i = 0; i < n; i += kMaxTensors)
    if (layout_of(tensors + i, std::min(kMaxTensors, n - i)).chunks > (int64_t)1 << 30) return MOE_LORA_ERR_DIMS;
  int sms;
  if ((rc = device_sms(&sms))) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  for (int i = 0; i < n; i += kMaxTensors)
    if ((rc = run_muon(o, tensors + i, std::min(kMaxTensors, n - i), static_cast<uint8_t*>(scratch), sms, s))) return rc;
  return MOE_LORA_OK;
}

extern "C" int moe_lora_muon_get_error(const void* scratch, void* stream) {
  if (!scratch) return MOE_LORA_ERR_NULL;
  int v = 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cudaMemcpyAsync(&v, scratch, sizeof v, cudaMemcpyDeviceToHost, s) != cudaSuccess || cudaStreamSynchronize(s) != cudaSuccess)
    return MOE_LORA_ERR_CUDA;
  return v;
}
