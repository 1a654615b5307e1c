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
// places of the long side, a piece a few chunks of a tile: the work of a block.
#include <math.h>

#include <algorithm>

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
// Powers of two that bring values into the middle of fp16's range.
constexpr float kXScale = 1024.f, kGScale = 256.f, kQScale = 64.f;

struct MuonTensor {
  void* p;
  float* master;
  const void* g;
  float* m;
  int64_t batch, tile0, piece0;  // matrices; first tile and piece of the launch
  int32_t s, L, tall;            // tall: [L, s] in memory
  int32_t per, pieces;           // matrices of a tile, pieces of a tile
  int32_t p_dtype, g_dtype;
  float decay, step;             // 1 - lr * weight_decay, lr * scale
};
struct MuonTable {
  int n, piece;                  // tensors; chunks of a piece
  int64_t tiles, pieces;
  float mu, nu, eps, a, b, c;    // nu = 1 - mu
  int nesterov;
  const float* gs;
  int* err;
  float *gram, *norm;            // [pieces][128][128], [tiles][128]: norm, factor of a row's matrix
  uint8_t *poly, *x;             // [tiles][kPoly], [chunks][kImage]
  MuonTensor t[kMaxTensors];
};
static_assert(sizeof(MuonTable) <= 32764, "kernel parameter limit");

struct Place {  // of a piece
  const MuonTensor* t;
  int64_t tile, image;  // of the launch; first chunk's image in the scratch
  int64_t first;        // first matrix
  int rows;             // short sides in use
  int c0, c1;           // chunks
};
__device__ __forceinline__ int64_t chunks_of(const MuonTensor& t) { return (t.L + kChunk - 1) / kChunk; }
__device__ __forceinline__ Place place_of(const MuonTable& tab, int64_t piece) {
  int lo = 0, hi = tab.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (piece >= tab.t[mid].piece0)
      lo = mid;
    else
      hi = mid - 1;
  }
  const MuonTensor& t = tab.t[lo];
  const int64_t tile = (piece - t.piece0) / t.pieces, part = (piece - t.piece0) % t.pieces;
  Place p;
  p.t = &t;
  p.tile = t.tile0 + tile;
  p.first = tile * t.per;
  p.rows = (int)min((int64_t)t.per, t.batch - p.first) * t.s;
  p.c0 = (int)part * tab.piece;
  p.c1 = min(p.c0 + tab.piece, (int)chunks_of(t));
  // images lie piece by piece, tab.piece to each
  p.image = piece * tab.piece;
  return p;
}

// ------------------------------------------------------------------ a thread's share of a chunk
// Quad i of a thread: four neighbouring elements in memory.  Rows of the short side [s, L]:
// along the long side; tall matrices [L, s]: along the short one.
struct Quad {
  int row, col;  // short side within the tile, long side within the chunk, of its first element
  __device__ __forceinline__ Quad(bool tall, int i) {
    if (tall) {
      row = (threadIdx.x & 31) * 4;
      col = i * (kThreads / 32) + (threadIdx.x >> 5);
    } else {
      row = i * (kThreads / 16) + (threadIdx.x >> 4);
      col = (threadIdx.x & 15) * 4;
    }
  }
};
// Element offset of (row, long index) from the tile's first matrix.
__device__ __forceinline__ int64_t offset_of(const MuonTensor& t, int row, int l) {
  if (!t.tall) return (int64_t)row * t.L + l;
  const int j = row / t.s;
  return ((int64_t)j * t.L + l) * t.s + (row - j * t.s);
}
// Whether all quads lie inside one matrix's run of memory and on 16 bytes (8 of 16-bit types).
__device__ __forceinline__ bool quads_aligned(const MuonTensor& t) { return t.tall ? t.s % 4 == 0 : t.L % 4 == 0; }

__device__ __forceinline__ float ld_one(const void* p, int dtype, int64_t i) {
  return dtype == MOE_LORA_F32    ? static_cast<const float*>(p)[i]
         : dtype == MOE_LORA_BF16 ? to_f32(static_cast<const __nv_bfloat16*>(p)[i])
                                  : to_f32(static_cast<const __half*>(p)[i]);
}
__device__ __forceinline__ void st_one(void* p, int dtype, int64_t i, float v) {
  if (dtype == MOE_LORA_F32)
    static_cast<float*>(p)[i] = v;
  else if (dtype == MOE_LORA_BF16)
    static_cast<__nv_bfloat16*>(p)[i] = from_f32<__nv_bfloat16>(v);
  else
    static_cast<__half*>(p)[i] = from_f32<__half>(v);
}
// Four elements as loaded, and widened.
__device__ __forceinline__ uint4 ld_quad(const void* p, int dtype, int64_t i) {
  if (dtype == MOE_LORA_F32) return *reinterpret_cast<const uint4*>(static_cast<const float*>(p) + i);
  const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i);
  return make_uint4(u.x, u.y, 0, 0);
}
__device__ __forceinline__ float4 widen(const uint4& u, int dtype) {
  if (dtype == MOE_LORA_F32)
    return make_float4(__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z), __uint_as_float(u.w));
  const float2 a = dtype == MOE_LORA_BF16 ? Two<__nv_bfloat16>::get(&u.x) : Two<__half>::get(&u.x);
  const float2 b = dtype == MOE_LORA_BF16 ? Two<__nv_bfloat16>::get(&u.y) : Two<__half>::get(&u.y);
  return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ void st_quad(void* p, int dtype, int64_t i, const float4& v) {
  if (dtype == MOE_LORA_F32) {
    *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = v;
    return;
  }
  uint2 u;
  if (dtype == MOE_LORA_BF16) {
    Two<__nv_bfloat16>::put(&u.x, make_float2(v.x, v.y));
    Two<__nv_bfloat16>::put(&u.y, make_float2(v.z, v.w));
  } else {
    Two<__half>::put(&u.x, make_float2(v.x, v.y));
    Two<__half>::put(&u.y, make_float2(v.z, v.w));
  }
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + i) = u;
}

// The gradient and momentum of a thread's quads of a chunk, on their way.
struct Loads {
  uint4 g[kQuads], m[kQuads];
};
__device__ __forceinline__ void load_chunk(const Place& pl, int c, bool aligned, bool with_g, Loads& ld) {
  const MuonTensor& t = *pl.t;
  const int64_t base = pl.first * t.s * t.L;
#pragma unroll
  for (int i = 0; i < kQuads; ++i) {
    const Quad q(t.tall, i);
    const int l = c * kChunk + q.col;
    ld.g[i] = ld.m[i] = make_uint4(0, 0, 0, 0);
    if (aligned) {
      if (q.row < pl.rows && l < t.L) {
        const int64_t at = base + offset_of(t, q.row, l);
        if (with_g) ld.g[i] = ld_quad(t.g, t.g_dtype, at);
        ld.m[i] = *reinterpret_cast<const uint4*>(t.m + at);
      }
    } else {  // widened at once
      float gv[4] = {}, mv[4] = {};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = q.row + (t.tall ? e : 0), k = l + (t.tall ? 0 : e);
        if (r < pl.rows && k < t.L) {
          const int64_t at = base + offset_of(t, r, k);
          if (with_g) gv[e] = ld_one(t.g, t.g_dtype, at);
          mv[e] = t.m[at];
        }
      }
      ld.g[i] = make_uint4(__float_as_uint(gv[0]), __float_as_uint(gv[1]), __float_as_uint(gv[2]), __float_as_uint(gv[3]));
      ld.m[i] = make_uint4(__float_as_uint(mv[0]), __float_as_uint(mv[1]), __float_as_uint(mv[2]), __float_as_uint(mv[3]));
    }
  }
}
__device__ __forceinline__ void store_m(const Place& pl, int c, bool aligned, int i, const float4& v) {
  const MuonTensor& t = *pl.t;
  const int64_t base = pl.first * t.s * t.L;
  const Quad q(t.tall, i);
  const int l = c * kChunk + q.col;
  if (aligned) {
    if (q.row < pl.rows && l < t.L) *reinterpret_cast<float4*>(t.m + base + offset_of(t, q.row, l)) = v;
    return;
  }
  const float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int r = q.row + (t.tall ? e : 0), k = l + (t.tall ? 0 : e);
    if (r < pl.rows && k < t.L) t.m[base + offset_of(t, r, k)] = x[e];
  }
}
// mu m + nu g, products and sum rounded one by one as the definition's are.
__device__ __forceinline__ float mix(float mu, float m, float nu, float g) { return __fadd_rn(__fmul_rn(mu, m), __fmul_rn(nu, g)); }
__device__ __forceinline__ float4 mix4(float mu, const float4& m, float nu, const float4& g) {
  return make_float4(mix(mu, m.x, nu, g.x), mix(mu, m.y, nu, g.y), mix(mu, m.z, nu, g.z), mix(mu, m.w, nu, g.w));
}
__device__ __forceinline__ float4 scale4(const float4& v, float f) { return make_float4(v.x * f, v.y * f, v.z * f, v.w * f); }

// ------------------------------------------------------------------ operands in shared memory
// All tiles have rows of 128 bytes whose 16-byte units are exchanged by row (unit ^ row % 8).
// A chunk of [s, L]: 128 rows of 64 long places.  Of [L, s]: two halves of 64 short places, a
// row per long place.
__device__ __forceinline__ uint32_t quad_at(bool tall, const Quad& q) {
  const uint32_t r = tall ? q.col : q.row, k = tall ? q.row % 64 : q.col, half = tall ? q.row / 64 * (kPart / 2) : 0;
  return half + r * 128 + ((((k >> 3) ^ (r & 7)) << 4) | ((k & 4) << 1));
}
__device__ __forceinline__ uint32_t hf2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return reinterpret_cast<const uint32_t&>(h);
}
// v -> its bf16 parts, each stored as eight bytes
__device__ __forceinline__ void put_bf16_parts(uint8_t* at, float4 v) {
#pragma unroll
  for (int p = 0; p < 3; ++p) {
    const uint2 u = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
    *reinterpret_cast<uint2*>(at + p * kPart) = u;
    if (p < 2) v = make_float4(v.x - bf16_lo(u.x), v.y - bf16_hi(u.x), v.z - bf16_lo(u.y), v.w - bf16_hi(u.y));
  }
}
// Two values to their fp16 parts.
__device__ __forceinline__ void fp16_parts(float a, float b, uint32_t& hi, uint32_t& lo) {
  hi = hf2(a, b);
  const float2 h = __half22float2(reinterpret_cast<const __half2&>(hi));
  lo = hf2(a - h.x, b - h.y);
}

// Instruction descriptor of kind::f16 with fp32 accumulation: fp16 operands (type code 0)
// instead of bf16 ones (1).
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, bool a_mn, bool b_mn) {
  return idesc_bf16_f32(M, N, a_mn, b_mn) & ~((1u << 7) | (1u << 10));
}

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
// All threads wait for the products committed to `bar`; false where they did not end in time.
__device__ __forceinline__ bool all_wait(uint64_t* bar, uint32_t parity, int* err) {
  const int ok = threadIdx.x == 0 ? mbar_wait(bar, parity, err) : 1;
  const bool all = __syncthreads_and(ok);
  tc_fence_after();
  return all;
}
// This thread's 32 columns from `col` on of its row: warps w and w + 4 have rows 32 (w % 4) + lane.
__device__ __forceinline__ void tmem_row32(uint32_t base, int col, float (&v)[32]) {
  const uint32_t lanes = ((threadIdx.x >> 5) & 3) * 32;
  tmem_ld32(base + (lanes << 16) + col, v);
}
__device__ __forceinline__ int my_row() { return ((threadIdx.x >> 5) & 3) * 32 + (threadIdx.x & 31); }
__device__ __forceinline__ int my_half() { return threadIdx.x >> 7; }

// ------------------------------------------------------------------ gram
constexpr int kGramStages = 2, kGramSmem = kGramStages * 3 * kPart + 1024;
constexpr int kGramCols = 256;

__device__ __forceinline__ uint8_t* aligned_smem(uint8_t* p) {
  return p + ((1024 - (smem_u32(p) & 1023)) & 1023);
}

__global__ void __launch_bounds__(kThreads, 2) muon_gram_kernel(const __grid_constant__ MuonTable tab) {
  extern __shared__ uint8_t muon_smem[];
  __shared__ uint64_t done[kGramStages];
  __shared__ uint32_t slot;
  uint8_t* sm = aligned_smem(muon_smem);
  const Place pl = place_of(tab, blockIdx.x);
  const MuonTensor& t = *pl.t;
  const bool aligned = quads_aligned(t), tall = t.tall;
  Loads ld;
  load_chunk(pl, pl.c0, aligned, true, ld);
  if (threadIdx.x == 0) {
    for (int i = 0; i < kGramStages; ++i) mbar_init(&done[i], 1);
    fence_mbar_init();
  }
  const uint32_t acc = tmem_open(&slot, kGramCols);
  const float gs = tab.gs ? *tab.gs : 1.f;
  bool ok = true;
  for (int c = pl.c0; c < pl.c1; ++c) {
    const int k = c - pl.c0, st = k % kGramStages;
    uint8_t* part = sm + st * 3 * kPart;
    if (k >= kGramStages && !(ok = all_wait(&done[st], (k / kGramStages - 1) & 1, tab.err))) break;
#pragma unroll
    for (int i = 0; i < kQuads; ++i) {
      const Quad q(tall, i);
      const float4 g = scale4(widen(ld.g[i], aligned ? t.g_dtype : MOE_LORA_F32), gs);
      const float4 m = mix4(tab.mu, widen(ld.m[i], MOE_LORA_F32), tab.nu, g);
      store_m(pl, c, aligned, i, m);
      put_bf16_parts(part + quad_at(tall, q), tab.nesterov ? mix4(tab.mu, m, tab.nu, g) : m);
    }
    if (c + 1 < pl.c1) load_chunk(pl, c + 1, aligned, true, ld);
    fence_proxy_async_smem();
    __syncthreads();
    if (threadIdx.x == 0) {
      tc_fence_after();
      const uint32_t h = smem_u32(part), m = h + kPart, l = m + kPart;
      const uint32_t id = idesc_bf16_f32(kTile, kTile, tall, tall);
#pragma unroll
      for (int kk = 0; kk < kChunk / 16; ++kk) {
        const uint32_t at = tall ? kk * 2048 : kk * 32, lbo = tall ? kPart / 2 : 16;
        const uint64_t dh = sw128_desc(h + at, lbo, 1024), dm = sw128_desc(m + at, lbo, 1024), dl = sw128_desc(l + at, lbo, 1024);
        const uint32_t more = k > 0 || kk > 0;
        mma_bf16(acc, dh, dh, id, more);
        mma_bf16(acc, dm, dm, id, 1);
        mma_bf16(acc + kTile, dh, dm, id, more);
        mma_bf16(acc + kTile, dh, dl, id, 1);
      }
      mma_commit(&done[st]);
    }
  }
  const int last = pl.c1 - pl.c0 - 1;
  if (ok) ok = all_wait(&done[last % kGramStages], (last / kGramStages) & 1, tab.err);
  // (hh + mm) / 2 + h(m + l): this and its transpose are added where it is read
  float* out = tab.gram + (int64_t)blockIdx.x * kTile * kTile + my_row() * kTile;
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const int col = my_half() * 64 + b * 32;
    float v[32], w[32];
    tmem_row32(acc, col, v);
    tmem_row32(acc + kTile, col, w);
#pragma unroll
    for (int i = 0; i < 32; i += 4)
      *reinterpret_cast<float4*>(out + col + i) = make_float4(0.5f * v[i] + w[i], 0.5f * v[i + 1] + w[i + 1], 0.5f * v[i + 2] + w[i + 2], 0.5f * v[i + 3] + w[i + 3]);
  }
  tmem_close(acc, kGramCols);
}

// ------------------------------------------------------------------ poly
// A block per tile.  A thread has half a row of each square matrix; they pass through
// shared memory as operands (fp16 parts of scaled values, zero outside the matrices' own
// blocks).
constexpr int kPolySmem = 3 * kPoly + 1024, kPolyCols = 256;

struct Block {  // columns [lo, hi) of this thread's row that belong to its matrix
  int lo, hi;
  __device__ __forceinline__ bool has(int col) const { return col >= lo && col < hi; }
};
// Writes this thread's half row, times `scale`, as fp16 parts of a square tile: two halves of 64
// columns, then the lower parts.
__device__ __forceinline__ void put_half_row(uint8_t* tile, const float (&v)[64], float scale) {
  const int r = my_row();
  uint8_t* at = tile + my_half() * kPart + r * 128;
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) fp16_parts(v[8 * u + 2 * i] * scale, v[8 * u + 2 * i + 1] * scale, hi[i], lo[i]);
    const int sw = (u ^ (r & 7)) << 4;
    *reinterpret_cast<uint4*>(at + sw) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(at + kTileBytes + sw) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
}
// D = A B^T of square tiles (both fp16 parts; the product of the lower parts is below fp32's rounding).
__device__ __forceinline__ void square_product(uint32_t d, uint32_t a, uint32_t b) {
  const uint32_t id = idesc_f16_f32(kTile, kTile, false, false);
#pragma unroll
  for (int p = 0; p < 3; ++p) {
    const uint32_t pa = a + (p == 2 ? kTileBytes : 0), pb = b + (p == 1 ? kTileBytes : 0);
#pragma unroll
    for (int kk = 0; kk < kTile / 16; ++kk) {
      const uint32_t at = kk / 4 * kPart + kk % 4 * 32;
      mma_bf16(d, sw128_desc(pa + at, 16, 1024), sw128_desc(pb + at, 16, 1024), id, p > 0 || kk > 0);
    }
  }
}
// This thread's half row of a product, times f, zero outside its block.
__device__ __forceinline__ void get_half_row(uint32_t d, const Block& blk, float f, float (&v)[64]) {
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    float w[32];
    tmem_row32(d, my_half() * 64 + b * 32, w);
#pragma unroll
    for (int i = 0; i < 32; ++i) v[b * 32 + i] = blk.has(my_half() * 64 + b * 32 + i) ? w[i] * f : 0.f;
  }
}

// `first`: G is of the update itself, whose norm is taken here.  Otherwise G is of X in the
// scratch, times kXScale^2.
__global__ void __launch_bounds__(kThreads, 1) muon_poly_kernel(const __grid_constant__ MuonTable tab, int steps, bool first) {
  extern __shared__ uint8_t muon_smem[];
  __shared__ uint64_t done;
  __shared__ uint32_t slot;
  __shared__ float diag[kTile];
  uint8_t* sm = aligned_smem(muon_smem);
  uint8_t *qt = sm, *gt = sm + kPoly, *pt = sm + 2 * kPoly;
  const int64_t tile = blockIdx.x;
  int ti = 0;
  while (ti + 1 < tab.n && tile >= tab.t[ti + 1].tile0) ++ti;
  const MuonTensor& t = tab.t[ti];
  const int rows = (int)min((int64_t)t.per, t.batch - (tile - t.tile0) * t.per) * t.s;
  const int row = my_row(), half = my_half();
  const Block blk{row < rows ? row / t.s * t.s : 0, row < rows ? row / t.s * t.s + t.s : 0};
  if (threadIdx.x == 0) {
    mbar_init(&done, 1);
    fence_mbar_init();
  }
  const uint32_t acc = tmem_open(&slot, kPolyCols);
  // G: the pieces' partial sums in order, each with its transpose
  float g[64];
#pragma unroll
  for (int i = 0; i < 64; ++i) g[i] = 0.f;
  const float* in = tab.gram + (t.piece0 + (tile - t.tile0) * t.pieces) * kTile * kTile;
  for (int p = 0; p < t.pieces; ++p, in += kTile * kTile) {
    const float* r = in + row * kTile + half * 64;
    const float* c = in + (int64_t)half * 64 * kTile + row;
#pragma unroll
    for (int i = 0; i < 64; i += 4) {
      const float4 u = *reinterpret_cast<const float4*>(r + i);
      g[i] += u.x + c[i * kTile];
      g[i + 1] += u.y + c[(i + 1) * kTile];
      g[i + 2] += u.z + c[(i + 2) * kTile];
      g[i + 3] += u.w + c[(i + 3) * kTile];
    }
  }
#pragma unroll
  for (int i = 0; i < 64; ++i)
    if (!blk.has(half * 64 + i)) g[i] = 0.f;
  float unit = 1.f / (kXScale * kXScale);  // X in the scratch is scaled
  if (first) {
#pragma unroll
    for (int i = 0; i < 64; ++i)
      if (half * 64 + i == row) diag[row] = g[i];
    __syncthreads();
    float n2 = 0.f;
    for (int i = blk.lo; i < blk.hi; ++i) n2 += diag[i];
    // a norm whose square fp32 does not hold: 0, or not finite, which is passed on as NaN
    const bool fine = n2 < INFINITY;
    const float norm = fine ? sqrtf(n2) : 0.f, inv = 1.f / (norm + tab.eps);
    // X = u / (norm + eps) = (u * up) * down, up a power of two that makes the matrix's norm 2^9 to 2^10
    float up = 0.f;
    if (norm > 0.f) up = ldexpf(1.f, 10 - (ilogbf(norm) + 1));
    unit = norm > 0.f ? inv * inv : 0.f;
    if (half == 0) {
      tab.norm[tile * 2 * kTile + row] = up;
      tab.norm[tile * 2 * kTile + kTile + row] = !fine ? NAN : norm > 0.f ? inv / up : 0.f;
    }
    if (!fine)
#pragma unroll
      for (int i = 0; i < 64; ++i) g[i] = 0.f;
  }
#pragma unroll
  for (int i = 0; i < 64; ++i) g[i] *= unit;
  uint32_t phase = 0;
  bool ok = true;
  // Runs products issued by one thread; operands are in shared memory.
  const auto products = [&](auto issue) {
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0) {
      tc_fence_after();
      issue();
      mma_commit(&done);
    }
    ok = all_wait(&done, phase, tab.err) && ok;
    phase ^= 1;
  };
  const uint32_t qa = smem_u32(qt), ga = smem_u32(gt), pa = smem_u32(pt);
  float v[64];
#pragma unroll
  for (int i = 0; i < 64; ++i) v[i] = blk.has(half * 64 + i) && half * 64 + i == row ? 1.f : 0.f;
  if (steps == 0) put_half_row(pt, v, kQScale);
  for (int k = 0; k < steps && ok; ++k) {
    put_half_row(gt, g, kGScale);
    products([&] { square_product(acc, ga, ga); });
    get_half_row(acc, blk, tab.c / (kGScale * kGScale), v);
#pragma unroll
    for (int i = 0; i < 64; ++i) {
      v[i] += tab.b * g[i];
      if (half * 64 + i == row && blk.has(row)) v[i] += tab.a;
    }
    put_half_row(qt, v, kQScale);
    if (k == 0) put_half_row(pt, v, kQScale);
    const bool last = k == steps - 1;
    if (last && k == 0) break;
    products([&] {
      if (!last) square_product(acc, qa, ga);
      if (k > 0) square_product(acc + kTile, qa, pa);
    });
    if (k > 0) {
      get_half_row(acc + kTile, blk, 1.f / (kQScale * kQScale), v);
      put_half_row(pt, v, kQScale);
    }
    if (last) break;
    get_half_row(acc, blk, 1.f / (kQScale * kGScale), v);
    put_half_row(gt, v, kGScale);
    products([&] { square_product(acc, qa, ga); });
    get_half_row(acc, blk, 1.f / (kQScale * kGScale), g);
  }
  __syncthreads();
  uint4* out = reinterpret_cast<uint4*>(tab.poly + tile * kPoly);
  for (int i = threadIdx.x; i < kPoly / 16; i += kThreads) out[i] = reinterpret_cast<const uint4*>(pt)[i];
  tmem_close(acc, kPolyCols);
}

// ------------------------------------------------------------------ apply and update
// D [128 x 64] = P X of a chunk.  X as two fp16 parts: rows of 64 long places (a short side
// each), or two halves of 64 short places (a row per long place).
__device__ __forceinline__ void poly_product(uint32_t d, uint32_t p, uint32_t x, bool tall) {
  const uint32_t id = idesc_f16_f32(kTile, kChunk, false, !tall);
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    const uint32_t a = p + (q == 2 ? kTileBytes : 0), b = x + (q == 1 ? kPart : 0);
#pragma unroll
    for (int kk = 0; kk < kTile / 16; ++kk) {
      const uint64_t ad = sw128_desc(a + kk / 4 * kPart + kk % 4 * 32, 16, 1024);
      const uint64_t bd = tall ? sw128_desc(b + kk / 4 * (kPart / 2) + kk % 4 * 32, 16, 1024) : sw128_desc(b + kk * 2048, 8192, 1024);
      mma_bf16(d, ad, bd, id, q > 0 || kk > 0);
    }
  }
}
__device__ __forceinline__ void copy_async(uint8_t* dst, const uint8_t* src, int bytes) {
  for (int i = threadIdx.x * 16; i < bytes; i += kThreads * 16) async_copy16(dst + i, src + i);
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
  const int64_t piece = tab.pieces - 1 - blockIdx.x;  // what the launch before it wrote last may still be in L2
  const Place pl = place_of(tab, piece);
  const MuonTensor& t = *pl.t;
  const bool aligned = quads_aligned(t), tall = t.tall, with_g = tab.nesterov;
  copy_async(pt, tab.poly + pl.tile * kPoly, kPoly);
  Loads ld;
  load_chunk(pl, pl.c0, aligned, with_g, ld);
  if (threadIdx.x == 0) {
    mbar_init(&done[0], 1);
    mbar_init(&done[1], 1);
    fence_mbar_init();
  }
  const float* norm = tab.norm + pl.tile * 2 * kTile;
  if (threadIdx.x < kTile) row_up[threadIdx.x] = norm[threadIdx.x];
  // P's scale, and the factor that makes the products X
  const float down = norm[kTile + my_row()] == norm[kTile + my_row()] ? norm[kTile + my_row()] * (kXScale / kQScale) : 0.f;
  const uint32_t acc = tmem_open(&slot, kApplyCols);
  const uint32_t gram = acc + 64;
  const float gs = tab.gs ? *tab.gs : 1.f;
  async_wait<0>();
  bool ok = true;
  for (int c = pl.c0; c < pl.c1; ++c) {
    const int k = c - pl.c0;
    if (k > 0 && !(ok = all_wait(&done[1], (k - 1) & 1, tab.err))) break;
#pragma unroll
    for (int i = 0; i < kQuads; ++i) {
      const Quad q(tall, i);
      float4 u = widen(ld.m[i], MOE_LORA_F32);
      if (with_g) u = mix4(tab.mu, u, tab.nu, scale4(widen(ld.g[i], aligned ? t.g_dtype : MOE_LORA_F32), gs));
      float f[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) f[e] = row_up[q.row + (tall ? e : 0)];
      // matrices without a norm (0, or not finite) take no part
      u = make_float4(f[0] > 0.f ? u.x * f[0] : 0.f, f[1] > 0.f ? u.y * f[1] : 0.f, f[2] > 0.f ? u.z * f[2] : 0.f, f[3] > 0.f ? u.w * f[3] : 0.f);
      uint2 hi, lo;
      fp16_parts(u.x, u.y, hi.x, lo.x);
      fp16_parts(u.z, u.w, hi.y, lo.y);
      uint8_t* at = xt + quad_at(tall, q);
      *reinterpret_cast<uint2*>(at) = hi;
      *reinterpret_cast<uint2*>(at + kPart) = lo;
    }
    fence_proxy_async_smem();
    __syncthreads();
    if (threadIdx.x == 0) {
      tc_fence_after();
      poly_product(acc, smem_u32(pt), smem_u32(xt), tall);
      mma_commit(&done[0]);
    }
    if (c + 1 < pl.c1) load_chunk(pl, c + 1, aligned, with_g, ld);
    if (!(ok = all_wait(&done[0], k & 1, tab.err))) break;
    // rows of 64 long places from here on: half a row each, to shared memory and to the scratch
    {
      float v[32];
      tmem_row32(acc, my_half() * 32, v);
      const int r = my_row();
      uint8_t* img = tab.x + (pl.image + k) * (int64_t)kImage;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        uint4 hi, lo;
        fp16_parts(v[8 * u] * down, v[8 * u + 1] * down, hi.x, lo.x);
        fp16_parts(v[8 * u + 2] * down, v[8 * u + 3] * down, hi.y, lo.y);
        fp16_parts(v[8 * u + 4] * down, v[8 * u + 5] * down, hi.z, lo.z);
        fp16_parts(v[8 * u + 6] * down, v[8 * u + 7] * down, hi.w, lo.w);
        const int at = r * 128 + (((my_half() * 4 + u) ^ (r & 7)) << 4);
        *reinterpret_cast<uint4*>(xt + at) = hi;
        *reinterpret_cast<uint4*>(xt + kPart + at) = lo;
        *reinterpret_cast<uint4*>(img + at) = hi;
        *reinterpret_cast<uint4*>(img + kPart + at) = lo;
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
        mma_bf16(gram, dh, dh, id, k > 0 || kk > 0);
        mma_bf16(gram, dh, dl, id, 1);
        mma_bf16(gram, dl, dh, id, 1);
      }
      mma_commit(&done[1]);
    }
  }
  const int last = pl.c1 - pl.c0 - 1;
  if (ok) all_wait(&done[1], last & 1, tab.err);
  float* out = tab.gram + piece * kTile * kTile + my_row() * kTile;
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const int col = my_half() * 64 + b * 32;
    float v[32];
    tmem_row32(gram, col, v);
#pragma unroll
    for (int i = 0; i < 32; i += 4)
      *reinterpret_cast<float4*>(out + col + i) = make_float4(0.5f * v[i], 0.5f * v[i + 1], 0.5f * v[i + 2], 0.5f * v[i + 3]);
  }
  tmem_close(acc, kApplyCols);
}

constexpr int kUpdateSmem = kPoly + kImage + 1024, kUpdateCols = 64;
constexpr int kPitch = 65;  // of the products in shared memory, fp32: rows and columns of a warp on different banks

// O = P X and the weights.
__global__ void __launch_bounds__(kThreads, 2) muon_update_kernel(const __grid_constant__ MuonTable tab) {
  extern __shared__ uint8_t muon_smem[];
  __shared__ uint64_t done;
  __shared__ uint32_t slot;
  uint8_t* sm = aligned_smem(muon_smem);
  uint8_t *pt = sm, *xt = sm + kPoly;
  const Place pl = place_of(tab, blockIdx.x);
  const MuonTensor& t = *pl.t;
  const bool aligned = quads_aligned(t), tall = t.tall;
  copy_async(pt, tab.poly + pl.tile * kPoly, kPoly);
  copy_async(xt, tab.x + pl.image * (int64_t)kImage, kImage);
  if (threadIdx.x == 0) {
    mbar_init(&done, 1);
    fence_mbar_init();
  }
  const float factor = tab.norm[pl.tile * 2 * kTile + kTile + my_row()];
  // NaN for a matrix whose norm is not finite
  const float f = (factor == factor ? 1.f : factor) * (1.f / (kXScale * kQScale));
  const uint32_t acc = tmem_open(&slot, kUpdateCols);
  const int64_t base = pl.first * t.s * t.L;
  const int wd = t.master ? MOE_LORA_F32 : t.p_dtype;
  const void* wp = t.master ? static_cast<const void*>(t.master) : t.p;
  for (int c = pl.c0; c < pl.c1; ++c) {
    async_wait<0>();
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0) {
      tc_fence_after();
      poly_product(acc, smem_u32(pt), smem_u32(xt), false);
      mma_commit(&done);
    }
    uint4 w[kQuads];
    if (aligned)
#pragma unroll
      for (int i = 0; i < kQuads; ++i) {
        const Quad q(tall, i);
        const int l = c * kChunk + q.col;
        if (q.row < pl.rows && l < t.L) w[i] = ld_quad(wp, wd, base + offset_of(t, q.row, l));
      }
    if (!all_wait(&done, (c - pl.c0) & 1, tab.err)) break;
    // the products change threads through shared memory, where X was
    float v[32];
    tmem_row32(acc, my_half() * 32, v);
    float* o = reinterpret_cast<float*>(xt);
#pragma unroll
    for (int half = 0; half < 2; ++half) {  // 64 rows at a time: kPitch * 128 floats are more than X's place
      if (my_row() / 64 == half)
#pragma unroll
        for (int i = 0; i < 32; ++i) o[(my_row() % 64) * kPitch + my_half() * 32 + i] = v[i] * f;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kQuads; ++i) {
        const Quad q(tall, i);
        const int l = c * kChunk + q.col;
        if (q.row / 64 != half) continue;
        float x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = o[(q.row % 64 + (tall ? e : 0)) * kPitch + q.col + (tall ? 0 : e)];
        if (aligned) {
          if (q.row < pl.rows && l < t.L) {
            const int64_t at = base + offset_of(t, q.row, l);
            float4 u = widen(w[i], wd);
            u = make_float4(u.x * t.decay - t.step * x[0], u.y * t.decay - t.step * x[1], u.z * t.decay - t.step * x[2], u.w * t.decay - t.step * x[3]);
            if (t.master) *reinterpret_cast<float4*>(t.master + at) = u;
            st_quad(t.p, t.p_dtype, at, u);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int r = q.row + (tall ? e : 0), k = l + (tall ? 0 : e);
            if (r < pl.rows && k < t.L) {
              const int64_t at = base + offset_of(t, r, k);
              const float u = ld_one(wp, wd, at) * t.decay - t.step * x[e];
              if (t.master) t.master[at] = u;
              st_one(t.p, t.p_dtype, at, u);
            }
          }
        }
      }
      __syncthreads();
    }
    if (c + 1 < pl.c1) copy_async(xt, tab.x + (pl.image + c + 1 - pl.c0) * (int64_t)kImage, kImage);
  }
  async_wait<0>();
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
// Chunks of a piece, from all tensors of a launch: enough pieces for two blocks on each of
// 152 SMs, and at most sixteen chunks (more than that adds up over a hundred products into one
// accumulator, whose additions the tensor cores cut off rather than round).
int piece_of(const moe_lora_muon_tensor* t, int n) {
  int64_t all = 0;
  for (int i = 0; i < n; ++i) all += shape_of(t[i]).tiles * shape_of(t[i]).chunks;
  return (int)std::min<int64_t>(16, std::max<int64_t>(1, (all + 303) / 304));
}
struct Layout {
  size_t err, norm, poly, gram, x, total;
  int piece;
  int64_t tiles, pieces;
};
Layout layout_of(const moe_lora_muon_tensor* t, int n) {
  Layout l = {};
  l.piece = piece_of(t, n);
  for (int i = 0; i < n; ++i) {
    const Shape h = shape_of(t[i]);
    l.tiles += h.tiles;
    l.pieces += h.tiles * ((h.chunks + l.piece - 1) / l.piece);
  }
  size_t o = 0;
  const auto take = [&](size_t bytes) { const size_t at = o; o = align_up(o + bytes, 256); return at; };
  l.err = take(16);
  l.norm = take(sizeof(float) * 2 * kTile * l.tiles);
  l.poly = take((size_t)kPoly * l.tiles);
  l.gram = take(sizeof(float) * kTile * kTile * l.pieces);
  l.x = take((size_t)kImage * l.pieces * l.piece);
  l.total = o;
  return l;
}

template <class K, class... A>
int launch_muon(int slot, K kernel, int64_t grid, size_t smem, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  prof_begin(slot, s);
  const cudaError_t e = launch_allowed(cfg, false, kernel, args...);
  prof_end(slot, s);
  return e == cudaSuccess ? MOE_LORA_OK : MOE_LORA_ERR_CUDA;
}

// The five launches over up to kMaxTensors tensors.
int run_muon(const moe_lora_muon* o, const moe_lora_muon_tensor* in, int n, uint8_t* ws, cudaStream_t s) {
  const Layout l = layout_of(in, n);
  if (l.tiles == 0) return MOE_LORA_OK;
  MuonTable tab;
  tab.n = 0;
  tab.piece = l.piece;
  tab.tiles = l.tiles;
  tab.pieces = l.pieces;
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
  int64_t tile = 0, piece = 0;
  for (int i = 0; i < n; ++i) {
    const Shape h = shape_of(in[i]);
    if (h.tiles == 0) continue;
    MuonTensor& t = tab.t[tab.n++];
    t = MuonTensor{in[i].p, in[i].master, in[i].g, in[i].m, in[i].batch, tile, piece, h.s, h.L, in[i].rows > in[i].cols, h.per,
                   (int)((h.chunks + l.piece - 1) / l.piece), in[i].p_dtype, in[i].g_dtype,
                   (float)(1 - in[i].lr * in[i].weight_decay), (float)(in[i].lr * in[i].scale)};
    tile += h.tiles;
    piece += h.tiles * t.pieces;
  }
  const int first = std::min(kFirstSteps, o->steps > 3 ? 2 : 1);
  int rc;
  if ((rc = launch_muon(K_MUON_GRAM, muon_gram_kernel, l.pieces, kGramSmem, s, tab)) ||
      (rc = launch_muon(K_MUON_POLY, muon_poly_kernel, l.tiles, kPolySmem, s, tab, first, true)) ||
      (rc = launch_muon(K_MUON_APPLY, muon_apply_kernel, l.pieces, kApplySmem, s, tab)) ||
      (rc = launch_muon(K_MUON_POLY, muon_poly_kernel, l.tiles, kPolySmem, s, tab, o->steps - first, false)) ||
      (rc = launch_muon(K_MUON_UPDATE, muon_update_kernel, l.pieces, kUpdateSmem, s, tab)))
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
  for (int i = 0; i < n; i += kMaxTensors) {
    const int64_t pieces = layout_of(tensors + i, std::min(kMaxTensors, n - i)).pieces;
    if (pieces > ((int64_t)1 << 31) - 1) return MOE_LORA_ERR_DIMS;
  }
  int sms;
  if ((rc = device_sms(&sms))) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  for (int i = 0; i < n; i += kMaxTensors)
    if ((rc = run_muon(o, tensors + i, std::min(kMaxTensors, n - i), static_cast<uint8_t*>(scratch), s))) return rc;
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
