// AdamW over many tensors in one launch, with moments in 32 or in 8 bits (definitions
// in include/moe_lora.h).
//
// Every element is read and written once: 18 bytes with 8-bit moments, fp32 gradients
// and master weights and a bf16 copy (and 16 per block for its scales), 22 with 32-bit
// moments, bf16 weights and gradients.  HBM is the bound; with 8-bit moments the
// instructions are close behind (69 per element and lane; the square root and the code
// conversions are half of them), and lead where weights and gradients have 16 bits.
// Measured on one GB300: 203 M elements with 8-bit moments 539 us (6.8 TB/s, the measured
// copy bandwidth); 96 tensors of 38.6 M elements with 32-bit moments 130 us (96% of it);
// 11.5 M elements of 10 bytes each, 8-bit moments with bf16 weights alone, 32 us (53%).
#include <float.h>
#include <math.h>

#include <type_traits>

#include "common.cuh"
#include "element.cuh"
#include "launch.h"
#include "prof.h"

namespace moelora {

namespace {

constexpr int kAdamWarps = 8, kAdamThreads = 32 * kAdamWarps;
constexpr int kAdamBlock = 256;  // elements of a warp's step = of one scale of an 8-bit state
constexpr int kAdamChunk = kAdamWarps * kAdamBlock;
// Tensors per launch.  The table travels in the kernel's parameters (32 KB at most), so
// nothing is copied to the device ahead of the launch and a graph captures it.
constexpr int kAdamFew = 40, kAdamSome = 128, kAdamMany = 352;

struct AdamTensor {
  void* p;
  float* master;
  const void* g;
  void* m;
  void* v;
  float* ms;
  float* vs;
  int64_t numel;
  float decay, lr;  // 1 - lr * weight_decay, lr / (1 - beta1^t)
  int32_t p_dtype, g_dtype;
};
struct AdamHyper {
  float b1, c1, b2, c2, rbc2, eps;  // c = 1 - b; rbc2 = 1 / sqrt(1 - beta2^t)
  float minus0;                     // -0, see adam_pair
  const float* gs;
};
template <int kCap>
struct AdamTable {
  int n;
  AdamHyper h;
  int64_t base[kCap + 1];  // first chunk (kAdamWarps blocks) of each tensor
  AdamTensor t[kCap];
};
static_assert(sizeof(AdamTable<kAdamMany>) <= 32764, "kernel parameter limit");

// Eight consecutive elements of a 16- or 32-bit type as loaded, and widened.  Loading and
// widening are apart so that all of a step's loads are under way before the first is used.
struct Raw8 {
  uint4 a, b;
  __device__ __forceinline__ void load(const void* p, int dtype, int64_t i) {
    const char* q = static_cast<const char*>(p) + (dtype == MOE_LORA_F32 ? 4 : 2) * i;
    a = *reinterpret_cast<const uint4*>(q);
    if (dtype == MOE_LORA_F32) b = *reinterpret_cast<const uint4*>(q + 16);
  }
  // this lane's eight of a warp's 256 elements in shared memory, 32 lanes' 16 bytes to a row
  __device__ __forceinline__ void get(const uint4* row, int dtype) {
    const int lane = threadIdx.x & 31;
    if (dtype == MOE_LORA_F32) {
      a = row[2 * lane];
      b = row[2 * lane + 1];
    } else {
      a = row[lane];
    }
  }
  __device__ __forceinline__ void widen(int dtype, float (&f)[8]) const {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    if (dtype == MOE_LORA_F32) {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 t = dtype == MOE_LORA_BF16 ? Two<__nv_bfloat16>::get(w + i) : Two<__half>::get(w + i);
        f[2 * i] = t.x;
        f[2 * i + 1] = t.y;
      }
    }
  }
};
__device__ __forceinline__ void store8(void* p, int dtype, int64_t i, const float (&f)[8]) {
  uint32_t w[8];
  if (dtype == MOE_LORA_F32) {
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
    q[0] = make_float4(f[0], f[1], f[2], f[3]);
    q[1] = make_float4(f[4], f[5], f[6], f[7]);
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 t = make_float2(f[2 * j], f[2 * j + 1]);
    if (dtype == MOE_LORA_BF16)
      Two<__nv_bfloat16>::put(w + j, t);
    else
      Two<__half>::put(w + j, t);
  }
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ float ld_any(const void* p, int dtype, int64_t i) {
  return dtype == MOE_LORA_F32    ? static_cast<const float*>(p)[i]
         : dtype == MOE_LORA_BF16 ? to_f32(static_cast<const __nv_bfloat16*>(p)[i])
                                  : to_f32(static_cast<const __half*>(p)[i]);
}
__device__ __forceinline__ void st_any(void* p, int dtype, int64_t i, float v) {
  if (dtype == MOE_LORA_F32)
    static_cast<float*>(p)[i] = v;
  else if (dtype == MOE_LORA_BF16)
    static_cast<__nv_bfloat16*>(p)[i] = from_f32<__nv_bfloat16>(v);
  else
    static_cast<__half*>(p)[i] = from_f32<__half>(v);
}
// Two E4M3 codes (the low byte first) to fp32, exactly.
__device__ __forceinline__ float2 from_e4m3x2(uint32_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)c));
  return __half22float2(reinterpret_cast<const __half2&>(h));
}

// Scale of a block from its largest finite magnitude `top`: codes are of x * inv, values
// code * scale.
__device__ __forceinline__ void block_scale(float top, float& inv, float& scale) {
  const bool some = top >= 7.888609052210118e-31f;  // 2^-100
  inv = some ? __fmul_rn(__frcp_rn(top), 448.f) : 0.f;
  scale = some ? __fmul_rn(top, 1.0f / 448.0f) : 0.f;
}
__device__ __forceinline__ uint32_t warp_max(float v) {  // v >= 0 or NaN: ordered as its bits, NaN last
  return __reduce_max_sync(0xffffffffu, __float_as_uint(v));
}
// Codes of a warp's block (this lane's eight values) and its scale.  All values are as
// good as always finite: the largest magnitude, NaN above all, tells, and only a block
// with one that is not looks at its elements one by one, for its scale and for the NaN
// codes (the conversion would saturate an infinity).
__device__ __forceinline__ uint2 encode8(const float (&x)[8], float& scale) {
  float t = 0.f, inv;
#pragma unroll
  for (int i = 0; i < 8; i += 2)
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(t) : "f"(t), "f"(x[i]), "f"(x[i + 1]));
  uint32_t top = warp_max(t), nan[2] = {0, 0};
  if (top >= 0x7f800000u) {
    t = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (fabsf(x[i]) < INFINITY)
        t = fmaxf(t, fabsf(x[i]));
      else
        nan[i >> 2] |= 0x7fu << (8 * (i & 3));
    }
    top = warp_max(t);
  }
  block_scale(__uint_as_float(top), inv, scale);
  float2 q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) q[i] = mul2(make_float2(x[2 * i], x[2 * i + 1]), both(inv));
  return make_uint2(e4m3x2(q[0].x, q[0].y) | e4m3x2(q[1].x, q[1].y) << 16 | nan[0],
                    e4m3x2(q[2].x, q[2].y) | e4m3x2(q[3].x, q[3].y) << 16 | nan[1]);
}

// 1 / d to one unit in the last place, for d in [2^-126, 2^126] (0 above it)
__device__ __forceinline__ float rcp_fast(float d) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
  return r;
}

// Two elements: new moments (v as its root r too) and weights.  Every product and sum is
// rounded on its own, so that the moments, and with them the 8-bit codes, are the
// formula's in fp32 bit for bit.  The assembler fuses mul.f32x2 with add.f32x2 (seen in
// results); a product with -0 added, a value it does not know, it leaves alone, and the
// -0 changes nothing.  The quotient is a product with the fast reciprocal, to 2 units in
// the last place of the update (203 M elements with 8-bit moments: 539 us, with
// __fdividef 546 us, and the correctly rounded quotient was 59 us slower than that); its
// divisor lies between eps (2^-126 at least) and 2^126, the range that rcp_fast takes.
__device__ __forceinline__ void adam_pair(const AdamHyper& h, float decay, float lr, float2 g, float2& m, float2& v,
                                          float2& r, float2& w) {
  const auto mul = [&](float2 a, float2 b) { return fma2(a, b, both(h.minus0)); };
  m = add2(mul(both(h.b1), m), mul(both(h.c1), g));
  v = add2(mul(both(h.b2), v), mul(mul(both(h.c2), g), g));
  r = make_float2(__fsqrt_rn(v.x), __fsqrt_rn(v.y));
  const float2 d = add2(mul(r, both(h.rbc2)), both(h.eps));
  const float2 u = mul(m, make_float2(rcp_fast(d.x), rcp_fast(d.y)));
  w = add2(mul(w, both(decay)), mul(both(-lr), u));
}

// A block takes chunks of eight 256-element blocks of one tensor in turn, a warp one of
// the eight, a lane eight consecutive elements of it.  The tensor is the same for the
// whole block: its table entry is read through the uniform path.
//
// 8-bit moments: their arithmetic is as long as the memory takes, so a warp's next block is
// copied into the warp's own shared memory (two stages) while it works on this one.  The 32
// lanes copy 512 bytes side by side and pick up their own eight elements afterwards; with
// two copies of 16 bytes a lane, 32 bytes apart, 203 M elements took 810 us.  Measured so,
// and loaded when needed: 203 M elements with fp32 gradients and master weights 539 and
// 578 us, 11.5 M with fp16 gradients and bf16 weights alone 32.0 and 32.9 us.  Three blocks
// an SM: with four the 203 M elements took 633 us (the reads ahead of all of them get in
// each other's way in memory).  With the stores through shared memory as well: 548 us.
// 32-bit moments: loaded when needed, four blocks an SM (38.6 M elements 130 us; copied
// ahead 142 us).
constexpr int kAdamSlots = 5;  // 16 bytes a lane: gradient, weight (two each), moments
using AdamRing = Ring<2, kAdamSlots>;
template <bool kEight>
constexpr int kAdamPerSm = kEight ? 3 : 4;  // blocks
template <bool kEight>
constexpr size_t kAdamSmem = kEight ? ring_bytes<2, kAdamSlots>(kAdamThreads) : 0;
static_assert(kAdamSmem<true> <= 48 << 10, "no launch option asked for");

// The tensor of chunk c, at or after `ti` in the table.
template <int kCap>
__device__ __forceinline__ int adam_tensor(const AdamTable<kCap>& tab, int64_t c, int ti) {
  if (c < tab.base[ti + 1]) return ti;
  int lo = ti + 1, hi = tab.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (c >= tab.base[mid])
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}
// Starts the copy of a warp's block, from element e on, of which `left` are inside the
// tensor: all whole units of 16 bytes (8 of codes), and so all lanes' whole eights.
__device__ __forceinline__ void adam_fetch(const AdamRing& ring, int stage, const AdamTensor& t, int64_t e,
                                           int64_t left) {
  const int lane = threadIdx.x & 31;
  const auto vec = [&](const void* p, int dtype, int at) {
    if (dtype == MOE_LORA_F32) {
      const float* q = static_cast<const float*>(p) + e + lane * 4;
      if (lane * 4 + 4 <= left) async_copy16(ring.slot(stage, at), q);
      if (lane * 4 + 132 <= left) async_copy16(ring.slot(stage, at + 1), q + 128);
    } else if (lane * 8 + 8 <= left) {
      async_copy16(ring.slot(stage, at), static_cast<const uint16_t*>(p) + e + lane * 8);
    }
  };
  vec(t.g, t.g_dtype, 0);
  if (t.master)
    vec(t.master, MOE_LORA_F32, 2);
  else
    vec(t.p, t.p_dtype, 2);
  if (lane * 8 + 8 <= left) {
    uint2* q = reinterpret_cast<uint2*>(ring.slot(stage, 4));
    async_copy8(q, static_cast<const uint8_t*>(t.m) + e + lane * 8);
    async_copy8(q + 1, static_cast<const uint8_t*>(t.v) + e + lane * 8);
  }
}

template <bool kEight, int kCap>
__global__ void __launch_bounds__(kAdamThreads, kAdamPerSm<kEight>)
    adamw_kernel(const __grid_constant__ AdamTable<kCap> tab) {
  extern __shared__ uint4 adam_smem[];
  const AdamRing ring(adam_smem);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const AdamHyper& h = tab.h;
  const float gs = h.gs ? *h.gs : 1.0f;
  const int64_t end = tab.base[tab.n];
  int ti = 0, next = 0, stage = 0;  // tensor of this chunk and of the next
  float sm = 0.f, sv = 0.f, next_sm = 0.f, next_sv = 0.f;
  const auto ahead = [&](int64_t c, int st) {
    if (c < end) {
      next = adam_tensor(tab, c, next);
      const AdamTensor& t = tab.t[next];
      const int64_t blk = (c - tab.base[next]) * kAdamWarps + warp, e = blk * kAdamBlock;
      adam_fetch(ring, st, t, e, t.numel - e);
      if (e < t.numel) {
        next_sm = t.ms[blk];
        next_sv = t.vs[blk];
      }
    }
    async_commit();
  };
  if constexpr (kEight) ahead(blockIdx.x, 0);
  for (int64_t c = blockIdx.x; c < end; c += gridDim.x, stage ^= 1) {
    if constexpr (kEight) {
      ti = next;
      sm = next_sm;
      sv = next_sv;
      __syncwarp();  // all lanes have read the stage that is filled next
      ahead(c + gridDim.x, stage ^ 1);
      async_wait<1>();
      __syncwarp();
    } else {
      ti = adam_tensor(tab, c, ti);
    }
    const AdamTensor& t = tab.t[ti];
    const int64_t blk = (c - tab.base[ti]) * kAdamWarps + warp, i = blk * kAdamBlock + lane * 8;
    if (blk * kAdamBlock >= t.numel) continue;
    const bool whole = i + 8 <= t.numel;
    float g[8], m[8], v[8], w[8];
    if (whole) {
      Raw8 rg, rw;
      const int wd = t.master ? MOE_LORA_F32 : t.p_dtype;
      if constexpr (kEight) {
        rg.get(ring.slot(stage, 0) - lane, t.g_dtype);
        rw.get(ring.slot(stage, 2) - lane, wd);
        const uint4 q = *ring.slot(stage, 4);
        const uint32_t code[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          const float2 a = from_e4m3x2(code[j >> 2] >> (8 * (j & 3)));
          const float2 b = from_e4m3x2(code[2 + (j >> 2)] >> (8 * (j & 3)));
          m[j] = a.x;
          m[j + 1] = a.y;
          v[j] = b.x;
          v[j + 1] = b.y;
        }
        rg.widen(t.g_dtype, g);
        rw.widen(wd, w);
      } else {
        Raw8 rm, rv;
        rg.load(t.g, t.g_dtype, i);
        if (t.master)
          rw.load(t.master, MOE_LORA_F32, i);
        else
          rw.load(t.p, t.p_dtype, i);
        rm.load(t.m, MOE_LORA_F32, i);
        rv.load(t.v, MOE_LORA_F32, i);
        rg.widen(t.g_dtype, g);
        rw.widen(wd, w);
        rm.widen(MOE_LORA_F32, m);
        rv.widen(MOE_LORA_F32, v);
      }
    } else {  // the end of a tensor, element by element
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const bool in = i + j < t.numel;
        g[j] = in ? ld_any(t.g, t.g_dtype, i + j) : 0.f;
        w[j] = !in ? 0.f : t.master ? t.master[i + j] : ld_any(t.p, t.p_dtype, i + j);
        if (kEight) {
          m[j] = in ? from_e4m3x2(static_cast<const uint8_t*>(t.m)[i + j]).x : 0.f;
          v[j] = in ? from_e4m3x2(static_cast<const uint8_t*>(t.v)[i + j]).x : 0.f;
        } else {
          m[j] = in ? static_cast<const float*>(t.m)[i + j] : 0.f;
          v[j] = in ? static_cast<const float*>(t.v)[i + j] : 0.f;
        }
      }
    }
    float r[8];
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      float2 mj = make_float2(m[j], m[j + 1]), vj = make_float2(v[j], v[j + 1]), wj = make_float2(w[j], w[j + 1]), rj;
      if (kEight) {
        mj = mul2(mj, both(sm));
        vj = mul2(vj, both(sv));
        vj = mul2(vj, vj);
      }
      adam_pair(h, t.decay, t.lr, mul2(make_float2(g[j], g[j + 1]), both(gs)), mj, vj, rj, wj);
      m[j] = mj.x;
      m[j + 1] = mj.y;
      v[j] = vj.x;
      v[j + 1] = vj.y;
      w[j] = wj.x;
      w[j + 1] = wj.y;
      r[j] = rj.x;
      r[j + 1] = rj.y;
    }
    uint2 cm, cv;
    if (kEight) {
      cm = encode8(m, sm);
      cv = encode8(r, sv);
      if (lane == 0) {
        t.ms[blk] = sm;
        t.vs[blk] = sv;
      }
    }
    if (whole) {
      if (t.master) store8(t.master, MOE_LORA_F32, i, w);
      store8(t.p, t.p_dtype, i, w);
      if (kEight) {
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(t.m) + i) = cm;
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(t.v) + i) = cv;
      } else {
        store8(t.m, MOE_LORA_F32, i, m);
        store8(t.v, MOE_LORA_F32, i, v);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (i + j >= t.numel) break;
        if (t.master) t.master[i + j] = w[j];
        st_any(t.p, t.p_dtype, i + j, w[j]);
        if (kEight) {
          static_cast<uint8_t*>(t.m)[i + j] = (uint8_t)((j < 4 ? cm.x : cm.y) >> (8 * (j & 3)));
          static_cast<uint8_t*>(t.v)[i + j] = (uint8_t)((j < 4 ? cv.x : cv.y) >> (8 * (j & 3)));
        } else {
          static_cast<float*>(t.m)[i + j] = m[j];
          static_cast<float*>(t.v)[i + j] = v[j];
        }
      }
    }
  }
}

int check_tensor(const moe_lora_adamw_tensor& t) {
  if (t.numel < 0 || t.numel > (int64_t)1 << 40) return MOE_LORA_ERR_DIMS;
  if (!dtype_ok(t.p_dtype) || !dtype_ok(t.g_dtype) || (t.state != 0 && t.state != 1)) return MOE_LORA_ERR_UNSUPPORTED;
  if (t.master && t.p_dtype == MOE_LORA_F32) return MOE_LORA_ERR_UNSUPPORTED;
  if (!isfinite(t.lr) || !isfinite(t.weight_decay)) return MOE_LORA_ERR_DIMS;
  if (t.numel == 0) return MOE_LORA_OK;
  int rc;
  if ((rc = check_ptr(t.p)) || (rc = check_ptr(t.g)) || (rc = check_ptr(t.m)) || (rc = check_ptr(t.v)) ||
      (rc = check_opt(t.master)))
    return rc;
  if (t.state == 1) {  // the scales are read one by one, and may be slices of larger arrays
    if (!t.m_scale || !t.v_scale) return MOE_LORA_ERR_NULL;
    if ((reinterpret_cast<uintptr_t>(t.m_scale) | reinterpret_cast<uintptr_t>(t.v_scale)) & 3u)
      return MOE_LORA_ERR_ALIGN;
  }
  return MOE_LORA_OK;
}

template <bool kEight, int kCap>
int launch_adamw(const AdamTable<kCap>& tab, int sms, cudaStream_t s) {
  const int64_t want = tab.base[tab.n], most = (int64_t)kAdamPerSm<kEight> * sms;
  prof_begin(K_ADAMW, s);
  adamw_kernel<kEight, kCap><<<(int)(want < most ? want : most), kAdamThreads, kAdamSmem<kEight>, s>>>(tab);
  prof_end(K_ADAMW, s);
  return cudaGetLastError() == cudaSuccess ? MOE_LORA_OK : MOE_LORA_ERR_CUDA;
}

// Launches over the tensors of one state kind, kCap at a time.
template <bool kEight, int kCap>
int run_adamw(const AdamHyper& h, double bc1, const moe_lora_adamw_tensor* tensors, int n, int sms, cudaStream_t s) {
  AdamTable<kCap> tab;
  tab.h = h;
  tab.n = 0;
  tab.base[0] = 0;
  for (int i = 0; i < n; ++i) {
    const moe_lora_adamw_tensor& t = tensors[i];
    if ((t.state == 1) != kEight || t.numel == 0) continue;
    tab.t[tab.n] = AdamTensor{t.p, t.master, t.g, t.m, t.v, t.m_scale, t.v_scale, t.numel,
                              (float)(1 - t.lr * t.weight_decay), (float)(t.lr / bc1), t.p_dtype, t.g_dtype};
    tab.base[tab.n + 1] = tab.base[tab.n] + (t.numel + kAdamChunk - 1) / kAdamChunk;
    if (++tab.n == kCap) {
      const int rc = launch_adamw<kEight>(tab, sms, s);
      if (rc) return rc;
      tab.n = 0;
    }
  }
  return tab.n ? launch_adamw<kEight>(tab, sms, s) : MOE_LORA_OK;
}

}  // namespace

}  // namespace moelora

using namespace moelora;

extern "C" int moe_lora_adamw_step(const moe_lora_adamw* o, const moe_lora_adamw_tensor* tensors, int32_t n,
                                   void* stream) {
  if (!o || (n > 0 && !tensors)) return MOE_LORA_ERR_NULL;
  if (n < 0 || o->step < 1) return MOE_LORA_ERR_DIMS;
  if (!(o->beta1 >= 0 && o->beta1 < 1) || !(o->beta2 >= 0 && o->beta2 < 1)) return MOE_LORA_ERR_DIMS;
  // A subnormal eps would be outside the fast quotient's range: 0 / eps would be NaN.
  if (!((float)o->eps >= FLT_MIN) || !isfinite((float)o->eps)) return MOE_LORA_ERR_DIMS;
  int rc;
  if (reinterpret_cast<uintptr_t>(o->grad_scale) & 3u) return MOE_LORA_ERR_ALIGN;  // a scalar, often inside a buffer
  for (int i = 0; i < n; ++i)
    if ((rc = check_tensor(tensors[i]))) return rc;
  int sms;
  if ((rc = device_sms(&sms))) return rc;
  const double bc1 = 1 - pow(o->beta1, (double)o->step), bc2 = 1 - pow(o->beta2, (double)o->step);
  const AdamHyper h{(float)o->beta1, (float)(1 - o->beta1), (float)o->beta2, (float)(1 - o->beta2),
                    (float)(1 / sqrt(bc2)), (float)o->eps, -0.f, o->grad_scale};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const auto run = [&](auto eight) {
    return n <= kAdamFew    ? run_adamw<eight, kAdamFew>(h, bc1, tensors, n, sms, s)
           : n <= kAdamSome ? run_adamw<eight, kAdamSome>(h, bc1, tensors, n, sms, s)
                            : run_adamw<eight, kAdamMany>(h, bc1, tensors, n, sms, s);
  };
  if ((rc = run(std::false_type{}))) return rc;
  return run(std::true_type{});
}
