// AdamW over many tensors in one launch, with moments in 32 or in 8 bits (definitions
// in include/moe_lora.h).
//
// Every element is read and written once: 18 bytes with 8-bit moments, fp32 gradients
// and master weights and a bf16 copy (and 16 per block for its scales), 22 with 32-bit
// moments, bf16 weights and gradients.  HBM is the bound, the instructions are
// close behind (about 60 per element and lane; the square root, the quotient and the
// code conversions are half of them).  Measured on one GB300: 203 M elements with 8-bit
// moments 570 us (6.4 TB/s, 95% of the measured copy bandwidth); 96 tensors of 38.6 M
// elements with 32-bit moments 130 us (96%).
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
__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a < INFINITY ? a : 0.f;
}
__device__ __forceinline__ float warp_top(float v) {  // v >= 0: ordered as its bits
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v)));
}
// Codes of a warp's block (this lane's eight values) and its scale.  x - x makes the NaN
// code of what is not finite; the conversion alone would saturate an infinity.
__device__ __forceinline__ uint2 encode8(const float (&x)[8], float& scale) {
  float top = 0.f, inv, q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) top = fmaxf(top, finite_abs(x[i]));
  block_scale(warp_top(top), inv, scale);
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = __fadd_rn(__fmul_rn(x[i], inv), __fsub_rn(x[i], x[i]));
  return make_uint2(e4m3x2(q[0], q[1]) | e4m3x2(q[2], q[3]) << 16, e4m3x2(q[4], q[5]) | e4m3x2(q[6], q[7]) << 16);
}

// Two elements: new moments (v as its root r too) and weights.  Every product and sum is
// rounded on its own, so that the moments, and with them the 8-bit codes, are the
// formula's in fp32 bit for bit.  The assembler fuses mul.f32x2 with add.f32x2 (seen in
// results); a product with -0 added, a value it does not know, it leaves alone, and the
// -0 changes nothing.  The quotient is
// the fast one, to 2 units in the last place of the update (203 M elements with 8-bit
// moments: 570 us against 629 us with the correctly rounded one); its divisor lies
// between eps (2^-126 at least) and 2^126, the range that the fast one takes.
__device__ __forceinline__ void adam_pair(const AdamHyper& h, float decay, float lr, float2 g, float2& m, float2& v,
                                          float2& r, float2& w) {
  const auto mul = [&](float2 a, float2 b) { return fma2(a, b, both(h.minus0)); };
  m = add2(mul(both(h.b1), m), mul(both(h.c1), g));
  v = add2(mul(both(h.b2), v), mul(mul(both(h.c2), g), g));
  r = make_float2(__fsqrt_rn(v.x), __fsqrt_rn(v.y));
  const float2 d = add2(mul(r, both(h.rbc2)), both(h.eps));
  const float2 u = make_float2(__fdividef(m.x, d.x), __fdividef(m.y, d.y));
  w = add2(mul(w, both(decay)), mul(both(-lr), u));
}

// A block takes chunks of eight 256-element blocks of one tensor in turn, a warp one of
// the eight, a lane eight consecutive elements of it.  The tensor is the same for the
// whole block: its table entry is read through the uniform path.
template <bool kEight, int kCap>
__global__ void __launch_bounds__(kAdamThreads, 4) adamw_kernel(const __grid_constant__ AdamTable<kCap> tab) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const AdamHyper& h = tab.h;
  const float gs = h.gs ? *h.gs : 1.0f;
  int ti = 0;
  for (int64_t c = blockIdx.x; c < tab.base[tab.n]; c += gridDim.x) {
    if (c >= tab.base[ti + 1]) {  // the tensor of chunk c, further on in the table
      int lo = ti + 1, hi = tab.n - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (c >= tab.base[mid])
          lo = mid;
        else
          hi = mid - 1;
      }
      ti = lo;
    }
    const AdamTensor& t = tab.t[ti];
    const int64_t blk = (c - tab.base[ti]) * kAdamWarps + warp, i = blk * kAdamBlock + lane * 8;
    if (blk * kAdamBlock >= t.numel) continue;
    const bool whole = i + 8 <= t.numel;
    float g[8], m[8], v[8], w[8], sm = 0.f, sv = 0.f;
    if (kEight) {
      sm = t.ms[blk];
      sv = t.vs[blk];
    }
    if (whole) {
      Raw8 rg, rw, rm, rv;
      rg.load(t.g, t.g_dtype, i);
      if (t.master)
        rw.load(t.master, MOE_LORA_F32, i);
      else
        rw.load(t.p, t.p_dtype, i);
      uint2 cm, cv;
      if (kEight) {
        cm = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(t.m) + i);
        cv = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(t.v) + i);
      } else {
        rm.load(t.m, MOE_LORA_F32, i);
        rv.load(t.v, MOE_LORA_F32, i);
      }
      rg.widen(t.g_dtype, g);
      rw.widen(t.master ? MOE_LORA_F32 : t.p_dtype, w);
      if (kEight) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 a = from_e4m3x2((j < 2 ? cm.x : cm.y) >> (16 * (j & 1)));
          const float2 c = from_e4m3x2((j < 2 ? cv.x : cv.y) >> (16 * (j & 1)));
          m[2 * j] = a.x;
          m[2 * j + 1] = a.y;
          v[2 * j] = c.x;
          v[2 * j + 1] = c.y;
        }
      } else {
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
  const auto kernel = adamw_kernel<kEight, kCap>;
  int per = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, kAdamThreads, 0) != cudaSuccess || per < 1)
    return MOE_LORA_ERR_CUDA;
  const int64_t want = tab.base[tab.n], most = (int64_t)per * sms;
  prof_begin(K_ADAMW, s);
  kernel<<<(int)(want < most ? want : most), kAdamThreads, 0, s>>>(tab);
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
