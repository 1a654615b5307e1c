// AdamW over many tensors in one launch, with moments in 32 or in 8 bits (definitions
// in include/moe_lora.h).
#include <math.h>

#include "common.cuh"
#include "element.cuh"
#include "launch.h"
#include "prof.h"

namespace moelora {

namespace {

constexpr int kAdamThreads = 256;
constexpr int kAdamBlock = 256;        // elements per warp step = per scale of an 8-bit state
constexpr int kAdamTensors = 352;      // per launch: the table travels in the kernel's parameters (32 KB at most)

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
  const float* gs;
};
struct AdamTable {
  int n;
  AdamHyper h;
  int64_t base[kAdamTensors + 1];  // first 256-element block of each tensor
  AdamTensor t[kAdamTensors];
};
static_assert(sizeof(AdamTable) <= 32764, "kernel parameter limit");

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
__device__ __forceinline__ float from_e4m3(uint8_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)c));
  return __half2float(__ushort_as_half((uint16_t)(h & 0xFFFFu)));
}

// Scale of a block from its largest finite magnitude `top`: codes are x * inv, values
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
// the NaN code where x is not finite (x - x is then NaN; the conversion alone would saturate an infinity)
__device__ __forceinline__ uint8_t to_e4m3(float x, float inv) {
  return (uint8_t)e4m3x2(__fadd_rn(__fmul_rn(x, inv), __fsub_rn(x, x)), 0.f);
}

template <bool kEight>
__global__ void __launch_bounds__(kAdamThreads) adamw_kernel(const __grid_constant__ AdamTable tab) {
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * (kAdamThreads / 32);
  const AdamHyper& h = tab.h;
  const float gs = h.gs ? *h.gs : 1.0f;
  int ti = 0;
  for (int64_t b = (int64_t)blockIdx.x * (kAdamThreads / 32) + (threadIdx.x >> 5); b < tab.base[tab.n]; b += warps) {
    while (b >= tab.base[ti + 1]) ++ti;
    const AdamTensor& t = tab.t[ti];
    const int64_t blk = b - tab.base[ti], i0 = blk * kAdamBlock + lane;
    float m[8], r[8];
    float tm = 0.f, tr = 0.f, sm = 0.f, sr = 0.f;
    if (kEight) {
      sm = t.ms[blk];
      sr = t.vs[blk];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t i = i0 + 32 * j;
      m[j] = r[j] = 0.f;
      if (i >= t.numel) continue;
      const float g = __fmul_rn(ld_any(t.g, t.g_dtype, i), gs);
      float m0, v0;
      if (kEight) {
        m0 = __fmul_rn(from_e4m3(static_cast<const uint8_t*>(t.m)[i]), sm);
        const float q = __fmul_rn(from_e4m3(static_cast<const uint8_t*>(t.v)[i]), sr);
        v0 = __fmul_rn(q, q);
      } else {
        m0 = static_cast<const float*>(t.m)[i];
        v0 = static_cast<const float*>(t.v)[i];
      }
      m0 = __fadd_rn(__fmul_rn(h.b1, m0), __fmul_rn(h.c1, g));
      v0 = __fadd_rn(__fmul_rn(h.b2, v0), __fmul_rn(__fmul_rn(h.c2, g), g));
      const float rt = __fsqrt_rn(v0);
      float w = t.master ? t.master[i] : ld_any(t.p, t.p_dtype, i);
      const float u = __fdiv_rn(m0, __fadd_rn(__fmul_rn(rt, h.rbc2), h.eps));
      w = __fsub_rn(__fmul_rn(w, t.decay), __fmul_rn(t.lr, u));
      if (t.master) t.master[i] = w;
      st_any(t.p, t.p_dtype, i, w);
      if (!kEight) {
        static_cast<float*>(t.m)[i] = m0;
        static_cast<float*>(t.v)[i] = v0;
      }
      m[j] = m0;
      r[j] = rt;
      tm = fmaxf(tm, finite_abs(m0));
      tr = fmaxf(tr, finite_abs(rt));
    }
    if (kEight) {
      float im, ir;
      block_scale(warp_top(tm), im, sm);
      block_scale(warp_top(tr), ir, sr);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int64_t i = i0 + 32 * j;
        if (i >= t.numel) continue;
        static_cast<uint8_t*>(t.m)[i] = to_e4m3(m[j], im);
        static_cast<uint8_t*>(t.v)[i] = to_e4m3(r[j], ir);
      }
      if (lane == 0) {
        t.ms[blk] = sm;
        t.vs[blk] = sr;
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
  if (t.state == 1 && ((rc = check_ptr(t.m_scale)) || (rc = check_ptr(t.v_scale)))) return rc;
  return MOE_LORA_OK;
}

// One launch over tab's tensors.
int launch_adamw(AdamTable& tab, int state, int sms, cudaStream_t s) {
  const int64_t blocks = tab.base[tab.n], per = kAdamThreads / 32;
  const int64_t want = (blocks + per - 1) / per;
  const int grid = (int)(want < 8LL * sms ? want : 8LL * sms);
  prof_begin(K_ADAMW, s);
  if (state)
    adamw_kernel<true><<<grid, kAdamThreads, 0, s>>>(tab);
  else
    adamw_kernel<false><<<grid, kAdamThreads, 0, s>>>(tab);
  prof_end(K_ADAMW, s);
  return cudaGetLastError() == cudaSuccess ? MOE_LORA_OK : MOE_LORA_ERR_CUDA;
}

}  // namespace

}  // namespace moelora

using namespace moelora;

extern "C" int moe_lora_adamw_step(const moe_lora_adamw* o, const moe_lora_adamw_tensor* tensors, int32_t n,
                                   void* stream) {
  if (!o || (n > 0 && !tensors)) return MOE_LORA_ERR_NULL;
  if (n < 0 || o->step < 1) return MOE_LORA_ERR_DIMS;
  if (!(o->beta1 >= 0 && o->beta1 < 1) || !(o->beta2 >= 0 && o->beta2 < 1) || !(o->eps > 0) || !isfinite(o->eps))
    return MOE_LORA_ERR_DIMS;
  int rc;
  if (reinterpret_cast<uintptr_t>(o->grad_scale) & 3u) return MOE_LORA_ERR_ALIGN;  // a scalar, often inside a buffer
  for (int i = 0; i < n; ++i)
    if ((rc = check_tensor(tensors[i]))) return rc;
  int sms;
  if ((rc = device_sms(&sms))) return rc;
  const double bc1 = 1 - pow(o->beta1, (double)o->step), bc2 = 1 - pow(o->beta2, (double)o->step);
  AdamTable tab;
  tab.h = AdamHyper{(float)o->beta1, (float)(1 - o->beta1), (float)o->beta2, (float)(1 - o->beta2),
                    (float)(1 / sqrt(bc2)), (float)o->eps, o->grad_scale};
  for (int state = 0; state < 2; ++state) {
    tab.n = 0;
    tab.base[0] = 0;
    for (int i = 0; i < n; ++i) {
      const moe_lora_adamw_tensor& t = tensors[i];
      if (t.state != state || t.numel == 0) continue;
      AdamTensor& d = tab.t[tab.n];
      d = AdamTensor{t.p, t.master, t.g, t.m, t.v, t.m_scale, t.v_scale, t.numel, (float)(1 - t.lr * t.weight_decay),
                     (float)(t.lr / bc1), t.p_dtype, t.g_dtype};
      tab.base[tab.n + 1] = tab.base[tab.n] + (t.numel + kAdamBlock - 1) / kAdamBlock;
      if (++tab.n == kAdamTensors) {
        if ((rc = launch_adamw(tab, state, sms, static_cast<cudaStream_t>(stream)))) return rc;
        tab.n = 0;
      }
    }
    if (tab.n && (rc = launch_adamw(tab, state, sms, static_cast<cudaStream_t>(stream)))) return rc;
  }
  return MOE_LORA_OK;
}
