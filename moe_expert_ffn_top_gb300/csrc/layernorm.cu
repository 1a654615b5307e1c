// Layer norm over rows of [rows, n], forward and backward (definitions in
// include/moe_lora.h).
#include "element.cuh"
#include "launch.h"
#include "prof.h"

namespace moelora {

namespace {

constexpr int kNormThreads = 256;
constexpr int kNormParts = 64;  // row slices of the weight gradients' sums

// Sum over the block, the same value in every thread.
__device__ __forceinline__ float block_sum(float v, float* sm) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.f;
  for (int w = 0; w < (int)(blockDim.x >> 5); ++w) s += sm[w];
  return s;
}

template <class T, class W>
__global__ void __launch_bounds__(kNormThreads) norm_fwd_kernel(moe_lora_norm nm, const T* x, const W* gamma,
                                                                const W* beta, T* y, float* mean, float* rstd) {
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
      yr[c] = from_f32<T>(h * (gamma ? to_f32(gamma[c]) : 1.f) + (beta ? to_f32(beta[c]) : 0.f));
    }
    if (mean && threadIdx.x == 0) {
      mean[r] = mu;
      rstd[r] = rs;
    }
  }
}

template <class T, class W>
__global__ void __launch_bounds__(kNormThreads) norm_bwd_kernel(moe_lora_norm nm, const T* x, const W* gamma,
                                                                const float* mean, const float* rstd, const T* dy,
                                                                const T* dres, T* dx) {
  __shared__ float sm[32];
  const int n = nm.n;
  for (int64_t r = blockIdx.x; r < nm.rows; r += gridDim.x) {
    const T *xr = x + r * nm.ldx, *gr = dy + r * nm.ldy;
    const float mu = mean[r], rs = rstd[r];
    float a = 0.f, b = 0.f;
    for (int c = threadIdx.x; c < n; c += blockDim.x) {
      const float u = to_f32(gr[c]) * (gamma ? to_f32(gamma[c]) : 1.f);
      a += u;
      b += u * ((to_f32(xr[c]) - mu) * rs);
    }
    a = block_sum(a, sm) / n;
    b = block_sum(b, sm) / n;
    for (int c = threadIdx.x; c < n; c += blockDim.x) {
      const float u = to_f32(gr[c]) * (gamma ? to_f32(gamma[c]) : 1.f), h = (to_f32(xr[c]) - mu) * rs;
      const float d = rs * (u - a - h * b) + (dres ? to_f32(dres[r * nm.lddres + c]) : 0.f);
      dx[r * nm.lddx + c] = from_f32<T>(d);
    }
  }
}

// Partial sums of the weight gradients over one slice of the rows: part[slice][2][n].
template <class T>
__global__ void __launch_bounds__(kNormThreads) norm_part_kernel(moe_lora_norm nm, const T* x, const float* mean,
                                                                 const float* rstd, const T* dy, float* part) {
  const int n = nm.n, c = blockIdx.x * blockDim.x + threadIdx.x;
  if (c >= n) return;
  const int64_t per = (nm.rows + gridDim.y - 1) / gridDim.y, r0 = blockIdx.y * per;
  const int64_t r1 = r0 + per < nm.rows ? r0 + per : nm.rows;
  float dg = 0.f, db = 0.f;
  for (int64_t r = r0; r < r1; ++r) {
    const float d = to_f32(dy[r * nm.ldy + c]);
    dg += d * ((to_f32(x[r * nm.ldx + c]) - mean[r]) * rstd[r]);
    db += d;
  }
  part[(int64_t)blockIdx.y * 2 * n + c] = dg;
  part[(int64_t)blockIdx.y * 2 * n + n + c] = db;
}

__global__ void __launch_bounds__(kNormThreads) norm_wgrad_kernel(int n, int parts, const float* part, float* dgamma,
                                                                  float* dbeta) {
  const int c = blockIdx.x * blockDim.x + threadIdx.x;
  if (c >= n) return;
  float dg = 0.f, db = 0.f;
  for (int p = 0; p < parts; ++p) {
    dg += part[(int64_t)p * 2 * n + c];
    db += part[(int64_t)p * 2 * n + n + c];
  }
  if (dgamma) dgamma[c] = dg;
  if (dbeta) dbeta[c] = db;
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

template <class T, class W>
int run_fwd(const moe_lora_norm& nm, const void* x, const void* gamma, const void* beta, void* y, float* mean,
            float* rstd, int sms, cudaStream_t s) {
  const int grid = (int)(nm.rows < 8LL * sms ? nm.rows : 8LL * sms);
  prof_begin(K_NORM_FWD, s);
  norm_fwd_kernel<T, W><<<grid, kNormThreads, 0, s>>>(nm, (const T*)x, (const W*)gamma, (const W*)beta, (T*)y, mean,
                                                     rstd);
  prof_end(K_NORM_FWD, s);
  return cudaGetLastError() == cudaSuccess ? MOE_LORA_OK : MOE_LORA_ERR_CUDA;
}

template <class T, class W>
int run_bwd(const moe_lora_norm& nm, const void* x, const void* gamma, const float* mean, const float* rstd,
            const void* dy, const void* dres, void* dx, float* dgamma, float* dbeta, float* part, int sms,
            cudaStream_t s) {
  const int cols = (nm.n + kNormThreads - 1) / kNormThreads;
  if (dgamma || dbeta) {  // before dx, which may overwrite dy
    prof_begin(K_NORM_WGRAD, s);
    norm_part_kernel<T><<<dim3(cols, kNormParts), kNormThreads, 0, s>>>(nm, (const T*)x, mean, rstd, (const T*)dy,
                                                                        part);
    prof_end(K_NORM_WGRAD, s);
    prof_begin(K_NORM_WGRAD, s);
    norm_wgrad_kernel<<<cols, kNormThreads, 0, s>>>(nm.n, kNormParts, part, dgamma, dbeta);
    prof_end(K_NORM_WGRAD, s);
  }
  const int grid = (int)(nm.rows < 8LL * sms ? nm.rows : 8LL * sms);
  prof_begin(K_NORM_BWD, s);
  norm_bwd_kernel<T, W><<<grid, kNormThreads, 0, s>>>(nm, (const T*)x, (const W*)gamma, mean, rstd, (const T*)dy,
                                                     (const T*)dres, (T*)dx);
  prof_end(K_NORM_BWD, s);
  return cudaGetLastError() == cudaSuccess ? MOE_LORA_OK : MOE_LORA_ERR_CUDA;
}

// CALL<T, W>(args) for the element types of nm.
#define NORM_DISPATCH(CALL, ...)                                                                          \
  (nm.dtype == MOE_LORA_F32    ? NORM_DISPATCH_W(CALL, float, __VA_ARGS__)                                \
   : nm.dtype == MOE_LORA_BF16 ? NORM_DISPATCH_W(CALL, __nv_bfloat16, __VA_ARGS__)                        \
                               : NORM_DISPATCH_W(CALL, __half, __VA_ARGS__))
#define NORM_DISPATCH_W(CALL, T, ...)                                        \
  (nm.wdtype == MOE_LORA_F32    ? CALL<T, float>(__VA_ARGS__)                \
   : nm.wdtype == MOE_LORA_BF16 ? CALL<T, __nv_bfloat16>(__VA_ARGS__)        \
                                : CALL<T, __half>(__VA_ARGS__))

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
  return NORM_DISPATCH(run_fwd, nm, x, gamma, beta, y, mean, rstd, sms, s);
}

size_t moe_lora_layernorm_scratch_bytes(const moe_lora_norm* in) {
  moe_lora_norm nm;
  return check_norm(in, &nm) ? 0 : (size_t)kNormParts * 2 * nm.n * sizeof(float);
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
  if (wgrad) {
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
  return NORM_DISPATCH(run_bwd, nm, x, gamma, mean, rstd, dy, dres, dx, dgamma, dbeta, static_cast<float*>(scratch),
                       sms, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
