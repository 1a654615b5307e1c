// Balance loss of the routing step with the per-expert counts and its gradient to the
// logits (definitions in include/moe_lora.h).
//
// Every adapter's tokens are cut into chunks whose length depends on that adapter's
// token count alone; a chunk's sum of probabilities is one partial row, and the
// partials are added in chunk order.
#include <algorithm>

#include "common.cuh"
#include "element.cuh"
#include "launch.h"
#include "prof.h"

namespace moelora {

namespace {

constexpr int kBalThreads = 256;
constexpr int kBalMaxE = 1024;
constexpr int kBalMinChunk = 64;    // tokens
constexpr int kBalMaxChunks = 304;  // per adapter: two blocks per SM

struct BalTable {
  int n;
  int tok_off[kMaxAdapters + 1];
  int chunk0[kMaxAdapters + 1];  // first chunk of each adapter
  int chunk[kMaxAdapters];       // tokens per chunk
};

struct BalLayout {
  size_t err, live, part, total;
};
BalLayout bal_layout(const moe_lora_dims* d) {
  BalLayout L;
  const int64_t chunks =
      std::min<int64_t>((int64_t)d->A * kBalMaxChunks, d->T / kBalMinChunk + d->A);
  size_t o = 0;
  auto take = [&](size_t bytes) { size_t at = o; o = align_up(o + bytes, 256); return at; };
  L.err = take(16);
  L.live = take(sizeof(int) * d->A);
  L.part = take(sizeof(float) * chunks * d->E);
  L.total = o;
  return L;
}

int check_balance_dims(const moe_lora_dims* d) {
  const int rc = check_dims(d);
  if (rc) return rc;
  return d->E > kBalMaxE ? MOE_LORA_ERR_UNSUPPORTED : MOE_LORA_OK;
}

struct Chunk {
  int a, t0, t1;
};
__device__ __forceinline__ Chunk chunk_of(const BalTable& bt, int c) {
  Chunk ch;
  ch.a = 0;
  while (ch.a + 1 < bt.n && c >= bt.chunk0[ch.a + 1]) ++ch.a;
  ch.t0 = bt.tok_off[ch.a] + (c - bt.chunk0[ch.a]) * bt.chunk[ch.a];
  ch.t1 = min(ch.t0 + bt.chunk[ch.a], bt.tok_off[ch.a + 1]);
  return ch;
}

// counts and live tokens, added with integer atomics (exact in any order)
__global__ void __launch_bounds__(kBalThreads) balance_count_kernel(BalTable bt, const int32_t* ids, int k, int E,
                                                                    int* counts, int* live, int* err) {
  __shared__ int hist[kBalMaxE];
  const Chunk ch = chunk_of(bt, blockIdx.x);
  for (int e = threadIdx.x; e < E; e += blockDim.x) hist[e] = 0;
  __syncthreads();
  int nl = 0;
  for (int t = ch.t0 + threadIdx.x; t < ch.t1; t += blockDim.x) {
    bool any = false;
    for (int j = 0; j < k; ++j) {
      const int e = ids[(int64_t)t * k + j];
      if (e >= 0 && e < E) {
        atomicAdd(&hist[e], 1);
        any = true;
      } else if (e != -1) {
        atomicOr(err, MOE_LORA_DEV_BAD_ID);
      }
    }
    nl += any;
  }
  if (nl) atomicAdd(&live[ch.a], nl);
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += blockDim.x)
    if (hist[e]) atomicAdd(&counts[ch.a * E + e], hist[e]);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// one warp per token of the chunk
template <class T>
__global__ void __launch_bounds__(kBalThreads) balance_prob_kernel(BalTable bt, const T* logits, int64_t ld,
                                                                   const int32_t* ids, int k, int E, float coef,
                                                                   const float* dloss, const int* counts,
                                                                   const int* live, float* part, float* dlogits) {
  constexpr int kW = kBalThreads / 32;
  __shared__ float acc[kW][kBalMaxE];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const Chunk ch = chunk_of(bt, blockIdx.x);
  for (int e = lane; e < E; e += 32) acc[w][e] = 0.f;
  const int* cnt = counts + ch.a * E;
  int R = 0;
  for (int e = lane; e < E; e += 32) R += cnt[e];
  R = __reduce_add_sync(0xffffffffu, R);
  const int N = live[ch.a];
  const float rR = 1.0f / max(R, 1), g = (dloss ? dloss[ch.a] : 1.f) * (coef * E) / max(N, 1);
  for (int t = ch.t0 + w; t < ch.t1; t += kW) {
    const T* row = logits + t * ld;
    bool any = false;
    for (int j = 0; j < k; ++j) {
      const int e = ids[(int64_t)t * k + j];
      any |= e >= 0 && e < E;
    }
    float mx = -INFINITY, z = 0.f, s = 0.f;
    if (any) {
      for (int e = lane; e < E; e += 32) mx = fmaxf(mx, to_f32(row[e]));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      // a row of -inf alone: exp(-inf - 0) = 0 everywhere
      if (mx == -INFINITY) mx = 0.f;
      for (int e = lane; e < E; e += 32) {
        const float p = expf(to_f32(row[e]) - mx);
        z += p;
        s += p * (cnt[e] * rR);
      }
      z = warp_sum(z);
      s = warp_sum(s);
    }
    const float rz = z == 0.f ? 0.f : 1.0f / z;
    s *= rz;
    for (int e = lane; e < E; e += 32) {
      const float p = any ? expf(to_f32(row[e]) - mx) * rz : 0.f;
      acc[w][e] += p;
      if (dlogits) dlogits[(int64_t)t * E + e] = any ? g * (p * (cnt[e] * rR - s)) : 0.f;
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    float v = 0.f;
    for (int i = 0; i < kW; ++i) v += acc[i][e];
    part[(int64_t)blockIdx.x * E + e] = v;
  }
}

__global__ void __launch_bounds__(kBalThreads) balance_loss_kernel(BalTable bt, int E, float coef, const int* counts,
                                                                   const int* live, const float* part, float* loss,
                                                                   float* prob) {
  __shared__ float sm[kBalThreads / 32][2];
  const int a = blockIdx.x, N = live[a];
  float s = 0.f, R = 0.f;
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    float v = 0.f;
    for (int c = bt.chunk0[a]; c < bt.chunk0[a + 1]; ++c) v += part[(int64_t)c * E + e];
    v /= max(N, 1);
    prob[a * E + e] = v;
    s += v * counts[a * E + e];
    R += counts[a * E + e];
  }
  s = warp_sum(s);
  R = warp_sum(R);
  if ((threadIdx.x & 31) == 0) {
    sm[threadIdx.x >> 5][0] = s;
    sm[threadIdx.x >> 5][1] = R;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    s = R = 0.f;
    for (int i = 0; i < kBalThreads / 32; ++i) {
      s += sm[i][0];
      R += sm[i][1];
    }
    loss[a] = coef * E * (s / fmaxf(R, 1.f));
  }
}

#define LAUNCH(call)                                     \
  do {                                                   \
    if ((call) != cudaSuccess) return MOE_LORA_ERR_CUDA; \
  } while (0)

template <class T>
int run_balance(const moe_lora_dims* d, const BalTable& bt, const void* logits, int64_t ld, const int32_t* ids,
                float coef, const float* dloss, float* loss, int32_t* counts, float* prob, float* dlogits,
                void* scratch, cudaStream_t s) {
  const BalLayout L = bal_layout(d);
  char* sc = static_cast<char*>(scratch);
  int *err = (int*)(sc + L.err), *live = (int*)(sc + L.live);
  float* part = (float*)(sc + L.part);
  const int chunks = bt.chunk0[bt.n];
  LAUNCH(cudaMemsetAsync(scratch, 0, L.part, s));
  LAUNCH(cudaMemsetAsync(counts, 0, sizeof(int) * (size_t)d->A * d->E, s));
  if (chunks) {
    prof_begin(K_BAL_COUNT, s);
    balance_count_kernel<<<chunks, kBalThreads, 0, s>>>(bt, ids, d->k, d->E, counts, live, err);
    prof_end(K_BAL_COUNT, s);
    prof_begin(K_BAL_PROB, s);
    balance_prob_kernel<T><<<chunks, kBalThreads, 0, s>>>(bt, (const T*)logits, ld, ids, d->k, d->E, coef, dloss,
                                                          counts, live, part, dlogits);
    prof_end(K_BAL_PROB, s);
  }
  prof_begin(K_BAL_LOSS, s);
  balance_loss_kernel<<<d->A, kBalThreads, 0, s>>>(bt, d->E, coef, counts, live, part, loss, prob);
  prof_end(K_BAL_LOSS, s);
  LAUNCH(cudaGetLastError());
  return MOE_LORA_OK;
}

}  // namespace

size_t balance_scratch_bytes(const moe_lora_dims* d) { return check_balance_dims(d) ? 0 : bal_layout(d).total; }

}  // namespace moelora

using namespace moelora;

extern "C" int moe_lora_balance_loss(const moe_lora_dims* d, const void* logits, int32_t dtype, int64_t ld,
                                     const int32_t* topk_ids, const int64_t* adapter_offsets, float coef,
                                     const float* dloss, float* loss, int32_t* counts, float* prob, float* dlogits,
                                     void* scratch, size_t scratch_bytes, void* stream) {
  int rc = check_balance_dims(d);
  if (rc) return rc;
  if (!dtype_ok(dtype)) return MOE_LORA_ERR_UNSUPPORTED;
  if (ld == 0) ld = d->E;
  if (ld < d->E || ld > (int64_t)1 << 32) return MOE_LORA_ERR_DIMS;
  AdapterTable at;
  if ((rc = make_adapter_table(d, adapter_offsets, &at))) return rc;
  if ((rc = check_ptr(scratch))) return rc;
  if (scratch_bytes < bal_layout(d).total) return MOE_LORA_ERR_WORKSPACE;
  if ((rc = check_ptr(loss)) || (rc = check_ptr(counts)) || (rc = check_ptr(prob)) || (rc = check_opt(dloss)) ||
      (rc = check_opt(dlogits)))
    return rc;
  if (d->T > 0 && ((rc = check_ptr(logits)) || (rc = check_ptr(topk_ids)))) return rc;
  int sms;
  if ((rc = device_sms(&sms))) return rc;
  BalTable bt = {};
  bt.n = d->A;
  for (int a = 0; a < d->A; ++a) {
    const int n = at.tok_off[a + 1] - at.tok_off[a];
    const int per = std::max(kBalMinChunk, (n + kBalMaxChunks - 1) / kBalMaxChunks);
    bt.tok_off[a] = at.tok_off[a];
    bt.chunk[a] = per;
    bt.chunk0[a + 1] = bt.chunk0[a] + (n + per - 1) / per;
  }
  bt.tok_off[d->A] = at.tok_off[d->A];
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const auto run = dtype == MOE_LORA_F32    ? run_balance<float>
                   : dtype == MOE_LORA_BF16 ? run_balance<__nv_bfloat16>
                                            : run_balance<__half>;
  return run(d, bt, logits, ld, topk_ids, coef, dloss, loss, counts, prob, dlogits, scratch, s);
}
