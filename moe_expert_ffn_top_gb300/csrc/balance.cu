// Balance loss of the routing step with the per-expert counts and its gradient to the
// logits (definitions in include/moe_lora.h).
//
// An adapter's tokens are cut into groups of eight chunks, in numbers that depend on that
// adapter's sizes alone.  A cluster of eight blocks works on a group, a block on a chunk:
// it keeps its sums of probabilities in registers, the cluster adds them through
// distributed shared memory in block order, and groups are added in order.
//
// Adapters of one group each (small batches): one launch.  The cluster counts its ids,
// meets, and every block has the counts it needs for the gradient.  Otherwise a first
// launch counts per group, and in the second the last cluster of an adapter to finish
// adds its groups.  Logits are read once, for the loss and the gradient together.
#include <algorithm>

#include "common.cuh"
#include "element.cuh"
#include "launch.h"
#include "prof.h"
#include "sm100_ptx.cuh"

namespace moelora {

namespace {

constexpr int kBalThreads = 256, kBalWarps = kBalThreads / 32;
constexpr int kBalMaxE = 1024;
constexpr int kBalCluster = 8;       // chunks per group
constexpr int kBalMaxChunk = 4096;   // tokens
constexpr int kBalMaxGroups = 38;    // 304 blocks, two per SM, unless the chunks get too long
constexpr int kBalGroupWork = 1 << 18;  // logits worth another group
constexpr int kBalStages = 3;

struct BalTable {
  int n;
  int tok_off[kMaxAdapters + 1];
  int group0[kMaxAdapters + 1];  // first group of each adapter
  int chunk[kMaxAdapters];       // tokens per chunk
};

// Groups of an adapter of n tokens: one per 2^18 logits up to 38, more only where a
// chunk would pass its limit.
int64_t bal_groups(int64_t n, int E) {
  const int64_t by_work = std::min<int64_t>((n * E + kBalGroupWork - 1) / kBalGroupWork, kBalMaxGroups);
  const int64_t by_size = (n + kBalCluster * kBalMaxChunk - 1) / (kBalCluster * kBalMaxChunk);
  return std::max<int64_t>(1, std::max(by_work, by_size));
}

struct BalLayout {
  size_t err, done, live, bad, counts, part, total;
};
BalLayout bal_layout(const moe_lora_dims* d) {
  BalLayout L;
  // ceil(a) + ceil(b) <= ceil(a + b) + 1, an adapter's groups
  const int64_t work = d->T * d->E / kBalGroupWork, size = d->T / (kBalCluster * kBalMaxChunk);
  const int64_t groups = std::min<int64_t>(work, (int64_t)d->A * kBalMaxGroups) + size + 2 * d->A;
  size_t o = 0;
  auto take = [&](size_t bytes) { size_t at = o; o = align_up(o + bytes, 256); return at; };
  L.err = take(sizeof(int) * d->A);
  L.done = take(sizeof(int) * d->A);
  L.live = take(sizeof(int) * groups);
  L.bad = take(sizeof(int) * groups);
  L.counts = take(sizeof(int) * groups * d->E);
  L.part = take(sizeof(float) * groups * d->E);
  L.total = o;
  return L;
}
// Device view of the scratch: per adapter an error word and the number of its groups that
// are done; per group its live tokens, error bits, counts [E] and sums of probabilities [E].
struct BalScratch {
  int *err, *done, *live, *bad, *counts;
  float* part;
};
BalScratch bal_scratch(const moe_lora_dims* d, void* p) {
  const BalLayout L = bal_layout(d);
  char* c = static_cast<char*>(p);
  return BalScratch{(int*)(c + L.err),  (int*)(c + L.done),   (int*)(c + L.live),
                    (int*)(c + L.bad), (int*)(c + L.counts), (float*)(c + L.part)};
}

int check_balance_dims(const moe_lora_dims* d) {
  const int rc = check_dims(d);
  if (rc) return rc;
  return d->E > kBalMaxE ? MOE_LORA_ERR_UNSUPPORTED : MOE_LORA_OK;
}

struct Chunk {
  int a, group, t0, len;  // adapter, group of all, first token, tokens
  __device__ __forceinline__ explicit Chunk(const BalTable& bt) {
    group = blockIdx.x / kBalCluster;
    a = 0;
    while (a + 1 < bt.n && group >= bt.group0[a + 1]) ++a;
    const int64_t at = (int64_t)(blockIdx.x - bt.group0[a] * kBalCluster) * bt.chunk[a];
    const int64_t left = bt.tok_off[a + 1] - bt.tok_off[a] - at;
    len = left <= 0 ? 0 : (int)(left < bt.chunk[a] ? left : bt.chunk[a]);
    t0 = bt.tok_off[a] + (int)(len ? at : 0);
  }
};

template <class V>
__device__ __forceinline__ V from_rank(const V* p, int rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v) : "r"(mapa_shared(smem_u32(p), rank)) : "memory");
  return reinterpret_cast<const V&>(v);
}

// What a block learns from the ids of its chunk.
struct IdScan {
  int hist[kBalMaxE];              // routes per expert (kCount)
  uint32_t live[kBalMaxChunk / 32];  // tokens with a route
  int nlive, bad;
};
template <bool kCount>
__device__ __forceinline__ void scan_ids(IdScan& sc, const Chunk& ch, const int32_t* ids, int k, int E) {
  if (kCount)
    for (int e = threadIdx.x; e < E; e += kBalThreads) sc.hist[e] = 0;
  for (int i = threadIdx.x; i < (ch.len + 31) / 32; i += kBalThreads) sc.live[i] = 0;
  if (threadIdx.x == 0) sc.nlive = sc.bad = 0;
  __syncthreads();
  const int32_t* p = ids + (int64_t)ch.t0 * k;
  const int routes = ch.len * k;
  for (int i = threadIdx.x; i < routes; i += kBalThreads) {
    const int e = p[i];
    if ((unsigned)e < (unsigned)E) {
      const int t = i / k;
      if (kCount) atomicAdd(&sc.hist[e], 1);
      atomicOr(&sc.live[t >> 5], 1u << (t & 31));
    } else if (e != -1) {
      sc.bad = MOE_LORA_DEV_BAD_ID;
    }
  }
  __syncthreads();
  if (kCount) {
    int n = 0;
    for (int i = threadIdx.x; i < (ch.len + 31) / 32; i += kBalThreads) n += __popc(sc.live[i]);
    n = __reduce_add_sync(0xffffffffu, n);
    if ((threadIdx.x & 31) == 0 && n) atomicAdd(&sc.nlive, n);
    __syncthreads();
  }
}

// First launch of larger batches: counts, live tokens and error bits per group.
__global__ void __cluster_dims__(kBalCluster, 1, 1) __launch_bounds__(kBalThreads)
    balance_count_kernel(const __grid_constant__ BalTable bt, const int32_t* ids, int k, int E, BalScratch out) {
  __shared__ IdScan sc;
  const Chunk ch(bt);
  const int rank = (int)cluster_rank();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  scan_ids<true>(sc, ch, ids, k, E);
  cluster_sync_all();
  const int per = (E + kBalCluster - 1) / kBalCluster;
  for (int e = rank * per + threadIdx.x; e < min(E, (rank + 1) * per); e += kBalThreads) {
    int c = 0;
    for (int r = 0; r < kBalCluster; ++r) c += from_rank(&sc.hist[e], r);
    out.counts[(int64_t)ch.group * E + e] = c;
  }
  if (rank == 0 && threadIdx.x == 0) {
    int n = 0, b = 0;
    for (int r = 0; r < kBalCluster; ++r) {
      n += from_rank(&sc.nlive, r);
      b |= from_rank(&sc.bad, r);
    }
    out.live[ch.group] = n;
    out.bad[ch.group] = b;
    if (ch.group == bt.group0[ch.a]) out.done[ch.a] = 0;
  }
  cluster_sync_all();  // nobody leaves while its counts are read
}

// Sum of v over the lanes that share a row.
__device__ __forceinline__ float lanes_sum(float v, int lpr) {
  for (int o = lpr >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

struct BalArgs {
  const void* logits;
  int64_t ld;
  const int32_t* ids;
  int k, E, lpr;  // lpr: lanes of a row
  float coef;
  const float* dloss;
  float* loss;
  int32_t* counts;
  float *prob, *dlogits;
  BalScratch sc;
};

// Loss, probabilities and the logits' gradient.  `lpr` lanes hold a row (4 to 32, so that
// a lane has at most kVals logits); a lane has the same experts in every row, whose f and
// sum of probabilities stay in its registers.  Vector rows come through a ring of
// asynchronous copies of the thread's own slots.
template <class T, int VL, int kVals, bool kOne>
__global__ void __cluster_dims__(kBalCluster, 1, 1) __launch_bounds__(kBalThreads, 2)
    balance_kernel(const __grid_constant__ BalTable bt, const __grid_constant__ BalArgs g) {
  constexpr int kP = Vec<T, VL>::kPairs, kSlots = kVals / (2 * kP);
  extern __shared__ __align__(16) uint8_t ring_sm[];
  __shared__ IdScan sc;
  __shared__ float fsm[kBalMaxE];  // f_e
  __shared__ float csm[kBalMaxE];  // this block's sums of probabilities
  __shared__ float lsm[kBalCluster];  // rank 0: the ranks' parts of the loss
  __shared__ int nsm[2], last, bad;  // R, N of the adapter; rank 0: this is its last group, error bits
  // per-warp sums of probabilities, half of the experts at a time, where the ring was
  float(*psm)[kBalMaxE / 2] = reinterpret_cast<float(*)[kBalMaxE / 2]>(ring_sm);
  const int E = g.E, lane = threadIdx.x % g.lpr, row = threadIdx.x / g.lpr, rows = kBalThreads / g.lpr;
  const int rank = (int)cluster_rank();
  const Chunk ch(bt);
  const Ring<kBalStages, kSlots> ring(ring_sm);
  const T* logits = static_cast<const T*>(g.logits);
  const auto copy_row = [&](int t, int s) {
    if (VL > 1) {
      if (t < ch.len) {
        const T* lr = logits + (ch.t0 + (int64_t)t) * g.ld;
#pragma unroll
        for (int i = 0; i < kSlots; ++i) {
          const SlotAt<VL> at(lane, i, g.lpr, E);
          if (at.in) async_copy16(ring.slot(s, i), lr + at.c);
        }
      }
      async_commit();
    }
  };
#pragma unroll
  for (int s = 0; s < kBalStages - 1; ++s) copy_row(row + s * rows, s);

  scan_ids<kOne>(sc, ch, g.ids, g.k, E);
  const int ng = bt.group0[ch.a + 1] - bt.group0[ch.a];
  if (threadIdx.x < 2) nsm[threadIdx.x] = 0;
  if (kOne)
    cluster_sync_all();
  else
    asm volatile("griddepcontrol.wait;" ::: "memory");
  __syncthreads();
  {
    const int* gc = g.sc.counts + (int64_t)bt.group0[ch.a] * E;
    int R = 0, N = 0;
    for (int e = threadIdx.x; e < E; e += kBalThreads) {
      int c = 0;
      if (kOne) {
        for (int r = 0; r < kBalCluster; ++r) c += from_rank(&sc.hist[e], r);
      } else {
#pragma unroll 8
        for (int i = 0; i < ng; ++i) c += gc[(int64_t)i * E + e];
      }
      fsm[e] = __int_as_float(c);
      R += c;
    }
    for (int i = threadIdx.x; i < (kOne ? kBalCluster : ng); i += kBalThreads)
      N += kOne ? from_rank(&sc.nlive, i) : g.sc.live[bt.group0[ch.a] + i];
    if (kOne && rank == 0 && threadIdx.x == 0) {
      bad = 0;
      for (int r = 0; r < kBalCluster; ++r) bad |= from_rank(&sc.bad, r);
    }
    R = __reduce_add_sync(0xffffffffu, R);
    N = __reduce_add_sync(0xffffffffu, N);
    if ((threadIdx.x & 31) == 0) {
      atomicAdd(&nsm[0], R);
      atomicAdd(&nsm[1], N);
    }
  }
  __syncthreads();
  const int N = nsm[1];
  const float rR = 1.0f / (float)max(nsm[0], 1), rN = 1.0f / (float)max(N, 1);
  const int per = (E + kBalCluster - 1) / kBalCluster, e0 = rank * per, e1 = min(E, e0 + per);
  for (int e = threadIdx.x; e < E; e += kBalThreads) {
    const int c = __float_as_int(fsm[e]);
    fsm[e] = (float)c * rR;
    if (e >= e0 && e < e1 && ch.group == bt.group0[ch.a]) g.counts[ch.a * E + e] = c;
  }
  __syncthreads();
  // f - 1/E instead of f: the gradient's difference f_e - <p, f> then loses less to cancellation
  const float mean = 1.0f / (float)E;
  const float up = (g.dlogits && g.dloss ? g.dloss[ch.a] : 1.f) * (g.coef * (float)E) * rN;
  float2 f[kSlots][kP], acc[kSlots][kP];
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
    const SlotAt<VL> at(lane, i, g.lpr, E);
#pragma unroll
    for (int j = 0; j < kP; ++j) {
      const int c = VL == 1 ? at.c : at.c + 2 * j, c2 = VL == 1 ? at.c + at.hop : c + 1;
      f[i][j] = at.in ? make_float2(fsm[c] - mean, fsm[c2] - mean) : both(0.f);
      acc[i][j] = both(0.f);
    }
  }
  int s = 0;
  for (int tb = 0; tb < ch.len; tb += rows) {
    const int t = tb + row;
    copy_row(t + (kBalStages - 1) * rows, s == 0 ? kBalStages - 1 : s - 1);
    const bool on = t < ch.len, alive = on && (sc.live[t >> 5] >> (t & 31) & 1);
    if (VL > 1) async_wait<kBalStages - 1>();
    float2 v[kSlots][kP];
    float mx = -INFINITY;
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
      const SlotAt<VL> at(lane, i, g.lpr, E);
      if (at.in && alive) {
        Vec<T, VL> w;
        if constexpr (VL > 1)
          w.from_smem(ring.slot(s, i));
        else
          w.load(logits + (ch.t0 + (int64_t)t) * g.ld + at.c, at.hop);
#pragma unroll
        for (int j = 0; j < kP; ++j) {
          v[i][j] = w.get(j);
          if (VL == 1 && !at.hop) v[i][j].y = -INFINITY;
          mx = fmaxf(mx, fmaxf(v[i][j].x, v[i][j].y));
        }
      } else {
#pragma unroll
        for (int j = 0; j < kP; ++j) v[i][j] = both(-INFINITY);
      }
    }
    for (int o = g.lpr >> 1; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if (mx == -INFINITY) mx = 0.f;  // nothing but -inf: exp(-inf) = 0 throughout
    float2 z = both(0.f), d = both(0.f);
#pragma unroll
    for (int i = 0; i < kSlots; ++i)
#pragma unroll
      for (int j = 0; j < kP; ++j) {
        const float2 x = mul2(add2(v[i][j], both(-mx)), both(1.4426950408889634f));
        v[i][j] = make_float2(exp2f(x.x), exp2f(x.y));
        z = add2(z, v[i][j]);
        d = fma2(v[i][j], f[i][j], d);
      }
    const float zs = lanes_sum(z.x + z.y, g.lpr);
    const float rz = zs == 0.f ? 0.f : 1.0f / zs;
    const float ds = lanes_sum(d.x + d.y, g.lpr) * rz;
    const float2 w = both(up * rz);
    float* dr = g.dlogits ? g.dlogits + (ch.t0 + (int64_t)t) * E : nullptr;
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
      const SlotAt<VL> at(lane, i, g.lpr, E);
      Vec<float, VL == 1 ? 1 : 4> o[VL == 8 ? 2 : 1];
#pragma unroll
      for (int j = 0; j < kP; ++j) {
        acc[i][j] = fma2(v[i][j], both(rz), acc[i][j]);
        o[VL == 8 ? j >> 1 : 0].put(VL == 8 ? j & 1 : j, mul2(mul2(v[i][j], w), add2(f[i][j], both(-ds))));
      }
      if (dr && on && at.in) {
        o[0].store(dr + at.c, at.hop);
        if (VL == 8) o[VL == 8 ? 1 : 0].store(dr + at.c + 4, 0);
      }
    }
    s = s == kBalStages - 1 ? 0 : s + 1;
  }
  async_wait<0>();
  __syncthreads();
  // the block's sums: rows of a warp by shuffles, warps in order
#pragma unroll
  for (int i = 0; i < kSlots; ++i)
#pragma unroll
    for (int j = 0; j < kP; ++j)
      for (int o = g.lpr; o < 32; o <<= 1) {
        acc[i][j].x += __shfl_xor_sync(0xffffffffu, acc[i][j].x, o);
        acc[i][j].y += __shfl_xor_sync(0xffffffffu, acc[i][j].y, o);
      }
  for (int h = 0; h < E; h += kBalMaxE / 2) {
    if ((threadIdx.x & 31) < g.lpr)
#pragma unroll
      for (int i = 0; i < kSlots; ++i) {
        const SlotAt<VL> at(lane, i, g.lpr, E);
        if (at.in)
#pragma unroll
          for (int j = 0; j < kP; ++j) {
            const int c = (VL == 1 ? at.c : at.c + 2 * j) - h, c2 = VL == 1 ? c + at.hop : c + 1;
            if ((unsigned)c2 < kBalMaxE / 2u && (VL > 1 || at.hop)) psm[threadIdx.x >> 5][c2] = acc[i][j].y;
            if ((unsigned)c < kBalMaxE / 2u) psm[threadIdx.x >> 5][c] = acc[i][j].x;
          }
      }
    __syncthreads();
    for (int e = h + threadIdx.x; e < min(E, h + kBalMaxE / 2); e += kBalThreads) {
      float p = 0.f;
#pragma unroll
      for (int w = 0; w < kBalWarps; ++w) p += psm[w][e - h];
      csm[e] = p;
    }
    __syncthreads();
  }
  cluster_sync_all();
  // the group's sums: this block's slice of the experts, blocks in order
  float part = 0.f;
  const auto finish = [&](int e, float p) {
    p *= rN;
    g.prob[ch.a * E + e] = p;
    part = fmaf(fsm[e], p, part);
  };
  for (int e = e0 + threadIdx.x; e < e1; e += kBalThreads) {
    float p = 0.f;
    for (int r = 0; r < kBalCluster; ++r) p += from_rank(&csm[e], r);
    if (kOne)
      finish(e, p);
    else
      g.sc.part[(int64_t)ch.group * E + e] = p;
  }
  bool ends = true;
  if (!kOne) {  // the adapter's last group adds them all
    __threadfence();
    cluster_sync_all();
    if (rank == 0 && threadIdx.x == 0) {
      __threadfence();
      const int is_last = atomicAdd(&g.sc.done[ch.a], 1) == ng - 1;
      __threadfence();
      last = is_last;
    }
    cluster_sync_all();
    ends = from_rank(&last, 0) != 0;
    if (ends) {
      __threadfence();
      const float* gp = g.sc.part + (int64_t)bt.group0[ch.a] * E;
      for (int e = e0 + threadIdx.x; e < e1; e += kBalThreads) {
        float p = 0.f;
#pragma unroll 8
        for (int i = 0; i < ng; ++i) p += __ldcg(gp + (int64_t)i * E + e);
        finish(e, p);
      }
    }
  }
  // the loss: threads in order within a warp (E <= 1024: a slice is one block's first 128 threads), warps, then ranks
  if (ends) {
    for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
    if ((threadIdx.x & 31) == 0) psm[threadIdx.x >> 5][0] = part;
    __syncthreads();
    if (threadIdx.x == 0) {
      float l = 0.f;
      for (int w = 0; w < kBalWarps; ++w) l += psm[w][0];
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(mapa_shared(smem_u32(&lsm[rank]), 0)), "f"(l) : "memory");
    }
  }
  cluster_sync_all();  // also: nobody leaves while its shared memory is read
  if (ends && rank == 0 && threadIdx.x == 0) {
    float l = 0.f;
    for (int r = 0; r < kBalCluster; ++r) l += lsm[r];
    g.loss[ch.a] = g.coef * (float)E * l;
    int b = kOne ? bad : 0;
    for (int i = 0; !kOne && i < ng; ++i) b |= g.sc.bad[bt.group0[ch.a] + i];
    g.sc.err[ch.a] = b;
  }
}

#define LAUNCH(call)                                     \
  do {                                                   \
    if ((call) != cudaSuccess) return MOE_LORA_ERR_CUDA; \
  } while (0)

template <class T, int VL, int kVals, bool kOne>
int launch_balance(const BalTable& bt, const BalArgs& a, cudaStream_t s) {
  const auto kernel = balance_kernel<T, VL, kVals, kOne>;
  const size_t ring = VL == 1 ? 0 : ring_bytes<kBalStages, kVals / VL>(kBalThreads);
  const size_t smem = std::max(ring, sizeof(float) * kBalWarps * (kBalMaxE / 2));
  LAUNCH(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem));
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)bt.group0[bt.n] * kBalCluster);
  cfg.blockDim = dim3(kBalThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = kOne ? 0 : 1;  // overlaps the counting launch before it
  prof_begin(K_BAL_LOSS, s);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, bt, a);
  prof_end(K_BAL_LOSS, s);
  return e == cudaSuccess ? MOE_LORA_OK : MOE_LORA_ERR_CUDA;
}

template <class T, int VL, int kVals>
int pick_groups(const BalTable& bt, const BalArgs& a, cudaStream_t s) {
  if (bt.group0[bt.n] == bt.n) return launch_balance<T, VL, kVals, true>(bt, a, s);
  prof_begin(K_BAL_COUNT, s);
  balance_count_kernel<<<bt.group0[bt.n] * kBalCluster, kBalThreads, 0, s>>>(bt, a.ids, a.k, a.E, a.sc);
  prof_end(K_BAL_COUNT, s);
  LAUNCH(cudaGetLastError());
  return launch_balance<T, VL, kVals, false>(bt, a, s);
}

template <class T>
int run_balance(const BalTable& bt, BalArgs a, cudaStream_t s) {
  constexpr int kVL = 16 / sizeof(T);
  const bool vec = (a.ld | a.E) % kVL == 0, few = a.E <= 64;
  a.lpr = few ? (a.E <= 32 ? 4 : 8) : a.E <= 128 ? 4 : a.E <= 256 ? 8 : a.E <= 512 ? 16 : 32;
  if (vec) return few ? pick_groups<T, kVL, 8>(bt, a, s) : pick_groups<T, kVL, 32>(bt, a, s);
  return few ? pick_groups<T, 1, 8>(bt, a, s) : pick_groups<T, 1, 32>(bt, a, s);
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
    const int64_t n = at.tok_off[a + 1] - at.tok_off[a], groups = bal_groups(n, d->E);
    bt.tok_off[a] = at.tok_off[a];
    bt.chunk[a] = (int)((n + groups * kBalCluster - 1) / (groups * kBalCluster));
    bt.group0[a + 1] = bt.group0[a] + (int)groups;
  }
  bt.tok_off[d->A] = at.tok_off[d->A];
  const BalArgs a{logits, ld, topk_ids, d->k, d->E, 0, coef, dloss, loss, counts, prob, dlogits, bal_scratch(d, scratch)};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return dtype == MOE_LORA_F32    ? run_balance<float>(bt, a, s)
         : dtype == MOE_LORA_BF16 ? run_balance<__nv_bfloat16>(bt, a, s)
                                  : run_balance<__half>(bt, a, s);
}

extern "C" int moe_lora_balance_get_error(const moe_lora_dims* d, const void* scratch, void* stream) {
  const int rc = check_balance_dims(d);
  if (rc) return rc;
  if (!scratch) return MOE_LORA_ERR_NULL;
  int v[kMaxAdapters], all = 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cudaMemcpyAsync(v, static_cast<const char*>(scratch) + bal_layout(d).err, sizeof(int) * d->A,
                      cudaMemcpyDeviceToHost, s) != cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess)
    return MOE_LORA_ERR_CUDA;
  for (int a = 0; a < d->A; ++a) all |= v[a];
  return all;
}
