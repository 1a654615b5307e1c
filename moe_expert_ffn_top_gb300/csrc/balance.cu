// Balance loss of the routing step with the per-expert counts and its gradient to the
// logits (definitions in include/moe_lora.h).
//
// An adapter's tokens are cut into groups of eight chunks, in numbers that depend on that
// adapter's sizes alone; a block works on a chunk and keeps its sums of probabilities in
// registers.  The sums of a group's chunks, then the groups', are added in order.
//
// Adapters of one group each (small batches): one launch.  A cluster of eight blocks
// counts the group's ids, meets, and every block has the counts that the gradient needs;
// the sums meet in distributed shared memory.  Otherwise a first launch counts, one
// cluster per group, and the second needs no cluster (its blocks fill every SM): the
// last block of a group to finish adds the group, the last group of an adapter the
// adapter.  Logits are read once, for the loss and the gradient together.
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
constexpr int kBalMaxChunk = 4096;   // tokens; a chunk is a multiple of 32 long
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
  size_t err, adone, gdone, live, bad, bits, counts, gpart, part, total;
};
BalLayout bal_layout(const moe_lora_dims* d) {
  BalLayout L;
  // ceil(a) + ceil(b) <= ceil(a + b) + 1, an adapter's groups
  const int64_t work = d->T * d->E / kBalGroupWork, size = d->T / (kBalCluster * kBalMaxChunk);
  const int64_t groups = std::min<int64_t>(work, (int64_t)d->A * kBalMaxGroups) + size + 2 * d->A;
  size_t o = 0;
  auto take = [&](size_t bytes) { size_t at = o; o = align_up(o + bytes, 256); return at; };
  L.err = take(sizeof(int) * d->A);
  L.adone = take(sizeof(int) * d->A);
  L.gdone = take(sizeof(int) * groups);
  L.live = take(sizeof(int) * groups);
  L.bad = take(sizeof(int) * groups);
  L.bits = take(sizeof(uint32_t) * (d->T / 32 + 1));
  L.counts = take(sizeof(int) * groups * d->E);
  L.gpart = take(sizeof(float) * groups * d->E);
  L.part = take(sizeof(float) * groups * kBalCluster * d->E);
  L.total = o;
  return L;
}
// Device view of the scratch.  Per adapter: an error word, how many of its groups are
// done.  Per group: how many of its chunks are done, its live tokens, error bits, counts
// [E], sums of probabilities [E]; per chunk such sums.  A bit per token: it is live.
struct BalScratch {
  int *err, *adone, *gdone, *live, *bad;
  uint32_t* bits;
  int* counts;
  float *gpart, *part;
};
BalScratch bal_scratch(const moe_lora_dims* d, void* p) {
  const BalLayout L = bal_layout(d);
  char* c = static_cast<char*>(p);
  return BalScratch{(int*)(c + L.err),  (int*)(c + L.adone),     (int*)(c + L.gdone),
                    (int*)(c + L.live), (int*)(c + L.bad),       (uint32_t*)(c + L.bits),
                    (int*)(c + L.counts), (float*)(c + L.gpart), (float*)(c + L.part)};
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
  int hist[kBalMaxE];                // routes per expert
  uint32_t live[kBalMaxChunk / 32];  // tokens with a route
  int nlive, bad;
};
__device__ __forceinline__ void scan_ids(IdScan& sc, const Chunk& ch, const int32_t* ids, int k, int E) {
  constexpr int kAhead = 4;  // loads under way per thread
  const int32_t* p = ids + (int64_t)ch.t0 * k;
  const int routes = ch.len * k, words = (ch.len + 31) / 32;
  int id[kAhead];
#pragma unroll
  for (int j = 0; j < kAhead; ++j) {
    const int i = threadIdx.x + j * kBalThreads;
    id[j] = i < routes ? p[i] : -1;
  }
  for (int e = threadIdx.x; e < E; e += kBalThreads) sc.hist[e] = 0;
  for (int i = threadIdx.x; i < words; i += kBalThreads) sc.live[i] = 0;
  if (threadIdx.x == 0) sc.nlive = sc.bad = 0;
  __syncthreads();
  for (int b = 0; b < routes; b += kAhead * kBalThreads) {
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int i = b + threadIdx.x + j * kBalThreads, e = id[j];
      if ((unsigned)e < (unsigned)E) {
        const int t = i / k;
        atomicAdd(&sc.hist[e], 1);
        atomicOr(&sc.live[t >> 5], 1u << (t & 31));
      } else if (e != -1) {
        sc.bad = MOE_LORA_DEV_BAD_ID;
      }
      const int next = i + kAhead * kBalThreads;
      id[j] = next < routes ? p[next] : -1;
    }
  }
  __syncthreads();
  int n = 0;
  for (int i = threadIdx.x; i < words; i += kBalThreads) n += __popc(sc.live[i]);
  n = __reduce_add_sync(0xffffffffu, n);
  if ((threadIdx.x & 31) == 0 && n) atomicAdd(&sc.nlive, n);
}

// First launch of larger batches: counts, live tokens and error bits of every group, and
// the tokens' live bits.
__global__ void __cluster_dims__(kBalCluster, 1, 1) __launch_bounds__(kBalThreads)
    balance_count_kernel(const __grid_constant__ BalTable bt, const int32_t* ids, int k, int E, BalScratch out) {
  __shared__ IdScan sc;
  const Chunk ch(bt);
  const int rank = (int)cluster_rank();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  scan_ids(sc, ch, ids, k, E);
  for (int i = threadIdx.x; i < (ch.len + 31) / 32; i += kBalThreads) out.bits[ch.t0 / 32 + i] = sc.live[i];
  cluster_sync_all();
  const int per = (E + kBalCluster - 1) / kBalCluster;
  for (int e = rank * per + threadIdx.x; e < min(E, (rank + 1) * per); e += kBalThreads) {
    int c = 0;
#pragma unroll
    for (int r = 0; r < kBalCluster; ++r) c += from_rank(&sc.hist[e], r);
    out.counts[(int64_t)ch.group * E + e] = c;
  }
  if (rank == 0 && threadIdx.x == 0) {
    int n = 0, b = 0;
#pragma unroll
    for (int r = 0; r < kBalCluster; ++r) {
      n += from_rank(&sc.nlive, r);
      b |= from_rank(&sc.bad, r);
    }
    out.live[ch.group] = n;
    out.bad[ch.group] = b;
    out.gdone[ch.group] = 0;
    if (ch.group == bt.group0[ch.a]) out.adone[ch.a] = 0;
  }
  cluster_sync_all();  // nobody leaves while its counts are read
}

// 2^x, to 2 units in the last place; results below 2^-126 become 0 (a probability that adds nothing).
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
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

// How a lane holds its logits: 16 bytes at a time, four (fp32 rows of any alignment,
// 16-bit rows of even length and stride), or element by element.  The first two come
// through a ring of asynchronous copies of the thread's own words.
enum RowMode { kVec16, kWord, kElement };

// A lane's kVals logits as pairs, and which experts they are.
template <class T, RowMode kMode>
struct Pairs {
  static constexpr int kPer = kMode == kVec16 ? 8 / (int)sizeof(T) : 1;  // pairs per vector (kVec16)
  int lane, lpr;
  // expert of the first of pair p, and the distance to the second
  __device__ __forceinline__ int first(int p) const {
    if (kMode == kVec16) return (lane + p / kPer * lpr) * 2 * kPer + 2 * (p % kPer);
    if (kMode == kWord && sizeof(T) == 2) return 2 * (lane + p * lpr);
    return lane + 2 * p * lpr;
  }
  __device__ __forceinline__ int apart() const { return kMode == kVec16 || (kMode == kWord && sizeof(T) == 2) ? 1 : lpr; }
};

// Adds in a fixed order over the block: threads of a warp, then warps.  One thread's result.
__device__ __forceinline__ float block_total(float v, float* sm) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.f;
  for (int w = 0; w < kBalWarps; ++w) v += sm[w];
  return v;
}

// Loss, probabilities and the logits' gradient.  `lpr` lanes hold a row (4 to 32, so that
// a lane has at most kVals logits); a lane has the same experts in every row, whose f and
// sum of probabilities stay in its registers (kFull: rows fill every lane).
template <class T, RowMode kMode, int kVals, bool kOne, bool kFull>
__global__ void __launch_bounds__(kBalThreads, 2)
    balance_kernel(const __grid_constant__ BalTable bt, const __grid_constant__ BalArgs g) {
  constexpr int kP = kVals / 2;
  constexpr int kWords = kVals * (int)sizeof(T) / 4;  // of a lane's row
  constexpr int kRows16 = kMode == kElement ? 1 : kWords / 4;
  extern __shared__ __align__(16) uint8_t ring_sm[];
  __shared__ IdScan sc;
  __shared__ float fsm[kBalMaxE];  // f_e
  __shared__ float csm[kBalMaxE];  // sums of probabilities: the block's; rank 0 of a cluster: the adapter's
  __shared__ float tsm[kBalWarps];
  __shared__ int nsm[2], last, bad;  // R, N of the adapter
  // per-warp sums of probabilities, half of the experts at a time, where the ring was
  float(*psm)[kBalMaxE / 2] = reinterpret_cast<float(*)[kBalMaxE / 2]>(ring_sm);
  const int E = g.E, row = threadIdx.x / g.lpr, rows = kBalThreads / g.lpr;
  const Pairs<T, kMode> pr{(int)threadIdx.x % g.lpr, g.lpr};
  const int rank = kOne ? (int)cluster_rank() : 0;
  const Chunk ch(bt);
  const Ring<kBalStages, kRows16> ring(ring_sm);
  const T* logits = static_cast<const T*>(g.logits) + (int64_t)ch.t0 * g.ld;
  const auto in = [&](int e) { return kFull || e < E; };
  // word w of the thread's row in stage s: words of a warp's lanes side by side (kWord)
  const auto word = [&](int s, int w) {
    return reinterpret_cast<uint32_t*>(ring.base - (threadIdx.x & 31) + s * kRows16 * 32) + w * 32 + (threadIdx.x & 31);
  };
  const auto copy_row = [&](int t, int s) {
    if (kMode == kElement) return;
    if (t < ch.len) {
      const T* lr = logits + (int64_t)t * g.ld;
      if (kMode == kVec16) {
#pragma unroll
        for (int i = 0; i < kRows16; ++i)
          if (in(pr.first(i * pr.kPer))) async_copy16(ring.slot(s, i), lr + pr.first(i * pr.kPer));
      } else {
#pragma unroll
        for (int w = 0; w < kWords; ++w) {
          const int e = sizeof(T) == 2 ? pr.first(w) : pr.lane + w * pr.lpr;
          if (in(e)) async_copy4(word(s, w), lr + e);
        }
      }
    }
    async_commit();
  };
#pragma unroll
  for (int s = 0; s < kBalStages - 1; ++s) copy_row(row + s * rows, s);

  const int ng = bt.group0[ch.a + 1] - bt.group0[ch.a];
  if (threadIdx.x < 2) nsm[threadIdx.x] = 0;
  if (kOne) {
    scan_ids(sc, ch, g.ids, g.k, E);
    cluster_sync_all();
  } else {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int i = threadIdx.x; i < (ch.len + 31) / 32; i += kBalThreads) sc.live[i] = g.sc.bits[ch.t0 / 32 + i];
    __syncthreads();
  }
  {
    const int* gc = g.sc.counts + (int64_t)bt.group0[ch.a] * E;
    int R = 0, N = 0;
    for (int e = threadIdx.x; e < E; e += kBalThreads) {
      int c = 0;
      if (kOne) {
#pragma unroll
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
      if (R) atomicAdd(&nsm[0], R);
      if (N) atomicAdd(&nsm[1], N);
    }
  }
  __syncthreads();
  const int N = nsm[1];
  const float rR = 1.0f / (float)max(nsm[0], 1), rN = 1.0f / (float)max(N, 1);
  const bool writes_counts = blockIdx.x == bt.group0[ch.a] * kBalCluster;
  for (int e = threadIdx.x; e < E; e += kBalThreads) {
    const int c = __float_as_int(fsm[e]);
    fsm[e] = (float)c * rR;
    if (writes_counts) g.counts[ch.a * E + e] = c;
  }
  __syncthreads();
  // f - 1/E instead of f: the gradient's difference f_e - <p, f> then loses less to cancellation
  const float mean = 1.0f / (float)E;
  const float up = (g.dlogits && g.dloss ? g.dloss[ch.a] : 1.f) * (g.coef * (float)E) * rN;
  float2 f[kP], acc[kP];
#pragma unroll
  for (int p = 0; p < kP; ++p) {
    const int e = pr.first(p), e2 = e + pr.apart();
    f[p] = make_float2(in(e) ? fsm[e] - mean : 0.f, in(e2) ? fsm[e2] - mean : 0.f);
    acc[p] = both(0.f);
  }
  int s = 0;
  for (int tb = 0; tb < ch.len; tb += rows) {
    const int t = tb + row;
    copy_row(t + (kBalStages - 1) * rows, s == 0 ? kBalStages - 1 : s - 1);
    const bool on = t < ch.len, alive = on && (sc.live[t >> 5] >> (t & 31) & 1);
    if (kMode != kElement) async_wait<kBalStages - 1>();
    float2 v[kP];
    float mx = -INFINITY;
#pragma unroll
    for (int p = 0; p < kP; ++p) v[p] = both(-INFINITY);
    if (alive) {
      if constexpr (kMode == kVec16) {
#pragma unroll
        for (int i = 0; i < kRows16; ++i)
          if (in(pr.first(i * pr.kPer))) {
            Vec<T, 16 / sizeof(T)> w;
            w.from_smem(ring.slot(s, i));
#pragma unroll
            for (int j = 0; j < pr.kPer; ++j) v[i * pr.kPer + j] = w.get(j);
          }
      } else {
        const T* lr = logits + (int64_t)t * g.ld;
#pragma unroll
        for (int p = 0; p < kP; ++p) {
          const int e = pr.first(p), e2 = e + pr.apart();
          if (!in(e)) continue;
          if constexpr (kMode == kElement) {
            v[p].x = to_f32(lr[e]);
            if (in(e2)) v[p].y = to_f32(lr[e2]);
          } else if constexpr (sizeof(T) == 2) {
            v[p] = Two<T>::get(word(s, p));
          } else {
            v[p].x = __uint_as_float(*word(s, 2 * p));
            if (in(e2)) v[p].y = __uint_as_float(*word(s, 2 * p + 1));
          }
        }
      }
#pragma unroll
      for (int p = 0; p < kP; ++p) mx = fmaxf(mx, fmaxf(v[p].x, v[p].y));
    }
    for (int o = g.lpr >> 1; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if (mx == -INFINITY) mx = 0.f;  // nothing but -inf: exp(-inf) = 0 throughout
    float2 z = both(0.f), d = both(0.f);
#pragma unroll
    for (int p = 0; p < kP; ++p) {
      const float2 x = mul2(add2(v[p], both(-mx)), both(1.4426950408889634f));
      v[p] = make_float2(ex2(x.x), ex2(x.y));
      z = add2(z, v[p]);
      d = fma2(v[p], f[p], d);
    }
    float zs = z.x + z.y, ds = d.x + d.y;
    for (int o = g.lpr >> 1; o > 0; o >>= 1) {
      zs += __shfl_xor_sync(0xffffffffu, zs, o);
      ds += __shfl_xor_sync(0xffffffffu, ds, o);
    }
    const float rz = zs == 0.f ? 0.f : 1.0f / zs;
    ds *= rz;
#pragma unroll
    for (int p = 0; p < kP; ++p) acc[p] = fma2(v[p], both(rz), acc[p]);
    if (g.dlogits && on) {
      const float2 w = both(up * rz), nd = both(-ds);
      float* dr = g.dlogits + (ch.t0 + (int64_t)t) * E;
#pragma unroll
      for (int p = 0; p < kP; ++p) v[p] = mul2(mul2(v[p], w), add2(f[p], nd));
      if constexpr (kMode == kVec16) {
#pragma unroll
        for (int p = 0; p < kP; p += 2)
          if (in(pr.first(p))) *reinterpret_cast<float4*>(dr + pr.first(p)) = make_float4(v[p].x, v[p].y, v[p + 1].x, v[p + 1].y);
      } else if constexpr (kMode == kWord && sizeof(T) == 2) {
#pragma unroll
        for (int p = 0; p < kP; ++p)
          if (in(pr.first(p))) *reinterpret_cast<float2*>(dr + pr.first(p)) = v[p];
      } else {
#pragma unroll
        for (int p = 0; p < kP; ++p) {
          const int e = pr.first(p), e2 = e + pr.apart();
          if (in(e)) dr[e] = v[p].x;
          if (in(e2)) dr[e2] = v[p].y;
        }
      }
    }
    s = s == kBalStages - 1 ? 0 : s + 1;
  }
  async_wait<0>();
  __syncthreads();
  // the block's sums: rows of a warp by shuffles, warps in order
#pragma unroll
  for (int p = 0; p < kP; ++p)
    for (int o = g.lpr; o < 32; o <<= 1) {
      acc[p].x += __shfl_xor_sync(0xffffffffu, acc[p].x, o);
      acc[p].y += __shfl_xor_sync(0xffffffffu, acc[p].y, o);
    }
  float* my_part = g.sc.part + (int64_t)blockIdx.x * E;
  for (int h = 0; h < E; h += kBalMaxE / 2) {
    const auto put = [&](int e, float x) {
      if (in(e) && (unsigned)(e - h) < kBalMaxE / 2u) psm[threadIdx.x >> 5][e - h] = x;
    };
    if ((int)(threadIdx.x & 31) < g.lpr)
#pragma unroll
      for (int p = 0; p < kP; ++p) {
        put(pr.first(p), acc[p].x);
        put(pr.first(p) + pr.apart(), acc[p].y);
      }
    __syncthreads();
    for (int e = h + threadIdx.x; e < min(E, h + kBalMaxE / 2); e += kBalThreads) {
      float p = 0.f;
#pragma unroll
      for (int w = 0; w < kBalWarps; ++w) p += psm[w][e - h];
      if (kOne)
        csm[e] = p;
      else
        my_part[e] = p;
    }
    __syncthreads();
  }
  // the group's, then the adapter's sums, and the loss
  float part = 0.f;
  if (kOne) {
    cluster_sync_all();
    const int per = (E + kBalCluster - 1) / kBalCluster;
    for (int e = rank * per + threadIdx.x; e < min(E, (rank + 1) * per); e += kBalThreads) {
      float p = 0.f;
#pragma unroll
      for (int r = 0; r < kBalCluster; ++r) p += from_rank(&csm[e], r);
      p *= rN;
      g.prob[ch.a * E + e] = p;
      // rank 0 needs them all; its psm is free
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(mapa_shared(smem_u32(&psm[0][0] + e), 0)), "f"(p) : "memory");
    }
    cluster_sync_all();  // also: nobody leaves while its shared memory is read
    if (rank != 0) return;
    for (int e = threadIdx.x; e < E; e += kBalThreads) part = fmaf(fsm[e], (&psm[0][0])[e], part);
  } else {
    // the last block of the group, then the last group of the adapter, go on
    const auto is_last = [&](int* counter, int of) {
      __threadfence();
      __syncthreads();
      if (threadIdx.x == 0) last = atomicAdd(counter, 1) == of - 1;
      __syncthreads();
      __threadfence();
      return last != 0;
    };
    if (!is_last(g.sc.gdone + ch.group, kBalCluster)) return;
    const float* cp = g.sc.part + (int64_t)ch.group * kBalCluster * E;
    for (int e = threadIdx.x; e < E; e += kBalThreads) {
      float p = 0.f;
#pragma unroll
      for (int r = 0; r < kBalCluster; ++r) p += __ldcg(cp + (int64_t)r * E + e);
      g.sc.gpart[(int64_t)ch.group * E + e] = p;
    }
    if (!is_last(g.sc.adone + ch.a, ng)) return;
    const float* gp = g.sc.gpart + (int64_t)bt.group0[ch.a] * E;
    for (int e = threadIdx.x; e < E; e += kBalThreads) {
      float p = 0.f;
#pragma unroll 8
      for (int i = 0; i < ng; ++i) p += __ldcg(gp + (int64_t)i * E + e);
      p *= rN;
      g.prob[ch.a * E + e] = p;
      part = fmaf(fsm[e], p, part);
    }
  }
  part = block_total(part, tsm);
  if (threadIdx.x == 0) {
    g.loss[ch.a] = g.coef * (float)E * part;
    int b = kOne ? bad : 0;
    for (int i = 0; !kOne && i < ng; ++i) b |= g.sc.bad[bt.group0[ch.a] + i];
    g.sc.err[ch.a] = b;
  }
}

#define LAUNCH(call)                                     \
  do {                                                   \
    if ((call) != cudaSuccess) return MOE_LORA_ERR_CUDA; \
  } while (0)

template <class T, RowMode kMode, int kVals, bool kOne>
int launch_balance(const BalTable& bt, const BalArgs& a, cudaStream_t s) {
  const auto kernel = kMode == kVec16 && a.E == a.lpr * kVals ? balance_kernel<T, kMode, kVals, kOne, kMode == kVec16>
                                                              : balance_kernel<T, kMode, kVals, kOne, false>;
  const size_t ring = kMode == kElement ? 0 : (size_t)kBalThreads * kBalStages * kVals * sizeof(T);
  const size_t smem = std::max(ring, sizeof(float) * kBalWarps * (kBalMaxE / 2));
  LAUNCH(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem));
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[1];
  if (kOne) {
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = kBalCluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  } else {  // overlaps the counting launch before it
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
  }
  cfg.gridDim = dim3((unsigned)bt.group0[bt.n] * kBalCluster);
  cfg.blockDim = dim3(kBalThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  prof_begin(K_BAL_LOSS, s);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, bt, a);
  prof_end(K_BAL_LOSS, s);
  return e == cudaSuccess ? MOE_LORA_OK : MOE_LORA_ERR_CUDA;
}

template <class T, RowMode kMode, int kVals>
int pick_groups(const BalTable& bt, const BalArgs& a, cudaStream_t s) {
  if (bt.group0[bt.n] == bt.n) return launch_balance<T, kMode, kVals, true>(bt, a, s);
  prof_begin(K_BAL_COUNT, s);
  balance_count_kernel<<<bt.group0[bt.n] * kBalCluster, kBalThreads, 0, s>>>(bt, a.ids, a.k, a.E, a.sc);
  prof_end(K_BAL_COUNT, s);
  LAUNCH(cudaGetLastError());
  return launch_balance<T, kMode, kVals, false>(bt, a, s);
}

template <class T, RowMode kMode>
int pick_vals(const BalTable& bt, BalArgs a, cudaStream_t s) {
  const bool few = a.E <= 64;
  a.lpr = few ? (a.E <= 32 ? 4 : 8) : a.E <= 128 ? 4 : a.E <= 256 ? 8 : a.E <= 512 ? 16 : 32;
  return few ? pick_groups<T, kMode, 8>(bt, a, s) : pick_groups<T, kMode, 32>(bt, a, s);
}

template <class T>
int run_balance(const BalTable& bt, const BalArgs& a, cudaStream_t s) {
  if ((a.ld | a.E) % (16 / sizeof(T)) == 0) return pick_vals<T, kVec16>(bt, a, s);
  if constexpr (sizeof(T) == 4) return pick_vals<T, kWord>(bt, a, s);
  return (a.ld | a.E) % 2 == 0 ? pick_vals<T, kWord>(bt, a, s) : pick_vals<T, kElement>(bt, a, s);
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
    bt.chunk[a] = (int)((n + groups * kBalCluster * 32 - 1) / (groups * kBalCluster * 32)) * 32;
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
