// Balance loss of the routing step with the per-expert counts and its gradient to the
// logits (definitions in include/moe_lora.h).
//
// An adapter's tokens are cut into groups of sixteen chunks, in numbers that depend on that
// adapter's sizes alone; a block works on a chunk and keeps its sums of probabilities in
// registers.  The sums of a group's chunks, then the groups', are added in order.
//
// Adapters of one group each (small batches): one launch.  A cluster of up to sixteen
// blocks counts the group's ids, meets, and every block has the counts that the gradient needs;
// the sums meet in distributed shared memory.  (Adapters of one chunk: no cluster.)
// Otherwise a first launch counts, a small cluster per group; the second needs no cluster, its
// blocks fill every SM; a third adds the chunks' sums.  Each is launched while the one
// before it still runs, and waits for it where it needs its results: the second has then
// its first logits under way.  Logits are read once, for the loss and the gradient
// together.
#include <algorithm>

#include "common.cuh"
#include "element.cuh"
#include "launch.h"
#include "prof.h"
#include "sm100_ptx.cuh"

namespace moelora {

namespace {

// Threads of the main kernel's blocks: many experts fill the registers of 256, up to 64
// experts (8 a lane) leave room for 512, whose iterations are half as many.
constexpr int block_threads(int vals) { return vals == 8 ? 512 : 256; }
constexpr int kSumPad = 16;
constexpr int kBalMaxE = 1024;
constexpr int kBalCluster = 16;      // chunks per group
constexpr int kBalMaxChunk = 4096;   // tokens; a chunk is a multiple of 32 long
constexpr int kBalMaxGroups = 19;    // 304 blocks, two per SM, unless the chunks get too long
constexpr int kBalGroupWork = 1 << 19;  // logits worth another group
constexpr int kBalGroupTokens = 1 << 13;  // tokens worth another group
constexpr int kBalFew = 8, kBalFewWork = 3 << 16, kBalFewTokens = 3 << 9;  // chunks of a small group, logits, tokens
constexpr int kBalChunkWork = 1 << 12;  // logits that one chunk takes alone
constexpr int kCountCluster = 4, kCountThreads = 512;
constexpr int kSumCluster = 8, kSumThreads = 1024;
constexpr int kBalStages = 3;

struct BalTable {
  int n;
  int tok_off[kMaxAdapters + 1];
  int group0[kMaxAdapters + 1];  // first group of each adapter
  int chunk[kMaxAdapters];       // tokens per chunk
};

// Groups of an adapter of n tokens: one per 2^19 logits and per 2^13 tokens up to 19, more
// only where a chunk would pass its limit.
int64_t bal_groups(int64_t n, int E) {
  const int64_t by_work = std::min<int64_t>(
      std::max<int64_t>((n * E + kBalGroupWork - 1) / kBalGroupWork, (n + kBalGroupTokens - 1) / kBalGroupTokens),
      kBalMaxGroups);
  const int64_t by_size = (n + kBalCluster * kBalMaxChunk - 1) / (kBalCluster * kBalMaxChunk);
  return std::max<int64_t>(1, std::max(by_work, by_size));
}

// Tokens per chunk of such an adapter: a sixteenth of a group; of one group and little
// work an eighth, of very little all.  The rule sees one adapter's sizes alone, so that its
// sums do not depend on the others.
// Clusters of eight against sixteen: one to four adapters of 1,024 x 128 8.5 and 7.6 us, of
// 2,048 x 128 11.4 and 8.8, of 512 x 16 6.4 and 6.4; sixteen adapters, whose clusters of
// sixteen do not all run together, 11.2 and 15.7, 15.6 and 20.6, 8.4 and 13.7.
// One block against a cluster of eight: 128 x 8 5.3 and 6.3 us, 512 x 8 7.5 and 6.9; 256 x 16
// 5.9 and 6.3, 512 x 16 7.3 and 6.5; 256 x 32 5.9 and 6.4; 64 x 64 5.1 and 6.5, 128 x 64 5.8
// and 6.4; 64 x 128 5.8 and 6.6.  They are level near 2,700 logits at 8 experts, 6,000 at 16,
// 10,000 at 32 and more: what one block takes alone is set for the few experts, and costs the
// others up to 1 us between 4,096 and 8,192 logits.
int bal_chunk(int64_t n, int64_t groups, int E) {
  const int64_t work = std::max(n * E, n * (kBalFewWork / kBalFewTokens));
  const int64_t chunks = groups > 1 || work > kBalFewWork ? groups * kBalCluster : n * E > kBalChunkWork ? kBalFew : 1;
  return (int)((n + chunks * 32 - 1) / (chunks * 32)) * 32;
}

struct BalLayout {
  size_t err, tokens, live, bad, bits, counts, part, total;
};
BalLayout bal_layout(const moe_lora_dims* d) {
  BalLayout L;
  // ceil(a) + ceil(b) <= ceil(a + b) + 1, an adapter's groups
  const int64_t work = d->T * d->E / kBalGroupWork + d->T / kBalGroupTokens, size = d->T / (kBalCluster * kBalMaxChunk);
  const int64_t groups = std::min<int64_t>(work, (int64_t)d->A * kBalMaxGroups) + size + 3 * d->A;
  size_t o = 0;
  auto take = [&](size_t bytes) { size_t at = o; o = align_up(o + bytes, 256); return at; };
  L.err = take(sizeof(int) * d->A);
  L.tokens = take(sizeof(int) * d->A);
  L.live = take(sizeof(int) * groups);
  L.bad = take(sizeof(int) * groups);
  L.bits = take(sizeof(uint32_t) * (d->T / 32 + 1));
  L.counts = take(sizeof(int) * groups * d->E);
  L.part = take(sizeof(float) * groups * kBalCluster * d->E);
  L.total = o;
  return L;
}
// Device view of the scratch.  Per adapter: an error word, its live tokens.  Per group: its
// live tokens, error bits, counts [E].  Per chunk: sums of probabilities [E].  A bit per
// token: it is live.
struct BalScratch {
  int *err, *tokens, *live, *bad;
  uint32_t* bits;
  int* counts;
  float* part;
};
BalScratch bal_scratch(const moe_lora_dims* d, void* p) {
  const BalLayout L = bal_layout(d);
  char* c = static_cast<char*>(p);
  return BalScratch{(int*)(c + L.err),  (int*)(c + L.tokens),    (int*)(c + L.live), (int*)(c + L.bad),
                    (uint32_t*)(c + L.bits), (int*)(c + L.counts), (float*)(c + L.part)};
}

int check_balance_dims(const moe_lora_dims* d) {
  const int rc = check_dims(d);
  if (rc) return rc;
  return d->E > kBalMaxE ? MOE_LORA_ERR_UNSUPPORTED : MOE_LORA_OK;
}

__device__ __forceinline__ int adapter_of(const BalTable& bt, int group) {
  int a = 0;
  while (a + 1 < bt.n && group >= bt.group0[a + 1]) ++a;
  return a;
}
// `chunks` consecutive chunks of an adapter from its chunk c0 on.
struct Span {
  int t0, len;  // first token, tokens
  __device__ __forceinline__ Span(const BalTable& bt, int a, int64_t c0, int chunks) {
    const int64_t at = c0 * bt.chunk[a], most = (int64_t)chunks * bt.chunk[a];
    const int64_t left = bt.tok_off[a + 1] - bt.tok_off[a] - at;
    len = left <= 0 ? 0 : (int)(left < most ? left : most);
    t0 = bt.tok_off[a] + (int)(len ? at : 0);
  }
};

template <class V>
__device__ __forceinline__ V from_rank(const V* p, int rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v) : "r"(mapa_shared(smem_u32(p), rank)) : "memory");
  return reinterpret_cast<const V&>(v);
}

// What a block learns from the ids of its tokens.
template <int kTokens>
struct IdScan {
  int hist[kBalMaxE];           // routes per expert
  uint32_t live[kTokens / 32];  // tokens with a route
  int nlive, bad;
};
// A thread takes a token's ids, a warp 32 tokens, whose live bits are then one ballot.
template <int kThreads, int kTokens>
__device__ __forceinline__ void scan_ids(IdScan<kTokens>& sc, const Span& sp, const int32_t* ids, int k, int E) {
  constexpr int kAhead = 8;  // loads under way per thread
  const int lane = threadIdx.x & 31, words = (sp.len + 31) / 32;
  int id[kAhead];
  const auto load = [&](int w, int j0) {
    const int t = w * 32 + lane;
    const int32_t* p = ids + ((int64_t)sp.t0 + t) * k + j0;
#pragma unroll
    for (int j = 0; j < kAhead; ++j) id[j] = t < sp.len && j0 + j < k ? p[j] : -1;
  };
  load(threadIdx.x >> 5, 0);
  for (int e = threadIdx.x; e < E; e += kThreads) sc.hist[e] = 0;
  if (threadIdx.x == 0) sc.nlive = sc.bad = 0;
  __syncthreads();
  int n = 0;
  for (int w = threadIdx.x >> 5; w < words; w += kThreads / 32) {
    bool any = false;
    for (int j0 = 0; j0 < k; j0 += kAhead) {
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        if ((unsigned)id[j] < (unsigned)E) {
          atomicAdd(&sc.hist[id[j]], 1);
          any = true;
        } else if (id[j] != -1) {
          sc.bad = MOE_LORA_DEV_BAD_ID;
        }
      }
      const bool more = j0 + kAhead < k;
      load(more ? w : w + kThreads / 32, more ? j0 + kAhead : 0);
    }
    const uint32_t bits = __ballot_sync(0xffffffffu, any);
    if (lane == 0) sc.live[w] = bits;
    n += __popc(bits);
  }
  if (lane == 0 && n) atomicAdd(&sc.nlive, n);
}

// First launch of larger batches: counts, live tokens and error bits of every group, and
// the tokens' live bits.  A group is a cluster's, an expert's count its blocks' sum.
__global__ void __cluster_dims__(kCountCluster, 1, 1) __launch_bounds__(kCountThreads)
    balance_count_kernel(const __grid_constant__ BalTable bt, const int32_t* ids, int k, int E, BalScratch out) {
  constexpr int kChunks = kBalCluster / kCountCluster;
  __shared__ IdScan<kChunks * kBalMaxChunk> sc;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int group = blockIdx.x / kCountCluster, a = adapter_of(bt, group), rank = (int)cluster_rank();
  const Span sp(bt, a, (int64_t)(group - bt.group0[a]) * kBalCluster + rank * kChunks, kChunks);
  scan_ids<kCountThreads>(sc, sp, ids, k, E);
  cluster_sync_all();
  for (int i = threadIdx.x; i < (sp.len + 31) / 32; i += kCountThreads) out.bits[sp.t0 / 32 + i] = sc.live[i];
  const int per = (E + kCountCluster - 1) / kCountCluster;
  for (int e = rank * per + threadIdx.x; e < min(E, (rank + 1) * per); e += kCountThreads) {
    int c = 0;
#pragma unroll
    for (int r = 0; r < kCountCluster; ++r) c += from_rank(&sc.hist[e], r);
    out.counts[(int64_t)group * E + e] = c;
  }
  if (rank == 0 && threadIdx.x == 0) {
    int n = 0, b = 0;
#pragma unroll
    for (int r = 0; r < kCountCluster; ++r) {
      n += from_rank(&sc.nlive, r);
      b |= from_rank(&sc.bad, r);
    }
    out.live[group] = n;
    out.bad[group] = b;
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
  __device__ __forceinline__ int apart() const {
    return kMode == kVec16 || (kMode == kWord && sizeof(T) == 2) ? 1 : lpr;
  }
};

// One expert's mean probability, also to the block that adds the loss (rank 0 of a
// cluster of kC).
template <int kC>
__device__ __forceinline__ void finish_prob(const BalArgs& g, int a, int e, float p, float* psm) {
  g.prob[a * g.E + e] = p;
  if (kC > 1)
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(mapa_shared(smem_u32(psm + e), 0)), "f"(p)
                 : "memory");
  else
    psm[e] = p;
}
// The loss from all of f and prob: 32 experts by a warp, the warps' sums in order.
template <int kThreads>
__device__ __forceinline__ void finish_loss(const BalArgs& g, int a, const float* f, const float* psm, float* tsm) {
  float t = 0.f;
  for (int b = 0; b < g.E; b += kThreads) {
    const int e = b + threadIdx.x;
    float v = e < g.E ? f[e] * psm[e] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) tsm[threadIdx.x >> 5] = v;
    __syncthreads();
    if (threadIdx.x == 0)
      for (int w = 0; w < min(kThreads, g.E - b + 31) / 32; ++w) t += tsm[w];
    __syncthreads();
  }
  if (threadIdx.x == 0) g.loss[a] = g.coef * (float)g.E * t;
}

// Loss, probabilities and the logits' gradient.  `lpr` lanes hold a row (4 to 32, so that
// a lane has at most kVals logits and a row's three reductions take few shuffles); a lane
// has the same experts in every row, whose f and sum of probabilities stay in its
// registers (kFull: rows fill every lane).
// kC: blocks of a cluster when one launch does it all, 0 as the second of three.
template <class T, RowMode kMode, int kVals, int kC, bool kFull>
__global__ void __launch_bounds__(block_threads(kVals), kVals == 8 ? 1 : 2)
    balance_kernel(const __grid_constant__ BalTable bt, const __grid_constant__ BalArgs g) {
  constexpr int kP = kVals / 2;
  constexpr int kWords = kVals * (int)sizeof(T) / 4;  // of a lane's row
  constexpr int kRows16 = kMode == kElement ? 1 : kWords / 4;
  constexpr bool kOne = kC > 0;
  constexpr int kT = block_threads(kVals);
  extern __shared__ __align__(16) uint8_t ring_sm[];
  __shared__ IdScan<kBalMaxChunk> sc;
  __shared__ float fsm[kBalMaxE];  // f_e
  __shared__ float csm[kBalMaxE];  // f_e - 1/E; then the block's sums of probabilities
  __shared__ float tsm[kT / 32];
  __shared__ int nsm[2], bad;  // R, N and error bits of the adapter
  // where the ring was: a row of sums per row group, rows apart so that float4 stores spread over the banks
  float* psm = reinterpret_cast<float*>(ring_sm);
  const int pitch = g.E + kSumPad;
  const int E = g.E, row = threadIdx.x / g.lpr, rows = kT / g.lpr;
  const Pairs<T, kMode> pr{(int)threadIdx.x % g.lpr, g.lpr};
  const int rank = kC > 1 ? (int)cluster_rank() : 0;
  const int group = kOne ? blockIdx.x / (kC ? kC : 1) : blockIdx.x / kBalCluster, a = adapter_of(bt, group);
  const int64_t chunk = kOne ? blockIdx.x % (kC ? kC : 1) : blockIdx.x - (int64_t)bt.group0[a] * kBalCluster;
  const Span ch(bt, a, chunk, 1);
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

  const int ng = bt.group0[a + 1] - bt.group0[a];
  if (threadIdx.x < 2) nsm[threadIdx.x] = 0;
  if (threadIdx.x == 0) bad = 0;
  int* cnt = reinterpret_cast<int*>(fsm);
  if (kOne) {
    scan_ids<kT>(sc, ch, g.ids, g.k, E);
    if (kC > 1)
      cluster_sync_all();
    else
      __syncthreads();
    for (int e = threadIdx.x; e < E; e += kT) {
      int c = kC > 1 ? 0 : sc.hist[e];
#pragma unroll
      for (int r = 0; r < (kC > 1 ? kC : 0); ++r) c += from_rank(&sc.hist[e], r);
      cnt[e] = c;
    }
    if (threadIdx.x < kC) {
      atomicAdd(&nsm[1], kC > 1 ? from_rank(&sc.nlive, threadIdx.x) : sc.nlive);
      atomicOr(&bad, kC > 1 ? from_rank(&sc.bad, threadIdx.x) : sc.bad);
    }
  } else {
    for (int e = threadIdx.x; e < E; e += kT) cnt[e] = 0;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __syncthreads();
    for (int i = threadIdx.x; i < (ch.len + 31) / 32; i += kT) sc.live[i] = g.sc.bits[ch.t0 / 32 + i];
    const int* gc = g.sc.counts + (int64_t)bt.group0[a] * E;
    // columns (four at a time where E allows) x slices of the groups, so that all loads are under way together
    const int wide = E % 4 == 0 ? 4 : 1, cols = E / wide, slices = max(1, kT / cols);
    for (int c = threadIdx.x; c < cols * slices; c += kT) {
      const int e = c % cols * wide;
      int4 v = make_int4(0, 0, 0, 0);
#pragma unroll 12
      for (int i = c / cols; i < ng; i += slices) {
        if (wide == 4) {
          const int4 u = *reinterpret_cast<const int4*>(gc + (int64_t)i * E + e);
          v.x += u.x;
          v.y += u.y;
          v.z += u.z;
          v.w += u.w;
        } else {
          v.x += gc[(int64_t)i * E + e];
        }
      }
      atomicAdd(&cnt[e], v.x);
      if (wide == 4) {
        atomicAdd(&cnt[e + 1], v.y);
        atomicAdd(&cnt[e + 2], v.z);
        atomicAdd(&cnt[e + 3], v.w);
      }
    }
    for (int i = threadIdx.x; i < ng; i += kT) {
      atomicAdd(&nsm[1], g.sc.live[bt.group0[a] + i]);
      atomicOr(&bad, g.sc.bad[bt.group0[a] + i]);
    }
  }
  __syncthreads();
  int R = 0;
  for (int e = threadIdx.x; e < E; e += kT) R += cnt[e];
  R = __reduce_add_sync(0xffffffffu, R);
  if ((threadIdx.x & 31) == 0 && R) atomicAdd(&nsm[0], R);
  __syncthreads();
  const int N = nsm[1];
  const float rR = 1.0f / (float)max(nsm[0], 1), rN = 1.0f / (float)max(N, 1);
  const bool first = chunk == 0;  // block of the adapter
  // f - 1/E instead of f for the gradient, which is the difference f_e - <p, f>: formed in
  // whole numbers, so that nothing cancels however even the counts are.
  const float rRE = rR * (1.0f / (float)E);
  for (int e = threadIdx.x; e < E; e += kT) {
    const int c = cnt[e];
    csm[e] = (float)((int64_t)c * E - nsm[0]) * rRE;
    fsm[e] = (float)c * rR;
    if (first) g.counts[a * E + e] = c;
  }
  if (first && threadIdx.x == 0) {
    g.sc.err[a] = bad;
    g.sc.tokens[a] = N;
  }
  __syncthreads();
  const float up = (g.dlogits && g.dloss ? g.dloss[a] : 1.f) * (g.coef * (float)E) * rN;
  float2 f[kP], acc[kP];
#pragma unroll
  for (int p = 0; p < kP; ++p) {
    const int e = pr.first(p), e2 = e + pr.apart();
    f[p] = make_float2(in(e) ? csm[e] : 0.f, in(e2) ? csm[e2] : 0.f);
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
      // rows without a probability (not live, or -inf throughout) have no gradient, also where dloss is not finite
      const float2 w = both(zs == 0.f ? 0.f : up * rz), nd = both(-ds);
      float* dr = g.dlogits + (ch.t0 + (int64_t)t) * E;
#pragma unroll
      for (int p = 0; p < kP; ++p) v[p] = mul2(mul2(v[p], w), add2(f[p], nd));
      if constexpr (kMode == kVec16) {
#pragma unroll
        for (int p = 0; p < kP; p += 2)
          if (in(pr.first(p)))
            *reinterpret_cast<float4*>(dr + pr.first(p)) = make_float4(v[p].x, v[p].y, v[p + 1].x, v[p + 1].y);
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
  // the block's sums over its row groups
#pragma unroll
  for (int p = 0; p < kP; ++p) {
    const int e = pr.first(p), e2 = e + pr.apart();
    if (kMode == kVec16) {
      if (p % 2 == 0 && in(e))
        *reinterpret_cast<float4*>(psm + row * pitch + e) = make_float4(acc[p].x, acc[p].y, acc[p + 1].x, acc[p + 1].y);
    } else {
      if (in(e)) psm[row * pitch + e] = acc[p].x;
      if (in(e2)) psm[row * pitch + e2] = acc[p].y;
    }
  }
  __syncthreads();
  const int slices = min(rows, max(1, kT / E));
  float* my_part = kOne ? csm : g.sc.part + (int64_t)blockIdx.x * E;
  if (slices > 1) {
    const int e = threadIdx.x % E, q = threadIdx.x / E;
    float p = 0.f;
    if (q < slices)
      for (int r = q; r < rows; r += slices) p += psm[r * pitch + e];
    __syncthreads();
    if (q < slices) psm[threadIdx.x] = p;
    __syncthreads();
    if (q == 0) {
      for (int i = 1; i < slices; ++i) p += psm[i * E + e];
      my_part[e] = p;
    }
  } else {
    for (int e = threadIdx.x; e < E; e += kT) {
      float p = 0.f;
      for (int r = 0; r < rows; ++r) p += psm[r * pitch + e];
      my_part[e] = p;
    }
  }
  if (!kOne) return;
  // the group's sums and the loss; psm: rank 0's, for all probabilities
  const int per = kC > 1 ? (E + kC - 1) / kC : E;
  if (kC > 1)
    cluster_sync_all();
  else
    __syncthreads();
  for (int e = rank * per + threadIdx.x; e < min(E, (rank + 1) * per); e += kT) {
    float p = kC > 1 ? 0.f : csm[e];
#pragma unroll
    for (int r = 0; r < (kC > 1 ? kC : 0); ++r) p += from_rank(&csm[e], r);
    finish_prob<kC>(g, a, e, p * rN, psm);
  }
  if (kC > 1)
    cluster_sync_all();  // also: nobody leaves while its shared memory is read
  else
    __syncthreads();
  if (rank == 0) finish_loss<kT>(g, a, fsm, psm, tsm);
}

// Third launch of larger batches: a cluster of eight blocks per adapter, an eighth of the
// experts each.  A group's chunks are added in order by one thread, the groups in order
// by another.
__global__ void __cluster_dims__(kSumCluster, 1, 1) __launch_bounds__(kSumThreads)
    balance_sum_kernel(const __grid_constant__ BalTable bt, const __grid_constant__ BalArgs g) {
  constexpr int kBatch = 64, kCols = kBalMaxE / kSumCluster;  // groups at a time, columns of a block
  __shared__ float gsm[kBatch][kCols];
  __shared__ float fsm[kBalMaxE], psm[kBalMaxE], tsm[kSumThreads / 32];
  __shared__ int nsm;
  const int E = g.E, a = blockIdx.x / kSumCluster, rank = (int)cluster_rank();
  const int per = (E + kSumCluster - 1) / kSumCluster, e0 = rank * per, cols = max(0, min(E - e0, per));
  const int slices = max(1, kSumThreads / max(cols, 1)), c = threadIdx.x % max(cols, 1), q = threadIdx.x / max(cols, 1);
  const int g0 = bt.group0[a], ng = bt.group0[a + 1] - g0;
  if (threadIdx.x == 0) nsm = 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __syncthreads();
  int R = 0;
  for (int e = threadIdx.x; e < E; e += kSumThreads) {
    const int n = g.counts[a * E + e];
    fsm[e] = (float)n;
    R += n;
  }
  R = __reduce_add_sync(0xffffffffu, R);
  if ((threadIdx.x & 31) == 0 && R) atomicAdd(&nsm, R);
  float p = 0.f;
  for (int b = 0; b < ng; b += kBatch) {
    const int m = min(kBatch, ng - b);
    if (c < cols && q < slices)
#pragma unroll 2
      for (int i = q; i < m; i += slices) {
        const float* cp = g.sc.part + (int64_t)(g0 + b + i) * kBalCluster * E + e0 + c;
        float v[kBalCluster];
#pragma unroll
        for (int r = 0; r < kBalCluster; ++r) v[r] = cp[(int64_t)r * E];
        float t = 0.f;
#pragma unroll
        for (int r = 0; r < kBalCluster; ++r) t += v[r];
        gsm[i][c] = t;
      }
    __syncthreads();
    if (q == 0 && c < cols)
      for (int i = 0; i < m; ++i) p += gsm[i][c];
    __syncthreads();
  }
  const float rR = 1.0f / (float)max(nsm, 1), rN = 1.0f / (float)max(g.sc.tokens[a], 1);
  for (int e = threadIdx.x; e < E; e += kSumThreads) fsm[e] *= rR;
  cluster_sync_all();  // rank 0 runs, its psm may be written
  if (q == 0 && c < cols) finish_prob<kSumCluster>(g, a, e0 + c, p * rN, psm);
  cluster_sync_all();
  if (rank == 0) finish_loss<kSumThreads>(g, a, fsm, psm, tsm);
}

#define LAUNCH(call)                                     \
  do {                                                   \
    if ((call) != cudaSuccess) return MOE_LORA_ERR_CUDA; \
  } while (0)

// A launch as a cluster, or overlapping the launch before it in the stream.
struct BalLaunch {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[1];
  BalLaunch(int64_t grid, int threads, size_t smem, int cluster, bool overlap, cudaStream_t s) {
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = at;
    if (overlap) {
      at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
      at[0].val.programmaticStreamSerializationAllowed = 1;
      cfg.numAttrs = 1;
    } else if (cluster > 1) {
      at[0].id = cudaLaunchAttributeClusterDimension;
      at[0].val.clusterDim.x = cluster;
      at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
      cfg.numAttrs = 1;
    }
  }
};

template <class T, RowMode kMode, int kVals, int kC>
int launch_balance(const BalTable& bt, const BalArgs& a, cudaStream_t s) {
  const auto kernel = kMode == kVec16 && a.E == a.lpr * kVals ? balance_kernel<T, kMode, kVals, kC, kMode == kVec16>
                                                              : balance_kernel<T, kMode, kVals, kC, false>;
  constexpr int kT = block_threads(kVals);
  const size_t ring = kMode == kElement ? 0 : (size_t)kT * kBalStages * kVals * sizeof(T);
  const size_t smem = std::max(ring, sizeof(float) * (kT / a.lpr) * (a.E + kSumPad));
  const BalLaunch l((int64_t)bt.group0[bt.n] * (kC ? kC : kBalCluster), kT, smem, kC, kC == 0, s);
  prof_begin(K_BAL_LOSS, s);
  const cudaError_t e = launch_allowed(l.cfg, (kC > 8), kernel, bt, a);
  prof_end(K_BAL_LOSS, s);
  return e == cudaSuccess ? MOE_LORA_OK : MOE_LORA_ERR_CUDA;
}

template <class T, RowMode kMode, int kVals>
int pick_groups(const BalTable& bt, const BalArgs& a, cudaStream_t s) {
  if (bt.group0[bt.n] == bt.n) {
    int most = 1;  // chunks of an adapter
    for (int i = 0; i < bt.n; ++i)
      if (bt.chunk[i]) most = std::max(most, (bt.tok_off[i + 1] - bt.tok_off[i] + bt.chunk[i] - 1) / bt.chunk[i]);
    return most == 1          ? launch_balance<T, kMode, kVals, 1>(bt, a, s)
           : most <= kBalFew ? launch_balance<T, kMode, kVals, kBalFew>(bt, a, s)
                             : launch_balance<T, kMode, kVals, kBalCluster>(bt, a, s);
  }
  prof_begin(K_BAL_COUNT, s);
  balance_count_kernel<<<bt.group0[bt.n] * kCountCluster, kCountThreads, 0, s>>>(bt, a.ids, a.k, a.E, a.sc);
  prof_end(K_BAL_COUNT, s);
  LAUNCH(cudaGetLastError());
  const int rc = launch_balance<T, kMode, kVals, 0>(bt, a, s);
  if (rc) return rc;
  const BalLaunch l((int64_t)bt.n * kSumCluster, kSumThreads, 0, 0, true, s);
  prof_begin(K_BAL_SUM, s);
  const cudaError_t e = cudaLaunchKernelEx(&l.cfg, balance_sum_kernel, bt, a);
  prof_end(K_BAL_SUM, s);
  return e == cudaSuccess ? MOE_LORA_OK : MOE_LORA_ERR_CUDA;
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
    bt.chunk[a] = bal_chunk(n, groups, d->E);
    bt.group0[a + 1] = bt.group0[a] + (int)groups;
  }
  bt.tok_off[d->A] = at.tok_off[d->A];
  const BalArgs a{logits, ld,   topk_ids, d->k, d->E,    0,
                  coef,   dloss, loss,    counts, prob, dlogits, bal_scratch(d, scratch)};
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
