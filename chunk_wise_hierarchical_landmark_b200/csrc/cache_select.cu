// Landmark scoring and selection of the decode step over a cache that grows
// token by token (model card "HiLS-Attention", section "What HiLS-Attention
// is"; molayo1419.me, "Core idea" step 1), with a length per sequence.
//
//   score[h][c] = scale <q_h, lmk_c>  for the completed chunks c < own
//   selection   the topk largest (score desc, chunk asc), the log-sum-exp of all
//   union       of the G heads of a KV head, the own chunk last
//
// cache_scores   bound by the landmark bytes.  The units of 8 KB of landmark rows
//                of all KV heads form one list; every warp takes an equal
//                contiguous range, so short sequences cost nothing.  Units
//                arrive by bulk copies through a ring of three per warp and are
//                multiplied as m16n8k16 (16 rows, the G <= 8 heads as columns).
// cache_select   a cluster of G CTAs per KV head, one head each, its scores in
//                registers (2, 8 or 32 per thread) as order-preserving keys.  A bound
//                that at least K of the threads' largest keys reach is one that
//                at least K scores reach: bisection over the threads' maxima
//                (a barrier that counts, no memory) finds one that few more
//                than K reach, and the scores at or above it, some 1.5 K, are
//                ranked exactly by (score, chunk).  Where too many scores tie,
//                the bisection goes on over all keys, down to the tie, whose
//                lowest chunks are taken.  The heads' bitmaps meet in
//                distributed shared memory: the union needs no launch of its
//                own.
//
// Measured (16 sequences of 512K, 32 / 8 heads, d = 128): scoring 51 us for 268
// MB (5.2 TB/s, 81 % of a plain copy, some 6 us of it start and end), selection
// and union 20 us, of it 16 us the latency of one cluster's chain.  A scoring
// kernel on tcgen05 with 128-landmark tiles takes the same 51 us at full
// batches and three times as long where lengths differ, since its grid follows
// the longest sequence; the tensor pipe is at 7 % here.
#include <cuda_bf16.h>

#include <algorithm>

#include "cache.h"
#include "common.cuh"
#include "pdl.cuh"
#include "sm100.cuh"

namespace hils {
namespace {

using namespace sm100;

constexpr int kC = 64;

__device__ __forceinline__ int seq_len(const DecodeSpec &ds, int b) {
  const int n = ds.lens[b];
  return n < 0 || n > ds.N ? 0 : n;  // out of bounds: an empty sequence
}
// completed chunks of sequence b
__device__ __forceinline__ int n_completed(const DecodeSpec &ds, int b) {
  const int n = seq_len(ds, b);
  return n > 0 ? (n - 1) / kC : 0;
}

// ---------------------------------------------------------------------------
constexpr int kScoreWarps = 4;
constexpr int kScoreCtas = 2;      // CTAs per SM (shared memory)
constexpr int kScoreSlots = 3;     // units in flight or in use per warp
constexpr int kUnitBytes = 8192;   // 32 landmark rows at d = 128, 64 at d = 64

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void bulk_g2s(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

template <int D>
struct ScoreLayout {
  static constexpr int ring = 0;  // [kScoreWarps][kScoreSlots][kUnitBytes]
  static constexpr int bars = kScoreWarps * kScoreSlots * kUnitBytes;
  static constexpr int misc = bars + kScoreWarps * kScoreSlots * 8;  // warp sums, abort flag
  static constexpr int total = misc + 32;
};

// Walks the list of units (b, hkv, first row) in order.
struct UnitWalk {
  int b = 0, before = 0, n_c = 0, nu = 0;  // sequence, units before it, its chunks, units of one head
};

template <int D>
__global__ void __launch_bounds__(kScoreWarps * 32) cache_scores_kernel(
    const DecodeSpec ds, const __nv_bfloat16 *__restrict__ q, const __nv_bfloat16 *__restrict__ lmk,
    float *__restrict__ scores, uint32_t *__restrict__ err) {
  using Lay = ScoreLayout<D>;
  constexpr int V = D / 32;                      // 16-byte pieces of a row per lane
  constexpr int kUnit = kUnitBytes / (2 * D);    // landmark rows per unit
  extern __shared__ __align__(128) unsigned char smem_sc[];
  unsigned char *smem = smem_sc;
  grid_dep_launch();  // the selection may launch (it waits for this grid's scores)
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int G = ds.Hq / ds.Hkv;
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Lay::bars) + warp * kScoreSlots;
  int *sums = reinterpret_cast<int *>(smem + Lay::misc);
  volatile int *abort_flag = sums + kScoreWarps;
  unsigned char *ring = smem + Lay::ring + warp * kScoreSlots * kUnitBytes;
  if (tid == 0) *abort_flag = 0;
  if (lane == 0) {
    for (int i = 0; i < kScoreSlots; ++i) mbar_init(&bars[i], 1);
    fence_mbar_init();
  }
  int total = 0;
  for (int b = tid; b < ds.B; b += kScoreWarps * 32) total += (n_completed(ds, b) + kUnit - 1) / kUnit;
  total = __reduce_add_sync(0xffffffffu, total);
  if (lane == 0) sums[warp] = total;
  __syncthreads();
  total = 0;
#pragma unroll
  for (int w = 0; w < kScoreWarps; ++w) total += sums[w];
  total *= ds.Hkv;
  const int W = min((int)gridDim.x * kScoreWarps, total), wid = blockIdx.x * kScoreWarps + warp;
  if (wid >= W) return;
  const int lo = (int)((long long)total * wid / W), hi = (int)((long long)total * (wid + 1) / W);
  // the sequence of unit lo, 32 sequences per step
  UnitWalk use;
  for (int b0 = 0;; b0 += 32) {
    const int bl = b0 + lane;
    const int nc = bl < ds.B ? n_completed(ds, bl) : 0;
    const int u = ((nc + kUnit - 1) / kUnit) * ds.Hkv;
    int x = u;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, use.before + x > lo);
    if (past) {
      const int l = __ffs(past) - 1;
      use.b = b0 + l;
      use.before += __shfl_sync(0xffffffffu, x - u, l);
      use.n_c = __shfl_sync(0xffffffffu, nc, l);
      break;
    }
    use.before += __shfl_sync(0xffffffffu, x, 31);
  }
  use.nu = (use.n_c + kUnit - 1) / kUnit;
  auto seek = [&](UnitWalk &w, int u) {  // to the sequence of unit u, not before w's
    while (u - w.before >= w.nu * ds.Hkv) {
      w.before += w.nu * ds.Hkv;
      w.n_c = n_completed(ds, ++w.b);
      w.nu = (w.n_c + kUnit - 1) / kUnit;
    }
  };
  UnitWalk ahead = use;  // lane 0's, of the copies
  int issued = lo;
  auto issue = [&]() {
    seek(ahead, issued);
    const int hkv = (issued - ahead.before) / ahead.nu, c0 = ((issued - ahead.before) % ahead.nu) * kUnit;
    const int s = (issued - lo) % kScoreSlots;
    const uint32_t bytes = (uint32_t)min(kUnit, ahead.n_c - c0) * (2 * D);
    mbar_expect_tx(&bars[s], bytes);
    bulk_g2s(ring + s * kUnitBytes, lmk + (((size_t)ahead.b * ds.Hkv + hkv) * ds.nlmk + c0) * D, bytes, &bars[s]);
    ++issued;
  };
  if (lane == 0)
    while (issued < min(hi, lo + kScoreSlots)) issue();
  int cur = -1;  // KV head whose queries are in qf
  uint4 qf[V];
  bool ok = true;
  for (int at = lo; at < hi; ++at) {
    seek(use, at);
    const int hkv = (at - use.before) / use.nu, c0 = ((at - use.before) % use.nu) * kUnit;
    const int bk = use.b * ds.Hkv + hkv, left = use.n_c - c0;
    if (bk != cur) {
      cur = bk;
      const __nv_bfloat16 *qrow = q + ((size_t)use.b * ds.Hq + hkv * G + (g < G ? g : 0)) * D;
#pragma unroll
      for (int i = 0; i < V; ++i)
        qf[i] = g < G ? *reinterpret_cast<const uint4 *>(qrow + 8 * (t + 4 * i)) : make_uint4(0u, 0u, 0u, 0u);
    }
    const int s = (at - lo) % kScoreSlots;
    ok = __all_sync(0xffffffffu, mbar_wait(&bars[s], ((at - lo) / kScoreSlots) & 1, abort_flag));
    if (!ok) break;
    const unsigned char *rows = ring + s * kUnitBytes;
    float acc[kUnit / 16][4];
#pragma unroll
    for (int mt = 0; mt < kUnit / 16; ++mt) {
      acc[mt][0] = acc[mt][1] = acc[mt][2] = acc[mt][3] = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        // rows past `left` hold an earlier unit's bytes: their scores are not written
        const unsigned char *p = rows + (mt * 16 + g) * (2 * D) + 16 * (t + 4 * i);
        const uint4 x = *reinterpret_cast<const uint4 *>(p), y = *reinterpret_cast<const uint4 *>(p + 16 * D);
        mma_bf16(acc[mt], x.x, y.x, x.y, y.y, qf[i].x, qf[i].y);
        mma_bf16(acc[mt], x.z, y.z, x.w, y.w, qf[i].z, qf[i].w);
      }
    }
    __syncwarp();
    if (lane == 0 && issued < hi) issue();
#pragma unroll
    for (int mt = 0; mt < kUnit / 16; ++mt) {
      const int row = mt * 16 + g;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (2 * t + h >= G) continue;
        float *dst = scores + ((size_t)bk * G + 2 * t + h) * ds.n_c + c0;
        if (row < left) dst[row] = acc[mt][h] * ds.scale;
        if (row + 8 < left) dst[row + 8] = acc[mt][2 + h] * ds.scale;
      }
    }
  }
  if (!ok && lane == 0) {
    // a wait gave up: every copy in flight must land before the CTA exits
    for (int u = max(lo, issued - kScoreSlots); u < issued; ++u)
      mbar_wait_bounded(&bars[(u - lo) % kScoreSlots], ((u - lo) / kScoreSlots) & 1);
    report(err, DEV_TIMEOUT);
  }
}

// ---------------------------------------------------------------------------
constexpr int kSelThreads = 256;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kMaxCand = 512;  // candidates ranked exactly
static_assert(kSelectMax == 32 * kSelThreads, "32 scores per thread at most");

// order-preserving 32-bit image of an fp32 score (-0 folded into +0), at least
// 1: 0 ranks below every score
__device__ __forceinline__ uint32_t score_key(float s) {
  const uint32_t x = __float_as_uint(s + 0.0f);
  return max(1u, (x & 0x80000000u) ? ~x : (x | 0x80000000u));
}

__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k);
}

__device__ __forceinline__ uint32_t map_peer(const void *p, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ uint32_t ld_peer(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

// Exclusive prefix of the popcounts of `words` (thread w < kWords passes its
// word); returns the total.  Two barriers.
template <int kWords>
__device__ __forceinline__ int popc_prefix(uint32_t word, int *prefix, int *warp_tot) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  static_assert(kWords <= kSelThreads, "a thread per word");
  const int c = tid < kWords ? __popc(word) : 0;
  int x = c;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_tot[warp] = x;
  __syncthreads();
  int base = 0, total = 0;
#pragma unroll
  for (int w = 0; w < (kWords + 31) / 32; ++w) {
    if (w < warp) base += warp_tot[w];
    total += warp_tot[w];
  }
  if (tid < kWords) prefix[tid] = base + x - c;
  __syncthreads();
  return total;
}

// The cluster's own scoring of a KV head with few chunks: 16 rows per warp and
// step, the scores through global memory to the heads' CTAs.
template <int D>
__device__ __forceinline__ void score_head(const DecodeSpec &ds, const __nv_bfloat16 *__restrict__ q,
                                           const __nv_bfloat16 *__restrict__ lmk, float *scores, int b,
                                           int bk, int rank, int n) {
  constexpr int V = D / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int G = ds.Hq / ds.Hkv, hkv = bk % ds.Hkv;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  const __nv_bfloat16 *qrow = q + ((size_t)b * ds.Hq + hkv * G + (g < G ? g : 0)) * D;
  for (int r0 = (rank * kSelWarps + warp) * 16; r0 < n; r0 += G * kSelWarps * 16) {
    const __nv_bfloat16 *rows = lmk + ((size_t)bk * ds.nlmk + r0) * D;
    uint4 x[V], y[V], w[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int col = 8 * (t + 4 * i);
      x[i] = r0 + g < n ? *reinterpret_cast<const uint4 *>(rows + g * D + col) : zero;
      y[i] = r0 + g + 8 < n ? *reinterpret_cast<const uint4 *>(rows + (g + 8) * D + col) : zero;
      w[i] = g < G ? *reinterpret_cast<const uint4 *>(qrow + col) : zero;
    }
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < V; ++i) {
      mma_bf16(s, x[i].x, y[i].x, x[i].y, y[i].y, w[i].x, w[i].y);
      mma_bf16(s, x[i].z, y[i].z, x[i].w, y[i].w, w[i].z, w[i].w);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (2 * t + h >= G) continue;
      float *dst = scores + ((size_t)bk * G + 2 * t + h) * ds.n_c + r0 + g;
      if (r0 + g < n) dst[0] = s[h] * ds.scale;
      if (r0 + g + 8 < n) dst[8] = s[2 + h] * ds.scale;
    }
  }
}

// kPer: scores per thread, for up to kPer * kSelThreads completed chunks.  D:
// the cluster scores its landmarks itself (0: the scores are there).
template <int kPer, int D>
__global__ void __launch_bounds__(kSelThreads, kPer > 8 || D > 0 ? 4 : 8) cache_select_kernel(
    const DecodeSpec ds, const CacheKV cache, const __nv_bfloat16 *__restrict__ q, float *scores,
    int32_t *__restrict__ sel, float *__restrict__ chunk_w, float *__restrict__ lse_lmk,
    int32_t *__restrict__ u_c, uint32_t *__restrict__ u_mask, float *__restrict__ u_logit,
    int32_t *__restrict__ u_count, uint4 *__restrict__ ent, int *__restrict__ next,
    uint32_t *__restrict__ err) {
  constexpr int kWords = kPer * kSelWarps;  // bitmap words
  __shared__ uint32_t keep[kWords];  // the head's selection, read by its cluster,
  __shared__ int place[kWords];      // and the chunks before each word of it
  __shared__ uint32_t eq[kWords];
  __shared__ int prefix[kWords];
  __shared__ int warp_tot[kSelWarps];
  __shared__ float redl[kSelWarps];
  __shared__ uint32_t redlo[kSelWarps], redhi[kSelWarps];
  __shared__ int cnt[2][kSelWarps], n_cand;
  __shared__ __align__(16) uint64_t cand[kMaxCand];  // (key, ~chunk): larger ranks first
  __shared__ uint32_t list[kSelectMaxG * 64];  // union chunks and their heads,
  __shared__ uint2 places[kSelectMaxG * 64];   // and their places in the heads' selections
  const int G = ds.Hq / ds.Hkv, K = ds.topk;
  const int bk = blockIdx.x / G, rank = blockIdx.x % G;  // one cluster per KV head
  const int b = bk / ds.Hkv, hkv = bk % ds.Hkv, h = b * ds.Hq + hkv * G + rank;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int len = seq_len(ds, b), own = len > 0 ? (len - 1) / kC : -1, n = max(0, own);
  const float *sc = scores + (size_t)h * ds.n_c;
  int32_t *srow = sel + (size_t)h * K;
  float *wrow = chunk_w + (size_t)h * K;
  grid_dep_launch();
  for (int i = tid; i < kWords; i += kSelThreads) keep[i] = 0u;
  if (tid == 0) n_cand = 0;
  if (n < K)  // padding
    for (int i = n + tid; i < K; i += kSelThreads) {
      srow[i] = -1;
      wrow[i] = -INFINITY;
    }
  if constexpr (D > 0) {
    score_head<D>(ds, q, static_cast<const __nv_bfloat16 *>(cache.lmk), scores, b, bk, rank, n);
    cluster_sync();
  } else {
    grid_dep_wait();  // the scores
  }
  // thread tid holds the keys of chunks i * kSelThreads + tid (0: none); the
  // log-sum-exp first, each thread's sum against its own maximum
  uint32_t key[kPer], top = 0u;
  float m = -INFINITY, l = 0.0f;
  {
    float v[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int c = i * kSelThreads + tid;
      v[i] = c < n ? sc[c] : -INFINITY;
      m = fmaxf(m, v[i]);
    }
    const float ref = m == -INFINITY ? 0.0f : m;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (i * kSelThreads < n) l += __expf(v[i] - ref);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      key[i] = i * kSelThreads + tid < n ? score_key(v[i]) : 0u;
      top = max(top, key[i]);
    }
  }
  // the block's largest key, and the least of the threads' largest ones (of the
  // min(n, 256) > K threads that have any, where there is something to select)
  const uint32_t wl = __reduce_min_sync(0xffffffffu, top ? top : 0xFFFFFFFFu);
  const uint32_t wh = __reduce_max_sync(0xffffffffu, top);
  if (lane == 0) {
    redlo[warp] = wl;
    redhi[warp] = wh;
  }
  __syncthreads();
  uint32_t lo = 0xFFFFFFFFu, hi = 0u;
#pragma unroll
  for (int w = 0; w < kSelWarps; ++w) {
    lo = min(lo, redlo[w]);
    hi = max(hi, redhi[w]);
  }
  {
    const float bm = key_value(hi);
    l = m == -INFINITY ? l : l * __expf(m - bm);
#pragma unroll
    for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (lane == 0) redl[warp] = l;
    __syncthreads();
    if (tid == 0 && lse_lmk) {
      float lt = 0.0f;
#pragma unroll
      for (int w = 0; w < kSelWarps; ++w) lt += redl[w];
      lse_lmk[h] = n > 0 ? bm + __logf(lt) : -INFINITY;
    }
  }
  int nc = kMaxCand + 1;  // candidates, when they were ranked
  if (n <= K) {
    // every completed chunk (they are the first thread-row's)
    const uint32_t kb = __ballot_sync(0xffffffffu, key[0] != 0u);
    if (lane == 0) keep[warp] = kb;
  } else {
    // at least K of the threads' maxima reach lo throughout
    uint32_t top_hi = hi;
    while (lo < top_hi) {
      const uint32_t mid = lo + (top_hi - lo + 1) / 2;
      const int c = __syncthreads_count(top >= mid);
      if (c < K) {
        top_hi = mid - 1;
      } else {
        lo = mid;
        if (c <= K + K / 4) break;
      }
    }
    // the candidates, in any order; ranked exactly below
    int mine_n = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) mine_n += key[i] >= lo && key[i] != 0u ? 1 : 0;
    if (mine_n) {
      int at = atomicAdd(&n_cand, mine_n);
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (key[i] >= lo && key[i] != 0u) {
          if (at < kMaxCand) cand[at] = ((uint64_t)key[i] << 32) | (0xFFFFFFFFu - (uint32_t)(i * kSelThreads + tid));
          ++at;
        }
    }
    __syncthreads();
    nc = n_cand;
    if (nc <= kMaxCand) {
      // four lanes per candidate, each against a quarter of the others
      for (int a0 = 0; a0 < nc; a0 += kSelThreads / 4) {
        const int a = a0 + (tid >> 2);
        const uint64_t x = a < nc ? cand[a] : ~0ull;
        int r = 0;
#pragma unroll 8
        for (int j = tid & 3; j < nc; j += 4) r += cand[j] > x ? 1 : 0;
        r += __shfl_xor_sync(0xffffffffu, r, 1);
        r += __shfl_xor_sync(0xffffffffu, r, 2);
        if (a < nc && (tid & 3) == 0 && r < K) {
          const uint32_t c = 0xFFFFFFFFu - (uint32_t)x;
          atomicOr(&keep[c >> 5], 1u << (c & 31u));
        }
      }
    } else {
      // many equal scores: the largest bound that at least K keys reach, by
      // bisection over all of them, then the lowest chunks of those on it
      int buf = 0;
      auto count = [&](uint32_t x) {
        int c = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) c += key[i] >= x ? 1 : 0;
        c = __reduce_add_sync(0xffffffffu, c);
        if (lane == 0) cnt[buf][warp] = c;
        __syncthreads();
        c = 0;
#pragma unroll
        for (int w = 0; w < kSelWarps; ++w) c += cnt[buf][w];
        buf ^= 1;
        return c;
      };
      lo = max(lo, 1u);
      while (lo < hi) {
        const uint32_t mid = lo + (hi - lo + 1) / 2;
        if (count(mid) >= K) lo = mid;
        else hi = mid - 1;
      }
      const int need = K - (lo == 0xFFFFFFFFu ? 0 : count(lo + 1));  // of the keys equal to lo
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const uint32_t kb = __ballot_sync(0xffffffffu, key[i] > lo), eb = __ballot_sync(0xffffffffu, key[i] == lo);
        if (lane == 0) {
          keep[i * kSelWarps + warp] = kb;
          eq[i * kSelWarps + warp] = eb;
        }
      }
      __syncthreads();
      popc_prefix<kWords>(tid < kWords ? eq[tid] : 0u, prefix, warp_tot);
      if (tid < kWords) {
        uint32_t e = eq[tid], take = 0u;
        for (int r = need - prefix[tid]; r > 0 && e; --r) {
          take |= e & (0u - e);
          e &= e - 1u;
        }
        keep[tid] |= take;
      }
    }
  }
  __syncthreads();
  // the selection in chunk order
  popc_prefix<kWords>(tid < kWords ? keep[tid] : 0u, place, warp_tot);
  auto put = [&](uint32_t k, int c) {
    const uint32_t word = keep[c >> 5];
    if ((word >> (c & 31)) & 1u) {
      const int pos = place[c >> 5] + __popc(word & ((1u << (c & 31)) - 1u));
      srow[pos] = c;
      wrow[pos] = key_value(k);
    }
  };
  if (nc <= kMaxCand) {
    for (int a = tid; a < nc; a += kSelThreads) put((uint32_t)(cand[a] >> 32), (int)(0xFFFFFFFFu - (uint32_t)cand[a]));
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (i * kSelThreads < n) put(key[i], i * kSelThreads + tid);
  }
  // ---- union of the cluster's heads
  static_assert(kSelectMax <= 1 << 16, "a chunk id in 16 bits");
  cluster_sync();
  uint32_t mine[kSelectMaxG], all = 0u;
  int at[kSelectMaxG];
#pragma unroll
  for (int g = 0; g < kSelectMaxG; ++g) {
    mine[g] = 0u;
    at[g] = 0;
    if (g < G && tid < kWords) {
      mine[g] = ld_peer(map_peer(&keep[tid], (uint32_t)g));
      if (ent) at[g] = (int)ld_peer(map_peer(&place[tid], (uint32_t)g));
    }
    all |= mine[g];
  }
  cluster_sync();  // every peer has been read: a CTA may end
  const int total = popc_prefix<kWords>(all, prefix, warp_tot);
  const size_t u0 = (size_t)bk * ds.ucap;
  if (tid < kWords) {
    int pos = prefix[tid];
    for (uint32_t rest = all; rest; rest &= rest - 1u, ++pos) {
      const int bit = __ffs(rest) - 1;
      uint32_t mask = 0u, lo8 = 0u, hi8 = 0u;
#pragma unroll
      for (int g = 0; g < kSelectMaxG; ++g) {
        const uint32_t in = (mine[g] >> bit) & 1u;
        mask |= in << g;
        (g < 4 ? lo8 : hi8) |= (uint32_t)at[g] << (8 * (g & 3));
        at[g] += (int)in;
      }
      list[pos] = (uint32_t)(tid * 32 + bit) | (mask << 16);
      places[pos] = make_uint2(lo8, hi8);
    }
  }
  __syncthreads();
  // the entries one by one, every G-th by this CTA
  for (int i = tid * G + rank; i < total; i += kSelThreads * G) {
    const int c = (int)(list[i] & 0xFFFFu);
    const uint32_t mask = list[i] >> 16;
    if (ent) {
      uint4 e = make_uint4((uint32_t)kEntNoPage, mask, 0u, 0u);
      const long long page = cache.table[(size_t)b * cache.max_pages + c];
      if (page >= 0 && page < cache.num_pages) {
        const size_t blk = (size_t)page * ds.Hkv + hkv;
        e.x = (uint32_t)blk;
        if (cache.q8) {
          e.z = __float_as_uint(cache.k_scale[blk]);
          e.w = __float_as_uint(cache.v_scale[blk]);
        }
      } else {
        report(err, DEV_BAD_INDEX);
      }
      ent[2 * (u0 + i)] = e;
      ent[2 * (u0 + i) + 1] = make_uint4(places[i].x, places[i].y, 0u, 0u);
    } else {
#pragma unroll
      for (int g = 0; g < kSelectMaxG; ++g)
        if ((mask >> g) & 1u) u_logit[(u0 + i) * G + g] = scores[((size_t)bk * G + g) * ds.n_c + c];
      u_c[u0 + i] = c;
      u_mask[u0 + i] = mask;
    }
  }
  if (rank == 0 && tid == 0) {
    if (own >= 0 && !ent) {  // every head attends its own chunk
      u_c[u0 + total] = own;
      u_mask[u0 + total] = (1u << G) - 1u;
    }
    u_count[bk] = own >= 0 ? total + 1 : 0;
    if (bk == 0 && next) *next = 0;
  }
}

}  // namespace

// Few enough landmarks per KV head for its cluster to score them itself, which
// saves a launch (a step of 1000 tokens 17.9 -> 16.9 us on the device, 45 ->
// 41 us with the host's part).  This and the scores per thread below go by ds.n_c,
// the bound that the call gives for its sequences; their lengths are on the device.
// Room for more costs a step of 1000 tokens 14.4 -> 15.6 us (128K), 17.0 us
// (512K) and, by the radix select past 8192 chunks, 19.7 us (1M), a batch of
// lengths up to 128K 88.5 -> 96.0 us (512K) and 100.6 us (1M).
bool cache_select_scores(const DecodeSpec &ds, bool bf16) { return bf16 && ds.n_c <= 2 * kSelThreads; }

cudaError_t cache_scores(const DecodeSpec &ds, const void *q, const void *lmk, float *scores,
                         uint32_t *err, cudaStream_t st) {
  const int unit = kUnitBytes / (2 * ds.d);
  const long long units = (long long)ds.B * ds.Hkv * ((ds.n_c + unit - 1) / unit);  // at most
  const unsigned ctas = (unsigned)std::min((units + kScoreWarps - 1) / kScoreWarps, (long long)148 * kScoreCtas);
  cudaError_t e;
#define HILS_SCORES(DD)                                                                          \
  do {                                                                                           \
    const size_t smem = ScoreLayout<DD>::total;                                                  \
    if ((e = cudaFuncSetAttribute(cache_scores_kernel<DD>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) != cudaSuccess) return e; \
    cache_scores_kernel<DD><<<ctas, kScoreWarps * 32, smem, st>>>(                               \
        ds, (const __nv_bfloat16 *)q, (const __nv_bfloat16 *)lmk, scores, err);                  \
  } while (0)
  if (ds.d == 64) HILS_SCORES(64); else HILS_SCORES(128);
#undef HILS_SCORES
  return cudaGetLastError();
}

cudaError_t cache_select(const DecodeSpec &ds, const CacheKV &cache, bool bf16, const void *q,
                         float *scores, int32_t *sel, float *w, float *lse_lmk, int32_t *u_c,
                         uint32_t *u_mask, float *u_logit, int32_t *u_count, uint4 *ent,
                         int *next, uint32_t *err, cudaStream_t st) {
  const int G = ds.Hq / ds.Hkv;
  const bool own_scores = cache_select_scores(ds, bf16);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(ds.B * ds.Hq));
  cfg.blockDim = dim3(kSelThreads);
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)G;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = ds.n_c > 0 && !own_scores ? 2 : 1;  // behind the scoring launch
  auto kern = own_scores ? (ds.d == 64 ? cache_select_kernel<2, 64> : cache_select_kernel<2, 128>)
              : ds.n_c <= 2 * kSelThreads ? cache_select_kernel<2, 0>
              : ds.n_c <= 8 * kSelThreads ? cache_select_kernel<8, 0> : cache_select_kernel<32, 0>;
  return cudaLaunchKernelEx(&cfg, kern, ds, cache, (const __nv_bfloat16 *)q, scores, sel, w, lse_lmk, u_c,
                            u_mask, u_logit, u_count, ent, next, err);
}

}  // namespace hils
