// Chunk attention of the decode step over a cache that grows token by token
// (aiweekly.co, mechanism paragraph: attention to each retrieved chunk
// independently, outputs fused by the chunk scores).  Per union entry (chunk
// c, heads that attend it) of a KV head:
//
//   x_j = scale <q, k_j>,  m = max x_j,  l = sum exp(x_j - m),
//   o = sum exp(x_j - m) v_j / l,  fusion logit = landmark logit, or m + log l
//   for the own chunk (its keys up to the newest token)
//
// and a combine fuses a head's chunks under their logits.  In the 8-bit
// form k_j = code * s_K, v_j = code * s_V with one power of two per block:
// s_K multiplies the logits and s_V the chunk's output, so the codes
// themselves enter the products.  The own chunk comes from the sequence's
// full-precision tail.  bf16 pages take the same kernel; fp32 pages take
// decode.cu's chunk attention.
//
// Bound by the bytes of the attended blocks.  Measured (16 sequences of 512K,
// 32 / 8 heads, d = 128, top 64, 8 bits): 93 us for 531 MB, 5.7 TB/s, 88 % of a
// plain copy; a quarter of the batch takes 32 us, so beyond some 12 us of start
// and end the rate is the copy's.  The tensor pipe is at 21 %: the G <= 8 heads
// of a KV head fill the 8 columns of m16n8k16, where a tcgen05 tile of 128 rows
// would be filled to a sixteenth by heads, or need the 64 keys of two chunks
// that other heads attend.
#include <cuda_bf16.h>

#include <algorithm>

#include "cache.h"
#include "common.cuh"
#include "e4m3.cuh"
#include "pdl.cuh"
#include "sm100.cuh"

namespace hils {
namespace {

using namespace sm100;

constexpr int kC = 64;
constexpr int kMaxG = 8;
constexpr int kMaxEntries = kCacheMaxEntries;  // union entries of an fp32 CTA's share
constexpr int kThreads = 128;

// Tokens of sequence b; a length outside [0, N] counts as an empty sequence.
__device__ __forceinline__ int seq_len(const DecodeSpec &ds, int b) {
  const int n = ds.lens[b];
  return n < 0 || n > ds.N ? 0 : n;
}

__device__ __forceinline__ void tma_load_3d(void *dst, const CUtensorMap *map, uint64_t *bar, int x,
                                            int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// Where the 64 rows of a union entry lie.
struct EntrySrc {
  const void *k, *v;  // [64][D] codes, or the tail's fp32 rows; nullptr: page outside the pool
  bool codes;
  float sk, sv;       // block scales (1 for the tail)
  int rows;           // valid rows (the own chunk of a sequence may be partial)
};

template <int D>
__device__ __forceinline__ EntrySrc entry_src(const DecodeSpec &ds, const CacheKV &c, int b,
                                              int hkv, int chunk, int len, uint32_t *err) {
  EntrySrc e;
  const int own = (len - 1) / kC;
  e.rows = chunk == own ? len - own * kC : kC;
  e.sk = e.sv = 1.0f;
  e.codes = chunk != own;
  if (chunk == own) {
    const size_t off = ((((size_t)b * 2 + (chunk & 1)) * ds.Hkv + hkv) * kC) * D;
    e.k = static_cast<const float *>(c.k_tail) + off;
    e.v = static_cast<const float *>(c.v_tail) + off;
    return e;
  }
  const long long page = c.table[(size_t)b * c.max_pages + chunk];
  if (page < 0 || page >= c.num_pages) {
    report(err, DEV_BAD_INDEX);
    e.k = e.v = nullptr;
    return e;
  }
  const size_t blk = (size_t)page * ds.Hkv + hkv;
  e.k = static_cast<const uint8_t *>(c.k_pages) + blk * kC * D;
  e.v = static_cast<const uint8_t *>(c.v_pages) + blk * kC * D;
  e.sk = c.k_scale[blk];
  e.sv = c.v_scale[blk];
  return e;
}

// ---------------------------------------------------------------------------
// CUDA-core form (fp32 parameters, for which the tensor cores have no exact
// product): a chunk is widened to fp32 in shared memory, then a thread
// per key for the logits, a warp per head for the softmax, a thread per
// column for P V.
template <int D>
struct SimtSmem {
  static constexpr int kRow = D + 4;  // padded row of K: 16-byte reads of 8 rows hit 32 banks
  float ks[kC * kRow];
  float vs[kC * D];
  float qs[kMaxG * D];
  float xs[kMaxG * kC];
  float so[kMaxG], sn[kMaxG], M[kMaxG], L[kMaxG];
  EntrySrc src[kMaxEntries];
};

// rows [64][D] into fp32 shared memory, zero past `rows`
template <int D>
__device__ __forceinline__ void stage_rows(const EntrySrc &e, const void *p, float *dst, int ld) {
  constexpr int kVec = D / 4;  // four elements at a time
  for (int i = threadIdx.x; i < kC * kVec; i += kThreads) {
    const int r = i / kVec, x = (i % kVec) * 4;
    float4 f = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (r < e.rows) {
      if (e.codes) {
        const uint32_t w = *reinterpret_cast<const uint32_t *>(static_cast<const uint8_t *>(p) + r * D + x);
        f = e4m3x4_to_f32(w);
      } else {
        f = *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + r * D + x);
      }
    }
    *reinterpret_cast<float4 *>(dst + r * ld + x) = f;
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads) cache_attn_simt_kernel(
    const DecodeSpec ds, const CacheKV c, const float *__restrict__ q,
    const int32_t *__restrict__ u_c, const uint32_t *__restrict__ u_mask,
    const float *__restrict__ u_logit, const int32_t *__restrict__ u_count,
    float *__restrict__ part, uint32_t *__restrict__ err) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  SimtSmem<D> &s = *reinterpret_cast<SimtSmem<D> *>(smem_raw);
  const int G = ds.Hq / ds.Hkv;
  const int qi = blockIdx.x, bk = blockIdx.y;
  const int b = bk / ds.Hkv, hkv = bk % ds.Hkv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int len = seq_len(ds, b), own = len > 0 ? (len - 1) / kC : -1;
  for (int i = tid; i < G * D; i += kThreads)
    s.qs[i] = q[((size_t)b * ds.Hq + hkv * G) * D + i] * ds.scale;
  if (tid < kMaxG) {
    s.M[tid] = -INFINITY;
    s.L[tid] = 0.0f;
  }
  if (qi == 0 && hkv == 0 && tid == 0 && (ds.lens[b] < 0 || ds.lens[b] > ds.N)) report(err, DEV_BAD_INDEX);
  grid_dep_launch();
  grid_dep_wait();  // the union
  const int i0 = qi * ds.epc, i1 = min(u_count[bk], i0 + ds.epc);
  if (tid < i1 - i0)
    s.src[tid] = entry_src<D>(ds, c, b, hkv, u_c[(size_t)bk * ds.ucap + i0 + tid], len, err);
  constexpr int NPART = kThreads / D < 1 ? 1 : kThreads / D;  // head groups of the P V pass
  constexpr int HPT = kMaxG / NPART;
  const int col = tid % D, hp = tid / D;
  float acc[HPT];
#pragma unroll
  for (int u = 0; u < HPT; ++u) acc[u] = 0.0f;
  __syncthreads();
  for (int i = i0; i < i1; ++i) {
    const EntrySrc &e = s.src[i - i0];
    if (!e.k) continue;  // a page outside the pool takes no part
    const size_t ue = (size_t)bk * ds.ucap + i;
    const uint32_t mask = u_mask[ue];
    stage_rows<D>(e, e.k, s.ks, SimtSmem<D>::kRow);
    stage_rows<D>(e, e.v, s.vs, D);
    __syncthreads();
    for (int g = tid / kC; g < G; g += kThreads / kC) {
      if (!((mask >> g) & 1u)) continue;
      const float *kr = s.ks + (tid % kC) * SimtSmem<D>::kRow, *qg = s.qs + g * D;
      float x = 0.0f;
#pragma unroll 8
      for (int d = 0; d < D; d += 4) {
        const float4 a = *reinterpret_cast<const float4 *>(kr + d), z = *reinterpret_cast<const float4 *>(qg + d);
        x = fmaf(a.x, z.x, x);
        x = fmaf(a.y, z.y, x);
        x = fmaf(a.z, z.z, x);
        x = fmaf(a.w, z.w, x);
      }
      s.xs[g * kC + tid % kC] = x * e.sk;
    }
    __syncthreads();
    for (int g = warp; g < G; g += kThreads / 32) {
      if (!((mask >> g) & 1u)) continue;
      const float x0 = lane < e.rows ? s.xs[g * kC + lane] : -INFINITY;
      const float x1 = lane + 32 < e.rows ? s.xs[g * kC + lane + 32] : -INFINITY;
      float m = fmaxf(x0, x1);
      for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      const float ref = m == -INFINITY ? 0.0f : m;  // every logit -inf: a sum of 0
      const float e0 = __expf(x0 - ref), e1 = __expf(x1 - ref);
      float l = e0 + e1;
      for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
      s.xs[g * kC + lane] = e0;
      s.xs[g * kC + lane + 32] = e1;
      if (lane == 0) {
        const int chunk = u_c[ue];
        const float lg = chunk == own ? m + __logf(l) : u_logit[ue * G + g];
        s.so[g] = 1.0f;
        s.sn[g] = 0.0f;
        if (lg != -INFINITY) {  // otherwise its weight is 0
          const float mn = fmaxf(s.M[g], lg);
          const float w = __expf(lg - mn);
          s.so[g] = __expf(s.M[g] - mn);
          s.sn[g] = w / l;
          s.L[g] = s.L[g] * s.so[g] + w;
          s.M[g] = mn;
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < HPT; ++u) {
      const int g = hp + u * NPART;
      if (g >= G || !((mask >> g) & 1u)) continue;
      float o = 0.0f;
#pragma unroll 8
      for (int j = 0; j < kC; ++j) o = fmaf(s.xs[g * kC + j], s.vs[j * D + col], o);
      // weight 0: no part of its values, also of infinities and NaN (0 times them is NaN)
      acc[u] = acc[u] * s.so[g] + (s.sn[g] == 0.0f ? 0.0f : s.sn[g] * (o * e.sv));
    }
    __syncthreads();
  }
  __syncthreads();
  const size_t rec = 2 + D;
#pragma unroll
  for (int u = 0; u < HPT; ++u) {
    const int g = hp + u * NPART;
    if (g < G) part[(((size_t)bk * ds.Q + qi) * G + g) * rec + 2 + col] = acc[u];
  }
  if (tid < G) {
    float *r = part + (((size_t)bk * ds.Q + qi) * G + tid) * rec;
    r[0] = s.M[tid];
    r[1] = s.L[tid];
  }
}

// ---------------------------------------------------------------------------
// Tensor-core form (bf16 parameters).  One warp takes a whole chunk; a CTA's
// four warps take the chunks of its share in turn.
//   copies   K and V blocks (64 d bytes each) arrive by tensor copies into a
//            ring of three slots per warp, so while a block is used the next
//            two are in flight; the hardware swizzle spreads the fragment
//            reads over the banks
//   logits   m16n8k16 with A = 16 keys x 16 dims, B = dims x 8 heads: e4m3
//            codes widen to fp16 exactly; the queries of a head are scaled by
//            a power of two to a largest value in [2^14, 2^15), so a bf16
//            query is exact in fp16 down to 2^-28 of it (below: 2^-39 of it)
//   softmax  the 64 logits of a head lie in the eight lanes of equal t
//   P V      A = 16 dims x 16 keys (two rows interleaved byte by byte), B =
//            keys x 8 heads, the logits' fragments transposed in registers;
//            probabilities times 2^15 in two fp16 parts (22 bits), accumulated
//            in fp32; 1 / l, of the same scaled probabilities in fp32, takes the
//            factor out again.  (One part, 11 bits, is off by up to 1.2e-4 of
//            the values' mean magnitude, two by 1e-8; its step of 16 x 512K
//            takes 166.2 instead of 167.1 us.)
// The order of the 16 keys of a step is free as long as K and V agree: row g
// of the fragment is key kperm(g), which keeps both the K reads (16 bytes of
// 8 rows) and the V reads clear of bank conflicts at d = 128.
constexpr int kWarps = kCacheWarps;
constexpr int kSlots = 3;
constexpr int kMaxSeg = 768;  // KV heads in a CTA's sight
static_assert(kMaxSeg >= kWarps * kCacheMaxPer + 8, "a CTA's part of the list");

__device__ __forceinline__ int kperm(int g) { return (g & 1) ? ((g - 1) ^ 5) : g; }

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// 8x8 transpose of 16-bit elements spread over the warp
__device__ __forceinline__ uint32_t movm(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t pack_h2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t pack_b2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}

template <int D, bool Q8>
struct MmaLayout {
  // an item is a K or V block of codes, or 64 columns of a bf16 one
  static constexpr int kItem = Q8 ? kC * D : kC * 128;
  static constexpr int kItems = Q8 ? 2 : 2 * (D / 64);  // items per entry, K first
  static constexpr int ring = 0;                        // [kWarps][kSlots][kItem]
  static constexpr int bars = ring + kWarps * kSlots * kItem;
  static constexpr int seg = bars + kWarps * kSlots * 8;  // KV heads of the CTA's range: index, first entry
  static constexpr int misc = seg + kMaxSeg * 8;
  static constexpr int total = misc + 64;
  static_assert(kItem % 1024 == 0, "swizzled blocks are 1024-byte aligned");
  static_assert(kWarps * kMaxG * (D + 2) * 4 <= bars, "the own chunk's merge uses the ring");
};

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Two heads' softmax over 16 MTS keys: s are the fragments of q k (rows =
// keys, columns = heads 2t, 2t+1; -inf: a masked key), f the positive factors
// that make logits of them.  On return s holds 2^kShift exp(x - m) and l its
// sum; m is the largest logit (natural units), -inf where no key is left.
template <int MTS, int kShift>
__device__ __forceinline__ void softmax_keys(float (&s)[MTS][4], const float (&f)[2], float (&m)[2],
                                             float (&l)[2]) {
  constexpr float kLog2e = 1.4426950408889634f;
  float off[2], f2[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float x = -INFINITY;
#pragma unroll
    for (int mt = 0; mt < MTS; ++mt) x = max3f(x, s[mt][h], s[mt][2 + h]);
#pragma unroll
    for (int o = 4; o <= 16; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    m[h] = x * f[h];
    f2[h] = f[h] * kLog2e;
    off[h] = x == -INFINITY ? 0.0f : x * f2[h] - (float)kShift;
    l[h] = 0.0f;
  }
#pragma unroll
  for (int mt = 0; mt < MTS; ++mt)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s[mt][i] = ex2(fmaf(s[mt][i], f2[i & 1], -off[i & 1]));
      l[i & 1] += s[mt][i];
    }
#pragma unroll
  for (int o = 4; o <= 16; o <<= 1) {
    l[0] += __shfl_xor_sync(0xffffffffu, l[0], o);
    l[1] += __shfl_xor_sync(0xffffffffu, l[1], o);
  }
}

// The own chunk of KV head bk: up to 64 bf16 rows of the tail or its page.  A warp takes
// 16 keys, its K and V rows requested together; the probabilities are split
// into two bf16 parts (16 bits); the warps meet in shared memory.  Depends on
// the step's inputs only, so it runs beside the selection.
template <int D, bool Q8>
__device__ __forceinline__ void own_chunk(const DecodeSpec &ds, const CacheKV &c,
                                          const __nv_bfloat16 *__restrict__ q, int bk,
                                          unsigned char *smem, float *__restrict__ rec,
                                          uint32_t *err) {
  constexpr int MT = D / 16, DG = D / 8, kRec = D + 2;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int G = ds.Hq / ds.Hkv, b = bk / ds.Hkv, hkv = bk % ds.Hkv;
  const int len = seq_len(ds, b);
  if (len == 0) return;
  const int own = (len - 1) / kC, rows = len - own * kC;
  size_t off = ((((size_t)b * 2 + (own & 1)) * ds.Hkv + hkv) * kC) * D;
  if (!Q8) {
    const long long page = c.table[(size_t)b * c.max_pages + own];
    if (page < 0 || page >= c.num_pages) {  // takes no part
      if (tid == 0) report(err, DEV_BAD_INDEX);
      for (int i = tid; i < G * kRec; i += kWarps * 32) rec[i] = i % kRec ? 0.0f : -INFINITY;
      return;
    }
    off = ((size_t)page * ds.Hkv + hkv) * kC * D;
  }
  const __nv_bfloat16 *kt = static_cast<const __nv_bfloat16 *>(Q8 ? c.k_tail : c.k_pages) + off;
  const __nv_bfloat16 *vt = static_cast<const __nv_bfloat16 *>(Q8 ? c.v_tail : c.v_pages) + off;
  const __nv_bfloat16 *qrow = q + ((size_t)b * ds.Hq + hkv * G + (g < G ? g : 0)) * D;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  const int k0 = warp * 16, ra = k0 + kperm(g);  // this lane's K rows: ra, ra + 8
  const int k4[4] = {k0 + kperm(2 * t), k0 + kperm(2 * t + 1), k0 + kperm(2 * t) + 8, k0 + kperm(2 * t + 1) + 8};
  uint4 x[D / 32], y[D / 32], w[D / 32], v[DG / 8][4];
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    const int col = 8 * (t + 4 * i);
    x[i] = ra < rows ? *reinterpret_cast<const uint4 *>(kt + ra * D + col) : zero;
    y[i] = ra + 8 < rows ? *reinterpret_cast<const uint4 *>(kt + (ra + 8) * D + col) : zero;
    w[i] = g < G ? *reinterpret_cast<const uint4 *>(qrow + col) : zero;
  }
#pragma unroll
  for (int h = 0; h < DG / 8; ++h)
#pragma unroll
    for (int u = 0; u < 4; ++u)
      v[h][u] = k4[u] < rows ? *reinterpret_cast<const uint4 *>(vt + k4[u] * D + DG * g + 8 * h) : zero;
  float s[1][4] = {{0.0f, 0.0f, 0.0f, 0.0f}};
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    mma_bf16(s[0], x[i].x, y[i].x, x[i].y, y[i].y, w[i].x, w[i].y);
    mma_bf16(s[0], x[i].z, y[i].z, x[i].w, y[i].w, w[i].z, w[i].w);
  }
  if (ra >= rows) s[0][0] = s[0][1] = -INFINITY;
  if (ra + 8 >= rows) s[0][2] = s[0][3] = -INFINITY;
  const float f[2] = {ds.scale, ds.scale};
  float m[2], l[2], o[MT][4];
  softmax_keys<1, 0>(s, f, m, l);
  uint32_t ph[2], pl[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const float a = s[0][2 * u], z = s[0][2 * u + 1];
    const uint32_t hi = pack_b2(a, z);
    ph[u] = movm(hi);
    pl[u] = movm(pack_b2(a - __uint_as_float(hi << 16), z - __uint_as_float(hi & 0xFFFF0000u)));
  }
#pragma unroll
  for (int h = 0; h < DG / 8; ++h) {
    uint32_t vw[4][4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      vw[u][0] = v[h][u].x;
      vw[u][1] = v[h][u].y;
      vw[u][2] = v[h][u].z;
      vw[u][3] = v[h][u].w;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t a0 = __byte_perm(vw[0][e], vw[1][e], 0x5410), a1 = __byte_perm(vw[0][e], vw[1][e], 0x7632);
      const uint32_t a2 = __byte_perm(vw[2][e], vw[3][e], 0x5410), a3 = __byte_perm(vw[2][e], vw[3][e], 0x7632);
      float (&oe)[4] = o[4 * h + e];
      oe[0] = oe[1] = oe[2] = oe[3] = 0.0f;
      mma_bf16(oe, a0, a1, a2, a3, ph[0], ph[1]);
      mma_bf16(oe, a0, a1, a2, a3, pl[0], pl[1]);
    }
  }
  float *fin = reinterpret_cast<float *>(smem);  // [kWarps][8][D + 2]: m, l, o
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float *r = fin + (warp * kMaxG + 2 * t + h) * kRec;
    if (g == 0) *reinterpret_cast<float2 *>(r) = make_float2(m[h], l[h]);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
      *reinterpret_cast<float2 *>(r + 2 + DG * g + 2 * mt) = make_float2(o[mt][h], o[mt][2 + h]);
  }
  __syncthreads();
  for (int i = tid; i < G * D; i += kWarps * 32) {
    const int hd = i / D, e = i % D;
    const float *r = fin + hd * kRec;
    float mm = r[0], ll = 0.0f, oo = 0.0f;  // the first warp has a key
#pragma unroll
    for (int wi = 1; wi < kWarps; ++wi) mm = fmaxf(mm, r[wi * kMaxG * kRec]);
#pragma unroll
    for (int wi = 0; wi < kWarps; ++wi) {
      const float *rw = r + wi * kMaxG * kRec;
      const float a = rw[0] == -INFINITY ? 0.0f : __expf(rw[0] - mm);
      ll += a * rw[1];
      oo += a * rw[2 + e];
    }
    // one entry of the fusion: logit m + log l, weight 1, output o / l (every
    // token's logit -inf: l = 0, the logit -inf, the output of no weight 0)
    rec[hd * kRec + 2 + e] = ll == 0.0f ? 0.0f : oo / ll;
    if (e == 0) *reinterpret_cast<float2 *>(rec + hd * kRec) = make_float2(mm + __logf(ll), 1.0f);
  }
}

// The first B Hkv CTAs take the own chunks (records of their own, own_part).
// The selected chunks of all KV heads form one list, in (b, hkv, chunk) order,
// which the warps of the other CTAs share out: half in equal parts, the rest in
// ever smaller claims on a counter, since SMs do not get equal shares of the
// memory (16 sequences of 512K: equal parts alone ended between 64 and 97 us
// after the start, 78 on average, with claims between 86 and 90; the step 172 ->
// 167 us).  Every chunk's output for a head is a record of its own, in the
// place of the chunk in the head's selection: who computes it leaves no trace
// in the result.  A warp's copies run on from claim to claim.  Past kMaxSeg KV
// heads the parts are equal and fixed.
template <int D, bool Q8>
__global__ void __launch_bounds__(kWarps * 32) cache_attn_mma_kernel(
    const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
    const DecodeSpec ds, const CacheKV c, const __nv_bfloat16 *__restrict__ q,
    const uint4 *__restrict__ ent, const int32_t *__restrict__ u_count, int *__restrict__ next,
    float *__restrict__ part, float *__restrict__ own_part, uint32_t *__restrict__ err) {
  using Lay = MmaLayout<D, Q8>;
  constexpr int MT = D / 16;  // 16-dim tiles of the output
  constexpr int DG = D / 8;   // dims of a lane group's V column
  constexpr int kRec = D + 2;
  extern __shared__ __align__(1024) unsigned char smem_mma[];
  unsigned char *smem = smem_mma;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (smem_u32(smem) & 1023u) {
    if (tid == 0) report(err, DEV_BAD_INDEX);
    grid_dep_wait();  // complete only after the kernels before it (the next ones rely on that)
    return;
  }
  const int g = lane >> 2, t = lane & 3;
  const int G = ds.Hq / ds.Hkv, BK = ds.B * ds.Hkv;
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Lay::bars) + warp * kSlots;
  int *seg_bk = reinterpret_cast<int *>(smem + Lay::seg), *seg_st = seg_bk + kMaxSeg;
  int *misc = reinterpret_cast<int *>(smem + Lay::misc);  // warp sums [kWarps], segment counts [kWarps]
  volatile int *abort_flag = misc + 2 * kWarps;
  unsigned char *ring = smem + Lay::ring + warp * kSlots * Lay::kItem;

  grid_dep_launch();
  if ((int)blockIdx.x < BK) {
    const int bk = blockIdx.x;
    if (tid == 0 && bk % ds.Hkv == 0 && (ds.lens[bk / ds.Hkv] < 0 || ds.lens[bk / ds.Hkv] > ds.N))
      report(err, DEV_BAD_INDEX);
    // no wait: it needs the step's inputs alone, and makes room for the others,
    // which do (the grid so ends after the kernels before it all the same)
    own_chunk<D, Q8>(ds, c, q, bk, smem, own_part + (size_t)bk * G * kRec, err);
    return;
  }
  if (tid == 0) {
    *abort_flag = 0;
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }
  if (lane == 0) {
    for (int i = 0; i < kSlots; ++i) mbar_init(&bars[i], 1);
    fence_mbar_init();
  }
  grid_dep_wait();  // the union
  // ---- the list: its length, and the KV heads of the part this CTA may see
  const int cnt0 = tid < BK ? max(0, u_count[tid] - 1) : 0;  // without the own chunk
  int total = cnt0;
  for (int i = tid + kWarps * 32; i < BK; i += kWarps * 32) total += max(0, u_count[i] - 1);
  total = __reduce_add_sync(0xffffffffu, total);
  if (lane == 0) misc[warp] = total;
  __syncthreads();
  total = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) total += misc[i];
  const int cta = (int)blockIdx.x - BK, wid = cta * kWarps + warp, W = ds.ctas * kWarps;
  const bool dynamic = BK <= kMaxSeg;
  auto first = [&](int w) { return (int)((long long)total * w / W); };
  const int see_lo = dynamic ? 0 : first(cta * kWarps), see_hi = dynamic ? total : first((cta + 1) * kWarps);
  if (see_lo >= see_hi) return;
  int n_seg = 0, run = 0;  // segments found, entries before the tile
  for (int i0 = 0; run < see_hi; i0 += kWarps * 32) {
    const int i = i0 + tid;
    const int cnt = i0 == 0 ? cnt0 : i < BK ? max(0, u_count[i] - 1) : 0;
    int x = cnt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    __syncthreads();  // misc is reused
    if (lane == 31) misc[warp] = x;
    __syncthreads();
    int st = run + x - cnt;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) st += misc[w];
      run += misc[w];
    }
    const bool in = cnt > 0 && st < see_hi && st + cnt > see_lo;
    const uint32_t bal = __ballot_sync(0xffffffffu, in);
    if (lane == 0) misc[kWarps + warp] = __popc(bal);
    __syncthreads();
    int at = n_seg + __popc(bal & ((1u << lane) - 1u));
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) at += misc[kWarps + w];
      n_seg += misc[kWarps + w];
    }
    if (in && at < kMaxSeg) {
      seg_bk[at] = i;
      seg_st[at] = st;
    }
  }
  n_seg = min(n_seg, kMaxSeg);
  __syncthreads();

  // claims of at most 32 entries, one per lane: the one in use and the next
  const int s0 = min(32, max(1, total / (2 * W)));  // the first, fixed
  int taken = dynamic ? wid * s0 : first(wid);      // where the last claim ended
  const int stop = dynamic ? total : first(wid + 1);
  bool started = false;
  auto claim = [&](int &at, int &n) {
    int size = 32;
    at = taken;
    if (dynamic && !started) {
      size = s0;
    } else if (dynamic) {
      size = min(32, max(1, (total - taken) / (4 * W)));
      if (lane == 0) at = W * s0 + atomicAdd(next, size);
      at = __shfl_sync(0xffffffffu, at, 0);
    }
    started = true;
    n = max(0, min(size, stop - at));
    taken = min(at + size, stop);
  };
  struct Batch {
    int n, bk, blk;
    uint32_t mask, slot_lo, slot_hi;
    float sk, sv;
  };
  auto load_batch = [&](Batch &r) {
    int at;
    claim(at, r.n);
    r.bk = 0;
    r.blk = kEntNoPage;
    r.mask = r.slot_lo = r.slot_hi = 0u;
    r.sk = r.sv = 0.0f;
    if (lane >= r.n) return;
    const int f = at + lane;
    int a = 0, z = n_seg;  // the last segment that starts at or before f
    while (z - a > 1) {
      const int mid = (a + z) >> 1;
      if (seg_st[mid] <= f) a = mid;
      else z = mid;
    }
    r.bk = seg_bk[a];
    const uint4 *e = ent + 2 * ((size_t)r.bk * ds.ucap + (f - seg_st[a]));
    const uint4 e0 = e[0], e1 = e[1];
    r.blk = (int)e0.x;
    r.mask = e0.y;
    r.sk = __uint_as_float(e0.z);
    r.sv = __uint_as_float(e0.w);
    r.slot_lo = e1.x;
    r.slot_hi = e1.y;
  };
  Batch cur, nxt;
  load_batch(cur);
  if (cur.n == 0) return;
  nxt = cur;
  nxt.n = 0;

  // copies: the items of the entries with a page, in order; at most kSlots are
  // ahead of the one in use.  e_next: the entry to request next, counted from
  // cur's first
  int issued = 0, done = 0, e_next = 0;
  auto pump = [&]() {
    while (issued < done + kSlots && e_next < cur.n + nxt.n) {
      const bool in_cur = e_next < cur.n;
      const int blk = __shfl_sync(0xffffffffu, in_cur ? cur.blk : nxt.blk, in_cur ? e_next : e_next - cur.n);
      if (blk >= 0) {
        if (lane == 0) {
          uint64_t *bar = &bars[issued % kSlots];
          mbar_expect_tx(bar, Lay::kItem);
          const int sub = issued % Lay::kItems;
          const bool is_v = sub >= Lay::kItems / 2;
          tma_load_3d(ring + (issued % kSlots) * Lay::kItem, is_v ? &tm_v : &tm_k, bar,
                      64 * (sub % (Lay::kItems / 2)), 0, blk);
        }
        ++issued;
        if (issued % Lay::kItems) continue;  // the rest of the entry comes next
      }
      ++e_next;
    }
  };
  pump();
  load_batch(nxt);
  pump();

  uint32_t qf[D / 16][2];  // the queries as B fragments: fp16, or as they are for bf16 pages
  float hf[2];             // logit factors of heads 2t, 2t+1
  int cur_bk = -1;
  // a new KV head: lane (g, t) holds head g's dims 16 (t + 4 i) .. + 15 as the B
  // fragments of four steps, scaled by the head's power of two (bf16 pages:
  // dims 8 (t + 4 i) .. + 7, two steps)
  auto start_head = [&](int bk) {
    cur_bk = bk;
    const int b = bk / ds.Hkv, hkv = bk % ds.Hkv;
    const __nv_bfloat16 *qrow = q + ((size_t)b * ds.Hq + hkv * G + (g < G ? g : 0)) * D;
    if constexpr (!Q8) {
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        uint4 w = make_uint4(0u, 0u, 0u, 0u);
        if (g < G) w = *reinterpret_cast<const uint4 *>(qrow + 8 * (t + 4 * i));
        qf[2 * i][0] = w.x;
        qf[2 * i][1] = w.y;
        qf[2 * i + 1][0] = w.z;
        qf[2 * i + 1][1] = w.w;
      }
      hf[0] = hf[1] = ds.scale;
      return;
    }
    float qv[D / 64][16];
    uint32_t mx = 0u;
#pragma unroll
    for (int i = 0; i < D / 64; ++i)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        uint4 w = make_uint4(0u, 0u, 0u, 0u);
        if (g < G) w = *reinterpret_cast<const uint4 *>(qrow + 16 * (t + 4 * i) + 8 * u);
        const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          qv[i][8 * u + 2 * e] = __uint_as_float(ww[e] << 16);
          qv[i][8 * u + 2 * e + 1] = __uint_as_float(ww[e] & 0xFFFF0000u);
          const uint32_t a = (ww[e] << 16) & 0x7FFFFFFFu, z = ww[e] & 0x7FFF0000u;
          mx = max(mx, max(a < 0x7F800000u ? a : 0u, z < 0x7F800000u ? z : 0u));
        }
      }
    mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    // 2^k brings the largest |q| = 1.m * 2^(e - 127) to [2^14, 2^15)
    const int k = mx == 0u ? 0 : min(126, max(-126, 14 - ((int)(mx >> 23) - 127)));
    const float up = pow2f(k), f = ds.scale * pow2f(-k);
#pragma unroll
    for (int i = 0; i < D / 64; ++i)
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        qf[4 * i + w][0] = pack_h2(qv[i][4 * w] * up, qv[i][4 * w + 1] * up);
        qf[4 * i + w][1] = pack_h2(qv[i][4 * w + 2] * up, qv[i][4 * w + 3] * up);
      }
    hf[0] = __shfl_sync(0xffffffffu, f, (2 * t) * 4);
    hf[1] = __shfl_sync(0xffffffffu, f, (2 * t + 1) * 4);
  };

  // keys of this lane in a 16-key step: A rows g, g + 8 of K; columns 2t, 2t+1 (+ 8) of V
  const int kr = kperm(g), va = kperm(2 * t), vb = kperm(2 * t + 1);

  bool ok = true;
  for (int src = 0;; ++src) {
    if (src == cur.n) {
      if (nxt.n == 0) break;
      e_next -= cur.n;
      src = 0;
      cur = nxt;
      load_batch(nxt);
      pump();
    }
    const int bk = __shfl_sync(0xffffffffu, cur.bk, src), blk = __shfl_sync(0xffffffffu, cur.blk, src);
    const uint32_t mask = __shfl_sync(0xffffffffu, cur.mask, src);
    const uint32_t slot_lo = __shfl_sync(0xffffffffu, cur.slot_lo, src), slot_hi = __shfl_sync(0xffffffffu, cur.slot_hi, src);
    const float sk = __shfl_sync(0xffffffffu, cur.sk, src), sv = __shfl_sync(0xffffffffu, cur.sv, src);
    if (bk != cur_bk) start_head(bk);
    // this lane's heads 2t, 2t+1: whether they attend the chunk, and their records
    bool att[2];
    float *rec[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int hd = 2 * t + h, slot = (int)(((t < 2 ? slot_lo : slot_hi) >> (8 * (hd & 3))) & 0xFFu);
      att[h] = ((mask >> hd) & 1u) != 0u;
      rec[h] = part + (((size_t)bk * G + hd) * ds.topk + slot) * D + (Q8 ? DG * g : 8 * g);
    }
    if (blk < 0) {  // a page outside the pool is not read
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (att[h])
#pragma unroll
          for (int mt = 0; mt < MT; mt += 2)
            *reinterpret_cast<float4 *>(rec[h] + (Q8 ? 2 * mt : 64 * (mt / 4) + 2 * (mt % 4))) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      pump();
      continue;
    }
    float s[4][4], o[MT][4], m[2], l[2];
#pragma unroll
    for (int mt = 0; mt < 4; ++mt)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[mt][i] = 0.0f;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[mt][i] = 0.0f;
    if constexpr (Q8) {
      // ---- logits
      int j = done;
      ok = __all_sync(0xffffffffu, mbar_wait(&bars[j % kSlots], (j / kSlots) & 1, abort_flag));
      if (!ok) break;
      const unsigned char *kb = ring + (j % kSlots) * Lay::kItem;
#pragma unroll
      for (int mt = 0; mt < 4; ++mt) {
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
          const int r = mt * 16 + kr;  // r and r + 8 share their swizzle
          const int off = D == 128 ? r * 128 + (((t + 4 * i) ^ (r & 7)) << 4)
                                   : r * 64 + ((t ^ ((r >> 1) & 3)) << 4);
          const uint4 x = *reinterpret_cast<const uint4 *>(kb + off);
          const uint4 y = *reinterpret_cast<const uint4 *>(kb + off + 8 * D);
          const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            uint32_t a0, a1, a2, a3;
            e4m3x4_to_f16x2(xw[w], a0, a2);
            e4m3x4_to_f16x2(yw[w], a1, a3);
            mma_f16(s[mt], a0, a1, a2, a3, qf[4 * i + w][0], qf[4 * i + w][1]);
          }
        }
      }
      __syncwarp();
      ++done;
      pump();
      const float f[2] = {hf[0] * sk, hf[1] * sk};
      softmax_keys<4, 15>(s, f, m, l);
      // ---- P V
      ++j;
      ok = __all_sync(0xffffffffu, mbar_wait(&bars[j % kSlots], (j / kSlots) & 1, abort_flag));
      if (!ok) break;
      const unsigned char *vbk = ring + (j % kSlots) * Lay::kItem;
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        uint32_t ph[2], pl[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint32_t top = pack_h2(s[ks][2 * u], s[ks][2 * u + 1]);
          const float2 r = __half22float2(*reinterpret_cast<const __half2 *>(&top));
          ph[u] = movm(top);
          pl[u] = movm(pack_h2(s[ks][2 * u] - r.x, s[ks][2 * u + 1] - r.y));
        }
        uint32_t w[4][DG / 4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int r = ks * 16 + ((u & 1) ? vb : va) + ((u & 2) ? 8 : 0);
          if constexpr (D == 128) {
            const uint4 x = *reinterpret_cast<const uint4 *>(vbk + r * 128 + ((g ^ (r & 7)) << 4));
            w[u][0] = x.x;
            w[u][1] = x.y;
            w[u][2] = x.z;
            w[u][3] = x.w;
          } else {
            const uint2 x = *reinterpret_cast<const uint2 *>(vbk + r * 64 + (((g >> 1) ^ ((r >> 1) & 3)) << 4) + (g & 1) * 8);
            w[u][0] = x.x;
            w[u][1] = x.y;
          }
        }
#pragma unroll
        for (int e = 0; e < DG / 4; ++e) {
          // four dims of two keys, byte by byte: (key a, key b) pairs of dims 4e .. 4e + 3
          const uint32_t x0 = __byte_perm(w[0][e], w[1][e], 0x5140), x1 = __byte_perm(w[0][e], w[1][e], 0x7362);
          const uint32_t y0 = __byte_perm(w[2][e], w[3][e], 0x5140), y1 = __byte_perm(w[2][e], w[3][e], 0x7362);
          uint32_t a0, a1, a2, a3;
          e4m3x4_to_f16x2(x0, a0, a1);
          e4m3x4_to_f16x2(y0, a2, a3);
          mma_f16(o[2 * e], a0, a1, a2, a3, ph[0], ph[1]);
          mma_f16(o[2 * e], a0, a1, a2, a3, pl[0], pl[1]);
          e4m3x4_to_f16x2(x1, a0, a1);
          e4m3x4_to_f16x2(y1, a2, a3);
          mma_f16(o[2 * e + 1], a0, a1, a2, a3, ph[0], ph[1]);
          mma_f16(o[2 * e + 1], a0, a1, a2, a3, pl[0], pl[1]);
        }
      }
      __syncwarp();
      ++done;
      pump();
    } else {
      // ---- the same on bf16 rows, 64 columns at a time; the probabilities are
      // split into two bf16 parts (16 bits)
#pragma unroll
      for (int half = 0; half < D / 64; ++half) {
        ok = __all_sync(0xffffffffu, mbar_wait(&bars[done % kSlots], (done / kSlots) & 1, abort_flag));
        if (!ok) break;
        const unsigned char *kb = ring + (done % kSlots) * Lay::kItem;
#pragma unroll
        for (int mt = 0; mt < 4; ++mt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int r = mt * 16 + kr, off = r * 128 + (((t + 4 * i) ^ (r & 7)) << 4), qi = 2 * (2 * half + i);
            const uint4 x = *reinterpret_cast<const uint4 *>(kb + off);
            const uint4 y = *reinterpret_cast<const uint4 *>(kb + off + 8 * 128);
            mma_bf16(s[mt], x.x, y.x, x.y, y.y, qf[qi][0], qf[qi][1]);
            mma_bf16(s[mt], x.z, y.z, x.w, y.w, qf[qi + 1][0], qf[qi + 1][1]);
          }
        __syncwarp();
        ++done;
        pump();
      }
      if (!ok) break;
      softmax_keys<4, 0>(s, hf, m, l);
      uint32_t ph[4][2], pl[4][2];
#pragma unroll
      for (int ks = 0; ks < 4; ++ks)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const float a = s[ks][2 * u], z = s[ks][2 * u + 1];
          const uint32_t top = pack_b2(a, z);
          ph[ks][u] = movm(top);
          pl[ks][u] = movm(pack_b2(a - __uint_as_float(top << 16), z - __uint_as_float(top & 0xFFFF0000u)));
        }
#pragma unroll
      for (int half = 0; half < D / 64; ++half) {
        ok = __all_sync(0xffffffffu, mbar_wait(&bars[done % kSlots], (done / kSlots) & 1, abort_flag));
        if (!ok) break;
        const unsigned char *vbk = ring + (done % kSlots) * Lay::kItem;
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          uint32_t w[4][4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int r = ks * 16 + ((u & 1) ? vb : va) + ((u & 2) ? 8 : 0);
            const uint4 x = *reinterpret_cast<const uint4 *>(vbk + r * 128 + ((g ^ (r & 7)) << 4));
            w[u][0] = x.x;
            w[u][1] = x.y;
            w[u][2] = x.z;
            w[u][3] = x.w;
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t a0 = __byte_perm(w[0][e], w[1][e], 0x5410), a1 = __byte_perm(w[0][e], w[1][e], 0x7632);
            const uint32_t a2 = __byte_perm(w[2][e], w[3][e], 0x5410), a3 = __byte_perm(w[2][e], w[3][e], 0x7632);
            mma_bf16(o[4 * half + e], a0, a1, a2, a3, ph[ks][0], ph[ks][1]);
            mma_bf16(o[4 * half + e], a0, a1, a2, a3, pl[ks][0], pl[ks][1]);
          }
        }
        __syncwarp();
        ++done;
        pump();
      }
      if (!ok) break;
    }
    // the records of the heads that attend it: the chunk's output
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (!att[h]) continue;
      // the scale apart: its product with 1 / l (down to 2^-21) would be subnormal
      // for the least scales and lose its bits
      const float inv = 1.0f / l[h], f = Q8 ? sv : 1.0f;
#pragma unroll
      for (int mt = 0; mt < MT; mt += 2)
        *reinterpret_cast<float4 *>(rec[h] + (Q8 ? 2 * mt : 64 * (mt / 4) + 2 * (mt % 4))) =
            make_float4(o[mt][h] * inv * f, o[mt][2 + h] * inv * f, o[mt + 1][h] * inv * f, o[mt + 1][2 + h] * inv * f);
    }
  }
  if (!ok && lane == 0) {
    // a wait gave up: every copy in flight must land before the CTA exits
    for (int j = max(0, issued - kSlots); j < issued; ++j)
      mbar_wait_bounded(&bars[j % kSlots], (j / kSlots) & 1);
    report(err, DEV_TIMEOUT);
  }
}

// The chunks of a head fused (one CTA per head): out = sum w_c o_c, w the
// softmax over the selected landmark logits and the own chunk's.  A logit of
// -inf weighs 0; a head that has no other gets out 0, lse -inf.  A warp sums
// every eighth record, a lane D / 32 columns, all its loads at once.
constexpr int kCombWarps = 8;
template <int D>
__global__ void __launch_bounds__(kCombWarps * 32) cache_combine_kernel(
    const DecodeSpec ds, const float *__restrict__ chunk_w, const int32_t *__restrict__ u_count,
    const float *__restrict__ part, const float *__restrict__ own_part,
    __nv_bfloat16 *__restrict__ out, float *__restrict__ lse) {
  constexpr int kRec = D + 2, V = D / 32, kMaxK = 64, kU = kMaxK / kCombWarps;
  __shared__ float wo[kCombWarps][D];
  const int G = ds.Hq / ds.Hkv, K = ds.topk;
  const int h = blockIdx.x, b = h / ds.Hq, hq = h % ds.Hq;
  const int bk = b * ds.Hkv + hq / G, hd = hq % G;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  grid_dep_wait();  // the chunk attention's records (and the selection before it)
  __nv_bfloat16 *orow = out + (size_t)h * D;
  if (u_count[bk] == 0) {  // an empty sequence: out 0, lse -inf
    if (tid < D) orow[tid] = __float2bfloat16_rn(0.0f);
    if (tid == 0) lse[h] = -INFINITY;
    return;
  }
  const float *own = own_part + ((size_t)bk * G + hd) * kRec;
  // the logits, every warp all of them (two per lane), and their softmax
  const float w0 = lane < K ? chunk_w[(size_t)h * K + lane] : -INFINITY;
  const float w1 = lane + 32 < K ? chunk_w[(size_t)h * K + lane + 32] : -INFINITY;
  const float wown = own[0];
  const float *r0 = part + (size_t)h * K * D + lane * V;
  float x[kU][V];
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const int k = warp + u * kCombWarps;
    const float w = __shfl_sync(0xffffffffu, k < 32 ? w0 : w1, k & 31);
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      const float2 y = w != -INFINITY ? *reinterpret_cast<const float2 *>(r0 + (size_t)k * D + i) : make_float2(0.0f, 0.0f);
      x[u][i] = y.x;
      x[u][i + 1] = y.y;
    }
  }
  float m = fmaxf(wown, fmaxf(w0, w1));
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float e0 = w0 == -INFINITY ? 0.0f : __expf(w0 - m), e1 = w1 == -INFINITY ? 0.0f : __expf(w1 - m);
  float l = e0 + e1;
#pragma unroll
  for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  const float eown = wown == -INFINITY ? 0.0f : __expf(wown - m);
  l += eown;  // at least 1, or 0 where every logit is -inf
  float acc[V];
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.0f;
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const int k = warp + u * kCombWarps;
    const float e = __shfl_sync(0xffffffffu, k < 32 ? e0 : e1, k & 31);
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] += e * x[u][i];
  }
#pragma unroll
  for (int i = 0; i < V; ++i) wo[warp][lane * V + i] = acc[i];
  __syncthreads();
  if (tid < D) {
    float y = eown * own[2 + tid];
#pragma unroll
    for (int w = 0; w < kCombWarps; ++w) y += wo[w][tid];
    orow[tid] = __float2bfloat16_rn(l == 0.0f ? 0.0f : y / l);
  }
  if (tid == 0) lse[h] = m + __logf(l);
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                  const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                  const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// A pool of blocks [blocks][64][d]: one block of codes per copy, its 16-byte
// pieces swizzled within 128 (d = 128) or 64 (d = 64) bytes; or 64 columns of a
// bf16 block, swizzled within 128 bytes.
cudaError_t make_tmap_blocks(CUtensorMap *map, const void *base, uint64_t blocks, int d, bool q8) {
  static EncodeTiledFn encode = nullptr;
  if (!encode) {
    void *fn = nullptr;
    cudaDriverEntryPointQueryResult r;
    cudaError_t e = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &r);
    if (e != cudaSuccess || r != cudaDriverEntryPointSuccess || !fn) return cudaErrorNotSupported;
    encode = reinterpret_cast<EncodeTiledFn>(fn);
  }
  const cuuint64_t dims[3] = {(cuuint64_t)d, kC, blocks};
  const cuuint64_t row = (cuuint64_t)d * (q8 ? 1 : 2);
  const cuuint64_t strides[2] = {row, row * kC};
  const cuuint32_t box[3] = {(cuuint32_t)(q8 ? d : 64), kC, 1}, estr[3] = {1, 1, 1};
  const CUresult r = encode(map, q8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                            const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                            q8 && d == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace

cudaError_t cache_attn(const DecodeSpec &ds, const CacheKV &c, const void *q, const uint4 *ent,
                       const int32_t *u_count, int *next, const float *chunk_w, float *part,
                       float *own_part, void *out, float *lse, uint32_t *err, cudaStream_t st) {
  cudaError_t e;
  CUtensorMap tk, tv;
  const uint64_t blocks = (uint64_t)c.num_pages * ds.Hkv;
  if ((e = make_tmap_blocks(&tk, c.k_pages, blocks, ds.d, c.q8)) != cudaSuccess) return e;
  if ((e = make_tmap_blocks(&tv, c.v_pages, blocks, ds.d, c.q8)) != cudaSuccess) return e;
#define HILS_MMA(DD, QQ)                                                                           \
  do {                                                                                           \
    auto kern = cache_attn_mma_kernel<DD, QQ>;                                                       \
    const size_t smem = MmaLayout<DD, QQ>::total;                                                    \
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) != cudaSuccess) return e; \
    if ((e = launch_dep(true, kern, dim3((unsigned)(ds.B * ds.Hkv + ds.ctas)), dim3(kWarps * 32), smem, \
                        st, tk, tv, ds, c, (const __nv_bfloat16 *)q, ent, u_count, next, part, \
                        own_part, err)) != cudaSuccess)                                          \
      return e;                                                                                  \
    return launch_dep(true, cache_combine_kernel<DD>, dim3((unsigned)(ds.B * ds.Hq)), dim3(kCombWarps * 32), 0, st, \
                      ds, chunk_w, u_count, (const float *)part, (const float *)own_part,        \
                      (__nv_bfloat16 *)out, lse);                                                \
  } while (0)
  if (ds.d == 64) { if (c.q8) HILS_MMA(64, true); else HILS_MMA(64, false); }
  if (c.q8) HILS_MMA(128, true);
  HILS_MMA(128, false);
#undef HILS_MMA
}

cudaError_t cache_attn_f32(const DecodeSpec &ds, const CacheKV &c, const void *q,
                           const int32_t *u_c, const uint32_t *u_mask, const float *u_logit,
                           const int32_t *u_count, float *part, uint32_t *err, cudaStream_t st) {
  const dim3 grid((unsigned)ds.Q, (unsigned)(ds.B * ds.Hkv));
  cudaError_t e;
#define HILS_SIMT(DD)                                                                            \
  do {                                                                                           \
    auto kern = cache_attn_simt_kernel<DD>;                                                      \
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,             \
                                  (int)sizeof(SimtSmem<DD>))) != cudaSuccess) return e;          \
    return launch_dep(true, kern, grid, dim3(kThreads), sizeof(SimtSmem<DD>), st, ds, c,         \
                      (const float *)q, u_c, u_mask, u_logit, u_count, part, err);               \
  } while (0)
  if (ds.d == 64) HILS_SIMT(64);
  HILS_SIMT(128);
#undef HILS_SIMT
}

}  // namespace hils
