// New keys and values entering the paged KV cache, with HoPE on the way
// (molayo1419.me, "Engineering details", HoPE: keys are rotated once, as they
// enter the cache; "Converting existing models": serving runs HiLS as an
// attention backend, whose cache this fills).  Per token and KV head:
//
//   key   y = R(p) x  (hope.cuh, the same arithmetic as hils_hope), rounded
//         to the parameter dtype;  value  unchanged
//
// written to a page of the dtype, or, in the 8-bit form, to the tail of its
// chunk; when the chunk's 64 tokens are complete they become one block of
// e4m3 codes with the scale s = 2^k, the smallest k >= -126 with
// max|x| <= 448 * 2^k over the block's finite values, code = rn(x / s).  A
// power of two moves no mantissa bit, so a value is rounded once, and the
// block is a function of its 64 keys alone: however the tokens arrived, one
// by one or as a prompt, the cache holds the same bits.  The landmark row of
// a completed chunk is the fp32 mean of its 64 keys as rounded to the dtype,
// its sum taken in a fixed order.
//
// Bound by bytes.  A CTA of 128 threads owns one (chunk, KV head, K or V) and
// reads its 64 rows (16 KB at bf16, d = 128) with every 16-byte load in
// flight; a thread holds the matching pieces of a row's two halves, so the
// pairs (i, i + d/2) of the rotation meet in its registers, and the codes,
// the block maximum and the column sums come from the same registers: the
// keys cross HBM once each way.  The queries' rotation rides in the same
// launch (rows 2 Hkv .. of the grid), so a decode step needs one launch here.
//
// Measured: a 128K prompt of 8 KV heads (d = 128, bf16 into e4m3) 145 us for
// 805 MB, 5.6 TB/s, 86 % of a plain copy; without the rotation the same launch
// runs at the copy's rate, so the sines and cosines (one pair of each per pair
// of elements and head) are what is left.  Sharing them between heads through
// shared memory cost more loads in flight than it saved (156 to 194 us).
#include <cuda_bf16.h>

#include <algorithm>

#include "cache.h"
#include "common.cuh"
#include "e4m3.cuh"
#include "hope.cuh"

namespace hils {
namespace {

constexpr int kC = 64;        // tokens per chunk
constexpr int kThreads = 128;

// A 16-byte piece of a row is four 32-bit words of N elements each.
template <typename T>
struct Word;
template <>
struct Word<__nv_bfloat16> {
  static constexpr int N = 2;
  static __device__ __forceinline__ void widen(uint32_t w, float (&f)[N]) {
    f[0] = __uint_as_float(w << 16);
    f[1] = __uint_as_float(w & 0xFFFF0000u);
  }
  static __device__ __forceinline__ uint32_t narrow(const float (&f)[N]) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f[0], f[1]);
    return *reinterpret_cast<const uint32_t *>(&h);
  }
  // the bits of the word's first n elements
  static __device__ __forceinline__ uint32_t mask(int n) {
    return n >= 2 ? 0xFFFFFFFFu : n == 1 ? 0xFFFFu : 0u;
  }
  // s += x * c per element, c a power of two (products exact in fp32); the
  // mixed-precision FMA widens on the way
  static __device__ __forceinline__ void fma(uint32_t x, uint16_t c, float *s) {
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "mov.b32 {lo, hi}, %2;\n\t"
        "fma.rn.f32.bf16 %0, lo, %3, %0;\n\t"
        "fma.rn.f32.bf16 %1, hi, %3, %1;\n\t}"
        : "+f"(s[0]), "+f"(s[1])
        : "r"(x), "h"(c));
  }
  // 2^k as the factor of fma, -126 <= k <= 127
  static __device__ __forceinline__ uint16_t pow2(int k) { return (uint16_t)((k + 127) << 7); }
};
template <>
struct Word<float> {
  static constexpr int N = 1;
  static __device__ __forceinline__ void widen(uint32_t w, float (&f)[N]) { f[0] = __uint_as_float(w); }
  static __device__ __forceinline__ uint32_t narrow(const float (&f)[N]) { return __float_as_uint(f[0]); }
  static __device__ __forceinline__ uint32_t mask(int n) { return n >= 1 ? 0xFFFFFFFFu : 0u; }
  static __device__ __forceinline__ void fma(uint32_t x, float c, float *s) {
    s[0] = fmaf(__uint_as_float(x), c, s[0]);
  }
  static __device__ __forceinline__ float pow2(int k) { return pow2f(k); }
};

// How 128 threads cover rows of D elements: LPR lanes per row, lane `col`
// holding elements [col E, col E + E) of both halves; RP rows per pass.
template <typename T, int D>
struct Lay {
  static constexpr int E = 16 / (int)sizeof(T);
  static constexpr int LPR = D / 2 / E;
  static constexpr int RP = kThreads / LPR;
  static constexpr int NP = kC / RP;  // passes of 64 rows
  static_assert(kThreads % LPR == 0 && kC % RP == 0 && 32 % LPR == 0, "row cover");
};

// A thread's share of 64 rows: pass i holds row i RP + rg.
template <typename T, int D>
struct Rows {
  uint32_t lo[Lay<T, D>::NP][4], hi[Lay<T, D>::NP][4];
  __device__ __forceinline__ void load(int i, const T *row, int col) {
    constexpr int E = Lay<T, D>::E;
    const uint4 a = *reinterpret_cast<const uint4 *>(row + col * E);
    const uint4 z = *reinterpret_cast<const uint4 *>(row + D / 2 + col * E);
    lo[i][0] = a.x; lo[i][1] = a.y; lo[i][2] = a.z; lo[i][3] = a.w;
    hi[i][0] = z.x; hi[i][1] = z.y; hi[i][2] = z.z; hi[i][3] = z.w;
  }
  __device__ __forceinline__ void clear(int i) {
#pragma unroll
    for (int w = 0; w < 4; ++w) lo[i][w] = hi[i][w] = 0u;
  }
  __device__ __forceinline__ void store(int i, T *row, int col) const {
    constexpr int E = Lay<T, D>::E;
    *reinterpret_cast<uint4 *>(row + col * E) = make_uint4(lo[i][0], lo[i][1], lo[i][2], lo[i][3]);
    *reinterpret_cast<uint4 *>(row + D / 2 + col * E) = make_uint4(hi[i][0], hi[i][1], hi[i][2], hi[i][3]);
  }
  // Rotates the rows r0 <= row < r1, row r at position p0 + r.  Pair by pair
  // over the passes: a pair's turn advances by RP positions per pass, one
  // 64-bit sum whose bits 32..63 are the fractional turn that hope_sincos
  // takes from the product (equal modulo 2^64, so the same bits).
  template <bool kFull>
  __device__ __forceinline__ void rotate(const HopeParams &hp, int p0, int r0, int r1, int col, int rg) {
    using L = Lay<T, D>;
    constexpr int N = Word<T>::N;
    uint32_t row_on[L::NP];
#pragma unroll
    for (int i = 0; i < L::NP; ++i) {
      const int r = i * L::RP + rg;
      row_on[i] = r >= r0 && r < r1 ? 0xFFFFFFFFu : 0u;
    }
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const int i0 = col * L::E + w * N;
      const uint32_t on = Word<T>::mask(hp.npairs - i0);  // the other pairs pass through
      unsigned long long th[N], turn[N];
#pragma unroll
      for (int u = 0; u < N; ++u) {
        th[u] = hp.turns[i0 + u];
        turn[u] = th[u] * (unsigned long long)(uint32_t)(p0 + rg);
      }
#pragma unroll
      for (int i = 0; i < L::NP; ++i) {
        if (kFull || (i * L::RP < r1 && (i + 1) * L::RP > r0)) {  // the same for the whole CTA
          float a[N], z[N], ya[N], yz[N];
          Word<T>::widen(lo[i][w], a);
          Word<T>::widen(hi[i][w], z);
#pragma unroll
          for (int u = 0; u < N; ++u) {
            float sn, cs;
            __sincosf((float)(int32_t)(uint32_t)(turn[u] >> 32) * kHopeTurnUnit, &sn, &cs);
            hope_rotate(a[u], z[u], sn, cs, ya[u], yz[u]);
          }
          const uint32_t m = kFull ? on : on & row_on[i];
          lo[i][w] = (Word<T>::narrow(ya) & m) | (lo[i][w] & ~m);
          hi[i][w] = (Word<T>::narrow(yz) & m) | (hi[i][w] & ~m);
        }
#pragma unroll
        for (int u = 0; u < N; ++u) turn[u] += th[u] * L::RP;
      }
    }
  }
};

// A thread's share of one row, rotated as Rows does.
template <typename T, int D>
struct OneRow {
  uint32_t lo[4] = {0u, 0u, 0u, 0u}, hi[4] = {0u, 0u, 0u, 0u};
  __device__ __forceinline__ void load(const T *row, int col) {
    constexpr int E = Lay<T, D>::E;
    const uint4 a = *reinterpret_cast<const uint4 *>(row + col * E);
    const uint4 z = *reinterpret_cast<const uint4 *>(row + D / 2 + col * E);
    lo[0] = a.x; lo[1] = a.y; lo[2] = a.z; lo[3] = a.w;
    hi[0] = z.x; hi[1] = z.y; hi[2] = z.z; hi[3] = z.w;
  }
  __device__ __forceinline__ void store(T *row, int col) const {
    constexpr int E = Lay<T, D>::E;
    *reinterpret_cast<uint4 *>(row + col * E) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    *reinterpret_cast<uint4 *>(row + D / 2 + col * E) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
  }
  __device__ __forceinline__ void rotate(const HopeParams &hp, int pos, int col) {
    constexpr int N = Word<T>::N;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const int i0 = col * Lay<T, D>::E + w * N;
      const uint32_t on = Word<T>::mask(hp.npairs - i0);  // the other pairs pass through
      float a[N], z[N], ya[N], yz[N];
      Word<T>::widen(lo[w], a);
      Word<T>::widen(hi[w], z);
#pragma unroll
      for (int u = 0; u < N; ++u) {
        float sn, cs;
        hope_sincos(hp.turns[i0 + u], pos, sn, cs);
        hope_rotate(a[u], z[u], sn, cs, ya[u], yz[u]);
      }
      lo[w] = (Word<T>::narrow(ya) & on) | (lo[w] & ~on);
      hi[w] = (Word<T>::narrow(yz) & on) | (hi[w] & ~on);
    }
  }
};

// Largest magnitude of the words added, as fp32 bits (infinity and NaN rank
// above every finite value).
template <typename T>
struct Amax;
template <>
struct Amax<__nv_bfloat16> {
  uint32_t m = 0u;  // two 15-bit magnitudes
  __device__ __forceinline__ void add(uint32_t w) { m = __vmaxu2(m, w & 0x7FFF7FFFu); }
  __device__ __forceinline__ uint32_t bits() const { return max(m & 0xFFFF0000u, m << 16); }
};
template <>
struct Amax<float> {
  uint32_t m = 0u;
  __device__ __forceinline__ void add(uint32_t w) { m = max(m, w & 0x7FFFFFFFu); }
  __device__ __forceinline__ uint32_t bits() const { return m; }
};

// the codes of the 4 / N words from w on, times inv = Word<T>::pow2(-k)
template <typename T, typename F>
__device__ __forceinline__ uint32_t codes4(const uint32_t *w, F inv) {
  float f[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < 4 / Word<T>::N; ++i) Word<T>::fma(w[i], inv, f + i * Word<T>::N);
  return e4m3x2(f[0], f[1]) | (e4m3x2(f[2], f[3]) << 16);
}

// Tokens [pos, end) of sequence b, or an empty range when its arguments are
// out of bounds: a negative or too large position or count, or an end past
// the longest sequence.
__device__ __forceinline__ bool token_range(const AppendSpec &as, int b, int &pos, int &n) {
  pos = as.pos[b];
  n = as.n_new ? as.n_new[b] : as.T;
  const bool ok = pos >= 0 && pos <= as.L && n >= 0 && n <= as.T && n <= as.L - pos;
  if (!ok) n = 0;
  return ok;
}

// Rows of one chunk of one (b, hkv), K or V.  r0 .. r1: its new rows; rows
// below r0 are older tokens.  kStore: the new rows are stored too (otherwise
// only what follows from a complete chunk).  kFull: all 64 rows are new.
template <typename T, int D, bool Q8, bool kStore, bool kFull>
__device__ __forceinline__ void append_chunk(const AppendSpec &as, const CacheKV &c,
                                             const HopeParams &hp, const T *__restrict__ src,
                                             long long src_st, bool is_k, int b, int hkv, int chunk,
                                             int pos, int end, uint32_t *err) {
  using L = Lay<T, D>;
  constexpr int E = L::E, N = Word<T>::N;
  __shared__ uint32_t red_max[kThreads / 32];
  __shared__ float red_sum[kThreads / 32][D];
  const int tid = threadIdx.x, col = tid % L::LPR, rg = tid / L::LPR;
  const int lane = tid & 31, warp = tid >> 5;
  const int t0 = chunk * kC;
  const int r0 = kFull ? 0 : max(0, pos - t0), r1 = kFull ? kC : min(kC, end - t0);
  const bool complete = kFull || r1 == kC;
  T *tail = nullptr;  // [64][D] of this chunk's half
  if (Q8)
    tail = static_cast<T *>(is_k ? c.k_tail : c.v_tail) +
           ((((size_t)b * 2 + (chunk & 1)) * as.Hkv + hkv) * kC) * D;
  // the page: read and written by a paged chunk, written by a complete 8-bit one
  long long page = -1;
  if (!Q8 || complete) {
    page = c.table[(size_t)b * c.max_pages + chunk];
    if (page < 0 || page >= c.num_pages) {
      if (tid == 0) report(err, DEV_BAD_INDEX);
      page = -1;
    }
  }
  const size_t blk = page < 0 ? 0 : (size_t)page * as.Hkv + hkv;
  const bool want_lmk = is_k && complete && c.lmk != nullptr;
  // older rows, needed when the chunk is complete: from the tail, or for the
  // landmark from the page
  const T *old = Q8 ? tail : (page < 0 ? nullptr : static_cast<const T *>(is_k ? c.k_pages : c.v_pages) + blk * kC * D);
  const bool need_old = !kFull && complete && r0 > 0 && (Q8 || want_lmk) && old != nullptr;

  Rows<T, D> x;
  if constexpr (kFull) {
    const T *row = src + (t0 + rg - pos) * src_st;
#pragma unroll
    for (int i = 0; i < L::NP; ++i, row += L::RP * src_st) x.load(i, row, col);
  } else {
#pragma unroll
    for (int i = 0; i < L::NP; ++i) {
      const int r = i * L::RP + rg;
      const T *row = nullptr;
      if (r >= r0 && r < r1) row = src + (long long)(t0 + r - pos) * src_st;
      else if (r < r0 && need_old) row = old + (size_t)r * D;
      if (row) x.load(i, row, col);
      else x.clear(i);
    }
  }
  if (is_k && hp.npairs > 0) x.template rotate<kFull>(hp, t0, r0, r1, col, rg);
  // the new rows in full precision: the tails of the last two chunks, or the page
  T *dst = nullptr;
  if (!kStore) {
  } else if (Q8) {
    if (chunk >= (end - 1) / kC - 1) dst = tail;
  } else if (page >= 0) {
    dst = static_cast<T *>(is_k ? c.k_pages : c.v_pages) + blk * kC * D;
  }
  if (dst) {
#pragma unroll
    for (int i = 0; i < L::NP; ++i) {
      const int r = i * L::RP + rg;
      if (kFull || (r >= r0 && r < r1)) x.store(i, dst + (size_t)r * D, col);
    }
  }
  if (!complete) return;
  if (Q8 && page >= 0) {
    // the block's largest magnitude (bits of non-negative floats order as integers)
    Amax<T> am;
#pragma unroll
    for (int i = 0; i < L::NP; ++i)
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        am.add(x.lo[i][w]);
        am.add(x.hi[i][w]);
      }
    uint32_t m = am.bits();
    m = __reduce_max_sync(0xffffffffu, m);
    if (lane == 0) red_max[warp] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) m = max(m, red_max[w]);
    if (m >= 0x7F800000u) {
      // infinities or NaN in the block: once more over the finite values alone
      m = 0u;
#pragma unroll
      for (int i = 0; i < L::NP; ++i)
#pragma unroll
        for (int w = 0; w < 8; ++w) {
          float f[N];
          Word<T>::widen(w < 4 ? x.lo[i][w & 3] : x.hi[i][w & 3], f);
#pragma unroll
          for (int u = 0; u < N; ++u) {
            const uint32_t v = __float_as_uint(f[u]) & 0x7FFFFFFFu;
            m = max(m, v < 0x7F800000u ? v : 0u);
          }
        }
      m = __reduce_max_sync(0xffffffffu, m);
      __syncthreads();  // red_max has been read
      if (lane == 0) red_max[warp] = m;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kThreads / 32; ++w) m = max(m, red_max[w]);
    }
    const int k = block_scale_exp(m);
    if (tid == 0) (is_k ? c.k_scale : c.v_scale)[blk] = pow2f(k);
    uint8_t *codes = static_cast<uint8_t *>(is_k ? c.k_pages : c.v_pages) + blk * kC * D;
    const auto inv = Word<T>::pow2(-k);
#pragma unroll
    for (int i = 0; i < L::NP; ++i) {
      uint8_t *row = codes + (size_t)(i * L::RP + rg) * D + col * E;
      if constexpr (E == 8) {
        *reinterpret_cast<uint2 *>(row) = make_uint2(codes4<T>(x.lo[i], inv), codes4<T>(x.lo[i] + 2, inv));
        *reinterpret_cast<uint2 *>(row + D / 2) = make_uint2(codes4<T>(x.hi[i], inv), codes4<T>(x.hi[i] + 2, inv));
      } else {
        *reinterpret_cast<uint32_t *>(row) = codes4<T>(x.lo[i], inv);
        *reinterpret_cast<uint32_t *>(row + D / 2) = codes4<T>(x.hi[i], inv);
      }
    }
  }
  if (want_lmk && (Q8 || page >= 0)) {
    if (chunk >= c.lmk_rows) {
      if (tid == 0) report(err, DEV_BAD_INDEX);
    } else {
      // column sums: a thread's rows in order, then the row groups of a warp,
      // then the warps, always in the same order
      const auto one = Word<T>::pow2(0);
      float sl[E], sh[E];
#pragma unroll
      for (int u = 0; u < E; ++u) sl[u] = sh[u] = 0.0f;
#pragma unroll
      for (int i = 0; i < L::NP; ++i)
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          Word<T>::fma(x.lo[i][w], one, sl + w * N);
          Word<T>::fma(x.hi[i][w], one, sh + w * N);
        }
#pragma unroll
      for (int o = 16; o >= L::LPR; o >>= 1) {
#pragma unroll
        for (int u = 0; u < E; ++u) {
          sl[u] += __shfl_xor_sync(0xffffffffu, sl[u], o);
          sh[u] += __shfl_xor_sync(0xffffffffu, sh[u], o);
        }
      }
      if (lane < L::LPR) {
#pragma unroll
        for (int u = 0; u < E; ++u) {
          red_sum[warp][col * E + u] = sl[u];
          red_sum[warp][D / 2 + col * E + u] = sh[u];
        }
      }
      __syncthreads();
      T *row = static_cast<T *>(c.lmk) + (((size_t)b * as.Hkv + hkv) * c.lmk_rows + chunk) * D;
      for (int e = tid; e < D; e += kThreads) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) s += red_sum[w][e];
        row[e] = from_f<T>(s * (1.0f / kC));
      }
    }
  }
}

// grid (chunks a sequence may touch, 2 Hkv + Hq, B): y < Hkv the keys of a
// head, y < 2 Hkv its values, the rest the queries' heads (64 new tokens per x).
template <typename T, int D, bool Q8>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 4 ? 3 : Q8 ? 8 : 7) kv_append_kernel(const AppendSpec as, const CacheKV c,
                                                             const RowsIn k, const RowsIn v,
                                                             const RowsIn q, T *__restrict__ q_out,
                                                             const HopeParams hp, uint32_t *err) {
  using L = Lay<T, D>;
  const int b = blockIdx.z, y = blockIdx.y, x = blockIdx.x;
  int pos, n;
  const bool ok = token_range(as, b, pos, n);
  if (x == 0 && y == 0 && threadIdx.x == 0) {
    if (!ok) report(err, DEV_BAD_INDEX);
    if (as.seq_lens) as.seq_lens[b] = ok ? pos + n : min(max(pos, 0), as.L);
  }
  if (y >= 2 * as.Hkv) {
    // queries: rotated into q_out; rows past the sequence's new tokens become zero
    const int hq = y - 2 * as.Hkv, col = threadIdx.x % L::LPR, rg = threadIdx.x / L::LPR;
    const T *src = static_cast<const T *>(q.p) + b * q.sb + hq * q.sh;
    T *dst = q_out + ((size_t)b * as.Hq + hq) * as.T * D;
    const int t0 = x * kC;
    Rows<T, D> r;
#pragma unroll
    for (int i = 0; i < L::NP; ++i) {
      const int t = t0 + i * L::RP + rg;
      if (t < n) r.load(i, src + t * q.st, col);
      else r.clear(i);
    }
    if (hp.npairs > 0) r.template rotate<false>(hp, pos + t0, 0, min(kC, n - t0), col, rg);
#pragma unroll
    for (int i = 0; i < L::NP; ++i) {
      const int t = t0 + i * L::RP + rg;
      if (t < as.T) r.store(i, dst + (size_t)t * D, col);
    }
    return;
  }
  if (n == 0) return;
  const bool is_k = y < as.Hkv;
  const int hkv = is_k ? y : y - as.Hkv;
  const RowsIn &in = is_k ? k : v;
  const T *src = static_cast<const T *>(in.p) + b * in.sb + hkv * in.sh;
  const int end = pos + n, c0 = pos / kC, cl = (end - 1) / kC;
  const int chunk = c0 + x;
  if (chunk > cl) return;
  // The first chunk's older rows lie in tail half c0 & 1.  A later chunk that
  // writes the same half (one of the last two, of c0's parity) is done by the
  // first chunk's CTA after it has read them.
  const int same = ((cl ^ c0) & 1) ? cl - 1 : cl;  // of the last two, the one of c0's parity
  const bool shared_half = Q8 && same > c0 && pos % kC != 0;
  if (shared_half && chunk == same) return;
  if (chunk * kC >= pos && (chunk + 1) * kC <= end) {
    append_chunk<T, D, Q8, true, true>(as, c, hp, src, in.st, is_k, b, hkv, chunk, pos, end, err);
    return;
  }
  append_chunk<T, D, Q8, true, false>(as, c, hp, src, in.st, is_k, b, hkv, chunk, pos, end, err);
  if (shared_half && chunk == c0) {
    __syncthreads();  // every thread has read the older rows
    append_chunk<T, D, Q8, true, false>(as, c, hp, src, in.st, is_k, b, hkv, same, pos, end, err);
  }
}

// Few new tokens (T <= kFew, so at most one chunk becomes complete): a CTA per
// 16 (bf16, d = 128) new rows of any kind, and behind them one per (b, KV head,
// K or V) that does a completed chunk's work, or has none.  The general grid
// spends a CTA of 64 rows on each head: 10.3 us for 64 sequences of 8 / 32
// heads against 3.6 us here (replayed from a graph).
constexpr int kFew = 64;
template <typename T, int D, bool Q8>
__global__ void __launch_bounds__(kThreads) kv_append_few_kernel(const AppendSpec as, const CacheKV c,
                                                                 const RowsIn k, const RowsIn v,
                                                                 const RowsIn q, T *__restrict__ q_out,
                                                                 const HopeParams hp, int row_ctas,
                                                                 uint32_t *err) {
  using L = Lay<T, D>;
  const int b = blockIdx.y;
  int pos, n;
  const bool ok = token_range(as, b, pos, n);
  const int end = pos + n;
  if ((int)blockIdx.x >= row_ctas) {
    const int y = (int)blockIdx.x - row_ctas, hkv = y % as.Hkv, chunk = pos / kC;
    const bool is_k = y < as.Hkv;
    if (n == 0 || (chunk + 1) * kC > end) return;
    if (!Q8 && (!is_k || !c.lmk)) return;  // full rows are all a page holds
    const RowsIn &in = is_k ? k : v;
    const T *src = static_cast<const T *>(in.p) + b * in.sb + hkv * in.sh;
    append_chunk<T, D, Q8, false, false>(as, c, hp, src, in.st, is_k, b, hkv, chunk, pos, end, err);
    return;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    if (!ok) report(err, DEV_BAD_INDEX);
    if (as.seq_lens) as.seq_lens[b] = ok ? end : min(max(pos, 0), as.L);
  }
  // row = head * T + token, heads in the order K, V, Q
  const int col = threadIdx.x % L::LPR, row = blockIdx.x * L::RP + threadIdx.x / L::LPR;
  const int y = row / as.T, i = row % as.T;
  const int kind = y < as.Hkv ? 0 : y < 2 * as.Hkv ? 1 : 2;  // K, V, Q
  if (y >= 2 * as.Hkv + (q.p ? as.Hq : 0) || (i >= n && kind != 2)) return;
  const int h = kind == 0 ? y : kind == 1 ? y - as.Hkv : y - 2 * as.Hkv;
  const T *src = kind == 0 ? static_cast<const T *>(k.p) + b * k.sb + h * k.sh + i * k.st
               : kind == 1 ? static_cast<const T *>(v.p) + b * v.sb + h * v.sh + i * v.st
                           : static_cast<const T *>(q.p) + b * q.sb + h * q.sh + i * q.st;
  const int p = pos + i, chunk = p / kC, r = p % kC;
  T *dst;
  if (kind == 2) {
    dst = q_out + (((size_t)b * as.Hq + h) * as.T + i) * D;
  } else if (Q8) {
    dst = static_cast<T *>(kind == 0 ? c.k_tail : c.v_tail) +
          ((((size_t)b * 2 + (chunk & 1)) * as.Hkv + h) * kC + r) * D;
  } else {
    const long long page = c.table[(size_t)b * c.max_pages + chunk];
    if (page < 0 || page >= c.num_pages) {
      report(err, DEV_BAD_INDEX);
      return;
    }
    dst = static_cast<T *>(kind == 0 ? c.k_pages : c.v_pages) + (((size_t)page * as.Hkv + h) * kC + r) * D;
  }
  OneRow<T, D> x;
  if (i < n) x.load(src, col);
  if (i < n && kind != 1 && hp.npairs > 0) x.rotate(hp, p, col);
  x.store(dst, col);
}

}  // namespace

cudaError_t kv_append(const AppendSpec &as, bool bf16, const CacheKV &c, const RowsIn &k,
                      const RowsIn &v, const RowsIn &q, void *q_out, const HopeParams &hp,
                      uint32_t *err, cudaStream_t st, int *launches) {
  if (as.T <= kFew) {
    const int rows = (2 * as.Hkv + (q.p ? as.Hq : 0)) * as.T;
#define HILS_FEW(T, DD)                                                                        \
  do {                                                                                         \
    const int row_ctas = (rows + Lay<T, DD>::RP - 1) / Lay<T, DD>::RP;                         \
    const dim3 grid((unsigned)(row_ctas + 2 * as.Hkv), (unsigned)as.B);                        \
    if (c.q8)                                                                                  \
      kv_append_few_kernel<T, DD, true><<<grid, kThreads, 0, st>>>(as, c, k, v, q, (T *)q_out, hp, row_ctas, err);  \
    else                                                                                       \
      kv_append_few_kernel<T, DD, false><<<grid, kThreads, 0, st>>>(as, c, k, v, q, (T *)q_out, hp, row_ctas, err); \
  } while (0)
    if (bf16) { if (as.d == 64) HILS_FEW(__nv_bfloat16, 64); else HILS_FEW(__nv_bfloat16, 128); }
    else { if (as.d == 64) HILS_FEW(float, 64); else HILS_FEW(float, 128); }
#undef HILS_FEW
    ++*launches;
    return cudaGetLastError();
  }
  // T tokens from any position touch at most this many chunks
  const unsigned nx = (unsigned)((as.T - 1) / kC + 2);
  const dim3 grid(nx, (unsigned)(2 * as.Hkv + (q.p ? as.Hq : 0)), (unsigned)as.B);
#define HILS_APPEND(T, DD)                                                                     \
  do {                                                                                         \
    if (c.q8)                                                                                  \
      kv_append_kernel<T, DD, true><<<grid, kThreads, 0, st>>>(as, c, k, v, q, (T *)q_out, hp, err);  \
    else                                                                                       \
      kv_append_kernel<T, DD, false><<<grid, kThreads, 0, st>>>(as, c, k, v, q, (T *)q_out, hp, err); \
  } while (0)
  if (bf16) { if (as.d == 64) HILS_APPEND(__nv_bfloat16, 64); else HILS_APPEND(__nv_bfloat16, 128); }
  else { if (as.d == 64) HILS_APPEND(float, 64); else HILS_APPEND(float, 128); }
#undef HILS_APPEND
  ++*launches;
  return cudaGetLastError();
}

}  // namespace hils
