// k_paged.cuh -- attention over raw rows held in 8 bits in a paged cache.
//
// Cache: pages of `page` rows in a pool, codes [n_pages, hkv, page, D] for
// keys and for values, one fp32 scale per block of `chunk` rows and kv head
// ([n_pages, hkv, page / chunk]); row r of sequence b lies in page
// table[b][r / page].  A row's value is scale * code.
//
// The product kernel of both readers (k_paged_attend: all rows of a
// sequence; k_paged_unfold: selected chunks and the own chunk of one query
// head) is one warp working through tiles of 32 rows:
//   z = K q        S^T[16 keys x 8 queries], mma.sync m16n8k32 on the codes as
//                  they are, the KEYS as the A operand: a kv head's 4..8 query
//                  heads fill the 8 columns, where queries as A would leave
//                  8..12 of 16 rows idle;
//   p = 2^(z - m)  lazy online softmax in fp32 (m raised when exceeded by
//                  kPgSlack), the scale of K applied to z, that of V to p;
//   O^T += V^T p   m16n8k32 with V^T as A (4 x 4 byte transposes of the codes
//                  in registers) and p as B (movmatrix turns the accumulator
//                  layout of S^T into it).
// The 8-bit operands of the other side are written as sums of 8-bit digits,
// one product each, so the codes need no conversion:
//   e4m3 (4 significant bits a digit): a bf16 query is 2 digits, the second
//     in an accumulator of its own at 2^4 times the scale; an fp32 one 3 + 3 at
//     2^12.  A row is scaled by a power of two so that its largest element
//     lies in [128, 256): digits end at 2^-10, 2^-22 (2^-30) of it.
//   int8 (7 bits a digit, fixed point): 3 digits for bf16 queries (2^-20 of the
//     row's largest element), 4 for fp32 (2^-28); sums are exact integers.
//   p times the scale of V is scaled by the largest of the tile's 32 in its
//     column: e4m3 3 digits (2^-12 of the weight, 2^-18 of the largest) or 6
//     (2^-22, 2^-30), int8 2 digits (2^-15 of the largest) or 3 (2^-22): the
//     fewer for bf16 outputs, whose own rounding is 2^-8.
// Statistics, sums of weights and the running output are fp32.
//
// What bounds it: HBM reads of the codes.  Every warp copies its tiles with
// 16-byte cp.async into its own ring, so there is no CTA-wide barrier in
// the loop; page-table entries are fetched one tile ahead of the copies,
// scales one tile behind them.
#pragma once

#include <type_traits>

#include "common.cuh"
#include "k_unfold.cuh"  // UnfoldArgs, ready list

namespace gsa {

// n / d for 0 <= n < 2^31 by a multiply and a shift (d >= 1 fixed at launch):
// with l = ceil(log2 d) and m = floor(2^32 (2^l - d) / d) + 1,
// n / d = (mulhi(m, n) + n) >> l  (Granlund and Montgomery, 1994).
struct FastDiv {
  uint32_t mul, shift, d;
  __host__ void init(uint32_t div) {
    d = div;
    shift = 0;
    while ((1ull << shift) < div) ++shift;
    mul = static_cast<uint32_t>((((1ull << shift) - div) << 32) / div + 1);
  }
  __device__ __forceinline__ uint32_t div(uint32_t n) const { return (__umulhi(mul, n) + n) >> shift; }
};

enum { kFmtI8 = 0, kFmtE4M3 = 1 };

struct PagedKV {
  const uint8_t *k, *v;       // [n_pages, hkv, page, D]
  const float *ks, *vs;       // [n_pages, hkv, page / chunk]
  const int32_t *table;       // [B, max_pages]
  int32_t n_pages, max_pages, hkv, blocks;  // blocks = page / chunk
  FastDiv page, chunk;
};

constexpr float kPgSlack = 16.0f;  // p <= 2^16 before the reference is raised (p is fp32)

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// c += A B on 8-bit codes (16 x 32 times 32 x 8).
__device__ __forceinline__ void mma_16832(float c[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint2 b) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b.x), "r"(b.y));
}
__device__ __forceinline__ void mma_16832(int c[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint2 b) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b.x), "r"(b.y));
}

// 8x8 block of 16-bit elements transposed across the warp's accumulator layout.
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// The larger, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// (a.x * b.x + c.x, a.y * b.y + c.y)
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(r)
      : "l"(*reinterpret_cast<const uint64_t *>(&a)), "l"(*reinterpret_cast<const uint64_t *>(&b)),
        "l"(*reinterpret_cast<const uint64_t *>(&c)));
  return *reinterpret_cast<const float2 *>(&r);
}

__device__ __forceinline__ float2 unpack_h2(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}

// e4m3 pair (16 bits) of an fp16 pair, and back.
__device__ __forceinline__ uint16_t h2_to_e4(__half2 x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(*reinterpret_cast<const uint32_t *>(&x)));
  return r;
}
__device__ __forceinline__ __half2 e4_to_h2(uint16_t x) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(x));
  return *reinterpret_cast<const __half2 *>(&r);
}

// N e4m3 digits of an fp16 pair: out[i] is the rounding of what out[0..i-1] left.  Returns the remainder (exact).
template <int N>
__device__ __forceinline__ __half2 e4_digits(__half2 x, uint16_t *out) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    out[i] = h2_to_e4(x);
    x = __hsub2(x, e4_to_h2(out[i]));
  }
  return x;
}

// Four codes -> two fp16 pairs (bytes 0,1 and bytes 2,3), exact.
template <int FMT>
__device__ __forceinline__ void codes_to_h2(uint32_t w, uint32_t &lo, uint32_t &hi) {
  if (FMT == kFmtI8) {
    // 0x6400 | u is the fp16 1024 + u for a byte u; u = code + 128
    const uint32_t u = w ^ 0x80808080u;
    const __half2 off = __half2half2(__ushort_as_half(0x6480));  // 1152
    uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 x = __hsub2(*reinterpret_cast<__half2 *>(&a), off);
    const __half2 y = __hsub2(*reinterpret_cast<__half2 *>(&b), off);
    lo = *reinterpret_cast<const uint32_t *>(&x);
    hi = *reinterpret_cast<const uint32_t *>(&y);
  } else {
    const __half2 x = e4_to_h2(static_cast<uint16_t>(w)), y = e4_to_h2(static_cast<uint16_t>(w >> 16));
    lo = *reinterpret_cast<const uint32_t *>(&x);
    hi = *reinterpret_cast<const uint32_t *>(&y);
  }
}

// One warp's ring: per stage K as [slot][lane] 16-byte pieces (each lane
// reads back what it copied), V as 32 rows with swizzled 16-byte pieces, the
// 64 scales of the tile (K then V) and the mask of live keys.
template <int D>
struct PgCfg {
  static constexpr int kStages = D == 64 ? 3 : 2;
  static constexpr int kCtas = D == 64 ? 4 : 3;  // of 4 warps on an SM
  static constexpr uint32_t kK = 32 * D, kScales = 64 * D, kMask = kScales + 256;
  static constexpr uint32_t kStage = kMask + 16;
  static constexpr uint32_t kRing = kStages * kStage;
};

// Offset of 16-byte piece p of row r inside a stage's V: lanes (g, t) read
// rows 2t (+1, +8, +9, ..) at dims g*D/8.., and the permutations below spread
// the 8 lanes of a shared-memory phase over all 32 banks.
template <int D>
__device__ __forceinline__ uint32_t v_off(uint32_t r, uint32_t p) {
  if (D == 128) return r * 128 + ((p ^ (((r >> 1) & 3) << 1)) << 4);
  return (r ^ ((r >> 2) & 1)) * 64 + ((p ^ (((r >> 1) & 1) << 1)) << 4);
}

// Digits of the queries: how many, and how they group into two accumulators
// (the value is acc[0] + acc[1] * kRest for e4m3, acc[0] * kTop + acc[1] for
// int8, whose first digits come first).
template <int FMT, bool QF32>
struct QDigits {
  static constexpr int kFirst = FMT == kFmtI8 ? 2 : (QF32 ? 3 : 1);  // digits of acc[0]
  static constexpr int kN = FMT == kFmtI8 ? (QF32 ? 4 : 3) : 2 * kFirst;
  static constexpr float kUp = QF32 ? 4096.f : 16.f;   // e4m3: scale of the second group
  static constexpr int kBits = 7 * kN - 1;             // int8: |fixed point| < 2^kBits
  static constexpr float kTop = kN == 4 ? 16384.f : 128.f;
};

// The queries of a segment in shared memory, as the B fragments of their
// digits: [NT][digit][k-step of 32 dims][lane], and the factor of each row's
// logits.  Row n (< 8 NT) is row(n), null when unused.
template <int D, int FMT, bool QF32, int NT>
struct PgQuery {
  using Dg = QDigits<FMT, QF32>;
  static constexpr int KS = D / 32;
  uint2 frag[NT][Dg::kN][KS][32];
  float f[8 * NT];

  // Group nt, by one warp.
  template <typename RowFn>
  __device__ __forceinline__ void load(int nt, RowFn row, float scale_log2) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const void *p = row(8 * nt + g);
    float x[D / 4];  // dims 64 c + 16 t + 0..15
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
#pragma unroll
      for (int v = 0; v < (QF32 ? 4 : 2); ++v) {
        const int e = (c * 64 + t * 16) + v * (QF32 ? 4 : 8);
        uint4 w = make_uint4(0, 0, 0, 0);
        if (p) w = __ldcg(reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(p) + e * (QF32 ? 4 : 2)));
        if (QF32)
          Vec16<float>::unpack(w, x + c * 16 + v * 4);
        else
          Vec16<__nv_bfloat16>::unpack(w, x + c * 16 + v * 8);
      }
    }
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < D / 4; ++i) a = max(a, __float_as_uint(x[i]) & 0x7fffffffu);
    a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
    a = max(a, __shfl_xor_sync(0xffffffffu, a, 2));
    // power of two that brings the row's maximum into [2^(top-1), 2^top); none for a row of zeros.  An inf or NaN
    // makes the row's logits NaN.
    constexpr int kTopExp = FMT == kFmtI8 ? Dg::kBits : 8;
    int sh = 0;
    if (a != 0 && a < 0x7f800000u) sh = min(kTopExp - 1 - (static_cast<int>(a >> 23) - 127), 120);
    const float up = __uint_as_float(static_cast<uint32_t>(127 + sh) << 23);
    const float down = __uint_as_float(static_cast<uint32_t>(127 - sh) << 23) * scale_log2;
    if (t == 0) f[8 * nt + g] = a < 0x7f800000u ? down : __uint_as_float(0x7fc00000u);
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      // words of b0 (dims 8 s' + 0..3) and b1 (+ 4..7) of this k-step
      uint32_t w[Dg::kN][2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float *y = x + 8 * s + 4 * h;
        if (FMT == kFmtI8) {
          uint32_t d[Dg::kN][4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            int v = __float2int_rn(y[i] * up);
#pragma unroll
            for (int k = Dg::kN - 1; k >= 0; --k) {  // last digit first; each in [-64, 63], the first takes the rest
              const int top = k == 0 ? v : ((v + 64) & 127) - 64;
              d[k][i] = static_cast<uint32_t>(top) & 0xffu;
              v = (v - top) >> 7;
            }
          }
#pragma unroll
          for (int k = 0; k < Dg::kN; ++k) w[k][h] = d[k][0] | d[k][1] << 8 | d[k][2] << 16 | d[k][3] << 24;
        } else {
          uint16_t d[2][Dg::kN];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float u = y[2 * i] * up, v = y[2 * i + 1] * up;
            const __half2 r = __floats2half2_rn(u, v);  // exact for bf16 down to fp16's subnormals
            const float2 rf = __half22float2(r);
            const float2 left = __half22float2(e4_digits<Dg::kFirst>(r, d[i]));
            e4_digits<Dg::kN - Dg::kFirst>(
                __floats2half2_rn(((u - rf.x) + left.x) * Dg::kUp, ((v - rf.y) + left.y) * Dg::kUp),
                d[i] + Dg::kFirst);
          }
#pragma unroll
          for (int k = 0; k < Dg::kN; ++k) w[k][h] = d[0][k] | static_cast<uint32_t>(d[1][k]) << 16;
        }
      }
#pragma unroll
      for (int k = 0; k < Dg::kN; ++k) frag[nt][k][s][lane] = make_uint2(w[k][0], w[k][1]);
    }
  }
};

// The state of one warp over a run of tiles; NT groups of 8 query columns.
template <int D, int FMT, bool QF32, bool HILO, int NT>
struct PgWarp {
  using Cfg = PgCfg<D>;
  using Query = PgQuery<D, FMT, QF32, NT>;
  using Dg = QDigits<FMT, QF32>;
  using Acc = typename std::conditional<FMT == kFmtI8, int, float>::type;
  static constexpr int S = Cfg::kStages;
  static constexpr int MT = D / 16;  // m-tiles of O^T
  // digits of a weight; int8: the first two share an accumulator
  static constexpr int PN = FMT == kFmtI8 ? (HILO ? 3 : 2) : (HILO ? 6 : 3);
  static constexpr float kPTop = FMT == kFmtI8 ? (HILO ? 2080768.f : 16256.f) : 448.f;  // 127 * 2^7 or 2^14

  float m[NT][2], l[NT][2];  // columns 2t, 2t + 1
  float2 o[NT][MT][2];       // O^T: dims g*D/8 + 2j and + 2j + 1, (column 2t, column 2t + 1)
  // the copy pipeline
  int32_t pid;     // page of this lane's key in the next tile to copy (-1: none)
  uint32_t off;    // its row in that page
  float sck, scv;  // scales of this lane's key in the tile copied last
  uint32_t ring;

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = neg_inf();
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int j = 0; j < MT; ++j) o[nt][j][0] = o[nt][j][1] = make_float2(0.f, 0.f);
    }
  }

  // Fetch the page of raw row r (< 0: no such key).
  __device__ __forceinline__ void fetch(const PagedKV &kv, const int32_t *table, int r) {
    pid = -1;
    off = 0;
    if (r >= 0) {
      const uint32_t p = kv.page.div(static_cast<uint32_t>(r));
      off = static_cast<uint32_t>(r) - p * kv.page.d;
      pid = __ldcg(table + p);
    }
  }

  // Copy the fetched tile into stage st.  A key whose page is not in the
  // pool is left out and flagged.
  __device__ __forceinline__ void copy(const PagedKV &kv, int kvh, int st, bool wanted, uint32_t *status) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const bool live = static_cast<uint32_t>(pid) < static_cast<uint32_t>(kv.n_pages);
    if (wanted && !live) flag_error(status, GSA_DEVERR_BAD_INDEX);
    const uint32_t ph = live ? static_cast<uint32_t>(pid) * kv.hkv + kvh : 0u;
    const uint32_t prow = live ? ph * kv.page.d + off : 0xffffffffu;
    sck = scv = 0.f;
    if (live) {
      const size_t i = static_cast<size_t>(ph) * kv.blocks + kv.chunk.div(off);
      sck = __ldcg(kv.ks + i);
      scv = __ldcg(kv.vs + i);
    }
    const uint32_t base = ring + st * Cfg::kStage;
    const uint32_t mask = __ballot_sync(0xffffffffu, live);
    if (lane == 0) asm volatile("st.shared.u32 [%0], %1;" ::"r"(base + Cfg::kMask), "r"(mask) : "memory");
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // keys g + 8 i
      const uint32_t r = __shfl_sync(0xffffffffu, prow, g + 8 * i);
      const uint32_t bytes = r != 0xffffffffu ? 16u : 0u;
      const size_t o8 = bytes ? static_cast<size_t>(r) * D + t * 16 : 0;
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        cp_async16(base + ((i * (D / 64) + c) * 32 + lane) * 16, kv.k + o8 + 64 * c, bytes);
        cp_async16(base + Cfg::kK + v_off<D>(g + 8 * i, t + 4 * c), kv.v + o8 + 64 * c, bytes);
      }
    }
  }

  __device__ __forceinline__ void put_scale(int st) {
    const uint32_t at = ring + st * Cfg::kStage + Cfg::kScales + (threadIdx.x & 31) * 4;
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(at), "f"(sck) : "memory");
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(at + 128), "f"(scv) : "memory");
  }

  __device__ __forceinline__ static void lds4(uint32_t at, uint32_t *w) {
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(at));
  }
  __device__ __forceinline__ static float ldsf(uint32_t at) {
    float x;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(at));
    return x;
  }

  // Work through the tile in stage st; key0: index of its first key, lim:
  // columns 2t, 2t + 1 see keys below lim (CAUSAL).
  template <bool CAUSAL>
  __device__ __forceinline__ void step(const Query &qs, int st, int key0, const int (*lim)[2]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint32_t base = ring + st * Cfg::kStage, scb = base + Cfg::kScales + 4 * g;
    uint32_t mask;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(mask) : "r"(base + Cfg::kMask));
    // ---- z: value e of half h: key 16 h + g + 8 (e >> 1), column 2 t + (e & 1)
    float z[2][NT][4];
    {
      Acc acc[2][NT][2][4];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[h][nt][k][e] = 0;
      uint32_t kw[D / 64][4][4];  // [piece][row g + 8 i][word]
#pragma unroll
      for (int c = 0; c < D / 64; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) lds4(base + ((i * (D / 64) + c) * 32 + lane) * 16, kw[c][i]);
#pragma unroll
      for (int k = 0; k < Dg::kN; ++k) {
        const int group = k < Dg::kFirst ? 0 : 1;
        if (FMT == kFmtI8 && k == (group ? Dg::kFirst + 1 : 1)) {  // second digit of its accumulator
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[h][nt][group][e] *= 128;
        }
#pragma unroll
        for (int s = 0; s < D / 32; ++s)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const uint2 b = qs.frag[nt][k][s][lane];
#pragma unroll
            for (int h = 0; h < 2; ++h)
              mma_16832(acc[h][nt][group], kw[s / 2][2 * h][2 * (s & 1)], kw[s / 2][2 * h + 1][2 * (s & 1)],
                        kw[s / 2][2 * h][2 * (s & 1) + 1], kw[s / 2][2 * h + 1][2 * (s & 1) + 1], b);
          }
      }
      bool over = false;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float kg[2] = {ldsf(scb + 64 * h), ldsf(scb + 64 * h + 32)};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float2 f = *reinterpret_cast<const float2 *>(&qs.f[8 * nt + 2 * t]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float v = FMT == kFmtI8 ? fmaf(static_cast<float>(acc[h][nt][0][e]), Dg::kTop,
                                                 static_cast<float>(acc[h][nt][1][e]))
                                          : fmaf(static_cast<float>(acc[h][nt][1][e]), 1.f / Dg::kUp,
                                                 static_cast<float>(acc[h][nt][0][e]));
            const int key = 16 * h + g + 8 * (e >> 1);
            bool see = (mask >> key) & 1u;
            if (CAUSAL) see = see && key0 + key < lim[nt][e & 1];
            z[h][nt][e] = see ? v * (kg[e >> 1] * (e & 1 ? f.y : f.x)) : neg_inf();
            over = over || z[h][nt][e] > m[nt][e & 1] + kPgSlack;
          }
        }
      }
      if (__any_sync(0xffffffffu, over)) {  // raise the references, rescale
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float c[2];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            float mx = fmaxf(fmaxf(z[0][nt][x], z[0][nt][x + 2]), fmaxf(z[1][nt][x], z[1][nt][x + 2]));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            c[x] = mx > m[nt][x] ? exp2_approx(m[nt][x] - mx) : 1.f;  // 0 when there was no reference
            l[nt][x] *= c[x];
            m[nt][x] = fmaxf(m[nt][x], mx);
          }
#pragma unroll
          for (int j = 0; j < MT; ++j)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              o[nt][j][y].x *= c[0];
              o[nt][j][y].y *= c[1];
            }
        }
      }
    }
    // ---- weights: p, times the scale of V, relative to the column's largest of the tile; their digits as B fragments
    uint2 pb[PN][NT];
    float2 back[NT];
    float vg[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) vg[i] = ldsf(scb + 128 + 32 * i);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float w[2][4], top[2];
      const float m0 = m[nt][0] == neg_inf() ? 0.f : m[nt][0], m1 = m[nt][1] == neg_inf() ? 0.f : m[nt][1];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float p = exp2_approx(z[h][nt][e] - (e & 1 ? m1 : m0));
          l[nt][e & 1] += p;
          w[h][e] = z[h][nt][e] == neg_inf() ? 0.f : p * vg[2 * h + (e >> 1)];  // (a scale of NaN stays with its keys)
        }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float a = max_nan(max_nan(w[0][x], w[0][x + 2]), max_nan(w[1][x], w[1][x + 2]));
        a = max_nan(a, __shfl_xor_sync(0xffffffffu, a, 4));
        a = max_nan(a, __shfl_xor_sync(0xffffffffu, a, 8));
        top[x] = max_nan(a, __shfl_xor_sync(0xffffffffu, a, 16));
      }
      // (weights whose reciprocal fp32 does not hold, below kPTop 2^-126, are zero)
      const float i0 = top[0] > kPTop * 1.18e-38f ? __fdividef(kPTop, top[0]) : 0.f;
      const float i1 = top[1] > kPTop * 1.18e-38f ? __fdividef(kPTop, top[1]) : 0.f;
      back[nt] = make_float2(top[0] * (1.f / kPTop), top[1] * (1.f / kPTop));
      // 16-bit element (key g, column): digits of keys g and g + 8 of the half
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t dig[PN];
        if (FMT == kFmtI8) {
          int v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = __float2int_rn(w[h][e] * (e & 1 ? i1 : i0));
#pragma unroll
          for (int k = PN - 1; k >= 0; --k) {
            // bytes: column 2t (keys g, g + 8), column 2t + 1 (keys g, g + 8); the last digit in [-64, 63]
            int r[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              r[e] = k == 0 ? v[e] : v[e] + 64;
              v[e] = r[e] >> 7;
              if (k > 0) r[e] = (r[e] & 127) - 64;
            }
            dig[k] = __byte_perm(__byte_perm(r[0], r[2], 0x0040), __byte_perm(r[1], r[3], 0x0040), 0x5410);
          }
        } else {
          uint16_t d0[PN], d1[PN];
          const float a0 = w[h][0] * i0, a2 = w[h][2] * i0, b0 = w[h][1] * i1, b2 = w[h][3] * i1;
          const __half2 ha = __floats2half2_rn(a0, a2), hb = __floats2half2_rn(b0, b2);
          const __half2 ra = e4_digits<3>(ha, d0), rb = e4_digits<3>(hb, d1);
          if (HILO) {
            const float2 fa = __half22float2(ha), fb = __half22float2(hb);
            const float2 la = __half22float2(ra), lb = __half22float2(rb);
            e4_digits<3>(__floats2half2_rn(((a0 - fa.x) + la.x) * 4096.f, ((a2 - fa.y) + la.y) * 4096.f),
                         d0 + (HILO ? 3 : 0));
            e4_digits<3>(__floats2half2_rn(((b0 - fb.x) + lb.x) * 4096.f, ((b2 - fb.y) + lb.y) * 4096.f),
                         d1 + (HILO ? 3 : 0));
          }
#pragma unroll
          for (int k = 0; k < PN; ++k) dig[k] = d0[k] | static_cast<uint32_t>(d1[k]) << 16;
        }
#pragma unroll
        for (int k = 0; k < PN; ++k) (h ? pb[k][nt].y : pb[k][nt].x) = movmatrix_trans(dig[k]);
      }
    }
    // ---- O^T += V^T p: dims in words of 4 codes, rows 2t, 2t+8, 2t+1, 2t+9 of each half
    constexpr int kW = D / 32;
    uint32_t vr[2][4][kW];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t r = 16 * h + 2 * t + (i >> 1) + 8 * (i & 1);
        if constexpr (D == 128) {
          lds4(base + Cfg::kK + v_off<D>(r, g), vr[h][i]);
        } else {
          asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];"
                       : "=r"(vr[h][i][0]), "=r"(vr[h][i][1])
                       : "r"(base + Cfg::kK + v_off<D>(r, g >> 1) + (g & 1) * 8));
        }
      }
#pragma unroll
    for (int w = 0; w < kW; ++w) {
      uint32_t a[2][4];  // [half][dim]: four keys' codes
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t x = __byte_perm(vr[h][0][w], vr[h][1][w], 0x5140);
        const uint32_t y = __byte_perm(vr[h][0][w], vr[h][1][w], 0x7362);
        const uint32_t u = __byte_perm(vr[h][2][w], vr[h][3][w], 0x5140);
        const uint32_t v = __byte_perm(vr[h][2][w], vr[h][3][w], 0x7362);
        a[h][0] = __byte_perm(x, u, 0x5410);
        a[h][1] = __byte_perm(x, u, 0x7632);
        a[h][2] = __byte_perm(y, v, 0x5410);
        a[h][3] = __byte_perm(y, v, 0x7632);
      }
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          constexpr int kAcc = HILO ? 2 : 1;
          Acc d[kAcc][4];
#pragma unroll
          for (int k = 0; k < kAcc; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) d[k][e] = 0;
#pragma unroll
          for (int k = 0; k < PN; ++k) {
            const int group = FMT == kFmtI8 ? k / 2 : k / 3;
            if (FMT == kFmtI8 && k == 1) {
#pragma unroll
              for (int e = 0; e < 4; ++e) d[0][e] *= 128;
            }
            mma_16832(d[group], a[0][2 * j], a[0][2 * j + 1], a[1][2 * j], a[1][2 * j + 1], pb[k][nt]);
          }
          float v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            v[e] = static_cast<float>(d[0][e]);
            if (HILO)
              v[e] = FMT == kFmtI8 ? fmaf(v[e], 128.f, static_cast<float>(d[kAcc - 1][e]))
                                   : fmaf(static_cast<float>(d[kAcc - 1][e]), 1.f / 4096.f, v[e]);
          }
          o[nt][2 * w + j][0] = fma2(back[nt], make_float2(v[0], v[1]), o[nt][2 * w + j][0]);
          o[nt][2 * w + j][1] = fma2(back[nt], make_float2(v[2], v[3]), o[nt][2 * w + j][1]);
        }
    }
  }

  // Run n tiles; raw(i) is this lane's key of tile i as a raw row (< 0:
  // none), key0(i) the index of the tile's first key; before() runs once
  // while the first copies are in flight (and makes qs ready).
  template <bool CAUSAL, typename RawFn, typename Key0Fn, typename BeforeFn>
  __device__ __forceinline__ void run(const PagedKV &kv, const int32_t *table, int kvh, int n, const Query &qs,
                                      RawFn raw, Key0Fn key0, const int (*lim)[2], uint32_t *status, BeforeFn before) {
    clear();
    int r = n > 0 ? raw(0) : -1;
    fetch(kv, table, r);
#pragma unroll
    for (int i = 0; i < S - 1; ++i) {
      if (i > 0 && i - 1 < n) put_scale(i - 1);
      if (i < n) {
        copy(kv, kvh, i, r >= 0, status);
        r = i + 1 < n ? raw(i + 1) : -1;
        fetch(kv, table, r);
      }
      cp_async_commit();
    }
    before();
    int st = 0, stc = S - 1;  // stage worked on, stage copied into
    for (int i = 0; i < n; ++i) {
      const int j = i + S - 1;  // tile copied in this turn
      if (j - 1 < n) put_scale(stc == 0 ? S - 1 : stc - 1);
      cp_async_wait<S - 2>();
      __syncwarp();
      if (j < n) {
        copy(kv, kvh, stc, r >= 0, status);
        r = j + 1 < n ? raw(j + 1) : -1;
        fetch(kv, table, r);
      }
      cp_async_commit();
      step<CAUSAL>(qs, st, key0(i), lim);
      st = st == S - 1 ? 0 : st + 1;
      stc = stc == S - 1 ? 0 : stc + 1;
    }
    cp_async_wait<0>();
    __syncwarp();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        l[nt][x] += __shfl_xor_sync(0xffffffffu, l[nt][x], 4);
        l[nt][x] += __shfl_xor_sync(0xffffffffu, l[nt][x], 8);
        l[nt][x] += __shfl_xor_sync(0xffffffffu, l[nt][x], 16);
      }
  }
};

// ------------------------------------------------------------ dense attention
// The rows of all (sequence, kv head, group of 8 NT query rows) segments, in
// steps of 32 rows a warp, form one line that the CTAs cut into equal parts
// (the lengths are on the device, so the cut is too): ragged batches and
// single long sequences load every SM alike.  A segment inside one CTA is
// written directly; one that several CTAs share is joined by the last of them
// to arrive (an atomic counter, no waiting) from partial records, in CTA
// order, so the result does not depend on who was last.  CTAs of 4 warps, 3
// or 4 on an SM: one joins its warps while the others stream.
constexpr int kPgWarps = 4;
constexpr int kPgThreads = 32 * kPgWarps;
constexpr int kPgStep = 32 * kPgWarps;  // rows of one CTA step
constexpr int kPgMaxCtas = 640;         // bound of the grid (partial slots in the workspace)
constexpr int kPgMaxBatch = 8192;       // prefix sums in shared memory
constexpr int kPgMaxRows = 16;          // query rows of a segment

struct PagedAttendArgs {
  PagedKV kv;
  const void *q;               // [B, n_q, hq, D]
  const int32_t *n_gists;      // or null
  const int32_t *own_len;
  int32_t B, n_q, hq, group, rg, chunk, n_max, t_max, min_steps;
  float scale_log2;
  float *part;                 // [ctas][2][8 NT][D + 4]
  uint32_t *counters;          // [B * hkv * rg]
  uint32_t *status;
  void *out;                   // [B, n_q, hq, D]
  int32_t out_bf16;
  float *lse;                  // [B, n_q, hq] or null
};

// Raw rows of sequence b: (n_gists ? N * chunk : 0) + own_len, clamped to t_max.
__device__ __forceinline__ int paged_len(const int32_t *n_gists, const int32_t *own_len, int b, int n_max, int chunk,
                                         int t_max) {
  int64_t n = max(__ldcg(own_len + b), 0);
  if (n_gists) n += static_cast<int64_t>(min(max(__ldcg(n_gists + b), 0), n_max)) * chunk;
  return static_cast<int>(n < t_max ? n : t_max);
}

// Exclusive prefix sums of count(b), b < B, in pre[0 .. B] (shared), by the
// whole CTA of NTHREADS threads.
template <int NTHREADS, typename CountFn>
__device__ void paged_prefix(uint32_t *pre, int B, CountFn count) {
  __shared__ uint32_t warp_sum[NTHREADS / 32];
  __shared__ uint32_t carry;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    carry = 0;
    pre[0] = 0;
  }
  __syncthreads();
  for (int b0 = 0; b0 < B; b0 += NTHREADS) {
    uint32_t x = b0 + tid < B ? count(b0 + tid) : 0u;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
    uint32_t add = carry;
    for (int w = 0; w < warp; ++w) add += warp_sum[w];
    if (b0 + tid < B) pre[b0 + tid + 1] = x + add;
    __syncthreads();
    if (tid == NTHREADS - 1) carry = x + add;
    __syncthreads();
  }
}

// The b with pre[b] <= p < pre[b + 1].
__device__ __forceinline__ int paged_find(const uint32_t *pre, int B, uint32_t p) {
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (pre[mid] <= p) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Dynamic shared memory: rings (over them, once drained, the warps' results
// and the weights of a join) | queries | prefix sums [B + 1] and lengths [B].
template <int D, int FMT, bool QF32, int NT>
__host__ __device__ constexpr uint32_t paged_attend_smem() {
  return kPgWarps * PgCfg<D>::kRing + sizeof(PgQuery<D, FMT, QF32, NT>);
}

template <int D, int FMT, bool QF32, bool HILO, int NT>
__global__ void __launch_bounds__(kPgThreads, PgCfg<D>::kCtas) k_paged_attend(const PagedAttendArgs a) {
  using Warp = PgWarp<D, FMT, QF32, HILO, NT>;
  using Query = typename Warp::Query;
  constexpr int R = 8 * NT, kRec = D + kPartHeader;
  static_assert(kPgWarps * PgCfg<D>::kRing >= (kPgWarps * R * kRec + 4 * kPgThreads) * 4, "results fit over the rings");
  static_assert(kPgWarps * PgCfg<D>::kRing >= (R * kPgMaxCtas + 4 * kPgThreads) * 4, "a join fits over the rings");
  extern __shared__ __align__(128) uint8_t smem[];
  Query &qs = *reinterpret_cast<Query *>(smem + kPgWarps * PgCfg<D>::kRing);
  uint32_t *pre = reinterpret_cast<uint32_t *>(smem + paged_attend_smem<D, FMT, QF32, NT>());
  int *lens = reinterpret_cast<int *>(pre + a.B + 1);
  float(*red)[R][kRec] = reinterpret_cast<float(*)[R][kRec]>(smem);
  __shared__ float wgt[R][kPgWarps], rowM[R], rowL[R];
  __shared__ int last_s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int per_b = a.kv.hkv * a.rg;
  pdl_wait();
  paged_prefix<kPgThreads>(pre, a.B, [&](int b) {
    const int len = paged_len(a.n_gists, a.own_len, b, a.n_max, a.chunk, a.t_max);
    lens[b] = len;
    return static_cast<uint32_t>(per_b) * static_cast<uint32_t>((len + kPgStep - 1) / kPgStep);
  });
  const uint32_t total = pre[a.B];
  const uint32_t ctas = min(gridDim.x, max(1u, (total + a.min_steps - 1) / a.min_steps));
  const uint32_t cta = blockIdx.x;
  // sequences without rows: zeros, ln of an empty sum
  for (int b = cta; b < a.B; b += gridDim.x)
    if (lens[b] == 0) {
      const size_t row0 = static_cast<size_t>(b) * a.n_q * a.hq;
      for (int i = tid; i < a.n_q * a.hq * D; i += kPgThreads) store_out(a.out, row0 * D + i, 0.f, a.out_bf16);
      if (a.lse)
        for (int i = tid; i < a.n_q * a.hq; i += kPgThreads) a.lse[row0 + i] = neg_inf();
    }
  if (cta >= ctas) return;
  const uint32_t p0 = static_cast<uint32_t>(static_cast<uint64_t>(total) * cta / ctas);
  const uint32_t p1 = static_cast<uint32_t>(static_cast<uint64_t>(total) * (cta + 1) / ctas);
  Warp w;
  w.ring = smem_u32(smem) + warp * PgCfg<D>::kRing;
  for (uint32_t p = p0; p < p1;) {
    const int b = paged_find(pre, a.B, p);
    const uint32_t steps = (pre[b + 1] - pre[b]) / per_b;
    const uint32_t seg = (p - pre[b]) / steps;
    const uint32_t seg0 = pre[b] + seg * steps, seg1 = seg0 + steps;
    const uint32_t s0 = p - seg0, s1 = min(p1, seg1) - seg0;
    p = seg0 + s1;
    const int kvh = seg / a.rg, rg = seg % a.rg;
    const int len = lens[b];
    const int rows = min(R, a.n_q * a.group - rg * R);
    // query row r of the segment -> its row in q and out
    auto out_row = [&](int r) {
      const int x = rg * R + r;
      return (static_cast<size_t>(b) * a.n_q + x / a.group) * a.hq + kvh * a.group + x % a.group;
    };
    int lim[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int x = 0; x < 2; ++x) lim[nt][x] = len - (a.n_q - 1) + (rg * R + 8 * nt + 2 * t + x) / a.group;
    const int n = static_cast<int>(s1 - s0);
    const int first = (static_cast<int>(s0) * kPgWarps + warp) * 32;
    int mine = 0;  // tiles of this warp that hold a row
    if (first < len) mine = min(n, (len - first + kPgStep - 1) / kPgStep);
    const int32_t *table = a.kv.table + static_cast<size_t>(b) * a.kv.max_pages;
    auto key0 = [&](int i) { return first + i * kPgStep; };
    auto raw = [&](int i) {
      const int k = key0(i) + lane;
      return k < len ? k : -1;
    };
    auto queries = [&] {
      if (warp < NT)
        qs.load(
            warp,
            [&](int r) -> const void * {
              return r < rows ? static_cast<const uint8_t *>(a.q) + out_row(r) * D * (QF32 ? 4 : 2) : nullptr;
            },
            a.scale_log2);
      __syncthreads();
    };
    if (a.n_q > 1)
      w.template run<true>(a.kv, table, kvh, mine, qs, raw, key0, lim, a.status, queries);
    else
      w.template run<false>(a.kv, table, kvh, mine, qs, raw, key0, lim, a.status, queries);
    __syncthreads();  // every ring is drained: red may overwrite them
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float *dst = red[warp][8 * nt + 2 * t + x];
#pragma unroll
        for (int j = 0; j < Warp::MT; ++j)
          *reinterpret_cast<float2 *>(dst + kPartHeader + g * (D / 8) + 2 * j) =
              x ? make_float2(w.o[nt][j][0].y, w.o[nt][j][1].y) : make_float2(w.o[nt][j][0].x, w.o[nt][j][1].x);
        if (g == 0) {
          dst[0] = w.m[nt][x];
          dst[1] = w.l[nt][x];
        }
      }
    __syncthreads();
    if (tid < R) {
      float M = neg_inf(), L = 0.f;
#pragma unroll
      for (int i = 0; i < kPgWarps; ++i) M = fmaxf(M, red[i][tid][0]);
#pragma unroll
      for (int i = 0; i < kPgWarps; ++i) {
        const float c = exp2_approx(red[i][tid][0] - (M == neg_inf() ? 0.f : M));
        wgt[tid][i] = c;
        L = fmaf(c, red[i][tid][1], L);
      }
      rowM[tid] = M;
      rowL[tid] = L;
    }
    __syncthreads();
    const uint32_t c0 = static_cast<uint32_t>(((static_cast<uint64_t>(seg0) + 1) * ctas - 1) / total);
    const uint32_t c1 = static_cast<uint32_t>((static_cast<uint64_t>(seg1) * ctas - 1) / total);
    const bool whole = c0 == c1;
    auto put = [&](int r, int d, float4 v, float M, float L) {  // 4 dims of a finished row
      const size_t o = out_row(r) * D + d;
      const float i = L != 0.f ? 1.f / L : 0.f;
      if (a.out_bf16) {
        __nv_bfloat162 *dst = reinterpret_cast<__nv_bfloat162 *>(static_cast<__nv_bfloat16 *>(a.out) + o);
        dst[0] = __floats2bfloat162_rn(v.x * i, v.y * i);
        dst[1] = __floats2bfloat162_rn(v.z * i, v.w * i);
      } else {
        *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + o) = make_float4(v.x * i, v.y * i, v.z * i, v.w * i);
      }
      if (d == 0 && a.lse) a.lse[out_row(r)] = L != 0.f ? (M + __log2f(L)) * kLn2 : neg_inf();
    };
    // this CTA's record: slot 1 if the segment starts in its part, else slot 0
    float *rec = a.part + (static_cast<size_t>(cta) * 2 + (cta == c0 ? 1 : 0)) * R * kRec;
    for (int i = tid; i < rows * (D / 4); i += kPgThreads) {
      const int r = i / (D / 4), d = 4 * (i % (D / 4));
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < kPgWarps; ++k) {
        const float4 x = *reinterpret_cast<const float4 *>(&red[k][r][kPartHeader + d]);
        const float c = wgt[r][k];
        v = make_float4(fmaf(c, x.x, v.x), fmaf(c, x.y, v.y), fmaf(c, x.z, v.z), fmaf(c, x.w, v.w));
      }
      if (whole) {
        put(r, d, v, rowM[r], rowL[r]);
      } else {
        float *dst = rec + static_cast<size_t>(r) * kRec;
        *reinterpret_cast<float4 *>(dst + kPartHeader + d) = v;
        if (d == 0) *reinterpret_cast<float2 *>(dst) = make_float2(rowM[r], rowL[r]);
      }
    }
    if (!whole) {
      __syncthreads();
      if (tid == 0) {
        __threadfence();
        uint32_t *counter = a.counters + (static_cast<size_t>(b) * per_b + seg);
        const bool last = atomicAdd(counter, 1u) == c1 - c0;
        if (last) {
          __threadfence();
          *counter = 0u;
        }
        last_s = last;
      }
      __syncthreads();
      if (last_s) {
        // join the records of CTAs c0 .. c1 (c0's in slot 1), in that order
        const int nr = static_cast<int>(c1 - c0) + 1;
        auto rec_of = [&](int k, int r) {
          return a.part + ((static_cast<size_t>(c0 + k) * 2 + (k == 0 ? 1 : 0)) * R + r) * kRec;
        };
        float *cw = reinterpret_cast<float *>(smem);                             // [rows][nr] weights
        float4 *sums = reinterpret_cast<float4 *>(smem) + (R * kPgMaxCtas) / 4;  // [kPgThreads]
        for (int r = warp; r < rows; r += kPgWarps) {
          float M = neg_inf(), L = 0.f;
          for (int k = lane; k < nr; k += 32) M = fmaxf(M, __ldcg(rec_of(k, r)));
          M = warp_max(M);
          const float mm = M == neg_inf() ? 0.f : M;
          for (int k = lane; k < nr; k += 32) {
            const float2 h = __ldcg(reinterpret_cast<const float2 *>(rec_of(k, r)));
            const float c = exp2_approx(h.x - mm);
            cw[r * nr + k] = c;
            L = fmaf(c, h.y, L);
          }
          L = warp_sum(L);
          if (lane == 0) {
            rowM[r] = M;
            rowL[r] = L;
          }
        }
        __syncthreads();
        // items of 4 dims; when they are few, several threads share an item's records
        const int items = rows * (D / 4);
        const int share = items >= kPgThreads ? 1 : kPgThreads / items;
        for (int i0 = 0; i0 < items; i0 += kPgThreads) {
          const int i = i0 + (share > 1 ? tid % items : tid), part = share > 1 ? tid / items : 0;
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
          const int r = i / (D / 4), d = 4 * (i % (D / 4));
          if (i < items && part < share) {
#pragma unroll 8
            for (int k = part; k < nr; k += share) {
              const float4 x = __ldcg(reinterpret_cast<const float4 *>(rec_of(k, r) + kPartHeader + d));
              const float c = cw[r * nr + k];
              v = make_float4(fmaf(c, x.x, v.x), fmaf(c, x.y, v.y), fmaf(c, x.z, v.z), fmaf(c, x.w, v.w));
            }
          }
          if (share > 1) {
            sums[tid] = v;
            __syncthreads();
            if (tid < items) {
              for (int k = 1; k < share; ++k) {
                const float4 x = sums[tid + k * items];
                v = make_float4(v.x + x.x, v.y + x.y, v.z + x.z, v.w + x.w);
              }
            }
          }
          if (i < items && part == 0) put(r, d, v, rowM[r], rowL[r]);
        }
      }
    }
    __syncthreads();  // results, queries and row sums are read: the next segment may overwrite them
  }
  pdl_trigger();
}

// ------------------------------------------------------------------ unfolding
// Grid (splits, hq, B) as k_unfold: split s of row (b, h) takes its share of
// the selected chunks; the last split also takes the own chunk.  The rows of
// the share, in list order, form the 32-row tiles of the warps (a tile may
// span chunks and pages); one of the 8 query columns is in use.  The gists
// of selected chunks (exclude mode) are summed on the CUDA cores while the
// first copies are in flight, as a record of their own.
struct PagedUnfoldArgs {
  UnfoldArgs u;  // raw_k, raw_v and the tensor maps unused
  PagedKV kv;
};

constexpr int kPuWarps = kUnfoldWarps;

// rings (over them, once drained, the warps' results) | queries | chunk ids | gist logits
template <int D, int FMT, bool QF32>
__host__ __device__ inline size_t paged_unfold_smem(int per) {
  return kPuWarps * PgCfg<D>::kRing + sizeof(PgQuery<D, FMT, QF32, 1>) + static_cast<size_t>(per) * 8;
}

// The CTA's partial (its 2 kPuWarps states in red) goes to the row's split
// slot; the CTA that arrives last at the row's counter joins all splits with
// the prior partials and writes the row.  A NaN among the attended values
// stays one.
template <int D>
__device__ void paged_unfold_finish(const UnfoldArgs &a, size_t row, int split, const float (*red)[2 + D],
                                    int &last_s) {
  constexpr int NW = 2 * kPuWarps, kRec = D + kPartHeader;
  const int tid = threadIdx.x;
  __syncthreads();
  float *rec = a.part + (row * a.n_split + split) * kRec;
  float M = neg_inf(), L = 0.f, x = 0.f;
#pragma unroll
  for (int w = 0; w < NW; ++w) M = fmaxf(M, red[w][0]);
  float mm = M == neg_inf() ? 0.f : M;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    const float c = exp2_approx(red[w][0] - mm);
    L = fmaf(c, red[w][1], L);
    if (tid < D) x = fmaf(c, red[w][2 + tid], x);
  }
  if (a.n_split > 1 || a.prior) {
    if (tid < D) rec[kPartHeader + tid] = x;
    if (tid == 0) {
      rec[0] = M;
      rec[1] = L;
    }
    __syncthreads();
    if (tid == 0) {
      int last = 1;
      if (a.n_split > 1) {
        __threadfence();
        last = atomicAdd(&a.counters[row], 1u) == static_cast<uint32_t>(a.n_split - 1);
        if (last) {
          __threadfence();
          a.counters[row] = 0u;
        }
      }
      last_s = last;
    }
    __syncthreads();
    if (!last_s) return;
    const float *recs[2] = {a.part + row * a.n_split * kRec, a.prior ? a.prior + row * a.n_prior * kRec : nullptr};
    const int counts[2] = {a.n_split, a.prior ? a.n_prior : 0};
    M = neg_inf();
    for (int li = 0; li < 2; ++li)
      for (int i = 0; i < counts[li]; ++i) M = fmaxf(M, __ldcg(recs[li] + static_cast<size_t>(i) * kRec));
    mm = M == neg_inf() ? 0.f : M;
    L = 0.f;
    x = 0.f;
    for (int li = 0; li < 2; ++li)
#pragma unroll 4
      for (int i = 0; i < counts[li]; ++i) {
        const float *r = recs[li] + static_cast<size_t>(i) * kRec;
        const float c = exp2_approx(__ldcg(r) - mm);
        L = fmaf(c, __ldcg(r + 1), L);
        if (tid < D) x = fmaf(c, __ldcg(r + kPartHeader + tid), x);
      }
  }
  if (tid < D) store_out(a.out, row * D + tid, L != 0.f ? x / L : 0.f, a.out_bf16);
  if (tid == 0 && a.lse) a.lse[row] = L != 0.f ? (M + __log2f(L)) * kLn2 : neg_inf();
}

template <int D, int FMT, bool QF32, bool HILO>
__global__ void __launch_bounds__(kUnfoldThreads, PgCfg<D>::kCtas)
    k_paged_unfold(const __grid_constant__ PagedUnfoldArgs pa) {
  using Warp = PgWarp<D, FMT, QF32, HILO, 1>;
  using Query = typename Warp::Query;
  const UnfoldArgs &a = pa.u;
  const PagedKV &kv = pa.kv;
  extern __shared__ __align__(128) uint8_t smem[];
  const int per = (a.k + a.n_split - 1) / a.n_split;
  Query &qs = *reinterpret_cast<Query *>(smem + kPuWarps * PgCfg<D>::kRing);
  int *items = reinterpret_cast<int *>(smem + kPuWarps * PgCfg<D>::kRing + sizeof(Query));
  float *item_z = reinterpret_cast<float *>(items + per);
  float(*red)[2 + D] = reinterpret_cast<float(*)[2 + D]>(smem);
  __shared__ int n_items_s, is_last_s, take_s[2];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  int split, h, b;
  if (a.ready.w) {
    if (tid == 0) {
      int sp = 0;
      take_s[0] = unfold_take_row(a, sp);
      take_s[1] = sp;
    }
    __syncthreads();
    if (take_s[0] < 0) {  // flagged: nothing to attend
      unfold_ready_done(a);
      return;
    }
    split = take_s[1];
    h = take_s[0] % a.hq;
    b = take_s[0] / a.hq;
  } else {
    pdl_wait();
    split = blockIdx.x;
    h = blockIdx.y;
    b = blockIdx.z;
  }
  const int kvh = h / a.group;
  const size_t row = static_cast<size_t>(b) * a.hq + h;
  const int N = min(min(max(__ldcg(a.n_gists + b), 0), a.n_max), a.t_max / a.chunk);
  int own = min(max(__ldcg(a.own_len + b), 0), a.chunk);
  if (static_cast<int64_t>(N) * a.chunk + own > a.t_max) own = max(0, a.t_max - N * a.chunk);
  if (split != a.n_split - 1) own = 0;

  // Selected chunks of this split, in list order (invalid entries dropped).
  const int i0 = min(a.k, split * per), i1 = min(a.k, i0 + per);
  if (warp == 0) {
    int cnt = 0;
    for (int base = i0; base < i1; base += 32) {
      const int i = base + lane;
      int m = -1;
      if (i < i1) {
        m = __ldcg(a.sel_idx + row * a.k + i);
        if (m >= N) {
          flag_error(a.status, GSA_DEVERR_BAD_INDEX);
          m = -1;
        }
      }
      const unsigned ball = __ballot_sync(0xffffffffu, m >= 0);
      if (m >= 0) {
        const int slot = cnt + __popc(ball & ((1u << lane) - 1u));
        items[slot] = m;
        if (a.exclude) item_z[slot] = __ldcg(a.sel_score + row * a.k + i) * kLog2e;
      }
      cnt += __popc(ball);
    }
    if (lane == 0) n_items_s = cnt;
  }
  Warp w;
  w.ring = smem_u32(smem) + warp * PgCfg<D>::kRing;
  if (warp == 1)
    qs.load(
        0,
        [&](int r) -> const void * {
          return r == 0 ? static_cast<const uint8_t *>(a.q) + row * D * (QF32 ? 4 : 2) : nullptr;
        },
        a.scale_log2);
  __syncthreads();
  const int n_sel = n_items_s, sel_rows = n_sel * a.chunk, n_keys = sel_rows + own;
  const int n_tiles = (n_keys + 31) >> 5;
  const int mine = n_tiles > warp ? (n_tiles - warp + kPuWarps - 1) / kPuWarps : 0;
  auto key0 = [&](int i) { return (warp + kPuWarps * i) * 32; };
  auto raw = [&](int i) {
    const int j = key0(i) + lane;
    if (j < sel_rows) {
      const int it = kv.chunk.div(j);
      return items[it] * a.chunk + (j - it * a.chunk);
    }
    return j < n_keys ? N * a.chunk + (j - sel_rows) : -1;
  };
  // gists of the selected chunks: D / 32 dims a lane
  constexpr int E = D / 32;
  float gm = neg_inf(), gl = 0.f, ga[E];
#pragma unroll
  for (int e = 0; e < E; ++e) ga[e] = 0.f;
  auto gists = [&] {
    if (!a.exclude) return;
    const size_t gv0 = (static_cast<size_t>(b) * a.hkv + kvh) * a.n_max;
#pragma unroll 4
    for (int i = warp; i < n_sel; i += kPuWarps) {
      const float z = item_z[i];
      const size_t at = (gv0 + items[i]) * D + E * lane;
      float v[E];
      if (QF32) {
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = __ldcg(static_cast<const float *>(a.gist_v) + at + e);
      } else {
        const uint32_t *p = reinterpret_cast<const uint32_t *>(static_cast<const __nv_bfloat16 *>(a.gist_v) + at);
#pragma unroll
        for (int e = 0; e < E / 2; ++e) {
          const uint32_t x = __ldcg(p + e);
          v[2 * e] = bf16_lo(x);
          v[2 * e + 1] = bf16_hi(x);
        }
      }
      if (z > gm + kRescaleSlack) {
        const float c = exp2_approx(gm - z);
        gl *= c;
#pragma unroll
        for (int e = 0; e < E; ++e) ga[e] *= c;
        gm = z;
      }
      const float p = exp2_approx(z - (gm == neg_inf() ? 0.f : gm));
      gl += p;
#pragma unroll
      for (int e = 0; e < E; ++e) ga[e] = fmaf(p, v[e], ga[e]);
    }
  };
  w.template run<false>(kv, kv.table + static_cast<size_t>(b) * kv.max_pages, kvh, mine, qs, raw, key0, nullptr,
                        a.status, gists);
  pdl_trigger();
  __syncthreads();  // every ring is drained: red may overwrite them
  if (t == 0) {     // column 0
#pragma unroll
    for (int j = 0; j < Warp::MT; ++j) {
      red[warp][2 + g * (D / 8) + 2 * j] = w.o[0][j][0].x;
      red[warp][2 + g * (D / 8) + 2 * j + 1] = w.o[0][j][1].x;
    }
    if (g == 0) {
      red[warp][0] = w.m[0][0];
      red[warp][1] = w.l[0][0];
    }
  }
#pragma unroll
  for (int e = 0; e < E; ++e) red[kPuWarps + warp][2 + E * lane + e] = ga[e];
  if (lane == 0) {
    red[kPuWarps + warp][0] = gm;
    red[kPuWarps + warp][1] = gl;
  }
  paged_unfold_finish<D>(a, row, split, red, is_last_s);
  if (a.ready.w) unfold_ready_done(a);
}

}  // namespace gsa
