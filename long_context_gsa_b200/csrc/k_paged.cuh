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
//   z = K q        S^T[16 keys x 8 queries] with mma.sync, the KEYS as the A
//                  operand: a kv head's 4..8 query heads fill the 8 columns,
//                  where queries as A would leave 8..12 of 16 rows idle;
//   p = 2^(z - m)  lazy online softmax in fp32 (m raised when exceeded by
//                  kPgSlack), the scale of K applied to z, that of V to p;
//   O^T += V^T p   V^T as A (the codes interleaved in registers) and p as B
//                  (movmatrix turns the accumulator layout of S^T into it).
// Operands: codes are exact in fp16 and in int8, queries and weights are sums of
// parts that hold about fp32's 24 bits:
//   int8 keys: m16n8k32 on the codes as they are; a query is 4 digits of 7 bits,
//     one product each, off by 2^-28 of the row's largest element at most (bf16:
//     exact down to 2^-19 of it); sums are exact integers.
//   e4m3 keys: m16n8k16 on fp16 (on sm_100a the e4m3 form of mma.sync runs as
//     conversions and two fp16 products, so the codes are converted once here);
//     queries as one fp16 term after a power-of-two scaling of the row to
//     [2^14, 2^15) (exact for bf16 down to 2^-31 of the scaling, off by 2^-39 of
//     it below), fp32 ones as two (2^-24 of the element, or 2^-39 again).
//   weights: two fp16 terms, relative to a power of two near the keys' scales of V
//     and to a reference weight (2^-24, or 2^-25 of the largest weight among keys
//     whose scales lie within 2^10 of the key's); bf16 outputs too, since what
//     their values cancel to is rounded, not the terms.  Tiles of scales farther
//     apart are taken in several turns (far_apart).
// Statistics, sums of weights and the running output are fp32.
//
// What bounds it: the reads of the codes, and the instructions that a tile of 32
// rows costs beside them.  Every warp copies its tiles with
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

constexpr float kPgSlack = 4.0f;     // p <= 2^4 before the reference is raised
// Weights in fp16: p <= 2^kPgSlack times a scale below 2 of the reference, up to 2^15 after a factor of 2^kPgUp.  With
// scales within 2^kPgBand of one another a weight of 1 (the reference's) is 1 at least there, and two terms hold it
// to 2^-24, smaller ones to 2^-25 of it.
constexpr uint32_t kPgUp = 10, kPgBand = 10;
constexpr uint32_t kPgLeast = 17u << 23, kPgInf = 0x7f800000u;  // bits of 2^-110, the least scale, and of infinity

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// c = A B (FIRST) or c += A B: fp16 16 x 16 times 16 x 8, int8 16 x 32 times 32 x 8.
template <bool FIRST>
__device__ __forceinline__ void mma_f16(float c[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  if (FIRST)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <bool FIRST>
__device__ __forceinline__ void mma_s8(int c[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  if (FIRST)
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=r"(c[0]), "=r"(c[1]), "=r"(c[2]), "=r"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "r"(0));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 8x8 block of 16-bit elements transposed across the warp's accumulator layout.
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
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

__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float2 unpack_h2(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2 *>(&w));
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
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}\n"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
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

// The queries of a segment in shared memory, as B fragments:
// [NT][term][k-step][lane], and the factor of each row's logits.  Row n
// (< 8 NT) is row(n), null when unused.
//   e4m3: kN fp16 terms, k-steps of 16 dims;
//   int8: kN digits of a fixed-point number |v| <= 2^kTopExp, k-steps of 32 dims.
template <int D, int FMT, bool QF32, int NT>
struct PgQuery {
  static constexpr bool kI8 = FMT == kFmtI8;
  static constexpr int kN = kI8 ? 4 : (QF32 ? 2 : 1);
  static constexpr int KS = kI8 ? D / 32 : D / 16;
  static constexpr int kTopExp = kI8 ? 7 * kN - 1 : 15;  // the row's largest is brought into [2^(kTopExp-1), 2^kTopExp)
  uint2 frag[NT][kN][KS][32];
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
    // a power of two; none for a row of zeros.  An inf or NaN makes the row's logits NaN.
    int sh = 0;
    if (a != 0 && a < 0x7f800000u) sh = min(kTopExp - 1 - (static_cast<int>(a >> 23) - 127), 120);
    const float up = __uint_as_float(static_cast<uint32_t>(127 + sh) << 23);
    const float down = __uint_as_float(static_cast<uint32_t>(127 - sh) << 23) * scale_log2;
    if (t == 0) f[8 * nt + g] = a < 0x7f800000u ? down : __uint_as_float(0x7fc00000u);
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      uint32_t w[kN][2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (kI8) {  // word h: dims 8 s + 4 h + 0..3
          const float *y = x + 8 * s + 4 * h;
          uint32_t d[kN][4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            int v = __float2int_rn(y[i] * up);
#pragma unroll
            for (int k = kN - 1; k >= 0; --k) {  // the last digit first; each in [-64, 63], the first takes the rest
              const int top = k == 0 ? v : ((v + 64) & 127) - 64;
              d[k][i] = static_cast<uint32_t>(top) & 0xffu;
              v = (v - top) >> 7;
            }
          }
#pragma unroll
          for (int k = 0; k < kN; ++k) w[k][h] = d[k][0] | d[k][1] << 8 | d[k][2] << 16 | d[k][3] << 24;
        } else {  // word h: dims 4 s + 2 h + 0, 1
          const float u = x[(4 * s + 2 * h) % (D / 4)] * up, v = x[(4 * s + 2 * h + 1) % (D / 4)] * up;
          w[0][h] = pack_h2(u, v);
          if (QF32) {
            const float2 r = unpack_h2(w[0][h]);
            w[kN - 1][h] = pack_h2(u - r.x, v - r.y);
          }
        }
      }
#pragma unroll
      for (int k = 0; k < kN; ++k) frag[nt][k][s][lane] = make_uint2(w[k][0], w[k][1]);
    }
  }
};

// The state of one warp over a run of tiles; NT groups of 8 query columns.
template <int D, int FMT, bool QF32, int NT>
struct PgWarp {
  using Cfg = PgCfg<D>;
  using Query = PgQuery<D, FMT, QF32, NT>;
  static constexpr int S = Cfg::kStages;
  static constexpr int MT = D / 16;           // m-tiles of O^T

  float m[NT][2], l[NT][2];  // columns 2t, 2t + 1
  float2 o[NT][MT][2];       // O^T: dims g*D/8 + 2j and + 2j + 1, (column 2t, column 2t + 1)
  // the copy pipeline
  int32_t pid;     // page of this lane's key in the next tile to copy (-1: none)
  uint32_t off;    // its row in that page
  float sck, scv;  // scales of this lane's key in the tile copied last (0 and -0: none)
  uint32_t ring;
  uint32_t low;    // bits of the least scale of V fetched so far
  static constexpr uint32_t kNoRow = 0xffffffffu;

  __device__ __forceinline__ void clear() {
    low = kPgInf;
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

  // The pool row of the fetched key, kNoRow without one (a page outside the
  // pool is flagged); its scales are fetched.
  __device__ __forceinline__ uint32_t locate(const PagedKV &kv, int kvh, bool wanted, uint32_t *status) {
    const bool live = static_cast<uint32_t>(pid) < static_cast<uint32_t>(kv.n_pages);
    if (wanted && !live) flag_error(status, GSA_DEVERR_BAD_INDEX);
    sck = 0.f;
    scv = -0.f;
    if (!live) return kNoRow;
    const uint32_t ph = static_cast<uint32_t>(pid) * kv.hkv + kvh;
    const size_t i = static_cast<size_t>(ph) * kv.blocks + kv.chunk.div(off);
    sck = __ldcg(kv.ks + i);
    scv = __ldcg(kv.vs + i);
    return ph * kv.page.d + off;
  }

  // Copy the tile whose keys lie at pool rows prow (one a lane) into stage st.
  __device__ __forceinline__ void copy(const PagedKV &kv, int st, uint32_t prow) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint32_t base = ring + st * Cfg::kStage;
    const uint32_t mask = __ballot_sync(0xffffffffu, prow != kNoRow);
    if (lane == 0) asm volatile("st.shared.u32 [%0], %1;" ::"r"(base + Cfg::kMask), "r"(mask) : "memory");
    // 32 rows one behind the other (a tile inside a page, or inside a chunk): one address and fixed steps
    const uint32_t row0 = __shfl_sync(0xffffffffu, prow, 0);
    if (__all_sync(0xffffffffu, prow == row0 + lane && prow != kNoRow)) {
      const size_t o8 = static_cast<size_t>(row0 + g) * D + t * 16;
      const uint8_t *k = kv.k + o8, *v = kv.v + o8;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          cp_async16(base + ((i * (D / 64) + c) * 32 + lane) * 16, k + 8 * i * D + 64 * c);
          cp_async16(base + Cfg::kK + v_off<D>(g + 8 * i, t + 4 * c), v + 8 * i * D + 64 * c);
        }
      return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // keys g + 8 i
      const uint32_t r = __shfl_sync(0xffffffffu, prow, g + 8 * i);
      const uint32_t bytes = r != kNoRow ? 16u : 0u;
      const size_t o8 = bytes ? static_cast<size_t>(r) * D + t * 16 : 0;
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        cp_async16(base + ((i * (D / 64) + c) * 32 + lane) * 16, kv.k + o8 + 64 * c, bytes);
        cp_async16(base + Cfg::kK + v_off<D>(g + 8 * i, t + 4 * c), kv.v + o8 + 64 * c, bytes);
      }
    }
  }

  // The scales of the tile in stage st, and how to take it: behind the mask the
  // bits of the power of two below its largest scale of V, or kPgInf when some
  // of them, or of earlier tiles', are too far apart for one reference (or NaN).
  __device__ __forceinline__ void put_scale(int st) {
    const int lane = threadIdx.x & 31;
    const uint32_t base = ring + st * Cfg::kStage, at = base + Cfg::kScales + lane * 4;
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(at), "f"(sck) : "memory");
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(at + 128), "f"(scv) : "memory");
    // bits order like the scales; the -0 of a key that is not there is below all others signed, above unsigned
    const int32_t top = max(static_cast<int32_t>(kPgLeast), __reduce_max_sync(0xffffffffu, __float_as_int(scv)));
    low = min(low, __reduce_min_sync(0xffffffffu, __float_as_uint(scv)));
    const uint32_t ref = static_cast<uint32_t>(top) > low + (kPgBand << 23) ? kPgInf : top & kPgInf;
    if (lane == 0) asm volatile("st.shared.u32 [%0], %1;" ::"r"(base + Cfg::kMask + 4), "r"(ref) : "memory");
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
  //
  // Weights enter the products as fp16, relative to a power of two near the
  // keys' largest scale of V and to each column's running reference m, as long
  // as every scale that the warp has met lies within 2^kPgBand of the others;
  // else far_apart takes the tile.
  template <bool CAUSAL>
  __device__ __forceinline__ void step(const Query &qs, int st, int key0, const int (*lim)[2]) {
    const uint32_t base = ring + st * Cfg::kStage;
    uint32_t mask, ref;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(mask), "=r"(ref) : "r"(base + Cfg::kMask));
    if (ref == kPgInf) {
      // on a copy of the state, so that nothing of the usual path's lives in memory
      PgWarp w = *this;
      int lim_[NT][2];
#pragma unroll
      for (int i = 0; i < NT; ++i)
        for (int x = 0; CAUSAL && x < 2; ++x) lim_[i][x] = lim[i][x];
      far_apart<CAUSAL>(w, qs, base, mask, key0, lim_);
      *this = w;
    } else {
      turn<CAUSAL, false>(qs, base, mask, ref, key0, lim);
    }
  }

  // A tile of scales that are far apart, or far from earlier ones: keys whose
  // scale is far below the largest are left for another turn, and each turn's
  // reference is its own largest logit.  A turn is to the running sums a tile
  // of its own, so no key is lost beside one of a larger scale, whatever their
  // weights.  16 x 32K rows take 98 us in the usual path (102 when every tile
  // looked for its largest logit), 136 here with one turn a tile and 233 with
  // two.
  template <bool CAUSAL>
  __device__ __noinline__ static void far_apart(PgWarp &w, const Query &qs, uint32_t base, uint32_t mask, int key0,
                                                const int (*lim)[2]) {
    const int lane = threadIdx.x & 31;
    const uint32_t own = __float_as_uint(ldsf(base + Cfg::kScales + 128 + 4 * lane)) & 0x7fffffffu;
    PgWarp s = w;
    do {
      const bool mine = (mask >> lane) & 1u;
      const uint32_t top = max(kPgLeast, __reduce_max_sync(0xffffffffu, mine && own < kPgInf ? own : 0u));
      // the key of the largest scale is among them, so the loop ends
      const uint32_t keys = __ballot_sync(0xffffffffu, mine && (own + (kPgBand << 23) >= top || top == kPgLeast));
      s.template turn<CAUSAL, true>(qs, base, keys, top & kPgInf, key0, lim);
      mask &= ~keys;
    } while (mask);
    w = s;
  }

  // The keys of the mask `keys` of a tile; ref: the power of two (its bits)
  // below the largest scale of V among them.
  template <bool CAUSAL, bool EXACT>
  __device__ __forceinline__ void turn(const Query &qs, uint32_t base, uint32_t keys, uint32_t ref, int key0,
                                       const int (*lim)[2]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint32_t scb = base + Cfg::kScales + 4 * g;
    // ---- z: value e of half h: key 16 h + g + 8 (e >> 1), column 2 t + (e & 1)
    float z[2][NT][4];
    logits(qs, base, z);
    bool masked = keys != 0xffffffffu;  // some key is not there, or not for every column
    if (CAUSAL) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) masked = masked || key0 + 32 > lim[nt][0] || key0 + 32 > lim[nt][1];
      masked = __any_sync(0xffffffffu, masked);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float kg[2] = {ldsf(scb + 64 * h), ldsf(scb + 64 * h + 32)};
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float2 f = *reinterpret_cast<const float2 *>(&qs.f[8 * nt + 2 * t]);
#pragma unroll
        for (int e = 0; e < 4; ++e)  // (in this order: kg f alone may pass fp32's range)
          z[h][nt][e] = z[h][nt][e] * (e & 1 ? f.y : f.x) * kg[e >> 1];
      }
    }
    if (masked) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int key = 16 * h + g + 8 * (e >> 1);
            if (!((keys >> key) & 1u) || (CAUSAL && key0 + key >= lim[nt][e & 1])) z[h][nt][e] = neg_inf();
          }
    }
    bool over = false;
    float mx[NT][2];
    auto across = [&] {  // the maxima over the lanes
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          mx[nt][x] = fmaxf(mx[nt][x], __shfl_xor_sync(0xffffffffu, mx[nt][x], 4));
          mx[nt][x] = fmaxf(mx[nt][x], __shfl_xor_sync(0xffffffffu, mx[nt][x], 8));
          mx[nt][x] = fmaxf(mx[nt][x], __shfl_xor_sync(0xffffffffu, mx[nt][x], 16));
        }
    };
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        mx[nt][x] = fmaxf(fmaxf(z[0][nt][x], z[0][nt][x + 2]), fmaxf(z[1][nt][x], z[1][nt][x + 2]));
        over = over || mx[nt][x] > m[nt][x] + kPgSlack;
      }
    if (EXACT) across();
    if (__any_sync(0xffffffffu, over)) {  // raise the references, rescale
      if (!EXACT) across();
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float c[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float v = mx[nt][x];
          c[x] = v > m[nt][x] ? exp2_approx(m[nt][x] - v) : 1.f;  // 0 when there was no reference
          l[nt][x] *= c[x];
          m[nt][x] = fmaxf(m[nt][x], v);
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
    // ---- weights: p = 2^(z - r) times the scale of V relative to ref (w <= 2^(kPgSlack + 1 + kPgUp)).
    // In exact turns f = 2^(r - m) takes the sums to the running reference, and with ref the products.
    const float up = __uint_as_float((254u << 23) + (kPgUp << 23) - ref);  // 2^kPgUp / ref
    float vg[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) vg[i] = ldsf(scb + 128 + 32 * i) * up;
    uint32_t pb[2][NT][2][2];  // [term][group][half]: B fragments, keys 2t, 2t + 1 and 2t + 8, 2t + 9
    float2 back[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float r[2], sum[2] = {0.f, 0.f};
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        r[x] = EXACT ? mx[nt][x] : m[nt][x];
        if (r[x] == neg_inf()) r[x] = 0.f;  // no key yet (or NaN alone, which p then is)
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float p = exp2_approx(z[h][nt][e] - r[e & 1]);
          (EXACT ? sum[e & 1] : l[nt][e & 1]) += p;
          w[e] = p * vg[2 * h + (e >> 1)];
        }
        if ((CAUSAL || EXACT) && masked) {  // scales of keys that a column does not see, or of other turns, stay out
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (z[h][nt][e] == neg_inf()) w[e] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t hi = pack_h2(w[2 * i], w[2 * i + 1]);
          pb[0][nt][h][i] = movmatrix_trans(hi);
          const float2 r = unpack_h2(hi);
          pb[1][nt][h][i] = movmatrix_trans(pack_h2(w[2 * i] - r.x, w[2 * i + 1] - r.y));
        }
      }
      const float down = __uint_as_float(ref) * (1.f / (1u << kPgUp));
      back[nt] = make_float2(down, down);
      if (EXACT) {
        float f[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          f[x] = mx[nt][x] == neg_inf() ? 0.f : exp2_approx(mx[nt][x] - m[nt][x]);
          l[nt][x] = fmaf(f[x], sum[x], l[nt][x]);
        }
        back[nt] = make_float2(f[0] * down, f[1] * down);
      }
    }
    // ---- O^T += V^T p: dims in words of 4 codes, rows 2t, 2t + 1, 2t + 8, 2t + 9 of each half
    constexpr int kW = D / 32;
    uint32_t vr[2][4][kW];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t r = 16 * h + 2 * t + (i & 1) + 8 * (i >> 1);
        if constexpr (D == 128) {
          lds4(base + Cfg::kK + v_off<D>(r, g), vr[h][i]);
        } else {
          asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];"
                       : "=r"(vr[h][i][0]), "=r"(vr[h][i][1])
                       : "r"(base + Cfg::kK + v_off<D>(r, g >> 1) + (g & 1) * 8));
        }
      }
#pragma unroll
    for (int w = 0; w < kW; ++w)
#pragma unroll
      for (int j = 0; j < 2; ++j) {  // dims 4 w + 2 j and + 1 of the lane's D / 8
        float d[NT][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t a0, a1, a2, a3;  // (row 2t, row 2t + 1) pairs of the two dims, then rows 2t + 8, 2t + 9
          codes_to_h2<FMT>(__byte_perm(vr[h][0][w], vr[h][1][w], j ? 0x7362 : 0x5140), a0, a1);
          codes_to_h2<FMT>(__byte_perm(vr[h][2][w], vr[h][3][w], j ? 0x7362 : 0x5140), a2, a3);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if (h == 0)
              mma_f16<true>(d[nt], a0, a1, a2, a3, pb[0][nt][h][0], pb[0][nt][h][1]);
            else
              mma_f16<false>(d[nt], a0, a1, a2, a3, pb[0][nt][h][0], pb[0][nt][h][1]);
            mma_f16<false>(d[nt], a0, a1, a2, a3, pb[1][nt][h][0], pb[1][nt][h][1]);
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          o[nt][2 * w + j][0] = fma2(back[nt], make_float2(d[nt][0], d[nt][1]), o[nt][2 * w + j][0]);
          o[nt][2 * w + j][1] = fma2(back[nt], make_float2(d[nt][2], d[nt][3]), o[nt][2 * w + j][1]);
        }
      }
  }

  // z[half][group][e] = codes . query terms (without the scales).
  __device__ __forceinline__ void logits(const Query &qs, uint32_t base, float (*z)[NT][4]) {
    const int lane = threadIdx.x & 31;
    uint32_t kw[D / 64][4][4];  // [piece][row g + 8 i][word]
#pragma unroll
    for (int c = 0; c < D / 64; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) lds4(base + ((i * (D / 64) + c) * 32 + lane) * 16, kw[c][i]);
    if constexpr (FMT == kFmtI8) {
      // digits 0, 1 share an accumulator (times 128 in between), so do 2, 3
      int acc[2][2][NT][4];
#pragma unroll
      for (int k = 0; k < Query::kN; ++k) {
        if (k & 1)
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[k / 2][h][nt][e] *= 128;
#pragma unroll
        for (int s = 0; s < D / 32; ++s)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const uint2 b = qs.frag[nt][k][s][lane];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t a0 = kw[s / 2][2 * h][2 * (s & 1)], a1 = kw[s / 2][2 * h + 1][2 * (s & 1)];
              const uint32_t a2 = kw[s / 2][2 * h][2 * (s & 1) + 1], a3 = kw[s / 2][2 * h + 1][2 * (s & 1) + 1];
              if (s == 0 && !(k & 1))
                mma_s8<true>(acc[k / 2][h][nt], a0, a1, a2, a3, b.x, b.y);
              else
                mma_s8<false>(acc[k / 2][h][nt], a0, a1, a2, a3, b.x, b.y);
            }
          }
      }
      static_assert(Query::kN == 4, "(d0 128 + d1) 2^14 + (d2 128 + d3)");
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            z[h][nt][e] = fmaf(static_cast<float>(acc[0][h][nt][e]), 16384.f, static_cast<float>(acc[1][h][nt][e]));
    } else {
#pragma unroll
      for (int s = 0; s < D / 16; ++s) {
        uint32_t a[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          codes_to_h2<FMT>(kw[s / 4][2 * h][s & 3], a[h][0], a[h][2]);
          codes_to_h2<FMT>(kw[s / 4][2 * h + 1][s & 3], a[h][1], a[h][3]);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < Query::kN; ++k) {
            const uint2 b = qs.frag[nt][k][s][lane];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if (s == 0 && k == 0)
                mma_f16<true>(z[h][nt], a[h][0], a[h][1], a[h][2], a[h][3], b.x, b.y);
              else
                mma_f16<false>(z[h][nt], a[h][0], a[h][1], a[h][2], a[h][3], b.x, b.y);
            }
          }
      }
    }
  }

  // Run n tiles whose keys are found through the page table: raw(i) is this
  // lane's key of tile i as a raw row (< 0: none), key0(i) the index of the
  // tile's first key; before() runs once while the first copies are in flight
  // (and makes qs ready).
  template <bool CAUSAL, typename RawFn, typename Key0Fn, typename BeforeFn>
  __device__ __forceinline__ void run(const PagedKV &kv, const int32_t *table, int kvh, int n, const Query &qs,
                                      RawFn raw, Key0Fn key0, const int (*lim)[2], uint32_t *status, BeforeFn before) {
    clear();
    int r = n > 0 ? raw(0) : -1;
    fetch(kv, table, r);
    auto next = [&](int j, int st) {  // copy tile j, fetch the pages of tile j + 1
      copy(kv, st, locate(kv, kvh, r >= 0, status));
      r = j + 1 < n ? raw(j + 1) : -1;
      fetch(kv, table, r);
    };
#pragma unroll
    for (int i = 0; i < S - 1; ++i) {
      if (i > 0 && i - 1 < n) put_scale(i - 1);
      if (i < n) next(i, i);
      cp_async_commit();
    }
    before();
    int st = 0, stc = S - 1;  // stage worked on, stage copied into
    for (int i = 0; i < n; ++i) {
      const int j = i + S - 1;  // tile copied in this turn
      if (j - 1 < n) put_scale(stc == 0 ? S - 1 : stc - 1);
      cp_async_wait<S - 2>();
      __syncwarp();
      if (j < n) next(j, stc);
      cp_async_commit();
      step<CAUSAL>(qs, st, key0(i), lim);
      st = st == S - 1 ? 0 : st + 1;
      stc = stc == S - 1 ? 0 : stc + 1;
    }
    finish();
  }

  // Run n tiles whose keys are known: row(i) gives this lane's key of tile i
  // as a pool row (kNoRow: none) and fetches its scales into sck, scv.
  template <typename RowFn, typename BeforeFn>
  __device__ __forceinline__ void run_known(const PagedKV &kv, int n, const Query &qs, RowFn row, BeforeFn before) {
    clear();
#pragma unroll
    for (int i = 0; i < S - 1; ++i) {
      if (i > 0 && i - 1 < n) put_scale(i - 1);
      if (i < n) copy(kv, i, row(i));
      cp_async_commit();
    }
    before();
    int st = 0, stc = S - 1;
    for (int i = 0; i < n; ++i) {
      const int j = i + S - 1;
      if (j - 1 < n) put_scale(stc == 0 ? S - 1 : stc - 1);
      cp_async_wait<S - 2>();
      __syncwarp();
      if (j < n) copy(kv, stc, row(j));
      cp_async_commit();
      step<false>(qs, st, 0, nullptr);
      st = st == S - 1 ? 0 : st + 1;
      stc = stc == S - 1 ? 0 : stc + 1;
    }
    finish();
  }

  // No copies in flight, the lanes' sums added up.
  __device__ __forceinline__ void finish() {
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
// single long sequences load every SM alike.  A segment begins with kPgHead
// empty steps on that line, about what starting one costs a CTA, and one of up
// to kPgWhole steps is not cut (64 ragged sequences of up to 3000 rows: 42 us
// with 0 head steps, 28 with 2, 31 with 8; 37 of up to 9001 rows with 4 fp32
// query tokens each: 67, 55, 62).  A segment inside one CTA is written
// directly; of one that several CTAs share each leaves a partial record, which
// k_paged_join adds up in CTA order.  (Joining by the last CTA to arrive took
// 10 us of 108 at 4 x 128K rows: 28 records of a segment, one dependent load
// of a CTA's 4 warps behind the other.)  CTAs of 4 warps, 3 or 4 on an SM: one
// joins its warps while the others stream.
// Measured, replayed from a graph / as calls one behind the other, where the
// power cap lowers the clock: 16 x 32K rows of e4m3 98 / 109 to 117 us (5.5 /
// 5.0 TB/s), 4 x 128K of int8 111 / 121 to 129 (4.8 / 4.4); DRAM is busy 58 and 50
// % of the kernel, issue slots 55 and 41 %, and most waits are for fixed
// latencies.  16 fp32 query rows (the 37 sequences above): 55 us for 18 us of
// bytes, tensor pipe 30 % and issue slots 44 % busy, 12 warps an SM too few to
// cover the rest.
constexpr int kPgWarps = 4;
constexpr int kPgThreads = 32 * kPgWarps;
constexpr int kPgStep = 32 * kPgWarps;  // rows of one CTA step
constexpr uint32_t kPgHead = 2;         // empty steps before a segment's rows
constexpr uint32_t kPgWhole = 4;        // steps of a segment that is not cut
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
  int4 *joins;                 // [ctas]: (b, segment, last CTA, 0) of the cut segment that begins in a CTA; b < 0: none
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

// Query row x (token x / group, head x % group of the kv head) of sequence b: its row in q and out.
__device__ __forceinline__ size_t paged_row(const PagedAttendArgs &a, int b, int kvh, int x) {
  return (static_cast<size_t>(b) * a.n_q + x / a.group) * a.hq + kvh * a.group + x % a.group;
}

// Four dims of a finished row: sum of weighted values v, base-2 maximum M and sum L of the weights.
template <int D>
__device__ __forceinline__ void paged_put(const PagedAttendArgs &a, size_t row, int d, float4 v, float M, float L) {
  const size_t o = row * D + d;
  const float i = L != 0.f ? 1.f / L : 0.f;
  if (a.out_bf16) {
    __nv_bfloat162 *dst = reinterpret_cast<__nv_bfloat162 *>(static_cast<__nv_bfloat16 *>(a.out) + o);
    dst[0] = __floats2bfloat162_rn(v.x * i, v.y * i);
    dst[1] = __floats2bfloat162_rn(v.z * i, v.w * i);
  } else {
    *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + o) = make_float4(v.x * i, v.y * i, v.z * i, v.w * i);
  }
  if (d == 0 && a.lse) a.lse[row] = L != 0.f ? (M + __log2f(L)) * kLn2 : neg_inf();
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

// Dynamic shared memory: rings (over them, once drained, the warps' results) |
// queries | prefix sums [B + 1] and lengths [B].
template <int D, int FMT, bool QF32, int NT>
__host__ __device__ constexpr uint32_t paged_attend_smem() {
  return kPgWarps * PgCfg<D>::kRing + sizeof(PgQuery<D, FMT, QF32, NT>);
}

template <int D, int FMT, bool QF32, int NT>
__global__ void __launch_bounds__(kPgThreads, PgCfg<D>::kCtas) k_paged_attend(const PagedAttendArgs a) {
  using Warp = PgWarp<D, FMT, QF32, NT>;
  using Query = typename Warp::Query;
  constexpr int R = 8 * NT, kRec = D + kPartHeader;
  static_assert(PgCfg<D>::kRing >= R * kRec * 4, "the warps' results fit over the rings");
  extern __shared__ __align__(128) uint8_t smem[];
  Query &qs = *reinterpret_cast<Query *>(smem + kPgWarps * PgCfg<D>::kRing);
  uint32_t *pre = reinterpret_cast<uint32_t *>(smem + paged_attend_smem<D, FMT, QF32, NT>());
  int *lens = reinterpret_cast<int *>(pre + a.B + 1);
  float(*red)[R][kRec] = reinterpret_cast<float(*)[R][kRec]>(smem);
  __shared__ float wgt[R][kPgWarps], rowM[R], rowL[R];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int per_b = a.kv.hkv * a.rg;
  pdl_wait();
  pdl_trigger();  // the join kernel waits for this grid; its CTAs fit once ours leave
  paged_prefix<kPgThreads>(pre, a.B, [&](int b) {
    const int len = paged_len(a.n_gists, a.own_len, b, a.n_max, a.chunk, a.t_max);
    lens[b] = len;
    const uint32_t steps = static_cast<uint32_t>((len + kPgStep - 1) / kPgStep);
    return static_cast<uint32_t>(per_b) * (steps ? steps + kPgHead : 0u);
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
  int4 join = make_int4(-1, 0, 0, 0);
  if (cta >= ctas) {
    if (tid == 0) a.joins[cta] = join;
    return;
  }
  // where CTA c's part begins: a cut inside a short segment moves to its start
  auto cut = [&](uint32_t c) {
    const uint32_t p = static_cast<uint32_t>(static_cast<uint64_t>(total) * c / ctas);
    if (p == total) return p;
    const int b = paged_find(pre, a.B, p);
    const uint32_t steps = (pre[b + 1] - pre[b]) / per_b;
    return steps > kPgWhole + kPgHead ? p : p - (p - pre[b]) % steps;
  };
  const uint32_t p0 = cut(cta), p1 = cut(cta + 1);
  Warp w;
  w.ring = smem_u32(smem) + warp * PgCfg<D>::kRing;
  for (uint32_t p = p0; p < p1;) {
    const int b = paged_find(pre, a.B, p);
    const uint32_t steps = (pre[b + 1] - pre[b]) / per_b;  // with the head
    const uint32_t seg = (p - pre[b]) / steps;
    const uint32_t seg0 = pre[b] + seg * steps + kPgHead, seg1 = seg0 + steps - kPgHead;  // its rows
    const uint32_t begin = max(p, seg0);
    p = min(p1, seg1);
    if (p <= begin) {  // this part ends inside the head
      p = p1;
      continue;
    }
    const uint32_t s0 = begin - seg0, s1 = p - seg0;
    const int kvh = seg / a.rg, rg = seg % a.rg;
    const int len = lens[b];
    const int rows = min(R, a.n_q * a.group - rg * R);
    auto out_row = [&](int r) { return paged_row(a, b, kvh, rg * R + r); };
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
    const bool whole = begin == seg0 && p == seg1;
    // this CTA's record: slot 1 if the segment starts in its part, else slot 0
    float *rec = a.part + (static_cast<size_t>(cta) * 2 + (begin == seg0 ? 1 : 0)) * R * kRec;
    if (!whole && begin == seg0)
      join = make_int4(b, static_cast<int>(seg),
                       static_cast<int>((static_cast<uint64_t>(seg1) * ctas - 1) / total), 0);
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
        paged_put<D>(a, out_row(r), d, v, rowM[r], rowL[r]);
      } else {
        float *dst = rec + static_cast<size_t>(r) * kRec;
        *reinterpret_cast<float4 *>(dst + kPartHeader + d) = v;
        if (d == 0) *reinterpret_cast<float2 *>(dst) = make_float2(rowM[r], rowL[r]);
      }
    }
    __syncthreads();  // results, queries and row sums are read: the next segment may overwrite them
  }
  if (tid == 0) a.joins[cta] = join;
}

// Grid (ctas, R / kRows) behind k_paged_attend: CTA (c, y) adds up kRows rows
// of the cut segment that begins in c's part, W warps a row.  The records
// lie equally spaced (the first one's in slot 1, the others in slot 0); a
// row's warps share them out (D / 4 lanes a record), the first kBatch of a lane
// fetched while the weights (a record a lane, by every warp for itself) are
// made.
template <int D, int NT, int W>
__global__ void __launch_bounds__(256) k_paged_join(const PagedAttendArgs a) {
  constexpr int R = 8 * NT, kRec = D + kPartHeader, kStride = 2 * R * kRec, kRows = 8 / W;
  constexpr int kSub = 128 / D, kBatch = 8, kEach = W * kSub;  // records side by side in a row's warps
  extern __shared__ float cw[];                                // [8][ctas] weights
  __shared__ float4 sums[8][32];
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, part = warp % W;
  const int r = kRows * blockIdx.y + warp / W;
  const int first = part * kSub + lane / (D / 4), d = 4 * (lane % (D / 4));
  const int c0 = blockIdx.x;
  const int4 join = __ldcg(a.joins + c0);
  if (join.x < 0) return;
  const int kvh = join.y / a.rg, x = (join.y % a.rg) * R + r;
  const bool on = x < a.n_q * a.group;  // (rows past the last: nothing to add)
  const int nr = on ? join.z - c0 + 1 : 0;
  const float *rec0 = a.part + static_cast<size_t>(c0) * kStride + r * kRec;
  auto rec_of = [&](int k) { return rec0 + (k == 0 ? R * kRec : static_cast<size_t>(k) * kStride); };
  float4 y[kBatch];
  auto fetch = [&](int k0) {
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int k = k0 + j * kEach + first;
      y[j] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (k < nr) y[j] = __ldcg(reinterpret_cast<const float4 *>(rec_of(k) + kPartHeader + d));
    }
  };
  fetch(0);
  float *w = cw + warp * gridDim.x;
  float M = neg_inf(), L = 0.f;
  for (int k = lane; k < nr; k += 32) {
    const float2 h = __ldcg(reinterpret_cast<const float2 *>(rec_of(k)));
    // one pass: the sum is kept relative to the largest so far
    const float mn = fmaxf(M, h.x), mm = mn == neg_inf() ? 0.f : mn;
    L = fmaf(L, exp2_approx(M - mm), exp2_approx(h.x - mm) * h.y);
    M = mn;
    w[k] = h.x;
  }
  const float mt = warp_max(M), mm = mt == neg_inf() ? 0.f : mt;
  L = warp_sum(L * exp2_approx(M - mm));
  for (int k = lane; k < nr; k += 32) w[k] = exp2_approx(w[k] - mm);
  __syncwarp();
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k0 = 0; k0 < nr; k0 += kBatch * kEach) {
    if (k0 > 0) fetch(k0);
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int k = k0 + j * kEach + first;
      const float c = k < nr ? w[k] : 0.f;
      v = make_float4(fmaf(c, y[j].x, v.x), fmaf(c, y[j].y, v.y), fmaf(c, y[j].z, v.z), fmaf(c, y[j].w, v.w));
    }
  }
  sums[warp][lane] = v;
  __syncthreads();
  if (on && part == 0 && lane < D / 4) {
#pragma unroll
    for (int k = 1; k < kEach; ++k) {
      const float4 u = sums[warp + k / kSub][lane + (k % kSub) * (D / 4)];
      v = make_float4(v.x + u.x, v.y + u.y, v.z + u.z, v.w + u.w);
    }
    paged_put<D>(a, paged_row(a, join.x, kvh, x), d, v, mt, L);
  }
}

// ------------------------------------------------------------------ unfolding
// Grid (splits, hq, B) as k_unfold: split s of row (b, h) takes its share of
// the selected chunks; the last split also takes the own chunk.  The rows of
// the share, in list order, form the 32-row tiles of the warps (a tile may
// span chunks and pages); one of the 8 query columns is in use.  The gists
// of selected chunks (exclude mode) are summed on the CUDA cores while the
// first copies are in flight, as a record of their own.  A CTA streams too
// little to hide its start and end: top-64 of 16 x 32K rows takes 15.8 us for
// 5.9 us of bytes, top-128 of 4 x 128K 26.7 for 9.6, 2 x 512K 17.3 for 5.3
// (neighbouring chunks in place of random ones: the same time).
struct PagedUnfoldArgs {
  UnfoldArgs u;  // raw_k, raw_v and the tensor maps unused
  PagedKV kv;
};

constexpr int kPuWarps = kUnfoldWarps;

// Zeroes the counters of rows whose splits are about to be joined.
__global__ void __launch_bounds__(256) k_paged_arm(uint32_t *counters, int rows) {
  pdl_wait();
  pdl_trigger();
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i < rows) counters[i] = 0u;
}

// rings (over them, once drained, the warps' results) | queries | items (the last one for the own chunk)
struct PagedItem {
  uint32_t prow;  // pool row of the chunk's first row, kNoRow: page outside the pool
  uint32_t si;    // place of its scales
  int32_t id;     // chunk
  float z;        // logit of its gist (exclude mode)
};

template <int D, int FMT, bool QF32>
__host__ __device__ inline size_t paged_unfold_smem(int per) {
  return kPuWarps * PgCfg<D>::kRing + sizeof(PgQuery<D, FMT, QF32, 1>) +
         (static_cast<size_t>(per) + 1) * sizeof(PagedItem);
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

template <int D, int FMT, bool QF32>
__global__ void __launch_bounds__(kUnfoldThreads, PgCfg<D>::kCtas)
    k_paged_unfold(const __grid_constant__ PagedUnfoldArgs pa) {
  using Warp = PgWarp<D, FMT, QF32, 1>;
  using Query = typename Warp::Query;
  const UnfoldArgs &a = pa.u;
  const PagedKV &kv = pa.kv;
  extern __shared__ __align__(128) uint8_t smem[];
  const int per = (a.k + a.n_split - 1) / a.n_split;
  Query &qs = *reinterpret_cast<Query *>(smem + kPuWarps * PgCfg<D>::kRing);
  PagedItem *items = reinterpret_cast<PagedItem *>(smem + kPuWarps * PgCfg<D>::kRing + sizeof(Query));
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
  // the list's first entries, asked for together with the counts (one latency)
  const int i0 = min(a.k, split * per), i1 = min(a.k, i0 + per);
  int m0 = -1;
  float z0 = 0.f;
  if (warp == 0 && i0 + lane < i1) {
    m0 = __ldcg(a.sel_idx + row * a.k + i0 + lane);
    if (a.exclude) z0 = __ldcg(a.sel_score + row * a.k + i0 + lane);
  }
  const int N = min(min(max(__ldcg(a.n_gists + b), 0), a.n_max), a.t_max / a.chunk);
  int own = min(max(__ldcg(a.own_len + b), 0), a.chunk);
  if (static_cast<int64_t>(N) * a.chunk + own > a.t_max) own = max(0, a.t_max - N * a.chunk);
  if (split != a.n_split - 1) own = 0;

  // Selected chunks of this split, in list order (invalid entries dropped), then the own chunk, each with its place
  // in the pool (a chunk lies in one page).
  const int32_t *table = kv.table + static_cast<size_t>(b) * kv.max_pages;
  auto item = [&](int slot, int m, float z) {
    const int r = m * a.chunk, p = kv.page.div(r), off = r - p * static_cast<int>(kv.page.d);
    const int pid = __ldcg(table + p);
    PagedItem it = {Warp::kNoRow, 0u, m, z};
    if (static_cast<uint32_t>(pid) < static_cast<uint32_t>(kv.n_pages)) {
      const uint32_t ph = static_cast<uint32_t>(pid) * kv.hkv + kvh;
      it.prow = ph * kv.page.d + off;
      it.si = ph * kv.blocks + kv.chunk.div(off);
    } else {
      flag_error(a.status, GSA_DEVERR_BAD_INDEX);
    }
    items[slot] = it;
  };
  if (warp == 0) {
    int cnt = 0;
    for (int base = i0; base < i1; base += 32) {
      const int i = base + lane;
      int m = m0;
      float z = z0;
      if (base > i0 && i < i1) {
        m = __ldcg(a.sel_idx + row * a.k + i);
        if (a.exclude) z = __ldcg(a.sel_score + row * a.k + i);
      }
      if (i >= i1) m = -1;
      if (m >= N) {
        flag_error(a.status, GSA_DEVERR_BAD_INDEX);
        m = -1;
      }
      const unsigned ball = __ballot_sync(0xffffffffu, m >= 0);
      if (m >= 0) item(cnt + __popc(ball & ((1u << lane) - 1u)), m, z * kLog2e);
      cnt += __popc(ball);
    }
    if (lane == 0) n_items_s = cnt;
  } else if (warp == 1) {
    qs.load(
        0,
        [&](int r) -> const void * {
          return r == 0 ? static_cast<const uint8_t *>(a.q) + row * D * (QF32 ? 4 : 2) : nullptr;
        },
        a.scale_log2);
  } else if (warp == 2 && lane == 0 && own > 0) {
    item(per, N, 0.f);  // the own chunk has the last place
  }
  Warp w;
  w.ring = smem_u32(smem) + warp * PgCfg<D>::kRing;
  __syncthreads();
  const int n_sel = n_items_s, sel_rows = n_sel * a.chunk, n_keys = sel_rows + own;
  const int n_tiles = (n_keys + 31) >> 5;
  const int mine = n_tiles > warp ? (n_tiles - warp + kPuWarps - 1) / kPuWarps : 0;
  auto key = [&](int i) {
    const int j = (warp + kPuWarps * i) * 32 + lane;
    w.sck = 0.f;
    w.scv = -0.f;
    if (j >= n_keys) return Warp::kNoRow;
    const int x = kv.chunk.div(j);
    const uint2 it = *reinterpret_cast<const uint2 *>(&items[x < n_sel ? x : per]);  // prow, si
    if (it.x == Warp::kNoRow) return Warp::kNoRow;
    w.sck = __ldcg(kv.ks + it.y);
    w.scv = __ldcg(kv.vs + it.y);
    return it.x + (j - x * a.chunk);
  };
  // gists of the selected chunks, relative to their own largest logit: kLpr lanes a row (16 bytes each), kRows rows a
  // warp at once, 8 such loads in flight a lane (one row behind the other took 5 us of 16 at 64 gists)
  using T = typename std::conditional<QF32, float, __nv_bfloat16>::type;
  constexpr int E = Vec16<T>::kElems, kLpr = D / E, kRows = 32 / kLpr;
  float gm = neg_inf(), gl = 0.f, ga[E];
#pragma unroll
  for (int e = 0; e < E; ++e) ga[e] = 0.f;
  auto gists = [&] {
    if (!a.exclude) return;
    for (int i = lane; i < n_sel; i += 32) gm = fmaxf(gm, items[i].z);
    gm = warp_max(gm);
    const float ref = gm == neg_inf() ? 0.f : gm;
    const T *gv = static_cast<const T *>(a.gist_v) + (static_cast<size_t>(b) * a.hkv + kvh) * a.n_max * D +
                  E * (lane % kLpr);
    for (int i0 = warp * kRows + lane / kLpr; i0 < n_sel; i0 += 8 * kPuWarps * kRows) {
      uint4 v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int i = i0 + j * kPuWarps * kRows;
        v[j] = make_uint4(0, 0, 0, 0);
        if (i < n_sel) v[j] = __ldcg(reinterpret_cast<const uint4 *>(gv + static_cast<size_t>(items[i].id) * D));
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int i = i0 + j * kPuWarps * kRows;
        if (i < n_sel) {
          const float p = exp2_approx(items[i].z - ref);
          float x[E];
          Vec16<T>::unpack(v[j], x);
          gl += p;
#pragma unroll
          for (int e = 0; e < E; ++e) ga[e] = fmaf(p, x[e], ga[e]);
        }
      }
    }
  };
  w.run_known(kv, mine, qs, key, gists);
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
  for (int o = kLpr; o < 32; o <<= 1) {
    gl += __shfl_xor_sync(0xffffffffu, gl, o);
#pragma unroll
    for (int e = 0; e < E; ++e) ga[e] += __shfl_xor_sync(0xffffffffu, ga[e], o);
  }
  if (lane < kLpr) {
#pragma unroll
    for (int e = 0; e < E; ++e) red[kPuWarps + warp][2 + E * lane + e] = ga[e];
    if (lane == 0) {
      red[kPuWarps + warp][0] = gm;
      red[kPuWarps + warp][1] = gl;
    }
  }
  paged_unfold_finish<D>(a, row, split, red, is_last_s);
  if (a.ready.w) unfold_ready_done(a);
}

}  // namespace gsa
