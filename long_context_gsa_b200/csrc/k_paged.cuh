// k_paged.cuh -- attention over raw rows held in 8 bits in a paged cache.
//
// Cache: pages of `page` rows in a pool, codes [n_pages, hkv, page, D] for
// keys and for values, one fp32 scale per block of `chunk` rows and kv head
// ([n_pages, hkv, page / chunk]); row r of sequence b lies in page
// table[b][r / page].  A row's value is scale * code.
//
// The product kernel of both readers (k_paged_attend: all rows of a
// sequence; k_paged_unfold: selected chunks and the own chunk of one query
// head) is one warp working through tiles of 16 rows:
//   z  = K q       S^T[16 keys x 8 queries], mma.sync m16n8k16 with the KEYS
//                  as the A operand: a kv head's 4..8 query heads fill the 8
//                  columns, where queries as A would leave 8..12 of 16 rows
//                  idle;
//   p  = 2^(z - m) lazy online softmax in fp32 (m raised when exceeded by
//                  kPgSlack), the scale of K applied to z;
//   O^T += V^T p   m16n8k16 with V^T as A (the tile's codes, transposed by
//                  byte permutes in registers) and p as B (movmatrix turns the
//                  accumulator layout of S^T into it).
// 8-bit codes are exact in fp16 (int8: |c| <= 127, e4m3: 4 significant bits
// within fp16's range), so K enters exactly.  Queries enter as fp16 after a
// power-of-two scaling of each row to [2^14, 2^15): exact for bf16 within 2^-38
// of the row's maximum; fp32 queries enter as two fp16 terms (22 bits).  p
// enters as one fp16 term when the output is bf16 (2^-12 relative, against
// the 2^-9 of the output's own rounding) and as two (2^-22) when it is
// fp32; the scale of V goes into p relative to the tile's largest scale,
// which is applied to the tile's product in fp32.  Statistics, sums and the
// running output are fp32.
//
// What bounds it: HBM reads of the codes.  Every warp copies its tiles with
// 16-byte cp.async into its own ring, so there is no CTA-wide barrier in
// the loop and 2 tiles of 4 KB (d = 128) or 4 of 2 KB (d = 64) are in flight
// for each of 16 warps on an SM; page-table entries are fetched one tile
// ahead of the copies, scales one tile behind them.
#pragma once

#include "common.cuh"
#include "k_unfold.cuh"  // UnfoldArgs, ready list, combine of partial records

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
constexpr float kPgPScale = 2048.f;  // p is scaled by 2^11 into fp16's range (<= 2^15)

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void mma_16816_f16(float c[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 8x8 fp16 block transposed across the warp's accumulator layout.
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
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
// reads back what it copied), V as 16 rows with swizzled 16-byte pieces, the
// 32 scales of the tile (K then V) and the mask of live keys.
template <int D>
struct PgCfg {
  static constexpr int kStages = D == 64 ? 5 : 3;
  static constexpr uint32_t kK = 16 * D, kV = 16 * D;
  static constexpr uint32_t kStage = kK + kV + 32 * 4 + 16;
  static constexpr uint32_t kRing = kStages * kStage;
};

// Offset of 16-byte piece p of row r inside a stage's V: lanes (g, t) read
// rows 2t (+1, +8, +9) at dims g*D/8.., and the permutations below spread the
// 8 lanes of a shared-memory phase over all 32 banks.
template <int D>
__device__ __forceinline__ uint32_t v_off(uint32_t r, uint32_t p) {
  if (D == 128) return r * 128 + ((p ^ (((r >> 1) & 3) << 1)) << 4);
  return (r ^ ((r >> 2) & 1)) * 64 + ((p ^ (((r >> 1) & 1) << 1)) << 4);
}

// The state of one warp over a run of tiles; NT groups of 8 query columns.
template <int D, int FMT, bool QF32, bool HILO, int NT>
struct PgWarp {
  using Cfg = PgCfg<D>;
  static constexpr int S = Cfg::kStages;
  static constexpr int KS = D / 16;          // k-steps of S^T, m-tiles of O^T
  static constexpr int QT = QF32 ? 2 : 1;    // fp16 terms of a query element

  uint32_t qf[QT][NT][KS][2];  // B fragments of the queries
  float f[NT][2];              // z factor of this lane's columns 2t, 2t + 1
  float m[NT][2], l[NT][2];
  float o[NT][KS][4];          // O^T: dims g*D/8 + 2j (+1), columns 2t, 2t + 1
  // the copy pipeline
  int32_t pid;                 // page of this lane's key in the next tile to copy (-1: none)
  uint32_t off;                // its row in that page
  float sc;                    // scale of the tile copied last (K: lanes 0..15, V: lanes 16..31)
  uint32_t ring;

  // Query column n (0 .. 8 NT - 1) is row(n), null when unused.
  template <typename RowFn>
  __device__ __forceinline__ void load_q(RowFn row, float scale_log2) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const void *p = row(8 * nt + g);
      float x[D / 4];
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
      // exponent shift that brings the row's maximum into [2^14, 2^15); none for zero, inf or NaN rows
      int sh = 0;
      if (a != 0 && a < 0x7f800000u) sh = min(14 - (static_cast<int>(a >> 23) - 127), 120);
      const float up = __uint_as_float(static_cast<uint32_t>(127 + sh) << 23);
      const float down = __uint_as_float(static_cast<uint32_t>(127 - sh) << 23) * scale_log2;
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float x0 = x[4 * s + 2 * h] * up, x1 = x[4 * s + 2 * h + 1] * up;
          qf[0][nt][s][h] = pack_h2(x0, x1);
          if (QF32) {
            const float2 r = unpack_h2(qf[0][nt][s][h]);
            qf[QT - 1][nt][s][h] = pack_h2(x0 - r.x, x1 - r.y);
          }
        }
      f[nt][0] = __shfl_sync(0xffffffffu, down, 8 * t);
      f[nt][1] = __shfl_sync(0xffffffffu, down, 8 * t + 4);
      m[nt][0] = m[nt][1] = neg_inf();
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int j = 0; j < KS; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][j][e] = 0.f;
    }
  }

  // Fetch the page of raw row r (< 0: no such key); lanes 16..31 hold the
  // same keys as lanes 0..15.
  __device__ __forceinline__ void fetch(const PagedKV &kv, const int32_t *table, int64_t r) {
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
    if (wanted && !live && lane < 16) flag_error(status, GSA_DEVERR_BAD_INDEX);
    const uint32_t ph = live ? static_cast<uint32_t>(pid) * kv.hkv + kvh : 0u;
    const uint32_t prow = live ? ph * kv.page.d + off : 0xffffffffu;
    sc = 0.f;
    if (live) sc = __ldcg((lane < 16 ? kv.ks : kv.vs) + (static_cast<size_t>(ph) * kv.blocks + kv.chunk.div(off)));
    const uint32_t base = ring + st * Cfg::kStage;
    const uint32_t mask = __ballot_sync(0xffffffffu, live) & 0xffffu;
    if (lane == 0) asm volatile("st.shared.u32 [%0], %1;" ::"r"(base + 32 * D + 128), "r"(mask) : "memory");
#pragma unroll
    for (int i = 0; i < 2; ++i) {  // keys g and g + 8
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
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(ring + st * Cfg::kStage + 32 * D + (threadIdx.x & 31) * 4), "f"(sc)
                 : "memory");
  }

  // Work through tile i in stage st; key0: index of its first key, lim:
  // columns 2t, 2t+1 see keys below lim (CAUSAL).
  template <bool CAUSAL>
  __device__ __forceinline__ void step(int st, int64_t key0, const int64_t (*lim)[2]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint32_t base = ring + st * Cfg::kStage, scb = base + 32 * D;
    float kg[2], vg[2];
    uint32_t mask;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(kg[0]) : "r"(scb + 4 * g));
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(kg[1]) : "r"(scb + 4 * g + 32));
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(vg[0]) : "r"(scb + 4 * g + 64));
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(vg[1]) : "r"(scb + 4 * g + 96));
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(mask) : "r"(scb + 128));
    float z[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) z[nt][e] = 0.f;
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
      uint32_t a[4], b[4];
      asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                   : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3])
                   : "r"(base + (c * 32 + lane) * 16));
      asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                   : "=r"(b[0]), "=r"(b[1]), "=r"(b[2]), "=r"(b[3])
                   : "r"(base + ((D / 64 + c) * 32 + lane) * 16));
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        uint32_t a0, a1, a2, a3;
        codes_to_h2<FMT>(a[w], a0, a2);
        codes_to_h2<FMT>(b[w], a1, a3);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int q = 0; q < QT; ++q)
            mma_16816_f16(z[nt], a0, a1, a2, a3, qf[q][nt][c * 4 + w][0], qf[q][nt][c * 4 + w][1]);
      }
    }
    const bool live0 = (mask >> g) & 1u, live1 = (mask >> (g + 8)) & 1u;
    bool over = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        bool see = e < 2 ? live0 : live1;
        if (CAUSAL) see = see && key0 + g + (e < 2 ? 0 : 8) < lim[nt][e & 1];
        z[nt][e] = see ? z[nt][e] * (kg[e >> 1] * f[nt][e & 1]) : neg_inf();
        over = over || z[nt][e] > m[nt][e & 1] + kPgSlack;
      }
    if (__any_sync(0xffffffffu, over)) {  // raise the references, rescale
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float mx = fmaxf(z[nt][x], z[nt][x + 2]);
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
          if (mx > m[nt][x]) {
            const float c = exp2_approx(m[nt][x] - mx);  // 0 when there was no reference
            l[nt][x] *= c;
#pragma unroll
            for (int j = 0; j < KS; ++j) {
              o[nt][j][x] *= c;
              o[nt][j][x + 2] *= c;
            }
            m[nt][x] = mx;
          }
        }
    }
    // the scale of V relative to the tile's largest (scales are >= 0, so their bits order like the values; fmaxf
    // drops a NaN scale here, which then reaches only the columns that see its keys)
    const float vmax =
        __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(fmaxf(vg[0], vg[1]), 0.f))));
    const float inv = vmax != 0.f ? __fdividef(kPgPScale, vmax) : 0.f;
    const float w0 = vg[0] * inv, w1 = vg[1] * inv;
    uint32_t pb[HILO ? 2 : 1][NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float p[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float mm = m[nt][e & 1];
        p[e] = exp2_approx(z[nt][e] - (mm == neg_inf() ? 0.f : mm));
      }
      l[nt][0] += p[0] + p[2];
      l[nt][1] += p[1] + p[3];
#pragma unroll
      for (int e = 0; e < 4; ++e) p[e] = z[nt][e] == neg_inf() ? 0.f : p[e] * (e < 2 ? w0 : w1);
      const uint32_t h0 = pack_h2(p[0], p[1]), h1 = pack_h2(p[2], p[3]);
      pb[0][nt][0] = movmatrix_trans(h0);
      pb[0][nt][1] = movmatrix_trans(h1);
      if (HILO) {
        const float2 r0 = unpack_h2(h0), r1 = unpack_h2(h1);
        pb[HILO ? 1 : 0][nt][0] = movmatrix_trans(pack_h2(p[0] - r0.x, p[1] - r0.y));
        pb[HILO ? 1 : 0][nt][1] = movmatrix_trans(pack_h2(p[2] - r1.x, p[3] - r1.y));
      }
    }
    const float back = vmax * (1.f / kPgPScale);
    constexpr int kW = D / 32;  // 32-bit words of a lane's D/8 codes of one row
    uint32_t vr[4][kW];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t r = 2 * t + (i & 1) + 8 * (i >> 1);
      if (D == 128)
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(vr[i][0]), "=r"(vr[i][1]), "=r"(vr[i][kW - 2]), "=r"(vr[i][kW - 1])
                     : "r"(base + Cfg::kK + v_off<D>(r, g)));
      else
        asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];"
                     : "=r"(vr[i][0]), "=r"(vr[i][1])
                     : "r"(base + Cfg::kK + v_off<D>(r, g >> 1) + (g & 1) * 8));
    }
#pragma unroll
    for (int w = 0; w < kW; ++w) {
      // (row 2t, row 2t+1) pairs of each dim, then rows 2t+8, 2t+9
      uint32_t a[2][2], c[2][2];
      codes_to_h2<FMT>(__byte_perm(vr[0][w], vr[1][w], 0x5140), a[0][0], a[0][1]);
      codes_to_h2<FMT>(__byte_perm(vr[0][w], vr[1][w], 0x7362), a[1][0], a[1][1]);
      codes_to_h2<FMT>(__byte_perm(vr[2][w], vr[3][w], 0x5140), c[0][0], c[0][1]);
      codes_to_h2<FMT>(__byte_perm(vr[2][w], vr[3][w], 0x7362), c[1][0], c[1][1]);
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float d[4] = {0.f, 0.f, 0.f, 0.f};
          mma_16816_f16(d, a[x][0], a[x][1], c[x][0], c[x][1], pb[0][nt][0], pb[0][nt][1]);
          if (HILO)
            mma_16816_f16(d, a[x][0], a[x][1], c[x][0], c[x][1], pb[HILO ? 1 : 0][nt][0], pb[HILO ? 1 : 0][nt][1]);
#pragma unroll
          for (int e = 0; e < 4; ++e) o[nt][2 * w + x][e] = fmaf(back, d[e], o[nt][2 * w + x][e]);
        }
    }
  }

  // Run n tiles; raw(i) is this lane's key (lane & 15) of tile i as a raw row
  // (< 0: none), key0(i) the index of the tile's first key; before() runs once
  // while the first copies are in flight.
  template <bool CAUSAL, typename RawFn, typename Key0Fn, typename BeforeFn>
  __device__ __forceinline__ void run(const PagedKV &kv, const int32_t *table, int kvh, int n, RawFn raw, Key0Fn key0,
                                      const int64_t (*lim)[2], uint32_t *status, BeforeFn before) {
    int64_t r = n > 0 ? raw(0) : -1;
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
      step<CAUSAL>(st, key0(i), lim);
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
// steps of 16 rows a warp, form one line that the CTAs cut into equal parts
// (the lengths are on the device, so the cut is too): ragged batches and
// single long sequences load every SM alike.  A segment inside one CTA is
// written directly; one that several CTAs share is joined by the last of them
// to arrive (an atomic counter, no waiting) from partial records, in CTA
// order, so the result does not depend on who was last.
constexpr int kPgWarps = 8;
constexpr int kPgThreads = 32 * kPgWarps;
constexpr int kPgStep = 16 * kPgWarps;  // rows of one CTA step
constexpr int kPgMaxCtas = 1024;        // bound of the grid (partial slots in the workspace)
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

template <int D, int NT>
__host__ __device__ constexpr uint32_t paged_attend_smem() {
  return kPgWarps * (PgCfg<D>::kRing > 8 * NT * (D + 4) * 4 ? PgCfg<D>::kRing : 8 * NT * (D + 4) * 4);
}

template <int D, int FMT, bool QF32, bool HILO, int NT>
__global__ void __launch_bounds__(kPgThreads, NT == 1 && !QF32 ? 2 : 1) k_paged_attend(const PagedAttendArgs a) {
  using Warp = PgWarp<D, FMT, QF32, HILO, NT>;
  constexpr int R = 8 * NT, kRec = D + kPartHeader;
  extern __shared__ __align__(128) uint8_t smem[];
  uint32_t *pre = reinterpret_cast<uint32_t *>(smem + paged_attend_smem<D, NT>());
  float(*red)[R][kRec] = reinterpret_cast<float(*)[R][kRec]>(smem);  // over the rings, once they are drained
  __shared__ float wgt[R][kPgWarps], rowM[R], rowL[R];
  __shared__ int last_s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int per_b = a.kv.hkv * a.rg;
  pdl_wait();
  paged_prefix<kPgThreads>(pre, a.B, [&](int b) {
    const int len = paged_len(a.n_gists, a.own_len, b, a.n_max, a.chunk, a.t_max);
    return static_cast<uint32_t>(per_b) * static_cast<uint32_t>((len + kPgStep - 1) / kPgStep);
  });
  const uint32_t total = pre[a.B];
  const uint32_t ctas = min(gridDim.x, max(1u, (total + a.min_steps - 1) / a.min_steps));
  const uint32_t cta = blockIdx.x;
  // sequences without rows: zeros, ln of an empty sum
  for (int b = cta; b < a.B; b += gridDim.x)
    if (pre[b] == pre[b + 1]) {
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
    const int len = paged_len(a.n_gists, a.own_len, b, a.n_max, a.chunk, a.t_max);
    const int rows = min(R, a.n_q * a.group - rg * R);
    // query row r of the segment -> its row in q and out
    auto out_row = [&](int r) {
      const int x = rg * R + r;
      return (static_cast<size_t>(b) * a.n_q + x / a.group) * a.hq + kvh * a.group + x % a.group;
    };
    w.load_q(
        [&](int r) -> const void * {
          return r < rows ? static_cast<const uint8_t *>(a.q) + out_row(r) * D * (QF32 ? 4 : 2) : nullptr;
        },
        a.scale_log2);
    int64_t lim[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int x = 0; x < 2; ++x)
        lim[nt][x] = static_cast<int64_t>(len) - (a.n_q - 1) + (rg * R + 8 * nt + 2 * t + x) / a.group;
    const int n = static_cast<int>(s1 - s0);
    const int64_t first = (static_cast<int64_t>(s0) * kPgWarps + warp) * 16;
    int mine = 0;  // tiles of this warp that hold a row
    if (first < len) mine = min(n, static_cast<int>((len - first + kPgStep - 1) / kPgStep));
    const int32_t *table = a.kv.table + static_cast<size_t>(b) * a.kv.max_pages;
    auto key0 = [&](int i) { return first + static_cast<int64_t>(i) * kPgStep; };
    auto raw = [&](int i) {
      const int64_t k = key0(i) + (lane & 15);
      return k < len ? k : static_cast<int64_t>(-1);
    };
    if (a.n_q > 1)
      w.template run<true>(a.kv, table, kvh, mine, raw, key0, lim, a.status, [] {});
    else
      w.template run<false>(a.kv, table, kvh, mine, raw, key0, lim, a.status, [] {});
    __syncthreads();  // every ring is drained: red may overwrite them
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float *dst = red[warp][8 * nt + 2 * t + x];
#pragma unroll
        for (int j = 0; j < Warp::KS; ++j)
          *reinterpret_cast<float2 *>(dst + kPartHeader + g * (D / 8) + 2 * j) =
              make_float2(w.o[nt][j][x], w.o[nt][j][x + 2]);
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
        L += c * red[i][tid][1];
      }
      rowM[tid] = M;
      rowL[tid] = L;
    }
    __syncthreads();
    const uint32_t c0 = static_cast<uint32_t>(((static_cast<uint64_t>(seg0) + 1) * ctas - 1) / total);
    const uint32_t c1 = static_cast<uint32_t>((static_cast<uint64_t>(seg1) * ctas - 1) / total);
    const bool whole = c0 == c1;
    // this CTA's record: slot 1 if the segment starts in its part, else slot 0
    float *rec = a.part + (static_cast<size_t>(cta) * 2 + (cta == c0 ? 1 : 0)) * R * kRec;
    for (int i = tid; i < rows * (D / 2); i += kPgThreads) {
      const int r = i / (D / 2), d = 2 * (i % (D / 2));
      float x = 0.f, y = 0.f;
#pragma unroll
      for (int k = 0; k < kPgWarps; ++k) {
        const float2 v = *reinterpret_cast<const float2 *>(&red[k][r][kPartHeader + d]);
        x = fmaf(wgt[r][k], v.x, x);
        y = fmaf(wgt[r][k], v.y, y);
      }
      if (whole) {
        const float L = rowL[r];
        const size_t o = out_row(r) * D + d;
        store_out(a.out, o, L != 0.f ? x / L : 0.f, a.out_bf16);
        store_out(a.out, o + 1, L != 0.f ? y / L : 0.f, a.out_bf16);
        if (d == 0 && a.lse) a.lse[out_row(r)] = L != 0.f ? (rowM[r] + __log2f(L)) * kLn2 : neg_inf();
      } else {
        *reinterpret_cast<float2 *>(rec + static_cast<size_t>(r) * kRec + kPartHeader + d) = make_float2(x, y);
        if (d == 0) {
          rec[static_cast<size_t>(r) * kRec] = rowM[r];
          rec[static_cast<size_t>(r) * kRec + 1] = rowL[r];
        }
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
        // records of CTAs c0 .. c1 (c0's in slot 1), in that order
        auto rec_of = [&](uint32_t c, int r) {
          return a.part + ((static_cast<size_t>(c) * 2 + (c == c0 ? 1 : 0)) * R + r) * kRec;
        };
        for (int i = tid; i < rows * (D / 2); i += kPgThreads) {
          const int r = i / (D / 2), d = 2 * (i % (D / 2));
          float M = neg_inf(), L = 0.f, x = 0.f, y = 0.f;
          for (uint32_t c = c0; c <= c1; ++c) M = fmaxf(M, __ldcg(rec_of(c, r)));
          const float mm = M == neg_inf() ? 0.f : M;
#pragma unroll 4
          for (uint32_t c = c0; c <= c1; ++c) {
            const float *q = rec_of(c, r);
            const float2 h = __ldcg(reinterpret_cast<const float2 *>(q));
            const float2 v = __ldcg(reinterpret_cast<const float2 *>(q + kPartHeader + d));
            const float k = exp2_approx(h.x - mm);
            L = fmaf(k, h.y, L);
            x = fmaf(k, v.x, x);
            y = fmaf(k, v.y, y);
          }
          const size_t o = out_row(r) * D + d;
          store_out(a.out, o, L != 0.f ? x / L : 0.f, a.out_bf16);
          store_out(a.out, o + 1, L != 0.f ? y / L : 0.f, a.out_bf16);
          if (d == 0 && a.lse) a.lse[out_row(r)] = L != 0.f ? (M + __log2f(L)) * kLn2 : neg_inf();
        }
      }
    }
    __syncthreads();  // red and the row sums are read: the rings may be used again
  }
  pdl_trigger();
}

// ------------------------------------------------------------------ unfolding
// Grid (splits, hq, B) as k_unfold: split s of row (b, h) takes its share of
// the selected chunks; the last split also takes the own chunk.  The rows of
// the share, in list order, form the 16-row tiles of the warps (a tile may
// span chunks and pages); one of the 8 query columns is in use.  The gists
// of selected chunks (exclude mode) are summed on the CUDA cores while the
// first copies are in flight, as a record of their own.
struct PagedUnfoldArgs {
  UnfoldArgs u;  // raw_k, raw_v and the tensor maps unused
  PagedKV kv;
};

constexpr int kPuWarps = kUnfoldWarps;

template <int D>
__host__ __device__ inline size_t paged_unfold_smem(int per) {
  return kPuWarps * PgCfg<D>::kRing + static_cast<size_t>(per) * 8;  // rings | chunk ids | gist logits
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
__global__ void __launch_bounds__(kUnfoldThreads, 4) k_paged_unfold(const __grid_constant__ PagedUnfoldArgs pa) {
  using Warp = PgWarp<D, FMT, QF32, HILO, 1>;
  const UnfoldArgs &a = pa.u;
  const PagedKV &kv = pa.kv;
  extern __shared__ __align__(128) uint8_t smem[];
  const int per = (a.k + a.n_split - 1) / a.n_split;
  int *items = reinterpret_cast<int *>(smem + kPuWarps * PgCfg<D>::kRing);
  float *item_z = reinterpret_cast<float *>(items + per);
  __shared__ int n_items_s, is_last_s, take_s[2];
  __shared__ float red[2 * kPuWarps][2 + D];
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
  w.load_q(
      [&](int r) -> const void * {
        return r == 0 ? static_cast<const uint8_t *>(a.q) + row * D * (QF32 ? 4 : 2) : nullptr;
      },
      a.scale_log2);
  __syncthreads();
  const int n_sel = n_items_s, sel_rows = n_sel * a.chunk, n_keys = sel_rows + own;
  const int n_tiles = (n_keys + 15) >> 4;
  const int mine = n_tiles > warp ? (n_tiles - warp + kPuWarps - 1) / kPuWarps : 0;
  auto key0 = [&](int i) { return static_cast<int64_t>((warp + kPuWarps * i) * 16); };
  auto raw = [&](int i) -> int64_t {
    const int j = static_cast<int>(key0(i)) + (lane & 15);
    if (j < sel_rows) {
      const int it = kv.chunk.div(j);
      return static_cast<int64_t>(items[it]) * a.chunk + (j - it * a.chunk);
    }
    return j < n_keys ? static_cast<int64_t>(N) * a.chunk + (j - sel_rows) : static_cast<int64_t>(-1);
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
  w.template run<false>(kv, kv.table + static_cast<size_t>(b) * kv.max_pages, kvh, mine, raw, key0, nullptr, a.status,
                        gists);
  pdl_trigger();
  if (t == 0) {  // column 0
#pragma unroll
    for (int j = 0; j < Warp::KS; ++j) {
      red[warp][2 + g * (D / 8) + 2 * j] = w.o[0][j][0];
      red[warp][2 + g * (D / 8) + 2 * j + 1] = w.o[0][j][2];
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
