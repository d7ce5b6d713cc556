// k_append.cuh -- new keys and values join a paged raw-token cache, with the
// position rotation applied on the way and 8-bit blocks quantised.
//
// A pair (x, y) of a head's rotated dims at position p and frequency w turns
// by the angle p w: (x cos - y sin, y cos + x sin).  The angle is reduced in
// 64 bits (p w / 2 pi loses whole turns in fp32 once p w passes about 10^5),
// the sine and cosine and the products are fp32.
//
// 8-bit caches: a block of `chunk` rows of one kv head has one fp32 scale s,
// codes round(x / s).  int8: s = max|x| / 127.  e4m3: s is the least power
// of two with max|x| / s <= 448, so x / s is exact, and moving codes to a
// larger scale loses only what falls into e4m3's subnormals.  A block whose
// max|x| is below 2^-100 has scale 0 and codes 0; one that receives an inf or
// NaN has scale NaN.  Rows that join a part-filled block can only raise its
// scale; the rows already held are then re-expressed (rounded once more).
//
// What bounds it: HBM (each new row read and written once) for long inputs,
// launch and three dependent loads for single tokens.  A CTA takes one block
// of one sequence for all heads (or a share of the heads when there are few
// blocks), so the sines of a row are computed once and every block of codes
// has one writer; a warp takes one (block, head) of keys or values, or one
// row's queries of a few heads, at a time.  A lane works on a unit of 16 dims,
// the 8 pairs that turn together, so nothing is loaded twice.  A block's first
// kHold passes of rows (8 rows of 64 dims or 4 of 128) stay in registers between
// its maximum and its codes, larger blocks are loaded and turned again (their
// second read from L2).  32768 tokens, 32 / 8 heads of 64 dims, e4m3 (369 MB):
// 127 us with 8 dims a lane, each lane loading its partner's too and an index
// division a row; 87 us so (4.2 TB/s).  CTAs of 128 threads, 5 on an SM: 256
// threads took 87..94 us, 64 threads as long; more queries in flight a lane
// spill.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"
#include "k_paged.cuh"

namespace gsa {

enum { kFmtPlain = 2 };

struct AppendArgs {
  const void *q, *k, *v;       // [n_tok, heads, D], rows q_stride / k_stride / v_stride elements apart; q may be null
  const int32_t *cu;           // [B + 1] or null (n_tok / B tokens each)
  const int32_t *pos;          // [n_tok] or null (the raw row)
  const float *inv_freq;       // [rot / 2]
  const int32_t *table;        // [B, max_pages]
  const int32_t *n_gists;      // or null
  int32_t *own_len;            // read; advanced by the last CTA when `advance`
  void *kp, *vp;               // pages
  float *ks, *vs;              // scales (8-bit)
  void *q_out;                 // [n_tok, hq, D]
  int32_t q_stride, k_stride, v_stride;
  int32_t n_tok, B, hq, hkv, n_max, t_max, n_pages, max_pages, blocks;
  int32_t rot, advance;
  FastDiv page, chunk;
  uint32_t *counter, *status;
};

constexpr int kApThreads = 128;
constexpr int kApWarps = kApThreads / 32;

// First new raw row and number of new rows of sequence b, cut at t_max.
__device__ __forceinline__ int append_span(const AppendArgs &a, int b, int &start, int &tok0) {
  int64_t s = max(__ldcg(a.own_len + b), 0);
  if (a.n_gists) s += static_cast<int64_t>(min(max(__ldcg(a.n_gists + b), 0), a.n_max)) * a.chunk.d;
  int n;
  if (a.cu) {
    tok0 = min(max(__ldcg(a.cu + b), 0), a.n_tok);
    n = min(max(__ldcg(a.cu + b + 1), 0), a.n_tok) - tok0;
  } else {
    n = a.n_tok / a.B;
    tok0 = b * n;
  }
  n = max(n, 0);
  start = static_cast<int>(s < a.t_max ? s : a.t_max);
  if (start + static_cast<int64_t>(n) > a.t_max) {
    flag_error(a.status, GSA_DEVERR_CAPACITY);
    n = a.t_max - start;
  }
  return n;
}

// A unit of 16 dims of a row as it lies in memory: dims A .. A + 7 and B ..
// B + 7 (see unit_dims).
template <typename T>
struct Raw16 {
  static constexpr int kVecs = sizeof(T) / 2;  // 16-byte loads of 8 dims
  uint4 a[kVecs], b[kVecs];
  __device__ __forceinline__ void load(const T *row, int A, int B) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      a[i] = ldg_nc_v4(row + A + i * 4);
      b[i] = ldg_nc_v4(row + B + i * 4);
    }
  }
  __device__ __forceinline__ void values(float *x) const {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      Vec16<T>::unpack(a[i], x + i * 4);
      Vec16<T>::unpack(b[i], x + 8 + i * 4);
    }
  }
};

// Dims of unit i: pairs of halves: 8 i and rot / 2 + 8 i; interleaved pairs,
// and dims that are not turned: 16 i and 16 i + 8.
template <bool INTER>
__device__ __forceinline__ void unit_dims(int i, int rot, int &A, int &B) {
  const bool halves = !INTER && i < (rot >> 4);
  A = halves ? 8 * i : 16 * i;
  B = halves ? (rot >> 1) + 8 * i : 16 * i + 8;
}

// The unit's 8 (cos, sin).  Dims that are not turned pass through as they are
// (times (1, 0) an inf would make its partner a NaN, and a -0 lose its sign);
// they load the 8 that the table begins with (its rows of rot / 2 follow).
struct Turn8 {
  float4 c[4];
  bool on;
  __device__ __forceinline__ void load(const float2 *cs, int r, int i, int rot) {
    on = i < (rot >> 4);
    const float4 *p = reinterpret_cast<const float4 *>(on ? cs + 8 + r * (rot >> 1) + 8 * i : cs);
#pragma unroll
    for (int k = 0; k < 4; ++k) c[k] = p[k];
  }
  // x[0..7] dims A.., x[8..15] dims B..
  template <bool INTER>
  __device__ __forceinline__ void turn(float *x) const {
    if (INTER) {
#pragma unroll
      for (int k = 0; k < 8; ++k) pair(k, x[2 * k], x[2 * k + 1]);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) pair(k, x[k], x[8 + k]);
    }
  }
  __device__ __forceinline__ void pair(int k, float &u, float &v) const {
    const float cs = k & 1 ? c[k / 2].z : c[k / 2].x, sn = k & 1 ? c[k / 2].w : c[k / 2].y;
    const float p = fmaf(u, cs, -(v * sn)), q = fmaf(v, cs, u * sn);
    u = on ? p : u;
    v = on ? q : v;
  }
};

// The larger, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Eight values to T at p.
template <typename T>
__device__ __forceinline__ void store8(T *p, const float *x) {
  if (sizeof(T) == 2) {
    uint4 w;
    uint32_t *u = &w.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      u[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    *reinterpret_cast<uint4 *>(p) = w;
  } else {
    float4 *f = reinterpret_cast<float4 *>(p);
    f[0] = make_float4(x[0], x[1], x[2], x[3]);
    f[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
}

template <int FMT>
__device__ __forceinline__ float block_scale(uint32_t amax_bits) {
  if (amax_bits >= 0x7f800000u) return __uint_as_float(0x7fc00000u);  // an inf or NaN among the values
  if (amax_bits < static_cast<uint32_t>(127 - 100) << 23) return 0.f;  // below 2^-100
  if (FMT == kFmtI8) return __fdiv_rn(__uint_as_float(amax_bits), 127.f);
  // amax = f 2^e, 1 <= f < 2; 448 = 1.75 * 2^8
  const int e = static_cast<int>(amax_bits >> 23) - 8 + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return __uint_as_float(static_cast<uint32_t>(e) << 23);
}

// Eight codes of x inv.  DIV: of x / s, inv the rounded 1 / s.  int8: x inv
// alone is off by up to 3 half units in the last place, which takes a quotient
// next to a half step to the wrong side; one correction by the remainder gives
// the nearest fp32 one.  (e4m3's scales are powers of two.)
template <int FMT, bool DIV = false>
__device__ __forceinline__ uint2 encode8(const float *x, float inv, float s = 0.f) {
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float *y = x + 4 * h;
    if (FMT == kFmtI8) {
      uint32_t u = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float v = y[i] * inv;
        if (DIV) v = fmaf(fmaf(-v, s, y[i]), inv, v);
        const int c = min(max(__float2int_rn(v), -127), 127);
        u |= (static_cast<uint32_t>(c) & 0xffu) << (8 * i);
      }
      w[h] = u;
    } else {
      const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(y[0] * inv, y[1] * inv), __NV_SATFINITE, __NV_E4M3);
      const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(y[2] * inv, y[3] * inv), __NV_SATFINITE, __NV_E4M3);
      w[h] = lo | (hi << 16);
    }
  }
  return make_uint2(w[0], w[1]);
}

template <int FMT>
__device__ __forceinline__ void decode8(uint2 c, float *x) {
  const uint32_t w[2] = {c.x, c.y};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t lo, hi;
    codes_to_h2<FMT>(w[h], lo, hi);
    const float2 a = unpack_h2(lo), b = unpack_h2(hi);
    x[4 * h] = a.x;
    x[4 * h + 1] = a.y;
    x[4 * h + 2] = b.x;
    x[4 * h + 3] = b.y;
  }
}

// One (block, kv head) of keys (TURN) or values: n new rows from token row
// `src` on (stride elements apart) go to page row `dst`.., `held` rows of the
// block come before them.
template <int D, typename T, int FMT, bool INTER, bool TURN>
__device__ __forceinline__ void append_block(const T *src, int stride, int n, int held, void *pages, uint32_t dst,
                                             float *scale, int rot, const float2 *cs) {
  constexpr int L = D / 16, RPW = 32 / L;        // lanes of a row, rows of a pass
  constexpr int kHold = 1;                       // passes held in registers
  const int lane = threadIdx.x & 31, sub = lane / L, unit = lane % L;
  int A, B;
  unit_dims<INTER>(unit, rot, A, B);
  auto turned = [&](const Raw16<T> &raw, int r, float *x) {
    raw.values(x);
    if (TURN) {
      Turn8 t;
      t.load(cs, r, unit, rot);
      t.turn<INTER>(x);
    }
  };
  if (FMT == kFmtPlain) {
    T *out = static_cast<T *>(pages) + static_cast<size_t>(dst) * D;
#pragma unroll 2
    for (int r = sub; r < n; r += RPW) {
      Raw16<T> raw;
      raw.load(src + static_cast<int64_t>(r) * stride, A, B);
      float x[16];
      turned(raw, r, x);
      store8(out + r * D + A, x);
      store8(out + r * D + B, x + 8);
    }
    return;
  }
  constexpr int F = FMT == kFmtPlain ? kFmtI8 : FMT;  // (the plain case has returned)
  const float old = held > 0 ? __ldcg(scale) : 0.f;
  float x[kHold][16], top = 0.f;
  // rows r0 + sub + RPW i of this lane, turned
  auto fetch = [&](int r0) {
    Raw16<T> raw[kHold];
#pragma unroll
    for (int i = 0; i < kHold; ++i)
      if (r0 + i * RPW + sub < n) raw[i].load(src + static_cast<int64_t>(r0 + i * RPW + sub) * stride, A, B);
#pragma unroll
    for (int i = 0; i < kHold; ++i)
      if (r0 + i * RPW + sub < n) turned(raw[i], r0 + i * RPW + sub, x[i]);
  };
#pragma unroll 1
  for (int r0 = 0; r0 < n; r0 += kHold * RPW) {
    fetch(r0);
#pragma unroll
    for (int i = 0; i < kHold; ++i)
      if (r0 + i * RPW + sub < n) {
#pragma unroll
        for (int k = 0; k < 16; ++k) top = max_nan(top, fabsf(x[i][k]));
      }
  }
  const uint32_t amax = __reduce_max_sync(0xffffffffu, __float_as_uint(top));  // (a NaN has the largest bits)
  float s = block_scale<F>(amax);
  if (!(s > old) && s == s) s = old;  // the larger; NaN from either stays
  uint8_t *out = static_cast<uint8_t *>(pages) + static_cast<size_t>(dst) * D;
  if (s > old && held > 0) {  // the rows already there, at the new scale
    const float ratio = old / s;
    uint8_t *first = out - held * D;
    for (int r = sub; r < held; r += RPW) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint2 *p = reinterpret_cast<uint2 *>(first + r * D + (h ? B : A));
        float y[8];
        decode8<F>(__ldcg(p), y);
        *p = encode8<F>(y, ratio);
      }
    }
  }
  // 0 for a scale of 0 or NaN: codes 0; a power of two is turned over in its exponent
  float inv = 0.f;
  if (s > 0.f) inv = F == kFmtI8 ? __frcp_rn(s) : __uint_as_float((254u << 23) - __float_as_uint(s));
#pragma unroll 1
  for (int r0 = 0; r0 < n; r0 += kHold * RPW) {
    if (n > kHold * RPW) fetch(r0);  // not held: read again
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
      const int r = r0 + i * RPW + sub;
      if (r < n) {
        uint2 c = make_uint2(0, 0), d = make_uint2(0, 0);
        if (inv > 0.f) {
          c = encode8<F, true>(x[i], inv, s);
          d = encode8<F, true>(x[i] + 8, inv, s);
        }
        *reinterpret_cast<uint2 *>(out + r * D + A) = c;
        *reinterpret_cast<uint2 *>(out + r * D + B) = d;
      }
    }
  }
  __syncwarp();
  if (lane == 0) *scale = s;
}

// kQPass passes of RPW heads of one row's queries, from head h0 on.
constexpr int kQPass = 2;
template <int D, typename T, bool INTER>
__device__ __forceinline__ void append_queries(const T *q, T *out, int r, int h0, int hq, int rot, const float2 *cs) {
  constexpr int L = D / 16, RPW = 32 / L;
  const int lane = threadIdx.x & 31, h = h0 + lane / L, unit = lane % L;
  int A, B;
  unit_dims<INTER>(unit, rot, A, B);
  Raw16<T> raw[kQPass];
#pragma unroll
  for (int i = 0; i < kQPass; ++i)
    if (h + i * RPW < hq) raw[i].load(q + (h + i * RPW) * D, A, B);
  Turn8 t;
  t.load(cs, r, unit, rot);
#pragma unroll
  for (int i = 0; i < kQPass; ++i)
    if (h + i * RPW < hq) {
      float x[16];
      raw[i].values(x);
      t.turn<INTER>(x);
      store8(out + (h + i * RPW) * D + A, x);
      store8(out + (h + i * RPW) * D + B, x + 8);
    }
}

// Grid (x, y): CTA x takes blocks x, x + gridDim.x, .. of the line of all
// sequences' touched blocks; the y CTAs share a block's heads.
template <int D, typename T, int FMT, bool INTER>
__global__ void __launch_bounds__(kApThreads, 5) k_paged_append(const AppendArgs a) {
  extern __shared__ __align__(128) uint8_t smem[];
  float2 *cs = reinterpret_cast<float2 *>(smem);  // [8 + chunk * rot / 2]
  uint32_t *pre = reinterpret_cast<uint32_t *>(cs + 8 + a.chunk.d * (a.rot / 2));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int chunk = a.chunk.d, half = a.rot >> 1;
  pdl_wait();
  paged_prefix<kApThreads>(pre, a.B, [&](int b) {
    int start, tok0;
    const int n = append_span(a, b, start, tok0);
    return n > 0 ? a.chunk.div(start + n - 1) - a.chunk.div(start) + 1 : 0u;
  });
  const uint32_t total = pre[a.B];
  // what a block is and where it goes; warp 0 works out the next one's while the others are at their tasks
  struct Unit {
    int tok, r0, rows, held, pid, off;
  };
  __shared__ Unit units[2];
  auto prepare = [&](uint32_t u, Unit &out) {
    if (u >= total) return;
    const int b = paged_find(pre, a.B, u);
    int start, tok0;
    const int n = append_span(a, b, start, tok0);
    const int blk = a.chunk.div(start) + (u - pre[b]);
    Unit x;
    x.r0 = max(start, blk * chunk);
    x.rows = min(start + n, (blk + 1) * chunk) - x.r0;  // (t_max <= 2^28)
    x.held = x.r0 - blk * chunk;
    x.tok = tok0 + (x.r0 - start);
    const uint32_t pg = a.page.div(x.r0);
    x.pid = __ldcg(a.table + static_cast<size_t>(b) * a.max_pages + pg);
    x.off = x.r0 - static_cast<int>(pg) * static_cast<int>(a.page.d);
    if (lane == 0) out = x;
  };
  if (warp == 0) prepare(blockIdx.x, units[0]);
  if (warp == 1 && lane < 8) cs[lane] = make_float2(1.f, 0.f);
  __syncthreads();
  int flip = 0;
  for (uint32_t u = blockIdx.x; u < total; u += gridDim.x, flip ^= 1) {
    const Unit x = units[flip];
    const int rows = x.rows, held = x.held, pid = x.pid, off = x.off;
    const int64_t tok = x.tok;
    const bool live = static_cast<uint32_t>(pid) < static_cast<uint32_t>(a.n_pages);
    if (!live && tid == 0) flag_error(a.status, GSA_DEVERR_BAD_INDEX);
    for (int i = tid; i < rows * half; i += kApThreads) {
      const int r = i / half, f = i - r * half;
      const int p = a.pos ? __ldcg(a.pos + tok + r) : x.r0 + r;
      // turns in 64 bits; the fraction of a turn as fp32 plus its remainder
      const double turns = static_cast<double>(p) * static_cast<double>(__ldcg(a.inv_freq + f)) * 0.15915494309189535;
      const double fr = 2.0 * (turns - rint(turns));
      const float hi = static_cast<float>(fr);
      const float lo = static_cast<float>(fr - static_cast<double>(hi)) * 3.14159265f;
      float sn, cn;
      sincospif(hi, &sn, &cn);
      cs[8 + i] = make_float2(fmaf(-lo, sn, cn), fmaf(lo, cn, sn));
    }
    __syncthreads();
    if (warp == 0) prepare(u + gridDim.x, units[flip ^ 1]);
    // tasks: K and V of each kv head, then the rows' queries in groups of kQPass passes
    constexpr int kHeads = kQPass * 32 / (D / 16);  // heads of a group
    const int kv_tasks = live ? 2 * a.hkv : 0;
    const int groups = a.q ? (a.hq + kHeads - 1) / kHeads : 0;
    const int tasks = kv_tasks + rows * groups;
    for (int i = blockIdx.y * kApWarps + warp; i < tasks; i += gridDim.y * kApWarps) {
      if (i < kv_tasks) {
        const bool is_v = i >= a.hkv;
        const int h = is_v ? i - a.hkv : i;
        const uint32_t ph = static_cast<uint32_t>(pid) * a.hkv + h, dst = ph * a.page.d + off;  // rows: 32 bits
        const uint32_t si = ph * a.blocks + a.chunk.div(off);
        if (is_v)
          append_block<D, T, FMT, INTER, false>(static_cast<const T *>(a.v) + tok * a.v_stride + h * D, a.v_stride,
                                                rows, held, a.vp, dst, a.vs + si, 0, nullptr);
        else
          append_block<D, T, FMT, INTER, true>(static_cast<const T *>(a.k) + tok * a.k_stride + h * D, a.k_stride, rows,
                                               held, a.kp, dst, a.ks + si, a.rot, cs);
      } else {
        const int r = (i - kv_tasks) / groups, grp = (i - kv_tasks) - r * groups;
        append_queries<D, T, INTER>(static_cast<const T *>(a.q) + (tok + r) * a.q_stride,
                                    static_cast<T *>(a.q_out) + (tok + r) * static_cast<int64_t>(a.hq) * D, r,
                                    grp * kHeads, a.hq, a.rot, cs);
      }
    }
    __syncthreads();  // the table of sines is read, the next unit is there
  }
  pdl_trigger();
  if (a.advance) {
    // every CTA has read the lengths: the last to arrive advances them
    __shared__ int last_s;
    __syncthreads();
    if (tid == 0) {
      __threadfence();
      const uint32_t all = gridDim.x * gridDim.y;
      last_s = atomicAdd(a.counter, 1u) == all - 1;
      if (last_s) {
        __threadfence();
        *a.counter = 0u;
      }
    }
    __syncthreads();
    if (last_s)
      for (int b = tid; b < a.B; b += kApThreads) {
        int start, tok0;
        const int n = append_span(a, b, start, tok0);
        if (n > 0) a.own_len[b] = max(__ldcg(a.own_len + b), 0) + n;
      }
  }
}

}  // namespace gsa
