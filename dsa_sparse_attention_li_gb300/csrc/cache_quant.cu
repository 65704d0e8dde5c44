// cache_quant.cu -- rows of activations into the quantised paged caches, and cache rows back out.
//
// "Inference Optimization for Kimi K3.1 Pro ...", section 4 (the latent cache in FP8 with one
// scale per token and 128-column tile; the index keys in FP8 with group scales): the formats that
// dsa_li_topk, dsa_sfa_* and dsa_mla_decode read.
//
// Quantisation of a group of columns with largest finite magnitude a:
//   FP8:    s = fp32(a / 448), 1 for a = 0, at least 2^-126;   c_i = e4m3(x_i / s)
//   MXFP8:  e = max(floor(log2 a) - 8, -127), 0 for a = 0;     c_i = e4m3(x_i 2^-e)
// e4m3() rounds to nearest even and saturates at 448.  x_i / s is not rounded before e4m3(): a
// quotient rounded to fp32 first can land exactly on the border between two codes.  The fast
// path multiplies by 1/s (1 - 2^-21) and 1/s (1 + 2^-21), between which the quotient lies, and keeps a
// code on which both agree; the few others, about one element in 2^16, take the sign of |x| - border * s,
// which one fused multiply-add keeps (see settle()).
//
// Both kernels move each byte once and are bound by HBM, with short rows by instruction issue (key rows: 70%
// of the issue slots).  The unit of work of a warp is 512 columns, two pieces of eight a lane (16- or
// 32-byte loads) out of one group, so that the group's maximum, its scale and the addresses are paid once
// for sixteen columns (eight a lane: 262,144 key rows 35 us instead of 31, 61,440 rows read 22 instead of
// 18).  A group is a segment of 2 to 16 lanes and its maximum a few shuffles.  A latent row is a unit and an
// eighth: the 64-column tails of eight rows share one, else most lanes of it would idle.  (A bf16 row has
// no groups and any width: units of 256 columns, four a warp.)
//
// A warp takes two units at once, each step of the chain seq, pos -> page table -> cache row issued for both
// before the next, beside the loads of the rows, which stay packed until they are quantised.  One unit a
// warp: 65,536 fp32 latent rows 33 against 31 us, 61,440 rows read 20 against 18; four: 35 and 18.  A write
// of less than a wave of warps takes one unit a warp, the shorter chain of instructions (one latent row 6
// us against 8, launch included; a read of 50 rows is 7 us either way).  Blocks of four warps: of eight,
// whose last warps hold the SM longer, 65,536 latent rows took 35 us.
//
// Measured, launch included, alone: 65,536 fp32 latent rows written in 31 us (6.1 TB/s; 34 to 35 us, 5.5 TB/s, in a
// run of calls), 262,144 fp16 key rows of 128 in 25 us (4.2 TB/s; the same), 61,440 latent rows read as
// bf16 in 18 us (5.9 TB/s; 20.5 us, 5.3 TB/s).
#include <type_traits>

#include "dsa_internal.h"
#include "ptx.cuh"

namespace dsa {
namespace cq {

constexpr int kThreads = 128;
constexpr int kUnits = 2;         // of a warp (a write's with many rows)
constexpr int kUnitsBf16 = 4;
constexpr int kLatent = 576;
constexpr int kLatentRow = 608;   // 576 codes, 5 fp32 scales, 12 zero bytes

struct Params {
  int n_rows, dim, B, page_size, max_pages, num_pages;
  int row_stride;        // elements
  uint32_t page_mul;     // j / page_size = j * page_mul >> page_shift for 0 <= j < 2^31
  int page_shift;
  long long units;
  uint8_t* rows;
  uint8_t* pool;
  float* scale_pool;
  uint8_t* sf_pool;
  const int* page_table;
  const int* seq;
  const int* pos;
  int* status;
};

// The row and the first column of a lane's columns in unit u; row < 0: none.  They are eight, and of a quantised
// format the eight that follow `step` columns on too, both of one group.
struct Place {
  int row, col, step;
};

// (units of a quantised format number at most 9/8 of the rows; a bf16 row may have any width)
template <int F>
using Unit = std::conditional_t<F == DSA_ROW_BF16, unsigned long long, uint32_t>;

template <int F>
DSA_DEV Place place(const Params& p, Unit<F> u, int lane) {
  if constexpr (F == DSA_ROW_BF16) {
    const int per = p.dim >> 3;             // lanes of a row
    const unsigned long long c = u * 32 + lane, row = c / per;
    return {row < (unsigned)p.n_rows ? (int)row : -1, (int)(c - row * per) * 8, 0};
  } else {
    uint32_t row;
    int col, step;
    if constexpr (F == DSA_ROW_LATENT_FP8) {
      const uint32_t blk = u / 9, k = u - blk * 9;   // eight rows are nine units
      row = blk * 8 + (k < 8 ? k : lane >> 2);
      col = k < 8 ? (lane >> 3) * 128 + (lane & 7) * 8 : 512 + (lane & 3) * 8;
      step = k < 8 ? 64 : 32;
    } else {                                // 2, 4, 8 or 16 lanes a row
      const int per = p.dim >> 4, l = lane & (per - 1), shift = 31 - __clz(per);
      row = (u << (5 - shift)) + (lane >> shift);
      col = F == DSA_ROW_MXFP8 ? (l >> 1) * 32 + (l & 1) * 8 : l * 8;
      step = F == DSA_ROW_MXFP8 ? 16 : p.dim >> 1;
    }
    return {row < (uint32_t)p.n_rows ? (int)row : -1, col, step};
  }
}

// Physical cache rows of N rows (-1: none, or out of range, which is reported), the loads of all of
// them in flight together.
template <int N>
DSA_DEV void cache_rows(const Params& p, const Place* w, int* at) {
  int b[N], j[N], slot[N], pg[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    b[i] = w[i].row >= 0 ? p.seq[w[i].row] : 0;
    j[i] = w[i].row >= 0 ? p.pos[w[i].row] : 0;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    slot[i] = (int)(((unsigned long long)(uint32_t)j[i] * p.page_mul) >> p.page_shift);
    const bool ok = w[i].row >= 0 && b[i] >= 0 && b[i] < p.B && j[i] >= 0 && slot[i] < p.max_pages;
    pg[i] = ok ? p.page_table[(long long)b[i] * p.max_pages + slot[i]] : -1;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const bool ok = pg[i] >= 0 && pg[i] < p.num_pages;
    at[i] = ok ? pg[i] * p.page_size + (j[i] - slot[i] * p.page_size) : -1;
    if (!ok && w[i].row >= 0) report(p.status, kStatusDeviceCheck);
  }
}

// Eight columns of a row as they lie there: half the registers of their fp32 values while 16-bit rows are on
// their way.
template <int E>
struct Eight {
  static constexpr int kWords = E == DSA_ELEM_FP32 ? 2 : 1;
  uint4 v[kWords];

  DSA_DEV void load(const uint8_t* base, long long at) {
    const uint4* s = reinterpret_cast<const uint4*>(base + at * (E == DSA_ELEM_FP32 ? 4 : 2));
#pragma unroll
    for (int k = 0; k < kWords; ++k) v[k] = __ldcs(s + k);
  }
  DSA_DEV void zero() {
#pragma unroll
    for (int k = 0; k < kWords; ++k) v[k] = make_uint4(0u, 0u, 0u, 0u);
  }
  DSA_DEV void values(float* x) const {
#pragma unroll
    for (int k = 0; k < kWords; ++k) {
      const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (E == DSA_ELEM_FP32) {
          x[4 * k + i] = __uint_as_float(w[i]);
        } else if constexpr (E == DSA_ELEM_BF16) {
          x[2 * i] = __uint_as_float(w[i] << 16);
          x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        } else {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
          x[2 * i] = f.x;
          x[2 * i + 1] = f.y;
        }
      }
    }
  }
};

template <int E>
DSA_DEV void store8(uint8_t* base, long long at, const float* y) {
  if constexpr (E == DSA_ELEM_FP32) {
    float4* d = reinterpret_cast<float4*>(base + at * 4);
    d[0] = make_float4(y[0], y[1], y[2], y[3]);
    d[1] = make_float4(y[4], y[5], y[6], y[7]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (E == DSA_ELEM_BF16) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(y[2 * i], y[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&v);
      } else {
        const __half2 v = __floats2half2_rn(y[2 * i], y[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&v);
      }
    }
    *reinterpret_cast<uint4*>(base + at * 2) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

DSA_DEV uint32_t e4m3x2(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

DSA_DEV float e4m3_value(uint32_t code) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)code, __NV_E4M3);
  return __half2float(*reinterpret_cast<const __half*>(&h));
}

// The code of x / s between its neighbours `lo` (toward zero) and `hi`, which differ by one: by the sign
// of |x| - border s, which one fused rounding keeps unless the scale is so small that it underflows.
// (16-bit rows meet exact borders often, about one element in 2^10.)
DSA_DEV uint32_t settle(float x, float s, uint32_t lo, uint32_t hi) {
  const float border = 0.5f * (e4m3_value(lo & 0x7f) + e4m3_value(hi & 0x7f));
  float d = fmaf(-border, s, fabsf(x));
  if (s < 0x1p-100f) d = fmaf(-border, s * 0x1p60f, fabsf(x) * 0x1p60f);  // both products exact
  const uint32_t even = (hi & 1u) ? lo : hi;
  return d > 0.f ? hi : d < 0.f ? lo : even;
}

// Eight columns with scale s, and inv about 1 / s -> eight codes.
DSA_DEV uint2 quantise8(const float* x, float s, float inv) {
  const float down = inv * (1.f - 0x1p-21f), up = inv * (1.f + 0x1p-21f);
  uint32_t lo[4], hi[4], differ = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 l = mul2(make_float2(x[2 * i], x[2 * i + 1]), down), h = mul2(make_float2(x[2 * i], x[2 * i + 1]), up);
    lo[i] = e4m3x2(l.x, l.y);
    hi[i] = e4m3x2(h.x, h.y);
    differ |= lo[i] ^ hi[i];
  }
  if (differ) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (lo[i] == hi[i]) continue;
      const uint32_t l0 = lo[i] & 0xff, h0 = hi[i] & 0xff, l1 = lo[i] >> 8, h1 = hi[i] >> 8;
      lo[i] = (l0 == h0 ? l0 : settle(x[2 * i], s, l0, h0)) | ((l1 == h1 ? l1 : settle(x[2 * i + 1], s, l1, h1)) << 8);
    }
  }
  return make_uint2(lo[0] | (lo[1] << 16), lo[2] | (lo[3] << 16));
}

// A lane's sixteen columns x of a row to cache row dst (< 0: nowhere).  The whole warp takes part.
template <int F>
DSA_DEV void write16(const Params& p, const Place& w, int row, const float* x) {
  const long long dst = row;
  // the group's largest finite magnitude: a NaN (which every maximum loses) or an infinity does not
  // cost its neighbours
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < 16; i += 2) a = max3(a, fabsf(x[i]), fabsf(x[i + 1]));
  if (a == INFINITY) {
    a = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) a = fmaxf(a, fabsf(x[i]) < INFINITY ? fabsf(x[i]) : 0.f);
  }
  constexpr int kMost = F == DSA_ROW_MXFP8 ? 2 : F == DSA_ROW_FP8 ? 16 : 8;   // lanes of a group
  const int lanes = F == DSA_ROW_MXFP8 ? 2 : w.step >> 3;
#pragma unroll
  for (int o = 1; o < kMost; o <<= 1) {
    if (F == DSA_ROW_FP8 && o >= lanes) break;   // (the same for the whole warp)
    const float m = __shfl_xor_sync(0xffffffffu, a, o);
    if (o < lanes) a = fmaxf(a, m);
  }
  if (dst < 0) return;
  if constexpr (F == DSA_ROW_MXFP8) {
    const int e = a > 0.f ? max((int)(__float_as_uint(a) >> 23) - 127 - 8, -127) : 0;
    // 2^-e with e in [-127, 119]: exact, and so is the product wherever e4m3 can tell
    const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
    uint32_t c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = e4m3x2(x[2 * i] * inv, x[2 * i + 1] * inv);
    uint8_t* d = p.pool + dst * p.dim + w.col;
    *reinterpret_cast<uint2*>(d) = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
    *reinterpret_cast<uint2*>(d + w.step) = make_uint2(c[4] | (c[5] << 16), c[6] | (c[7] << 16));
    if ((w.col & 31) == 0) p.sf_pool[dst * (p.dim >> 5) + (w.col >> 5)] = (uint8_t)(e + 127);
  } else {
    const float s = a > 0.f ? fmaxf(__fdiv_rn(a, 448.f), 0x1p-126f) : 1.f;
    float inv;   // within 2^-23; with the two roundings that follow, well inside 2^-21
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
    uint8_t* d = p.pool + dst * (F == DSA_ROW_FP8 ? p.dim : kLatentRow);
    *reinterpret_cast<uint2*>(d + w.col) = quantise8(x, s, inv);
    *reinterpret_cast<uint2*>(d + w.col + w.step) = quantise8(x + 8, s, inv);
    if constexpr (F == DSA_ROW_FP8) {
      if (w.col == 0) p.scale_pool[dst] = s;
    } else {
      if ((w.col & 127) == 0) *reinterpret_cast<float*>(d + kLatent + (w.col >> 7) * 4) = s;
      if (w.col >= 520) *reinterpret_cast<uint32_t*>(d + kLatent + 20 + (w.col - 520) / 2) = 0u;
    }
  }
}

template <int F, int E, int N>
__global__ void __launch_bounds__(kThreads) write_kernel(const __grid_constant__ Params p) {
  const Unit<F> u = ((Unit<F>)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * N;
  const int lane = threadIdx.x & 31;
  Place w[N];
  Eight<E> x[N][2];
  int dst[N];
#pragma unroll
  for (int n = 0; n < N; ++n) {
    w[n] = place<F>(p, u + n, lane);
    x[n][0].zero();
    x[n][1].zero();
    if (w[n].row < 0) continue;
    const long long at = (long long)w[n].row * p.row_stride + w[n].col;
    x[n][0].load(p.rows, at);
    x[n][1].load(p.rows, at + w[n].step);
  }
  cache_rows<N>(p, w, dst);
#pragma unroll
  for (int n = 0; n < N; ++n) {
    float y[16];
    x[n][0].values(y);
    x[n][1].values(y + 8);
    write16<F>(p, w[n], dst[n], y);
  }
}

// A lane's columns of a cache row as they lie there, and their scale: eight bf16, or twice eight codes.
struct Packed {
  uint4 bits;
  float scale;
};

template <int F, int E, int N>
__global__ void __launch_bounds__(kThreads) read_kernel(const __grid_constant__ Params p) {
  const Unit<F> u = ((Unit<F>)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * N;
  const int lane = threadIdx.x & 31;
  Place w[N];
  int src[N];
  Packed v[N];
#pragma unroll
  for (int n = 0; n < N; ++n) w[n] = place<F>(p, u + n, lane);
  cache_rows<N>(p, w, src);
#pragma unroll
  for (int n = 0; n < N; ++n) {
    v[n].bits = make_uint4(0u, 0u, 0u, 0u);
    v[n].scale = 0.f;
    if (src[n] < 0) continue;
    if constexpr (F == DSA_ROW_BF16) {
      v[n].bits = __ldcs(reinterpret_cast<const uint4*>(p.pool + ((long long)src[n] * p.dim + w[n].col) * 2));
    } else {
      const uint8_t* row = p.pool + (long long)src[n] * (F == DSA_ROW_LATENT_FP8 ? kLatentRow : p.dim);
      const uint2 a = __ldcs(reinterpret_cast<const uint2*>(row + w[n].col));
      const uint2 b = __ldcs(reinterpret_cast<const uint2*>(row + w[n].col + w[n].step));
      v[n].bits = make_uint4(a.x, a.y, b.x, b.y);
      if constexpr (F == DSA_ROW_LATENT_FP8) {
        v[n].scale = *reinterpret_cast<const float*>(row + kLatent + (w[n].col >> 7) * 4);
      } else if constexpr (F == DSA_ROW_FP8) {
        v[n].scale = p.scale_pool[src[n]];
      } else {
        const uint32_t e = p.sf_pool[(long long)src[n] * (p.dim >> 5) + (w[n].col >> 5)];
        v[n].scale = e == 255u ? __uint_as_float(0x7fffffffu)      // not a valid scale: NaN
                               : e == 0u ? 0x1p-127f : __uint_as_float(e << 23);
      }
    }
  }
#pragma unroll
  for (int n = 0; n < N; ++n) {
    if (w[n].row < 0) continue;
    const uint32_t bits[4] = {v[n].bits.x, v[n].bits.y, v[n].bits.z, v[n].bits.w};
    const long long at = (long long)w[n].row * p.row_stride + w[n].col;
    float y[8];
    if constexpr (F == DSA_ROW_BF16) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        y[2 * i] = __uint_as_float(bits[i] << 16);
        y[2 * i + 1] = __uint_as_float(bits[i] & 0xffff0000u);
      }
      store8<E>(p.rows, at, y);
    } else {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t two = (bits[2 * k + (i >> 1)] >> ((i & 1) * 16)) & 0xffffu;
          const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
          const float2 m = mul2(f, v[n].scale);
          y[2 * i] = m.x;
          y[2 * i + 1] = m.y;
        }
        store8<E>(p.rows, at + k * w[n].step, y);
      }
    }
  }
}

using Kernel = void (*)(Params);

template <int N>
Kernel write_variant(int format, int elem) {
  static const Kernel k[3][3] = {
      {write_kernel<DSA_ROW_FP8, 0, N>, write_kernel<DSA_ROW_FP8, 1, N>, write_kernel<DSA_ROW_FP8, 2, N>},
      {write_kernel<DSA_ROW_MXFP8, 0, N>, write_kernel<DSA_ROW_MXFP8, 1, N>, write_kernel<DSA_ROW_MXFP8, 2, N>},
      {write_kernel<DSA_ROW_LATENT_FP8, 0, N>, write_kernel<DSA_ROW_LATENT_FP8, 1, N>,
       write_kernel<DSA_ROW_LATENT_FP8, 2, N>}};
  return k[format - 1][elem];
}

Kernel read_variant(int format, int elem) {
  constexpr int N = kUnits, M = kUnitsBf16;
  static const Kernel k[4][3] = {
      {read_kernel<DSA_ROW_BF16, 0, M>, read_kernel<DSA_ROW_BF16, 1, M>, read_kernel<DSA_ROW_BF16, 2, M>},
      {read_kernel<DSA_ROW_FP8, 0, N>, read_kernel<DSA_ROW_FP8, 1, N>, read_kernel<DSA_ROW_FP8, 2, N>},
      {read_kernel<DSA_ROW_MXFP8, 0, N>, read_kernel<DSA_ROW_MXFP8, 1, N>, read_kernel<DSA_ROW_MXFP8, 2, N>},
      {read_kernel<DSA_ROW_LATENT_FP8, 0, N>, read_kernel<DSA_ROW_LATENT_FP8, 1, N>,
       read_kernel<DSA_ROW_LATENT_FP8, 2, N>}};
  return k[format][elem];
}

}  // namespace cq

dsa_status launch_cache_rows(const dsa_cache_rows_args& a, bool write, cudaStream_t stream,
                             std::string& err) {
  using namespace cq;
  Params p;
  p.n_rows = a.n_rows;
  p.dim = a.dim;
  p.B = a.B;
  p.page_size = a.page_size;
  p.max_pages = a.max_pages;
  p.num_pages = a.num_pages;
  p.row_stride = (int)a.row_stride;
  int shift = 0;   // 2^shift >= page_size
  while ((1LL << shift) < a.page_size) ++shift;
  p.page_shift = 31 + shift;
  p.page_mul = (uint32_t)((((unsigned long long)1 << p.page_shift) + a.page_size - 1) / a.page_size);
  p.rows = reinterpret_cast<uint8_t*>(a.rows);
  p.pool = reinterpret_cast<uint8_t*>(a.pool);
  p.scale_pool = a.scale_pool;
  p.sf_pool = a.sf_pool;
  p.page_table = a.page_table;
  p.seq = a.seq;
  p.pos = a.pos;
  p.status = a.status;
  const int cols = a.format == DSA_ROW_BF16 ? 256 : 512;   // of a unit
  p.units = a.format == DSA_ROW_LATENT_FP8 ? ((long long)a.n_rows + 7) / 8 * 9
                                           : ((long long)a.n_rows * a.dim + cols - 1) / cols;
  DeviceInfo dev;
  if (!device_info(dev, err)) return DSA_ERR_CUDA;
  const bool few = write && p.units <= (long long)dev.sm_count * 64;   // less than a wave of warps
  const int each = few ? 1 : a.format == DSA_ROW_BF16 ? kUnitsBf16 : kUnits;
  const long long warps = (p.units + each - 1) / each;
  const long long blocks = (warps + kThreads / 32 - 1) / (kThreads / 32);
  if (blocks > 0x7fffffffLL) {
    err = "cache rows: too many rows for one launch";
    return DSA_ERR_UNSUPPORTED;
  }
  const Kernel k = !write ? read_variant(a.format, a.elem)
                   : few ? write_variant<1>(a.format, a.elem) : write_variant<kUnits>(a.format, a.elem);
  k<<<(unsigned)blocks, kThreads, 0, stream>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, write ? "cache_write_quant: launch" : "cache_read: launch", err);
  return DSA_OK;
}

}  // namespace dsa
