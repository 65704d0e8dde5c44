// norm_quant.cu -- rows to e4m3 codes with one fp32 scale per 128 columns, after a root-mean-square norm with the
// residual's addition (rms_norm_quant) or as they are (quant_rows): the left operand of dsa_matmul_fp8.
//
//   h = T(x + residual),  r = 1 / sqrt(mean(h^2) + eps),  v = h w r;   per group: s = fp32(max|v| / 448),  c = e4m3(v / s)
//
// h w is exact in fp32 for 16-bit types, and r, which the group's values share, is kept as the sum of two floats, so that
// s and the codes are those of the formula but where the sum of squares (fp32) is off by enough to tell: v and v / s
// have no rounding of their own (quant.cuh).
//
// Every byte moves once: a row stays in registers, packed, between the sum and the quantisation.  A lane has units of
// sixteen columns, two pieces of eight 64 apart in one group, so that a group is eight lanes and its maximum three
// shuffles.  A row of up to 512 columns is 8, 16 or 32 lanes of a warp, a longer one a block.
#include "dsa_internal.h"
#include "quant.cuh"

namespace dsa {
namespace nq {

constexpr int kGroup = 128;

struct NormParams {
  int n_rows, dim, lanes;
  float eps;
  long long x_stride, residual_stride, sum_stride, y_stride, codes_stride, scale_stride;
  const uint8_t* x;
  const uint8_t* weight;
  const uint8_t* residual;
  uint8_t* sum;
  uint8_t* y;
  uint8_t* codes;
  float* scale;
};

struct QuantParams {
  int n_rows, dim, groups;
  long long units;
  long long x_stride, codes_stride, scale_stride;
  const uint8_t* x;
  uint8_t* codes;
  float* scale;
};

// The sum of two floats, and what its rounding lost.
DSA_DEV float two_sum(float a, float b, float& lost) {
  const float s = a + b, t = s - a;
  lost = (a - (s - t)) + (b - t);
  return s;
}

// 1 / sqrt(hi + lo), as the sum of two floats.
DSA_DEV float inverse_root(float hi, float lo, float& rest) {
  const float r = __frsqrt_rn(hi);
  const float p = r * r, pe = fmaf(r, r, -p);
  const float e = fmaf(-hi, p, 1.f) - fmaf(hi, pe, lo * p);
  rest = 0.5f * r * e;
  if (!(fabsf(rest) <= r)) rest = 0.f;   // r is 0, infinite or NaN, or its square is
  return r;
}

// The code of u r / s, r = hi + lo, between its neighbours: by the sign of |u| r - border s.
DSA_DEV uint32_t settle_by(float u, float hi, float rest, float s, uint32_t lo, uint32_t up) {
  const float border = 0.5f * (e4m3_value(lo & 0x7f) + e4m3_value(up & 0x7f));
  u = fabsf(u);
  if (s < 0x1p-100f) {   // products of this size would lose their last bits
    u *= 0x1p60f;
    s *= 0x1p60f;
  }
  const float p = u * hi, q = border * s;
  const float d = (p - q) + ((fmaf(u, hi, -p) + u * rest) - fmaf(border, s, -q));
  const uint32_t even = (up & 1u) ? lo : up;
  return d > 0.f ? up : d < 0.f ? lo : even;
}

// The largest of a group, which is eight lanes.
DSA_DEV float group_max(float a) {
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
  return a;
}

// E: type of the rows; WE: of the weight; C: units of a lane.
template <int E, int WE, int C>
__global__ void __launch_bounds__(1024) norm_kernel(const __grid_constant__ NormParams p) {
  __shared__ float part[32];
  const int tid = threadIdx.x;
  const bool shared = p.lanes <= 32;   // (rows that share a warp or a block)
  const long long row = shared ? ((long long)blockIdx.x * blockDim.x + tid) / p.lanes : blockIdx.x;
  const int l = shared ? tid & (p.lanes - 1) : tid;
  const bool live = row < p.n_rows;
  auto column = [&](int c, int k) { return ((l + c * p.lanes) >> 3) * kGroup + (l & 7) * 8 + k * 64; };

  Eight<E> x[C][2];
  Eight<WE> w[C][2];
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      x[c][k].zero();
      w[c][k].zero();
      if (live && column(c, k) < p.dim) {
        x[c][k].load(p.x, row * p.x_stride + column(c, k));
        w[c][k].load_shared(p.weight, column(c, k));
      }
    }
  if (p.residual) {
    Eight<E> r[C][2];
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        r[c][k].zero();
        if (live && column(c, k) < p.dim) r[c][k].load(p.residual, row * p.residual_stride + column(c, k));
      }
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float a[8], b[8];
        x[c][k].values(a);
        r[c][k].values(b);
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] += b[i];
        x[c][k].round(a);
        if (live && column(c, k) < p.dim) x[c][k].store(p.sum, row * p.sum_stride + column(c, k));
      }
  }

  float2 ss = make_float2(0.f, 0.f);
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float a[8];
      x[c][k].values(a);
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        ss.x = fmaf(a[i], a[i], ss.x);
        ss.y = fmaf(a[i + 1], a[i + 1], ss.y);
      }
    }
  float total = ss.x + ss.y, lost = 0.f;
  for (int o = 1; o < min(p.lanes, 32); o <<= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  if (!shared) {
    if ((tid & 31) == 0) part[tid >> 5] = total;
    __syncthreads();
    total = part[0];
    for (int i = 1; i < (int)(blockDim.x >> 5); ++i) {
      float e;
      total = two_sum(total, part[i], e);
      lost += e;
    }
  }
  const float d = (float)p.dim, mean = __fdiv_rn(total, d);
  float more;
  const float t = two_sum(mean, p.eps, more);
  more += __fdiv_rn(fmaf(-mean, d, total) + lost, d);
  if (!(fabsf(more) <= t)) more = 0.f;   // (an infinite or NaN sum)
  float rest;
  const float r = inverse_root(t, more, rest);

#pragma unroll
  for (int c = 0; c < C; ++c) {
    float u[16], v[16], f[8];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      x[c][k].values(u + 8 * k);
      w[c][k].values(f);
      if (r == 0.f)   // what is finite becomes 0 here too where h w is not
#pragma unroll
        for (int i = 0; i < 8; ++i) u[8 * k + i] *= 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) u[8 * k + i] *= f[i];
    }
    const float a = group_max(finite_max16(u));
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      const float2 m = mul2(make_float2(u[i], u[i + 1]), r);
      v[i] = m.x;
      v[i + 1] = m.y;
    }
    const float top = a * r;
    float s = 1.f;
    if (top > 0.f) {
      const float q = __fdiv_rn(top, 448.f), e = fmaf(a, r, -top) + a * rest;
      s = fmaxf(fmaf(fmaf(-q, 448.f, top) + e, 1.f / 448.f, q), 0x1p-126f);
    }
    const float inv = fast_inverse(s);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int col = column(c, k);
      if (!live || col >= p.dim) continue;
      const uint2 codes = quantise8_by(v + 8 * k, inv, [&](int i, uint32_t lo, uint32_t up) {
        return settle_by(u[8 * k + i], r, rest, s, lo, up);
      });
      *reinterpret_cast<uint2*>(p.codes + row * p.codes_stride + col) = codes;
      if (p.y) store8<E>(p.y, row * p.y_stride + col, v + 8 * k);
      if ((l & 7) == 0 && k == 0) p.scale[row * p.scale_stride + (col >> 7)] = s;
    }
  }
}

// E: type of the rows; C: units of a lane.
template <int E, int C>
__global__ void __launch_bounds__(128) quant_kernel(const __grid_constant__ QuantParams p) {
  const long long first = (long long)blockIdx.x * (C * 128) + threadIdx.x;
  Eight<E> x[C][2];
  long long row[C];
  int col[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const long long u = first + c * 128;
    const long long g = u >> 3;   // groups, row after row
    row[c] = g / p.groups;
    col[c] = (int)(g - row[c] * p.groups) * kGroup + (int)(u & 7) * 8;
    if (u >= p.units) col[c] = p.dim;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      x[c][k].zero();
      if (col[c] + k * 64 < p.dim) x[c][k].load(p.x, row[c] * p.x_stride + col[c] + k * 64);
    }
  }
#pragma unroll
  for (int c = 0; c < C; ++c) {
    float v[16];
    x[c][0].values(v);
    x[c][1].values(v + 8);
    const float a = group_max(finite_max16(v));
    const float s = a > 0.f ? fmaxf(__fdiv_rn(a, 448.f), 0x1p-126f) : 1.f, inv = fast_inverse(s);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int at = col[c] + k * 64;
      if (at >= p.dim) continue;
      *reinterpret_cast<uint2*>(p.codes + row[c] * p.codes_stride + at) = quantise8(v + 8 * k, s, inv);
      if ((at & 127) == 0) p.scale[row[c] * p.scale_stride + (at >> 7)] = s;
    }
  }
}

using NormKernel = void (*)(NormParams);

template <int C>
NormKernel norm_variant(int elem, int weight_elem) {
  if (elem == DSA_ELEM_BF16)
    return weight_elem == elem ? norm_kernel<DSA_ELEM_BF16, DSA_ELEM_BF16, C> : norm_kernel<DSA_ELEM_BF16, DSA_ELEM_FP32, C>;
  if (elem == DSA_ELEM_FP16)
    return weight_elem == elem ? norm_kernel<DSA_ELEM_FP16, DSA_ELEM_FP16, C> : norm_kernel<DSA_ELEM_FP16, DSA_ELEM_FP32, C>;
  return norm_kernel<DSA_ELEM_FP32, DSA_ELEM_FP32, C>;
}

}  // namespace nq

dsa_status launch_rms_norm_quant(const dsa_rms_norm_quant_args& a, cudaStream_t stream, std::string& err) {
  using namespace nq;
  NormParams p;
  p.n_rows = a.n_rows;
  p.dim = a.dim;
  p.eps = a.eps;
  p.x_stride = a.x_stride;
  p.residual_stride = a.residual_stride;
  p.sum_stride = a.sum_stride;
  p.y_stride = a.y_stride;
  p.codes_stride = a.codes_stride;
  p.scale_stride = a.scale_stride;
  p.x = reinterpret_cast<const uint8_t*>(a.x);
  p.weight = reinterpret_cast<const uint8_t*>(a.weight);
  p.residual = reinterpret_cast<const uint8_t*>(a.residual);
  p.sum = reinterpret_cast<uint8_t*>(a.sum);
  p.y = reinterpret_cast<uint8_t*>(a.y);
  p.codes = reinterpret_cast<uint8_t*>(a.codes);
  p.scale = a.scale;
  const int units = (a.dim + kGroup - 1) / kGroup * 8;   // of a row
  const int each = units > 1024 ? 2 : 1;
  int threads, rows = 1;   // of a block
  if (units <= 32) {
    p.lanes = units <= 8 ? 8 : units <= 16 ? 16 : 32;
    threads = 128;
    rows = threads / p.lanes;
  } else {
    threads = p.lanes = ((units + each - 1) / each + 31) / 32 * 32;
  }
  const long long blocks = ((long long)a.n_rows + rows - 1) / rows;
  const NormKernel k = each == 1 ? norm_variant<1>(a.elem, a.weight_elem) : norm_variant<2>(a.elem, a.weight_elem);
  k<<<(unsigned)blocks, threads, 0, stream>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "rms_norm_quant: launch", err);
  return DSA_OK;
}

dsa_status launch_quant_rows(const dsa_quant_rows_args& a, cudaStream_t stream, std::string& err) {
  using namespace nq;
  QuantParams p;
  p.n_rows = a.n_rows;
  p.dim = a.dim;
  p.groups = (a.dim + kGroup - 1) / kGroup;
  p.units = (long long)a.n_rows * p.groups * 8;
  p.x_stride = a.x_stride;
  p.codes_stride = a.codes_stride;
  p.scale_stride = a.scale_stride;
  p.x = reinterpret_cast<const uint8_t*>(a.x);
  p.codes = reinterpret_cast<uint8_t*>(a.codes);
  p.scale = a.scale;
  constexpr int kUnits = 1;
  const long long blocks = (p.units + kUnits * 128 - 1) / (kUnits * 128);
  if (blocks > 0x7fffffffLL) {
    err = "quant_rows: too many rows for one launch";
    return DSA_ERR_UNSUPPORTED;
  }
  const auto k = a.elem == DSA_ELEM_BF16   ? quant_kernel<DSA_ELEM_BF16, kUnits>
                 : a.elem == DSA_ELEM_FP16 ? quant_kernel<DSA_ELEM_FP16, kUnits>
                                           : quant_kernel<DSA_ELEM_FP32, kUnits>;
  k<<<(unsigned)blocks, 128, 0, stream>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "quant_rows: launch", err);
  return DSA_OK;
}

}  // namespace dsa
