// norm_quant.cu -- rows to e4m3 codes with one fp32 scale per 128 columns, after a root-mean-square norm with the
// residual's addition (rms_norm_quant) or as they are (quant_rows): the left operand of dsa_matmul_fp8.
//
//   h = T(x + residual),  r = 1 / sqrt(mean(h^2) + eps),  v = h w r;   per group: s = fp32(max|v| / 448),  c = e4m3(v / s)
//
// h w is exact in fp32 for 16-bit types, and r, which the group's values share, is kept as the sum of two floats, so that
// s and the codes are those of the formula but where the sum of squares (fp32) is off by enough to tell: v and v / s
// have no rounding of their own (quant.cuh).
//
// Every byte moves once: a row stays in registers between the sum and the quantisation.  A lane has a unit of 32 columns,
// four pieces of eight 32 apart, so that a group is four lanes: its maximum, scale and reciprocal are paid once for 32
// columns (sixteen a lane: 240 us for 16,384 rows of 7,168 bf16 with residual, 54 for 4,095 rows of 16,384).  A row of up to
// 1,024 columns is 4 to 32 lanes of a warp, a longer one a block; its warps' sums meet in shared memory, where one warp
// makes r of them for all.
//
// Bound by HBM with a residual (16,384 rows of 7,168 bf16 in 122 us in a run of calls, 6.8 TB/s) and for 32-bit rows as they
// are (4,095 of 16,384 in 48 us, 6.9 TB/s, above the rate of a copy as four of five bytes are read); 16-bit rows as they are
// are near both HBM's and the issue's limit (4,095 of 16,384 bf16 in 33.5 us, 6.0 TB/s; 67% of the issue slots): a conversion
// takes two roundings of every value (see quant.cuh).  A norm without a residual fills neither (16,384 of 7,168 bf16 in 88 us,
// 4.0 TB/s; 56% of the issue slots): a row's loads, two barriers and conversion follow one another in its block, and nothing
// of the next row is on its way meanwhile.
#include "dsa_internal.h"
#include "quant.cuh"

namespace dsa {
namespace nq {

constexpr int kGroup = 128;

constexpr int kUnit = 32, kPieces = 4, kLanes = kGroup / kUnit;   // columns and pieces of a lane, lanes of a group

struct NormParams {
  int n_rows, dim, lanes;   // lanes of a row: 4, 8, 16, 32, or a block's
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
  int dim, groups;
  uint32_t units;            // of all rows
  uint32_t row_mul;          // g / groups = g * row_mul >> row_shift for 0 <= g < 2^31
  int row_shift;
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

// The largest finite magnitude of a group, from its lanes' units.
DSA_DEV float group_max(const uint64_t* x) {
  float f[kUnit];
#pragma unroll
  for (int i = 0; i < kUnit; i += 2) {
    const float2 two = unpack2(x[i / 2]);
    f[i] = two.x;
    f[i + 1] = two.y;
  }
  float a = fmaxf(finite_max16(f), finite_max16(f + 16));
#pragma unroll
  for (int o = 1; o < kLanes; o <<= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
  return a;
}

template <int E>
DSA_DEV float value_at(const uint8_t* base, long long at) {
  if constexpr (E == DSA_ELEM_FP32) return reinterpret_cast<const float*>(base)[at];
  const uint16_t v = reinterpret_cast<const uint16_t*>(base)[at];
  if constexpr (E == DSA_ELEM_BF16) return __uint_as_float((uint32_t)v << 16);
  return __half2float(*reinterpret_cast<const __half*>(&v));
}

// The columns whose codes codes8() left open, in turn: code(off) gives that of the column `off` columns on.  (With 16-bit
// rows every 2^10th quotient is next to a border, one in most warps: eight columns at a time, with both codes and the
// values in registers, they took as long as all the rest, 54 us instead of 47 for 4,095 x 16,384 bf16.)
template <class Code>
DSA_DEV void settle_open(uint32_t open, int pieces, uint8_t* codes, Code&& code) {
  while (open) {
    const int bit = __ffs((int)open) - 1, four = bit & 7, off = (four >> 1) * 32 + (four & 1) * 4 + (bit >> 3);
    open &= open - 1u;
    if ((four >> 1) < pieces) codes[off] = (uint8_t)code(off);
  }
}

// 1 / sqrt(total / d + eps), as the sum of two floats, where the sum of squares is total + lost.
DSA_DEV float2 root_of(float total, float lost, int dim, float eps) {
  const float d = (float)dim, mean = __fdiv_rn(total, d);
  float more;
  const float t = two_sum(mean, eps, more);
  more += __fdiv_rn(fmaf(-mean, d, total) + lost, d);
  if (!(fabsf(more) <= t)) more = 0.f;   // (an infinite or NaN sum)
  float2 r;
  r.x = inverse_root(t, more, r.y);
  return r;
}

// Most threads of a block of the variant with registers for two such blocks (16-bit rows, 72 of them; four blocks of 7,168
// columns) or as many as it wants (32-bit rows, 90).  A longer row's block, of up to 1,024 threads, leaves each 64 at most,
// which spill, and fits an SM once: 8,192 rows of 14,344 bf16 with residual take 155 us against 131 of 14,336, 4,096 of 16,392
// fp32 227 against 146 of 16,384 (floors 121 and 129), 2,048 of 32,768 fp32 211.  The same variant for shorter rows: 16,384 of
// 7,168 bf16 with residual 134 against 122, without 96 against 88, 11,969 of 1,536 fp32 45 against 31.  (76 registers, three
// blocks of 7,168 columns: 162.)
template <int E>
constexpr int kFew = E == DSA_ELEM_FP32 ? 512 : 448;

// E: type of the rows; WE: of the weight; kMost: most threads of a block.
template <int E, int WE, int kMost>
__global__ void __launch_bounds__(kMost, kMost == kFew<DSA_ELEM_BF16> ? 2 : 1) norm_kernel(const __grid_constant__ NormParams p) {
  __shared__ float part[32];
  __shared__ float2 root;
  const int tid = threadIdx.x;
  const bool shared = p.lanes <= 32;   // (rows that share a warp or a block)
  const long long row = shared ? ((long long)blockIdx.x * blockDim.x + tid) / p.lanes : blockIdx.x;
  const int l = shared ? tid & (p.lanes - 1) : tid;
  const int col = (l / kLanes) * kGroup + (l % kLanes) * 8;   // the unit's columns: eight from here on, and 32, 64 and 96 on
  const int pieces = row < p.n_rows && col < p.dim ? min(kPieces, (p.dim - col + 31) / 32) : 0;

  griddep_wait();   // nothing above reads global memory
  uint64_t h[kUnit / 2];   // two columns each
  {
    Eight<E> x[kPieces];
    const long long at = row * p.x_stride + col;
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
      x[k].zero();
      if (k < pieces) x[k].load_shared(p.x, at + k * 32);
    }
    if (p.residual) {
      Eight<E> r[kPieces];
      const long long from = row * p.residual_stride + col, to = row * p.sum_stride + col;
#pragma unroll
      for (int k = 0; k < kPieces; ++k) {
        r[k].zero();
        if (k < pieces) r[k].load(p.residual, from + k * 32);
      }
#pragma unroll
      for (int k = 0; k < kPieces; ++k) {
        x[k].add(r[k]);
        if (k < pieces) x[k].store(p.sum, to + k * 32);
      }
    }
#pragma unroll
    for (int k = 0; k < kPieces; ++k) x[k].pairs(h + 4 * k);
  }

  uint64_t ss = 0u;   // two sums
#pragma unroll
  for (int i = 0; i < kUnit / 2; ++i) ss = fma2(h[i], h[i], ss);
  float total = unpack2(ss).x + unpack2(ss).y;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1)
    if (o < p.lanes) total += __shfl_xor_sync(0xffffffffu, total, o);
  // (on their way while the sums meet; 32-bit ones beside 16-bit rows, which would not find the registers, later)
  constexpr bool kEarly = E == WE;
  Eight<WE> w[kPieces];
  auto load_weight = [&](int k) {
    w[k].zero();
    if (k < pieces) w[k].load_shared(p.weight, col + k * 32);
  };
  if (kEarly) {
#pragma unroll
    for (int k = 0; k < kPieces; ++k) load_weight(k);
  }
  float2 r;
  if (shared) {
    r = root_of(total, 0.f, p.dim, p.eps);
  } else {
    if ((tid & 31) == 0) part[tid >> 5] = total;
    __syncthreads();
    if (tid < 32) {
      float sum = tid < (int)(blockDim.x >> 5) ? part[tid] : 0.f, lost = 0.f;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        float e;
        const float other = __shfl_xor_sync(0xffffffffu, sum, o), others = __shfl_xor_sync(0xffffffffu, lost, o);
        sum = two_sum(sum, other, e);
        lost += others + e;
      }
      if (tid == 0) root = root_of(sum, lost, p.dim, p.eps);
    }
    __syncthreads();
    r = root;
  }

  // h w in h's place
  if (r.x == 0.f) {   // what is finite becomes 0 where h w is not
#pragma unroll
    for (int i = 0; i < kUnit / 2; ++i) h[i] = mul2(h[i], 0u);
  }
#pragma unroll
  for (int k = 0; k < kPieces; ++k) {
    uint64_t f[4];
    if (!kEarly) load_weight(k);
    w[k].pairs(f);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[4 * k + i] = mul2(h[4 * k + i], f[i]);
  }
  float a = group_max(h), top = a * r.x;
  // v is beyond fp32 where h w is not: the largest of the others.  (By the whole warp: groups alone cost registers.)
  if (__any_sync(0xffffffffu, top == INFINITY)) {
    a = 0.f;
#pragma unroll
    for (int i = 0; i < kUnit / 2; ++i) {
      const float2 two = unpack2(h[i]);
      a = fmaxf(a, fabsf(two.x) * r.x < INFINITY ? fabsf(two.x) : 0.f);
      a = fmaxf(a, fabsf(two.y) * r.x < INFINITY ? fabsf(two.y) : 0.f);
    }
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    top = a * r.x;
  }
  float s = 1.f;
  if (top > 0.f) {
    const float q = __fdiv_rn(top, 448.f), e = fmaf(a, r.x, -top) + a * r.y;
    s = fmaxf(fmaf(fmaf(-q, 448.f, top) + e, 1.f / 448.f, q), 0x1p-126f);
  }
  const float inv = fast_inverse(s);
  uint8_t* codes = p.codes + row * p.codes_stride + col;
  // v in h's place
  const uint64_t rr = pack2(r.x, r.x), down = pack2(inv * kDown, inv * kDown), up = pack2(inv * kUp, inv * kUp);
#pragma unroll
  for (int i = 0; i < kUnit / 2; ++i) h[i] = mul2(h[i], rr);
  uint32_t open = 0;
#pragma unroll
  for (int k = 0; k < kPieces; ++k) {
    const uint2 c = codes8(h + 4 * k, down, up, 2 * k, open);
    if (k < pieces) *reinterpret_cast<uint2*>(codes + k * 32) = c;
  }
  settle_open(open, pieces, codes, [&](int off) {
    // (the column is read again: registers have no index)
    const float u = p.residual ? value_at<E>(p.sum, row * p.sum_stride + col + off) : value_at<E>(p.x, row * p.x_stride + col + off);
    const float uw = (r.x == 0.f ? u * 0.f : u) * value_at<WE>(p.weight, col + off);
    const uint32_t lo = e4m3x2(uw * r.x * (inv * kDown), 0.f) & 0xffu;
    return settle_by(uw, r.x, r.y, s, lo, lo + 1);
  });
  if (p.y) {   // (after the columns were read again: it may be x itself)
#pragma unroll
    for (int k = 0; k < kPieces; ++k)
      if (k < pieces) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          const float2 two = unpack2(h[(8 * k + i) / 2]);
          v[i] = two.x;
          v[i + 1] = two.y;
        }
        store8<E>(p.y, row * p.y_stride + col + k * 32, v);
      }
  }
  if (pieces > 0 && l % kLanes == 0) p.scale[row * p.scale_stride + col / kGroup] = s;
}

// E: type of the rows; N: units of a lane, whose loads are all on their way before the first is used.
template <int E, int N>
__global__ void __launch_bounds__(128) quant_kernel(const __grid_constant__ QuantParams p) {
  uint32_t row[N];
  int group[N], pieces[N];
  Eight<E> x[N][kPieces];
  const int in = (int)(threadIdx.x % kLanes) * 8;   // of the group's columns
  griddep_wait();   // nothing above reads global memory
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const uint32_t u = blockIdx.x * (N * 128u) + n * 128u + threadIdx.x, g = u / kLanes;   // groups, row after row
    row[n] = (uint32_t)(((unsigned long long)g * p.row_mul) >> p.row_shift);
    group[n] = (int)(g - row[n] * (uint32_t)p.groups);
    const int col = group[n] * kGroup + in;
    pieces[n] = u < p.units && col < p.dim ? min(kPieces, (p.dim - col + 31) / 32) : 0;
    const long long at = row[n] * p.x_stride + col;
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
      x[n][k].zero();
      if (k < pieces[n]) x[n][k].load_shared(p.x, at + k * 32);
    }
  }
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const int col = group[n] * kGroup + in;
    uint64_t v[kUnit / 2];
#pragma unroll
    for (int k = 0; k < kPieces; ++k) x[n][k].pairs(v + 4 * k);
    const float a = group_max(v);
    const float s = a > 0.f ? fmaxf(__fdiv_rn(a, 448.f), 0x1p-126f) : 1.f, inv = fast_inverse(s);
    uint8_t* codes = p.codes + row[n] * p.codes_stride + col;
    const uint64_t down = pack2(inv * kDown, inv * kDown), up = pack2(inv * kUp, inv * kUp);
    uint32_t open = 0;
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
      const uint2 c = codes8(v + 4 * k, down, up, 2 * k, open);
      if (k < pieces[n]) *reinterpret_cast<uint2*>(codes + k * 32) = c;
    }
    settle_open(open, pieces[n], codes, [&](int off) {
      const float y = value_at<E>(p.x, row[n] * p.x_stride + col + off);
      const uint32_t lo = e4m3x2(y * (inv * kDown), 0.f) & 0xffu;
      return settle(y, s, lo, lo + 1);
    });
    if (pieces[n] > 0 && in == 0) p.scale[row[n] * p.scale_stride + group[n]] = s;
  }
}

using NormKernel = void (*)(NormParams);

template <int E, int WE>
NormKernel norm_variant(int threads) {
  return threads <= kFew<E> ? norm_kernel<E, WE, kFew<E>> : norm_kernel<E, WE, 1024>;
}

// A launch that may begin while the kernel before it ends (the kernels wait for that before they read anything).
template <class Params>
cudaError_t launch_early(void (*k)(Params), unsigned blocks, int threads, cudaStream_t stream, const Params& p) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, p);
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
  const int units = (a.dim + kGroup - 1) / kGroup * kLanes;   // of a row
  int threads, rows = 1;   // of a block
  if (units <= 32) {
    for (p.lanes = kLanes; p.lanes < units; p.lanes *= 2) {
    }
    threads = 128;
    rows = threads / p.lanes;
  } else {
    threads = p.lanes = (units + 31) / 32 * 32;
  }
  const long long blocks = ((long long)a.n_rows + rows - 1) / rows;
  const bool same = a.weight_elem == a.elem;
  const NormKernel k =
      a.elem == DSA_ELEM_FP32   ? norm_variant<DSA_ELEM_FP32, DSA_ELEM_FP32>(threads)
      : a.elem == DSA_ELEM_BF16 ? same ? norm_variant<DSA_ELEM_BF16, DSA_ELEM_BF16>(threads) : norm_variant<DSA_ELEM_BF16, DSA_ELEM_FP32>(threads)
      : same                    ? norm_variant<DSA_ELEM_FP16, DSA_ELEM_FP16>(threads) : norm_variant<DSA_ELEM_FP16, DSA_ELEM_FP32>(threads);
  const cudaError_t e = launch_early(k, (unsigned)blocks, threads, stream, p);
  if (e != cudaSuccess) return cuda_fail(e, "rms_norm_quant: launch", err);
  return DSA_OK;
}

dsa_status launch_quant_rows(const dsa_quant_rows_args& a, cudaStream_t stream, std::string& err) {
  using namespace nq;
  QuantParams p;
  p.dim = a.dim;
  p.groups = (a.dim + kGroup - 1) / kGroup;
  const long long groups = (long long)a.n_rows * p.groups;
  if (groups * kLanes > 0x7fffffffLL) {
    err = "quant_rows: rows times their groups of 128 columns must number below 2^29";
    return DSA_ERR_UNSUPPORTED;
  }
  p.units = (uint32_t)groups * kLanes;
  int shift = 0;   // 2^shift >= groups of a row
  while ((1LL << shift) < p.groups) ++shift;
  p.row_shift = 31 + shift;
  p.row_mul = (uint32_t)((((unsigned long long)1 << p.row_shift) + p.groups - 1) / p.groups);
  p.x_stride = a.x_stride;
  p.codes_stride = a.codes_stride;
  p.scale_stride = a.scale_stride;
  p.x = reinterpret_cast<const uint8_t*>(a.x);
  p.codes = reinterpret_cast<uint8_t*>(a.codes);
  p.scale = a.scale;
  constexpr int N = 2;
  const unsigned blocks = (p.units + N * 128 - 1) / (N * 128);
  const auto k = a.elem == DSA_ELEM_BF16   ? quant_kernel<DSA_ELEM_BF16, N>
                 : a.elem == DSA_ELEM_FP16 ? quant_kernel<DSA_ELEM_FP16, N>
                                           : quant_kernel<DSA_ELEM_FP32, N>;
  const cudaError_t e = launch_early(k, blocks, 128, stream, p);
  if (e != cudaSuccess) return cuda_fail(e, "quant_rows: launch", err);
  return DSA_OK;
}

}  // namespace dsa
