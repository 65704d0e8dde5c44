// matmul_fp8.cu -- product of e4m3 rows with one fp32 scale per 128 columns and e4m3 weights with one per block of
// 128 x 128:
//   out[m][n] = sum_b a_scale[m][b] b_scale[n / 128][b] sum_{k in block b} a[m][k] b[n][k]
//
// Simple form: a block of 256 threads has 64 x 64 outputs, a thread 4 x 4, over blocks of 128 columns whose codes it
// turns into fp32 in shared memory.
#include "dsa_internal.h"
#include "quant.cuh"

namespace dsa {
namespace mm {

constexpr int kTile = 64, kBlock = 128, kPitch = kBlock + 1;

struct Params {
  int M, N, K;
  long long a_stride, a_scale_stride, b_stride, b_scale_stride, out_stride;
  const uint8_t* a;
  const float* a_scale;
  const uint8_t* b;
  const float* b_scale;
  uint8_t* out;
};

template <int E>
__global__ void __launch_bounds__(256) simple_kernel(const __grid_constant__ Params p) {
  extern __shared__ float smem[];
  float* as = smem;
  float* bs = smem + kTile * kPitch;
  const int tid = threadIdx.x, m0 = blockIdx.y * kTile, n0 = blockIdx.x * kTile;
  const int tm = (tid >> 4) * 4, tn = (tid & 15) * 4;
  float acc[4][4] = {};
  for (int k0 = 0; k0 < p.K; k0 += kBlock) {
    for (int i = tid; i < kTile * kBlock; i += 256) {
      const int r = i >> 7, k = i & 127;
      const bool in = k0 + k < p.K;
      as[r * kPitch + k] = in && m0 + r < p.M ? e4m3_value(p.a[(long long)(m0 + r) * p.a_stride + k0 + k]) : 0.f;
      bs[r * kPitch + k] = in && n0 + r < p.N ? e4m3_value(p.b[(long long)(n0 + r) * p.b_stride + k0 + k]) : 0.f;
    }
    __syncthreads();
    float part[4][4] = {};
    for (int k = 0; k < kBlock; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) part[i][j] = fmaf(as[(tm + i) * kPitch + k], bs[(tn + j) * kPitch + k], part[i][j]);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int m = m0 + tm + i, n = n0 + tn + j;
        if (m >= p.M || n >= p.N) continue;
        const float s = p.a_scale[m * p.a_scale_stride + (k0 >> 7)] * p.b_scale[(n >> 7) * p.b_scale_stride + (k0 >> 7)];
        acc[i][j] = fmaf(s, part[i][j], acc[i][j]);
      }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int m = m0 + tm + i, n = n0 + tn + j;
      if (m >= p.M || n >= p.N) continue;
      const long long at = m * p.out_stride + n;
      if constexpr (E == DSA_ELEM_FP32)
        reinterpret_cast<float*>(p.out)[at] = acc[i][j];
      else if constexpr (E == DSA_ELEM_BF16)
        reinterpret_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(acc[i][j]);
      else
        reinterpret_cast<__half*>(p.out)[at] = __float2half_rn(acc[i][j]);
    }
}

}  // namespace mm

dsa_status launch_matmul_fp8(const dsa_matmul_fp8_args& a, cudaStream_t stream, std::string& err) {
  using namespace mm;
  Params p;
  p.M = a.M;
  p.N = a.N;
  p.K = a.K;
  p.a_stride = a.a_stride;
  p.a_scale_stride = a.a_scale_stride;
  p.b_stride = a.b_stride;
  p.b_scale_stride = a.b_scale_stride;
  p.out_stride = a.out_stride;
  p.a = reinterpret_cast<const uint8_t*>(a.a);
  p.a_scale = a.a_scale;
  p.b = reinterpret_cast<const uint8_t*>(a.b);
  p.b_scale = a.b_scale;
  p.out = reinterpret_cast<uint8_t*>(a.out);
  const dim3 grid((a.N + kTile - 1) / kTile, (a.M + kTile - 1) / kTile);
  if (grid.y > 65535) {
    err = "matmul_fp8: too many rows for one launch";
    return DSA_ERR_UNSUPPORTED;
  }
  const int smem = 2 * kTile * kPitch * 4;
  const auto k = a.elem == DSA_ELEM_BF16   ? simple_kernel<DSA_ELEM_BF16>
                 : a.elem == DSA_ELEM_FP16 ? simple_kernel<DSA_ELEM_FP16>
                                           : simple_kernel<DSA_ELEM_FP32>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return cuda_fail(e, "matmul_fp8: set shared memory size", err);
  k<<<grid, 256, smem, stream>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "matmul_fp8: launch", err);
  return DSA_OK;
}

}  // namespace dsa
