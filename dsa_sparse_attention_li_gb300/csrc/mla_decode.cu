// mla_decode.cu -- dense latent attention over the paged cache, absorbed form.
//
// One warp per (token, head): 18 of the 576 columns a lane, online softmax over the positions.
#include "dsa_internal.h"
#include "ptx.cuh"

namespace dsa {
namespace mlad {

constexpr int kWarps = 8;

struct Params {
  int B, n_q, H, max_pages, num_pages;
  float scale_log2;
  const __nv_bfloat16* q;
  const uint8_t* kv;
  const int* page_table;
  const int* seq_lens;
  const int* q_start;
  __nv_bfloat16* out;
  float* lse;
  int* status;
};

template <bool KV8>
__global__ void __launch_bounds__(kWarps * 32) mla_decode_kernel(const Params p) {
  const int lane = threadIdx.x & 31;
  const long long w = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < p.B; i += kWarps * 32)
      if (p.q_start[i] < 0 || p.q_start[i + 1] < p.q_start[i] || p.q_start[i + 1] > p.n_q)
        report(p.status, kStatusDeviceCheck);
  const int t = (int)(w / p.H);
  if (t >= p.n_q) return;
  int lo = 0, hi = p.B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.q_start[mid] <= t) lo = mid; else hi = mid - 1;
  }
  const int b = lo, s0 = p.q_start[b], s1 = p.q_start[b + 1];
  if (s0 < 0 || s1 > p.n_q || t < s0 || t >= s1) return;
  int len = p.seq_lens[b];
  if (len < 0 || len > p.max_pages * 64) {
    if (lane == 0) report(p.status, kStatusDeviceCheck);
    len = max(0, min(len, p.max_pages * 64));
  }
  const int seen = len - (s1 - s0) + (t - s0) + 1;
  float q[18], o[16], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < 18; ++i) q[i] = __bfloat162float(p.q[w * 576 + i * 32 + lane]);
#pragma unroll
  for (int i = 0; i < 16; ++i) o[i] = 0.f;
  for (int j = 0; j < seen; ++j) {
    const int pg = p.page_table[(long long)b * p.max_pages + (j >> 6)];
    if (pg < 0 || pg >= p.num_pages) {
      if (lane == 0) report(p.status, kStatusDeviceCheck);
      continue;
    }
    const long long row = (long long)pg * 64 + (j & 63);
    float k[18], z = 0.f;
#pragma unroll
    for (int i = 0; i < 18; ++i) {
      if constexpr (KV8) {
        const uint8_t* r = p.kv + row * 608;
        const __half_raw h = __nv_cvt_fp8_to_halfraw(r[i * 32 + lane], __NV_E4M3);
        const float s = reinterpret_cast<const float*>(r + 576)[i >> 2];
        k[i] = __bfloat162float(__float2bfloat16_rn(__half2float(*reinterpret_cast<const __half*>(&h)) * s));
      } else {
        k[i] = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p.kv)[row * 576 + i * 32 + lane]);
      }
      z += q[i] * k[i];
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) z += __shfl_xor_sync(0xffffffffu, z, x);
    z *= p.scale_log2;
    const float m2 = fmaxf(m, z);
    const float a = m == m2 ? 1.f : exp2f(m - m2), e = exp2f(z - m2);
    m = m2;
    l = l * a + e;
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] = o[i] * a + e * k[i];
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int i = 0; i < 16; ++i) p.out[w * 512 + i * 32 + lane] = __float2bfloat16_rn(o[i] * inv);
  if (lane == 0 && p.lse) p.lse[w] = l == 0.f ? -INFINITY : m * 0.69314718055994531f + logf(l);
}

}  // namespace mlad

size_t mla_decode_workspace_bytes(const dsa_mla_decode_args&) { return 0; }

dsa_status launch_mla_decode(const dsa_mla_decode_args& a, cudaStream_t stream, std::string& err) {
  using namespace mlad;
  Params p = {a.B, a.n_q, a.H, a.max_pages, a.num_pages, a.softmax_scale * 1.4426950408889634f,
              (const __nv_bfloat16*)a.q, (const uint8_t*)a.kv_pool, a.page_table, a.seq_lens, a.q_start,
              (__nv_bfloat16*)a.out, a.lse, a.status};
  const unsigned blocks = (unsigned)(((long long)a.n_q * a.H + kWarps - 1) / kWarps);
  if (a.kv_dtype == DSA_FP8_E4M3)
    mla_decode_kernel<true><<<blocks, kWarps * 32, 0, stream>>>(p);
  else
    mla_decode_kernel<false><<<blocks, kWarps * 32, 0, stream>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "mla_decode: launch", err);
  return DSA_OK;
}

}  // namespace dsa
