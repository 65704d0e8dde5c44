// mla_prefill.cu -- dense latent attention, expanded form.
//
// One warp per (token, head): online softmax over the keys the token sees.
#include "dsa_internal.h"
#include "ptx.cuh"

namespace dsa {
namespace mlap {

constexpr int kWarps = 8;

struct Params {
  int B, n_q, n_kv, H, max_q;
  float scale_log2;
  long long rope_stride;
  const __nv_bfloat16* q;
  const __nv_bfloat16* kv;
  const __nv_bfloat16* rope;
  const int* q_start;
  const int* kv_start;
  __nv_bfloat16* out;
  float* lse;
  int* status;
};

__global__ void __launch_bounds__(kWarps * 32) mla_prefill_kernel(const Params p) {
  const int lane = threadIdx.x & 31;
  const long long w = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < p.B; i += kWarps * 32)
      if (p.q_start[i] < 0 || p.q_start[i + 1] < p.q_start[i] || p.q_start[i + 1] > p.n_q)
        report(p.status, kStatusDeviceCheck);
  const int t = (int)(w / p.H), h = (int)(w % p.H);
  if (t >= p.n_q) return;
  int lo = 0, hi = p.B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.q_start[mid] <= t) lo = mid; else hi = mid - 1;
  }
  const int b = lo, s0 = p.q_start[b], s1 = p.q_start[b + 1];
  if (s0 < 0 || s1 > p.n_q || t < s0 || t >= s1) return;
  const int k0 = p.kv_start[b], k1 = p.kv_start[b + 1];
  if (k0 < 0 || k1 < k0 || k1 > p.n_kv || t - s0 >= p.max_q) {
    if (lane == 0) report(p.status, kStatusDeviceCheck);
    return;
  }
  const int seen = k1 - k0 - (s1 - s0) + (t - s0) + 1;
  float q[6], o[4] = {0.f, 0.f, 0.f, 0.f}, m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < 6; ++i) q[i] = __bfloat162float(p.q[w * 192 + i * 32 + lane]);
  for (int j = k0; j < k0 + seen; ++j) {
    const __nv_bfloat16* row = p.kv + ((long long)j * p.H + h) * 256;
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) z += q[i] * __bfloat162float(row[i * 32 + lane]);
#pragma unroll
    for (int i = 0; i < 2; ++i) z += q[4 + i] * __bfloat162float(p.rope[j * p.rope_stride + i * 32 + lane]);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) z += __shfl_xor_sync(0xffffffffu, z, x);
    z *= p.scale_log2;
    const float m2 = fmaxf(m, z);
    const float a = m == m2 ? 1.f : exp2f(m - m2), e = exp2f(z - m2);
    m = m2;
    l = l * a + e;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = o[i] * a + e * __bfloat162float(row[128 + i * 32 + lane]);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int i = 0; i < 4; ++i) p.out[w * 128 + i * 32 + lane] = __float2bfloat16_rn(o[i] * inv);
  if (lane == 0 && p.lse) p.lse[w] = l == 0.f ? -INFINITY : m * 0.69314718055994531f + logf(l);
}

}  // namespace mlap

dsa_status launch_mla_prefill(const dsa_mla_prefill_args& a, cudaStream_t stream, std::string& err) {
  using namespace mlap;
  Params p = {a.B, a.n_q, a.n_kv, a.H, a.max_q_per_seq, a.softmax_scale * 1.4426950408889634f, a.k_rope_stride,
              (const __nv_bfloat16*)a.q, (const __nv_bfloat16*)a.kv, (const __nv_bfloat16*)a.k_rope, a.q_start,
              a.kv_start, (__nv_bfloat16*)a.out, a.lse, a.status};
  const long long blocks = ((long long)a.n_q * a.H + kWarps - 1) / kWarps;
  mla_prefill_kernel<<<(unsigned)blocks, kWarps * 32, 0, stream>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "mla_prefill: launch", err);
  return DSA_OK;
}

}  // namespace dsa
