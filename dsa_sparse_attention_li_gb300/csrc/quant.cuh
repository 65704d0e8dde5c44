// quant.cuh -- rows of activations to e4m3 codes: loads and stores of eight columns of a row, and the
// conversion of a group of columns with one fp32 scale.
//
// Of a group whose largest finite magnitude is a:  s = fp32(a / 448), 1 for a = 0, at least 2^-126, and
// c_i = e4m3(x_i / s), to nearest even, saturated at 448.  x_i / s is not rounded before e4m3(): a quotient
// rounded to fp32 first can land exactly on the border between two codes.  The fast path multiplies by
// 1/s (1 - 2^-21) and 1/s (1 + 2^-21), between which the quotient lies, and keeps a code on which both agree;
// the few others, about one element in 2^16, are settled by the sign of |x| - border * s.
#pragma once

#include "dsa.h"
#include "ptx.cuh"

namespace dsa {

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
  // (of memory that other rows read too)
  DSA_DEV void load_shared(const uint8_t* base, long long at) {
    const uint4* s = reinterpret_cast<const uint4*>(base + at * (E == DSA_ELEM_FP32 ? 4 : 2));
#pragma unroll
    for (int k = 0; k < kWords; ++k) v[k] = *(s + k);
  }
  DSA_DEV void zero() {
#pragma unroll
    for (int k = 0; k < kWords; ++k) v[k] = make_uint4(0u, 0u, 0u, 0u);
  }
  DSA_DEV void store(uint8_t* base, long long at) const {
    uint4* d = reinterpret_cast<uint4*>(base + at * (E == DSA_ELEM_FP32 ? 4 : 2));
#pragma unroll
    for (int k = 0; k < kWords; ++k) d[k] = v[k];
  }
  // Takes the values y, rounded to nearest even.
  DSA_DEV void round(const float* y) {
#pragma unroll
    for (int k = 0; k < kWords; ++k) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (E == DSA_ELEM_FP32) {
          w[i] = __float_as_uint(y[4 * k + i]);
        } else if constexpr (E == DSA_ELEM_BF16) {
          w[i] = pack_bf16(y[2 * i], y[2 * i + 1]);
        } else {
          const __half2 h = __floats2half2_rn(y[2 * i], y[2 * i + 1]);
          w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
      }
      v[k] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  // The same as four packed pairs.
  DSA_DEV void pairs(uint64_t* x) const {
    float f[8];
    values(f);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = pack2(f[2 * i], f[2 * i + 1]);
  }
  // Adds other columns, each sum rounded once to the type.
  DSA_DEV void add(const Eight& o) {
#pragma unroll
    for (int k = 0; k < kWords; ++k) {
      uint32_t a[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
      const uint32_t b[4] = {o.v[k].x, o.v[k].y, o.v[k].z, o.v[k].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (E == DSA_ELEM_FP32) {
          a[i] = __float_as_uint(__fadd_rn(__uint_as_float(a[i]), __uint_as_float(b[i])));
        } else if constexpr (E == DSA_ELEM_BF16) {
          const __nv_bfloat162 s = __hadd2_rn(*reinterpret_cast<const __nv_bfloat162*>(&a[i]), *reinterpret_cast<const __nv_bfloat162*>(&b[i]));
          a[i] = *reinterpret_cast<const uint32_t*>(&s);
        } else {
          const __half2 s = __hadd2_rn(*reinterpret_cast<const __half2*>(&a[i]), *reinterpret_cast<const __half2*>(&b[i]));
          a[i] = *reinterpret_cast<const uint32_t*>(&s);
        }
      }
      v[k] = make_uint4(a[0], a[1], a[2], a[3]);
    }
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
  Eight<E> v;
  v.round(y);
  v.store(base, at);
}

DSA_DEV uint32_t e4m3x2(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

DSA_DEV float e4m3_value(uint32_t code) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)code, __NV_E4M3);
  return __half2float(*reinterpret_cast<const __half*>(&h));
}

// The quotient lies between x inv kDown and x inv kUp: inv is off by 2^-23 of itself and the two products by 2^-24 each;
// x is exact, or after a norm off by 2^-23 (its product with 1 / sqrt as one float, and what that float leaves).  3 * 2^-23
// in all, of 4.
constexpr float kDown = 1.f - 0x1p-21f, kUp = 1.f + 0x1p-21f;

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
  const float down = inv * kDown, up = inv * kUp;
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

// Eight columns (packed pairs) x and their factors down and up, about 1 / s on either side -> the codes toward zero, and in
// `open` the columns that have another: two codes that differ by one differ in their last bit, and column i's, the j-th
// four's (i & 3)-th, gets bit 8 (i & 3) + j.
DSA_DEV uint2 codes8(const uint64_t* x, uint64_t down, uint64_t up, int j, uint32_t& open) {
  uint32_t word[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    uint32_t lo[2], hi[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 l = unpack2(mul2(x[2 * k + i], down)), h = unpack2(mul2(x[2 * k + i], up));
      lo[i] = e4m3x2(l.x, l.y);
      hi[i] = e4m3x2(h.x, h.y);
    }
    word[k] = __byte_perm(lo[0], lo[1], 0x5410);
    open |= ((word[k] ^ __byte_perm(hi[0], hi[1], 0x5410)) & 0x01010101u) << (j + k);
  }
  return make_uint2(word[0], word[1]);
}

// Largest finite magnitude of sixteen columns: a NaN (which every maximum loses) or an infinity does not cost
// its neighbours.
DSA_DEV float finite_max16(const float* x) {
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < 16; i += 2) a = max3(a, fabsf(x[i]), fabsf(x[i + 1]));
  if (a == INFINITY) {
    a = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) a = fmaxf(a, fabsf(x[i]) < INFINITY ? fabsf(x[i]) : 0.f);
  }
  return a;
}

// About 1 / s, within 2^-23.
DSA_DEV float fast_inverse(float s) {
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
  return inv;
}

}  // namespace dsa
