// fp8.h -- e4m3 values with power-of-two block scales (e8m0), and 8-element
// accesses of rows that need not be aligned.
#pragma once

#include "dev_math.h"

namespace mssm {

// Columns that share one scale.
constexpr int kScaleBlock = 128;

// Biased exponent of the smallest power of two s with amax / s <= 448, the
// largest finite e4m3 value.  448 is 1.75 * 2^8, so with amax = m * 2^e and m
// in [1, 2) s is 2^(e-8) up to m = 1.75 and 2^(e-7) above it: adding the
// mantissa's distance from 0.75 to 1 (less one unit) carries into the
// exponent exactly there.  An all-zero block gets the smallest scale.  A
// power of two divides the values without rounding them, and the matrix
// instructions take such scales themselves.
__device__ __forceinline__ uint32_t scale_code(float amax) {
  const int32_t c = (int32_t)((__float_as_uint(amax) + 0x1FFFFFu) >> 23) - 8;
  return (uint32_t)max(c, 0);
}
// 1 / s.  amax is finite, so the code is at most 247 and the power normal.
__device__ __forceinline__ float scale_inverse(uint32_t code) {
  return __uint_as_float((254u - code) << 23);
}

// An infinity has no e4m3 value; it becomes NaN here, so that it neither
// decides a block's scale (fmaxf passes NaN over) nor saturates.
__device__ __forceinline__ float finite_or_nan(float v) {
  return fabsf(v) <= 3.402823466e38f ? v : __builtin_nanf("");
}

// Four values within +-448 (or NaN) to e4m3, round to nearest even.
__device__ __forceinline__ uint32_t pack_fp8x4(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
  return (uint32_t)w;
}

// Wide accesses at any element's alignment: the type's alignment of 1 lets
// the compiler use one global access of its full width, which gfx950 takes at
// every byte address.
struct __attribute__((packed, aligned(1))) Any4 { uint32_t w; };
struct __attribute__((packed, aligned(1))) Any8 { uint32_t w[2]; };
struct __attribute__((packed, aligned(1))) Any16 { uint32_t w[4]; };

// v[0..7] = p[i..i+7], the values past `n` >= 1 of them zero.  (Written without
// loops: an array filled in loops of two branches was put into scratch memory.)
template <bool BF16>
__device__ __forceinline__ void load8(float (&v)[8], const void* p, int64_t i, int n) {
  uint32_t w0, w1, w2, w3, w4, w5, w6, w7;
  if constexpr (BF16) {
    const uint16_t* q = static_cast<const uint16_t*>(p) + i;
    if (n >= 8) {
      const Any16 a = *reinterpret_cast<const Any16*>(q);
      w0 = a.w[0], w1 = a.w[1], w2 = a.w[2], w3 = a.w[3];
    } else {
      const auto at = [&](int j) { return j < n ? (uint32_t)q[min(j, n - 1)] : 0u; };
      w0 = at(0) | at(1) << 16, w1 = at(2) | at(3) << 16;
      w2 = at(4) | at(5) << 16, w3 = at(6);
    }
    v[0] = bf16_lo(w0), v[1] = bf16_hi(w0), v[2] = bf16_lo(w1), v[3] = bf16_hi(w1);
    v[4] = bf16_lo(w2), v[5] = bf16_hi(w2), v[6] = bf16_lo(w3), v[7] = bf16_hi(w3);
  } else {
    const uint32_t* q = static_cast<const uint32_t*>(p) + i;
    if (n >= 8) {
      const Any16 a = reinterpret_cast<const Any16*>(q)[0];
      const Any16 b = reinterpret_cast<const Any16*>(q)[1];
      w0 = a.w[0], w1 = a.w[1], w2 = a.w[2], w3 = a.w[3];
      w4 = b.w[0], w5 = b.w[1], w6 = b.w[2], w7 = b.w[3];
    } else {
      const auto at = [&](int j) { return j < n ? q[min(j, n - 1)] : 0u; };
      w0 = at(0), w1 = at(1), w2 = at(2), w3 = at(3), w4 = at(4), w5 = at(5), w6 = at(6), w7 = 0;
    }
    v[0] = __uint_as_float(w0), v[1] = __uint_as_float(w1), v[2] = __uint_as_float(w2);
    v[3] = __uint_as_float(w3), v[4] = __uint_as_float(w4), v[5] = __uint_as_float(w5);
    v[6] = __uint_as_float(w6), v[7] = __uint_as_float(w7);
  }
}

// 8 elements as they lie in memory, for loads that are to be in flight together.
template <bool BF16>
struct Raw8 {
  Any16 a[BF16 ? 1 : 2];
};
template <bool BF16>
__device__ __forceinline__ Raw8<BF16> load_raw8(const void* p, int64_t i) {
  return *reinterpret_cast<const Raw8<BF16>*>(static_cast<const char*>(p) + i * (BF16 ? 2 : 4));
}
template <bool BF16>
__device__ __forceinline__ void unpack8(float (&v)[8], const Raw8<BF16>& r) {
  if constexpr (BF16) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = bf16_lo(r.a[0].w[j]);
      v[2 * j + 1] = bf16_hi(r.a[0].w[j]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(r.a[j >> 2].w[j & 3]);
  }
}

template <bool BF16>
__device__ __forceinline__ void store8(void* p, int64_t i, int n, const float (&v)[8]) {
  if constexpr (BF16) {
    uint16_t* q = static_cast<uint16_t*>(p) + i;
    if (n >= 8) {
      Any16 a;
#pragma unroll
      for (int j = 0; j < 4; ++j) a.w[j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
      *reinterpret_cast<Any16*>(q) = a;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < n) q[j] = to_bf16(v[j]);
    }
  } else {
    float* q = static_cast<float*>(p) + i;
    if (n >= 8) {
      Any16 a, b;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        a.w[j] = __float_as_uint(v[j]);
        b.w[j] = __float_as_uint(v[4 + j]);
      }
      reinterpret_cast<Any16*>(q)[0] = a;
      reinterpret_cast<Any16*>(q)[1] = b;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < n) q[j] = v[j];
    }
  }
}

// The same past the caches, for results too many to be found there again.
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(1)));
template <bool BF16>
__device__ __forceinline__ void store8_past(void* p, int64_t i, int n, const float (&v)[8]) {
  if (n < 8) {
    store8<BF16>(p, i, n, v);
  } else if constexpr (BF16) {
    const u32x4_any a = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                         pack_bf16x2(v[6], v[7])};
    __builtin_nontemporal_store(a, reinterpret_cast<u32x4_any*>(static_cast<uint16_t*>(p) + i));
  } else {
    u32x4_any* q = reinterpret_cast<u32x4_any*>(static_cast<float*>(p) + i);
    const u32x4_any a = {__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                         __float_as_uint(v[3])};
    const u32x4_any b = {__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]),
                         __float_as_uint(v[7])};
    __builtin_nontemporal_store(a, q);
    __builtin_nontemporal_store(b, q + 1);
  }
}

__device__ __forceinline__ void store8_fp8(uint8_t* p, int n, uint32_t lo, uint32_t hi) {
  if (n >= 8) {
    *reinterpret_cast<Any8*>(p) = Any8{{lo, hi}};
  } else {
    const uint64_t w = (uint64_t)hi << 32 | lo;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) p[j] = (uint8_t)(w >> (8 * j));
  }
}

// Largest / sum over aligned groups of 16 lanes (DPP moves inside a row of 16
// lanes: a quad's lanes, then the mirrored lane of each 8 and of each 16),
// every lane getting the result; fmaxf passes a NaN over.
template <int CTRL>
__device__ __forceinline__ float dpp_row(float v) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xF, 0xF, true));
}
__device__ __forceinline__ float max16(float v) {
  v = fmaxf(v, dpp_row<0xB1>(v));
  v = fmaxf(v, dpp_row<0x4E>(v));
  v = fmaxf(v, dpp_row<0x141>(v));
  return fmaxf(v, dpp_row<0x140>(v));
}
__device__ __forceinline__ float sum16(float v) {
  v += dpp_row<0xB1>(v);
  v += dpp_row<0x4E>(v);
  v += dpp_row<0x141>(v);
  return v + dpp_row<0x140>(v);
}
__device__ __forceinline__ float sum64(float v) {
  v = sum16(v);
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}

}  // namespace mssm
