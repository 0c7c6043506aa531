// adamw.hip -- the AdamW step of many tensors in one launch, states in fp32 or
// in 8 bits.  Each value is read and written once: HBM bounds both (129M
// parameters with fp32 states and a bf16 copy 673 us, 209M with 8-bit ones 630: 5.4
// TB/s), the vector ALU the second nearly so.
//
//   m = b1 m + (1 - b1) g;  v = b2 v + (1 - b2) g^2
//   p = p (1 - lr decay) - lr (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps)
//
// The 8-bit states are e4m3 values of m and sqrt(v), not v: the root halves the
// range in powers of two, and e4m3 with a block's scale spans 2^18 below the
// block's largest.  Each block of 128 has an fp32 scale, its largest value times
// 1/448, so that a block whose values all fall by a thousandth does so in its
// scale.  A value goes to one of its two neighbours by a fraction u that has
// each value's mean kept (rounding to nearest would never let a moment move by
// less than half a unit, 3% to 6% of it, in a step).  u walks through the
// elements as a sequence of equal steps modulo 1 (2^32 / golden ratio, and 2^32
// times the root of 2's fraction for the second state), shifted by a hash of
// the seed and the step; for one element it is spread evenly over the steps.
//
// A last bit decides there whether a value moves by a whole unit, a 16th to an 8th
// of itself, which every later step then starts from.  So each fp32 operation from
// the old states and the gradient to the new states is fixed by the definition and
// rounded to nearest: nothing is contracted or approximated on that way, and equal
// inputs give equal states by any route.  (The parameter's step feeds nothing back.)
#include "fp8.h"
#include "mssm_internal.h"

namespace mssm {
namespace {

// 4 elements a thread, so that a wave's accesses are of whole neighbouring lines
// (1 KB of fp32); 32 lanes hold a block.  A workgroup of more passes spreads the
// finding of its tensor over more elements, but its loads wait for the last pass's
// stores: four passes with fp32 states 734 us for 129M elements, one 676; with
// 8-bit states 645 and 641 for 209M.
constexpr int kThreads = 256, kPer = 4;
constexpr int kElements = kThreads * kPer;  // of a workgroup
constexpr int kBlockLanes = kScaleBlock / kPer;
constexpr float kSmallest = 0x1p-100f, kMost8 = 448.0f, kInvMost8 = 1.0f / 448.0f;
constexpr uint32_t kStrideM = 0x9E3779B9u, kStrideV = 0x6A09E667u;

// v[0..3] = p[i..i+3], the values past `n` >= 1 of them zero.
template <bool BF16>
__device__ __forceinline__ void load4(float (&v)[4], const void* p, int64_t i, int n) {
  if constexpr (BF16) {
    const uint16_t* q = static_cast<const uint16_t*>(p) + i;
    uint32_t a, b;
    if (n >= 4) {
      const Any8 w = *reinterpret_cast<const Any8*>(q);
      a = w.w[0], b = w.w[1];
    } else {
      a = q[0] | (n > 1 ? (uint32_t)q[1] << 16 : 0u);
      b = n > 2 ? q[2] : 0u;
    }
    v[0] = bf16_lo(a), v[1] = bf16_hi(a), v[2] = bf16_lo(b), v[3] = bf16_hi(b);
  } else {
    const float* q = static_cast<const float*>(p) + i;
    if (n >= 4) {
      const Any16 w = *reinterpret_cast<const Any16*>(q);
      v[0] = __uint_as_float(w.w[0]), v[1] = __uint_as_float(w.w[1]);
      v[2] = __uint_as_float(w.w[2]), v[3] = __uint_as_float(w.w[3]);
    } else {
      v[0] = q[0], v[1] = n > 1 ? q[1] : 0.0f, v[2] = n > 2 ? q[2] : 0.0f, v[3] = 0.0f;
    }
  }
}
// Past the caches: a large step's data are more than they hold, and not read again
// soon.  (Through them 129M parameters 698 us, past them 670; from 6M to 47M the same,
// also with a read of the copy after the step; below, that read is 1 us slower.)
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(1)));
template <bool BF16>
__device__ __forceinline__ void store4(void* p, int64_t i, int n, const float (&v)[4]) {
  if constexpr (BF16) {
    uint16_t* q = static_cast<uint16_t*>(p) + i;
    if (n >= 4) {
      const u32x2_any w = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
      __builtin_nontemporal_store(w, reinterpret_cast<u32x2_any*>(q));
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < n) q[j] = to_bf16(v[j]);
    }
  } else {
    float* q = static_cast<float*>(p) + i;
    if (n >= 4) {
      const u32x4_any w = {__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                           __float_as_uint(v[3])};
      __builtin_nontemporal_store(w, reinterpret_cast<u32x4_any*>(q));
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < n) q[j] = v[j];
    }
  }
}

struct Rates {
  float lr, grad_scale, inv_c1, inv_c2;
  uint32_t shift_m, shift_v;
};
__device__ __forceinline__ Rates rates_of(const AdamParams& p) {
  Rates r;
  r.lr = p.lr_value ? *p.lr_value : p.lr;
  r.grad_scale = p.grad_scale_value ? *p.grad_scale_value : p.grad_scale;
  r.inv_c1 = p.inv_c1;
  r.inv_c2 = p.inv_c2;
  int64_t step = p.step;
  if (p.step_value) {
    step = *p.step_value;
    // 1 - b^t; expm1 keeps its digits where b^t is close to 1
    r.inv_c1 = 1.0f / -expm1f((float)step * p.log_beta1);
    r.inv_c2 = 1.0f / sqrtf(-expm1f((float)step * p.log_beta2));
  }
  uint64_t x = (p.seed + (uint64_t)step) * 0x9E3779B97F4A7C15ull;
  x = (x ^ x >> 32) * 0x6A09E667F3BCC909ull;
  x ^= x >> 32;
  r.shift_m = (uint32_t)x;
  r.shift_v = (uint32_t)(x >> 32);
  return r;
}

__device__ __forceinline__ void load4_fp8(float (&v)[4], const void* p, int64_t i) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  const int w = *reinterpret_cast<const int*>(static_cast<const uint8_t*>(p) + i);
  const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(w, false);
  const f32x2 b = __builtin_amdgcn_cvt_pk_f32_fp8(w, true);
  v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
}

// x, of the block that 32 neighbouring lanes hold, as e4m3 at p + i.  CAREFUL: with
// infinities or NaN among them, which become NaN and leave the block's scale
// alone.  (The vector ALU is what the 8-bit step has least of: 109 instructions an
// element with these cases everywhere and the compiler's root, 668 us for 209M
// elements; 92 and 635 with them, and roots below 2^-48, in the waves that hold any.)
template <bool POSITIVE, bool CAREFUL>
__device__ __forceinline__ void store4_rounded(void* p, float* scales, int64_t i,
                                               const float (&x)[4], uint32_t u, uint32_t stride) {
  float most = 0.0f;
#pragma unroll
  for (int j = 0; j < 4; ++j) most = fmaxf(most, fabsf(CAREFUL ? finite_or_nan(x[j]) : x[j]));
  most = max16(most);
  most = fmaxf(most, __shfl_xor(most, 16));
  if (most < kSmallest) most = 0.0f;
  const float up = most > 0.0f ? kMost8 * (1.0f / most) : 0.0f;
  if ((threadIdx.x & (kBlockLanes - 1)) == 0) scales[i / kScaleBlock] = most * kInvMost8;
  float q[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float y = x[j] * up;
    // y's power of two, 2^-6 at least; its unit is an eighth of it (3 mantissa bits)
    const float power = fmaxf(__uint_as_float(__float_as_uint(y) & 0x7F800000u), 0x1p-6f);
    const float per = __uint_as_float(0x80800000u - __float_as_uint(power));  // 8 / power
    const float dither = (float)((u + j * stride) >> 8);
    // |y| per is exact and below 16: one rounding, of the sum
    float units = floorf(fmaf(dither, 0x1p-24f, fabsf(y) * per));
    // a root above zero is 2^-75 or more
    if (POSITIVE) units = fmaxf(units, __builtin_amdgcn_fmed3f(x[j] * 0x1p126f, 0.0f, 1.0f));
    q[j] = fminf(units * (power * 0.125f), kMost8);
    if (!POSITIVE) q[j] = copysignf(q[j], y);
    if (CAREFUL && !(fabsf(x[j]) <= 3.402823466e38f)) q[j] = __builtin_nanf("");
  }
  __builtin_nontemporal_store(pack_fp8x4(q[0], q[1], q[2], q[3]),
                              reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p) + i));
}

__device__ __forceinline__ uint64_t of_lane(uint64_t v, int lane) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, lane);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), lane);
  return (uint64_t)hi << 32 | lo;
}

// The root of x, rounded to nearest: of the hardware's (a unit off at most) and its
// two neighbours the one that x's distance from their products picks.  For 0, and from
// 2^-96 on, below which those distances are not exact.
constexpr uint32_t kLeastSquare = (127u - 96u) << 23;
__device__ __forceinline__ float near_root(float x) {
  const float s = __builtin_amdgcn_sqrtf(x);
  const float down = __uint_as_float(__float_as_uint(s) - 1);
  const float up = __uint_as_float(__float_as_uint(s) + 1);
  const float y = fmaf(-down, s, x) <= 0.0f ? down : s;
  return fmaf(-up, s, x) > 0.0f ? up : y;
}

template <bool EIGHT>
__global__ void __launch_bounds__(kThreads) adamw_kernel(AdamParams p) {
#pragma clang fp contract(off)
  // the tensor whose workgroup this is: the last that begins at or before it.
  // Lane i holds the table's entry i, so that finding the tensor and reading its
  // entry is one wait.
  const int lane = threadIdx.x & 63;
  const int at_most = lane < p.count ? lane : p.count - 1;
  const AdamTensor mine = p.tensors[at_most];
  const uint32_t first = lane < p.count ? p.first[lane] : 0xFFFFFFFFu;
  const int which = __popcll(__ballot(first <= blockIdx.x)) - 1;
  AdamTensor t;
  t.param = (float*)of_lane((uint64_t)mine.param, which);
  t.grad = (const void*)of_lane((uint64_t)mine.grad, which);
  t.copy = (void*)of_lane((uint64_t)mine.copy, which);
  t.size = (int64_t)of_lane((uint64_t)mine.size, which);
  t.at = (int64_t)of_lane((uint64_t)mine.at, which);
  t.decay = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(mine.decay), which));
  t.grad_bf16 = __builtin_amdgcn_readlane(mine.grad_bf16, which);
  const uint32_t begins = (uint32_t)__builtin_amdgcn_readlane((int)first, which);
  const int64_t begin = (int64_t)(blockIdx.x - begins) * kElements;
  const Rates r = rates_of(p);
  const float keep = 1.0f - r.lr * t.decay;
  const int64_t i = begin + threadIdx.x * kPer;
  const int64_t left = t.size - i;
  // the states go on to the end of the last block of 128
  if (begin + (int64_t)(threadIdx.x & ~(kBlockLanes - 1)) * kPer >= t.size) return;
  const int n = (int)min((int64_t)kPer, left);
  float w[4], g[4], m[4], v[4];
  if (n > 0) {
    load4<false>(w, t.param, i, n);
    if (t.grad_bf16)
      load4<true>(g, t.grad, i, n);
    else
      load4<false>(g, t.grad, i, n);
  } else {
#pragma unroll
    for (int j = 0; j < kPer; ++j) w[j] = g[j] = 0.0f;
  }
  const int64_t at = t.at + i;
  if constexpr (EIGHT) {
    load4_fp8(m, p.m, at);
    load4_fp8(v, p.v, at);
    const float ms = p.m_scales[at / kScaleBlock], vs = p.v_scales[at / kScaleBlock];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      m[j] *= ms;
      v[j] *= vs;
      v[j] *= v[j];
    }
  } else {
    load4<false>(m, p.m, at, 4);
    load4<false>(v, p.v, at, 4);
  }
  float root[4], all = 0.0f;
  uint32_t least = 0xFFFFFFFFu;  // the smallest nonzero v's bits, less one
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    // each product rounded by itself, as the definition reads
    const float s = g[j] * r.grad_scale;
    m[j] = m[j] * p.beta1 + s * p.rest1;
    v[j] = v[j] * p.beta2 + s * s * p.rest2;
  }
  if (n < kPer) {  // behind the tensor's end zeros stay zeros, also with a scale of infinity
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (j >= n) m[j] = v[j] = 0.0f;
  }
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    if constexpr (EIGHT) {
      root[j] = near_root(v[j]);
      all = fmaf(m[j], 0.0f, fmaf(v[j], 0.0f, all));
      least = min(least, __float_as_uint(v[j]) - 1);
    } else {
      root[j] = sqrtf(v[j]);
    }
  }
  if constexpr (EIGHT) {
    if (__ballot(least < kLeastSquare - 1)) {
#pragma unroll
      for (int j = 0; j < kPer; ++j) root[j] = sqrtf(v[j]);
    }
  }
  // The parameter's step.  With fp32 states a rounded division, which waits for HBM
  // anyway; with 8-bit ones, whose vector instructions nearly bound the call, a
  // product with the hardware's reciprocal, a unit off at most: 640 us, divided 690.
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const float moved = r.lr * r.inv_c1 * m[j], by = fmaf(root[j], r.inv_c2, p.eps);
    w[j] = EIGHT ? fmaf(-moved, hw_rcp(by), w[j] * keep) : w[j] * keep - moved / by;
  }
  if (n > 0) {
    store4<false>(t.param, i, n, w);
    if (t.copy) store4<true>(t.copy, i, n, w);
  }
  if constexpr (EIGHT) {
    const uint32_t um = r.shift_m + (uint32_t)i * kStrideM, uv = r.shift_v + (uint32_t)i * kStrideV;
    if (__ballot(!(all == 0.0f))) {  // infinity or NaN in this wave
      store4_rounded<false, true>(p.m, p.m_scales, at, m, um, kStrideM);
      store4_rounded<true, true>(p.v, p.v_scales, at, root, uv, kStrideV);
    } else {
      store4_rounded<false, false>(p.m, p.m_scales, at, m, um, kStrideM);
      store4_rounded<true, false>(p.v, p.v_scales, at, root, uv, kStrideV);
    }
  } else {
    store4<false>(p.m, at, 4, m);
    store4<false>(p.v, at, 4, v);
  }
}

}  // namespace

int64_t adamw_block_elements() { return kElements; }

hipError_t launch_adamw(const AdamParams& p, bool eight, hipStream_t st) {
  auto kernel = eight ? adamw_kernel<true> : adamw_kernel<false>;
  hipLaunchKernelGGL(kernel, dim3(p.blocks), dim3(kThreads), 0, st, p);
  return hipGetLastError();
}

}  // namespace mssm
