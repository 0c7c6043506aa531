// fp8_matmul.hip -- the product of two e4m3 matrices with a power-of-two
// scale for each block of 128 along the summed axis:
//
//   out[m, n] = sum_kb sa[m, kb] sb[n', kb] sum_{k in block kb} a[m, k] b[n, k]
//
// a is (M, K), b is (N, K) (a linear layer's weight as it is stored), n' is n
// or the 128-row block of n.  The scales go into the matrix instruction
// (v_mfma_scale_f32_*_f8f6f4), which multiplies them into the products it adds
// to the fp32 sums: no scaling pass and no second set of sums.
//
// An 8-bit matrix instruction aligns its products to the largest of them and
// keeps about 18 bits below it: sums of random products came out 1.5e-5 of
// their size off (32x32x64 and 16x16x128 alike, and the older 8-bit forms),
// against 3e-8 for the bf16 instructions.  That is 1/100 of a bf16 result's
// own rounding, so bf16 outputs use it; an fp32 output is wanted for its
// precision, and there the e4m3 values are widened to bf16, scale included
// (exact: 4 significant bits and a power of two), and multiplied by the bf16
// instructions at half the rate.
//
// b's rows are the instruction's rows and a's its columns, so that a lane
// ends with neighbouring n of one m.  Both operands put the same k in the same
// lane and register, and a whole block of 128 has one scale, so any order of
// k inside the block gives the same sum.
#include "fp8.h"
#include "mssm_internal.h"

namespace mssm {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

union Frag {
  i32x8 v;
  i32x4 h[2];
};

__device__ __forceinline__ f32x16 mfma32(const Frag& a, const Frag& b, f32x16 c, int sa, int sb) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a.v, b.v, c, 0, 0, 0, sa, 0, sb);
}
__device__ __forceinline__ f32x4 mfma16(const Frag& a, const Frag& b, f32x4 c, int sa, int sb) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a.v, b.v, c, 0, 0, 0, sa, 0, sb);
}

// The scale of an e8m0 byte as fp32.
__device__ __forceinline__ float scale_value(int code) {
  return __uint_as_float(code ? (uint32_t)code << 23 : 0x00400000u);
}

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2v __attribute__((ext_vector_type(2)));

// Values 8q .. 8q+7 of a fragment in bf16, times its scale.
__device__ __forceinline__ bf16x8 widen8(const Frag& f, int q, float s) {
  union {
    bf16x2v h[4];
    bf16x8 v;
  } u;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t w = (uint32_t)f.v[2 * q + i];
    u.h[2 * i] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, false);
    u.h[2 * i + 1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, true);
  }
  return u.v;
}

// 16 bytes of a row at column k, zeros from K on.
__device__ __forceinline__ i32x4 load16(const uint8_t* row, int64_t k, int64_t K) {
  const int64_t n = K - k;
  if (n >= 16) {
    const Any16 a = *reinterpret_cast<const Any16*>(row + k);
    return i32x4{(int)a.w[0], (int)a.w[1], (int)a.w[2], (int)a.w[3]};
  }
  uint32_t w[4] = {0, 0, 0, 0};
  for (int i = 0; i < 16; ++i)
    if (i < n) w[i >> 2] |= (uint32_t)row[k + i] << (8 * (i & 3));
  return i32x4{(int)w[0], (int)w[1], (int)w[2], (int)w[3]};
}

template <bool BF16>
__device__ __forceinline__ void store4(void* out, int64_t at, int n, float a, float b, float c,
                                       float d) {
  if constexpr (BF16) {
    uint16_t* p = static_cast<uint16_t*>(out) + at;
    if (n >= 4) {
      *reinterpret_cast<Any8*>(p) = Any8{{pack_bf16x2(a, b), pack_bf16x2(c, d)}};
    } else {
      if (n > 0) p[0] = to_bf16(a);
      if (n > 1) p[1] = to_bf16(b);
      if (n > 2) p[2] = to_bf16(c);
    }
  } else {
    float* p = static_cast<float*>(out) + at;
    if (n >= 4) {
      *reinterpret_cast<Any16*>(p) = Any16{{__float_as_uint(a), __float_as_uint(b),
                                            __float_as_uint(c), __float_as_uint(d)}};
    } else {
      if (n > 0) p[0] = a;
      if (n > 1) p[1] = b;
      if (n > 2) p[2] = c;
    }
  }
}

// ---------------------------------------------------------------- few rows of a
//
// A workgroup takes 16 rows of b and all of a's rows (MT tiles of 16); its 8
// waves take every 8th block of 128, straight from memory into the
// instruction's registers, and their sums meet in LDS.  b is read once: its
// bytes bound the kernel.
constexpr int kFewWaves = 8;

template <bool BF16, int MT>
__global__ void __launch_bounds__(64 * kFewWaves) fp8_few_kernel(MatmulParams p) {
  __shared__ float part[kFewWaves][MT][64][4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const int64_t kbs = (p.K + kScaleBlock - 1) / kScaleBlock;
  // rows past the last read the last one; what they give is not stored
  const int64_t nr = min(n0 + (lane & 15), p.N - 1);
  const uint8_t* brow = p.b + nr * p.K;
  const uint8_t* bs = p.b_scales + (nr / p.b_rows) * kbs;
  const uint8_t* arow[MT];
  const uint8_t* as[MT];
  f32x4 acc[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int64_t m = min((int64_t)i * 16 + (lane & 15), p.M - 1);
    arow[i] = p.a + m * p.K;
    as[i] = p.a_scales + m * kbs;
    acc[i] = f32x4{0, 0, 0, 0};
  }
  for (int64_t kb = wave; kb < kbs; kb += kFewWaves) {
    const int64_t k = kb * kScaleBlock + (lane >> 4) * 32;
    Frag b, a[MT];
    b.h[0] = load16(brow, k, p.K);
    b.h[1] = load16(brow, k + 16, p.K);
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      a[i].h[0] = load16(arow[i], k, p.K);
      a[i].h[1] = load16(arow[i], k + 16, p.K);
    }
    const int sb = bs[kb];
    if constexpr (BF16) {
#pragma unroll
      for (int i = 0; i < MT; ++i) acc[i] = mfma16(b, a[i], acc[i], sb, as[i][kb]);
    } else {
      float sa[MT];
#pragma unroll
      for (int i = 0; i < MT; ++i) sa[i] = scale_value(as[i][kb]);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const bf16x8 bw = widen8(b, q, scale_value(sb));
#pragma unroll
        for (int i = 0; i < MT; ++i)
          acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bw, widen8(a[i], q, sa[i]), acc[i], 0, 0, 0);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) part[wave][i][lane][j] = acc[i][j];
  __syncthreads();
  if (wave >= MT) return;
  float s[4] = {0, 0, 0, 0};
#pragma unroll
  for (int w = 0; w < kFewWaves; ++w)
#pragma unroll
    for (int j = 0; j < 4; ++j) s[j] += part[w][wave][lane][j];
  const int64_t m = wave * 16 + (lane & 15), n = n0 + 4 * (lane >> 4);
  if (m < p.M && n < p.N)
    store4<BF16>(p.out, m * p.N + n, (int)min((int64_t)4, p.N - n), s[0], s[1], s[2], s[3]);
}

// ---------------------------------------------------------------- tiles
//
// A workgroup of WM x WN waves takes a BM x BN tile of out, in steps of one
// block of 128 along k.  A step's BM + BN rows of 128 bytes are staged in LDS
// in two buffers, the next step's loads in flight while this one's products
// run.  A row is 8 pieces of 16 bytes; row r keeps piece c in place
// c ^ ((r >> 1) & 7), so that the same piece of 16 neighbouring rows covers all
// 64 banks.
template <int BM, int BN, int WM, int WN>
struct Tile {
  static constexpr int kWaves = WM * WN, kThreads = 64 * kWaves;
  static constexpr int kRows = BM + BN;           // a's rows, then b's
  static constexpr int kFm = BM / WM / 32, kFn = BN / WN / 32;
  static constexpr int kPieces = kRows * 8 / kThreads;  // 16-byte pieces a thread stages
};

__device__ __forceinline__ int piece_at(int row, int c) {
  return row * 128 + ((c ^ ((row >> 1) & 7)) << 4);
}

template <bool BF16, int BM, int BN, int WM, int WN>
__global__ void __launch_bounds__(64 * WM * WN) fp8_tile_kernel(MatmulParams p) {
  using T = Tile<BM, BN, WM, WN>;
  __shared__ __attribute__((aligned(16))) uint8_t lds[2][T::kRows * 128];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t tiles_m = (p.M + BM - 1) / BM;
  const int64_t m0 = (int64_t)(blockIdx.x % tiles_m) * BM, n0 = (int64_t)(blockIdx.x / tiles_m) * BN;
  const int wm = (wave % WM) * (BM / WM), wn = (wave / WM) * (BN / WN);
  const int64_t kbs = (p.K + kScaleBlock - 1) / kScaleBlock;

  auto stage = [&](int64_t kb, uint8_t* to) {
#pragma unroll
    for (int i = 0; i < T::kPieces; ++i) {
      const int at = i * T::kThreads + threadIdx.x;
      const int row = at >> 3, c = at & 7;
      const bool isa = row < BM;
      const int64_t g = isa ? m0 + row : n0 + row - BM;
      i32x4 v = i32x4{0, 0, 0, 0};
      if (g < (isa ? p.M : p.N))
        v = load16((isa ? p.a : p.b) + g * p.K, kb * kScaleBlock + c * 16, p.K);
      *reinterpret_cast<i32x4*>(to + piece_at(row, c)) = v;
    }
  };

  const uint8_t* as[T::kFm];
  const uint8_t* bs[T::kFn];
#pragma unroll
  for (int i = 0; i < T::kFm; ++i)
    as[i] = p.a_scales + min(m0 + wm + 32 * i + (lane & 31), p.M - 1) * kbs;
#pragma unroll
  for (int j = 0; j < T::kFn; ++j)
    bs[j] = p.b_scales + min(n0 + wn + 32 * j + (lane & 31), p.N - 1) / p.b_rows * kbs;

  f32x16 acc[T::kFm][T::kFn];
#pragma unroll
  for (int i = 0; i < T::kFm; ++i)
#pragma unroll
    for (int j = 0; j < T::kFn; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

  stage(0, lds[0]);
  __syncthreads();
  for (int64_t kb = 0; kb < kbs; ++kb) {
    if (kb + 1 < kbs) stage(kb + 1, lds[(kb + 1) & 1]);
    const uint8_t* at = lds[kb & 1];
    int sa[T::kFm], sb[T::kFn];
#pragma unroll
    for (int i = 0; i < T::kFm; ++i) sa[i] = as[i][kb];
#pragma unroll
    for (int j = 0; j < T::kFn; ++j) sb[j] = bs[j][kb];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      Frag a[T::kFm], b[T::kFn];
      const int c = 4 * h + 2 * (lane >> 5);
#pragma unroll
      for (int i = 0; i < T::kFm; ++i) {
        const int row = wm + 32 * i + (lane & 31);
        a[i].h[0] = *reinterpret_cast<const i32x4*>(at + piece_at(row, c));
        a[i].h[1] = *reinterpret_cast<const i32x4*>(at + piece_at(row, c + 1));
      }
#pragma unroll
      for (int j = 0; j < T::kFn; ++j) {
        const int row = BM + wn + 32 * j + (lane & 31);
        b[j].h[0] = *reinterpret_cast<const i32x4*>(at + piece_at(row, c));
        b[j].h[1] = *reinterpret_cast<const i32x4*>(at + piece_at(row, c + 1));
      }
      if constexpr (BF16) {
#pragma unroll
        for (int i = 0; i < T::kFm; ++i)
#pragma unroll
          for (int j = 0; j < T::kFn; ++j) acc[i][j] = mfma32(b[j], a[i], acc[i][j], sb[j], sa[i]);
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          bf16x8 aw[T::kFm], bw[T::kFn];
#pragma unroll
          for (int i = 0; i < T::kFm; ++i) aw[i] = widen8(a[i], q, scale_value(sa[i]));
#pragma unroll
          for (int j = 0; j < T::kFn; ++j) bw[j] = widen8(b[j], q, scale_value(sb[j]));
#pragma unroll
          for (int i = 0; i < T::kFm; ++i)
#pragma unroll
            for (int j = 0; j < T::kFn; ++j)
              acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(bw[j], aw[i], acc[i][j], 0, 0, 0);
        }
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < T::kFm; ++i) {
    const int64_t m = m0 + wm + 32 * i + (lane & 31);
    if (m >= p.M) continue;
#pragma unroll
    for (int j = 0; j < T::kFn; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int64_t n = n0 + wn + 32 * j + 8 * q + 4 * (lane >> 5);
        if (n < p.N)
          store4<BF16>(p.out, m * p.N + n, (int)min((int64_t)4, p.N - n), acc[i][j][4 * q],
                       acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]);
      }
  }
}

template <bool BF16, int BM, int BN, int WM, int WN>
void launch_tile(const MatmulParams& p, hipStream_t st) {
  const int64_t tiles = ((p.M + BM - 1) / BM) * ((p.N + BN - 1) / BN);
  hipLaunchKernelGGL((fp8_tile_kernel<BF16, BM, BN, WM, WN>), dim3((unsigned)tiles),
                     dim3(64 * WM * WN), 0, st, p);
}

template <bool BF16>
void launch(const MatmulParams& p, hipStream_t st) {
  if (p.M <= 64) {
    const dim3 grid((unsigned)((p.N + 15) / 16)), block(64 * kFewWaves);
    if (p.M <= 16) hipLaunchKernelGGL((fp8_few_kernel<BF16, 1>), grid, block, 0, st, p);
    else if (p.M <= 32) hipLaunchKernelGGL((fp8_few_kernel<BF16, 2>), grid, block, 0, st, p);
    else hipLaunchKernelGGL((fp8_few_kernel<BF16, 4>), grid, block, 0, st, p);
    return;
  }
  launch_tile<BF16, 128, 128, 2, 2>(p, st);
}

}  // namespace

hipError_t launch_fp8_matmul(const MatmulParams& p, bool bf16, hipStream_t st) {
  bf16 ? launch<true>(p, st) : launch<false>(p, st);
  return hipGetLastError();
}

}  // namespace mssm
