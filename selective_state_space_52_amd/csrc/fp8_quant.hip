// fp8_quant.hip -- values to e4m3 with one power-of-two scale (e8m0) for each
// block of 128 along a row, of 128 down a column (the output transposed), or
// of 128 x 128.
//
//   s = the smallest power of two with max |block| / s <= 448;  q = e4m3(x / s)
//
// The division is by a power of two, so each value is rounded once.  An
// infinity becomes NaN; it and NaN leave the block's scale alone.  The
// kernels read and write each value once: HBM bounds large ones along rows (4096 x
// 3352 bf16: 8.7 us, 4.7 TB/s).  A workgroup of the others loads, waits and stores
// its 128 rows once: 12 us transposed (15 with the workgroups in row order), 12.7 for
// 128 x 128 blocks, 9.8 for those transposed, 3.2 to 4.2 TB/s.
#include "fp8.h"
#include "mssm_internal.h"

namespace mssm {
namespace {

// Blocks along a row: 8 neighbouring columns a thread, 16 threads a block.
template <bool BF16>
__global__ void __launch_bounds__(256) quant_rows_kernel(QuantParams p) {
  const int64_t block = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
  const int64_t kb = (p.cols + kScaleBlock - 1) / kScaleBlock;
  if (block >= p.rows * kb) return;  // the 16 lanes of a block together
  const int64_t row = block / kb;
  const int64_t col = (block - row * kb) * kScaleBlock + (threadIdx.x & 15) * 8;
  const int n = (int)min((int64_t)8, p.cols - col);
  float v[8];
  float amax = 0.0f;
  if (n > 0) load8<BF16>(v, p.x, row * p.x_stride + col, n);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    v[j] = n > 0 ? finite_or_nan(v[j]) : 0.0f;
    amax = fmaxf(amax, fabsf(v[j]));
  }
  const uint32_t code = scale_code(max16(amax));
  const float inv = scale_inverse(code);
  if (n > 0)
    store8_fp8(p.q + row * p.cols + col, n,
               pack_fp8x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
               pack_fp8x4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
  if ((threadIdx.x & 15) == 0) p.scales[block] = (uint8_t)code;
}

// A tile of 128 rows a workgroup: thread (r, g) holds rows 4r..4r+3 of columns
// 8g..8g+7, so that four rows of a column pack into one word of the
// transposed tile, which is turned in LDS.  A pitch of 33 words puts the 8 x 8
// lanes of a wave's store on 64 banks.
// SQUARE: 128 columns and one scale for them all; else 64, a scale for each.
template <bool BF16, bool SQUARE, bool TRANSPOSE>
__global__ void __launch_bounds__(SQUARE ? 512 : 256) quant_tile_kernel(QuantParams p) {
  constexpr int kPitch = 33, kWide = SQUARE ? 2 : 1, kCols = 64 * kWide;
  __shared__ float part[8][kCols];
  __shared__ uint32_t tile[TRANSPOSE ? kCols * kPitch : 1];
  // lanes: 8 column groups by 8 row groups; waves: kWide by 4
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int g = (lane & 7) + 8 * (wave % kWide), r = (lane >> 3) + 8 * (wave / kWide);
  // down the columns first where the output is transposed: workgroups side by
  // side would write at multiples of the row count, often of the same channel
  const int64_t tiles_c = (p.cols + kCols - 1) / kCols;
  const int64_t tall = (p.rows + kScaleBlock - 1) / kScaleBlock;
  const int64_t tr = TRANSPOSE ? blockIdx.x % tall : blockIdx.x / tiles_c;
  const int64_t tc = TRANSPOSE ? blockIdx.x / tall : blockIdx.x - tr * tiles_c;
  const int64_t row0 = tr * kScaleBlock, col0 = tc * kCols;
  const int64_t row = row0 + 4 * r, col = col0 + 8 * g;
  const int n = (int)min((int64_t)8, p.cols - col);
  float v[4][8], amax[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) amax[j] = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool in = n > 0 && row + i < p.rows;
    if (in) load8<BF16>(v[i], p.x, (row + i) * p.x_stride + col, n);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[i][j] = in ? finite_or_nan(v[i][j]) : 0.0f;
      amax[j] = fmaxf(amax[j], fabsf(v[i][j]));
    }
  }
  if constexpr (SQUARE) {
    float m = amax[0];
#pragma unroll
    for (int j = 1; j < 8; ++j) m = fmaxf(m, amax[j]);
#pragma unroll
    for (int d = 1; d < 64; d *= 2) m = fmaxf(m, __shfl_xor(m, d));
    if (lane == 0) part[0][wave] = m;
    __syncthreads();
    m = part[0][0];
    for (int w = 1; w < 8; ++w) m = fmaxf(m, part[0][w]);
#pragma unroll
    for (int j = 0; j < 8; ++j) amax[j] = m;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
#pragma unroll
      for (int d = 8; d < 64; d *= 2) amax[j] = fmaxf(amax[j], __shfl_xor(amax[j], d));
      if (lane < 8) part[wave / kWide][8 * g + j] = amax[j];
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      amax[j] = part[0][8 * g + j];
#pragma unroll
      for (int w = 1; w < 4; ++w) amax[j] = fmaxf(amax[j], part[w][8 * g + j]);
    }
  }
  uint32_t code[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    code[j] = scale_code(amax[j]);
    const float inv = scale_inverse(code[j]);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i][j] *= inv;
  }
  if constexpr (SQUARE) {
    if (threadIdx.x == 0)
      p.scales[TRANSPOSE ? tc * tall + tr : (int64_t)blockIdx.x] = (uint8_t)code[0];
  } else if (r == 0) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) p.scales[(col + j) * tall + tr] = (uint8_t)code[j];
  }
  if constexpr (!TRANSPOSE) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n > 0 && row + i < p.rows)
        store8_fp8(p.q + (row + i) * p.cols + col, n,
                   pack_fp8x4(v[i][0], v[i][1], v[i][2], v[i][3]),
                   pack_fp8x4(v[i][4], v[i][5], v[i][6], v[i][7]));
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      tile[(8 * g + j) * kPitch + r] = pack_fp8x4(v[0][j], v[1][j], v[2][j], v[3][j]);
    __syncthreads();
    // 8 16-byte pieces a column, two a thread
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int c = (threadIdx.x >> 3) + kCols / 2 * k, piece = threadIdx.x & 7;
      const int64_t at = row0 + 16 * piece;
      const int left = (int)min((int64_t)16, p.rows - at);
      if (col0 + c >= p.cols || left <= 0) continue;
      Any16 w;
#pragma unroll
      for (int q = 0; q < 4; ++q) w.w[q] = tile[c * kPitch + 4 * piece + q];
      uint8_t* to = p.q + (col0 + c) * p.rows + at;
      if (left == 16) {
        *reinterpret_cast<Any16*>(to) = w;
      } else {
#pragma unroll
        for (int b = 0; b < 16; ++b)
          if (b < left) to[b] = (uint8_t)(w.w[b >> 2] >> (8 * (b & 3)));
      }
    }
  }
}

template <bool BF16>
void launch(const QuantParams& p, hipStream_t st) {
  const int64_t kb = (p.cols + kScaleBlock - 1) / kScaleBlock;
  const int64_t tall = (p.rows + kScaleBlock - 1) / kScaleBlock;
  const int64_t tiles = kb * tall, halves = tall * ((p.cols + 63) / 64);
  if (!p.square && !p.transpose)
    hipLaunchKernelGGL((quant_rows_kernel<BF16>), dim3((unsigned)((p.rows * kb + 15) / 16)),
                       dim3(256), 0, st, p);
  else if (!p.square)
    hipLaunchKernelGGL((quant_tile_kernel<BF16, false, true>), dim3((unsigned)halves), dim3(256), 0,
                       st, p);
  else if (p.transpose)
    hipLaunchKernelGGL((quant_tile_kernel<BF16, true, true>), dim3((unsigned)tiles), dim3(512), 0,
                       st, p);
  else
    hipLaunchKernelGGL((quant_tile_kernel<BF16, true, false>), dim3((unsigned)tiles), dim3(512), 0,
                       st, p);
}

}  // namespace

hipError_t launch_quantize_fp8(const QuantParams& p, bool bf16, hipStream_t st) {
  bf16 ? launch<true>(p, st) : launch<false>(p, st);
  return hipGetLastError();
}

}  // namespace mssm
