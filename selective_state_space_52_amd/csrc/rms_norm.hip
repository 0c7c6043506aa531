// rms_norm.hip -- root-mean-square norm with the residual stream's addition,
// its output in the io dtype or as e4m3 with a power-of-two scale for each
// 128 columns, and its backward.
//
// Per row of `dim` columns, in fp32:
//   r    = x + residual                 (written in the residual's dtype)
//   rstd = 1 / sqrt(mean(r^2) + eps)
//   y    = r * rstd * weight
// and for dy = dLoss/dy, ds = dLoss/dr from the stream's later uses:
//   xhat = r * rstd
//   dr   = rstd * (w dy - xhat * mean(w dy xhat)) + ds
//   dw   = sum over rows of dy * xhat
// The sum of squares is of the unrounded r; the backward starts from r as it
// was written.
//
// Both directions read and write each value once, so HBM bounds them: at 8192
// rows of 2560 (bf16 x, fp32 stream) 40 us into 8 bits (5.8 TB/s) and 67 us back
// (5.0 TB/s), where a copy of 512 MB reaches 5.4.  The backward keeps a row's
// values and its columns' sums in registers; above 16384 columns (4 passes of 1024
// threads, 128 registers each) 187 to 275 of them are spilled: 2048 x 16384 124 us,
// 2048 x 32768 497.
#include "fp8.h"
#include "mssm_internal.h"

namespace mssm {
namespace {

// A row belongs to T threads (a multiple of 64), 8 neighbouring columns each
// in each of CH passes, which stay in registers between the sum and the
// output.  16 lanes hold one scale block.  Rows of up to 512 columns take one
// wave and need no barrier; four of them share a workgroup.
constexpr int kMaxThreads = 1024;

__device__ __forceinline__ float row_total(float v, int waves, float* lds) {
  v = sum64(v);
  if (waves == 1) return v;
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.0f;
  for (int i = 0; i < waves; ++i) s += lds[i];
  return s;
}

// RES: 0 no residual, 1 bf16, 2 fp32.
template <bool BF16, int RES, bool FP8, int CH>
__global__ void __launch_bounds__(kMaxThreads) rms_norm_kernel(NormParams p) {
  __shared__ float lds[kMaxThreads / 64];
  const int T = p.threads;
  const int t = T == 64 ? threadIdx.x & 63 : threadIdx.x;
  const int64_t row = T == 64 ? (int64_t)blockIdx.x * (blockDim.x >> 6) + (threadIdx.x >> 6)
                              : (int64_t)blockIdx.x;
  if (row >= p.rows) return;  // whole waves, and only where there is no barrier
  const int dim = p.dim;
  float r[CH][8];
  float ss = 0.0f;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int i = (c * T + t) * 8, n = dim - i;
    if (n > 0) {
      load8<BF16>(r[c], p.x, row * p.x_stride + i, n);
      if constexpr (RES != 0) {
        float q[8];
        load8<RES == 1>(q, p.residual, row * dim + i, n);
#pragma unroll
        for (int j = 0; j < 8; ++j) r[c][j] += q[j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) r[c][j] = 0.0f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(r[c][j], r[c][j], ss);
  }
  const float total = row_total(ss, T >> 6, lds);
  const float rstd = rsqrtf(total * p.inv_dim + p.eps);
  if (p.rstd && t == 0) p.rstd[row] = rstd;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int i = (c * T + t) * 8, n = dim - i;
    float y[8];
    if (n > 0) {
      if (p.residual_out) {
        if constexpr (RES == 1)
          store8<true>(p.residual_out, row * dim + i, n, r[c]);
        else if constexpr (RES == 2)
          store8<false>(p.residual_out, row * dim + i, n, r[c]);
      }
      load8<false>(y, p.weight, i, n);
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] *= r[c][j] * rstd;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = 0.0f;
    }
    if constexpr (FP8) {
      float amax = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        y[j] = finite_or_nan(y[j]);
        amax = fmaxf(amax, fabsf(y[j]));
      }
      const uint32_t code = scale_code(max16(amax));
      const float inv = scale_inverse(code);
      if (n > 0) {
        const uint32_t lo = pack_fp8x4(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv);
        const uint32_t hi = pack_fp8x4(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv);
        store8_fp8(static_cast<uint8_t*>(p.out) + row * dim + i, n, lo, hi);
        if ((t & 15) == 0)
          p.scales[row * p.scale_cols + i / kScaleBlock] = (uint8_t)code;
      }
    } else if (n > 0) {
      store8<BF16>(p.out, row * dim + i, n, y);
    }
  }
}

// The backward's first launch: a workgroup takes every gridDim-th row (each
// of its waves every 4 gridDim-th one for one-wave rows), writes dr, and keeps
// its columns' sums of dy xhat, written as one row of partial sums at its end.
// Two to four workgroups a CU: more of them write more partial sums (768
// workgroups 67 us, 1536: 96 at 8192 x 2560); the next row's loads ahead of
// this one's sum cost registers and gained nothing (92 us).
template <bool BF16, int RES, int CH>
__global__ void __launch_bounds__(kMaxThreads) rms_norm_bwd_kernel(NormBwdParams p) {
  __shared__ float lds[2][kMaxThreads / 64];
  const int T = p.threads;
  const int t = T == 64 ? threadIdx.x & 63 : threadIdx.x;
  const int per = T == 64 ? blockDim.x >> 6 : 1;
  const int64_t first = (int64_t)blockIdx.x * per + (T == 64 ? threadIdx.x >> 6 : 0);
  const int64_t step = (int64_t)gridDim.x * per;
  const int dim = p.dim;
  constexpr bool kKeepW = CH < 4;  // at 4 the weights are read again for each row
  float w[CH][8], dw[CH][8];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int i = (c * T + t) * 8, n = dim - i;
    if (kKeepW && n > 0) load8<false>(w[c], p.weight, i, n);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (n <= 0) w[c][j] = 0.0f;
      dw[c][j] = 0.0f;
    }
  }
  int buf = 0;
  for (int64_t row = first; row < p.rows; row += step) {
    float g[CH][8], xh[CH][8];
    float dot = 0.0f;
    const float rstd = p.rstd[row];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = (c * T + t) * 8, n = dim - i;
      if (n > 0) {
        if (!kKeepW) load8<false>(w[c], p.weight, i, n);
        load8<BF16>(g[c], p.dout, row * dim + i, n);
        load8<RES == 0 ? BF16 : RES == 1>(xh[c], p.r, row * dim + i, n);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) g[c][j] = xh[c][j] = 0.0f;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        xh[c][j] *= rstd;
        dw[c][j] = fmaf(g[c][j], xh[c][j], dw[c][j]);
        g[c][j] *= w[c][j];
        dot = fmaf(g[c][j], xh[c][j], dot);
      }
    }
    // two buffers: a wave may reach the next row's sum while another still
    // reads this one's, but not the one after it
    const float mean = row_total(dot, T >> 6, lds[buf]) * p.inv_dim;
    buf ^= 1;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = (c * T + t) * 8, n = dim - i;
      if (n <= 0) continue;
      float dr[8], ds[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        ds[j] = 0.0f;
        dr[j] = rstd * (g[c][j] - xh[c][j] * mean);
      }
      if constexpr (RES != 0) {
        if (p.dresidual) load8<RES == 1>(ds, p.dresidual, row * dim + i, n);
#pragma unroll
        for (int j = 0; j < 8; ++j) dr[j] += ds[j];
        if (p.dr) store8<RES == 1>(p.dr, row * dim + i, n, dr);
      }
      store8<BF16>(p.dx, row * dim + i, n, dr);
    }
  }
  float* part = p.partial + first * dim;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int i = (c * T + t) * 8, n = dim - i;
    if (n > 0) store8<false>(part, i, n, dw[c]);
  }
}

// The second launch: dw[i] = sum of the partial rows, in a fixed order.  A
// workgroup takes 16 columns, each of its 64 groups of 16 threads every 64th row.
constexpr int kDwCols = 16, kDwGroups = 64;
__global__ void __launch_bounds__(kDwCols* kDwGroups)
    rms_norm_dw_kernel(const float* __restrict__ partial, float* __restrict__ dw, int dim, int rows) {
  __shared__ float lds[kDwGroups][kDwCols + 1];
  const int c = threadIdx.x % kDwCols, part = threadIdx.x / kDwCols;
  const int col = blockIdx.x * kDwCols + c;
  float s = 0.0f;
  if (col < dim) {
#pragma unroll 8
    for (int r = part; r < rows; r += kDwGroups) s += partial[(int64_t)r * dim + col];
  }
  lds[part][c] = s;
  __syncthreads();
  for (int half = kDwGroups / 2; half > 0; half /= 2) {
    if (part < half) lds[part][c] += lds[part + half][c];
    __syncthreads();
  }
  if (part == 0 && col < dim) dw[col] = lds[0][c];
}

struct Shape {
  int threads, chunks, block;
};
Shape shape_of(int dim) {
  const int groups = (dim + 7) / 8;
  const int ch = groups <= kMaxThreads ? 1 : groups <= 2 * kMaxThreads ? 2 : 4;
  const int threads = ((groups + ch - 1) / ch + 63) / 64 * 64;
  return Shape{threads, ch, threads == 64 ? 256 : threads};
}

template <bool BF16, int RES, bool FP8>
void launch_fwd(const NormParams& p, Shape s, dim3 grid, hipStream_t st) {
  if (s.chunks == 1)
    hipLaunchKernelGGL((rms_norm_kernel<BF16, RES, FP8, 1>), grid, dim3(s.block), 0, st, p);
  else if (s.chunks == 2)
    hipLaunchKernelGGL((rms_norm_kernel<BF16, RES, FP8, 2>), grid, dim3(s.block), 0, st, p);
  else
    hipLaunchKernelGGL((rms_norm_kernel<BF16, RES, FP8, 4>), grid, dim3(s.block), 0, st, p);
}
template <bool BF16, int RES>
void launch_fwd(const NormParams& p, Shape s, dim3 grid, hipStream_t st) {
  if (p.scales)
    launch_fwd<BF16, RES, true>(p, s, grid, st);
  else
    launch_fwd<BF16, RES, false>(p, s, grid, st);
}
template <bool BF16, int RES>
void launch_bwd(const NormBwdParams& p, Shape s, dim3 grid, hipStream_t st) {
  if (s.chunks == 1)
    hipLaunchKernelGGL((rms_norm_bwd_kernel<BF16, RES, 1>), grid, dim3(s.block), 0, st, p);
  else if (s.chunks == 2)
    hipLaunchKernelGGL((rms_norm_bwd_kernel<BF16, RES, 2>), grid, dim3(s.block), 0, st, p);
  else
    hipLaunchKernelGGL((rms_norm_bwd_kernel<BF16, RES, 4>), grid, dim3(s.block), 0, st, p);
}

}  // namespace

int rms_norm_max_dim() { return 4 * kMaxThreads * 8; }

// res: 0 no residual, 1 bf16, 2 fp32.
hipError_t launch_rms_norm(NormParams p, bool bf16, int res, hipStream_t st) {
  const Shape s = shape_of(p.dim);
  p.threads = s.threads;
  p.inv_dim = 1.0f / (float)p.dim;
  const int64_t per = s.threads == 64 ? s.block / 64 : 1;
  const dim3 grid((unsigned)((p.rows + per - 1) / per));
  if (bf16)
    res == 0 ? launch_fwd<true, 0>(p, s, grid, st)
             : res == 1 ? launch_fwd<true, 1>(p, s, grid, st) : launch_fwd<true, 2>(p, s, grid, st);
  else
    res == 0 ? launch_fwd<false, 0>(p, s, grid, st)
             : res == 1 ? launch_fwd<false, 1>(p, s, grid, st) : launch_fwd<false, 2>(p, s, grid, st);
  return hipGetLastError();
}

// Workgroups of the backward's first launch.
static int64_t bwd_blocks(int64_t rows, Shape s, int cus) {
  const int64_t per = s.threads == 64 ? s.block / 64 : 1;
  const int64_t resident = (int64_t)cus * (s.block >= 512 ? 2 : 1024 / s.block);
  const int64_t need = (rows + per - 1) / per;
  return need < resident ? need : resident;
}

int64_t rms_norm_bwd_workspace(int64_t rows, int dim, int cus) {
  const Shape s = shape_of(dim);
  return bwd_blocks(rows, s, cus) * (s.threads == 64 ? s.block / 64 : 1) * dim * 4;
}

hipError_t launch_rms_norm_bwd(NormBwdParams p, bool bf16, int res, int cus, hipStream_t st) {
  const Shape s = shape_of(p.dim);
  p.threads = s.threads;
  p.inv_dim = 1.0f / (float)p.dim;
  const int64_t blocks = bwd_blocks(p.rows, s, cus);
  const dim3 grid((unsigned)blocks);
  if (bf16)
    res == 0 ? launch_bwd<true, 0>(p, s, grid, st)
             : res == 1 ? launch_bwd<true, 1>(p, s, grid, st) : launch_bwd<true, 2>(p, s, grid, st);
  else
    res == 0 ? launch_bwd<false, 0>(p, s, grid, st)
             : res == 1 ? launch_bwd<false, 1>(p, s, grid, st) : launch_bwd<false, 2>(p, s, grid, st);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int parts = (int)(blocks * (s.threads == 64 ? s.block / 64 : 1));
  hipLaunchKernelGGL(rms_norm_dw_kernel, dim3((unsigned)((p.dim + kDwCols - 1) / kDwCols)),
                     dim3(kDwCols * kDwGroups), 0, st, p.partial, p.dw, p.dim, parts);
  return hipGetLastError();
}

}  // namespace mssm
