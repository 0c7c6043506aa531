// mamba2_step.hip -- the single-token step of a Mamba-2 block: the causal
// convolution of the new token's x, B and C channels against the kept window,
// and the state update and readout.
//
// Per sequence, with v the window's inputs and the new one:
//   u      = silu(conv_bias + sum_k conv_weight[k] v_k),  the window moves on
//   Delta  = softplus(dt[h] + dt_bias[h])
//   h[d,n] <- exp(Delta A[h]) h[d,n] + Delta u_x[d] u_B[g,n]
//   out[d] = (sum_n u_C[g,n] h[d,n] + D[h] u_x[d]) * silu(z[d])
//
// The fp32 state is read and written once and is nearly all of the bytes: HBM
// bounds a batch, the two launches a single sequence.
#include "fp8.h"
#include "mssm_internal.h"

namespace mssm {
namespace {

// The state's row of sequence b, or -1 where its slot names none.
__device__ __forceinline__ int64_t slot_of(const Mamba2StepParams& p, int64_t b) {
  if (!p.slots) return b;
  const int64_t s = p.slots[b];
  return s >= 0 && s < p.cache ? s : -1;
}

template <bool BF16>
__device__ __forceinline__ float ld(const void* p, int64_t i) {
  if constexpr (BF16) return bf16_bits(static_cast<const uint16_t*>(p)[i]);
  else return static_cast<const float*>(p)[i];
}

// One channel a thread: its conv output in fp32 to the workspace, its window
// moved on by one.
template <bool BF16, int W>
__global__ void __launch_bounds__(256) step_conv_kernel(Mamba2StepParams p) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= p.batch * p.channels) return;
  const int64_t b = i / p.channels, c = i - b * p.channels;
  const int64_t slot = slot_of(p, b);
  if (slot < 0) return;
  const int64_t at = (slot * p.channels + c) * (W - 1);
  float v[W];
#pragma unroll
  for (int k = 0; k < W - 1; ++k) v[k] = ld<BF16>(p.conv_state, at + k);
  v[W - 1] = ld<BF16>(p.xbc, b * p.xbc_stride + c);
  float u = p.conv_bias ? p.conv_bias[c] : 0.0f;
#pragma unroll
  for (int k = 0; k < W; ++k) u = fmaf(p.conv_weight[c * W + k], v[k], u);
  p.u[i] = silu_f32(u);
#pragma unroll
  for (int k = 0; k < W - 1; ++k) {
    if constexpr (BF16) static_cast<uint16_t*>(p.conv_state)[at + k] = to_bf16(v[k + 1]);
    else static_cast<float*>(p.conv_state)[at + k] = v[k + 1];
  }
}

// ITEMS * 256 / (N / 4) channels of one head a workgroup: N / 4 lanes share a
// channel, 4 states each, and every load is issued before the first is used.
template <bool BF16, int N, int ITEMS>
__global__ void __launch_bounds__(256) step_state_kernel(Mamba2StepParams p) {
  constexpr int LPR = N / 4, ROWS = 256 / LPR;
  constexpr int P = 64, PIECES = P / (ROWS * ITEMS);
  const int64_t unit = blockIdx.x / PIECES;
  const int part = (int)(blockIdx.x - unit * PIECES);
  const int64_t b = unit / p.nheads;
  const int h = (int)(unit - b * p.nheads);
  const int64_t slot = slot_of(p, b);
  const int lane_n = (threadIdx.x % LPR) * 4;
  const int row0 = part * ROWS * ITEMS + threadIdx.x / LPR;
  const int64_t dim = (int64_t)p.nheads * P, d0 = (int64_t)h * P + row0;
  if (slot < 0) {
    if (lane_n == 0)
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
        const int64_t o = b * dim + d0 + i * ROWS;
        if constexpr (BF16) static_cast<uint16_t*>(p.out)[o] = 0;
        else static_cast<float*>(p.out)[o] = 0.0f;
      }
    return;
  }
  float* st = p.state + (slot * dim + d0) * N + lane_n;
  Any16 raw[ITEMS];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i)
    raw[i] = *reinterpret_cast<const Any16*>(st + (int64_t)i * ROWS * N);
  const float* u = p.u + b * p.channels;
  const int g = h / (p.nheads / p.ngroups);
  const float* ub = u + dim + (int64_t)g * N + lane_n;
  const float* uc = ub + (int64_t)p.ngroups * N;
  float B[4], C[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    B[j] = ub[j];
    C[j] = uc[j];
  }
  const float raw_dt = ld<BF16>(p.dt, b * p.dt_stride + h) + (p.dt_bias ? p.dt_bias[h] : 0.0f);
  const float dt = p.softplus ? softplus_f32(raw_dt) : raw_dt;
  const float decay = hw_exp2(dt * p.A[h] * kLog2e);
  const float D = p.D ? p.D[h] : 0.0f;
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int64_t d = d0 + i * ROWS;
    const float x = u[d], w = dt * x;
    float y = 0.0f;
    Any16 now;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float s = fmaf(decay, __uint_as_float(raw[i].w[j]), w * B[j]);
      now.w[j] = __float_as_uint(s);
      y = fmaf(C[j], s, y);
    }
    *reinterpret_cast<Any16*>(st + (int64_t)i * ROWS * N) = now;
    y = sum16(y);
    if constexpr (LPR == 32) y += __shfl_xor(y, 16);
    if (lane_n == 0) {
      y = fmaf(D, x, y);
      if (p.z) y *= silu_f32(ld<BF16>(p.z, b * p.z_stride + d));
      if constexpr (BF16) static_cast<uint16_t*>(p.out)[b * dim + d] = to_bf16(y);
      else static_cast<float*>(p.out)[b * dim + d] = y;
    }
  }
}

template <bool BF16, int N>
void launch_state(const Mamba2StepParams& p, int cus, hipStream_t st) {
  // the largest piece of a head that still gives every CU four workgroups
  const int64_t units = p.batch * p.nheads;
  constexpr int ROWS = 256 / (N / 4), MOST = 64 / ROWS;
  if (units >= 4 * cus)
    hipLaunchKernelGGL((step_state_kernel<BF16, N, MOST>), dim3((unsigned)units), dim3(256), 0, st,
                       p);
  else
    hipLaunchKernelGGL((step_state_kernel<BF16, N, 1>), dim3((unsigned)(units * MOST)), dim3(256),
                       0, st, p);
}

template <bool BF16>
hipError_t launch(const Mamba2StepParams& p, int cus, hipStream_t st) {
  const dim3 grid((unsigned)((p.batch * p.channels + 255) / 256)), block(256);
  if (p.width == 2) hipLaunchKernelGGL((step_conv_kernel<BF16, 2>), grid, block, 0, st, p);
  else if (p.width == 3) hipLaunchKernelGGL((step_conv_kernel<BF16, 3>), grid, block, 0, st, p);
  else hipLaunchKernelGGL((step_conv_kernel<BF16, 4>), grid, block, 0, st, p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (p.N == 64) launch_state<BF16, 64>(p, cus, st);
  else launch_state<BF16, 128>(p, cus, st);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mamba2_step(const Mamba2StepParams& p, bool bf16, int cus, hipStream_t st) {
  return bf16 ? launch<true>(p, cus, st) : launch<false>(p, cus, st);
}

}  // namespace mssm
