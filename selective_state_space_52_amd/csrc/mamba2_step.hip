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
// One launch: a workgroup takes a head, or a piece of its channels where there
// are few heads, and computes for itself the convolution of its x channels and
// of its group's B and C.  The windows of B and C are moved on by the last of
// a group's workgroups to have read them, told by a counter that it sets back
// to zero.  (The convolution in a launch of its own, its outputs in a
// workspace, was 283 us against 240 for 256 sequences of 80 heads.)
//
// Workgroups go round the 8 XCDs; XCD x takes the x-th eighth of the heads, so
// that a group's windows and counter stay with one XCD (266 us without), and the
// state passes the caches by (260 us without).
//
// The fp32 state is read and written once and is nearly all of the bytes: HBM
// bounds a batch (5.6 TB/s of the state at 256 sequences of 80 heads, N = 128),
// the launch a single sequence.
#include "fp8.h"  // sum16
#include "mssm_internal.h"

namespace mssm {
namespace {

// The state's row of sequence b, or -1 where its slot names none.
__device__ __forceinline__ int64_t slot_of(const Mamba2StepParams& p, int64_t b) {
  if (!p.slots) return b;
  const int64_t s = p.slots[b];
  return s >= 0 && s < p.cache ? s : -1;
}

// The state, past the caches.
typedef float f32x4n __attribute__((ext_vector_type(4), aligned(4)));
__device__ __forceinline__ f32x4n state_load(const float* p) {
  return __builtin_nontemporal_load(reinterpret_cast<const f32x4n*>(p));
}
__device__ __forceinline__ void state_store(float* p, f32x4n v) {
  __builtin_nontemporal_store(v, reinterpret_cast<f32x4n*>(p));
}

template <bool BF16>
__device__ __forceinline__ float ld(const void* p, int64_t i) {
  if constexpr (BF16) return bf16_bits(static_cast<const uint16_t*>(p)[i]);
  else return static_cast<const float*>(p)[i];
}

// Channel c of sequence b: the window's inputs, the new one last.
template <bool BF16, int W>
__device__ __forceinline__ void window_of(const Mamba2StepParams& p, int64_t b, int64_t slot, int c,
                                          float (&v)[W]) {
  const int64_t at = (slot * p.channels + c) * (W - 1);
#pragma unroll
  for (int k = 0; k < W - 1; ++k) v[k] = ld<BF16>(p.conv_state, at + k);
  v[W - 1] = ld<BF16>(p.xbc, b * p.xbc_stride + c);
}
template <int W>
__device__ __forceinline__ float conv_of(const Mamba2StepParams& p, int c, const float (&v)[W]) {
  float u = p.conv_bias ? p.conv_bias[c] : 0.0f;
#pragma unroll
  for (int k = 0; k < W; ++k) u = fmaf(p.conv_weight[(int64_t)c * W + k], v[k], u);
  return silu_f32(u);
}
template <bool BF16, int W>
__device__ __forceinline__ void move_window(const Mamba2StepParams& p, int64_t slot, int c,
                                            const float (&v)[W]) {
  const int64_t at = (slot * p.channels + c) * (W - 1);
#pragma unroll
  for (int k = 0; k < W - 1; ++k) {
    if constexpr (BF16) static_cast<uint16_t*>(p.conv_state)[at + k] = to_bf16(v[k + 1]);
    else static_cast<float*>(p.conv_state)[at + k] = v[k + 1];
  }
}

// ITEMS * 256 / (N / 4) channels of one head a workgroup: N / 4 lanes share a
// channel, 4 states each, and every load of the state is issued before the
// convolution.
template <bool BF16, int N, int W, int ITEMS>
__global__ void __launch_bounds__(256) step_kernel(Mamba2StepParams p) {
  constexpr int LPR = N / 4, ROWS = 256 / LPR, MINE = ROWS * ITEMS;
  constexpr int P = 64, PIECES = P / MINE;
  __shared__ float u[2 * N + MINE];  // the group's B and C, this piece's x
  __shared__ int is_last;
  const int t = threadIdx.x;
  const unsigned xcd = blockIdx.x % 8, rest = gridDim.x % 8;
  const unsigned id = xcd * (gridDim.x / 8) + min(xcd, rest) + blockIdx.x / 8;
  const int64_t unit = id / PIECES;
  const int part = (int)(id - unit * PIECES);
  const int64_t b = unit / p.nheads;
  const int h = (int)(unit - b * p.nheads);
  const int heads_per_group = p.nheads / p.ngroups, g = h / heads_per_group;
  const int64_t slot = slot_of(p, b);
  const int lane_n = (t % LPR) * 4, row0 = t / LPR;
  const int dim = p.nheads * P, d0 = h * P + part * MINE;
  if (slot < 0) {
    if (t < MINE) {
      const int64_t o = b * dim + d0 + t;
      if constexpr (BF16) static_cast<uint16_t*>(p.out)[o] = 0;
      else static_cast<float*>(p.out)[o] = 0.0f;
    }
    return;
  }
  float* st = p.state + (slot * dim + d0 + row0) * N + lane_n;
  f32x4n state[ITEMS];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) state[i] = state_load(st + i * ROWS * N);

  // threads 0 .. 2N - 1: a channel of B or C; threads X0 .. X0 + MINE - 1: one of x
  constexpr int X0 = 2 * N + MINE <= 256 ? 2 * N : 0;
  const int cbc = dim + (t < N ? g * N + t : (p.ngroups + g) * N + t - N);
  const int cx = d0 + t - X0;
  const bool has_x = t >= X0 && t < X0 + MINE;
  float vbc[W], vx[W];
  if (t < 2 * N) window_of<BF16, W>(p, b, slot, cbc, vbc);
  if (has_x) window_of<BF16, W>(p, b, slot, cx, vx);
  const float raw_dt = ld<BF16>(p.dt, b * p.dt_stride + h) + (p.dt_bias ? p.dt_bias[h] : 0.0f);
  const float A = p.A[h], D = p.D ? p.D[h] : 0.0f;
  if (t < 2 * N) u[t] = conv_of<W>(p, cbc, vbc);
  if (has_x) {
    u[2 * N + t - X0] = conv_of<W>(p, cx, vx);
    move_window<BF16, W>(p, slot, cx, vx);
  }
  __syncthreads();  // the windows have been read
  if (t == 0) {
    const int arrivals = heads_per_group * PIECES;
    unsigned* counter = p.counters + b * p.ngroups + g;
    // No data passes between the workgroups, so the count needs no fence: this
    // one's reads have returned, and the last one's writes follow its count.
    is_last = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
              (unsigned)arrivals - 1;
    if (is_last) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  const float dt = p.softplus ? softplus_f32(raw_dt) : raw_dt;
  const float decay = hw_exp2(dt * A * kLog2e);
  float B[4], C[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    B[j] = u[lane_n + j];
    C[j] = u[N + lane_n + j];
  }
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int row = row0 + i * ROWS;
    const float x = u[2 * N + row], w = dt * x;
    float y = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      state[i][j] = fmaf(decay, state[i][j], w * B[j]);
      y = fmaf(C[j], state[i][j], y);
    }
    state_store(st + i * ROWS * N, state[i]);
    y = sum16(y);
    if constexpr (LPR == 32) y += __shfl_xor(y, 16);
    if (lane_n == 0) {
      const int64_t d = d0 + row;
      y = fmaf(D, x, y);
      if (p.z) y *= silu_f32(ld<BF16>(p.z, b * p.z_stride + d));
      if constexpr (BF16) static_cast<uint16_t*>(p.out)[b * dim + d] = to_bf16(y);
      else static_cast<float*>(p.out)[b * dim + d] = y;
    }
  }
  __syncthreads();
  if (is_last && t < 2 * N) move_window<BF16, W>(p, slot, cbc, vbc);
}

template <bool BF16, int N, int W>
void launch(const Mamba2StepParams& p, int cus, hipStream_t st) {
  // A head a workgroup; half of one where that leaves most CUs idle (24 heads,
  // us: 6.7, halves 5.2, quarters 5.2; 80 heads: 7.0, 6.9, 7.9; 1280: 27, 40, 66,
  // more workgroups at each counter).
  const int64_t units = p.batch * p.nheads;
  constexpr int MOST = 64 / (256 / (N / 4));
  if (4 * units >= cus)
    hipLaunchKernelGGL((step_kernel<BF16, N, W, MOST>), dim3((unsigned)units), dim3(256), 0, st, p);
  else
    hipLaunchKernelGGL((step_kernel<BF16, N, W, MOST / 2>), dim3((unsigned)(units * 2)), dim3(256), 0,
                       st, p);
}
template <bool BF16, int N>
void launch(const Mamba2StepParams& p, int cus, hipStream_t st) {
  if (p.width == 2) launch<BF16, N, 2>(p, cus, st);
  else if (p.width == 3) launch<BF16, N, 3>(p, cus, st);
  else launch<BF16, N, 4>(p, cus, st);
}
template <bool BF16>
hipError_t launch(const Mamba2StepParams& p, int cus, hipStream_t st) {
  if (p.N == 64) launch<BF16, 64>(p, cus, st);
  else launch<BF16, 128>(p, cus, st);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mamba2_step(const Mamba2StepParams& p, bool bf16, int cus, hipStream_t st) {
  return bf16 ? launch<true>(p, cus, st) : launch<false>(p, cus, st);
}

}  // namespace mssm
