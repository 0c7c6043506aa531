// token_loss.hip -- log-probabilities of given tokens, the policy and
// preference losses on them, and the gradients by the logits.
//
// With the row's largest logit m, z_j = (l_j - m) / T and s = sum_j exp(z_j):
//   logp      = z_token - log(s)
//   dlogits_j = c / T ([j = token] - exp(z_j - log(s))),  c = dloss/dlogp
// The difference to the largest logit is taken before anything is multiplied,
// so logits up to the type's lowest value neither overflow nor lose their
// distance.  Everything is fp32 but the result's one rounding.
#include "fp8.h"
#include "mssm_internal.h"

namespace mssm {
namespace {

constexpr float kLowest = -3.402823466e38f;

// 8 columns of a row from i on, -infinity (of probability zero) past its end.
template <bool BF16>
__device__ __forceinline__ Raw8<BF16> load_columns(const void* p, int64_t from, int i, int vocab) {
  Raw8<BF16> r;
  const int n = vocab - i;
  if (n >= 8) {
    r = load_raw8<BF16>(p, from + i);
  } else if constexpr (BF16) {
    const uint16_t* q = static_cast<const uint16_t*>(p) + from + i;
    const auto at = [&](int j) { return j < n ? (uint32_t)q[j] : 0xFF80u; };
    r.a[0].w[0] = at(0) | at(1) << 16, r.a[0].w[1] = at(2) | at(3) << 16;
    r.a[0].w[2] = at(4) | at(5) << 16, r.a[0].w[3] = at(6) | 0xFF800000u;
  } else {
    const uint32_t* q = static_cast<const uint32_t*>(p) + from + i;
    const auto at = [&](int j) { return j < n ? q[j] : 0xFF800000u; };
    r.a[0].w[0] = at(0), r.a[0].w[1] = at(1), r.a[0].w[2] = at(2), r.a[0].w[3] = at(3);
    r.a[1].w[0] = at(4), r.a[1].w[1] = at(5), r.a[1].w[2] = at(6), r.a[1].w[3] = 0xFF800000u;
  }
  return r;
}

template <bool BF16>
__device__ __forceinline__ float logit(const void* p, int64_t i) {
  if constexpr (BF16) return bf16_bits(static_cast<const uint16_t*>(p)[i]);
  else return static_cast<const float*>(p)[i];
}

// Values that the compiler is to take for new ones: packed ones are unpacked
// again where they are used, in place of as many more registers in between (101
// for 64 of them, with which one workgroup of 1024 threads fits a CU and not two).
template <bool BF16, int N>
__device__ __forceinline__ void opaque(Raw8<BF16> (&raw)[N]) {
#pragma unroll
  for (int c = 0; c < N; ++c)
#pragma unroll
    for (int j = 0; j < 4; ++j) asm("" : "+v"(raw[c].a[0].w[j]));
}

// A maximum and the sum of exp((l - max) / T) below it; k = log2(e) / T.
// fmaxf passes a NaN over, and the sum becomes NaN.
struct Running {
  float top, sum;
};
template <bool BF16, int N>
__device__ __forceinline__ void take(Running& r, Raw8<BF16> (&raw)[N], float k) {
  float top = r.top;
#pragma unroll
  for (int c = 0; c < N; ++c) {
    float v[8];
    unpack8<BF16>(v, raw[c]);
#pragma unroll
    for (int j = 0; j < 8; ++j) top = fmaxf(top, v[j]);
  }
  float s = r.sum * hw_exp2((r.top - top) * k);
  if constexpr (BF16) opaque(raw);
#pragma unroll
  for (int c = 0; c < N; ++c) {
    float v[8];
    unpack8<BF16>(v, raw[c]);
#pragma unroll
    for (int j = 0; j < 8; ++j) s += hw_exp2((v[j] - top) * k);
  }
  r.top = top;
  r.sum = s;
}

// The workgroup's, from its threads'.
template <int WAVES>
__device__ __forceinline__ Running of_workgroup(Running r, float k) {
  __shared__ Running part[WAVES];
  const float own = r.top;
  float top = max16(own);
  top = fmaxf(top, __shfl_xor(top, 16));
  top = fmaxf(top, __shfl_xor(top, 32));
  const float sum = sum64(r.sum * hw_exp2((own - top) * k));
  if (WAVES == 1) return Running{top, sum};
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = Running{top, sum};
  __syncthreads();
  const int i = threadIdx.x & 15;
  r = part[i % WAVES];
  top = max16(r.top);
  return Running{top, sum16(i < WAVES ? r.sum * hw_exp2((r.top - top) * k) : 0.0f)};
}

// What follows from a row's sum: its outputs, and the gradient's factor.
struct Row {
  float top, log_sum, factor;
};
__device__ __forceinline__ Row finish_row(const LogprobParams& p, int64_t row, bool live, Running r,
                                          float taken) {
  float logp = 0.0f, log_sum = 0.0f, loss = 0.0f, slope = 0.0f;
  if (live) {
    log_sum = logf(r.sum);
    logp = (taken - r.top) * p.inv_temperature - log_sum;
    if (p.old_logprobs) {
      const float ratio = expf(logp - p.old_logprobs[row]), adv = p.advantages[row];
      const float open = ratio * adv, held = fminf(fmaxf(ratio, p.clip_lo), p.clip_hi) * adv;
      loss = -(held < open ? held : open);
      slope = held < open ? 0.0f : -open;
      if (p.ref_logprobs) {
        const float x = p.ref_logprobs[row] - logp, e = expm1f(x);
        loss += p.kl_coef * (e - x);
        slope -= p.kl_coef * e;
      }
      if (p.weights) slope *= p.weights[row];
    }
  }
  if (threadIdx.x == 0) {
    p.logprobs[row] = logp;
    if (p.loss) p.loss[row] = loss;
    if (p.stats) {
      p.stats[2 * row] = live ? r.top : 0.0f;
      p.stats[2 * row + 1] = log_sum;
    }
  }
  return Row{r.top, log_sum, slope * p.inv_temperature};
}

// factor * ([i = token] - softmax) of 8 columns from i on.
template <bool BF16>
__device__ __forceinline__ void store_slope(const LogprobParams& p, int64_t to, int i, int token,
                                            const Raw8<BF16>& raw, Row r, float k) {
  float v[8];
  unpack8<BF16>(v, raw);
  const float log_sum2 = r.log_sum * kLog2e;
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = hw_exp2((v[j] - r.top) * k - log_sum2);
  const uint32_t own = (uint32_t)(token - i);
  if (own < 8) {  // one thread of a row
#pragma unroll
    for (uint32_t j = 0; j < 8; ++j)
      if (j == own) v[j] -= 1.0f;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] *= -r.factor;
  if (p.past)
    store8_past<BF16>(p.dlogits, to + i, p.vocab - i, v);
  else
    store8<BF16>(p.dlogits, to + i, p.vocab - i, v);
}
template <bool BF16>
__device__ __forceinline__ void store_zeros(const LogprobParams& p, int64_t to, int i, int end,
                                            int step) {
  const float zero[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  for (; i < end; i += step) {
    if (p.past)
      store8_past<BF16>(p.dlogits, to + i, p.vocab - i, zero);
    else
      store8<BF16>(p.dlogits, to + i, p.vocab - i, zero);
  }
}

// One workgroup of T threads a row that stays in its registers, NV times 8
// columns a thread: read once.
template <bool BF16, int T, int NV>
__global__ void __launch_bounds__(T) logprob_held_kernel(LogprobParams p) {
  const int64_t row = blockIdx.x, from = row * p.logits_stride, to = row * p.grad_stride;
  const int64_t token = p.tokens[row];
  const bool live = token >= 0 && token < p.vocab;
  const float k = p.inv_temperature * kLog2e;
  Raw8<BF16> raw[NV];
  Running r{kLowest, 0.0f};
  float taken = 0.0f;
  if (live) {
#pragma unroll
    for (int c = 0; c < NV; ++c)
      raw[c] = load_columns<BF16>(p.logits, from, min((c * T + (int)threadIdx.x) * 8, p.vocab), p.vocab);
    taken = logit<BF16>(p.logits, from + token);
    take<BF16, NV>(r, raw, k);
    r = of_workgroup<T / 64>(r, k);
  }
  const Row w = finish_row(p, row, live, r, taken);
  if (!p.dlogits) return;
  if (w.factor == 0.0f) {
    store_zeros<BF16>(p, to, threadIdx.x * 8, p.vocab, T * 8);
    return;
  }
  if constexpr (BF16) opaque(raw);
#pragma unroll
  for (int c = 0; c < NV; ++c) {
    const int i = (c * T + threadIdx.x) * 8;
    if (i < p.vocab) store_slope<BF16>(p, to, i, (int)token, raw[c], w, k);
  }
}

// One workgroup a longer row, which is read again for its gradient.
constexpr int kThreads = 1024, kFlight = 4;
template <bool BF16>
__global__ void __launch_bounds__(kThreads) logprob_kernel(LogprobParams p) {
  const int64_t row = blockIdx.x, from = row * p.logits_stride, to = row * p.grad_stride;
  const int64_t token = p.tokens[row];
  const bool live = token >= 0 && token < p.vocab;
  const float k = p.inv_temperature * kLog2e;
  Running r{kLowest, 0.0f};
  float taken = 0.0f;
  Raw8<BF16> raw[kFlight];
  const auto load = [&](int i) {
#pragma unroll
    for (int c = 0; c < kFlight; ++c)
      raw[c] = load_columns<BF16>(p.logits, from, min(i + c * kThreads * 8, p.vocab), p.vocab);
  };
  if (live) {
    for (int i = threadIdx.x * 8; i < p.vocab; i += kFlight * kThreads * 8) {
      load(i);
      take<BF16, kFlight>(r, raw, k);
    }
    taken = logit<BF16>(p.logits, from + token);
    r = of_workgroup<kThreads / 64>(r, k);
  }
  const Row w = finish_row(p, row, live, r, taken);
  if (!p.dlogits) return;
  if (w.factor == 0.0f) {
    store_zeros<BF16>(p, to, threadIdx.x * 8, p.vocab, kThreads * 8);
    return;
  }
  for (int i = threadIdx.x * 8; i < p.vocab; i += kFlight * kThreads * 8) {
    load(i);
#pragma unroll
    for (int c = 0; c < kFlight; ++c) {
      const int at = i + c * kThreads * 8;
      if (at < p.vocab) store_slope<BF16>(p, to, at, (int)token, raw[c], w, k);
    }
  }
}

// The gradient alone: a workgroup takes kColumns columns of a row.
constexpr int kBwdThreads = 256, kBwdFlight = 4, kColumns = kBwdThreads * 8 * kBwdFlight;
template <bool BF16>
__global__ void __launch_bounds__(kBwdThreads) logprob_bwd_kernel(LogprobParams p, int parts) {
  const int64_t row = blockIdx.x / parts;
  const int first = (int)(blockIdx.x % parts) * kColumns + threadIdx.x * 8;
  const int end = min(p.vocab, (int)(blockIdx.x % parts) * kColumns + kColumns);
  const int64_t token = p.tokens[row], from = row * p.logits_stride, to = row * p.grad_stride;
  const bool live = token >= 0 && token < p.vocab;
  const Row w{p.stats[2 * row], p.stats[2 * row + 1],
              live ? p.dlogprobs[row] * p.inv_temperature : 0.0f};
  if (w.factor == 0.0f) {
    store_zeros<BF16>(p, to, first, end, kBwdThreads * 8);
    return;
  }
  Raw8<BF16> raw[kBwdFlight];
#pragma unroll
  for (int c = 0; c < kBwdFlight; ++c)
    raw[c] = load_columns<BF16>(p.logits, from, min(first + c * kBwdThreads * 8, p.vocab), p.vocab);
#pragma unroll
  for (int c = 0; c < kBwdFlight; ++c) {
    const int i = first + c * kBwdThreads * 8;
    if (i < end)
      store_slope<BF16>(p, to, i, (int)token, raw[c], w, p.inv_temperature * kLog2e);
  }
}

// One workgroup a pair.
constexpr int kPairThreads = 256;
__device__ __forceinline__ double block_sum(double v, double* lds) {
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0.0;
  for (int w = 0; w < kPairThreads / 64; ++w) v += lds[w];
  return v;
}
__global__ void __launch_bounds__(kPairThreads) preference_kernel(PreferenceParams p) {
  __shared__ double lds[kPairThreads / 64];
  const int pair = blockIdx.x;
  int64_t at[3];
  for (int i = 0; i < 3; ++i)
    at[i] = min(max(p.offsets[2 * pair + i], 0), p.rows);
  double d = 0.0;
  for (int64_t i = at[0] + threadIdx.x; i < at[1]; i += kPairThreads)
    d += (double)p.logprobs[i] - (double)p.ref_logprobs[i];
  for (int64_t i = at[1] + threadIdx.x; i < at[2]; i += kPairThreads)
    d -= (double)p.logprobs[i] - (double)p.ref_logprobs[i];
  const float x = (float)(block_sum(d, lds) * p.beta);
  // -log sigmoid(x) = softplus(-x); its slope is sigmoid(x) - 1
  const float e = expf(-fabsf(x)), both = log1pf(e);
  const float minus = fmaxf(-x, 0.0f) + both, plus = fmaxf(x, 0.0f) + both;
  const float against = (x > 0.0f ? e : 1.0f) / (1.0f + e);  // sigmoid(-x)
  if (threadIdx.x == 0)
    p.loss[pair] = (1.0f - p.smoothing) * minus + p.smoothing * plus;
  const float w = p.weights ? p.weights[pair] : 1.0f;
  const float slope = (p.smoothing - against) * p.beta * w;
  for (int64_t i = at[0] + threadIdx.x; i < at[1]; i += kPairThreads) p.dlogprobs[i] = slope;
  for (int64_t i = at[1] + threadIdx.x; i < at[2]; i += kPairThreads) p.dlogprobs[i] = -slope;
  if (pair == 0)
    for (int64_t i = threadIdx.x; i < at[0]; i += kPairThreads) p.dlogprobs[i] = 0.0f;
  if (pair == p.pairs - 1)
    for (int64_t i = at[2] + threadIdx.x; i < p.rows; i += kPairThreads) p.dlogprobs[i] = 0.0f;
}

}  // namespace

template <bool BF16>
static void launch_row(const LogprobParams& p, hipStream_t st) {
  const dim3 grid((unsigned)p.rows);
  if (!p.dlogits && p.vocab > 16384) {
    hipLaunchKernelGGL((logprob_kernel<BF16>), grid, dim3(kThreads), 0, st, p);
    return;
  }
  const auto go = [&](auto kernel, int threads) {
    hipLaunchKernelGGL(kernel, grid, dim3(threads), 0, st, p);
  };
  if (p.vocab <= 256 * 8)
    go(logprob_held_kernel<BF16, 256, 1>, 256);
  else if (p.vocab <= 256 * 8 * 2)
    go(logprob_held_kernel<BF16, 256, 2>, 256);
  else if (p.vocab <= 256 * 8 * 4)
    go(logprob_held_kernel<BF16, 256, 4>, 256);
  else if (p.vocab <= 1024 * 8 * 2)
    go(logprob_held_kernel<BF16, 1024, 2>, 1024);
  else if (p.vocab <= 1024 * 8 * 4)
    go(logprob_held_kernel<BF16, 1024, 4>, 1024);
  else if (p.vocab <= 1024 * 8 * 8)
    go(logprob_held_kernel<BF16, 1024, 8>, 1024);
  else
    go(logprob_kernel<BF16>, kThreads);
}

// Gradients of more than 64 MB go past the caches, which would be left full of
// lines to write back.
static bool goes_past(const LogprobParams& p, bool bf16) {
  return p.rows * p.vocab * (bf16 ? 2 : 4) > (int64_t)64 << 20;
}

hipError_t launch_logprobs(LogprobParams p, bool bf16, hipStream_t st) {
  p.past = goes_past(p, bf16);
  bf16 ? launch_row<true>(p, st) : launch_row<false>(p, st);
  return hipGetLastError();
}

hipError_t launch_logprobs_bwd(LogprobParams p, bool bf16, hipStream_t st) {
  p.past = goes_past(p, bf16);
  const int64_t parts = (p.vocab + kColumns - 1) / kColumns;
  auto kernel = bf16 ? logprob_bwd_kernel<true> : logprob_bwd_kernel<false>;
  hipLaunchKernelGGL(kernel, dim3((unsigned)(p.rows * parts)), dim3(kBwdThreads), 0, st, p,
                     (int)parts);
  return hipGetLastError();
}

hipError_t launch_preference(const PreferenceParams& p, hipStream_t st) {
  hipLaunchKernelGGL(preference_kernel, dim3((unsigned)p.pairs), dim3(kPairThreads), 0, st, p);
  return hipGetLastError();
}

}  // namespace mssm
