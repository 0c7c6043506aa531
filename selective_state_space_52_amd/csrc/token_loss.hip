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

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr float kLowest = -3.402823466e38f;

// A maximum and the sum of exp((l - max) / T) below it.
struct Running {
  float top, sum;
};
__device__ __forceinline__ Running join(Running a, Running b, float k) {
  const float top = fmaxf(a.top, b.top);
  // a sum of nothing stays 0 whatever its top is
  return Running{top, a.sum * hw_exp2((a.top - top) * k) + b.sum * hw_exp2((b.top - top) * k)};
}

template <bool BF16>
__device__ __forceinline__ void take(Running& r, const float (&v)[8], int n, float k) {
  float top = r.top;
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < n) top = fmaxf(top, v[j]);
  float s = r.sum * hw_exp2((r.top - top) * k);
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < n) s += hw_exp2((v[j] - top) * k);
  r.top = top;
  r.sum = s;
}

template <bool BF16>
__device__ __forceinline__ float logit(const void* p, int64_t i) {
  if constexpr (BF16) return bf16_bits(static_cast<const uint16_t*>(p)[i]);
  else return static_cast<const float*>(p)[i];
}

// factor * ([i = token] - softmax) for 8 columns
__device__ __forceinline__ void slope8(float (&v)[8], int i, int token, float top, float log_sum2,
                                       float k, float factor) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float p = hw_exp2((v[j] - top) * k - log_sum2);
    v[j] = factor * ((i + j == token ? 1.0f : 0.0f) - p);
  }
}

// One workgroup a row.
template <bool BF16>
__global__ void __launch_bounds__(kThreads) logprob_kernel(LogprobParams p) {
  __shared__ Running part[kWaves];
  const int64_t row = blockIdx.x;
  const int64_t from = row * p.logits_stride;
  const int64_t token = p.tokens[row];
  const bool live = token >= 0 && token < p.vocab;
  const float k = p.inv_temperature * kLog2e;
  Running r{kLowest, 0.0f};
  float logp = 0.0f, log_sum = 0.0f, factor = 0.0f;
  if (live) {
    for (int i = threadIdx.x * 8; i < p.vocab; i += kThreads * 8) {
      float v[8];
      load8<BF16>(v, p.logits, from + i, p.vocab - i);
      take<BF16>(r, v, p.vocab - i, k);
    }
    for (int d = 1; d < 64; d <<= 1)
      r = join(r, Running{__shfl_xor(r.top, d), __shfl_xor(r.sum, d)}, k);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = r;
    const float taken = logit<BF16>(p.logits, from + token);
    __syncthreads();
    r = part[0];
    for (int w = 1; w < kWaves; ++w) r = join(r, part[w], k);
    log_sum = logf(r.sum);
    logp = (taken - r.top) * p.inv_temperature - log_sum;
  }
  const bool policy = p.old_logprobs != nullptr;
  if (policy && live) {
    const float ratio = expf(logp - p.old_logprobs[row]), adv = p.advantages[row];
    const float open = ratio * adv, held = fminf(fmaxf(ratio, p.clip_lo), p.clip_hi) * adv;
    float loss = -(held < open ? held : open);
    float slope = held < open ? 0.0f : -open;
    if (p.ref_logprobs) {
      const float x = p.ref_logprobs[row] - logp, e = expm1f(x);
      loss += p.kl_coef * (e - x);
      slope -= p.kl_coef * e;
    }
    if (p.weights) slope *= p.weights[row];
    factor = slope * p.inv_temperature;
    if (threadIdx.x == 0) p.loss[row] = loss;
  } else if (policy && threadIdx.x == 0) {
    p.loss[row] = 0.0f;
  }
  if (threadIdx.x == 0) {
    p.logprobs[row] = logp;
    if (p.stats) {
      p.stats[2 * row] = r.top;
      p.stats[2 * row + 1] = log_sum;
    }
  }
  if (!p.dlogits) return;
  const int64_t to = row * p.grad_stride;
  const float log_sum2 = log_sum * kLog2e;
  for (int i = threadIdx.x * 8; i < p.vocab; i += kThreads * 8) {
    float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (factor != 0.0f) {
      load8<BF16>(v, p.logits, from + i, p.vocab - i);
      slope8(v, i, (int)token, r.top, log_sum2, k, factor);
    }
    store8<BF16>(p.dlogits, to + i, p.vocab - i, v);
  }
}

// The gradient alone: a workgroup takes kColumns columns of a row.
constexpr int kBwdThreads = 256, kColumns = kBwdThreads * 8 * 4;
template <bool BF16>
__global__ void __launch_bounds__(kBwdThreads) logprob_bwd_kernel(LogprobParams p, int parts) {
  const int64_t row = blockIdx.x / parts;
  const int first = (int)(blockIdx.x % parts) * kColumns;
  const int end = min(p.vocab, first + kColumns);
  const int64_t token = p.tokens[row], from = row * p.logits_stride, to = row * p.grad_stride;
  const bool live = token >= 0 && token < p.vocab;
  const float factor = live ? p.dlogprobs[row] * p.inv_temperature : 0.0f;
  const float top = p.stats[2 * row], log_sum2 = p.stats[2 * row + 1] * kLog2e;
  const float k = p.inv_temperature * kLog2e;
  for (int i = first + threadIdx.x * 8; i < end; i += kBwdThreads * 8) {
    float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (factor != 0.0f) {
      load8<BF16>(v, p.logits, from + i, p.vocab - i);
      slope8(v, i, (int)token, top, log_sum2, k, factor);
    }
    store8<BF16>(p.dlogits, to + i, p.vocab - i, v);
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

hipError_t launch_logprobs(const LogprobParams& p, bool bf16, hipStream_t st) {
  auto kernel = bf16 ? logprob_kernel<true> : logprob_kernel<false>;
  hipLaunchKernelGGL(kernel, dim3((unsigned)p.rows), dim3(kThreads), 0, st, p);
  return hipGetLastError();
}

hipError_t launch_logprobs_bwd(const LogprobParams& p, bool bf16, hipStream_t st) {
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
