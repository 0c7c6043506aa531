// token_loss.hip -- log-probabilities of given tokens, the policy and
// preference losses on them, and the gradients by the logits.
//
// With the row's largest logit m, z_j = (l_j - m) / T and s = sum_j exp(z_j):
//   logp      = z_token - log(s)
//   dlogits_j = c / T ([j = token] - exp(z_j - log(s))),  c = dloss/dlogp
// The difference to the largest logit is taken before anything is multiplied,
// so logits up to the type's lowest value neither overflow nor lose their
// distance.  Everything is fp32 but the result's one rounding.
//
// Reading the logits and writing their gradient bounds the calls: the policy loss
// of 4096 rows of 50304 (bf16, a fourth without a token) 131 us, 5.5 TB/s where a copy
// reaches 4.9 to 5.3; a forward pass 5.4 TB/s, a gradient alone 5.6.  What decides
// that: a row held in registers between its sum and its gradient (read twice: 175
// us), loads of 4 to 8 times 16 bytes a thread in flight, gradients past the caches
// (138 us through them).  A row too long for that is read twice, by two launches
// (1000 x 200003 198 us; the second read costs as much as the first, also when
// the rows are taken in groups that the 256 MB cache holds).  fp32 rows above 32768
// leave room for one workgroup a CU: 2048 x 50304 200 us, 4.1 TB/s, in parts 243.
#include "fp8.h"
#include "mssm_internal.h"

namespace mssm {
namespace {

constexpr float kLowest = -3.402823466e38f;

// A row as the threads see it.  Loads of 16 bytes run at full rate from every
// multiple of 4 bytes, not from the odd bf16 addresses that every second row of an
// odd vocabulary begins at (1000 x 200000 80 us, 200003: 108); such a row is taken
// from the element before it on, which is neither read nor written.
struct Columns {
  int64_t from, to;  // of place 0 in the logits and the gradient
  int skip;          // places before the first column: 0 or 1
  int end;           // the place behind the last column
};
template <bool BF16>
__device__ __forceinline__ Columns columns_of(const LogprobParams& p, int64_t row) {
  const int64_t from = row * p.logits_stride;
  const int skip = BF16 && p.odd ? (int)(((uint64_t)p.logits / 2 + (uint64_t)from) & 1) : 0;
  return Columns{from - skip, row * p.grad_stride - skip, skip, p.vocab + skip};
}

// 8 places from i on, -infinity (of probability zero) where there is no column.
template <bool BF16>
__device__ __forceinline__ Raw8<BF16> load_columns(const void* p, const Columns& c, int i) {
  Raw8<BF16> r;
  if (i >= c.skip && i + 8 <= c.end) {
    r = load_raw8<BF16>(p, c.from + i);
  } else if constexpr (BF16) {
    const uint16_t* q = static_cast<const uint16_t*>(p) + c.from + i;
    const auto at = [&](int j) {
      return i + j >= c.skip && i + j < c.end ? (uint32_t)q[j] : 0xFF80u;
    };
    r.a[0].w[0] = at(0) | at(1) << 16, r.a[0].w[1] = at(2) | at(3) << 16;
    r.a[0].w[2] = at(4) | at(5) << 16, r.a[0].w[3] = at(6) | at(7) << 16;
  } else {
    const uint32_t* q = static_cast<const uint32_t*>(p) + c.from + i;
    const auto at = [&](int j) { return i + j < c.end ? q[j] : 0xFF800000u; };
    r.a[0].w[0] = at(0), r.a[0].w[1] = at(1), r.a[0].w[2] = at(2), r.a[0].w[3] = at(3);
    r.a[1].w[0] = at(4), r.a[1].w[1] = at(5), r.a[1].w[2] = at(6), r.a[1].w[3] = at(7);
  }
  return r;
}

// Values at the 8 places from i on.
template <bool BF16>
__device__ __forceinline__ void store_columns(const LogprobParams& p, const Columns& c, int i,
                                              const float (&v)[8]) {
  if (i < c.skip) {
#pragma unroll
    for (int j = 1; j < 8; ++j) {
      if (i + j >= c.end) break;
      if constexpr (BF16) static_cast<uint16_t*>(p.dlogits)[c.to + i + j] = to_bf16(v[j]);
      else static_cast<float*>(p.dlogits)[c.to + i + j] = v[j];
    }
  } else if (p.past) {
    store8_past<BF16>(p.dlogits, c.to + i, c.end - i, v);
  } else {
    store8<BF16>(p.dlogits, c.to + i, c.end - i, v);
  }
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
// Adds kFlight times 8 columns, as every kernel here does, so that a row's sum has
// the same bits in all of them, and in calls of any number of rows.  (A bf16 row that
// begins at an odd address is grouped from one column earlier than one that does not:
// the same row at addresses of both parities may differ in its sum's last bits.)
constexpr int kFlight = 4;
template <bool BF16, int N>
__device__ __forceinline__ void take(Running& r, Raw8<BF16> (&raw)[N], float k) {
  static_assert(N <= kFlight, "columns that are added together");
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

// The wave's and the workgroup's, from their threads'.
__device__ __forceinline__ Running of_wave(Running r, float k) {
  float top = max16(r.top);
  top = fmaxf(top, __shfl_xor(top, 16));
  top = fmaxf(top, __shfl_xor(top, 32));
  return Running{top, sum64(r.sum * hw_exp2((r.top - top) * k))};
}
template <int WAVES>
__device__ __forceinline__ Running of_workgroup(Running r, float k) {
  __shared__ Running part[WAVES];
  r = of_wave(r, k);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = r;
  __syncthreads();
  const int i = threadIdx.x & 15;
  r = part[i % WAVES];
  const float top = max16(r.top);
  return Running{top, sum16(i < WAVES ? r.sum * hw_exp2((r.top - top) * k) : 0.0f)};
}

// What follows from a row's sum: its outputs, and the gradient's factor.
struct Row {
  float top, log_sum, factor;
};
__device__ __forceinline__ Row finish_row(const LogprobParams& p, int64_t row, bool live, Running r,
                                          float taken, bool writes) {
  float logp = 0.0f, log_sum = 0.0f, loss = 0.0f, slope = 0.0f;
  if (live) {
    log_sum = logf(r.sum);
    logp = (taken - r.top) * p.inv_temperature - log_sum;
    if (p.old_logprobs) {
      const float ratio = expf(logp - p.old_logprobs[row]), adv = p.advantages[row];
      // an advantage of 0 is none, however large the ratio
      const float open = adv == 0.0f && ratio > 1.0f ? 0.0f : ratio * adv;
      const float held = fminf(fmaxf(ratio, p.clip_lo), p.clip_hi) * adv;
      loss = -(held < open ? held : open);
      slope = held < open ? 0.0f : -open;
      if (p.ref_logprobs) {
        const float x = p.ref_logprobs[row] - logp, e = expm1f(x);
        loss += p.kl_coef * (x < __builtin_inff() ? e - x : x);  // infinite, not inf - inf
        slope -= p.kl_coef * e;
      }
      if (p.weights) {
        // a weight of 0 takes the row out, whatever the loss is there
        const float w = p.weights[row];
        slope = w == 0.0f ? 0.0f : slope * w;
      }
    }
  }
  if (writes) {
    p.logprobs[row] = logp;
    if (p.loss) p.loss[row] = loss;
    if (p.stats) {
      p.stats[2 * row] = live ? r.top : 0.0f;
      p.stats[2 * row + 1] = log_sum;
    }
  }
  return Row{r.top, log_sum, slope * p.inv_temperature};
}

// factor * ([column = token] - softmax) at the 8 places from i on.
template <bool BF16>
__device__ __forceinline__ void store_slope(const LogprobParams& p, const Columns& c, int i,
                                            int token, const Raw8<BF16>& raw, Row r, float k) {
  float v[8];
  unpack8<BF16>(v, raw);
  const float log_sum2 = r.log_sum * kLog2e;
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = hw_exp2((v[j] - r.top) * k - log_sum2);
  const uint32_t own = (uint32_t)(token + c.skip - i);
  if (own < 8) {  // one thread of a row
#pragma unroll
    for (uint32_t j = 0; j < 8; ++j)
      if (j == own) v[j] -= 1.0f;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] *= -r.factor;
  store_columns<BF16>(p, c, i, v);
}
template <bool BF16>
__device__ __forceinline__ void store_zeros(const LogprobParams& p, const Columns& c, int i, int end,
                                            int step) {
  const float zero[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  for (; i < end; i += step) store_columns<BF16>(p, c, i, zero);
}

// One workgroup of T threads a row that stays in its registers, NV times 8
// columns a thread: read once.
template <bool BF16, int T, int NV>
__global__ void __launch_bounds__(T) logprob_held_kernel(LogprobParams p) {
  const int64_t row = blockIdx.x;
  const Columns at = columns_of<BF16>(p, row);
  const int64_t token = p.tokens[row];
  const bool live = token >= 0 && token < p.vocab;
  const float k = p.inv_temperature * kLog2e;
  constexpr int kGroups = (NV + kFlight - 1) / kFlight, kEach = NV / kGroups;
  Raw8<BF16> raw[kGroups][kEach];
  Running r{kLowest, 0.0f};
  float taken = 0.0f;
  if (live) {
#pragma unroll
    for (int c = 0; c < NV; ++c)
      raw[c / kEach][c % kEach] =
          load_columns<BF16>(p.logits, at, min((c * T + (int)threadIdx.x) * 8, at.end));
    taken = logit<BF16>(p.logits, at.from + at.skip + token);
#pragma unroll
    for (int g = 0; g < kGroups; ++g) take<BF16, kEach>(r, raw[g], k);
    r = of_workgroup<T / 64>(r, k);
  }
  const Row w = finish_row(p, row, live, r, taken, threadIdx.x == 0);
  if (!p.dlogits) return;
  if (w.factor == 0.0f) {
    store_zeros<BF16>(p, at, threadIdx.x * 8, at.end, T * 8);
    return;
  }
  if constexpr (BF16) {
#pragma unroll
    for (int g = 0; g < kGroups; ++g) opaque(raw[g]);
  }
#pragma unroll
  for (int c = 0; c < NV; ++c) {
    const int i = (c * T + threadIdx.x) * 8;
    if (i < at.end) store_slope<BF16>(p, at, i, (int)token, raw[c / kEach][c % kEach], w, k);
  }
}

// One workgroup a row of which nothing is kept: without the gradient.
constexpr int kThreads = 1024;
template <bool BF16>
__global__ void __launch_bounds__(kThreads) logprob_kernel(LogprobParams p) {
  const int64_t row = blockIdx.x;
  const Columns at = columns_of<BF16>(p, row);
  const int64_t token = p.tokens[row];
  const bool live = token >= 0 && token < p.vocab;
  const float k = p.inv_temperature * kLog2e;
  Running r{kLowest, 0.0f};
  float taken = 0.0f;
  if (live) {
    for (int i = threadIdx.x * 8; i < at.end; i += kFlight * kThreads * 8) {
      Raw8<BF16> raw[kFlight];
#pragma unroll
      for (int c = 0; c < kFlight; ++c)
        raw[c] = load_columns<BF16>(p.logits, at, min(i + c * kThreads * 8, at.end));
      take<BF16, kFlight>(r, raw, k);
    }
    taken = logit<BF16>(p.logits, at.from + at.skip + token);
    r = of_workgroup<kThreads / 64>(r, k);
  }
  finish_row(p, row, live, r, taken, threadIdx.x == 0);
}

// ---- Longer rows: parts of them by workgroups of their own, whose sums a second
// launch joins and, for the gradient, reads the logits again.
constexpr int kPartThreads = 256, kColumns = kPartThreads * 8 * kFlight;

// A workgroup sums kColumns columns, so that a row's sum goes by its length alone and
// not by how many rows the call has (2 to 8 times as many columns for a workgroup
// where the rows are many: 1000 x 200003 204 to 212 us, so 202).  The first of a row
// keeps the token's logit too (the gradient may take the logits' place).
template <bool BF16>
__global__ void __launch_bounds__(kPartThreads) logprob_part_kernel(LogprobParams p) {
  const int64_t row = blockIdx.x / p.parts;
  const Columns at = columns_of<BF16>(p, row);
  const int part = (int)(blockIdx.x % p.parts);
  const int64_t token = p.tokens[row];
  if (token < 0 || token >= p.vocab) return;
  const float k = p.inv_temperature * kLog2e;
  Running r{kLowest, 0.0f};
  const int first = part * kColumns + threadIdx.x * 8;
  Raw8<BF16> raw[kFlight];
#pragma unroll
  for (int c = 0; c < kFlight; ++c)
    raw[c] = load_columns<BF16>(p.logits, at, min(first + c * kPartThreads * 8, at.end));
  take<BF16, kFlight>(r, raw, k);
  r = of_workgroup<kPartThreads / 64>(r, k);
  if (threadIdx.x != 0) return;
  float* out = p.partial + row * (2 * p.parts + 1);
  out[2 * part] = r.top;
  out[2 * part + 1] = r.sum;
  if (part == 0) out[2 * p.parts] = logit<BF16>(p.logits, at.from + at.skip + token);
}

// The row's, by a wave.
__device__ __forceinline__ Running join_parts(const LogprobParams& p, int64_t row, float k) {
  const float* in = p.partial + row * (2 * p.parts + 1);
  Running r{kLowest, 0.0f};
  for (int i = threadIdx.x & 63; i < p.parts; i += 64) {
    const Running o{in[2 * i], in[2 * i + 1]};
    const float top = fmaxf(r.top, o.top);
    r = Running{top, r.sum * hw_exp2((r.top - top) * k) + o.sum * hw_exp2((o.top - top) * k)};
  }
  return of_wave(r, k);
}

// Without the gradient: a wave a row.
__global__ void __launch_bounds__(kPartThreads) logprob_join_kernel(LogprobParams p) {
  const int64_t row = (int64_t)blockIdx.x * (kPartThreads / 64) + (threadIdx.x >> 6);
  if (row >= p.rows) return;
  const int64_t token = p.tokens[row];
  const bool live = token >= 0 && token < p.vocab;
  Running r{kLowest, 0.0f};
  if (live) r = join_parts(p, row, p.inv_temperature * kLog2e);
  finish_row(p, row, live, r, live ? p.partial[row * (2 * p.parts + 1) + 2 * p.parts] : 0.0f,
             (threadIdx.x & 63) == 0);
}

// The gradient: a workgroup takes kColumns columns of a row, whose statistics it
// has from the forward call (STATS) or joins.
template <bool BF16, bool STATS>
__global__ void __launch_bounds__(kPartThreads) logprob_bwd_kernel(LogprobParams p, int pieces) {
  const int64_t row = blockIdx.x / pieces;
  const int piece = (int)(blockIdx.x % pieces);
  const Columns at = columns_of<BF16>(p, row);
  const int first = piece * kColumns + threadIdx.x * 8, end = min(at.end, (piece + 1) * kColumns);
  const int64_t token = p.tokens[row];
  const bool live = token >= 0 && token < p.vocab;
  const float k = p.inv_temperature * kLog2e;
  Row w;
  if constexpr (STATS) {
    w = Row{p.stats[2 * row], p.stats[2 * row + 1],
            live ? p.dlogprobs[row] * p.inv_temperature : 0.0f};
  } else {
    Running r{kLowest, 0.0f};
    if (live) r = join_parts(p, row, k);
    w = finish_row(p, row, live, r, live ? p.partial[row * (2 * p.parts + 1) + 2 * p.parts] : 0.0f,
                   piece == 0 && threadIdx.x == 0);
  }
  if (w.factor == 0.0f) {
    store_zeros<BF16>(p, at, first, end, kPartThreads * 8);
    return;
  }
  Raw8<BF16> raw[kFlight];
#pragma unroll
  for (int c = 0; c < kFlight; ++c)
    raw[c] = load_columns<BF16>(p.logits, at, min(first + c * kPartThreads * 8, at.end));
#pragma unroll
  for (int c = 0; c < kFlight; ++c) {
    const int i = first + c * kPartThreads * 8;
    if (i < end) store_slope<BF16>(p, at, i, (int)token, raw[c], w, k);
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
  // a side of weight 0 counts nothing, also where it is infinite
  if (threadIdx.x == 0)
    p.loss[pair] = (p.smoothing < 1.0f ? (1.0f - p.smoothing) * minus : 0.0f) +
                   (p.smoothing > 0.0f ? p.smoothing * plus : 0.0f);
  const float w = p.weights ? p.weights[pair] : 1.0f;
  const float slope = w == 0.0f ? 0.0f : (p.smoothing - against) * p.beta * w;
  for (int64_t i = at[0] + threadIdx.x; i < at[1]; i += kPairThreads) p.dlogprobs[i] = slope;
  for (int64_t i = at[1] + threadIdx.x; i < at[2]; i += kPairThreads) p.dlogprobs[i] = -slope;
  if (pair == 0)
    for (int64_t i = threadIdx.x; i < at[0]; i += kPairThreads) p.dlogprobs[i] = 0.0f;
  if (pair == p.pairs - 1)
    for (int64_t i = at[2] + threadIdx.x; i < p.rows; i += kPairThreads) p.dlogprobs[i] = 0.0f;
}

}  // namespace

// Columns that a workgroup of 1024 threads can hold.
constexpr int64_t kHeld = 1024 * 8 * 8;

static int parts_of(int64_t vocab) {
  return vocab <= kHeld ? 0 : (int)((vocab + 1 + kColumns - 1) / kColumns);  // one place more: odd rows
}
int64_t logprob_workspace(int64_t rows, int64_t vocab) {
  const int64_t parts = parts_of(vocab);
  return parts ? rows * (2 * parts + 1) * 4 : 0;
}

template <bool BF16>
static hipError_t launch_row(const LogprobParams& p, hipStream_t st) {
  const dim3 grid((unsigned)p.rows);
  const auto go = [&](auto kernel, int threads) {
    hipLaunchKernelGGL(kernel, grid, dim3(threads), 0, st, p);
    return hipGetLastError();
  };
  if (p.parts) {
    hipLaunchKernelGGL(logprob_part_kernel<BF16>, dim3((unsigned)(p.rows * p.parts)),
                       dim3(kPartThreads), 0, st, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int pieces = (p.vocab + p.odd + kColumns - 1) / kColumns;
    if (p.dlogits)
      hipLaunchKernelGGL((logprob_bwd_kernel<BF16, false>), dim3((unsigned)(p.rows * pieces)),
                         dim3(kPartThreads), 0, st, p, pieces);
    else
      hipLaunchKernelGGL(logprob_join_kernel, dim3((unsigned)((p.rows + 3) / 4)),
                         dim3(kPartThreads), 0, st, p);
    return hipGetLastError();
  }
  const int places = p.vocab + p.odd;
  if (places <= 256 * 8) return go(logprob_held_kernel<BF16, 256, 1>, 256);
  if (places <= 256 * 8 * 2) return go(logprob_held_kernel<BF16, 256, 2>, 256);
  if (places <= 256 * 8 * 4) return go(logprob_held_kernel<BF16, 256, 4>, 256);
  if (places <= 1024 * 8 * 2) return go(logprob_held_kernel<BF16, 1024, 2>, 1024);
  if (!p.dlogits) return go(logprob_kernel<BF16>, kThreads);
  if (places <= 1024 * 8 * 4) return go(logprob_held_kernel<BF16, 1024, 4>, 1024);
  return go(logprob_held_kernel<BF16, 1024, 8>, 1024);
}

// Gradients of more than 64 MB go past the caches, which would be left full of
// lines to write back.
static bool goes_past(const LogprobParams& p, bool bf16) {
  return p.rows * p.vocab * (bf16 ? 2 : 4) > (int64_t)64 << 20;
}

// Whether rows may begin at odd bf16 addresses.  (Where one place more is more than
// a workgroup holds, they are taken as they lie.)
static int odd_rows(const LogprobParams& p, bool bf16) {
  return bf16 && (((uint64_t)p.logits / 2 | (uint64_t)p.logits_stride) & 1) && p.vocab != kHeld;
}

hipError_t launch_logprobs(LogprobParams p, bool bf16, hipStream_t st) {
  p.odd = odd_rows(p, bf16);
  p.past = goes_past(p, bf16);
  p.parts = parts_of(p.vocab);
  return bf16 ? launch_row<true>(p, st) : launch_row<false>(p, st);
}

hipError_t launch_logprobs_bwd(LogprobParams p, bool bf16, hipStream_t st) {
  p.past = goes_past(p, bf16);
  p.odd = odd_rows(p, bf16);
  const int pieces = (p.vocab + p.odd + kColumns - 1) / kColumns;
  auto kernel = bf16 ? logprob_bwd_kernel<true, true> : logprob_bwd_kernel<false, true>;
  hipLaunchKernelGGL(kernel, dim3((unsigned)(p.rows * pieces)), dim3(kPartThreads), 0, st, p, pieces);
  return hipGetLastError();
}

hipError_t launch_preference(const PreferenceParams& p, hipStream_t st) {
  hipLaunchKernelGGL(preference_kernel, dim3((unsigned)p.pairs), dim3(kPairThreads), 0, st, p);
  return hipGetLastError();
}

}  // namespace mssm
