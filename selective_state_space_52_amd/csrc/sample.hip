// sample.hip -- the next token of each row of logits from given random
// numbers: temperature, then the k likeliest, then the likeliest up to a
// probability mass p of those, then those of at least min_p times the
// likeliest one's probability.
//
// With m the row's largest logit, w_i = exp((l_i - m) / T) and the tokens in
// order of falling logit, ties by rising index:
//   top-k   keeps the first k
//   top-p   keeps a token while the mass before it is below p times the mass
//           of the first k
//   min-p   keeps w_i >= min_p (the first token's w is 1); the first stays
// and of the kept tokens the one with the largest w_i / -log(u_i) is taken,
// for u uniform on (0, 1) (each w_i / -log(u_i) exceeds the others with
// probability w_i / sum w); its log-probability is
// (l - m) / T - log(sum of the kept w).
//
// Masses are sums of w in units of 2^-40 in 64-bit integers: they are exact
// whatever the order of the additions, so equal calls give equal tokens.
#include "fp8.h"
#include "mssm_internal.h"

namespace mssm {
namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64, kBins = 256;
constexpr float kUnits = 1099511627776.0f;  // 2^40

// Unsigned order of floats: larger value, larger key.  Both zeros are equal;
// NaN counts as -infinity.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}

template <bool BF16>
__device__ __forceinline__ float logit(const void* row, int64_t i) {
  float x;
  if constexpr (BF16) x = bf16_bits(static_cast<const uint16_t*>(row)[i]);
  else x = static_cast<const float*>(row)[i];
  return x == x ? x : -__builtin_inff();
}

__device__ __forceinline__ uint64_t max_u64(uint64_t a, uint64_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint64_t shfl_xor_u64(uint64_t v, int d) {
  const uint32_t lo = __shfl_xor((uint32_t)v, d), hi = __shfl_xor((uint32_t)(v >> 32), d);
  return (uint64_t)hi << 32 | lo;
}

struct Shared {
  uint64_t mass[kBins];
  uint32_t count[kBins];
  uint64_t red[kWaves];
  uint64_t found_mass;
  uint32_t found_bin, found_count;
};

template <typename F>
__device__ uint64_t block_reduce(uint64_t v, Shared& s, F f) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) v = f(v, shfl_xor_u64(v, d));
  __syncthreads();
  if ((threadIdx.x & 63) == 0) s.red[threadIdx.x >> 6] = v;
  __syncthreads();
  v = s.red[0];
  for (int w = 1; w < kWaves; ++w) v = f(v, s.red[w]);
  return v;
}

struct Weight {
  float max, inv_t;
  __device__ __forceinline__ float scaled(float x) const {
    return x == max ? 0.0f : (x - max) * inv_t;
  }
  __device__ __forceinline__ float of(float x) const { return hw_exp2(scaled(x) * kLog2e); }
  __device__ __forceinline__ uint64_t units(float x) const {
    const float v = of(x);
    return v > 0.0f ? (uint64_t)(v * kUnits + 0.5f) : 0u;  // a NaN weight counts nothing
  }
};

// A place in the row's order: the tokens with a larger key, and the first
// `ties` (by index) of those with this key.
struct Place {
  uint32_t key;
  uint32_t ties;
};

// The last place whose count (BY_MASS: the mass before whose last token) is
// below a bound, found digit by digit of the key, from the top.
template <bool BF16, bool BY_MASS>
__device__ Place find_place(const void* row, int V, const Weight& w, uint64_t want, Shared& s) {
  uint32_t prefix = 0, mask = 0;
  uint64_t above = 0;  // count or mass of the keys above the prefix
  uint32_t ties = 0;
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = threadIdx.x; i < kBins; i += kThreads) s.mass[i] = s.count[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < V; i += kThreads) {
      const float x = logit<BF16>(row, i);
      const uint32_t key = key_of(x);
      if ((key & mask) != prefix) continue;
      const uint32_t bin = (key >> shift) & 255u;
      atomicAdd(&s.count[bin], 1u);
      if constexpr (BY_MASS) atomicAdd((unsigned long long*)&s.mass[bin], (unsigned long long)w.units(x));
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      // the bin that holds the last token whose predecessors sum below want
      uint64_t sum = above;
      uint32_t last = 0, n = 0;
      uint64_t before = above;
      for (int bin = kBins - 1; bin >= 0; --bin) {
        const uint32_t c = s.count[bin];
        if (c == 0) continue;
        if (sum >= want && n) break;
        last = (uint32_t)bin;
        before = sum;
        n = c;
        sum += BY_MASS ? s.mass[bin] : (uint64_t)c;
      }
      s.found_bin = last;
      s.found_mass = before;
      s.found_count = n;
    }
    __syncthreads();
    above = s.found_mass;
    ties = s.found_count;
    prefix |= s.found_bin << shift;
    mask |= 255u << shift;
    __syncthreads();
  }
  const uint64_t each = BY_MASS ? w.units(value_of(prefix)) : 1u;
  const uint64_t room = want > above ? want - above : 0;
  const uint64_t n = each ? (room + each - 1) / each : ties;
  return Place{prefix, (uint32_t)(n < ties ? (n ? n : 1) : ties)};
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads) sample_kernel(SampleParams p) {
  __shared__ Shared s;
  const int64_t r = blockIdx.x;
  const int V = p.vocab;
  const void* row = static_cast<const char*>(p.logits) + r * p.logits_stride * (BF16 ? 2 : 4);
  const float* noise = p.noise + r * p.noise_stride;
  const float T = p.temperature_row ? p.temperature_row[r] : p.temperature;
  const int top_k = p.top_k_row ? p.top_k_row[r] : p.top_k;
  const float top_p = p.top_p_row ? p.top_p_row[r] : p.top_p;
  const float min_p = p.min_p_row ? p.min_p_row[r] : p.min_p;
  const auto most = [](uint64_t a, uint64_t b) { return max_u64(a, b); };
  const auto sum = [](uint64_t a, uint64_t b) { return a + b; };

  // the first token of the order: largest key, lowest index
  uint64_t best = 0;
  for (int i = threadIdx.x; i < V; i += kThreads)
    best = max_u64(best, (uint64_t)key_of(logit<BF16>(row, i)) << 32 | (0xFFFFFFFFu - (uint32_t)i));
  best = block_reduce(best, s, most);
  const uint32_t top_key = (uint32_t)(best >> 32);
  const int first = (int)(0xFFFFFFFFu - (uint32_t)best);
  const Weight w{value_of(top_key), 1.0f / T};
  if (w.max == -__builtin_inff()) {  // nothing to choose from
    if (threadIdx.x == 0) {
      p.tokens[r] = -1;
      p.logprobs[r] = -__builtin_inff();
    }
    return;
  }
  if (!(T > 0.0f) || top_k == 1) {
    if (threadIdx.x == 0) {
      p.tokens[r] = first;
      p.logprobs[r] = 0.0f;
    }
    return;
  }
  Place end{0u, 0xFFFFFFFFu};
  if (top_k > 0 && top_k < V) end = find_place<BF16, false>(row, V, w, (uint64_t)top_k, s);
  if (top_p < 1.0f) {
    uint64_t mass = 0;
    for (int i = threadIdx.x; i < V; i += kThreads) {
      const float x = logit<BF16>(row, i);
      if (key_of(x) > end.key) mass += w.units(x);
    }
    mass = block_reduce(mass, s, sum);
    if (end.key) mass += end.ties * w.units(value_of(end.key));
    const double bound = (double)fmaxf(top_p, 0.0f) * (double)mass;
    uint64_t want = (uint64_t)ceil(bound);
    const Place q = find_place<BF16, true>(row, V, w, want ? want : 1u, s);
    if (q.key > end.key || (q.key == end.key && q.ties < end.ties)) end = q;
  }
  // the tie that is the last one kept: the index up to which ties count
  int last = V;
  if (end.key && end.ties != 0xFFFFFFFFu) {
    int lo = 0, hi = V;  // smallest `last` with `ties` ties below it
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      uint64_t n = 0;
      for (int i = threadIdx.x; i < mid; i += kThreads) n += key_of(logit<BF16>(row, i)) == end.key;
      n = block_reduce(n, s, sum);
      if (n >= end.ties) hi = mid;
      else lo = mid + 1;
    }
    last = lo;
  }
  uint64_t kept = 0, win = 0;
  for (int i = threadIdx.x; i < V; i += kThreads) {
    const float x = logit<BF16>(row, i);
    const uint32_t key = key_of(x);
    if (key < end.key || (key == end.key && i >= last)) continue;
    const float wi = w.of(x);
    if (i != first && (!(wi > 0.0f) || wi < min_p)) continue;
    kept += w.units(x);
    const float u = noise[i];
    const float e = u > 0.0f ? fmaxf(-hw_log2(u), 0.0f) : __builtin_inff();
    float score = wi / e;
    if (!(score >= 0.0f)) score = 0.0f;
    win = max_u64(win, (uint64_t)__float_as_uint(score) << 32 | (0xFFFFFFFFu - (uint32_t)i));
  }
  kept = block_reduce(kept, s, sum);
  win = block_reduce(win, s, most);
  if (threadIdx.x == 0) {
    const int token = (int)(0xFFFFFFFFu - (uint32_t)win);
    p.tokens[r] = token;
    p.logprobs[r] = w.scaled(logit<BF16>(row, token)) - hw_log2((float)kept / kUnits) * kLn2;
  }
}

}  // namespace

hipError_t launch_sample(const SampleParams& p, bool bf16, hipStream_t st) {
  const dim3 grid((unsigned)p.rows);
  if (bf16) hipLaunchKernelGGL((sample_kernel<true>), grid, dim3(kThreads), 0, st, p);
  else hipLaunchKernelGGL((sample_kernel<false>), grid, dim3(kThreads), 0, st, p);
  return hipGetLastError();
}

}  // namespace mssm
