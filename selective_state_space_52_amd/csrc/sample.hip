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
// One workgroup takes a row and reads it three to five times, from L2 after the
// first (held in registers instead, unrolled, it was 78 us against 51 for 256
// rows of 50304: the code no longer fit the instruction cache).  Sorting a row
// would move it many times over; what is wanted is the last kept token, in
// steps that each leave few tokens:
//   top-k up to kRank: of the threads' largest logits the k-th is no larger
//     than the row's k-th, so the tokens from its bin up hold the first k.  Of
//     random logits they are few more; they go to a list in LDS, and where it
//     holds them (no more than kRank; top-k up to 180 of 50304), the rest is done
//     there: 256 rows 22 us at top-k 100, 33 the other way.  A list too long is a
//     pass for nothing: 5 us of 40 at top-k 200, so larger top-k do not try.
//   otherwise: the row's counts or masses in bins of the distance below the
//     largest logit (32 to each power of two) give the bin in which the last
//     kept token lies; its tokens go to the list, and if they are many once
//     more through 512 bins of their own.
//   A list of up to kRank tokens is ranked by comparing all pairs, a longer one
//     is sorted.  Where a list would hold more than kList tokens (many equal
//     logits, or a bin of a large vocabulary: normal logits of deviation 2.5 pass
//     it from about 100000 tokens on, earlier the closer top-p is to 1), the
//     boundary is found digit by digit of the logits' keys, in four passes over
//     the row for each (64 rows of 128256, top-p 0.95: 99 us; 0.99: 680).
//
// The vector instructions of the passes bound a batch of rows, latency a
// single row.  Sums are in a fixed order or, where the order may differ, in
// units of 2^-41 in 64-bit integers, so equal calls give equal tokens.
#include "fp8.h"
#include "mssm_internal.h"

namespace mssm {
namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kBins = 256;   // of one digit of a key
constexpr int kFine = 512;   // of the distance below the largest logit
constexpr int kList = 4096;  // tokens of the list in LDS
constexpr int kRank = 256;   // ... that are ranked by comparing all pairs
constexpr int kPer = kList / kThreads;
constexpr double kUnits = 2199023255552.0;  // 2^41: 2^22 tokens of w = 1 sum to 2^63

// Unsigned order of floats: larger value, larger key.  Both zeros are equal.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}
// A token's place in the order as one number, larger first.
__device__ __forceinline__ uint64_t entry_of(uint32_t key, int i) {
  return (uint64_t)key << 32 | (0xFFFFFFFFu - (uint32_t)i);
}
__device__ __forceinline__ int index_of(uint64_t e) { return (int)(0xFFFFFFFFu - (uint32_t)e); }
__device__ __forceinline__ float value_of(uint64_t e) { return value_of((uint32_t)(e >> 32)); }

__device__ __forceinline__ float no_nan(float x) { return x == x ? x : -__builtin_inff(); }
template <bool BF16>
__device__ __forceinline__ float logit(const void* row, int64_t i) {
  if constexpr (BF16) return no_nan(bf16_bits(static_cast<const uint16_t*>(row)[i]));
  else return no_nan(static_cast<const float*>(row)[i]);
}

struct Shared {
  union {
    uint64_t list[kList];  // entries
    struct {
      uint64_t mass[kBins];
      uint32_t count[kBins];
    };
  };
  uint64_t fine[kFine];
  uint64_t units[kRank];
  uint64_t red[2][kWaves];
  uint64_t found_mass;
  uint32_t found_bin, found_count;
  uint32_t listed;
};

// ---- reductions: DPP moves inside each 16 lanes, two shuffles, and one round
// through LDS, whose two buffers take turns so that one barrier is enough.
template <int CTRL>
__device__ __forceinline__ uint64_t dpp64(uint64_t v) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_mov_dpp((int)(v >> 32), CTRL, 0xF, 0xF, true);
  return (uint64_t)hi << 32 | lo;
}
__device__ __forceinline__ uint64_t shfl_xor_u64(uint64_t v, int d) {
  const uint32_t lo = __shfl_xor((uint32_t)v, d), hi = __shfl_xor((uint32_t)(v >> 32), d);
  return (uint64_t)hi << 32 | lo;
}
__device__ __forceinline__ uint64_t shfl_up_u64(uint64_t v, int d) {
  const uint32_t lo = __shfl_up((uint32_t)v, d), hi = __shfl_up((uint32_t)(v >> 32), d);
  return (uint64_t)hi << 32 | lo;
}
template <typename F>
__device__ __forceinline__ uint64_t reduce16(uint64_t v, F f) {
  v = f(v, dpp64<0xB1>(v));
  v = f(v, dpp64<0x4E>(v));
  v = f(v, dpp64<0x141>(v));
  return f(v, dpp64<0x140>(v));
}
struct Max { __device__ uint64_t operator()(uint64_t a, uint64_t b) const { return a > b ? a : b; } };
struct Min { __device__ uint64_t operator()(uint64_t a, uint64_t b) const { return a < b ? a : b; } };
struct Sum { __device__ uint64_t operator()(uint64_t a, uint64_t b) const { return a + b; } };
struct SumF64 {
  __device__ uint64_t operator()(uint64_t a, uint64_t b) const {
    return __builtin_bit_cast(uint64_t, __builtin_bit_cast(double, a) + __builtin_bit_cast(double, b));
  }
};
struct Block {
  Shared& s;
  int turn = 0;
  template <typename F>
  __device__ __forceinline__ uint64_t reduce(uint64_t v, F f) {
    v = reduce16(v, f);
    v = f(v, shfl_xor_u64(v, 16));
    v = f(v, shfl_xor_u64(v, 32));
    if ((threadIdx.x & 63) == 0) s.red[turn][threadIdx.x >> 6] = v;
    __syncthreads();
    v = s.red[turn][threadIdx.x & 15];
    turn ^= 1;
    return reduce16(v, f);
  }
  __device__ __forceinline__ double sum(double v) {
    return __builtin_bit_cast(double, reduce(__builtin_bit_cast(uint64_t, v), SumF64()));
  }
  // The sum of v over the threads before this one.
  __device__ __forceinline__ uint64_t before(uint64_t v) {
    uint64_t upto = v;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const uint64_t o = shfl_up_u64(upto, d);
      if ((threadIdx.x & 63) >= d) upto += o;
    }
    if ((threadIdx.x & 63) == 63) s.red[turn][threadIdx.x >> 6] = upto;
    __syncthreads();
    uint64_t sum = upto - v;
    for (int q = 0; q < (int)(threadIdx.x >> 6); ++q) sum += s.red[turn][q];
    turn ^= 1;
    return sum;
  }
};

struct Weight {
  float max, inv_t;
  __device__ __forceinline__ float scaled(float x) const {
    return x == max ? 0.0f : (x - max) * inv_t;
  }
  __device__ __forceinline__ float of(float x) const { return hw_exp2(scaled(x) * kLog2e); }
  // w in units of 2^-41, rounded to the nearest: V roundings, all of one sign
  // where many logits are equal, are at most V 2^-42 of the largest token's mass
  // (1e-6 for 2^22 tokens; in units of 2^-31 a tail of that many tokens could
  // weigh 1e-3 and count nothing).  By halves, whole 2^-9 and the rest, which is
  // exact and never rounds up to 2^32 (by a sum with 2^11 in 64-bit floats rows
  // decided digit by digit took 3% longer).  A NaN weight counts nothing: the
  // conversions give 0.
  __device__ __forceinline__ uint64_t units(float x) const { return units_of(of(x)); }
  static __device__ __forceinline__ uint64_t units_of(float v) {
    const float a = v * 512.0f;
    const uint32_t hi = (uint32_t)a;
    const uint32_t lo = (uint32_t)fmaf(a - (float)hi, 4294967296.0f, 0.5f);
    return (uint64_t)hi << 32 | lo;
  }
  // The same without the look at the largest logit, which `scaled` needs where
  // that is infinite, or 1 / T nearly.
  __device__ __forceinline__ float fast(float x) const {
    return hw_exp2((x - max) * (inv_t * kLog2e));
  }
  __device__ __forceinline__ bool plain() const {
    return fabsf(max) <= 3.402823466e38f && inv_t <= 2e38f;
  }
};

// The bin of a token that lies d below the largest: equal steps of 1/32 of
// each power of two from 2^-5 to 2^11, the rest in the first and the last.
// Monotone in x, as the rounded difference is.
__device__ __forceinline__ uint32_t distance(float top, float x) {
  return __float_as_uint(top - x);
}
__device__ __forceinline__ int bin_of(float top, float x) {
  const int b = (int)(distance(top, x) >> 18) - (((127 - 5) << 5) - 1);
  return min(max(b, 0), kFine - 1);
}

// w / -log(u), which orders like the race; w is positive.
__device__ __forceinline__ float race(float w, float u) {
  return w * hw_rcp(fmaxf(-hw_log2(fmaxf(u, 0.0f)), 0.0f));
}

// A row's tokens, 8 neighbours a thread at a time.  NaN counts as -infinity, and
// so does what lies past the row's end in its last 8.
template <bool BF16>
struct Row {
  static constexpr int kWords = BF16 ? 4 : 8, kStep = kThreads * 8;
  const void* row;
  int V;

  __device__ __forceinline__ void load(float (&x)[8], int i) const {
    uint32_t w[kWords];
    if (i + 8 <= V) {
#pragma unroll
      for (int h = 0; h < kWords / 4; ++h) {
        const Any16 a = reinterpret_cast<const Any16*>(static_cast<const char*>(row) +
                                                       (int64_t)i * (BF16 ? 2 : 4))[h];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[4 * h + j] = a.w[j];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float v = !BF16 ? __uint_as_float(w[j % kWords])
                              : j & 1 ? bf16_hi(w[j / 2]) : bf16_lo(w[j / 2]);
        x[j] = fmaxf(v, -__builtin_inff());
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float v = logit<BF16>(row, min(i + j, V - 1));
        x[j] = i + j < V ? v : -__builtin_inff();
      }
    }
  }
  // f(values, index of the first) for each 8 of this thread's tokens, in rising
  // order, the loads of two at a time
  template <typename F>
  __device__ __forceinline__ void eights(F f) const {
    for (int i = threadIdx.x * 8; i < V; i += 2 * kStep) {
      float x[8], y[8];
      load(x, i);
      const bool two = i + kStep < V;
      if (two) load(y, i + kStep);
      f(x, i);
      if (two) f(y, i + kStep);
    }
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
__device__ __forceinline__ Place find_place(const void* row, int V, const Weight& w, uint64_t want, Shared& s) {
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

// list[0..size) in falling order, size a power of two.
__device__ __forceinline__ void sort_list(int size, uint64_t* list) {
  for (int k = 2; k <= size; k *= 2)
    for (int d = k / 2; d > 0; d /= 2) {
      __syncthreads();
      for (int p = threadIdx.x; p < size / 2; p += kThreads) {
        const int i = 2 * p - (p & (d - 1)), j = i + d;
        const uint64_t a = list[i], b = list[j];
        if ((a < b) == ((i & k) == 0)) {
          list[i] = b;
          list[j] = a;
        }
      }
    }
  __syncthreads();
}

// The boundary digit by digit, and the race over the whole row: for rows of
// which too many tokens stay for the list.
template <bool BF16>
__device__ __forceinline__ void sample_by_digits(const SampleParams& p, const void* row,
                                              const float* noise, Weight w, int top_k,
                                              float top_p, float min_p, Shared& s) {
  const int64_t r = blockIdx.x;
  const int V = p.vocab;
  Block block{s};
  __syncthreads();

  Place end{0u, 0xFFFFFFFFu};
  if (top_k > 0 && top_k < V) end = find_place<BF16, false>(row, V, w, (uint64_t)top_k, s);
  if (top_p < 1.0f) {
    uint64_t mass = 0;
    for (int i = threadIdx.x; i < V; i += kThreads) {
      const float x = logit<BF16>(row, i);
      if (key_of(x) > end.key) mass += w.units(x);
    }
    mass = block.reduce(mass, Sum());
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
      n = block.reduce(n, Sum());
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
    if (!(wi > 0.0f) || wi < min_p) continue;
    kept += w.units(x);
    win = Max()(win, entry_of(__float_as_uint(race(wi, noise[i])), i));
  }
  kept = block.reduce(kept, Sum());
  win = block.reduce(win, Max());
  if (threadIdx.x == 0) {
    const int token = index_of(win);
    p.tokens[r] = token;
    p.logprobs[r] = w.scaled(logit<BF16>(row, token)) - hw_log2((float)((double)kept / kUnits)) * kLn2;
  }
}


// The last bin of `fine` with less than `limit` in it before it (`ahead` before
// the first), and what is before it: s.found_bin, s.found_mass.  Empty bins are
// passed over.
__device__ __forceinline__ void find_bin(Shared& s, uint64_t ahead, uint64_t limit) {
  const int t = threadIdx.x;
  if (t < 64) {
    constexpr int kEach = kFine / 64;
    uint64_t mine[kEach], sum = 0;
#pragma unroll
    for (int q = 0; q < kEach; ++q) {
      mine[q] = s.fine[t * kEach + q];
      sum += mine[q];
    }
    uint64_t upto = sum;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const uint64_t o = shfl_up_u64(upto, d);
      if (t >= d) upto += o;
    }
    uint64_t before = ahead + upto - sum, at = 0;
    int found = -1;
#pragma unroll
    for (int q = 0; q < kEach; ++q) {
      if (mine[q] > 0 && before < limit) {
        found = t * kEach + q;
        at = before;
      }
      before += mine[q];
    }
    const uint64_t whose = __ballot(found >= 0);
    if (t == 63 - (whose ? __builtin_clzll(whose) : 63)) {
      s.found_bin = (uint32_t)(found < 0 ? 0 : found);
      s.found_mass = at;
    }
  }
  __syncthreads();
}

// What a token counts for: one, or its mass.
__device__ __forceinline__ uint64_t counts_for(bool mass, const Weight& w, float x) {
  return mass ? Weight::units_of(w.fast(x)) : 1;
}

// The last entry of s.list[0..n) with less than `limit` before it, `ahead`
// being before the list.  n is at most kList.
__device__ __forceinline__ uint64_t last_of(Shared& s, Block& block, int n, bool mass, const Weight& w,
                            uint64_t ahead, uint64_t limit) {
  const int t = threadIdx.x;
  uint64_t low = ~0ull;
  if (n <= kRank) {
    const uint64_t mine = t < n ? s.list[t] : 0;
    if (t < n) s.units[t] = counts_for(mass, w, value_of(mine));
    __syncthreads();
    if (t < n) {
      uint64_t before = ahead;
#pragma unroll 4
      for (int j = 0; j < n; ++j) before += s.list[j] > mine ? s.units[j] : 0;
      if (before < limit) low = mine;
    }
  } else {
    int size = 2 * kRank;
    while (size < n) size *= 2;
    for (int i = n + t; i < size; i += kThreads) s.list[i] = 0;
    sort_list(size, s.list);
    const int per = (size + kThreads - 1) / kThreads;
    uint64_t e[kPer], each[kPer], part = 0;
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      const int at = t * per + q;
      e[q] = q < per && at < n ? s.list[at] : 0;
      each[q] = e[q] ? counts_for(mass, w, value_of(e[q])) : 0;
      part += each[q];
    }
    uint64_t before = ahead + block.before(part);
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      if (e[q] && before < limit) low = e[q];
      before += each[q];
    }
  }
  return block.reduce(low, Min());
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads) sample_kernel(SampleParams p) {
  __shared__ Shared s;
  Block block{s};
  const int64_t r = blockIdx.x;
  const int V = p.vocab, t = threadIdx.x;
  const Row<BF16> row{static_cast<const char*>(p.logits) + r * p.logits_stride * (BF16 ? 2 : 4), V};
  const float* noise = p.noise + r * p.noise_stride;
  const float T = p.temperature_row ? p.temperature_row[r] : p.temperature;
  const int top_k = p.top_k_row ? p.top_k_row[r] : p.top_k;
  const float top_p = p.top_p_row ? p.top_p_row[r] : p.top_p;
  const float min_p = p.min_p_row ? p.min_p_row[r] : p.min_p;

  float top = -__builtin_inff();  // of this thread
  row.eights([&](const float (&x)[8], int) {
#pragma unroll
    for (int j = 0; j < 8; ++j) top = fmaxf(top, x[j]);
  });
  const Weight w{value_of((uint32_t)block.reduce((uint64_t)key_of(top), Max())), 1.0f / T};
  if (w.max == -__builtin_inff()) {  // nothing to choose from
    if (t == 0) {
      p.tokens[r] = -1;
      p.logprobs[r] = -__builtin_inff();
    }
    return;
  }
  if (!(T > 0.0f) || top_k == 1 || top_p <= 0.0f || min_p > 1.0f) {
    // only the first token of the order: largest logit, lowest index
    uint64_t lowest = ~0ull;
    if (top == w.max)
      row.eights([&](const float (&x)[8], int i) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (x[j] == w.max) lowest = Min()(lowest, (uint64_t)(i + j));
      });
    lowest = block.reduce(lowest, Min());
    if (t == 0) {
      p.tokens[r] = (int64_t)lowest;
      p.logprobs[r] = 0.0f;
    }
    return;
  }

  const bool by_k = top_k > 0 && top_k < V, by_p = top_p < 1.0f;
  const float mass_p = top_p;
  // The winner so far of this thread, its score below 0 where it has none; the
  // sum of the kept w.
  float score = -1.0f;
  int winner = 0;
  double kept = 0.0;
  const auto run = [&](float wi, int i, float u) {
    const float here = race(wi, u);
    if (here > score) {  // a thread's tokens come in rising order
      score = here;
      winner = i;
    }
  };
  // The tokens of one bin, or of it and those above, to the list (n of them,
  // the first `most` kept).  Few are: two comparisons a token, a little wider
  // than the bin, pass over most of them.
  const auto gather = [&](int bin, bool above, uint64_t least, int most) {
    const int bits = (bin + ((127 - 5) << 5) - 1) << 18;
    const float near = __uint_as_float(bits), far = __uint_as_float(bits + (1 << 18));
    const float high = bin == 0 || above ? w.max : w.max - near * 0.999f;
    const float low = bin == kFine - 1 ? -__builtin_inff() : w.max - far * 1.001f;
    row.eights([&](const float (&x)[8], int i) {
      uint32_t in = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) in |= x[j] >= low && x[j] <= high ? 1u << j : 0u;
      for (; in; in &= in - 1) {  // the token again from the cache: any of the eight registers
        const int k = i + __builtin_ctz(in);
        const float v = k < V ? logit<BF16>(row.row, k) : -__builtin_inff();
        const int b = bin_of(w.max, v);
        const uint64_t e = entry_of(key_of(v), k);
        if ((above ? b > bin : b != bin) || e < least) continue;
        const uint32_t at = atomicAdd(&s.listed, 1u);
        if (at < (uint32_t)most) s.list[at] = e;
      }
    });
    __syncthreads();
    return (int)s.listed;
  };

  bool listed = false, fits = w.plain();
  if (fits && by_k && top_k <= kRank) {
    for (int i = t; i < kFine; i += kThreads) s.fine[i] = 0;
    if (t == 0) s.listed = 0;
    __syncthreads();
    atomicAdd((unsigned long long*)&s.fine[bin_of(w.max, top)], 1ull);
    __syncthreads();
    find_bin(s, 0, (uint64_t)top_k);
    const int n = gather((int)s.found_bin, true, 0, kRank);
    __syncthreads();  // s.listed may be cleared below
    listed = n <= kRank;
    if (listed) {
      // each token's rank and the mass before it
      const uint64_t mine = t < n ? s.list[t] : 0;
      const float wi = t < n ? w.fast(value_of(mine)) : 0.0f;
      const uint64_t units = Weight::units_of(wi);
      if (t < n) s.units[t] = units;
      __syncthreads();
      uint64_t before = 0;
      int rank = 0;
      if (t < n)
#pragma unroll 4
        for (int j = 0; j < n; ++j) {
          const bool ahead = s.list[j] > mine;
          rank += ahead;
          before += ahead ? s.units[j] : 0;
        }
      bool in = t < n && rank < top_k;
      const uint64_t all = block.reduce(in ? units : 0, Sum());
      if (by_p) in = in && (rank == 0 || before < (uint64_t)ceil((double)mass_p * (double)all));
      in = in && wi > 0.0f && !(wi < min_p);
      if (in) run(wi, index_of(mine), noise[index_of(mine)]);
      kept = (double)block.reduce(in ? units : 0, Sum()) * (1.0 / kUnits);
    }
  }
  if (!listed) {
    uint64_t last = 0;  // the last kept token's entry
    for (int turn = by_k ? 0 : 1; turn < (by_p ? 2 : 1) && fits; ++turn) {
      // turn 0: the first k; turn 1: those up to the mass p of what is left
      const bool mass = turn == 1;
      for (int i = t; i < kFine; i += kThreads) s.fine[i] = 0;
      if (t == 0) s.listed = 0;
      __syncthreads();
      row.eights([&](const float (&x)[8], int i) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (last && entry_of(key_of(x[j]), i + j) < last) continue;
          atomicAdd((unsigned long long*)&s.fine[bin_of(w.max, x[j])],
                    (unsigned long long)counts_for(mass, w, x[j]));
        }
      });
      __syncthreads();
      uint64_t limit = (uint64_t)top_k;
      if (mass) {
        const uint64_t all = block.reduce(t < kFine ? s.fine[t] : 0, Sum());
        limit = (uint64_t)ceil((double)mass_p * (double)all);
      }
      find_bin(s, 0, limit);
      const int bin = (int)s.found_bin;
      uint64_t ahead = s.found_mass;
      int n = gather(bin, false, last, kList);
      fits = n <= kList;
      if (!fits) break;
      if (n > kRank && bin > 0 && bin < kFine - 1) {
        // all of one bin: the next 9 bits of the distance
        const auto sub = [&](uint64_t e) { return (int)(distance(w.max, value_of(e)) >> 9 & (kFine - 1)); };
        uint64_t e[kPer];
        for (int i = t; i < kFine; i += kThreads) s.fine[i] = 0;
        __syncthreads();
#pragma unroll
        for (int q = 0; q < kPer; ++q) {
          e[q] = q * kThreads + t < n ? s.list[q * kThreads + t] : 0;
          if (e[q])
            atomicAdd((unsigned long long*)&s.fine[sub(e[q])],
                      (unsigned long long)counts_for(mass, w, value_of(e[q])));
        }
        if (t == 0) s.listed = 0;
        __syncthreads();
        find_bin(s, ahead, limit);
        ahead = s.found_mass;
#pragma unroll
        for (int q = 0; q < kPer; ++q)
          if (e[q] && sub(e[q]) == (int)s.found_bin) s.list[atomicAdd(&s.listed, 1u)] = e[q];
        __syncthreads();
        n = (int)s.listed;
      }
      last = Max()(last, last_of(s, block, n, mass, w, ahead, limit));
      __syncthreads();
    }
    if (!fits)
      return sample_by_digits<BF16>(p, row.row, noise, w, by_k ? top_k : 0, top_p, min_p, s);

    // The noise of 8 tokens is read whole where one of them is kept, that of
    // four eights at a time.
    const float last_x = last ? value_of(last) : -__builtin_inff();
    const int last_i = last ? index_of(last) : V;
    constexpr int G = 4;
    for (int i0 = t * 8; i0 < V; i0 += G * row.kStep) {
      float x[G][8], u[G][8];
      uint32_t in[G];
#pragma unroll
      for (int g = 0; g < G; ++g)
        if (i0 + g * row.kStep < V) row.load(x[g], i0 + g * row.kStep);
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const int i = i0 + g * row.kStep;
        in[g] = 0;
        if (i >= V) continue;
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (x[g][j] > last_x || (x[g][j] == last_x && i + j <= last_i)) in[g] |= 1u << j;
        if (in[g] == 0) continue;
        if (i + 8 <= V) {
          const Any16 a = reinterpret_cast<const Any16*>(noise + i)[0];
          const Any16 b = reinterpret_cast<const Any16*>(noise + i)[1];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            u[g][j] = __uint_as_float(a.w[j]);
            u[g][4 + j] = __uint_as_float(b.w[j]);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) u[g][j] = noise[min(i + j, V - 1)];
        }
      }
#pragma unroll
      for (int g = 0; g < G; ++g) {
        if (in[g] == 0) continue;
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int i = i0 + g * row.kStep + j;
          const float wi = w.fast(x[g][j]);
          if ((in[g] >> j & 1) && wi > 0.0f && !(wi < min_p)) {
            sum += wi;
            run(wi, i, u[g][j]);
          }
        }
        kept += sum;
      }
    }
    kept = block.sum(kept);
  }
  const uint64_t win = block.reduce(
      score >= 0.0f ? entry_of(__float_as_uint(score), winner) : 0, Max());
  if (t == 0) {
    const int token = index_of(win);  // some token is always kept
    p.tokens[r] = token;
    p.logprobs[r] = w.scaled(logit<BF16>(row.row, token)) - hw_log2((float)kept) * kLn2;
  }
}

}  // namespace

hipError_t launch_sample(const SampleParams& p, bool bf16, hipStream_t st) {
  const dim3 grid((unsigned)p.rows), block(kThreads);
  if (bf16) hipLaunchKernelGGL((sample_kernel<true>), grid, block, 0, st, p);
  else hipLaunchKernelGGL((sample_kernel<false>), grid, block, 0, st, p);
  return hipGetLastError();
}

}  // namespace mssm
