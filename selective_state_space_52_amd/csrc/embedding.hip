// embedding.hip -- rows of a table by token, and the table's gradient.
//
//   out[i]    = scale * table[tokens[i]]
//   dtable[v] = scale * sum of dout[i] over the i with tokens[i] = v  (+ dtable[v])
//
// A token outside the table is padding: a zero row, and no gradient.
//
// Both move each value once; HBM bounds the large calls, and a call's few waits
// one after another the small ones.  8192 tokens of a 50304 x 2560 bf16 table 11.5 us
// (a text's spread names 3360 rows: 17 MB read and 42 written, 5.1 TB/s); the
// gradient of such a table in fp32 124 us: 515 MB are the table's rows, most of them
// cleared beside the sums (12 us the order, 107 sums and clearing at 5.3 TB/s, 6 the
// join).  1777 tokens added to a 50257 x 769 table 21 us, 7.5 + 9.6 + 4.5 in three
// launches.
#include <type_traits>

#include "fp8.h"
#include "mssm_internal.h"

namespace mssm {
namespace {

constexpr int kThreads = 256;

// A row belongs to `lanes` neighbouring lanes (a power of two up to 64), 8
// columns each in each pass.
template <bool TBF, bool OBF>
__global__ void __launch_bounds__(kThreads) embedding_kernel(EmbedParams p, int lanes_log2) {
  const int lanes = 1 << lanes_log2;
  const int64_t row = (int64_t)blockIdx.x * (kThreads >> lanes_log2) + (threadIdx.x >> lanes_log2);
  if (row >= p.rows) return;
  const int64_t token = p.tokens[row];
  const bool live = token >= 0 && token < p.vocab;
  const int64_t from = live ? token * p.dim : 0, to = row * p.io_stride;
  for (int i = (threadIdx.x & (lanes - 1)) * 8; i < p.dim; i += lanes * 8) {
    const int n = p.dim - i;
    float v[8];
    if (live) {
      load8<TBF>(v, p.table, from + i, n);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= p.scale;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = 0.0f;
    }
    store8<OBF>(p.out, to + i, n, v);
  }
}

// ---- Backward.  Three launches: the rows' indices in order of their tokens
// (equal tokens by rising index), sums over pieces of that order, and the sums
// of the tokens that lie across pieces.

// The order's workgroups divide the table's rows among them.  Each reads every
// token: it counts those below its own and each of its own, which gives its
// place in the order without a word from the others, and then puts its own
// there.  One launch in place of the several of a digit-by-digit sort; the
// tokens come from L2.
constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64;
constexpr int kSortRange = 512;  // most rows of the table a workgroup: 32 KB of counts
constexpr int kSortBits = 10;    // of a row among them, and of none

struct SortPlan {
  int groups, range;
};
SortPlan sort_plan(int64_t vocab) {
  int64_t range = (vocab + 255) / 256;
  if (range > kSortRange) range = kSortRange;
  return SortPlan{(int)((vocab + range - 1) / range), (int)range};
}

// A wave's tokens from i on, 64 apart, as loads that are in flight together; -1
// past the end.
constexpr int kBatch = 8;
__device__ __forceinline__ void load_tokens(int64_t (&t)[kBatch], const int64_t* tokens, int64_t i,
                                            int64_t end) {
#pragma unroll
  for (int b = 0; b < kBatch; ++b) {
    const int64_t at = i + b * 64;
    t[b] = tokens[at < end ? at : end - 1];
    if (at >= end) t[b] = -1;
  }
}

__global__ void __launch_bounds__(kSortThreads)
    embedding_sort_kernel(const int64_t* __restrict__ tokens, int rows, int vocab, int range,
                          int* __restrict__ order, int* __restrict__ named, int* __restrict__ count,
                          uint8_t* __restrict__ present) {
  extern __shared__ uint32_t cursor[];  // [kSortWaves][range]
  __shared__ uint32_t part[kSortWaves], below_part[kSortWaves];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int first = blockIdx.x * range;
  const int mine = min(range, vocab - first);
  // each wave takes a run of neighbouring tokens; the first batch stays
  const int run = ((rows + kSortThreads - 1) / kSortThreads) * 64;
  const int64_t begin = min((int64_t)rows, (int64_t)wave * run);
  const int64_t end = min((int64_t)rows, begin + run);
  int64_t held[kBatch];
  if (begin < end) load_tokens(held, tokens, begin + lane, end);
  for (int i = threadIdx.x; i < kSortWaves * range; i += kSortThreads) cursor[i] = 0;
  __syncthreads();
  uint32_t below = 0;
  for (int64_t i = begin; i < end; i += 64 * kBatch) {
    int64_t t[kBatch];
    if (i == begin) {
#pragma unroll
      for (int b = 0; b < kBatch; ++b) t[b] = held[b];
    } else {
      load_tokens(t, tokens, i + lane, end);
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      if (t[b] >= 0 && t[b] < first) ++below;
      const int64_t at = t[b] - first;
      if (at >= 0 && at < mine) atomicAdd(&cursor[wave * range + (int)at], 1u);
    }
  }
  for (int d = 32; d > 0; d >>= 1) below += __shfl_xor(below, d);
  if (lane == 0) below_part[wave] = below;
  __syncthreads();
  // thread v: where row v's tokens begin, for each wave
  uint32_t total = 0;
  const int v = threadIdx.x;
  if (v < mine)
    for (int w = 0; w < kSortWaves; ++w) total += cursor[w * range + v];
  uint32_t upto = total;
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t o = __shfl_up(upto, d);
    if (lane >= d) upto += o;
  }
  if (lane == 63) part[wave] = upto;
  __syncthreads();
  uint32_t base = 0;
  for (int w = 0; w < kSortWaves; ++w) {
    base += below_part[w];
    if (w < wave) base += part[w];
  }
  uint32_t at = base + upto - total;
  if (v < mine)
    for (int w = 0; w < kSortWaves; ++w) {
      const uint32_t c = cursor[w * range + v];
      cursor[w * range + v] = at;
      at += c;
    }
  if (blockIdx.x == gridDim.x - 1 && v == mine - 1) *count = (int)at;
  if (present && v < mine) present[first + v] = total != 0;
  __syncthreads();
  for (int64_t i = begin; i < end; i += 64 * kBatch) {
    int64_t t[kBatch];
    if (i == begin) {
#pragma unroll
      for (int b = 0; b < kBatch; ++b) t[b] = held[b];
    } else {
      load_tokens(t, tokens, i + lane, end);
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int64_t own = t[b] - first;
      const bool in = own >= 0 && own < mine;
      const uint64_t any = __ballot(in);
      if (!any) continue;
      if (__popcll(any) <= 2) {
        for (uint64_t left = any; left; left &= left - 1) {
          const int who = __builtin_ctzll(left);
          if (lane == who) {
            const uint32_t to = atomicAdd(&cursor[wave * range + (int)own], 1u);
            order[to] = (int)(i + b * 64 + lane);
            named[to] = first + (int)own;
          }
        }
        continue;
      }
      // the lanes with this lane's token, from a ballot for each of its bits; the
      // first of them takes places for all.  (One lane a turn, as above, takes 470 us
      // for 65536 tokens half of which fall in one range, as a vocabulary in order of
      // frequency has it, and both 68.  This alone 9 and 35 us for 8192 and 65536
      // evenly spread tokens, both 7.3 and 26; for 8192 of a text 11.5 and 11.6.)
      const uint32_t id = in ? (uint32_t)own : (uint32_t)kSortRange;
      uint64_t same = ~0ull;
#pragma unroll
      for (int bit = 0; bit < kSortBits; ++bit) {
        const uint64_t has = __ballot(id >> bit & 1);
        same &= id >> bit & 1 ? has : ~has;
      }
      const int leader = __builtin_ctzll(same);
      uint32_t place = 0;
      if (in && lane == leader)
        place = atomicAdd(&cursor[wave * range + (int)own], (uint32_t)__popcll(same));
      place = (uint32_t)__shfl((int)place, leader);
      if (in) {
        const uint32_t to = place + (uint32_t)__popcll(same & ((1ull << lane) - 1));
        order[to] = (int)(i + b * 64 + lane);
        named[to] = first + (int)own;
      }
    }
  }
}

// A piece of `len` places of the order and 8 columns a lane, 512 a wave.
struct Pieces {
  const int* order;
  const int* named;
  const int* count;
  const uint8_t* present;
  float* head;   // (pieces, dim): the sum of the token that came in from the piece before
  float* tail;   // (pieces, dim): of the one that goes on into the next
  int len, slices;
  int sums;      // workgroups that sum; those after them clear
  U32Div chunks; // 16 bytes each, of a row of the gradient
};

// The token's row from its sum, and from what it held (ADD).
template <bool TBF, bool ADD>
__device__ __forceinline__ void finish(const EmbedBwdParams& p, int token, int col, float (&sum)[8],
                                       const float (&old)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) sum[j] = ADD ? sum[j] * p.scale + old[j] : sum[j] * p.scale;
  store8<TBF>(p.dtable, (int64_t)token * p.dim + col, p.dim - col, sum);
}

// Clears the rows that no token names, in pieces of 16 bytes: kClear a thread.
constexpr int kClear = 16;
template <bool TBF, typename Present>
__device__ __forceinline__ void clear_rows(const EmbedBwdParams& p, U32Div div, int64_t block,
                                           Present present) {
  constexpr int kCols = TBF ? 8 : 4;
  typedef typename std::conditional<TBF, uint16_t, uint32_t>::type T;
  const int chunks = (p.dim + kCols - 1) / kCols;
  const int64_t first = block * (kThreads * kClear);
  const int64_t row0 = first / chunks;
  const uint32_t at0 = (uint32_t)(first - row0 * chunks) + threadIdx.x;
#pragma unroll 4
  for (int c = 0; c < kClear; ++c) {
    const uint32_t at = at0 + c * kThreads, down = udiv(at, div);
    const int64_t row = row0 + down;
    if (row >= p.vocab) return;
    const int col = (int)(at - down * chunks) * kCols, n = p.dim - col;
    if (present(row, down)) continue;
    T* to = static_cast<T*>(p.dtable) + row * p.dim + col;
    if (n >= kCols) {
      *reinterpret_cast<Any16*>(to) = Any16{{0, 0, 0, 0}};
    } else {
      for (int j = 0; j < n; ++j) to[j] = 0;
    }
  }
}

constexpr int kRows = 8;  // whose loads are in flight together

// One wave a piece and slice of columns.  Its lanes hold the piece's rows and
// tokens; 8 rows' loads are in flight together.
template <bool TBF, bool OBF, bool ADD>
__global__ void __launch_bounds__(kThreads) embedding_sum_kernel(EmbedBwdParams p, Pieces q) {
  if ((int)blockIdx.x >= q.sums) {
    clear_rows<TBF>(p, q.chunks, (int)blockIdx.x - q.sums,
                    [&](int64_t row, uint32_t) { return q.present[row] != 0; });
    return;
  }
  const int64_t item = (int64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6);
  const int64_t piece = item / q.slices;
  const int lane = threadIdx.x & 63;
  const int col = (int)(item % q.slices) * 512 + lane * 8;
  const int64_t begin = piece * q.len, last_row = p.rows - 1;
  // one wait for all of them: places behind the count are in the arrays, and what
  // they hold is not used
  const int64_t at = min(begin + lane, last_row);
  const int count = __builtin_amdgcn_readfirstlane(*q.count);
  const int rows = q.order[at], names = q.named[at];
  const int prior = q.named[begin > 0 ? min(begin - 1, last_row) : 0];
  const int next = q.named[min(begin + q.len, last_row)];
  if (begin >= count) return;
  const int len = (int)min((int64_t)q.len, count - begin);
  bool came_in = begin > 0 && prior == __builtin_amdgcn_readfirstlane(names);
  const bool goes_on =
      begin + len < count && next == __builtin_amdgcn_readlane(names, len - 1);
  const int n = p.dim - col;
  const bool whole = n >= 8;
  float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  for (int i = 0; i < len; i += kRows) {
    Raw8<OBF> raw[kRows];
    Raw8<TBF> held_old[kRows];
    if (whole) {
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const int64_t row = __builtin_amdgcn_readlane(rows, min(i + r, len - 1));
        raw[r] = load_raw8<OBF>(p.dout, row * p.io_stride + col);
      }
      if constexpr (ADD) {
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          // what the row of a token that ends here holds
          const int name = __builtin_amdgcn_readlane(names, min(i + r, len - 1));
          if (i + r >= len - 1 || name != __builtin_amdgcn_readlane(names, i + r + 1))
            held_old[r] = load_raw8<TBF>(p.dtable, (int64_t)name * p.dim + col);
        }
      }
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      if (i + r >= len) break;
      float v[8];
      if (whole)
        unpack8<OBF>(v, raw[r]);
      else if (n > 0)
        load8<OBF>(v, p.dout, (int64_t)__builtin_amdgcn_readlane(rows, i + r) * p.io_stride + col, n);
      else
        for (int j = 0; j < 8; ++j) v[j] = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[j] += v[j];
      const bool last = i + r == len - 1;
      const int token = __builtin_amdgcn_readlane(names, i + r);
      if (!last && token == __builtin_amdgcn_readlane(names, i + r + 1)) continue;
      if (n > 0) {
        if (came_in) {
          store8<false>(q.head, piece * p.dim + col, n, sum);
        } else if (last && goes_on) {
          store8<false>(q.tail, piece * p.dim + col, n, sum);
        } else {
          float old[8];
          if constexpr (ADD) {
            if (whole)
              unpack8<TBF>(old, held_old[r]);
            else
              load8<TBF>(old, p.dtable, (int64_t)token * p.dim + col, n);
          }
          finish<TBF, ADD>(p, token, col, sum, old);
        }
      }
      came_in = false;
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[j] = 0.0f;
    }
  }
}

// The piece in which a token across pieces begins adds up its sums: a workgroup
// for it and a slice of columns, whose waves take runs of the pieces, 8 loads in
// flight, and are added in order.
constexpr int kJoinWaves = kThreads / 64;
template <bool TBF, bool ADD>
__global__ void __launch_bounds__(kThreads) embedding_join_kernel(EmbedBwdParams p, Pieces q) {
  __shared__ float part[kJoinWaves][64][9];
  const int64_t piece = blockIdx.x / q.slices;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int col = (int)(blockIdx.x % q.slices) * 512 + lane * 8;
  const int count = *q.count;
  const int64_t begin = piece * q.len, end = begin + q.len;
  if (end >= count) return;
  const int token = q.named[end];
  if (q.named[end - 1] != token) return;                 // nothing goes on
  if (begin > 0 && q.named[begin - 1] == token) return;  // it began earlier
  // the pieces that it reaches: 64 of their first places a turn
  int64_t pieces = 0;
  for (;;) {
    const int64_t at = end + (pieces + lane) * q.len;
    const uint64_t in = __ballot(at < count && q.named[at < count ? at : 0] == token);
    if (in != ~0ull) {
      pieces += __builtin_ctzll(~in);
      break;
    }
    pieces += 64;
  }
  const int n = p.dim - col;
  const int64_t each = (pieces + kJoinWaves - 1) / kJoinWaves;
  const int64_t from = wave * each, to = min(pieces, from + each);
  float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  float old[8];
  if (n > 0) {
    if (wave == 0) load8<false>(sum, q.tail, piece * p.dim + col, n);
    if (ADD && wave == 0) load8<TBF>(old, p.dtable, (int64_t)token * p.dim + col, n);
    const int64_t at = (piece + 1) * p.dim + col;
    for (int64_t i = from; i < to; i += kRows) {
      float v[kRows][8];
#pragma unroll
      for (int r = 0; r < kRows; ++r) load8<false>(v[r], q.head, at + min(i + r, to - 1) * p.dim, n);
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        if (i + r >= to) break;
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[j] += v[r][j];
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) part[wave][lane][j] = sum[j];
  __syncthreads();
  if (wave != 0 || n <= 0) return;
  for (int w = 1; w < kJoinWaves; ++w)
#pragma unroll
    for (int j = 0; j < 8; ++j) sum[j] += part[w][lane][j];
  finish<TBF, ADD>(p, token, col, sum, old);
}

// Few rows: one launch and no order (81 rows into 28638 x 270: 8 us a call, 24 with
// the three launches; the comparisons grow with the square of the rows).  A
// workgroup takes a row and 512 columns and
// compares the row's token with all others; where no earlier row has it, its
// waves add up the rows that have it (in parts, added in order).
constexpr int kDirect = 512;
template <bool TBF, bool OBF, bool ADD>
__global__ void __launch_bounds__(kThreads)
    embedding_direct_kernel(EmbedBwdParams p, int slices, int sums, U32Div chunks) {
  __shared__ uint64_t same[kDirect / 64];
  __shared__ float part[kJoinWaves][64][9];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int rows = (int)p.rows;
  if ((int)blockIdx.x >= sums) {
    __shared__ uint8_t named[kThreads * kClear + 8];
    const int64_t block = (int)blockIdx.x - sums;
    for (int i = threadIdx.x; i < kThreads * kClear + 8; i += kThreads) named[i] = 0;
    __syncthreads();
    constexpr int kCols = TBF ? 8 : 4;
    const int64_t row0 = block * (kThreads * kClear) / ((p.dim + kCols - 1) / kCols);
    for (int i = threadIdx.x; i < rows; i += kThreads) {
      const int64_t at = p.tokens[i] - row0;
      if (at >= 0 && at < kThreads * kClear + 8) named[at] = 1;
    }
    __syncthreads();
    clear_rows<TBF>(p, chunks, block, [&](int64_t, uint32_t down) { return named[down] != 0; });
    return;
  }
  const int row = (int)(blockIdx.x / slices);
  const int col = (int)(blockIdx.x % slices) * 512 + lane * 8, n = p.dim - col;
  const int64_t token = p.tokens[row];
  if (token < 0 || token >= p.vocab) return;
  const int words = (rows + 63) / 64;
  for (int k = wave; k < words; k += kJoinWaves) {
    const int i = k * 64 + lane;
    const uint64_t m = __ballot(i < rows && p.tokens[min(i, rows - 1)] == token);
    if (lane == 0) same[k] = m;
  }
  float old[8];
  if (ADD && wave == 0 && n > 0) load8<TBF>(old, p.dtable, token * p.dim + col, n);
  __syncthreads();
  int total = 0;
  for (int k = 0; k < words; ++k) total += __popcll(same[k]);
  int before = __popcll(same[row >> 6] & ((1ull << (row & 63)) - 1));
  for (int k = 0; k < row >> 6; ++k) before += __popcll(same[k]);
  total = __builtin_amdgcn_readfirstlane(total);
  if (__builtin_amdgcn_readfirstlane(before)) return;
  const bool alone = total <= kRows;  // the first wave's
  const int each = alone ? total : (total + kJoinWaves - 1) / kJoinWaves;
  int left = min(each, total - wave * each);
  if (alone && wave != 0) return;
  // from this wave's first of the rows
  int word = 0, skip = wave * each;
  uint64_t bits = 0;
  if (left > 0) {
    bits = same[0];
    while (skip >= __popcll(bits)) {
      skip -= __popcll(bits);
      bits = same[++word];
    }
    for (; skip > 0; --skip) bits &= bits - 1;
  }
  float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  while (left > 0) {
    const int now = min(left, kRows);
    int at[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      if (r < now) {
        while (bits == 0) bits = same[++word];
        at[r] = word * 64 + __builtin_ctzll(bits);
        bits &= bits - 1;
      } else {
        at[r] = at[r ? r - 1 : 0];
      }
    }
    if (n >= 8) {
      Raw8<OBF> raw[kRows];
#pragma unroll
      for (int r = 0; r < kRows; ++r)
        raw[r] = load_raw8<OBF>(p.dout, (int64_t)at[r] * p.io_stride + col);
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        if (r >= now) break;
        float v[8];
        unpack8<OBF>(v, raw[r]);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[j] += v[j];
      }
    } else if (n > 0) {
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        if (r >= now) break;
        float v[8];
        load8<OBF>(v, p.dout, (int64_t)at[r] * p.io_stride + col, n);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[j] += v[j];
      }
    }
    left -= now;
  }
  if (!alone) {
#pragma unroll
    for (int j = 0; j < 8; ++j) part[wave][lane][j] = sum[j];
    __syncthreads();
    if (wave != 0) return;
    for (int w = 1; w < kJoinWaves; ++w)
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[j] += part[w][lane][j];
  }
  if (n > 0) finish<TBF, ADD>(p, (int)token, col, sum, old);
}

// Places of a piece: 8 at least, 64 (its wave's lanes) at most, in between as
// many as give 2048 waves.
int len_of(int64_t rows, int64_t dim) {
  const int64_t waves = rows * ((dim + 511) / 512);
  int len = 8;
  while (len < 64 && waves / len > 2048) len *= 2;
  return len;
}
int64_t pieces_of(int64_t rows, int64_t dim) {
  const int len = len_of(rows, dim);
  return (rows + len - 1) / len;
}
int64_t round256(int64_t n) { return (n + 255) / 256 * 256; }

}  // namespace

hipError_t launch_embedding(const EmbedParams& p, bool table_bf16, bool io_bf16, hipStream_t st) {
  int log2 = 0;
  while (log2 < 6 && (8 << log2) < p.dim) ++log2;
  const int64_t per = kThreads >> log2;
  const dim3 grid((unsigned)((p.rows + per - 1) / per));
  auto kernel = table_bf16 ? (io_bf16 ? embedding_kernel<true, true> : embedding_kernel<true, false>)
                           : (io_bf16 ? embedding_kernel<false, true> : embedding_kernel<false, false>);
  hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, st, p, log2);
  return hipGetLastError();
}

int64_t embedding_bwd_workspace(int64_t rows, int64_t vocab, int64_t dim) {
  if (rows <= kDirect) return 0;
  return 256 + 2 * round256(rows * 4) + round256(vocab) +
         2 * round256(pieces_of(rows, dim) * dim * 4);
}

template <bool TBF, bool OBF, bool ADD>
static hipError_t launch_bwd(const EmbedBwdParams& p, hipStream_t st) {
  const int64_t chunks = TBF ? (p.dim + 7) / 8 : (p.dim + 3) / 4;
  const int64_t clears = ADD ? 0 : (p.vocab * chunks + kThreads * kClear - 1) / (kThreads * kClear);
  const U32Div div = make_u32div((uint32_t)chunks);
  const int slices = (p.dim + 511) / 512;
  if (p.rows <= kDirect) {
    const int64_t sums = p.rows * slices;
    hipLaunchKernelGGL((embedding_direct_kernel<TBF, OBF, ADD>), dim3((unsigned)(sums + clears)),
                       dim3(kThreads), 0, st, p, slices, (int)sums, div);
    return hipGetLastError();
  }
  char* ws = static_cast<char*>(p.workspace);
  int* count = reinterpret_cast<int*>(ws);
  ws += 256;
  int* order = reinterpret_cast<int*>(ws);
  ws += round256(p.rows * 4);
  int* named = reinterpret_cast<int*>(ws);
  ws += round256(p.rows * 4);
  uint8_t* present = ADD ? nullptr : reinterpret_cast<uint8_t*>(ws);
  ws += round256(p.vocab);
  const int64_t pieces = pieces_of(p.rows, p.dim);
  Pieces q;
  q.head = reinterpret_cast<float*>(ws);
  q.tail = reinterpret_cast<float*>(ws + round256(pieces * p.dim * 4));
  q.order = order; q.named = named; q.count = count; q.present = present;
  q.len = len_of(p.rows, p.dim);
  q.slices = slices;
  q.chunks = div;
  const SortPlan s = sort_plan(p.vocab);
  hipLaunchKernelGGL(embedding_sort_kernel, dim3((unsigned)s.groups), dim3(kSortThreads),
                     (size_t)kSortWaves * s.range * 4, st, p.tokens, (int)p.rows, p.vocab, s.range,
                     order, named, count, present);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t per = kThreads / 64;
  q.sums = (int)((pieces * slices + per - 1) / per);
  hipLaunchKernelGGL((embedding_sum_kernel<TBF, OBF, ADD>), dim3((unsigned)(q.sums + clears)),
                     dim3(kThreads), 0, st, p, q);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((embedding_join_kernel<TBF, ADD>), dim3((unsigned)((pieces - 1) * slices)),
                     dim3(kThreads), 0, st, p, q);
  return hipGetLastError();
}

hipError_t launch_embedding_bwd(const EmbedBwdParams& p, bool table_bf16, bool io_bf16,
                                hipStream_t st) {
  if (p.add)
    return table_bf16 ? (io_bf16 ? launch_bwd<true, true, true>(p, st) : launch_bwd<true, false, true>(p, st))
                      : (io_bf16 ? launch_bwd<false, true, true>(p, st) : launch_bwd<false, false, true>(p, st));
  return table_bf16 ? (io_bf16 ? launch_bwd<true, true, false>(p, st) : launch_bwd<true, false, false>(p, st))
                    : (io_bf16 ? launch_bwd<false, true, false>(p, st) : launch_bwd<false, false, false>(p, st));
}

}  // namespace mssm
