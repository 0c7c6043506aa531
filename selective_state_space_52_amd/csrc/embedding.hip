// embedding.hip -- rows of a table by token, and the table's gradient.
//
//   out[i]    = scale * table[tokens[i]]
//   dtable[v] = scale * sum of dout[i] over the i with tokens[i] = v  (+ dtable[v])
//
// A token outside the table is padding: a zero row, and no gradient.
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
constexpr int kSortRange = 1024;  // most rows of the table a workgroup

struct SortPlan {
  int groups, range;
};
SortPlan sort_plan(int64_t vocab) {
  int64_t range = (vocab + 255) / 256;
  if (range > kSortRange) range = kSortRange;
  return SortPlan{(int)((vocab + range - 1) / range), (int)range};
}

template <bool TBF>
__global__ void __launch_bounds__(kSortThreads)
    embedding_sort_kernel(const int64_t* __restrict__ tokens, int rows, int vocab, int range,
                          int* __restrict__ order, int* __restrict__ named, int* __restrict__ count,
                          void* __restrict__ dtable, int dim) {
  extern __shared__ uint32_t cursor[];  // [kSortWaves][range]
  __shared__ uint32_t part[kSortWaves], below_part[kSortWaves];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int first = blockIdx.x * range;
  const int mine = min(range, vocab - first);
  for (int i = threadIdx.x; i < kSortWaves * range; i += kSortThreads) cursor[i] = 0;
  __syncthreads();
  // each wave takes a run of neighbouring tokens
  const int run = ((rows + kSortThreads - 1) / kSortThreads) * 64;
  const int64_t begin = min((int64_t)rows, (int64_t)wave * run);
  const int64_t end = min((int64_t)rows, begin + run);
  uint32_t below = 0;
  for (int64_t i = begin + lane; i < end; i += 64) {
    const int64_t t = tokens[i];
    if (t >= 0 && t < first) ++below;
    const int64_t at = t - first;
    if (at >= 0 && at < mine) atomicAdd(&cursor[wave * range + (int)at], 1u);
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
  // rows that no token names are cleared here
  __shared__ uint32_t empty[kSortRange / 32];
  const uint64_t none = __ballot(v < mine && total == 0);
  if (lane == 0) empty[wave * 2] = (uint32_t)none, empty[wave * 2 + 1] = (uint32_t)(none >> 32);
  __syncthreads();
  for (int64_t i = begin; i < end; i += 64) {
    const int64_t t = i + lane < end ? tokens[i + lane] : -1;
    const int64_t own = t - first;
    const bool in = own >= 0 && own < mine;
    uint64_t left = __ballot(in);
    while (left) {  // one different token of the 64 a turn
      const int leader = __ffsll((unsigned long long)left) - 1;
      const int token = __builtin_amdgcn_readlane((int)own, leader);
      const uint64_t same = __ballot(in && (int)own == token);
      uint32_t place = 0;
      if (lane == leader)
        place = atomicAdd(&cursor[wave * range + token], (uint32_t)__popcll(same));
      place = __builtin_amdgcn_readlane((int)place, leader);
      if (same >> lane & 1) {
        const uint32_t to = place + (uint32_t)__popcll(same & ((1ull << lane) - 1));
        order[to] = (int)(i + lane);
        named[to] = first + token;
      }
      left &= ~same;
    }
  }
  if (dtable == nullptr) return;
  for (int r = wave; r < mine; r += kSortWaves) {
    if (!(empty[r >> 5] >> (r & 31) & 1)) continue;
    const float zero[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    const int64_t to = (int64_t)(first + r) * dim;
    for (int i = lane * 8; i < dim; i += 512) store8<TBF>(dtable, to + i, dim - i, zero);
  }
}

// A piece of `len` places of the order and 8 columns a lane, 512 a wave.
struct Pieces {
  const int* order;
  const int* named;
  const int* count;
  float* head;   // (pieces, dim): the sum of the token that came in from the piece before
  float* tail;   // (pieces, dim): of the one that goes on into the next
  int len, slices;
};

template <bool TBF>
__device__ __forceinline__ void finish(const EmbedBwdParams& p, int token, int col, float (&sum)[8]) {
  const int n = p.dim - col;
  const int64_t to = (int64_t)token * p.dim + col;
#pragma unroll
  for (int j = 0; j < 8; ++j) sum[j] *= p.scale;
  if (p.add) {
    float old[8];
    load8<TBF>(old, p.dtable, to, n);
#pragma unroll
    for (int j = 0; j < 8; ++j) sum[j] += old[j];
  }
  store8<TBF>(p.dtable, to, n, sum);
}

template <bool TBF, bool OBF>
__global__ void __launch_bounds__(kThreads) embedding_sum_kernel(EmbedBwdParams p, Pieces q) {
  const int64_t item = (int64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6);
  const int64_t piece = item / q.slices;
  const int col = (int)(item % q.slices) * 512 + (threadIdx.x & 63) * 8;
  const int count = *q.count;
  const int64_t begin = piece * q.len, end = min((int64_t)count, begin + q.len);
  if (begin >= count || col >= p.dim) return;
  const int n = p.dim - col;
  bool came_in = begin > 0 && q.named[begin - 1] == q.named[begin];
  const bool goes_on = end < count && q.named[end] == q.named[end - 1];
  float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  int token = q.named[begin];
  for (int64_t i = begin; i < end; ++i) {
    const int next = q.named[i];
    if (next != token) {
      if (came_in)
        store8<false>(q.head, piece * p.dim + col, n, sum);
      else
        finish<TBF>(p, token, col, sum);
      came_in = false;
      token = next;
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[j] = 0.0f;
    }
    float v[8];
    load8<OBF>(v, p.dout, (int64_t)q.order[i] * p.io_stride + col, n);
#pragma unroll
    for (int j = 0; j < 8; ++j) sum[j] += v[j];
  }
  if (came_in)
    store8<false>(q.head, piece * p.dim + col, n, sum);
  else if (goes_on)
    store8<false>(q.tail, piece * p.dim + col, n, sum);
  else
    finish<TBF>(p, token, col, sum);
}

// The piece in which a token across pieces begins adds up its sums, in order.
template <bool TBF>
__global__ void __launch_bounds__(kThreads) embedding_join_kernel(EmbedBwdParams p, Pieces q) {
  const int64_t item = (int64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6);
  const int64_t piece = item / q.slices;
  const int col = (int)(item % q.slices) * 512 + (threadIdx.x & 63) * 8;
  const int count = *q.count;
  const int64_t begin = piece * q.len, end = begin + q.len;
  if (end >= count || col >= p.dim) return;
  const int token = q.named[end];
  if (q.named[end - 1] != token) return;                    // nothing goes on
  if (begin > 0 && q.named[begin - 1] == token) return;     // it began earlier
  const int n = p.dim - col;
  float sum[8];
  load8<false>(sum, q.tail, piece * p.dim + col, n);
  for (int64_t at = end; at < count && q.named[at] == token; at += q.len) {
    float v[8];
    load8<false>(v, q.head, at / q.len * p.dim + col, n);
#pragma unroll
    for (int j = 0; j < 8; ++j) sum[j] += v[j];
  }
  finish<TBF>(p, token, col, sum);
}

constexpr int kLen = 32;
int64_t pieces_of(int64_t rows) { return (rows + kLen - 1) / kLen; }
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
  (void)vocab;
  return 256 + 2 * round256(rows * 4) + 2 * round256(pieces_of(rows) * dim * 4);
}

hipError_t launch_embedding_bwd(const EmbedBwdParams& p, bool table_bf16, bool io_bf16,
                                hipStream_t st) {
  char* ws = static_cast<char*>(p.workspace);
  Pieces q;
  int* count = reinterpret_cast<int*>(ws);
  ws += 256;
  int* order = reinterpret_cast<int*>(ws);
  ws += round256(p.rows * 4);
  int* named = reinterpret_cast<int*>(ws);
  ws += round256(p.rows * 4);
  const int64_t pieces = pieces_of(p.rows);
  q.head = reinterpret_cast<float*>(ws);
  q.tail = reinterpret_cast<float*>(ws + round256(pieces * p.dim * 4));
  q.order = order; q.named = named; q.count = count;
  q.len = kLen;
  q.slices = (p.dim + 511) / 512;
  const SortPlan s = sort_plan(p.vocab);
  const size_t lds = (size_t)kSortWaves * s.range * 4;
  auto sort = table_bf16 ? embedding_sort_kernel<true> : embedding_sort_kernel<false>;
  hipLaunchKernelGGL(sort, dim3((unsigned)s.groups), dim3(kSortThreads), lds, st, p.tokens,
                     (int)p.rows, p.vocab, s.range, order, named, count,
                     p.add ? nullptr : p.dtable, p.dim);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t per = kThreads / 64;
  const dim3 grid((unsigned)((pieces * q.slices + per - 1) / per));
  auto sum = table_bf16 ? (io_bf16 ? embedding_sum_kernel<true, true> : embedding_sum_kernel<true, false>)
                        : (io_bf16 ? embedding_sum_kernel<false, true> : embedding_sum_kernel<false, false>);
  hipLaunchKernelGGL(sum, grid, dim3(kThreads), 0, st, p, q);
  e = hipGetLastError();
  if (e != hipSuccess || pieces == 1) return e;
  auto join = table_bf16 ? embedding_join_kernel<true> : embedding_join_kernel<false>;
  hipLaunchKernelGGL(join, grid, dim3(kThreads), 0, st, p, q);
  return hipGetLastError();
}

}  // namespace mssm
