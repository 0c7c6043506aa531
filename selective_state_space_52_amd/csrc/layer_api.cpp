// layer_api.cpp -- the C ABI of the layer's operators around the scans
// (declared in include/mssm.h): argument validation, always before the first
// HIP call, and dispatch on the caller's stream.
#include <hip/hip_runtime.h>

#include <cstring>
#include <initializer_list>

#include "mssm.h"
#include "mssm_internal.h"

namespace {

constexpr int64_t kMost = INT64_MAX / 16;  // elements of one array
constexpr int64_t kGrid = INT32_MAX;       // workgroups of one launch
constexpr int64_t kItems = UINT32_MAX;     // threads of one launch

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
int64_t blocks128(int64_t n) { return (n + 127) / 128; }
int64_t size_of(int32_t dtype) { return dtype == MSSM_BF16 ? 2 : 4; }
bool known(int32_t dtype) { return dtype == MSSM_F32 || dtype == MSSM_BF16; }

// a * b <= limit for positive a, b.
bool fits(int64_t a, int64_t b, int64_t limit = kMost) { return a > 0 && b > 0 && a <= limit / b; }

struct Range {
  uintptr_t lo, hi;  // [lo, hi)
};
Range range(const void* p, int64_t bytes) {
  return p && bytes > 0 ? Range{(uintptr_t)p, (uintptr_t)p + (uintptr_t)bytes} : Range{0, 0};
}
// Rows of `cols` elements, `stride` apart.
Range rows_range(const void* p, int64_t rows, int64_t cols, int64_t stride, int64_t size) {
  return range(p, ((rows - 1) * stride + cols) * size);
}
bool overlap(Range a, Range b) {
  return a.lo != a.hi && b.lo != b.hi && a.lo < b.hi && b.lo < a.hi;
}
// Whether an output overlaps an input or another output.
bool aliased(std::initializer_list<Range> outs, std::initializer_list<Range> ins) {
  for (const Range* o = outs.begin(); o != outs.end(); ++o) {
    for (const Range& i : ins)
      if (overlap(*o, i)) return true;
    for (const Range* q = o + 1; q != outs.end(); ++q)
      if (overlap(*o, *q)) return true;
  }
  return false;
}
bool all_aligned(std::initializer_list<const void*> ps, size_t a) {
  for (const void* p : ps)
    if (p && !aligned(p, a)) return false;
  return true;
}

int done(hipError_t e, const char* what) {
  if (e == hipSuccess) return MSSM_OK;
  mssm::set_hip_error(what, e);
  return MSSM_ERR_HIP;
}

int check_norm_dims(const mssm_norm_dims* d) {
  if (!d) return MSSM_ERR_NULL;
  if (!known(d->io_dtype) || !known(d->res_dtype)) return MSSM_ERR_UNSUPPORTED;
  if (d->rows <= 0 || d->dim <= 0 || d->rows > kGrid || !fits(d->rows, d->dim))
    return MSSM_ERR_DIMS;
  if (d->dim > mssm::rms_norm_max_dim()) return MSSM_ERR_UNSUPPORTED;
  if (!fits(d->rows, (d->dim / 8 + 256) / 64 * 64, kItems)) return MSSM_ERR_DIMS;
  if (d->x_stride != 0 && (d->x_stride < d->dim || !fits(d->rows, d->x_stride)))
    return MSSM_ERR_DIMS;
  return MSSM_OK;
}

int norm_fwd(const void* x, const void* residual, const float* weight, void* out, void* scales,
             bool fp8, void* residual_out, float* rstd, const mssm_norm_dims* dims, void* stream) {
  const int rc = check_norm_dims(dims);
  if (rc != MSSM_OK) return rc;
  if (!x || !weight || !out || (fp8 && !scales)) return MSSM_ERR_NULL;
  if (residual_out && !residual) return MSSM_ERR_NULL;
  if (!(dims->eps >= 0.0f)) return MSSM_ERR_DIMS;
  const int64_t rows = dims->rows, dim = dims->dim;
  const int64_t stride = dims->x_stride ? dims->x_stride : dim;
  const int64_t io = size_of(dims->io_dtype), rs = size_of(dims->res_dtype);
  if (!aligned(x, io) || !all_aligned({residual, residual_out}, rs) ||
      !all_aligned({weight, rstd}, 4) || (!fp8 && !aligned(out, io)))
    return MSSM_ERR_ALIGN;
  const Range r_res = range(residual, rows * dim * rs);
  const Range r_out = range(out, rows * dim * (fp8 ? 1 : io));
  const Range r_sc = range(fp8 ? scales : nullptr, rows * blocks128(dim));
  const Range r_rstd = range(rstd, rows * 4);
  const Range r_x = rows_range(x, rows, dim, stride, io), r_w = range(weight, dim * 4);
  // the stream may be updated in place
  const Range r_ro = residual_out == residual ? Range{0, 0} : range(residual_out, rows * dim * rs);
  if (aliased({r_out, r_sc, r_rstd, r_ro}, {r_x, r_res, r_w})) return MSSM_ERR_ALIAS;
  if (residual_out == residual && aliased({r_res}, {r_x, r_w})) return MSSM_ERR_ALIAS;
  mssm::NormParams p;
  std::memset(&p, 0, sizeof(p));
  p.x = x; p.residual = residual; p.weight = weight; p.out = out;
  p.scales = fp8 ? static_cast<uint8_t*>(scales) : nullptr;
  p.residual_out = residual_out; p.rstd = rstd;
  p.rows = rows; p.dim = (int32_t)dim; p.x_stride = stride; p.scale_cols = blocks128(dim);
  p.eps = dims->eps;
  const int res = !residual ? 0 : dims->res_dtype == MSSM_BF16 ? 1 : 2;
  return done(mssm::launch_rms_norm(p, dims->io_dtype == MSSM_BF16, res, (hipStream_t)stream),
              "rms norm launch");
}

int check_step_dims(const mssm_step_dims* d) {
  if (!d) return MSSM_ERR_NULL;
  if (!known(d->io_dtype)) return MSSM_ERR_UNSUPPORTED;
  if (d->batch <= 0 || d->nheads <= 0 || d->ngroups <= 0 || d->cache <= 0) return MSSM_ERR_DIMS;
  if (d->headdim != 64 || (d->dstate != 64 && d->dstate != 128) || d->width < 2 || d->width > 4 ||
      d->nheads % d->ngroups != 0)
    return MSSM_ERR_UNSUPPORTED;
  // a head, or half of one, a workgroup
  if (!fits(d->nheads, 64, INT32_MAX / 8) || !fits(d->ngroups, 2 * d->dstate, INT32_MAX / 8) ||
      !fits(d->batch, d->nheads * 2, kItems / 256))
    return MSSM_ERR_DIMS;
  const int64_t channels = d->nheads * 64 + 2 * d->ngroups * d->dstate;
  if (!fits(d->batch, channels) || !fits(d->cache, channels, kMost / 4) ||
      !fits(d->cache, d->nheads * 64 * d->dstate))
    return MSSM_ERR_DIMS;
  const int64_t least[3] = {channels, d->nheads, d->nheads * 64};
  const int64_t strides[3] = {d->xbc_stride, d->dt_stride, d->z_stride};
  for (int i = 0; i < 3; ++i)
    if (strides[i] != 0 && (strides[i] < least[i] || !fits(d->batch, strides[i])))
      return MSSM_ERR_DIMS;
  return MSSM_OK;
}

}  // namespace

extern "C" {

int mssm_rms_norm_fwd(const void* x, const void* residual, const float* weight, void* out,
                      void* residual_out, float* rstd, const mssm_norm_dims* dims, void* stream) {
  return norm_fwd(x, residual, weight, out, nullptr, false, residual_out, rstd, dims, stream);
}

int mssm_rms_norm_fwd_fp8(const void* x, const void* residual, const float* weight, void* q,
                          void* scales, void* residual_out, float* rstd,
                          const mssm_norm_dims* dims, void* stream) {
  return norm_fwd(x, residual, weight, q, scales, true, residual_out, rstd, dims, stream);
}

int mssm_rms_norm_bwd_workspace(const mssm_norm_dims* dims, int64_t* bytes) {
  if (!bytes) return MSSM_ERR_NULL;
  const int rc = check_norm_dims(dims);
  if (rc != MSSM_OK) return rc;
  *bytes = mssm::rms_norm_bwd_workspace(dims->rows, (int)dims->dim, mssm::compute_units());
  return MSSM_OK;
}

int mssm_rms_norm_bwd(const void* dout, const void* r, const float* weight, const float* rstd,
                      const void* dresidual, void* dx, void* dr, float* dweight, void* workspace,
                      int64_t workspace_bytes, const mssm_norm_dims* dims, int has_residual,
                      void* stream) {
  int rc = check_norm_dims(dims);
  if (rc != MSSM_OK) return rc;
  if (!dout || !r || !weight || !rstd || !dx || !dweight) return MSSM_ERR_NULL;
  if (!has_residual && (dresidual || dr)) return MSSM_ERR_NULL;
  if (dims->x_stride != 0 && dims->x_stride != dims->dim) return MSSM_ERR_DIMS;
  const int64_t rows = dims->rows, dim = dims->dim;
  const int64_t io = size_of(dims->io_dtype);
  const int64_t rs = has_residual ? size_of(dims->res_dtype) : io;
  if (!all_aligned({dout, dx}, io) || !all_aligned({r, dresidual, dr}, rs) ||
      !all_aligned({weight, rstd, dweight}, 4))
    return MSSM_ERR_ALIGN;
  const Range r_dx = range(dx, rows * dim * io), r_dr = range(dr, rows * dim * rs);
  const Range r_dw = range(dweight, dim * 4);
  const Range r_dout = range(dout, rows * dim * io), r_r = range(r, rows * dim * rs);
  const Range r_w = range(weight, dim * 4), r_rstd = range(rstd, rows * 4);
  const Range r_dres = range(dresidual, rows * dim * rs);
  if (aliased({r_dx, r_dr, r_dw}, {r_dout, r_r, r_w, r_rstd, r_dres})) return MSSM_ERR_ALIAS;
  // one that is missing or misaligned, whatever the size
  rc = mssm::check_workspace(workspace, workspace_bytes, 1);
  if (rc != MSSM_OK) return rc;
  // the first HIP call: the size goes by the device's compute units
  const int cus = mssm::compute_units();
  const int64_t need = mssm::rms_norm_bwd_workspace(rows, (int)dim, cus);
  rc = mssm::check_workspace(workspace, workspace_bytes, need);
  if (rc != MSSM_OK) return rc;
  if (aliased({range(workspace, need)}, {r_dx, r_dr, r_dw, r_dout, r_r, r_w, r_rstd, r_dres}))
    return MSSM_ERR_ALIAS;
  mssm::NormBwdParams p;
  std::memset(&p, 0, sizeof(p));
  p.dout = dout; p.r = r; p.weight = weight; p.rstd = rstd; p.dresidual = dresidual;
  p.dx = dx; p.dr = dr; p.dw = dweight; p.partial = static_cast<float*>(workspace);
  p.rows = rows; p.dim = (int32_t)dim;
  const int res = !has_residual ? 0 : dims->res_dtype == MSSM_BF16 ? 1 : 2;
  return done(mssm::launch_rms_norm_bwd(p, dims->io_dtype == MSSM_BF16, res, cus,
                                        (hipStream_t)stream),
              "rms norm backward launch");
}

int mssm_quantize_fp8(const void* x, void* q, void* scales, const mssm_quant_dims* dims,
                      void* stream) {
  if (!dims) return MSSM_ERR_NULL;
  if (!known(dims->io_dtype) || (dims->block_rows != 1 && dims->block_rows != 128))
    return MSSM_ERR_UNSUPPORTED;
  const int64_t rows = dims->rows, cols = dims->cols;
  const int64_t stride = dims->x_stride ? dims->x_stride : cols;
  if (!fits(rows, cols) || stride < cols || !fits(rows, stride)) return MSSM_ERR_DIMS;
  const bool square = dims->block_rows == 128, t = dims->transpose != 0;
  const bool rowwise = !square && !t;
  const int64_t nb = rowwise ? rows * blocks128(cols) / 16 : blocks128(rows) * blocks128(cols);
  if (nb >= kItems / 512) return MSSM_ERR_DIMS;
  if (!x || !q || !scales) return MSSM_ERR_NULL;
  const int64_t io = size_of(dims->io_dtype);
  if (!aligned(x, io)) return MSSM_ERR_ALIGN;
  const int64_t sr = square ? blocks128(t ? cols : rows) : t ? cols : rows;
  const int64_t sc = blocks128(t ? rows : cols);
  if (aliased({range(q, rows * cols), range(scales, sr * sc)},
              {rows_range(x, rows, cols, stride, io)}))
    return MSSM_ERR_ALIAS;
  const mssm::QuantParams p{x, static_cast<uint8_t*>(q), static_cast<uint8_t*>(scales), rows, cols,
                            stride, square, t};
  return done(mssm::launch_quantize_fp8(p, dims->io_dtype == MSSM_BF16, (hipStream_t)stream),
              "quantize launch");
}

int mssm_fp8_matmul(const void* a, const void* a_scales, const void* b, const void* b_scales,
                    void* out, const mssm_matmul_dims* dims, void* stream) {
  if (!dims) return MSSM_ERR_NULL;
  if (!known(dims->out_dtype) || (dims->b_block_rows != 1 && dims->b_block_rows != 128))
    return MSSM_ERR_UNSUPPORTED;
  const int64_t M = dims->m, N = dims->n, K = dims->k;
  if (!fits(M, N) || !fits(M, K) || !fits(N, K) || K > (1 << 22) ||
      (M + 63) / 64 > kItems / 256 / ((N + 63) / 64) || N / 16 >= kItems / 512)
    return MSSM_ERR_DIMS;
  if (!a || !a_scales || !b || !b_scales || !out) return MSSM_ERR_NULL;
  const int64_t size = size_of(dims->out_dtype);
  if (!aligned(out, size)) return MSSM_ERR_ALIGN;
  const int64_t kb = blocks128(K), nb = dims->b_block_rows == 128 ? blocks128(N) : N;
  if (aliased({range(out, M * N * size)},
              {range(a, M * K), range(a_scales, M * kb), range(b, N * K), range(b_scales, nb * kb)}))
    return MSSM_ERR_ALIAS;
  const mssm::MatmulParams p{static_cast<const uint8_t*>(a), static_cast<const uint8_t*>(a_scales),
                             static_cast<const uint8_t*>(b), static_cast<const uint8_t*>(b_scales),
                             out, M, N, K, dims->b_block_rows};
  return done(mssm::launch_fp8_matmul(p, dims->out_dtype == MSSM_BF16, mssm::compute_units(),
                                      (hipStream_t)stream),
              "fp8 product launch");
}

int mssm_sample(const void* logits, const float* noise, int64_t* tokens, float* logprobs,
                const mssm_sample_args* args, void* stream) {
  if (!args) return MSSM_ERR_NULL;
  if (!known(args->io_dtype)) return MSSM_ERR_UNSUPPORTED;
  const int64_t rows = args->rows, V = args->vocab;
  const int64_t ls = args->logits_stride ? args->logits_stride : V;
  const int64_t ns = args->noise_stride ? args->noise_stride : V;
  if (rows <= 0 || V <= 0 || rows > kItems / 1024 || V > (1 << 22) || ls < V || ns < V ||
      !fits(rows, ls) || !fits(rows, ns))
    return MSSM_ERR_DIMS;
  if (!logits || !noise || !tokens || !logprobs) return MSSM_ERR_NULL;
  const int64_t io = size_of(args->io_dtype);
  if (!aligned(logits, io) || !aligned(tokens, 8) ||
      !all_aligned({noise, logprobs, args->temperature_row, args->top_k_row, args->top_p_row,
                    args->min_p_row}, 4))
    return MSSM_ERR_ALIGN;
  if (aliased({range(tokens, rows * 8), range(logprobs, rows * 4)},
              {rows_range(logits, rows, V, ls, io), rows_range(noise, rows, V, ns, 4),
               range(args->temperature_row, rows * 4), range(args->top_k_row, rows * 4),
               range(args->top_p_row, rows * 4), range(args->min_p_row, rows * 4)}))
    return MSSM_ERR_ALIAS;
  mssm::SampleParams p;
  std::memset(&p, 0, sizeof(p));
  p.logits = logits; p.noise = noise; p.tokens = tokens; p.logprobs = logprobs;
  p.rows = rows; p.logits_stride = ls; p.noise_stride = ns; p.vocab = (int32_t)V;
  p.temperature = args->temperature; p.top_p = args->top_p; p.min_p = args->min_p;
  p.top_k = args->top_k;
  p.temperature_row = args->temperature_row; p.top_k_row = args->top_k_row;
  p.top_p_row = args->top_p_row; p.min_p_row = args->min_p_row;
  return done(mssm::launch_sample(p, args->io_dtype == MSSM_BF16, (hipStream_t)stream),
              "sample launch");
}

int mssm_mamba2_state_update_workspace(const mssm_step_dims* dims, int64_t* bytes) {
  if (!bytes) return MSSM_ERR_NULL;
  const int rc = check_step_dims(dims);
  if (rc != MSSM_OK) return rc;
  *bytes = dims->batch * dims->ngroups * 4;
  return MSSM_OK;
}

int mssm_mamba2_state_update(float* state, void* conv_state, const void* xbc, const void* dt,
                             const float* conv_weight, const float* conv_bias, const float* A,
                             const float* D, const void* z, const float* dt_bias, int softplus,
                             const int32_t* slots, void* out, void* workspace,
                             int64_t workspace_bytes, const mssm_step_dims* dims, void* stream) {
  int rc = check_step_dims(dims);
  if (rc != MSSM_OK) return rc;
  if (!state || !conv_state || !xbc || !dt || !conv_weight || !A || !out) return MSSM_ERR_NULL;
  if (!slots && dims->cache != dims->batch) return MSSM_ERR_DIMS;
  const int64_t io = size_of(dims->io_dtype);
  if (!all_aligned({conv_state, xbc, dt, z, out}, io) ||
      !all_aligned({state, conv_weight, conv_bias, A, D, dt_bias, slots}, 4))
    return MSSM_ERR_ALIGN;
  const int64_t batch = dims->batch, H = dims->nheads, N = dims->dstate, dim = H * 64;
  const int64_t ch = dim + 2 * dims->ngroups * N;
  const int64_t xs = dims->xbc_stride ? dims->xbc_stride : ch;
  const int64_t ds = dims->dt_stride ? dims->dt_stride : H;
  const int64_t zs = dims->z_stride ? dims->z_stride : dim;
  int64_t need = 0;
  mssm_mamba2_state_update_workspace(dims, &need);
  const Range r_state = range(state, dims->cache * dim * N * 4);
  const Range r_conv = range(conv_state, dims->cache * ch * (dims->width - 1) * io);
  const Range r_out = range(out, batch * dim * io), r_ws = range(workspace, need);
  if (aliased({r_state, r_conv, r_out, r_ws},
              {rows_range(xbc, batch, ch, xs, io), rows_range(dt, batch, H, ds, io),
               rows_range(z, batch, dim, zs, io), range(conv_weight, ch * dims->width * 4),
               range(conv_bias, ch * 4), range(A, H * 4), range(D, H * 4), range(dt_bias, H * 4),
               range(slots, batch * 4)}))
    return MSSM_ERR_ALIAS;
  rc = mssm::check_workspace(workspace, workspace_bytes, need);
  if (rc != MSSM_OK) return rc;
  mssm::Mamba2StepParams p;
  std::memset(&p, 0, sizeof(p));
  p.state = state; p.conv_state = conv_state; p.xbc = xbc; p.dt = dt; p.z = z;
  p.conv_weight = conv_weight; p.conv_bias = conv_bias; p.A = A; p.D = D; p.dt_bias = dt_bias;
  p.slots = slots; p.out = out; p.counters = static_cast<uint32_t*>(workspace);
  p.batch = batch; p.cache = dims->cache; p.channels = ch;
  p.xbc_stride = xs; p.dt_stride = ds; p.z_stride = zs;
  p.nheads = (int32_t)H; p.ngroups = (int32_t)dims->ngroups; p.N = (int32_t)N;
  p.width = dims->width; p.softplus = softplus ? 1 : 0;
  return done(mssm::launch_mamba2_step(p, dims->io_dtype == MSSM_BF16, mssm::compute_units(),
                                       (hipStream_t)stream),
              "Mamba-2 step launch");
}

}  // extern "C"
