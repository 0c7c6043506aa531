// train_api.cpp -- the C ABI of the ends of a training step (declared in
// include/mssm.h): argument validation, always before the first HIP call, and
// dispatch on the caller's stream.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <memory>
#include <new>

#include "api_checks.h"

using namespace mssm::api;

namespace {

int check_embed_dims(const mssm_embed_dims* d) {
  if (!d) return MSSM_ERR_NULL;
  if (!known(d->table_dtype) || !known(d->io_dtype)) return MSSM_ERR_UNSUPPORTED;
  if (d->rows <= 0 || d->rows > INT32_MAX || d->vocab <= 0 || d->vocab > (1 << 22) || d->dim <= 0 ||
      d->dim > (1 << 20))
    return MSSM_ERR_DIMS;
  if (d->io_stride != 0 && (d->io_stride < d->dim || !fits(d->rows, d->io_stride)))
    return MSSM_ERR_DIMS;
  // at most a workgroup for each 512 columns of a row of few, a wave of many, and in
  // the backward a thread for 64 columns of the table
  if (!fits(d->rows, (d->dim + 511) / 512 * 64, kItems / 4) ||
      !fits(d->vocab, (d->dim + 3) / 4, kItems / 2 * 16 - 4096))
    return MSSM_ERR_DIMS;
  return MSSM_OK;
}

int check_logprob_dims(const mssm_logprob_dims* d, bool grad) {
  if (!d) return MSSM_ERR_NULL;
  if (!known(d->io_dtype)) return MSSM_ERR_UNSUPPORTED;
  if (d->rows <= 0 || d->rows > kItems / 1024 || d->vocab <= 0 || d->vocab > (1 << 22))
    return MSSM_ERR_DIMS;
  if (d->logits_stride != 0 && (d->logits_stride < d->vocab || !fits(d->rows, d->logits_stride)))
    return MSSM_ERR_DIMS;
  if (grad && d->grad_stride != 0 &&
      (d->grad_stride < d->vocab || !fits(d->rows, d->grad_stride)))
    return MSSM_ERR_DIMS;
  // workgroups of 256 threads take 8192 columns, one column more of odd rows
  if (!fits(d->rows, (d->vocab + 8192) / 8192, kItems / 256)) return MSSM_ERR_DIMS;
  // the kernels multiply by log2(e) / temperature
  if (!(d->temperature > 0.0f) || !std::isfinite(1.4426950408889634f * (1.0f / d->temperature)) ||
      1.0f / d->temperature == 0.0f)
    return MSSM_ERR_DIMS;
  return MSSM_OK;
}

// The ranges of logits and their gradient, which may be the logits in place.
struct LogitRanges {
  Range logits, grad;
  bool in_place;
};
LogitRanges logit_ranges(const void* logits, const void* dlogits, const mssm_logprob_dims* d) {
  const int64_t io = size_of(d->io_dtype);
  const int64_t ls = d->logits_stride ? d->logits_stride : d->vocab;
  const int64_t gs = d->grad_stride ? d->grad_stride : d->vocab;
  LogitRanges r;
  r.logits = rows_range(logits, d->rows, d->vocab, ls, io);
  r.grad = rows_range(dlogits, d->rows, d->vocab, gs, io);
  r.in_place = dlogits == logits && (ls == gs || d->rows == 1);
  return r;
}

mssm::LogprobParams logprob_params(const mssm_logprob_dims* d) {
  mssm::LogprobParams p;
  std::memset(&p, 0, sizeof(p));
  p.rows = d->rows;
  p.vocab = (int32_t)d->vocab;
  p.logits_stride = d->logits_stride ? d->logits_stride : d->vocab;
  p.grad_stride = d->grad_stride ? d->grad_stride : d->vocab;
  p.inv_temperature = 1.0f / d->temperature;
  return p;
}

}  // namespace

extern "C" {

int mssm_embedding_fwd(const int64_t* tokens, const void* table, void* out,
                       const mssm_embed_dims* dims, void* stream) {
  const int rc = check_embed_dims(dims);
  if (rc != MSSM_OK) return rc;
  if (!tokens || !table || !out) return MSSM_ERR_NULL;
  const int64_t ts = size_of(dims->table_dtype), io = size_of(dims->io_dtype);
  const int64_t stride = dims->io_stride ? dims->io_stride : dims->dim;
  if (!aligned(tokens, 8) || !aligned(table, ts) || !aligned(out, io)) return MSSM_ERR_ALIGN;
  if (aliased({rows_range(out, dims->rows, dims->dim, stride, io)},
              {range(tokens, dims->rows * 8), range(table, dims->vocab * dims->dim * ts)}))
    return MSSM_ERR_ALIAS;
  const mssm::EmbedParams p{tokens, table, out, dims->rows, stride, (int32_t)dims->vocab,
                            (int32_t)dims->dim, dims->scale};
  return done(mssm::launch_embedding(p, dims->table_dtype == MSSM_BF16, dims->io_dtype == MSSM_BF16,
                                     (hipStream_t)stream),
              "embedding launch");
}

int mssm_embedding_bwd_workspace(const mssm_embed_dims* dims, int64_t* bytes) {
  if (!bytes) return MSSM_ERR_NULL;
  const int rc = check_embed_dims(dims);
  if (rc != MSSM_OK) return rc;
  *bytes = mssm::embedding_bwd_workspace(dims->rows, dims->vocab, dims->dim);
  return MSSM_OK;
}

int mssm_embedding_bwd(const int64_t* tokens, const void* dout, void* dtable, void* workspace,
                       int64_t workspace_bytes, const mssm_embed_dims* dims, void* stream) {
  int rc = check_embed_dims(dims);
  if (rc != MSSM_OK) return rc;
  if (!tokens || !dout || !dtable) return MSSM_ERR_NULL;
  const int64_t ts = size_of(dims->table_dtype), io = size_of(dims->io_dtype);
  const int64_t stride = dims->io_stride ? dims->io_stride : dims->dim;
  if (!aligned(tokens, 8) || !aligned(dout, io) || !aligned(dtable, ts)) return MSSM_ERR_ALIGN;
  const int64_t need = mssm::embedding_bwd_workspace(dims->rows, dims->vocab, dims->dim);
  if (aliased({range(dtable, dims->vocab * dims->dim * ts), range(workspace, need)},
              {range(tokens, dims->rows * 8),
               rows_range(dout, dims->rows, dims->dim, stride, io)}))
    return MSSM_ERR_ALIAS;
  rc = mssm::check_workspace(workspace, workspace_bytes, need);
  if (rc != MSSM_OK) return rc;
  const mssm::EmbedBwdParams p{tokens, dout, dtable, workspace, dims->rows, stride,
                               (int32_t)dims->vocab, (int32_t)dims->dim, dims->scale,
                               dims->add ? 1 : 0};
  return done(mssm::launch_embedding_bwd(p, dims->table_dtype == MSSM_BF16,
                                         dims->io_dtype == MSSM_BF16, (hipStream_t)stream),
              "embedding backward launch");
}

int mssm_token_logprobs_workspace(const mssm_logprob_dims* dims, int64_t* bytes) {
  if (!bytes) return MSSM_ERR_NULL;
  const int rc = check_logprob_dims(dims, false);
  if (rc != MSSM_OK) return rc;
  *bytes = mssm::logprob_workspace(dims->rows, dims->vocab);
  return MSSM_OK;
}

int mssm_token_logprobs_fwd(const void* logits, const int64_t* tokens, float* logprobs,
                            float* stats, void* workspace, int64_t workspace_bytes,
                            const mssm_logprob_dims* dims, void* stream) {
  int rc = check_logprob_dims(dims, false);
  if (rc != MSSM_OK) return rc;
  if (!logits || !tokens || !logprobs) return MSSM_ERR_NULL;
  if (!aligned(logits, size_of(dims->io_dtype)) || !aligned(tokens, 8) ||
      !all_aligned({logprobs, stats}, 4))
    return MSSM_ERR_ALIGN;
  const int64_t rows = dims->rows, need = mssm::logprob_workspace(rows, dims->vocab);
  if (aliased({range(logprobs, rows * 4), range(stats, rows * 8), range(workspace, need)},
              {logit_ranges(logits, nullptr, dims).logits, range(tokens, rows * 8)}))
    return MSSM_ERR_ALIAS;
  rc = mssm::check_workspace(workspace, workspace_bytes, need);
  if (rc != MSSM_OK) return rc;
  mssm::LogprobParams p = logprob_params(dims);
  p.partial = static_cast<float*>(workspace);
  p.logits = logits; p.tokens = tokens; p.logprobs = logprobs; p.stats = stats;
  return done(mssm::launch_logprobs(p, dims->io_dtype == MSSM_BF16, (hipStream_t)stream),
              "log-probability launch");
}

int mssm_token_logprobs_bwd(const void* logits, const int64_t* tokens, const float* stats,
                            const float* dlogprobs, void* dlogits, const mssm_logprob_dims* dims,
                            void* stream) {
  const int rc = check_logprob_dims(dims, true);
  if (rc != MSSM_OK) return rc;
  if (!logits || !tokens || !stats || !dlogprobs || !dlogits) return MSSM_ERR_NULL;
  const int64_t io = size_of(dims->io_dtype), rows = dims->rows;
  if (!all_aligned({logits, dlogits}, io) || !aligned(tokens, 8) ||
      !all_aligned({stats, dlogprobs}, 4))
    return MSSM_ERR_ALIGN;
  const LogitRanges r = logit_ranges(logits, dlogits, dims);
  if (aliased({r.grad}, {r.in_place ? Range{0, 0} : r.logits, range(tokens, rows * 8),
                         range(stats, rows * 8), range(dlogprobs, rows * 4)}))
    return MSSM_ERR_ALIAS;
  mssm::LogprobParams p = logprob_params(dims);
  p.logits = logits; p.tokens = tokens; p.stats = const_cast<float*>(stats);
  p.dlogprobs = dlogprobs; p.dlogits = dlogits;
  return done(mssm::launch_logprobs_bwd(p, dims->io_dtype == MSSM_BF16, (hipStream_t)stream),
              "log-probability backward launch");
}

int mssm_policy_loss(const void* logits, const int64_t* tokens, const float* old_logprobs,
                     const float* advantages, const float* ref_logprobs, const float* weights,
                     float* loss, float* logprobs, void* dlogits, void* workspace,
                     int64_t workspace_bytes, const mssm_policy_args* args, void* stream) {
  if (!args) return MSSM_ERR_NULL;
  const mssm_logprob_dims* d = &args->dims;
  int rc = check_logprob_dims(d, dlogits != nullptr);
  if (rc != MSSM_OK) return rc;
  if (!(args->clip_low >= 0.0f) || !(args->clip_high >= 0.0f) || !(args->kl_coef >= 0.0f) ||
      !std::isfinite(args->kl_coef))
    return MSSM_ERR_DIMS;
  if (!logits || !tokens || !old_logprobs || !advantages || !loss || !logprobs)
    return MSSM_ERR_NULL;
  const int64_t io = size_of(d->io_dtype), rows = d->rows;
  if (!all_aligned({logits, dlogits}, io) || !aligned(tokens, 8) ||
      !all_aligned({old_logprobs, advantages, ref_logprobs, weights, loss, logprobs}, 4))
    return MSSM_ERR_ALIGN;
  const LogitRanges r = logit_ranges(logits, dlogits, d);
  const Range r_loss = range(loss, rows * 4), r_logp = range(logprobs, rows * 4);
  const Range r_tok = range(tokens, rows * 8), r_old = range(old_logprobs, rows * 4);
  const Range r_adv = range(advantages, rows * 4), r_ref = range(ref_logprobs, rows * 4);
  const Range r_w = range(weights, rows * 4);
  const int64_t need = mssm::logprob_workspace(rows, d->vocab);
  const Range r_ws = range(workspace, need);
  if (aliased({r_loss, r_logp, r_ws}, {r.logits, r_tok, r_old, r_adv, r_ref, r_w}) ||
      aliased({r.grad, r_loss, r_logp, r_ws},
              {r.in_place ? Range{0, 0} : r.logits, r_tok, r_old, r_adv, r_ref, r_w}))
    return MSSM_ERR_ALIAS;
  rc = mssm::check_workspace(workspace, workspace_bytes, need);
  if (rc != MSSM_OK) return rc;
  mssm::LogprobParams p = logprob_params(d);
  p.partial = static_cast<float*>(workspace);
  p.logits = logits; p.tokens = tokens; p.logprobs = logprobs;
  p.old_logprobs = old_logprobs; p.advantages = advantages;
  p.ref_logprobs = args->kl_coef > 0.0f ? ref_logprobs : nullptr;  // else no KL term: 0 * inf
  p.weights = weights; p.loss = loss; p.dlogits = dlogits;
  p.clip_lo = 1.0f - args->clip_low; p.clip_hi = 1.0f + args->clip_high;
  p.kl_coef = args->kl_coef;
  return done(mssm::launch_logprobs(p, d->io_dtype == MSSM_BF16, (hipStream_t)stream),
              "policy loss launch");
}

int mssm_preference_loss(const float* logprobs, const float* ref_logprobs, const int32_t* offsets,
                         const float* weights, float* loss, float* dlogprobs,
                         const mssm_preference_args* args, void* stream) {
  if (!args) return MSSM_ERR_NULL;
  if (args->rows <= 0 || args->rows > INT32_MAX || args->pairs <= 0 || args->pairs > (1 << 20) ||
      !std::isfinite(args->beta) || !(args->label_smoothing >= 0.0f && args->label_smoothing <= 1.0f))
    return MSSM_ERR_DIMS;
  if (!logprobs || !ref_logprobs || !offsets || !loss || !dlogprobs) return MSSM_ERR_NULL;
  if (!all_aligned({logprobs, ref_logprobs, offsets, weights, loss, dlogprobs}, 4))
    return MSSM_ERR_ALIGN;
  const int64_t rows = args->rows, pairs = args->pairs;
  if (aliased({range(loss, pairs * 4), range(dlogprobs, rows * 4)},
              {range(logprobs, rows * 4), range(ref_logprobs, rows * 4),
               range(offsets, (2 * pairs + 1) * 4), range(weights, pairs * 4)}))
    return MSSM_ERR_ALIAS;
  const mssm::PreferenceParams p{logprobs, ref_logprobs, offsets, weights, loss, dlogprobs,
                                 (int32_t)rows, (int32_t)pairs, args->beta, args->label_smoothing};
  return done(mssm::launch_preference(p, (hipStream_t)stream), "preference loss launch");
}

int mssm_adamw(const mssm_adamw_tensor* tensors, int64_t count, void* m, void* v, float* m_scales,
               float* v_scales, const mssm_adamw_args* args, void* stream) {
  if (!args || !tensors || !m || !v) return MSSM_ERR_NULL;
  if (args->state_bits != 32 && args->state_bits != 8) return MSSM_ERR_UNSUPPORTED;
  const bool eight = args->state_bits == 8;
  if (eight && (!m_scales || !v_scales)) return MSSM_ERR_NULL;
  if (!eight && (m_scales || v_scales)) return MSSM_ERR_UNSUPPORTED;
  if (count <= 0 || !(args->beta1 >= 0.0 && args->beta1 < 1.0) ||
      !(args->beta2 >= 0.0 && args->beta2 < 1.0) || !(args->eps >= 0.0) ||
      (!args->step_value && args->step < 1) || count > (1 << 24))
    return MSSM_ERR_DIMS;
  if (!all_aligned({m, v}, 16) || !all_aligned({m_scales, v_scales, args->lr_value,
                                                args->grad_scale_value}, 4) ||
      !aligned(args->step_value, 8))
    return MSSM_ERR_ALIGN;
  int64_t total = 0;
  for (int64_t i = 0; i < count; ++i) {
    const mssm_adamw_tensor& t = tensors[i];
    if (!t.param || !t.grad) return MSSM_ERR_NULL;
    if (!known(t.grad_dtype)) return MSSM_ERR_UNSUPPORTED;
    // 2^33 elements of one tensor are 2^23 workgroups or fewer
    if (t.size <= 0 || t.size > (int64_t)1 << 33 || total > (int64_t)1 << 50) return MSSM_ERR_DIMS;
    if (!aligned(t.param, 4) || !aligned(t.grad, size_of(t.grad_dtype)) || !aligned(t.copy, 2))
      return MSSM_ERR_ALIGN;
    total += blocks128(t.size) * 128;
  }
  const int64_t each = eight ? 1 : 4;
  // No output (params, copies, states) may overlap another or an input: all
  // ranges in order of address.
  struct Item {
    Range r;
    bool out;
  };
  const int64_t most_items = 3 * count + 7;
  std::unique_ptr<Item[]> items(new (std::nothrow) Item[(size_t)most_items]);
  if (!items) return MSSM_ERR_WORKSPACE;
  int64_t n = 0;
  const auto put = [&](const void* q, int64_t bytes, bool out) {
    if (q) items[n++] = Item{range(q, bytes), out};
  };
  for (int64_t i = 0; i < count; ++i) {
    const mssm_adamw_tensor& t = tensors[i];
    put(t.param, t.size * 4, true);
    put(t.copy, t.size * 2, true);
    put(t.grad, t.size * size_of(t.grad_dtype), false);
  }
  put(m, total * each, true);
  put(v, total * each, true);
  put(m_scales, total / 128 * 4, true);
  put(v_scales, total / 128 * 4, true);
  put(args->lr_value, 4, false);
  put(args->grad_scale_value, 4, false);
  put(args->step_value, 8, false);
  std::sort(items.get(), items.get() + n,
            [](const Item& a, const Item& b) { return a.r.lo < b.r.lo; });
  uintptr_t outs = 0, ins = 0;  // the ends of those so far
  for (int64_t i = 0; i < n; ++i) {
    const Item& a = items[i];
    if (a.r.lo < outs || (a.out && a.r.lo < ins)) return MSSM_ERR_ALIAS;
    (a.out ? outs : ins) = std::max(a.out ? outs : ins, a.r.hi);
  }
  mssm::AdamParams p;
  std::memset(&p, 0, sizeof(p));
  p.m = m; p.v = v; p.m_scales = m_scales; p.v_scales = v_scales;
  p.lr_value = args->lr_value; p.grad_scale_value = args->grad_scale_value;
  p.step_value = args->step_value;
  p.seed = args->seed; p.step = args->step;
  p.lr = (float)args->lr; p.grad_scale = (float)args->grad_scale;
  // the hardware's reciprocal of less is infinite, and its product with a step of 0 NaN
  p.eps = args->eps > 0.0 ? std::max((float)args->eps, 0x1p-126f) : 0.0f;
  // 1 - beta from the double: from the rounded float it would be 2e-7 off
  p.beta1 = (float)args->beta1; p.rest1 = (float)(1.0 - args->beta1);
  p.beta2 = (float)args->beta2; p.rest2 = (float)(1.0 - args->beta2);
  p.log_beta1 = (float)std::log(args->beta1); p.log_beta2 = (float)std::log(args->beta2);
  if (!args->step_value) {
    p.inv_c1 = (float)(1.0 / (1.0 - std::pow(args->beta1, (double)args->step)));
    p.inv_c2 = (float)(1.0 / std::sqrt(1.0 - std::pow(args->beta2, (double)args->step)));
  }
  // a launch takes tensors up to its table's length and its grid's threads
  const int64_t per = mssm::adamw_block_elements(), most = kItems / 256;
  int64_t at = 0, next = 0;
  while (next < count) {
    int64_t blocks = 0;
    p.count = 0;
    while (next < count && p.count < mssm::kAdamTensors) {
      const mssm_adamw_tensor& t = tensors[next];
      const int64_t need = (t.size + per - 1) / per;
      if (need > most - blocks) break;
      p.tensors[p.count] = mssm::AdamTensor{t.param, t.grad, t.copy, t.size, at, t.weight_decay,
                                            t.grad_dtype == MSSM_BF16};
      p.first[p.count++] = (uint32_t)blocks;
      blocks += need;
      at += blocks128(t.size) * 128;
      ++next;
    }
    p.blocks = (uint32_t)blocks;
    const int rc = done(mssm::launch_adamw(p, eight, (hipStream_t)stream), "AdamW launch");
    if (rc != MSSM_OK) return rc;
  }
  return MSSM_OK;
}

}  // extern "C"
