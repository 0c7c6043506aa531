"""A small Mamba-2 language model with 8-bit projections and random weights: a
prompt through the convolution and the scan, then single tokens through the
step, the next token sampled on the GPU; the training step of a layer's norm and
input projection; and training steps of a small policy from rewards and from
preferences, its table shared by the embedding and the output projection.

Run: python examples/mamba2_generate.py
"""
import math
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import selective_state_space_52_amd as mssm  # noqa: E402


class Model:
    """`layers` Mamba-2 layers of width `dim` with dim // 32 heads of 64 channels
    (an expansion of 2), one group of B and C with N states, a width-4
    convolution.  The residual stream is fp32, activations bf16, the
    projections e4m3 with a scale for each 128 x 128 block."""

    def __init__(self, dim=256, layers=2, vocab=1000, N=128, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def randn(*shape, scale=1.0):
            return torch.randn(*shape, generator=g, device=device) * scale
        self.dim, self.N, self.vocab = dim, N, vocab
        self.heads, self.inner = dim // 32, 2 * dim
        self.channels = self.inner + 2 * N          # of the convolution: x, B, C
        self.embedding = randn(vocab, dim).bfloat16()
        self.layers = []
        for _ in range(layers):
            rows = self.inner + self.channels + self.heads      # z | x, B, C | dt
            step = torch.exp(torch.rand(self.heads, generator=g, device=device) * math.log(100.0)
                             + math.log(1e-3))
            self.layers.append(dict(
                norm=torch.ones(dim, device=device),
                in_proj=mssm.quantize_fp8(randn(rows, dim, scale=dim ** -0.5), block_rows=128),
                conv_weight=randn(self.channels, 4, scale=0.5),
                conv_bias=randn(self.channels, scale=0.1),
                A=-1.0 - 15.0 * torch.rand(self.heads, generator=g, device=device),
                D=torch.ones(self.heads, device=device),
                dt_bias=step + torch.log(-torch.expm1(-step)),
                out_norm=torch.ones(self.inner, device=device),
                out_proj=mssm.quantize_fp8(randn(dim, self.inner, scale=self.inner ** -0.5),
                                           block_rows=128)))
        self.norm = torch.ones(dim, device=device)
        self.head = mssm.quantize_fp8(randn(vocab, dim, scale=dim ** -0.5), block_rows=128)

    def states(self, sequences):
        """The layers' states, one row for each sequence: (state, window)."""
        dev = self.embedding.device
        return [(torch.zeros(sequences, self.inner, self.N, device=dev),
                 torch.zeros(sequences, self.channels, 3, dtype=torch.bfloat16, device=dev))
                for _ in self.layers]

    def _project(self, layer, x, residual):
        q, scales, residual, _ = mssm.rms_norm_fwd_fp8(x, layer["norm"], residual=residual)
        p = mssm.fp8_matmul(q, scales, *layer["in_proj"])
        return p[:, :self.inner], p[:, self.inner:-self.heads], p[:, -self.heads:], residual

    def _finish(self, layer, y):
        q, scales, _, _ = mssm.rms_norm_fwd_fp8(y, layer["out_norm"])
        return mssm.fp8_matmul(q, scales, *layer["out_proj"])

    def _logits(self, x, residual):
        q, scales, _, _ = mssm.rms_norm_fwd_fp8(x, self.norm, residual=residual)
        return mssm.fp8_matmul(q, scales, *self.head, out_dtype=torch.float32)

    def prompt(self, tokens):
        """tokens (batch, L), L >= 3.  Returns the last tokens' logits and the states."""
        batch, L = tokens.shape
        x = mssm.embedding_fwd(tokens.flatten(), self.embedding)
        residual = torch.zeros(batch * L, self.dim, device=x.device)
        states = []
        for layer in self.layers:
            z, xbc, dt, residual = self._project(layer, x, residual)
            z, xbc, dt = (t.contiguous() for t in (z, xbc, dt))   # the scan takes whole tensors
            xbc = xbc.view(batch, L, self.channels)
            u = mssm.causal_conv1d_fwd(xbc, layer["conv_weight"], layer["conv_bias"], layout="bld")
            xs, B, C = (t.contiguous() for t in u.split([self.inner, self.N, self.N], dim=2))
            last = torch.empty(batch, self.inner, self.N, device=x.device)
            y = mssm.mamba2_scan_fwd(
                xs.view(batch, L, self.heads, 64), dt.view(batch, L, self.heads), layer["A"],
                B.unsqueeze(2), C.unsqueeze(2), D=layer["D"],
                z=z.view(batch, L, self.heads, 64), dt_bias=layer["dt_bias"], last_state=last)
            states.append((last, xbc[:, -3:].transpose(1, 2).contiguous()))
            x = self._finish(layer, y.view(batch * L, self.inner))
        end = torch.arange(L - 1, batch * L, L, device=x.device)
        return self._logits(x[end], residual[end]), states

    def step(self, tokens, states, slots=None):
        """tokens (batch,): one more of each sequence; the states are updated in
        place (rows `slots` of them, where given).  Returns the logits."""
        x = mssm.embedding_fwd(tokens.contiguous(), self.embedding)
        residual = torch.zeros(len(tokens), self.dim, device=x.device)
        for layer, (state, window) in zip(self.layers, states):
            z, xbc, dt, residual = self._project(layer, x, residual)
            y = mssm.mamba2_state_update(state, window, xbc, dt, layer["conv_weight"], layer["A"],
                                         conv_bias=layer["conv_bias"], D=layer["D"], z=z,
                                         dt_bias=layer["dt_bias"], slots=slots)
            x = self._finish(layer, y)
        return self._logits(x, residual)

    def generate(self, tokens, count, seed=0, **sampling):
        """`count` sampled tokens after the prompt, (batch, count)."""
        g = torch.Generator(device=tokens.device).manual_seed(seed)
        logits, states = self.prompt(tokens)
        out = []
        for i in range(count):
            noise = torch.rand(logits.shape, generator=g, device=logits.device)
            token, _ = mssm.sample_tokens(logits, noise, **sampling)
            out.append(token)
            if i + 1 < count:
                logits = self.step(token, states)
        return torch.stack(out, 1)


class NormLinear(torch.autograd.Function):
    """out = norm(x + residual) w^T with the product in 8 bits, and the new
    residual stream; the gradients through the 8-bit products and the norm."""

    @staticmethod
    def forward(ctx, x, residual, norm, w):
        y, stream, rstd = mssm.rms_norm_fwd(x, norm, residual=residual, want_rstd=True)
        out = mssm.fp8_matmul(*mssm.quantize_fp8(y), *mssm.quantize_fp8(w, block_rows=128))
        ctx.save_for_backward(y, stream, rstd, norm, w)
        return out, stream

    @staticmethod
    def backward(ctx, dout, dstream):
        y, stream, rstd, norm, w = ctx.saved_tensors
        dout = dout.contiguous()
        dy = mssm.fp8_matmul(*mssm.quantize_fp8(dout),
                             *mssm.quantize_fp8(w, block_rows=128, transpose=True))
        dw = mssm.fp8_matmul(*mssm.quantize_fp8(dout, transpose=True),
                             *mssm.quantize_fp8(y, transpose=True), out_dtype=torch.float32)
        dx, dresidual, dnorm = mssm.rms_norm_bwd(dy, stream, norm, rstd,
                                                 dresidual=dstream.contiguous())
        return dx, dresidual, dnorm, dw


class Policy:
    """Logits of the next token from the last one: a table of `vocab` rows, a norm,
    and the table again.  Parameters fp32 with a bf16 copy of the table for the
    lookup; the products in 8 bits; AdamW's states in `bits` bits."""

    def __init__(self, dim=128, vocab=500, bits=8, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        self.vocab = vocab
        self.table = torch.randn(vocab, dim, generator=g, device=device) * 0.05
        self.norm = torch.ones(dim, device=device)
        self.params = [self.table, self.norm]
        self.copies = [self.table.bfloat16(), None]
        self.moments = mssm.adamw_state(self.params, bits)
        # on the device, so that a captured step finds them new in every replay
        self.step = torch.zeros(1, dtype=torch.int64, device=device)
        self.lr = torch.full((1,), 1e-3, device=device)

    def logits(self, tokens):
        """Of tokens (rows,), and what the backward needs."""
        x = mssm.embedding_fwd(tokens, self.copies[0])
        y, _, rstd = mssm.rms_norm_fwd(x, self.norm, want_rstd=True)
        out = mssm.fp8_matmul(*mssm.quantize_fp8(y), *mssm.quantize_fp8(self.table, block_rows=128),
                              out_dtype=torch.float32)
        return out, (tokens, x, y, rstd)

    def gradients(self, saved, dlogits):
        """Of the table and the norm, for the logits' gradient."""
        tokens, x, y, rstd = saved
        dy = mssm.fp8_matmul(*mssm.quantize_fp8(dlogits),
                             *mssm.quantize_fp8(self.table, block_rows=128, transpose=True))
        dtable = mssm.fp8_matmul(*mssm.quantize_fp8(dlogits, transpose=True),
                                 *mssm.quantize_fp8(y, transpose=True), out_dtype=torch.float32)
        dx, _, dnorm = mssm.rms_norm_bwd(dy, x, self.norm, rstd)
        mssm.embedding_bwd(tokens, dx, self.vocab, add_to=dtable)
        return [dtable, dnorm]

    def update(self, grads):
        m, v, m_scales, v_scales = self.moments
        self.step += 1
        mssm.adamw_step(self.params, grads, m, v, step=self.step, lr=self.lr,
                        weight_decay=[0.1, 0.0], m_scales=m_scales, v_scales=v_scales,
                        copies=self.copies)

    def answer(self, tokens, noise):
        """Sampled next tokens, and their log-probabilities."""
        logits, _ = self.logits(tokens)
        taken, _ = mssm.sample_tokens(logits, noise)
        return taken, mssm.token_logprobs_fwd(logits, taken)[0]

    def reward_step(self, tokens, taken, old_logprobs, advantages, ref_logprobs, weights):
        """One step on the clipped policy loss; taken is -1 in a prompt's rows.
        Returns each row's loss and the gradients."""
        logits, saved = self.logits(tokens)
        loss, _, dlogits = mssm.policy_loss(logits, taken, old_logprobs, advantages,
                                            ref_logprobs=ref_logprobs, weights=weights,
                                            kl_coef=0.05, out=logits)
        grads = self.gradients(saved, dlogits)
        self.update(grads)
        return loss, grads

    def preference_step(self, tokens, taken, ref_logprobs, offsets):
        """One step on the preference loss of packed pairs.  Returns each pair's
        loss and the gradients."""
        logits, saved = self.logits(tokens)
        logprobs, stats = mssm.token_logprobs_fwd(logits, taken)
        loss, dlogprobs = mssm.preference_loss(logprobs, ref_logprobs, offsets)
        dlogits = mssm.token_logprobs_bwd(logits, taken, stats, dlogprobs, out=logits)
        grads = self.gradients(saved, dlogits)
        self.update(grads)
        return loss, grads


def main():
    model = Model()
    prompt = torch.randint(0, model.vocab, (4, 32), device="cuda")
    print(model.generate(prompt, 16, temperature=0.8, top_k=50, top_p=0.95))
    policy = Policy()
    tokens = torch.randint(0, policy.vocab, (64,), device="cuda")
    taken, old = policy.answer(tokens, torch.rand(64, policy.vocab, device="cuda"))
    advantages = (taken % 2).float() * 2 - 1
    for _ in range(3):
        loss, _ = policy.reward_step(tokens, taken, old, advantages, old,
                                     torch.full_like(old, 1 / 64))
        print(loss.mean().item())


if __name__ == "__main__":
    main()
