"""The ends of a training step together, as the example runs them."""
import pytest
import torch

from tests import train_common as tc
from tests.test_gpu_layer_path import ex, rel  # noqa: F401

pytestmark = pytest.mark.gpu
ROWS = 150


def batch(ex, policy, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    tokens = torch.randint(0, policy.vocab, (ROWS,), generator=g, device="cuda")
    taken, old = policy.answer(tokens, torch.rand(ROWS, policy.vocab, generator=g, device="cuda"))
    taken[::7] = -1                                        # prompts
    old = old - 0.05 * torch.randn(ROWS, generator=g, device="cuda")
    adv = torch.randn(ROWS, generator=g, device="cuda")
    ref = old + 0.2 * torch.randn(ROWS, generator=g, device="cuda")
    return tokens, taken, old, adv, ref


def exact_gradients(table, copy, norm, tokens, dlogits):
    """Of the exact layer in 64 bits, for a gradient of its logits."""
    t, w, n = (x.double().cpu().requires_grad_() for x in (copy, table, norm))
    x = t[tokens.cpu()]
    y = x * torch.rsqrt(x.square().mean(1, keepdim=True) + 1e-5) * n
    (y @ w.t()).backward(dlogits)
    return t.grad + w.grad, n.grad


def check(got, before, tokens, dlogits):
    """e4m3 rounds each operand by 2^-5.3 of it in the mean square: two operands a
    product, three products (the logits' is in dlogits already) and the norm's
    backward after one of them: 0.1."""
    for a, b in zip(got, exact_gradients(*before, tokens, dlogits)):
        assert rel(a.cpu(), b) < 0.1


def test_reward_gradients(ex):  # noqa: F811
    policy = ex.Policy()
    tokens, taken, old, adv, ref = batch(ex, policy)
    w = torch.full((ROWS,), 1 / ROWS, device="cuda")
    before = [policy.table.clone(), policy.copies[0].clone(), policy.norm.clone()]
    # the loss's gradient at the logits that the step itself sees, ratios far from the clip
    logits = policy.logits(tokens)[0].cpu()
    cpu = taken.cpu()
    logp, _, _, p = tc.logprobs(logits, cpu, 1.0)
    old = (logp - (logp - old.cpu().double()).clamp(-0.15, 0.15)).float().cuda()
    loss, grads = policy.reward_step(tokens, taken, old, adv, ref, w)
    want, slope = tc.policy(logp, cpu, policy.vocab, old.cpu(), adv.cpu(), ref.cpu(), 0.2, 0.2, 0.05)
    assert rel(loss.cpu(), want) < 1e-5
    check(grads, before, tokens, tc.softmax_slope(p, cpu, slope / ROWS))
    assert (loss.cpu()[cpu < 0] == 0).all() and int(policy.step) == 1
    # the step moved every parameter with a gradient, and the copy follows
    assert torch.equal(policy.copies[0], policy.table.bfloat16())
    assert float((policy.norm - before[2]).abs().min()) > 0.0


def test_preference_gradients(ex):  # noqa: F811
    policy = ex.Policy(bits=32)
    tokens, taken, old, adv, ref = batch(ex, policy, seed=3)
    ref = torch.where(taken >= 0, ref, 0.0)
    at = torch.tensor([0, 30, 70, 90, 140], dtype=torch.int32, device="cuda")
    before = [policy.table.clone(), policy.copies[0].clone(), policy.norm.clone()]
    logits = policy.logits(tokens)[0].cpu()
    cpu = taken.cpu()
    logp, _, _, p = tc.logprobs(logits, cpu, 1.0)
    loss, grads = policy.preference_step(tokens, taken, ref, at)
    want, slope, _ = tc.preference(logp, ref.cpu(), at.cpu(), None, 0.1, 0.0)
    assert rel(loss.cpu(), want) < 1e-5
    check(grads, before, tokens, tc.softmax_slope(p, cpu, torch.where(cpu >= 0, slope, 0.0)))


@pytest.mark.parametrize("bits", [32, 8])
def test_steps_in_a_graph(ex, bits):  # noqa: F811
    """A captured step, replayed with the program's own work in between, does what
    the eager step does each time: the same kernels on the same inputs."""
    a, b = ex.Policy(bits=bits), ex.Policy(bits=bits)
    tokens, taken, old, adv, ref = batch(ex, a)
    w = torch.full((ROWS,), 1 / ROWS, device="cuda")
    warm = ex.Policy(bits=bits)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        warm.reward_step(tokens, taken, old, adv, ref, w)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            loss, grads = a.reward_step(tokens, taken, old, adv, ref, w)
    torch.cuda.current_stream().wait_stream(side)
    for k in range(1, 5):
        a.lr.fill_(1e-3 / k)
        b.lr.fill_(1e-3 / k)
        graph.replay()
        torch.cuda.synchronize()
        want, want_grads = b.reward_step(tokens, taken, old, adv, ref, w)
        assert torch.equal(loss, want) and all(torch.equal(x, y) for x, y in zip(grads, want_grads))
        assert all(torch.equal(x, y) for x, y in zip(a.params, b.params))
        for x, y in zip(a.moments, b.moments):
            assert x is None or torch.equal(x.view(torch.uint8), y.view(torch.uint8))
        assert int(a.step) == k
        tokens.copy_(tokens.flip(0))


def test_example_runs(ex):  # noqa: F811
    ex.main()
