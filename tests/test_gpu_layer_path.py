"""The layer's operators together, as the example runs them."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "mamba2_generate.py")


@pytest.fixture(scope="module")
def ex():
    spec = importlib.util.spec_from_file_location("mamba2_generate", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def rel(a, b):
    return float((a.double() - b.double()).norm() / b.double().norm())


def test_steps_continue_the_prompt(ex):
    """Logits after prompt and steps against those of the whole text as a prompt.
    The step keeps the convolution's output in fp32 and the prompt in bf16 (2^-8),
    which moves some e4m3 roundings (2^-4 at most, 2^-5.3 in the mean square) at
    each of five products: 0.1 covers all of them moving."""
    model = ex.Model()
    tokens = torch.randint(0, model.vocab, (3, 12), device="cuda")
    logits, states = model.prompt(tokens[:, :9])
    for t in range(9, 12):
        logits = model.step(tokens[:, t], states)
    want, want_states = model.prompt(tokens)
    assert rel(logits, want) < 0.1
    for (s, w), (s2, w2) in zip(states, want_states):
        assert rel(s, s2) < 0.1 and rel(w.float(), w2.float()) < 0.1


def test_slots(ex):
    """The same steps with the sequences in slots of a larger cache: the same bits."""
    model = ex.Model(layers=1)
    tokens = torch.randint(0, model.vocab, (2, 8), device="cuda")
    _, states = model.prompt(tokens)
    cache = model.states(5)
    slots = torch.tensor([3, 1], dtype=torch.int32, device="cuda")
    for (s, w), (cs, cw) in zip(states, cache):
        cs[slots.long()], cw[slots.long()] = s, w
    nxt = torch.tensor([5, 6], device="cuda")
    a = model.step(nxt, states)
    b = model.step(nxt, cache, slots=slots)
    assert torch.equal(a, b)
    assert torch.equal(cache[0][0][slots.long()], states[0][0])
    assert float(cache[0][0][[0, 2, 4]].abs().max()) == 0.0


def test_generate_is_repeatable(ex):
    model = ex.Model(dim=128, layers=1, vocab=500)
    prompt = torch.randint(0, 500, (2, 7), device="cuda")
    a = model.generate(prompt, 6, temperature=0.8, top_k=50, top_p=0.95)
    b = model.generate(prompt, 6, temperature=0.8, top_k=50, top_p=0.95)
    assert torch.equal(a, b) and a.shape == (2, 6) and int(a.min()) >= 0 and int(a.max()) < 500


def test_steps_in_a_graph(ex):
    """A captured step, replayed with the program's own work in between, gives
    what the eager step gives each time."""
    model = ex.Model(dim=128, layers=1, vocab=500)
    prompt = torch.randint(0, 500, (2, 5), device="cuda")
    _, states = model.prompt(prompt)
    other = [(s.clone(), w.clone()) for s, w in states]
    token = torch.tensor([3, 4], device="cuda")
    noise = torch.rand(2, 500, device="cuda")
    import selective_state_space_52_amd as mssm
    warm = [(s.clone(), w.clone()) for s, w in states]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        model.step(token, warm)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            logits = model.step(token, states)
            picked = mssm.sample_tokens(logits, noise, temperature=0.9, top_p=0.9)[0]
    torch.cuda.current_stream().wait_stream(side)
    for _ in range(4):
        graph.replay()
        torch.cuda.synchronize()
        want = model.step(token, other)
        want_token, _ = mssm.sample_tokens(want, noise, temperature=0.9, top_p=0.9)
        assert torch.equal(logits, want) and torch.equal(picked, want_token)
        for (s, w), (s2, w2) in zip(states, other):
            assert torch.equal(s, s2) and torch.equal(w, w2)
        token.copy_(want_token)


def test_norm_linear_gradients(ex):
    """Against the gradients of the exact layer in 64 bits: e4m3 rounds each
    operand by 2^-5.3 of it in the mean square, two operands a product and the
    norm's backward after it: 0.1."""
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, res, norm, w = r(96, 256).bfloat16(), r(96, 256), 1 + 0.1 * r(256), r(200, 256) / 16
    dout, dstream = r(96, 200).bfloat16(), 0.1 * r(96, 256)
    leaves = [t.clone().requires_grad_() for t in (x, res, norm, w)]
    out, stream = ex.NormLinear.apply(*leaves)
    torch.autograd.backward([out, stream], [dout, dstream])
    out, stream = out.detach(), stream.detach()
    exact = [t.double().requires_grad_() for t in (x, res, norm, w)]
    s = exact[0] + exact[1]
    y = s * torch.rsqrt(s.square().mean(1, keepdim=True) + 1e-5) * exact[2]
    want = y @ exact[3].t()
    torch.autograd.backward([want, s], [dout.double(), dstream.double()])
    assert rel(out, want.detach()) < 0.1 and rel(stream, s.detach()) < 1e-6
    for a, b in zip(leaves, exact):
        assert rel(a.grad, b.grad) < 0.1
