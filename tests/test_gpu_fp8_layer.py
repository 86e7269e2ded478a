"""The 8-bit operators and the whole layer for few tokens as a program uses them together: training steps with products in 8 bits, then
the same layer held in 8 bits for a prompt and for the tokens behind it; a training step in a captured graph; on streams of its own."""
import pytest
import torch
from torch.nn import functional as F

from gpu_util import dev, say
from sparse_gemm_amd import expert_layer, experts, fp8
from sparse_gemm_amd.expert_layer import ExpertFFN

pytestmark = pytest.mark.gpu


def layer(dim=256, hidden=208, E=6, k=2, seed=0, **kw):
    torch.manual_seed(seed)
    return ExpertFFN(dim, hidden, E, k, bias=True, device=dev(), **kw)


def step(m, x, t):
    """The gradients of a loss."""
    return torch.autograd.grad((m(x).float() - t).square().sum(), [x, *m.parameters()])


def by_hand(m, x, t):
    """step from the single calls, without the autograd of this library: the gradients of the products in 8 bits are products in 8 bits."""
    B = lambda v: v.to(torch.bfloat16)   # noqa: E731
    with torch.no_grad():
        logits = F.linear(x, m.router)
        index, weight = experts.router_fwd(logits, m.k, m.renormalize)
        p = experts.ExpertPlan.from_index(index, m.num_experts)
        (uq, ut), (dq, dt) = fp8.quantize_blocks(m.up.data, transposed=True), fp8.quantize_blocks(m.down.data, transposed=True)
        z = fp8.expert_fwd(p, fp8.quantize_rows(x), uq, m.up_bias)
    z.requires_grad_(True)
    gate, up = z.chunk(2, dim=1)
    h = F.silu(gate) * up
    with torch.no_grad():
        hd = h.detach().contiguous()
        y = fp8.expert_fwd(p, fp8.quantize_rows(hd), dq, m.down_bias, gather=False)
        out = experts.combine_fwd(p, y, weight)
        dout = B(2 * (out.float() - t))
        dy, dw = experts.combine_bwd(p, dout, y, weight)
        dh = fp8.expert_fwd(p, fp8.quantize_rows(dy), dt, gather=False)
        ddown, ddown_bias = experts.expert_bwd_weight(p, dy, hd, False, True)
    dz, = torch.autograd.grad(h, z, dh)
    with torch.no_grad():
        dx = experts.combine_fwd(p, fp8.expert_fwd(p, fp8.quantize_rows(dz.contiguous()), ut, gather=False))
        dup, dup_bias = experts.expert_bwd_weight(p, dz.contiguous(), x, True, True)
        dlogits = experts.router_bwd(logits, index, weight, dw, m.renormalize)
        return [dx + dlogits @ m.router, dlogits.t() @ x, dup, ddown, dup_bias, ddown_bias]


@pytest.mark.parametrize("T", [1, 90, 700])
def test_training_then_prompt_then_tokens(T):
    m = layer(fp8=True, decode_tokens=16)
    g = torch.Generator(device=dev()).manual_seed(T)
    t = torch.randn(T, 256, generator=g, device=dev())
    for _ in range(3):
        x = torch.randn(T, 256, generator=g, device=dev()).bfloat16().requires_grad_(True)
        got, want = step(m, x, t), by_hand(m, x.detach(), t)
        for a, b, q in zip(got, want, [x, *m.parameters()]):
            assert a.shape == q.shape
            # the same kernels on the same values; library products and sums of x's two parts may round once each in another order
            assert float((a.double() - b.double()).norm()) <= 2.0 ** -7 * float(b.double().norm()) + 2.0 ** -126
        with torch.no_grad():
            for q, d in zip(m.parameters(), got[1:]):
                q -= 0.01 * d / (1 + d.float().norm())
        del got, want
    with torch.no_grad():
        prompt = torch.randn(100, 256, generator=g, device=dev()).bfloat16()
        trained = m(prompt)                     # still on bf16 weights, products in 8 bits
        m.quantize_("fp8")
        served = m(prompt)                      # quantised once: the same codes
        assert torch.equal(trained, served)
        m.prompt_tokens = 1000
        exact = m(prompt).double()              # activations in bf16
        tokens = torch.cat([m(prompt[a:a + n]) for a, n in ((0, 1), (1, 2), (3, 16), (19, 8), (27, 9))]).double()
        rel = float((tokens - exact[:36]).norm() / exact[:36].norm())
        say(f"    tokens against the batch {rel:.2e}")
        # logits, h, y of the batch are rounded to bf16 where the whole layer keeps 32 bits: 2^-8 each at most; the weights pass on the
        # logits' 2^-8, whose magnitude is below 4 here, twice
        assert float(F.linear(prompt, m.router).abs().max()) < 4
        assert rel < (2 * 4 + 4) * 2.0 ** -8


@pytest.mark.parametrize("T", [5, 300])
def test_a_captured_training_step(T):
    """Forward and backward in one graph, replayed with other inputs and weights. (No eager graph of the same leaves may live then: the
    step works on leaves of its own.)"""
    m, other = layer(fp8=True), layer(fp8=True)
    x, t = torch.randn(T, 256, device=dev()).bfloat16().requires_grad_(True), torch.randn(T, 256, device=dev())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(2):
            step(m, x, t)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(m, x, t)
    for i in range(3):
        with torch.no_grad():
            x.copy_(torch.randn(T, 256, device=dev()))
            t.copy_(torch.randn(T, 256, device=dev()))
            for q, r in zip(m.parameters(), other.parameters()):
                q.mul_(0.9)
                r.copy_(q)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, step(other, x.detach().clone().requires_grad_(True), t)):
            assert torch.equal(a, b)


def test_on_streams_of_its_own():
    """Calls on two streams at once, their inputs made there, against the same calls one after the other."""
    T, K, N, E = 400, 528, 272, 5
    p = experts.ExpertPlan.from_index(torch.randint(0, E, (T, 2), device=dev(), dtype=torch.int32), E)
    W = [torch.randn(E, N, K, device=dev()).bfloat16() for _ in range(2)]
    x = [torch.randn(T, K, device=dev()).bfloat16() for _ in range(2)]

    def run(i):
        a = (x[i].float() * 2).bfloat16()
        q, t = fp8.quantize_blocks(W[i], transposed=True)
        y = fp8.expert_fwd(p, fp8.quantize_rows(a), q)
        return y, fp8.expert_fwd(p, a, q), fp8.expert_fwd(p, fp8.quantize_rows(y), t, gather=False)

    want = [run(i) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [None, None]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = run(i)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_frozen_parts_get_no_gradient():
    """Weights alone, inputs alone, the bias alone."""
    T, K, N, E = 50, 64, 48, 3
    p = experts.ExpertPlan.from_index(torch.randint(0, E, (T, 1), device=dev(), dtype=torch.int32), E)
    x, W, b = (torch.randn(*s, device=dev()).bfloat16() for s in ((T, K), (E, N, K), (E, N)))
    dY = torch.randn(T, N, device=dev()).bfloat16()
    leaves = [v.clone().requires_grad_(True) for v in (x, W, b)]
    full = torch.autograd.grad(expert_layer.expert_linear_fp8(p, *leaves), leaves, dY)
    for i in range(3):
        mine = [v.clone().requires_grad_(j == i) for j, v in enumerate((x, W, b))]
        one, = torch.autograd.grad(expert_layer.expert_linear_fp8(p, *mine), [mine[i]], dY)
        assert torch.equal(one, full[i])
    expanded = torch.ones(1, 1, dtype=torch.bfloat16, device=dev()).expand(T, N)   # the gradient of a sum: strides of 0
    a, = torch.autograd.grad(expert_layer.expert_linear_fp8(p, leaves[0], W, b), [leaves[0]], expanded)
    c, = torch.autograd.grad(expert_layer.expert_linear_fp8(p, leaves[0], W, b), [leaves[0]], expanded.contiguous())
    assert torch.equal(a, c)


def test_the_example_in_8_bits():
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import expert_ffn
    got = expert_ffn.main(3, "fp8")
    # of x, W, h and the second W each value is rounded to E4M3, 2^-4 of it at most, and the activation passes its factors' on twice
    assert len(got["losses"]) == 3 and got["prompt"] < 6 * 2.0 ** -4 and got["token"] < 6 * 2.0 ** -4


def test_an_empty_batch():
    m = layer(fp8=True, decode_tokens=4)
    x = torch.zeros(0, 256, dtype=torch.bfloat16, device=dev(), requires_grad=True)
    got = step(m, x, torch.zeros(0, 256, device=dev()))
    for a, q in zip(got, [x, *m.parameters()]):
        assert a.shape == q.shape and not a.any()
    with torch.no_grad():
        assert m(x).shape == (0, 256) and m.quantize_("fp8")(x).shape == (0, 256)
