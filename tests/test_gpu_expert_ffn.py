"""A whole layer of experts for a few tokens against the definition in 64 bits, on weights in bf16, MXFP4 and 8 bits."""
import math

import numpy as np
import pytest
import torch

import fp8_ref
from expert_ref import f64
from gpu_util import dev, say
from sparse_gemm_amd import _lib, expert_layer, few_tokens, fp8, mx4

pytestmark = pytest.mark.gpu

HOLD = {"bf16": lambda W: W, "mx4": mx4.quantize, "fp8": fp8.quantize_blocks}
VALUES = {"bf16": lambda W: W, "mx4": mx4.dequantize, "fp8": fp8.dequantize}


def gen(seed):
    return torch.Generator().manual_seed(seed)


class Layer:
    """Inputs of a case on the CPU, what is held on the GPU, and the values that it stands for."""

    def __init__(self, form, T, dim, hidden, E, k, renorm, bias, seed=0):
        g = gen(seed + T + dim + hidden + E + k)
        bf = lambda *s, std=1.0: (torch.randn(s, generator=g) * std).bfloat16()   # noqa: E731
        self.k, self.renorm, self.form = k, renorm, form
        self.router = bf(E, dim, std=dim ** -0.5)
        self.x = bf(T, dim)
        self.up = HOLD[form](bf(E, 2 * hidden, dim, std=dim ** -0.5).to(dev()))
        self.down = HOLD[form](bf(E, dim, hidden, std=hidden ** -0.5).to(dev()))
        self.up_bias, self.down_bias = (bf(E, 2 * hidden, std=0.3), bf(E, dim, std=0.3)) if bias else (None, None)
        self.upv, self.downv = f64(VALUES[form](self.up)), f64(VALUES[form](self.down))
        for _ in range(50):   # tokens whose choice 32-bit sums cannot change
            near = torch.from_numpy(self.want()[3] < 1.0)
            if not near.any():
                break
            self.x = torch.where(near[:, None], bf(T, dim), self.x)
        else:
            raise AssertionError("no such tokens")

    def want(self):
        o = lambda t: None if t is None else f64(t)   # noqa: E731
        return fp8_ref.layer(f64(self.x), f64(self.router), lambda e: self.upv[e], lambda e: self.downv[e], self.k, self.renorm,
                             o(self.up_bias), o(self.down_bias))

    def args(self):
        o = lambda t: None if t is None else t.to(dev())   # noqa: E731
        return dict(x=self.x.to(dev()), router=self.router.to(dev()), up=self.up, down=self.down, k=self.k, renormalize=self.renorm,
                    up_bias=o(self.up_bias), down_bias=o(self.down_bias))

    def check(self, got):
        out, tol, _, _ = self.want()
        off = np.abs(f64(got) - out)
        assert np.isfinite(f64(got)).all()
        assert (off <= tol).all(), f"worst {np.max(off / tol):.3f} of the tolerance at {np.unravel_index(np.argmax(off / tol), out.shape)}"
        say(f"    worst {np.max(off / tol):.3f} of the tolerance")


STEP = {"bf16": 8, "fp8": 16, "mx4": 32}
#        T, dim, hidden (in steps of the form), E, k, renormalize, bias
CASES = [(1, 1, 1, 1, 1, True, False), (1, 8, 4, 8, 2, True, True), (3, 9, 7, 4, 4, False, True), (16, 5, 11, 60, 4, True, False),
         (16, 17, 3, 8, 2, False, True), (7, 33, 13, 64, 8, False, False), (2, 40, 67, 128, 8, True, True), (5, 3, 5, 200, 32, True, False),
         (16, 4, 2, 1024, 32, False, True), (16, 2, 9, 12, 12, True, True), (9, 130, 21, 16, 1, False, False), (4, 19, 300, 4, 2, True, False),
         (8, 12, 1, 256, 32, True, True), (8, 40, 1, 256, 32, False, False), (8, 100, 1, 256, 32, True, False), (16, 40, 3, 256, 24, True, True),
         (12, 100, 1, 256, 24, False, True), (8, 5, 1, 64, 8, True, True), (16, 5, 1, 64, 4, False, True)] + [(T, 20, hidden, 200, k, T > 8, False) for T, k in ((8, 32), (12, 20)) for hidden in (1, 2, 4)]


@pytest.mark.parametrize("T,dim,hidden,E,k,renorm,bias", CASES)
@pytest.mark.parametrize("form", ["bf16", "mx4", "fp8"])
def test_layer(form, T, dim, hidden, E, k, renorm, bias):
    dim, hidden = dim * STEP[form], hidden * STEP[form]
    say(f"case expert_ffn {form} T={T} dim={dim} hidden={hidden} E={E} k={k} renorm={renorm} bias={bias}")
    m = Layer(form, T, dim, hidden, E, k, renorm, bias)
    a = m.args()
    got = expert_layer.expert_ffn(**a)
    m.check(got)
    room = torch.full((T + 2, dim), math.nan, dtype=torch.bfloat16, device=dev())
    again = few_tokens.expert_ffn(**a, out=room[:T])
    assert torch.equal(again, got)   # and the same bits each time
    assert torch.isnan(room[T:]).all()


WIDE_CASES = [(1, 2048, 1024, 8, 2), (4, 4096, 1792, 8, 2), (16, 4128, 288, 16, 4), (3, 8224, 96, 4, 2), (11, 4096, 64, 24, 3), (2, 4096, 256, 4, 1), (16, 2048, 96, 64, 8), (2, 1536, 640, 8, 4)]

# weights of 256 MB and more, rows of whole lines
STREAMED = [("bf16", T, *c) for T in (5, 9) for c in ((4096, 5504, 2, 2), (8192, 2752, 2, 2), (2560, 4416, 4, 2), (1536, 3648, 8, 4), (1024, 5504, 8, 4))]
STREAMED += [(form, 8 if form == "fp8" else 10, 1024, hidden, 8, 4) for form, hidden in (("fp8", 11008), ("mx4", 22016))]
STREAMED += [(form, 3 if form == "mx4" else 12, 4864, hidden, 2, 2) for form, hidden in (("fp8", 9344), ("mx4", 18688))]


@pytest.mark.parametrize("form", ["bf16", "mx4", "fp8"])
@pytest.mark.parametrize("T,dim,hidden,E,k", WIDE_CASES)
def test_wide_layer(form, T, dim, hidden, E, k):
    say(f"case expert_ffn {form} T={T} dim={dim} hidden={hidden} E={E} k={k}")
    m = Layer(form, T, dim, hidden, E, k, True, False)
    m.check(expert_layer.expert_ffn(**m.args()))


@pytest.mark.parametrize("form,T,dim,hidden,E,k", STREAMED)
def test_large_layer(form, T, dim, hidden, E, k):
    say(f"case expert_ffn {form} T={T} dim={dim} hidden={hidden} E={E} k={k}")
    m = Layer(form, T, dim, hidden, E, k, True, True)
    m.check(expert_layer.expert_ffn(**m.args()))


@pytest.mark.parametrize("form", ["bf16", "mx4", "fp8"])
@pytest.mark.parametrize("T,first", [(9, 1), (9, 8), (9, 9), (16, 7), (16, 8), (16, 0), (13, 8), (8, 8)])
@pytest.mark.parametrize("dim", [1, 128])
def test_tokens_of_one_expert(form, T, first, dim):
    """Up to 8 tokens of an expert share an operand: `first` tokens choose one expert, the others the other."""
    dim *= 32
    m = Layer(form, T, dim, 96, 3, 1, True, True)
    m.router = torch.zeros(3, dim).bfloat16()
    m.router[1, 5], m.router[2, 5] = 4.0, -4.0
    order = torch.randperm(T, generator=gen(first))
    m.x[:, 5] = -1.0
    m.x[order[:first], 5] = 1.0
    assert m.want()[2].reshape(-1).tolist().count(1) == first
    m.check(expert_layer.expert_ffn(**m.args()))


def test_ties_go_to_the_lowest_expert():
    m = Layer("bf16", 6, 136, 24, 16, 3, True, False)
    m.router = m.router[torch.arange(16) // 2 * 2]   # pairs of equal logits
    want = m.want()
    assert all(len(set(i // 2 for i in row)) == 2 for row in want[2].tolist())
    m.check(expert_layer.expert_ffn(**m.args()))


@pytest.mark.parametrize("form", ["bf16", "mx4", "fp8"])
def test_values_that_are_not_finite_stay_where_they_are(form):
    """A token of NaN has a result of NaN, and no other has; the weights of experts that no token chose are not read, and NaN
    weights reach only the tokens of their expert."""
    m = Layer(form, 9, 160, 96, 32, 2, True, False)
    index = m.want()[2]
    a = m.args()
    clean = expert_layer.expert_ffn(**a)
    a["x"][4] = math.nan
    got = expert_layer.expert_ffn(**a)
    others = torch.arange(9) != 4
    assert torch.isnan(got[4]).all() and torch.equal(got[others], clean[others])
    a = m.args()
    unused = [e for e in range(32) if e not in set(index.reshape(-1).tolist())]
    chosen = int(index[0, 0])
    for name in ("up", "down"):
        W = VALUES[form](a[name]).clone()
        W[unused] = math.nan
        if name == "down":
            W[chosen] = math.nan
        a[name] = HOLD[form](W)
    got = expert_layer.expert_ffn(**a)
    hit = torch.from_numpy((index == chosen).any(1))
    assert unused and torch.isnan(got[hit]).all() and torch.equal(got[~hit], clean[~hit])


@pytest.mark.parametrize("form", ["bf16", "mx4", "fp8"])
@pytest.mark.parametrize("T", [3, 12])
@pytest.mark.parametrize("E", [6, 70, 300])
def test_experts_out_of_reach(form, T, E):
    """A logit of -infinity: its expert is not chosen, and a token without any has a result of zeros."""
    m = Layer(form, T, 96, 64, E, 3, True, True)
    a = m.args()
    near = [1, E - 2]
    a["x"][:, 7] = 1.0
    a["router"][:, 7] = -math.inf
    assert not expert_layer.expert_ffn(**a).any()
    a["router"][near, 7] = 0.5
    got = expert_layer.expert_ffn(**a).double()
    pick = (lambda W: W[near]) if form == "bf16" else (lambda W: type(W)(W.codes[near].contiguous(), W.scales[near].contiguous()))
    want = expert_layer.expert_ffn(a["x"], a["router"][near].contiguous(), pick(a["up"]), pick(a["down"]), 2, True,
                                   a["up_bias"][near].contiguous(), a["down_bias"][near].contiguous()).double()
    # sums in another order: h and the result may each round to a neighbour, 2 * 2^-8 of a value
    assert float((got - want).norm()) <= 4 * 2.0 ** -8 * float(want.norm())
    far = a["x"].clone()
    far[0, 7] = -1.0   # the signs of token 0 turn: all but two are +infinity, NaN weights
    assert torch.equal(expert_layer.expert_ffn(**{**a, "x": far})[1:].double(), got[1:])


def test_no_tokens():
    m = Layer("bf16", 1, 64, 32, 4, 2, True, False)
    a = m.args()
    a["x"] = a["x"][:0]
    assert expert_layer.expert_ffn(**a).shape == (0, 64)


@pytest.mark.parametrize("form", ["bf16", "mx4", "fp8"])
def test_captured_and_replayed(form):
    m = Layer(form, 5, 288, 160, 16, 4, True, True)
    a = m.args()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        expert_layer.expert_ffn(**a)
    torch.cuda.current_stream().wait_stream(s)
    first, second = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(first):
        one = expert_layer.expert_ffn(**a)
    with torch.cuda.graph(second):
        two = expert_layer.expert_ffn(**{**a, "x": one})   # the layer after it
    for i in range(4):
        a["x"].copy_(torch.randn(a["x"].shape, generator=gen(i)))
        first.replay()
        second.replay()
        torch.cuda.synchronize()
        want = expert_layer.expert_ffn(**a)
        assert torch.equal(one, want)
        assert torch.equal(two, expert_layer.expert_ffn(**{**a, "x": want}))


def test_two_streams_at_once():
    """Calls on two streams have a workspace each."""
    ms = [Layer(form, 16, 512, 512, 16, 4, True, False, seed) for seed, form in enumerate(("bf16", "fp8"))]
    args = [m.args() for m in ms]
    want = [expert_layer.expert_ffn(**a) for a in args]
    streams = [torch.cuda.Stream() for _ in ms]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(expert_layer.expert_ffn(**args[i]))
    torch.cuda.synchronize()
    for w, gs in zip(want, got):
        assert all(torch.equal(w, x) for x in gs)


@pytest.mark.parametrize("form", ["bf16", "mx4", "fp8"])
def test_the_layer_module_calls_it(form):
    """ExpertFFN with decode_tokens: few tokens without a gradient take the whole layer, up to the roundings that the single calls
    make between; more tokens, and tokens that want gradients, take those."""
    torch.manual_seed(4)
    m = expert_layer.ExpertFFN(128, 192, 8, 2, bias=True, device=dev(), decode_tokens=8)
    plain = expert_layer.ExpertFFN(128, 192, 8, 2, bias=True, device=dev())
    plain.load_state_dict(m.state_dict())
    if form != "bf16":
        m.quantize_(form), plain.quantize_(form)
    x = torch.randn(2, 3, 128, device=dev()).bfloat16()
    with torch.no_grad():
        few, single = m(x), plain(x)
        assert few.shape == x.shape and torch.equal(m(x.repeat(2, 1, 1)), plain(x.repeat(2, 1, 1)))
    held = m._held() if m.quantized else (m.up.detach(), m.down.detach())
    direct = few_tokens.expert_ffn(x.reshape(6, 128), m.router.detach(), *held, 2, True, m.up_bias.detach(), m.down_bias.detach())
    assert torch.equal(direct.reshape(x.shape), few)
    # the single calls round logits (2^-8 of up to 3: a weight is off by 2^-6), gate, up, silu, their product and each expert's row
    rel = float((few.double() - single.double()).norm() / single.double().norm())
    say(f"    relative difference {rel:.2e}")
    assert rel < 2.0 ** -5
    if form == "bf16":
        assert torch.equal(m(x), plain(x))   # parameters that want gradients
        with pytest.raises(RuntimeError):
            expert_layer.expert_ffn(x.reshape(6, 128), m.router, m.up, m.down, 2)


def test_refusals():
    m = Layer("fp8", 2, 64, 32, 4, 2, True, False)
    a = m.args()
    call = lambda **kw: few_tokens.expert_ffn(**{**a, **kw})   # noqa: E731
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device=dev())   # noqa: E731
    with pytest.raises(ValueError, match="at most 16"):
        call(x=bf(17, 64))
    with pytest.raises(TypeError, match="same form"):
        call(down=bf(4, 64, 32))
    with pytest.raises(ValueError):
        call(x=bf(2, 128))
    with pytest.raises(ValueError):
        call(down=fp8.quantize_blocks(bf(4, 64, 48)))
    with pytest.raises(ValueError):
        call(up_bias=bf(4, 32))
    with pytest.raises(TypeError):
        call(x=bf(2, 64).float())
    with pytest.raises(ValueError):
        call(router=bf(4, 64).cpu())
    with pytest.raises(_lib.BsrError, match="k must"):
        call(k=5)
    with pytest.raises(_lib.BsrError, match="multiples of 16"):
        few_tokens.expert_ffn(bf(2, 64), bf(4, 64), fp8.quantize_blocks(bf(4, 48, 64)),
                              fp8.Fp8Blocks(torch.zeros((4, 64, 24), dtype=torch.uint8, device=dev()),
                                            torch.zeros((4, 1, 1), dtype=torch.uint8, device=dev())), 2)
