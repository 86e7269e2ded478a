"""Forward-mode derivatives: a tangent is refused by every path of an expert layer, whatever holds the weights and however many tokens
there are, instead of being dropped (a stand-in for the library records the calls; no GPU)."""
import pytest
import torch
from torch.autograd import forward_ad

from sparse_gemm_amd import expert_layer, fp8, mx4
from test_expert_calls_cpu import bf
from test_fp8_blocks_cpu import library  # noqa: F401

FORMS = ["bf16", "mx4", "fp8"]


def layer(form, decode_tokens=8):
    m = expert_layer.ExpertFFN(64, 64, 4, 2, bias=True, device="cpu", decode_tokens=decode_tokens)
    return m if form == "bf16" else m.quantize_(form)


def put(m, name):
    """A dual tensor in the place of a parameter."""
    p = getattr(m, name).detach()
    delattr(m, name)
    setattr(m, name, forward_ad.make_dual(p, torch.ones_like(p)))


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("decode_tokens", [0, 8])
@pytest.mark.parametrize("grad", [False, True])
def test_a_layer_refuses_tangents_of_its_input(library, form, decode_tokens, grad):  # noqa: F811
    m = layer(form, decode_tokens)
    for tokens in (1, 8, 9):
        with forward_ad.dual_level(), torch.set_grad_enabled(grad):
            x = forward_ad.make_dual(bf(tokens, 64), torch.ones(tokens, 64).bfloat16())
            with pytest.raises(NotImplementedError):
                m(x)
            assert m(forward_ad.unpack_dual(x).primal).shape == (tokens, 64)   # without a tangent


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("decode_tokens", [0, 8])
@pytest.mark.parametrize("name", ["router", "up", "down", "up_bias", "down_bias"])
def test_a_layer_refuses_tangents_of_its_parameters(library, form, decode_tokens, name):  # noqa: F811
    m = layer(form, decode_tokens)
    if getattr(m, name) is None:
        pytest.skip("held without it")
    with forward_ad.dual_level(), torch.no_grad():
        put(m, name)
        with pytest.raises(NotImplementedError):
            m(bf(3, 64))


@pytest.mark.parametrize("form", FORMS)
def test_the_whole_layer_refuses_tangents(library, form):  # noqa: F811
    hold = {"bf16": lambda W: W, "mx4": mx4.quantize, "fp8": fp8.quantize_blocks}[form]
    args = dict(x=bf(3, 64), router=bf(4, 64), up=hold(bf(4, 128, 64)), down=hold(bf(4, 64, 64)), up_bias=bf(4, 128), down_bias=bf(4, 64))
    for name in args:
        with forward_ad.dual_level():
            if not isinstance(args[name], torch.Tensor):
                continue
            dual = forward_ad.make_dual(args[name], torch.ones_like(args[name]))
            library.calls.clear()
            with pytest.raises(NotImplementedError, match="forward-mode"):
                expert_layer.expert_ffn(**{**args, name: dual}, k=2)
            assert not library.calls
            assert expert_layer.expert_ffn(**args, k=2).shape == (3, 64)
    assert expert_layer.expert_ffn(**args, k=2).shape == (3, 64)
