"""What the Python face of the expert layers passes to the library, without a GPU: tensors on the CPU pass for
tensors on GPU 0, and a stand-in for the library records the arguments of each call."""
import copy
import ctypes
import os
import pickle
import subprocess
import sys

import pytest
import torch

from conftest import ROOT
from sparse_gemm_amd import _lib, expert_layer, experts, mx4
from sparse_gemm_amd.experts import ExpertPlan


class Recorder:
    """Every function returns status 0 and leaves (name, arguments) in `calls`."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


@pytest.fixture
def library(monkeypatch):
    rec = Recorder()
    for module in (experts, mx4):
        monkeypatch.setattr(module, "C", rec)
        monkeypatch.setattr(module, "current_device", lambda: 0)
        monkeypatch.setattr(module, "raw_stream", lambda d: None)
        monkeypatch.setattr(module, "empty_strided", lambda shape, strides, dtype: torch.empty_strided(shape, strides, dtype=dtype))
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 0)
    return rec


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def a_plan(T=4, k=2, E=3):
    return ExpertPlan(torch.zeros(E + 1, dtype=torch.int32), torch.zeros(T * k, dtype=torch.int32),
                      torch.zeros((T, k), dtype=torch.int32))


def plan_calls(plan):
    """Every call that takes a plan, as (the call, the plan's tensors that it passes)."""
    T, k, E, R, N, K = plan.T, plan.k, plan.E, plan.R, 64, 64
    W, q = bf(E, N, K), mx4.Mx4(torch.zeros((E, N, K // 2), dtype=torch.uint8), torch.zeros((E, 1, N, 8), dtype=torch.uint8))
    x4 = mx4.Mx4(torch.zeros((T, K // 2), dtype=torch.uint8), torch.zeros((1, T, 8), dtype=torch.uint8))
    return [(lambda: experts.expert_fwd(plan, bf(T, K), W), ("offsets", "row_token")),
            (lambda: experts.expert_fwd(plan, bf(R, K), W, gather=False), ("offsets",)),
            (lambda: experts.expert_bwd_input(plan, bf(R, N), W), ("offsets",)),
            (lambda: experts.expert_bwd_weight(plan, bf(R, N), bf(T, K)), ("offsets", "row_token")),
            (lambda: experts.combine_fwd(plan, bf(R, N)), ("slot_row",)),
            (lambda: experts.combine_bwd(plan, bf(T, N), bf(R, N)), ("offsets", "slot_row")),
            (lambda: mx4.expert_fwd(plan, bf(T, K), q), ("offsets", "row_token")),
            (lambda: mx4.expert_fwd(plan, x4, q), ("offsets", "row_token"))]


def built(library):
    return ExpertPlan.from_index(torch.zeros((4, 2), dtype=torch.int32), 3)


@pytest.mark.parametrize("make", [lambda library: a_plan(), built], ids=["tensors", "index"])
@pytest.mark.parametrize("copied", [copy.copy, copy.deepcopy, lambda p: pickle.loads(pickle.dumps(p)),
                                    lambda p: copy.deepcopy({"plan": [p]})["plan"][0]], ids=["copy", "deepcopy", "pickle", "nested"])
def test_a_copied_plan_passes_its_own_memory(library, make, copied):
    original = make(library)
    plan = copied(original)
    assert (plan.T, plan.k, plan.E, plan.R, plan.device) == (4, 2, 3, 8, 0)
    for call, names in plan_calls(plan):
        library.calls.clear()
        call()
        (name, args), = library.calls
        for n in names:
            assert getattr(plan, n).data_ptr() in args, (name, n)
        if copied is not copy.copy:
            for n in ("offsets", "row_token", "slot_row"):
                assert getattr(original, n).data_ptr() not in args, (name, n)


def test_a_plan_keeps_its_tensors(library):
    plan = a_plan()
    for n in ("offsets", "row_token", "slot_row"):
        with pytest.raises(AttributeError):
            setattr(plan, n, torch.zeros(1, dtype=torch.int32))


def test_a_plan_without_its_gpu_is_refused(library, monkeypatch):
    """A plan's copy is checked like a plan from tensors: one whose tensors came back on the CPU is no plan."""
    data = pickle.dumps(a_plan())
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: -1)
    with pytest.raises(ValueError):
        pickle.loads(data)


@pytest.mark.parametrize("E,rows,K", [(3, 5, 32), (3, 41, 32), (2, 3, 256), (3, 7, 544), (1, 3, 32), (3, 5, 288), (3, 40, 320), (2, 0, 32)])
def test_every_experts_scales_are_aligned(library, E, rows, K):
    """[E, rows, K] goes to the library expert by expert, whose scales need not lie on whole 16 bytes among all experts'.
    Stand-ins write the expert's number into its scales, and read it."""
    c, n = mx4.chunks(K), rows * mx4.chunks(K) * 8
    read = []

    def quantize(x, r, k, codes, scales, values, stream):
        assert (r, k) == (rows, K) and x % 16 == codes % 16 == scales % 16 == 0
        ctypes.memset(scales, len(library.calls) + 1, n)
        library.calls.append(scales)
        return 0

    def dequantize(codes, scales, r, k, values, stream):
        assert (r, k) == (rows, K) and codes % 16 == scales % 16 == values % 16 == 0
        read.append(ctypes.string_at(scales, n))
        return 0

    library.bsr_mx4_quantize, library.bsr_mx4_dequantize = quantize, dequantize
    q = mx4.quantize(bf(E, rows, K))
    assert len(library.calls) == E and q.scales.shape == (E, c, rows, 8)
    for e in range(E):
        assert (q.scales[e] == e + 1).all()
    mx4.dequantize(q)
    assert read == [bytes([e + 1]) * n for e in range(E)]


def off_by_one(t):
    """t's values in contiguous memory that is not 16-byte aligned."""
    flat = torch.empty(t.numel() + 8, dtype=t.dtype)
    at = 1 if flat.data_ptr() % 16 == 0 else 0
    v = flat[at:at + t.numel()].view(t.shape)
    v.copy_(t)
    assert v.is_contiguous() and v.data_ptr() % 16
    return v


def test_autograd_functions_take_contiguous_slices(library, monkeypatch):
    """Slices of odd sizes are contiguous and not 16-byte aligned, which the library refuses: inputs, and incoming gradients
    (the gradient of a concatenation's part is such a slice), are copied where that is so."""
    T, k, E, N, K = 3, 1, 3, 64, 64

    def aligned(rec, name):
        def call(*args):
            rec.calls.append(name)
            bad = [a for a in args if isinstance(a, int) and a > 1 << 20 and a % 16]
            assert not bad, name
            return 0
        return call

    monkeypatch.setattr(Recorder, "__getattr__", aligned)
    plan = a_plan(T, k, E)
    logits = off_by_one(torch.zeros(T, E)).requires_grad_()
    index, weight = expert_layer.route(logits, k)
    weight.backward(off_by_one(torch.ones(T, k)))
    x, W, b = off_by_one(bf(T, K)).requires_grad_(), bf(E, N, K).requires_grad_(), bf(E, N).requires_grad_()
    expert_layer.expert_linear(plan, x, W, b).backward(off_by_one(bf(T * k, N)))
    y, w = off_by_one(bf(T * k, N)).requires_grad_(), off_by_one(torch.ones(T, k)).requires_grad_()
    expert_layer.combine(plan, y, w).backward(off_by_one(bf(T, N)))
    assert library.calls == ["bsr_router_fwd", "bsr_router_bwd", "bsr_expert_fwd", "bsr_expert_bwd_input", "bsr_expert_combine_fwd",
                             "bsr_expert_bwd_weight", "bsr_expert_combine_fwd", "bsr_expert_combine_bwd"]


def test_autograd_functions_do_not_copy_aligned_tensors(library):
    plan, T, N = a_plan(4, 2, 3), 4, 64
    x, W, y, w = bf(T, N), bf(3, N, N), bf(8, N), torch.ones(4, 2)
    logits = torch.zeros(4, 3)
    expert_layer.route(logits, 2)
    expert_layer.expert_linear(plan, x, W)
    expert_layer.combine(plan, y, w)
    for (name, args), tensors in zip(library.calls, ([logits], [x, W], [y, w])):
        for t in tensors:
            assert t.data_ptr() in args, name


@pytest.mark.parametrize("tokens", [3, 100])
def test_a_quantised_layer_trains_nothing(library, tokens):
    """quantize_() freezes what is left of the parameters, so that a model's optimiser finds no gradients missing; a layer
    that is asked to train after all refuses, whether its input wants a gradient or not."""
    m = expert_layer.ExpertFFN(64, 64, 4, 2, bias=True, device="cpu").quantize_()
    x = bf(tokens, 64)
    assert {n for n, _ in m.named_parameters()} == {"router", "up_bias", "down_bias"}
    assert not any(p.requires_grad for p in m.parameters())
    assert not m(x).requires_grad
    with pytest.raises(RuntimeError, match="no backward"):
        m(x.clone().requires_grad_())
    for name in ("router", "up_bias", "down_bias"):
        m.requires_grad_(False)
        getattr(m, name).requires_grad_()
        with pytest.raises(RuntimeError, match="no backward"):
            m(x)
        with torch.no_grad():
            assert m(x).shape == (tokens, 64)


@pytest.mark.parametrize("train_W", [False, True])
@pytest.mark.parametrize("train_b", [False, True])
def test_only_wanted_gradients_are_computed(library, train_W, train_b):
    plan, T, R, E, N, K = a_plan(), 4, 8, 3, 64, 64
    x, W, b = bf(T, K).requires_grad_(), bf(E, N, K).requires_grad_(train_W), bf(E, N).requires_grad_(train_b)
    y = expert_layer.expert_linear(plan, x, W, b)
    library.calls.clear()
    y.backward(bf(R, N))
    calls = dict(library.calls)
    assert ("bsr_expert_bwd_weight" in calls) == (train_W or train_b)
    if train_W or train_b:
        dW, db = calls["bsr_expert_bwd_weight"][9:11]
        assert (dW is not None) == train_W and (db is not None) == train_b
    assert (W.grad is not None) == train_W and (b.grad is not None) == train_b


def test_sizes_past_32_bits_are_refused(library):
    """The library takes widths, experts and slots as 32-bit numbers; a larger one would reach it cut to its low bits."""
    big = (1 << 32) + 64
    meta = lambda *s, dtype=torch.bfloat16: torch.empty(s, dtype=dtype, device="meta")   # noqa: E731
    plan = a_plan(1, 1, 1)
    u8, i32, f32 = torch.uint8, torch.int32, torch.float32
    calls = [lambda: mx4.quantize(meta(1, big)), lambda: mx4.quantize(meta(2, 1, big)),
             lambda: mx4.dequantize(mx4.Mx4(meta(1, big // 2 + 32, dtype=u8), meta(big // 256, 1, 8, dtype=u8))),
             lambda: experts.router_fwd(meta(1, big, dtype=f32), 2),
             lambda: experts.router_bwd(meta(1, big, dtype=f32), meta(1, 2, dtype=i32), meta(1, 2, dtype=f32), meta(1, 2, dtype=f32)),
             lambda: ExpertPlan.from_index(meta(1, big, dtype=i32), 8),
             lambda: ExpertPlan(meta(big, dtype=i32), meta(2, dtype=i32), meta(1, 2, dtype=i32)),
             lambda: experts.expert_fwd(plan, meta(1, 64), meta(1, big, 64)),
             lambda: experts.expert_fwd(plan, meta(1, big), meta(1, 64, big)),
             lambda: experts.expert_bwd_input(plan, meta(1, big), meta(1, big, 64)),
             lambda: experts.expert_bwd_weight(plan, meta(1, big), meta(1, 64)),
             lambda: experts.expert_bwd_weight(plan, meta(1, 64), meta(1, big)),
             lambda: experts.combine_fwd(plan, meta(1, big)), lambda: experts.combine_bwd(plan, meta(1, big), meta(1, big)),
             lambda: mx4.expert_fwd(plan, meta(1, 64), mx4.Mx4(meta(1, big, 32, dtype=u8), meta(1, 1, big, 8, dtype=u8)))]
    for i, call in enumerate(calls):
        with pytest.raises(ValueError, match="2\\^31"):
            call()
        assert not library.calls, i


def test_slots_and_experts_reach_the_library_whole(library, monkeypatch):
    """k and E come from the caller, and are refused by the library, not cut."""
    monkeypatch.setattr(experts, "empty_strided", lambda shape, strides, dtype: torch.empty(4, dtype=dtype))
    experts.router_fwd(torch.zeros(1, 8), (1 << 32) + 2)
    ExpertPlan.from_index(torch.zeros((1, 2), dtype=torch.int32), (1 << 32) + 8)
    (_, router), (_, plan) = library.calls
    assert router[4] == plan[3] == (1 << 31) - 1


@pytest.mark.filterwarnings("ignore:Accessing the data pointer")
def test_tensors_without_memory_are_refused(library, monkeypatch):
    """Fake tensors (torch's tracing) have no address, and the library itself refuses that before anything is enqueued."""
    from torch._subclasses.fake_tensor import FakeTensorMode
    plan, real = a_plan(), experts._Calls()
    monkeypatch.setattr(experts, "C", real)
    monkeypatch.setattr(mx4, "C", real)
    with FakeTensorMode(allow_non_fake_inputs=True):
        calls = [lambda: experts.router_fwd(torch.zeros(4, 3), 2), lambda: ExpertPlan.from_index(torch.zeros((4, 2), dtype=torch.int32), 3),
                 lambda: experts.expert_fwd(plan, bf(4, 64), bf(3, 64, 64)), lambda: experts.combine_fwd(plan, bf(8, 64)),
                 lambda: mx4.quantize(bf(4, 64))]
        for call in calls:
            with pytest.raises(_lib.BsrError, match="is NULL"):
                call()


def test_the_module_needs_no_private_names():
    """Without torch's private calls for stream, device and allocation the public ones take their place."""
    code = """
import torch
for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
if hasattr(torch._C._dynamo.guards, "_empty_strided_cuda"):
    del torch._C._dynamo.guards._empty_strided_cuda
from sparse_gemm_amd import experts, mx4
assert experts.current_device is torch.cuda.current_device
torch.cuda.current_stream = lambda d: type("Stream", (), {"cuda_stream": 70 + d})
assert experts.raw_stream(1) == mx4.raw_stream(1) == 71
try:
    experts.router_fwd(torch.zeros(4, 8), 2)
except ValueError:
    print("refused")
"""
    env = {**os.environ, "PYTHONPATH": ROOT}
    out = subprocess.run([sys.executable, "-c", code], env=env, capture_output=True, text=True, timeout=300)
    assert out.stdout.strip() == "refused", out.stderr
