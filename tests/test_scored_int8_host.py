"""Host-side checks of scored routing and the int8 layer that need no GPU: every
refusal comes back as a status before anything is launched, and the references
the GPU tests use agree with independent formulas."""
import ctypes

import numpy as np
import pytest
import torch

import sparse_mixture_experts_05_b200 as moe
from sparse_mixture_experts_05_b200 import binding

import _scored as ref

P = ctypes.c_void_p
GOOD = P(1 << 20)           # never dereferenced: validation fails first
BAD = P((1 << 20) + 8)      # not 16-byte aligned
BIG = ctypes.c_size_t(1 << 40)


def _call(fn, *args):
    return getattr(binding.lib(), fn)(*args)


def _S(*shape):
    return binding.MoeShape(*shape)


@pytest.mark.parametrize("shape,code", [
    ((64, 128, 256, 8, 2), moe.MOE_OK),
    ((0, 16, 16, 1, 1), moe.MOE_OK),
    ((4096, 4096, 14336, 512, 16), moe.MOE_OK),
    ((1 << 27, 131072, 16, 1, 1), moe.MOE_OK),
    ((-1, 128, 256, 8, 2), moe.MOE_ERR_INVALID_ARG),
    ((64, 128, 256, 8, 0), moe.MOE_ERR_INVALID_ARG),
    ((64, 128, 256, 8, 9), moe.MOE_ERR_INVALID_ARG),
    ((64, 0, 256, 8, 2), moe.MOE_ERR_INVALID_ARG),
    ((64, 128, -16, 8, 2), moe.MOE_ERR_INVALID_ARG),
    ((64, 120, 256, 8, 2), moe.MOE_ERR_UNSUPPORTED),
    ((64, 128, 264, 8, 2), moe.MOE_ERR_UNSUPPORTED),
    ((64, 131088, 256, 8, 2), moe.MOE_ERR_UNSUPPORTED),
    ((64, 128, 256, 513, 2), moe.MOE_ERR_UNSUPPORTED),
    ((64, 128, 256, 32, 17), moe.MOE_ERR_UNSUPPORTED),
    (((1 << 26) + 1, 128, 256, 8, 2), moe.MOE_ERR_UNSUPPORTED),
])
def test_shape_checks(shape, code):
    assert moe.moe_check_shape_int8(shape) == code
    ws = moe.moe_forward_int8_workspace_bytes(shape)
    assert (ws > 0) == (code == moe.MOE_OK)
    assert (moe.moe_expert_swiglu_int8_workspace_bytes(shape) > 0) == (code == moe.MOE_OK)


@pytest.mark.parametrize("k,E,scoring,code", [
    (8, 256, dict(n_group=8, topk_group=4, group_top=2), moe.MOE_OK),
    (16, 512, dict(n_group=32, topk_group=1), moe.MOE_OK),
    (2, 8, dict(n_group=3), moe.MOE_ERR_INVALID_ARG),                  # 8 experts, 3 groups
    (2, 8, dict(n_group=0), moe.MOE_ERR_INVALID_ARG),
    (2, 8, dict(n_group=4, topk_group=5), moe.MOE_ERR_INVALID_ARG),
    (2, 8, dict(n_group=4, topk_group=0), moe.MOE_ERR_INVALID_ARG),
    (3, 8, dict(n_group=4, topk_group=1), moe.MOE_ERR_INVALID_ARG),     # 2 experts for 3 slots
    (2, 8, dict(group_top=0), moe.MOE_ERR_INVALID_ARG),
    (2, 8, dict(group_top=3), moe.MOE_ERR_INVALID_ARG),
    (2, 8, dict(scale=float("nan")), moe.MOE_ERR_INVALID_ARG),
    (2, 8, dict(scale=float("inf")), moe.MOE_ERR_INVALID_ARG),
    (2, 64, dict(n_group=64, topk_group=8), moe.MOE_ERR_UNSUPPORTED),
    (2, 513, dict(), moe.MOE_ERR_UNSUPPORTED),
    (17, 64, dict(), moe.MOE_ERR_UNSUPPORTED),
    (9, 8, dict(), moe.MOE_ERR_INVALID_ARG),
])
def test_scoring_checks(k, E, scoring, code):
    sc = moe.MoeScoring(**scoring)
    assert moe.moe_check_scoring((4, 0, 0, E, k), sc) == code
    if code != moe.MOE_OK:
        S = _S(4, 128, 128, E, k)
        assert _call("moe_route_scored", S, sc, GOOD, 0, None, None, GOOD, GOOD, None) == code
        assert _call("moe_route_scored_backward", S, sc, GOOD, 0, GOOD, GOOD, GOOD, None) == code
        assert _call("moe_forward_int8", S, GOOD, GOOD, 0, sc, None, None, *([GOOD] * 6), GOOD, None,
                     None, GOOD, BIG, None) == code


def test_unknown_scores():
    with pytest.raises(ValueError):
        moe.MoeScoring(score="tanh")
    sc = moe.MoeScoring()
    sc.score = 2
    assert moe.moe_check_scoring((4, 0, 0, 8, 2), sc) == moe.MOE_ERR_INVALID_ARG


def test_routing_pointers():
    S, sc = _S(4, 128, 128, 8, 2), moe.MoeScoring()
    bad = moe.MOE_ERR_INVALID_ARG
    args = [GOOD, 0, GOOD, GOOD, GOOD, GOOD]
    for i in (0, 4, 5):
        for p in (None, BAD):
            a = list(args)
            a[i] = p
            assert _call("moe_route_scored", S, sc, *a, None) == bad
    for i in (2, 3):
        a = list(args)
        a[i] = BAD
        assert _call("moe_route_scored", S, sc, *a, None) == bad
    assert _call("moe_route_scored", S, sc, GOOD, 2, None, None, GOOD, GOOD, None) == bad
    args = [GOOD, 0, GOOD, GOOD, GOOD]
    for i in (0, 2, 3, 4):
        for p in (None, BAD):
            a = list(args)
            a[i] = p
            assert _call("moe_route_scored_backward", S, sc, *a, None) == bad
    assert _call("moe_route_scored_backward", S, sc, GOOD, -1, GOOD, GOOD, GOOD, None) == bad
    # nothing to do
    E0 = _S(0, 128, 128, 8, 2)
    assert _call("moe_route_scored", E0, sc, None, 0, None, None, None, None, None) == moe.MOE_OK
    assert _call("moe_route_scored_backward", E0, sc, None, 0, None, None, None, None) == moe.MOE_OK


def test_int8_pointers_and_workspaces():
    S, sc = _S(64, 128, 256, 8, 2), moe.MoeScoring()
    bad = moe.MOE_ERR_INVALID_ARG
    for p in (None, BAD):
        for i in range(3):
            a = [GOOD] * 3
            a[i] = p
            assert _call("moe_quantize_weights_int8", 2, 128, 64, *a, None) == bad
            a = [GOOD] * 4
            a[i] = p
            assert _call("moe_combine_bf16", S, *a, None) == bad
        for i in range(7):
            a = [GOOD] * 7
            a[i] = p
            assert _call("moe_dispatch_int8", S, *a, None) == bad
        for i in range(11):
            a = [GOOD] * 11
            a[i] = p
            assert _call("moe_expert_swiglu_int8", S, *a, BIG, None) == bad
    assert _call("moe_quantize_weights_int8", 0, 128, 64, GOOD, GOOD, GOOD, None) == bad
    for e, k, n in ((513, 128, 64), (2, 120, 64), (2, 128, 72), (2, 131088, 64)):
        assert _call("moe_quantize_weights_int8", e, k, n, GOOD, GOOD, GOOD, None) == \
            moe.MOE_ERR_UNSUPPORTED
    need = moe.moe_expert_swiglu_int8_workspace_bytes((64, 128, 256, 8, 2))
    assert _call("moe_expert_swiglu_int8", S, *([GOOD] * 11), ctypes.c_size_t(need - 1), None) == \
        moe.MOE_ERR_WORKSPACE
    t = ctypes.c_uint64(10 ** 6)
    assert _call("moe_expert_swiglu_int8_stall_test", S, *([GOOD] * 11), BIG, -1, t, None) == bad
    assert _call("moe_expert_swiglu_int8_stall_test", S, *([GOOD] * 11), BIG, 0,
                 ctypes.c_uint64(10), None) == bad
    need = moe.moe_forward_int8_workspace_bytes((64, 128, 256, 8, 2))

    def forward(args, nbytes=BIG, kind=0):
        x, logits, bias, mask, w, y, idx, gate, ws = args
        return _call("moe_forward_int8", S, x, logits, kind, sc, bias, mask, *([w] * 6), y, idx, gate,
                     ws, nbytes, None)
    args = [GOOD, GOOD, None, None, GOOD, GOOD, None, None, GOOD]
    assert forward(args, ctypes.c_size_t(need - 1)) == moe.MOE_ERR_WORKSPACE
    assert forward(args, kind=3) == bad
    for i in range(9):
        a = list(args)
        a[i] = BAD
        assert forward(a) == bad
    for i in (0, 1, 4, 5, 8):
        a = list(args)
        a[i] = None
        assert forward(a) == bad


def test_binding_refuses_wrong_tensors():
    sc = moe.MoeScoring()
    with pytest.raises(ValueError):
        moe.moe_route_scored((4, 128, 128, 8, 2), torch.zeros(4, 8, dtype=torch.float16), sc)
    with pytest.raises(ValueError):
        moe.moe_route_scored((4, 128, 128, 8, 2), torch.zeros(4, 8), sc)       # not on a GPU
    with pytest.raises(ValueError):
        moe.moe_quantize_weights_int8(torch.zeros(2, 16, 16, dtype=torch.bfloat16))


# ------------------------------------------------------------------ the references themselves

def test_quotients_round_alike_in_32_and_64_bits():
    """rint(x * 127 / amax) from one product with 127 / amax rounded up, as the
    kernels form it, against the exact integers, for every pair of bf16 significands."""
    from fractions import Fraction
    for A in range(128, 256):
        for shift in (0, 1, 3, 6, 9):
            xs = np.arange(0, 256) if shift else np.arange(0, A + 1)
            xs = xs[xs <= A * 2 ** shift]
            exact = [Fraction(int(X) * 127, A * 2 ** shift) for X in xs]
            want = np.array([round(f) for f in exact])  # ties to even
            r = np.float32(127.0 / A)
            if float(r) < 127.0 / A:
                r = np.nextafter(r, np.float32(np.inf), dtype=np.float32)
            prod = xs.astype(np.float64) / 2 ** shift * float(r)     # exact: 8 + 24 bits
            assert np.array_equal(np.rint(prod).astype(int), want)   # the fused add rounds it once


def test_ties_are_at_half_the_largest_value_or_have_an_exact_multiplier():
    """127 X / (A 2^shift) half way between two whole numbers, for all bf16 significands: X is half of A's
    value, or 127 divides A and 127 / A is a power of two."""
    kinds = set()
    for A in range(128, 256):
        for shift in range(0, 9):
            for X in range(1, 256):
                if X <= A << shift and (2 * 127 * X) % (A << shift) == 0 and (2 * 127 * X // (A << shift)) % 2:
                    kinds.add("half" if 2 * X == A << shift else "exact")
                    assert 2 * X == A << shift or A == 254
    assert kinds == {"half", "exact"}


def test_reference_gates_by_torch():
    l = torch.randn(6, 12, generator=torch.Generator().manual_seed(1))
    for score in ("softmax", "sigmoid"):
        p = torch.softmax(l.double(), 1) if score == "softmax" else torch.sigmoid(l.double())
        for renorm in (True, False):
            idx, gate = ref.route(l, 3, dict(score=score, renorm=renorm, scale=1.5))
            v, i = torch.topk(p, 3)
            assert np.array_equal(i.numpy(), idx)
            w = v / v.sum(1, keepdim=True) if renorm else v
            assert np.allclose(gate, 1.5 * w.numpy(), rtol=1e-12)


def test_reference_gradient_by_autograd():
    l = torch.randn(5, 10, generator=torch.Generator().manual_seed(2))
    dg = torch.randn(5, 4, generator=torch.Generator().manual_seed(3))
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            sc = dict(score=score, renorm=renorm, scale=2.0)
            idx, _ = ref.route(l, 4, sc)
            x = l.double().requires_grad_()
            p = torch.softmax(x, 1) if score == "softmax" else torch.sigmoid(x)
            w = p.gather(1, torch.as_tensor(idx))
            if renorm:
                w = w / w.sum(1, keepdim=True)
            (2.0 * w * dg.double()).sum().backward()
            got, _ = ref.route_backward(l, torch.as_tensor(idx), dg, sc)
            assert np.allclose(got, x.grad.numpy(), rtol=1e-9, atol=1e-12)


def test_binding_refuses_a_stream_of_another_device():
    class Stream:
        device_index, cuda_stream = 1, 0
    with pytest.raises(ValueError, match="cuda:1"):
        binding._queue(Stream(), 0)
    assert binding._queue(Stream(), 1) == 0


def test_a_shape_is_read_anew_by_every_call():
    T = torch.tensor(4)
    shape = [T, 128, np.int64(128), 8, 2]
    assert binding._shape(shape).T == 4
    T.add_(1)
    assert binding._shape(shape).T == 5


@pytest.mark.parametrize("shape", [(4, 128, 128, 8), (4, 128, 128, 8, 2, 1), ()])
def test_a_shape_of_another_length_is_a_value_error(shape):
    for call in (moe.moe_check_shape, moe.moe_check_shape_int8, moe.moe_forward_workspace_bytes):
        with pytest.raises(ValueError):
            call(shape)
