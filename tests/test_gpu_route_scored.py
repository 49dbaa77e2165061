"""Scored routing and its gradient against float64 references: score kinds, biases,
groups, top-k, renormalisation, logits that are infinite, NaN or masked, ties
closer than float32 resolves, strides past 32 bits, streams and graphs."""
import numpy as np
import pytest
import torch

import sparse_mixture_experts_05_b200 as moe

import _scored as ref

pytestmark = pytest.mark.gpu

INF = float("inf")


def _logits(T, E, seed, dtype=torch.float32):
    gen = torch.Generator("cuda").manual_seed(seed)
    return (2.0 * torch.randn(T, E, generator=gen, device="cuda")).to(dtype)


def _gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def _run(l, k, sc, bias=None, mask=None):
    T, E = l.shape
    return moe.moe_route_scored((T, 128, 128, E, k), l, moe.MoeScoring(**sc), bias=bias, mask=mask)


def _check(l, k, sc, bias=None, mask=None):
    idx, gate = _run(l, k, sc, bias, mask)
    r_idx, r_gate = ref.route(l, k, sc, bias, mask)
    assert np.array_equal(idx.cpu().numpy(), r_idx)
    g = gate.double().cpu().numpy()
    ln = l.double().cpu().numpy()
    fin = np.where(np.isfinite(ln), ln, 0.0)
    spread = (fin.max(1) - fin.min(1))[:, None]
    # gates below float32's smallest normal number are off by its spacing
    bound = np.abs(r_gate) * ref.gate_rel(spread, l.shape[1]) + 2.0 ** -140
    assert np.all(np.abs(g - r_gate) <= bound), float(np.max(np.abs(g - r_gate) / bound))
    return idx, gate


CASES = [
    # E, k, scoring
    (1, 1, dict(score="softmax")),
    (2, 2, dict(score="sigmoid", renorm=False)),
    (8, 2, dict(score="softmax")),
    (8, 2, dict(score="softmax", renorm=False, scale=0.5)),
    (16, 16, dict(score="sigmoid")),
    (31, 5, dict(score="softmax", renorm=False)),
    (32, 4, dict(score="softmax", n_group=8, topk_group=3)),
    (33, 7, dict(score="sigmoid", n_group=3, topk_group=2, group_top=2)),
    (60, 4, dict(score="softmax", n_group=6, topk_group=2, group_top=2)),
    (64, 6, dict(score="softmax", n_group=8, topk_group=3, group_top=1, scale=16.0)),
    (100, 9, dict(score="sigmoid", n_group=10, topk_group=4, group_top=2)),
    (128, 8, dict(score="sigmoid", n_group=32, topk_group=4, group_top=2)),
    (160, 6, dict(score="softmax", n_group=8, topk_group=3, renorm=False)),
    (256, 8, dict(score="sigmoid", n_group=8, topk_group=4, group_top=2, scale=2.5)),
    (257, 3, dict(score="sigmoid")),
    (300, 10, dict(score="softmax", n_group=5, topk_group=5, group_top=2)),
    (512, 16, dict(score="sigmoid", n_group=16, topk_group=2, group_top=2)),
    (512, 8, dict(score="softmax", renorm=False)),
    (16, 2, dict(score="sigmoid", n_group=16, topk_group=7)),
    (48, 3, dict(score="softmax", n_group=3, topk_group=1, group_top=2)),
    (504, 8, dict(score="sigmoid", n_group=9, topk_group=4, group_top=2)),
    (510, 12, dict(score="softmax", n_group=17, topk_group=8, group_top=2)),
    (500, 7, dict(score="sigmoid", n_group=2, topk_group=1)),
    (62, 2, dict(score="sigmoid", n_group=31, topk_group=9, group_top=2)),
    (256, 13, dict(score="softmax", n_group=8, topk_group=4)),
]


@pytest.mark.parametrize("biased", [False, True], ids=["plain", "biased"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_routing_against_float64(case, dtype, biased):
    E, k, sc = CASES[case]
    for T in (1, 67):
        l = _logits(T, E, 100 + case, dtype)
        bias = None
        if biased:
            gen = torch.Generator("cuda").manual_seed(case)
            bias = 0.3 * torch.randn(E, generator=gen, device="cuda")
        _check(l, k, sc, bias)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("grouped", [False, True])
@pytest.mark.parametrize("biased", [False, True])
def test_infinite_nan_and_lowest_logits(score, renorm, grouped, biased):
    E, k = 24, 5
    l = _logits(12, E, 7)
    lowest = torch.finfo(torch.float32).min
    l[0] = -INF                       # nothing is left
    l[1, 3:] = -INF                   # fewer experts than slots
    l[2] = lowest                     # all at the type's lowest value
    l[3, ::2] = lowest
    l[4] = float("nan")
    l[5, 1::2] = float("nan")
    l[6, :3] = INF                    # several infinities share the softmax
    l[7] = -300.0 - torch.arange(E, device="cuda")  # sigmoids below float32's range
    l[8] = 200.0
    l[9, :12] = -INF                  # whole groups gone
    l[10, 5] = INF
    l[11] = 0.0
    l[11, 4] = -0.0                   # the two zeros tie
    sc = dict(score=score, renorm=renorm, scale=1.5)
    if grouped:
        sc.update(n_group=4, topk_group=2, group_top=2)
    bias = None
    if biased:
        bias = torch.linspace(-0.2, 0.3, E, device="cuda")
        bias[20] = -INF               # an expert taken out by its bias
    idx, gate = _check(l, k, sc, bias)
    assert torch.all(idx[0] == -1) and torch.all(gate[0] == 0)
    assert torch.all(idx[4] == -1)
    if renorm and not biased:
        assert abs(float(gate[7].sum()) - 1.5) < 1e-5


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_sigmoids_below_the_smallest_normal_number(dtype):
    """Gates and gradients of logits from -80 to -104, whose sigmoids reach float32's smallest
    subnormals; sums of them in the gates are the renormalised ones' (tested above)."""
    E, k = 40, 6
    l = -(80.0 + 24.0 * torch.rand(30, E, generator=_gen(1), device="cuda")).to(dtype)
    sc = dict(score="sigmoid", renorm=False)
    idx, gate = _check(l, k, sc)
    assert torch.all(gate[l.gather(1, idx.long()) > -100] > 0)
    _check(l, k, sc, torch.linspace(-0.3, 0.3, E, device="cuda"))
    dgate = torch.randn(30, k, generator=_gen(2), device="cuda")
    got = moe.moe_route_scored_backward((30, 128, 128, E, k), l, moe.MoeScoring(**sc), idx, dgate)
    want, bound = ref.route_backward(l, idx, dgate, sc)
    step = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    # below the smallest normal number a value is off by its type's spacing, 2^-133 or 2^-149, in
    # the result and a few times 2^-149 before it
    least = 2.0 ** -133 if dtype == torch.bfloat16 else 2.0 ** -145
    assert np.all(np.abs(got.double().cpu().numpy() - want) <= bound + np.abs(want) * step + least)


@pytest.mark.parametrize("biases", [100.0, -100.0])
def test_groups_at_the_end_of_the_keys_range(biases):
    """Group 0 holds the row's largest choice; the two best of group 1 and of group 2 lie 4 below
    it, on the border of what the keys tell apart, with sums 1e-7 from each other."""
    T, ulp = 6000, 2.0 ** -17             # the spacing of float32 between 64 and 128
    u = (torch.rand(T, 2, generator=_gen(1), device="cuda", dtype=torch.float64) - 0.5) * 3e-7
    half = ulp / 2                        # biased choices round up from here
    # group 1's choices round up into the range, group 2's down out of it
    s = torch.stack([0.5 + half + u[:, 0], 0.5 - half + u[:, 1]], 1)
    logit = torch.log(s / (1.0 - s)).float()
    l = torch.zeros(T, 6, device="cuda")
    l[:, 2:4] = logit[:, :1]
    l[:, 4:6] = logit[:, 1:]
    bias = torch.tensor([biases, biases, biases - 4.0, biases - 4.0, biases - 4.0 + ulp, biases - 4.0 + ulp],
                        device="cuda")
    for top in (1, 2):
        idx, _ = _check(l, 4, dict(score="sigmoid", n_group=3, topk_group=2, group_top=top), bias)
        second = idx[:, 2] // 2
        assert 1000 < int((second == 2).sum()) < 5000


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,G,k", [(256, 8, 8), (60, 6, 4), (96, 3, 12), (16, 16, 2), (510, 17, 6)])
def test_groups_switched_off(E, G, k, score, dtype):
    """Groups at -inf, at the type's lowest value, far below the others, with one live expert, and
    rows that leave fewer live groups than stay, or none: by the logits, and by the bias."""
    w = E // G
    l = _logits(40, E, 77, dtype)
    off = _logits(40, E, 77, dtype)
    for t in range(40):
        for g in range(G):
            if (t * 7 + g * 5) % (2 + t % 4) == 0 or t in (30, 31):
                off[t, g * w:(g + 1) * w] = (-INF, torch.finfo(dtype).min, -60.0, -200.0)[t % 4]
                if t >= 20 and t != 30:
                    off[t, g * w + t % w] = l[t, g * w + t % w]
    by_bias = torch.zeros(E, device="cuda")
    by_bias[:w] = -INF
    by_bias[(G - 1) * w:] = -1e9
    for top in (1, 2):
        for kept in (1, (G + 1) // 2, G):
            if k > kept * w:
                continue
            sc = dict(score=score, n_group=G, topk_group=kept, group_top=top)
            _check(off, k, sc)
            _check(off, k, sc, torch.linspace(-0.2, 0.2, E, device="cuda"))
            _check(l, k, sc, by_bias)


def _time_route(l, sc, bias, idx, gate):
    T, E = l.shape
    best = INF
    for _ in range(12):
        begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        torch.cuda._sleep(400000)            # the calls are queued before the first begins
        begin.record()
        for _ in range(8):
            moe.moe_route_scored((T, 128, 128, E, idx.shape[1]), l, sc, bias=bias, idx=idx, gate=gate)
        end.record()
        end.synchronize()
        best = min(best, begin.elapsed_time(end))
    return best


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,G,k", [(64, 1, 6), (256, 8, 8), (60, 6, 12), (8, 1, 2), (300, 5, 16)])
def test_rows_with_fewer_live_experts_than_slots(E, G, k, score, dtype):
    """0 to 9 experts above the others, which are at -inf, far below, or both."""
    gen = _gen(E + k)
    l = _logits(80, E, 5, dtype)
    for t in range(80):
        at = torch.randperm(E, generator=gen, device="cuda")
        rest = at[min(t % 10, E):]
        l[t, rest] = (-INF, -70.0, -90.0, -INF)[t // 20]
        if t >= 60 and len(rest) > 3:
            l[t, rest[:2]] = torch.tensor([-55.0, -80.0], device="cuda").to(dtype)
    for top in (1, 2):
        sc = dict(score=score, n_group=G, topk_group=(G + 1) // 2, group_top=top)
        for renorm in (True, False):
            sc["renorm"] = renorm
            _check(l, k, sc)
            _check(l, k, sc, torch.linspace(-0.2, 0.2, E, device="cuda"))
            _check(l, k, sc, torch.linspace(-9.0, 9.0, E, device="cuda"))


@pytest.mark.parametrize("score,top,biased", [("softmax", 1, False), ("softmax", 2, False), ("sigmoid", 1, True),
                                              ("softmax", 0, False), ("sigmoid", 0, True)])
def test_groups_switched_off_cost_no_more_than_live_ones(score, top, biased):
    """16384 rows of 256 experts with and without a group at -inf: about the same time (a row that goes
    to the last attempt for its dead group made it five times as long).  The same without
    groups (top 0) and with fewer live experts than slots."""
    E, k = 256, 8
    if top == 0:
        sc = moe.MoeScoring(score=score)
        bias = 0.05 * torch.randn(E, generator=_gen(2), device="cuda") if biased else None
        l = _logits(16384, E, 1)
        off = l.clone()
        off[:, 5:] = -INF
        idx, gate = _run(off, k, dict(score=score), bias)
        assert torch.all(idx[:, :5] >= 0) and torch.all(idx[:, 5:] == -1)
        assert _time_route(off, sc, bias, idx, gate) < 2.0 * _time_route(l, sc, bias, idx, gate)
        return
    sc = moe.MoeScoring(score=score, n_group=8, topk_group=4, group_top=top)
    bias = 0.05 * torch.randn(E, generator=_gen(2), device="cuda") if biased else None
    l = _logits(16384, E, 1)
    off = l.clone()
    off[:, :32] = -INF
    idx, gate = _run(l, k, dict(score=score, n_group=8, topk_group=4, group_top=top), bias)
    assert _time_route(off, sc, bias, idx, gate) < 2.0 * _time_route(l, sc, bias, idx, gate)


def test_masked_rows_get_no_expert_whatever_they_hold():
    l = _logits(40, 64, 3)
    mask = torch.ones(40, dtype=torch.uint8, device="cuda")
    mask[30:] = 0
    mask[4] = 0
    l[30:] = float("nan")
    l[4] = INF
    idx, gate = _check(l, 6, dict(score="softmax", renorm=False), mask=mask)
    assert torch.all(idx[30:] == -1) and torch.all(gate[30:] == 0) and torch.all(idx[4] == -1)
    mask.zero_()
    idx, gate = _check(l, 6, dict(score="sigmoid"), mask=mask)
    assert torch.all(idx == -1) and torch.all(gate == 0)


@pytest.mark.parametrize("E,groups", [(64, 1), (256, 8)])
def test_choices_closer_than_float32_resolves(E, groups):
    """Sigmoids of 18 .. 34 are all 1 in float32 but distinct in float64; biased
    choices that differ by 1e-9 likewise."""
    T = 50
    gen = torch.Generator("cuda").manual_seed(5)
    steps = torch.linspace(18.0, 34.0, E, device="cuda")
    l = torch.stack([steps[torch.randperm(E, generator=gen, device="cuda")] for _ in range(T)])
    sc = dict(score="sigmoid", n_group=groups, topk_group=max(1, groups // 2), group_top=2)
    _check(l, 8, sc, torch.zeros(E, device="cuda"))
    _check(l, 8, sc)
    # s + b nearly equal for all experts: b = 1 - s rounded to float32
    l = _logits(T, E, 6)
    l[:] = l[0]
    bias = (1.0 - torch.sigmoid(l[0].double())).float()
    _check(l, 8, sc, bias)
    sc["score"] = "softmax"
    bias = (1.0 - torch.softmax(l[0].double(), 0)).float()
    _check(l, 8, sc, bias)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("scale", [1e-43, 1e-3, 30.0, 1e4])
@pytest.mark.parametrize("tops", [1, 2])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_logits_of_every_size(score, tops, scale, dtype):
    """Mostly negative logits, subnormal to huge, with groups valued by their logits or by
    sums of scores; a biased selection on the same."""
    E, groups = 128, 16
    l = ((torch.randn(60, E, generator=_gen(3), device="cuda") - 1.5) * scale).to(dtype)
    sc = dict(score=score, n_group=groups, topk_group=5, group_top=tops)
    _check(l, 6, sc)
    _check(l, 6, sc, torch.linspace(-0.3, 0.3, E, device="cuda"))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,groups", [(64, 6, 1), (64, 6, 16), (256, 8, 8), (256, 8, 1), (40, 12, 5), (24, 2, 4),
                                        (512, 16, 32), (8, 2, 1)])
@pytest.mark.parametrize("levels", [2, 9, 40])
def test_rows_with_many_nearly_equal_choices(score, E, k, groups, levels):
    """A few levels of logits, equal or a few units of the last place apart, some experts
    masked out: ties at the k-th place, between groups, and within their best two."""
    gen = torch.Generator("cuda").manual_seed(levels)
    T = 33
    level = 1.0 + torch.randn(levels, generator=gen, device="cuda")
    l = level[torch.randint(levels, (T, E), generator=gen, device="cuda")]
    l = l * (1.0 + 2.0 ** -23 * torch.randint(-2, 3, (T, E), generator=gen, device="cuda"))
    l[3, ::3] = -INF
    l[4, E // 8:] = -INF
    bias = 2.0 ** -3 * torch.randint(0, 3, (E,), generator=gen, device="cuda").float()
    for top in (1, 2):
        sc = dict(score=score, n_group=groups, topk_group=(groups + 1) // 2, group_top=top)
        for b in (None, bias, torch.zeros(E, device="cuda")):
            _check(l, k, sc, b)


# all ways to cut these numbers of experts into groups: where a group's experts do not fill its
# lanes, the places behind them count past the last expert (in 21 of these pairs past 511)
RAGGED = [(E, G) for E in (501, 504, 505, 506, 507, 510, 511, 512) for G in range(2, 33) if E % G == 0]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("E,G", RAGGED)
def test_groups_that_do_not_fill_their_lanes(E, G, dtype):
    gen = torch.Generator("cuda").manual_seed(E + G)
    bias = 0.3 * torch.randn(E, generator=gen, device="cuda")
    l = _logits(7, E, 31 * E + G, dtype)
    l[4] = -9.0                          # equal choices
    l[5, :E - 3] = -INF                  # the last group alone
    l[6, E // G:] = -INF                 # the first
    for score in ("softmax", "sigmoid"):
        for top in (1, 2):
            sc = dict(score=score, n_group=G, topk_group=(G + 1) // 2, group_top=top)
            for k in (8, 12):
                _check(l, k, sc)
                _check(l, k, sc, bias)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,G,k", [(510, 15, 8), (510, 30, 16), (511, 7, 8), (507, 3, 12), (504, 6, 2), (501, 3, 5)])
@pytest.mark.parametrize("ties", [2, 20, 40])
def test_ties_at_the_last_place_in_groups_that_do_not_fill_their_lanes(score, E, G, k, ties):
    """`ties` equal choices, spread over the groups, around the k-th place: fewer than the slots,
    a few more, and more than a warp decides at once."""
    gen = torch.Generator("cuda").manual_seed(E + ties)
    l = -2.0 - torch.rand(9, E, generator=gen, device="cuda")
    for t in range(9):
        at = torch.randperm(E, generator=gen, device="cuda")
        l[t, at[:k // 2]] = 1.0 + torch.rand(k // 2, generator=gen, device="cuda")
        l[t, at[k // 2:k // 2 + ties]] = 0.5
    for top in (1, 2):
        sc = dict(score=score, n_group=G, topk_group=G, group_top=top)
        _check(l, k, sc)
        _check(l, k, sc, torch.zeros(E, device="cuda"))


def test_equal_choices_go_to_the_lower_index():
    l = torch.zeros(3, 256, device="cuda")
    l[1, 100:] = 1.0
    l[2, ::7] = 2.0
    for sc in (dict(score="softmax"), dict(score="sigmoid", n_group=8, topk_group=4, group_top=2)):
        idx, _ = _check(l, 8, sc)
        assert idx[0].tolist() == list(range(8))
        _check(l, 8, sc, torch.full((256,), 0.25, device="cuda"))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("E,k,groups", [(33, 2, 1), (60, 4, 1), (60, 4, 6), (100, 9, 10), (160, 6, 8), (256, 8, 1),
                                        (256, 8, 8), (300, 12, 5), (500, 2, 1), (510, 8, 15), (512, 16, 16)])
def test_a_rows_bits_do_not_depend_on_the_number_of_rows(E, k, groups, dtype):
    """Few rows take 32 lanes each, many 8 or 16; the softmax's sum is the same tree."""
    l = _logits(5000, E, E, dtype)
    bias = 0.1 * torch.randn(E, generator=_gen(1), device="cuda")
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            sc = dict(score=score, renorm=renorm, n_group=groups, topk_group=(groups + 1) // 2,
                      group_top=2 if groups > 1 else 1)
            for b in (None, bias):
                idx, gate = _run(l, k, sc, b)
                for T in (1, 77, 500, 900):
                    s_idx, s_gate = _run(l[:T].clone(), k, sc, b)
                    assert torch.equal(s_idx, idx[:T])
                    assert torch.equal(s_gate, gate[:T]), (score, renorm, b is None, T)


def test_rows_past_32_bit_offsets():
    E, k = 512, 4
    T = (1 << 31) // E + 77
    l = torch.zeros(T, E, dtype=torch.bfloat16, device="cuda")
    l[-80:] = _logits(80, E, 9, torch.bfloat16)
    sc = dict(score="softmax", renorm=False)
    idx, gate = _run(l, k, sc)
    r_idx, r_gate = ref.route(l[-80:], k, sc)
    assert np.array_equal(idx[-80:].cpu().numpy(), r_idx)
    assert np.allclose(gate[-80:].cpu().numpy(), r_gate, rtol=1e-5)
    dgate = torch.ones(T, k, device="cuda")
    grad = moe.moe_route_scored_backward((T, 128, 128, E, k), l, moe.MoeScoring(**sc), idx, dgate)
    r_grad, bound = ref.route_backward(l[-80:], idx[-80:], dgate[-80:], sc)
    g = grad[-80:].double().cpu().numpy()
    assert np.all(np.abs(g - r_grad) <= bound + np.abs(r_grad) * 2.0 ** -8 + 1e-38)


# ------------------------------------------------------------------ gradient

@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_gradient_against_float64(case, dtype):
    E, k, sc = CASES[case]
    for T in (1, 67):
        l = _logits(T, E, 300 + case, dtype)
        idx, _ = _run(l, k, sc)
        gen = torch.Generator("cuda").manual_seed(case)
        dgate = torch.randn(T, k, generator=gen, device="cuda")
        if T > 1:
            idx[5] = -1                     # a masked row
            idx[6, 0] = -1                  # an unfilled slot
            dgate[5] = float("nan")         # ... whose gradient is not looked at
            dgate[6, 0] = INF
            l[5] = float("nan")
            if k > 1:
                idx[7, 1] = idx[7, 0]       # the same expert twice
            idx[8, 0] = E                   # outside the experts
        got = torch.full((T, E), 7.0, dtype=dtype, device="cuda")
        moe.moe_route_scored_backward((T, 128, 128, E, k), l, moe.MoeScoring(**sc), idx, dgate,
                                      dlogits=got)
        want, bound = ref.route_backward(l, idx, dgate, sc)
        g = got.double().cpu().numpy()
        step = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
        bound = bound + np.abs(want) * step + 2.0 ** -133
        assert np.all(np.abs(g - want) <= bound), float(np.max(np.abs(g - want) / bound))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_against_differences(score, renorm):
    """Central differences of the float64 gates, step 1e-6: truncation below
    1e-11, rounding below 1e-9, against float32's bound of about 1e-6."""
    E, k, T = 20, 4, 6
    sc = dict(score=score, renorm=renorm, scale=2.0)
    l = _logits(T, E, 11)
    idx, _ = _run(l, k, sc)
    dgate = torch.randn(T, k, generator=torch.Generator("cuda").manual_seed(1), device="cuda")
    got = moe.moe_route_scored_backward((T, 128, 128, E, k), l, moe.MoeScoring(**sc), idx, dgate)
    ln, ix, dg = l.double().cpu().numpy(), idx.cpu().numpy(), dgate.double().cpu().numpy()

    def loss(row, t):
        return 2.0 * float((ref._weights(row, ix[t], score, renorm) * dg[t]).sum())
    want = np.zeros((T, E))
    for t in range(T):
        for i in range(E):
            up, down = ln[t].copy(), ln[t].copy()
            up[i] += 1e-6
            down[i] -= 1e-6
            want[t, i] = (loss(up, t) - loss(down, t)) / 2e-6
    assert np.all(np.abs(got.cpu().numpy() - want) <= 1e-5)


def test_infinite_logits_in_the_gradient():
    l = _logits(4, 16, 2)
    l[0, 3:] = -INF
    l[1, 2] = INF
    l[2, ::2] = float("nan")
    for sc in (dict(score="softmax", renorm=False), dict(score="softmax"),
               dict(score="sigmoid"), dict(score="sigmoid", renorm=False)):
        idx, _ = _run(l, 4, sc)
        dgate = torch.ones(4, 4, device="cuda")
        dgate[:, 1] = -2.0
        got = moe.moe_route_scored_backward((4, 128, 128, 16, 4), l, moe.MoeScoring(**sc), idx, dgate)
        want, bound = ref.route_backward(l, idx, dgate, sc)
        assert np.all(np.abs(got.double().cpu().numpy() - want) <= bound + 1e-37)


# ------------------------------------------------------------------ streams, graphs, layer

def test_graph_replay_and_other_streams():
    T, E, k = 300, 256, 8
    sc = moe.MoeScoring(score="sigmoid", n_group=8, topk_group=4, group_top=2, scale=2.5)
    shape = (T, 128, 128, E, k)
    bias = 0.1 * torch.randn(E, device="cuda")
    static, dgate = _logits(T, E, 1), torch.randn(T, k, device="cuda")
    idx = torch.empty(T, k, dtype=torch.int32, device="cuda")
    gate = torch.empty(T, k, device="cuda")
    grad = torch.empty(T, E, device="cuda")

    def step(l, i, g, dl):
        moe.moe_route_scored(shape, l, sc, bias=bias, idx=i, gate=g)
        moe.moe_route_scored_backward(shape, l, sc, i, dgate, dlogits=dl)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(static, idx, gate, grad)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(static, idx, gate, grad)
    for seed in (2, 3):
        l = _logits(T, E, seed)
        static.copy_(l)
        graph.replay()
        e_idx, e_gate = moe.moe_route_scored(shape, l, sc, bias=bias)
        e_grad = moe.moe_route_scored_backward(shape, l, sc, e_idx, dgate)
        torch.cuda.synchronize()
        assert torch.equal(idx, e_idx) and torch.equal(gate, e_gate) and torch.equal(grad, e_grad)


def test_equals_the_layers_router_on_its_logits():
    """Softmax over the selected two: the same experts, gates within both kernels'
    float32 error (1e-6), as moe_route gives."""
    T, d, E, k = 257, 256, 8, 2
    gen = torch.Generator("cuda").manual_seed(4)
    x = torch.randn(T, d, generator=gen, device="cuda").bfloat16()
    Wg = (torch.randn(d, E, generator=gen, device="cuda") / 16).bfloat16()
    shape = (T, d, 256, E, k)
    idx, gate, logits = moe.moe_route(shape, x, Wg, want_logits=True)
    s_idx, s_gate = moe.moe_route_scored(shape, logits, moe.MoeScoring())
    assert torch.equal(idx, s_idx)
    assert float((gate - s_gate).abs().max()) <= 1e-6
