"""The int8 layer against float64 references: quantised rows and channels, dispatch
for many experts, the experts' products, the combine, and a run of all of them."""
import numpy as np
import pytest
import torch

import sparse_mixture_experts_05_b200 as moe

import _scored as ref

pytestmark = pytest.mark.gpu

INF = float("inf")


def _gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def _x(T, d, seed):
    return torch.randn(T, d, generator=_gen(seed), device="cuda").bfloat16()


def _idx(T, E, k, seed, skew=0.0):
    """k distinct experts a token."""
    g = _gen(seed)
    score = torch.rand(T, E, generator=g, device="cuda") + skew * torch.rand(E, generator=g, device="cuda")
    return torch.topk(score, k, dim=1).indices.to(torch.int32)


def _tricky_rows(T, d, seed):
    x = _x(T, d, seed)
    x[0] = 0.0
    if T > 1:
        x[1] = 2.0 ** -133          # subnormal bf16
    if T > 2:
        x[2] = 3.0e38
    if T > 3:                       # ties: half of the largest value
        x[3] = 1.0
        x[3, 0] = -2.0
        x[3, 1::3] = -1.0
    if T > 4:
        x[4, d // 2] = INF
    if T > 5:
        x[5, 0] = float("nan")
    if T > 6:
        x[6] = x[6] * 1e-36         # 127 / amax leaves the float range
    if T > 7:
        x[7] = torch.arange(d, device="cuda").bfloat16() * 2.0 ** -130
    return x


# ------------------------------------------------------------------ rows and channels

@pytest.mark.parametrize("T,d,E,k", [
    (1, 16, 1, 1), (9, 128, 8, 2), (130, 48, 5, 3), (33, 4096, 64, 6), (700, 272, 300, 16),
    (12, 4112, 32, 8), (20, 16400, 33, 1), (2500, 32, 512, 4), (9000, 16, 256, 8)])
def test_dispatch_and_quantised_rows(T, d, E, k):
    x = _tricky_rows(T, d, 1)
    idx = _idx(T, E, k, 2, skew=0.5)
    if T > 8:
        idx[7, 0] = -1                       # an unfilled slot
        idx[8] = E                           # outside the experts: no rows
        if k > 1:
            idx[6, 1] = idx[6, 0]            # the same expert twice
    shape = (T, d, 128, E, k)
    xq = torch.full((T * k, d), 99, dtype=torch.int8, device="cuda")
    xs = torch.full((T * k,), -5.0, device="cuda")
    offsets, perm, inv, xq, xs = moe.moe_dispatch_int8(shape, idx, x, xq=xq, xs=xs)
    r_off, r_perm, r_inv = ref.dispatch(idx, E)
    n = int(r_off[-1])
    assert np.array_equal(offsets.cpu().numpy(), r_off)
    assert np.array_equal(perm.cpu().numpy()[:n], r_perm)
    assert np.array_equal(inv.cpu().numpy(), r_inv)
    q, s = ref.quantize(x)
    rows = torch.as_tensor(r_perm, device="cuda")
    assert torch.equal(xq[:n].double(), q[rows])
    assert torch.equal(torch.nan_to_num(xs[:n], nan=-1.0), torch.nan_to_num(s[rows], nan=-1.0))
    assert torch.all(xq[n:] == 99) and torch.all(xs[n:] == -5.0)


@pytest.mark.parametrize("E,K,N", [(1, 16, 16), (3, 128, 64), (2, 272, 80), (5, 144, 400),
                                   (2, 4096, 48)])
def test_quantised_weights(E, K, N):
    W = _tricky_rows(E * N, K, 3).view(E, N, K).transpose(1, 2).contiguous()
    q, s = moe.moe_quantize_weights_int8(W)
    r_q, r_s = ref.quantize(W.transpose(1, 2))
    assert torch.equal(q.double(), r_q)
    assert torch.equal(torch.nan_to_num(s, nan=-1.0), torch.nan_to_num(r_s, nan=-1.0))


def _rows_of_ties():
    """Rows whose largest value has the significand 254 (or its half, 127): quotients by it are halves and
    quarters of the other significands, so that every odd one ties; two rows that tie at 63.5."""
    rows = []
    for p in (-130, -126, -100, -7, 0, 40, 120):
        for step in (1.0, 0.5, 0.25):
            v = torch.arange(128, 255, dtype=torch.float64) * step     # 8-bit significands
            v = torch.cat([v, -v, torch.tensor([254.0, -127.0])])
            rows.append(torch.nn.functional.pad(v, (0, 272 - v.numel())) * 2.0 ** p)
    for big in (2.0, 3.0):
        rows.append(torch.full((272,), big / 2, dtype=torch.float64))
        rows[-1][5], rows[-1][::2] = -big, -big / 2
    return torch.stack(rows).float().bfloat16().cuda()


def test_ties_between_two_8_bit_values():
    x = _rows_of_ties()
    T = x.shape[0]
    q, s = ref.quantize(x)
    f = x.double() * 127.0 / x.double().abs().amax(1, keepdim=True)
    assert int((f - f.floor() == 0.5).sum()) > 1000        # ties there are
    idx = torch.zeros(T, 1, dtype=torch.int32, device="cuda")
    for reps in (1, 80):                                   # both of the dispatch's forms
        xr = x.repeat(reps, 1)
        _, _, _, xq, xs = moe.moe_dispatch_int8((T * reps, 272, 128, 1, 1), idx.repeat(reps, 1), xr)
        assert torch.equal(xq.double(), q.repeat(reps, 1)) and torch.equal(xs, s.repeat(reps))
    W = x[:T // 16 * 16].T.contiguous()[None]
    wq, ws = moe.moe_quantize_weights_int8(W)
    assert torch.equal(wq[0].double(), q[:T // 16 * 16]) and torch.equal(ws[0], s[:T // 16 * 16])


# ------------------------------------------------------------------ products

def _check_experts(shape, idx, x, weights, seed=0):
    T, d, d_ff, E, k = shape
    offsets, perm, inv, xq, xs = moe.moe_dispatch_int8(shape, idx, x)
    o = torch.full((T * k, d), -7.0, dtype=torch.bfloat16, device="cuda")
    o, ws = moe.moe_expert_swiglu_int8(shape, xq, xs, offsets, *weights, o=o)
    assert moe.moe_read_device_status(ws) == moe.MOE_OK
    n = int(offsets[-1])
    want, tol = ref.experts(xq[:n].double(), xs[:n], offsets.cpu(), *weights)
    got = o[:n].double()
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan)
    off = torch.where(nan, 0.0, (got - want).abs() / tol)
    assert float(off.max() if off.numel() else 0) <= 1.0, float(off.max())
    assert torch.all(o[n:] == -7.0)
    return o, (offsets, xq, xs)


SHAPES = [
    (1, 128, 256, 8, 2), (1, 16, 16, 1, 1), (3, 48, 80, 4, 4), (16, 256, 512, 8, 2),
    (17, 272, 400, 5, 3), (33, 1024, 144, 64, 6), (64, 128, 128, 2, 1), (129, 144, 272, 3, 2),
    (200, 512, 1424, 16, 8), (300, 400, 336, 300, 16), (700, 256, 512, 8, 2),
    (520, 640, 768, 4, 2), (1100, 128, 256, 33, 5), (2600, 1024, 256, 8, 2), (513, 528, 528, 2, 2)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_products_against_float64(shape):
    T, d, d_ff, E, k = shape
    _check_experts(shape, _idx(T, E, k, 5, skew=1.0), _x(T, d, 6), ref.random_weights(E, d, d_ff, 7))


@pytest.mark.parametrize("T", [40, 900])
def test_products_with_missing_rows_and_experts(T):
    """Slots without an expert, experts without rows, one expert with nearly all rows,
    a token sent twice to the same expert, rows of zeros, infinities and NaN."""
    shape = (T, 256, 384, 20, 3)
    idx = _idx(T, 20, 3, 1)
    idx[:, 0] = 13
    idx[::5, 1] = -1
    idx[1::7, 2] = 13
    idx[idx == 4] = 13
    idx[9] = -1
    _check_experts(shape, idx, _tricky_rows(T, 256, 2), ref.random_weights(20, 256, 384, 3))


@pytest.mark.parametrize("T,k", [(20, 2), (600, 1)])
def test_all_slots_empty(T, k):
    shape = (T, 128, 128, 8, k)
    idx = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
    _check_experts(shape, idx, _x(T, 128, 1), ref.random_weights(8, 128, 128, 2))


@pytest.mark.parametrize("T", [5, 300])
def test_sums_past_24_bits(T):
    """All values at +-127 over K = 16384: sums of 2.6e8, past float32's integers."""
    d = 16384
    shape = (T, d, 64, 2, 1)
    W1, W3, W2 = ref.random_weights(2, d, 64, 1)
    W1[0].fill_(127)
    W3[0].fill_(-127)
    W1[1].fill_(1.0 / (127.0 * d))
    W3[1].fill_(3.0 / (127.0 * d))
    x = torch.ones(T, d, device="cuda").bfloat16()
    x[::2, ::5] = 0.75
    _check_experts(shape, _idx(T, 2, 1, 1), x, (W1, W3, W2))


@pytest.mark.parametrize("T", [400, 60000])
def test_swiglu_is_float32_exact_far_from_zero_too(T):
    """Every h within 10 2^-24 of SiLU(a) b, rounded once, for a down to -80: all 16 channels of a row
    hold one h, so its 8-bit values are +-127, and a weight of 127 scaled by
    1 / 127 brings it back as o (three float32 roundings, which bf16 does not show).  a and b
    are exact: whole sums times powers of two.  11 2^-24 allows for this test's own
    rounding by way of float32."""
    xq = torch.randint(-127, 128, (T, 16), generator=_gen(1), device="cuda").to(torch.int8)
    w1 = torch.randint(-127, 128, (16,), generator=_gen(2), device="cuda").to(torch.int8)
    w3 = torch.randint(-127, 128, (16,), generator=_gen(3), device="cuda").to(torch.int8)
    xs = torch.exp2(-torch.randint(9, 12, (T,), generator=_gen(4), device="cuda").float())
    a = (xq.double() @ w1.double()) * xs.double()
    b = (xq.double() @ w3.double()) * xs.double()
    keep = (a > -80) & (a < 80) & (b.abs() > 1.0)
    xq[~keep] = 0
    one = torch.ones(1, 16, device="cuda")
    W2 = torch.zeros(1, 16, 16, dtype=torch.int8, device="cuda")
    W2[:, :, 3] = 127
    weights = ((w1.expand(1, 16, 16).contiguous(), one), (w3.expand(1, 16, 16).contiguous(), one),
               (W2, one / 127.0))
    offsets = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    o, ws = moe.moe_expert_swiglu_int8((T, 16, 16, 1, 1), xq, xs, offsets, *weights)
    assert moe.moe_read_device_status(ws) == moe.MOE_OK
    h = torch.where(keep, a * torch.sigmoid(a) * b, 0.0)
    ends = torch.stack([(h * (1.0 + s * 11 * 2.0 ** -24)).bfloat16() for s in (-1, 1)]).double()
    got = o.double()
    assert torch.all((got >= ends.amin(0)[:, None]) & (got <= ends.amax(0)[:, None]))
    assert T < 1000 or int((keep & (a < -20)).sum()) > 5000


@pytest.mark.parametrize("T", [100, 600])
def test_swiglu_where_the_exponential_overflows(T):
    """a from -88 to -10000, where e^-a or the quotient leaves float32's range: h is 0 or next to it, never NaN."""
    xq = torch.full((T, 16), 100, dtype=torch.int8, device="cuda")
    xs = torch.linspace(88.0, 10000.0, T, device="cuda") / (16 * 100 * 100)
    W = torch.full((1, 16, 16), 100, dtype=torch.int8, device="cuda")
    one = torch.ones(1, 16, device="cuda")
    offsets = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    for up in (one, -one):
        o, _ = moe.moe_expert_swiglu_int8((T, 16, 16, 1, 1), xq, xs, offsets, (W, -one), (W, up), (W, one))
        assert torch.all(o.float().abs() <= 1e-20)
    o, _ = moe.moe_expert_swiglu_int8((T, 16, 16, 1, 1), xq, xs, offsets, (W, one), (W, one), (W, one))
    assert torch.all(torch.isfinite(o)) and torch.all(o > 0)         # SiLU(a) = a on the other side


@pytest.mark.parametrize("T", [24, 640])
def test_same_bits_whatever_else_is_in_the_batch(T):
    shape = (T, 512, 768, 8, 2)
    weights = ref.random_weights(8, 512, 768, 3)
    x, l = _x(T, 512, 1), torch.randn(T, 8, generator=_gen(2), device="cuda")
    sc = moe.MoeScoring(score="sigmoid")
    y = moe.moe_forward_int8(shape, x, l, sc, *weights)
    for _ in range(3):
        assert torch.equal(y, moe.moe_forward_int8(shape, x, l, sc, *weights))
    for t in (0, 11, T - 1):
        one = moe.moe_forward_int8((1, 512, 768, 8, 2), x[t:t + 1].clone(), l[t:t + 1].clone(), sc, *weights)
        assert torch.equal(y[t], one[0])


def test_same_bits_in_batches_of_every_size_with_softmax_gates():
    shape = (700, 256, 144, 60, 4)
    weights = ref.random_weights(60, 256, 144, 3)
    x, l = _x(700, 256, 1), torch.randn(700, 60, generator=_gen(2), device="cuda")
    sc = moe.MoeScoring(renorm=False)
    y = moe.moe_forward_int8(shape, x, l, sc, *weights)
    for T in (1, 30, 500):
        part = moe.moe_forward_int8((T, 256, 144, 60, 4), x[:T].clone(), l[:T].clone(), sc, *weights)
        assert torch.equal(part, y[:T])


@pytest.mark.parametrize("T,d,d_ff", [(16, 512, 1024), (900, 256, 512), (1000, 128, 3600)])
def test_calls_back_to_back_on_one_workspace(T, d, d_ff):
    """Up to 2048 rows, so the down product starts beside the quantisation of h: two batches in
    turn, whose row scales differ by 2^6, leave nothing of one another."""
    shape = (T, d, d_ff, 8, 2)
    weights = ref.random_weights(8, d, d_ff, 3)
    rows = []
    for s in range(2):
        idx = _idx(T, 8, 2, s)
        offsets, _, _, xq, xs = moe.moe_dispatch_int8(shape, idx, _x(T, d, s) * (1.0 if s else 64.0))
        rows.append((xq, xs, offsets))
    want = [moe.moe_expert_swiglu_int8(shape, *r, *weights)[0] for r in rows]
    ws = moe.workspace(moe.moe_expert_swiglu_int8_workspace_bytes(shape), "cuda")
    outs = [torch.empty_like(want[0]) for _ in range(40)]
    for j, o in enumerate(outs):
        moe.moe_expert_swiglu_int8(shape, *rows[j % 2], *weights, o=o, ws=ws)
    for j, o in enumerate(outs):
        assert torch.equal(o, want[j % 2])


@pytest.mark.parametrize("d,d_ff,E", [(3312, 848, 1), (944, 9184, 1), (2048, 8192, 4)])
def test_few_rows_take_no_longer_than_many(d, d_ff, E):
    """Rows below 512 may have their tiles cut along K; where that does not pay they are not: at no
    number of rows does the call take much longer than with 512 (it took up to five times as
    long for 22 rows of one expert)."""
    weights = ref.random_weights(E, d, d_ff, 3)

    def time(R):
        shape = (R, d, d_ff, E, 1)
        offsets, _, _, xq, xs = moe.moe_dispatch_int8(shape, _idx(R, E, 1, R), _x(R, d, 1))
        o, ws = moe.moe_expert_swiglu_int8(shape, xq, xs, offsets, *weights)
        best = INF
        for _ in range(12):
            begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            torch.cuda._sleep(400000)            # the calls are queued before the first begins
            begin.record()
            for _ in range(5):
                moe.moe_expert_swiglu_int8(shape, xq, xs, offsets, *weights, o=o, ws=ws)
            end.record()
            end.synchronize()
            best = min(best, begin.elapsed_time(end))
        return best
    many = time(512)
    for R in (1, 4, 22, 64, 200):
        assert time(R) < 1.4 * many, R


# ------------------------------------------------------------------ combine

@pytest.mark.parametrize("T,d,k", [(1, 16, 1), (5, 48, 2), (70, 272, 3), (300, 1024, 8), (64, 128, 16)])
def test_combine_of_bf16_outputs(T, d, k):
    o = _x(T * k, d, 1)
    inv = torch.randperm(T * k, generator=_gen(2), device="cuda").to(torch.int32).view(T, k)
    gate = torch.rand(T, k, generator=_gen(3), device="cuda")
    inv[0, 0] = -1
    if T > 3:
        inv[3] = -1                            # a token without any row
    y = moe.moe_combine_bf16((T, d, 128, 16, k), o, inv, gate)
    want = torch.zeros(T, d, device="cuda")
    for s in range(k):                         # the same float32 products and sums
        has = (inv[:, s] >= 0)[:, None]
        term = gate[:, s:s + 1] * o[inv[:, s].clamp_min(0).long()].float()
        want = torch.where(has, want + term, want)
    assert torch.equal(y, want.bfloat16())


# ------------------------------------------------------------------ all of it

LAYERS = [
    ((1, 256, 512, 8, 2), dict(score="softmax")),
    ((16, 1024, 512, 8, 2), dict(score="softmax", renorm=False)),
    ((65, 272, 400, 60, 4), dict(score="sigmoid", n_group=6, topk_group=3, group_top=2)),
    ((700, 512, 256, 128, 8), dict(score="sigmoid", n_group=8, topk_group=4, group_top=2, scale=2.5)),
    ((1025, 256, 768, 16, 3), dict(score="softmax", n_group=4, topk_group=2))]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("n", range(len(LAYERS)))
def test_layer_against_float64_and_its_steps(n, dtype):
    shape, sc = LAYERS[n]
    T, d, d_ff, E, k = shape
    W = [(0.05 * torch.randn(E, a, b, generator=_gen(40 + i), device="cuda")).bfloat16()
         for i, (a, b) in enumerate(((d, d_ff), (d, d_ff), (d_ff, d)))]
    weights = [moe.moe_quantize_weights_int8(w) for w in W]
    x = _x(T, d, 8)
    logits = torch.randn(T, E, generator=_gen(9), device="cuda").to(dtype)
    bias = 0.1 * torch.randn(E, generator=_gen(10), device="cuda") if n % 2 else None
    mask = torch.ones(T, dtype=torch.uint8, device="cuda")
    mask[T - T // 5:] = 0
    scoring = moe.MoeScoring(**sc)
    idx = torch.empty(T, k, dtype=torch.int32, device="cuda")
    gate = torch.empty(T, k, device="cuda")
    y = moe.moe_forward_int8(shape, x, logits, scoring, *weights, route_bias=bias, mask=mask,
                             idx_out=idx, gate_out=gate)
    # the steps, one by one: the same bits
    s_idx, s_gate = moe.moe_route_scored(shape, logits, scoring, bias=bias, mask=mask)
    offsets, _, inv, xq, xs = moe.moe_dispatch_int8(shape, s_idx, x)
    o, ws = moe.moe_expert_swiglu_int8(shape, xq, xs, offsets, *weights)
    assert torch.equal(idx, s_idx) and torch.equal(gate, s_gate)
    assert torch.equal(y, moe.moe_combine_bf16(shape, o, inv, s_gate))
    # routing and output in 64 bits
    r_idx, _ = ref.route(logits, k, sc, bias, mask)
    assert np.array_equal(idx.cpu().numpy(), r_idx)
    want, tol = ref.layer(x, idx, gate, *weights, E)
    assert torch.all((y.double() - want).abs() <= tol)
    assert torch.all(y[T - T // 5:] == 0)


def test_close_to_the_bf16_layer():
    """The same weights through moe_forward: 8-bit rows and channels each carry
    half a step of at most 1/127 of their largest value, about 1 % of an output's
    rms for bell-shaped data; 5 % bounds three such products."""
    T, d, d_ff, E, k = 256, 512, 1024, 8, 2
    from sparse_mixture_experts_05_b200.inputs import make_inputs
    inp = make_inputs(T, d, d_ff, E, k, 5, device="cuda")
    shape = inp["shape"]
    y = moe.moe_forward(shape, inp["x"], inp["Wg"], None, inp["W1"], inp["W3"], inp["W2"])
    _, _, logits = moe.moe_route(shape, inp["x"], inp["Wg"], want_logits=True)
    weights = [moe.moe_quantize_weights_int8(inp[n]) for n in ("W1", "W3", "W2")]
    y8 = moe.moe_forward_int8(shape, inp["x"], logits, moe.MoeScoring(), *weights)
    rel = float((y8.double() - y.double()).norm() / y.double().norm())
    assert rel <= 0.05, rel


def test_empty_batch():
    weights = ref.random_weights(8, 128, 128, 1)
    x = torch.empty(0, 128, dtype=torch.bfloat16, device="cuda")
    l = torch.empty(0, 8, device="cuda")
    y = moe.moe_forward_int8((0, 128, 128, 8, 2), x, l, moe.MoeScoring(), *weights)
    assert y.shape == (0, 128)
    idx = torch.empty(0, 2, dtype=torch.int32, device="cuda")
    offsets = moe.moe_dispatch_int8((0, 128, 128, 8, 2), idx, x)[0]
    assert torch.all(offsets == 0)
    idx = torch.empty(0, 2, dtype=torch.int32, device="cuda")
    offsets = moe.moe_dispatch_int8((0, 128, 128, 100, 2), idx, x)[0]
    assert torch.all(offsets == 0)


@pytest.mark.parametrize("T", [16, 700])
def test_layer_replays_in_a_graph_and_runs_on_two_streams(T):
    shape = (T, 256, 512, 8, 2)
    weights = ref.random_weights(8, 256, 512, 3)
    sc = moe.MoeScoring(score="sigmoid")
    nbytes = moe.moe_forward_int8_workspace_bytes(shape)
    batches = [(_x(T, 256, s), torch.randn(T, 8, generator=_gen(s), device="cuda")) for s in range(4)]
    want = [moe.moe_forward_int8(shape, x, l, sc, *weights) for x, l in batches]
    # two streams at once, each with its own workspace
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [moe.workspace(nbytes, "cuda") for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got.append(moe.moe_forward_int8(shape, *batches[i], sc, *weights, ws=spaces[i]))
    torch.cuda.synchronize()
    for j, y in enumerate(got):
        assert torch.equal(y, want[j % 2])
    # a graph, replayed on new inputs; its workspace holds an earlier call's contents
    x, l = batches[0][0].clone(), batches[0][1].clone()
    y = torch.empty_like(x)
    spaces[0].fill_(255)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_forward_int8(shape, x, l, sc, *weights, y=y, ws=spaces[0])
    for j in (2, 3):
        x.copy_(batches[j][0])
        l.copy_(batches[j][1])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[j])
        assert moe.moe_read_device_status(spaces[0]) == moe.MOE_OK


@pytest.mark.parametrize("T", [16, 700])
def test_expired_waits_are_reported_and_the_next_call_is_exact(T):
    shape = (T, 2048, 1024, 8, 2)   # several stages for every CTA
    weights = ref.random_weights(8, 2048, 1024, 3)
    idx, x = _idx(T, 8, 2, 1), _x(T, 2048, 2)
    offsets, _, _, xq, xs = moe.moe_dispatch_int8(shape, idx, x)
    want, ws = moe.moe_expert_swiglu_int8(shape, xq, xs, offsets, *weights)
    for stall in (0, 1, 3):
        moe.moe_expert_swiglu_int8_stall_test(shape, xq, xs, offsets, *weights, stall, 2_000_000, ws=ws)
        assert moe.moe_read_device_status(ws) == moe.MOE_ERR_DEVICE_TIMEOUT
    o, _ = moe.moe_expert_swiglu_int8(shape, xq, xs, offsets, *weights, ws=ws)
    assert moe.moe_read_device_status(ws) == moe.MOE_OK
    assert torch.equal(o, want)


# ------------------------------------------------------------------ borders

@pytest.mark.parametrize("T,E,k", [(1024, 8, 1), (1025, 8, 1), (128, 32, 8), (205, 32, 5), (128, 33, 8),
                                   (205, 33, 5), (64, 512, 16), (65, 512, 16), (2, 40, 16),
                                   (70, 16, 16), (200, 32, 16)])
def test_dispatch_where_the_kernels_change(T, E, k):
    """1024 slots and one more, 32 experts and one more, the most experts and slots."""
    x, idx = _x(T, 64, 1), _idx(T, E, k, 2)
    offsets, perm, inv, xq, xs = moe.moe_dispatch_int8((T, 64, 128, E, k), idx, x)
    r_off, r_perm, r_inv = ref.dispatch(idx, E)
    assert np.array_equal(offsets.cpu().numpy(), r_off)
    assert np.array_equal(perm.cpu().numpy(), r_perm)
    assert np.array_equal(inv.cpu().numpy(), r_inv)
    q, s = ref.quantize(x)
    rows = torch.as_tensor(r_perm, device="cuda")
    assert torch.equal(xq.double(), q[rows]) and torch.equal(xs, s[rows])


@pytest.mark.parametrize("shape", [(511, 192, 160, 7, 1), (256, 192, 160, 7, 2), (400, 3520, 144, 2, 2),
                                   (1600, 3520, 3520, 1, 1)], ids=str)
def test_products_where_the_plans_change(shape):
    """511 and 512 rows; K on both sides of the pairs' rule, for both products."""
    T, d, d_ff, E, k = shape
    _check_experts(shape, _idx(T, E, k, 5), _x(T, d, 6), ref.random_weights(E, d, d_ff, 7))


@pytest.mark.parametrize("T", [12, 640])
def test_a_batch_of_nothing_but_padding(T):
    shape = (T, 256, 512, 8, 2)
    weights = ref.random_weights(8, 256, 512, 3)
    ws = moe.workspace(moe.moe_forward_int8_workspace_bytes(shape), "cuda").fill_(255)
    x = torch.full((T, 256), float("nan"), device="cuda").bfloat16()
    y = moe.moe_forward_int8(shape, x, torch.full((T, 8), float("nan"), device="cuda"),
                             moe.MoeScoring(), *weights, ws=ws,
                             mask=torch.zeros(T, dtype=torch.uint8, device="cuda"))
    assert torch.all(y == 0)
    assert moe.moe_read_device_status(ws) == moe.MOE_OK


@pytest.mark.parametrize("T", [24, 700])
def test_offsets_that_do_not_ascend_stay_within_the_buffers(T):
    shape = (T, 256, 400, 8, 2)
    R = 2 * T
    weights = ref.random_weights(8, 256, 400, 3)
    idx, x = _idx(T, 8, 2, 1), _x(T, 256, 2)
    offsets, _, _, xq, xs = moe.moe_dispatch_int8(shape, idx, x)
    n = moe.moe_expert_swiglu_int8_workspace_bytes(shape)
    ws = torch.full((n + 4096,), 77, dtype=torch.uint8, device="cuda")
    o = torch.full((R + 8, 256), -7.0, dtype=torch.bfloat16, device="cuda")
    for wild in ([0, R, 0, R, 0, R, 0, R, 0], [-5, 3 * R, R // 2, -(1 << 31), (1 << 31) - 1, 0, 7, R, 1 << 30]):
        wild = torch.tensor(wild, dtype=torch.int32, device="cuda")
        moe.moe_expert_swiglu_int8(shape, xq, xs, wild, *weights, o=o[:R], ws=ws[:n])
        assert moe.moe_read_device_status(ws) == moe.MOE_OK
        assert torch.all(o[R:] == -7.0) and torch.all(ws[n:] == 77)
    want, _ = moe.moe_expert_swiglu_int8(shape, xq, xs, offsets, *weights)
    got, _ = moe.moe_expert_swiglu_int8(shape, xq, xs, offsets, *weights, ws=ws[:n])
    assert torch.equal(got, want)


def test_rows_past_32_bit_offsets():
    """Rows whose values lie past 2^31 elements and 2^32 bytes, of every tensor of the
    layer: the last tokens have the bits that they have alone."""
    T, n = 530000, 200
    shape = (T, 4096, 4096, 2, 2)
    weights = ref.random_weights(2, 4096, 4096, 3)
    x = torch.zeros(T, 4096, dtype=torch.bfloat16, device="cuda")
    x[-n:] = _x(n, 4096, 1)
    logits = torch.randn(T, 2, generator=_gen(2), device="cuda")
    sc = moe.MoeScoring(score="sigmoid", renorm=False)
    y = moe.moe_forward_int8(shape, x, logits, sc, *weights)
    one = moe.moe_forward_int8((n, 4096, 4096, 2, 2), x[-n:].clone(), logits[-n:].clone(), sc, *weights)
    assert torch.equal(y[-n:], one)
    assert not torch.any(y[:-n]) and torch.any(one != 0)


@pytest.mark.parametrize("T", [3, 300])
def test_weights_past_32_bit_offsets(T):
    """An expert whose weights begin past 2^31 bytes, against the same weights alone."""
    E, d, d_ff = 40, 4096, 14336
    last = [moe.moe_quantize_weights_int8((0.02 * torch.randn(1, a, b, generator=_gen(i), device="cuda")).bfloat16())
            for i, (a, b) in enumerate(((d, d_ff), (d, d_ff), (d_ff, d)))]
    weights = []
    for q, s in last:
        Q = torch.zeros(E, *q.shape[1:], dtype=torch.int8, device="cuda")
        S = torch.zeros(E, s.shape[1], device="cuda")
        Q[-1], S[-1] = q[0], s[0]
        weights.append((Q, S))
    x = _x(T, d, 9)
    outs = []
    for experts, w in ((E, weights), (1, last)):
        shape = (T, d, d_ff, experts, 1)
        idx = torch.full((T, 1), experts - 1, dtype=torch.int32, device="cuda")
        offsets, _, _, xq, xs = moe.moe_dispatch_int8(shape, idx, x)
        outs.append(moe.moe_expert_swiglu_int8(shape, xq, xs, offsets, *w)[0])
    assert torch.equal(*outs) and torch.any(outs[0] != 0)
    W = torch.zeros(E, d, d_ff, dtype=torch.bfloat16, device="cuda")     # 2^32 bytes and more
    W[-1] = _x(d, d_ff, 4)
    q, s = moe.moe_quantize_weights_int8(W)
    q1, s1 = moe.moe_quantize_weights_int8(W[-1:].clone())
    assert torch.equal(q[-1], q1[0]) and torch.equal(s[-1], s1[0]) and not torch.any(q[:-1])


# ------------------------------------------------------------------ how it is called

def test_memory_of_a_call_on_another_stream_is_not_handed_out_early():
    shape = (16, 256, 512, 8, 2)
    weights = ref.random_weights(8, 256, 512, 3)
    x, l = _x(16, 256, 1), torch.randn(16, 8, generator=_gen(2), device="cuda")
    sc = moe.MoeScoring()
    want = moe.moe_forward_int8(shape, x, l, sc, *weights)
    nbytes = moe.moe_forward_int8_workspace_bytes(shape)
    stream = torch.cuda.Stream()
    for _ in range(3):
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        with torch.cuda.stream(stream):
            torch.cuda._sleep(20_000_000)            # the call's kernels begin later
        y = moe.moe_forward_int8(shape, x, l, sc, *weights, stream=stream)
        junk = [moe.workspace(nbytes, "cuda").fill_(255) for _ in range(4)]
        torch.cuda.synchronize()
        assert torch.equal(y, want)
        del junk


@pytest.mark.parametrize("T", [16, 700])
def test_two_graphs_share_a_workspace(T):
    sc = moe.MoeScoring(score="sigmoid")
    shapes = [(T, 256, 512, 8, 2), (T // 2, 256, 512, 8, 2)]
    weights = ref.random_weights(8, 256, 512, 3)
    ws = moe.workspace(moe.moe_forward_int8_workspace_bytes(shapes[0]), "cuda").fill_(255)
    runs = []
    for s in shapes:
        x, l = _x(s[0], 256, s[0]), torch.randn(s[0], 8, generator=_gen(s[0]), device="cuda")
        want = moe.moe_forward_int8(s, x, l, sc, *weights)
        y = torch.empty_like(x)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            moe.moe_forward_int8(s, x, l, sc, *weights, y=y, ws=ws)
        runs.append((graph, x, l, y, want))
    for i in (0, 1, 1, 0, 1, 0, 0):
        graph, _, _, y, want = runs[i]
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)


_FIRST_CALL = """
import torch
import sparse_mixture_experts_05_b200 as moe
T, d, d_ff, E, k = shape = (%d, 256, 512, 64, 4)
g = torch.Generator("cuda").manual_seed(1)
W = [(torch.randint(-127, 128, (E, b, a), generator=g, device="cuda").to(torch.int8),
      torch.rand(E, b, generator=g, device="cuda")) for a, b in ((d, d_ff), (d, d_ff), (d_ff, d))]
x = torch.randn(T, d, generator=g, device="cuda").bfloat16()
l = torch.randn(T, E, generator=g, device="cuda")
ws = moe.workspace(moe.moe_forward_int8_workspace_bytes(shape), "cuda")
y = torch.empty_like(x)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    moe.moe_forward_int8(shape, x, l, moe.MoeScoring(), *W, y=y, ws=ws)
graph.replay()
torch.cuda.synchronize()
assert torch.equal(y, moe.moe_forward_int8(shape, x, l, moe.MoeScoring(), *W))
assert torch.any(y != 0)
"""


@pytest.mark.parametrize("T", [16, 700])
def test_a_process_may_begin_with_a_capture(T):
    import pathlib
    import subprocess
    import sys
    out = subprocess.run([sys.executable, "-c", _FIRST_CALL % T], capture_output=True, text=True, timeout=300,
                         cwd=pathlib.Path(__file__).resolve().parent.parent)
    assert out.returncode == 0, out.stderr[-2000:]
