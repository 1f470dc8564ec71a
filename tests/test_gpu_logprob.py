"""GPU parity of the log probabilities of given tokens, entropy and top alternatives, and of their gradient, with the
float64 oracle.

Tolerances, from the arithmetic: x = scale logit, the maximum m and d = x - m are rounded once each to 24 bits (2^-24 of |x|,
|m|, |d|); an exponential of d is off by 2^-22 and by 2^-23 |d| relative to itself, which weighted by the probabilities is at
most 2^-22 (1 + H + ln z) of a sum; sums of positive terms run through fewer than 2^8 additions (at most 128 in a
thread, a tree of 6, 8 waves, a tree of 6 parts): 2^-16 of them.  So ln z is off by 2^-16 + 2^-22 (1 + H + ln z), the mean of d likewise times
its size.  Gradients: a probability is off by 2^-22 + 2^-23 (|x| + |m| + 2 |d|) of itself, the factor beside it by 2^-22 of
what it adds, and the result is rounded to its type."""
import math

import numpy as np
import pytest
import torch

import bit_nf4_quantized_11_amd as Q
from helpers import host, log, require_gpu
from oracle import rows as oracle

pytestmark = pytest.mark.gpu

# rows, vocab, dtype, scale, top, masked, pad: one part and many, every number of loads, rows that start anywhere
CASES = [
    (1, 1, "bf16", 1.0, 1, False, 0),
    (3, 7, "fp32", 1.0, 7, False, 0),
    (2, 63, "bf16", 0.5, 32, True, 1),
    (5, 1000, "fp32", 1.25, 5, True, 3),
    (130, 4096, "bf16", 1.0, 20, False, 0),
    (129, 4097, "bf16", 1.0, 1, False, 0),
    (1, 32000, "bf16", 0.7, 20, False, 0),
    (4, 32001, "fp32", 1.0, 32, True, 0),
    (128, 32768, "bf16", 1.0, 3, False, 8),
    (128, 32769, "fp32", 2.0, 32, True, 5),
    (140, 50001, "bf16", 1.0, 0, True, 0),
    (2, 131073, "bf16", 1.0, 20, False, 7),
    (130, 70001, "fp32", 0.8, 4, False, 0),
    (1, 1 << 20, "bf16", 1.0, 32, False, 0),
    (600, 333, "bf16", 1.0, 0, False, 1),
]


def _make(case, seed=0):
    n, v, dtype, scale, top, masked, pad = case
    gen = torch.Generator().manual_seed(seed + n + v)
    x = torch.randn((n, v + pad), generator=gen) * 3
    token = torch.randint(0, v, (n,), generator=gen)
    if masked:
        hidden = torch.rand(x.shape, generator=gen) < 0.4
        hidden[torch.arange(n)[1:], token[1:]] = False
        if n > 2:
            hidden[n // 2] = True
        x = x.masked_fill(hidden, -math.inf)
    if n > 3:
        token[3] = -100
    x = x.to(torch.bfloat16 if dtype == "bf16" else torch.float32).cuda()[:, :v]
    return x, token.cuda()


def _f64(x):
    return x.double().cpu().numpy()


def _s(scale):
    return float(np.float32(scale))


@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward(case):
    require_gpu()
    log("logprob", case)
    n, v, dtype, scale, top, masked, pad = case
    x, token = _make(case)
    lp, stats, ent, tlp, tix = Q.qlora_token_logprob(x, token, scale, entropy=True, top=top)
    want = oracle.token_logprob(_f64(x), token.cpu().numpy(), _s(scale), top)
    w_lp, m, z, w_ent, w_tlp, w_tix = want
    with np.errstate(invalid="ignore", divide="ignore"):
        lnz = np.where(z > 0, np.log(z), 0)
        off_z = 2.0 ** -16 + 2.0 ** -22 * (1 + w_ent + lnz)
    same = lambda got, ref: np.array_equal(got[~np.isfinite(ref)], ref[~np.isfinite(ref)], equal_nan=True)

    def near(got, ref, tol):
        got = host(got).astype(np.float64)
        f = np.isfinite(ref)
        assert same(got, ref) and np.all(np.abs(got - ref)[f] <= np.broadcast_to(tol, ref.shape)[f])

    fin = np.where(np.isfinite(m), np.abs(m), 0)
    near(stats[:, 0], m, 2.0 ** -24 * fin)
    near(stats[:, 1], z, z * (off_z + 2.0 ** -23 * fin))
    # x_t = m + logprob + ln z: the rounding of x, m and d
    around = lambda l: off_z.reshape(-1, *[1] * (l.ndim - 1)) + 2.0 ** -22 * (
        (fin + lnz).reshape(-1, *[1] * (l.ndim - 1)) + np.abs(np.where(np.isfinite(l), l, 0)))
    near(lp, w_lp, around(w_lp))
    near(ent, w_ent, off_z + 2.0 ** -15 * (w_ent + lnz) + 2.0 ** -22 * fin)
    if top:
        assert np.array_equal(host(tix), w_tix)
        near(tlp, w_tlp, around(w_tlp))
    else:
        assert tlp is None and tix is None
    # fewer outputs: the same bits
    a = Q.qlora_token_logprob(x, token, scale)
    assert torch.equal(a[0], lp) and torch.equal(a[1], stats) and a[2] is None
    b = Q.qlora_token_logprob(x, None, scale, entropy=True, top=top)
    assert b[0] is None and torch.equal(b[2], ent) and (not top or torch.equal(b[3], tlp))


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("form", ["logprob", "entropy", "both"])
def test_backward(case, form):
    require_gpu()
    log("logprob_bwd", case, form)
    n, v, dtype, scale, top, masked, pad = case
    x, token = _make(case, 7)
    gen = torch.Generator().manual_seed(n)
    dlp = torch.randn(n, generator=gen).cuda() if form != "entropy" else None
    dent = torch.randn(n, generator=gen).cuda() if form != "logprob" else None
    _, stats, ent, _, _ = Q.qlora_token_logprob(x, token, scale, entropy=True)
    got = Q.qlora_token_logprob_bwd(x, token, stats, dlp, ent, dent, scale)
    assert got.dtype == x.dtype and got.shape == x.shape
    xs = _f64(x) * _s(scale)
    f = lambda t: None if t is None else t.double().cpu().numpy()
    want = oracle.token_logprob_bwd(_f64(x), token.cpu().numpy(), _s(scale), f(dlp), f(dent))
    lp, m, z = oracle.log_softmax(xs)
    live = np.isfinite(lp)
    p = np.where(live, np.exp(np.where(live, lp, 0)), 0)
    H = -(p * np.where(live, lp, 0)).sum(-1, keepdims=True)
    a1 = np.zeros(n) if dlp is None else np.abs(f(dlp))
    a2 = np.zeros(n) if dent is None else np.abs(f(dent))
    mm = np.where(np.isfinite(m), np.abs(m), 0)[:, None]
    xx, ll = np.where(live, np.abs(xs), 0), np.where(live, np.abs(lp), 0)
    lnz = np.log(np.maximum(z, 1))[:, None]
    # z and the entropy come from the forward, with its errors
    off_z = 2.0 ** -16 + 2.0 ** -22 * (1 + H + lnz)
    off_p = p * (2.0 ** -22 + 2.0 ** -23 * (xx + mm + 2 * ll + 2 * lnz) + off_z)
    off_H = off_z + 2.0 ** -15 * (H + lnz) + 2.0 ** -22 * mm
    off = off_p * (a1[:, None] + a2[:, None] * (ll + H)) * 1.1
    off += p * a2[:, None] * (off_H + off_z + 2.0 ** -22 * (ll + H + lnz + xx + mm)) + 2.0 ** -23 * a1[:, None] * p
    off[np.arange(n), np.clip(token.cpu().numpy(), 0, v - 1)] += 2.0 ** -23 * a1
    step = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -23
    d = np.abs(f(got) - want)
    assert np.all(d <= _s(scale) * off * (1 + step) + step * np.abs(want) + 2.0 ** -126)
    # over the logits themselves, and into rows of a wider buffer: the same bits
    wide = torch.full((n, v + 3), 7.0, dtype=x.dtype, device="cuda")
    Q.qlora_token_logprob_bwd(x, token, stats, dlp, ent, dent, scale, out=wide[:, :v])
    assert torch.equal(wide[:, :v], got) and torch.all(wide[:, v:] == 7)
    y = x.clone()
    assert Q.qlora_token_logprob_bwd(y, token, stats, dlp, ent, dent, scale, out=y) is y and torch.equal(y, got)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("n,v", [(3, 5000), (140, 5000), (2, 40000), (130, 40000)])
def test_top_with_ties_and_nothing(dtype, n, v):
    """Equal logits in numbers past any list, both zeros, rows of one value, of -infinity, and with the large ones in one
    thread's loads: the lower index first."""
    require_gpu()
    gen = torch.Generator().manual_seed(v)
    rows = [torch.zeros(v), torch.full((v,), -math.inf), torch.randint(0, 3, (v,), generator=gen).float(),
            torch.where(torch.rand(v, generator=gen) < 0.5, 0.0, -0.0), torch.arange(v).float(), -torch.arange(v).float(),
            torch.full((v,), -math.inf).index_fill(0, torch.tensor([17, v - 1, 4000]), 2.0),
            torch.randn(v, generator=gen).index_add(0, torch.arange(1000, 1040), torch.full((40,), 30.0))]
    x = torch.stack([rows[i % len(rows)] for i in range(n)]).to(dtype).cuda()
    for k in (1, 20, 32):
        _, stats, ent, tlp, tix = Q.qlora_token_logprob(x, None, entropy=True, top=k)
        order = torch.sort(x.float().cpu(), dim=1, descending=True, stable=True)[1][:, :k]
        assert torch.equal(tix.cpu(), order)
        lp = oracle.log_softmax(_f64(x))[0]
        ref = np.take_along_axis(lp, order.numpy(), 1)
        got = host(tlp).astype(np.float64)
        f = np.isfinite(ref)
        assert np.array_equal(got[~f], ref[~f])
        # (logits up to v in size are exact here; ln z as above)
        assert np.all(np.abs(got - ref)[f] <= (2.0 ** -15 + 2.0 ** -22 * (16 + np.abs(ref)))[f])


def test_nan_infinity_and_wrong_tokens():
    require_gpu()
    for v in (700, 50000):
        for dtype in (torch.bfloat16, torch.float32):
            x = torch.randn(6, v, generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
            x[1, 5] = math.nan
            x[2, 9] = math.inf
            x[4, v - 1] = -math.nan
            x[4, 11] = math.nan
            token = torch.tensor([3, 3, 3, v, 3, -1], device="cuda")
            lp, stats, ent, tlp, tix = Q.qlora_token_logprob(x, token, entropy=True, top=4)
            assert lp[[1, 2, 3, 4]].isnan().all() and lp[0].isfinite() and lp[5] == 0
            assert ent[[1, 2, 4]].isnan().all() and ent[[0, 3, 5]].isfinite().all()
            want = torch.sort(torch.where(x.float().isnan(), math.inf, x.float()), dim=1, descending=True, stable=True)[1][:, :4]
            assert torch.equal(tix, want) and tlp[[1, 4]].isnan().all() and tlp[[0, 3, 5]].isfinite().all()
            g = Q.qlora_token_logprob_bwd(x, token, stats, torch.ones(6, device="cuda"))
            assert g[[1, 3, 4]].isnan().all() and torch.all(g[5] == 0) and g[0].isfinite().all() and g[2, 9].isnan()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
def test_masks_of_the_lowest_value_and_infinite_products(dtype):
    """A mask of the type's lowest number: beside other logits it has probability 0; a whole row of it is uniform, and with
    a scale that makes it -infinity in fp32 a row of nothing.  A logit whose product is +infinity makes its row NaN."""
    require_gpu()
    low = torch.finfo(dtype).min
    for n, v in ((4, 100), (4, 40000), (200, 20000)):
        x = torch.randn(n, v, generator=torch.Generator().manual_seed(v)).to(dtype)
        x[0] = low
        x[1, ::2] = low
        x[2, 7] = -low
        x = x.cuda()
        token = torch.full((n,), 1, device="cuda")
        lp, stats, ent, tlp, tix = Q.qlora_token_logprob(x, token, entropy=True, top=3)
        assert abs(lp[0].item() + math.log(v)) < 1e-4 and abs(ent[0].item() - math.log(v)) < 1e-4 and stats[0, 1] == v
        assert tix[0].tolist() == [0, 1, 2] and tix[2, 0] == 7
        want = oracle.token_logprob(_f64(x[1:2])[:, 1::2], np.array([0]), 1.0, 0)
        assert abs(lp[1].item() - want[0][0]) < 1e-4 and abs(ent[1].item() - want[3][0]) < 1e-3
        assert lp[2] == -math.inf or lp[2].item() < -1e38       # (the given token beside one that is everything)
        g = Q.qlora_token_logprob_bwd(x, token, stats, torch.ones(n, device="cuda"), ent, torch.ones(n, device="cuda"))
        assert g[[0, 1]].isfinite().all() and torch.all(g[1, ::2] == 0)
        lp, stats, ent, tlp, tix = Q.qlora_token_logprob(x, token, 2.0, entropy=True, top=3)
        assert lp[0] == -math.inf and ent[0] == 0 and stats[0, 0] == -math.inf and stats[0, 1] == 0 and torch.all(tlp[0] == -math.inf)
        assert lp[1].isfinite() and lp[2].isnan() and ent[2].isnan()
        g = Q.qlora_token_logprob_bwd(x, token, stats, torch.ones(n, device="cuda"), ent, torch.ones(n, device="cuda"), 2.0)
        assert torch.all(g[0] == 0) and g[1].isfinite().all() and g[2].isnan().any()


def test_rows_past_32_bit_offsets():
    """Rows 2^31 + 40 elements apart: the last one lies 8.6 GB behind the first."""
    require_gpu()
    v, stride = 3000, (1 << 31) + 40
    buf = torch.zeros(2 * stride + v, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((3, v), (stride, 1))
    small = torch.randn(3, v, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    x.copy_(small)
    token = torch.tensor([0, 5, v - 1], device="cuda")
    a, b = Q.qlora_token_logprob(x, token, entropy=True, top=4), Q.qlora_token_logprob(small, token, entropy=True, top=4)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    d = torch.randn(3, device="cuda")
    want = Q.qlora_token_logprob_bwd(small, token, b[1], d)
    assert Q.qlora_token_logprob_bwd(x, token, b[1], d, out=x) is x and torch.equal(x, want)
    assert buf[v:stride].abs().max() == 0 and buf[stride + v:2 * stride].abs().max() == 0


def test_difference():
    """The gradient against differences of the forward: float32 logits, a step of 2^-7 along a random direction; the values
    are exact to 2^-16 (module's head), so the quotient to 2^-8 per row, and the curvature adds 2^-13."""
    require_gpu()
    n, v = 8, 1000
    gen = torch.Generator().manual_seed(3)
    x, d = torch.randn(n, v, generator=gen).cuda(), torch.randn(n, v, generator=gen).cuda()
    token = torch.randint(0, v, (n,), generator=gen).cuda()
    _, stats, ent, _, _ = Q.qlora_token_logprob(x, token, entropy=True)
    ones = torch.ones(n, device="cuda")
    up, down = (Q.qlora_token_logprob(x + s * 2.0 ** -7 * d, token, entropy=True) for s in (1, -1))
    for args, i in (((ones, None, None), 0), ((None, ent, ones), 2)):
        g = Q.qlora_token_logprob_bwd(x, token, stats, *args)
        assert torch.all(((up[i] - down[i]) * 2.0 ** 6 - (g * d).sum(1)).abs() <= 2.0 ** -7 + 2.0 ** -12)


def test_no_rows_strides_captured_and_other_streams():
    require_gpu()
    e = torch.empty(0, 10, device="cuda")
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    lp, stats, _, tlp, tix = Q.qlora_token_logprob(e, none, top=3)
    assert lp.shape == (0,) and stats.shape == (0, 2) and tlp.shape == tix.shape == (0, 3)
    assert Q.qlora_token_logprob_bwd(e, none, stats, lp).shape == (0, 10)
    one = torch.randn(1, 777, device="cuda").bfloat16().expand(9, 777)   # rows that are one and the same
    token = torch.arange(9, device="cuda")
    a, b = Q.qlora_token_logprob(one, token, top=5), Q.qlora_token_logprob(one.contiguous(), token, top=5)
    assert all(torch.equal(x, y) for x, y in zip(a, b) if x is not None)
    assert torch.equal(Q.qlora_token_logprob_bwd(one, token, a[1], torch.ones(9, device="cuda")),
                       Q.qlora_token_logprob_bwd(one.contiguous(), token, a[1], torch.ones(9, device="cuda")))
    for n, v in ((5, 40001), (200, 3000)):
        x, token = torch.randn(n, v, device="cuda"), torch.randint(0, v, (n,), device="cuda")
        dlp, dent = torch.randn(n, device="cuda"), torch.randn(n, device="cuda")
        ws = torch.empty(Q.qlora_token_logprob_workspace(n, v, 8), dtype=torch.uint8, device="cuda")

        def run():
            out = Q.qlora_token_logprob(x, token, 0.9, entropy=True, top=8, workspace=ws)
            return (*out, Q.qlora_token_logprob_bwd(x, token, out[1], dlp, out[2], dent, 0.9))

        run()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            captured = run()
        for k in range(3):
            x.copy_(torch.randn(n, v, device="cuda"))
            token.copy_(torch.randint(0, v, (n,), device="cuda"))
            eager = [t.clone() for t in run()]
            ws.fill_(0xFF)
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(p, q) for p, q in zip(captured, eager))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        out = Q.qlora_token_logprob(x, token, 0.9, entropy=True, top=8, stream=side)
        g = Q.qlora_token_logprob_bwd(x, token, out[1], dlp, out[2], dent, 0.9, stream=side)
        side.synchronize()
        assert all(torch.equal(p, q) for p, q in zip((*out, g), eager))


def test_binding_refusals():
    require_gpu()
    x = torch.zeros(4, 50, device="cuda")
    t = torch.zeros(4, dtype=torch.int64, device="cuda")
    s, d = torch.ones(4, 2, device="cuda"), torch.ones(4, device="cuda")
    for bad in (x.double(), x.half(), x.cpu(), x[0], x[:, ::2], x.t()):
        with pytest.raises(Q.QLoRAError):
            Q.qlora_token_logprob(bad, t)
        with pytest.raises(Q.QLoRAError):
            Q.qlora_token_logprob_bwd(bad, t, s, d)
    for bad in (t.int(), t[:3], t.cpu(), t[:, None]):
        with pytest.raises(Q.QLoRAError):
            Q.qlora_token_logprob(x, bad)
    for kw in ({"top": 33}, {"top": -1}, {"top": 51}, {"scale": 0.0}, {"scale": float("nan")}):
        with pytest.raises(Q.QLoRAError):
            Q.qlora_token_logprob(x, t, **kw)
    for args in ((None, s, d), (t, s[:3], d), (t, s.double(), d), (t, s, d[:3]), (t, s, None), (t, s, None, None, d),
                 (t, s, d, d[:2], d)):
        with pytest.raises(Q.QLoRAError):
            Q.qlora_token_logprob_bwd(x, *args)
    for out in (x.bfloat16(), x[:3], x.cpu(), torch.zeros(4, 100, device="cuda")[:, ::2], torch.zeros(1, 50, device="cuda").expand(4, 50)):
        with pytest.raises(Q.QLoRAError):
            Q.qlora_token_logprob_bwd(x, t, s, d, out=out)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("n,v", [(6, 700), (6, 3000), (6, 9000), (6, 32001), (140, 20000), (6, 150000)])
def test_top_wherever_the_large_ones_lie(dtype, n, v):
    """Rows whose large logits lie together, in one thread's elements, spread over all waves, at the row's end, or fewer than the
    alternatives above equal ones: the first of a stable sort in descending order."""
    require_gpu()
    gen = torch.Generator().manual_seed(v)
    x = torch.randn(n, v, generator=gen)
    k = 32
    x[0, 8:8 + 100] += 10                                    # neighbouring threads of one wave
    x[1, ::8192 if v > 8192 else 64] += 10                   # one thread, or one of each wave
    x[2, v - 40:] = 5 + torch.arange(40) % 7 / 8             # the end, with equal ones
    x[3, torch.randperm(v, generator=gen)[:k]] = 9.0         # k equal ones and no others
    x[4] = x[4].clamp(max=0.0)                               # half of them equal
    x[4, torch.randperm(v, generator=gen)[:5]] = 3.0
    x[5] = -torch.arange(v) // 3 / 16.0
    x = x.to(dtype)
    want = torch.sort(x.double(), dim=1, descending=True, stable=True)[1][:, :k]
    token = torch.zeros(n, dtype=torch.int64, device="cuda")
    for top in (1, 7, k):
        _, _, _, tlp, tix = Q.qlora_token_logprob(x.cuda(), token, top=top)
        assert torch.equal(tix.cpu(), want[:, :top]), top
        exact = torch.log_softmax(x.double(), 1).gather(1, want[:, :top])
        # (the distance from the largest logit is exact to 2^-24 of it, the sum's logarithm to 2^-18)
        assert torch.all((tlp.double().cpu() - exact).abs() <= 2.0 ** -18 + 2.0 ** -22 * (16 + exact.abs()))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("v", [40, 300, 5000, 32001, 150000])
def test_top_of_rows_with_few_tokens_left(dtype, v):
    """Masks that leave fewer tokens than the alternatives, as many, a few more, or tokens in the first places of the row
    only: the allowed ones by their logits, then those of -infinity by their index."""
    require_gpu()
    gen = torch.Generator().manual_seed(v)
    counts = (0, 1, 3, 19, 20, 21, 31, 32, 33, 36)
    for n in (len(counts), 130):
        x = torch.full((n, v), -math.inf)
        for i in range(n):
            k = counts[i % len(counts)]
            at = torch.randperm(v, generator=gen)[:k] if i % 3 else torch.randperm(min(v, 40), generator=gen)[:k]
            x[i, at] = torch.randn(len(at), generator=gen)
        x = x.to(dtype)
        want = torch.sort(x.double(), dim=1, descending=True, stable=True)[1]
        token = torch.zeros(n, dtype=torch.int64, device="cuda")
        for top in (1, 20, 32):
            _, _, _, tlp, tix = Q.qlora_token_logprob(x.cuda(), token, top=top)
            assert torch.equal(tix.cpu(), want[:, :top]), (n, top)
            exact = torch.log_softmax(x.double(), 1).gather(1, want[:, :top])
            exact[torch.isinf(x).all(1)] = -math.inf
            got = tlp.double().cpu()
            assert torch.equal(torch.isinf(got), torch.isinf(exact))
            assert torch.all(((got - exact).abs() <= 2.0 ** -18 + 2.0 ** -22 * (16 + exact.abs())) | torch.isinf(exact))
