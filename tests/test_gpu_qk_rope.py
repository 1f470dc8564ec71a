"""GPU parity of the head norm and rotation and of its backward with the float64 oracle.

Tolerances, from the arithmetic: the result is rounded once to bf16 (half a step: 2^-8 of the value);
before that it is a handful of fp32 operations (2^-24 each) on sine and cosine, whose argument is exact
to 2^-25 revolutions (2^-22.3 radians) and which the sine instruction gives to better than 2^-20: in all at
most 2^-18 of the magnitudes that are added, |a| + |b| of the pair (and, in the backward, the mean term).
Weight gradients are fp32 sums of N terms that carry such an error each, added in a tree whose longest
chain is below 2^9 additions: 2^-15 of the sum of magnitudes."""
import numpy as np
import pytest
import torch

import bit_nf4_quantized_11_amd as Q
from helpers import dev_bf16, host, log, require_gpu
from kv_cases import bits
from oracle import kv

pytestmark = pytest.mark.gpu

BF16, FP32 = 2.0 ** -8, 2.0 ** -18

# rows, q heads, k heads, dim, rot, norm of q, norm of k, interleaved, far
CASES = [
    (1, 1, 1, 64, 64, False, False, False, 10),
    (1, 64, 8, 128, 128, True, True, False, 4096),
    (3, 5, 0, 128, 64, True, False, False, 1 << 26),
    (7, 3, 2, 64, 32, False, True, True, 1000),
    (33, 9, 3, 256, 256, True, True, True, 1000000),
    (130, 32, 1, 128, 16, True, True, False, 100),
    (17, 4, 4, 256, 0, True, True, False, 1),
    (2100, 2, 1, 64, 48, True, True, False, 131072),
]


def _inputs(case, seed=0):
    rows, hq, hk, dim, rot, nq, nk, inter, far = case
    rng = np.random.default_rng(seed + rows + dim)
    x = {"q": bits(seed + 1, (rows, hq, dim), 1.5), "k": bits(seed + 2, (rows, hk, dim), 1.5) if hk else None}
    w = {"q": bits(seed + 3, (dim,), 1.0) if nq else None, "k": bits(seed + 4, (dim,), 1.0) if nk and hk else None}
    pos = rng.integers(-far if far > 10 else 0, far, rows)
    half = rot // 2
    freq = (10000.0 ** (-np.arange(half) / max(half, 1))).astype(np.float32)
    return x, w, pos, freq


def _dev(u16):
    return None if u16 is None else dev_bf16(u16)


def _pair_sum(mag, rot, inter):
    """|a| + |b| of each element's pair."""
    out = mag.copy()
    half = rot // 2
    if inter:
        s = mag[..., 0:rot:2] + mag[..., 1:rot:2]
        out[..., 0:rot:2], out[..., 1:rot:2] = s, s
    else:
        s = mag[..., :half] + mag[..., half:rot]
        out[..., :half], out[..., half:rot] = s, s
    return out


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("eps", [1e-6])
def test_forward(case, eps):
    require_gpu()
    log("qk forward", case)
    rows, hq, hk, dim, rot, nq, nk, inter, far = case
    x, w, pos, freq = _inputs(case)
    q, k = Q.qlora_qk_norm_rope(_dev(x["q"]), _dev(x["k"]), torch.from_numpy(pos).cuda() if rot else None,
                                torch.from_numpy(freq).cuda() if rot else None, _dev(w["q"]), _dev(w["k"]), eps, inter)
    assert (k is None) == (hk == 0)
    for t, got in (("q", q), ("k", k)):
        if got is None:
            continue
        xf, wf = kv.f64(x[t]), None if w[t] is None else kv.f64(w[t])
        want = kv.norm_rope(xf, wf, pos, freq, eps, inter)
        before = np.abs(kv.norm_rope(xf, wf, pos * 0, freq, eps, inter))   # not rotated
        d = np.abs(host(got.float()).astype(np.float64) - want)
        assert np.all(d <= BF16 * np.abs(want) + FP32 * _pair_sum(before, rot, inter)), (t, d.max())


@pytest.mark.parametrize("case", CASES, ids=str)
def test_backward(case):
    require_gpu()
    log("qk backward", case)
    rows, hq, hk, dim, rot, nq, nk, inter, far = case
    eps = 1e-5
    x, w, pos, freq = _inputs(case, 100)
    dy = {"q": bits(7, (rows, hq, dim)), "k": bits(8, (rows, hk, dim)) if hk else None}
    got = Q.qlora_qk_norm_rope_bwd(_dev(dy["q"]), _dev(dy["k"]), _dev(x["q"]), _dev(x["k"]),
                                   torch.from_numpy(pos).cuda() if rot else None,
                                   torch.from_numpy(freq).cuda() if rot else None, _dev(w["q"]), _dev(w["k"]), eps, inter)
    for t, dx, dw in (("q", got[0], got[2]), ("k", got[1], got[3])):
        assert (dw is None) == (w[t] is None)
        if dy[t] is None:
            assert dx is None
            continue
        xf, wf, df = kv.f64(x[t]), None if w[t] is None else kv.f64(w[t]), kv.f64(dy[t])
        want, want_w = kv.norm_rope_bwd(df, xf, wf, pos, freq, eps, inter)
        mag = _pair_sum(np.abs(df), rot, inter)
        if wf is not None:
            r = 1 / np.sqrt((xf * xf).mean(-1, keepdims=True) + eps)
            gmag = mag
            mag = r * (np.abs(wf) * mag + np.abs(xf) * r * r * (np.abs(wf) * mag * np.abs(xf)).mean(-1, keepdims=True))
            dwm = (gmag * np.abs(xf) * r).sum((0, 1))
            assert np.all(np.abs(host(dw).astype(np.float64) - want_w) <= 2.0 ** -15 * dwm)
        d = np.abs(host(dx.float()).astype(np.float64) - want)
        assert np.all(d <= BF16 * np.abs(want) + FP32 * mag), (t, d.max())


def test_strided_views_in_place_and_repeated():
    """q and k as slices of one projection, written over themselves; head-major outputs; broadcast gradients; and
    the same bits every time."""
    require_gpu()
    rows, hq, hk, dim = 37, 6, 2, 128
    joint = dev_bf16(bits(1, (rows, (hq + 2 * hk) * dim)))
    q, k, v = (t.unflatten(1, (-1, dim)) for t in joint.split([hq * dim, hk * dim, hk * dim], 1))
    pos = torch.arange(rows, device="cuda") * 5
    freq = torch.tensor(10000.0 ** (-np.arange(64) / 64), dtype=torch.float32, device="cuda")
    wq, wk = dev_bf16(bits(2, (dim,))), dev_bf16(bits(3, (dim,)))
    want = Q.qlora_qk_norm_rope(q.contiguous(), k.contiguous(), pos, freq, wq, wk)
    qo = torch.empty(hq, rows, dim, dtype=torch.bfloat16, device="cuda").transpose(0, 1)   # [heads][rows][dim]
    ko = torch.empty(rows, hk, dim + 8, dtype=torch.bfloat16, device="cuda")[..., :dim]
    Q.qlora_qk_norm_rope(q, k, pos, freq, wq, wk, q_out=qo, k_out=ko)
    assert torch.equal(qo, want[0]) and torch.equal(ko, want[1])
    before = v.clone()
    x, y = q.clone(), k.clone()
    Q.qlora_qk_norm_rope(q, k, pos, freq, wq, wk, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(v, before)
    one = dev_bf16(bits(4, (1, 1, dim)))
    g = (one.expand(rows, hq, dim), one.expand(rows, hk, dim))
    ref = Q.qlora_qk_norm_rope_bwd(g[0].contiguous(), g[1].contiguous(), x, y, pos, freq, wq, wk)
    for _ in range(3):
        got = Q.qlora_qk_norm_rope_bwd(*g, x, y, pos, freq, wq, wk)
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
    gq, gk = g[0].contiguous(), g[1].contiguous()
    got = Q.qlora_qk_norm_rope_bwd(gq, gk, x, y, pos, freq, wq, wk, dq=gq, dk=gk)
    assert all(torch.equal(a, b) for a, b in zip(got, ref))


def test_gradient_against_differences():
    """The backward's gradient along a direction, against the float64 forward's differences (the kernel's own
    outputs are rounded to bf16 and cannot be differenced finely)."""
    require_gpu()
    rows, hq, hk, dim, rot = 6, 3, 2, 64, 32
    case = (rows, hq, hk, dim, rot, True, True, False, 500)
    x, w, pos, freq = _inputs(case, 50)
    dy = {t: bits(9 + i, x[t].shape) for i, t in enumerate("qk")}
    got = Q.qlora_qk_norm_rope_bwd(_dev(dy["q"]), _dev(dy["k"]), _dev(x["q"]), _dev(x["k"]),
                                   torch.from_numpy(pos).cuda(), torch.from_numpy(freq).cuda(), _dev(w["q"]), _dev(w["k"]),
                                   1e-5)
    rng = np.random.default_rng(5)
    h = 1e-5
    for t, dx, dw in (("q", got[0], got[2]), ("k", got[1], got[3])):
        xf, wf, df = kv.f64(x[t]), kv.f64(w[t]), kv.f64(dy[t])
        f = lambda a, b: (kv.norm_rope(a, b, pos, freq, 1e-5) * df).sum()
        gx, gw = host(dx.float()).astype(np.float64), host(dw).astype(np.float64)
        for _ in range(5):
            d, e = rng.standard_normal(xf.shape), rng.standard_normal(wf.shape)
            num = (f(xf + h * d, wf) - f(xf - h * d, wf)) / (2 * h)
            # each of dx's elements is off by at most 2^-8 of itself (and 2^-18 of larger terms)
            assert abs(num - (gx * d).sum()) <= 1.1 * BF16 * np.abs(gx * d).sum() + 1e-6 * abs(num)
            num = (f(xf, wf + h * e) - f(xf, wf - h * e)) / (2 * h)
            assert abs(num - (gw * e).sum()) <= 2.0 ** -15 * np.abs(gw * e).sum() * 8 + 1e-6 * abs(num)


def test_no_rows_and_non_finite_heads():
    require_gpu()
    dim = 128
    e = torch.empty(0, 4, dim, dtype=torch.bfloat16, device="cuda")
    w = dev_bf16(bits(3, (dim,)))
    q, k = Q.qlora_qk_norm_rope(e, e, None, None, w, w)
    assert q.shape == e.shape
    g = Q.qlora_qk_norm_rope_bwd(e, e, e, e, None, None, w, w, dq_weight=torch.full((dim,), 7.0, device="cuda"))
    assert torch.all(g[2] == 0) and torch.all(g[3] == 0)
    # a head with an infinity touches itself alone; without a norm, itself means its pair
    x = dev_bf16(bits(4, (2, 3, dim)))
    x[0, 1, 5] = float("inf")
    pos = torch.tensor([3, 4], device="cuda")
    freq = torch.ones(16, device="cuda")
    q, _ = Q.qlora_qk_norm_rope(x, None, pos, freq)
    bad = ~torch.isfinite(q.float())
    assert bad.sum() == 2 and bad[0, 1, 5] and bad[0, 1, 21]
    q, _ = Q.qlora_qk_norm_rope(x, None, pos, freq, w)
    good = torch.isfinite(q.float()).all(-1)
    assert good.sum() == 5 and not good[0, 1]


def test_captured_forward_and_backward():
    """Both in one captured graph with the workspace passed in, replayed with other inputs, positions and eager calls
    between (which use the same workspace): the eager bits every time."""
    require_gpu()
    rows, hq, hk, dim = 300, 6, 2, 64
    t = [dev_bf16(bits(i, (rows, h, dim))) for i, h in enumerate((hq, hk, hq, hk))]
    new = [[dev_bf16(bits(10 * j + i, x.shape)) for i, x in enumerate(t)] for j in (1, 2, 3)]
    pos = torch.arange(rows, device="cuda")
    freq = torch.tensor(10000.0 ** (-np.arange(32) / 32), dtype=torch.float32, device="cuda")
    w = [dev_bf16(bits(40 + i, (dim,))) for i in range(2)]
    ws = torch.empty(Q.qlora_qk_norm_rope_bwd_workspace(rows, hq, hk, dim), dtype=torch.uint8, device="cuda")

    def run():
        return (*Q.qlora_qk_norm_rope(t[0], t[1], pos, freq, *w),
                *Q.qlora_qk_norm_rope_bwd(t[2], t[3], t[0], t[1], pos, freq, *w, workspace=ws))

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = run()
    for values in new:
        for x, y in zip(t, values):
            x.copy_(y)
        pos.add_(77)
        eager = [x.clone() for x in run()]
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(captured, eager))


def test_binding_refusals():
    """What the binding refuses before any launch."""
    require_gpu()
    x = torch.zeros(5, 3, 64, dtype=torch.bfloat16, device="cuda")
    pos, freq = torch.arange(5, device="cuda"), torch.ones(16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    for bad in (x.float(), x.cpu(), x[0], x[0, 0], x[..., ::2], torch.zeros(5, 3, 96, dtype=torch.bfloat16, device="cuda")):
        with pytest.raises(Q.QLoRAError):
            Q.qlora_qk_norm_rope(bad, None, pos, freq)
        with pytest.raises(Q.QLoRAError):
            Q.qlora_qk_norm_rope(x, None, pos, freq, q_out=bad)
        with pytest.raises(Q.QLoRAError):
            Q.qlora_qk_norm_rope_bwd(x, None, bad, None, pos, freq, w)
    for args in ((None, freq), (pos.int(), freq), (pos[:4], freq), (pos.cpu(), freq), (pos, freq.double()),
                 (pos, freq.cpu()), (pos, torch.ones(12, device="cuda")), (pos, torch.ones(40, device="cuda"))):
        with pytest.raises(Q.QLoRAError):
            Q.qlora_qk_norm_rope(x, x, *args)
    for bad in (w.float(), w[:32], w.cpu()):
        with pytest.raises(Q.QLoRAError):
            Q.qlora_qk_norm_rope(x, None, pos, freq, bad)
    for kw in ({"k_weight": w}, {"k_out": x.clone()}, {"eps": -1.0}, {"eps": float("nan")}):
        with pytest.raises(Q.QLoRAError):
            Q.qlora_qk_norm_rope(x, None, pos, freq, **kw)
    for bad in (x[:4], x[0], x[0, 0], x.cpu(), torch.zeros(5, 3, 128, dtype=torch.bfloat16, device="cuda")):
        with pytest.raises(Q.QLoRAError):
            Q.qlora_qk_norm_rope(x, bad, pos, freq)
        with pytest.raises(Q.QLoRAError):
            Q.qlora_qk_norm_rope_bwd(x, bad, None, None, pos, freq)
    for kw in ({"q_weight": w}, {"k_weight": w}, {"dk": x.clone()}, {"dq_weight": torch.zeros(64, device="cuda")},
               {"q_weight": w, "dq_weight": torch.zeros(32, device="cuda")},
               {"q_weight": w, "workspace": torch.empty(64, dtype=torch.uint8, device="cuda")}):
        q = x if "dq_weight" in kw or "workspace" in kw else None
        with pytest.raises(Q.QLoRAError):
            Q.qlora_qk_norm_rope_bwd(x, None, q, None, pos, freq, **kw)
