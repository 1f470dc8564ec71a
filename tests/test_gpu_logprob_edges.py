"""Log probabilities and their gradient at the ends of their ranges: NaN in rows that have nothing else, NaN at the first
token, gradients of the entropy of any size, rows without a token, scales of any size.  (The sums of ordinary rows are in
test_gpu_logprob.py, whose tolerances are used here.)"""
import math

import numpy as np
import pytest
import torch

import bit_nf4_quantized_11_amd as Q
from helpers import log, require_gpu
from oracle import rows as oracle

pytestmark = pytest.mark.gpu

NAN, INF = math.nan, math.inf
TYPES = [torch.bfloat16, torch.float32]
# rows, vocab: a wave to a row, one part of several waves, several parts, parts of many rows
SHAPES = [(8, 40), (8, 700), (8, 9000), (8, 50000), (136, 40000)]


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("n,v", SHAPES)
def test_nan_without_a_logit(dtype, n, v):
    """A NaN makes its row NaN also where nothing else of the row is above -infinity; without one such a row is empty."""
    require_gpu()
    log("logprob nan", dtype, n, v)
    x = torch.full((n, v), -INF)
    x[0] = NAN
    x[1, v // 2] = NAN
    x[2, v - 1] = NAN
    x[3, 1:4] = -NAN
    x[5] = torch.finfo(dtype).min            # (its products with the scale are -infinity)
    x[6] = torch.finfo(dtype).min
    x[6, v // 3] = NAN
    x[7, 5] = 1.0
    x = x.to(dtype).cuda()
    token = torch.full((n,), 7, device="cuda")
    token[2] = -1
    for top in (0, 1, 20):
        lp, stats, ent, tlp, tix = Q.qlora_token_logprob(x, token, 2.0, entropy=True, top=top)
        bad, empty = [0, 1, 2, 3, 6], [4, 5]
        assert ent[bad].isnan().all() and stats[bad, 1].isnan().all()
        assert lp[[0, 1, 3, 6]].isnan().all() and lp[2] == 0
        assert torch.all(ent[empty] == 0) and torch.all(lp[empty] == -INF)
        assert torch.all(stats[empty, 0] == -INF) and torch.all(stats[empty, 1] == 0)
        assert lp[7] == -INF and ent[7] == 0 and stats[7].tolist() == [2.0, 1.0]
        if top:
            assert tlp[bad].isnan().all() and torch.all(tlp[empty] == -INF) and tlp[7, 0] == 0
            assert tix[[1, 2, 3, 6, 7], 0].tolist() == [v // 2, v - 1, 1, v // 3, 5]
    one = torch.ones(n, device="cuda")
    for args in ((one, None, None), (None, ent, one), (one, ent, one)):
        g = Q.qlora_token_logprob_bwd(x, token, stats, *args, 2.0)
        assert g[[0, 1, 3, 6]].isnan().all() and torch.all(g[empty] == 0) and g[7].isfinite().all()
        if args[2] is not None:
            assert g[2].isnan().all()


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("n,v", [(4, 1), (4, 3), (4, 32), *SHAPES])
def test_nan_at_the_first_token(dtype, n, v):
    """NaN before all else, equal ones by the lower index, from token 0 on; as many alternatives as tokens."""
    require_gpu()
    log("logprob first nan", dtype, n, v)
    x = torch.randn(n, v, generator=torch.Generator().manual_seed(v))
    x[0] = NAN
    x[1, 0] = NAN
    x[2, 0] = -NAN
    x[2, v - 1] = NAN
    x = x.to(dtype)
    key = torch.where(x.isnan(), INF, x.double())
    want = torch.sort(key, dim=1, descending=True, stable=True)[1]
    for top in {1, min(v, 3), min(v, 32)}:
        _, _, _, tlp, tix = Q.qlora_token_logprob(x.cuda(), None, top=top)
        assert torch.equal(tix.cpu(), want[:, :top]), top
        assert tlp[:3].isnan().all() and tlp[3].isfinite().all()


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("size", [1e-30, 1.0, 3e8, 1e20, 1e30, 1e37])
def test_entropy_gradients_of_any_size(dtype, size):
    """-dent p (ln p + H) and dlp (1[v] - p) where p is 0 (masked and far tokens) and where it is not."""
    require_gpu()
    log("logprob dent", dtype, size)
    n, v = 6, 3000
    gen = torch.Generator().manual_seed(1)
    x = torch.randn(n, v, generator=gen) * 2
    x[:, ::3] = -INF
    x[1, 1::3] = torch.finfo(dtype).min
    x[2, 1::3] = -1e4
    x[3] = -INF
    x = x.to(dtype)
    token = torch.tensor([1, 2, 5, 1, -1, 8])
    d1, d2 = (torch.randn(n, generator=gen) * size for _ in range(2))
    _, stats, ent, _, _ = Q.qlora_token_logprob(x.cuda(), token.cuda(), entropy=True)
    x64, f64 = x.double().numpy(), lambda t: t.double().numpy()
    lp = oracle.log_softmax(x64)[0]
    live = np.isfinite(lp)
    p, ll = np.where(live, np.exp(np.where(live, lp, 0)), 0), np.where(live, np.abs(lp), 0)
    plp = p * np.minimum(ll, 1e6)
    H = plp.sum(-1, keepdims=True)
    for a1, a2 in ((d1, d2), (None, d2), (d1, None)):
        got = Q.qlora_token_logprob_bwd(x.cuda(), token.cuda(), stats, None if a1 is None else a1.cuda(), ent,
                                        None if a2 is None else a2.cuda())
        want = oracle.token_logprob_bwd(x64, token.numpy(), 1.0, None if a1 is None else f64(a1), None if a2 is None else f64(a2))
        # logits below 16 and ln p above -2^5 where p counts: z is 2^-16 off and the entropy 2^-14 (H and ln z below 2^3), so p, and
        # what it is multiplied by, less than 2^-13 of p and of their terms; then one rounding of the type
        b1 = np.zeros((n, 1)) if a1 is None else np.abs(f64(a1))[:, None]
        b2 = np.zeros((n, 1)) if a2 is None else np.abs(f64(a2))[:, None]
        tol = 2.0 ** -13 * (p * b1 + b2 * (plp + p * (H + 1)))
        tol[np.arange(n), np.maximum(token.numpy(), 0)] += 2.0 ** -23 * b1[:, 0]
        step = torch.finfo(dtype).eps / 2
        got = got.double().cpu().numpy()
        assert np.all(np.abs(got - want) <= tol * (1 + step) + step * np.abs(want) + 2.0 ** -126)
        assert np.all(got[~live & (np.arange(v) != token.numpy()[:, None])] == 0)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("n,v", SHAPES)
def test_rows_without_a_token(dtype, n, v):
    """A row without a token has no gradient of its log probability, whatever its logits and its dlogprob are: the padding
    of a batch may hold anything."""
    require_gpu()
    log("logprob no token", dtype, n, v)
    gen = torch.Generator().manual_seed(v)
    x = torch.randn(n, v, generator=gen)
    x[1] = NAN
    x[2, 5] = INF
    x[3, v - 1] = NAN
    x[4] = -INF
    x = x.to(dtype).cuda()
    token = torch.randint(0, v, (n,), generator=gen).cuda()
    token[1:6] = -100
    lp, stats, _, _, _ = Q.qlora_token_logprob(x, token)
    assert torch.all(lp[1:6] == 0)
    d = torch.randn(n, generator=gen).cuda()
    d[2], d[5] = INF, NAN
    g = Q.qlora_token_logprob_bwd(x, token, stats, d)
    assert torch.all(g[1:6] == 0) and g[0].isfinite().all() and g[6:].isfinite().all()
    y = x.clone()
    assert torch.equal(Q.qlora_token_logprob_bwd(y, token, stats, d, out=y), g)
    # beside the entropy's gradient: that one alone
    ent = Q.qlora_token_logprob(x, token, entropy=True)[2]
    e = torch.randn(n, generator=gen).cuda()
    both, alone = (Q.qlora_token_logprob_bwd(x, token, stats, a, ent, e) for a in (d, None))
    assert torch.equal(both[4:6], alone[4:6]) and both[5].isfinite().all() and both[[1, 2, 3]].isnan().any(1).all()


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_empty_rows_have_no_gradient(dtype):
    """Also where what comes back for their log probability of -infinity is infinite or NaN; a token past the vocabulary stays NaN."""
    require_gpu()
    n, v = 6, 3000
    x = torch.full((n, v), -INF, dtype=dtype, device="cuda")
    x[1] = torch.finfo(dtype).min            # (times the scale)
    x[5, 3] = 0.0
    token = torch.tensor([0, 1, 2, -1, v, 3], device="cuda")
    _, stats, ent, _, _ = Q.qlora_token_logprob(x, token, 2.0, entropy=True)
    d, e = torch.tensor([INF, NAN, -INF, 1.0, 1.0, 1.0], device="cuda"), torch.tensor([NAN, 1.0, INF, NAN, 0.0, 1.0], device="cuda")
    for a, b in ((d, None), (None, e), (d, e)):
        g = Q.qlora_token_logprob_bwd(x, token, stats, a, ent, b, 2.0)
        assert torch.all(g[:4] == 0) and torch.all(g[5] == 0)
        assert g[4].isnan().all() if a is not None else torch.all(g[4] == 0)


# scale, logits of size: products of ordinary size from factors at the ends of fp32, sums of logits past it, products past it
SCALES = [(1.5 * 2.0 ** 127, 2.0 ** -126), (2.4e38, 0.0), (3e30, 1e-30), (1e-28, 1e28), (1e-33, 2e33), (1e-38, 3e38), (2.0 ** -127, 2e38),
          (1e-38, 1.0)]


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("n,v", [(3, 40), (3, 9000), (3, 50000), (130, 40000)])
@pytest.mark.parametrize("scale,size", SCALES)
def test_scales_of_any_size(scale, size, n, v, dtype):
    """Everything is of x = fl32(scale logit): forward and backward agree on it however large or small the factors are."""
    require_gpu()
    log("logprob scale", scale, size, n, v, dtype)
    gen = torch.Generator().manual_seed(v)
    x = ((torch.rand(n, v, generator=gen) * 2 - 1) * size).to(dtype)
    x[1, ::2] = -INF
    x[2, 1] = 0.0
    token = torch.full((n,), 1)
    s32 = np.float32(scale)
    xs = (x.float().numpy() * s32).astype(np.float64)   # rounded to fp32, as defined
    k = min(v, 8)
    lp, stats, ent, tlp, tix = Q.qlora_token_logprob(x.cuda(), token.cuda(), scale, entropy=True, top=k)
    w_lp, m, z, w_ent, _, _ = oracle.token_logprob(xs, token.numpy(), 1.0, k)
    order = torch.sort(x.double(), dim=1, descending=True, stable=True)[1][:, :k]
    w_tlp = np.take_along_axis(oracle.log_softmax(xs)[0], order.numpy(), 1)
    h = lambda t: t.double().cpu().numpy()
    # |x| at most 3: sums 2^-16 off, so logarithms 2^-15, and the entropy by twice that of the mean of d (at most 6): below 2^-12
    assert np.array_equal(h(stats[:, 0]), m) and np.all(np.abs(h(stats[:, 1]) - z) <= 2.0 ** -15 * z)
    assert np.all(np.abs(h(ent) - w_ent) <= 2.0 ** -12) and torch.equal(tix.cpu(), order)
    f = np.isfinite(w_lp)
    assert np.all(np.abs(h(lp) - w_lp)[f] <= 2.0 ** -14) and np.all(h(lp)[~f] == w_lp[~f])
    assert np.all(np.abs(h(tlp) - w_tlp) <= 2.0 ** -14)
    d1, d2 = torch.randn(n, generator=gen), torch.randn(n, generator=gen)
    g = Q.qlora_token_logprob_bwd(x.cuda(), token.cuda(), stats, d1.cuda(), ent, d2.cuda(), scale)
    want = oracle.token_logprob_bwd(xs, token.numpy(), 1.0, d1.double().numpy(), d2.double().numpy())
    p = np.exp(oracle.log_softmax(xs)[0])
    # (before the product with the scale; the factors of p are below 2^5 in all, and 2^-12 off; results of less than the least
    # normal number may be anything between 0 and it)
    tol = 2.0 ** -10 * p * (np.abs(d1.numpy()) + np.abs(d2.numpy()))[:, None]
    tol[:, 1] += 2.0 ** -22 * np.abs(d1.numpy())
    step = torch.finfo(dtype).eps / 2
    s64 = float(s32)
    with np.errstate(over="ignore"):
        big = np.abs(want) * s64 > 2.0 ** 127
        assert np.all((np.abs(h(g) - want * s64) <= 1.01 * s64 * tol + 1.01 * step * s64 * np.abs(want) + 2.0 ** -126)[~big])
