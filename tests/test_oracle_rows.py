"""The oracle of the residual norm, the gated block and the log probabilities: against torch's float64 functions and
autograd, and central differences."""
import numpy as np
import pytest
import torch

from oracle import rows

# float64 against float64: sums of at most a few hundred terms
TIGHT = 1e-12


def _near(a, b, tol=TIGHT):
    a, b = np.asarray(a), np.asarray(b)
    assert a.shape == b.shape and np.all(np.abs(a - b) <= tol * (1 + np.abs(b)))


def _differences(f, x, d, h=1e-6):
    """d/dx of f at x along d, by central differences (error h^2 and rounding / h)."""
    return (f(x + h * d) - f(x - h * d)) / (2 * h)


def test_bf16_matches_torch():
    x = np.concatenate([np.random.default_rng(0).standard_normal(4096).astype(np.float32) * 10.0 ** np.arange(-8, 8).repeat(256),
                        np.float32([0.0, -0.0, 1 + 2 ** -8, 1 + 3 * 2 ** -8, 1e-40])]).astype(np.float32)
    _near(rows.bf16(x), torch.from_numpy(x).bfloat16().double().numpy(), 0)


@pytest.mark.parametrize("weight", [False, True])
@pytest.mark.parametrize("dh", [False, True])
def test_rms_norm(weight, dh):
    rng = np.random.default_rng(1)
    h, dy = rng.standard_normal((5, 24)), rng.standard_normal((5, 24))
    w = rng.standard_normal(24) if weight else None
    g = rng.standard_normal((5, 24)) if dh else None
    th = torch.from_numpy(h).requires_grad_()
    tw = torch.ones(24, dtype=torch.float64) if w is None else torch.from_numpy(w)
    tw.requires_grad_()
    y = torch.nn.functional.rms_norm(th, (24,), tw, 1e-5)
    loss = (y * torch.from_numpy(dy)).sum() + (0 if g is None else (th * torch.from_numpy(g)).sum())
    gh, gw = torch.autograd.grad(loss, (th, tw))
    got, kept = rows.rms_norm(h, None, w, 1e-5)
    assert kept is h
    _near(got, y.detach().numpy())
    dx, dw = rows.rms_norm_bwd(dy, h, w, g, 1e-5)
    _near(dx, gh.numpy())
    _near(dw, gw.numpy())
    d = rng.standard_normal(h.shape)
    f = lambda v: (rows.rms_norm(v, None, w, 1e-5)[0] * dy).sum() + (0 if g is None else (v * g).sum())
    assert abs(_differences(f, h, d) - (dx * d).sum()) < 1e-6


def test_rms_norm_residual_is_rounded_once():
    x, r = rows.bf16(np.random.default_rng(2).standard_normal((3, 16))), rows.bf16(np.random.default_rng(3).standard_normal((3, 16)))
    y, h = rows.rms_norm(x, r, None, 0.0)
    _near(h, (torch.from_numpy(x).bfloat16() + torch.from_numpy(r).bfloat16()).double().numpy(), 0)
    _near((y * y).mean(-1), np.ones(3))


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_gated(kind):
    rng = np.random.default_rng(4)
    G, U, dH = (rng.standard_normal((4, 40)) * s for s in (3, 2, 1))
    tg, tu = torch.from_numpy(G).requires_grad_(), torch.from_numpy(U).requires_grad_()
    a = torch.nn.functional.silu(tg) if kind == "silu" else torch.nn.functional.gelu(tg, approximate="tanh")
    H = a * tu
    dg, du = torch.autograd.grad(H, (tg, tu), torch.from_numpy(dH))
    for got, want in zip(rows.gated_bwd(dH, G, U, kind), (dg, du, H)):
        _near(got, want.detach().numpy())
    d = rng.standard_normal(G.shape)
    f = lambda v: (rows.activation(v, kind)[0] * U * dH).sum()
    assert abs(_differences(f, G, d) - (rows.gated_bwd(dH, G, U, kind)[0] * d).sum()) < 1e-6


def test_token_logprob():
    rng = np.random.default_rng(5)
    x = rng.standard_normal((6, 50)) * 3
    x[1, ::3] = -np.inf
    x[2] = -np.inf
    x[3, 4:9] = x[3].max() + 1   # ties
    token = np.array([3, 1, 0, 8, -100, 50])
    lp, m, z, ent, tlp, tix = rows.token_logprob(x, token, 0.7, 9)
    want = torch.log_softmax(torch.from_numpy(x) * 0.7, -1).numpy()
    for i in (0, 1, 3):
        assert abs(lp[i] - want[i, token[i]]) < TIGHT * 10
        assert abs(m[i] + np.log(z[i]) - torch.logsumexp(torch.from_numpy(x[i]) * 0.7, 0).item()) < TIGHT * 10
        p = np.exp(want[i][np.isfinite(want[i])])
        assert abs(ent[i] + (p * np.log(p)).sum()) < TIGHT * 10
        _near(tlp[i], want[i][tix[i]])
    assert lp[2] == -np.inf and ent[2] == 0 and m[2] == -np.inf and z[2] == 0 and lp[4] == 0 and np.isnan(lp[5])
    assert list(tix[2]) == list(range(9)) and list(tix[3][:5]) == [4, 5, 6, 7, 8] and np.all(tlp[2] == -np.inf)


@pytest.mark.parametrize("entropy", [False, True])
@pytest.mark.parametrize("prob", [False, True])
def test_token_logprob_bwd(entropy, prob):
    if not (entropy or prob):
        return
    rng = np.random.default_rng(6)
    x = rng.standard_normal((4, 30)) * 2
    token = np.array([3, 29, -1, 0])
    dlp = rng.standard_normal(4) if prob else None
    dent = rng.standard_normal(4) if entropy else None
    g = rows.token_logprob_bwd(x, token, 1.3, dlp, dent)
    d = rng.standard_normal(x.shape)

    def f(v):
        lp, _, _, ent, _, _ = rows.token_logprob(v, token, 1.3, 0)
        return (lp * dlp).sum() * prob + (ent * dent).sum() * entropy if prob and entropy else \
            (lp * dlp).sum() if prob else (ent * dent).sum()

    assert abs(_differences(f, x, d) - (g * d).sum()) < 1e-6
    y = x.copy()
    y[1, 5] = -np.inf
    y[3] = -np.inf
    g = rows.token_logprob_bwd(y, np.array([3, 30, -1, 0]), 1.3, dlp, dent)
    assert np.all(g[3] == 0) and np.all(np.isfinite(g[[0, 2]])) and np.all(np.isnan(g[1])) == prob
