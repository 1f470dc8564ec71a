"""Argument checks of the residual norm, the gated block and the log probabilities, and the properties of their
workspace sizes.  No kernel is launched here: every call is refused, or has no rows."""
import ctypes as C

import pytest

from bit_nf4_quantized_11_amd import _lib

OK, NULL, SHAPE, ALIGN, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3, 4, 5
P, Q, R, S = 0x10000, 0x20000, 0x30000, 0x40000   # never read: refused before any launch


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def test_rms_norm_validation(lib):
    def f(x=P, sx=64, r=None, sr=0, rows=3, dim=64, w=Q, eps=1e-6, y=R, sy=64, h=None, sh=0):
        return lib.qlora_rms_norm(x, sx, r, sr, rows, dim, w, eps, y, sy, h, sh, None)

    assert f(rows=0) == OK and f(rows=0, x=None, y=None) == OK and f(rows=0, r=P, h=None) == OK
    assert f(x=None) == NULL and f(y=None) == NULL and f(r=S, sr=64) == NULL and f(h=S, sh=64) == NULL
    for dim in (0, -8, 4, 12, 32776):
        assert f(dim=dim) == SHAPE and f(rows=0, dim=dim) == SHAPE
    assert f(rows=-1) == SHAPE and f(rows=1 << 22) == SHAPE
    assert f(sx=-8) == SHAPE and f(sx=1 << 36) == SHAPE and f(sy=56) == SHAPE and f(sy=0) == SHAPE
    assert f(r=S, sr=-8, h=P, sh=64) == SHAPE and f(r=S, sr=64, h=P, sh=56) == SHAPE
    assert f(r=S, sr=64, h=R, sh=64) == SHAPE                     # y and sum the same
    assert f(x=P + 8) == ALIGN and f(y=R + 2) == ALIGN and f(w=Q + 8) == ALIGN and f(sx=68) == ALIGN and f(sy=68) == ALIGN
    assert f(r=S + 8, sr=64, h=P, sh=64) == ALIGN and f(r=S, sr=60, h=P, sh=64) == ALIGN
    for eps in (-1e-6, float("nan"), float("inf")):
        assert f(eps=eps) == UNSUPPORTED


def test_rms_norm_bwd_validation(lib):
    need = lib.qlora_rms_norm_bwd_workspace(3, 64)

    def f(dy=P, sg=64, h=Q, sh=64, dh=None, sd=0, rows=3, dim=64, w=Q, eps=1e-6, dx=R, sx=64, dw=S, ws=S, n=need):
        return lib.qlora_rms_norm_bwd(dy, sg, h, sh, dh, sd, rows, dim, w, eps, dx, sx, dw, ws, n, None)

    assert need > 0 and need % 256 == 0
    assert f(rows=0, dw=None) == OK
    assert f(dy=None) == NULL and f(h=None) == NULL and f(dx=None) == NULL and f(w=None) == NULL   # (a gradient without weight)
    assert f(dim=20) == SHAPE and f(rows=-1) == SHAPE and f(sx=32) == SHAPE and f(sh=-8) == SHAPE and f(dh=P, sd=1 << 36) == SHAPE
    assert f(dy=P + 8) == ALIGN and f(dw=S + 2) == ALIGN and f(ws=S + 8) == ALIGN and f(dh=P + 2, sd=64) == ALIGN
    assert f(eps=-1.0) == UNSUPPORTED
    assert f(n=need - 1) == WORKSPACE and f(ws=None) == WORKSPACE
    for bad in ((-1, 64), (1 << 22, 64), (3, 4), (3, 12), (3, 32776)):
        assert lib.qlora_rms_norm_bwd_workspace(*bad) == 0


def test_rms_norm_bwd_workspace_grows_with_the_rows(lib):
    for dim in (8, 64, 512, 520, 1024, 2048, 2056, 4096, 8192, 8200, 16384, 32768):
        got = [lib.qlora_rms_norm_bwd_workspace(n, dim) for n in list(range(0, 40)) + [100, 255, 256, 257, 1000, 5000, 1 << 20]]
        assert got == sorted(got) and got[0] > 0 and got[-1] <= 256 << 20


def _w(rows=128, cols=64, dq=0, cb=0, block=64, codes=P):
    return _lib.qlora_nf4(rows, cols, dq, cb, block, 0, codes, Q, Q, Q)


def test_gated_fwd_validation(lib):
    need = lib.qlora_gated_workspace(3, 64, 128, 8)
    assert need > 0

    def f(X=P, M=3, gate=_w(), up=_w(), Ag=P, Bg=P, Au=P, Bu=P, r=8, act=0, H=R, G=None, U=None, Tg=None, Tu=None, ws=S, n=need):
        return lib.qlora_gated_fwd(X, M, None if gate is None else C.byref(gate), None if up is None else C.byref(up), Ag, Bg,
                                   Au, Bu, r, 0.5, act, H, G, U, Tg, Tu, ws, n, None)

    assert f(M=0, X=None, H=None) == OK
    for name in ("X", "gate", "up", "Ag", "Bg", "Au", "Bu", "H"):
        assert f(**{name: None}) == NULL
    assert f(G=P) == NULL and f(U=P) == NULL and f(Tg=P) == NULL and f(Tu=P) == NULL and f(up=_w(codes=None)) == NULL
    assert f(M=-1) == SHAPE and f(M=1 << 26) == SHAPE and f(up=_w(rows=136)) == SHAPE and f(up=_w(cols=128)) == SHAPE
    assert f(gate=_w(rows=132), up=_w(rows=132)) == SHAPE and f(gate=_w(cols=96), up=_w(cols=96)) == SHAPE
    for up in (_w(dq=1), _w(cb=1), _w(block=32)):
        assert f(up=up) == UNSUPPORTED
    assert f(act=2) == UNSUPPORTED and f(act=-1) == UNSUPPORTED and f(r=12) == UNSUPPORTED and f(r=264) == UNSUPPORTED
    for name in ("X", "Ag", "Bg", "Au", "Bu", "H"):
        assert f(**{name: P + 8}) == ALIGN
    assert f(G=P, U=P + 8) == ALIGN and f(Tg=P, Tu=P + 2) == ALIGN and f(ws=S + 8) == ALIGN
    assert f(n=need - 1) == WORKSPACE and f(ws=None) == WORKSPACE
    # 0 and 64 are the same block size
    assert f(up=_w(block=0), n=need - 1) == WORKSPACE
    for bad in ((-1, 64, 128, 8), (1 << 26, 64, 128, 8), (3, 32, 128, 8), (3, 64, 4, 8), (3, 64, 128, 4), (3, 64, 128, 300),
                (3, (1 << 22) + 64, 128, 8), (3, 64, (1 << 22) + 8, 8)):
        assert lib.qlora_gated_workspace(*bad) == 0


def test_gated_bwd_validation(lib):
    def f(dH=P, G=Q, U=R, M=3, n=64, act=1, dG=S, dU=P, H=None):
        return lib.qlora_gated_bwd(dH, G, U, M, n, act, dG, dU, H, None)

    assert f(M=0) == OK and f(M=0, dH=None, G=None, U=None, dG=None, dU=None) == OK
    for name in ("dH", "G", "U", "dG", "dU"):
        assert f(**{name: None}) == NULL
    assert f(dH=None, dG=None, dU=None) == NULL and f(dH=None, dU=None, H=S) == NULL      # H alone, or all
    assert f(M=-1) == SHAPE and f(M=1 << 26) == SHAPE and f(n=0) == SHAPE and f(n=12) == SHAPE and f(n=(1 << 22) + 8) == SHAPE
    assert f(dG=P, dU=P) == SHAPE and f(H=S) == SHAPE and f(H=P) == SHAPE            # one output twice
    for name in ("dH", "G", "U", "dG", "dU", "H"):
        assert f(**{name: 0x50008}) == ALIGN
    assert f(act=2) == UNSUPPORTED and f(act=-1) == UNSUPPORTED


def test_token_logprob_validation(lib):
    need = lib.qlora_token_logprob_workspace(3, 40000, 5)
    assert need > 0

    def f(x=P, sx=40000, rows=3, vocab=40000, dt=1, tok=P, scale=1.0, top=5, lp=Q, st=Q, ent=None, tlp=R, tix=R, ws=S, n=need):
        return lib.qlora_token_logprob(x, sx, rows, vocab, dt, tok, scale, top, lp, st, ent, tlp, tix, ws, n, None)

    assert f(rows=0, x=None, st=None) == OK
    assert f(x=None) == NULL and f(st=None) == NULL and f(tok=None) == NULL and f(tlp=None) == NULL and f(tix=None) == NULL
    assert f(rows=-1) == SHAPE and f(rows=1 << 22) == SHAPE and f(vocab=0) == SHAPE and f(vocab=(1 << 20) + 1) == SHAPE
    assert f(rows=(1 << 22) - 1, vocab=1 << 14) == SHAPE and f(top=33) == SHAPE and f(top=-1) == SHAPE and f(vocab=4) == SHAPE
    assert f(sx=-1) == SHAPE and f(sx=1 << 36) == SHAPE
    assert f(x=P + 2) == ALIGN and f(x=P + 1, dt=0) == ALIGN and f(tok=P + 4) == ALIGN and f(tix=R + 4) == ALIGN and f(st=Q + 2) == ALIGN
    assert f(ent=Q + 1) == ALIGN and f(lp=Q + 2) == ALIGN and f(tlp=R + 2) == ALIGN and f(ws=S + 8) == ALIGN
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert f(scale=scale) == UNSUPPORTED
    assert f(dt=2) == UNSUPPORTED and f(dt=-1) == UNSUPPORTED
    assert f(ws=None) == WORKSPACE and f(n=0) == WORKSPACE
    for bad in ((-1, 5, 0), (1 << 22, 5, 0), (3, 0, 0), (3, (1 << 20) + 1, 0), (3, 5, 33), (3, 5, -1), ((1 << 22) - 1, 1 << 14, 0)):
        assert lib.qlora_token_logprob_workspace(*bad) == 0


def test_token_logprob_workspace_grows_and_suffices(lib):
    """The query never falls with rows, vocab or top; and a call is never refused for the workspace that its own query
    gave (a call with a bad pointer behind that check says ALIGN, not WORKSPACE)."""
    vocabs = [1, 7, 100, 4096, 4097, 16384, 32000, 32768, 32769, 50001, 65536, 65537, 131072, 200000, 1 << 20]
    before = None
    for rows in (0, 1, 2, 3, 7, 8, 31, 64, 100, 127, 128, 129, 255, 300, 5000):
        got = [[lib.qlora_token_logprob_workspace(rows, v, top) for v in vocabs] for top in (0, 1, 20, 32)]
        assert all(g == sorted(g) for g in got) and all(a <= b for x, y in zip(got, got[1:]) for a, b in zip(x, y))
        assert before is None or all(a <= b for x, y in zip(before, got) for a, b in zip(x, y))
        before = got
        for v in vocabs:
            for dt in (0, 1):
                for top in (0, min(v, 32)):
                    if rows:
                        n = lib.qlora_token_logprob_workspace(rows, v, top)
                        st = lib.qlora_token_logprob(P, v, rows, v, dt, P, 1.0, top, Q, Q, None, R, R, S + 8, n, None)
                        assert st == ALIGN, (rows, v, dt, top)


def test_token_logprob_bwd_validation(lib):
    def f(x=P, sx=100, rows=3, vocab=100, dt=1, tok=P, scale=1.0, st=Q, dlp=Q, ent=None, dent=None, dx=R, sd=100):
        return lib.qlora_token_logprob_bwd(x, sx, rows, vocab, dt, tok, scale, st, dlp, ent, dent, dx, sd, None)

    assert f(rows=0, x=None, dx=None) == OK
    assert f(x=None) == NULL and f(dx=None) == NULL and f(st=None) == NULL and f(tok=None) == NULL and f(dent=Q) == NULL
    assert f(dlp=None) == NULL
    assert f(sd=99) == SHAPE and f(vocab=0) == SHAPE and f(rows=1 << 22) == SHAPE and f(sd=-100) == SHAPE
    assert f(dx=R + 2) == ALIGN and f(tok=P + 4) == ALIGN and f(dlp=Q + 2) == ALIGN and f(ent=Q, dent=Q + 2) == ALIGN
    assert f(scale=0.0) == UNSUPPORTED and f(dt=3) == UNSUPPORTED


def test_outputs_that_would_overlap(lib):
    """Rows written where inputs begin, at another stride, and one tensor for two outputs."""
    n = lib.qlora_rms_norm_bwd_workspace(3, 64)

    def norm(y=R, sy=64, h=S, sh=64):
        return lib.qlora_rms_norm(P, 64, Q, 72, 3, 64, None, 0.0, y, sy, h, sh, None)

    assert norm(y=P, sy=72) == SHAPE and norm(y=Q, sy=64) == SHAPE and norm(h=P, sh=72) == SHAPE and norm(h=Q, sh=64) == SHAPE
    assert lib.qlora_rms_norm(P, 64, None, 0, 3, 64, None, 0.0, P, 128, None, 0, None) == SHAPE
    for src in (P, Q, R):
        st = lib.qlora_rms_norm_bwd(P, 64, Q, 64, R, 64, 3, 64, None, 0.0, src, 128, None, None, n, None)
        assert st == SHAPE
    assert lib.qlora_token_logprob_bwd(P, 100, 3, 100, 1, Q, 1.0, Q, Q, None, None, P, 101, None) == SHAPE
    w = _w()
    need = lib.qlora_gated_workspace(3, 64, 128, 8)
    for H, G, U, Tg, Tu in ((P, None, None, None, None), (R, P, S, None, None), (R, S, P, None, None), (R, R, S, None, None),
                            (R, S, R, None, None), (R, S, S, None, None), (R, None, None, S, S)):
        st = lib.qlora_gated_fwd(P, 3, C.byref(w), C.byref(w), P, P, P, P, 8, 0.5, 0, H, G, U, Tg, Tu, S, need, None)
        assert st == SHAPE


def test_token_logprob_without_workspace(lib):
    """None up to 32768 logits a row, or 16384 from 128 rows on: then a call of 0 bytes passes the check of its size (and is
    refused for its alignment behind that)."""
    for rows, most in ((1, 32768), (127, 32768), (128, 16384), (5000, 16384)):
        for dt in (0, 1):
            for v in (1, 4097, 8192, 8193, 16384, most):
                assert lib.qlora_token_logprob_workspace(rows, v, 1) == 0
                assert lib.qlora_token_logprob(P, v, rows, v, dt, P, 1.0, 1, Q, Q, None, R, R, P + 8, 0, None) == ALIGN
        assert lib.qlora_token_logprob_workspace(rows, most + 1, 0) > 0
