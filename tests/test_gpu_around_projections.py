"""Uses of the residual norm, the gated block and the log probabilities that go past one call: two streams at once, captured
graphs that share a workspace, saved outputs in part, one weight on both sides, and the largest row counts and offsets."""
import ctypes as C

import pytest
import torch

import bit_nf4_quantized_11_amd as Q
from bit_nf4_quantized_11_amd import _lib
from helpers import dev_bf16, require_gpu
from kv_cases import bits

pytestmark = pytest.mark.gpu

BF16, FP32 = 2.0 ** -8, 2.0 ** -24
K, N, R, V = 512, 1032, 24, 40000
TOKENS = (5, 150, 1200)   # a pass over the weights, K-slices, whole tiles


class Layer:
    def __init__(self, seed):
        self.w = [Q.qlora_quantize_nf4(dev_bf16(bits(seed + i, (N, K), 0.05))) for i in range(2)]
        self.A = [dev_bf16(bits(seed + 2 + i, (K, R), 0.05)) for i in range(2)]
        self.B = [dev_bf16(bits(seed + 4 + i, (R, N), 0.05)) for i in range(2)]

    def __call__(self, X, **kw):
        return Q.qlora_gated_fwd(X, self.w[0], self.w[1], self.A[0], self.B[0], self.A[1], self.B[1], 0.5, **kw)


def _workspaces(M):
    """One for each of a step's calls that take one: gated block, norm's backward, log probabilities."""
    sizes = (Q.qlora_gated_workspace(M, K, N, R), Q.qlora_rms_norm_bwd_workspace(M, K), Q.qlora_token_logprob_workspace(min(M, 64), V, 9))
    return [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes]


def _inputs(seed, M):
    gen = torch.Generator().manual_seed(seed)
    n = min(M, 64)
    return {"x": dev_bf16(bits(seed, (M, K))), "res": dev_bf16(bits(seed + 1, (M, K))), "d": dev_bf16(bits(seed + 2, (M, N))),
            "logits": torch.randn(n, V, generator=gen).cuda(), "token": torch.randint(0, V, (n,), generator=gen).cuda(),
            "dlp": torch.randn(n, generator=gen).cuda(), "w": (1 + 0.2 * dev_bf16(bits(seed + 3, (K,))).float()).bfloat16()}


def _step(layer, t, ws, stream=None):
    y, h = Q.qlora_rms_norm(t["x"], t["w"], t["res"], stream=stream)
    H, G, U, Tg, Tu = layer(y, workspace=ws[0], stream=stream)
    g = Q.qlora_gated_bwd(t["d"], G, U, H=True, stream=stream)
    n = Q.qlora_rms_norm_bwd(y, h, t["w"], t["res"], workspace=ws[1], stream=stream)
    lp = Q.qlora_token_logprob(t["logits"], t["token"], 0.7, entropy=True, top=9, workspace=ws[2], stream=stream)
    dl = Q.qlora_token_logprob_bwd(t["logits"], t["token"], lp[1], t["dlp"], scale=0.7, stream=stream)
    return (y, h, H, G, U, Tg, Tu, *g, *n, *lp, dl)


def _same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("M", TOKENS)
def test_two_streams_at_once(M):
    """Each with its own workspaces: the bits of one after the other."""
    require_gpu()
    layers, inputs = [Layer(10), Layer(20)], [_inputs(30, M), _inputs(40, M)]
    ws = [_workspaces(M), _workspaces(M)]
    want = [_step(layers[i], inputs[i], ws[i]) for i in range(2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(4):
        for i, s in enumerate(streams):
            got[i].append(_step(layers[i], inputs[i], ws[i], s))
    for s in streams:
        s.synchronize()
    for i in range(2):
        assert all(_same(want[i], g) for g in got[i])


def test_captured_graphs_share_workspaces():
    """Three graphs of different sizes on the largest of their workspaces, replayed in turn: no replay depends on what another
    one left there."""
    require_gpu()
    layer = Layer(50)
    ws = [max((t[i] for t in map(_workspaces, TOKENS)), key=lambda t: t.numel()) for i in range(3)]
    inputs = [_inputs(60 + 10 * i, M) for i, M in enumerate(TOKENS)]
    for t in inputs:
        _step(layer, t, ws)
    torch.cuda.synchronize()
    graphs, out = [], []
    for t in inputs:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            out.append(_step(layer, t, ws))
    for k in range(3):
        want = []
        for i, t in enumerate(inputs):
            new = _inputs(1000 + 100 * k + 10 * i, TOKENS[i])
            for name in t:
                t[name].copy_(new[name])
            want.append([v.clone() for v in _step(layer, t, _workspaces(TOKENS[i]))])
        for i in (2, 0, 1, 0, 2):
            for v in out[i]:
                v.zero_()
            graphs[i].replay()
            torch.cuda.synchronize()
            assert _same(out[i], want[i]), (k, i)


@pytest.mark.parametrize("M", TOKENS)
def test_saved_in_part(M):
    """G and U without T, T without G and U, and neither: the outputs that are asked for are those of the whole call."""
    require_gpu()
    layer, X = Layer(70), dev_bf16(bits(71, (M, K)))
    want = layer(X)
    lib = _lib.load()
    ws = _workspaces(M)[0]
    g, u = (w.desc() for w in layer.w)
    for parts in ((), (1, 2), (3, 4)):
        out = [torch.full_like(t, 7.0) for t in want]
        p = [out[i].data_ptr() if i == 0 or i in parts else None for i in range(5)]
        st = lib.qlora_gated_fwd(X.data_ptr(), M, C.byref(g), C.byref(u), layer.A[0].data_ptr(), layer.B[0].data_ptr(),
                                 layer.A[1].data_ptr(), layer.B[1].data_ptr(), R, 0.5, 0, *p, ws.data_ptr(), ws.nbytes,
                                 torch.cuda.current_stream().cuda_stream)
        assert st == 0
        torch.cuda.synchronize()
        for i, t in enumerate(out):
            assert torch.equal(t, want[i]) if i == 0 or i in parts else torch.all(t == 7.0)


@pytest.mark.parametrize("M", TOKENS)
def test_one_weight_on_both_sides(M):
    require_gpu()
    layer = Layer(80)
    layer.w[1], layer.A[1], layer.B[1] = layer.w[0], layer.A[0], layer.B[0]
    H, G, U, Tg, Tu = layer(dev_bf16(bits(81, (M, K))))
    assert torch.equal(G, U) and torch.equal(Tg, Tu)
    # g^2 s of an unrounded g, and of its rounding: g off by 2^-8 twice over, s by |g| 2^-8 / 4 at most, and one rounding
    g = G.float()
    assert torch.all((H.float() - g * g * torch.sigmoid(g)).abs() <= (3 * BF16 + g.abs() * BF16 / 4 + 2 * BF16 * BF16) * (g * g) + 2.0 ** -126)


def test_largest_gated_block():
    """260000 tokens of 8008 features, each output close below the 4 GiB that the products take (more is refused).  Its last rows are
    those of a call on these rows alone, up to the rounding of T, where another order of its sums may end, and the output's
    own: 2^-8 of a part of G or U each, fewer than eight of these in a product."""
    require_gpu()
    M, k, n, tail = 260000, 64, 8008, 300
    w = [Q.qlora_quantize_nf4(dev_bf16(bits(90 + i, (n, k), 0.1))) for i in range(2)]
    A, B = [dev_bf16(bits(92 + i, (k, 8), 0.1)) for i in range(2)], [dev_bf16(bits(94 + i, (8, n), 0.1)) for i in range(2)]
    X = torch.zeros(M + 10000, k, dtype=torch.bfloat16, device="cuda")
    X[M - tail:M] = dev_bf16(bits(96, (tail, k)))
    X[:tail] = X[M - tail:M].flip(0)
    call = lambda X: Q.qlora_gated_fwd(X, w[0], w[1], A[0], B[0], A[1], B[1], 1.0)
    with pytest.raises(Q.QLoRAError):
        call(X)
    H, G, U, _, _ = call(X[:M])
    h, g, u, _, _ = call(X[M - tail:M].contiguous())
    for big, small in ((H, h), (G, g), (U, u)):
        for part in (big[-tail:], big[:tail].flip(0)):
            assert (part.float() - small.float()).norm() <= 8 * BF16 * small.float().norm()
        assert big[tail:tail + 1000].abs().max() == 0 and big[-tail - 1000:-tail].abs().max() == 0


def test_gated_backward_past_32_bit_offsets():
    """2.2e9 elements, in place, more than one round of the largest launch."""
    require_gpu()
    M, n, tail = 270000, 8008, 300
    dH, G, U = (torch.zeros(M, n, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    for i, t in enumerate((dH, G, U)):
        t[-tail:] = t[:tail] = dev_bf16(bits(97 + i, (tail, n)))
    want = Q.qlora_gated_bwd(*(t[:tail].clone() for t in (dH, G, U)), H=True)
    got = Q.qlora_gated_bwd(dH, G, U, dG=G, dU=U, H=dH)
    for a, b in zip(got, want):
        assert torch.equal(a[-tail:], b) and torch.equal(a[:tail], b) and a[M // 2].abs().max() == 0


def test_most_rows():
    """As many rows as a call takes, of the fewest elements."""
    require_gpu()
    n = (1 << 22) - 1
    x, r, dy = (dev_bf16(bits(100 + i, (1 << 10, 8))).repeat(1 << 12, 1)[:n] for i in range(3))
    w = torch.ones(8, dtype=torch.bfloat16, device="cuda")
    y, h = Q.qlora_rms_norm(x, w, r)
    small = Q.qlora_rms_norm(x[:1024], w, r[:1024])
    for big, s in ((y, small[0]), (h, small[1])):
        assert torch.equal(big[:1024], s) and torch.equal(big[-1023:], s[:1023]) and torch.equal(big[1 << 21:][:1024], s)
    dx, dw = Q.qlora_rms_norm_bwd(dy, h, w)
    sx, sw = Q.qlora_rms_norm_bwd(dy[:1024], h[:1024], w)
    assert torch.equal(dx[:1024], sx) and torch.equal(dx[-1023:], sx[:1023])
    # the sum of n terms: a thread adds n / 2048 of them, then 512 partials and 4 waves are added
    f = h.double()
    terms = dy.double() * f * (f.pow(2).mean(1, keepdim=True) + 1e-6).rsqrt()
    assert torch.all((dw.double() - terms.sum(0)).abs() <= (n / 2048 + 512 + 4 + 8) * FP32 * terms.abs().sum(0))
    for dtype in (torch.bfloat16, torch.float32):
        logits = dy.to(dtype)[:, :5]
        token = torch.arange(n, device="cuda") % 5
        lp, stats, ent, tlp, tix = Q.qlora_token_logprob(logits, token, entropy=True, top=2)
        few = Q.qlora_token_logprob(logits[-1000:], token[-1000:], entropy=True, top=2)
        assert _same([t[-1000:] for t in (lp, stats, ent, tlp, tix)], few)
        all_lp = torch.log_softmax(logits.double(), 1)
        assert (lp - all_lp.gather(1, token[:, None])[:, 0]).abs().max() < 1e-5
        d = Q.qlora_token_logprob_bwd(logits, token, stats, torch.ones(n, device="cuda"))
        want = torch.nn.functional.one_hot(token, 5) - all_lp.exp()
        assert (d.double() - want).abs().max() <= (BF16 if dtype == torch.bfloat16 else 0) + 1e-5


@pytest.mark.parametrize("rows", [1, 130])
def test_largest_vocabulary(rows):
    """2^20 fp32 logits to a row and 32 alternatives, the last and the first among them, in the most parts of a row."""
    require_gpu()
    v = 1 << 20
    x = torch.randn(rows, v, generator=torch.Generator("cuda").manual_seed(3), device="cuda")
    place = torch.arange(32, device="cuda") * (v // 31 - 1)
    place[-1] = v - 1
    x[:, place] = 20.0 + torch.arange(32, device="cuda") / 64.0
    token = torch.full((rows,), v - 1, device="cuda")
    lp, stats, ent, tlp, tix = Q.qlora_token_logprob(x, token, entropy=True, top=32)
    assert torch.equal(tix, place.flip(0).expand(rows, 32))
    for i in (0, rows - 1):
        all_lp = torch.log_softmax(x[i].double(), 0)
        # (the sums are of positive terms in trees of fewer than 2^10 additions in a row)
        assert (tlp[i] - all_lp[tix[i]]).abs().max() <= 2.0 ** -13 and (lp[i] - all_lp[-1]).abs() <= 2.0 ** -13
        assert (ent[i] + (all_lp.exp() * all_lp).sum()).abs() <= 2.0 ** -10


@pytest.mark.parametrize("rows,dim", [(5000, 64), (4500, 1024), (2100, 2048), (1200, 4096), (1100, 5000), (1100, 8192), (600, 16384),
                                      (600, 16392)], ids=str)
def test_norm_in_place_over_many_rows(rows, dim):
    """Every workgroup goes over several rows: each output on each input, at every number of threads of a row."""
    require_gpu()
    x, r, dh, dy = (dev_bf16(bits(110 + i, (64, dim))).repeat(rows // 64 + 1, 1)[:rows] for i in range(4))
    w = (1 + 0.2 * dev_bf16(bits(120, (dim,))).float()).bfloat16()
    y, h = Q.qlora_rms_norm(x, w, r)
    a, b = x.clone(), r.clone()
    assert _same(Q.qlora_rms_norm(a, w, b, out=b, sum_out=a), (y, h))
    a = x.clone()
    assert torch.equal(Q.qlora_rms_norm(a, w, out=a)[0], Q.qlora_rms_norm(x, w)[0])
    for given in (None, dh):
        want = Q.qlora_rms_norm_bwd(dy, h, w, given)
        assert torch.equal(want[0], want[0][:64].repeat(rows // 64 + 1, 1)[:rows])
        for i in range(2 if given is None else 3):
            t = [v.clone() for v in ((dy, h) if given is None else (dy, h, dh))]
            assert _same(Q.qlora_rms_norm_bwd(t[0], t[1], w, *t[2:], dx=t[i]), want) if given is not None else \
                _same(Q.qlora_rms_norm_bwd(t[0], t[1], w, dx=t[i]), want)
