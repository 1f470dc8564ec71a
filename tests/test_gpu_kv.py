"""GPU parity of the 4-bit cache (written, read back: bit for bit) and of the attention over it.

Attention's tolerance, from the roundings on its path (fp16: half a step is 2^-11 of a normal value, 2^-25 below
2^-14).  Levels are held in fp16 times a constant that makes FP4's and Int4's exact: TAB below.  A logit is then off by
at most TAB * scale * sum |q k| plus fp32 errors and what a row's elements below 2^-17 of its largest lose (2^-16 of
that sum is ample), so p / sum p by twice that (relatively).  p is rounded to fp16 and multiplied with a power-of-two
share of the value's scale, rounded again: 2 * 2^-11, or, where small, at most 3 * 2^-25 of the largest such product's
unit, which is 2^-13 of the largest scale: 3 * 2^-38 * max|v| for each of n tokens.  With E = the logit's error
  |o - want| <= (2 E + 2^-10 + TAB) (1 + small) sum p|v| + 3 n 2^-38 max|v| + 2^-8 |want|.
Errors of different elements are independent, so over a whole output they come to far less: relative Frobenius
error at most 3e-3 (2^-8 / sqrt 3 = 2.3e-3 is the most that the output's own rounding to bf16 can come to for any
distribution of its significands, 0.3e-3 each for p, values and logits of unit spread), asserted for ordinary data."""
import math

import numpy as np
import pytest
import torch

import bit_nf4_quantized_11_amd as Q
from helpers import dev_bf16, host, host_u16, log, require_gpu
from kv_cases import CODEBOOKS, bits, device_batch, fill_cache, i32, layout
from oracle import kv

pytestmark = pytest.mark.gpu

TAB = {"nf4": 2.0 ** -11, "fp4": 2.0 ** -22, "int4": 2.0 ** -22}
P16 = 2.0 ** -10
FAULT_START, FAULT_LENGTH, FAULT_PAGE = 1, 2, 4


def _word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ---- write and read ----------------------------------------------------------------------------------------
STORE = [
    # lens, new, heads, dim, block, page, book
    ([1], [1], 1, 64, 64, 16, "nf4"),
    ([17, 5], [17, 5], 3, 128, 64, 16, "nf4"),
    ([40, 0, 33, 7], [9, 0, 33, 1], 2, 64, 32, 16, "fp4"),
    ([70], [40], 1, 256, 128, 32, "int4"),
    ([3, 100, 1], [2, 50, 1], 2, 256, 32, 64, "nf4"),
    ([130], [130], 1, 128, 128, 128, "fp4"),
    ([20, 30], [20, 30], 5, 128, 32, 16, "int4"),
]


@pytest.mark.parametrize("lens,new,heads,dim,block,page,book", STORE, ids=str)
def test_write_and_read_back(lens, new, heads, dim, block, page, book):
    require_gpu()
    log("kv write/read", lens, new, heads, dim, block, page, book)
    h = layout(lens, new, page, sum(lens) + dim)
    rows = h.rows + 3                                        # rows behind the last sequence
    x = {"k": bits(1, (rows, heads, dim), 3.0), "v": bits(2, (rows, heads, dim))}
    x["k"][0, 0, :block] = 0                                 # a block of zeros
    x["v"][0, 0, 3] = 0x8001                                 # and a subnormal among ordinary values
    cache = Q.kv_alloc(h.pages, page, heads, dim, block, CODEBOOKS[book])
    for t in (cache.k_codes, cache.v_codes):
        t.fill_(0xA5)
    for t in (cache.k_scale, cache.v_scale):
        t.fill_(3.0)
    fault = _word()
    batch = device_batch(h, fault)
    Q.qlora_kv_write(dev_bf16(x["k"]), dev_bf16(x["v"]), cache, batch)
    got = {"k": (host(cache.k_codes), host_u16(cache.k_scale)), "v": (host(cache.v_codes), host_u16(cache.v_scale))}
    out = {t: torch.full((rows, heads, dim), 7.0, dtype=torch.bfloat16, device="cuda") for t in "kv"}
    Q.qlora_kv_read(cache, batch, rows, out["k"], out["v"])
    touched = np.zeros((h.pages, page), bool)
    for t in "kv":
        back = host_u16(out[t])
        for b, (n, m) in enumerate(zip(lens, new)):
            for i in range(m):
                p = n - m + i
                pg, off, row = h.table[b, p // page], p % page, h.start[b] + i
                touched[pg, off] = True
                for hd in range(heads):
                    c, s = kv.quantize_row(x[t][row, hd], block, book)
                    assert np.array_equal(got[t][0][pg, hd, off], kv.pack_row(c, t == "k")), (t, b, i, hd)
                    assert np.array_equal(got[t][1][pg, hd, off], s), (t, b, i, hd)
                    assert np.array_equal(back[row, hd], kv.row_bf16(c, s, book)), (t, b, i, hd)
        # no other slot and no other row is touched
        assert np.all(got[t][0].transpose(0, 2, 1, 3)[~touched] == 0xA5)
        assert np.all(got[t][1].transpose(0, 2, 1, 3)[~touched] == 0x4040)
        assert torch.all(out[t][h.rows:] == 7.0)
    assert fault.item() == 0


def test_every_bf16_share_gets_the_weight_quantizers_code():
    """Rows whose first element is 1 and the others sweep the bf16 values up to it, in both signs: the same
    codes as the weight quantizer's on the same blocks."""
    require_gpu()
    vals = np.arange(0x3600, 0x3F81, dtype=np.uint16)        # 2^-19 .. 1
    vals = np.concatenate([vals, vals | 0x8000])
    vals = np.concatenate([vals, np.zeros(-len(vals) % 63, np.uint16)]).reshape(-1, 63)
    x = np.concatenate([np.full((len(vals), 1), 0x3F80, np.uint16), vals], 1)
    for book, cb in CODEBOOKS.items():
        h = layout([len(x)], [len(x)], 64, cb)
        cache = Q.kv_alloc(h.pages, 64, 1, 64, 64, cb)
        d = dev_bf16(x[:, None])
        Q.qlora_kv_write(d, d, cache, device_batch(h))
        w = Q.qlora_quantize_nf4(d.view(len(x), 64), double_quant=False, codebook=cb)
        got = cache.v_codes[torch.from_numpy(h.table[0, :-1].astype(np.int64)).cuda(), 0].flatten(0, 1)[:len(x)]
        assert torch.equal(got.flatten(), w.codes), book


def test_non_finite_rows_and_strides():
    require_gpu()
    heads, dim, block = 2, 128, 32
    h = layout([6], [6], 16, 0)
    joint = dev_bf16(bits(3, (6, 3 * heads * dim)))          # q, k, v of one projection
    k, v = (joint[:, i * heads * dim:(i + 1) * heads * dim].unflatten(1, (heads, dim)) for i in (1, 2))
    k[2, 1, 40] = float("inf")
    k[3, 0, 0] = float("nan")
    cache = Q.kv_alloc(h.pages, 16, heads, dim, block)
    batch = device_batch(h)
    Q.qlora_kv_write(k, v, cache, batch)
    ko = torch.empty(heads, 6, dim, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    vo = torch.empty(6, heads, dim + 24, dtype=torch.bfloat16, device="cuda")[..., 8:dim + 8]
    Q.qlora_kv_read(cache, batch, 6, ko, vo)
    bad = torch.isnan(ko.float())
    assert bad[2, 1, 32:64].all() and bad[3, 0, :32].all() and bad.sum() == 64
    cache2 = Q.kv_alloc(h.pages, 16, heads, dim, block)
    Q.qlora_kv_write(k.contiguous(), v.contiguous(), cache2, batch)
    k2, v2 = Q.qlora_kv_read(cache2, batch, 6)
    assert torch.equal(v2, vo) and torch.equal(torch.nan_to_num(k2), torch.nan_to_num(ko))


def test_wrong_entries_are_reported_and_touch_nothing():
    """Pages, lengths and starts out of range: checked by the kernels, the bit set, nothing written, NaN read."""
    require_gpu()
    heads, dim, page, pages = 1, 64, 16, 4
    k = dev_bf16(bits(1, (4, heads, dim)))

    def run(start, length, table):
        cache = Q.kv_alloc(pages, page, heads, dim)
        for t in (cache.k_codes, cache.v_codes, cache.k_scale, cache.v_scale):
            t.zero_()
        fault = _word()
        batch = Q.KVBatch(i32(start), i32(length), i32(table), fault)
        Q.qlora_kv_write(k, k, cache, batch)
        wrote = int(fault.item())
        fault.zero_()
        out = torch.full((4, heads, dim), 5.0, dtype=torch.bfloat16, device="cuda")
        o, lse = torch.full_like(out, 5.0), torch.full((4, heads), 5.0, device="cuda")
        Q.qlora_kv_read(cache, batch, 4, out, out.clone())
        read = int(fault.item())
        fault.zero_()
        Q.qlora_kv_attn(k, cache, batch, out=o, lse=lse)
        return wrote, read, int(fault.item()), cache, out.float()[:, 0], o.float()[:, 0], lse[:, 0]

    # a page past the end, and a negative one, under the second and third row
    for bad in (pages, -1, -2 ** 31, 2 ** 31 - 1):
        w, r, a, cache, out, o, lse = run([0, 4], [18], [[3, bad]])     # positions 14..17
        assert (w, r, a) == (FAULT_PAGE,) * 3
        assert torch.isfinite(out[:2]).all() and torch.isnan(out[2:]).all()
        assert torch.isfinite(o[:2]).all() and torch.isnan(o[2:]).all() and torch.isnan(lse[2:]).all()
        assert torch.count_nonzero(cache.k_scale) == 2
    for bad in (33, -1, 2 ** 31 - 1):                                  # two columns of 16 tokens
        w, r, a, cache, out, o, lse = run([0, 1, 4], [5, bad], [[0, 1], [2, 3]])
        assert (w, r, a) == (FAULT_LENGTH,) * 3
        assert torch.isfinite(out[0]).all() and torch.isnan(out[1:]).all()
        assert torch.isfinite(o[0]).all() and torch.isnan(o[1:]).all() and torch.isnan(lse[1:]).all()
        assert torch.count_nonzero(cache.k_scale) == 1
    for start in ([0, 5], [-1, 4], [3, 1], [0, -7], [0, 2 ** 31 - 1]):  # past the rows, before them, out of order
        w, r, a, cache, out, o, lse = run(start, [8], [[0, 1]])
        assert (w, r, a) == (FAULT_START,) * 3
        assert torch.all(out == 5.0) and torch.all(o == 5.0) and torch.all(lse == 5.0)
        assert torch.count_nonzero(cache.k_scale) == 0
    # a sequence that is in order beside one that is not
    w, r, a, cache, out, o, lse = run([0, 2, 9], [2, 7], [[0, 1], [2, 3]])
    assert (w, r, a) == (FAULT_START,) * 3 and torch.isfinite(o[:2]).all() and torch.all(o[2:] == 5.0)


# ---- attention ---------------------------------------------------------------------------------------------------
def check_attention(h, heads, group, dim, block, book, seed=0, causal=True, window=0, scale=None, q_std=1.0, k_gain=1.0,
                    fro=True, cache=None):
    scale = dim ** -0.5 if scale is None else scale
    cache, ks, vs = cache or fill_cache(h, heads, dim, block, book, seed, k_gain)
    rows = h.rows + 2
    q = bits(seed + 5, (rows, heads * group, dim), q_std)
    o = torch.full((rows, heads * group, dim), 9.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((rows, heads * group), 9.0, device="cuda")
    fault = _word()
    batch = device_batch(h, fault)
    Q.qlora_kv_attn(dev_bf16(q), cache, batch, scale, causal, window, out=o, lse=lse)
    assert fault.item() == 0
    assert torch.all(o[h.rows:] == 9.0) and torch.all(lse[h.rows:] == 9.0)
    got, gl = host(o.float()).astype(np.float64)[:h.rows], host(lse).astype(np.float64)[:h.rows]
    want, wl, bound = np.zeros_like(got), np.zeros_like(gl), np.zeros_like(got)
    err = np.zeros_like(gl)
    for b, (n, m) in enumerate(zip(h.lens, h.new)):
        r = slice(h.start[b], h.start[b + 1])
        qf = kv.f64(q[r])
        want[r], wl[r], bound[r] = kv.attention(qf, ks[b], vs[b], n, scale, causal, window)
        if n and m:
            mag = np.einsum("nhd,lhd->nhl", np.abs(qf), np.abs(np.repeat(ks[b], group, 1))).max(-1)
            err[r] = (TAB[book] + 2.0 ** -16) * scale * mag
    e = err[..., None]
    tol = (np.expm1(2 * e) + P16 + TAB[book]) * 1.02 * bound + 2.0 ** -8 * np.abs(want) * 1.02
    for b, n in enumerate(h.lens):
        if n:
            tol[h.start[b]:h.start[b + 1]] += 3 * n * 2.0 ** -38 * np.abs(vs[b]).max()
    d = np.abs(got - want)
    assert np.all(np.isfinite(got))
    assert np.all(d <= tol), (d.max(), (d / np.maximum(tol, 1e-30)).max())
    empty = np.isneginf(wl)
    assert np.array_equal(empty, np.isneginf(gl)) and np.all(got[empty] == 0)
    gl, wl = np.where(empty, 0, gl), np.where(empty, 0, wl)
    assert np.all(np.abs(gl - wl)[~empty] <= err[~empty] + 2.0 ** -20 * (1 + np.abs(wl[~empty])))
    if fro and np.linalg.norm(want) > 0:
        rel = np.linalg.norm(d) / np.linalg.norm(want)
        log(f"  rel fro {rel:.2e}")
        assert rel <= 3e-3, rel
    return cache


DECODE = [
    # lens, new, heads, group, dim, block, page, book
    ([1], [1], 1, 1, 64, 64, 16, "nf4"),
    ([63, 64, 65], [1, 1, 1], 2, 4, 128, 64, 16, "nf4"),
    ([255, 256, 257, 1], [1, 1, 1, 1], 1, 8, 128, 32, 32, "fp4"),
    ([700], [1], 1, 5, 128, 128, 16, "int4"),
    ([300, 0, 129], [1, 0, 1], 2, 16, 64, 32, 64, "nf4"),
    ([40, 333], [1, 1], 1, 20, 64, 64, 16, "int4"),
    ([270, 15], [1, 1], 2, 3, 256, 128, 16, "nf4"),
    ([200], [1], 1, 2, 256, 32, 128, "fp4"),
    ([100, 31], [1, 1], 1, 1, 256, 64, 16, "int4"),
]


@pytest.mark.parametrize("lens,new,heads,group,dim,block,page,book", DECODE, ids=str)
def test_decode(lens, new, heads, group, dim, block, page, book):
    require_gpu()
    log("attn decode", lens, heads, group, dim, block, page, book)
    check_attention(layout(lens, new, page, dim + group), heads, group, dim, block, book)


ROWS = [
    # lens, new, heads, group, dim, block, page, book, causal, window
    ([70, 9], [5, 9], 2, 4, 128, 64, 16, "nf4", True, 0),
    ([300], [300], 1, 2, 64, 64, 16, "nf4", True, 0),
    ([200, 31, 77], [180, 31, 1], 1, 3, 128, 32, 32, "int4", True, 0),
    ([290], [33], 1, 4, 256, 64, 16, "fp4", True, 0),
    ([150, 20], [150, 20], 2, 1, 128, 128, 64, "nf4", False, 0),
    ([40, 100], [7, 90], 1, 7, 64, 32, 16, "nf4", False, 0),
    ([300, 100], [1, 40], 1, 4, 128, 64, 16, "nf4", True, 50),
    ([280], [280], 1, 1, 64, 64, 16, "fp4", True, 1),
    ([333, 64], [64, 64], 2, 2, 128, 64, 32, "int4", True, 64),
    ([500], [3], 1, 8, 128, 64, 16, "nf4", True, 300),
]


@pytest.mark.parametrize("lens,new,heads,group,dim,block,page,book,causal,window", ROWS, ids=str)
def test_rows_masks_and_windows(lens, new, heads, group, dim, block, page, book, causal, window):
    require_gpu()
    log("attn rows", lens, new, heads, group, dim, block, page, book, causal, window)
    check_attention(layout(lens, new, page, dim + group), heads, group, dim, block, book, causal=causal, window=window)


def test_rows_without_a_token():
    """More rows than tokens: the first rows have negative positions and attend nothing."""
    require_gpu()
    for causal in (True, False):
        check_attention(layout([3, 0, 20], [5, 4, 24], 16, 1), 2, 2, 128, 64, "nf4", causal=causal)


def test_no_rows_no_sequences():
    require_gpu()
    h = layout([5, 7], [0, 0], 16, 1)
    cache, _, _ = fill_cache(h, 1, 64, 64, "nf4", 0)
    o = torch.full((3, 2, 64), 4.0, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros_like(o)
    Q.qlora_kv_attn(q, cache, device_batch(h), out=o)                         # sequences, none with a row
    none = Q.KVBatch(i32([0]), i32([]), torch.empty(0, 1, dtype=torch.int32, device="cuda"))
    Q.qlora_kv_attn(q, cache, none, out=o)                                    # no sequence
    Q.qlora_kv_read(cache, none, 3, o[:, :1], o[:, :1].clone())
    Q.qlora_kv_write(o[:, :1], o[:, :1], cache, none)
    assert torch.all(o == 4.0)
    assert Q.qlora_kv_attn(q[:0], cache, device_batch(h))[0].shape == (0, 2, 64)


@pytest.mark.parametrize("book", ["nf4", "int4"])
def test_strong_logits(book):
    """Logits of hundreds: the softmax is close to one-hot, and the running maximum moves between tiles."""
    require_gpu()
    check_attention(layout([600], [2], 16, 3), 1, 4, 128, 64, book, q_std=8.0, k_gain=8.0, fro=False)


def test_many_sequences():
    """More sequences than one pass of the scheduler's scan takes, with empty ones among them."""
    require_gpu()
    rng = np.random.default_rng(0)
    lens = [int(n) for n in rng.integers(0, 40, 700)]
    new = [int(min(n, m)) for n, m in zip(lens, rng.integers(0, 3, 700))]
    check_attention(layout(lens, new, 16, 2), 1, 2, 64, 64, "nf4")


def test_what_a_row_does_not_see_does_not_reach_it():
    """NaN in later tokens of the same call (stored with a NaN scale) stays with the rows that see them."""
    require_gpu()
    dim, n = 128, 40
    h = layout([n], [n], 16, 0)
    cache = Q.kv_alloc(h.pages, 16, 1, dim)
    x = dev_bf16(bits(1, (n, 1, dim)))
    v = dev_bf16(bits(2, (n, 1, dim)))
    batch = device_batch(h)
    Q.qlora_kv_write(x, v, cache, batch)
    q = dev_bf16(bits(3, (n, 4, dim)))
    ref, _ = Q.qlora_kv_attn(q, cache, batch)
    kb, vb = x.clone(), v.clone()
    kb[30] = float("nan")
    vb[20, 0, 70] = float("inf")
    Q.qlora_kv_write(kb, vb, cache, batch)
    o, _ = Q.qlora_kv_attn(q, cache, batch)
    assert torch.equal(o[:20], ref[:20])
    assert torch.equal(o[20:30, :, :64], ref[20:30, :, :64]) and torch.isnan(o[20:30, :, 64:]).all()
    assert torch.isnan(o[30:]).all()
    ow, _ = Q.qlora_kv_attn(q, cache, batch, window=5)
    refw = Q.qlora_kv_attn(q, cache, batch, window=5)[0]
    assert torch.equal(torch.nan_to_num(ow), torch.nan_to_num(refw))
    assert torch.isfinite(ow[35:]).all() and torch.isnan(ow[30:35]).all() and torch.isfinite(ow[25:30]).all()


def test_strided_q_and_output():
    require_gpu()
    h = layout([90, 31], [4, 2], 16, 5)
    cache, _, _ = fill_cache(h, 2, 128, 64, "nf4", 3)
    joint = dev_bf16(bits(8, (6, 8 * 128 + 64)))
    q = joint[:, 64:].unflatten(1, (8, 128))
    batch = device_batch(h)
    want, wl = Q.qlora_kv_attn(q.contiguous(), cache, batch, lse=True)
    out = torch.zeros(8, 6, 136, dtype=torch.bfloat16, device="cuda")[..., :128].transpose(0, 1)
    got, gl = Q.qlora_kv_attn(q, cache, batch, out=out, lse=True)
    assert got is out and torch.equal(got, want) and torch.equal(gl, wl)


def test_cache_past_32_bit_offsets():
    """A cache of more than 4 GiB of codes: pages at its end are found."""
    require_gpu()
    heads, dim, page = 8, 128, 1024
    pages = (5 << 30) // (heads * page * dim // 2)
    cache = Q.kv_alloc(pages, page, heads, dim)
    assert cache.k_codes.nbytes > 1 << 32
    n = 1500
    far = Q.KVBatch(i32([0, n]), i32([n]), i32([[pages - 1, pages - 2]]))
    near = Q.KVBatch(i32([0, n]), i32([n]), i32([[0, 1]]))
    k, v = dev_bf16(bits(1, (n, heads, dim))), dev_bf16(bits(2, (n, heads, dim)))
    q = dev_bf16(bits(3, (n, heads, dim)))
    res = []
    for b in (near, far):
        Q.qlora_kv_write(k, v, cache, b)
        res.append((Q.qlora_kv_attn(q[-3:], cache, Q.KVBatch(i32([0, 3]), b.length, b.table))[0],
                    *Q.qlora_kv_read(cache, b, n)))
    assert all(torch.equal(x, y) for x, y in zip(*res))
    assert torch.equal(cache.v_scale[pages - 1], cache.v_scale[0])


def test_same_bits_on_another_stream_and_with_one_workspace_for_two_calls():
    require_gpu()
    h = layout([900, 333, 50], [1, 1, 1], 16, 5)
    cache, _, _ = fill_cache(h, 1, 64, 64, "nf4", 3)
    batch = device_batch(h)
    q = [dev_bf16(bits(20 + i, (3, 8, 64))) for i in range(3)]
    want = [Q.qlora_kv_attn(x, cache, batch)[0] for x in q]
    ws = torch.empty(Q.qlora_kv_attn_workspace(cache, batch, 3, 8), dtype=torch.uint8, device="cuda").fill_(0xFF)
    for _ in range(3):
        got = [Q.qlora_kv_attn(x, cache, batch, workspace=ws)[0] for x in q]
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = [Q.qlora_kv_attn(x, cache, batch, stream=s)[0] for x in q]
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


# ---- all of it, as a decoding step uses it ----------------------------------------------------------------------
def _chain(x, lin, cache, batch, pos, freq, wq, wk, heads, kv_heads, dim, ws):
    """Projection -> norm and rotation -> cache -> attention -> projection."""
    w, A, B, wo, Ao, Bo = lin
    y, _ = Q.qlora_linear_fwd(x, w, A, B, 0.25, save_T=False, workspace=ws["lin"])
    q, k, v = y.split([heads * dim, kv_heads * dim, kv_heads * dim], 1)
    q, k, v = q.unflatten(1, (heads, dim)), k.unflatten(1, (kv_heads, dim)), v.unflatten(1, (kv_heads, dim))
    q, k = Q.qlora_qk_norm_rope(q, k, pos, freq, wq, wk)
    Q.qlora_kv_write(k, v, cache, batch)
    o, _ = Q.qlora_kv_attn(q, cache, batch, workspace=ws["attn"])
    return Q.qlora_linear_fwd(o.flatten(1), wo, Ao, Bo, 0.25, save_T=False, workspace=ws["lin2"])[0], q, k, v, o


def test_decoding_steps_eager_and_captured():
    """A prompt, then single tokens, of three sequences: the attention of every step against the oracle on the
    values that the cache holds, and the same steps replayed from one captured graph, whose lengths, positions
    and inputs change in place, bit for bit (three replays, with eager work between)."""
    require_gpu()
    torch.manual_seed(0)
    heads, kv_heads, dim, hidden, page, steps = 4, 2, 64, 256, 16, 4
    dev = torch.device("cuda", 0)
    r = lambda *s, std=0.05: (torch.randn(*s, device=dev) * std).bfloat16()
    width = (heads + 2 * kv_heads) * dim
    lin = (Q.qlora_quantize_nf4(r(width, hidden)), r(hidden, 8), r(8, width), Q.qlora_quantize_nf4(r(hidden, heads * dim)),
           r(heads * dim, 8), r(8, hidden))
    wq, wk = r(dim, std=1.0), r(dim, std=1.0)
    freq = torch.tensor(10000.0 ** (-np.arange(dim // 2) / (dim // 2)), dtype=torch.float32, device=dev)
    prompt = [13, 16, 31]
    table = torch.arange(12, device=dev).flip(0).to(torch.int32).view(3, 4)

    def fresh():
        c = Q.kv_alloc(12, page, kv_heads, dim)
        for t in (c.k_codes, c.v_codes, c.k_scale, c.v_scale):
            t.zero_()
        return c

    def workspaces(n, cache, batch):
        return {"lin": torch.empty(Q.qlora_fwd_workspace(n, hidden, width, 8), dtype=torch.uint8, device=dev),
                "lin2": torch.empty(Q.qlora_fwd_workspace(n, heads * dim, hidden, 8), dtype=torch.uint8, device=dev),
                "attn": torch.empty(Q.qlora_kv_attn_workspace(cache, batch, n, heads), dtype=torch.uint8, device=dev)}

    xp = r(sum(prompt), hidden, std=1.0)
    xs = [r(3, hidden, std=1.0) for _ in range(steps)]
    pos_p = torch.cat([torch.arange(n) for n in prompt]).cuda()
    bp = Q.KVBatch(i32(np.concatenate([[0], np.cumsum(prompt)])), i32(prompt), table)
    args = (freq, wq, wk, heads, kv_heads, dim)

    cache = fresh()
    y, q, k, v, o = _chain(xp, lin, cache, bp, pos_p, *args, workspaces(len(xp), cache, bp))
    eager = []
    all_k = [[k[s:e]] for s, e in zip(np.cumsum([0] + prompt)[:-1], np.cumsum(prompt))]
    all_v = [[v[s:e]] for s, e in zip(np.cumsum([0] + prompt)[:-1], np.cumsum(prompt))]
    for i in range(steps):
        lens = [n + i + 1 for n in prompt]
        b1 = Q.KVBatch(i32([0, 1, 2, 3]), i32(lens), table)
        y, q, k, v, o = _chain(xs[i], lin, cache, b1, i32(lens).long() - 1, *args, workspaces(3, cache, b1))
        eager.append((y, o))
        for b in range(3):
            all_k[b].append(k[b:b + 1])
            all_v[b].append(v[b:b + 1])
            vals = []
            for rows in (all_k[b], all_v[b]):
                u = host_u16(torch.cat(rows))
                vals.append(np.stack([[kv.row_values(*kv.quantize_row(u[t, hd], 64, "nf4"), "nf4")
                                       for hd in range(kv_heads)] for t in range(len(u))]))
            want, _, bound = kv.attention(kv.f64(host_u16(q[b:b + 1])), *vals, lens[b], dim ** -0.5)
            d = np.abs(host(o[b:b + 1].float()).astype(np.float64) - want)
            mag = np.abs(kv.f64(host_u16(q[b]))).sum(-1).max() * np.abs(vals[0]).max() * dim ** -0.5
            assert np.all(d <= (np.expm1(2 * TAB["nf4"] * mag) + P16 + TAB["nf4"]) * 1.02 * bound + 2.0 ** -8 * np.abs(want))

    # the same from a captured step
    cache2 = fresh()
    _chain(xp, lin, cache2, bp, pos_p, *args, workspaces(len(xp), cache2, bp))
    x, length = torch.zeros_like(xs[0]), i32(prompt)
    b1 = Q.KVBatch(i32([0, 1, 2, 3]), length, table)
    pos = torch.zeros(3, dtype=torch.int64, device=dev)
    ws = workspaces(3, cache2, b1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        yg, _, _, _, og = _chain(x, lin, cache2, b1, pos, *args, ws)
    for i in range(steps):
        length.add_(1)
        pos.copy_(length.long() - 1)
        x.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(og, eager[i][1]) and torch.equal(yg, eager[i][0]), f"replay {i}"
        (torch.randn(100, 100, device=dev) @ torch.randn(100, 100, device=dev)).sum().item()
    for a, b in ((cache.k_codes, cache2.k_codes), (cache.v_codes, cache2.v_codes), (cache.k_scale, cache2.k_scale)):
        assert torch.equal(a, b)
