"""Attention over the 4-bit cache with many rows of a sequence: the kernel for prompts, its parts joined, both kernels
in one call, and the wider tiles of the one for few rows.

Tolerance: as derived for single tokens, with three terms more.  Keys are rounded to fp16 after the multiplication with
their scale: 2^-11 more for a logit (values are so too, in place of the product that is rounded there).  A probability is held times 2^7 relative to a maximum
that may be up to 2^6 too small, so one that rounds as a subnormal is off by 2^-25 where the sum is at least 2^7, and
the value it meets is below 2 in units of the largest value scale so far: 2^-31 max|v| for each of n tokens.  A value
(level times scale) that is small beside the largest of its 64 tokens is off by 2^-25 of a unit that is at most the
largest scale, as is an element of a key: 2^-25 max|v| over all tokens, whose probabilities sum to 1, and
2^-25 scale sum|q| max|k| for a logit."""
import numpy as np
import pytest
import torch

import bit_nf4_quantized_11_amd as Q
from helpers import dev_bf16, host, log, require_gpu
from kv_cases import Host, bits, device_batch, fill_cache, i32, layout
from oracle import kv

pytestmark = pytest.mark.gpu

TAB = {"nf4": 2.0 ** -11, "fp4": 2.0 ** -22, "int4": 2.0 ** -22}
P16 = 2.0 ** -10
FAULT_START, FAULT_LENGTH, FAULT_PAGE = 1, 2, 4


def _word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def tolerance(h, q, ks, vs, group, book, scale, want, bound):
    """(tolerance of the outputs, of the logits) as above."""
    tol, err = np.zeros_like(want), np.zeros(want.shape[:2])
    for b, (n, m) in enumerate(zip(h.lens, h.new)):
        if not (n and m):
            continue
        r = slice(h.start[b], h.start[b + 1])
        qa, ka = np.abs(kv.f64(q[r])), np.repeat(np.abs(ks[b]), group, 1)
        mag = np.stack([(qa[:, x] @ ka[:, x].T).max(-1) for x in range(qa.shape[1])], 1)
        err[r] = scale * ((TAB[book] + 2.0 ** -11 + 2.0 ** -16) * mag + 2.0 ** -25 * qa.sum(-1) * ka.max())
        tol[r] = (np.expm1(2 * err[r])[..., None] + P16 + TAB[book]) * 1.02 * bound[r] + \
            1.02 * 2.0 ** -8 * np.abs(want[r]) + (n * 2.0 ** -31 + 2.0 ** -25) * np.abs(vs[b]).max()
    return tol, err


def check(h, heads, group, dim, block, book, seed=0, causal=True, window=0, q_std=1.0, k_gain=1.0, fro=True, cache=None):
    scale = dim ** -0.5
    cache, ks, vs = cache or fill_cache(h, heads, dim, block, book, seed, k_gain)
    rows = h.rows + 3
    q = bits(seed + 5, (rows, heads * group, dim), q_std)
    o = torch.full((rows, heads * group, dim), 9.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((rows, heads * group), 9.0, device="cuda")
    fault = _word()
    Q.qlora_kv_attn(dev_bf16(q), cache, device_batch(h, fault), scale, causal, window, out=o, lse=lse)
    assert fault.item() == 0
    assert torch.all(o[h.rows:] == 9.0) and torch.all(lse[h.rows:] == 9.0)
    got, gl = host(o.float()).astype(np.float64)[:h.rows], host(lse).astype(np.float64)[:h.rows]
    want, wl, bound = np.zeros_like(got), np.zeros_like(gl), np.zeros_like(got)
    for b in range(len(h.lens)):
        r = slice(h.start[b], h.start[b + 1])
        want[r], wl[r], bound[r] = kv.attention(kv.f64(q[r]), ks[b], vs[b], h.lens[b], scale, causal, window)
    tol, err = tolerance(h, q, ks, vs, group, book, scale, want, bound)
    d = np.abs(got - want)
    assert np.all(np.isfinite(got)) and np.all(d <= tol), (d.max(), (d / np.maximum(tol, 1e-300)).max())
    empty = np.isneginf(wl)
    assert np.array_equal(empty, np.isneginf(gl)) and np.all(got[empty] == 0)
    gl, wl = np.where(empty, 0, gl), np.where(empty, 0, wl)
    assert np.all(np.abs(gl - wl)[~empty] <= err[~empty] + 2.0 ** -20 * (1 + np.abs(wl[~empty])))
    if fro and np.linalg.norm(want) > 0:
        rel = np.linalg.norm(d) / np.linalg.norm(want)
        log(f"  rel fro {rel:.2e}")
        assert rel <= 3e-3, rel


MANY = [
    # lens, new, heads, group, dim, block, page, book, causal, window
    ([130], [130], 1, 1, 64, 64, 16, "nf4", True, 0),
    ([257], [257], 2, 1, 64, 32, 32, "fp4", True, 0),
    ([333, 129], [200, 129], 1, 3, 128, 128, 16, "int4", True, 0),
    ([190, 300, 65], [190, 100, 65], 2, 2, 128, 64, 64, "nf4", True, 0),
    ([260], [70], 1, 5, 128, 32, 16, "fp4", True, 0),
    ([150], [129], 1, 1, 256, 128, 16, "nf4", True, 0),
    ([97, 140], [97, 70], 1, 2, 256, 64, 32, "int4", True, 0),
    ([200], [40], 2, 4, 256, 32, 16, "nf4", True, 0),
    # one cached head for 20 query heads
    ([75], [30], 1, 20, 64, 64, 16, "int4", True, 0),
    # no mask; windows narrower than a tile, of one token, wider than the cache
    ([90, 201], [90, 80], 1, 2, 128, 64, 16, "nf4", False, 0),
    ([300], [300], 1, 1, 128, 64, 16, "nf4", True, 17),
    ([300], [280], 1, 2, 64, 32, 16, "int4", True, 1),
    ([200], [150], 1, 2, 256, 64, 64, "fp4", True, 100),
    ([260], [260], 1, 1, 128, 128, 128, "nf4", True, 5000),
    # the tokens of a tile in parts, joined: long caches under few tiles
    ([1500], [40], 1, 2, 128, 64, 64, "nf4", True, 0),
    ([1027], [70], 2, 1, 64, 32, 16, "fp4", True, 0),
    ([1027], [150], 2, 1, 64, 32, 16, "fp4", True, 0),
    ([800], [45], 1, 3, 64, 64, 64, "nf4", False, 0),
    ([900], [35], 1, 2, 256, 128, 128, "int4", False, 0),
    ([1400, 1, 600], [90, 1, 100], 1, 2, 128, 32, 16, "nf4", True, 700),
    ([2000], [66], 1, 1, 128, 64, 256, "int4", True, 64),
    ([2100], [230], 1, 1, 128, 32, 64, "int4", True, 0),
    ([2200, 2070], [120, 130], 1, 2, 64, 64, 64, "nf4", True, 0),
]


@pytest.mark.parametrize("lens,new,heads,group,dim,block,page,book,causal,window", MANY, ids=str)
def test_many_rows(lens, new, heads, group, dim, block, page, book, causal, window):
    require_gpu()
    log("attn many rows", lens, new, heads, group, dim, block, page, book, causal, window)
    check(layout(lens, new, page, dim + group), heads, group, dim, block, book, causal=causal, window=window)


WIDE = [
    # lens, new, heads, group, dim, block, page, book, window: tables long enough for tiles of 32 rows
    ([300, 80], [5, 9], 2, 4, 128, 64, 64, "nf4", 0),
    ([700, 1, 0, 333], [40, 1, 0, 33], 1, 1, 128, 32, 64, "fp4", 0),
    ([520], [3], 3, 8, 128, 128, 64, "int4", 0),
    ([100, 400], [20, 11], 2, 2, 64, 64, 64, "int4", 0),
    ([640, 31], [17, 31], 2, 1, 64, 32, 64, "nf4", 40),
]


@pytest.mark.parametrize("lens,new,heads,group,dim,block,page,book,window", WIDE, ids=str)
def test_tiles_of_32_rows(lens, new, heads, group, dim, block, page, book, window):
    require_gpu()
    log("attn wide tiles", lens, new, heads, group, dim, block, page, book, window)
    check(layout(lens, new, page, dim + group, spare_cols=4200), heads, group, dim, block, book, window=window)


@pytest.mark.parametrize("dim", [64, 128])
def test_many_rows_of_some_among_many_sequences(dim):
    """More sequences than one pass of the scan takes: most with a few rows, ten with many, so both kernels run."""
    require_gpu()
    rng = np.random.default_rng(1)
    lens = [int(n) for n in rng.integers(0, 30, 600)]
    new = [int(min(n, m)) for n, m in zip(lens, rng.integers(0, 3, 600))]
    for i in (0, 5, 255, 256, 300, 511, 512, 513, 577, 599):
        lens[i], new[i] = 470 + i % 7, 460
    check(layout(lens, new, 16, 2), 1, 8, dim, 64, "nf4")


@pytest.mark.parametrize("dim,rows", [(64, 300), (128, 300), (256, 300), (128, 200)], ids=str)
def test_one_prompt_among_single_tokens(dim, rows):
    """A low mean of rows with one sequence of many: both kernels, or the one for few rows alone."""
    require_gpu()
    rng = np.random.default_rng(6)
    lens = [int(n) for n in rng.integers(1, 90, 41)]
    new = [1] * 41
    lens[17], new[17] = rows + 30, rows
    check(layout(lens, new, 16, 6), 1, 4, dim, 64, "int4")


def test_capacities_near_the_largest():
    """Tables for 2^30 tokens a sequence, few of them used: the units of work get larger, so that their number fits 32
    bits.  Four pages of 2^20 tokens that 300 sequences share, single tokens; then some with many rows."""
    require_gpu()
    dim, page, cols = 64, 1 << 20, 1024
    four = layout([600] * 4, [600] * 4, 16, 3)          # (for its values alone)
    rng = np.random.default_rng(4)
    lens = [int(n) for n in rng.integers(1, 601, 300)]
    _, ks, vs = fill_cache(layout([600], [1], 16, 3), 1, dim, 64, "nf4", 11)
    cache = Q.kv_alloc(4, page, 1, dim)
    x = {}
    for t, seed in (("k", 11), ("v", 12)):
        x[t] = dev_bf16(np.concatenate([bits(seed, (600, 1, dim))] * 4))
    Q.qlora_kv_write(x["k"], x["v"], cache, Q.KVBatch(i32(four.start), i32([600] * 4), i32([[p] for p in range(4)])))
    for new in ([1] * 300, [120] * 3 + [1] * 297):
        n = [max(a, b) for a, b in zip(lens, new)]
        table = np.full((300, cols), 2 ** 31 - 1, np.int32)
        table[:, 0] = np.arange(300) % 4
        h = Host(n, new, np.concatenate([[0], np.cumsum(new)]).astype(np.int32), table, 4, page)
        check(h, 1, 4, dim, 64, "nf4", seed=5, cache=(cache, [ks[0][:a] for a in n], [vs[0][:a] for a in n]))


def test_rows_without_a_token():
    """More rows than tokens: the first rows have negative positions and attend nothing."""
    require_gpu()
    for causal in (True, False):
        check(layout([3, 0, 20], [150, 90, 80], 16, 1), 2, 2, 128, 64, "nf4", causal=causal)
        check(layout([64], [200], 16, 1), 1, 1, 256, 64, "nf4", causal=causal)


def test_windows_that_are_none():
    """The widest window there is, also where rows have negative positions, is no window."""
    require_gpu()
    h = layout([20, 150], [90, 100], 16, 1)
    cache, _, _ = fill_cache(h, 1, 64, 64, "nf4", 0)
    for n in (190, 6):
        q = dev_bf16(bits(3, (n, 2, 64)))
        batch = device_batch(h) if n == 190 else Q.KVBatch(i32([0, 4, 6]), i32([3, 150]), i32(h.table))
        want = Q.qlora_kv_attn(q, cache, batch, lse=True)
        for window in (2 ** 32 + 5, 2 ** 31 - 1, 2 ** 31 - 2, 2 ** 30, h.table.shape[1] * 16):
            got = Q.qlora_kv_attn(q, cache, batch, window=window, lse=True)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("book", ["nf4", "int4"])
def test_strong_logits(book):
    """The softmax is close to one-hot, and the maximum moves from tile to tile."""
    require_gpu()
    check(layout([700], [130], 16, 3), 1, 2, 128, 64, book, q_std=8.0, k_gain=8.0, fro=False)


@pytest.mark.parametrize("dim,block,new", [(64, 32, 1), (128, 64, 1), (256, 64, 1), (64, 64, 150), (128, 32, 150), (256, 128, 80)],
                         ids=str)
def test_scales_of_all_sizes(dim, block, new):
    """Key and value scales that change by powers of two up to 2^24 from token to token and from block to block,
    and values near both ends of the range."""
    require_gpu()
    n, heads = 200, 1
    for base in (0, 96, -80):
        h = layout([n], [new], 16, 4)
        rng = np.random.default_rng(dim + base + 100)
        shape = (h.pages, heads, 16)
        arr = {t + "c": np.full(shape + (dim // 2,), 0xFF, np.uint8) for t in "kv"}
        arr.update({t + "s": np.full(shape + (dim // block,), kv.NAN16, np.uint16) for t in "kv"})
        vals = {}
        for t in "kv":
            x = rng.integers(0, 16, (n, dim))
            e = rng.integers(-24, 1, (n, dim // block)) + (base if t == "v" else 0)
            s = ((127 + e) << 7 | rng.integers(0, 128, e.shape)).astype(np.uint16)
            vals[t] = np.stack([kv.row_values(x[p], s[p], "nf4") for p in range(n)])[:, None]
            for p in range(n):
                at = h.table[0, p // 16], 0, p % 16
                arr[t + "c"][at], arr[t + "s"][at] = kv.pack_row(x[p], t == "k"), s[p]
        dev = {k: torch.from_numpy(a).cuda() if a.dtype == np.uint8 else dev_bf16(a) for k, a in arr.items()}
        cache = Q.KVCache(dev["kc"], dev["ks"], dev["vc"], dev["vs"], block, 0)
        log("scales", dim, block, new, base)
        check(h, heads, 1, dim, block, "nf4", fro=False, cache=(cache, [vals["k"]], [vals["v"]]))


@pytest.mark.parametrize("dim,prefix", [(64, 0), (128, 0), (256, 0), (128, 1500), (128, 2000), (64, 2000), (256, 500)], ids=str)
def test_what_a_row_does_not_see_does_not_reach_it(dim, prefix):
    """NaN in later tokens of the same call stays with the rows and the blocks that see them, also where the tokens
    are attended in parts."""
    require_gpu()
    m, new = prefix, 120
    n = m + new
    h = layout([n], [new], 16, 0)
    cache = Q.kv_alloc(h.pages, 16, 1, dim)
    x, v = dev_bf16(bits(1, (n, 1, dim))), dev_bf16(bits(2, (n, 1, dim)))
    batch = device_batch(h)
    everything = Q.KVBatch(i32([0, n]), batch.length, batch.table)
    q = dev_bf16(bits(3, (new, 2, dim)))
    Q.qlora_kv_write(x, v, cache, everything)
    ref, refw = (Q.qlora_kv_attn(q, cache, batch, window=w)[0] for w in (0, 30))
    kb, vb = x.clone(), v.clone()
    kb[m + 90] = float("nan")
    vb[m + 40, 0, dim - 1] = float("inf")
    Q.qlora_kv_write(kb, vb, cache, everything)
    o, ow = (Q.qlora_kv_attn(q, cache, batch, window=w)[0] for w in (0, 30))
    cut = dim - 64
    assert torch.equal(o[:40], ref[:40])
    assert torch.equal(o[40:90, :, :cut], ref[40:90, :, :cut]) and torch.isnan(o[40:90, :, cut:]).all()
    assert torch.isnan(o[90:]).all()
    assert torch.equal(ow[:40], refw[:40]) and torch.isnan(ow[40:70, :, cut:]).all()
    assert torch.equal(ow[70:90], refw[70:90]) and torch.isnan(ow[90:]).all()


@pytest.mark.parametrize("dim", [64, 128])
def test_wrong_entries_are_reported(dim):
    """Pages, lengths and starts out of range: the bit set, NaN where a row needs what is not there, nothing else touched."""
    require_gpu()
    page, pages, rows = 16, 16, 150
    q = dev_bf16(bits(1, (rows, 2, dim)))
    x = dev_bf16(bits(2, (256, 1, dim)))
    cache = Q.kv_alloc(pages, page, 1, dim)
    good = np.arange(16)[None, :]
    Q.qlora_kv_write(x, x, cache, Q.KVBatch(i32([0, 256]), i32([256]), i32(good)))

    def run(start, length, table):
        fault = _word()
        o, lse = torch.full_like(q, 5.0), torch.full((rows, 2), 5.0, device="cuda")
        Q.qlora_kv_attn(q, cache, Q.KVBatch(i32(start), i32(length), i32(table), fault), out=o, lse=lse)
        return int(fault.item()), o.float(), lse

    ref = run([0, rows], [256], good)
    assert ref[0] == 0
    for bad in (pages, -1, -2 ** 31, 2 ** 31 - 1):      # the page of tokens 128 .. 143: rows 22 on see it
        t = good.copy()
        t[0, 8] = bad
        f, o, lse = run([0, rows], [256], t)
        assert f == FAULT_PAGE and torch.equal(o[:22], ref[1][:22]) and torch.isnan(o[22:]).all() and torch.isnan(lse[22:]).all()
    for bad in (257, -1, 2 ** 31 - 1):
        f, o, lse = run([0, rows], [bad], good)
        assert f == FAULT_LENGTH and torch.isnan(o).all() and torch.isnan(lse).all()
    for start in ([0, rows + 1], [-1, rows], [rows, 0], [0, 2 ** 31 - 1]):
        f, o, lse = run(start, [256], good)
        assert f == FAULT_START and torch.all(o == 5.0) and torch.all(lse == 5.0)
    # starts that go back: the rows of the sequences in order are done, some by two sequences with the same result: that
    # of three sequences of which two are empty (of one sequence alone another kernel may take the rows, other bits)
    three = run([0, rows, rows, rows], [256] * 3, np.repeat(good, 3, 0))
    assert three[0] == 0
    f, o, lse = run([0, rows, 0, rows], [256] * 3, np.repeat(good, 3, 0))
    assert f == FAULT_START and torch.equal(o, three[1]) and torch.equal(lse, three[2])


def test_strides_streams_and_one_workspace_for_two_calls():
    require_gpu()
    h = layout([900, 333], [100, 77], 16, 5)
    cache, _, _ = fill_cache(h, 2, 128, 64, "nf4", 3)
    batch = device_batch(h)
    joint = [dev_bf16(bits(8 + i, (177, 4 * 128 + 64))) for i in range(2)]
    q = [j[:, 64:].unflatten(1, (4, 128)) for j in joint]
    want = [Q.qlora_kv_attn(x.contiguous(), cache, batch, lse=True) for x in q]
    ws = torch.empty(Q.qlora_kv_attn_workspace(cache, batch, 177, 4), dtype=torch.uint8, device="cuda").fill_(0xFF)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for stream in (None, s, s):
        got = []
        for x in q:
            out = torch.zeros(6, 177, 136, dtype=torch.bfloat16, device="cuda")[:4, :, :128].transpose(0, 1)
            s.wait_stream(torch.cuda.current_stream())
            got.append(Q.qlora_kv_attn(x, cache, batch, out=out, lse=True, workspace=ws, stream=stream))
        s.synchronize()
        torch.cuda.synchronize()
        for (a, la), (b, lb) in zip(got, want):
            assert torch.equal(a, b) and torch.equal(la, lb)


def test_captured_prompts_with_one_workspace_for_two_graphs():
    """Two captured calls that share a workspace, replayed in turn with eager calls between, lengths, tables and rows
    changed in place: the same bits as eager calls."""
    require_gpu()
    heads, group, dim, page = 1, 2, 128, 16
    cases = [layout([600, 200], [90, 60], page, 1, spare_cols=10), layout([333, 700], [50, 100], page, 2, spare_cols=4)]
    cache, _, _ = fill_cache(layout([704, 704], [1, 1], page, 7, spare_pages=0), heads, dim, 64, "nf4", 0)
    cols = max(c.table.shape[1] for c in cases)
    tables = []
    for c in cases:
        t = np.full((2, cols), 2 ** 31 - 1, np.int32)
        t[:, :c.table.shape[1]] = c.table
        tables.append(i32(t))
    start, length, table = i32(cases[0].start), i32(cases[0].lens), tables[0].clone()
    batch = Q.KVBatch(start, length, table)
    qs = [dev_bf16(bits(30 + i, (160, heads * group, dim))) for i in range(2)]
    q = qs[0].clone()
    ws = torch.empty(Q.qlora_kv_attn_workspace(cache, batch, 160, heads * group), dtype=torch.uint8, device="cuda")
    outs = [torch.zeros_like(q) for _ in range(2)]
    lses = [torch.zeros(160, heads * group, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    graphs = []
    for i, window in enumerate((0, 150)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            Q.qlora_kv_attn(q, cache, batch, window=window, out=outs[i], lse=lses[i], workspace=ws)
        graphs.append(g)
    for step in range(4):
        c = cases[step % 2]
        start.copy_(i32(c.start))
        length.copy_(i32(c.lens))
        table.copy_(tables[step % 2])
        q.copy_(qs[(step // 2) % 2])
        eager = [Q.qlora_kv_attn(q, cache, batch, window=w, lse=True) for w in (0, 150)]
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(outs[i][:c.rows], eager[i][0][:c.rows]), step
            assert torch.equal(lses[i][:c.rows], eager[i][1][:c.rows]), step


def test_binding_refusals():
    """What the binding refuses before any launch."""
    require_gpu()
    cache = Q.kv_alloc(4, 16, 2, 64)
    batch = Q.KVBatch(i32([0, 3]), i32([3]), i32([[0, 1]]))
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    bad = [x.float(), x.cpu(), x[..., ::2], x[0], x[0, 0], x[0, 0, 0], torch.zeros(3, 3, 64, dtype=torch.bfloat16, device="cuda"),
           torch.zeros(3, 2, 128, dtype=torch.bfloat16, device="cuda")]
    for b in bad:
        with pytest.raises(Q.QLoRAError):
            Q.qlora_kv_write(b, x, cache, batch)
        with pytest.raises(Q.QLoRAError):
            Q.qlora_kv_write(x, b, cache, batch)
        with pytest.raises(Q.QLoRAError):
            Q.qlora_kv_read(cache, batch, 3, b, x)
        with pytest.raises(Q.QLoRAError):
            Q.qlora_kv_attn(b, cache, batch)
        with pytest.raises(Q.QLoRAError):
            Q.qlora_kv_attn(x, cache, batch, out=b)
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    for ws in (small, small.cpu(), torch.empty(1 << 20, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(Q.QLoRAError):
            Q.qlora_kv_attn(x, cache, batch, workspace=ws)
    for kw in ({"window": -1}, {"window": 5 - 2 ** 32}, {"window": 4, "causal": False}, {"lse": torch.zeros(3, 3, device="cuda")},
               {"lse": torch.zeros(3, 2, dtype=torch.bfloat16, device="cuda")}):
        with pytest.raises(Q.QLoRAError):
            Q.qlora_kv_attn(x, cache, batch, **kw)
    for args in (([0, 3], [3], [0, 1]), ([0], [3], [[0, 1]]), ([0, 3, 4], [3], [[0, 1]])):
        with pytest.raises(Q.QLoRAError):
            Q.KVBatch(*(i32(a) for a in args))
    with pytest.raises(Q.QLoRAError):
        Q.KVBatch(torch.tensor([0, 3], device="cuda"), i32([3]), i32([[0, 1]]))      # int64
    with pytest.raises(Q.QLoRAError):
        Q.KVBatch(i32([0, 3]).cpu(), i32([3]), i32([[0, 1]]))
    for shape in ((4, 24, 2, 64), (4, 8, 2, 64), (0, 16, 2, 64), (4, 16, 0, 64), (4, 16, 2, 96)):
        with pytest.raises(Q.QLoRAError):
            Q.kv_alloc(*shape)
    with pytest.raises(Q.QLoRAError):
        Q.kv_alloc(4, 16, 2, 64, 128)
