"""The 4-bit cache and its attention where ordinary data does not lead: rows of zeros and of infinities, scales at both
ends, entries behind a window, starts out of order, workspaces of other calls."""
import copy
import pickle

import numpy as np
import pytest
import torch

import bit_nf4_quantized_11_amd as Q
import test_gpu_kv_many as many
from helpers import dev_bf16, host, log, require_gpu
from kv_cases import Host, bits, device_batch, i32, layout
from oracle import kv

pytestmark = pytest.mark.gpu

FAULT_START, FAULT_LENGTH, FAULT_PAGE = 1, 2, 4


def _word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def written(h: Host, k16, v16, heads, dim, block):
    """A cache that holds k16, v16 [b] -> [len][heads][dim] (bf16 bits), and what its rows stand for in float64."""
    cache = Q.kv_alloc(h.pages, h.page, heads, dim, block)
    for t in (cache.k_scale, cache.v_scale):
        t.fill_(float("nan"))
    full = Q.KVBatch(i32(np.concatenate([[0], np.cumsum(h.lens)])), i32(h.lens), i32(h.table))
    Q.qlora_kv_write(*(dev_bf16(np.concatenate(x)) for x in (k16, v16)), cache, full)
    value = lambda x: np.stack([[kv.row_values(*kv.quantize_row(r, block, "nf4"), "nf4") for r in t] for t in x])
    return cache, [value(x) for x in k16], [value(x) for x in v16]


def against_oracle(h, q16, cache, ks, vs, causal=True, window=0, scale=None):
    """The attention of q16 [rows][q_heads][dim] within the tolerance derived for many rows (which holds for few)."""
    heads, dim = cache.heads, cache.head_dim
    scale = dim ** -0.5 if scale is None else scale
    fault = _word()
    o, lse = Q.qlora_kv_attn(dev_bf16(q16), cache, device_batch(h, fault), scale, causal, window, lse=True)
    assert fault.item() == 0
    got, gl = host(o.float()).astype(np.float64), host(lse).astype(np.float64)
    want, wl, bound = np.zeros_like(got), np.zeros_like(gl), np.zeros_like(got)
    for b in range(len(h.lens)):
        r = slice(h.start[b], h.start[b + 1])
        want[r], wl[r], bound[r] = kv.attention(kv.f64(q16[r]), ks[b], vs[b], h.lens[b], scale, causal, window)
    tol, err = many.tolerance(h, q16, ks, vs, q16.shape[1] // heads, "nf4", scale, want, bound)
    d = np.abs(got - want)
    assert np.all(np.isfinite(got)), np.argwhere(~np.isfinite(got))[:3]
    assert np.all(d <= tol), (d.max(), (d / np.maximum(tol, 1e-300)).max())
    empty = np.isneginf(wl)
    assert np.array_equal(empty, np.isneginf(gl)) and np.all(got[empty] == 0)
    assert np.all(np.abs(gl - wl)[~empty] <= err[~empty] + 2.0 ** -20 * (1 + np.abs(wl[~empty])))


ZERO = [
    # dim, block, lens, new, causal, window: the kernel for many rows (and, for the last, both)
    (64, 64, [150], [150], True, 0),
    (128, 64, [333], [200], True, 0),
    (256, 32, [130], [130], True, 0),
    (64, 32, [201], [140], False, 0),
    (128, 128, [201, 90], [80, 90], False, 0),
    (256, 64, [100], [70], False, 0),
    (128, 32, [300], [280], True, 17),
    (64, 64, [300], [140], True, 100),
    (128, 64, [1500], [40], True, 0),        # in parts
    (256, 128, [900], [35], False, 0),       # in parts
    (128, 64, [90, 150, 70], [1, 150, 3], True, 0),
]


@pytest.mark.parametrize("what", ["all", "tail", "tiny"])
@pytest.mark.parametrize("dim,block,lens,new,causal,window", ZERO, ids=str)
def test_zero_queries_over_zero_keys(dim, block, lens, new, causal, window, what):
    """All queries and keys zero; those of the last 70 rows and tokens (padding); or both so small (2^-75) that their product
    is no fp32 number.  Such rows attend what they see evenly."""
    require_gpu()
    log("zeros", dim, block, lens, new, causal, window, what)
    heads, group = 1, 2
    h = layout(lens, new, 16, dim + sum(new))
    std = 2.0 ** -75 if what == "tiny" else 1.0
    k = [bits(3 + b, (n, heads, dim), std) for b, n in enumerate(lens)]
    v = [bits(30 + b, (n, heads, dim)) for b, n in enumerate(lens)]
    q = bits(9, (h.rows, heads * group, dim), std)
    for b, n in enumerate(new):
        if what != "tiny":
            at = 0 if what == "all" else max(0, n - 70)
            q[h.start[b] + at:h.start[b + 1]] = 0
            k[b][0 if what == "all" else max(0, lens[b] - 70):] = 0
    against_oracle(h, q, *written(h, k, v, heads, dim, block), causal, window)


@pytest.mark.parametrize("dim,new", [(64, 1), (128, 5), (256, 1), (64, 150), (128, 150), (256, 80)], ids=str)
@pytest.mark.parametrize("scale", [1e-20, 2.0 ** -149, 2.0 ** 127], ids=str)
def test_scales_at_the_ends_of_their_range(dim, new, scale):
    """Rows of zeros, whose logits are zero under any scale; and under a tiny one, ordinary rows."""
    require_gpu()
    log("scale", dim, new, scale)
    h = layout([200], [new], 16, dim)
    k, v = ([bits(s, (200, 1, dim))] for s in (3, 4))
    q = bits(9, (new, 2, dim), 1.0 if scale < 1 else 0.0)
    q[::2] = 0
    against_oracle(h, q, *written(h, k, v, 1, dim, 64), scale=scale)


@pytest.mark.parametrize("dim,new", [(64, 3), (128, 3), (256, 3), (64, 150), (128, 150), (256, 80)], ids=str)
def test_infinite_queries(dim, new):
    """A row of q with an infinity has no softmax, also where every product is -infinity: NaN if it sees a token, nothing
    if it sees none, and no other row is touched."""
    require_gpu()
    n = new - 1                              # the first row has no token
    h = layout([n], [new], 16, dim)
    k, v = ([bits(s, (n, 1, dim))] for s in (3, 4))
    k[0][:, 0, 5] = 0x3F80                   # element 5 of every key is positive
    cache, _, _ = written(h, k, v, 1, dim, 64)
    q = bits(9, (new, 2, dim))
    batch = device_batch(h)
    ref, rl = Q.qlora_kv_attn(dev_bf16(q), cache, batch, lse=True)
    for value in (0xFF80, 0x7F80, 0x7FC0):
        x = q.copy()
        for row in (0, 1, new - 1):
            x[row, 1, 5] = value
        o, lse = Q.qlora_kv_attn(dev_bf16(x), cache, batch, lse=True)
        bad = torch.zeros(new, 2, dtype=torch.bool, device="cuda")
        bad[1, 1] = bad[new - 1, 1] = True
        assert torch.isnan(o[bad]).all() and torch.isnan(lse[bad]).all()
        assert torch.equal(o[~bad], ref[~bad]) and torch.equal(lse[~bad], rl[~bad])
        assert torch.all(o[0] == 0) and torch.isneginf(lse[0]).all()


def test_starts_that_go_back_stay_inside_the_workspace():
    """Starts that name the same 1500 rows eleven times: more tiles than the workspace of a call in order has room for
    when they are cut into parts.  They are left whole, nothing is written past the workspace, and the rows hold the result."""
    require_gpu()
    dim, page, rows, length = 128, 64, 1500, 4096
    one = layout([length], [rows], page, 5, spare_cols=0)
    q = bits(9, (rows, 1, dim))
    cache, ks, vs = written(one, [bits(3, (length, 1, dim))], [bits(4, (length, 1, dim))], 1, dim, 64)
    start = [0, rows] * 11
    n = len(start) - 1
    fault = _word()
    batch = Q.KVBatch(i32(start), i32([length] * n), i32(np.repeat(one.table, n, 0)), fault)
    need = Q.qlora_kv_attn_workspace(cache, batch, rows, 1)
    guarded = torch.full((need + (1 << 20),), 0xA5, dtype=torch.uint8, device="cuda")
    o, lse = Q.qlora_kv_attn(dev_bf16(q), cache, batch, lse=True, workspace=guarded[:need])
    assert fault.item() == FAULT_START
    assert torch.all(guarded[need:] == 0xA5)
    want, wl, bound = kv.attention(kv.f64(q), ks[0], vs[0], length, dim ** -0.5)
    tol, err = many.tolerance(one, q, ks, vs, 1, "nf4", dim ** -0.5, want, bound)
    assert np.all(np.abs(host(o.float()) - want) <= tol)
    assert np.all(np.abs(host(lse) - wl) <= err + 2.0 ** -20 * (1 + np.abs(wl)))


BEHIND = [
    # dim, page, lens, new, window: both kernels, with and without parts
    (128, 16, [777], [1], 100),
    (64, 32, [500, 90], [5, 2], 70),
    (256, 16, [300], [3], 33),
    (64, 16, [420], [150], 45),
    (128, 32, [730], [140], 90),
    (256, 16, [300], [70], 21),
    (128, 16, [1400, 1, 600], [90, 1, 100], 700),
]


def _first_seen(h, b, window):
    return max(0, h.lens[b] - h.new[b] + 1 - window)


@pytest.mark.parametrize("dim,page,lens,new,window", BEHIND, ids=str)
def test_pages_behind_the_window_may_be_gone(dim, page, lens, new, window):
    """Pages that lie behind the window of every row, given back and their entries set to -1, are not needed."""
    require_gpu()
    log("behind", dim, page, lens, new, window)
    h = layout(lens, new, page, dim)
    k, v = ([bits(s + b, (n, 1, dim)) for b, n in enumerate(lens)] for s in (3, 30))
    cache, ks, vs = written(h, k, v, 1, dim, 64)
    q = bits(9, (h.rows, 4, dim))
    want = Q.qlora_kv_attn(dev_bf16(q), cache, device_batch(h), window=window, lse=True)
    gone = 0
    for b in range(len(lens)):
        first = _first_seen(h, b, window) // page
        h.table[b, :first] = -1
        gone += first
    assert gone
    fault = _word()
    got = Q.qlora_kv_attn(dev_bf16(q), cache, device_batch(h, fault), window=window, lse=True)
    assert fault.item() == 0
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    against_oracle(h, q, cache, ks, vs, True, window)


@pytest.mark.parametrize("dim,page,lens,new,window", BEHIND, ids=str)
@pytest.mark.parametrize("what", [2.0 ** 40, float("nan")], ids=str)
def test_tokens_behind_the_window_do_not_reach_a_row(dim, page, lens, new, window, what):
    """Slots behind the window of every row may hold anything, far larger scales among it: the same bits."""
    require_gpu()
    h = layout(lens, new, page, dim)
    k, v = ([bits(s + b, (n, 1, dim)) for b, n in enumerate(lens)] for s in (3, 30))
    cache, _, _ = written(h, k, v, 1, dim, 64)
    q = dev_bf16(bits(9, (h.rows, 4, dim)))
    want = Q.qlora_kv_attn(q, cache, device_batch(h), window=window, lse=True)
    for b in range(len(lens)):
        for p in range(_first_seen(h, b, window)):
            at = int(h.table[b, p // page]), slice(None), p % page
            cache.k_scale[at] *= what
            cache.v_scale[at] *= what
    got = Q.qlora_kv_attn(q, cache, device_batch(h), window=window, lse=True)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


STARTS = [
    # start, the sequence whose row each of 24 rows is (-1: none; rows that several name are the first one's)
    ([0, 100, 5, 20, 24], [-1] * 5 + [2] * 15 + [3] * 4),             # one entry past the rows
    ([0, -3, 5, 20, 24], [-1] * 5 + [2] * 15 + [3] * 4),              # before them
    ([0, 10, 5, 20, 24], [0] * 10 + [2] * 10 + [3] * 4),              # out of order
    ([7, 2, 9, 9, 16], [-1] * 2 + [1] * 7 + [3] * 7 + [-1] * 8),      # back before the first
    ([0, 24, 3, 24, 24], [0] * 24),
    ([3, 3, 8, 12, 20], [-1] * 3 + [1] * 5 + [2] * 4 + [3] * 8 + [-1] * 4),
]


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("start,owner", STARTS, ids=str)
def test_a_wrong_start_leaves_the_other_sequences_alone(start, owner, dim):
    """Written and read: sequences whose own entries are in order have their rows, whatever stands before them."""
    require_gpu()
    rows, page, n = 24, 16, len(start) - 1
    x = {t: bits(i, (rows, 1, dim)) for i, t in enumerate("kv")}
    cache = Q.kv_alloc(2 * n, page, 1, dim)
    for t in (cache.k_codes, cache.v_codes, cache.k_scale, cache.v_scale):
        t.zero_()
    fault = _word()
    table = np.arange(2 * n).reshape(n, 2)
    batch = Q.KVBatch(i32(start), i32([30] * n), i32(table), fault)
    Q.qlora_kv_write(dev_bf16(x["k"]), dev_bf16(x["v"]), cache, batch)
    order = all(0 <= a <= b <= rows for a, b in zip(start, start[1:]))
    assert fault.item() == (0 if order else FAULT_START)
    out = [torch.full((rows, 1, dim), 7.0, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    Q.qlora_kv_read(cache, batch, rows, *out)
    slots = set()
    for i, b in enumerate(owner):
        if b < 0:
            assert torch.all(out[0][i] == 7.0) and torch.all(out[1][i] == 7.0), i
            continue
        p = 30 - (start[b + 1] - i)
        slots.add((int(table[b, p // page]), p % page))
        for t, o in zip("kv", out):
            want = kv.row_bf16(*kv.quantize_row(x[t][i, 0], 64, "nf4"), "nf4")
            assert np.array_equal(host(o[i, 0].view(torch.int16)).view(np.uint16), want), (i, t)
    held = torch.nonzero(cache.k_scale[:, 0, :, 0])
    assert {tuple(s) for s in held.tolist()} == slots


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_one_workspace_for_the_largest_call_and_smaller_ones(dim):
    """A workspace made for a prompt that is not cut into parts serves drafts, single tokens and short prompts, which are."""
    require_gpu()
    h = layout([2500, 300], [1, 1], 16, dim)
    k, v = ([bits(s + b, (n, 1, dim)) for b, n in enumerate(h.lens)] for s in (3, 30))
    cache, _, _ = written(h, k, v, 1, dim, 64)
    table = i32(h.table)
    need = Q.qlora_kv_attn_workspace(cache, Q.KVBatch(i32([0, 0, 0]), i32(h.lens), table), 40000, 4)
    guarded = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    for new in ([1, 1], [9, 3], [40, 0], [150, 100], [2500, 1]):
        rows = sum(new)
        batch = Q.KVBatch(i32(np.concatenate([[0], np.cumsum(new)])), i32(h.lens), table)
        q = dev_bf16(bits(9, (rows, 4, dim)))
        want = Q.qlora_kv_attn(q, cache, batch, lse=True)
        got = Q.qlora_kv_attn(q, cache, batch, lse=True, workspace=guarded[:need])
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert torch.all(guarded[need:] == 0xA5)


def test_one_workspace_for_the_largest_backward_and_smaller_ones():
    require_gpu()
    hq, hk, dim = 32, 32, 128
    need = Q.qlora_qk_norm_rope_bwd_workspace(2048, hq, hk, dim)
    guarded = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    w = [dev_bf16(bits(i, (dim,))) for i in (1, 2)]
    t = [dev_bf16(bits(3 + i, (2048, h, dim))) for i, h in enumerate((hq, hk, hq, hk))]
    for rows in (2048, 2047, 700, 1):
        args = [x[:rows] for x in t]
        want = Q.qlora_qk_norm_rope_bwd(*args, None, None, *w)
        got = Q.qlora_qk_norm_rope_bwd(*args, None, None, *w, workspace=guarded[:need])
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert torch.all(guarded[need:] == 0xA5)


def test_copies_and_pickles_of_a_cache_and_a_batch():
    """Copies have buffers of their own and describe those."""
    require_gpu()
    h = layout([40, 9], [3, 1], 16, 1)
    k, v = ([bits(s + b, (n, 1, 64)) for b, n in enumerate(h.lens)] for s in (3, 30))
    cache, _, _ = written(h, k, v, 1, 64, 32)
    batch = device_batch(h, _word())
    q = dev_bf16(bits(9, (h.rows, 2, 64)))
    want = Q.qlora_kv_attn(q, cache, batch)[0]
    copies = [(copy.deepcopy(cache), copy.deepcopy(batch)), pickle.loads(pickle.dumps((cache, batch)))]
    shared = copy.copy(cache), copy.copy(batch)
    assert shared[0].k_codes is cache.k_codes and shared[1].table is batch.table
    for c, b in copies + [shared]:
        assert (c.block, c.codebook, c.pages, c.heads, c.page_size, c.head_dim) == (32, 0, h.pages, 1, 16, 64)
        assert torch.equal(Q.qlora_kv_attn(q, c, b)[0], want)
    for c, b in copies:
        assert c.k_codes.data_ptr() != cache.k_codes.data_ptr() and b.table.data_ptr() != batch.table.data_ptr()
    for t in (cache.k_codes, cache.k_scale, cache.v_codes, cache.v_scale, batch.table):
        t.zero_()
    for c, b in copies:                      # (the first ones' buffers are not looked at)
        assert torch.equal(Q.qlora_kv_attn(q, c, b)[0], want)


def test_the_largest_batch():
    """65536 sequences of one token, attended and read back: the bits of calls with a thousand of them."""
    require_gpu()
    n, page, pages, dim = 65536, 64, 8, 64
    rng = np.random.default_rng(0)
    cache = Q.kv_alloc(pages, page, 1, dim)
    k, v = (dev_bf16(bits(s, (pages * page, 1, dim))) for s in (1, 2))
    Q.qlora_kv_write(k, v, cache, Q.KVBatch(i32([0, pages * page]), i32([pages * page]), i32([list(range(pages))])))
    lens, table = i32(rng.integers(1, page + 1, n)), i32(rng.integers(0, pages, (n, 1)))
    start = torch.arange(n + 1, dtype=torch.int32, device="cuda")
    q = dev_bf16(bits(3, (n, 2, dim)))
    fault = _word()
    batch = Q.KVBatch(start, lens, table, fault)
    o, lse = Q.qlora_kv_attn(q, cache, batch, lse=True)
    back = Q.qlora_kv_read(cache, batch, n)
    for i in range(0, n, 1024):
        part = Q.KVBatch(start[:1025], lens[i:i + 1024], table[i:i + 1024])
        po, pl = Q.qlora_kv_attn(q[i:i + 1024], cache, part, lse=True)
        assert torch.equal(o[i:i + 1024], po) and torch.equal(lse[i:i + 1024], pl), i
        for a, b in zip(back, Q.qlora_kv_read(cache, part, 1024)):
            assert torch.equal(a[i:i + 1024], b), i
    assert fault.item() == 0


@pytest.mark.parametrize("dim,new", [(64, [2, 3]), (128, [150, 1]), (256, [70, 80])], ids=str)
def test_rows_before_the_first_sequence_and_queries_of_one_row(dim, new):
    """Starts that begin behind row 0, rows behind the last one, and q broadcast over rows (a stride of 0)."""
    require_gpu()
    h = layout([200, 90], new, 16, dim)
    k, v = ([bits(s + b, (n, 1, dim)) for b, n in enumerate(h.lens)] for s in (3, 30))
    cache, _, _ = written(h, k, v, 1, dim, 64)
    rows = h.rows + 9
    one = dev_bf16(bits(9, (1, 4, dim)))
    ahead = Q.KVBatch(i32(h.start + 5), i32(h.lens), i32(h.table))
    o, lse = torch.full((rows, 4, dim), 6.0, dtype=torch.bfloat16, device="cuda"), torch.full((rows, 4), 6.0, device="cuda")
    Q.qlora_kv_attn(one.expand(rows, 4, dim), cache, ahead, out=o, lse=lse)
    want, wl = Q.qlora_kv_attn(one.expand(h.rows, 4, dim).contiguous(), cache, device_batch(h), lse=True)
    assert torch.equal(o[5:-4], want) and torch.equal(lse[5:-4], wl)
    for t in (o, lse):
        assert torch.all(t[:5] == 6.0) and torch.all(t[-4:] == 6.0)


@pytest.mark.parametrize("dim,batch", [(64, 1), (128, 3), (256, 2)])
def test_a_thousand_query_heads_of_one_cached_head(dim, batch):
    require_gpu()
    lens = [130, 1, 67][:batch]
    h = layout(lens, [1] * batch, 16, dim)
    k, v = ([bits(s + b, (n, 1, dim)) for b, n in enumerate(lens)] for s in (3, 30))
    against_oracle(h, bits(9, (batch, 1024, dim)), *written(h, k, v, 1, dim, 64))
