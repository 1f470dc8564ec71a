"""The operators between a projection and the next one: per-head norm and rotary positions of
queries and keys, the key/value cache held in 4 bits (written and read back), and the attention
that reads it.  Each in its plain form (elementary torch operations in 32 bits) and as the
library's calls, with the inputs that both take.

The cache: pages of `page` tokens; codes [pages][heads][page][D/2] bytes and one bf16 scale per
`block` elements, for keys and for values.  A dword of codes holds 8 consecutive elements: byte i
holds element i in its low and element i + 4 in its high nibble.  The dwords of a value row are in
element order; those of a key row are transposed, within 32 n elements (n = 4, or 2 where D = 64)
dword n*g + k holds elements 8*(4k + g) .. + 7, g < 4, k < n."""
import math

import torch

own = False

NAN = float("nan")

# levels in ascending order, as the fp32 values nearest to the decimals
LEVELS = {
    "nf4": [-1.0, -0.69619292, -0.525073051, -0.394917488, -0.284441352, -0.18477343, -0.0910499915, 0.0,
            0.0795803294, 0.160930172, 0.246112287, 0.337915182, 0.4407098, 0.562616944, 0.722956717, 1.0],
    "fp4": [-4 / 3, -1.0, -4 / 6, -3 / 6, -2 / 6, -1.5 / 6, -1 / 6, -0.5 / 6, 0.0, 0.5 / 6, 1 / 6, 1.5 / 6, 2 / 6,
            3 / 6, 4 / 6, 1.0],
    "int4": [k / 7 for k in range(-8, 8)],
}
CODEBOOK = {"nf4": 0, "fp4": 1, "int4": 2}


# ---- cases -------------------------------------------------------------------------------------
def _qk(op, tokens, q_heads, k_heads, dim, rot, norm, interleaved, far, name=None):
    case = dict(op=op, tokens=tokens, q_heads=q_heads, k_heads=k_heads, dim=dim, rot=rot, norm=norm,
                interleaved=interleaved, far=far)
    return dict(case, name=name) if name else case


def _kv(op, lens, new, q_heads, k_heads, dim, block, page, book, causal=True, window=0, name=None):
    case = dict(op=op, lens=lens, new=new, q_heads=q_heads, k_heads=k_heads, dim=dim, block=block, page=page,
                book=book, causal=causal, window=window)
    return dict(case, name=name) if name else case


def _text(values):
    return ",".join(str(v) for v in values)


def _ints(text):
    return [int(v) for v in text.split(",")]


def listed():
    return [
        # 16 sequences decode one token each, 65B head shapes: latency
        _qk("qk", 16, 64, 64, 128, 128, False, False, 4096, "rope_decode_16"),
        # a training batch behind 7B projections, with per-head norms
        _qk("qk", 4096, 32, 32, 128, 128, True, False, 4096, "qk_norm_rope_train_4096"),
        # its backward at 65B head shapes
        _qk("qk_bwd", 2048, 64, 64, 128, 128, True, False, 2048, "qk_norm_rope_bwd_2048"),
        # backward of a ragged batch: grouped heads, half of each head rotated, interleaved pairs, far positions
        _qk("qk_bwd", 1531, 24, 6, 64, 32, True, True, 1000000, "qk_norm_rope_bwd_ragged"),
        # one new token for each of 64 sequences written, and read back
        _kv("store", _text(range(100, 100 + 64 * 17, 17)), _text([1] * 64), 8, 8, 128, 64, 16, "nf4",
            name="kv_store_decode_64"),
        # prompts of a ragged batch written (7B heads, finer blocks), and read back
        _kv("store", "4096,1777,333,1,1985", "4096,1777,333,1,1985", 32, 32, 128, 32, 64, "fp4", name="kv_store_prompts"),
        # a cached prefix read back: small
        _kv("read", "515,77", "515,77", 8, 8, 64, 64, 16, "int4", name="kv_read_small"),
        # a long cached prefix read back
        _kv("read", "16384,9001", "16384,9001", 16, 16, 128, 64, 256, "nf4", name="kv_read_long"),
        # decode, one sequence, short cache: latency
        _kv("attn", "777", "1", 32, 8, 128, 64, 16, "nf4", name="kv_attn_decode_1"),
        # decode, a ragged batch with long caches, grouped heads
        _kv("attn", "32768,30011,16384,12000,32001,8192,501,20480,28000,32768,1,25013,16001,4096,31000,19999",
            _text([1] * 16), 64, 8, 128, 64, 64, "nf4", name="kv_attn_decode_16_long"),
        # drafted tokens checked, 8 sequences, one cached head for each query head (7B), sliding window
        _kv("attn", "5000,4097,6100,333,2048,8191,64,3001", _text([5, 3, 8, 1, 4, 5, 7, 2]), 32, 32, 128, 32, 32, "int4",
            window=2048, name="kv_attn_draft_8"),
        # prompts attended through the cache that they were written to
        _kv("attn", "4096,1500,2600", "4096,1000,2600", 32, 8, 128, 64, 64, "nf4", name="kv_attn_prompt"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["qk", "qk_bwd", "store", "read", "attn", "attn", "attn"])
    dim = rng.choice([64, 128, 128, 256])
    if op in ("qk", "qk_bwd"):
        k_heads = rng.choice([1, 2, 3, 4, 8, 16])
        q_heads = k_heads * rng.choice([1, 2, 4, 5])
        tokens = _log(rng, 1, max(1, min(4096, (1 << 25) // ((q_heads + k_heads) * dim))))
        norm = rng.random() < 0.7
        rot = rng.choice([dim, dim, dim // 2, 32])
        return _qk(op, tokens, q_heads, k_heads, dim, rot, norm, rng.random() < 0.4, rng.choice([4096, 200000, 1000000]))
    book = rng.choice(["nf4", "nf4", "fp4", "int4"])
    block = rng.choice([b for b in (32, 64, 64, 128) if b <= dim])
    page = rng.choice([16, 32, 64, 256])
    k_heads = rng.choice([1, 2, 4, 5, 8])
    q_heads = k_heads * rng.choice([1, 2, 3, 4, 6, 8])
    batch = _log(rng, 1, 32)
    if op != "attn":
        lens = [_log(rng, 1, 12000 // batch + 1) for _ in range(batch)]
        new = list(lens) if op == "read" or rng.random() < 0.5 else [_log(rng, 1, n) for n in lens]
        return _kv(op, _text(lens), _text(new), q_heads, k_heads, dim, block, page, book)
    form = rng.choice(["decode", "decode", "draft", "prompt"])
    if form == "prompt":
        batch = min(batch, 4)
        lens = [_log(rng, 16, 3500) for _ in range(batch)]
        new = [min(n, _log(rng, 16, 3000)) for n in lens]
    else:
        lens = [_log(rng, 1, 120000 // batch) for _ in range(batch)]
        new = [1 if form == "decode" else min(n, rng.randint(1, 9)) for n in lens]
    causal = rng.random() < 0.85
    window = rng.choice([0, 0, 0, 100, 1000]) if causal else 0
    return _kv(op, _text(lens), _text(new), q_heads, k_heads, dim, block, page, book, causal, window)


def work(case):
    dim = case["dim"]
    if case["op"] in ("qk", "qk_bwd"):
        rows = case["tokens"] * (case["q_heads"] + case["k_heads"])
        weights = 2 * dim if case["norm"] else 0
        table = case["tokens"] * 8 + case["rot"] * 2
        if case["op"] == "qk":
            return {"bytes": rows * dim * 4 + weights * 2 + table, "flops": rows * (4 * dim * case["norm"] + 3 * case["rot"])}
        # the saved inputs are only needed where there is a norm
        reads = 4 if case["norm"] else 2
        return {"bytes": rows * dim * (reads + 2) + weights * 6 + table,
                "flops": rows * (9 * dim * case["norm"] + 3 * case["rot"])}
    lens, new = _ints(case["lens"]), _ints(case["new"])
    per_token = 2 * case["k_heads"] * (dim // 2 + 2 * (dim // case["block"]))   # cache bytes, keys and values
    values = 2 * case["k_heads"] * dim * 2
    tables = sum(-(-n // case["page"]) for n in lens) * 4 + 8 * len(lens) + 4
    if case["op"] == "store":
        return {"bytes": sum(new) * (2 * values + 2 * per_token) + tables, "flops": sum(new) * values * 4}
    if case["op"] == "read":
        return {"bytes": sum(new) * (values + per_token) + tables, "flops": sum(new) * values // 2}
    pairs = seen = 0
    for length, n in zip(lens, new):
        first, last = length - n, length - 1
        lo = max(0, first + 1 - case["window"]) if case["window"] else 0
        seen += length - lo
        if not case["causal"]:
            pairs += n * length
        else:
            pairs += sum(min(p + 1, case["window"]) if case["window"] else p + 1 for p in range(first, last + 1))
    return {"bytes": seen * per_token + sum(new) * case["q_heads"] * dim * 4 + tables,
            "flops": 4 * dim * case["q_heads"] * pairs}


# ---- the 4-bit format, plain ---------------------------------------------------------------------
def _levels(book, device, dtype=torch.float32):
    return torch.tensor(LEVELS[book], dtype=torch.float32, device=device).to(dtype)


def _key_order(dim, device):
    """Position of each dword (8 elements) of a key row."""
    n = min(dim, 128) // 32
    e = torch.arange(dim // 8, device=device)
    r = e % (4 * n)
    return e - r + (r % 4) * n + r // 4


def _encode(x, block, book):
    """bf16 [..., D] -> (codes [..., D] as whole numbers, scale [..., D / block] bf16)."""
    lv = _levels(book, x.device, torch.float64)
    mid = (lv[1:] + lv[:-1]) / 2
    near = mid.float()
    thr = torch.where(near.double() > mid, torch.nextafter(near, torch.full_like(near, -2.0)), near)
    b = x.float().unflatten(-1, (-1, block))
    a = b.abs().amax(-1, keepdim=True)
    a = torch.where(a < 2.0 ** -126, torch.zeros_like(a), a)
    inv = torch.where(a > 0, (1.0 / a.double()).float(), torch.zeros_like(a))
    # the product of a bf16 and an fp32 value is exact in 64 bits: rounded to 32 once
    y = (b.double() * inv.double()).float()
    codes = torch.bucketize(y, thr)   # the number of thresholds below y: ties go to the lower code
    return codes.flatten(-2), a.squeeze(-1).bfloat16()


def _pack(codes, key):
    c = codes.to(torch.uint8).unflatten(-1, (-1, 8))
    if key:
        order = _key_order(codes.shape[-1], codes.device)
        out = torch.empty_like(c)
        out[..., order, :] = c
        c = out
    return (c[..., :4] | (c[..., 4:] << 4)).flatten(-2)


def _unpack(data, key):
    """Packed rows [..., D/2] -> codes [..., D]."""
    b = data.unflatten(-1, (-1, 4))
    c = torch.cat([b & 15, b >> 4], -1)
    if key:
        c = c[..., _key_order(2 * data.shape[-1], data.device), :]
    return c.flatten(-2)


def _values(data, scale, book, key):
    """fp32 values [..., D] that packed rows stand for."""
    lv = _levels(book, data.device)
    c = lv[_unpack(data, key).int()].unflatten(-1, (scale.shape[-1], -1))
    return (c * scale.float().unsqueeze(-1)).flatten(-2)


# ---- inputs ----------------------------------------------------------------------------------------
def _normal(gen, shape, std=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * std).bfloat16()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dim, hq, hk = case["dim"], case["q_heads"], case["k_heads"]
    state = {"case": case}
    if case["op"] in ("qk", "qk_bwd"):
        n = case["tokens"]
        # q, k as a joint projection leaves them: slices of one row
        joint = _normal(gen, (n, (hq + hk) * dim), 1.5)
        state["q"], state["k"] = joint[:, :hq * dim].view(n, hq, dim), joint[:, hq * dim:].view(n, hk, dim)
        state["pos"] = torch.randint(0, case["far"], (n,), generator=gen, device="cuda")
        half = case["rot"] // 2
        state["freq"] = torch.tensor([10000.0 ** (-i / half) for i in range(half)], dtype=torch.float32, device="cuda")
        state["wq"] = (1 + 0.2 * torch.randn(dim, generator=gen, device="cuda")).bfloat16() if case["norm"] else None
        state["wk"] = (1 + 0.2 * torch.randn(dim, generator=gen, device="cuda")).bfloat16() if case["norm"] else None
        if case["op"] == "qk_bwd":
            state["dq"], state["dk"] = _normal(gen, (n, hq, dim)), _normal(gen, (n, hk, dim))
        if own:
            import bit_nf4_quantized_11_amd as Q
            state["Q"] = Q
            if case["op"] == "qk_bwd":
                state["ws"] = torch.empty(Q.qlora_qk_norm_rope_bwd_workspace(n, hq, hk, dim), dtype=torch.uint8,
                                          device="cuda")
        return state
    lens, new = _ints(case["lens"]), _ints(case["new"])
    page, block = case["page"], case["block"]
    counts = [-(-n // page) for n in lens]
    pages = sum(counts) + 3
    rows = sum(new)
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.zeros((len(lens), max(counts)), dtype=torch.int32, device="cuda")
    at = 0
    for b, c in enumerate(counts):
        table[b, :c] = order[at:at + c]
        at += c
    start = [0]
    for n in new:
        start.append(start[-1] + n)
    state.update(table=table, start=torch.tensor(start, dtype=torch.int32, device="cuda"),
                 length=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    shape = (pages, hk, page)
    for t in "kv":
        # what a torch.empty cache may hold in slots that nothing was written to yet
        state[t + "_codes"] = torch.full(shape + (dim // 2,), 0x99, dtype=torch.uint8, device="cuda")
        state[t + "_scale"] = torch.full(shape + (dim // block,), NAN, dtype=torch.bfloat16, device="cuda")
    # keys have a few strong channels
    gain = 1 + 3 * (torch.rand(hk, 1, dim, generator=gen, device="cuda") < 0.03).float()
    if case["op"] == "store":
        state["k"] = (torch.randn(rows, hk, dim, generator=gen, device="cuda") * gain[:, 0]).bfloat16()
        state["v"] = _normal(gen, (rows, hk, dim))
    else:
        step = max(1, (1 << 24) // (hk * page * dim))
        for t in "kv":
            for p in range(0, pages, step):
                x = torch.randn((min(step, pages - p),) + shape[1:] + (dim,), generator=gen, device="cuda")
                x = (x * gain).bfloat16() if t == "k" else x.bfloat16()
                codes, scale = _encode(x, block, case["book"])
                state[t + "_codes"][p:p + step] = _pack(codes, t == "k")
                state[t + "_scale"][p:p + step] = scale
        # slots behind each sequence's end hold nothing
        for b, (n, c) in enumerate(zip(lens, counts)):
            if n % page:
                last = int(table[b, c - 1])
                state["k_scale"][last, :, n % page:] = NAN
                state["v_scale"][last, :, n % page:] = NAN
    if case["op"] == "attn":
        state["q"] = _normal(gen, (rows, hq, dim), 1.5)
    if own:
        import bit_nf4_quantized_11_amd as Q
        state["Q"] = Q
        state["cache"] = Q.KVCache(state["k_codes"], state["k_scale"], state["v_codes"], state["v_scale"], block,
                                   CODEBOOK[case["book"]])
        state["batch"] = Q.KVBatch(state["start"], state["length"], table)
        if case["op"] == "attn":
            state["ws"] = torch.empty(Q.qlora_kv_attn_workspace(state["cache"], state["batch"], rows, hq),
                                      dtype=torch.uint8, device="cuda")
    return state


# ---- plain forms --------------------------------------------------------------------------------------
def _turn(x, cos, sin, interleaved, back=False):
    """x [n][heads][D] rotated; cos, sin [n][1][R/2]."""
    rot = 2 * cos.shape[-1]
    if back:
        sin = -sin
    r, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([r, rest], -1)


def _angles(state):
    # angles of far positions need 64 bits
    t = state["pos"].double()[:, None] * state["freq"].double()
    return t.cos().float()[:, None], t.sin().float()[:, None]


EPS = 1e-6


def _run_qk(state):
    case = state["case"]
    cos, sin = _angles(state)
    out = []
    for x, w in ((state["q"], state["wq"]), (state["k"], state["wk"])):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
        out.append(_turn(x, cos, sin, case["interleaved"]).bfloat16())
    return out


def _run_qk_bwd(state):
    case = state["case"]
    cos, sin = _angles(state)
    grads, weights = [], []
    for x, w, dy in ((state["q"], state["wq"], state["dq"]), (state["k"], state["wk"], state["dk"])):
        g = _turn(dy.float(), cos, sin, case["interleaved"], True)
        if w is not None:
            x = x.float()
            r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
            weights.append((g * x * r).sum((0, 1)))
            g = g * w.float()
            g = r * (g - x * (r * r) * (g * x).mean(-1, keepdim=True))
        grads.append(g.bfloat16())
    return grads + weights


def _slots(state):
    """Page and offset of every row."""
    rows = torch.arange(sum(_ints(state["case"]["new"])), device="cuda")
    seq = torch.searchsorted(state["start"][1:], rows, right=True)
    p = state["length"][seq] - state["start"][seq + 1] + rows
    page = state["case"]["page"]
    return state["table"][seq, p // page].long(), p % page


def _read_back(state):
    page, offset = _slots(state)
    book = state["case"]["book"]
    return [_values(state[t + "_codes"][page, :, offset], state[t + "_scale"][page, :, offset], book, t == "k").bfloat16()
            for t in "kv"]


def _run_store(state):
    case = state["case"]
    page, offset = _slots(state)
    for t in "kv":
        codes, scale = _encode(state[t], case["block"], case["book"])
        state[t + "_codes"][page, :, offset] = _pack(codes, t == "k")
        state[t + "_scale"][page, :, offset] = scale
    return _read_back(state)


def _run_attn(state):
    case = state["case"]
    lens, new = _ints(case["lens"]), _ints(case["new"])
    hk, dim = case["k_heads"], case["dim"]
    group = case["q_heads"] // hk
    out = torch.empty_like(state["q"])
    at = 0
    for b, (length, n) in enumerate(zip(lens, new)):
        pages = state["table"][b, :-(-length // case["page"])].long()
        kv = []
        for t in "kv":   # [heads][length][D]
            x = _values(state[t + "_codes"][pages], state[t + "_scale"][pages], case["book"], t == "k")
            kv.append(x.transpose(0, 1).reshape(hk, -1, dim)[:, :length])
        k, v = kv
        v = v.contiguous()
        kt = k.transpose(1, 2).contiguous()
        key = torch.arange(length, device="cuda")
        step = max(1, (1 << 28) // (case["q_heads"] * length))
        for i in range(0, n, step):
            m = min(step, n - i)
            q = state["q"][at + i:at + i + m].float().view(m, hk, group, dim).permute(1, 0, 2, 3).reshape(hk, m * group, dim)
            s = torch.matmul(q, kt) * (1 / math.sqrt(dim))
            pos = torch.arange(length - n + i, length - n + i + m, device="cuda").repeat_interleave(group)[:, None]
            if case["causal"]:
                hidden = key > pos
                if case["window"]:
                    hidden |= key <= pos - case["window"]
                s = s.masked_fill(hidden, -math.inf)
            p = torch.exp(s - s.amax(-1, keepdim=True))
            o = torch.matmul(p, v) / p.sum(-1, keepdim=True)
            out[at + i:at + i + m] = o.view(hk, m, group, dim).permute(1, 0, 2, 3).reshape(m, -1, dim).bfloat16()
        at += n
    return out


def run(state):
    case = state["case"]
    op = case["op"]
    if not own:
        return {"qk": _run_qk, "qk_bwd": _run_qk_bwd, "store": _run_store, "read": _read_back, "attn": _run_attn}[op](state)
    Q = state["Q"]
    if op == "qk":
        return list(Q.qlora_qk_norm_rope(state["q"], state["k"], state["pos"], state["freq"], state["wq"], state["wk"],
                                         eps=EPS, interleaved=case["interleaved"]))
    if op == "qk_bwd":
        g = Q.qlora_qk_norm_rope_bwd(state["dq"], state["dk"], state["q"], state["k"], state["pos"], state["freq"],
                                     state["wq"], state["wk"], eps=EPS, interleaved=case["interleaved"],
                                     workspace=state["ws"])
        return [t for t in g if t is not None]
    if op == "store":
        Q.qlora_kv_write(state["k"], state["v"], state["cache"], state["batch"])
        return list(Q.qlora_kv_read(state["cache"], state["batch"], state["k"].shape[0]))
    if op == "read":
        return list(Q.qlora_kv_read(state["cache"], state["batch"], sum(_ints(case["new"]))))
    return Q.qlora_kv_attn(state["q"], state["cache"], state["batch"], causal=case["causal"], window=case["window"],
                           workspace=state["ws"])[0]


# ---- the definitions in 64 bits ---------------------------------------------------------------------------
def _exact_levels(book):
    """fp32 levels from their definitions: normal quantiles with the tails pulled in, E2M1 sixths, sevenths."""
    if book == "nf4":
        q = 0.9677083
        pos = torch.special.ndtri(torch.linspace(q, 0.5, 9, dtype=torch.float64)[:-1])
        neg = -torch.special.ndtri(torch.linspace(q, 0.5, 8, dtype=torch.float64)[:-1])
        lv = torch.cat([pos, neg, torch.zeros(1, dtype=torch.float64)]).sort().values
        lv = lv / lv.abs().max()
    elif book == "fp4":
        half = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
        lv = torch.tensor([-8.0] + [-h for h in half[:0:-1]] + half, dtype=torch.float64) / 6
    else:
        lv = torch.arange(-8, 8, dtype=torch.float64) / 7
    return lv.float().double().cuda()


def _exact_rows(data, scale, book, key):
    """float64 values of packed rows, element by element: which byte and which nibble holds it."""
    dim = data.shape[-1] * 2
    lv = _exact_levels(book)
    byte, shift = [], []
    for d in range(dim):
        word, j = divmod(d, 8)
        if key:
            n = 2 if dim == 64 else 4
            section, r = divmod(word, 4 * n)
            word = section * 4 * n + n * (r % 4) + r // 4
        byte.append(4 * word + j % 4)
        shift.append(4 * (j // 4))
    code = (data[..., torch.tensor(byte, device="cuda")] >> torch.tensor(shift, dtype=torch.uint8, device="cuda")) & 15
    return lv[code.long()] * scale.double().repeat_interleave(dim // scale.shape[-1], -1)


def _exact_quantized(x, block, book):
    """The value each element stands for once stored: nearest level of the block's share, ties to the lower."""
    lv = _exact_levels(book)
    b = x.double().unflatten(-1, (-1, block))
    a = b.abs().amax(-1, keepdim=True)
    # the definition rounds the reciprocal and the share to 32 bits
    share = (b * torch.where(a > 0, 1.0 / a, torch.zeros_like(a)).float().double()).float().double()
    best = torch.zeros_like(share)
    gap = torch.full_like(share, math.inf)
    for level in lv:
        d = (share - level).abs()
        nearer = d < gap
        best = torch.where(nearer, level, best)
        gap = torch.where(nearer, d, gap)
    return (best * a).flatten(-2)


def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    op = case["op"]
    if op in ("qk", "qk_bwd"):
        angle = s["pos"].double()[:, None, None] * s["freq"].double()
        turn = torch.polar(torch.ones_like(angle), angle)
        rot = case["rot"]

        def rotate(x, turn):
            r = x[..., :rot]
            if case["interleaved"]:
                z = torch.view_as_real(torch.view_as_complex(r.unflatten(-1, (-1, 2)).contiguous()) * turn).flatten(-2)
            else:
                z = torch.complex(r[..., :rot // 2].contiguous(), r[..., rot // 2:].contiguous()) * turn
                z = torch.cat([z.real, z.imag], -1)
            return torch.cat([z, x[..., rot:]], -1)

        outs, weights = [], []
        for t in "qk":
            x, w = s[t].double(), s["w" + t]
            inv = 1 / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS)
            if op == "qk":
                outs.append(rotate(x if w is None else x * inv * w.double(), turn))
                continue
            g = rotate(s["d" + t].double(), turn.conj())
            if w is not None:
                hat = x * inv
                weights.append((g * hat).sum(1).sum(0))
                g = g * w.double()
                g = inv * (g - hat * (g * hat).mean(-1, keepdim=True))
            outs.append(g)
        return outs + weights
    page = case["page"]
    lens, new = _ints(case["lens"]), _ints(case["new"])
    if op == "store":
        return [_exact_quantized(s[t], case["block"], case["book"]) for t in "kv"]
    outs = {"k": [], "v": [], "o": []}
    group = case["q_heads"] // case["k_heads"]
    at = 0
    for b, (length, n) in enumerate(zip(lens, new)):
        pages = s["table"][b, :-(-length // page)].long()
        o = torch.empty((n, case["q_heads"], case["dim"]), dtype=torch.float64, device="cuda") if op == "attn" else None
        heads = {"k": [], "v": []}
        for h in range(case["k_heads"]):
            k, v = (_exact_rows(s[t + "_codes"][pages, h].flatten(0, 1)[:length],
                                s[t + "_scale"][pages, h].flatten(0, 1)[:length], case["book"], t == "k") for t in "kv")
            if op == "read":
                heads["k"].append(k[length - n:])
                heads["v"].append(v[length - n:])
                continue
            key = torch.arange(length, device="cuda")
            pos = torch.arange(length - n, length, device="cuda")[:, None]
            seen = key <= pos if case["causal"] else torch.ones((n, length), dtype=torch.bool, device="cuda")
            if case["window"]:
                seen = seen & (key + case["window"] > pos)
            for g in range(h * group, (h + 1) * group):
                logit = s["q"][at:at + n, g].double() @ k.t() / math.sqrt(case["dim"])
                o[:, g] = torch.softmax(logit.masked_fill(~seen, -math.inf), -1) @ v
        at += n
        if op == "read":
            for t in "kv":
                outs[t].append(torch.stack(heads[t], 1))
        else:
            outs["o"].append(o)
    return [torch.cat(outs[t]) for t in "kv"] if op == "read" else torch.cat(outs["o"])
