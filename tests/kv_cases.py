"""A random cache and batch for the cache and attention tests, on the host: what the device gets as
arrays and what it stands for in float64."""
from dataclasses import dataclass

import numpy as np
import torch

import bit_nf4_quantized_11_amd as Q
import workloads
from helpers import dev_bf16
from oracle import kv

CODEBOOKS = {"nf4": 0, "fp4": 1, "int4": 2}


def bits(seed, shape, std=1.0):
    return workloads.normal_bf16(seed, shape, std)


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


@dataclass
class Host:
    lens: list
    new: list
    start: np.ndarray
    table: np.ndarray
    pages: int
    page: int

    @property
    def rows(self):
        return int(self.start[-1])


def layout(lens, new, page, seed, spare_pages=2, spare_cols=1):
    """Pages dealt out at random, table entries past a sequence's end out of range."""
    rng = np.random.default_rng(seed)
    counts = [-(-n // page) for n in lens]
    pages = sum(counts) + spare_pages
    order = rng.permutation(pages)
    table = np.full((len(lens), max(counts + [1]) + spare_cols), 2 ** 31 - 1, np.int32)
    at = 0
    for b, c in enumerate(counts):
        table[b, :c] = order[at:at + c]
        at += c
    start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    return Host(list(lens), list(new), start, table, pages, page)


def device_batch(h: Host, fault=None):
    return Q.KVBatch(i32(h.start), i32(h.lens), i32(h.table), fault)


def fill_cache(h: Host, heads, dim, block, book, seed, k_gain=1.0):
    """A cache whose tokens are quantized normal values, NaN scales and 0xFF codes in every slot that
    holds none.  Returns (device cache, k [b] -> [len][heads][dim] float64, v likewise)."""
    shape = (h.pages, heads, h.page)
    arr = {t + "c": np.full(shape + (dim // 2,), 0xFF, np.uint8) for t in "kv"}
    arr.update({t + "s": np.full(shape + (dim // block,), kv.NAN16, np.uint16) for t in "kv"})
    values = {"k": [], "v": []}
    for b, n in enumerate(h.lens):
        for t in "kv":
            x = bits(seed + 10 * b + (t == "v"), (max(n, 1), heads, dim), k_gain if t == "k" else 1.0)
            out = np.zeros((n, heads, dim))
            for p in range(n):
                pg, off = h.table[b, p // h.page], p % h.page
                for hd in range(heads):
                    c, s = kv.quantize_row(x[p, hd], block, book)
                    arr[t + "c"][pg, hd, off] = kv.pack_row(c, t == "k")
                    arr[t + "s"][pg, hd, off] = s
                    out[p, hd] = kv.row_values(c, s, book)
            values[t].append(out)
    dev = {n: torch.from_numpy(a).cuda() if a.dtype == np.uint8 else dev_bf16(a) for n, a in arr.items()}
    cache = Q.KVCache(dev["kc"], dev["ks"], dev["vc"], dev["vs"], block, CODEBOOKS[book])
    return cache, values["k"], values["v"]
