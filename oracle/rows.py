"""Oracle: residual RMS norm, the gated block's activation and product, and log probabilities of given tokens, each
with its backward, in float64.

TEST INFRASTRUCTURE ONLY (see the package docstring).  Written from the definitions in the public header.
"""
from __future__ import annotations

import math

import numpy as np


def bf16(x) -> np.ndarray:
    """float64 of the bf16 value next to each fp32 value (ties to even)."""
    b = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    b = ((b + 0x7FFF + ((b >> 16) & 1)) >> 16 << 16).astype(np.uint32)
    return b.view(np.float32).astype(np.float64)


# ---- residual addition and norm ---------------------------------------------------------------------
def rms_norm(x, residual, w, eps):
    """(y, h): h is the bf16 of the fp32 sum."""
    h = x if residual is None else bf16(x.astype(np.float32) + residual.astype(np.float32))
    y = h / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    return (y if w is None else y * w), h


def rms_norm_bwd(dy, h, w, dh, eps):
    """(dx, dw) of <y, dy> + <h, dh>."""
    r = 1 / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    g = dy if w is None else dy * w
    dx = r * (g - h * r * r * (g * h).mean(-1, keepdims=True))
    return (dx if dh is None else dx + dh), (dy * h * r).sum(0)


# ---- gated block ----------------------------------------------------------------------------------------
def activation(g, kind):
    """(act(g), act'(g))."""
    if kind == "silu":
        s = 1 / (1 + np.exp(-g))
        return g * s, s * (1 + g * (1 - s))
    c = math.sqrt(2 / math.pi)
    # (1 + tanh t) / 2 as 1 / (1 + e^-2t): far below zero the sum 1 + tanh t has no digits left in float64
    s = 1 / (1 + np.exp(-2 * c * (g + 0.044715 * g ** 3)))
    return g * s, s + 2 * g * s * (1 - s) * c * (1 + 3 * 0.044715 * g * g)


def gated_bwd(dH, G, U, kind):
    """(dG, dU, H)."""
    a, slope = activation(G, kind)
    return dH * U * slope, dH * a, a * U


# ---- log probabilities ----------------------------------------------------------------------------------
def log_softmax(x):
    """Rows of -infinity stay so."""
    m = x.max(-1, keepdims=True)
    with np.errstate(divide="ignore", invalid="ignore"):
        d = np.where(m == -np.inf, x, x - m)
        z = np.exp(d).sum(-1, keepdims=True)
        return np.where(z == 0, x, d - np.log(z)), m[..., 0], z[..., 0]


def token_logprob(logits, token, scale, top):
    """(logprob, m, z, entropy, top_logprob, top_index); logits without NaN."""
    lp, m, z = log_softmax(logits * scale)
    rows = np.arange(len(logits))
    p = np.exp(lp)
    entropy = -np.where(p > 0, p * np.where(p > 0, lp, 0), 0).sum(-1)
    at = np.where(token >= 0, lp[rows, np.clip(token, 0, lp.shape[1] - 1)], 0.0)
    at = np.where(token >= lp.shape[1], np.nan, at)
    index = np.argsort(-logits, axis=1, kind="stable")[:, :top]
    return at, m, z, entropy, np.take_along_axis(lp, index, 1), index


def token_logprob_bwd(logits, token, scale, dlp, dent):
    """Gradient of <logprob, dlp> + <entropy, dent>; a row without a logit above -infinity has none."""
    lp, m, z = log_softmax(logits * scale)
    p = np.exp(lp)
    hit = np.zeros_like(p)
    given = (token >= 0) & (token < lp.shape[1])
    hit[np.nonzero(given)[0], token[given]] = 1
    g = np.where(given, 0.0 if dlp is None else dlp, 0.0)[:, None] * (hit - p)
    if dent is not None:
        plp = np.where(p > 0, p * np.where(p > 0, lp, 0), 0)
        entropy = -plp.sum(-1, keepdims=True)
        g = g - dent[:, None] * (plp + p * entropy)
    g[z == 0] = 0
    if dlp is not None:
        g[token >= lp.shape[1]] = np.nan
    return g * scale
