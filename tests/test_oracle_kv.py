"""The oracle of the head norms, rotation, cache and attention against what mathematics fixes."""
import numpy as np
import pytest

from oracle import kv, nf4


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_rotation(interleaved):
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 2, 64))
    pos, freq = np.array([0, 1, 7, 1000, 123456]), (10000.0 ** (-np.arange(16) / 16)).astype(np.float32)
    y = kv.rotate(x, pos, freq, interleaved)
    assert np.array_equal(y[0], x[0]) and np.array_equal(y[..., 32:], x[..., 32:])
    np.testing.assert_allclose((y * y).sum(-1), (x * x).sum(-1), rtol=1e-12)
    np.testing.assert_allclose(kv.rotate(y, pos, freq, interleaved, -1.0), x, atol=1e-12)
    # the product of two rotated vectors depends on the distance of their positions alone
    a, b = x[:, 0], x[:, 1]
    d1 = (kv.rotate(a[:, None], pos + 3, freq, interleaved) * kv.rotate(b[:, None], pos, freq, interleaved)).sum(-1)
    d2 = (kv.rotate(a[:, None], pos * 0 + 3, freq, interleaved) * b[:, None]).sum(-1)
    np.testing.assert_allclose(d1, d2, atol=1e-9)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_norm_rope_gradient_against_differences(norm, interleaved):
    rng = np.random.default_rng(1)
    x, dy = rng.standard_normal((3, 2, 64)), rng.standard_normal((3, 2, 64))
    w = 1 + 0.3 * rng.standard_normal(64) if norm else None
    pos, freq = np.array([3, 50, 900]), (100.0 ** (-np.arange(24) / 24)).astype(np.float32)
    dx, dw = kv.norm_rope_bwd(dy, x, w, pos, freq, 1e-3, interleaved)
    f = lambda x, w: (kv.norm_rope(x, w, pos, freq, 1e-3, interleaved) * dy).sum()
    h = 1e-5
    for _ in range(20):
        d = rng.standard_normal(x.shape)
        num = (f(x + h * d, w) - f(x - h * d, w)) / (2 * h)
        assert abs(num - (dx * d).sum()) <= 1e-7 * max(1.0, abs(num))
    if norm:
        d = rng.standard_normal(w.shape)
        num = (f(x, w + h * d) - f(x, w - h * d)) / (2 * h)
        assert abs(num - (dw * d).sum()) <= 1e-7 * max(1.0, abs(num))


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_key_order_is_a_permutation_within_blocks_of_its_section(dim):
    order = [kv.key_dword(e, dim) for e in range(dim // 8)]
    assert sorted(order) == list(range(dim // 8))
    codes = np.random.default_rng(dim).integers(0, 16, dim)
    for key in (False, True):
        assert np.array_equal(kv.unpack_row(kv.pack_row(codes, key), key), codes)


@pytest.mark.parametrize("book", ["nf4", "fp4", "int4"])
@pytest.mark.parametrize("block", [32, 64, 128])
def test_row_format_is_the_weight_quantizers(book, block):
    x = nf4.f32_to_bf16(np.random.default_rng(2).standard_normal(256).astype(np.float32))
    ref = nf4.quantize(x.reshape(1, 256), False, codebook=book, block=block)
    codes, scales = kv.quantize_row(x, block, book)
    assert np.array_equal(codes, nf4.unpack_nibbles(ref["codes"], 256))
    assert np.array_equal(nf4.bf16_to_f32(scales), nf4.blockwise_absmax(x.reshape(1, 256), block))
    assert np.array_equal(kv.pack_row(codes, False), ref["codes"])


def test_blocks_of_zeros_and_of_non_finite_values():
    x = np.zeros(64, np.uint16)
    x[3], x[40] = 0x7F80, 0x0001
    codes, scales = kv.quantize_row(x, 32, "nf4")
    assert list(scales) == [kv.NAN16, 0] and set(codes) == {7}
    assert np.all(kv.row_bf16(codes, scales, "nf4")[:32] == kv.NAN16)
    assert np.all(kv.row_bf16(codes, scales, "nf4")[32:] == 0)


def test_attention_of_what_is_seen():
    rng = np.random.default_rng(3)
    k, v, q = rng.standard_normal((9, 2, 8)), rng.standard_normal((9, 2, 8)), rng.standard_normal((3, 4, 8))
    o, lse, _ = kv.attention(q, k, v, 9, 0.3)
    for i in range(3):
        o1, l1, _ = kv.attention(q[i:i + 1], k[:7 + i], v[:7 + i], 7 + i, 0.3)   # the same row as the last of a shorter cache
        np.testing.assert_allclose(o[i], o1[0], rtol=1e-13)
        np.testing.assert_allclose(lse[i], l1[0], rtol=1e-13)
    ow, _, _ = kv.attention(q, k, v, 9, 0.3, window=1)
    np.testing.assert_allclose(ow, np.repeat(v[6:9], 2, axis=1))      # one token seen: its value
    oe, le, be = kv.attention(rng.standard_normal((4, 4, 8)), k[:2], v[:2], 2, 0.3)
    assert np.all(oe[:2] == 0) and np.all(le[:2] == -np.inf) and np.all(oe[2] != 0)   # more rows than tokens
