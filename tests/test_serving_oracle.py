"""The oracle of the cache, the plan, attention and the norms, pinned on the CPU: hand values
and identities that do not come from its own code."""
import numpy as np
import pytest

from oracle import serving_oracle as S


def test_bf16_round():
    x = np.array([1.0, 1.0 + 2.0 ** -8, 1.0 + 3 * 2.0 ** -8, -3.14159, 0.0], np.float32)
    assert np.array_equal(S.bf16_round(x), np.array([1.0, 1.0, 1.0 + 2.0 ** -6, -3.140625, 0.0], np.float32))


def test_quant_hand_values():
    x = np.arange(64, dtype=np.float16)[None]          # 0 .. 63: s = fp16(4.2), m = 0
    c, s, m = S.kv4_quant(x)
    assert m[0, 0] == 0 and s[0, 0] == np.float16(4.2)
    assert c[0, 0, 0] == 0 and c[0, 0, 63] == 15 and c[0, 0, 3] == 1
    c, s, m = S.kv4_quant(np.full((1, 64), 2.5, np.float16))   # constant: exact
    assert s[0, 0] == 0 and m[0, 0] == np.float16(2.5) and not c.any()
    x = np.zeros((1, 64), np.float16)
    x[0, 7] = 2.0 ** -24                               # a scale that underflows
    c, s, m = S.kv4_quant(x)
    assert s[0, 0] == np.float16(2.0 ** -24) and c[0, 0, 7] == 1
    bad = np.zeros((1, 64), np.float32)
    bad[0, :3] = [np.nan, np.inf, -np.inf]
    c, s, m = S.kv4_quant(bad)
    assert m[0, 0] == -65504 and np.isfinite(s[0, 0])
    assert abs(S.kv4_values(c, s, m)[0, 0]) <= float(s[0, 0])


def test_quant_error_is_at_most_about_half_a_step():
    """|x - (m + s c)| <= s / 2 plus what rounding s and m to fp16 moves: s is off by at most
    2^-11 of itself (15 codes), m is exact for fp16 inputs; the clamp at 15 adds the same."""
    rng = np.random.default_rng(0)
    x = rng.normal(0, 1, (50, 3, 128)).astype(np.float16)
    c, s, m = S.kv4_quant(x)
    err = np.abs(S.kv4_values(c, s, m) - x.astype(np.float64)).reshape(50, 3, 2, 64)
    assert np.all(err <= s.astype(np.float64)[..., None] * (0.5 + 15 * 2.0 ** -11 + 1e-6))


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_layout_places_every_nibble_once(dim):
    """Writing one token changes exactly its own bytes, every code lands where the layout's
    formula says, and two tokens share no byte."""
    page, heads = 16, 2
    cache = np.zeros((2, heads, page * dim * 9 // 8), np.uint8)
    x = np.zeros((1, heads, dim), np.float16)
    x[0, 1] = np.tile(np.arange(16), dim // 16)
    S.kv4_write(cache, [16 + 5], x, x, page)
    assert not cache[0].any() and not cache[1, 0].any()   # another page; a head of zeros
    kc, vc, kp, vp = S.kv4_block(cache, 1, 1, page, dim)
    row = kc.reshape(page, dim // 2)
    assert not np.delete(row, 5, 0).any()
    nib = np.stack([row[5] & 15, row[5] >> 4], -1).reshape(4, dim // 32, 8)   # [c][s][j]
    assert np.array_equal(nib.transpose(1, 0, 2).reshape(-1), np.tile(np.arange(16), dim // 16))
    words = vc.reshape(page // 4, 16, 4, dim // 32)
    mine = words[1, :, 1]
    other = words.copy()
    other[1, :, 1] = 0
    assert not other.any()
    nib = np.stack([mine & 15, mine >> 4], -1).reshape(16, dim // 16)         # [n][j]
    assert np.array_equal(nib, np.tile(np.arange(16)[:, None], (1, dim // 16)))
    par = kp.view(np.float16).reshape(page, 2, dim // 64)
    assert np.all(par[5, 0] == 1) and np.all(par[5, 1] == 0)


def test_plan_hand_values():
    page, pages = 16, 100
    table = np.full((4, 4), -1, np.int32)
    table[0, :2], table[1, 0], table[2, :1] = [7, 9], 3, 5
    pool = np.array([20, 21, 22, 0, 0, 0], np.int32)
    r = S.kv_plan([1, -1, 17, 2], [32, 16, 15, 0], table, pool, 3, page, pages, 24)
    assert list(r["pool"][:5]) == [20, 21, 22, 3, 0]      # request 1's page on top
    assert list(r["table"][0]) == [7, 9, 3, -1]           # taken from the top
    assert list(r["table"][2]) == [5, 22, -1, -1]         # 15 + 17 = 32 tokens: one more page
    assert list(r["table"][3]) == [21, -1, -1, -1]
    assert list(r["lens_out"]) == [33, 0, 32, 2] and list(r["count_out"]) == [1, 0]
    assert list(r["cu"]) == [0, 1, 1, 18, 20]
    assert list(r["slots"][:3]) == [3 * 16, 5 * 16 + 15, 22 * 16] and list(r["slots"][18:]) == [336, 337, -1, -1, -1, -1]
    assert list(r["pos"][:3]) == [32, 15, 16] and list(r["pos"][20:]) == [0] * 4


def test_plan_refusals():
    table = np.full((4, 2), -1, np.int32)
    table[0, 0] = 1
    pool = np.array([4, 5], np.int32)
    r = S.kv_plan([40, 17, 1, 1], [10, 0, 0, 0], table, pool, 2, 16, 10, 60)
    # request 0 outgrows its row; 1 takes both pages; 2 and 3 find none
    assert list(r["lens_out"]) == [10, 17, 0, 0] and list(r["count_out"]) == [0, 3]
    assert list(r["slots"][:40]) == [-1] * 40 and r["slots"][40] == 5 * 16 and list(r["slots"][57:]) == [-1] * 3


def test_attention_identities():
    rng = np.random.default_rng(1)
    q = rng.normal(size=(3, 4, 64))
    k, v = rng.normal(size=(10, 2, 64)), rng.normal(size=(10, 2, 64))
    out, lse, mass, _ = S.attention(q, k, v, 10, 0.1)
    # one token: the output is its value; equal keys: the mean of the values
    o1, l1, _, _ = S.attention(q[:1], k[:1], v[:1], 1, 0.1)
    assert np.allclose(o1[0, 3], v[0, 1]) and np.allclose(l1[0, 3], 0.1 * (k[0, 1] @ q[0, 3]))
    o2, l2, _, _ = S.attention(q, np.repeat(k[:1], 10, 0), v, 10, 0.1)
    assert np.allclose(o2[2, 0], v[:, 0].mean(0)) and np.allclose(o2[0, 0], v[:8, 0].mean(0))
    # a window of one token; a row before the first token sees nothing
    o3, _, _, _ = S.attention(q, k, v, 10, 0.1, window=1)
    assert np.allclose(o3[0, 0], v[7, 0]) and np.allclose(o3[2, 2], v[9, 1])
    o4, l4, _, _ = S.attention(q, k, v, 2, 0.1)
    assert not o4[0].any() and np.all(np.isneginf(l4[0])) and np.allclose(o4[1, 0], v[0, 0])
    assert np.all(np.abs(out) <= mass + 1e-12)


def test_residual_norm_identities():
    rng = np.random.default_rng(2)
    h = rng.normal(size=(3, 50))
    one = np.ones(50)
    hh, y, _ = S.residual_norm(None, h, one, eps=0.0)
    assert np.array_equal(hh, h) and np.allclose((y * y).mean(-1), 1.0)
    x = rng.normal(size=(3, 50))
    hh, _, _ = S.residual_norm(x, h, one, post=2 * one, gate=0.5 * one, alpha=3.0, beta=-1.0, eps=0.0)
    assert np.allclose((((3.0 * h - hh)) ** 2).mean(-1), 1.0)
