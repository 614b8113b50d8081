"""Calls of the 4-bit cache's operators at the ends of what their documentation allows: row
buffers shorter than the requests' rows, memory that no token was written to inside a page that
is read, scores near the ends of fp32.  Tolerances as in test_gpu_kv4.py."""
import numpy as np
import pytest

from oracle import serving_oracle as S
from tests import gpu_util as U
from tests import test_gpu_kv4 as K

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def L():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    from weight_activation_quantized_amd import mixllm
    return mixllm


def call(L, q, dev, table, lens, cu, page, max_rows, max_len, scale, window=0):
    """Attention of the rows q [T], whatever cu says; out and lse as they are left."""
    out = torch.full_like(q, 9.0)
    lse = torch.full(q.shape[:2], 9.0, device="cuda")
    size = L.mixllm_kv4_attention_workspace_bytes(q.shape[0], len(lens), q.shape[1], dev.shape[1], q.shape[2], max_rows,
                                                  max_len, window)
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda") if size else None
    L.mixllm_kv4_attention(q, dev, K.cuda(table), K.i32(lens), K.i32(cu), out, page, max_rows, max_len, scale=scale,
                           window=window, lse=lse, workspace=ws)
    return out, lse


@pytest.mark.parametrize("before", [0, 2994])
@pytest.mark.parametrize("window", [0, 5])
@pytest.mark.parametrize("group", [1, 4])
def test_rows_behind_the_buffer_do_not_move_the_others(L, before, window, group):
    """10 rows, of which 8 fit: they have the positions of the first 8, and the two tokens that no
    row wrote (their memory holds NaN) are not seen.  A request all behind the buffer is left out."""
    U.say("attention rows behind the buffer", before, window, group)
    n, dtype = before + 8, torch.float16
    dev, table, kv = K.build([n, 20], 2, 128, 16, dtype, 61)
    q = K.rounded(np.random.default_rng(4).normal(size=(8, 2 * group, 128)).astype(np.float32), dtype)
    # the table's rows as they stand: two more tokens stay inside the request's last page
    assert (n + 2 + 15) // 16 == (n + 15) // 16
    out, lse = call(L, K.cuda(q, dtype), dev, table, [n + 2, 20], [0, 10, 13], 16, 10, n + 2, 0.1, window)
    K.compare(out, lse, q, kv, [n], [8], dtype, 0.1, window)


def test_row_bounds_far_behind_the_buffer(L):
    """Row bounds that saturate, as a plan of too many tokens leaves them."""
    U.say("attention saturated bounds")
    dtype = torch.bfloat16
    dev, table, kv = K.build([40, 30], 2, 64, 16, dtype, 62)
    q = K.rounded(np.random.default_rng(4).normal(size=(3, 4, 64)).astype(np.float32), dtype)
    for cu, window in (([0, 1, 2 ** 31 - 1], 0), ([0, 1, 2 ** 31 - 1], 2 ** 30 - 1)):
        out, lse = call(L, K.cuda(q, dtype), dev, table, [40, 30], cu, 16, 2000, 40, 0.1, window)
        K.compare(out[:1], lse[:1], q[:1], kv, [40], [1], dtype, 0.1, window)
        # the second request's rows stand far before its first token: they see nothing
        assert not out[1:].any() and torch.isneginf(lse[1:]).all()
    for cu in ([0, 1, 1], [2 ** 31 - 1] * 3, [5, 9, 12]):
        out, lse = call(L, K.cuda(q, dtype), dev, table, [40, 30], cu, 16, 2000, 40, 0.1)
        K.compare(out[:cu[1] if cu[0] == 0 else 0], lse, q, kv, [40], [1 if cu[0] == 0 else 0], dtype, 0.1)
        assert torch.all(out[1 if cu[0] == 0 else 0:] == 9.0)


@pytest.mark.parametrize("dim,heads,rows", [(64, 2, 1), (64, 8, 3), (128, 2, 1), (128, 8, 1), (128, 16, 1), (128, 8, 40),
                                            (256, 2, 1), (256, 8, 5)])
@pytest.mark.parametrize("length", [300, 3000])
def test_tokens_before_the_window_need_not_be_written(L, dim, heads, rows, length):
    """Only the tokens that a row sees are in the cache (a long prompt under a window appends no
    others): the memory before them, in the same page, holds NaN.  The rows are those of a
    cache that has all tokens, bit for bit."""
    U.say("attention unwritten tokens before the window", dim, heads, rows, length)
    window, dtype = 77, torch.float16
    dev, table, kv = K.build([length], 2, dim, 64, dtype, 63)
    first = length - rows - window + 1
    assert first % 16                              # inside a run of 16 tokens, and of a page
    pos = np.arange(first, length)
    slots = K.i32(table[0, pos // 64] * 64 + pos % 64)
    k = torch.zeros((len(pos), 2, dim), dtype=dtype, device="cuda")
    v = torch.zeros_like(k)
    holes = torch.full_like(dev, 255)
    # the seen tokens' own bytes, from the definition of the cache's layout
    part = np.full(holes.shape, 255, np.uint8)
    kk, vv = K.key_values(length, 2, dim, dtype, 63 * 100)
    S.kv4_write(part, slots.tolist(), kk[first:], vv[first:], 64)
    holes.copy_(torch.from_numpy(part))
    L.mixllm_kv4_read(holes, slots, k, v, 64)
    assert torch.isfinite(k).all() and torch.isfinite(v).all()
    q = K.cuda(K.rounded(np.random.default_rng(5).normal(size=(rows, heads, dim)).astype(np.float32), dtype), dtype)
    full = call(L, q, dev, table, [length], [0, rows], 64, rows, length, 0.1, window)
    for t in (table, np.where(np.arange(table.shape[1]) < first // 64, -1, table)):
        got = call(L, q, holes, t, [length], [0, rows], 64, rows, length, 0.1, window)
        assert torch.equal(got[0], full[0]) and torch.equal(got[1], full[1])
    K.compare(*full, q.float().cpu().numpy(), kv, [length], [rows], dtype, 0.1, window,
              picks=lambda n: {0, n // 2, n - 1})


def constant_keys(n, heads, dim, dtype, level, vscale, seed):
    """Keys that are one number per token (held exactly: s = 0), values of a given size."""
    k = np.broadcast_to(np.asarray(level, np.float64)[:, None, None], (n, heads, dim)).astype(np.float32)
    v = vscale * (np.random.default_rng(seed).normal(size=(n, heads, dim)) + 0.3)
    return k, K.rounded(v.astype(np.float32), dtype)


def cached(L, k, v, dtype, page=16):
    n, heads, dim = k.shape
    pages = -(-n // page) + 1
    cache = torch.full((pages, heads, page * dim * 9 // 8), 255, dtype=torch.uint8, device="cuda")
    L.mixllm_kv4_append(K.cuda(k, dtype), K.cuda(v, dtype), K.i32(np.arange(n)), cache, page)
    return cache, np.arange(pages, dtype=np.int32)[None], S.kv4_values(*S.kv4_quant(v))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("vscale", [2.0 ** -19, 0.002, 0.1, 3.0, 9000.0])
@pytest.mark.parametrize("dim,heads", [(64, 8), (128, 8), (256, 4)])
def test_scores_of_any_size(L, dtype, vscale, dim, heads):
    """Scores from 1e6 to 1e14, where a step of fp32 is larger than a power that keeps weights in
    fp16.  The tokens with the largest key share its score to the last bit, all others are so far
    below that their weights are zero: the output is the mean of 1 or 2 values.  Everything
    before the output's rounding is a sum of at most two terms with weights that are powers of
    two: 4 fp32 roundings of |m| + 15 s, and for the values' sum the two fp16 operands' 2^-22
    (fp16) or one operand's 2^-11 (bf16) of its s c where a weight times a scale is subnormal: a
    step of 2^-24 beside 2^-24 of the smallest scale, less than one step of its code: s.
    lse: the score, 2 D + 16 roundings of equal terms of one sign."""
    U.say("attention large scores", dtype, vscale, dim, heads)
    n = 700
    level = np.full(n, 100.0)
    level[200:400] = 700.0                       # the running maximum moves by large steps
    level[[450, 451, 452]] = [800.0, 900.0, 1000.0]
    level[[500, 650]] = 1200.0                   # the largest, in two places
    k, v = constant_keys(n, 2, dim, dtype, level, vscale, 5)
    cache, table, vv = cached(L, k, v, dtype)
    c, s, m = S.kv4_quant(v)
    most = np.repeat(15 * s.astype(np.float64) + np.abs(m.astype(np.float64)), 64, -1).reshape(v.shape)
    step = np.repeat(s.astype(np.float64), 64, -1).reshape(v.shape)
    q = np.full((1, heads, dim), 2000.0, np.float32)
    for upto, tops in ((700, [500, 650]), (600, [500])):
        for e in range(-8, 20, 2):
            scale = 2.0 ** e * 128 / dim
            out, lse = call(L, K.cuda(q, dtype), cache, table, [upto], [0, 1], 16, 1, upto, scale)
            k16 = K.rounded(np.float32([1200.0]), dtype).astype(np.float64)[0]
            score = scale * dim * 2000.0 * k16
            o = out.float().cpu().numpy().astype(np.float64)[0].reshape(2, heads // 2, dim)
            want, f = vv[tops].mean(0)[:, None], torch.finfo(dtype)
            tol = 4 * 2.0 ** -24 * most[tops].max(0)[:, None] + 2.0 ** -11 * step[tops].max(0)[:, None] * 15
            tol = tol + f.eps / 2 * (np.abs(want) + tol) + float(f.smallest_normal) * f.eps / 2
            err = np.abs(o - want)
            assert np.all(err <= tol), (upto, e, (err / tol).max())
            ls = lse.cpu().numpy().astype(np.float64)
            assert np.all(np.abs(ls - score) <= (2 * dim + 20) * 2.0 ** -24 * score + 1), (upto, e)


@pytest.mark.parametrize("top,scale", [(119.9, 0.0884), (119.9, 0.99), (100, 2.0 ** 19), (-90, 2.0 ** 119)])
@pytest.mark.parametrize("dim,heads", [(64, 8), (128, 2), (128, 40)])
def test_queries_to_the_ends_of_their_range(L, top, scale, dim, heads):
    """bf16 queries up to 2^120 and scales up to it: over keys of zero every score is zero, and the
    outputs are the mean of the values; keys that bring the scores back to ordinary sizes give
    ordinary results."""
    U.say("attention large queries", top, scale, dim, heads)
    dtype, n, rows = torch.bfloat16, 300, 2
    rng = np.random.default_rng(6)
    g = rng.normal(size=(rows, heads, dim))
    q = K.rounded((2.0 ** top * g / np.abs(g).max()).astype(np.float32), dtype)
    for level in (np.zeros(n), np.where(np.arange(n) % 3 == 1, 2.0 ** -24, 0.0)):
        if level.any() and top + np.log2(scale) > 30:
            continue                                # no fp16 key makes these scores small
        k, v = constant_keys(n, 1, dim, dtype, level, 0.7, 7)
        cache, table, vv = cached(L, k, v, dtype)
        c, s, m = S.kv4_quant(v)
        vmost = np.repeat(15 * s.astype(np.float64) + np.abs(m.astype(np.float64)), 64, -1).reshape(v.shape)
        kv = [[k.astype(np.float64), np.abs(k).astype(np.float64), vv, vmost]]
        out, lse = call(L, K.cuda(q, dtype), cache, table, [n], [0, rows], 16, rows, n, scale)
        K.compare(out, lse, q, kv, [n], [rows], dtype, scale)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_a_large_scale_and_small_queries(L, dtype):
    """scale 2^115 with bf16 queries of 2^-115, 2^14 with fp16 ones of 2^-14: ordinary scores."""
    e = 115 if dtype == torch.bfloat16 else 14
    U.say("attention large scale", dtype)
    dev, table, kv = K.build([90], 2, 128, 16, dtype, 64)
    q = K.rounded((np.random.default_rng(3).normal(size=(3, 8, 128)) * 2.0 ** -e).astype(np.float32), dtype)
    out, lse = call(L, K.cuda(q, dtype), dev, table, [90], [0, 3], 16, 3, 90, 0.1 * 2.0 ** e)
    K.compare(out, lse, q, kv, [90], [3], dtype, 0.1 * 2.0 ** e)


@pytest.mark.parametrize("hq,hkv,dim", [(32, 8, 128), (24, 3, 64), (16, 2, 256)])
def test_bf16_outputs_of_single_rows_are_nearly_rounded(L, hq, hkv, dim):
    """At most one in 20 is another number than the exact output rounded once.  What the two
    operands of a weight add is 9e-5 of an output's size (see the fp16 test of the same name): beside
    a step of 2^-8 to 2^-7 of the value, on average 0.0054, and an error of 0.8 of its root mean
    square on average, a share a / x of the outputs of size x, a = 0.8 9e-5 / 0.0054 = 0.013, and
    over normally distributed ones 0.8 a (1 + ln(1 / a)) = 5.6%, less what is lost above x = 1: 5%.
    A weight in one operand adds more than twice of that."""
    lens = [100] * 12
    dev, table, kv = K.build(lens, hkv, dim, 16, torch.bfloat16, 71)
    q = K.rounded(np.random.default_rng(8).normal(size=(len(lens), hq, dim)).astype(np.float32), torch.bfloat16)
    U.say("attention bf16 outputs", hq, hkv, dim)
    out, _ = K.attend(L, q, dev, table, lens, [1] * len(lens), 16, torch.bfloat16, dim ** -0.5)
    want = np.stack([S.attention(q[b:b + 1], kv[b][0], kv[b][2], 100, dim ** -0.5, 0, ())[0][0] for b in range(len(lens))])
    differ = np.mean(out.float().cpu().numpy() != S.bf16_round(want.astype(np.float32)))
    assert differ <= 0.05, differ


def test_rows_that_belong_to_no_request_are_left(L):
    """Row bounds that start behind the first row and end before the last, long and short."""
    U.say("attention rows of no request")
    dtype = torch.bfloat16
    dev, table, kv = K.build([40, 2100], 2, 128, 16, dtype, 65)
    q = K.rounded(np.random.default_rng(4).normal(size=(9, 8, 128)).astype(np.float32), dtype)
    for max_len in (2100, 40000):
        out, lse = call(L, K.cuda(q, dtype), dev, table, [40, 2100], [3, 5, 6], 16, 2, max_len, 0.1)
        K.compare(out[3:6], lse[3:6], q[3:6], kv, [40, 2100], [2, 1], dtype, 0.1)
        for rest in (slice(0, 3), slice(6, 9)):
            assert torch.all(out[rest] == 9.0) and torch.all(lse[rest] == 9.0)
