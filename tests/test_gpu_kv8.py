"""The 8-bit cache on the GPU: write, read and attention against the oracle.

Write and read are exact.  Attention, counted per output element against the values the cache
stands for (64 bits), as for the 4-bit cache (`test_gpu_kv4.compare`, with |x| up to 127 s):
* a score is an fp32 sum of products of exact codes with the query in at most 2 D + 16 roundings,
  each at most 2^-24 of the sum of |q| 127 s: relative error of a probability <= e := 3 (2 D + 16)
  2^-24 size + 2^-21 (exp2 and its argument);
* a weight times a value's scale is rounded once to fp16, 2^-11 at most, and sums over the tokens
  in fp32 add below 2^-13 in all here: |out - exact| <= (2^-11 + 2^-13 + 2 e) (mass of P 127 s),
  plus half a step of the output's type;
* lse: e + 2^-20 (1 + |lse|)."""
import numpy as np
import pytest

from oracle import eight_bit_oracle as E
from oracle import serving_oracle as S
from tests import gpu_util as U
from tests import test_gpu_kv4 as K
from tests.test_gpu_kv4 import cuda, i32, key_values, rounded

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def L():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    from weight_activation_quantized_amd import mixllm
    return mixllm


def new_cache(pages, heads, page, dim, seed=0):
    """Memory that holds anything, NaN scales among it."""
    rng = np.random.default_rng(seed)
    return rng.integers(0, 256, (pages, heads, E.block_bytes(page, dim)), dtype=np.uint8)


def slots_of(table, pos, page):
    pos = np.asarray(pos)
    return (table[pos // page] * page + pos % page).astype(np.int32)


# ------------------------------------------------------------------------- write and read

# tokens that a request adds call by call
STEPS = {"one by one": [1] * 37, "prompt": [50], "prompt, then single": [37] + [1] * 14, "pieces": [3, 13, 16, 5, 11, 40, 1],
         "long": [200, 1, 7]}


def same_runs(got, want, page, dim, heads, slots):
    """Codes and scales of the runs of these slots are the same."""
    for run in {int(s) // E.RUN for s in slots}:
        p, r = divmod(run, page // E.RUN)
        for h in range(heads):
            for (gc, gs), (wc, ws) in zip(E.run_views(got, p, h, r, page, dim), E.run_views(want, p, h, r, page, dim)):
                assert gs.view(np.uint32) == ws.view(np.uint32), (run, h, gs, ws)
                assert np.array_equal(gc, wc), (run, h, np.argwhere(gc != wc)[:4].ravel())


@pytest.mark.parametrize("dim,heads,page", [(64, 3, 16), (128, 2, 64), (256, 1, 32), (128, 1, 1024)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("name", STEPS)
def test_append_step_by_step(L, dim, heads, page, dtype, name):
    """Two requests that go on side by side; every byte of the cache is the oracle's after every
    call, runs that no token went to among them."""
    U.say("append8", dim, heads, page, dtype, name)
    total, pages = sum(STEPS[name]), 2 * -(-sum(STEPS[name]) // page) + 2
    rng = np.random.default_rng(dim + total)
    table = rng.permutation(pages)
    table = table[:2 * -(-total // page)].reshape(2, -1)
    want = new_cache(pages, heads, page, dim)
    dev = cuda(want)
    at = 0
    for i, n in enumerate(STEPS[name]):
        slots, rows = [], []
        for b in range(2):
            slots += list(slots_of(table[b], np.arange(at, at + n), page)) + ([-1] if i % 3 == 0 else [])
        at += n
        t = len(slots)
        k, v = key_values(t, heads, dim, dtype, 100 * i + dim)
        grow = (1 + 0.3 * rng.random((t, 1, 1))).astype(np.float32)    # scales that grow and that do not
        k, v = rounded(k * grow, dtype), rounded(v / grow, dtype)
        if i == 0:
            k[0], v[-2] = 0.0, 0.0
        row = torch.full((t, 2 * heads * dim + 64), 3.0, dtype=dtype, device="cuda")
        kd, vd = row[:, 64:64 + heads * dim].view(t, heads, dim), row[:, 64 + heads * dim:].view(t, heads, dim)
        kd.copy_(cuda(k, dtype))
        vd.copy_(cuda(v, dtype))
        L.mixllm_kv8_append(kd, vd, i32(slots), dev, page)
        E.kv8_write(want, slots, k, v, page)
        got = dev.cpu().numpy()
        same_runs(got, want, page, dim, heads, [s for s in slots if s >= 0])
        assert np.array_equal(got, want), (i, np.argwhere(got != want)[:5])
    # and back
    slots = np.concatenate([slots_of(table[b], np.arange(at), page) for b in range(2)] + [[-1, pages * page, -2 ** 31]])
    ko = torch.full((len(slots), heads, dim), 9.0, dtype=dtype, device="cuda")
    vo = torch.full_like(ko, 9.0)
    L.mixllm_kv8_read(dev, i32(slots), ko, vo, page)
    vals, _ = E.kv8_values(want, slots[:-3], page, dim)
    for got, val in zip((ko, vo), vals):
        exact = rounded(val.astype(np.float32), dtype)
        assert np.array_equal(got[:-3].float().cpu().numpy(), exact)
        assert torch.all(got[-3:] == 9.0)


def test_read_into_slices(L):
    dim, heads, page, dtype = 128, 2, 32, torch.bfloat16
    cache = new_cache(2, heads, page, dim)
    k, v = key_values(20, heads, dim, dtype, 5)
    E.kv8_write(cache, np.arange(20), k, v, page)
    row = torch.full((20, 2 * heads * dim + 24), 9.0, dtype=dtype, device="cuda")
    ko, vo = row[:, 8:8 + heads * dim].view(20, heads, dim), row[:, 16 + heads * dim:16 + 2 * heads * dim].view(20, heads, dim)
    L.mixllm_kv8_read(cuda(cache), i32(list(range(19, -1, -1))), ko, vo, page)
    vals, _ = E.kv8_values(cache, np.arange(20)[::-1], page, dim)
    assert np.array_equal(ko.float().cpu().numpy(), rounded(vals[0].astype(np.float32), dtype))
    assert np.array_equal(vo.float().cpu().numpy(), rounded(vals[1].astype(np.float32), dtype))
    assert torch.all(row[:, :8] == 9.0) and torch.all(row[:, -8:] == 9.0)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_append_numbers_that_are_none(L, dtype):
    """NaN counts as 0, infinities and what is beyond fp16 as its largest; tiny values keep a
    scale of their own; a held scale that is no positive number counts as none."""
    dim, heads, page = 64, 2, 16
    k, v = key_values(9, heads, dim, dtype, 1)
    k[0, 0, :4] = [np.nan, np.inf, -np.inf, 1.0]
    v[0, 1] = np.nan
    if dtype == torch.bfloat16:
        k[1, 0, 5], v[2, 0, 7] = 3e38, -1e30
    v[3:] = rounded(v[3:] * np.float32(1e-6), dtype)
    want = new_cache(4, heads, page, dim, 3)
    dev = cuda(want)
    # rows 0..2 begin a run, 3.. another, 5.. go on in a run that nothing began, under any scale
    for bad in (np.nan, np.inf, -1.0, 0.0):
        for slots in ([0, 1, 2, 16, 17, 37, 38, 39, 40],):
            for c in (want,):
                for h in range(heads):
                    for _, s in E.run_views(c, 2, h, 0, page, dim):
                        s[0] = bad
            dev.copy_(cuda(want))
            L.mixllm_kv8_append(cuda(k, dtype), cuda(v, dtype), i32(slots), dev, page)
            E.kv8_write(want, slots, k, v, page)
            assert np.array_equal(dev.cpu().numpy(), want), bad
    vals, _ = E.kv8_values(want, [0, 1, 2, 16, 17], page, dim)
    assert np.isfinite(vals).all()


def test_append_nothing(L):
    cache = L.kv8_cache(2, 16, 2, 64)
    before = cache.clone()
    e = torch.empty((0, 2, 64), dtype=torch.float16, device="cuda")
    L.mixllm_kv8_append(e, e, i32([]), cache, 16)
    x = torch.ones((3, 2, 64), dtype=torch.float16, device="cuda")
    L.mixllm_kv8_append(x, x, i32([-1, -1, 32]), cache, 16)
    assert torch.equal(cache, before)


def test_rows_that_share_a_run_out_of_order_touch_no_other_run(L):
    """A slot given twice, and rows of a run in another order or apart: that run is unspecified, the
    others are as if they had been written alone."""
    dim, heads, page = 128, 2, 64
    k, v = key_values(45, heads, dim, torch.float16, 3)
    want = new_cache(3, heads, page, dim, 1)
    dev = cuda(want)
    slots = np.array([5] * 20 + [9, 8, 7] + list(range(64, 80)) + [2, 100, 101, 102, 96, 97], np.int32)
    L.mixllm_kv8_append(cuda(k[:45], torch.float16), cuda(v[:45], torch.float16), i32(slots), dev, page)
    keep = [i for i, s in enumerate(slots) if s // 16 in (4,)]
    E.kv8_write(want, slots[keep], k[keep], v[keep], page)
    got = dev.cpu().numpy()
    same_runs(got, want, page, dim, heads, slots[keep])
    for run in set(range(3 * page // 16)) - {0, 4, 6}:
        p, r = divmod(run, page // 16)
        for h in range(heads):
            for (gc, gs), (wc, ws) in zip(E.run_views(got, p, h, r, page, dim), E.run_views(want, p, h, r, page, dim)):
                assert np.array_equal(gc, wc) and gs.view(np.uint32) == ws.view(np.uint32), run


# ------------------------------------------------------------------------------ attention

def build(lens, heads, dim, page, dtype, seed, spare=2, poison=255, kv=key_values):
    """A cache with the given requests on shuffled pages, written by the library; what nothing was
    written to is 0xFF (NaN scales).  Returns (cache, table, values of keys and values with their
    largest sizes 127 s, per request)."""
    from weight_activation_quantized_amd import mixllm
    rng = np.random.default_rng(seed)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + spare
    order = rng.permutation(pages)
    table = np.full((len(lens), max(need + [1])), -1, np.int32)
    dev, at, out = cuda(np.full((pages, heads, E.block_bytes(page, dim)), poison, np.uint8)), 0, []
    for b, n in enumerate(lens):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
        k, v = kv(n, heads, dim, dtype, seed * 100 + b)
        if n:
            mixllm.mixllm_kv8_append(cuda(k, dtype), cuda(v, dtype), i32(slots_of(table[b], np.arange(n), page)), dev, page)
    cache = dev.cpu().numpy()
    for b, n in enumerate(lens):
        out.append(values_of(cache, table[b], n, page, dim))
    return dev, table, out


def values_of(cache, row, n, page, dim):
    """[keys, their largest size, values, theirs] of a request's tokens, by whole runs."""
    heads, parts = cache.shape[1], []
    ch, t = np.arange(dim), np.arange(E.RUN)[:, None]
    runs = -(-n // E.RUN)
    for part in range(2):
        x, most = np.zeros((runs * E.RUN, heads, dim)), np.zeros((runs * E.RUN, heads, dim))
        for r in range(runs):
            for h in range(heads):
                codes, s = E.run_views(cache, row[r * E.RUN // page], h, r % (page // E.RUN), page, dim)[part]
                at = slice(r * E.RUN, (r + 1) * E.RUN)
                x[at, h] = (codes[E.code_byte(part, t, ch)].astype(np.float64) - 128) * float(s[0])
                most[at, h] = 127 * float(s[0])
        parts += [x[:n], most[:n]]
    return parts


def attend(L, q, dev, table, lens, rows, page, dtype, scale, window=0, max_rows=None, max_len=None, pad=0, stream=None):
    t = q.shape[0] + pad
    cu = np.concatenate([[0], np.cumsum(rows)])
    qd = torch.full((t, *q.shape[1:]), 5.0, dtype=dtype, device="cuda")
    qd[:q.shape[0]] = cuda(q, dtype)
    out, ls = torch.full_like(qd, 9.0), torch.full(qd.shape[:2], 9.0, device="cuda")
    mr, ml = max_rows or max(rows), max_len or max(lens)
    size = L.mixllm_kv8_attention_workspace_bytes(t, len(lens), q.shape[1], dev.shape[1], q.shape[2], mr, ml, window)
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda") if size else None
    L.mixllm_kv8_attention(qd, dev, cuda(table), i32(lens), i32(cu), out, page, mr, ml, scale=scale, window=window, lse=ls,
                           workspace=ws, stream=stream)
    assert torch.all(out[q.shape[0]:] == 9.0) and torch.all(ls[q.shape[0]:] == 9.0)
    return out[:q.shape[0]], ls[:q.shape[0]]


def queries(t, hq, dim, dtype, seed, size=1.0):
    return rounded((size * np.random.default_rng(seed).normal(size=(t, hq, dim))).astype(np.float32), dtype)


HEADS = [(32, 8, 128), (8, 8, 64), (24, 2, 128), (16, 1, 256), (5, 5, 256), (40, 1, 64)]


@pytest.mark.parametrize("hq,hkv,dim", HEADS)
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("page", [16, 64])
def test_single_rows(L, hq, hkv, dim, dtype, page):
    lens = [1, 2, 15, 16, 17, 31, 33, 64, 100, 129, 257]
    U.say("attention8 rows", hq, hkv, dim, dtype, page)
    dev, table, kv = build(lens, hkv, dim, page, dtype, dim + page)
    q = queries(len(lens), hq, dim, dtype, 5)
    rows = [1] * len(lens)
    out, lse = attend(L, q, dev, table, lens, rows, page, dtype, dim ** -0.5, pad=3)
    K.compare(out, lse, q, kv, lens, rows, dtype, dim ** -0.5)


@pytest.mark.parametrize("hq,hkv,dim", HEADS[:4])
@pytest.mark.parametrize("window", [0, 1, 20, 150])
def test_rows_of_prompts(L, hq, hkv, dim, window):
    """Several rows per request: tiles that mix tokens and heads, requests without rows, rows
    before the first token, windows that cut the front."""
    dtype, page = torch.float16, 32
    lens, rows = [7, 40, 300, 3, 90, 0], [7, 5, 9, 5, 0, 2]
    U.say("attention8 prompt", hq, hkv, dim, window)
    dev, table, kv = build(lens, hkv, dim, page, dtype, 7)
    q = queries(sum(rows), hq, dim, dtype, 6)
    out, lse = attend(L, q, dev, table, lens, rows, page, dtype, 0.11, window, pad=2)
    K.compare(out, lse, q, kv, lens, rows, dtype, 0.11, window)


@pytest.mark.parametrize("rows,length", [([130, 70], [130, 333]), ([257], [600]), ([64, 1, 200], [64, 500, 201]),
                                         ([513, 300], [513, 777])])
@pytest.mark.parametrize("hq,hkv,dim", [(8, 2, 128), (4, 4, 64), (4, 1, 256)])
@pytest.mark.parametrize("dtype,window", [(torch.bfloat16, 0), (torch.bfloat16, 77), (torch.float16, 0)])
def test_long_prompts(L, rows, length, hq, hkv, dim, dtype, window):
    page = 16
    U.say("attention8 long prompt", rows, length, hq, hkv, dim, dtype, window)
    dev, table, kv = build(length, hkv, dim, page, dtype, 11)
    q = queries(sum(rows), hq, dim, dtype, 8)
    out, lse = attend(L, q, dev, table, length, rows, page, dtype, 0.08, window)
    K.compare(out, lse, q, kv, length, rows, dtype, 0.08, window,
              picks=lambda n: set(range(0, n, 37)) | {n - 1, n // 2, 15, 16, 63, 64})


@pytest.mark.parametrize("dim,dtype", [(64, torch.float16), (128, torch.bfloat16), (256, torch.float16)])
@pytest.mark.parametrize("window", [0, 700])
def test_long_context(L, dim, dtype, window):
    """One row over thousands of tokens: chunks joined by the second launch."""
    lens = [5003, 2600]
    U.say("attention8 long", dim, dtype, window)
    dev, table, kv = build(lens, 2, dim, 64, dtype, 13)
    q = queries(2, 8, dim, dtype, 9, 2.0)
    out, lse = attend(L, q, dev, table, lens, [1, 1], 64, dtype, dim ** -0.5, window)
    K.compare(out, lse, q, kv, lens, [1, 1], dtype, dim ** -0.5, window)


@pytest.mark.parametrize("rows", [1, 40, 64])
def test_pages_that_are_not_there(L, rows):
    """Negative page numbers and ones past the cache: their tokens count as absent; requests of
    which nothing is left give 0 and -inf."""
    dim, page, dtype, lens = 128, 16, torch.float16, [100, 70, 64]
    hq = 8 if rows == 64 else 4
    dev, table, kv = build(lens, 2, dim, page, dtype, 17)
    gone = [set(), set(), set()]
    for b, js in ((0, (0, 3, 6)), (1, (4,)), (2, (0, 1, 2, 3))):
        for j in js:
            table[b, j] = [-1, 10 ** 6, -2 ** 31, 2 ** 31 - 1][j % 4]
            gone[b] |= set(range(j * page, (j + 1) * page))
    q = queries(3 * rows, hq, dim, dtype, 2)
    out, lse = attend(L, q, dev, table, lens, [rows] * 3, page, dtype, 0.1)
    K.compare(out, lse, q, kv, lens, [rows] * 3, dtype, 0.1, absent=gone)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("rows", [1, 30, 90])
def test_runs_of_far_apart_sizes(L, dtype, rows):
    """Values whose runs differ by up to 2^30 and keys that make the small ones count: what a weight
    loses goes by the row's own largest product, not by the largest scale that it passes."""
    dim, page, n = 128, 16, 200

    def kv(t, heads, d, dt, seed):
        k, v = key_values(t, heads, d, dt, seed)
        run = np.arange(t) // 16
        v = v * np.float32(2.0) ** (np.array([13, -14, 0, 6, -10])[run % 5])[:, None, None].astype(np.float32)
        k[run % 5 != 1] -= 3.0      # with a query of one sign the second runs' scores are far above
        return rounded(k.astype(np.float32), dt), rounded(v.astype(np.float32), dt)

    dev, table, vals = build([n], 2, dim, page, dtype, 19, kv=kv)
    q = np.abs(queries(rows, 4, dim, dtype, 3))
    out, lse = attend(L, q, dev, table, [n], [rows], page, dtype, 0.12)
    K.compare(out, lse, q, vals, [n], [rows], dtype, 0.12)
    # the outputs are those of the second runs: as exact as their own size lets them be
    want, _, _, _ = S.attention(q[-1:], vals[0][0], vals[0][2], n, 0.12)
    err = np.abs(out[-1].double().cpu().numpy() - want[0])
    scale = np.abs(want[0]).max()
    assert scale < 1.0 and err.max() <= (torch.finfo(dtype).eps / 2 + 2.0 ** -10) * scale, (err.max(), scale)


@pytest.mark.parametrize("rows", [1, 7, 40])
def test_scores_of_any_size(L, rows):
    """Large scores (a few tokens take everything), and values of zero."""
    dim, page, dtype, lens = 64, 32, torch.float16, [150, 90]
    dev, table, kv = build(lens, 1, dim, page, dtype, 23)
    q = queries(2 * rows, 4, dim, dtype, 4)
    for scale in (0.0, 3.0, -2.0, 300.0):
        out, lse = attend(L, q, dev, table, lens, [rows] * 2, page, dtype, scale)
        K.compare(out, lse, q, kv, lens, [rows] * 2, dtype, scale)

    def zero(t, heads, d, dt, seed):
        k, v = key_values(t, heads, d, dt, seed)
        return k, np.where(np.arange(t)[:, None, None] // 16 % 2 == 0, 0, v).astype(np.float32)

    dev, table, kv = build(lens, 1, dim, page, dtype, 29, kv=zero)
    out, lse = attend(L, q, dev, table, lens, [rows] * 2, page, dtype, 0.1)
    K.compare(out, lse, q, kv, lens, [rows] * 2, dtype, 0.1)

    def none(t, heads, d, dt, seed):
        k, v = key_values(t, heads, d, dt, seed)
        return k, 0 * v

    dev, table, kv = build(lens, 1, dim, page, dtype, 29, kv=none)
    out, lse = attend(L, q, dev, table, lens, [rows] * 2, page, dtype, 0.1)
    assert not out.any()
    K.compare(out, lse, q, kv, lens, [rows] * 2, dtype, 0.1)


@pytest.mark.parametrize("hq,hkv,dim,rows,window", [(8, 2, 128, 64, 0), (4, 1, 256, 33, 0), (8, 1, 64, 20, 900), (32, 1, 128, 9, 0)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_many_rows_over_a_long_context(L, hq, hkv, dim, rows, window, dtype):
    """Tiles of many rows whose tokens are split among workgroups."""
    page, lens = 64, [4000, 1531]
    U.say("attention8 many rows, long", hq, hkv, dim, rows, window, dtype)
    dev, table, kv = build(lens, hkv, dim, page, dtype, 53)
    q = queries(2 * rows, hq, dim, dtype, 5)
    out, lse = attend(L, q, dev, table, lens, [rows] * 2, page, dtype, dim ** -0.5, window)
    K.compare(out, lse, q, kv, lens, [rows] * 2, dtype, dim ** -0.5, window, picks=lambda n: {0, 7, n - 1})


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("rows", [1, 100])
def test_a_row_without_numbers_spoils_no_other(L, dtype, rows):
    dim, page, lens = 128, 16, [200, 120]
    dev, table, kv = build(lens, 2, dim, page, dtype, 31)
    q = queries(2 * rows, 8, dim, dtype, 5)
    want, wl = attend(L, q, dev, table, lens, [rows] * 2, page, dtype, 0.09)
    q[rows - 1, 2, 7], q[rows, 5, 0] = np.nan, np.inf
    out, lse = attend(L, q, dev, table, lens, [rows] * 2, page, dtype, 0.09)
    ok = torch.ones(out.shape[:2], dtype=torch.bool, device="cuda")
    ok[rows - 1, 2] = ok[rows, 5] = False
    assert torch.equal(out[ok], want[ok]) and torch.equal(lse[ok], wl[ok])
    assert out[rows - 1, 2].isnan().all()


MIXES = {  # rows of each request: prompts among requests of few rows, some without any
    "one prompt, 68 of few rows": ([1, 16, 15, 17, 0, 2, 1, 40] * 8 + [0, 300, 1, 16, 1], 2),
    "two prompts, 130 single rows": ([1] * 60 + [129] + [1] * 69 + [258, 1], 2),
    "few requests": ([1, 0, 700, 3, 2], 4),
    "the prompt last": ([1] * 90 + [333], 1),
}


@pytest.mark.parametrize("mix", MIXES)
@pytest.mark.parametrize("dim,dtype,window", [(64, torch.float16, 0), (128, torch.bfloat16, 0), (128, torch.float16, 90),
                                              (256, torch.bfloat16, 0)])
def test_prompts_among_single_rows(L, mix, dim, dtype, window):
    """One call whose largest request has many rows and most others few: tiles by the rows of the
    call, and a launch for the requests of few rows where the batch is large; rows that the call
    does not have stay as they were."""
    rows, group = MIXES[mix]
    hkv = 1 if len(rows) < 10 else 3 if len(rows) > 80 else 4
    lens = [max(0, n - 3) if b % 9 == 5 else n + (b * 67) % 400 for b, n in enumerate(rows)]
    U.say("attention8 mix", mix, dim, dtype, window)
    dev, table, kv = build(lens, hkv, dim, 32, dtype, 41)
    q = queries(sum(rows), hkv * group, dim, dtype, 14)
    out, lse = attend(L, q, dev, table, lens, rows, 32, dtype, 0.09, window, pad=4)
    K.compare(out, lse, q, kv, lens, rows, dtype, 0.09, window,
              picks=lambda n: set(range(n)) if n <= 17 else set(range(0, n, 43)) | {n - 1, n // 2, 15, 16, 63, 64} & set(range(n)))


def test_a_replayed_call_of_prompts_among_single_rows(L):
    """The same graph for another step: which requests have many rows is read on the GPU."""
    hq, hkv, dim, page, dtype = 8, 4, 64, 16, torch.float16
    steps = [[1] * 30 + [200] + [1] * 39, [2] * 50 + [150, 0] + [1] * 18, [0] * 69 + [260]]
    lens = [[(b * 31) % 300 + n for b, n in enumerate(rows)] for rows in steps]
    dev, table, kv = build([max(x) for x in zip(*lens)], hkv, dim, page, dtype, 43)
    t, b = 300, 70
    q, cu, ln = torch.zeros(t, hq, dim, dtype=dtype, device="cuda"), i32([0] * (b + 1)), i32([0] * b)
    out, tab = torch.empty_like(q), cuda(table)
    size = L.mixllm_kv8_attention_workspace_bytes(b * 260, b, hq, hkv, dim, 260, 600)  # of the largest step
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    assert size
    call = lambda: L.mixllm_kv8_attention(q, dev, tab, ln, cu, out, page, 260, 600, scale=0.1, workspace=ws)  # noqa: E731
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for i, (rows, held) in enumerate(zip(steps * 2, lens * 2)):
        x = queries(t, hq, dim, dtype, 50 + i)
        q.copy_(cuda(x, dtype))
        cu.copy_(i32(np.concatenate([[0], np.cumsum(rows)])))
        ln.copy_(i32(held))
        out.fill_(9.0)
        g.replay()
        torch.cuda.synchronize()
        n = sum(rows)
        got = out[:n].clone()
        assert torch.all(out[n:] == 9.0)
        out.fill_(9.0)
        call()
        torch.cuda.synchronize()
        assert torch.equal(out[:n], got)
        alone, lse = attend(L, x[:n], dev, table, held, rows, page, dtype, 0.1, max_rows=260, max_len=600)
        K.compare(got, lse, x[:n], [tuple(a[:m] for a in one) for one, m in zip(kv, held)], held, rows, dtype, 0.1,
                  picks=lambda n: set(range(n)) if n <= 17 else set(range(0, n, 43)) | {n - 1})


@pytest.mark.parametrize("max_rows,max_len", [(3, 500), (1, 100), (9, 40)])
def test_promises_that_are_too_small(L, max_rows, max_len):
    """Rows past max_rows are left out, lengths past max_len count as that."""
    dim, page, dtype, lens, rows = 64, 16, torch.float16, [90, 200], [2, 6]
    dev, table, kv = build(lens, 2, dim, page, dtype, 37)
    q = queries(sum(rows), 4, dim, dtype, 6)
    out, lse = attend(L, q, dev, table, lens, rows, page, dtype, 0.1, max_rows=max_rows, max_len=max_len)
    at = 0
    for b in range(2):
        n = min(lens[b], max_len)
        for i in range(rows[b]):
            if i >= max_rows:
                assert torch.all(out[at + i] == 9.0) and torch.all(lse[at + i] == 9.0)
                continue
            upto = n - rows[b] + i + 1
            part = [x[:upto] for x in kv[b]]
            K.compare(out[at + i:at + i + 1], lse[at + i:at + i + 1], q[at + i:at + i + 1], [part], [upto], [1], dtype, 0.1)
        at += rows[b]


def test_strided_rows_and_tables(L):
    dim, hq, hkv, page, dtype, lens = 128, 6, 2, 32, torch.bfloat16, [40, 100, 7]
    dev, table, kv = build(lens, hkv, dim, page, dtype, 41)
    q = queries(3, hq, dim, dtype, 7)
    row = torch.full((3, hq * dim + 32), 2.0, dtype=dtype, device="cuda")
    row[:, 16:16 + hq * dim] = cuda(q, dtype).flatten(1)
    res = torch.full((3, hq * dim + 8), 9.0, dtype=dtype, device="cuda")
    wide = torch.full((5, table.shape[1] + 3), -7, dtype=torch.int32, device="cuda")
    wide[:3, :table.shape[1]] = cuda(table)
    lse = torch.empty((3, hq), device="cuda")
    L.mixllm_kv8_attention(row[:, 16:16 + hq * dim].view(3, hq, dim), dev, wide[:, :table.shape[1]], i32(lens), i32([0, 1, 2, 3]),
                           res[:, :hq * dim].view(3, hq, dim), page, 1, 100, lse=lse)
    K.compare(res[:, :hq * dim].view(3, hq, dim), lse, q, kv, lens, [1, 1, 1], dtype, dim ** -0.5)
    assert torch.all(res[:, hq * dim:] == 9.0)


def test_fp16_outputs_have_the_error_of_their_own_rounding(L):
    """Decodes over long contexts, where outputs are small sums of many values."""
    dim, page, dtype, lens = 128, 64, torch.float16, [6000]
    dev, table, kv = build(lens, 2, dim, page, dtype, 43)
    q = queries(1, 16, dim, dtype, 8)
    out, lse = attend(L, q, dev, table, lens, [1], page, dtype, dim ** -0.5)
    want, wl, _, _ = S.attention(q, kv[0][0], kv[0][2], 6000, dim ** -0.5)
    rms = lambda x: float(np.sqrt((x ** 2).mean()))  # noqa: E731
    err = rms(out.double().cpu().numpy() - want)
    own = rms(want.astype(np.float16).astype(np.float64) - want)
    assert err <= 1.2 * own, (err, own)
    assert np.abs(lse.double().cpu().numpy() - wl).max() < 1e-5


def test_two_graphs_and_an_eager_call(L):
    """Calls captured with a workspace each, replayed on two streams beside eager work."""
    dim, page, dtype, lens = 128, 64, torch.bfloat16, [3000, 1500]
    dev, table, kv = build(lens, 2, dim, page, dtype, 47)
    tab, ln, cu = cuda(table), i32(lens), i32([0, 1, 2])
    size = L.mixllm_kv8_attention_workspace_bytes(2, 2, 8, 2, dim, 1, 3000, 0)
    assert size
    sides = []
    for seed in (1, 2):
        q = cuda(queries(2, 8, dim, dtype, seed), dtype)
        out, ws = torch.empty_like(q), torch.empty(size, dtype=torch.uint8, device="cuda")
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        call = lambda q=q, out=out, ws=ws, s=s: L.mixllm_kv8_attention(q, dev, tab, ln, cu, out, page, 1, 3000, workspace=ws,  # noqa: E731
                                                                       stream=s)
        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            call()
        sides.append((q, out, s, g))
    ws, want = torch.empty(size, dtype=torch.uint8, device="cuda"), torch.empty((2, 8, dim), dtype=dtype, device="cuda")
    for i in range(6):
        for q, out, s, g in sides:
            q.mul_(1.02)
            out.fill_(0)
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                g.replay()
        for q, out, s, g in sides:
            torch.cuda.current_stream().wait_stream(s)
            L.mixllm_kv8_attention(q, dev, tab, ln, cu, want, page, 1, 3000, workspace=ws)
            torch.cuda.synchronize()
            assert torch.equal(out, want), i


def test_binding_refuses(L):
    cache = L.kv8_cache(4, 16, 2, 64)
    x = torch.zeros((3, 2, 64), dtype=torch.float16, device="cuda")
    s = i32([0, 1, 2])
    four = L.kv4_cache(4, 16, 2, 64)
    for call in (lambda: L.mixllm_kv8_append(x, x, s, four, 16), lambda: L.mixllm_kv8_append(x, x, s, cache, 32),
                 lambda: L.mixllm_kv4_append(x, x, s, cache, 16), lambda: L.mixllm_kv8_append(x, x[:2], s, cache, 16),
                 lambda: L.mixllm_kv8_append(x, x, s[:2], cache, 16), lambda: L.mixllm_kv8_append(x, x.bfloat16(), s, cache, 16),
                 lambda: L.mixllm_kv8_read(cache, s.long(), x, x, 16), lambda: L.mixllm_kv8_append(x[:, :1], x[:, :1], s, cache, 16),
                 lambda: L.mixllm_kv8_attention(x, four, s[None], s[:1], s[:2], x, 16, 1, 16),
                 lambda: L.mixllm_kv8_attention(x, cache, s[None], s[:1], s[:1], x, 16, 1, 16),
                 lambda: L.mixllm_kv8_attention(x, cache, s[None], s[:1], s[:2], x.bfloat16(), 16, 1, 16),
                 lambda: L.mixllm_kv8_attention(x, cache, s[None], s[:1], s[:2], x, 16, 1, 16, lse=torch.zeros((3, 1), device="cuda")),
                 lambda: L.mixllm_kv8_attention(x, cache, s[None], s[:1], s[:2], x, 16, 1, 2 ** 32 + 16)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(L.MixLLMError):      # splits need a workspace
        L.mixllm_kv8_attention(x[:1], cache, i32([[0] * 256]), s[:1], s[:2], torch.empty_like(x[:1]), 16, 1, 4096)


def some_table(requests, per, page, seed):
    rng = np.random.default_rng(seed)
    return rng.permutation(requests * per + 3)[:requests * per].reshape(requests, per)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("dim,heads,requests", [(64, 8, 600), (128, 3, 1400), (256, 2, 2100)])
def test_append_of_many_requests(L, dim, heads, requests, dtype):
    """Steps of single tokens and of a few each, of so many requests that workgroups take many rows."""
    U.say("append8 many", dim, heads, requests, dtype)
    page, held = 16, np.arange(requests) * 5 % 23
    table = some_table(requests, 3, page, 1)
    want = new_cache(3 * requests + 3, heads, page, dim)
    dev = cuda(want)
    for i, most in enumerate((23, 1, 3)):
        add = held if i == 0 else 1 + np.arange(requests) * 7 % most
        at = np.zeros(requests, int) if i == 0 else held
        slots = np.concatenate([slots_of(table[b], np.arange(at[b], at[b] + add[b]), page) for b in range(requests)])
        held = at + add
        k, v = key_values(len(slots), heads, dim, dtype, i)
        L.mixllm_kv8_append(cuda(k, dtype), cuda(v, dtype), i32(slots), dev, page)
        E.kv8_write(want, slots, k, v, page)
        got = dev.cpu().numpy()
        assert np.array_equal(got, want), (i, np.argwhere(got != want)[:5])


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_quotients_at_halves(L, dtype):
    """Values whose quotients are halves or next to them, over many scales: rounded as the division says."""
    dim, heads, page, runs = 64, 2, 64, 40
    rng = np.random.default_rng(4)
    x = (rng.integers(-254, 255, (16 * runs, heads, dim)) / 2).astype(np.float32)
    x[::16, :, 0] = 127
    s = np.exp2(rng.integers(-9, 6, (runs, heads)).astype(np.float32)) * rng.choice([1, 1.0009765625, 0.99951171875, 1.25], (runs, heads))
    x = rounded((x.reshape(runs, 16, heads, dim) * s[:, None, :, None]).reshape(-1, heads, dim).astype(np.float32), dtype)
    v = rounded(x[::-1] * np.float32(0.37), dtype)
    want = new_cache(runs * 16 // page, heads, page, dim)
    dev = cuda(want)
    slots = np.arange(16 * runs, dtype=np.int32)
    L.mixllm_kv8_append(cuda(x, dtype), cuda(v, dtype), i32(slots), dev, page)
    E.kv8_write(want, slots, x, v, page)
    assert np.array_equal(dev.cpu().numpy(), want)
