"""The 4-bit cache on the GPU: plan, write, read and attention against the oracle.

Plan, write and read are exact.  Attention, counted per output element against the values
the cache stands for (64 bits):
* a score is an fp32 sum of products of exact codes with the query (fp16, exact up to a power
  of two; bf16 fits it too), in at most 2 D + 16 roundings, each at most 2^-24 of the sum of
  |q| (s c + |m|) <= 3 |q| |k|-like terms; `size` bounds that sum with c up to 15:
  relative error of a probability <= e := (2 D + 16) 2^-24 size + 2^-21 (exp2 and its argument);
* a weight s P is rounded once to fp16: 2^-11 of s c P, with s c <= |v| + |m|; sums over the
  tokens in fp32 add 2^-24 per token and step of the tree, below 2^-13 in all here;
* the matrix instruction cuts its products (of subnormal codes) at 2^10 2^-24 2^-p of a code
  beside its largest factor, p the lowest bit the codes are at: keys (p = 4) 2^-18 / 15 of the
  largest term, D times at most, which is less than the 3 (2 D + 16) 2^-24 that the bound below
  takes of `size`; values (p = 2) 2^-16 s of the largest weight, 32 times, where its mass is s c +
  |m| with |m| > 5 s here: below the 2^-13;
* so |out - exact| <= (2^-11 + 2^-13 + 2 e) (mass of P (s c + |m|)), plus half a step of the
  output's type;
* lse: e + 2^-20 (1 + |lse|).
"""
import numpy as np
import pytest

from oracle import serving_oracle as S
from tests import gpu_util as U

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def L():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    from weight_activation_quantized_amd import mixllm
    return mixllm


def cuda(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if dtype is None else t.to(dtype)


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def rounded(x, dtype):
    """fp32 values of x rounded to a 16-bit type."""
    return x.astype(np.float16).astype(np.float32) if dtype == torch.float16 else S.bf16_round(x)


def key_values(t, heads, dim, dtype, seed):
    rng = np.random.default_rng(seed)
    k = rng.normal(size=(t, heads, dim)) + 0.5 * rng.normal(size=(1, heads, dim))
    k[:, :, 3::41] *= 7
    v = 0.7 * rng.normal(size=(t, heads, dim))
    return rounded(k.astype(np.float32), dtype), rounded(v.astype(np.float32), dtype)


# ------------------------------------------------------------------------- write and read

@pytest.mark.parametrize("dim,heads", [(64, 3), (128, 8), (256, 1)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("t,page", [(1, 16), (37, 32), (3, 1024)])
def test_append_and_read(L, dim, heads, dtype, t, page):
    U.say("append", dim, heads, dtype, t, page)
    pages = 5
    rng = np.random.default_rng(t + dim)
    k, v = key_values(t, heads, dim, dtype, 1)
    k[0, 0, :64], v[0, 0] = 2.5, 0.0                       # constant groups
    k[-1, -1, :4] = [np.nan, np.inf, -np.inf, 1.0]
    v[-1, -1, 64:] *= 1e-7                                 # a scale that underflows fp16
    v = rounded(v, dtype)
    slots = rng.permutation(pages * page)[:t].astype(np.int32)
    if t > 4:
        slots[2], slots[4], slots[5] = -1, pages * page, -2 ** 31   # no token there
    cache = rng.integers(0, 256, (pages, heads, page * dim * 9 // 8), dtype=np.uint8)
    dev = cuda(cache)
    # keys and values as slices of one wider row, as a q/k/v GEMM leaves them
    row = torch.full((t, 2 * heads * dim + 64), 3.0, dtype=dtype, device="cuda")
    kd, vd = row[:, 64:64 + heads * dim].view(t, heads, dim), row[:, 64 + heads * dim:].view(t, heads, dim)
    kd.copy_(cuda(k, dtype))
    vd.copy_(cuda(v, dtype))
    L.mixllm_kv4_append(kd, vd, i32(slots), dev, page)
    S.kv4_write(cache, slots, k, v, page)
    got = dev.cpu().numpy()
    assert np.array_equal(got, cache), np.argwhere(got != cache)[:5]

    ko, vo = torch.full_like(row, 9.0), torch.full((t, heads, dim), 9.0, dtype=dtype, device="cuda")
    kov = ko[:, 64:64 + heads * dim].view(t, heads, dim)
    L.mixllm_kv4_read(dev, i32(slots), kov, vo, page)
    for x, o in ((k, kov), (v, vo)):
        want = S.kv4_values(*S.kv4_quant(x)).astype(np.float32)
        want = rounded(want, dtype)
        live = (slots >= 0) & (slots < pages * page)
        assert np.array_equal(o.float().cpu().numpy()[live], want[live])
        assert np.all(o.float().cpu().numpy()[~live] == 9.0)
    assert torch.all(ko[:, :64] == 9.0)


def test_append_nothing(L):
    cache = L.kv4_cache(2, 16, 2, 64)
    before = cache.clone()
    e = torch.empty((0, 2, 64), dtype=torch.float16, device="cuda")
    L.mixllm_kv4_append(e, e, i32([]), cache, 16)
    x = torch.ones((3, 2, 64), dtype=torch.float16, device="cuda")
    L.mixllm_kv4_append(x, x, i32([-1, -1, 32]), cache, 16)
    assert torch.equal(cache, before)


def test_same_slot_twice_touches_no_other_token(L):
    cache = torch.zeros((2, 2, 16 * 72), dtype=torch.uint8, device="cuda")
    k, v = key_values(20, 2, 64, torch.float16, 3)
    L.mixllm_kv4_append(cuda(k, torch.float16), cuda(v, torch.float16), i32([5] * 20), cache, 16)
    ko = torch.full((31, 2, 64), 9.0, dtype=torch.float16, device="cuda")
    vo = ko.clone()
    L.mixllm_kv4_read(cache, i32([s for s in range(32) if s != 5]), ko, vo, 16)
    assert not ko.any() and not vo.any()


# ------------------------------------------------------------------------------- the plan

def plan_case(fresh, lens, width, page, pages, pool_size, free, tokens, seed, in_place=False):
    rng = np.random.default_rng(seed)
    order = rng.permutation(pages).astype(np.int32)
    table = rng.integers(-5, pages + 5, (len(fresh), width)).astype(np.int32)  # entries past a length: anything
    at = 0
    for b, n in enumerate(lens):
        have = -(-min(max(n, 0), width * page) // page)
        table[b, :have] = order[np.arange(at, at + have) % pages]
        at += have
    pool = np.full(pool_size, -7, np.int32)
    n = min(free, pool_size, max(pages - at, 0))
    pool[:n] = order[at:at + n]
    return table, pool, n


def run_plan(L, fresh, lens, table, pool, count, page, pages, tokens, in_place=False):
    f, n, t, p, c = i32(fresh), i32(lens), cuda(table), cuda(pool), i32([count, 99])
    lo = n if in_place else torch.full_like(n, -9)
    co = c if in_place else i32([-9, -9])
    cu, slots, pos = i32([-9] * (len(fresh) + 1)), i32([-9] * tokens), i32([-9] * tokens)
    L.mixllm_kv_plan(f, n, t, p, c, page, pages, lo, co, cu, slots, pos)
    return dict(table=t, pool=p, lens_out=lo, count_out=co, cu=cu, slots=slots, pos=pos)


PLANS = {
    "one": ([1], [0], 4, 16, 10, 10, 10, 1),
    "empty requests": ([0, 0, 3, 0], [0, 5, 0, 16], 4, 16, 10, 10, 10, 8),
    "ends": ([-1, 1, -1, 1, -1], [33, 15, 64, 16, 0], 4, 16, 30, 30, 5, 4),
    "all end": ([-1, -1], [40, 17], 4, 16, 30, 30, 0, 0),
    "pool too small for what comes back": ([-1, -1], [64, 64], 4, 16, 30, 6, 1, 3),
    "pool runs out": ([20, 1, 33, 1, 0, 16], [0, 15, 0, 16, 3, 1], 4, 16, 30, 30, 3, 90),
    "row full": ([1, 1, 70, 2 ** 31 - 1, 1], [64, 63, 0, 3, 9], 4, 16, 30, 30, 20, 100),
    "lengths out of range": ([1, 1, -1], [-5, 1000, 2000], 4, 16, 40, 40, 10, 6),
    "rows cut short": ([30, 30], [0, 0], 4, 16, 30, 30, 20, 37),
    "none": ([], [], 4, 16, 10, 10, 4, 3),
    "prompts": ([5000, 1, 1, 7000, 1], [0, 100, 31, 1000, 64], 300, 32, 900, 900, 700, 12010),
    "big pages": ([1500, 3], [2, 1023], 4, 1024, 9, 9, 4, 1600),
}


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("name", PLANS)
def test_plan(L, name, in_place):
    U.say("plan", name, in_place)
    fresh, lens, width, page, pages, size, free, tokens = PLANS[name]
    table, pool, count = plan_case(*PLANS[name][:6], free, tokens, 3)
    want = S.kv_plan(fresh, lens, table, pool, count, page, pages, tokens)
    got = run_plan(L, fresh, lens, table, pool, count, page, pages, tokens, in_place)
    for k, v in want.items():
        assert np.array_equal(got[k].cpu().numpy(), v), k


@pytest.mark.parametrize("b,prompt,free", [(1023, 1, 2000), (1024, 1, 40), (1025, 40, 3000), (2500, 7, 9000), (2100, 2, 4000),
                                           (1024, 300, 9000)])
def test_plan_of_many_requests(L, b, prompt, free):
    """More requests than the sums' workgroup has threads, with ends, prompts and refusals."""
    U.say("plan many", b, prompt, free)
    rng = np.random.default_rng(b)
    fresh = rng.choice([-1, 0, 1, 1, 1, prompt], b)
    lens = rng.integers(0, 130, b)
    pages = 16000
    tokens = int(np.maximum(fresh, 0).sum()) + 3
    table, pool, count = plan_case(fresh, lens, 12, 16, pages, pages, free, tokens, b)
    want = S.kv_plan(fresh, lens, table, pool, count, 16, pages, tokens)
    got = run_plan(L, fresh, lens, table, pool, count, 16, pages, tokens)
    for k, v in want.items():
        assert np.array_equal(got[k].cpu().numpy(), v), k


def test_plan_with_pages_that_do_not_exist(L):
    """A table or pool with numbers outside the cache gives no slot, never a wrong one."""
    table = np.array([[3, 900, -1], [-4, 2, -1], [1, -1, -1]], np.int32)
    pool = np.array([5, 77, 6], np.int32)
    args = ([18, 20, 40], [14, 3, 0], table, pool, 3, 16, 10, 80)
    want, got = S.kv_plan(*args), run_plan(L, *args)
    for k, v in want.items():
        assert np.array_equal(got[k].cpu().numpy(), v), k


# ------------------------------------------------------------------------------ attention

def build(lens, heads, dim, page, dtype, seed, spare=2, poison=255):
    """A cache with the given requests on shuffled pages; memory no token was written to is
    0xFF (fp16 NaN).  Returns (cache, table, values of each request's keys and values, |m| + 15 s)."""
    rng = np.random.default_rng(seed)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + spare
    order = rng.permutation(pages)
    table = np.full((len(lens), max(need + [1])), -1, np.int32)
    cache = np.full((pages, heads, page * dim * 9 // 8), poison, np.uint8)
    dev, at, kv = cuda(cache), 0, []
    from weight_activation_quantized_amd import mixllm
    for b, n in enumerate(lens):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
        k, v = key_values(n, heads, dim, dtype, seed * 100 + b)
        if n:
            pos = np.arange(n)
            slots = table[b, pos // page] * page + pos % page
            mixllm.mixllm_kv4_append(cuda(k, dtype), cuda(v, dtype), i32(slots), dev, page)
        parts = []
        for x in (k, v):
            c, s, m = S.kv4_quant(x)
            bound = np.repeat(15 * s.astype(np.float64) + np.abs(m.astype(np.float64)), 64, -1)
            parts += [S.kv4_values(c, s, m), bound.reshape(n, heads, dim)]
        kv.append(parts)
    return dev, table, kv


def attend(L, q, dev, table, lens, rows, page, dtype, scale, window=0, max_rows=None, max_len=None, pad=0, lse=True):
    t = q.shape[0] + pad
    cu = np.concatenate([[0], np.cumsum(rows)])
    qd = torch.full((t, *q.shape[1:]), 5.0, dtype=dtype, device="cuda")
    qd[:q.shape[0]] = cuda(q, dtype)
    out = torch.full_like(qd, 9.0)
    ls = torch.full(qd.shape[:2], 9.0, device="cuda") if lse else None
    mr, ml = max_rows or max(rows), max_len or max(lens)
    size = L.mixllm_kv4_attention_workspace_bytes(t, len(lens), q.shape[1], dev.shape[1], q.shape[2], mr, ml, window)
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda") if size else None
    L.mixllm_kv4_attention(qd, dev, cuda(table), i32(lens), i32(cu), out, page, mr, ml, scale=scale, window=window, lse=ls,
                           workspace=ws)
    assert torch.all(out[q.shape[0]:] == 9.0) and (ls is None or torch.all(ls[q.shape[0]:] == 9.0))
    return out[:q.shape[0]], None if ls is None else ls[:q.shape[0]]


def compare(out, lse, q, kv, lens, rows, dtype, scale, window=0, absent=None, picks=None):
    o, ls = out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    d, at = q.shape[2], 0
    for b, n in enumerate(lens):
        kval, kmost, vval, vmost = kv[b]
        for i in range(rows[b]):
            if picks is not None and i not in picks(rows[b]):
                continue
            upto = n - rows[b] + i + 1   # one row: a request of that length
            qr = q[at + i:at + i + 1]
            if upto <= 0:
                assert not o[at + i].any() and np.all(np.isneginf(ls[at + i])), (b, i)
                continue
            gone = absent[b] if absent else ()
            want, wl, _, _ = S.attention(qr, kval[:upto], vval[:upto], upto, scale, window, gone)
            _, _, mass, size = S.attention(qr, kval[:upto], vmost[:upto], upto, scale, window, gone)
            size = (np.abs(scale) * np.einsum("td,xd->xt", kmost[:upto].max(1), np.abs(qr[0]).astype(np.float64))).max(-1)
            e = (2 * d + 16) * 2.0 ** -24 * 3 * size + 2.0 ** -21
            f = torch.finfo(dtype)
            tol = (2.0 ** -11 + 2.0 ** -13 + 2 * e)[:, None] * mass[0]
            tol = tol + f.eps / 2 * (np.abs(want[0]) + tol) + float(f.smallest_normal) * f.eps / 2
            err = np.abs(o[at + i] - want[0])
            assert np.all(err <= tol), (b, i, (err / tol).max())
            seen = np.isfinite(wl[0])
            assert np.array_equal(np.isneginf(ls[at + i]), ~seen)
            le = np.abs(ls[at + i][seen] - wl[0][seen])
            assert np.all(le <= e[seen] + 2.0 ** -20 * (1 + np.abs(wl[0][seen]))), (b, i, le.max())
        at += rows[b]


HEADS = [(32, 8, 128), (8, 8, 64), (24, 2, 128), (16, 1, 256), (5, 5, 256), (40, 1, 64)]


@pytest.mark.parametrize("hq,hkv,dim", HEADS)
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("page", [16, 64])
def test_single_rows(L, hq, hkv, dim, dtype, page):
    lens = [1, 2, 15, 16, 17, 31, 33, 64, 100, 129, 257]
    U.say("attention rows", hq, hkv, dim, dtype, page)
    dev, table, kv = build(lens, hkv, dim, page, dtype, dim + page)
    q = rounded(np.random.default_rng(5).normal(size=(len(lens), hq, dim)).astype(np.float32), dtype)
    rows = [1] * len(lens)
    out, lse = attend(L, q, dev, table, lens, rows, page, dtype, dim ** -0.5, pad=3)
    compare(out, lse, q, kv, lens, rows, dtype, dim ** -0.5)


@pytest.mark.parametrize("hq,hkv,dim", HEADS[:4])
@pytest.mark.parametrize("window", [0, 1, 20, 150])
def test_rows_of_prompts(L, hq, hkv, dim, window):
    """Several rows per request: tiles that mix tokens and heads, requests without rows, rows
    before the first token, windows that cut the front."""
    dtype, page = torch.float16, 32
    lens, rows = [7, 40, 300, 3, 90, 0], [7, 5, 9, 5, 0, 2]
    U.say("attention prompt", hq, hkv, dim, window)
    dev, table, kv = build(lens, hkv, dim, page, dtype, 7)
    q = rounded(np.random.default_rng(6).normal(size=(sum(rows), hq, dim)).astype(np.float32), dtype)
    out, lse = attend(L, q, dev, table, lens, rows, page, dtype, 0.11, window, pad=2)
    compare(out, lse, q, kv, lens, rows, dtype, 0.11, window)


@pytest.mark.parametrize("rows,length", [([130, 70], [130, 333]), ([257], [600]), ([64, 1, 200], [64, 500, 201])])
@pytest.mark.parametrize("hq,hkv,dim", [(8, 2, 128), (4, 4, 64), (4, 1, 256)])
@pytest.mark.parametrize("window", [0, 77])
def test_long_prompts(L, rows, length, hq, hkv, dim, window):
    dtype, page = torch.bfloat16, 16
    U.say("attention long prompt", rows, length, hq, hkv, dim, window)
    dev, table, kv = build(length, hkv, dim, page, dtype, 11)
    q = rounded(np.random.default_rng(8).normal(size=(sum(rows), hq, dim)).astype(np.float32), dtype)
    out, lse = attend(L, q, dev, table, length, rows, page, dtype, 0.08, window)
    compare(out, lse, q, kv, length, rows, dtype, 0.08, window,
            picks=lambda n: set(range(0, n, 37)) | {n - 1, n // 2, 15, 16, 63, 64})


@pytest.mark.parametrize("dim,dtype", [(64, torch.float16), (128, torch.bfloat16), (256, torch.float16)])
@pytest.mark.parametrize("window", [0, 700])
def test_long_context(L, dim, dtype, window):
    """One row over thousands of tokens: chunks joined by the second launch."""
    lens = [5003, 2600]
    U.say("attention long", dim, dtype, window)
    dev, table, kv = build(lens, 2, dim, 64, dtype, 13)
    q = rounded(2 * np.random.default_rng(9).normal(size=(2, 8, dim)).astype(np.float32), dtype)
    out, lse = attend(L, q, dev, table, lens, [1, 1], 64, dtype, dim ** -0.5, window)
    compare(out, lse, q, kv, lens, [1, 1], dtype, dim ** -0.5, window)


@pytest.mark.parametrize("length", [64, 3000])
def test_promised_bounds_larger_than_the_truth(L, length):
    """max_rows and max_len above the real ones (a captured launch): the same results."""
    lens, rows = [length, 5, 0], [2, 1, 0]
    dev, table, kv = build(lens, 2, 128, 16, torch.float16, 17)
    q = rounded(np.random.default_rng(3).normal(size=(3, 8, 128)).astype(np.float32), torch.float16)
    for mr, ml in ((2, length), (5, 10000), (40, 40000)):
        U.say("attention bounds", length, mr, ml)
        out, lse = attend(L, q, dev, table, lens, rows, 16, torch.float16, 0.1, 0, mr, ml, pad=5)
        compare(out, lse, q, kv, lens, rows, torch.float16, 0.1)


def test_lengths_past_the_promise_are_cut(L):
    """A length above max_len or the table counts as that bound: nothing past it is read."""
    dev, table, kv = build([64], 2, 128, 16, torch.float16, 19)
    q = rounded(np.random.default_rng(3).normal(size=(1, 8, 128)).astype(np.float32), torch.float16)
    for length, ml, eff in ((1000, 48, 48), (1000, 4000, 64), (2 ** 31 - 1, 64, 64), (-3, 64, 0)):
        U.say("attention cut", length, ml)
        out, lse = attend(L, q, dev, table, [length], [1], 16, torch.float16, 0.1, 0, 1, ml)
        compare(out, lse, q, kv, [eff], [1], torch.float16, 0.1)


@pytest.mark.parametrize("length", [100, 4000])
def test_pages_that_do_not_exist_hide_their_tokens(L, length):
    lens = [length, length]
    dev, table, kv = build(lens, 2, 128, 16, torch.float16, 23)
    table[0, 2], table[0, length // 16 - 1], table[1, :] = -1, dev.shape[0], 2 ** 31 - 1
    gone = [set(range(32, 48)) | set(range((length // 16 - 1) * 16, length // 16 * 16)), set(range(length))]
    q = rounded(np.random.default_rng(3).normal(size=(2, 4, 128)).astype(np.float32), torch.float16)
    U.say("attention absent pages", length)
    out, lse = attend(L, q, dev, table, lens, [1, 1], 16, torch.float16, 0.1)
    compare(out, lse, q, kv, lens, [1, 1], torch.float16, 0.1, absent=gone)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("vscale,qscale", [(1e-4, 1.0), (3000.0, 1.0), (1.0, 3e4), (1.0, 1e-6), ("rising", 1.0),
                                           ("falling", 1.0), ("zeros", 0.0), ("groups", 1.0)])
def test_extreme_values(L, dtype, vscale, qscale):
    """Values tiny, huge or of changing size along the context, queries at the ends of the
    type, a maximum that keeps rising: the probabilities' fp16 operands must not lose it."""
    n, dim, hq, hkv = 900, 128, 8, 2
    U.say("attention extremes", dtype, vscale, qscale)
    rng = np.random.default_rng(31)
    k, v = rng.normal(size=(n, hkv, dim)), rng.normal(size=(n, hkv, dim))
    if vscale == "rising":
        v *= (2.0 ** (np.arange(n) / 60 - 12))[:, None, None]
        k *= (np.arange(n) / n)[:, None, None] * 3
    elif vscale == "falling":
        v *= (2.0 ** (-np.arange(n) / 60 + 8))[:, None, None]
    elif vscale == "zeros":
        v *= 0
    elif vscale == "groups":     # the second group of channels far larger than the first
        v[:, :, 64:] *= 2000.0
        k[:, :, 64:] *= 0.01
    else:
        v *= vscale
    k, v = rounded(k.astype(np.float32), dtype), rounded(v.astype(np.float32), dtype)
    cache = torch.full((60, hkv, 16 * 144), 255, dtype=torch.uint8, device="cuda")
    table = np.random.default_rng(1).permutation(60)[:57].astype(np.int32)[None]
    pos = np.arange(n)
    L.mixllm_kv4_append(cuda(k, dtype), cuda(v, dtype), i32(table[0, pos // 16] * 16 + pos % 16), cache, 16)
    parts = []
    for x in (k, v):
        c, s, m = S.kv4_quant(x)
        parts += [S.kv4_values(c, s, m), np.repeat(15 * s.astype(np.float64) + np.abs(m.astype(np.float64)), 64, -1).reshape(n, hkv, dim)]
    q = rounded((qscale * rng.normal(size=(1, hq, dim))).clip(-60000, 60000).astype(np.float32), dtype)
    scale = 0.09 / max(qscale, 1.0)
    out, lse = attend(L, q, cache, table, [n], [1], 16, dtype, scale)
    compare(out, lse, q, [parts], [n], [1], dtype, scale)


@pytest.mark.parametrize("hq,hkv,dim", [(32, 8, 128), (24, 3, 64), (16, 1, 256), (40, 1, 128)])
def test_half_outputs_are_nearly_rounded(L, hq, hkv, dim):
    """fp16 outputs have the error of their own rounding and little else: 1.1 times it, that is
    0.45 of it added in squares, 0.45 * 2^-11 / sqrt(3) / 1.44 = 9e-5 of an output.  What is added:
    the two operands of a weight hold it to 2^-22; a product of codes at bit 2 of a subnormal
    operand is cut below 2^10 2^-24 2^-2 = 2^-16 of the largest w s beside it, by half of that
    where it is cut at all, of 100 weights whose products with codes are 1 to 15: 100 2^-17 / 15 =
    5e-5 of the largest weight's share at the most; scores are off by 2^-19 or less.  A weight
    in one fp16 operand adds up to 2^-11 / sqrt(3) / 1.44 = 2e-4: up to 1.4 times."""
    lens = [100] * 6
    dev, table, kv = build(lens, hkv, dim, 16, torch.float16, 71)
    q = rounded(np.random.default_rng(8).normal(size=(len(lens), hq, dim)).astype(np.float32), torch.float16)
    U.say("attention half outputs", hq, hkv, dim)
    out, _ = attend(L, q, dev, table, lens, [1] * len(lens), 16, torch.float16, dim ** -0.5)
    out = out.float().cpu().numpy().astype(np.float64)
    want = np.stack([S.attention(q[b:b + 1], kv[b][0], kv[b][2], 100, dim ** -0.5, 0, ())[0][0] for b in range(len(lens))])
    own, rounding = np.square(out - want).mean(), np.square(want.astype(np.float16) - want).mean()
    assert own <= 1.1 ** 2 * rounding, (own / rounding) ** 0.5


@pytest.mark.parametrize("scale", [-0.1, 0.0, 2.0])
@pytest.mark.parametrize("rows", [1, 3, 40])
def test_any_finite_scale(L, scale, rows):
    """A negative scale turns the order of the scores, zero makes them equal; 2.0 makes them peaked."""
    lens = [300]
    dev, table, kv = build(lens, 2, 128, 16, torch.float16, 29)
    q = rounded(np.random.default_rng(3).normal(size=(rows, 8, 128)).astype(np.float32), torch.float16)
    U.say("attention scale", scale, rows)
    out, lse = attend(L, q, dev, table, lens, [rows], 16, torch.float16, scale)
    compare(out, lse, q, kv, lens, [rows], torch.float16, scale, picks=lambda n: {0, n // 2, n - 1})


def test_rows_past_the_promise_are_left(L):
    """More rows than max_rows: the first ones are computed at their own positions, the others of
    out and lse stay."""
    dev, table, kv = build([100], 2, 128, 16, torch.float16, 29)
    q = rounded(np.random.default_rng(3).normal(size=(9, 8, 128)).astype(np.float32), torch.float16)
    full, lf = attend(L, q, dev, table, [100], [9], 16, torch.float16, 0.1)
    for mr in (1, 2, 5):
        U.say("attention rows cut", mr)
        out, lse = attend(L, q, dev, table, [100], [9], 16, torch.float16, 0.1, 0, mr)
        # another number of rows is another cut of the work: equal up to its rounding
        compare(out[:mr], lse[:mr], q[:mr], [[x[:100 - 9 + mr] for x in kv[0]]], [100 - 9 + mr], [mr], torch.float16, 0.1)
        assert torch.all(out[mr:] == 9.0) and torch.all(lse[mr:] == 9.0)
    compare(full, lf, q, kv, [100], [9], torch.float16, 0.1)


def test_calls_side_by_side(L):
    """Attention and appends on two streams at once, each with its own workspace and cache: the
    results of running them one after the other."""
    lens = [6000, 900, 3000]
    sides = []
    for i in range(2):
        dev, table, _ = build(lens, 4, 128, 64, torch.bfloat16, 51 + i)
        q = cuda(rounded(np.random.default_rng(i).normal(size=(3, 16, 128)).astype(np.float32), torch.bfloat16), torch.bfloat16)
        size = L.mixllm_kv4_attention_workspace_bytes(3, 3, 16, 4, 128, 1, 6000)
        assert size
        sides.append(dict(q=q, dev=dev, table=cuda(table), out=torch.empty_like(q),
                          ws=torch.empty(size, dtype=torch.uint8, device="cuda"), stream=torch.cuda.Stream()))
    ln, cu = i32(lens), i32([0, 1, 2, 3])
    k = torch.randn(3, 4, 128, device="cuda").bfloat16()

    def run(s, stream):
        slots = s["table"][:, 0] * 64
        L.mixllm_kv4_append(k, k, slots, s["dev"], 64, stream=stream)
        L.mixllm_kv4_attention(s["q"], s["dev"], s["table"], ln, cu, s["out"], 64, 1, 6000, workspace=s["ws"], stream=stream)

    want = []
    for s in sides:
        run(s, None)
        want.append(s["out"].clone())
    torch.cuda.synchronize()
    U.say("attention side by side")
    for rep in range(20):
        for s in sides:
            s["out"].fill_(float("nan"))
        torch.cuda.synchronize()
        for s in sides:
            with torch.cuda.stream(s["stream"]):
                run(s, s["stream"] if rep % 2 else s["stream"].cuda_stream)
        torch.cuda.synchronize()
        for s, w in zip(sides, want):
            assert torch.equal(s["out"], w), rep


def test_a_row_that_is_not_finite_stays_alone(L):
    dev, table, kv = build([200], 2, 128, 16, torch.float16, 37)
    q = rounded(np.random.default_rng(3).normal(size=(5, 8, 128)).astype(np.float32), torch.float16)
    bad = q.copy()
    bad[2, 3, 7], bad[4, 0, 0] = np.nan, np.inf
    a, la = attend(L, q, dev, table, [200], [5], 16, torch.float16, 0.1)
    b, lb = attend(L, bad, dev, table, [200], [5], 16, torch.float16, 0.1)
    same = torch.ones(5, 8, dtype=torch.bool, device="cuda")
    same[2, 3] = same[4, 0] = False
    assert torch.equal(a[same], b[same]) and torch.equal(la[same], lb[same])
    assert not torch.isfinite(b[2, 3]).any()


def test_strided_query_and_output_and_no_lse(L):
    """q as a slice of a q/k/v row, out inside a wider buffer, no lse: the same bits."""
    lens, rows = [100, 40], [2, 1]
    dev, table, kv = build(lens, 2, 128, 16, torch.float16, 41)
    q = rounded(np.random.default_rng(3).normal(size=(3, 8, 128)).astype(np.float32), torch.float16)
    ref, _ = attend(L, q, dev, table, lens, rows, 16, torch.float16, 0.1)
    wide = torch.zeros((3, 8 * 128 + 512), dtype=torch.float16, device="cuda")
    qv = wide[:, :1024].view(3, 8, 128)
    qv.copy_(cuda(q, torch.float16))
    buf = torch.full((3, 2048), 9.0, dtype=torch.float16, device="cuda")
    big = cuda(np.concatenate([table, np.full((2, 9), 10 ** 9, np.int32)], 1))   # a table with wider rows
    L.mixllm_kv4_attention(qv, dev, big[:, :table.shape[1]], i32(lens), i32([0, 2, 3]), buf[:, 512:1536].view(3, 8, 128), 16, 2,
                           100, scale=0.1)
    assert torch.equal(buf[:, 512:1536].view(3, 8, 128), ref)
    assert torch.all(buf[:, :512] == 9.0) and torch.all(buf[:, 1536:] == 9.0)


def test_results_repeat_and_streams(L):
    """The same call twice gives the same bits, also on a stream of the caller's."""
    lens = [3000, 70]
    dev, table, _ = build(lens, 8, 128, 64, torch.bfloat16, 43)
    q = rounded(np.random.default_rng(3).normal(size=(2, 32, 128)).astype(np.float32), torch.bfloat16)
    a, la = attend(L, q, dev, table, lens, [1, 1], 64, torch.bfloat16, 0.1)
    b, lb = attend(L, q, dev, table, lens, [1, 1], 64, torch.bfloat16, 0.1)
    assert torch.equal(a, b) and torch.equal(la, lb)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c, lc = attend(L, q, dev, table, lens, [1, 1], 64, torch.bfloat16, 0.1)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(a, c) and torch.equal(la, lc)


def test_offsets_past_32_bits(L):
    """A cache over 4 GiB: pages at its far end are written, read and attended."""
    page, heads, dim = 1024, 8, 256
    pages = 2000
    cache = L.kv4_cache(pages, page, heads, dim)            # 4.7 GB
    assert cache.numel() > 1 << 32
    n = 1030
    table = np.array([[pages - 1, 0]], np.int32)
    k, v = key_values(n, heads, dim, torch.float16, 3)
    pos = np.arange(n)
    slots = i32(table[0, pos // page] * page + pos % page)
    U.say("attention far", cache.numel())
    L.mixllm_kv4_append(cuda(k, torch.float16), cuda(v, torch.float16), slots, cache, page)
    ko, vo = torch.empty((n, heads, dim), dtype=torch.float16, device="cuda"), torch.empty((n, heads, dim), dtype=torch.float16, device="cuda")
    L.mixllm_kv4_read(cache, slots, ko, vo, page)
    parts = []
    for x, o in ((k, ko), (v, vo)):
        c, s, m = S.kv4_quant(x)
        val = S.kv4_values(c, s, m)
        assert np.array_equal(o.cpu().numpy(), val.astype(np.float32).astype(np.float16))
        parts += [val, np.repeat(15 * s.astype(np.float64) + np.abs(m.astype(np.float64)), 64, -1).reshape(n, heads, dim)]
    q = rounded(np.random.default_rng(3).normal(size=(1, 8, dim)).astype(np.float32), torch.float16)
    out, lse = attend(L, q, cache, table, [n], [1], page, torch.float16, 0.06)
    compare(out, lse, q, [parts], [n], [1], torch.float16, 0.06)


def test_binding_refusals(L):
    dev, table, _ = build([40], 2, 128, 16, torch.float16, 1)
    q = torch.zeros((1, 8, 128), dtype=torch.float16, device="cuda")
    out, tb, lens, cu = torch.empty_like(q), cuda(table), i32([40]), i32([0, 1])
    ok = dict(q=q, cache=dev, table=tb, lens=lens, cu=cu, out=out, page=16, max_rows=1, max_len=40)
    L.mixllm_kv4_attention(**ok)
    for bad in (dict(q=q.float()), dict(out=out.bfloat16()), dict(page=32), dict(cache=dev.cpu()), dict(table=tb.long()),
                dict(lens=lens.long()), dict(cu=cu[:1]), dict(out=out[:, :4]), dict(lse=torch.empty(1, 8, dtype=torch.float64)),
                dict(table=tb.t().expand(3, 3))):
        with pytest.raises(ValueError):
            L.mixllm_kv4_attention(**{**ok, **bad})
    with pytest.raises(L.MixLLMError):
        L.mixllm_kv4_attention(**{**ok, "max_len": 9000})       # needs a workspace
    k = torch.zeros((2, 2, 128), dtype=torch.float16, device="cuda")
    for bad in (dict(k=k[:, :1]), dict(v=k.bfloat16()), dict(slots=i32([1])), dict(page=64),
                dict(k=k.transpose(0, 1).contiguous().transpose(0, 1))):
        with pytest.raises(ValueError):
            L.mixllm_kv4_append(**{**dict(k=k, v=k, slots=i32([1, 2]), cache=dev, page=16), **bad})
