"""The loops that long calls of the 8-bit kernels spend their time in, on the GPU against the oracle:
batches of pages that follow one another, stages that come round again, head groups that one wave
takes in turn.

Sizes are chosen by what one workgroup is left with, which each test works out from the workspace
(chunks along the tokens) or from the kernels' own rules and asserts.  Tolerances are those of the
operators' own tests; fp16 outputs are held to the error of their own rounding too: a weight times a
value's scale is kept to 2^-22, so what is left beside the output's rounding are fp32 sums, whose
error may add 0.66 of it in the squares (1.2^2 = 1 + 0.66^2).  With weights of 11 bits, whose roundings
an output of many values sums up to about its own rounding, it would be 1.4."""
import numpy as np
import pytest

from oracle import eight_bit_oracle as E
from oracle import serving_oracle as S
from tests import gpu_util as U
from tests import test_gpu_gemm8 as G
from tests import test_gpu_kv4 as K
from tests import test_gpu_kv8 as V
from tests import test_gpu_rotate as O
from tests.test_eight_bit_tiles import LOOPS, STRIDED, picked
from tests.test_gpu_kv4 import cuda

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def L():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    from weight_activation_quantized_amd import mixllm
    return mixllm


def chunks(L, t, b, hq, hkv, dim, rows, length, window, tile_rows):
    """Along the tokens of a tile, from the workspace of all chunks' rows."""
    tiles = -(-rows * (hq // hkv) // tile_rows)
    size = L.mixllm_kv8_attention_workspace_bytes(t, b, hq, hkv, dim, rows, length, window)
    return max(size // (b * tiles * hkv * tile_rows * (dim + 2) * 4), 1)


def own_rounding(out, q, kv, lens, rows, scale, window, picks):
    """Root mean squares of the outputs' error and of that of the exact outputs' rounding to fp16."""
    err, own, at = [], [], 0
    o = out.double().cpu().numpy()
    for b, n in enumerate(lens):
        for i in range(rows[b]):
            upto = n - rows[b] + i + 1
            if i in picks(rows[b]) and upto > 200:
                want = S.attention(q[at + i:at + i + 1], kv[b][0][:upto], kv[b][2][:upto], upto, scale, window)[0][0]
                err.append(o[at + i] - want)
                own.append(want.astype(np.float16).astype(np.float64) - want)
        at += rows[b]
    return [float(np.sqrt(np.mean(np.square(x)))) for x in (err, own)]


# (heads of queries, key/value heads, dim, rows, requests, rows of a tile)
SINGLES = [(16, 8, 128, 1, 64, 16), (32, 2, 64, 1, 256, 16), (6, 3, 256, 2, 171, 16), (24, 4, 64, 4, 128, 32),
           (20, 4, 128, 8, 64, 32), (12, 4, 256, 8, 64, 16)]


@pytest.mark.parametrize("hq,hkv,dim,rows,requests,tile_rows", SINGLES)
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("window", [0, 4500])
def test_decodes_that_no_chunk_cuts(L, hq, hkv, dim, rows, requests, tile_rows, dtype, window):
    """Workgroups that walk thousands of tokens: many steps of a wave, and more than the 4096 tokens
    whose pages and scales it fetches at once, twice over for the longest request."""
    page = 64
    lens = [8700, 4097 + rows, 4224, 700] + [1 + (b * 7) % 40 for b in range(requests - 4)]
    rng = np.random.default_rng(dim + rows)
    order = rng.permutation(requests)
    lens = [lens[i] for i in order]
    U.say("attention8 unsplit", hq, hkv, dim, rows, requests, dtype, window)
    dev, table, kv = V.build(lens, hkv, dim, page, dtype, 61)
    q = V.queries(requests * rows, hq, dim, dtype, 15)
    assert chunks(L, len(q), requests, hq, hkv, dim, rows, max(lens), window, tile_rows) == 1
    out, lse = V.attend(L, q, dev, table, lens, [rows] * requests, page, dtype, dim ** -0.5, window)
    K.compare(out, lse, q, kv, lens, [rows] * requests, dtype, dim ** -0.5, window)
    if dtype == torch.float16:
        err, own = own_rounding(out, q, kv, lens, [rows] * requests, dim ** -0.5, window, range)
        assert err <= 1.2 * own, (err, own)


# (group, key/value heads, rows of the largest request, requests, window, chunks); 1024 tokens' pages at once
PROMPTS = [(4, 16, 40, 9, 0, 1), (4, 16, 40, 9, 1300, 1), (2, 4, 150, 40, 0, 1), (4, 16, 40, 6, 0, 2), (1, 5, 200, 25, 2100, 2)]


@pytest.mark.parametrize("group,hkv,rows,requests,window,splits", PROMPTS)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_prompts_over_more_than_one_batch_of_pages(L, group, hkv, rows, requests, window, splits, dim, dtype):
    page, hq = 32, hkv * group
    lens = [2500, 4700, 1025, 3333] + [rows + (b * 13) % 50 for b in range(requests - 4)]
    fresh = [rows, rows - 7, rows, rows - 1] + [rows - b % 9 for b in range(requests - 4)]
    U.say("attention8 long chunks", group, hkv, rows, requests, window, dim, dtype)
    tile = 128 if dim == 256 else 256
    if dim == 256 and splits == 2:
        requests = max(4, requests // -(-rows * group // tile))
        lens, fresh = lens[:requests], fresh[:requests]
    got = chunks(L, sum(fresh), requests, hq, hkv, dim, rows, 4700, window, tile)
    assert got == splits and (min(4700, window + rows if window else 4700) // got) > 1024, got
    dev, table, kv = V.build(lens, hkv, dim, page, dtype, 67)
    q = V.queries(sum(fresh), hq, dim, dtype, 16)
    out, lse = V.attend(L, q, dev, table, lens, fresh, page, dtype, dim ** -0.5, window, max_rows=rows)
    picks = lambda n: {0, n // 3, n - 1}  # noqa: E731
    K.compare(out[:sum(fresh[:5])], lse[:sum(fresh[:5])], q, kv[:5], lens[:5], fresh[:5], dtype, dim ** -0.5, window, picks=picks)
    if dtype == torch.float16:
        err, own = own_rounding(out, q, kv[:4], lens[:4], fresh[:4], dim ** -0.5, window, picks)
        assert err <= 1.2 * own, (err, own)


@pytest.mark.parametrize("t,hq,hkv,dim,rot", [(4100, 40, 8, 64, 64), (2100, 60, 9, 128, 128), (4100, 25, 4, 128, 64),
                                              (1500, 14, 3, 256, 256), (4100, 5, 4, 512, 512), (4100, 64, 8, 64, 0)])
@pytest.mark.parametrize("neighbours", [False, True])
@pytest.mark.parametrize("inside", [False, True])
def test_head_groups_in_turn(L, t, hq, hkv, dim, rot, neighbours, inside):
    """Waves that take two head groups and more, whose loads run two ahead of what is written (also
    where that is the input)."""
    dtype = torch.bfloat16 if neighbours else torch.float16
    per = 64 // {64: 4, 128: 8, 256: 16, 512: 32}[dim]        # heads that a wave takes at a time
    groups = -(-(hq + hkv) // per)
    parts = min(-(-4096 // t), groups)
    assert -(-groups // parts) >= 2
    U.say("rotate groups", t, hq, hkv, dim, rot, neighbours, inside)
    gen = torch.Generator("cuda").manual_seed(t + dim)
    q, k, wq, wk = ((torch.randn(shape, generator=gen, device="cuda") + at).to(dtype)
                    for shape, at in (((t, hq, dim), 0), ((t, hkv, dim), 0), ((dim,), 1), ((dim,), 1)))
    pos = torch.randint(0, 100000, (t,), generator=gen, device="cuda").to(torch.int32)
    freq = cuda(O.frequencies(rot)) if rot else None
    qo, ko = (x.clone() if inside else torch.full_like(x, 7.0) for x in (q, k))
    L.mixllm_head_norm_rotate(*((qo, ko) if inside else (q, k)), pos, freq, qo, ko, wq, wk, neighbours=neighbours)
    some = sorted({*range(64), *range(t - 64, t), *range(0, t, 37)})       # a wave has one token: all are alike
    host = [None if x is None else x.float().cpu().numpy() for x in (q[some], k[some], pos[some], freq, wq, wk)]
    O.check(qo[some], host[0], host[2].astype(np.int32), host[3], host[4], 1e-6, neighbours, dtype)
    O.check(ko[some], host[1], host[2].astype(np.int32), host[3], host[5], 1e-6, neighbours, dtype)


def product(m, n, k, seed):
    rng = np.random.default_rng(seed)
    return (G.codes(rng, m, k), G.codes(rng, n, k), (rng.random(m) * 2e-4 + 1e-5).astype(np.float32),
            (rng.random(n) * 2e-3 + 1e-5).astype(np.float32))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("tile,m,n,k", LOOPS)
def test_stages_that_come_round(L, tile, m, n, k, dtype):
    assert picked(m, n, k) == tile
    U.say("gemm8 stages", tile, m, n, k, dtype)
    aq, w, sa, sw = product(m, n, k, m + n + k)
    y = torch.full((m, n), 9.0, dtype=dtype, device="cuda")
    L.mixllm_gemm_w8a8(cuda(aq), cuda(sa), cuda(w), cuda(sw), y)
    G.check(y, aq, sa, w, sw, dtype)


@pytest.mark.parametrize("tile,m,n,k", STRIDED)
@pytest.mark.parametrize("pad", [(16, 16, 1), (32, 48, 8), (16, 0, 3)])
def test_stages_of_rows_inside_wider_ones(L, tile, m, n, k, pad):
    assert picked(m, n, k) == tile
    U.say("gemm8 stages, strided", tile, m, n, k, pad)
    aq, w, sa, sw = product(m, n, k, m + n)
    a2 = torch.full((m, k + pad[0]), 101, dtype=torch.int8, device="cuda")
    w2 = torch.full((n, k + pad[1]), 99, dtype=torch.int8, device="cuda")
    y2 = torch.full((m, n + pad[2] + 2), 9.0, dtype=torch.float16, device="cuda")
    a2[:, :k], w2[:, :k] = cuda(aq), cuda(w)
    y = y2[:, pad[2]:pad[2] + n]
    L.mixllm_gemm_w8a8(a2[:, :k], cuda(sa), w2[:, :k], cuda(sw), y)
    G.check(y, aq, sa, w, sw, torch.float16)
    assert torch.all(y2[:, :pad[2]] == 9.0) and torch.all(y2[:, pad[2] + n:] == 9.0)
