"""The norms of queries and keys with the rotation by position, on the GPU against the oracle.

Per element, with e = 2^-24: the sum of a head's squares is off by at most (dim / 2 + 8) e of itself (each
lane adds at most 8 products, the lanes are a tree: 16 roundings at most; dim / 2 + 8 is more), its
root by half that, the products with the weight by 3 e; the reduced angle is rounded once to fp32 (pi
e) and its cosine and sine are within 4 e; each result is a sum of two products.  So |out - exact| <=
(dim / 4 + 16) e (|a| + |b|) before the last rounding, which adds half a step of the type."""
import numpy as np
import pytest

from oracle import eight_bit_oracle as E
from tests import gpu_util as U
from tests.test_gpu_kv4 import cuda, i32, rounded

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def L():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    from weight_activation_quantized_amd import mixllm
    return mixllm


def inputs(t, hq, hkv, dim, dtype, seed, norm=True):
    rng = np.random.default_rng(seed)
    q, k = (rounded((rng.normal(size=(t, h, dim)) * rng.choice([0.1, 1, 30], size=(t, h, 1))).astype(np.float32), dtype)
            for h in (hq, hkv))
    w = [rounded((1 + 0.3 * rng.normal(size=dim)).astype(np.float32), dtype) if norm else None for _ in range(2)]
    return q, k, w[0], w[1]


def check(got, x, pos, freq, norm, eps, neighbours, dtype):
    want, size = E.head_norm_rotate(x, pos, freq, norm, eps, neighbours)
    f = torch.finfo(dtype)
    tol = (x.shape[-1] / 4 + 16) * 2.0 ** -24 * size
    tol = tol + f.eps / 2 * (np.abs(want) + tol) + float(f.smallest_normal) * f.eps / 2
    err = np.abs(got.double().cpu().numpy() - want)
    assert np.all(err <= tol), (np.unravel_index((err - tol).argmax(), err.shape), (err / tol).max())


def run(L, q, k, pos, freq, wq, wk, dtype, eps=1e-6, neighbours=False, **kw):
    q, k = (None if x is None else cuda(x, dtype) for x in (q, k))
    w = [None if x is None else cuda(x, dtype) for x in (wq, wk)]
    f = None if freq is None else cuda(np.asarray(freq, np.float32))
    qo, ko = (None if x is None else torch.full_like(x, 7.0) for x in (q, k))
    L.mixllm_head_norm_rotate(q, k, i32(pos), f, qo, ko, *w, eps=eps, neighbours=neighbours, **kw)
    return qo, ko


def frequencies(rot, base=10000.0):
    return (base ** (-np.arange(0, rot, 2) / max(rot, 1))).astype(np.float32)


@pytest.mark.parametrize("neighbours", [False, True])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("hq,hkv,dim,rot", [(32, 8, 128, 128), (5, 1, 64, 64), (4, 2, 256, 64), (3, 3, 80, 80), (2, 1, 96, 40),
                                            (1, 1, 512, 512), (1, 1, 8, 8), (1, 1, 2, 2), (7, 2, 50, 50), (2, 2, 66, 14),
                                            (3, 1, 40, 12), (9, 5, 128, 0), (64, 8, 128, 128), (2, 1, 510, 510)])
def test_norm_and_rotation(L, hq, hkv, dim, rot, dtype, neighbours):
    U.say("rotate", hq, hkv, dim, rot, dtype, neighbours)
    t = 5
    q, k, wq, wk = inputs(t, hq, hkv, dim, dtype, dim + rot)
    pos = np.array([0, 1, 77, 131071, 2 ** 20 + 3], np.int32)
    freq = frequencies(rot) if rot else None
    qo, ko = run(L, q, k, pos, freq, wq, wk, dtype, 1e-5, neighbours)
    check(qo, q, pos, freq, wq, 1e-5, neighbours, dtype)
    check(ko, k, pos, freq, wk, 1e-5, neighbours, dtype)


@pytest.mark.parametrize("which", ["both", "queries", "keys", "none"])
@pytest.mark.parametrize("dim", [128, 50])
def test_norms_that_are_not_there(L, which, dim):
    dtype = torch.float16
    q, k, wq, wk = inputs(3, 6, 2, dim, dtype, 4)
    wq, wk = wq if which in ("both", "queries") else None, wk if which in ("both", "keys") else None
    pos, freq = [3, 4, 5], frequencies(dim)
    qo, ko = run(L, q, k, pos, freq, wq, wk, dtype)
    check(qo, q, pos, freq, wq, 1e-6, False, dtype)
    check(ko, k, pos, freq, wk, 1e-6, False, dtype)


@pytest.mark.parametrize("t", [1, 2, 1023, 1024, 1500])
def test_numbers_of_tokens(L, t):
    U.say("rotate tokens", t)
    dtype = torch.bfloat16
    q, k, wq, wk = inputs(t, 9, 2, 64, dtype, t)
    pos = np.random.default_rng(t).integers(0, 5000, t).astype(np.int32)
    qo, ko = run(L, q, k, pos, frequencies(64), wq, wk, dtype)
    check(qo, q, pos, frequencies(64), wq, 1e-6, False, dtype)
    check(ko, k, pos, frequencies(64), wk, 1e-6, False, dtype)


def test_far_and_negative_positions(L):
    """Angles of many turns: the last frequencies of fp32 would leave them off by whole radians."""
    dtype = torch.float16
    pos = np.array([2 ** 31 - 1, -2 ** 31, -1, -5000, 2 ** 30 + 12345, 16777217], np.int32)
    freq = np.array([1.0, 0.99999994, 0.333333343, 1e-3, 7.0, 0.0], np.float32)
    q, k, _, _ = inputs(len(pos), 2, 1, 16, dtype, 9, norm=False)
    for neighbours in (False, True):
        qo, ko = run(L, q, k, pos, freq, None, None, dtype, neighbours=neighbours)
        check(qo, q, pos, freq, None, 0, neighbours, dtype)
        check(ko, k, pos, freq, None, 0, neighbours, dtype)


def test_queries_or_keys_alone(L):
    dtype = torch.float16
    q, k, wq, wk = inputs(4, 3, 2, 128, dtype, 1)
    qo, none = run(L, q, None, [1, 2, 3, 4], frequencies(128), wq, None, dtype)
    assert none is None
    check(qo, q, [1, 2, 3, 4], frequencies(128), wq, 1e-6, False, dtype)
    none, ko = run(L, None, k, [1, 2, 3, 4], frequencies(128), None, wk, dtype)
    check(ko, k, [1, 2, 3, 4], frequencies(128), wk, 1e-6, False, dtype)


@pytest.mark.parametrize("dim,pad", [(128, 0), (128, 3), (96, 8), (34, 1)])
def test_slices_of_one_row_in_place(L, dim, pad):
    """Queries and keys as slices of a q/k/v product, turned where they are; what lies beside
    them stays."""
    U.say("rotate in place", dim, pad)
    dtype, t, hq, hkv = torch.float16, 6, 5, 2
    q, k, wq, wk = inputs(t, hq, hkv, dim, dtype, 3)
    row = torch.full((t, pad + (hq + 2 * hkv) * dim + 5), 3.0, dtype=dtype, device="cuda")
    qv = row[:, pad:pad + hq * dim].view(t, hq, dim)
    kv = row[:, pad + hq * dim:pad + (hq + hkv) * dim].view(t, hkv, dim)
    qv.copy_(cuda(q, dtype))
    kv.copy_(cuda(k, dtype))
    pos = [9, 8, 7, 6, 5, 4]
    L.mixllm_head_norm_rotate(qv, kv, i32(pos), cuda(frequencies(dim)), q_norm=cuda(wq, dtype), k_norm=cuda(wk, dtype))
    check(qv, q, pos, frequencies(dim), wq, 1e-6, False, dtype)
    check(kv, k, pos, frequencies(dim), wk, 1e-6, False, dtype)
    assert torch.all(row[:, :pad] == 3.0) and torch.all(row[:, pad + (hq + hkv) * dim:] == 3.0)


@pytest.mark.parametrize("dim", [128, 50])
def test_one_heads_numbers_stay_there(L, dim):
    """A head of infinities or NaN, or of zeros, leaves the others as they are."""
    dtype = torch.float16
    q, k, wq, wk = inputs(4, 4, 2, dim, dtype, 8)
    pos, freq = [0, 5, 6, 7], frequencies(dim)
    want, _ = run(L, q, k, pos, freq, wq, wk, dtype)
    q2 = q.copy()
    q2[1, 1, 3], q2[2, 0, 0], q2[3, 3] = np.inf, np.nan, 0.0
    got, _ = run(L, q2, k, pos, freq, wq, wk, dtype)
    same = torch.ones(4, 4, dtype=torch.bool)
    same[1, 1] = same[2, 0] = same[3, 3] = False
    assert torch.equal(got[same.cuda()], want[same.cuda()])
    assert got[2, 0].isnan().all() and not got[3, 3].any()


def test_nothing_to_do(L):
    q = torch.empty((0, 4, 64), dtype=torch.float16, device="cuda")
    L.mixllm_head_norm_rotate(q, None, i32([]), cuda(frequencies(64)))
    q = torch.ones((3, 4, 64), dtype=torch.float16, device="cuda")
    L.mixllm_head_norm_rotate(q, None, None, None)       # no norm, no rotation
    assert torch.all(q == 1.0)


def test_refuses(L):
    q = torch.zeros((3, 4, 64), dtype=torch.float16, device="cuda")
    pos, f = i32([0, 1, 2]), cuda(frequencies(64))
    bad = [lambda: L.mixllm_head_norm_rotate(q, q[:2], pos, f), lambda: L.mixllm_head_norm_rotate(q, None, pos[:2], f),
           lambda: L.mixllm_head_norm_rotate(q, None, pos.long(), f), lambda: L.mixllm_head_norm_rotate(q, None, pos, f.double()),
           lambda: L.mixllm_head_norm_rotate(q, None, None, f), lambda: L.mixllm_head_norm_rotate(None, None, pos, f),
           lambda: L.mixllm_head_norm_rotate(q.float(), None, pos, f), lambda: L.mixllm_head_norm_rotate(q.cpu(), None, pos, f),
           lambda: L.mixllm_head_norm_rotate(q, q.bfloat16(), pos, f), lambda: L.mixllm_head_norm_rotate(q[0], None, pos, f),
           lambda: L.mixllm_head_norm_rotate(q, None, pos, f, q_norm=f[:8].half()),
           lambda: L.mixllm_head_norm_rotate(q, None, pos, f, k_norm=q[0, 0]),
           lambda: L.mixllm_head_norm_rotate(q.transpose(1, 2), None, pos, f)]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    for kw in (dict(inv_freq=cuda(frequencies(66))), dict(inv_freq=f, eps=-1.0)):
        with pytest.raises(L.MixLLMError):
            L.mixllm_head_norm_rotate(q, None, pos, **kw)


def test_replayed_beside_eager_calls_on_another_stream(L):
    """A captured call in a graph, replayed while eager calls run on another stream."""
    dtype = torch.float16
    q, k, wq, wk = inputs(40, 8, 2, 128, dtype, 2)
    pos, f = i32(np.arange(40)), cuda(frequencies(128))
    q, k, wq, wk = (cuda(x, dtype) for x in (q, k, wq, wk))
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    want = [torch.empty_like(q), torch.empty_like(k)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    L.mixllm_head_norm_rotate(q, k, pos, f, qo, ko, wq, wk, stream=s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        L.mixllm_head_norm_rotate(q, k, pos, f, qo, ko, wq, wk)
    for i in range(5):
        q.mul_(1.01)
        qo.fill_(0)
        g.replay()
        L.mixllm_head_norm_rotate(q, k, pos, f, *want, wq, wk)
        torch.cuda.synchronize()
        assert torch.equal(qo, want[0]) and torch.equal(ko, want[1]), i
