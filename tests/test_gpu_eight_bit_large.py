"""The 8-bit operators where places in their tensors pass 32 bits: caches of more than 4 GB, rows far
behind one another, products with more outputs than that.  Only some rows are computed again; tolerances
are those of the operators' own tests."""
import numpy as np
import pytest

from oracle import eight_bit_oracle as E
from tests import gpu_util as U
from tests import test_gpu_gemm8 as G
from tests import test_gpu_kv4 as K
from tests import test_gpu_kv8 as V
from tests import test_gpu_rotate as O
from tests.test_gpu_kv4 import cuda, i32, key_values, rounded

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def L():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    from weight_activation_quantized_amd import mixllm
    return mixllm


@pytest.mark.parametrize("dim,heads,page", [(128, 8, 1024), (64, 2, 64), (256, 4, 16)])
@pytest.mark.parametrize("rows", [1, 70])
def test_a_cache_of_more_than_4_gb(L, dim, heads, page, rows):
    dtype, group = torch.float16, 2
    per = heads * E.block_bytes(page, dim)
    pages = (5 << 30) // per
    U.say("cache of 5 GB", dim, heads, page, rows)
    cache = torch.full((pages, heads, E.block_bytes(page, dim)), 255, dtype=torch.uint8, device="cuda")
    n, used = 150, -(-150 // page)
    # requests in the first pages, on both sides of 2^31 and of 2^32 bytes, and in the last ones
    at = [0, (1 << 31) // per - 1, (1 << 31) // per + used, (1 << 32) // per - 1, (1 << 32) // per + used, pages - used]
    table = np.array([np.arange(p, p + used) for p in at], np.int32)
    kv = [key_values(n, heads, dim, dtype, 3 + b) for b in range(len(at))]
    slots = np.concatenate([V.slots_of(t, np.arange(n), page) for t in table])
    k, v = (cuda(np.concatenate([x[part] for x in kv]), dtype) for part in range(2))
    L.mixllm_kv8_append(k, v, i32(slots), cache, page)
    small = cache[torch.from_numpy(table).long().flatten().cuda()].cpu().numpy()
    want = np.full_like(small, 255)
    mine = np.arange(len(at) * used).reshape(len(at), used)
    E.kv8_write(want, np.concatenate([V.slots_of(t, np.arange(n), page) for t in mine]), k.float().cpu().numpy(),
                v.float().cpu().numpy(), page)
    assert np.array_equal(small, want)
    ko, vo = torch.full_like(k, 9.0), torch.full_like(v, 9.0)
    L.mixllm_kv8_read(cache, i32(slots), ko, vo, page)
    vals, _ = E.kv8_values(want, np.concatenate([V.slots_of(t, np.arange(n), page) for t in mine]), page, dim)
    for got, val in zip((ko, vo), vals):
        assert np.array_equal(got.float().cpu().numpy(), rounded(val.astype(np.float32), dtype))
    lens, fresh = [n] * len(at), [rows] * len(at)
    q = V.queries(sum(fresh), heads * group, dim, dtype, 5)
    out, lse = V.attend(L, q, cache, table, lens, fresh, page, dtype, 0.1)
    K.compare(out, lse, q, [V.values_of(want, t, n, page, dim) for t in mine], lens, fresh, dtype, 0.1,
              picks=lambda m: {0, m // 2, m - 1})
    # nothing else was written: what lies in between, by blocks of 256 pages
    left = torch.ones(pages, dtype=torch.bool, device="cuda")
    left[torch.from_numpy(table).long().flatten().cuda()] = False
    words = cache.view(pages, -1)
    assert all(bool((words[i:i + 256][left[i:i + 256]] == 255).all()) for i in range(0, pages, 256))


@pytest.mark.parametrize("dim", [128, 50])
def test_rows_of_the_rotation_that_lie_far_apart(L, dim):
    t, hq, hkv, step, dtype = 300, 4, 2, 1 << 24, torch.float16
    U.say("rotate, far apart", dim)
    q, k, wq, wk = O.inputs(t, hq, hkv, dim, dtype, 5)
    memory = torch.zeros((t, step), dtype=dtype, device="cuda")          # 10 GB; the last rows begin behind 2^32 values
    qd, kd = memory[:, :hq * dim].view(t, hq, dim), memory[:, 8192:8192 + hkv * dim].view(t, hkv, dim)
    qd.copy_(cuda(q, dtype))
    kd.copy_(cuda(k, dtype))
    pos, f = np.arange(t, dtype=np.int32), O.frequencies(dim)
    L.mixllm_head_norm_rotate(qd, kd, i32(pos), cuda(f), q_norm=cuda(wq, dtype), k_norm=cuda(wk, dtype))
    O.check(qd, q, pos, f, wq, 1e-6, False, dtype)
    O.check(kd, k, pos, f, wk, 1e-6, False, dtype)


def test_rows_of_the_cache_calls_that_lie_far_apart(L):
    t, heads, dim, page, dtype = 300, 2, 64, 16, torch.bfloat16
    U.say("append8, read8, far apart")
    k, v = key_values(t, heads, dim, dtype, 5)
    memory = torch.zeros((t, 1 << 24), dtype=dtype, device="cuda")
    kd, vd = memory[:, :heads * dim].view(t, heads, dim), memory[:, 8192:8192 + heads * dim].view(t, heads, dim)
    kd.copy_(cuda(k, dtype))
    vd.copy_(cuda(v, dtype))
    want = V.new_cache(20, heads, page, dim)
    cache, slots = cuda(want), np.arange(t)
    L.mixllm_kv8_append(kd, vd, i32(slots), cache, page)
    E.kv8_write(want, slots, k, v, page)
    assert np.array_equal(cache.cpu().numpy(), want)
    kd.zero_()
    vd.zero_()
    L.mixllm_kv8_read(cache, i32(slots), kd, vd, page)
    for got, val in zip((kd, vd), E.kv8_values(want, slots, page, dim)[0]):
        assert np.array_equal(got.float().cpu().numpy(), rounded(val.astype(np.float32), dtype))


@pytest.mark.parametrize("m,n,k", [(36000, 300, 131072), (300, 36000, 131072), (70000, 40000, 16)])
def test_products_and_rows_past_32_bits(L, m, n, k):
    """Activations, weights or outputs of more than 4 GB."""
    dtype = torch.bfloat16
    U.say("gemm8, past 32 bits", m, n, k)
    gen = torch.Generator("cuda").manual_seed(m)
    make = lambda r: torch.randint(-127, 128, (r, k), dtype=torch.int8, device="cuda", generator=gen)  # noqa: E731
    aq, w = make(m), make(n)
    sa, sw = (torch.rand(x, device="cuda", generator=gen) * 1e-3 + 1e-5 for x in (m, n))
    y = torch.full((m, n), 9.0, dtype=dtype, device="cuda")
    L.mixllm_gemm_w8a8(aq, sa, w, sw, y)
    pick = lambda x: torch.tensor(sorted({0, 1, x // 2, *range(x - 40, x)}), device="cuda")  # noqa: E731
    i, j = pick(m), pick(n)
    host = lambda x: x.cpu().numpy()  # noqa: E731
    G.check(y[i][:, j], host(aq[i]), host(sa[i]), host(w[j]), host(sw[j]), dtype)
    assert not bool((y == 9.0).all(1).any())


def test_quantized_rows_past_32_bits(L):
    m, k, dtype = 40000, 131072, torch.float16
    U.say("quant rows, past 32 bits")
    gen = torch.Generator("cuda").manual_seed(1)
    a = torch.empty((m, k), dtype=dtype, device="cuda").normal_(generator=gen)
    q, s = torch.full((m, k), 77, dtype=torch.int8, device="cuda"), torch.zeros(m, device="cuda")
    L.mixllm_quant_rows(a, q, s)
    i = torch.tensor([0, 16383, 16384, 32767, 32768, m - 1], device="cuda")
    wq, ws = E.quant_rows(a[i].float().cpu().numpy())
    assert np.array_equal(q[i].cpu().numpy(), wq) and np.array_equal(s[i].cpu().numpy(), ws) and bool((s > 0).all())
