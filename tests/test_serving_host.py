"""The norm's, the plan's and the cache calls' refusals, on the host: every bad argument comes
back as its status before any HIP call, so nothing here needs a GPU."""
import ctypes

import pytest

L = pytest.importorskip("weight_activation_quantized_amd.mixllm")

P = ctypes.c_void_p(0x10000)     # never dereferenced
ODD = ctypes.c_void_p(0x10001)
P4 = ctypes.c_void_p(0x10004)
P8 = ctypes.c_void_p(0x10008)
P2 = ctypes.c_void_p(0x10002)
NULL, SHAPE, GROUP, SPACE = -1, -2, -3, -5


def call(fn, base, **over):
    """`fn` with the named arguments of `base`, some replaced."""
    assert set(over) <= set(base), over
    return fn(*{**base, **over}.values())


NORM = dict(x=P, ldx=256, post=P, gate=P, ldgate=0, res=P, ldr=256, res_out=P, ldro=256, pre=P, y=P, ldy=256, aq=P,
            sa=P, asum=P, rowop=P, m=4, n=256, group=128, dtype=0, res_dtype=0, eps=1e-5, alpha=1.0, beta=1.0,
            stream=None)


@pytest.mark.parametrize("over,status", [
    (dict(group=64), GROUP), (dict(m=-1), SHAPE), (dict(n=0), SHAPE), (dict(n=65664), SHAPE), (dict(dtype=2), SHAPE),
    (dict(dtype=-1), SHAPE), (dict(res_dtype=1), SHAPE), (dict(dtype=1, res_dtype=0), SHAPE), (dict(res_dtype=3), SHAPE),
    (dict(eps=-1.0), SHAPE), (dict(eps=float("nan")), SHAPE), (dict(res=None), NULL), (dict(x=None), NULL),
    (dict(y=None, aq=None, sa=None, asum=None, rowop=None), NULL), (dict(pre=None), NULL), (dict(sa=None), NULL),
    (dict(aq=None), NULL), (dict(pre=None, y=None, aq=None, sa=None, asum=None, rowop=None, res_out=None), NULL),
    (dict(ldr=255), SHAPE), (dict(ldro=248), SHAPE), (dict(ldx=0), SHAPE), (dict(ldy=1), SHAPE), (dict(ldgate=128), SHAPE),
    (dict(x=ODD), SHAPE), (dict(res_dtype=2, res=P2), SHAPE), (dict(x=P2), SHAPE),            # int8 outputs: aligned
    (dict(ldx=257), SHAPE), (dict(n=200), SHAPE), (dict(aq=P8), SHAPE),
    (dict(m=0), 0), (dict(m=0, res=None), 0),
])
def test_norm_refusals(over, status):
    assert call(L.library_handle().mixllm_residual_norm, NORM, **over) == status


PLAN = dict(fresh=P, lens=P, b=4, table=P, ldt=8, width=8, pool=P, f=10, count=P, page=16, pages=64, lens_out=P,
            count_out=P, cu=P, slots=P, pos=P, tokens=7, stream=None)


@pytest.mark.parametrize("over,status", [
    (dict(b=-1), SHAPE), (dict(tokens=-1), SHAPE), (dict(f=-1), SHAPE), (dict(width=0), SHAPE), (dict(ldt=7), SHAPE),
    (dict(page=0), SHAPE), (dict(page=8), SHAPE), (dict(page=48), SHAPE), (dict(page=2048), SHAPE),
    (dict(page=-16), SHAPE), (dict(pages=0), SHAPE), (dict(pages=1 << 28, page=1024), SHAPE),
    (dict(width=1 << 27, ldt=1 << 27), SHAPE), (dict(b=1 << 29), SHAPE), (dict(fresh=None), NULL), (dict(lens=None), NULL),
    (dict(table=None), NULL), (dict(pool=None), NULL), (dict(count=None), NULL), (dict(lens_out=None), NULL),
    (dict(count_out=None), NULL), (dict(cu=None), NULL), (dict(slots=None), NULL), (dict(pos=None), NULL),
    (dict(slots=P2), SHAPE), (dict(table=ODD), SHAPE), (dict(b=0, tokens=0, cu=None), NULL),
])
def test_plan_refusals(over, status):
    assert call(L.library_handle().mixllm_kv_plan, PLAN, **over) == status


APPEND = dict(k=P, ldk=1024, v=P, ldv=1024, dtype=0, slots=P4, t=5, cache=P, nbytes=1 << 30, pages=64, page=16, heads=8,
              dim=128, stream=None)
READ = dict(cache=P, nbytes=1 << 30, pages=64, page=16, heads=8, dim=128, slots=P4, t=5, k=P, ldk=1024, v=P, ldv=1024,
            dtype=0, stream=None)


@pytest.mark.parametrize("over,status", [
    (dict(t=-1), SHAPE), (dict(dtype=2), SHAPE), (dict(dim=96), SHAPE), (dict(dim=0), SHAPE), (dict(page=24), SHAPE),
    (dict(heads=0), SHAPE), (dict(pages=0), SHAPE), (dict(heads=-8), SHAPE), (dict(cache=None), NULL), (dict(cache=P8), SHAPE),
    (dict(nbytes=64 * 8 * 16 * 144 - 1), SPACE), (dict(ldk=1016), SHAPE), (dict(ldv=1028), SHAPE), (dict(ldk=-1024), SHAPE),
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(slots=None), NULL), (dict(k=P8), SHAPE), (dict(slots=P2), SHAPE),
    (dict(heads=1 << 16, ldk=1 << 23, ldv=1 << 23, nbytes=1 << 60), SHAPE), (dict(pages=1 << 27), SHAPE), (dict(t=0), 0),
    (dict(t=0, k=None, cache=None), 0),
])
@pytest.mark.parametrize("base", [APPEND, READ], ids=["append", "read"])
def test_token_refusals(base, over, status):
    fn = L.library_handle().mixllm_kv4_append if base is APPEND else L.library_handle().mixllm_kv4_read
    assert call(fn, base, **over) == status


ATT = dict(q=P, ldq=4096, dtype=0, t=4, hq=32, cache=P, nbytes=1 << 40, pages=64, page=16, heads=8, dim=128, table=P4,
           ldt=16, width=16, lens=P4, cu=P4, b=4, max_rows=1, max_len=256, scale=0.1, window=0, out=P, ldo=4096, lse=P4,
           ws=P, ws_bytes=1 << 40, stream=None)


@pytest.mark.parametrize("over,status", [
    (dict(t=-1), SHAPE), (dict(b=-1), SHAPE), (dict(hq=0), SHAPE), (dict(hq=33), SHAPE), (dict(hq=4), SHAPE),
    (dict(heads=0), SHAPE), (dict(dim=80), SHAPE), (dict(page=20), SHAPE), (dict(pages=-1), SHAPE), (dict(dtype=2), SHAPE),
    (dict(max_rows=-1), SHAPE), (dict(max_len=-1), SHAPE), (dict(max_len=1 << 30), SHAPE), (dict(window=-1), SHAPE),
    (dict(width=0), SHAPE), (dict(ldt=15), SHAPE), (dict(ldq=4088), SHAPE), (dict(ldq=4100), SHAPE), (dict(ldo=0), SHAPE),
    (dict(q=None), NULL), (dict(cache=None), NULL), (dict(table=None), NULL), (dict(lens=None), NULL), (dict(cu=None), NULL),
    (dict(out=None), NULL), (dict(q=P8), SHAPE), (dict(out=P8), SHAPE), (dict(lse=P2), SHAPE), (dict(ws=P8), SHAPE),
    (dict(nbytes=64 * 8 * 16 * 144 - 1), SPACE), (dict(b=1 << 20, max_rows=1 << 20), SHAPE),
    (dict(max_len=8192, ws=None), NULL), (dict(max_len=8192, ws_bytes=16), SPACE),
    (dict(t=0), 0), (dict(b=0), 0), (dict(max_rows=0, q=None), 0),
])
def test_attention_refusals(over, status):
    assert call(L.library_handle().mixllm_kv4_attention, ATT, **over) == status


@pytest.mark.parametrize("over", [dict(t=1 << 30), dict(window=1 << 30), dict(b=65536), dict(max_rows=1 << 28),
                                  dict(b=60000, max_rows=2000)])
def test_attention_limits(over):
    assert call(L.library_handle().mixllm_kv4_attention, ATT, **over) == SHAPE


def test_sizes():
    assert L.mixllm_kv4_page_bytes(16, 8, 128) == 16 * 8 * 144
    assert L.mixllm_kv4_page_bytes(64, 1, 64) == 64 * 72
    for bad in ((15, 8, 128), (16, 0, 128), (16, 8, 100), (0, 8, 128)):
        assert L.mixllm_kv4_page_bytes(*bad) == 0
    ws = L.mixllm_kv4_attention_workspace_bytes
    assert ws(1, 1, 32, 8, 128, 1, 77) == 0                 # one workgroup per head does
    assert ws(0, 1, 32, 8, 128, 1, 100000) == 0
    assert ws(1, 1, 32, 7, 128, 1, 100000) == 0             # refused shapes have none
    long = ws(1, 1, 32, 8, 128, 1, 100000)
    assert 0 < long < 1 << 26
    # a window bounds what is read, whatever the length
    assert ws(1, 1, 32, 8, 128, 1, 100000, 64) == ws(1, 1, 32, 8, 128, 1, 1000, 64)


def test_binding_refuses_what_is_not_a_gpu_tensor():
    torch = pytest.importorskip("torch")
    z = torch.zeros(4, 256, dtype=torch.float16)
    with pytest.raises(ValueError):
        L.mixllm_residual_norm(z, z, z[0], y=z)
    with pytest.raises(ValueError):
        L.mixllm_residual_norm(None, z, None, y=z)
    with pytest.raises(ValueError):
        L.mixllm_kv4_append(z.view(4, 2, 128), z.view(4, 2, 128), torch.zeros(4, dtype=torch.int32),
                            torch.zeros(1, 2, 16 * 144, dtype=torch.uint8), 16)
    with pytest.raises(ValueError):
        L.kv4_cache(4, 20, 8, 128, device="cpu")
    assert L.kv4_cache(3, 16, 2, 64, device="cpu").shape == (3, 2, 16 * 72)
