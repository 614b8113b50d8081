"""The refusals of the 8-bit operators, on the host: every bad argument comes back as its status
before any HIP call, so nothing here needs a GPU.  And the oracle's own hand cases."""
import numpy as np
import pytest

from oracle import eight_bit_oracle as E
from tests.test_serving_host import APPEND, ATT, NULL, ODD, P, P2, P4, P8, READ, SHAPE, SPACE, call

L = pytest.importorskip("weight_activation_quantized_amd.mixllm")

ROTATE = dict(q=P, ldq=4096, k=P, ldk=1024, qo=P, ldqo=4096, ko=P, ldko=1024, pos=P4, freq=P4, qn=P, kn=P, t=5, hq=32, hkv=8,
              dim=128, rot=128, neighbours=0, dtype=0, eps=1e-6, stream=None)


@pytest.mark.parametrize("over,status", [
    (dict(t=-1), SHAPE), (dict(hq=-1), SHAPE), (dict(hkv=-1), SHAPE), (dict(dim=0), SHAPE), (dict(dim=127), SHAPE),
    (dict(dim=514, rot=2, ldq=1 << 20, ldqo=1 << 20, ldk=1 << 20, ldko=1 << 20), SHAPE), (dict(rot=-2), SHAPE), (dict(rot=130), SHAPE),
    (dict(rot=3), SHAPE), (dict(neighbours=2), SHAPE), (dict(dtype=2), SHAPE), (dict(eps=-1.0), SHAPE),
    (dict(eps=float("nan")), SHAPE), (dict(hq=65536, ldq=1 << 30, ldqo=1 << 30), SHAPE), (dict(t=1 << 24), SHAPE),
    (dict(t=1 << 22), SHAPE), (dict(q=None), NULL), (dict(k=None), NULL), (dict(qo=None), NULL), (dict(ko=None), NULL),
    (dict(pos=None), NULL), (dict(freq=None), NULL), (dict(hq=0), NULL), (dict(hkv=0), NULL), (dict(ldq=4095), SHAPE),
    (dict(ldqo=0), SHAPE), (dict(ldk=-1), SHAPE), (dict(ldko=1023), SHAPE), (dict(q=ODD), SHAPE), (dict(kn=ODD), SHAPE),
    (dict(pos=P2), SHAPE), (dict(freq=P2), SHAPE), (dict(t=0), 0), (dict(t=0, q=None), 0), (dict(hq=0, hkv=0, qn=None, kn=None), 0),
])
def test_rotate_refusals(over, status):
    assert call(L.library_handle().mixllm_head_norm_rotate, ROTATE, **over) == status


BLOCK = 2 * 16 * 128 + 128


@pytest.mark.parametrize("over,status", [
    (dict(t=-1), SHAPE), (dict(dtype=2), SHAPE), (dict(dim=96), SHAPE), (dict(dim=0), SHAPE), (dict(page=24), SHAPE),
    (dict(page=8), SHAPE), (dict(page=2048), SHAPE),
    (dict(heads=0), SHAPE), (dict(pages=0), SHAPE), (dict(heads=-8), SHAPE), (dict(cache=None), NULL), (dict(cache=P8), SHAPE),
    (dict(nbytes=64 * 8 * BLOCK - 1), SPACE), (dict(ldk=1016), SHAPE), (dict(ldv=1028), SHAPE), (dict(ldk=-1024), SHAPE),
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(slots=None), NULL), (dict(k=P8), SHAPE), (dict(slots=P2), SHAPE),
    (dict(heads=1 << 16, ldk=1 << 23, ldv=1 << 23, nbytes=1 << 60), SHAPE), (dict(pages=1 << 27), SHAPE),
    (dict(t=1 << 25, heads=64, ldk=8192, ldv=8192), SHAPE), (dict(t=0), 0), (dict(t=0, k=None, cache=None), 0),
])
@pytest.mark.parametrize("base", [APPEND, READ], ids=["append", "read"])
def test_token_refusals(base, over, status):
    fn = L.library_handle().mixllm_kv8_append if base is APPEND else L.library_handle().mixllm_kv8_read
    assert call(fn, base, **over) == status


@pytest.mark.parametrize("over,status", [
    (dict(t=-1), SHAPE), (dict(b=-1), SHAPE), (dict(hq=0), SHAPE), (dict(hq=33), SHAPE), (dict(hq=4), SHAPE),
    (dict(heads=0), SHAPE), (dict(dim=80), SHAPE), (dict(page=20), SHAPE), (dict(pages=-1), SHAPE), (dict(dtype=2), SHAPE),
    (dict(max_rows=-1), SHAPE), (dict(max_len=-1), SHAPE), (dict(max_len=1 << 30), SHAPE), (dict(window=-1), SHAPE),
    (dict(width=0), SHAPE), (dict(ldt=15), SHAPE), (dict(ldq=4088), SHAPE), (dict(ldq=4100), SHAPE), (dict(ldo=0), SHAPE),
    (dict(q=None), NULL), (dict(cache=None), NULL), (dict(table=None), NULL), (dict(lens=None), NULL), (dict(cu=None), NULL),
    (dict(out=None), NULL), (dict(q=P8), SHAPE), (dict(out=P8), SHAPE), (dict(lse=P2), SHAPE), (dict(ws=P8), SHAPE),
    (dict(nbytes=64 * 8 * BLOCK - 1), SPACE), (dict(b=1 << 20, max_rows=1 << 20), SHAPE),
    (dict(max_len=8192, ws=None), NULL), (dict(max_len=8192, ws_bytes=16), SPACE), (dict(t=1 << 30), SHAPE),
    (dict(window=1 << 30), SHAPE), (dict(b=65536), SHAPE), (dict(max_rows=1 << 28), SHAPE), (dict(b=60000, max_rows=2000), SHAPE),
    (dict(t=0), 0), (dict(b=0), 0), (dict(max_rows=0, q=None), 0),
])
def test_attention_refusals(over, status):
    assert call(L.library_handle().mixllm_kv8_attention, ATT, **over) == status


ROWS = dict(a=P, lda=4096, dtype=0, m=4, k=4096, q=P, ldq=4096, s=P4, stream=None)
GEMM = dict(aq=P, lda=4096, sa=P4, w=P, ldw=4096, sw=P4, m=4, n=100, k=4096, y=P2, ldy=100, dtype=0, stream=None)


@pytest.mark.parametrize("over,status", [
    (dict(m=-1), SHAPE), (dict(m=1 << 22), SHAPE), (dict(k=0), SHAPE), (dict(k=4095), SHAPE), (dict(k=4088), SHAPE),
    (dict(k=131088, lda=1 << 18, ldq=1 << 18), SHAPE), (dict(dtype=2), SHAPE), (dict(lda=4088), SHAPE), (dict(lda=4100), SHAPE),
    (dict(ldq=4080), SHAPE), (dict(ldq=4104), SHAPE), (dict(a=None), NULL), (dict(q=None), NULL), (dict(s=None), NULL),
    (dict(a=P8), SHAPE), (dict(q=P8), SHAPE), (dict(s=P2), SHAPE), (dict(m=0, a=None), 0),
])
def test_quant_rows_refusals(over, status):
    assert call(L.library_handle().mixllm_quant_rows, ROWS, **over) == status


@pytest.mark.parametrize("over,status", [
    (dict(m=-1), SHAPE), (dict(n=0), SHAPE), (dict(n=-5), SHAPE), (dict(k=0), SHAPE), (dict(k=24, lda=32, ldw=32), SHAPE),
    (dict(k=131088, lda=1 << 18, ldw=1 << 18), SHAPE), (dict(dtype=2), SHAPE), (dict(lda=4080), SHAPE), (dict(lda=4104), SHAPE),
    (dict(ldw=4080), SHAPE), (dict(ldw=4104), SHAPE), (dict(ldy=99), SHAPE), (dict(aq=None), NULL), (dict(sa=None), NULL),
    (dict(w=None), NULL), (dict(sw=None), NULL), (dict(y=None), NULL), (dict(aq=P8), SHAPE), (dict(w=P8), SHAPE),
    (dict(sa=P2), SHAPE), (dict(sw=ODD), SHAPE), (dict(y=ODD), SHAPE), (dict(m=1 << 30, n=1 << 10, ldy=1 << 10), SHAPE), (dict(lda=1 << 23), SHAPE), (dict(ldw=1 << 23), SHAPE),
    (dict(m=0, aq=None), 0),
])
def test_gemm_refusals(over, status):
    assert call(L.library_handle().mixllm_gemm_w8a8, GEMM, **over) == status


def test_sizes():
    assert L.mixllm_kv8_page_bytes(16, 8, 128) == 8 * BLOCK
    assert L.mixllm_kv8_page_bytes(64, 1, 64) == 2 * 64 * 64 + 128
    assert L.mixllm_kv8_page_bytes(1024, 3, 256) == 3 * (2 * 1024 * 256 + 512)
    for page in (16, 32, 64, 128, 256, 512, 1024):
        assert L.mixllm_kv8_page_bytes(page, 1, 128) == E.block_bytes(page, 128)
    for bad in ((15, 8, 128), (16, 0, 128), (16, 8, 100), (0, 8, 128)):
        assert L.mixllm_kv8_page_bytes(*bad) == 0
    ws = L.mixllm_kv8_attention_workspace_bytes
    assert ws(1, 1, 32, 8, 128, 1, 77) == 0                 # one workgroup per head does
    assert ws(0, 1, 32, 8, 128, 1, 100000) == 0
    assert ws(1, 1, 32, 7, 128, 1, 100000) == 0             # refused shapes have none
    assert 0 < ws(1, 1, 32, 8, 128, 1, 100000) < 1 << 26
    assert ws(1, 1, 32, 8, 128, 1, 100000, 64) == ws(1, 1, 32, 8, 128, 1, 1000, 64)
    # 70 requests, one of many rows: room for two chunks of each of the others
    assert ws(400, 70, 8, 4, 64, 300, 600) == 70 * 4 * 2 * 32 * (64 + 2) * 4
    assert ws(70 * 300, 70, 8, 4, 64, 300, 600) == ws(400, 70, 8, 4, 64, 300, 600)  # serves calls of fewer rows
    assert ws(400, 60, 8, 4, 64, 300, 600) == 0             # fewer requests stay in the one launch
    with pytest.raises(ValueError):
        L.kv8_cache(4, 20, 8, 128, device="cpu")
    assert L.kv8_cache(3, 16, 2, 64, device="cpu").shape == (3, 2, 2 * 16 * 64 + 128)


def test_places_of_a_run_are_all_different():
    for dim in (64, 128, 256):
        for part in range(2):
            at = {E.code_byte(part, t, ch) for t in range(16) for ch in range(dim)}
            assert at == set(range(16 * dim))


def test_a_scale_that_grows_by_hand():
    """One channel takes 1, then 2: the first token's code 127 becomes 64 (127 / 2 = 63.5, to even)."""
    cache = np.full((1, 1, E.block_bytes(16, 64)), 255, np.uint8)
    x = np.zeros((1, 1, 64), np.float32)
    x[..., 5] = 1.0
    E.kv8_write(cache, [0], x, x, 16)
    (codes, scale), _ = E.run_views(cache, 0, 0, 0, 16, 64)
    assert scale[0] == np.float32(1) / np.float32(127) and codes[E.code_byte(0, 0, 5)] == 255
    E.kv8_write(cache, [1], 2 * x, x, 16)
    assert scale[0] == np.float32(2) / np.float32(127)
    assert codes[E.code_byte(0, 0, 5)] == 128 + 64 and codes[E.code_byte(0, 1, 5)] == 255
    (_, _), (vcodes, vscale) = E.run_views(cache, 0, 0, 0, 16, 64)
    assert vscale[0] == np.float32(1) / np.float32(127) and vcodes[E.code_byte(1, 0, 5)] == vcodes[E.code_byte(1, 1, 5)] == 255
    E.kv8_write(cache, [0], x / 4, x, 16)                    # begun anew: the second token is gone
    assert scale[0] == np.float32(0.25) / np.float32(127) and codes[E.code_byte(0, 1, 5)] == 128


def test_rotation_by_hand():
    x = np.zeros((1, 1, 4))
    x[0, 0] = [1, 2, 3, 4]
    quarter = np.array([np.pi / 2], np.float32)
    y, _ = E.head_norm_rotate(x, [1], quarter)
    assert np.allclose(y, [[[-2, 1, 3, 4]]], atol=1e-7)
    y, _ = E.head_norm_rotate(x, [1], np.array([0, np.pi / 2], np.float32))
    assert np.allclose(y, [[[1, -4, 3, 2]]], atol=1e-6)
    y, _ = E.head_norm_rotate(x, [1], np.array([0, np.pi / 2], np.float32), neighbours=True)
    assert np.allclose(y, [[[1, 2, -4, 3]]], atol=1e-6)
    y, _ = E.head_norm_rotate(x, [3], None, norm=[1, 1, 1, 2], eps=0)
    assert np.allclose(y, x / np.sqrt(7.5) * [1, 1, 1, 2])


def test_rows_and_their_product_by_hand():
    q, s = E.quant_rows([[127, 1.5, -0.5, 0], [0, 0, 0, 0], [-2, 2, 1, 0.5]])
    assert q.tolist() == [[127, 2, 0, 0], [0, 0, 0, 0], [-127, 127, 64, 32]]
    assert s.tolist() == [1.0, 0.0, np.float32(2) / np.float32(127)]
    y = E.gemm_w8a8(q, s, q[:1], np.array([0.5], np.float32))
    assert y[0, 0] == (127 * 127 + 4) * 0.5 and y[1, 0] == 0
