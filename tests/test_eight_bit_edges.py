"""Calls at the edges of what the 8-bit operators allow: streams, rows that hold no number, values whose
scales are far apart, sizes past a launch."""
import contextlib

import numpy as np
import pytest

from oracle import eight_bit_oracle as E
from tests import gpu_util as U
from tests import test_gpu_gemm8 as G
from tests import test_gpu_kv4 as K
from tests import test_gpu_kv8 as V
from tests.test_eight_bit_host import ROTATE
from tests.test_gpu_kv4 import cuda, rounded
from tests.test_serving_host import SHAPE, call

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def L():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    from weight_activation_quantized_amd import mixllm
    return mixllm


@pytest.mark.gpu
@pytest.mark.parametrize("times", [1, 2, 3])
def test_a_layer_used_on_another_stream_at_once(L, times):
    """The constructor's stream is busy when a layer is made; its weights are there for any stream
    afterwards, without a wait of the caller's."""
    rng = np.random.default_rng(times)
    w = rounded(rng.normal(size=(512, 1024)).astype(np.float32), torch.float16)
    dev = cuda(w, torch.float16)                  # on the GPU already: nothing else makes the constructor wait
    a = cuda(rng.normal(size=(8, 1024)).astype(np.float32), torch.float16)
    wq, sw = E.quant_rows(w)
    aq, sa = E.quant_rows(a.float().cpu().numpy())
    busy, s = torch.ones((4096, 4096), device="cuda"), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        busy = (busy @ busy).clamp_(max=1.0)
    layer = L.RowLinear(dev)
    with torch.cuda.stream(s):
        y = layer.forward(a, stream=s)
    s.synchronize()
    assert np.array_equal(layer.w.cpu().numpy(), wq) and np.array_equal(layer.sw.cpu().numpy(), sw)
    G.check(y, aq, sa, wq, sw, torch.float16)


def test_rows_without_numbers_by_hand():
    q, s = E.quant_rows([[1, np.nan, -2], [np.inf, 0, 1], [1, -np.inf, np.nan], [-2, 1, 0]])
    assert np.isnan(s[:3]).all() and not q[:3].any()
    assert s[3] == np.float32(2) / np.float32(127) and q[3].tolist() == [-127, 64, 0]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("m,k", [(9, 16), (9, 1040), (9, 4096), (9, 8208), (9, 16400), (9, 40000), (1030, 2032), (1030, 4096)])
def test_a_row_that_holds_no_number(L, m, k, dtype):
    """NaN or an infinity anywhere in a row: its scale is NaN and its codes are 0, so its outputs are
    NaN, and no other row's."""
    U.say("quant rows, none", m, k, dtype)
    rng = np.random.default_rng(k)
    a = rounded(rng.normal(size=(m, k)).astype(np.float32), dtype)
    a[1, 0], a[2, k - 1], a[3, k // 2], a[m - 1, 15] = np.nan, np.inf, -np.inf, np.nan
    a[5], a[6, ::3], a[7] = np.nan, -np.inf, 0.0
    largest = float(torch.finfo(dtype).max)
    a[0, 3] = largest                                          # a number, if the largest
    q = torch.full((m, k), 77, dtype=torch.int8, device="cuda")
    s = torch.full((m,), 9.0, device="cuda")
    L.mixllm_quant_rows(cuda(a, dtype), q, s)
    want_q, want_s = E.quant_rows(a)
    bad = [1, 2, 3, 5, 6, m - 1]
    assert np.isnan(want_s[bad]).all() and np.isfinite(np.delete(want_s, bad)).all()
    assert np.array_equal(s.cpu().numpy(), want_s, equal_nan=True)
    assert np.array_equal(q.cpu().numpy(), want_q)
    w, sw = cuda(rng.integers(-127, 128, (33, k)).astype(np.int8)), torch.full((33,), 1e-6, device="cuda")
    sw[4] = 0.0
    y = torch.empty((m, 33), dtype=torch.bfloat16, device="cuda")
    L.mixllm_gemm_w8a8(q, s, w, sw, y)
    ok = torch.ones(m, dtype=torch.bool)
    ok[bad] = False
    assert y[~ok.cuda()].isnan().all() and y[ok.cuda()].isfinite().all()


@pytest.mark.gpu
@pytest.mark.parametrize("apart", [-40, -75, -110, -125, -133])
@pytest.mark.parametrize("rows", [1, 9, 40])
def test_values_whose_scales_are_far_apart(L, apart, rows):
    """Every second run's values are 2^apart of the others': they count as next to nothing in the
    outputs, and in full in what the outputs are divided by."""
    dim, page, dtype, lens = 128, 16, torch.bfloat16, [300, 200]
    U.say("attention8 scales apart", apart, rows)

    def kv(t, heads, d, dt, seed):
        k, v = K.key_values(t, heads, d, dt, seed)
        v = np.where(np.arange(t)[:, None, None] // 16 % 2, v.astype(np.float64) * 2.0 ** apart, v)
        return k, rounded(v.astype(np.float32), dt)

    dev, table, vals = V.build(lens, 2, dim, page, dtype, 71, kv=kv)
    q = V.queries(2 * rows, 8, dim, dtype, 17)
    out, lse = V.attend(L, q, dev, table, lens, [rows] * 2, page, dtype, 0.09)
    K.compare(out, lse, q, vals, lens, [rows] * 2, dtype, 0.09)


@pytest.mark.parametrize("t,heads", [(24573, 2731), (1082401, 62), (1 << 20, 64), (671089, 100)])
def test_more_heads_of_tokens_than_one_launch_has_threads(t, heads):
    """From 2^26 - 3 on the last workgroup would be the launch's 2^32nd thread."""
    assert t * heads > (1 << 26) - 4
    lib = pytest.importorskip("weight_activation_quantized_amd.mixllm").library_handle()
    wide = heads * 50
    assert call(lib.mixllm_head_norm_rotate, ROTATE, t=t, hq=heads - 1, hkv=1, dim=50, rot=50, ldq=wide, ldqo=wide) == SHAPE


@pytest.mark.parametrize("kind", ["packed", "rows"])
def test_buffers_of_a_call_are_the_streams(monkeypatch, kind):
    """A call without buffers makes them while its stream is the current one, so that what it frees on
    return is reused behind its work only."""
    lib = pytest.importorskip("weight_activation_quantized_amd.mixllm")
    for name in ("mixllm_quant_act", "mixllm_gemm_w4w8a8", "mixllm_quant_rows", "mixllm_gemm_w8a8"):
        monkeypatch.setattr(lib, name, lambda *a, **k: None)
    now, made = [None], []

    @contextlib.contextmanager
    def current(stream, dev):
        now[0] = stream
        yield
        now[0] = None

    monkeypatch.setattr(lib, "_current", current)
    w = np.zeros((64, 256), np.float16)
    layer = lib.RowLinear(w, "cpu") if kind == "rows" else lib.PackedLinear(w, [3], "cpu")
    own = layer.buffers
    monkeypatch.setattr(layer, "buffers", lambda m: made.append(now[0]) or own(m))
    a = torch.zeros((5, 256), dtype=torch.float16)
    layer.forward(a, stream="a stream")
    layer.forward(a)
    layer.forward(a, own(5), "another")
    assert made == ["a stream", None]


@pytest.mark.gpu
def test_memory_of_a_call_is_not_given_away_before_it_ran(L):
    """Work that the current stream does while a layer waits on its own stream leaves the layer's codes alone."""
    rng = np.random.default_rng(5)
    w = rounded(rng.normal(size=(512, 2048)).astype(np.float32), torch.float16)
    layer, a = L.RowLinear(torch.from_numpy(w).half()), cuda(rng.normal(size=(64, 2048)).astype(np.float32), torch.float16)
    aq, sa = E.quant_rows(a.float().cpu().numpy())
    wq, sw = E.quant_rows(w)
    s, busy = torch.cuda.Stream(), torch.ones((4096, 4096), device="cuda")
    for _ in range(3):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            work = busy
            for _ in range(10):
                work = (work @ busy).clamp_(max=1.0)
        y = layer.forward(a, stream=s)
        others = [torch.full((64, 2048), 77, dtype=torch.int8, device="cuda") for _ in range(8)]
        others += [torch.full((64,), 1e9, device="cuda") for _ in range(8)]
        torch.cuda.synchronize()
        G.check(y, aq, sa, wq, sw, torch.float16)
        assert all(bool((x == (77 if x.dtype == torch.int8 else 1e9)).all()) for x in others)
