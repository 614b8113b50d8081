"""The layers' own checks, on the host: a call that cannot be right is refused before anything
is launched.  The library's calls are replaced by ones that note their names, so nothing here
needs a GPU."""
import numpy as np
import pytest

from tests import test_serving_host as H
from weight_activation_quantized_amd import workloads as WL

L = pytest.importorskip("weight_activation_quantized_amd.mixllm")
torch = pytest.importorskip("torch")

H_WIDE = dict(ldx=16512, ldr=16512, ldro=16512, ldy=16512)


@pytest.fixture
def calls(monkeypatch):
    """Names and arguments of the device calls made, which do nothing."""
    made = []
    for name in ("mixllm_quant_act", "mixllm_silu_mul_quant", "mixllm_gemm_w4w8a8", "mixllm_residual_norm", "mixllm_kv_plan_fit",
                 "mixllm_kv4_append", "mixllm_kv4_attention"):
        monkeypatch.setattr(L, name, lambda *a, _name=name, **k: made.append((_name, a)))
    return made


def weights(n, k, seed):
    return WL.make_weights(n, k, (seed,)), WL.make_idx8(n, 5, (seed,))


def layers():
    (wq, iq), (wk, ik), (wv, iv) = (weights(n, 256, i) for i, n in enumerate((128, 64, 64)))
    (wg, ig), (wu, iu), (wd, idn) = weights(128, 256, 3), weights(128, 256, 4), weights(256, 128, 5)
    return {"linear": L.PackedLinear(wq, iq, "cpu"), "qkv": L.QKVProjection(wq, wk, wv, iq, ik, iv, "cpu"),
            "mlp": L.MLPBlock(wg, wu, wd, ig, iu, idn, "cpu")}


@pytest.mark.parametrize("name", ["linear", "qkv", "mlp"])
@pytest.mark.parametrize("rows", [3, 8])
def test_buffers_of_another_number_of_rows(calls, name, rows):
    """Quantization packs its scales by the input's rows, the GEMM reads them by the buffers'."""
    layer = layers()[name]
    a = torch.zeros((rows, 256), dtype=torch.float16)
    with pytest.raises(ValueError, match="rows"):
        layer.forward(a, layer.buffers(5))
    assert not calls
    layer.forward(a, layer.buffers(rows))
    assert [a[4] for n, a in calls if n == "mixllm_gemm_w4w8a8"] == [rows] * (2 if name == "mlp" else 1)


@pytest.mark.parametrize("name", ["linear", "qkv", "mlp"])
def test_no_rows_are_no_rows_in_any_buffers(calls, name):
    layer = layers()[name]
    layer.forward(torch.zeros((0, 256), dtype=torch.float16), layer.buffers(5))
    assert {a[4] for n, a in calls if n == "mixllm_gemm_w4w8a8"} == {0}


def test_blocks_buffers_that_do_not_fit_each_other(calls):
    mlp = layers()["mlp"]
    bufs = dict(mlp.buffers(4), h=mlp.down.buffers(6))
    for run in (lambda: mlp.forward(torch.zeros((4, 256), dtype=torch.float16), bufs), lambda: mlp.forward_quantized(bufs)):
        with pytest.raises(ValueError, match="rows"):
            run()
        assert not calls


def test_a_plan_needs_a_count_for_every_request(calls):
    """The row bounds of the requests behind a shorter `fresh` would stay those of the step before,
    and their rows overlap the new ones'."""
    req = L.RequestPages(3, 8, 16, 64, 20, device="cpu")
    for size in (2, 4, 0):
        with pytest.raises(ValueError, match="fresh"):
            req.plan(torch.zeros(size, dtype=torch.int32))
    assert not calls
    req.plan(torch.zeros(3, dtype=torch.int32))
    assert [n for n, _ in calls] == ["mixllm_kv_plan_fit"]


def attention_block(page=16, pages=6, **kw):
    (wq, iq), (wk, ik), (wv, iv), (wo, io) = (weights(n, k, i) for i, (n, k) in enumerate(
        ((256, 256), (128, 256), (128, 256), (256, 256))))
    norm = torch.ones(256, dtype=torch.float16)
    return L.AttentionBlock(wq, wk, wv, wo, iq, ik, iv, io, norm, 4, 2, pages, page, device="cpu", **kw)


@pytest.mark.parametrize("page,pages,fits", [(16, 6, True), (16, 5, True), (32, 3, False), (16, 7, False), (8, 6, False)])
def test_requests_of_other_pages(calls, page, pages, fits):
    """Slots and page numbers mean what they mean only for caches of the same pages; a cache may have
    more of them than the requests use."""
    att = attention_block()
    req = L.RequestPages(2, pages, page, 60, 10, device="cpu")
    h = torch.zeros((3, 256), dtype=torch.float16)
    if fits:
        att.forward(None, h, att.buffers(3, 2, 2, 60), req)
        assert [n for n, _ in calls][2:4] == ["mixllm_kv4_append", "mixllm_kv4_attention"]
    else:
        with pytest.raises(ValueError, match="pages"):
            att.forward(None, h, att.buffers(3, 2, 2, 60), req)
        assert not calls


@pytest.mark.parametrize("value", [2 ** 31, 2 ** 32, 2 ** 32 + 16, -2 ** 31 - 1, -2 ** 32])
def test_numbers_past_32_bits(value):
    """They would reach the library as their low 32 bits: a longest length of 2^32 as 0."""
    z = torch.zeros((1, 4, 128), dtype=torch.float16)
    i = torch.zeros(1, dtype=torch.int32)
    att = dict(q=z, cache=torch.zeros((1, 2, 16 * 144), dtype=torch.uint8), table=i[None], lens=i, cu=i, out=z, page=16,
               max_rows=1, max_len=16, window=0)
    for name in ("max_rows", "max_len", "window"):
        with pytest.raises(ValueError, match="32 bits"):
            L.mixllm_kv4_attention(**{**att, name: value})
    sizes = dict(t=1, b=1, q_heads=4, kv_heads=2, dim=128, max_rows=1, max_len=9000, window=0)
    assert L.mixllm_kv4_attention_workspace_bytes(**sizes) > 0
    for name in sizes:
        with pytest.raises(ValueError, match="32 bits"):
            L.mixllm_kv4_attention_workspace_bytes(**{**sizes, name: value})
    for fn in (L.mixllm_kv_plan, L.mixllm_kv_plan_fit):
        for page, pages in ((value, 4), (16, value)):
            with pytest.raises(ValueError, match="32 bits"):
                fn(i, i, i[None], i, i, page, pages, i, i, i, i, i)
    for args in ((value, 8, 128), (16, value, 128), (16, 8, value)):
        with pytest.raises(ValueError, match="32 bits"):
            L.mixllm_kv4_page_bytes(*args)


def test_device_calls_run_on_their_tensors_device(monkeypatch):
    """On the stream of the device that holds the tensors, not of the current one."""
    made = []
    monkeypatch.setattr(L, "_on", lambda dev, stream, fn, *args: made.append((dev, stream, fn.__name__)))
    monkeypatch.setattr(L, "_gpu", lambda t, name: 1)
    monkeypatch.setattr(L, "_need", lambda *a, **k: None)
    monkeypatch.setattr(L, "_gemm_inputs", lambda *a: None)
    a, y = torch.zeros((3, 256), dtype=torch.float16), torch.zeros((3, 64), dtype=torch.float16)
    w, idx = weights(64, 256, 1)
    blob = L.DeviceBlob(L.mixllm_pack_weights(w, idx), "cpu")
    for stream in (None, 5):
        del made[:]
        L.mixllm_quant_act(a, a, a, stream=stream)
        L.mixllm_silu_mul_quant(a, a, a, a, stream=stream)
        L.mixllm_gemm_w4w8a8(a, a, a, a, 3, 64, 256, 5, blob, y, stream=stream)
        L.mixllm_gemm_w4w8a8_partials(a, a, a, a, 3, 64, 256, 5, blob, 0, 64, y, stream=stream)
        assert [m[:2] for m in made] == [(1, stream)] * 4
        assert [m[2] for m in made] == ["mixllm_quant_act", "mixllm_silu_mul_quant", "mixllm_gemm_w4w8a8",
                                        "mixllm_gemm_w4w8a8_partials"]


def test_tensors_on_the_host_are_refused(monkeypatch):
    """Every call on a device pointer names a tensor that has none."""
    made = []
    monkeypatch.setattr(L, "_on", lambda *a: made.append(a))
    a = torch.zeros((3, 256), dtype=torch.float16)
    w, idx = weights(64, 256, 1)
    blob = L.DeviceBlob(L.mixllm_pack_weights(w, idx), "cpu")
    monkeypatch.setattr(L, "_need", lambda *a, **k: None)
    monkeypatch.setattr(L, "_gemm_inputs", lambda *a: None)
    for run in (lambda: L.mixllm_quant_act(a, a, a), lambda: L.mixllm_silu_mul_quant(a, a, a, a),
                lambda: L.mixllm_gemm_w4w8a8(a, a, a, a, 3, 64, 256, 5, blob, a),
                lambda: L.mixllm_gemm_w4w8a8_partials(a, a, a, a, 3, 64, 256, 5, blob, 0, 64, a)):
        with pytest.raises(ValueError, match="CUDA"):
            run()
    assert not made


@pytest.mark.parametrize("name,over", [
    ("mixllm_residual_norm", dict(m=1 << 26)), ("mixllm_residual_norm", dict(m=1 << 24, n=640, **H_WIDE)), ("mixllm_residual_norm", dict(m=1 << 23, n=4224, **H_WIDE)),
    ("mixllm_residual_norm", dict(m=1 << 22, n=16512, **H_WIDE)), ("mixllm_kv4_append", dict(t=(1 << 25) - 15)),
    ("mixllm_kv4_read", dict(t=1 << 30)), ("mixllm_kv4_append", dict(t=2 ** 31 - 1))])
def test_more_rows_than_a_launch_has_threads(name, over):
    """Refused on the host, before any launch."""
    base = {"mixllm_residual_norm": H.NORM, "mixllm_kv4_append": H.APPEND, "mixllm_kv4_read": H.READ}[name]
    assert H.call(getattr(L.library_handle(), name), base, **over) == H.SHAPE
