"""Calls at the edges of what the 8-bit operators allow."""
import numpy as np
import pytest

from oracle import eight_bit_oracle as E
from tests import test_gpu_gemm8 as G
from tests.test_gpu_kv4 import cuda, rounded

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
