"""How a decoder layer calls what it is made of, on the GPU: streams, and its attention against
the definition with the operator's own bounds."""
import numpy as np
import pytest

from oracle import serving_oracle as S
from tests import gpu_util as U
from tests import test_gpu_decoder as D
from tests import test_gpu_kv4 as K

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def L():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    from weight_activation_quantized_amd import mixllm
    return mixllm


def inputs(m, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(m, D.HIDDEN, generator=g) * 0.5).half().cuda()


@pytest.mark.parametrize("kind", ["none", "stream", "handle", "default handle"])
def test_positions_are_embedded_on_the_layers_stream(L, kind):
    U.say("layer stream", kind)
    layer, _ = D.make_layer(L, 8, 2, 64, 8)
    req = L.RequestPages(2, 8, D.PAGE, 60, 8)
    bufs = layer.buffers(4, 2, 3, 60)
    h, fresh = inputs(4, 1), K.i32([1, 3])
    stream_h = h.clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    stream, want = {"none": (None, torch.cuda.current_stream()), "stream": (side, side),
                    "handle": (side.cuda_stream, side), "default handle": (0, torch.cuda.default_stream())}[kind]
    seen = []

    def rotate(q, k, pos):
        seen.append(torch.cuda.current_stream().cuda_stream)
        D.rotation(q, k, pos)

    before = torch.cuda.current_stream()
    req.plan(fresh, stream)
    y = layer.forward(None, stream_h, bufs, req, rotate, stream)
    torch.cuda.synchronize()
    assert seen == [want.cuda_stream] and torch.cuda.current_stream() == before
    # the same step on the current stream
    other = L.RequestPages(2, 8, D.PAGE, 60, 8).plan(fresh)
    again = layer.forward(None, h, layer.buffers(4, 2, 3, 60), other, D.rotation)
    assert torch.equal(y, again)


@pytest.mark.parametrize("hq,hkv,dim,window", [(8, 2, 64, 0), (4, 4, 128, 0), (16, 2, 64, 21)])
def test_a_layers_attention_within_the_operators_bounds(L, hq, hkv, dim, window):
    """Prompts and decodes: what reaches the output projection is attention over the codes of the
    keys and values that the projections left."""
    U.say("layer attention", hq, hkv, dim, window)
    layer, _ = D.make_layer(L, hq, hkv, dim, 30, window)
    att, req = layer.attention, L.RequestPages(3, 30, D.PAGE, 100, 60)
    held = [[np.zeros((0, hkv, dim), np.float32)] * 2 for _ in range(3)]
    for n, fresh in enumerate(([40, 1, 18], [1, 2, 0], [1, 1, 30])):
        rows = sum(fresh)
        bufs = layer.buffers(rows, 3, max(fresh), 100)
        req.plan(K.i32(fresh))
        layer.forward(None, inputs(rows, n), bufs, req, D.rotation)
        q, k, v = (t.unflatten(1, (-1, dim)) for t in att.qkv.split(bufs["attention"]["qkv"]["y"]))
        at, kv = 0, []
        for b in range(3):
            parts = []
            for i, new in enumerate((k, v)):
                held[b][i] = np.concatenate([held[b][i], new[at:at + fresh[b]].float().cpu().numpy()])
                c, s, m = S.kv4_quant(held[b][i])
                most = np.repeat(15 * s.astype(np.float64) + np.abs(m.astype(np.float64)), 64, -1)
                parts += [S.kv4_values(c, s, m), most.reshape(held[b][i].shape)]
            kv.append(parts)
            at += fresh[b]
        lens = req.lens.tolist()
        out, lse = torch.empty_like(q), torch.empty((rows, hq), device="cuda")
        L.mixllm_kv4_attention(q, att.cache, req.table, req.lens, req.cu, out, D.PAGE, max(fresh), 100, window=window, lse=lse,
                               workspace=bufs["attention"]["ws"])
        assert torch.equal(out, bufs["attention"]["attn"])
        K.compare(out, lse, q.float().cpu().numpy(), kv, lens, fresh, torch.float16, dim ** -0.5, window)


def test_a_gate_is_per_channel_or_per_token(L):
    """A gate of any other shape is refused, and weights of another number of channels: only the
    first N numbers of them would be read."""
    m, n = 4, 256
    x, one = torch.ones((m, n), dtype=torch.float16, device="cuda"), torch.ones(n, dtype=torch.float16, device="cuda")
    y = torch.empty_like(x)
    L.mixllm_residual_norm(x, x, one, y=y, gate=one, post_weight=one)
    L.mixllm_residual_norm(x, x, one, y=y, gate=x, post_weight=one)
    more = torch.ones(m * n, dtype=torch.float16, device="cuda")
    for bad in (dict(gate=x[None]), dict(gate=more), dict(gate=one[:1]), dict(post_weight=more), dict(post_weight=x),
                dict(pre_weight=more), dict(gate=torch.ones((), dtype=torch.float16, device="cuda"))):
        with pytest.raises(ValueError):
            L.mixllm_residual_norm(**{**dict(x=x, res=x, pre_weight=one, y=y), **bad})


def test_scales_and_sums_without_codes_are_refused(L):
    """They belong to the codes: without them they would be left unwritten."""
    m, n = 4, 256
    x, one = torch.ones((m, n), dtype=torch.float16, device="cuda"), torch.ones(n, dtype=torch.float16, device="cuda")
    y = torch.empty_like(x)
    for bad in (dict(sa=torch.empty((2, m), device="cuda")), dict(asum=torch.empty((2, m), dtype=torch.int32, device="cuda")),
                dict(rowop=L.rowop_buffer(m, n))):
        with pytest.raises(ValueError, match="aq"):
            L.mixllm_residual_norm(x, x, one, y=y, **bad)
