"""The 8-bit operators as a decoder uses them together: AttentionBlock with norms of its heads, the
rotation, the cache in 8 bits and an output projection in 8 bits, over steps of prompts and single
tokens, eager and replayed as a HIP graph.

As for the 4-bit layer (`test_gpu_decoder`) each operator is compared with the oracle applied to
its own input on the GPU, with its own test's tolerance."""
import numpy as np
import pytest

from oracle import eight_bit_oracle as E
from oracle import serving_oracle as S
from tests import gpu_util as U
from tests import test_gpu_decoder as T
from tests import test_gpu_gemm8 as G
from tests import test_gpu_kv4 as K
from tests import test_gpu_kv8 as V
from tests import test_gpu_rotate as O

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

HIDDEN, PAGE = T.HIDDEN, T.PAGE


@pytest.fixture(scope="module")
def L():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    from weight_activation_quantized_amd import mixllm
    return mixllm


def make(L, hq, hkv, dim, pages, norms=True, rot=None, neighbours=False, packed_o=False, window=0, seed=70):
    g = torch.Generator().manual_seed(seed)
    w = {}
    for i, (name, n, k, n8) in enumerate((("q", hq * dim, HIDDEN, 20), ("k", hkv * dim, HIDDEN, 7), ("v", hkv * dim, HIDDEN, 60),
                                          ("o", HIDDEN, hq * dim, 30))):
        w[name] = T.weights(n, k, n8, seed + i)
    norm = lambda n: (1 + 0.2 * torch.randn(n, generator=g)).half().cuda()  # noqa: E731
    rot = dim if rot is None else rot
    att = L.AttentionBlock(*(w[x][0] for x in "qkvo"), *(w[x][1] for x in "qkv"), w["o"][1] if packed_o else None, norm(HIDDEN),
                           hq, hkv, pages, PAGE, window=window, cache_bits=8, q_norm=norm(dim) if norms else None,
                           k_norm=norm(dim) if norms else None,
                           inv_freq=K.cuda(O.frequencies(rot)) if rot else None, neighbours=neighbours)
    att.cache.fill_(255)
    return att, w


@pytest.mark.parametrize("hq,hkv,dim,norms,rot,neighbours,packed_o,window", [
    (8, 2, 64, True, 64, False, False, 0), (4, 4, 128, True, 64, True, False, 21), (16, 2, 64, False, 64, False, True, 0),
    (6, 1, 128, True, 0, False, False, 0)])
def test_steps_of_an_attention_block(L, hq, hkv, dim, norms, rot, neighbours, packed_o, window):
    U.say("attention block 8", hq, hkv, dim, norms, rot, neighbours, packed_o, window)
    b, pages, tokens = 4, 40, 60
    att, w = make(L, hq, hkv, dim, pages, norms, rot, neighbours, packed_o, window)
    req = L.RequestPages(b, pages, PAGE, 200, tokens)
    host = att.cache.cpu().numpy().copy()
    rng = np.random.default_rng(3)
    for n, fresh in enumerate([[30, 1, 17, 0], [1, 1, 1, 40], [1, -1, 1, 1], [1, 3, 5, 1], [1, 1, 1, 1]]):
        m = sum(max(f, 0) for f in fresh) + (3 if n == 3 else 0)   # one step with padding rows
        bufs = att.buffers(m, b, max(max(fresh), 1), 200)
        h = torch.from_numpy(rng.normal(size=(m, HIDDEN)).astype(np.float16)).cuda()
        req.plan(K.i32(fresh))
        y = att.forward(None, h, bufs, req)
        slots, pos = req.slots.cpu().numpy()[:m], req.pos.cpu().numpy()[:m]
        # the product before the rotation, again into another output
        again = dict(bufs["qkv"], y=torch.empty_like(bufs["qkv"]["y"]))
        att.qkv.layer.gemm(again)
        before = [t.unflatten(1, (-1, dim)) for t in att.qkv.split(again["y"])]
        after = [t.unflatten(1, (-1, dim)) for t in att.qkv.split(bufs["qkv"]["y"])]
        for x, z, wt in zip(before[:2], after[:2], (att.q_norm, att.k_norm)):
            O.check(z, x.float().cpu().numpy(), pos, O.frequencies(rot) if rot else None,
                    None if wt is None else wt.float().cpu().numpy(), att.eps, neighbours, torch.float16)
        assert torch.equal(before[2], after[2])
        # the cache, byte by byte
        E.kv8_write(host, slots, after[1].float().cpu().numpy(), after[2].float().cpu().numpy(), PAGE)
        assert np.array_equal(att.cache.cpu().numpy(), host), n
        # attention over what the cache stands for
        lens, table = req.lens.cpu().numpy(), req.table.cpu().numpy()
        kv = [V.values_of(host, table[i], int(lens[i]), PAGE, dim) for i in range(b)]
        rows = [max(f, 0) for f in fresh]
        total = sum(rows)
        qs = after[0][:total].float().cpu().numpy()
        lse = torch.empty((m, hq), device="cuda")
        ws = bufs["ws"]
        out = torch.full_like(bufs["attn"], 5.0)
        L.mixllm_kv8_attention(after[0], att.cache, req.table, req.lens, req.cu, out, PAGE, bufs["max_rows"], 200, window=window,
                               lse=lse, workspace=ws)
        assert torch.equal(out[:total], bufs["attn"][:total])
        K.compare(out[:total], lse[:total], qs, kv, [int(x) for x in lens], rows, torch.float16, dim ** -0.5, window)
        assert not bufs["attn"][total:].any()                             # padding rows: as they were
        # the output projection
        flat = bufs["attn"].flatten(1).float().cpu().numpy()
        if packed_o:
            U.assert_y_close(y.cpu().numpy(), U.oracle_at(flat.astype(np.float16), w["o"][0], w["o"][1])["y16"], "o")
        else:
            aq, sa = E.quant_rows(flat)
            wq, sw = E.quant_rows(w["o"][0].astype(np.float32))
            assert np.array_equal(att.o.w.cpu().numpy(), wq) and np.array_equal(bufs["o"]["aq"].cpu().numpy(), aq)
            G.check(y, aq, sa, wq, sw, torch.float16)


def test_decode_steps_replayed_as_a_graph(L):
    """Plan and block captured once; every replay is the next decode step, equal bit for bit to eager
    steps on a state of its own, with other work between.  The runs' scales grow on the way."""
    b, pages = 3, 64
    U.say("attention block 8 graph")
    sides = [(make(L, 8, 2, 64, pages)[0], L.RequestPages(b, pages, PAGE, 600, 320)) for _ in range(2)]
    rng = np.random.default_rng(5)
    prompt = torch.from_numpy(rng.normal(size=(310, HIDDEN)).astype(np.float16)).cuda()
    x = torch.from_numpy(rng.normal(size=(b, HIDDEN)).astype(np.float16)).cuda()
    fresh, state = K.i32([1] * b), []

    def run(att, req, bufs, h, f):
        req.plan(f)
        return att.forward(None, h, bufs, req)

    for att, req in sides:
        run(att, req, att.buffers(310, b, 300, 600), prompt, K.i32([300, 2, 8]))
        state.append((att.buffers(b, b, 1, 600), torch.empty_like(x)))
    (a0, r0), (a1, r1) = sides
    (b0, h0), (b1, h1) = state
    assert torch.equal(a0.cache, a1.cache)
    kept = (r1.lens, r1.table, r1.pool, r1.count, a1.cache)
    snap = [t.clone() for t in kept]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        h1.copy_(x)
        run(a1, r1, b1, h1, fresh)            # warm-up outside the capture, then taken back
        for t, o in zip(kept, snap):
            t.copy_(o)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        run(a1, r1, b1, h1, fresh)
    other = torch.randn(1 << 20, device="cuda")
    for i in range(20):
        for h in (h0, h1):
            h.copy_(x).mul_(1 + 0.1 * i)
        b1["o"]["y"].fill_(float("nan"))
        g.replay()
        other.mul_(1.0001).add_(1.0)
        y = run(a0, r0, b0, h0, fresh)
        torch.cuda.synchronize()
        assert torch.equal(y, b1["o"]["y"]) and torch.equal(a0.cache, a1.cache), i
        assert torch.equal(r0.lens, r1.lens) and torch.equal(r0.slots, r1.slots), i
    assert r0.lens.tolist() == [320, 22, 28]


def test_on_another_stream(L):
    """The whole block on a stream given by the caller."""
    att, _ = make(L, 8, 2, 64, 20)
    req = L.RequestPages(2, 20, PAGE, 100, 30)
    h = torch.randn((30, HIDDEN), device="cuda").half()
    bufs = att.buffers(30, 2, 20, 100)
    req.plan(K.i32([20, 10]))
    want = att.forward(None, h.clone(), bufs, req).clone()
    cache = att.cache.clone()
    att.cache.fill_(255)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = att.forward(None, h.clone(), bufs, req, stream=s)
    s.synchronize()
    assert torch.equal(got, want) and torch.equal(att.cache, cache)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_row_linear(L, dtype):
    rng = np.random.default_rng(2)
    w = torch.from_numpy(rng.normal(size=(300, 256)).astype(np.float32)).to(dtype)
    layer = L.RowLinear(w, dtype=dtype)
    a = K.cuda(rng.normal(size=(37, 256)).astype(np.float32), dtype)
    y = layer.forward(a)
    aq, sa = E.quant_rows(a.float().cpu().numpy())
    wq, sw = E.quant_rows(w.float().numpy())
    G.check(y, aq, sa, wq, sw, dtype)
    bufs = layer.buffers(37)
    assert torch.equal(layer.forward(a, bufs), y) and torch.equal(layer.gemm(bufs), y)
    with pytest.raises(ValueError, match="rows"):
        layer.forward(a[:5], bufs)
    assert layer.forward(a[:0], bufs) is bufs["y"]


def test_refuses(L):
    for kw in (dict(cache_bits=5), dict(q_norm=torch.ones(7, device="cuda")), dict(inv_freq=torch.ones(65, device="cuda"))):
        with pytest.raises(ValueError):
            ws = [T.weights(n, k, 5, 1) for n, k in ((256, 256), (128, 256), (128, 256), (256, 256))]
            L.AttentionBlock(*(x[0] for x in ws), *(x[1] for x in ws), torch.ones(256, device="cuda").half(), 2, 1, 4, 16, **kw)
