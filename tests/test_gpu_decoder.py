"""The operators between the packed layers as a decoder uses them: steps of prompts and of
single tokens, requests that end and begin, through AttentionBlock and DecoderLayer, eager and
replayed as a HIP graph.

Each operator is compared with the oracle applied to its own input on the GPU (the steps round
in between, so this is how a pipeline's parity is checked), with its own test's tolerance."""
import numpy as np
import pytest

from oracle import serving_oracle as S
from tests import gpu_util as U
from tests import test_gpu_kv4 as K
from tests import test_gpu_norm as N
from weight_activation_quantized_amd import workloads as WL

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

HIDDEN, INTER, PAGE = 512, 384, 16


@pytest.fixture(scope="module")
def L():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    from weight_activation_quantized_amd import mixllm
    return mixllm


def weights(n, k, n8, seed):
    return WL.make_weights(n, k, (seed,)) * np.float16(2), WL.make_idx8(n, n8, (seed,))


def make_layer(L, hq, hkv, dim, pages, window=0, post=False, seed=70):
    g = torch.Generator().manual_seed(seed)
    w = {}
    for i, (name, n, k, n8) in enumerate((("q", hq * dim, HIDDEN, 20), ("k", hkv * dim, HIDDEN, 7), ("v", hkv * dim, HIDDEN, 60),
                                          ("o", HIDDEN, hq * dim, 30), ("gate", INTER, HIDDEN, 5), ("up", INTER, HIDDEN, 40),
                                          ("down", HIDDEN, INTER, 100))):
        w[name] = weights(n, k, n8, seed + i)
    norm = lambda: (1 + 0.2 * torch.randn(HIDDEN, generator=g)).half().cuda()  # noqa: E731
    att = L.AttentionBlock(*(w[x][0] for x in "qkvo"), *(w[x][1] for x in "qkvo"), norm(), hq, hkv, pages, PAGE,
                           post_norm=norm() if post else None, window=window)
    att.cache.fill_(255)
    mlp = L.MLPBlock(*(w[x][0] for x in ("gate", "up", "down")), *(w[x][1] for x in ("gate", "up", "down")))
    return L.DecoderLayer(att, mlp, norm(), norm() if post else None), w


def rotation(q, k, pos):
    """A rotation of channel pairs by the position, in place."""
    d = q.shape[-1]
    a = pos.double()[:, None, None] * 0.7 ** torch.arange(d // 2, device=q.device)
    for t in (q, k):
        x, y = t[..., :d // 2].double(), t[..., d // 2:].double()
        t[..., :d // 2], t[..., d // 2:] = (x * a.cos() - y * a.sin()).half(), (x * a.sin() + y * a.cos()).half()


def state_of(req):
    return {k: getattr(req, k).cpu().numpy().copy() for k in ("table", "pool", "lens", "count")}


@pytest.mark.parametrize("hq,hkv,dim,window,post", [(8, 2, 64, 0, False), (4, 4, 128, 0, True), (16, 2, 64, 21, True)])
def test_steps_of_a_decoder_layer(L, hq, hkv, dim, window, post):
    U.say("decoder layer", hq, hkv, dim, window, post)
    b, pages = 4, 40
    layer, w = make_layer(L, hq, hkv, dim, pages, window, post)
    att = layer.attention
    steps = [[30, 1, 17, 0], [1, 1, 1, 40], [1, -1, 1, 1], [1, 3, 5, 1], [1, 1, 1, 1]]
    tokens = 60
    req = L.RequestPages(b, pages, PAGE, 200, tokens)
    host_cache = att.cache.cpu().numpy().copy()
    rng = np.random.default_rng(3)
    for n, fresh in enumerate(steps):
        m = sum(max(f, 0) for f in fresh) + (3 if n == 3 else 0)   # one step with padding rows
        bufs = layer.buffers(m, b, max(max(fresh), 1), 200)
        x = torch.from_numpy((0.3 * rng.normal(size=(m, HIDDEN))).astype(np.float16)).cuda() if n else None
        h = torch.from_numpy(rng.normal(size=(m, HIDDEN)).astype(np.float16)).cuda()
        h0, before = h.clone(), state_of(req)
        req.plan(K.i32(fresh))
        want = S.kv_plan(fresh, before["lens"], before["table"], before["pool"], before["count"][0], PAGE, pages, tokens)
        got = state_of(req)
        for a, c in (("table", "table"), ("pool", "pool"), ("lens", "lens_out"), ("count", "count_out")):
            assert np.array_equal(got[a], want[c]), (n, a)
        slots = req.slots.cpu().numpy()
        assert np.array_equal(slots, want["slots"]) and np.array_equal(req.cu.cpu().numpy(), want["cu"])

        y = layer.forward(x, h, bufs, req, rotation)
        ba, bm = bufs["attention"], bufs["mlp"]
        # first norm: its codes are those of a 16-bit y from the same call
        h1, y1 = torch.empty_like(h), torch.empty_like(h)
        L.mixllm_residual_norm(x, h0, att.norm, h1 if x is not None else None, y=y1,
                               post_weight=att.post_norm if x is not None else None)
        if x is None:
            h1 = h0
        N.check(dict(x=x, res=h0, pre=att.norm, post=att.post_norm if x is not None else None, gate=None),
                h1 if x is not None else None, y1, 1.0, 1.0, 1e-5)
        y16 = y1.cpu().numpy()
        wq, iq, bounds = L.concat_layers([w[c][0] for c in "qkv"], [w[c][1] for c in "qkv"])
        ref = U.oracle_at(y16, wq, iq)
        assert np.array_equal(ba["qkv"]["aq"].cpu().numpy(), ref["aq"])
        # the GEMM, before the rotation: again on its own, into another output
        again = dict(ba["qkv"], y=torch.empty_like(ba["qkv"]["y"]))
        att.qkv.layer.gemm(again)
        U.assert_y_close(again["y"].cpu().numpy(), ref["y16"], "q/k/v")
        q, k, v = att.qkv.split(again["y"])
        q, k, v = (t.unflatten(1, (-1, dim)) for t in (q, k, v))
        rotation(q, k, req.pos[:m])
        assert torch.equal(again["y"], ba["qkv"]["y"])
        # the cache, byte by byte
        S.kv4_write(host_cache, slots[:m], k.float().cpu().numpy(), v.float().cpu().numpy(), PAGE)
        assert np.array_equal(att.cache.cpu().numpy(), host_cache), n
        # attention over what the cache stands for
        kv, lens = [], got["lens"]
        for i in range(b):
            pos = np.arange(lens[i])
            s = K.i32(got["table"][i][pos // PAGE] * PAGE + pos % PAGE)
            parts = []
            ko = torch.zeros((len(pos), hkv, dim), dtype=torch.float16, device="cuda")
            vo = ko.clone()
            L.mixllm_kv4_read(att.cache, s, ko, vo, PAGE)   # rounded to fp16: half a step of it below
            for t in (ko, vo):
                val = t.cpu().numpy().astype(np.float64)
                parts += [val, np.abs(val) * (1 + 2.0 ** -11) + 15 * 0.5]
            kv.append(parts)
        rows = [max(f, 0) for f in fresh]
        at = 0
        out = ba["attn"].cpu().numpy().astype(np.float64)
        for i in range(b):
            if rows[i]:
                o, _, mass, size = S.attention(q[at:at + rows[i]].cpu().numpy(), kv[i][0], kv[i][2], int(lens[i]), dim ** -0.5,
                                               window)
                # the read's rounding of keys and values (2^-11 each) on top of the kernel's own
                e = (2.0 ** -11 * 2 + 2.0 ** -10) * (1 + size[..., None]) * (mass + np.abs(o) + 1.0)
                err = np.abs(out[at:at + rows[i]] - o)
                assert np.all(err <= e), (n, i, (err / e).max())
            at += rows[i]
        assert not out[at:].any()                                     # padding rows: as they were
        ref = U.oracle_at(ba["attn"].flatten(1).cpu().numpy(), w["o"][0], w["o"][1])
        U.assert_y_close(ba["o"]["y"].cpu().numpy(), ref["y16"], "o")
        # second norm, MLP
        h2, y2 = torch.empty_like(h), torch.empty_like(h)
        L.mixllm_residual_norm(ba["o"]["y"], h1, layer.norm, h2, y=y2, post_weight=layer.post_norm)
        assert torch.equal(h, h2)
        N.check(dict(x=ba["o"]["y"], res=h1, pre=layer.norm, post=layer.post_norm, gate=None), h2, y2, 1.0, 1.0, 1e-5)
        want_y = layer.mlp.forward(y2, layer.mlp.buffers(m))
        assert torch.equal(y, want_y)


def test_decode_steps_replayed_as_a_graph(L):
    """Plan, two layers and the last norm captured once; every replay is the next decode step,
    equal bit for bit to eager steps on a state of its own, with other work between."""
    b, pages = 3, 64
    U.say("decoder graph")
    sides = []
    for _ in range(2):
        layers = [make_layer(L, 8, 2, 64, pages, seed=s)[0] for s in (70, 90)]
        req = L.RequestPages(b, pages, PAGE, 600, 320)
        sides.append((layers, req))
    rng = np.random.default_rng(5)
    prompt = torch.from_numpy(rng.normal(size=(310, HIDDEN)).astype(np.float16)).cuda()
    x = torch.from_numpy(rng.normal(size=(b, HIDDEN)).astype(np.float16)).cuda()
    fresh = K.i32([1] * b)
    last = torch.ones(HIDDEN, dtype=torch.float16, device="cuda")

    def run(layers, req, bufs, h, y, f):
        req.plan(f)
        out = None
        for layer, buf in zip(layers, bufs):
            out = layer.forward(out, h, buf, req)
        L.mixllm_residual_norm(out, h, last, h, y=y)

    state = []
    for layers, req in sides:
        bufs = [l.buffers(310, b, 300, 600) for l in layers]
        run(layers, req, bufs, prompt.clone(), torch.empty_like(prompt), K.i32([300, 2, 8]))
        bufs = [l.buffers(b, b, 1, 600) for l in layers]
        # the two layers run one after the other: one workspace does
        for u in bufs[1:]:
            u["attention"]["ws"] = bufs[0]["attention"]["ws"]
        state.append((bufs, torch.empty_like(x), torch.empty_like(x)))
    assert torch.equal(sides[0][1].lens, sides[1][1].lens)
    (l0, r0), (l1, r1) = sides
    (b0, h0, y0), (b1, h1, y1) = state

    snap = [t.clone() for t in (r1.lens, r1.table, r1.pool, r1.count)] + [l.attention.cache.clone() for l in l1]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        h1.copy_(x)
        run(l1, r1, b1, h1, y1, fresh)            # warm-up outside the capture, then taken back
        for t, o in zip([r1.lens, r1.table, r1.pool, r1.count] + [l.attention.cache for l in l1], snap):
            t.copy_(o)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        run(l1, r1, b1, h1, y1, fresh)
    other = torch.randn(1 << 20, device="cuda")
    for i in range(20):
        for h in (h0, h1):
            h.copy_(x).mul_(1 + 0.01 * i)
        y1.fill_(float("nan"))
        g.replay()
        other.mul_(1.0001).add_(1.0)
        run(l0, r0, b0, h0, y0, fresh)
        torch.cuda.synchronize()
        assert torch.equal(y0, y1) and torch.equal(h0, h1), i
        assert torch.equal(r0.lens, r1.lens) and torch.equal(r0.slots, r1.slots) and torch.equal(r0.count, r1.count), i
        assert torch.equal(l0[1].attention.cache, l1[1].attention.cache), i
    assert r0.lens.tolist() == [320, 22, 28]


def test_request_pages_refuses(L):
    with pytest.raises(ValueError):
        L.RequestPages(2, 0, 16, 100, 10)
    req = L.RequestPages(2, 4, 16, 64, 100)
    req.plan(K.i32([50, 50]))                     # four pages each: the second finds none
    assert req.lens.tolist() == [50, 0] and req.count.tolist() == [0, 1]
    assert req.slots[50:].tolist() == [-1] * 50
    with pytest.raises(L.MixLLMError):
        L.RequestPages(2, 4, 24, 64, 100).plan(K.i32([1, 1]))
    with pytest.raises(ValueError):
        req.plan(torch.tensor([1, 1], device="cuda"))
