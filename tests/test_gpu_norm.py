"""The fused norms on the GPU against the definition in 64 bits.

Tolerances, counted in fp32 roundings (u = 2^-24) and half steps of the output type:
* a row's mean of squares is a sum of N non-negative terms: each thread adds at most 64 in
  sequence, then 6 steps across lanes and at most 16 waves: relative error <= 90 u; with the
  division, the square root and the reciprocal 1 / rms is within (45 + 4) u, below 64 u;
* h' has the block's term with 1 / rms of x, three products and one fused sum:
  |h' - exact| <= (64 + 5) u size, size the unsigned sum of its terms;
* y = h' w / rms(h'): the error of h' moves an element by itself and through the mean, which
  is at most the row's rms of it: (69 u) (size + |h'| rms(size) / rms(h')) w / rms(h'), plus
  64 u + 3 u of y itself;
* one rounding to the output type: half a step, eps / 2, relative; below the smallest normal
  value half the smallest step.
"""
import numpy as np
import pytest

import oracle as O
from oracle import serving_oracle as S
from tests import gpu_util as U

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
u = 2.0 ** -24


@pytest.fixture(scope="module")
def L():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    from weight_activation_quantized_amd import mixllm
    return mixllm


def half_step(v, dtype):
    f = torch.finfo(dtype)
    return f.eps / 2 * np.abs(v) + float(f.smallest_normal) * f.eps / 2


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def make(m, n, dtype, res, post, gate, seed):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    h = 2 * r(m, n)
    h[:, ::97] *= 15
    d = dict(x=(1.5 * r(m, n)).to(dtype), res=h.to(torch.float32 if res == "fp32" else dtype), pre=(1 + 0.2 * r(n)).to(dtype),
             post=(1 + 0.2 * r(n)).to(dtype) if post else None,
             gate={"none": None, "channel": r(n).to(dtype), "token": r(m, n).to(dtype)}[gate])
    return {k: v if v is None else v.cuda() for k, v in d.items()}


def check(d, h_out, y, alpha, beta, eps):
    h, yy, size = S.residual_norm(*(None if d[k] is None else host(d[k]) for k in ("x", "res", "pre", "post", "gate")),
                                  alpha=alpha, beta=beta, eps=eps)
    if h_out is not None:
        tol = 69 * u * size + (half_step(h, h_out.dtype) if h_out.dtype != torch.float32 else u * np.abs(h))
        err = np.abs(host(h_out) - h)
        assert np.all(err <= tol), (err / tol).max()
    if y is not None:
        rms = np.sqrt((h * h).mean(-1, keepdims=True) + eps)
        w = np.abs(host(d["pre"]))
        moved = 69 * u * (size + np.abs(h) * np.sqrt((size * size).mean(-1, keepdims=True)) / rms) * w / rms
        tol = moved + 67 * u * np.abs(yy)
        tol = tol + half_step(np.abs(yy) + tol, y.dtype)
        err = np.abs(host(y) - yy)
        assert np.all(err <= tol), (err / tol).max()


SIZES = [(1, 1), (1, 64), (3, 65), (2, 512), (5, 513), (4, 2048), (2, 2056), (3, 4096), (1, 5000), (2, 8192), (2, 8200),
         (1, 16384), (1, 16392), (2, 32768), (1, 40000), (1, 65536), (130, 1408)]


@pytest.mark.parametrize("m,n", SIZES)
@pytest.mark.parametrize("dtype,res,post,gate", [
    (torch.float16, "same", True, "channel"), (torch.bfloat16, "fp32", True, "token"),
    (torch.float16, "fp32", False, "none"), (torch.bfloat16, "same", False, "channel")])
def test_sixteen_bit_output(L, m, n, dtype, res, post, gate):
    U.say("norm", m, n, dtype, res, post, gate)
    d = make(m, n, dtype, res, post, gate, m * 1000 + n)
    h_out, y = torch.empty_like(d["res"]), torch.empty_like(d["x"])
    L.mixllm_residual_norm(d["x"], d["res"], d["pre"], h_out, y=y, post_weight=d["post"], gate=d["gate"], alpha=1.25,
                           beta=0.5, eps=1e-5)
    check(d, h_out, y, 1.25, 0.5, 1e-5)


@pytest.mark.parametrize("m,n", [(1, 128), (5, 384), (3, 4096), (65, 1408), (2, 14336), (1, 65536)])
@pytest.mark.parametrize("dtype,res", [(torch.float16, "same"), (torch.bfloat16, "fp32")])
def test_int8_outputs_are_those_of_its_y(L, m, n, dtype, res):
    """Codes, scales, code sums and row operands equal quantizing the 16-bit y, bit for bit."""
    U.say("norm int8", m, n, dtype)
    d = make(m, n, dtype, res, True, "channel", n)
    g = n // 128
    y, h_out = torch.empty_like(d["x"]), torch.empty_like(d["res"])
    aq = torch.empty((m, n), dtype=torch.int8, device="cuda")
    sa = torch.empty((g, m), device="cuda")
    asum = torch.empty((g, m), dtype=torch.int32, device="cuda")
    ro = L.rowop_buffer(m, n)
    kw = dict(post_weight=d["post"], gate=d["gate"], beta=0.3)
    L.mixllm_residual_norm(d["x"], d["res"], d["pre"], h_out, y=y, aq=aq, sa=sa, asum=asum, rowop=ro, **kw)
    check(d, h_out, y, 1.0, 0.3, 1e-5)
    yf = y.float().cpu().numpy()
    gr = yf.reshape(m, g, 128)
    s = (np.abs(gr).max(-1) / np.float32(127)).astype(np.float32)
    q = np.where(s[..., None] > 0, np.clip(np.rint(gr / np.where(s > 0, s, np.float32(1))[..., None]), -127, 127), 0)
    if dtype == torch.float16:
        oq, osa, _ = O.quant_act(yf.astype(np.float16))
        assert np.array_equal(oq.reshape(m, g, 128), q) and np.array_equal(osa, s)
    assert np.array_equal(aq.cpu().numpy().reshape(m, g, 128), q)
    assert np.array_equal(sa.cpu().numpy().T, s)
    qs = q.astype(np.int64).sum(-1).astype(np.int32)
    assert np.array_equal(asum.cpu().numpy().T, qs)
    assert np.array_equal(ro.cpu().numpy().view(np.uint32), U.rowop_records(s.T, qs.T.astype(np.float32) * s.T))
    # without the 16-bit copy, and without the optional outputs: the same codes
    aq2, sa2 = torch.empty_like(aq), torch.empty_like(sa)
    L.mixllm_residual_norm(d["x"], d["res"], d["pre"], aq=aq2, sa=sa2, **kw)
    assert torch.equal(aq, aq2) and torch.equal(sa, sa2)


def test_first_norm_has_no_block_and_zero_rows_stay_zero(L):
    d = make(4, 1024, torch.float16, "same", False, "none", 5)
    d["res"][1] = 0
    y = torch.empty_like(d["res"])
    L.mixllm_residual_norm(None, d["res"], d["pre"], y=y)
    check({**d, "x": None}, None, y, 1.0, 1.0, 1e-5)
    assert not y[1].any()
    L.mixllm_residual_norm(None, d["res"], d["pre"], y=y, eps=0.0)  # 0 / 0 in a row touches no other row
    check({**d, "x": None, "res": d["res"][[0, 2, 3]]}, None, y[[0, 2, 3]], 1.0, 1.0, 0.0)
    # the last residual sum, without a second norm
    h_out = torch.empty_like(d["res"])
    L.mixllm_residual_norm(d["x"], d["res"], None, h_out, alpha=0.5)
    check(d, h_out, None, 0.5, 1.0, 1e-5)


@pytest.mark.parametrize("off", [0, 1])
def test_strided_rows_in_place_and_neighbours_untouched(L, off):
    """Rows inside wider buffers (16-byte aligned, or shifted by one element), the residual
    updated in place: the same results, and nothing else in the buffers changes."""
    m, n, ld = 5, 512, 768
    d = make(m, n, torch.bfloat16, "same", True, "token", 9)
    h_ref, y_ref = torch.empty_like(d["res"]), torch.empty_like(d["x"])
    kw = dict(post_weight=d["post"], beta=0.7)
    L.mixllm_residual_norm(d["x"], d["res"], d["pre"], h_ref, y=y_ref, gate=d["gate"], **kw)
    wide = {k: torch.full((m, ld), 7.0, dtype=torch.bfloat16, device="cuda") for k in ("x", "res", "gate", "y")}
    view = {k: v[:, off:off + n] for k, v in wide.items()}
    for k in ("x", "res", "gate"):
        view[k].copy_(d[k])
    L.mixllm_residual_norm(view["x"], view["res"], d["pre"], view["res"], y=view["y"], gate=view["gate"], **kw)
    check(d, view["res"], view["y"], 1.0, 0.7, 1e-5)
    if off == 0:
        assert torch.equal(view["res"], h_ref) and torch.equal(view["y"], y_ref)
    for v in wide.values():
        assert torch.all(v[:, :off] == 7.0) and torch.all(v[:, off + n:] == 7.0)


def test_binding_refusals(L):
    d = make(4, 256, torch.float16, "same", True, "channel", 1)
    y = torch.empty_like(d["x"])
    ok = dict(y=y, post_weight=d["post"], gate=d["gate"])
    bad = [dict(x=d["x"][:3]), dict(res=d["res"].bfloat16()), dict(y=y.float()), dict(gate=d["gate"][:128]),
           dict(post_weight=d["post"].float()), dict(x=d["x"].t().contiguous().t()), dict(y=y.cpu()),
           dict(res=d["res"][:1].expand(4, 256)), dict(res_out=d["res"].float()),
           dict(aq=torch.empty(4, 256, dtype=torch.int8, device="cuda"))]
    for b in bad:
        args = {**dict(x=d["x"], res=d["res"], pre_weight=d["pre"]), **ok, **b}
        with pytest.raises(ValueError):
            L.mixllm_residual_norm(**args)
    e = torch.empty(0, 256, dtype=torch.float16, device="cuda")
    L.mixllm_residual_norm(e, e, d["pre"], e, y=e)  # no rows: nothing to do
