"""The plan that refuses what has no rows: its refusals on the host, its oracle by hand, and the
kernel against the oracle."""
import numpy as np
import pytest

from oracle import serving_oracle as S
from tests import gpu_util as U
from tests import test_gpu_kv4 as K
from tests import test_serving_host as H

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def L():
    from weight_activation_quantized_amd import mixllm
    return mixllm


@pytest.mark.parametrize("over,status", [
    (dict(b=-1), H.SHAPE), (dict(tokens=-1), H.SHAPE), (dict(ldt=7), H.SHAPE), (dict(page=48), H.SHAPE),
    (dict(fresh=None), H.NULL), (dict(slots=None), H.NULL), (dict(cu=None), H.NULL), (dict(pos=H.P2), H.SHAPE)])
def test_refusals(L, over, status):
    assert H.call(L.library_handle().mixllm_kv_plan_fit, H.PLAN, **over) == status


def test_oracle_by_hand():
    table, pool = np.full((5, 2), -1, np.int32), np.array([4, 5, 6], np.int32)
    r = S.kv_plan([3, 6, 0, 1, -1], [0, 0, 7, 0, 0], table, pool, 3, 16, 10, 8, fit=True)
    # 3 rows fit, 6 more end behind 8; one that adds nothing is none the worse, the next comes behind them
    assert list(r["lens_out"]) == [3, 0, 7, 0, 0] and list(r["count_out"]) == [2, 2]
    assert list(r["cu"]) == [0, 3, 9, 9, 10, 10]
    assert list(r["slots"]) == [96, 97, 98] + [-1] * 5 and list(r["pos"]) == [0, 1, 2, 0, 1, 2, 3, 4]
    exact = S.kv_plan([3, 5, 0, 0, 0], [0, 0, 7, 0, 0], table, pool, 3, 16, 10, 8, fit=True)
    assert list(exact["lens_out"]) == [3, 5, 7, 0, 0] and list(exact["count_out"]) == [1, 0]


def run(L, fresh, lens, table, pool, count, page, pages, tokens):
    b = len(fresh)
    out = dict(table=K.cuda(table), pool=K.cuda(pool), lens_out=K.i32([-9] * b), count_out=K.i32([-9, -9]),
               cu=K.i32([-9] * (b + 1)), slots=K.i32([-9] * tokens), pos=K.i32([-9] * tokens))
    L.mixllm_kv_plan_fit(K.i32(fresh), K.i32(lens), out["table"], out["pool"], K.i32([count, 99]), page, pages,
                         out["lens_out"], out["count_out"], out["cu"], out["slots"], out["pos"])
    return out


def check(L, case, seed):
    fresh, lens, width, page, pages, size, free, tokens = case
    table, pool, count = K.plan_case(fresh, lens, width, page, pages, size, free, tokens, seed)
    want = S.kv_plan(fresh, lens, table, pool, count, page, pages, tokens, fit=True)
    got = run(L, fresh, lens, table, pool, count, page, pages, tokens)
    for k, v in want.items():
        assert np.array_equal(got[k].cpu().numpy(), v), k


@pytest.mark.gpu
@pytest.mark.parametrize("name", K.PLANS)
def test_plan(L, name):
    U.say("plan fit", name)
    check(L, K.PLANS[name], 3)


@pytest.mark.gpu
@pytest.mark.parametrize("tokens", [0, 1, 29, 30, 37, 59, 60, 4095, 5000])
def test_rows_that_do_not_fit(L, tokens):
    U.say("plan fit rows", tokens)
    check(L, ([30, 0, 30, -1, 5000, 1], [0, 9, 4, 33, 2, 70], 400, 16, 700, 700, 600, tokens), 5)


@pytest.mark.gpu
@pytest.mark.parametrize("b,prompt,tokens", [(1024, 3, 700), (1025, 40, 1024), (2500, 7, 1500), (2100, 200, 9000)])
def test_many_requests(L, b, prompt, tokens):
    U.say("plan fit many", b, prompt, tokens)
    rng = np.random.default_rng(b)
    fresh, lens = rng.choice([-1, 0, 1, 1, prompt], b), rng.integers(0, 130, b)
    assert np.maximum(fresh, 0).sum() > tokens
    check(L, (fresh, lens, 24, 16, 16000, 16000, 5000, tokens), b)


@pytest.mark.gpu
def test_request_pages_has_a_row_for_every_token(L):
    """A step of more tokens than rows: the requests that have no room stay as they were and can be
    asked for again."""
    U.say("request pages rows")
    req = L.RequestPages(3, 40, 16, 200, 50)
    req.plan(K.i32([20, 31, 1]))                       # 20 fit; 51 do not, nor what comes behind them
    assert req.lens.tolist() == [20, 0, 0] and req.count.tolist() == [38, 2]
    assert (req.slots[:20] >= 0).all() and (req.slots[20:] == -1).all()
    req.plan(K.i32([1, 31, 18]))
    assert req.lens.tolist() == [21, 31, 18] and req.count[1].item() == 0 and (req.slots >= 0).all()
