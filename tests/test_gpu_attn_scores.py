"""GPU tests of paged attention whose scores are infinite or NaN: a row whose every score is -infinity is 0, as
one that sees no token; among other scores -infinity weighs nothing; +infinity and NaN reach the row, and no
other row."""

import numpy as np
import pytest

from tests import attn_util as au
from tests.gpu_util import mol_lib, torch_cuda
from tests.test_gpu_attn import attend

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def env():
    return torch_cuda(), mol_lib()


def problem(torch, lens, D, page, score_of):
    """Keys whose first value is score_of(sequence, position) and the rest finite, queries whose first value
    is positive and whose others are finite: products of the first values decide."""
    p = au.problem(torch, D, lens, 8, 2, D, page)
    k, _ = au.caches(p, "cpu")
    p["q"][..., 0] = 2.0
    for b, (_, kv) in enumerate(lens):
        for j in range(kv):
            k[int(p["table"][b, j // page]), j % page, :, 0] = score_of(b, j)
    return p


# few rows (16 and 32 a block), many (tensor copies, gathered tokens), 256 values a head; undivided and in parts
FORMS = [(1, 64, 16), (1, 128, 16), (1, 256, 16), (6, 64, 16), (60, 64, 16), (60, 64, 5), (60, 128, 16), (90, 256, 16)]


@pytest.mark.parametrize("n,D,page", FORMS)
@pytest.mark.parametrize("kv", [90, 2100])
def test_scores_of_minus_infinity(env, n, D, page, kv):
    torch, _ = env
    lens = [(n, kv)] * 4
    # sequence 0: all; 1: all but the first token; 2: all but the last; 3: none
    p = problem(torch, lens, D, page, lambda b, j: -INF if b == 0 or (b == 1 and j > 0) or (b == 2 and j < kv - 1) else 1.0)
    got = attend(env, p)
    want, spread, reach = (np.array(x) for x in au.oracle(dict(p, k=torch.nan_to_num(p["k"], neginf=0.0)), D ** -0.5))
    _, v = au.caches(p, "cpu")

    def value(b, j):  # of every head's key head
        return v[int(p["table"][b, j // page]), j % page].double().numpy().repeat(4, 0)

    want[:n], spread[:n] = 0.0, 0.0
    want[n:2 * n], spread[n:2 * n] = value(1, 0), np.abs(value(1, 0))
    want[2 * n:3 * n], spread[2 * n:3 * n] = 0.0, 0.0  # (the last token is the last row's alone)
    want[3 * n - 1], spread[3 * n - 1] = value(2, kv - 1), np.abs(value(2, kv - 1))
    au.check(got, want, spread, reach)
    assert bool((got[:n] == 0).all()) and bool((got[2 * n:3 * n - 1] == 0).all())


@pytest.mark.parametrize("n,D,page", FORMS)
@pytest.mark.parametrize("bad", [INF, NAN])
@pytest.mark.parametrize("kv", [90, 2100])
def test_scores_of_infinity_and_nan(env, n, D, page, kv, bad):
    torch, _ = env
    lens = [(n, kv)] * 3
    # sequence 0: the first token; 1: a token that the rows from the middle on see; 2: none
    at = kv - 1 - (n - 1) // 2
    clean = problem(torch, lens, D, page, lambda b, j: 1.0)
    hurt = problem(torch, lens, D, page, lambda b, j: bad if (b, j) in ((0, 0), (1, at)) else 1.0)
    got = attend(env, hurt)
    want, spread, reach = au.oracle(clean, D ** -0.5)
    sees = np.concatenate([np.full(n, True), np.arange(kv - n, kv) >= at, np.full(n, False)])
    assert bool(torch.isnan(got[torch.from_numpy(sees)]).all())
    au.check(got, np.where(sees[:, None, None], np.nan, want), spread, reach)
