"""Attention under score rules and over a shared prefix where lengths, positions and schedules go to their ends, on the
GPU against 64-bit references; tolerances as in test_attn_rules."""
import numpy as np
import pytest

from tests.test_attn_rules import ALIBI, Tables, check_shared, shared, with_prefix
from tests.test_layer_ops import BF16, DT, F16, F32, L, dev  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(params=[False, True], ids=["held", "room"])
def room(request):
    Tables.room = request.param
    yield request.param
    Tables.room = False


@pytest.mark.usefixtures("room")
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("window", [0, 20, 2000])
@pytest.mark.parametrize("biased", [False, True])
def test_prefix_lengths_that_cannot_be(L, dtype, window, biased):  # noqa: F811
    """Nobody sees such a prefix, and positions are not counted from it, under windows and biases too.  Rows before the
    first sequence's, between sequences (one has more queries than max_q) and behind the last are left."""
    rng = np.random.default_rng(window)
    B, Hq, D, P = 60, 4, 64, 100
    new = np.full(B, 2)
    new[10] = 9
    ctx = [int(x) for x in new + rng.integers(0, 30, B)]
    cu = 5 + np.concatenate([[0], np.cumsum(new)])
    c, t, desc, front, table = with_prefix(L, P, ctx, 16, 1, D, rng)
    q = dev(rng.standard_normal((int(cu[-1]), Hq, D)), DT[dtype])
    kw = dict(slopes=ALIBI(Hq) * 0.1) if biased else {}
    for bad in (P, 2 ** 31 - 1, 2 ** 31 - 20, 10 ** 9, -1, -2 ** 31):
        out, lse, st = shared(L, desc, 1, front, bad, table, ctx, cu, q, dtype, window, max_q=2, **kw)
        assert st == L.E0_ST_BAD_LENGTH
        for rows in (slice(0, 5), slice(cu[10], cu[11]), slice(cu[-1], None)):
            assert (out[rows] == -7).all() and (lse[rows] == -7).all()
        check_shared(c, front, P if bad == P else 0, table, ctx, cu, q, out, lse, dtype, window, skip=(10,), **kw)
