"""Attention under score rules and over a shared prefix where lengths, positions and schedules go to their ends, on the
GPU against 64-bit references; tolerances as in test_attn_rules."""
import numpy as np
import pytest

from tests.test_attn_rules import (ALIBI, Tables, check_shared, compare, rules_ref, shared, weights_of,
                                   with_prefix)
from tests.test_layer_ops import BF16, DT, EPS, F16, F32, L, dev, f64  # noqa: F401

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


@pytest.mark.usefixtures("room")
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("P", [0, 1, 2])
def test_queries_before_the_first_position(L, D, dtype, P):  # noqa: F811
    """Sequences with more queries than tokens: their queries' positions are -1 and less, counted from an empty or a short
    prefix.  Their rows are written all the same: with the prefix, or with zeros where there is none."""
    rng = np.random.default_rng(D + P)
    B, Hq = 72, 4
    new = rng.integers(1, 4, B)
    ctx = np.where(np.arange(B) % 3 == 0, 0, new + rng.integers(0, 30, B))
    tokens = ctx.copy()  # what the device is told: some lengths that cannot be
    tokens[3], tokens[6] = -5, 10 ** 9
    cu = np.concatenate([[0], np.cumsum(new)])
    c, t, desc, front, table = with_prefix(L, P, [int(x) for x in ctx], 16, 1, D, rng)
    table[[b for b in range(B) if ctx[b] == 0]] = -1
    q = dev(rng.standard_normal((int(cu[-1]), Hq, D)), DT[dtype])
    out, lse, st = shared(L, desc, 1, front, P, table, tokens, cu, q, dtype)
    assert st == L.E0_ST_BAD_LENGTH
    none = [b for b in range(B) if ctx[b] == 0]
    check_shared(c, front, P, table, ctx, cu, q, out, lse, dtype, skip=none)
    pk, pv = c.row(front, P)
    werr, quantum = weights_of(dtype, dtype != F32, dtype == BF16, c.vs)
    for b in none:
        rows = slice(cu[b], cu[b + 1])
        if P == 0:
            assert (out[rows] == 0).all() and torch.isneginf(lse[rows]).all(), b
            continue
        want = rules_ref(f64(q[rows]), pk, pv, float(np.float32(D ** -0.5)), np.zeros(new[b]), np.ones((new[b], P), bool),
                         weight_err=werr + 32 * EPS, quantum=quantum)
        compare(f64(out[rows]), f64(lse[rows]), (*want[:3], want[3] + 32 * EPS * (1 + np.abs(want[1]))), dtype, b)
