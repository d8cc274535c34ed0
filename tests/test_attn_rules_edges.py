"""Attention under score rules and over a shared prefix where lengths, positions and schedules go to their ends, on the
GPU against 64-bit references; tolerances as in test_attn_rules."""
import numpy as np
import pytest

from tests.test_attn_rules import (ALIBI, Tables, check_scored, check_shared, compare, rules_ref, scored, shared,
                                   weights_of, with_prefix)
from tests.test_layer_ops import BF16, DT, EPS, F16, F32, L, dev, f64, filled_cache, status  # noqa: F401

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


@pytest.mark.usefixtures("room")
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("kw", [{}, dict(window=333), dict(cap=6.0, biased=True)])
def test_prompts_behind_a_prefix(L, dtype, kw):  # noqa: F811
    """Sequences whose own new tokens are hundreds, some of them behind cached ones."""
    rng = np.random.default_rng(17)
    kw = dict(kw)
    new, held = [400, 1, 130, 0, 257], [0, 90, 300, 4, 1]
    ctx = [n + h for n, h in zip(new, held)]
    cu = np.concatenate([[0], np.cumsum(new)])
    Hq, Hkv, D, P = 4, 2, 64, 300
    if kw.pop("biased", False):
        kw["slopes"] = ALIBI(Hq) * 0.1
    c, t, desc, front, table = with_prefix(L, P, ctx, 32, Hkv, D, rng)
    q = dev(rng.standard_normal((int(cu[-1]), Hq, D)), DT[dtype])
    out, lse, st = shared(L, desc, Hkv, front, P, table, ctx, cu, q, dtype, **kw)
    assert st == 0
    check_shared(c, front, P, table, ctx, cu, q, out, lse, dtype, **kw)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("P", [0, 1, 300])
def test_more_tiles_than_blocks_behind_a_prefix(L, D, dtype, P):  # noqa: F811
    """So many rows that a block has several tiles: the results come together in a kernel of their own, without a window."""
    rng = np.random.default_rng(D + P)
    B, Hq, Hkv = 40, 32, 8
    new = rng.integers(20, 45, B)
    ctx = [int(x) for x in new + rng.integers(0, 30, B)]
    cu = np.concatenate([[0], np.cumsum(new)])
    c, t, desc, front, table = with_prefix(L, P, ctx, 64, Hkv, D, rng)
    q = dev(rng.standard_normal((int(cu[-1]), Hq, D)), DT[dtype])
    Tables.room = True
    try:
        out, lse, st = shared(L, desc, Hkv, front, P, table, ctx, cu, q, dtype)
    finally:
        Tables.room = False
    assert st == 0
    check_shared(c, front, P, table, ctx, cu, q, out, lse, dtype)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("Hq,Hkv,D", [(64, 1, 64), (200, 1, 128), (300, 1, 64), (130, 2, 256), (513, 1, 64)])
@pytest.mark.parametrize("cap", [0.0, 5.0])
def test_many_heads_of_a_kv_head(L, Hq, Hkv, D, dtype, cap):  # noqa: F811
    """Single tokens whose heads alone fill a tile, or do not divide one; cu_q may be NULL then."""
    rng = np.random.default_rng(Hq)
    B = 9
    ctx = [int(x) for x in rng.integers(1, 700, B)]
    ctx[3] = 1
    c, t, desc, table = filled_cache(L, B, 16, Hkv, D, ctx, rng)
    q = dev(rng.standard_normal((B, Hq, D)), DT[dtype])
    room = np.pad(table, ((0, 0), (0, 512 - table.shape[1])), constant_values=-1)  # for 8192 positions
    out, ls = torch.full((B + 1, Hq, D), -7.0, dtype=DT[dtype], device="cuda"), torch.full((B + 1, Hq), -7.0, device="cuda")
    wsb = L.e0_attn_scored_workspace_size(B, Hq, Hkv, D, 1)
    ws, st = torch.full((wsb,), 255, dtype=torch.uint8, device="cuda"), status()
    L.e0_attn_scored(desc, dev(room), 512, dev(np.asarray(ctx, np.int32)), None, B, 1, q, dtype, Hq * D, Hq, D ** -0.5,
                     L.AttnRules(cap), out, Hq * D, ls, ws, wsb, st)
    assert L.e0_read_status(st) == 0
    check_scored(c, table, ctx, np.arange(B + 1), q, out, ls, dtype, cap=cap, tiles=dtype != F32)


@pytest.mark.usefixtures("room")
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_first_and_open_at_their_types_ends(L, dtype):  # noqa: F811
    """Any 32-bit number may stand in first and open_len, and the largest window."""
    rng = np.random.default_rng(23)
    new, ctx = [70, 1, 100], [300, 40, 100]
    cu = np.concatenate([[0], np.cumsum(new)])
    c, t, desc, table = filled_cache(L, 3, 16, 1, 64, ctx, rng)
    q = dev(rng.standard_normal((int(cu[-1]), 4, 64)), DT[dtype])
    ends = np.array([-2 ** 31, -1, 0, 1, 50, 2 ** 31 - 1, 2 ** 31 - 64, 299])
    first = ends[rng.integers(0, len(ends), int(cu[-1]))]
    for opens in ([-2 ** 31, 2 ** 31 - 1, 60], [2 ** 31 - 1, -1, 2 ** 30]):
        for window in (0, 37, 2 ** 31 - 1):
            kw = dict(first=first, opens=opens, window=window)
            out, lse, st = scored(L, desc, 1, table, ctx, cu, q, dtype, **kw)
            assert st == 0
            check_scored(c, table, ctx, cu, q, out, lse, dtype, **kw)


@pytest.mark.usefixtures("room")
@pytest.mark.parametrize("bad", [-2 ** 31, -2 ** 31 + 1, -1, 2 ** 31 - 1])
def test_any_block_id_that_is_none(L, bad):  # noqa: F811
    """Every 32-bit number that is no block's is reported, in a sequence's table and in a prefix'."""
    rng = np.random.default_rng(31)
    n, ctx, P = 90, [90], 60
    c, t, desc, front, table = with_prefix(L, P, ctx, 16, 1, 64, rng)
    q = dev(rng.standard_normal((n, 4, 64)), torch.float16)
    hole = table.copy()
    hole[0, 2] = bad
    out, lse, st = scored(L, desc, 1, hole, ctx, [0, n], q, F16)
    assert st == L.E0_ST_BAD_BLOCK
    check_scored(c, np.where((hole < 0) | (hole >= c.n), -1, hole), ctx, [0, n], q, out, lse, F16)
    hole = front.copy()
    hole[1] = bad
    out, lse, st = shared(L, desc, 1, hole, P, table, ctx, [0, n], q, F16)
    assert st == L.E0_ST_BAD_BLOCK
    check_shared(c, np.where((hole < 0) | (hole >= c.n), -1, hole), P, table, ctx, [0, n], q, out, lse, F16)


@pytest.mark.usefixtures("room")
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_blocks_that_nobody_sees_may_be_gone(L, dtype):  # noqa: F811
    """Prefix blocks before every window, and blocks before every document: their ids are not looked at."""
    rng = np.random.default_rng(37)
    B, Hq, D, P, window = 40, 4, 64, 400, 100
    new = rng.integers(1, 4, B)
    ctx = [int(x) for x in new + rng.integers(0, 20, B)]
    cu = np.concatenate([[0], np.cumsum(new)])
    c, t, desc, front, table = with_prefix(L, P, ctx, 16, 1, D, rng)
    q = dev(rng.standard_normal((int(cu[-1]), Hq, D)), DT[dtype])
    least = P + min(x - n for x, n in zip(ctx, new)) - window + 1
    gone = front.copy()
    gone[:least // 16] = -1
    assert least // 16 > 15
    out, lse, st = shared(L, desc, 1, gone, P, table, ctx, cu, q, dtype, window)
    assert st == 0
    check_shared(c, front, P, table, ctx, cu, q, out, lse, dtype, window)
    q = torch.cat([q[:7], q])  # rows of no sequence see nothing either
    out, lse, st = shared(L, desc, 1, gone, P, table, ctx, 7 + cu, q, dtype, window)
    assert st == 0 and (out[:7] == -7).all()
    check_shared(c, front, P, table, ctx, 7 + cu, q, out, lse, dtype, window)
    n, ctx = 60, [500]
    c, t, desc, table = filled_cache(L, 1, 16, 1, D, ctx, rng)
    q = dev(rng.standard_normal((n, Hq, D)), DT[dtype])
    first = rng.integers(300, 440, n)
    gone = table.copy()
    gone[0, :first.min() // 16] = -1
    out, lse, st = scored(L, desc, 1, gone, ctx, [0, n], q, dtype, first=first)
    assert st == 0
    check_scored(c, table, ctx, [0, n], q, out, lse, dtype, first=first)
    for m in (1, 3, n):  # documents that begin behind everything there is
        first = np.full(m, 501)
        out, lse, st = scored(L, desc, 1, np.full_like(table, -1), ctx, [0, m], q[:m], dtype, first=first)
        assert st == 0 and (out[:m] == 0).all() and torch.isneginf(lse[:m]).all()
    # windows that end before their prefix' last block does
    c, t, desc, front, table = with_prefix(L, 390, [20], 16, 1, D, rng)
    out, lse, st = shared(L, desc, 1, np.full_like(front, -1), 390, table, [20], [0, 1], q[:1], dtype, 20)
    assert st == 0
    check_shared(c, front, 390, table, [20], [0, 1], q[:1], out, lse, dtype, 20)
