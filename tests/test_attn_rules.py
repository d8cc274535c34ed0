"""Attention under score rules (a cap, a bias by distance, documents, open prefixes) and
over a prefix that the batch shares, on the GPU against 64-bit references.

Tolerances: EPS = 2^-23 is one step of fp32, H[dtype] half a step of an output's type; `rules_ref`
says what it counts."""
import numpy as np
import pytest

from tests import layer_ref as R
from tests.test_layer_ops import (BF16, DT, EPS, F16, F32, H, TINY16, L, attend, cache_dev, dev, f64,  # noqa: F401
                                  filled_cache, status)

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

TILE_ROWS = 64  # rows of a KV head from which 16-bit queries can go through the tiles
ROOM = 8192     # positions: with tables of as many, calls of some hundred rows do
WORTH = 5_000_000  # pairs of rows and positions from which all do


class Tables:
    """Tables as long as what the cache holds, or with room for more, where calls of few rows go another way."""
    room = False

    @classmethod
    def widen(cls, table, bs):
        table = np.atleast_2d(np.asarray(table, np.int32))
        n = ROOM // bs - table.shape[1] if cls.room else 0
        return np.pad(table, ((0, 0), (0, max(n, 0))), constant_values=-1)


@pytest.fixture(params=[False, True], ids=["held", "room"])
def room(request):
    Tables.room = request.param
    yield request.param
    Tables.room = False


def rules_ref(q, k, v, scale, p, seen, cap=0.0, slopes=None, weight_err=0.0, quantum=0.0, more=0.0):
    """q [n][Hq][D] at the positions p, k and v [S][Hkv][D] (NaN: not there), seen [n][S].  Returns out, lse and what
    they may be off by; `more`: of a score, beside its own."""
    n, Hq, D = q.shape
    G = Hq // k.shape[1]
    j = np.arange(len(k))
    out, lse = np.zeros(q.shape), np.full((n, Hq), -np.inf)
    tol, ltol = np.zeros(q.shape), np.zeros((n, Hq))
    there = ~np.isnan(k[:, 0, 0]) if len(k) else np.zeros(0, bool)
    see = seen & there[None, :]
    rows = see.any(1)
    if not rows.any():
        return out, lse, tol, ltol
    k, v = np.where(there[:, None, None], k, 0.0), np.where(there[:, None, None], v, 0.0)
    count = see.sum(1)
    for h in range(Hq):
        kk, vv = k[:, h // G], v[:, h // G]
        s = q[:, h] @ kk.T * scale
        mag = np.abs(q[:, h]) @ np.abs(kk).T * abs(scale)
        # a score: D products of operands of 22 bits and more, summed in fp32, and factors of three roundings
        off = (D + 16) * EPS * mag + (4 * EPS + more) * np.abs(s)
        if cap:
            s = cap * np.tanh(s / cap)
            off = off + 4 * EPS * cap  # the cap's own steps: an exponential, a division, two products
        if slopes is not None:
            bias = slopes[h] * np.abs(p[:, None] - j[None, :])
            s = s - bias
            off = off + 2 * EPS * (bias + np.abs(s))
        s = np.where(see, s, -np.inf)
        m = np.where(rows, s.max(1), 0.0)
        e = np.exp(s - m[:, None])
        z = np.where(rows, e.sum(1), 1.0)
        w = e / z[:, None]
        out[:, h] = w @ vv
        lse[rows, h] = (m + np.log(z))[rows]
        ds = np.where(see, off, 0.0).max(1) + 4 * EPS * np.where(see, np.abs(s), 0.0).max(1)
        rel = 2 * ds + (count / 4 + 64) * EPS  # exp2's argument and result; sums over the positions
        tol[:, h] = (rel + weight_err)[:, None] * (w @ np.abs(vv)) + (count * quantum)[:, None]
        ltol[:, h] = rel + 4 * EPS * np.abs(np.where(rows, lse[:, h], 0.0))
    return out, lse, tol, ltol


def weights_of(dtype, tiles, wide, vs):
    """How far the weights' rounding is off: as a share of a weight, and for each position in units of the output.
    Tiles: fp16 with bf16 outputs, 22 bits with fp16 ones; weights are at most 2^15 and the largest at least 2^-1, so
    what falls below fp16's steps (2^-24, half of one lost) is 2^-24 of the largest's code, 448 of a scale."""
    if tiles:
        return (2.0 ** -11 if dtype == BF16 else 2.0 ** -21), 2.0 ** -24 * 448 * float(np.nanmax(vs))
    return (2.0 ** -11, 2.0 ** -24 * 448 * float(np.nanmax(vs))) if wide else (0.0, 0.0)


def compare(got, gl, want, dtype, where=""):
    o, l, tol, ltol = want
    if dtype == F16:  # beyond fp16's largest number and half a step the result is infinity
        assert np.isinf(got[np.abs(o) > 65520 + tol]).all(), where
        over = np.isinf(got) & (np.abs(o) > 65520 - tol) & (np.sign(got) == np.sign(o))
        got, o = np.where(over, 0.0, got), np.where(over, 0.0, o)
    assert (np.abs(got - o) <= tol + H[dtype] * np.abs(o) * 1.0001 + TINY16[dtype]).all(), \
        (where, np.abs(got - o).max(), np.argwhere(~(np.abs(got - o) <= tol + H[dtype] * np.abs(o) * 1.0001 + TINY16[dtype]))[:4])
    if gl is not None:
        none = np.isneginf(l)
        assert np.isneginf(gl[none]).all() and (np.abs(gl[~none] - l[~none]) <= ltol[~none]).all(), where


def scored(L, desc, Hkv, table, ctx, cu, q, dtype, window=0, cap=0.0, slopes=None, first=None, opens=None,  # noqa: F811
           scale=None, out=None, lse=True, pad=2, max_q=None, stream=None, rows=0):
    T, Hq, D = q.shape
    B = len(ctx)
    n = np.diff(cu)
    if max_q is None:
        max_q = max(1, int(n.max()))
        if Tables.room and B * Hq < WORTH:
            max_q = max(max_q, TILE_ROWS)
            while B * max_q * Hq * min(ROOM, window + max_q if window else ROOM) < WORTH:
                max_q *= 2
    table = Tables.widen(table, desc.block_tokens)
    if out is None:
        out = torch.full((T + pad, Hq, D), -7.0, dtype=DT[dtype], device="cuda")
    ls = torch.full((T + pad, Hq), -7.0, device="cuda") if lse else None
    keep = [None if x is None else dev(np.asarray(x, t)) for x, t in
            ((slopes, np.float32), (first, np.int32), (opens, np.int32))]
    rules = L.AttnRules(cap, window, *[L.ptr(x) for x in keep], rows)
    wsb = L.e0_attn_scored_workspace_size(B, Hq, Hkv, D, max_q)
    ws = torch.full((wsb,), 255, dtype=torch.uint8, device="cuda")
    st = status()
    L.e0_attn_scored(desc, dev(table), table.shape[1], dev(np.asarray(ctx, np.int32)),
                     dev(np.asarray(cu, np.int32)), B, max_q, q, dtype, q.stride(0), Hq, scale or 1 / np.sqrt(D), rules, out,
                     out.stride(0), ls, ws, wsb, st, stream=stream)
    return out, ls, L.e0_read_status(st)


def check_scored(c, table, ctx, cu, q, out, lse, dtype, window=0, cap=0.0, slopes=None, first=None, opens=None, scale=None,
                 more=0.0, tiles=None):
    T, Hq, D = q.shape
    scale = float(np.float32(scale or 1 / np.sqrt(D)))
    slopes = None if slopes is None else np.asarray(slopes, np.float32).astype(np.float64)
    got, gl, qv = f64(out), f64(lse) if lse is not None else None, f64(q)
    rows = int(np.diff(cu).max()) * (Hq // c.H)
    tiles = dtype != F32 and (rows >= TILE_ROWS or Tables.room) if tiles is None else tiles
    werr, quantum = weights_of(dtype, tiles, dtype == BF16 and rows > 8, c.vs)
    for b in range(len(ctx)):
        at = slice(cu[b], cu[b + 1])
        n = cu[b + 1] - cu[b]
        if n == 0:
            continue
        k, v = c.row(table[b], int(ctx[b]))
        p, j = ctx[b] - n + np.arange(n), np.arange(ctx[b])
        seen = j[None, :] <= p[:, None]
        if opens is not None:
            seen = seen | (j < opens[b])[None, :]
        if first is not None:
            seen = seen & (j[None, :] >= np.asarray(first)[at][:, None])
        if window:
            seen = seen & (j[None, :] > p[:, None] - window)
        want = rules_ref(qv[at], k, v, scale, p, seen, cap, slopes, werr, quantum, more)
        compare(got[at], None if gl is None else gl[at], want, dtype, (b, n, ctx[b]))
    end = cu[-1]
    assert (got[end:] == -7).all() and (gl is None or (gl[end:] == -7).all())


ALIBI = lambda Hq: 2.0 ** (-8.0 * np.arange(1, Hq + 1) / Hq)  # noqa: E731


# ------------------------------------------------------------------ tiles: the plain case first


@pytest.mark.usefixtures("room")
@pytest.mark.parametrize("D", [128, 64, 256])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_prompt_of_one_tile(L, D, dtype):  # noqa: F811
    rng = np.random.default_rng(D)
    ctx, cu = [64], [0, 64]
    c, t, desc, table = filled_cache(L, 1, 64, 1, D, ctx, rng)
    q = dev(rng.standard_normal((64, 1, D)), DT[dtype])
    out, lse, st = scored(L, desc, 1, table, ctx, cu, q, dtype)
    assert st == 0
    check_scored(c, table, ctx, cu, q, out, lse, dtype)


@pytest.mark.usefixtures("room")
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("bs", [16, 128])
def test_prompts_of_many_lengths(L, D, dtype, bs):  # noqa: F811
    """Around the edges of tiles, units and blocks; behind cached tokens and from nothing; none at all."""
    rng = np.random.default_rng(D + bs)
    new = [1, 0, 31, 64, 65, 127, 128, 129, 200, 300]
    held = [5, 9, 0, 64, 1, 0, 128, 500, 0, 77]
    ctx = [a + b for a, b in zip(new, held)]
    cu = np.concatenate([[0], np.cumsum(new)])
    c, t, desc, table = filled_cache(L, len(ctx), bs, 2, D, ctx, rng)
    q = dev(rng.standard_normal((int(cu[-1]), 6, D)) * 1.5, DT[dtype])
    out, lse, st = scored(L, desc, 2, table, ctx, cu, q, dtype)
    assert st == 0
    check_scored(c, table, ctx, cu, q, out, lse, dtype)


@pytest.mark.usefixtures("room")
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 8), (4, 1), (24, 3), (20, 1), (7, 1), (40, 2)])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("window", [0, 1, 90])
def test_prompts_heads_and_windows(L, Hq, Hkv, dtype, window):  # noqa: F811
    rng = np.random.default_rng(Hq * 7 + window)
    new, ctx = [70, 3, 140], [270, 3, 1140]
    cu = np.concatenate([[0], np.cumsum(new)])
    c, t, desc, table = filled_cache(L, 3, 32, Hkv, 64, ctx, rng)
    q = dev(rng.standard_normal((int(cu[-1]), Hq, 64)) * 2, DT[dtype])
    out, lse, st = scored(L, desc, Hkv, table, ctx, cu, q, dtype, window)
    assert st == 0
    check_scored(c, table, ctx, cu, q, out, lse, dtype, window)


# ------------------------------------------------------------------ rules, for single tokens and for prompts


@pytest.mark.usefixtures("room")
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("new", [[1, 1, 1, 1, 1], [3, 0, 2, 1, 4], [40, 1, 130, 66, 0]])
@pytest.mark.parametrize("rule", ["cap", "slopes", "both"])
def test_capped_and_biased_scores(L, D, dtype, new, rule):  # noqa: F811
    rng = np.random.default_rng(D + sum(new))
    ctx = [max(n, x) for n, x in zip(new, (1, 30, 130, 700, 2000))]
    cu = np.concatenate([[0], np.cumsum(new)])
    c, t, desc, table = filled_cache(L, 5, 32, 2, D, ctx, rng)
    q = dev(rng.standard_normal((int(cu[-1]), 8, D)) * 3, DT[dtype])
    kw = dict(cap=5.0 if rule != "slopes" else 0.0, slopes=ALIBI(8) * (-1) ** np.arange(8) * 0.1 if rule != "cap" else None)
    out, lse, st = scored(L, desc, 2, table, ctx, cu, q, dtype, **kw)
    assert st == 0
    check_scored(c, table, ctx, cu, q, out, lse, dtype, **kw)


@pytest.mark.usefixtures("room")
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("long", [False, True])
def test_documents_and_open_prefixes(L, D, dtype, long):  # noqa: F811
    """Documents in any order of first positions, rows that see nothing, open prefixes before, around and behind the
    queries, and all of it within a window."""
    rng = np.random.default_rng(D + long)
    new = [150, 1, 333, 40, 64] if long else [2, 1, 5, 3, 0]
    ctx = [n + x for n, x in zip(new, (50, 300, 0, 1000, 0))]
    cu = np.concatenate([[0], np.cumsum(new)])
    c, t, desc, table = filled_cache(L, 5, 16, 2, D, ctx, rng)
    T = int(cu[-1])
    q = dev(rng.standard_normal((T, 4, D)) * 1.5, DT[dtype])
    seq = np.repeat(np.arange(5), new)
    pos = np.concatenate([ctx[b] - new[b] + np.arange(new[b]) for b in range(5)])
    first = rng.integers(-5, np.asarray(ctx)[seq] + 1)  # some beyond their own position
    first[::3] = np.maximum(pos[::3] - rng.integers(0, 20, len(first[::3])), 0)
    opens = [100, 0, 333, 20, 5] if long else [1, 301, 3, 2000, 0]
    for kw in (dict(first=first), dict(opens=opens), dict(first=first, opens=opens), dict(first=first, opens=opens, window=30),
               dict(opens=opens, window=64, cap=7.0, slopes=ALIBI(4) * 0.05)):
        out, lse, st = scored(L, desc, 2, table, ctx, cu, q, dtype, **kw)
        assert st == 0
        check_scored(c, table, ctx, cu, q, out, lse, dtype, **kw)


@pytest.mark.usefixtures("room")
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("D,Hq,Hkv", [(128, 8, 1), (64, 4, 2), (256, 2, 1)])
def test_long_contexts_cut_among_blocks(L, D, Hq, Hkv, dtype):  # noqa: F811
    """Few rows, contexts long enough for every block of the GPU to have a part."""
    rng = np.random.default_rng(D + Hq)
    new, ctx = [70, 100], [9000, 4000]
    cu = [0, 70, 170]
    c, t, desc, table = filled_cache(L, 2, 64, Hkv, D, ctx, rng)
    q = dev(rng.standard_normal((170, Hq, D)) * 2, DT[dtype])
    for kw in (dict(), dict(window=3000), dict(cap=20.0)):
        out, lse, st = scored(L, desc, Hkv, table, ctx, cu, q, dtype, **kw)
        assert st == 0
        check_scored(c, table, ctx, cu, q, out, lse, dtype, **kw)
        again, _, _ = scored(L, desc, Hkv, table, ctx, cu, q, dtype, **kw)
        assert torch.equal(out, again)


@pytest.mark.usefixtures("room")
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_caps_of_any_size(L, dtype):  # noqa: F811
    """A cap that makes all scores alike, below fp32's normal numbers too, and one that no score comes near."""
    rng = np.random.default_rng(11)
    ctx, cu = [300, 90], np.array([0, 70, 140])
    c, t, desc, table = filled_cache(L, 2, 16, 2, 64, ctx, rng)
    q = dev(rng.standard_normal((140, 4, 64)) * 2, DT[dtype])
    q[3] = 0
    for cap in (1e-42, 1e-38, 1e-20):  # scores of that size: their weights are equal to 2^-60
        out, lse, st = scored(L, desc, 2, table, ctx, cu, q, dtype, cap=cap)
        assert st == 0
        check_scored(c, table, ctx, cu, torch.zeros_like(q), out, lse, dtype)
    for cap in (1e20, 3e38):  # s^3 / (3 cap^2) is less than 2^-100 of s = 1000
        out, lse, st = scored(L, desc, 2, table, ctx, cu, q, dtype, cap=cap)
        assert st == 0
        # the score through the cap and back: a product with its inverse, the tangent's factor, a product with it
        check_scored(c, table, ctx, cu, q, out, lse, dtype, more=4 * EPS)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_few_rows_in_all(L, dtype):  # noqa: F811
    """Where the rows in all are told, a step of single tokens takes the path for few rows, whatever max_q is."""
    rng = np.random.default_rng(12)
    ctx, cu = [int(x) for x in rng.integers(1, 900, 20)], np.arange(21)
    c, t, desc, table = filled_cache(L, 20, 32, 2, 128, ctx, rng)
    q = dev(rng.standard_normal((20, 8, 128)), DT[dtype])
    wide = np.pad(table, ((0, 0), (0, 256 - table.shape[1])), constant_values=-1)
    a, la, _ = attend(L, c, desc, wide, ctx, cu, q, dtype, max_q=512)  # that path by itself; bf16's bits know max_q there, too
    b, lb, st = scored(L, desc, 2, wide, ctx, cu, q, dtype, max_q=512, rows=20)
    assert st == 0 and torch.equal(a, b) and torch.equal(la, lb)
    b, lb, st = scored(L, desc, 2, wide, ctx, cu, q, dtype, max_q=512)
    assert st == 0
    check_scored(c, table, ctx, cu, q, b, lb, dtype, tiles=dtype != F32)


def test_no_rules_is_plain_attention(L):  # noqa: F811
    rng = np.random.default_rng(1)
    ctx, cu = [100, 1, 2000], [0, 1, 2, 3]
    c, t, desc, table = filled_cache(L, 3, 64, 2, 128, ctx, rng)
    for dtype in (F32, F16, BF16):
        q = dev(rng.standard_normal((3, 8, 128)), DT[dtype])
        a, la, _ = attend(L, c, desc, table, ctx, np.asarray(cu), q, dtype)
        b, lb, st = scored(L, desc, 2, table, ctx, cu, q, dtype)
        assert st == 0 and torch.equal(a, b) and torch.equal(la, lb)


@pytest.mark.usefixtures("room")
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_tiles_of_far_scales_and_large_scores(L, dtype):  # noqa: F811
    """Value scales 2^40 apart, scores of hundreds that grow along the context, queries of any size."""
    rng = np.random.default_rng(2)
    D, n, ctx = 128, 80, [700]
    c, t, desc, table = filled_cache(L, 1, 16, 1, D, ctx, rng)
    c.vs[:] = np.where(np.isnan(c.vs), c.vs, c.vs * 2.0 ** rng.integers(-20, 20, c.vs.shape))
    c.ks[table[0, :44], 0] *= np.linspace(0.1, 8, 44).astype(np.float32)
    t, desc = cache_dev(L, c)
    size = 10.0 ** rng.uniform(-3, 3, (n, 1, 1)) if dtype == BF16 else 10.0 ** rng.uniform(-2, 2, (n, 1, 1))
    q = dev(rng.standard_normal((n, 1, D)) * size, DT[dtype])
    out, lse, st = scored(L, desc, 1, table, ctx, [0, n], q, dtype)
    assert st == 0
    check_scored(c, table, ctx, [0, n], q, out, lse, dtype)


@pytest.mark.usefixtures("room")
@pytest.mark.parametrize("n", [1, 90])
def test_non_finite_queries_and_codes_that_nobody_sees(L, n):  # noqa: F811
    """A query's NaN stays in its row; NaN codes behind a row's position or before its document do not reach it."""
    rng = np.random.default_rng(3)
    D, ctx = 64, [n + 50]
    c, t, desc, table = filled_cache(L, 1, 16, 1, D, ctx, rng)
    blk = table[0, 1]
    c.k[blk, :, 3], c.v[blk, :, 3] = 0x7F, 0xFF  # position 19
    t, desc = cache_dev(L, c)
    q = dev(rng.standard_normal((n, 2, D)), torch.float16)
    q[0, 1, 5] = float("nan")
    first = np.full(n, 20)
    out, lse, st = scored(L, desc, 1, table, ctx, [0, n], q, F16, first=first)
    assert st == 0 and out[0, 1].isnan().all() and lse[0, 1].isnan()
    ok = q.clone()
    ok[0, 1] = 0
    c.k[blk, :, 3] = c.v[blk, :, 3] = 0
    t2, desc2 = cache_dev(L, c)
    ref, rl, _ = scored(L, desc2, 1, table, ctx, [0, n], ok, F16, first=first)
    keep = torch.ones((n, 2), dtype=torch.bool, device="cuda")
    keep[0, 1] = False
    assert torch.equal(out[:n][keep], ref[:n][keep]) and torch.equal(lse[:n][keep], rl[:n][keep])


@pytest.mark.usefixtures("room")
@pytest.mark.parametrize("n", [1, 3, 90])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_capped_scores_know_nothing_of_one_another(L, n, dtype):  # noqa: F811
    """Scores far beyond the cap in places that a row does not see, or in other rows, leave no trace in its bits; a
    query's NaN stays NaN beside scores beyond the cap."""
    rng = np.random.default_rng(n)
    D, ctx, Hq = 64, [n + 50], 4
    c, t, desc, table = filled_cache(L, 1, 16, 2, D, ctx, rng)
    c.k[:] = R.encode(rng.standard_normal(c.k.shape) * 0.1)
    c.ks[np.isnan(c.ks)] = c.vs[np.isnan(c.vs)] = 1.0
    c.ks[:] = 1.0
    t, desc = cache_dev(L, c)
    q = dev(rng.standard_normal((n, Hq, D)), DT[dtype])
    first = np.full(n, 20)
    kw = dict(cap=4.0, first=first)
    a, la, st = scored(L, desc, 2, table, ctx, [0, n], q, dtype, **kw)
    assert st == 0
    check_scored(c, table, ctx, [0, n], q, a, la, dtype, **kw)
    blk, last = table[0, 1], table[0, (ctx[0] - 1) // 16]
    c.k[blk, :, :4] = 0x7E  # positions 16 to 19: 448
    if ctx[0] % 16:
        c.k[last, :, ctx[0] % 16:] = 0x7E  # behind the last one
    t2, desc2 = cache_dev(L, c)
    b, lb, _ = scored(L, desc2, 2, table, ctx, [0, n], q, dtype, **kw)
    assert torch.equal(a, b) and torch.equal(la, lb)
    large = q.clone()
    large[0, 1] *= 100  # its own scores are beyond the cap
    b, lb, _ = scored(L, desc2, 2, table, ctx, [0, n], large, dtype, **kw)
    keep = torch.ones((n, Hq), dtype=torch.bool, device="cuda")
    keep[0, 1] = False
    assert torch.equal(a[:n][keep], b[:n][keep]) and torch.equal(la[:n][keep], lb[:n][keep])
    large[0, 1, 3] = float("nan")
    large[0, 0] *= 100
    b, lb, _ = scored(L, desc2, 2, table, ctx, [0, n], large, dtype, **kw)
    assert b[0, 1].isnan().all() and lb[0, 1].isnan() and b[0, 0].isfinite().all()


@pytest.mark.usefixtures("room")
@pytest.mark.parametrize("n", [2, 100])
def test_bad_lengths_and_blocks(L, n):  # noqa: F811
    rng = np.random.default_rng(4)
    D, ctx = 64, [n + 60, n + 10, n + 40]
    cu = [0, n, 2 * n, 3 * n]
    c, t, desc, table = filled_cache(L, 3, 16, 1, D, ctx, rng)
    q = dev(rng.standard_normal((3 * n, 2, D)), torch.float16)
    bad = table.copy()
    bad[0, 2], bad[2, 0] = c.n + 5, -9
    out, lse, st = scored(L, desc, 1, bad, ctx, cu, q, F16)
    assert st == L.E0_ST_BAD_BLOCK
    check_scored(c, np.where((bad < 0) | (bad >= c.n), -1, bad), ctx, cu, q, out, lse, F16)  # their tokens are not seen
    long = [ctx[0], 10 ** 9, -3]
    out, lse, st = scored(L, desc, 1, table, long, cu, q, F16)
    assert st == L.E0_ST_BAD_LENGTH
    check_scored(c, table, ctx[:1], cu[:2], q[:n], out[:n], lse[:n], F16)
    assert (out[n:3 * n] == 0).all() and torch.isneginf(lse[n:3 * n]).all()
    worse = [0, n, n - 1, 3 * n]  # falls; then more than max_q
    out, lse, st = scored(L, desc, 1, table, ctx, worse, q, F16, max_q=n)
    assert st == L.E0_ST_BAD_LENGTH and (out[n:] == -7).all()
    check_scored(c, table, ctx[:1], cu[:2], q[:n], out[:n], lse[:n], F16)


@pytest.mark.usefixtures("room")
@pytest.mark.parametrize("D", [64, 128, 256])
def test_strided_queries_and_unaligned_outputs(L, D):  # noqa: F811
    """Queries inside a projection's rows, outputs at odd addresses and strides, no lse."""
    rng = np.random.default_rng(D)
    n, Hq, ctx = 75, 4, [200]
    c, t, desc, table = filled_cache(L, 1, 32, 2, D, ctx, rng)
    for dtype in (F16, BF16):
        wide = dev(rng.standard_normal((n, Hq + 4, D)), DT[dtype])
        q = wide[:, :Hq]
        buf = torch.full((n * (Hq * D + 3) + 1 + Hq * D,), -7.0, dtype=DT[dtype], device="cuda")
        out = torch.as_strided(buf, (n, Hq, D), (Hq * D + 3, D, 1), 1)
        scored(L, desc, 2, table, ctx, [0, n], q, dtype, out=out, lse=False)
        want, _, _ = scored(L, desc, 2, table, ctx, [0, n], q.contiguous(), dtype)
        assert torch.equal(out, want[:n])
        mask = torch.ones_like(buf, dtype=torch.bool)
        torch.as_strided(mask, (n, Hq, D), (Hq * D + 3, D, 1), 1).fill_(False)
        assert (buf[mask] == -7).all()


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("D,Hq,Hkv", [(128, 16, 4), (64, 8, 2)])
@pytest.mark.parametrize("open_part", [False, True])
def test_short_last_tiles_between_long_prompts(L, D, Hq, Hkv, dtype, open_part):  # noqa: F811
    """Tiles of which only the first half has rows, several heads of them before tiles of two halves: whoever works on
    the second half is there early, and has to wait for its own queries."""
    rng = np.random.default_rng(D + open_part)
    new = [714, 33, 70, 1500, 10, 17, 918, 30, 800, 95, 954]
    held = [774, 100, 0, 585, 745, 3, 632, 175, 0, 40, 859]
    ctx = [a + b for a, b in zip(new, held)]
    cu = np.concatenate([[0], np.cumsum(new)])
    c, t, desc, table = filled_cache(L, len(new), 32, Hkv, D, ctx, rng)
    # queries of many sizes: each row's own factor counts
    q = dev(rng.standard_normal((int(cu[-1]), Hq, D)) * 2.0 ** rng.integers(-6, 2, (int(cu[-1]), 1, 1)), DT[dtype])
    kw = dict(opens=[int(0.4 * x) for x in ctx], cap=30.0) if open_part else {}
    for _ in range(4):
        out, lse, st = scored(L, desc, Hkv, table, ctx, cu, q, dtype, **kw)
        assert st == 0
        if _ == 0:
            check_scored(c, table, ctx, cu, q, out, lse, dtype, **kw)
            first = out, lse
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])


@pytest.mark.usefixtures("room")
def test_many_sequences_of_prompts(L):  # noqa: F811
    rng = np.random.default_rng(6)
    B = 1100
    new = rng.integers(0, 3, B)
    new[[3, 500, 1099]] = [70, 65, 130]
    ctx = [int(n + x) for n, x in zip(new, rng.integers(0, 40, B))]
    cu = np.concatenate([[0], np.cumsum(new)])
    c, t, desc, table = filled_cache(L, B, 16, 1, 64, ctx, rng)
    q = dev(rng.standard_normal((int(cu[-1]), 1, 64)), torch.bfloat16)
    out, lse, st = scored(L, desc, 1, table, ctx, cu, q, BF16)
    assert st == 0
    check_scored(c, table, ctx, cu, q, out, lse, BF16)


# ------------------------------------------------------------------ a prefix in common


def shared(L, desc, Hkv, ptable, P, table, ctx, cu, q, dtype, window=0, cap=0.0, slopes=None, T=None, scale=None,  # noqa: F811
           max_q=None, pad=2, lse=True, plen=None, stream=None):
    rows, Hq, D = q.shape
    B = len(ctx)
    T = rows if T is None else T
    n = np.diff(cu)
    max_q = max(1, int(n.max())) if max_q is None else max_q
    out = torch.full((rows + pad, Hq, D), -7.0, dtype=DT[dtype], device="cuda")
    ls = torch.full((rows + pad, Hq), -7.0, device="cuda") if lse else None
    sl = None if slopes is None else dev(np.asarray(slopes, np.float32))
    rules = L.AttnRules(cap, window, L.ptr(sl), None, None) if cap or window or slopes is not None else None
    wsb = L.e0_attn_shared_workspace_size(B, T, Hq, Hkv, D, max_q)
    ws = torch.full((wsb,), 255, dtype=torch.uint8, device="cuda")
    st = status()
    pl = dev(np.array([P], np.int32)) if plen is None else plen
    ptable = Tables.widen(ptable, desc.block_tokens)[0]
    L.e0_attn_shared(desc, dev(ptable), len(ptable), pl, dev(np.asarray(table, np.int32)),
                     np.asarray(table).shape[1], dev(np.asarray(ctx, np.int32)), dev(np.asarray(cu, np.int32)), B, T, max_q, q,
                     dtype, Hq * D, Hq, scale or 1 / np.sqrt(D), rules, out, Hq * D, ls, ws, wsb, st, stream=stream)
    return out, ls, L.e0_read_status(st)


def check_shared(c, ptable, P, table, ctx, cu, q, out, lse, dtype, window=0, cap=0.0, slopes=None, skip=()):
    T, Hq, D = q.shape
    scale = float(np.float32(1 / np.sqrt(D)))
    slopes = None if slopes is None else np.asarray(slopes, np.float32).astype(np.float64)
    got, gl, qv = f64(out), f64(lse) if lse is not None else None, f64(q)
    werr, quantum = weights_of(dtype, dtype != F32, dtype == BF16, c.vs)
    # the two results, normed, are joined in fp32: exponentials, a division, products, beside each one's own
    werr += 16 * EPS
    pk, pv = c.row(ptable, P)
    for b in range(len(ctx)):
        n = cu[b + 1] - cu[b]
        if n == 0 or b in skip:
            continue
        k, v = c.row(table[b], int(ctx[b]))
        k, v = np.concatenate([pk, k]), np.concatenate([pv, v])
        p, j = P + ctx[b] - n + np.arange(n), np.arange(len(k))
        seen = j[None, :] <= p[:, None]
        if window:
            seen = seen & (j[None, :] > p[:, None] - window)
        o, l, tol, ltol = rules_ref(qv[cu[b]:cu[b + 1]], k, v, scale, p, seen, cap, slopes, werr, quantum)
        tol = tol + 16 * EPS * np.abs(np.where(np.isneginf(l), 0, l))[:, :, None] * np.nanmax(np.abs(v))  # lse's own steps
        compare(got[cu[b]:cu[b + 1]], None if gl is None else gl[cu[b]:cu[b + 1]], (o, l, tol, ltol + 16 * EPS * (1 + np.abs(
            np.where(np.isneginf(l), 0, l)))), dtype, (b, n, ctx[b]))
    end = cu[-1]
    assert (got[end:] == -7).all() and (gl is None or (gl[end:] == -7).all())


def with_prefix(L, P, ctx, bs, Hkv, D, rng):  # noqa: F811
    """A pool that holds a prefix and the sequences; the prefix as the last row of the table."""
    c, t, desc, table = filled_cache(L, len(ctx) + 1, bs, Hkv, D, list(ctx) + [P], rng)
    front = table[-1, :max(1, -(-P // bs))]
    return c, t, desc, np.maximum(front, -1), table[:-1]


@pytest.mark.usefixtures("room")
@pytest.mark.parametrize("D", [128, 64, 256])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("P", [1, 16, 100, 128, 129, 700])
def test_shared_prefix(L, D, dtype, P):  # noqa: F811
    """Prefixes that end inside blocks and tiles, sequences of one token and more, some without queries, few rows and many."""
    rng = np.random.default_rng(D + P)
    for B, Hq, Hkv in ((5, 4, 2), (40, 8, 2)):
        new = rng.integers(0, 3, B)
        new[0] = 1
        ctx = [int(max(n, x)) for n, x in zip(new, rng.integers(0, 60, B))]
        cu = np.concatenate([[0], np.cumsum(new)])
        c, t, desc, front, table = with_prefix(L, P, ctx, 16, Hkv, D, rng)
        q = dev(rng.standard_normal((int(cu[-1]), Hq, D)) * 1.5, DT[dtype])
        out, lse, st = shared(L, desc, Hkv, front, P, table, ctx, cu, q, dtype)
        assert st == 0
        check_shared(c, front, P, table, ctx, cu, q, out, lse, dtype)


@pytest.mark.usefixtures("room")
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("window", [0, 1, 40, 600])
def test_shared_prefix_rules(L, dtype, window):  # noqa: F811
    """Windows that reach the prefix for some queries only, caps, biases by the distance over both parts."""
    rng = np.random.default_rng(window)
    B, Hq, Hkv, D, P = 30, 6, 2, 64, 333
    new = rng.integers(0, 4, B)
    new[1] = 3
    ctx = [int(max(n, x)) for n, x in zip(new, rng.integers(0, 100, B))]
    cu = np.concatenate([[0], np.cumsum(new)])
    c, t, desc, front, table = with_prefix(L, P, ctx, 32, Hkv, D, rng)
    q = dev(rng.standard_normal((int(cu[-1]), Hq, D)) * 2, DT[dtype])
    for kw in (dict(window=window), dict(window=window, cap=4.0), dict(window=window, slopes=ALIBI(Hq) * 0.1)):
        out, lse, st = shared(L, desc, Hkv, front, P, table, ctx, cu, q, dtype, **kw)
        assert st == 0
        check_shared(c, front, P, table, ctx, cu, q, out, lse, dtype, **kw)


@pytest.mark.usefixtures("room")
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_shared_long_prefix_and_equal_bits(L, dtype):  # noqa: F811
    rng = np.random.default_rng(7)
    B, Hq, Hkv, D, P = 24, 8, 1, 128, 9000
    ctx = [int(x) for x in rng.integers(1, 300, B)]
    cu = np.arange(B + 1)
    c, t, desc, front, table = with_prefix(L, P, ctx, 64, Hkv, D, rng)
    q = dev(rng.standard_normal((B, Hq, D)) * 2, DT[dtype])
    out, lse, st = shared(L, desc, Hkv, front, P, table, ctx, cu, q, dtype)
    assert st == 0
    check_shared(c, front, P, table, ctx, cu, q, out, lse, dtype)
    again, l2, _ = shared(L, desc, Hkv, front, P, table, ctx, cu, q, dtype)
    assert torch.equal(out, again) and torch.equal(lse, l2)


@pytest.mark.usefixtures("room")
def test_shared_prefix_of_nothing_and_bad_lengths(L):  # noqa: F811
    rng = np.random.default_rng(8)
    B, Hq, Hkv, D, P = 40, 4, 1, 64, 50
    ctx = [int(x) for x in rng.integers(1, 60, B)]
    cu = np.arange(B + 1)
    c, t, desc, front, table = with_prefix(L, P, ctx, 16, Hkv, D, rng)
    for dtype in (F16, F32):
        q = dev(rng.standard_normal((B, Hq, D)), DT[dtype])
        none, lse, st = shared(L, desc, Hkv, front, 0, table, ctx, cu, q, dtype)
        assert st == 0
        check_shared(c, front, 0, table, ctx, cu, q, none, lse, dtype)
        for bad in (-1, len(Tables.widen(front, 16)[0]) * 16 + 1, 2 ** 31 - 1):
            out, lse, st = shared(L, desc, Hkv, front, bad, table, ctx, cu, q, dtype)
            assert st == L.E0_ST_BAD_LENGTH and torch.equal(out, none)
        holes = front.copy()
        holes[1] = c.n
        out, lse, st = shared(L, desc, Hkv, holes, P, table, ctx, cu, q, dtype)
        assert st == L.E0_ST_BAD_BLOCK
        check_shared(c, np.where(holes >= c.n, -1, holes), P, table, ctx, cu, q, out, lse, dtype)
        # fewer rows than cu_q gives: the last sequence's rows are left
        out, lse, st = shared(L, desc, Hkv, front, P, table, ctx, cu, q, dtype, T=B - 1)
        assert st == L.E0_ST_BAD_LENGTH and (out[B - 1] == -7).all() and (lse[B - 1] == -7).all()
        check_shared(c, front, P, table, ctx[:-1], cu[:-1], q, out, lse, dtype)
        long = list(ctx)
        long[4] = 10 ** 8  # no tokens of its own are seen, the prefix is
        out, lse, st = shared(L, desc, Hkv, front, P, table, long, cu, q, dtype)
        assert st == L.E0_ST_BAD_LENGTH
        check_shared(c, front, P, table, ctx, cu, q, out, lse, dtype, skip=(4,))
        pk, pv = c.row(front, P)
        werr, quantum = weights_of(dtype, dtype != F32, False, c.vs)
        want = rules_ref(f64(q[4:5]), pk, pv, float(np.float32(D ** -0.5)), np.array([P]), np.ones((1, P), bool),
                         weight_err=werr + 32 * EPS, quantum=quantum)
        compare(f64(out[4:5]), None, want, dtype)


def test_a_captured_prefix_that_changes_and_two_streams(L):  # noqa: F811
    """The prefix's length and the lengths are read on the device; calls on two streams have a workspace each."""
    rng = np.random.default_rng(9)
    B, Hq, Hkv, D = 40, 4, 1, 128
    ctx = [int(x) for x in rng.integers(1, 60, B)]
    cu = np.arange(B + 1)
    c, t, desc, front, table = with_prefix(L, 400, ctx, 16, Hkv, D, rng)
    q = dev(rng.standard_normal((B, Hq, D)), torch.bfloat16)
    wsb = L.e0_attn_shared_workspace_size(B, B, Hq, Hkv, D, 1)
    bufs = [(torch.empty_like(q), torch.zeros(wsb, dtype=torch.uint8, device="cuda")) for _ in range(2)]
    plen, st = torch.tensor([400], dtype=torch.int32, device="cuda"), status()
    dt, dc, dcu, df = dev(table), dev(np.asarray(ctx, np.int32)), dev(np.asarray(cu, np.int32)), dev(front)

    def call(i, stream=None):
        L.e0_attn_shared(desc, df, len(front), plen, dt, table.shape[1], dc, dcu, B, B, 1, q, BF16, Hq * D, Hq, D ** -0.5, None,
                         bufs[i][0], Hq * D, None, bufs[i][1], wsb, st, stream=stream)

    call(0)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(0)
    for P in (400, 17, 0, 390):
        plen.fill_(P)
        g.replay()
        assert torch.equal(bufs[0][0], shared(L, desc, Hkv, front, P, table, ctx, cu, q, BF16)[0][:B])
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        call(0, a)
        call(1, b)
    torch.cuda.synchronize()
    assert torch.equal(bufs[0][0], bufs[1][0]) and L.e0_read_status(st) == 0
