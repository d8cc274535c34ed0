"""The bits that attention keeps of its weights, on the GPU against 64-bit references."""
import numpy as np
import pytest

from tests.test_attn_rules import Tables, rules_ref, scored, shared, with_prefix
from tests.test_layer_ops import BF16, DT, F16, L, dev, f64, filled_cache  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def between(got, want, tol, dtype):
    """Outputs are the rounded values of something within tol of the reference: rounding keeps the order."""
    lo, hi = (torch.from_numpy(want + s * tol).to(DT[dtype]).double().numpy() for s in (-1, 1))
    assert ((lo <= got) & (got <= hi)).all(), (np.mean((got < lo) | (hi < got)), np.abs(got - want).max(), tol.max())


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_weights_in_tiles(L, D, dtype):  # noqa: F811
    """Rows that see one to six positions, whose weights' roundings hardly cancel: 2^-21 of a weight at most.  Small
    scores, so that what they may be off by is less than that of weights of 11 bits."""
    rng = np.random.default_rng(D)
    n, Hq = 700, 8
    c, t, desc, table = filled_cache(L, 1, 32, 2, D, [n], rng)
    q = dev(rng.standard_normal((n, Hq, D)) * 0.05, DT[dtype])
    p = np.arange(n)
    first = np.maximum(p - rng.integers(0, 6, n), 0)
    Tables.room = True
    try:
        out, _, st = scored(L, desc, 2, table, [n], [0, n], q, dtype, first=first)
    finally:
        Tables.room = False
    assert st == 0
    k, v = c.row(table[0], n)
    seen = (p[None, :] <= p[:, None]) & (p[None, :] >= first[:, None])
    o, _, tol, _ = rules_ref(f64(q), k, v, float(np.float32(D ** -0.5)), p, seen, weight_err=2.0 ** -21,
                             quantum=2.0 ** -24 * 448 * float(np.nanmax(c.vs)))
    between(f64(out)[:n], o, tol, dtype)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_weights_behind_a_prefix(L, D, dtype):  # noqa: F811
    """Single tokens behind a prefix of a few positions, which goes through the tiles for its table's room."""
    rng = np.random.default_rng(D + 1)
    B, Hq, P = 80, 4, 5
    ctx = [1] * B
    cu = np.arange(B + 1)
    c, t, desc, front, table = with_prefix(L, P, ctx, 16, 1, D, rng)
    q = dev(rng.standard_normal((B, Hq, D)) * 0.05, DT[dtype])
    Tables.room = True
    try:
        out, lse, st = shared(L, desc, 1, front, P, table, ctx, cu, q, dtype)
    finally:
        Tables.room = False
    assert st == 0
    pk, pv = c.row(front, P)
    for b in range(B):
        k, v = c.row(table[b], 1)
        k, v = np.concatenate([pk, k]), np.concatenate([pv, v])
        # the parts' join: factors of an exponential, a division and products of the lses' own steps
        o, l, tol, _ = rules_ref(f64(q[b:b + 1]), k, v, float(np.float32(D ** -0.5)), np.array([P]), np.ones((1, P + 1), bool),
                                 weight_err=2.0 ** -21 + 32 * 2.0 ** -23, quantum=2.0 ** -24 * 448 * float(np.nanmax(c.vs)))
        between(f64(out[b:b + 1]), o, tol + 16 * 2.0 ** -23 * np.abs(l)[:, :, None] * np.abs(v).max(), dtype)
