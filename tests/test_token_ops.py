"""Rotation of queries and keys with their norms, and sampling, on the GPU against
64-bit references.

Tolerances: eps = 2^-23 is one step of fp32, H[dtype] half a step of an output's
type; each test says what it counts."""
import math

import numpy as np
import pytest

from tests.test_layer_ops import BF16, DT, EPS, F16, F32, H, TINY16, L, dev, f64, status  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

# ------------------------------------------------------------------ rotation


def rope_of(L, D, rot, freq, axis=None, wq=None, wk=None, axes=1, adjacent=False, norm=False, eps=1e-6):  # noqa: F811
    r = L.Rope(L.ptr(freq), L.ptr(axis), L.ptr(wq), L.ptr(wk), D, rot, axes,
               (L.E0_ROPE_ADJACENT if adjacent else 0) | (L.E0_QK_NORM if norm else 0), eps)
    r._keep = (freq, axis, wq, wk)
    return r


def rope_ref(x, Hq, pos, freq, axis, rot, adjacent, norm, wq, wk, eps):
    """x float64 [T][heads][D]; the result, and a bound on what fp32 may be off by (without the output's rounding)."""
    h = x.copy()
    if norm:
        h = h / np.sqrt((h ** 2).mean(2, keepdims=True) + eps)
        if wq is not None:
            h[:, :Hq] *= wq
        if wk is not None:
            h[:, Hq:] *= wk
    half = rot // 2
    i = np.arange(half)
    e0, e1 = (2 * i, 2 * i + 1) if adjacent else (i, i + half)
    turns = pos[axis].T.astype(object)  # whole numbers: angles modulo a turn exactly enough
    a = np.array([[float(math.fmod(int(turns[t, k]) * float(freq[k]), 2 * math.pi)) if abs(int(turns[t, k])) < 2 ** 24
                   else angle(int(turns[t, k]), float(freq[k])) for k in range(half)] for t in range(len(x))])
    a = a.reshape(len(x), half)
    c, s = np.cos(a)[:, None], np.sin(a)[:, None]
    y = h.copy()
    y[:, :, e0] = h[:, :, e0] * c - h[:, :, e1] * s
    y[:, :, e1] = h[:, :, e1] * c + h[:, :, e0] * s
    # a norm: 16 products in a lane and 4 additions across lanes, all of one sign, a mean, a root of 2 steps, two products;
    # the sine of 2 steps at an angle off by 2^-22; two products and their sum
    rel = ((20 / 2 + 6) * EPS if norm else 0.0) + 2.0 ** -22 + 4 * EPS
    mag = np.abs(h)
    big = mag.copy()
    big[:, :, e0] = big[:, :, e1] = mag[:, :, e0] + mag[:, :, e1]
    return y, rel * big


def angle(p, f):
    """p * f modulo a turn for whole p, f an fp32 number: by whole numbers, with 2 pi to 200 bits."""
    from fractions import Fraction
    tau = Fraction(2 * 0x3243F6A8885A308D313198A2E03707344A4093822299F31D008, 16 ** 50)
    v = Fraction(p) * Fraction(f)
    return float(v - (v // tau) * tau)


@pytest.mark.parametrize("T,Hq,Hk,D,rot", [(1, 1, 0, 64, 64), (8, 16, 2, 256, 64), (5, 0, 3, 128, 128), (3, 6, 2, 80, 80),
                                           (2, 5, 1, 96, 32), (4, 3, 3, 128, 64), (7, 2, 1, 66, 22), (1, 9, 9, 2, 2),
                                           (300, 4, 1, 64, 64), (2600, 3, 1, 128, 128), (3, 70, 1, 16, 16),
                                           (2, 3, 2, 48, 0), (2, 2, 2, 254, 254), (5, 33, 2, 192, 96)])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("adjacent,norm", [(False, True), (True, False), (True, True), (False, False)])
def test_rope(L, T, Hq, Hk, D, rot, dtype, adjacent, norm):  # noqa: F811
    rng = np.random.default_rng(T * 1009 + D + Hq)
    x = dev(rng.standard_normal((T, Hq + Hk, D)) * np.exp(rng.standard_normal((T, Hq + Hk, 1))), DT[dtype])
    axes = 1 + (T + D) % 3
    half = rot // 2
    freq = (1e4 ** (-np.arange(half) / max(half, 1))).astype(np.float32)
    axis = rng.integers(0, axes, half).astype(np.uint8)
    pos = rng.integers(0, 300000, (axes, T)).astype(np.int32)
    pos[1:] -= 1000
    wq = 1 + 0.3 * rng.standard_normal(D).astype(np.float32) if T % 2 else None
    wk = 1 + 0.3 * rng.standard_normal(D).astype(np.float32)
    r = rope_of(L, D, rot, dev(freq) if rot else None, dev(axis) if axes > 1 else None, None if wq is None else dev(wq),
                dev(wk), axes, adjacent, norm)
    y, st = torch.full_like(x, 7.0), status()
    ld = (Hq + Hk) * D
    L.e0_qk_rope(x, dtype, ld, T, Hq, Hk, r, dev(pos), T, y, ld, st)
    assert L.e0_read_status(st) == 0
    want, tol = rope_ref(f64(x), Hq, pos, freq, axis if axes > 1 else np.zeros(half, int), rot, adjacent, norm, wq, wk, 1e-6)
    assert (np.abs(f64(y) - want) <= tol + H[dtype] * np.abs(want) * 1.0001 + TINY16[dtype]).all()
    if not norm and rot < D:
        assert torch.equal(y[:, :, rot:], x[:, :, rot:])
    L.e0_qk_rope(x, dtype, ld, T, Hq, Hk, r, dev(pos), T, x, ld, st)  # in place
    assert torch.equal(x, y)


def test_rope_inside_longer_rows_and_unaligned(L):  # noqa: F811
    """The heads of a projection's rows, at strides and starts that vectors do and do not fit."""
    rng = np.random.default_rng(5)
    freq = (1e4 ** (-np.arange(32) / 32)).astype(np.float32)
    for dtype, ld, skip in ((F16, 5 * 64, 0), (F32, 400, 4), (BF16, 331, 1), (F32, 321, 3), (F16, 328, 8)):
        T, Hq, Hk, D = 6, 3, 1, 64
        big = dev(rng.standard_normal(T * ld + 16), DT[dtype])
        was = big.clone()
        pos = np.array([[0, 5, -1, 9000, 2, -1]], np.int32)
        r = rope_of(L, D, 64, dev(freq), norm=True)
        L.e0_qk_rope(big[skip:], dtype, ld, T, Hq, Hk, r, dev(pos), T, big[skip:], ld)
        rows, before = (torch.as_strided(t[skip:], (T, 4, D), (ld, D, 1)) for t in (big, was))
        want, tol = rope_ref(f64(before), Hq, np.maximum(pos, 0), freq, np.zeros(32, int), 64, False, True, None, None, 1e-6)
        at = pos[0] >= 0
        assert (np.abs(f64(rows) - want) <= tol + H[dtype] * np.abs(want) * 1.0001 + TINY16[dtype])[at].all()
        assert torch.equal(rows[torch.from_numpy(~at).cuda()], before[torch.from_numpy(~at).cuda()])
        mask = torch.ones_like(big, dtype=torch.bool)
        torch.as_strided(mask[skip:], (T, 4, D), (ld, D, 1)).fill_(False)
        assert torch.equal(big[mask], was[mask])  # what stands between the rows


def test_rope_far_positions_and_queries_and_keys_apart(L):  # noqa: F811
    rng = np.random.default_rng(6)
    T, D = 5, 128
    freq = np.concatenate([[6.5, -1.0, 3.0e5, 1.5e-9], 1e4 ** (-np.arange(60) / 60)]).astype(np.float32)
    pos = np.array([[0, 1, 2 ** 30, 2 ** 31 - 1, 999999937]], np.int32)
    x = dev(rng.standard_normal((T, 5, D)), torch.float32)
    want, tol = rope_ref(f64(x), 4, pos, freq, np.zeros(64, int), D, False, False, None, None, 1e-6)
    r = rope_of(L, D, D, dev(freq))
    y = torch.empty_like(x)
    L.e0_qk_rope(x, F32, 5 * D, T, 4, 1, r, dev(pos), T, y, 5 * D)
    assert (np.abs(f64(y) - want) <= tol + H[F32] * np.abs(want)).all()
    a, b = x.clone(), x.clone()  # queries and keys in calls of their own, keys by their address
    L.e0_qk_rope(a, F32, 5 * D, T, 4, 0, r, dev(pos), T, a, 5 * D)
    L.e0_qk_rope(b.view(-1)[4 * D:], F32, 5 * D, T, 0, 1, r, dev(pos), T, b.view(-1)[4 * D:], 5 * D)
    assert torch.equal(a[:, :4], y[:, :4]) and torch.equal(a[:, 4], x[:, 4])
    assert torch.equal(b[:, 4], y[:, 4]) and torch.equal(b[:, :4], x[:, :4])


def test_rope_zero_and_non_finite_heads(L):  # noqa: F811
    x = torch.randn((4, 2, 64), generator=torch.Generator().manual_seed(1)).cuda()
    x[0, 0] = 0
    x[1, 1, 5] = float("nan")
    x[2, 0, 0] = float("inf")
    x[3, 1] = 2.0 ** 70  # its sum of squares is beyond fp32
    freq = dev((1e4 ** (-np.arange(32) / 32)).astype(np.float32))
    pos = torch.arange(4, dtype=torch.int32, device="cuda")
    y, st = torch.empty_like(x), status()
    L.e0_qk_rope(x, F32, 128, 4, 1, 1, rope_of(L, 64, 64, freq, norm=True), pos, 4, y, 128, st)
    assert L.e0_read_status(st) == L.E0_ST_NONFINITE
    assert (y[0, 0] == 0).all() and y[1, 1].isnan().all() and y[2, 0, 0].isnan() and (y[3, 1] == 0).all()
    for t, h in ((0, 1), (1, 0), (2, 1), (3, 0)):
        assert y[t, h].isfinite().all() and (y[t, h] != 0).any()
    st.zero_()
    L.e0_qk_rope(x, F32, 128, 4, 1, 1, rope_of(L, 64, 64, freq), pos, 4, y, 128, st)  # without a norm: what the products give
    assert L.e0_read_status(st) == 0 and (y[1, 1].isnan().sum() == 2)


# ------------------------------------------------------------------ sampling


def rules_of(L, **rules):  # noqa: F811
    t = {k: dev(np.asarray(v, np.int32 if k == "top_k" else np.float32)) for k, v in rules.items()}
    r = L.Sampling(**{k: v.data_ptr() for k, v in t.items()})
    r._keep = t
    return r


def draw(L, x, u, dtype, rules, ld=None, with_outputs=True):  # noqa: F811
    T, V = x.shape
    tok = torch.full((T,), -7, dtype=torch.int32, device="cuda")
    logp, kept, st = torch.empty(T, device="cuda"), torch.full((T,), -7, dtype=torch.int32, device="cuda"), status()
    L.e0_sample(x, dtype, x.stride(0) if ld is None else ld, T, V, rules, dev(np.asarray(u, np.float32)), tok,
                logp if with_outputs else None, kept if with_outputs else None, st)
    return tok.cpu().numpy(), f64(logp), kept.cpu().numpy(), L.e0_read_status(st)


def row_ref(x, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """Token, ln p, number kept of one row (x float64), and how near the cuts and the draw are to their borders, as shares
    of the sums."""
    order = np.lexsort((np.arange(len(x)), -x))
    order = order[x[order] > -np.inf]
    w = np.exp((x[order] - x[order[0]]) / temperature)
    if top_k > 0:
        order, w = order[:top_k], w[:top_k]
    n, near = len(w), 1.0
    if top_p < 1:
        cum = np.cumsum(w)
        n = 1 + int(np.searchsorted(cum, max(top_p, 0) * cum[-1])) if top_p > 0 else 1
        near = min(near, np.abs(cum - max(top_p, 0) * cum[-1]).min() / cum[-1])
    if min_p > 0:
        least = min(float(min_p), 1.0)
        n = min(n, max(1, int((w >= least).sum())))
        off = np.abs(w[1:] - least) / least  # a weight is compared by itself: its own error counts, not a sum's
        near = min(near, off.min() if len(off) else 1.0)
    n = min(n, len(w))
    who = np.sort(order[:n])
    w = np.exp((x[who] - x[order[0]]) / temperature)
    cum = np.cumsum(w)
    at = min(int(np.searchsorted(cum, u * cum[-1], side="right")), n - 1)
    near = min(near, np.abs(cum[:-1] - u * cum[-1]).min() / cum[-1] if n > 1 else 1.0)
    return who[at], math.log(w[at] / cum[-1]), n, near


# weights are off by 2^-28 of themselves at most, so a running sum and the total that it is compared with by as much of
# themselves, 2^-27 of the total together: cuts and draws nearer than that to a border may go either way
NEAR = 2.0 ** -27


def check_draw(L, x, u, dtype, **rules):  # noqa: F811
    got, logp, kept, st = draw(L, x, u, dtype, rules_of(L, **rules) if rules else None)
    assert st == 0
    xv, sure = f64(x), 0
    for t in range(len(u)):
        of = {k: float(np.float32(v[t])) if k != "top_k" else int(v[t]) for k, v in rules.items()}
        w_tok, w_logp, w_n, near = row_ref(xv[t], float(np.float32(u[t])), **of)
        if near < NEAR + xv.shape[1] * 2.0 ** -44:
            continue
        sure += 1
        assert got[t] == w_tok and kept[t] == w_n, (t, got[t], w_tok, kept[t], w_n)
        # the ratio of two sums, a logarithm of 2 steps
        assert abs(logp[t] - w_logp) <= 6 * EPS * max(abs(w_logp), 0.0) + 4 * EPS * (1 if w_logp < -0.6 else 0) + 1e-9
    assert sure >= len(u) - 2 - len(u) // 50
    return got, kept


@pytest.mark.parametrize("V", [1, 2, 31, 100, 2048, 2049, 5000, 32000, 40001, 131071, 262144])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_draws_by_all_rules(L, V, dtype):  # noqa: F811
    rng = np.random.default_rng(V)
    T = 24
    x = rng.standard_normal((T, V)) * 2.5
    x[np.arange(T), rng.integers(0, V, T)] += 6
    x = dev(x, DT[dtype])
    u = rng.random(T).astype(np.float32) * 0.999
    check_draw(L, x, u, dtype)
    check_draw(L, x, u, dtype, temperature=0.3 + rng.random(T))
    check_draw(L, x, u, dtype, top_k=rng.integers(-1, 60, T))
    check_draw(L, x, u, dtype, top_p=rng.random(T) * 1.1)
    check_draw(L, x, u, dtype, min_p=rng.random(T) * 0.2 - 0.02)
    check_draw(L, x, u, dtype, top_k=rng.integers(1, max(2, V), T), top_p=0.3 + 0.69 * rng.random(T))
    got, kept = check_draw(L, x, u, dtype, temperature=0.5 + rng.random(T), top_k=rng.integers(1, max(2, V), T),
                           top_p=0.5 + 0.5 * rng.random(T), min_p=rng.random(T) ** 3 * 0.1)
    assert (got >= 0).all() and (got < V).all() and (kept >= 1).all()


@pytest.mark.parametrize("V", [3000, 30000, 131072])
def test_many_equal_logits(L, V):  # noqa: F811
    """Ties go to the lower token: among a few values, and where a bin holds many different ones."""
    rng = np.random.default_rng(V + 1)
    T = 12
    u = rng.random(T).astype(np.float32)
    k = rng.integers(1, V, T)
    coarse = dev(np.round(rng.standard_normal((T, V)) * 2) / 2, torch.float32)
    check_draw(L, coarse, u, F32, top_k=k)
    check_draw(L, coarse, u, F32, top_p=0.05 + 0.9 * rng.random(T))
    check_draw(L, coarse, u, F32, top_k=k, top_p=0.3 + 0.6 * rng.random(T), min_p=np.full(T, 1e-3))
    same = torch.full((T, V), -3.25, device="cuda")
    got, kept = check_draw(L, same, u, F32, top_k=k)
    assert np.array_equal(kept, k) and (got < k).all()
    got, _, kept, _ = draw(L, same, u, F32, rules_of(L, top_p=np.full(T, 0.5)))  # exactly half of them
    assert np.array_equal(kept, np.full(T, -(-V // 2)))
    # logits so near one another that one bin has them all, each a number of its own
    close = torch.from_numpy((1.0 + np.stack([rng.permutation(V) for _ in range(T)]) * 2.0 ** -23).astype(np.float32)).cuda()
    check_draw(L, close, u, F32, top_k=k)
    got, kept, st = draw(L, close, u, F32, rules_of(L, top_p=np.full(T, 0.25)))[0::2] + (0,)
    assert (np.abs(kept - V / 4) <= V * 0.01 + 1).all()


def test_far_logits_and_masked_tokens(L):  # noqa: F811
    rng = np.random.default_rng(3)
    V, T = 9001, 10
    x = rng.standard_normal((T, V)).astype(np.float32) * 200
    x[:, rng.permutation(V)[:4000]] = -np.inf
    x[1] = -np.inf
    x[1, 77] = -5e30
    x[2, :] = np.where(np.arange(V) % 2, 3.0e38, -3.0e38)
    x[3, 5:] = -np.inf
    xd = dev(x)
    u = rng.random(T).astype(np.float32)
    got, kept = check_draw(L, xd, u, F32, top_k=np.full(T, 3000))
    assert got[1] == 77 and kept[1] == 1 and kept[3] == np.isfinite(x[3]).sum()
    check_draw(L, xd, u, F32, top_p=np.full(T, 0.9))
    check_draw(L, xd, u, F32, temperature=np.full(T, 50.0))
    got, _ = check_draw(L, xd, u, F32)
    assert np.isfinite(x[np.arange(T), got]).all()


def test_greedy_and_edges_of_the_rules(L):  # noqa: F811
    rng = np.random.default_rng(4)
    V, T = 5000, 8
    x = np.round(rng.standard_normal((T, V)) * 4).astype(np.float32)  # ties for the largest
    x[0, 17] = x[0, 3000] = 50
    xd = dev(x)
    u = np.array([0, 1, 0.5, 0.25, 1, 0, 0.999, 1e-7], np.float32)
    best = x.argmax(1)
    for rules in (dict(temperature=np.zeros(T)), dict(top_k=np.ones(T)), dict(top_p=np.zeros(T)),
                  dict(temperature=np.full(T, 1e-31))):
        got, logp, kept, st = draw(L, xd, u, F32, rules_of(L, **rules))
        assert st == 0 and np.array_equal(got, best) and (logp == 0).all() and (kept == 1).all()
    got, logp, kept, st = draw(L, xd, u, F32, rules_of(L, min_p=np.full(T, 7.0)))  # 1: all that are as likely as the first
    assert st == 0 and np.array_equal(kept, (x == x.max(1, keepdims=True)).sum(1)) and got[0] == 17
    got, logp, kept, st = draw(L, xd, u, F32, None)
    assert got[5] == 0 and got[1] == V - 1 and (kept == V).all()  # u = 0: the first; u = 1: the last
    assert draw(L, xd, u, F32, None, with_outputs=False)[0].tolist() == got.tolist()


def test_rows_that_cannot_be_drawn_from(L):  # noqa: F811
    V = 6000
    x = torch.randn((9, V), generator=torch.Generator().manual_seed(2)).cuda()
    x[0, 5999] = float("nan")
    x[1, 3] = float("inf")
    x[2] = -float("inf")
    u = np.array([.5, .5, .5, -0.1, 1.5, np.nan, .5, .5, .5], np.float32)
    temp = np.ones(9, np.float32)
    temp[6], temp[7] = -1, np.nan
    got, logp, kept, st = draw(L, x, u, F32, rules_of(L, temperature=temp, top_p=np.full(9, 0.8)))
    assert st == L.E0_ST_NONFINITE
    assert (got[:8] == -1).all() and (kept[:8] == 0).all() and np.isneginf(logp[:8]).all() and got[8] >= 0
    for bad in (dict(top_p=np.full(9, np.nan)), dict(min_p=np.full(9, np.nan)), dict(temperature=np.full(9, np.inf))):
        got, _, kept, st = draw(L, x, u, F32, rules_of(L, **bad))
        assert st == L.E0_ST_NONFINITE and (got == -1).all()


def test_strided_and_unaligned_rows_and_equal_calls(L):  # noqa: F811
    rng = np.random.default_rng(9)
    for dtype, V, ld, skip in ((F32, 5003, 5010, 3), (F16, 70001, 70003, 1), (BF16, 4096, 4096, 5), (F32, 2048, 2052, 0)):
        T = 7
        buf = dev(rng.standard_normal(T * ld + 16) * 3, DT[dtype])
        x = torch.as_strided(buf, (T, V), (ld, 1), skip)
        u = rng.random(T).astype(np.float32)
        rules = dict(top_k=np.full(T, 500), top_p=np.full(T, 0.9))
        a = check_draw(L, x, u, dtype, **rules)
        b = check_draw(L, x, u, dtype, **rules)
        assert np.array_equal(a[0], b[0])
    L.e0_sample(None, F32, 8, 0, 8, None, None, None)


def test_draws_follow_the_weights(L):  # noqa: F811
    """Evenly spread u give every token its share: the definition, counted."""
    V, T = 50, 20000
    x = torch.randn((1, V), generator=torch.Generator().manual_seed(5)).cuda().repeat(T, 1)
    u = (np.arange(T) + 0.5) / T
    got = draw(L, x, u, F32, rules_of(L, temperature=np.full(T, 0.7)))[0]
    p = np.exp(f64(x)[0] / float(np.float32(0.7)))
    p /= p.sum()
    assert (np.abs(np.bincount(got, minlength=V) - p * T) <= 1.01).all() and (np.diff(got) >= 0).all()


def test_a_captured_draw_and_another_stream(L):  # noqa: F811
    V, T = 33000, 5
    g = torch.Generator(device="cuda").manual_seed(3)
    x, u = torch.randn((T, V), generator=g, device="cuda"), torch.rand(T, generator=g, device="cuda")
    rules = rules_of(L, top_k=np.full(T, 40), top_p=np.full(T, 0.9))
    tok, st = torch.empty(T, dtype=torch.int32, device="cuda"), status()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    L.e0_sample(x, F32, V, T, V, rules, u, tok, None, None, st, stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.e0_sample(x, F32, V, T, V, rules, u, tok, None, None, st)
    for _ in range(5):
        x.copy_(torch.randn((T, V), generator=g, device="cuda"))
        u.copy_(torch.rand(T, generator=g, device="cuda"))
        graph.replay()
        assert tok.tolist() == draw(L, x, u.cpu().numpy(), F32, rules)[0].tolist()
