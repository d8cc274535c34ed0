"""Rotation and sampling where their inputs go to the ends of their ranges, on the GPU against 64-bit references."""
import numpy as np
import pytest

from tests.test_layer_ops import BF16, DT, EPS, F16, F32, H, L, dev, f64, status  # noqa: F401
from tests.test_token_ops import NEAR, draw, rope_of, rope_ref, row_ref, rules_of

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("V", [2049, 4097, 8193, 16385])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_the_largest_of_many_short_rows(L, V, dtype):  # noqa: F811
    """Rows of a few thousand tokens, many of them, on clusters of two to eight blocks that come to their first meeting at
    different times: every block's largest logit counts."""
    T = 2500
    rng = np.random.default_rng(V)
    x = torch.randn((T, V), generator=torch.Generator(device="cuda").manual_seed(V), device="cuda").clamp_(-3, 3)
    at = rng.integers(0, V, T)
    at[:40] = np.arange(40) * V // 40
    x[torch.arange(T), torch.from_numpy(at).cuda()] = 9
    x = x.to(DT[dtype])
    for rules in (dict(top_k=np.ones(T)), dict(top_k=np.full(T, 2), top_p=np.full(T, 0.5))):
        got, logp, kept, st = draw(L, x, np.full(T, 0.4), dtype, rules_of(L, **rules))
        assert st == 0 and np.array_equal(got, at) and (kept == 1).all() and (logp == 0).all()


@pytest.mark.parametrize("V", [3, 200, 3000, 40000])
@pytest.mark.parametrize("temp", [1.0, 0.37, 60.0])
@pytest.mark.parametrize("rules", ["none", "top_k", "top_p"])
def test_the_probability_of_rare_tokens(L, V, temp, rules):  # noqa: F811
    """The last token, drawn by u = 1, has a weight of 2^-1 to 2^-43.9: ln p is its logit's, not that of the few bits that
    its weight has as a whole number of 2^-44."""
    rng = np.random.default_rng(V)
    y = np.concatenate([np.linspace(1, 43.9, 60), [30, 35.5, 40.5, 41.9, 42.9, 43.5]])
    T = len(y)
    temp = float(np.float32(temp))
    x = np.minimum(rng.standard_normal((T, V)), 2.9) * 2 * temp
    if rules != "none":  # few tokens that come before it, so that the first block ends the row
        x = x - 200 * temp
    x[:, 0] = 6 * temp
    x[:, V - 1] = 6 * temp - y * np.log(2) * temp
    x = dev(x, torch.float32)
    kw = dict(temperature=np.full(T, temp))
    if rules == "top_k":
        kw["top_k"] = np.full(T, 2)
    if rules == "top_p":
        kw["top_p"] = np.full(T, 1 - 2.0 ** -24)  # the last token is needed up to a weight of 2^-24
    got, logp, kept, st = draw(L, x, np.ones(T), F32, rules_of(L, **kw))
    assert st == 0
    xv = f64(x)
    for t in range(T):
        if rules == "top_p" and y[t] > 23:
            continue
        assert got[t] == V - 1, (t, y[t])
        d = (xv[t] - xv[t].max()) / temp
        w = np.exp(d if rules == "none" else d[[0, V - 1]])
        want = d[V - 1] - np.log(w.sum())
        # 4 steps of fp32, of which the test's own 64 bits take none; weights are whole numbers of 2^-44
        assert abs(logp[t] - want) <= 4 * EPS * abs(want) + V * 2.0 ** -44, (t, y[t], logp[t], want)


@pytest.mark.parametrize("temp", [2.0 ** 100, 1e31, 2.0 ** 116, 1e37, 1.3e38, 3.4e38])
@pytest.mark.parametrize("size", [1.0, 1e31, 3e35, 3e38])
def test_the_hottest_temperatures(L, temp, size):  # noqa: F811
    """Temperatures beyond 2^116 count as that: the weights keep their bits, and logits whose differences pass fp32's range
    are told apart."""
    rng = np.random.default_rng(int(np.log2(temp)))
    V, T = 3000, 60
    x = rng.uniform(-1, 1, (T, V)) * size
    x = dev(x.astype(np.float32))
    u = rng.random(T).astype(np.float32) * 0.999
    got, logp, kept, st = draw(L, x, u, F32, rules_of(L, temperature=np.full(T, temp), top_p=np.full(T, 0.7)))
    assert st == 0
    xv, sure = f64(x), 0
    for t in range(T):
        tok, want, n, near = row_ref(xv[t], float(u[t]), min(float(np.float32(temp)), 2.0 ** 116), 0, float(np.float32(0.7)))
        if near < NEAR + V * 2.0 ** -44:
            continue
        sure += 1
        assert got[t] == tok and kept[t] == n
        assert abs(logp[t] - want) <= 4 * EPS * abs(want) + V * 2.0 ** -44
    assert sure >= T - 3


@pytest.mark.parametrize("eps", [0.0, 2.0 ** -140, 1e-38, 2.0 ** -100, 1e-12])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D", [64, 80])
def test_norms_of_the_smallest_heads(L, eps, dtype, D):  # noqa: F811
    """Heads whose squares are below fp32's normal numbers, with an eps that does not hide them."""
    rng = np.random.default_rng(D)
    size = 2.0 ** np.array([0, -20, -49.5, -50, -51, -60, -66, -70, -75, -90, -110, -120, -130])  # (bf16 and fp32 alike)
    T = len(size)
    x = dev(rng.uniform(0.5, 1, (T, 3, D)) * rng.choice([-1, 1], (T, 3, D)) * size[:, None, None], DT[dtype])
    x[0, 0] = 0
    eps = float(np.float32(eps))
    freq = (1e4 ** (-np.arange(D // 2) / (D // 2))).astype(np.float32)
    pos = np.arange(T, dtype=np.int32)[None] * 100
    y, st = torch.full_like(x, 7.0), status()
    L.e0_qk_rope(x, dtype, 3 * D, T, 2, 1, rope_of(L, D, D, dev(freq), norm=True, eps=eps), dev(pos), T, y, 3 * D, st)
    assert L.e0_read_status(st) == 0
    want, tol = rope_ref(f64(x), 2, pos, freq, np.zeros(D // 2, int), D, False, True, None, None, eps if eps else 1e-300)
    got = f64(y)
    if not eps:  # 0 / 0
        assert np.isnan(got[0, 0]).all()
        got[0, 0] = want[0, 0] = tol[0, 0] = 0
    assert (np.abs(got - want) <= tol + H[dtype] * np.abs(want) * 1.0001 + 2.0 ** -126).all()
