"""The operators around the MoE block on the GPU against 64-bit references:
residual norm with e4m3 output, int4 linear, paged 8-bit KV cache, attention.

Tolerances: eps = 2^-23 is one step of fp32, H[dtype] half a step of an output's
type; each test says what it counts."""
import os

import numpy as np
import pytest

from tests import layer_ref as R

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

EPS = 2.0 ** -23
F32, F16, BF16, E4M3 = 0, 1, 2, 3
H = {F32: 2.0 ** -24, F16: 2.0 ** -11, BF16: 2.0 ** -8}
DT = {F32: torch.float32, F16: torch.float16, BF16: torch.bfloat16}
TINY16 = {F32: 0.0, F16: 2.0 ** -25, BF16: 0.0}  # half a step of fp16's subnormals


@pytest.fixture(scope="module")
def L():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from int4_gathered_expert_gb300 import build, lib
    if not os.path.exists(lib.LIB_PATH):
        build.build()
    lib.load()
    return lib


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).cuda()


def f64(t):
    return t.double().cpu().numpy()


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ norm


@pytest.mark.parametrize("T,H_", [(1, 64), (8, 2048), (3, 1536), (5, 100), (2, 1), (2, 63), (7, 65), (3, 4104), (1300, 512),
                                  (1300, 136), (1400, 1544),
                                  (2, 8200), (1, 16384), (300, 256), (2, 5001)])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("with_d,with_w", [(True, True), (False, False)])
def test_norm(L, T, H_, dtype, with_d, with_w):
    rng = np.random.default_rng(T * 10007 + H_)
    r = dev(rng.standard_normal((T, H_)), DT[dtype])
    d = dev(rng.standard_normal((T, H_)), DT[dtype]) if with_d else None
    w = dev(1 + 0.3 * rng.standard_normal(H_), torch.float32) if with_w else None
    ro, h = torch.empty_like(r), torch.empty_like(r)
    ng = -(-H_ // 64)
    q = torch.empty((T, H_), dtype=torch.uint8, device="cuda")
    qs = torch.empty((T, ng), device="cuda")
    st = status()
    L.e0_rmsnorm_q8(r, d, w, T, H_, dtype, 1e-6, H_, H_, ro, h, q, qs, st)
    assert L.e0_read_status(st) == 0
    s = (r.float() + d.float()).to(DT[dtype]) if with_d else r  # one fp32 addition, one rounding
    assert torch.equal(ro, s)
    x = f64(s)
    want = x / np.sqrt((x ** 2).mean(1, keepdims=True) + 1e-6)
    if with_w:
        want = want * f64(w)
    # a sum of squares in fp32: at most 8 * 4 products in a thread, 5 + 16 additions across the block, all of one
    # sign; then the mean, the root, the division and two products
    rel = (32 + 21) / 2 * EPS + 5 * EPS
    assert (np.abs(f64(h) - want) <= (rel + H[dtype]) * np.abs(want) * 1.0001 + TINY16[dtype]).all()
    pad = np.zeros((T, ng * 64))
    pad[:, :H_] = want
    m = np.abs(pad.reshape(T, ng, 64)).max(2) / 448
    assert (np.abs(f64(qs) - m) <= (rel + EPS) * m).all()
    scaled = (pad.reshape(T, ng, 64) / np.where(m > 0, m, 1)[:, :, None]).reshape(T, ng * 64)[:, :H_]
    code = q.cpu().numpy()
    sure = R.border_distance(scaled) > 2 * rel + 4 * EPS  # away from a rounding border the code is decided
    assert np.array_equal(code[sure], R.encode(scaled)[sure])
    step = np.maximum(np.abs(scaled) * 2.0 ** -4, 2.0 ** -10)
    assert (np.abs(R.decode(code) - scaled) <= step * (1 + 1e-5)).all()


def test_norm_in_place_strided_and_unaligned(L):
    rng = np.random.default_rng(3)
    for dtype, H_, ld, skip in ((F32, 256, 256, 0), (BF16, 256, 320, 8), (F16, 130, 131, 1), (F32, 64, 67, 3)):
        big = dev(rng.standard_normal((6, ld + 16)), DT[dtype])
        dd = dev(rng.standard_normal((6, ld + 16)), DT[dtype])
        r, d = big.view(-1)[skip:], dd.view(-1)[skip:]
        rows = torch.as_strided(r, (4, H_), (ld, 1)).float() + torch.as_strided(d, (4, H_), (ld, 1)).float()
        want = rows.to(DT[dtype])
        ro = torch.empty((4, H_), dtype=DT[dtype], device="cuda")
        L.e0_rmsnorm_q8(r, d, None, 4, H_, dtype, 1e-6, ld, ld, ro, None, None, None)
        assert torch.equal(ro, want)
    r = dev(rng.standard_normal((5, 192)), torch.float32)
    d = dev(rng.standard_normal((5, 192)), torch.float32)
    for over in ("r", "d"):
        a, b = r.clone(), d.clone()
        h = torch.empty_like(r)
        L.e0_rmsnorm_q8(a, b, None, 5, 192, F32, 1e-6, 192, 192, a if over == "r" else b, h, None, None)
        assert torch.equal(a if over == "r" else b, r + d)
        s = r + d
        assert torch.allclose(h, s / torch.sqrt((s * s).mean(1, keepdim=True) + 1e-6), rtol=1e-5, atol=1e-6)


def test_norm_zero_tiny_and_non_finite_rows(L):
    r = torch.randn((5, 128), generator=torch.Generator().manual_seed(1)).cuda()
    r[0] = 0
    r[1, :64] = 0
    r[2] *= 1e-30
    r[3, 70] = float("nan")
    r[4, 3] = float("inf")
    h, q = torch.empty_like(r), torch.empty((5, 128), dtype=torch.uint8, device="cuda")
    qs, st = torch.empty((5, 2), device="cuda"), status()
    L.e0_rmsnorm_q8(r, None, None, 5, 128, F32, 1e-6, 128, 0, None, h, q, qs, st)
    assert L.e0_read_status(st) == L.E0_ST_NONFINITE
    assert (h[0] == 0).all() and (q[0] == 0).all() and (qs[0] == 0).all()
    assert qs[1, 0] == 0 and qs[1, 1] > 0 and (q[1, :64] == 0).all()
    assert torch.allclose(h[2], r[2] * 1e3, rtol=1e-5) and (qs[2] > 0).all()
    assert h[3].isnan().all() and (q[3] == 0).all() and (qs[3] == 0).all()
    # an infinity leaves a root of infinity: its own place is NaN, all others 0
    assert h[4, 3].isnan() and (h[4, 4:] == 0).all() and (qs[4] == 0).all() and (q[4] == 0).all()
    L.e0_rmsnorm_q8(r, None, None, 0, 128, F32, 1e-6, 128, 0, None, h, None, None)


@pytest.mark.parametrize("T,H_", [(3, 256), (3, 65), (1300, 64), (2, 8200)])
def test_norm_says_where_the_sum_of_squares_overflows(L, T, H_):
    """2^63.5 squared, twice, is 2^128; a row of 2^60 is still a row."""
    r = torch.zeros((T, H_), device="cuda")
    r[:, 0], r[:, 1] = 2.0 ** 60, -2.0 ** 60
    h, q = torch.empty_like(r), torch.empty((T, H_), dtype=torch.uint8, device="cuda")
    qs, st = torch.empty((T, -(-H_ // 64)), device="cuda"), status()
    L.e0_rmsnorm_q8(r, None, None, T, H_, F32, 1e-6, H_, 0, None, h, q, qs, st)
    assert L.e0_read_status(st) == 0
    assert torch.allclose(h[:, 0], torch.full((T,), (H_ / 2) ** 0.5, device="cuda"), rtol=1e-6) and (q[:, 0] == 0x7E).all()
    r[T - 1, :3] = 2.0 ** 64
    for outs in ((h, None, None), (None, q, qs), (h, q, qs)):
        st.zero_()
        L.e0_rmsnorm_q8(r, None, None, T, H_, F32, 1e-6, H_, 0, None, *outs, st)
        assert L.e0_read_status(st) == L.E0_ST_NONFINITE
    assert (h[T - 1] == 0).all() and (q[T - 1] == 0).all() and (qs[T - 1] == 0).all()
    assert (h[:T - 1, 0] > 1).all() and (q[:T - 1, 0] == 0x7E).all()
    st.zero_()
    L.e0_rmsnorm_q8(r, None, None, T, H_, F32, 1e-6, H_, 0, h, None, None, None, st)  # no norm is asked for
    assert L.e0_read_status(st) == 0 and torch.equal(h, r)


@pytest.mark.parametrize("T,H_", [(4, 128), (3, 65), (1300, 64), (2, 4104)])
def test_norm_up_to_the_largest_numbers(L, T, H_):
    """Weights that bring h close to fp32's largest value: codes and scales as at any size."""
    rng = np.random.default_rng(H_)
    v = rng.uniform(-1, 1, (T, H_))
    v[:, ::64] = 1  # every group's maximum
    r = dev(v, torch.float32)
    x = f64(r)
    root = np.sqrt((x ** 2).mean(1, keepdims=True) + 1e-6)
    w = dev(np.full(H_, 3.3e38 * root.min()), torch.float32)
    want = x / root * f64(w)
    assert 3e38 < np.abs(want).max() < 3.4e38
    h, q = torch.empty_like(r), torch.empty((T, H_), dtype=torch.uint8, device="cuda")
    ng = -(-H_ // 64)
    qs, st = torch.empty((T, ng), device="cuda"), status()
    L.e0_rmsnorm_q8(r, None, w, T, H_, F32, 1e-6, H_, 0, None, h, q, qs, st)
    assert L.e0_read_status(st) == 0
    rel = (32 + 21) / 2 * EPS + 5 * EPS  # as in test_norm
    assert (np.abs(f64(h) - want) <= (rel + H[F32]) * np.abs(want) * 1.0001).all()
    pad = np.zeros((T, ng * 64))
    pad[:, :H_] = want
    m = np.abs(pad.reshape(T, ng, 64)).max(2) / 448
    assert (np.abs(f64(qs) - m) <= (rel + EPS) * m).all()
    scaled = (pad.reshape(T, ng, 64) / m[:, :, None]).reshape(T, ng * 64)[:, :H_]
    code = q.cpu().numpy()
    sure = R.border_distance(scaled) > 2 * rel + 4 * EPS
    assert sure.mean() > 0.99 and np.array_equal(code[sure], R.encode(scaled)[sure])
    step = np.maximum(np.abs(scaled) * 2.0 ** -4, 2.0 ** -10)
    assert (np.abs(R.decode(code) - scaled) <= step * (1 + 1e-5)).all()


# ------------------------------------------------------------------ linear


def make_linear(L, N, K, rng, q=None):
    q = rng.integers(0, 16, (N, K)).astype(np.uint8) if q is None else q
    scale = np.abs(rng.normal(0, 0.02, (N, K // 64))).astype(np.float16)
    bias = (-8 * scale + rng.normal(0, 1e-3, scale.shape)).astype(np.float16)
    codes = dev(q[:, 0::2] | (q[:, 1::2] << 4))
    s, b = dev(scale), dev(bias)
    w = torch.empty(L.e0_linear_bytes(N, K), dtype=torch.uint8, device="cuda")
    L.e0_pack_linear(L.QTensor(codes.data_ptr(), s.data_ptr(), b.data_ptr()), N, K, w)
    return w, q.astype(np.float64), scale.astype(np.float64), bias.astype(np.float64), (codes, s, b)


def linear_ref(q, s, b, x):
    """y and the magnitude sum that its rounding goes by."""
    N, K = q.shape
    G = K // 64
    y, mag = np.zeros((len(x), N)), np.zeros((len(x), N))
    for g in range(G):
        xx = x[:, g * 64:(g + 1) * 64]
        qq = q[:, g * 64:(g + 1) * 64]
        y += (xx @ qq.T) * s[:, g] + xx.sum(1, keepdims=True) * b[:, g]
        mag += (np.abs(xx) @ qq.T) * s[:, g] + np.abs(xx).sum(1, keepdims=True) * np.abs(b[:, g])
    return y, mag


def make_x(T, K, xt, rng, ld=None, skip=0):
    ld = K if ld is None else ld
    v = rng.standard_normal((T, ld))
    if xt == E4M3:
        code = R.encode(v * 100).astype(np.uint8)
        xs = np.abs(rng.normal(0.01, 0.003, (T, K // 64))).astype(np.float32)
        flat = torch.zeros(skip + T * ld, dtype=torch.uint8, device="cuda")
        flat[skip:] = dev(code).view(-1)
        x = R.decode(code)[:, :K].reshape(T, K // 64, 64) * xs[:, :, None].astype(np.float64)
        return flat[skip:], dev(xs), x.reshape(T, K)
    flat = torch.zeros(skip + T * ld, dtype=DT[xt], device="cuda")
    flat[skip:] = dev(v, DT[xt]).view(-1)
    return flat[skip:], None, f64(flat[skip:].view(T, ld))[:, :K]


@pytest.mark.parametrize("T,N,K", [(1, 64, 64), (1, 1, 128), (3, 17, 192), (8, 2048, 2048), (9, 100, 512),
                                   (2, 1000, 6400), (33, 130, 1024), (64, 48, 320), (1, 20000, 64), (5, 19500, 128)])
@pytest.mark.parametrize("xt", [F32, F16, BF16, E4M3])
def test_linear(L, T, N, K, xt):
    rng = np.random.default_rng(N * 31 + K)
    w, q, s, b, keep = make_linear(L, N, K, rng)
    x, xs, xv = make_x(T, K, xt, rng)
    want, mag = linear_ref(q, s, b, xv)
    yt = {F32: F32, F16: F16, BF16: BF16, E4M3: F32}[xt]
    for add in (False, True):
        y = torch.full((T, N), float("nan"), dtype=DT[yt], device="cuda")
        a = dev(rng.standard_normal((T, N)), DT[yt]) if add else None
        L.e0_linear_forward(w, N, K, x, xt, K, xs, T, a, N, y, yt, N)
        ref = want + (f64(a) if add else 0)
        # 64 products of a group and the sum before each, K/64 groups, 8 warps, 8 blocks, 3 scalings
        tol = (64 + 4 + K / 64 + 8 + 8 + 3) * EPS * mag + (H[yt] + EPS) * np.abs(ref) * 1.0001 + TINY16[yt]
        assert (np.abs(f64(y) - ref) <= tol).all()


@pytest.mark.parametrize("T,N,K", [(16, 10240, 2560), (40, 7168, 2048), (20, 11008, 1536), (64, 2500, 2048),
                                   (16, 300, 640), (17, 300, 640), (48, 300, 640), (49, 300, 640), (12, 40000, 512), (15, 1000, 4160),
                                   (1, 5120, 5120), (8, 4500, 7168), (2, 12500, 3200)])
@pytest.mark.parametrize("xt", [F32, F16, E4M3])
def test_linear_clusters(L, T, N, K, xt):
    """K split over numbers of blocks that divide neither its groups nor the rows that they finish."""
    rng = np.random.default_rng(N + K)
    w, q, s, b, keep = make_linear(L, N, K, rng)
    x, xs, xv = make_x(T, K, xt, rng)
    want, mag = linear_ref(q, s, b, xv)
    y = torch.full((T + 1, N), -7.0, device="cuda")
    L.e0_linear_forward(w, N, K, x, xt, K, xs, T, None, 0, y, F32, N)
    # as in test_linear
    tol = (64 + 4 + K / 64 + 8 + 8 + 3) * EPS * mag + 2 * EPS * np.abs(want) * 1.0001
    assert (np.abs(f64(y)[:T] - want) <= tol).all() and (y[T] == -7).all()
    z = torch.empty((T, N), device="cuda")
    L.e0_linear_forward(w, N, K, x, xt, K, xs, T, None, 0, z, F32, N)
    assert torch.equal(z, y[:T])


@pytest.mark.parametrize("xt", [F32, F16, BF16, E4M3])
def test_linear_strides_alignment_and_untouched_rows(L, xt):
    rng = np.random.default_rng(9)
    T, N, K = 5, 70, 256
    w, q, s, b, keep = make_linear(L, N, K, rng)
    for ld, skip in ((K, 0), (K + 64, 0), (K + 3, 1)):
        x, xs, xv = make_x(T, K, xt, rng, ld, skip)
        y = torch.full((T + 2, N + 5), -7.0, dtype=torch.bfloat16, device="cuda")
        L.e0_linear_forward(w, N, K, x, xt, ld, xs, T, None, 0, y, BF16, N + 5)
        want, mag = linear_ref(q, s, b, xv)
        got = f64(y)
        assert (np.abs(got[:T, :N] - want) <= 100 * EPS * mag + H[BF16] * np.abs(want) * 1.01).all()
        assert (got[:T, N:] == -7).all() and (got[T:] == -7).all()
    # y over add; equal calls give equal bits; a row does not depend on the others in its tile
    x, xs, xv = make_x(T, K, xt, rng)
    y0 = dev(rng.standard_normal((T, N)), torch.float32)
    ya, yb = y0.clone(), y0.clone()
    L.e0_linear_forward(w, N, K, x, xt, K, xs, T, ya, N, ya, F32, N)
    L.e0_linear_forward(w, N, K, x, xt, K, xs, T, y0, N, yb, F32, N)
    assert torch.equal(ya, yb)


@pytest.mark.parametrize("xt", [F32, F16, BF16])
def test_linear_extreme_and_non_finite_inputs(L, xt):
    rng = np.random.default_rng(4)
    T, N, K = 4, 32, 128
    w, q, s, b, keep = make_linear(L, N, K, rng)
    v = rng.standard_normal((T, K))
    big = {F32: 1e30, F16: 3e4, BF16: 1e30}[xt]
    v[0] *= big / 8
    v[1] *= {F32: 1e-30, F16: 1e-6, BF16: 1e-30}[xt]
    x = dev(v, DT[xt])
    x[2, 5], x[3, 64] = float("nan"), float("inf")
    y = torch.empty((T, N), device="cuda")
    L.e0_linear_forward(w, N, K, x, xt, K, None, T, None, 0, y, F32, N)
    xv = f64(x)[:2]
    want, mag = linear_ref(q, s, b, xv)
    assert (np.abs(f64(y)[:2] - want) <= 100 * EPS * mag).all()
    assert not torch.isfinite(y[2:]).any()


@pytest.mark.parametrize("T", [5, 12, 33, 70])
@pytest.mark.parametrize("xt", [F32, F16, BF16, E4M3])
@pytest.mark.parametrize("more,skip", [(0, 0), (64, 0), (3, 1)])
def test_linear_rows_of_any_kind(L, T, xt, more, skip):
    """Strided and unaligned rows for few and for many of them, y over add in rows longer than N, K split over a cluster;
    a row's values, a NaN or an infinity among them, do not reach the other rows."""
    rng = np.random.default_rng(T + more)
    N, K = 300, 1344
    w, q, s, b, keep = make_linear(L, N, K, rng)
    ld = K + more
    x, xs, xv = make_x(T, K, xt, rng, ld, skip)
    a = dev(rng.standard_normal((T + 2, N + 5)), torch.float32)
    y = a.clone()
    L.e0_linear_forward(w, N, K, x, xt, ld, xs, T, y, N + 5, y, F32, N + 5)
    want, mag = linear_ref(q, s, b, xv)
    want = want + f64(a)[:T, :N]
    # as in test_linear
    tol = (64 + 4 + K / 64 + 8 + 8 + 3) * EPS * mag + 2 * EPS * np.abs(want) * 1.0001
    assert (np.abs(f64(y)[:T, :N] - want) <= tol).all()
    assert torch.equal(y[:T, N:], a[:T, N:]) and torch.equal(y[T:], a[T:])
    rows = torch.as_strided(x, (T, K), (ld, 1))
    for row, value in ((0, 2.0), (T - 1, float("nan")), (T // 2, float("inf"))):
        kept = rows[row].clone()
        if xt != E4M3:
            rows[row, 70] = value
        else:
            rows[row, 70] = 0x40 if value == 2 else 0x7F  # 2 and NaN; there is no infinity
        z = a.clone()
        L.e0_linear_forward(w, N, K, x, xt, ld, xs, T, z, N + 5, z, F32, N + 5)
        others = torch.arange(T + 2, device="cuda") != row
        assert torch.equal(z[others], y[others])
        assert (torch.isfinite(z[row, :N]).all() and not torch.equal(z[row], y[row])) if value == 2 else \
            not torch.isfinite(z[row, :N]).any()
        rows[row] = kept


@pytest.mark.parametrize("T,N,K", [(1, 40, 128), (8, 300, 4160), (12, 300, 640), (40, 130, 4096)])
@pytest.mark.parametrize("xt", [F32, BF16])
@pytest.mark.parametrize("add", [False, True])
def test_linear_large_values_of_one_sign(L, T, N, K, xt, add):
    """Values near fp32's end whose sums with the codes pass it, and y does not."""
    rng = np.random.default_rng(N + K)
    q = rng.integers(0, 16, (N, K)).astype(np.uint8)
    scale = rng.uniform(1e-4, 2e-4, (N, K // 64)).astype(np.float16)
    bias = (-7.5 * scale).astype(np.float16)
    codes, s, b = dev(q[:, 0::2] | (q[:, 1::2] << 4)), dev(scale), dev(bias)
    w = torch.empty(L.e0_linear_bytes(N, K), dtype=torch.uint8, device="cuda")
    L.e0_pack_linear(L.QTensor(codes.data_ptr(), s.data_ptr(), b.data_ptr()), N, K, w)
    x = dev(rng.uniform(1e38, 3.3e38, (T, K)), DT[xt])
    a = dev(rng.uniform(-1e36, 1e36, (T, N)), torch.float32) if add else None
    y = torch.empty((T, N), device="cuda")
    L.e0_linear_forward(w, N, K, x, xt, K, None, T, a, N, y, F32, N)
    want, mag = linear_ref(q.astype(np.float64), scale.astype(np.float64), bias.astype(np.float64), f64(x))
    want = want + (f64(a) if add else 0)
    assert np.isfinite(want.astype(np.float32)).all()
    # as in test_linear; with codes as 16 + code a weight's part of the sums is up to 31 scales, and so is the bias's
    big = np.abs(f64(x)).reshape(T, K // 64, 64).sum(2) @ (31 * scale.astype(np.float64).T)
    tol = (64 + 4 + K / 64 + 8 + 8 + 3) * EPS * (mag + big) + 2 * EPS * np.abs(want) * 1.0001
    assert (np.abs(f64(y) - want) <= tol).all()


def test_linear_codes_reach_their_places(L):
    """Weights that single out one input each: every nibble of the layout is found."""
    rng = np.random.default_rng(5)
    N, K = 128, 128
    q = np.zeros((N, K), np.uint8)
    q[np.arange(N), rng.permutation(K)] = rng.integers(1, 16, N)
    codes = dev(q[:, 0::2] | (q[:, 1::2] << 4))
    s, b = torch.ones((N, 2), dtype=torch.half, device="cuda"), torch.zeros((N, 2), dtype=torch.half, device="cuda")
    w = torch.empty(L.e0_linear_bytes(N, K), dtype=torch.uint8, device="cuda")
    L.e0_pack_linear(L.QTensor(codes.data_ptr(), s.data_ptr(), b.data_ptr()), N, K, w)
    x = dev(rng.integers(-99, 100, (3, K)), torch.float32)
    y = torch.empty((3, N), device="cuda")
    L.e0_linear_forward(w, N, K, x, F32, K, None, 3, None, 0, y, F32, N)
    assert np.array_equal(f64(y), f64(x) @ q.T.astype(np.float64))


# ------------------------------------------------------------------ plan and release


class Kv:
    """Sequences, their blocks and the free stack, on the host and on the device."""

    def __init__(self, L, B, bs, max_blocks, n_blocks, rng, held=None):
        self.L, self.B, self.bs, self.M, self.n = L, B, bs, max_blocks, n_blocks
        ids = list(rng.permutation(n_blocks))
        self.ctx = np.zeros(B, np.int32) if held is None else np.asarray(held, np.int32)
        self.table = np.full((B, max_blocks), -1, np.int32)
        for b in range(B):
            for j in range(-(-int(self.ctx[b]) // bs)):
                self.table[b, j] = ids.pop()
        self.free = ids
        self.d_table, self.d_ctx = dev(self.table), dev(self.ctx)
        fl = np.full(n_blocks, -5, np.int32)
        fl[:len(ids)] = ids
        self.d_free, self.d_count = dev(fl), dev(np.array([len(ids)], np.int32))
        self.desc = L.KvState(self.d_table.data_ptr(), self.d_ctx.data_ptr(), self.d_free.data_ptr(),
                              self.d_count.data_ptr(), B, max_blocks, bs, n_blocks)

    def plan_ref(self, new):
        slots, pos, seq = [], [], []
        for b in range(self.B):
            for i in range(int(new[b])):
                p = int(self.ctx[b]) + i
                if p % self.bs == 0:
                    self.table[b, p // self.bs] = self.free.pop()
                slots.append(int(self.table[b, p // self.bs]) * self.bs + p % self.bs)
                pos.append(p)
                seq.append(b)
            self.ctx[b] += int(new[b])
        return slots, pos, seq

    def check(self):
        assert np.array_equal(self.d_table.cpu().numpy(), self.table)
        assert np.array_equal(self.d_ctx.cpu().numpy(), self.ctx)
        assert int(self.d_count.item()) == len(self.free)
        assert np.array_equal(self.d_free.cpu().numpy()[:len(self.free)], np.array(self.free, np.int32))


def plan(L, kv, new, T_cap, apart=False):
    B = kv.B
    o = {"cu": torch.full((B + 1,), -9, dtype=torch.int32, device="cuda"),
         "slots": torch.full((max(T_cap, 1),), -9, dtype=torch.int64, device="cuda"),
         "pos": torch.full((max(T_cap, 1),), -9, dtype=torch.int32, device="cuda"),
         "seq": torch.full((max(T_cap, 1),), -9, dtype=torch.int32, device="cuda"), "st": status()}
    ctx = torch.empty_like(kv.d_ctx) if apart else kv.d_ctx
    count = torch.empty_like(kv.d_count) if apart else kv.d_count
    L.e0_kv_plan(kv.desc, dev(np.asarray(new, np.int32)), T_cap, ctx, count, o["cu"], o["slots"], o["pos"], o["seq"],
                 o["st"])
    if apart:
        kv.d_ctx.copy_(ctx)
        kv.d_count.copy_(count)
    return o


@pytest.mark.parametrize("B,bs,top,pad", [(1, 16, 1, 0), (1, 128, 300, 5), (64, 64, 1, 0), (64, 64, 1, 64), (7, 32, 90, 3),
                                          (300, 16, 60, 100), (1500, 16, 3, 0), (4096, 16, 2, 1), (3, 64, 6000, 7)])
@pytest.mark.parametrize("apart", [False, True])
def test_plan_steps(L, B, bs, top, pad, apart):
    rng = np.random.default_rng(B + top)
    steps = 3
    M = -(-steps * (top + 1) // bs) + 4
    kv = Kv(L, B, bs, M, B * M + 3, rng, rng.integers(0, 2 * bs, B))
    for step in range(steps):
        new = rng.integers(0, top + 1, B) if top > 1 else np.ones(B, int)
        T = int(new.sum())
        o = plan(L, kv, new, T + pad, apart)
        slots, pos, seq = kv.plan_ref(new)
        assert L.e0_read_status(o["st"]) == 0
        assert np.array_equal(o["cu"].cpu().numpy(), np.concatenate([[0], np.cumsum(new)]))
        for name, want in (("slots", slots), ("pos", pos), ("seq", seq)):
            got = o[name].cpu().numpy()[:T + pad]
            assert np.array_equal(got[:T], np.array(want, got.dtype)) and (got[T:] == -1).all(), name
        kv.check()


def test_plan_is_all_or_nothing(L):
    rng = np.random.default_rng(2)
    cases = [  # new lengths, T_cap, what is raised
        ([100, 0, 0, 1], 200, "E0_ST_POOL_FULL"),   # 2 + 5 + 0: more blocks than are free
        ([3, 3, 3, 3], 11, "E0_ST_POOL_FULL"),      # more tokens than T_cap
        ([1, -1, 0, 0], 10, "E0_ST_BAD_LENGTH"),
        ([0, 0, 0, 200], 400, "E0_ST_BAD_LENGTH"),  # beyond max_blocks
        ([2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1, 5], 10, "E0_ST_BAD_LENGTH")]
    for new, cap, bit in cases:
        for apart in (False, True):
            kv = Kv(L, 4, 16, 10, 12, rng, [5, 16, 33, 70])  # 1 + 1 + 3 + 5 blocks held, 2 free
            o = plan(L, kv, new, cap, apart)
            assert L.e0_read_status(o["st"]) == getattr(L, bit)
            assert (o["cu"] == 0).all()
            assert (o["slots"][:cap] == -1).all() and (o["pos"][:cap] == -1).all() and (o["seq"][:cap] == -1).all()
            kv.check()
    kv = Kv(L, 4, 16, 10, 12, rng, [5, 16, 33, 70])
    kv.d_ctx[2] = -3
    o = plan(L, kv, [1, 1, 1, 1], 4)
    assert L.e0_read_status(o["st"]) == L.E0_ST_BAD_LENGTH and (o["slots"] == -1).all()
    kv = Kv(L, 2, 16, 4, 6, rng, [0, 0])
    kv.d_count.fill_(7)  # a stack higher than the pool
    o = plan(L, kv, [1, 1], 2)
    assert L.e0_read_status(o["st"]) == L.E0_ST_BAD_LENGTH and (o["slots"] == -1).all()


def test_plan_ids_out_of_range_and_empty_calls(L):
    rng = np.random.default_rng(8)
    kv = Kv(L, 2, 16, 4, 8, rng, [4, 16])
    kv.d_table[0, 0] = 8                       # a held block that cannot be
    top = int(kv.d_count.item()) - 1
    kv.d_free[top] = -2                        # a free one that cannot be
    o = plan(L, kv, [2, 1], 3)
    assert L.e0_read_status(o["st"]) == L.E0_ST_BAD_BLOCK
    assert (o["slots"] == -1).all() and o["pos"].tolist() == [4, 5, 16]
    kv = Kv(L, 2, 16, 4, 8, rng, [4, 16])
    o = plan(L, kv, [0, 0], 0)
    assert L.e0_read_status(o["st"]) == 0 and (o["cu"] == 0).all()
    kv.check()
    empty = L.KvState(None, None, kv.d_free.data_ptr(), kv.d_count.data_ptr(), 0, 4, 16, 8)
    cu = torch.full((1,), -9, dtype=torch.int32, device="cuda")
    count = kv.d_count.clone()
    L.e0_kv_plan(empty, None, 0, None, count, cu, None)
    assert cu.item() == 0 and count.item() == kv.d_count.item()


@pytest.mark.parametrize("B,bs,longest", [(1, 16, 1), (5, 32, 200), (64, 64, 1000), (900, 16, 200)])
@pytest.mark.parametrize("apart", [False, True])
def test_release_and_reuse(L, B, bs, longest, apart):
    rng = np.random.default_rng(B)
    held = rng.integers(0, longest + 1, B)
    M = -(-longest // bs) + 2
    kv = Kv(L, B, bs, M, int((-(-held // bs)).sum()) + 4, rng, held)
    mask = rng.integers(0, 2, B).astype(np.uint8) * 3
    mask[0] = 1
    ctx = torch.empty_like(kv.d_ctx) if apart else kv.d_ctx
    count = torch.empty_like(kv.d_count) if apart else kv.d_count
    st = status()
    L.e0_kv_release(kv.desc, dev(mask), ctx, count, st)
    kv.d_ctx.copy_(ctx), kv.d_count.copy_(count)
    assert L.e0_read_status(st) == 0
    for b in range(B):
        if mask[b]:
            n = -(-int(kv.ctx[b]) // bs)
            kv.free += list(kv.table[b, :n])
            kv.table[b, :n] = -1
            kv.ctx[b] = 0
    kv.check()
    new = np.where(mask > 0, bs + 1, 0)
    if 2 * (mask > 0).sum() <= len(kv.free):
        o = plan(L, kv, new, int(new.sum()))
        kv.plan_ref(new)
        assert L.e0_read_status(o["st"]) == 0
        kv.check()


def test_release_refuses_what_cannot_be(L):
    rng = np.random.default_rng(1)
    kv = Kv(L, 2, 16, 4, 8, rng, [30, 64])
    for ctx, count in (([65, 64], 2), ([-1, 64], 2), ([30, 64], 3)):  # 2 + 4 blocks held, 2 free
        kv.d_ctx.copy_(dev(np.array(ctx, np.int32)))
        kv.d_count.fill_(count)
        st = status()
        L.e0_kv_release(kv.desc, dev(np.ones(2, np.uint8)), kv.d_ctx, kv.d_count, st)
        assert L.e0_read_status(st) == L.E0_ST_BAD_LENGTH
        assert kv.d_ctx.tolist() == ctx and kv.d_count.item() == count
        assert np.array_equal(kv.d_table.cpu().numpy(), kv.table)


@pytest.mark.parametrize("B,bs,longest,wide", [(3, 16, 100, 0), (40, 16, 300, 0), (40, 16, 300, 300), (700, 16, 200, 0)])
@pytest.mark.parametrize("bad", [False, True])
@pytest.mark.parametrize("apart", [False, True])
def test_release_passes_over_places_without_a_block(L, B, bs, longest, wide, bad, apart):
    """Rows whose early blocks are gone (-1), or that hold ids that cannot be: what goes onto the stack are blocks of the
    pool, in order, and a plan that takes them all gives every token a place.  wide: a table with many more places."""
    rng = np.random.default_rng(B + wide)
    held = rng.integers(1, longest + 1, B)
    M = -(-longest // bs) + 2 + wide
    kv = Kv(L, B, bs, M, int((-(-held // bs)).sum()) + 4, rng, held)
    mask = rng.integers(0, 4, B).astype(np.uint8)
    mask[0] = 1
    gone = []
    for b in range(B):
        n = -(-int(kv.ctx[b]) // bs)
        k = int(rng.integers(0, n + 1)) if mask[b] else 0
        gone += list(kv.table[b, :k])  # given back by hand, in what order ever
        kv.table[b, :k] = -1
    kv.free = gone[::-1] + kv.free
    junk = [kv.n, -2, 2 ** 31 - 1, -2 ** 31] if bad else []
    at = [(b, j) for b in range(B) if mask[b] for j in range(-(-int(kv.ctx[b]) // bs)) if kv.table[b, j] == -1][:len(junk)]
    dirty = kv.table.copy()
    for (b, j), x in zip(at, junk):
        dirty[b, j] = x
    kv.d_table.copy_(dev(dirty))
    kv.d_free[:len(kv.free)] = dev(np.array(kv.free, np.int32))
    kv.d_count.fill_(len(kv.free))
    ctx = torch.empty_like(kv.d_ctx) if apart else kv.d_ctx
    count = torch.empty_like(kv.d_count) if apart else kv.d_count
    st = status()
    L.e0_kv_release(kv.desc, dev(mask), ctx, count, st)
    kv.d_ctx.copy_(ctx), kv.d_count.copy_(count)
    assert L.e0_read_status(st) == (L.E0_ST_BAD_BLOCK if at else 0)
    for b in range(B):
        if mask[b]:
            kv.free += [int(x) for x in kv.table[b] if x >= 0]
            kv.table[b] = -1
            kv.ctx[b] = 0
    kv.check()
    new = np.zeros(B, int)  # all the blocks that there are, one sequence after another
    left = len(kv.free)
    for b in np.flatnonzero(mask):
        k = min(left, M)
        new[b], left = k * bs, left - k
    o = plan(L, kv, new, int(new.sum()))
    slots, _, _ = kv.plan_ref(new)
    assert L.e0_read_status(o["st"]) == 0 and np.array_equal(o["slots"].cpu().numpy()[:len(slots)], np.array(slots))
    kv.check()


def test_release_of_the_most_places(L):
    """2^30 places without a block are passed over; more are refused."""
    per = 1 << 26
    table = torch.full((17, per), -1, dtype=torch.int32, device="cuda")
    table[3, per - 1], table[15, 0], table[15, per - 1] = 5, 2, 7
    ctx = torch.full((17,), 1 << 30, dtype=torch.int32, device="cuda")
    free = torch.full((8,), -5, dtype=torch.int32, device="cuda")
    free[:2] = torch.tensor([1, 6])
    count = torch.full((1,), 2, dtype=torch.int32, device="cuda")
    kv = L.KvState(table.data_ptr(), ctx.data_ptr(), free.data_ptr(), count.data_ptr(), 17, per, 16, 8)
    mask, st = torch.ones(17, dtype=torch.uint8, device="cuda"), status()
    L.e0_kv_release(kv, mask, ctx, count, st)
    assert L.e0_read_status(st) == L.E0_ST_BAD_LENGTH
    assert (ctx == 1 << 30).all() and count.item() == 2 and table[3, per - 1].item() == 5
    mask[16] = 0
    st.zero_()
    L.e0_kv_release(kv, mask, ctx, count, st)
    assert L.e0_read_status(st) == 0 and ctx.tolist() == [0] * 16 + [1 << 30]
    assert count.item() == 5 and free.tolist() == [1, 6, 5, 2, 7, -5, -5, -5]
    assert table[3, per - 1].item() == table[15, 0].item() == table[15, per - 1].item() == -1


@pytest.mark.parametrize("B,M", [(3, 8), (200, 40)])
def test_a_captured_plan_and_release(L, B, M):
    """Sequences that come and go by the same graph, on a stream of its own, lengths and stack in place."""
    rng = np.random.default_rng(M)
    kv = Kv(L, B, 16, M, B * M // 2, rng, rng.integers(0, 30, B))
    new, mask = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.uint8, device="cuda")
    cap = 40 * B
    cu, slots = torch.zeros(B + 1, dtype=torch.int32, device="cuda"), torch.zeros(cap, dtype=torch.int64, device="cuda")
    st, stream = status(), torch.cuda.Stream()

    def step(s=None):
        L.e0_kv_release(kv.desc, mask, kv.d_ctx, kv.d_count, st, s)
        L.e0_kv_plan(kv.desc, new, cap, kv.d_ctx, kv.d_count, cu, slots, status=st, stream=s)

    torch.cuda.synchronize()
    step(stream)  # the first call of everything: nothing comes, nothing goes
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        step()
    for _ in range(12):
        gone = (rng.random(B) < 0.3) | (kv.ctx > 16 * M - 60)
        for b in np.flatnonzero(gone):
            kv.free += [int(x) for x in kv.table[b] if x >= 0]
            kv.table[b], kv.ctx[b] = -1, 0
        lens = rng.integers(0, 40, B)
        lens[np.cumsum(lens // 16 + 2) > len(kv.free)] = 0
        mask.copy_(dev(gone.astype(np.uint8)))
        new.copy_(dev(lens.astype(np.int32)))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        want, _, _ = kv.plan_ref(lens)
        assert L.e0_read_status(st) == 0 and slots[:len(want)].tolist() == want and (slots[len(want):] == -1).all()
        kv.check()


# ------------------------------------------------------------------ append


def cache_dev(L, c):
    t = [dev(c.k), dev(c.v), dev(c.ks), dev(c.vs)]
    return t, L.KvCache(*[x.data_ptr() for x in t], c.n, c.H, c.bs, c.D)


def same_cache(t, c, blocks):
    """Codes that stand for the same numbers (0 and -0 are one), scales equal."""
    k, v, ks, vs = [x.cpu().numpy() for x in t]
    b = sorted(blocks)
    assert np.array_equal(ks[b], c.ks[b]) and np.array_equal(vs[b], c.vs[b])
    assert np.array_equal(R.decode(k), R.decode(c.k)) and np.array_equal(R.decode(v), R.decode(c.v))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("bs,Hkv", [(16, 1), (64, 3), (128, 2)])
def test_append_steps(L, D, dtype, bs, Hkv):
    """Prompts, then single tokens whose size grows and shrinks, into blocks that
    hold anything before: codes and scales equal the reference's."""
    rng = np.random.default_rng(D + bs)
    B = 5
    c = R.Cache(60, Hkv, bs, D, rng)
    t, desc = cache_dev(L, c)
    kv = Kv(L, B, bs, 12, 60, rng)
    touched = set()
    for step in range(6):
        new = rng.integers(0, 3 * bs // 2, B) if step in (0, 3) else np.ones(B, int)
        slots, _, _ = kv.plan_ref(new)
        T = len(slots) + 2
        slots = np.array([-1] + slots + [-1], np.int64)  # padding is skipped
        size = np.exp(rng.normal(0, 2, (T, 2, Hkv, 1)))
        x = dev(rng.standard_normal((T, 2, Hkv, D)) * size, DT[dtype])
        st = status()
        row = 2 * Hkv * D
        L.e0_kv_append(desc, x, x[:, 1], dtype, row, row, dev(slots), T, st)
        assert L.e0_read_status(st) == 0
        xv = f64(x)
        c.append(xv[:, 0], xv[:, 1], slots)
        touched |= {int(s) // bs for s in slots if s >= 0}
        same_cache(t, c, touched)


def test_append_unaligned_rows_bad_slots_and_non_finite_values(L):
    rng = np.random.default_rng(11)
    c = R.Cache(6, 2, 16, 64, rng)
    t, desc = cache_dev(L, c)
    T, ld = 5, 2 * 64 + 1
    flat = dev(rng.standard_normal(2 * T * ld + 2), torch.bfloat16)
    k, v = flat[1:], flat[1 + T * ld:]
    slots = np.array([16, 17, 6 * 16, 95, 48], np.int64)  # the third beyond the cache, the fourth a block's last place
    st = status()
    L.e0_kv_append(desc, k, v, BF16, ld, ld, dev(slots), T, st)
    assert L.e0_read_status(st) == L.E0_ST_BAD_BLOCK
    kk = f64(torch.as_strided(k, (T, 2, 64), (ld, 64, 1)))
    vv = f64(torch.as_strided(v, (T, 2, 64), (ld, 64, 1)))
    c.ks[5], c.vs[5] = 2.0 ** 60, 2.0 ** 60  # block 5 holds 15 tokens already, at a scale that stays
    t[2][5], t[3][5] = 2.0 ** 60, 2.0 ** 60
    t2, desc2 = cache_dev(L, c)
    L.e0_kv_append(desc2, k, v, BF16, ld, ld, dev(slots), T, None)
    c.append(kk, vv, slots)
    same_cache(t2, c, {1, 3, 5})
    x = dev(rng.standard_normal((2, 2, 64)), torch.float32)
    x[0, 0, 3], x[1, 1, 0], x[1, 1, 1] = float("nan"), float("inf"), float("-inf")
    st = status()
    L.e0_kv_append(desc2, x, x, F32, 128, 128, dev(np.array([0, 1], np.int64)), 2, st)
    assert L.e0_read_status(st) == L.E0_ST_NONFINITE
    xv = f64(x)
    c.append(xv, xv, [0, 1])
    same_cache(t2, c, {0, 1, 3, 5})
    zero = torch.zeros((1, 2, 64), device="cuda")
    L.e0_kv_append(desc2, zero, zero, F32, 128, 128, dev(np.array([32], np.int64)), 1, None)
    assert (t2[2][2] == 2.0 ** -100).all() and (t2[0][2, :, 0] == 0).all()


# ------------------------------------------------------------------ attention


def attend(L, c, desc, table, ctx, cu, q, dtype, window=0, scale=None, lse=True, pad_rows=2, out=None, max_q=None):
    T, Hq, D = q.shape
    B = len(ctx)
    n = np.diff(cu)
    max_q = max(1, int(n.max())) if max_q is None else max_q
    row = Hq * D
    if out is None:
        out = torch.full((T + pad_rows, Hq, D), -7.0, dtype=DT[dtype], device="cuda")
    ls = torch.full((T + pad_rows, Hq), -7.0, device="cuda") if lse else None
    wsb = L.e0_attn_workspace_size(B, Hq, c.H, D, max_q)
    ws = torch.full((wsb,), 255, dtype=torch.uint8, device="cuda")
    st = status()
    L.e0_attn_decode(desc, dev(np.asarray(table, np.int32)), np.asarray(table).shape[1], dev(np.asarray(ctx, np.int32)),
                     dev(np.asarray(cu, np.int32)), B, max_q, q, dtype, row, Hq, scale or 1 / np.sqrt(D), window, out,
                     row, ls, ws, wsb, st)
    return out, ls, L.e0_read_status(st)


def filled_cache(L, B, bs, Hkv, D, ctx, rng, extra=2):
    """A pool whose used places hold normal values (sizes by block and head) and whose other places hold anything."""
    need = [-(-int(x) // bs) for x in ctx]
    c = R.Cache(sum(need) + extra, Hkv, bs, D, rng)
    ids = rng.permutation(c.n)
    table = np.full((B, max(max(need), 1) + 1), -1, np.int32)
    at = 0
    for b in range(B):
        for j in range(need[b]):
            blk = int(ids[at])
            at += 1
            table[b, j] = blk
            m = min(bs, int(ctx[b]) - j * bs)
            for codes, scale in ((c.k, c.ks), (c.v, c.vs)):
                size = np.exp(rng.normal(0, 0.7, Hkv))
                x = rng.standard_normal((Hkv, m, D)) * size[:, None, None]
                s = np.array([R.pow2_scale(np.abs(x[h]).max()) for h in range(Hkv)])
                scale[blk] = s
                codes[blk, :, :m] = R.encode(x / s[:, None, None])
    t, desc = cache_dev(L, c)
    return c, t, desc, table


def check_attention(c, table, ctx, cu, q, out, lse, dtype, window=0, scale=None):
    T, Hq, D = q.shape
    scale = float(np.float32(scale or 1 / np.sqrt(D)))
    got, gl, qv = f64(out), f64(lse) if lse is not None else None, f64(q)
    for b in range(len(ctx)):
        n = cu[b + 1] - cu[b]
        if n == 0:
            continue
        k, v = c.row(table[b], int(ctx[b]))
        # bf16 with more than 8 query rows a KV head: weights rounded to fp16, half a step at most
        wide = dtype == BF16 and int(np.diff(cu).max()) * (Hq // c.H) > 8
        o, l, tol, ltol = R.attention(qv[cu[b]:cu[b + 1]], k, v, scale, int(ctx[b]), window,
                                      2.0 ** -11 if wide else 0.0)
        g = got[cu[b]:cu[b + 1]]
        assert (np.abs(g - o) <= tol + H[dtype] * np.abs(o) * 1.0001 + TINY16[dtype]).all(), b
        if gl is not None:
            x = gl[cu[b]:cu[b + 1]]
            none = np.isneginf(l)
            assert np.isneginf(x[none]).all() and (np.abs(x[~none] - l[~none]) <= ltol[~none]).all(), b
    end = cu[-1]
    assert (got[end:] == -7).all() and (gl is None or (gl[end:] == -7).all())


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("bs", [16, 32, 64, 128])
def test_attention_lengths(L, D, dtype, bs):
    """Lengths from one token on, around block and unit edges, one query each."""
    rng = np.random.default_rng(D + bs)
    ctx = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200, 333, 1000]
    c, t, desc, table = filled_cache(L, len(ctx), bs, 2, D, ctx, rng)
    cu = np.arange(len(ctx) + 1)
    q = dev(rng.standard_normal((len(ctx), 6, D)), DT[dtype])
    out, lse, st = attend(L, c, desc, table, ctx, cu, q, dtype)
    assert st == 0
    check_attention(c, table, ctx, cu, q, out, lse, dtype)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 8), (4, 1), (6, 2), (24, 3), (32, 2), (20, 1)])
@pytest.mark.parametrize("window", [0, 1, 50])
def test_attention_heads_and_runs_of_queries(L, Hq, Hkv, window):
    """Several queries a sequence, none for some, more rows than a tile."""
    rng = np.random.default_rng(Hq * 7 + window)
    new = [1, 0, 5, 9, 2, 0]
    ctx = [40, 30, 5, 300, 70, 0]
    cu = np.concatenate([[0], np.cumsum(new)])
    c, t, desc, table = filled_cache(L, len(ctx), 32, Hkv, 64, ctx, rng)
    q = dev(rng.standard_normal((int(cu[-1]), Hq, 64)) * 2, torch.float16)
    out, lse, st = attend(L, c, desc, table, ctx, cu, q, F16, window)
    assert st == 0
    check_attention(c, table, ctx, cu, q, out, lse, F16, window)


@pytest.mark.parametrize("Hq,Hkv,D", [(16, 1, 64), (24, 1, 128), (32, 2, 256), (9, 1, 128)])
@pytest.mark.parametrize("window", [0, 60])
def test_attention_many_rows_bf16(L, Hq, Hkv, D, window):
    """More than 8 query rows a KV head: tiles of 16, the last one part empty; sequences on one and on several blocks."""
    rng = np.random.default_rng(Hq + D)
    new = [1, 3, 0, 5, 1]
    ctx = [1, 700, 9, 64, 3000]
    cu = np.concatenate([[0], np.cumsum(new)])
    c, t, desc, table = filled_cache(L, len(ctx), 16, Hkv, D, ctx, rng)
    q = dev(rng.standard_normal((int(cu[-1]), Hq, D)) * 1.5, torch.bfloat16)
    out, lse, st = attend(L, c, desc, table, ctx, cu, q, BF16, window)
    assert st == 0
    check_attention(c, table, ctx, cu, q, out, lse, BF16, window)
    q[0, 8] = float("nan")  # one head of the upper rows
    out2, lse2, _ = attend(L, c, desc, table, ctx, cu, q, BF16, window)
    assert out2[0, 8].isnan().all() and torch.equal(out2[1:], out[1:]) and torch.equal(out2[0, :8], out[0, :8])


@pytest.mark.parametrize("B,longest,Hq,Hkv,D", [(1, 9000, 8, 1, 128), (1, 20000, 4, 2, 64), (3, 5000, 16, 2, 256), (1, 12000, 32, 2, 128),
                                                (40, 900, 8, 4, 64), (300, 60, 2, 2, 64)])
def test_attention_splits(L, B, longest, Hq, Hkv, D):
    """Long sequences split over many blocks, many short ones packed into each."""
    rng = np.random.default_rng(B)
    ctx = [longest] if B == 1 else rng.integers(1, longest + 1, B)
    cu = np.arange(B + 1)
    c, t, desc, table = filled_cache(L, B, 64, Hkv, D, ctx, rng)
    q = dev(rng.standard_normal((B, Hq, D)) * 1.5, torch.bfloat16)
    out, lse, st = attend(L, c, desc, table, ctx, cu, q, BF16)
    assert st == 0
    check_attention(c, table, ctx, cu, q, out, lse, BF16)
    again, _, _ = attend(L, c, desc, table, ctx, cu, q, BF16)
    assert torch.equal(out, again)


@pytest.mark.parametrize("D,most", [(64, 1280), (128, 768), (256, 384)])
@pytest.mark.parametrize("more", [-1, 0, 1, 40])
@pytest.mark.parametrize("windowed", [False, True])
def test_attention_few_short_jobs(L, D, most, more, windowed):
    """A long sequence among short ones, around the longest that tables or windows may hold for calls without a join."""
    rng = np.random.default_rng(D + more)
    window = most + more - 1 - (128 if D < 256 else 64) if windowed else 0
    ctx = [1, most + more + (5000 if windowed else 0), 3]
    cu = np.arange(4)
    c, t, desc, table = filled_cache(L, 3, 16, 2, D, ctx, rng)
    table = np.ascontiguousarray(table[:, :-(-ctx[1] // 16)])
    q = dev(rng.standard_normal((3, 4, D)), torch.float16)
    out, lse, st = attend(L, c, desc, table, ctx, cu, q, F16, window)
    assert st == 0
    check_attention(c, table, ctx, cu, q, out, lse, F16, window)


@pytest.mark.parametrize("D,unit", [(64, 128), (128, 128), (256, 64)])
@pytest.mark.parametrize("more", [-1, 0, 1])
def test_attention_a_unit_a_block(L, D, unit, more):
    """Sequences that come to as many units as there are blocks, to one fewer and to one more."""
    blocks = 2 * torch.cuda.get_device_properties(0).multi_processor_count
    rng = np.random.default_rng(D + more)
    units = blocks // 2 - 2  # of two heads, beside two sequences of one unit
    ctx = [3, (units // 2 + more) * unit - 5, unit, (units - units // 2) * unit]
    cu = np.array([0, 1, 2, 3, 4])
    c, t, desc, table = filled_cache(L, 4, 64, 2, D, ctx, rng)
    q = dev(rng.standard_normal((4, 16, D)) * 1.5, torch.float32)
    out, lse, st = attend(L, c, desc, table, ctx, cu, q, F32)
    assert st == 0
    check_attention(c, table, ctx, cu, q, out, lse, F32)
    again, _, _ = attend(L, c, desc, table, ctx, cu, q, F32)
    assert torch.equal(out, again)


def test_attention_without_cu_q_or_lse_and_strided(L):
    rng = np.random.default_rng(6)
    B, Hq, Hkv, D, bs = 5, 4, 2, 64, 16
    ctx = [3, 100, 16, 1, 47]
    c, t, desc, table = filled_cache(L, B, bs, Hkv, D, ctx, rng)
    big = dev(rng.standard_normal((B, 3 * Hq * D)), torch.float32)
    q = big[:, Hq * D:2 * Hq * D].reshape(B, Hq, D)
    out = torch.full((B, Hq * D + 8), -7.0, device="cuda")
    wsb = L.e0_attn_workspace_size(B, Hq, Hkv, D, 1)
    ws = torch.empty(wsb, dtype=torch.uint8, device="cuda")
    L.e0_attn_decode(desc, dev(table), table.shape[1], dev(np.array(ctx, np.int32)), None, B, 1, big[:, Hq * D:], F32,
                     3 * Hq * D, Hq, 0.125, 0, out, Hq * D + 8, None, ws, wsb)
    assert (out[:, Hq * D:] == -7).all()
    check_attention(c, table, ctx, np.arange(B + 1), q, out[:, :Hq * D].reshape(B, Hq, D), None, F32)


def test_attention_rows_that_see_nothing(L):
    """Lengths of zero, queries before the first position, blocks that are not there, lengths that cannot be."""
    rng = np.random.default_rng(7)
    Hq, Hkv, D, bs = 4, 2, 64, 16
    ctx = [0, 2, 40, 33, 20]
    new = [2, 4, 1, 1, 1]   # sequence 1 has more queries than positions: its first two see nothing
    cu = np.concatenate([[0], np.cumsum(new)])
    c, t, desc, table = filled_cache(L, 5, bs, Hkv, D, ctx, rng)
    q = dev(rng.standard_normal((int(cu[-1]), Hq, D)), torch.float32)
    out, lse, st = attend(L, c, desc, table, ctx, cu, q, F32)
    assert st == 0
    check_attention(c, table, ctx, cu, q, out, lse, F32)
    assert (out[:4] == 0).all() and torch.isneginf(lse[:4]).all()
    # block ids out of range: their tokens are not seen
    table[2, 1], table[3, 0], table[3, 1], table[3, 2] = c.n, -1, 2 ** 31 - 1, -2 ** 31
    out, lse, st = attend(L, c, desc, table, ctx, cu, q, F32)
    assert st == L.E0_ST_BAD_BLOCK
    check_attention(c, table, ctx, cu, q, out, lse, F32)
    assert (out[7] == 0).all() and torch.isneginf(lse[7]).all()
    # lengths that cannot be: nothing is seen, the other sequences are as before
    want = out.clone()
    for bad in (-1, table.shape[1] * bs + 1, 2 ** 31 - 1):
        out, lse, st = attend(L, c, desc, table, [0, 2, 40, 33, bad], cu, q, F32)
        assert st == L.E0_ST_BAD_LENGTH | L.E0_ST_BAD_BLOCK
        assert (out[8] == 0).all() and torch.isneginf(lse[8]).all() and torch.equal(out[:8], want[:8])
    # more queries than max_q, a cu_q that falls: those rows are left as they were
    out, lse, st = attend(L, c, desc, table, ctx, cu, q, F32, max_q=3)
    assert st == L.E0_ST_BAD_LENGTH | L.E0_ST_BAD_BLOCK
    assert (out[2:6] == -7).all() and torch.equal(out[6:9], want[6:9])
    falls = cu.copy()
    falls[2] = 1
    out, lse, st = attend(L, c, desc, table, ctx, falls, q, F32, max_q=9)
    assert st & L.E0_ST_BAD_LENGTH


def test_attention_row_numbers_that_wrap(L):
    """A cu_q whose neighbours differ by more than 32 bits hold: -2^31 - (2^31 - 1) is 1 in 32 bits, and 2^31 - 1 no row."""
    rng = np.random.default_rng(18)
    Hq, Hkv, D, bs = 4, 2, 64, 16
    ctx, cu = [20, 33], np.array([0, 1, 2])
    c, t, desc, table = filled_cache(L, 2, bs, Hkv, D, ctx, rng)
    q = dev(rng.standard_normal((2, Hq, D)), torch.float32)
    want, _, st = attend(L, c, desc, table, ctx, cu, q, F32)
    assert st == 0
    top = 2 ** 31 - 1
    for bad in ([top, -top - 1, 2], [top - 1, -top, 1], [top, -top + 1, -top + 1], [1, -top, -top + 2]):
        out, lse, st = attend(L, c, desc, table, ctx, np.array(bad), q, F32, max_q=3)
        assert st == L.E0_ST_BAD_LENGTH and (out == -7).all() and (lse == -7).all()
    out, _, st = attend(L, c, desc, table, ctx, np.array([-top - 1, 1, 2]), q, F32, max_q=3)
    assert st == L.E0_ST_BAD_LENGTH and torch.equal(out[1], want[1]) and (out[0] == -7).all()


@pytest.mark.parametrize("bs", [16, 64])
def test_attention_window_over_released_blocks(L, bs):
    """Blocks that lie wholly before the window may be gone: ids out of range, scales that are not numbers."""
    rng = np.random.default_rng(bs)
    Hq, Hkv, D, window = 4, 2, 64, 70
    ctx, cu = [500, 130, 69], np.array([0, 1, 4, 6])
    c, t, desc, table = filled_cache(L, 3, bs, Hkv, D, ctx, rng)
    q = dev(rng.standard_normal((6, Hq, D)), torch.float32)
    out, lse, st = attend(L, c, desc, table, ctx, cu, q, F32, window)
    check_attention(c, table, ctx, cu, q, out, lse, F32, window)
    for b in range(3):
        first = max(0, ctx[b] - (cu[b + 1] - cu[b]) + 1 - window)
        for j in range(first // bs):
            blk = int(table[b, j])
            t[2][blk], t[3][blk], t[0][blk], t[1][blk] = float("nan"), float("inf"), 127, 127
            if j % 2:
                table[b, j] = -1
    again, lse2, st = attend(L, c, desc, table, ctx, cu, q, F32, window)
    assert st == 0 and torch.equal(out, again) and torch.equal(lse, lse2)


def test_attention_masked_garbage_and_non_finite_queries(L):
    """What stands behind a sequence's end (NaN codes and scales) or outside a window does not matter; a query that is not
    finite spoils its own head only."""
    rng = np.random.default_rng(12)
    Hq, Hkv, D, bs = 4, 2, 128, 64
    ctx, cu = [70, 5], np.array([0, 3, 4])
    c, t, desc, table = filled_cache(L, 2, bs, Hkv, D, ctx, rng)
    q = dev(rng.standard_normal((4, Hq, D)), torch.float32)
    out, lse, st = attend(L, c, desc, table, ctx, cu, q, F32)
    check_attention(c, table, ctx, cu, q, out, lse, F32)
    for b in range(2):
        blk, off = table[b, (ctx[b] - 1) // bs], ctx[b] % bs
        t[0][blk, :, off:], t[1][blk, :, off:] = 127, 255
    again, _, _ = attend(L, c, desc, table, ctx, cu, q, F32)
    assert torch.equal(out, again)
    q[1, 2, 7], q[3, 0, 0] = float("nan"), float("inf")
    out2, lse2, _ = attend(L, c, desc, table, ctx, cu, q, F32)
    assert out2[1, 2].isnan().all() and lse2[1, 2].isnan() and out2[3, 0].isnan().all()
    ok = torch.ones((4, Hq), dtype=torch.bool, device="cuda")
    ok[1, 2] = ok[3, 0] = False
    assert torch.equal(out2[:4][ok], out[:4][ok]) and torch.equal(lse2[:4][ok], lse[:4][ok])


def test_attention_scores_and_scales_far_apart(L):
    """Scores in the hundreds, queries and blocks whose sizes differ by powers of two far beyond fp16's range."""
    rng = np.random.default_rng(13)
    Hq, Hkv, D, bs = 4, 1, 64, 16
    ctx, cu = [200, 64], np.array([0, 1, 2])
    c, t, desc, table = filled_cache(L, 2, bs, Hkv, D, ctx, rng)
    c.vs[table[0, :13]] *= np.exp2(rng.integers(-30, 30, (13, 1))).astype(np.float32)
    c.vs[table[1, 0]] = 2.0 ** -60
    c.ks[table[0, 5]] *= 32
    t, desc = cache_dev(L, c)
    for size in (1e-20, 1.0, 60.0):
        q = dev(rng.standard_normal((2, Hq, D)) * size, torch.float32)
        out, lse, st = attend(L, c, desc, table, ctx, cu, q, F32)
        check_attention(c, table, ctx, cu, q, out, lse, F32)


@pytest.mark.parametrize("Hq,dtype", [(1, F32), (4, F16), (16, BF16)])
def test_attention_lse_over_values_of_zero(L, Hq, dtype):
    """A long context of zero values (scales of 2^-100): the softmax's sum stays in range, with scores that rise by almost
    the running maximum's slack after each warp's first step, as with equal ones."""
    B, n, D, bs = 300, 1 << 14, 64, 128
    c = R.Cache(n // bs, 1, bs, D)
    c.k[1:, :, :, 0] = 0x38  # 1.0; the first 128 positions have scores of 0
    c.ks[:], c.vs[:] = 1, 2.0 ** -100
    t, desc = cache_dev(L, c)
    table = np.tile(np.arange(n // bs, dtype=np.int32), (B, 1))
    q = torch.zeros((B, Hq, D), dtype=DT[dtype], device="cuda")
    q[:, :, 0] = 43.75  # times 0.125: 7.89 in log2
    ctx, cu = [n] * B, np.arange(B + 1)
    out, lse, st = attend(L, c, desc, table, ctx, cu, q, dtype)
    assert st == 0 and (out[:B] == 0).all()
    want = np.log(128 + (n - 128) * np.exp(43.75 * 0.125))
    # in log2: t, the maximum's part, log2 of the sum and their own sum are below 2^7, so half a step is 2^-18; log2f
    # may be off by a step; exp2 by 2 ulp and n positive terms in 304 blocks of 4 warps of 8 lanes are summed in fp32
    tol = (3 * 2.0 ** -18 + 2.0 ** -17) * np.log(2) + (2 + n / 32 + 64) * EPS + 4 * EPS * want
    assert (np.abs(f64(lse)[:B] - want) <= tol).all()
    # a sequence of 2^21 positions: the same blocks again and again, all scores equal
    m = (1 << 21) + 1000
    table = np.zeros((1, -(-m // bs)), np.int32)
    out, lse, st = attend(L, c, desc, table, [m], np.arange(2), q[:1], dtype)
    assert st == 0 and (out[:1] == 0).all()
    tol = (3 * 2.0 ** -18 + 2.0 ** -17) * np.log(2) + (2 + m / 32 / 150 + 304 + 64) * EPS + 4 * EPS * np.log(m)
    assert (np.abs(f64(lse)[:1] - np.log(m)) <= tol).all()


@pytest.mark.parametrize("Hq,dtype", [(2, F32), (16, BF16)])
def test_attention_values_of_the_largest_scales(L, Hq, dtype):
    """Values up to fp32's end: the inverse of the softmax's sum stays in range."""
    rng = np.random.default_rng(19)
    ctx, cu = [1, 70, 900], np.arange(4)
    c, t, desc, table = filled_cache(L, 3, 16, 1, 64, ctx, rng)
    c.v &= 0xF7  # codes of at most 240
    c.vs[:] = 2.0 ** 119
    t, desc = cache_dev(L, c)
    q = dev(rng.standard_normal((3, Hq, 64)) * 1.5, DT[dtype])
    out, lse, st = attend(L, c, desc, table, ctx, cu, q, dtype)
    assert st == 0 and torch.isfinite(out.float()).all()
    check_attention(c, table, ctx, cu, q, out, lse, dtype)


def test_attention_offsets_beyond_32_bits(L):
    """A pool of more than 2^31 code bytes: blocks at its end."""
    Hkv, D, bs = 8, 256, 128
    n = (1 << 31) // (Hkv * D * bs) + 600
    k = torch.zeros(n * Hkv * bs * D, dtype=torch.uint8, device="cuda")
    v = torch.zeros_like(k)
    ks, vs = torch.ones((n, Hkv), device="cuda"), torch.ones((n, Hkv), device="cuda")
    rng = np.random.default_rng(14)
    small, t, _, table = filled_cache(L, 2, bs, Hkv, D, [300, 129], rng)
    far = n - small.n
    per = Hkv * bs * D
    k[far * per:] = t[0].view(-1)
    v[far * per:] = t[1].view(-1)
    ks[far:], vs[far:] = t[2], t[3]
    desc = L.KvCache(k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(), n, Hkv, bs, D)
    q = dev(rng.standard_normal((2, 8, D)), torch.float16)
    cu = np.arange(3)
    out, lse, st = attend(L, small, desc, np.where(table >= 0, table + far, -1), [300, 129], cu, q, F16)
    assert st == 0
    check_attention(small, table, [300, 129], cu, q, out, lse, F16)
    x = dev(rng.standard_normal((1, Hkv, D)), torch.float16)
    at = (n - 1) * bs
    L.e0_kv_append(desc, x, x, F16, Hkv * D, Hkv * D, dev(np.array([at], np.int64)), 1, None)
    s = ks[n - 1].double().cpu().numpy()
    got = R.decode(k[(n - 1) * per:].view(Hkv, bs, D)[:, 0].cpu().numpy()) * s[:, None]
    assert np.array_equal(got, R.decode(R.encode(f64(x)[0] / s[:, None])) * s[:, None])


# ------------------------------------------------------------------ all of them


def test_attention_most_sequences_and_a_window_without_end(L):
    """As many sequences as a call takes, most of them empty or one token long; a window that covers everything is none."""
    rng = np.random.default_rng(16)
    B, Hq, Hkv, D, bs = 4096, 2, 1, 64, 16
    ctx = rng.integers(0, 3, B)
    ctx[[0, 1000, 4095]] = [40, 300, 17]
    new = np.minimum(ctx, 1)
    cu = np.concatenate([[0], np.cumsum(new)])
    c, t, desc, table = filled_cache(L, B, bs, Hkv, D, ctx, rng)
    q = dev(rng.standard_normal((int(cu[-1]), Hq, D)), torch.float32)
    out, lse, st = attend(L, c, desc, table, ctx, cu, q, F32)
    assert st == 0
    check_attention(c, table, ctx, cu, q, out, lse, F32)
    for window in (2 ** 31 - 1, table.shape[1] * bs):
        again, _, _ = attend(L, c, desc, table, ctx, cu, q, F32, window)
        assert torch.equal(out, again)


def test_calls_at_once_on_two_streams(L):
    """The same operators on two streams, workspaces of their own: what each leaves is what it leaves alone."""
    rng = np.random.default_rng(17)
    jobs = []
    for ctx in ([2500, 64, 900], [70, 3100, 1]):
        c, t, desc, table = filled_cache(L, 3, 64, 2, 128, ctx, rng)
        w, *_, keep = make_linear(L, 3000, 1024, rng)
        q = dev(rng.standard_normal((3, 8, 128)), torch.float16)
        x = dev(rng.standard_normal((12, 1024)), torch.float16)
        wsb = L.e0_attn_workspace_size(3, 8, 2, 128, 1)
        jobs.append(dict(desc=desc, t=t, table=dev(table), M=table.shape[1], ctx=dev(np.array(ctx, np.int32)), q=q, x=x, w=w,
                         keep=keep, ws=torch.empty(wsb, dtype=torch.uint8, device="cuda"), wsb=wsb, o=torch.empty_like(q),
                         y=torch.empty((12, 3000), device="cuda"), n8=torch.empty((12, 1024), dtype=torch.uint8, device="cuda"),
                         ns=torch.empty((12, 16), device="cuda")))

    def run(j, stream=None):
        L.e0_attn_decode(j["desc"], j["table"], j["M"], j["ctx"], None, 3, 1, j["q"], F16, 1024, 8, 0.1, 0, j["o"], 1024,
                         None, j["ws"], j["wsb"], None, stream)
        L.e0_rmsnorm_q8(j["x"], None, None, 12, 1024, F16, 1e-6, 1024, 0, None, None, j["n8"], j["ns"], None, stream)
        L.e0_linear_forward(j["w"], 3000, 1024, j["n8"], E4M3, 1024, j["ns"], 12, None, 0, j["y"], F32, 3000, stream)

    want = []
    for j in jobs:
        run(j)
        want.append((j["o"].clone(), j["y"].clone()))
        j["o"].zero_(), j["y"].zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for j, s in zip(jobs, streams):
            run(j, s)
    torch.cuda.synchronize()
    for j, (o, y) in zip(jobs, want):
        assert torch.equal(j["o"], o) and torch.equal(j["y"], y)


def test_streams_and_graphs_share_a_workspace(L):
    """Two captured attention steps over one workspace, replayed in turn, and the same on another stream, equal the eager calls."""
    rng = np.random.default_rng(15)
    Hq, Hkv, D, bs = 8, 2, 128, 64
    sets = []
    wsb = L.e0_attn_workspace_size(3, Hq, Hkv, D, 1)
    ws = torch.empty(wsb, dtype=torch.uint8, device="cuda")
    for ctx in ([3000, 10, 700], [1, 4000, 64]):
        c, t, desc, table = filled_cache(L, 3, bs, Hkv, D, ctx, rng)
        q = dev(rng.standard_normal((3, Hq, D)), torch.bfloat16)
        sets.append((c, t, desc, dev(table), table.shape[1], dev(np.array(ctx, np.int32)), q, torch.empty_like(q)))

    def step(x, out, stream=None):
        _, _, desc, table, M, ctx, q, _ = x
        L.e0_attn_decode(desc, table, M, ctx, None, 3, 1, q, BF16, Hq * D, Hq, 0.09, 0, out, Hq * D, None, ws, wsb,
                         None, stream)

    want = []
    for x in sets:
        step(x, x[7])
        want.append(x[7].clone())
    graphs = []
    for x in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(x, x[7])
        graphs.append(g)
    for x in sets:
        x[7].zero_()
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for x, y in zip(sets, want):
        assert torch.equal(x[7], y)
    other = torch.cuda.Stream()
    for x, y in zip(sets, want):
        x[7].zero_()
        torch.cuda.synchronize()
        step(x, x[7], other)
        other.synchronize()
        assert torch.equal(x[7], y)
