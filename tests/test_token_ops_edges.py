"""Rotation and sampling where their inputs go to the ends of their ranges, on the GPU against 64-bit references."""
import numpy as np
import pytest

from tests.test_layer_ops import BF16, DT, F16, F32, L  # noqa: F401
from tests.test_token_ops import draw, rules_of

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
