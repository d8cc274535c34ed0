"""Host-side argument checks of e0_attn_scored and e0_attn_shared: every refusal comes before a launch, so a CPU is
enough; and the arithmetic of the cap's polynomial."""
import numpy as np
import pytest

from tests.test_layer_ops_cpu import L, P, call  # noqa: F401


def cache(L, **c):  # noqa: F811
    f = dict(k=P, v=P, k_scale=P, v_scale=P, n_blocks=8, Hkv=2, block_tokens=16, D=64)
    f.update(c)
    return L.KvCache(**f)


SCORED = dict(cache=None, block_table=P, max_blocks=4, ctx_len=P, cu_q=P, B=2, max_q=2, q=P, dtype=1, q_ld=256, Hq=4,
              scale=0.125, rules=None, out=2 * P, out_ld=256, lse=None, ws=P, ws_bytes=1 << 34, status=None)
SHARED = dict(cache=None, prefix_table=P, prefix_blocks=4, prefix_len=P, block_table=P, max_blocks=4, ctx_len=P, cu_q=P, B=2,
              T=4, max_q=2, q=P, dtype=1, q_ld=256, Hq=4, scale=0.125, rules=None, out=2 * P, out_ld=256, lse=None, ws=P,
              ws_bytes=1 << 34, status=None)

BOTH = [
    (dict(B=-1), "ARG"), (dict(max_blocks=0), "ARG"), (dict(max_q=0), "ARG"), (dict(dtype=3), "ARG"), (dict(Hq=3), "ARG"),
    (dict(Hq=0), "ARG"), (dict(scale=float("nan")), "ARG"), (dict(cu_q=None), "ARG"), (dict(B=4097), "UNSUPPORTED"),
    (dict(max_blocks=1 << 27), "UNSUPPORTED"), (dict(max_q=1 << 29), "UNSUPPORTED"), (dict(block_table=None), "NULL"),
    (dict(ctx_len=None), "NULL"), (dict(q=None), "NULL"), (dict(out=None), "NULL"), (dict(ws=None), "NULL"),
    (dict(q_ld=255), "ARG"), (dict(out_ld=255), "ARG"), (dict(q=P + 8), "ARG"), (dict(q_ld=260), "ARG"), (dict(out=P + 1), "ARG"),
    (dict(ws=P + 128), "ARG"), (dict(ws_bytes=100), "ARG"), (dict(lse=P + 2), "ARG"), (dict(B=0, q=None), "OK")]


@pytest.mark.parametrize("change,code", BOTH)
def test_scored_and_shared_refusals(L, change, code):  # noqa: F811
    want = L.E0_OK if code == "OK" else getattr(L, "E0_ERR_" + code)
    assert call(L.e0_attn_scored, dict(SCORED, cache=cache(L)), **change) == want
    assert call(L.e0_attn_shared, dict(SHARED, cache=cache(L)), **change) == want


@pytest.mark.parametrize("change,code", [
    (dict(T=0), "ARG"), (dict(prefix_blocks=0), "ARG"), (dict(prefix_blocks=1 << 26), "UNSUPPORTED"),
    (dict(prefix_blocks=(1 << 26) - 4 + 1), "UNSUPPORTED"), (dict(prefix_blocks=(1 << 31) - 1), "UNSUPPORTED"),
    (dict(T=1 << 29), "UNSUPPORTED"), (dict(prefix_table=None), "NULL"), (dict(prefix_len=None), "NULL"),
    (dict(prefix_table=P + 2), "ARG"), (dict(prefix_len=P + 2), "ARG")])
def test_shared_refusals(L, change, code):  # noqa: F811
    assert call(L.e0_attn_shared, dict(SHARED, cache=cache(L)), **change) == getattr(L, "E0_ERR_" + code)


@pytest.mark.parametrize("field,value,scored,shared", [
    ("cap", -1.0, "ARG", "ARG"), ("cap", float("nan"), "ARG", "ARG"), ("cap", float("inf"), "ARG", "ARG"),
    ("window", -1, "ARG", "ARG"), ("rows", -1, "ARG", "ARG"), ("slopes", P + 2, "ARG", "ARG"), ("first", P + 1, "ARG", "ARG"), ("open_len", P + 1, "ARG", "ARG"),
    ("first", P, None, "UNSUPPORTED"), ("open_len", P, None, "UNSUPPORTED")])
def test_rules_refusals(L, field, value, scored, shared):  # noqa: F811
    rules = L.AttnRules(**{field: value})
    if scored:
        assert call(L.e0_attn_scored, dict(SCORED, cache=cache(L)), rules=rules) == getattr(L, "E0_ERR_" + scored)
    assert call(L.e0_attn_shared, dict(SHARED, cache=cache(L)), rules=rules) == getattr(L, "E0_ERR_" + shared)


@pytest.mark.parametrize("c,code", [(dict(D=96), "UNSUPPORTED"), (dict(block_tokens=8), "UNSUPPORTED"), (dict(k=None), "NULL"),
                                    (dict(k=P + 8), "ARG"), (dict(n_blocks=0), "ARG")])
def test_cache_refusals(L, c, code):  # noqa: F811
    for fn, base in ((L.e0_attn_scored, SCORED), (L.e0_attn_shared, SHARED)):
        assert call(fn, dict(base, cache=cache(L, **c))) == getattr(L, "E0_ERR_" + code)


def test_workspace_sizes(L):  # noqa: F811
    few, many = L.e0_attn_scored_workspace_size(2, 4, 2, 64, 4), L.e0_attn_scored_workspace_size(2, 4, 2, 64, 1000)
    assert few == L.e0_attn_workspace_size(2, 4, 2, 64, 4) and many > few
    assert L.e0_attn_scored_workspace_size(2, 4, 2, 64, 2000) >= many
    assert L.e0_attn_shared_workspace_size(2, 2000, 4, 2, 64, 4) > L.e0_attn_shared_workspace_size(2, 4, 4, 2, 64, 4) > few
    for bad in ((0, 4, 2, 64, 1), (4097, 4, 2, 64, 1), (1, 3, 2, 64, 1), (1, 4, 2, 96, 1), (1, 4, 2, 64, 0), (1, 4, 2, 64, 1 << 29)):
        assert L.e0_attn_scored_workspace_size(*bad) == 0
    assert L.e0_attn_shared_workspace_size(1, 0, 4, 2, 64, 1) == L.e0_attn_shared_workspace_size(1, 1 << 29, 4, 2, 64, 1) == 0


def test_the_caps_polynomial():
    """tanh(u) / u up to u = 1, the factors as the kernels have them, in fp32 steps: 1.5e-7 of itself."""
    import os
    import re
    here = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "int4_gathered_expert_gb300", "csrc")
    src = open(os.path.join(here, "e0_attn.cuh")).read()
    body = src[src.index("tanh_of(int i)"):]
    c = [np.float32(x) for x in re.findall(r"[?:] (-?\d+\.\d+)f", body[:body.index("}")])]
    assert len(c) == 8
    u = np.linspace(0, 1, 100001).astype(np.float32)[1:]
    v = (u * u).astype(np.float32)
    p = np.full_like(v, c[7])
    for k in c[6::-1]:
        p = (p.astype(np.float64) * v + np.float64(k)).astype(np.float32)
    want = np.tanh(u.astype(np.float64))
    assert (np.abs((p * u).astype(np.float32) / want - 1) < 1.5e-7).all()
