"""Host-side argument checks of e0_qk_rope and e0_sample: every refusal comes before a
launch, so a CPU is enough."""
import pytest

from tests.test_layer_ops_cpu import L, P, call  # noqa: F401

ROPE = dict(x=P, dtype=0, x_ld=192, T=1, Hq=2, Hk=1, rope=None, positions=P, pos_ld=1, y=2 * P, y_ld=192, status=None)


def rope(L, **c):  # noqa: F811
    f = dict(freq=P, axis=None, q_norm=None, k_norm=None, D=64, rot=64, n_axes=1, flags=0, eps=1e-6)
    f.update(c)
    return L.Rope(**f)


@pytest.mark.parametrize("change,of_rope,code", [
    (dict(T=-1), {}, "ARG"), (dict(Hq=-1), {}, "ARG"), (dict(Hk=-1), {}, "ARG"), (dict(Hq=0, Hk=0), {}, "ARG"),
    (dict(dtype=3), {}, "ARG"), (dict(dtype=-1), {}, "ARG"), ({}, dict(D=0), "ARG"), ({}, dict(D=63), "ARG"),
    ({}, dict(rot=66), "ARG"), ({}, dict(rot=-2), "ARG"), ({}, dict(rot=31), "ARG"), ({}, dict(n_axes=0), "ARG"),
    ({}, dict(n_axes=5), "ARG"), ({}, dict(flags=4), "ARG"), ({}, dict(eps=-1.0), "ARG"),
    ({}, dict(eps=float("nan")), "ARG"), (dict(x_ld=800, y_ld=800), dict(D=258, rot=64), "UNSUPPORTED"),
    (dict(T=(1 << 30) + 1), {}, "UNSUPPORTED"), (dict(Hq=65536), {}, "UNSUPPORTED"), (dict(x=None), {}, "NULL"),
    (dict(y=None), {}, "NULL"), (dict(positions=None), {}, "NULL"), ({}, dict(freq=None), "NULL"),
    (dict(x_ld=191), {}, "ARG"), (dict(y_ld=191), {}, "ARG"), (dict(T=2), dict(n_axes=2), "ARG"),
    (dict(x=P + 2), {}, "ARG"), (dict(dtype=1, y=P + 1), {}, "ARG"), (dict(positions=P + 2), {}, "ARG"),
    ({}, dict(freq=P + 1), "ARG"), ({}, dict(q_norm=P + 2), "ARG"), ({}, dict(k_norm=P + 2), "ARG"),
    (dict(y=P, y_ld=256), {}, "ARG"), (dict(T=0, x=None), {}, "OK")])
def test_rope_refusals(L, change, of_rope, code):  # noqa: F811
    want = L.E0_OK if code == "OK" else getattr(L, "E0_ERR_" + code)
    assert call(L.e0_qk_rope, dict(ROPE, rope=rope(L, **of_rope)), **change) == want


def test_rope_wants_a_description(L):  # noqa: F811
    assert L.load().e0_qk_rope(P, 0, 192, 1, 2, 1, None, P, 1, P, 192, None, None) == L.E0_ERR_NULL


SAMPLE = dict(x=P, dtype=0, ld=100, T=2, V=100, rules=None, u=P, token=P, logp=None, kept=None, status=None)


@pytest.mark.parametrize("change,code", [
    (dict(T=-1), "ARG"), (dict(V=0), "ARG"), (dict(dtype=3), "ARG"), (dict(V=(1 << 18) + 1, ld=1 << 19), "UNSUPPORTED"),
    (dict(T=(1 << 24) + 1), "UNSUPPORTED"), (dict(x=None), "NULL"), (dict(u=None), "NULL"), (dict(token=None), "NULL"),
    (dict(ld=99), "ARG"), (dict(x=P + 2), "ARG"), (dict(dtype=2, x=P + 1), "ARG"), (dict(u=P + 2), "ARG"),
    (dict(token=P + 2), "ARG"), (dict(logp=P + 1), "ARG"), (dict(kept=P + 1), "ARG"), (dict(T=0, x=None), "OK")])
def test_sample_refusals(L, change, code):  # noqa: F811
    want = L.E0_OK if code == "OK" else getattr(L, "E0_ERR_" + code)
    assert call(L.e0_sample, SAMPLE, **change) == want


@pytest.mark.parametrize("field", ["temperature", "top_k", "top_p", "min_p"])
def test_sample_refuses_rules_that_do_not_align(L, field):  # noqa: F811
    rules = L.Sampling(**{field: P + 2})
    assert call(L.e0_sample, SAMPLE, rules=rules) == L.E0_ERR_ARG
