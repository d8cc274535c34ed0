"""Host-side argument checks of the operators around the MoE block: every
refusal comes before a launch, so a CPU is enough."""
import os

import numpy as np
import pytest

from tests.layer_ref import E4M3, decode, encode, pow2_scale

P = 4096  # an address that is never read


@pytest.fixture(scope="module")
def L():
    from int4_gathered_expert_gb300 import build, lib
    if not os.path.exists(lib.LIB_PATH):
        try:
            build.nvcc()
        except RuntimeError:
            pytest.skip("nvcc unavailable and the library is not built")
        build.build()
    lib.load()
    return lib


def call(fn, base, **change):
    names = list(base)
    assert set(change) <= set(names)
    return fn(*[change.get(n, base[n]) for n in names], stream=0, raise_on_error=False)


NORM = dict(r=P, d=None, w=None, T=1, H=64, dtype=0, eps=1e-6, r_ld=64, d_ld=0, r_out=None, h=2 * P, q=None,
            q_scale=None, status=None)


@pytest.mark.parametrize("change,code", [
    (dict(T=-1), "ARG"), (dict(H=0), "ARG"), (dict(dtype=3), "ARG"), (dict(dtype=-1), "ARG"), (dict(eps=-1.0), "ARG"),
    (dict(eps=float("nan")), "ARG"), (dict(H=16385, r_ld=16385), "UNSUPPORTED"), (dict(T=(1 << 30) + 1), "UNSUPPORTED"),
    (dict(r=None), "NULL"),
    (dict(h=None), "NULL"), (dict(q=P), "NULL"), (dict(q_scale=P), "NULL"), (dict(r_ld=63), "ARG"),
    (dict(d=3 * P, d_ld=63), "ARG"), (dict(r=P + 2), "ARG"), (dict(dtype=1, r=P + 1), "ARG"), (dict(w=P + 2), "ARG"),
    (dict(h=P), "ARG"), (dict(d=2 * P, d_ld=64), "ARG"), (dict(r_out=2 * P), "ARG"),
    (dict(r_out=P, r_ld=128), "ARG"), (dict(d=3 * P, d_ld=65, r_out=3 * P), "ARG"), (dict(T=0, r=None), "OK")])
def test_norm_refusals(L, change, code):
    want = L.E0_OK if code == "OK" else getattr(L, "E0_ERR_" + code)
    assert call(L.e0_rmsnorm_q8, NORM, **change) == want


LIN = dict(w=P, N=64, K=128, x=P, x_type=0, x_ld=128, x_scale=None, T=1, add=None, add_ld=0, y=2 * P, y_type=0,
           y_ld=64)


@pytest.mark.parametrize("change,code", [
    (dict(T=-1), "ARG"), (dict(N=0), "ARG"), (dict(K=0), "ARG"), (dict(K=100), "ARG"), (dict(x_type=4), "ARG"),
    (dict(y_type=3), "ARG"), (dict(w=None), "NULL"), (dict(x=None), "NULL"), (dict(y=None), "NULL"),
    (dict(x_type=3), "NULL"), (dict(x_ld=127), "ARG"), (dict(y_ld=63), "ARG"), (dict(add=P, add_ld=63), "ARG"),
    (dict(w=P + 8), "ARG"), (dict(x=P + 2), "ARG"), (dict(y=P + 2), "ARG"), (dict(add=2 * P, add_ld=65), "ARG"),
    (dict(x_type=3, x_scale=P + 1), "ARG"), (dict(T=524281), "UNSUPPORTED"),
    (dict(K=(1 << 20) + 64, x_ld=1 << 21), "UNSUPPORTED"), (dict(N=(1 << 28) + 1, y_ld=1 << 29), "UNSUPPORTED"),
    (dict(T=0, x=None), "OK")])
def test_linear_refusals(L, change, code):
    want = L.E0_OK if code == "OK" else getattr(L, "E0_ERR_" + code)
    assert call(L.e0_linear_forward, LIN, **change) == want


def test_pack_linear_refusals_and_sizes(L):
    assert L.e0_linear_bytes(1, 64) == L.e0_linear_bytes(128, 64) == 8 * 576
    assert L.e0_linear_bytes(129, 128) == 2 * 2 * 8 * 576
    assert L.e0_linear_bytes(131072, 8192) == 8192 * 128 * 576
    for n, k in ((0, 64), (1, 0), (1, 63), (-1, 64), ((1 << 28) + 1, 64), (1, (1 << 20) + 64)):
        assert L.e0_linear_bytes(n, k) == 0
    q = L.QTensor(P, P, P)
    no = dict(stream=0, raise_on_error=False)
    assert L.e0_pack_linear(L.QTensor(None, P, P), 16, 64, P, **no) == L.E0_ERR_NULL
    assert L.e0_pack_linear(L.QTensor(P, P, None), 16, 64, P, **no) == L.E0_ERR_NULL
    assert L.e0_pack_linear(q, 16, 64, None, **no) == L.E0_ERR_NULL
    assert L.e0_pack_linear(q, 0, 64, P, **no) == L.E0_ERR_ARG
    assert L.e0_pack_linear(q, 16, 65, P, **no) == L.E0_ERR_ARG
    assert L.e0_pack_linear(q, (1 << 28) + 1, 64, P, **no) == L.E0_ERR_UNSUPPORTED
    assert L.e0_pack_linear(q, 16, 64, P + 8, **no) == L.E0_ERR_ARG
    assert L.e0_pack_linear(L.QTensor(P, P + 1, P), 16, 64, P, **no) == L.E0_ERR_ARG


FIRST = r"""
#include <cstdio>
#include "e0_first.h"
int main() {
    e0::FirstAnswer<9> a;
    int asked = 0;
    const auto says = [&](int n) { return [&asked, n]() { ++asked; return n; }; };
    printf("%d ", a.get(0, 3, 38, says(0)));    // no answer: the other number
    printf("%d ", a.get(0, 3, 38, says(50)));   // ... and the same one ever after
    printf("%d ", a.get(0, 4, 38, says(50)));   // another question
    printf("%d ", a.get(1, 3, 38, says(44)));   // another device
    printf("%d ", a.get(1, 3, 38, says(45)));
    printf("%d %d ", a.get(-1, 3, 38, says(50)), a.get(64, 3, 38, says(50)));
    printf("%d ", a.get(2, 3, 38, [&]() { return a.get(2, 3, 38, says(41)) + 1; }));  // the answer of a call in between
    printf("%d\n", asked);
}
"""


def test_the_first_answer_for_a_device_stays(tmp_path):
    """How many parts K is split into, and so the order of the linear's sums, goes by what the runtime said first."""
    import shutil
    import subprocess
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host compiler")
    (tmp_path / "first.cpp").write_text(FIRST)
    csrc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "int4_gathered_expert_gb300", "csrc")
    exe = str(tmp_path / "first")
    subprocess.run([cxx, "-std=c++17", "-I", csrc, str(tmp_path / "first.cpp"), "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True, check=True).stdout
    assert out.split() == ["38", "38", "50", "44", "44", "38", "38", "41", "4"]


def state(L, **c):
    f = dict(block_table=P, ctx_len=P, free_list=P, free_count=P, B=2, max_blocks=4, block_tokens=16, n_blocks=8)
    f.update(c)
    return L.KvState(*f.values())


@pytest.mark.parametrize("change,code", [
    (dict(B=-1), "ARG"), (dict(max_blocks=0), "ARG"), (dict(n_blocks=0), "ARG"), (dict(block_tokens=8), "ARG"),
    (dict(block_tokens=48), "ARG"), (dict(B=4097), "UNSUPPORTED"), (dict(block_table=None), "NULL"),
    (dict(max_blocks=(1 << 26) + 1), "UNSUPPORTED"), (dict(n_blocks=(1 << 30) + 1), "UNSUPPORTED"),
    (dict(ctx_len=None), "NULL"), (dict(free_list=None), "NULL"), (dict(free_count=None), "NULL"),
    (dict(ctx_len=P + 2), "ARG")])
def test_plan_and_release_refuse_a_bad_state(L, change, code):
    s = state(L, **change)
    want = getattr(L, "E0_ERR_" + code)
    assert L.e0_kv_plan(s, P, 4, P, P, P, P, stream=0, raise_on_error=False) == want
    assert L.e0_kv_release(s, P, P, P, stream=0, raise_on_error=False) == want


def test_plan_and_release_refusals(L):
    s = state(L)
    no = dict(stream=0, raise_on_error=False)
    assert L.e0_kv_plan(s, P, -1, P, P, P, P, **no) == L.E0_ERR_ARG
    assert L.e0_kv_plan(s, P, (1 << 30) + 1, P, P, P, P, **no) == L.E0_ERR_UNSUPPORTED
    assert L.e0_kv_plan(s, None, 4, P, P, P, P, **no) == L.E0_ERR_NULL
    assert L.e0_kv_plan(s, P, 4, None, P, P, P, **no) == L.E0_ERR_NULL
    assert L.e0_kv_plan(s, P, 4, P, None, P, P, **no) == L.E0_ERR_NULL
    assert L.e0_kv_plan(s, P, 4, P, P, None, P, **no) == L.E0_ERR_NULL
    assert L.e0_kv_plan(s, P, 4, P, P, P, None, **no) == L.E0_ERR_NULL
    assert L.e0_kv_plan(s, P, 4, P, P, P, P + 4, **no) == L.E0_ERR_ARG
    assert L.e0_kv_plan(s, P, 4, P, P, P, P, P + 1, **no) == L.E0_ERR_ARG
    assert L.e0_kv_release(s, None, P, P, **no) == L.E0_ERR_NULL
    assert L.e0_kv_release(s, P, P, None, **no) == L.E0_ERR_NULL
    assert L.load().e0_kv_plan(None, P, 4, P, P, P, P, None, None, None, None) == L.E0_ERR_NULL


def cache(L, **c):
    f = dict(k=P, v=P, k_scale=P, v_scale=P, n_blocks=4, Hkv=2, block_tokens=16, D=64)
    f.update(c)
    return L.KvCache(*f.values())


@pytest.mark.parametrize("change,code", [
    (dict(k=None), "NULL"), (dict(v_scale=None), "NULL"), (dict(n_blocks=0), "ARG"), (dict(Hkv=0), "ARG"),
    (dict(Hkv=32768), "UNSUPPORTED"), (dict(block_tokens=24), "UNSUPPORTED"), (dict(D=96), "UNSUPPORTED"),
    (dict(D=512), "UNSUPPORTED"),
    (dict(v=P + 8), "ARG"), (dict(k_scale=P + 2), "ARG")])
def test_append_and_attention_refuse_a_bad_cache(L, change, code):
    c = cache(L, **change)
    want = getattr(L, "E0_ERR_" + code)
    assert L.e0_kv_append(c, P, P, 0, 1024, 1024, P, 4, stream=0, raise_on_error=False) == want
    assert call(L.e0_attn_decode, dict(ATT, cache=c, Hq=2 * max(c.Hkv, 1))) == want


APP = dict(k=P, v=P, dtype=0, k_ld=128, v_ld=128, slots=P, T=4)


@pytest.mark.parametrize("change,code", [
    (dict(T=-1), "ARG"), (dict(dtype=3), "ARG"), (dict(k=None), "NULL"), (dict(v=None), "NULL"),
    (dict(slots=None), "NULL"), (dict(k_ld=127), "ARG"), (dict(v_ld=0), "ARG"), (dict(k=P + 2), "ARG"),
    (dict(slots=P + 4), "ARG"), (dict(T=0, k=None), "OK"), (dict(T=(1 << 30) + 1), "UNSUPPORTED")])
def test_append_refusals(L, change, code):
    want = L.E0_OK if code == "OK" else getattr(L, "E0_ERR_" + code)
    c = cache(L)
    assert call(lambda *a, **k: L.e0_kv_append(c, *a, **k), APP, **change) == want


ATT = dict(cache=None, block_table=P, max_blocks=4, ctx_len=P, cu_q=P, B=2, max_q=1, q=P, dtype=1, q_ld=256, Hq=4,
           scale=1.0, window=0, out=P, out_ld=256, lse=None, ws=P, ws_bytes=1 << 30, status=None)


@pytest.mark.parametrize("change,code", [
    (dict(B=-1), "ARG"), (dict(max_blocks=0), "ARG"), (dict(max_q=0), "ARG"), (dict(dtype=3), "ARG"),
    (dict(window=-1), "ARG"), (dict(Hq=3), "ARG"), (dict(Hq=1), "ARG"), (dict(scale=float("nan")), "ARG"),
    (dict(cu_q=None, max_q=2), "ARG"), (dict(B=4097), "UNSUPPORTED"), (dict(max_q=1 << 30), "UNSUPPORTED"),
    (dict(max_blocks=(1 << 26) + 1), "UNSUPPORTED"), (dict(block_table=None), "NULL"), (dict(ctx_len=None), "NULL"),
    (dict(q=None), "NULL"), (dict(out=None), "NULL"),
    (dict(ws=None), "NULL"), (dict(q_ld=255), "ARG"), (dict(q_ld=257), "ARG"), (dict(out_ld=255), "ARG"),
    (dict(q=P + 8), "ARG"), (dict(out=P + 1), "ARG"), (dict(lse=P + 2), "ARG"), (dict(ws=P + 128), "ARG"),
    (dict(ws_bytes=1), "ARG"), (dict(B=0, q=None), "OK")])
def test_attention_refusals(L, change, code):
    want = L.E0_OK if code == "OK" else getattr(L, "E0_ERR_" + code)
    assert call(L.e0_attn_decode, dict(ATT, cache=cache(L)), **change) == want


def test_attention_workspace_sizes(L):
    assert L.e0_attn_workspace_size(1, 8, 2, 128, 1) > 0
    for bad in ((0, 8, 2, 128, 1), (1, 8, 3, 128, 1), (1, 1, 2, 128, 1), (1, 8, 2, 96, 1), (1, 8, 2, 128, 0),
                (5000, 8, 2, 128, 1)):
        assert L.e0_attn_workspace_size(*bad) == 0


def test_reference_number_format():
    assert len(E4M3) == 127 and E4M3[-1] == 448 and E4M3[1] == 2.0 ** -9 and E4M3[8] == 2.0 ** -6
    c = np.arange(256).astype(np.uint8)
    num = (c & 127) != 127
    assert np.array_equal(encode(decode(c))[num], c[num])
    assert encode(np.array([1e9]))[0] == 126 and encode(np.array([2.0 ** -10]))[0] == 0  # tie to even
    assert encode(np.array([17.0]))[0] == encode(np.array([16.0]))[0]                    # tie to even
    assert pow2_scale(448) == 1 and pow2_scale(449) == 2 and pow2_scale(0) == 2.0 ** -100
    torch = pytest.importorskip("torch")
    x = torch.randn(4096, dtype=torch.float64, generator=torch.Generator().manual_seed(1)) * 50
    assert np.array_equal(encode(x.float().double().numpy()), x.float().to(torch.float8_e4m3fn).view(torch.uint8).numpy())
