"""Rotation, score rules, a prefix in common and sampling together, as a batch's generation
uses them (BatchDecoder, KvCacheDev.share, QkRope, Sampler): every stage against a 64-bit reference fed
with what the stage before left, and captured steps against eager ones."""
import numpy as np
import pytest

from int4_gathered_expert_gb300 import synth
from tests import layer_ref as R
from tests.test_attn_rules import compare, rules_ref
from tests.test_batch_decoder import L, f64  # noqa: F401
from tests.test_layer_ops import EPS, F16, H, TINY16
from tests.test_token_ops import rope_ref, row_ref

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def parts(n_layers, a, seed=21):
    from int4_gathered_expert_gb300.model import StackDev
    shape = synth.StackShape(layer=synth.TINY, n_layers=n_layers, owners=(), shared_expert=True, seed=seed)
    m = synth.stack_model(shape, n_tokens=1, threads=2)
    return StackDev(m), [synth.attention(seed, l, synth.TINY.H, a) for l in range(n_layers)]


def freqs(D, base=100.0):
    return (base ** (-np.arange(D // 2) / (D // 2))).astype(np.float32)


def held(c, layer):
    """The cache's codes and scales as the reference's cache."""
    ref = R.Cache(c.n_blocks, c.k.shape[2], c.block_tokens, c.k.shape[4])
    ref.k, ref.v = c.k[layer].cpu().numpy(), c.v[layer].cpu().numpy()
    ref.ks, ref.vs = c.k_scale[layer].cpu().numpy(), c.v_scale[layer].cpu().numpy()
    return ref


@pytest.mark.parametrize("prefix_tokens", [0, 9, 40])
@pytest.mark.parametrize("rules", ["none", "cap", "slopes"])
def test_steps_behind_a_prefix(L, prefix_tokens, rules):  # noqa: F811
    """One layer: a sequence becomes the prefix, the others go on behind it; queries and keys are normed and turned at
    positions that count the prefix, and what attention gives is that of prefix and own tokens."""
    from int4_gathered_expert_gb300.model import BatchDecoder, KvCacheDev, QkRope
    a = synth.AttnShape(Hq=6, Hkv=2, D=64, block_tokens=16)
    B, T, Hh = 4, 40, synth.TINY.H
    rng = np.random.default_rng(prefix_tokens)
    sd, attn = parts(1, a)
    cache = KvCacheDev(1, B, 40, 8, a.Hkv, a.D, a.block_tokens)
    qn, kn = 1 + 0.2 * rng.standard_normal(64).astype(np.float32), 1 + 0.2 * rng.standard_normal(64).astype(np.float32)
    rope, seen = QkRope(a, freqs(64), 1, q_norm=[qn], k_norm=[kn]), []

    def edit(layer, qkv, positions):
        was = qkv.clone()
        rope(layer, qkv, positions)
        seen.append((was, qkv.clone(), positions.clone()))

    kw = dict(cap=3.0 if rules == "cap" else 0.0, slopes=0.05 * np.arange(1, 7) if rules == "slopes" else None)
    bd = BatchDecoder(sd, attn, a, cache, T, edit=edit, prefix=True, **kw)

    def x():
        return torch.from_numpy(rng.standard_normal((T, Hh)).astype(np.float32)).cuda()

    def lens(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    if prefix_tokens:
        bd.step(x(), lens([0, 0, prefix_tokens, 0]))
        assert cache.ctx.tolist() == [0, 0, prefix_tokens, 0]
        cache.share(2)
    assert cache.prefix_len.tolist() == [prefix_tokens] and cache.ctx.tolist() == [0] * B
    ctx = np.zeros(B, int)
    for new in ([1, 3, 0, 20], [1, 1, 1, 1], [0, 2, 5, 1]):
        seen.clear()
        bd.step(x(), lens(new))
        assert L.e0_read_status(bd.status) == 0 and L.e0_read_status(rope.status) == 0
        ctx += new
        n = sum(new)
        cu = np.concatenate([[0], np.cumsum(new)])
        at = np.concatenate([prefix_tokens + ctx[b] - new[b] + np.arange(new[b]) for b in range(B)])
        was, qkv, positions = seen[0]
        assert positions.tolist() == list(at) + [-1] * (T - n)
        # norms and rotation
        heads = f64(was)[:n, :8 * 64].reshape(n, 8, 64)
        want, tol = rope_ref(heads, 6, at[None].astype(np.int32), freqs(64), np.zeros(32, int), 64, False, True, qn.astype(
            np.float64), kn.astype(np.float64), 1e-6)
        got = f64(qkv)[:n, :8 * 64].reshape(n, 8, 64)
        assert (np.abs(got - want) <= tol + H[F16] * np.abs(want) * 1.0001 + TINY16[F16]).all()
        assert torch.equal(qkv[:, 8 * 64:], was[:, 8 * 64:]) and torch.equal(qkv[n:], was[n:])
        # attention over prefix and own tokens
        ref, table = held(cache, 0), cache.table.cpu().numpy()
        pk, pv = ref.row(cache.prefix_table[0].cpu().numpy(), prefix_tokens)
        o = f64(bd.o).reshape(T, 6, 64)
        for b in range(B):
            if not new[b]:
                continue
            k, v = ref.row(table[b], int(ctx[b]))
            k, v = np.concatenate([pk, k]), np.concatenate([pv, v])
            p = prefix_tokens + ctx[b] - new[b] + np.arange(new[b])
            sees = np.arange(len(k))[None, :] <= p[:, None]
            sl = None if kw["slopes"] is None else kw["slopes"].astype(np.float32).astype(np.float64)
            w_o, w_l, tol, ltol = rules_ref(got[cu[b]:cu[b + 1], :6], k, v, float(np.float32(0.125)), p, sees, kw["cap"], sl,
                                            2.0 ** -21 + 16 * EPS, 2.0 ** -24 * 448 * float(ref.vs.max()))
            tol = tol + 16 * EPS * np.abs(w_l)[:, :, None] * np.abs(v).max()
            compare(o[cu[b]:cu[b + 1]], None, (w_o, w_l, tol, ltol), F16, (b, new))
        assert (o[n:] == 0).all()
    # another prefix in the place of this one, whose blocks are free again
    cache.release(torch.ones(B, dtype=torch.uint8, device="cuda"), bd.status)
    bd.step(x(), lens([0, 17, 0, 0]))
    cache.share(1)
    assert cache.prefix_len.tolist() == [17] and cache.free_count.tolist() == [38] and cache.ctx.tolist() == [0] * B
    # everything goes back
    cache.release(torch.ones(B, dtype=torch.uint8, device="cuda"), bd.status)
    cache.unshare(bd.status)
    assert L.e0_read_status(bd.status) == 0 and cache.free_count.tolist() == [40] and cache.prefix_len.tolist() == [0]
    assert sorted(cache.free.tolist()) == list(range(40))


def test_capped_steps_without_a_prefix(L):  # noqa: F811
    from int4_gathered_expert_gb300.model import BatchDecoder, KvCacheDev
    a = synth.AttnShape(Hq=4, Hkv=2, D=64, block_tokens=16)
    B, T = 2, 6
    sd, attn = parts(1, a)
    cache = KvCacheDev(1, B, 20, 6, a.Hkv, a.D, 16)
    bd = BatchDecoder(sd, attn, a, cache, T, cap=2.0)
    rng = np.random.default_rng(4)
    ctx = np.zeros(B, int)
    for new in ([4, 2], [1, 1], [0, 6]):
        bd.step(torch.from_numpy(rng.standard_normal((T, 256)).astype(np.float32)).cuda(), torch.tensor(
            new, dtype=torch.int32, device="cuda"), window=5)
        ctx += new
        cu = np.concatenate([[0], np.cumsum(new)])
        ref, table, o = held(cache, 0), cache.table.cpu().numpy(), f64(bd.o).reshape(T, 4, 64)
        q = f64(bd.x_qkv)[:, :256].reshape(T, 4, 64)
        for b in range(B):
            if not new[b]:
                continue
            k, v = ref.row(table[b], int(ctx[b]))
            p, j = ctx[b] - new[b] + np.arange(new[b]), np.arange(ctx[b])
            sees = (j[None] <= p[:, None]) & (j[None] > p[:, None] - 5)
            compare(o[cu[b]:cu[b + 1]], None, rules_ref(q[cu[b]:cu[b + 1]], k, v, 0.125, p, sees, 2.0), F16, (b, new))
    assert L.e0_read_status(bd.status) == 0


def test_generation_captured_and_eager(L):  # noqa: F811
    """Whole tokens: embedding, two layers behind a prefix, logits, a draw, the next embedding; a captured step replayed
    gives the tokens that eager ones give, and each draw is the definition's."""
    from int4_gathered_expert_gb300.model import BatchDecoder, KvCacheDev, LinearDev, QkRope, Sampler
    a = synth.AttnShape(Hq=8, Hkv=2, D=64, block_tokens=16)
    B, V, Hh = 5, 3001, synth.TINY.H
    g = np.random.default_rng(6)
    embed = torch.from_numpy(g.standard_normal((V, Hh)).astype(np.float32)).cuda()
    head = LinearDev(synth.qtensor(np.random.default_rng(8), V, Hh))
    runs = []
    for captured in (False, True):
        sd, attn = parts(2, a)
        cache = KvCacheDev(2, B, 64, 8, a.Hkv, a.D, 16)
        rope = QkRope(a, freqs(64), 2, adjacent=True)
        first = BatchDecoder(sd, attn, a, cache, 32, edit=rope, prefix=True)
        bd = BatchDecoder(sd, attn, a, cache, B, edit=rope, prefix=True)
        rng = np.random.default_rng(7)
        first.step(embed[torch.from_numpy(rng.integers(0, V, 32)).cuda()], torch.tensor([29, 0, 0, 0, 0], dtype=torch.int32,
                                                                                     device="cuda"))
        cache.share(0)
        temp, top_p = torch.full((B,), 0.8, device="cuda"), torch.full((B,), 0.9, device="cuda")
        top_k = torch.full((B,), 200, dtype=torch.int32, device="cuda")
        sample = Sampler(B, V, temperature=temp, top_k=top_k, top_p=top_p)
        one = torch.ones(B, dtype=torch.int32, device="cuda")
        u, x, logits = torch.zeros(B, device="cuda"), torch.zeros((B, Hh), device="cuda"), torch.zeros((B, V), device="cuda")
        sample.tokens.copy_(torch.arange(B, dtype=torch.int32))

        def step():
            torch.index_select(embed, 0, sample.tokens, out=x)
            r = bd.step(x, one)
            L.e0_linear_forward(head.data, V, Hh, r, L.E0_F32, Hh, None, B, None, 0, logits, L.E0_F32, V)
            sample(logits, u)

        us = np.random.default_rng(9).random((12, B)).astype(np.float32)
        said, graph = [], None
        for i in range(12):
            u.copy_(torch.from_numpy(us[i]))
            if captured and i == 2:
                torch.cuda.synchronize()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    step()
            graph.replay() if graph else step()
            said.append(sample.tokens.tolist())
            for t in range(B):
                tok, logp, n, near = row_ref(f64(logits)[t], float(us[i, t]), float(np.float32(0.8)), 200, float(np.float32(0.9)))
                if near > 2.0 ** -26:
                    assert said[-1][t] == tok and int(sample.kept[t]) == n
        assert L.e0_read_status(bd.status) == 0 and L.e0_read_status(sample.status) == 0
        assert cache.ctx.tolist() == [12] * B and cache.prefix_len.tolist() == [29]
        runs.append(said)
    assert runs[0] == runs[1] and len({tuple(r) for r in runs[0]}) > 3


def test_what_does_not_fit_is_refused(L):  # noqa: F811
    from int4_gathered_expert_gb300.model import BatchDecoder, KvCacheDev, QkRope, Sampler
    a = synth.AttnShape(Hq=4, Hkv=2, D=64, block_tokens=16)
    sd, attn = parts(1, a)
    cache = KvCacheDev(1, 2, 8, 4, a.Hkv, a.D, 16)
    for kw in (dict(cap=-1.0), dict(cap=float("inf")), dict(slopes=np.ones(3))):
        with pytest.raises(ValueError):
            BatchDecoder(sd, attn, a, cache, 2, **kw)
    with pytest.raises(ValueError):
        cache.share(2)
    with pytest.raises(ValueError):
        QkRope(a, freqs(64), 1, q_norm=[np.ones(63, np.float32)])
    with pytest.raises(ValueError):
        QkRope(a, freqs(64), 1, axis=np.full(32, 2), n_axes=2)
    rope = QkRope(a, freqs(64))
    pos = torch.zeros(3, dtype=torch.int32, device="cuda")
    for qkv in (torch.zeros((3, 512), device="cuda"), torch.zeros((3, 500), dtype=torch.float16, device="cuda")):
        with pytest.raises(ValueError):
            rope(0, qkv, pos)
    with pytest.raises(ValueError):
        rope(0, torch.zeros((2, 512), dtype=torch.float16, device="cuda"), pos)
    with pytest.raises(ValueError):
        Sampler(3, 10, top_k=torch.zeros(3, device="cuda"))
    sample = Sampler(3, 10)
    with pytest.raises(ValueError):
        sample(torch.zeros((3, 11), device="cuda"), torch.zeros(3, device="cuda"))
    with pytest.raises(ValueError):
        sample(torch.zeros((3, 10), device="cuda"), torch.zeros(3, dtype=torch.float64, device="cuda"))
