"""The attention half and the MoE half of layers together (BatchDecoder): every
stage against a 64-bit reference fed with what the stage before left, sequences
that come, grow, end and come again, a captured step, a pool that runs out."""
import os

import numpy as np
import pytest

from int4_gathered_expert_gb300 import synth
from oracle import e0_oracle as O
from tests import layer_ref as R
from tests.parity import REL_L2, rel_l2

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

EPS = 2.0 ** -23


@pytest.fixture(scope="module")
def L():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from int4_gathered_expert_gb300 import build, lib
    if not os.path.exists(lib.LIB_PATH):
        build.build()
    lib.load()
    return lib


def decoder(n_layers, B, T, n_blocks, max_blocks, a, seed=21, shared=True):
    from int4_gathered_expert_gb300.model import BatchDecoder, KvCacheDev, StackDev
    shape = synth.StackShape(layer=synth.TINY, n_layers=n_layers, owners=(), shared_expert=shared, seed=seed)
    m = synth.stack_model(shape, n_tokens=1, threads=2)
    attn = [synth.attention(seed, l, synth.TINY.H, a) for l in range(n_layers)]
    cache = KvCacheDev(n_layers, B, n_blocks, max_blocks, a.Hkv, a.D, a.block_tokens)
    return m, attn, BatchDecoder(StackDev(m), attn, a, cache, T)


def f64(t):
    return t.double().cpu().numpy()


def codes_of(t):
    return R.decode(t.cpu().numpy())


def test_one_layer_stage_by_stage(L):
    a = synth.AttnShape(Hq=6, Hkv=2, D=64, block_tokens=16)
    B, T, H = 3, 12, synth.TINY.H
    m, attn, bd = decoder(1, B, T, 24, 12, a)
    c = bd.cache
    ref = R.Cache(24, a.Hkv, 16, a.D)
    ref.k, ref.v = c.k[0].cpu().numpy(), c.v[0].cpu().numpy()
    rng = np.random.default_rng(3)
    ctx = np.zeros(B, int)
    for new in ([7, 3, 0], [1, 1, 1], [0, 1, 9], [1, 1, 1], [5, 0, 1]):
        x = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).cuda()
        out = bd.step(x, torch.tensor(new, dtype=torch.int32, device="cuda"))
        assert L.e0_read_status(bd.status) == 0
        n = sum(new)
        ctx += new
        assert c.ctx.tolist() == list(ctx)
        # the norm's codes and scales give h back to half a step
        xv = f64(x)
        h = xv / np.sqrt((xv ** 2).mean(1, keepdims=True) + 1e-6) * attn[0]["norm"].astype(np.float64)
        hq = (codes_of(bd.q8).reshape(T, -1, 64) * f64(bd.q8_scale)[:, :, None]).reshape(T, H)
        step = np.maximum(np.abs(h) * 2.0 ** -4, np.repeat(f64(bd.q8_scale), 64, 1) * 2.0 ** -10)
        assert (np.abs(hq - h) <= step * (1 + 1e-4) + 1e-5 * np.abs(h)).all()
        # queries, keys, values: fp32 sums of exact products, one rounding to fp16
        W = O.dequant(attn[0]["qkv"])
        want = hq @ W.T
        mag = np.abs(hq) @ (15 * np.repeat(attn[0]["qkv"]["scale"].astype(np.float64), 64, 1)
                            + np.abs(np.repeat(attn[0]["qkv"]["bias"].astype(np.float64), 64, 1))).T
        qkv = f64(bd.x_qkv)
        assert (np.abs(qkv - want) <= 90 * EPS * mag + 2.0 ** -11 * np.abs(want) * 1.001 + 2.0 ** -25).all()
        # the cache holds them
        slots = bd.slots.cpu().numpy()
        assert (slots[n:] == -1).all()
        k = qkv[:, a.Hq * a.D:(a.Hq + a.Hkv) * a.D].reshape(T, a.Hkv, a.D)
        v = qkv[:, (a.Hq + a.Hkv) * a.D:].reshape(T, a.Hkv, a.D)
        ref.append(k, v, slots)
        used = np.unique(slots[:n] // 16)
        assert np.array_equal(codes_of(c.k[0]), R.decode(ref.k)) and np.array_equal(codes_of(c.v[0]), R.decode(ref.v))
        assert np.array_equal(c.k_scale[0].cpu().numpy()[used], ref.ks[used])
        # attention over it
        table, cu = c.table.cpu().numpy(), bd.cu_q.cpu().numpy()
        o = f64(bd.o).reshape(T, a.Hq, a.D)
        for b in range(B):
            if new[b]:
                kk, vv = ref.row(table[b], ctx[b])
                q = qkv[cu[b]:cu[b + 1], :a.Hq * a.D].reshape(-1, a.Hq, a.D)
                wo, _, tol, _ = R.attention(q, kk, vv, float(np.float32(a.D ** -0.5)), ctx[b], 0)
                assert (np.abs(o[cu[b]:cu[b + 1]] - wo) <= tol + 2.0 ** -11 * np.abs(wo) * 1.001 + 2.0 ** -25).all()
        # back onto the stream, and the MoE half
        r = xv + f64(bd.o) @ O.dequant(attn[0]["out"]).T
        assert rel_l2(f64(bd.r)[:n], r[:n]) <= 1e-5
        hh = O.rmsnorm(f64(bd.r)[:n])
        y = O.moe_block(hh, O.BankExperts(m.banks[0]), bd.inds.cpu().numpy()[:n], f64(bd.w)[:n], m.shared[0])
        assert rel_l2(f64(bd.y)[:n], y) <= REL_L2
        assert torch.equal(out, bd.r + bd.y)


def decoder_with(edit, n_layers, B, T, n_blocks, max_blocks, a):
    """The same as decoder's, with an edit."""
    from int4_gathered_expert_gb300.model import BatchDecoder, KvCacheDev
    _, attn, bd = decoder(n_layers, B, T, n_blocks, max_blocks, a)
    cache = KvCacheDev(n_layers, B, n_blocks, max_blocks, a.Hkv, a.D, a.block_tokens)
    return BatchDecoder(bd.sd, attn, a, cache, T, edit=edit)


def rotary(a, base=100.0):
    """Rotary embeddings of queries and keys, as an edit of BatchDecoder."""
    freq = base ** (-torch.arange(a.D // 2, device="cuda", dtype=torch.float64) / (a.D // 2))

    def edit(layer, qkv, positions):
        angle = positions.clamp(min=0).double()[:, None, None] * freq * (layer + 1)
        n = (a.Hq + a.Hkv) * a.D
        x = qkv[:, :n].reshape(len(qkv), -1, 2, a.D // 2).double()
        c, s = angle.cos(), angle.sin()
        out = torch.stack([x[:, :, 0] * c - x[:, :, 1] * s, x[:, :, 1] * c + x[:, :, 0] * s], 2)
        qkv[:, :n] = out.reshape(len(qkv), n).half()

    return edit


@pytest.mark.parametrize("how", ["current", "stream"])
def test_rotary_embeddings_between_projection_and_cache(L, how):
    """What the edit leaves is what is cached and asked with; it sees each row's position, and the step's stream."""
    a = synth.AttnShape(Hq=4, Hkv=2, D=64, block_tokens=16)
    B, T, H = 2, 9, synth.TINY.H
    seen, rope = [], rotary(a)

    def edit(layer, qkv, positions):
        was = qkv.clone()
        rope(layer, qkv, positions)
        seen.append((layer, was, qkv.clone(), positions.clone(), torch.cuda.current_stream().cuda_stream))

    stream = torch.cuda.Stream() if how == "stream" else None
    bd = decoder_with(edit, 2, B, T, 12, 6, a)
    _, _, plain = decoder(2, B, T, 12, 6, a)
    c = bd.cache
    ref = [R.Cache(12, a.Hkv, 16, a.D) for _ in range(2)]
    rng = np.random.default_rng(8)
    ctx = np.zeros(B, int)
    for new in ([5, 3], [1, 1], [8, 0], [0, 9], [1, 1]):
        x = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).cuda()
        lens = torch.tensor(new, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        seen.clear()
        bd.step(x, lens, stream=stream)
        torch.cuda.synchronize()
        assert L.e0_read_status(bd.status) == 0 and [e[0] for e in seen] == [0, 1]
        n = sum(new)
        want = [int(ctx[b]) + i for b in range(B) for i in range(new[b])] + [-1] * (T - n)
        ctx += new
        slots, table, cu = bd.slots.cpu().numpy(), c.table.cpu().numpy(), bd.cu_q.cpu().numpy()
        for layer, was, qkv, pos, on in seen:
            assert pos.tolist() == want
            assert on == (stream or torch.cuda.current_stream()).cuda_stream
            v = f64(qkv)
            ref[layer].append(v[:, a.Hq * a.D:(a.Hq + a.Hkv) * a.D].reshape(T, a.Hkv, a.D),
                              v[:, (a.Hq + a.Hkv) * a.D:].reshape(T, a.Hkv, a.D), slots)
            assert np.array_equal(codes_of(c.k[layer]), R.decode(ref[layer].k))
            assert np.array_equal(codes_of(c.v[layer]), R.decode(ref[layer].v))
        o, q = f64(bd.o).reshape(T, a.Hq, a.D), f64(seen[1][2])[:, :a.Hq * a.D].reshape(T, a.Hq, a.D)
        for b in range(B):
            if new[b]:
                kk, vv = ref[1].row(table[b], ctx[b])
                wo, _, tol, _ = R.attention(q[cu[b]:cu[b + 1]], kk, vv, float(np.float32(a.D ** -0.5)), ctx[b], 0)
                assert (np.abs(o[cu[b]:cu[b + 1]] - wo) <= tol + 2.0 ** -11 * np.abs(wo) * 1.001 + 2.0 ** -25).all()
        plain.step(x, lens)
        assert torch.equal(plain.positions, bd.positions)
        moved = [p > 0 for p in want[:n]]
        assert not np.array_equal(f64(seen[0][1])[:n][moved], f64(seen[0][2])[:n][moved])


def test_a_captured_step_with_an_edit(L):
    a = synth.AttnShape(Hq=4, Hkv=2, D=64, block_tokens=16)
    B, T = 3, 4
    eager, graph = decoder_with(rotary(a), 2, B, T, 20, 6, a), decoder_with(rotary(a), 2, B, T, 20, 6, a)
    x = torch.zeros((T, 256), device="cuda")
    new = torch.zeros(B, dtype=torch.int32, device="cuda")
    graph.step(x, new)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        graph.step(x, new)
    rng = np.random.default_rng(9)
    for _ in range(10):
        x.copy_(torch.from_numpy(rng.standard_normal((T, 256)).astype(np.float32)))
        lens = rng.multinomial(T, np.ones(B) / B)
        new.copy_(torch.from_numpy(lens.astype(np.int32)))
        g.replay()
        assert torch.equal(graph.r_out, eager.step(x, new))
    assert L.e0_read_status(graph.status) == 0 and torch.equal(graph.cache.ctx, eager.cache.ctx)


def test_layers_follow_one_another(L):
    """Two layers equal the second layer alone fed with the first one's output."""
    a = synth.AttnShape(Hq=4, Hkv=1, D=64, block_tokens=16)
    B, T = 4, 4
    m, attn, two = decoder(2, B, T, 16, 4, a)
    from int4_gathered_expert_gb300.model import BatchDecoder, KvCacheDev
    halves = []
    for l in range(2):
        sd = two.sd
        import copy
        one = copy.copy(sd)
        one.L, one.pools, one.routers, one.shared = 1, [sd.pools[l]], [sd.routers[l]], [sd.shared[l]]
        halves.append(BatchDecoder(one, [attn[l]], a, KvCacheDev(1, B, 16, 4, 1, 64, 16), T))
    rng = np.random.default_rng(5)
    new = torch.ones(B, dtype=torch.int32, device="cuda")
    for _ in range(20):
        x = torch.from_numpy(rng.standard_normal((T, 256)).astype(np.float32)).cuda()
        got = two.step(x, new).clone()
        mid = halves[0].step(x, new)
        assert torch.equal(got, halves[1].step(mid, new))
    assert L.e0_read_status(two.status) == 0
    assert torch.equal(two.cache.k[1], halves[1].cache.k[0])


def test_a_captured_step_replays(L):
    a = synth.AttnShape(Hq=8, Hkv=2, D=128, block_tokens=16)
    B, T = 5, 8
    _, _, eager = decoder(2, B, T, 40, 8, a)
    _, _, graph = decoder(2, B, T, 40, 8, a)
    x = torch.zeros((T, 256), device="cuda")
    new = torch.zeros(B, dtype=torch.int32, device="cuda")
    graph.step(x, new)  # nothing joins: the first call of everything
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        graph.step(x, new)
    rng = np.random.default_rng(6)
    for i in range(25):
        x.copy_(torch.from_numpy(rng.standard_normal((T, 256)).astype(np.float32)))
        lens = rng.multinomial(T, np.ones(B) / B) if i % 3 == 0 else np.ones(B, int)
        new.copy_(torch.from_numpy(lens.astype(np.int32)))
        if i == 15:  # two sequences end; others come in their place
            for d in (eager, graph):
                d.cache.release(torch.tensor([1, 0, 0, 1, 0], dtype=torch.uint8, device="cuda"), d.status)
        g.replay()
        n = int(lens.sum())
        assert torch.equal(graph.r_out[:n], eager.step(x, new)[:n])
    assert L.e0_read_status(graph.status) == 0
    assert torch.equal(graph.cache.table, eager.cache.table) and torch.equal(graph.cache.ctx, eager.cache.ctx)


def test_many_query_rows_over_a_long_context(L):
    """Several new tokens of wide groups on contexts of thousands: more than a tile of query rows a KV head."""
    a = synth.AttnShape(Hq=16, Hkv=2, D=64, block_tokens=64)
    B, T = 3, 60
    m, attn, bd = decoder(1, B, T, 130, 60, a)
    c = bd.cache
    ctx = np.array([3500, 40, 2000])
    need = -(-ctx // 64)
    rng = np.random.default_rng(11)
    ref = R.Cache(130, 2, 64, 64)
    for x, codes, dst, scale in ((ref.k, c.k, 0, ref.ks), (ref.v, c.v, 1, ref.vs)):  # what earlier steps left
        x[:] = R.encode(rng.standard_normal(x.shape) * 100)
        codes[0].copy_(torch.from_numpy(x))
        scale[:] = 2.0 ** -7
        (c.v_scale if dst else c.k_scale)[0].copy_(torch.from_numpy(scale))
    ids = c.free.cpu().numpy()[::-1].copy()
    at = 0
    for b in range(B):
        c.table[b, :need[b]] = torch.from_numpy(ids[at:at + need[b]]).cuda()
        at += need[b]
    c.free_count.fill_(130 - at)
    c.ctx.copy_(torch.from_numpy(ctx.astype(np.int32)))
    for new in ([20, 1, 30], [1, 1, 1]):
        x = torch.from_numpy(rng.standard_normal((T, 256)).astype(np.float32)).cuda()
        bd.step(x, torch.tensor(new, dtype=torch.int32, device="cuda"))
        assert L.e0_read_status(bd.status) == 0
        ctx = ctx + new
        qkv, slots = f64(bd.x_qkv), bd.slots.cpu().numpy()
        ref.append(qkv[:, 1024:1152].reshape(T, 2, 64), qkv[:, 1152:].reshape(T, 2, 64), slots)
        table, cu, o = c.table.cpu().numpy(), bd.cu_q.cpu().numpy(), f64(bd.o).reshape(T, 16, 64)
        for b in range(B):
            kk, vv = ref.row(table[b], ctx[b])
            q = qkv[cu[b]:cu[b + 1], :1024].reshape(-1, 16, 64)
            wo, _, tol, _ = R.attention(q, kk, vv, 0.125, ctx[b], 0)
            assert (np.abs(o[cu[b]:cu[b + 1]] - wo) <= tol + 2.0 ** -11 * np.abs(wo) * 1.001 + 2.0 ** -25).all()


def test_a_full_pool_caches_nothing(L):
    a = synth.AttnShape(Hq=2, Hkv=2, D=64, block_tokens=16)
    m, attn, bd = decoder(1, 2, 40, 4, 8, a)
    x = torch.randn((40, 256), generator=torch.Generator().manual_seed(1)).cuda()
    bd.step(x, torch.tensor([20, 18], dtype=torch.int32, device="cuda"))
    assert L.e0_read_status(bd.status) == 0 and bd.cache.free_count.item() == 0
    before = [t.clone() for t in (bd.cache.k, bd.cache.v, bd.cache.table, bd.cache.ctx, bd.cache.k_scale)]
    bd.step(x, torch.tensor([1, 20], dtype=torch.int32, device="cuda"))
    assert L.e0_read_status(bd.status) == L.E0_ST_POOL_FULL
    for t, w in zip((bd.cache.k, bd.cache.v, bd.cache.table, bd.cache.ctx, bd.cache.k_scale), before):
        assert torch.equal(t, w)
    bd.status.zero_()
    bd.cache.release(torch.tensor([1, 0], dtype=torch.uint8, device="cuda"), bd.status)
    bd.step(x, torch.tensor([1, 14], dtype=torch.int32, device="cuda"))
    assert L.e0_read_status(bd.status) == 0 and bd.cache.ctx.tolist() == [1, 32]


@pytest.mark.parametrize("how", ["current", "stream", "handle"])
def test_a_row_that_overflowed_does_not_stay(L, how):
    """A query beyond fp16 spoils its own row; a step with fewer tokens after it raises nothing and is as it would be
    without."""
    a = synth.AttnShape(Hq=2, Hkv=2, D=64, block_tokens=16)
    stream = {"current": None, "stream": torch.cuda.Stream(), "handle": torch.cuda.Stream()}[how]
    arg = stream.cuda_stream if how == "handle" else stream
    pair = []
    for _ in range(2):
        m, attn, bd = decoder(1, 2, 8, 8, 4, a)
        bd.norm[0][0] = 1e9  # the first column, times this, passes fp16
        pair.append(bd)
    x = torch.randn((8, 256), generator=torch.Generator().manual_seed(2)).cuda()
    x[:, 0] = 0
    wild = x.clone()
    wild[6, 0] = 1
    torch.cuda.synchronize()

    def step(bd, x, lens):
        new = torch.tensor(lens, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        out = bd.step(x, new, stream=arg)
        torch.cuda.synchronize()
        st = L.e0_read_status(bd.status)
        bd.status.zero_()
        return out.clone(), st

    _, st = step(pair[0], wild, [3, 5])
    assert st & L.E0_ST_NONFINITE
    assert step(pair[1], x, [3, 5])[1] == 0
    for lens in ([2, 0], [1, 0]):
        got, st = step(pair[0], x, lens)
        want, _ = step(pair[1], x, lens)
        n = sum(lens)
        assert st == 0 and torch.isfinite(got).all() and torch.equal(got[:n], want[:n])


def test_a_new_cache_is_ready_for_any_stream(L):
    """What fills it is not still waiting on the stream that was current."""
    from int4_gathered_expert_gb300.model import KvCacheDev
    other = torch.cuda.Stream()
    new = torch.full((3,), 20, dtype=torch.int32, device="cuda")
    cu, slots = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(60, dtype=torch.int64, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    keep = KvCacheDev(1, 3, 100, 8, 2, 64, 16)
    keep.plan(new, 60, cu, slots, status=st, stream=other)  # the first call of everything
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)  # a tenth of a second of work that the constructor's comes after
    c = KvCacheDev(1, 3, 100, 8, 2, 64, 16)
    c.plan(new, 60, cu, slots, status=st, stream=other)
    torch.cuda.synchronize()
    assert L.e0_read_status(st) == 0
    assert c.ctx.tolist() == [20] * 3 and c.free_count.item() == 94 and c.table[:, :2].flatten().tolist() == list(range(6))


def test_decoder_refuses(L):
    from int4_gathered_expert_gb300.model import BatchDecoder
    a = synth.AttnShape(Hq=2, Hkv=2, D=64, block_tokens=16)
    _, attn, bd = decoder(1, 2, 4, 4, 8, a)
    with pytest.raises(ValueError):
        BatchDecoder(bd.sd, attn + attn, a, bd.cache, 4)
    with pytest.raises(ValueError):
        BatchDecoder(bd.sd, attn, a, bd.cache, 65)


def test_decoder_refuses_what_does_not_fit(L):
    """Caches, weights and inputs whose sizes the kernels would read past."""
    from int4_gathered_expert_gb300.model import BatchDecoder, KvCacheDev
    a = synth.AttnShape(Hq=2, Hkv=2, D=64, block_tokens=16)
    _, attn, bd = decoder(1, 2, 4, 4, 8, a)
    for cache in (KvCacheDev(1, 2, 4, 8, 4, 64, 16), KvCacheDev(1, 2, 4, 8, 2, 128, 16), KvCacheDev(0, 2, 4, 8, 2, 64, 16)):
        with pytest.raises(ValueError):
            BatchDecoder(bd.sd, attn, a, cache, 4)
    BatchDecoder(bd.sd, attn, a, KvCacheDev(2, 2, 4, 8, 2, 64, 16), 4)  # more layers than are used
    other = synth.attention(1, 0, synth.TINY.H, synth.AttnShape(Hq=4, Hkv=2, D=64))
    narrow = synth.attention(1, 0, 128, a)
    for half in (other, narrow, dict(attn[0], out=other["out"]), dict(attn[0], norm=attn[0]["norm"][:-1])):
        with pytest.raises(ValueError):
            BatchDecoder(bd.sd, [half], a, bd.cache, 4)
    x = torch.zeros((4, 256), device="cuda")
    new = torch.ones(2, dtype=torch.int32, device="cuda")
    for bad in (x[:3], x.half(), x[:, :128], x.cpu(), torch.zeros((256, 4), device="cuda").t(), x.view(-1)):
        with pytest.raises(ValueError):
            bd.step(bad, new)
    for bad in (new.long(), new[:1], new.cpu(), torch.ones(4, dtype=torch.int32, device="cuda")[::2]):
        with pytest.raises(ValueError):
            bd.step(x, bad)
    bd.step(x, new)
    assert L.e0_read_status(bd.status) == 0 and bd.cache.ctx.tolist() == [1, 1]
