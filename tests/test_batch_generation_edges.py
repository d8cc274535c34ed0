"""A batch's generation where its parts meet in ways that test_batch_generation does not use."""
import numpy as np
import pytest

from int4_gathered_expert_gb300 import synth
from tests.test_batch_decoder import L, f64  # noqa: F401
from tests.test_batch_generation import freqs, parts
from tests.test_layer_ops import F16, H, TINY16
from tests.test_token_ops import rope_ref

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def lens(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("axes", [2, 3, 4])
def test_steps_on_several_axes(L, axes):  # noqa: F811
    """A decoder knows the positions in the row; whoever knows the other axes' hands all of them to the rotation."""
    from int4_gathered_expert_gb300.model import BatchDecoder, KvCacheDev, QkRope
    a = synth.AttnShape(Hq=6, Hkv=2, D=64, block_tokens=16)
    B, T = 3, 12
    rng = np.random.default_rng(axes)
    sd, attn = parts(1, a)
    cache = KvCacheDev(1, B, 20, 6, a.Hkv, a.D, 16)
    axis = rng.integers(0, axes, 32)
    rope = QkRope(a, freqs(64), 1, axis=axis, n_axes=axes)
    grid = torch.zeros((axes, T), dtype=torch.int32, device="cuda")
    seen = []

    def edit(layer, qkv, positions):
        grid[0].copy_(positions)
        for i in range(1, axes):
            grid[i].copy_(positions % (3 * i + 1))
        was = qkv.clone()
        rope(layer, qkv, grid)
        seen.append((was, qkv.clone(), grid.cpu().numpy()))

    bd = BatchDecoder(sd, attn, a, cache, T, edit=edit)
    for new in ([5, 4, 3], [1, 0, 2]):
        seen.clear()
        bd.step(torch.from_numpy(rng.standard_normal((T, synth.TINY.H)).astype(np.float32)).cuda(), lens(new))
        assert L.e0_read_status(bd.status) == 0 and L.e0_read_status(rope.status) == 0
        n = sum(new)
        was, qkv, pos = seen[0]
        assert (pos[0, :n] >= 0).all() and (pos[0, n:] == -1).all() and (pos[1:] != pos[0]).any()
        want, tol = rope_ref(f64(was)[:n, :8 * 64].reshape(n, 8, 64), 6, pos[:, :n], freqs(64), axis, 64, False, True, None, None, 1e-6)
        got = f64(qkv)[:n, :8 * 64].reshape(n, 8, 64)
        assert (np.abs(got - want) <= tol + H[F16] * np.abs(want) * 1.0001 + TINY16[F16]).all()
        assert torch.equal(qkv[:, 8 * 64:], was[:, 8 * 64:]) and torch.equal(qkv[n:], was[n:])
    with pytest.raises(ValueError):  # the row's positions alone do not say where it is on the others
        rope(0, torch.zeros((T, 640), dtype=torch.float16, device="cuda"), torch.zeros(T, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("captured", [False, True])
def test_a_prefix_is_shared_where_the_others_are_empty(L, captured):  # noqa: F811
    """Tokens that another sequence has would silently stand behind it: the cache, and a prefix there was, stay as they are."""
    from int4_gathered_expert_gb300.model import BatchDecoder, KvCacheDev
    a = synth.AttnShape(Hq=4, Hkv=2, D=64, block_tokens=16)
    B, T = 3, 40
    sd, attn = parts(1, a)
    cache = KvCacheDev(1, B, 20, 4, a.Hkv, a.D, 16)
    first, bd = BatchDecoder(sd, attn, a, cache, T), BatchDecoder(sd, attn, a, cache, T, prefix=True)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    graph, side = None, torch.cuda.Stream()

    def share():
        if graph:
            graph.replay()
        else:
            cache.share(1, status=st)

    def all_of():
        return [t.clone() for t in (cache.table, cache.ctx, cache.prefix_table, cache.prefix_len, cache.free_count)]

    if captured:
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            cache.share(1, status=st)
        assert cache.prefix_len.tolist() == [0] and L.e0_read_status(st) == 0
    x = torch.randn((T, synth.TINY.H), generator=torch.Generator().manual_seed(1)).cuda()
    first.step(x, lens([0, 17, 0]))
    row = cache.table[1].clone()
    share()
    assert L.e0_read_status(st) == 0 and cache.prefix_len.tolist() == [17] and cache.ctx.tolist() == [0] * B
    assert torch.equal(cache.prefix_table[0], row) and (cache.table == -1).all()
    bd.step(x, lens([1, 0, 1]))
    for new in ([0, 0, 0], [0, 18, 0]):  # an empty sequence as another prefix; one with tokens
        if sum(new):
            bd.step(x, lens(new))
        was = all_of()
        share()
        assert L.e0_read_status(st) == L.E0_ST_BAD_LENGTH and all(torch.equal(p, q) for p, q in zip(was, all_of()))
        st.zero_()
    cache.release(torch.tensor([1, 0, 1], dtype=torch.uint8, device="cuda"), st)
    share()  # the others are empty now
    assert cache.prefix_len.tolist() == [18] and cache.free_count.tolist() == [18] and cache.ctx.tolist() == [0] * B
    torch.cuda.synchronize()
    cache.share(0, stream=side)  # nothing as the prefix, on a stream of its own
    cache.share(0, stream=side.cuda_stream)
    side.synchronize()
    assert L.e0_read_status(st) == 0 and cache.prefix_len.tolist() == [0] and sorted(cache.free.tolist()) == list(range(20))
    assert cache.free_count.tolist() == [20]
