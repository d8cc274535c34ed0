"""Device-resident weights for the C ABI: uploads the canonical tensors drawn
by ``synth``, packs experts into slot pools with e0_pack_experts and keeps the
ctypes descriptors (and the torch tensors they point into) alive.  PyTorch is
used for device memory and streams only; all arithmetic runs in libe0moe.
"""
from __future__ import annotations

import contextlib
import ctypes as C
from typing import Callable, Dict, List, Optional

import numpy as np
import torch

from . import lib as L


def _dev(a: np.ndarray, device) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(a)).to(device, non_blocking=False)


def _on(stream):
    """torch's calls on the stream that a call takes (None: the current one)."""
    if stream is None:
        return contextlib.nullcontext()
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


class DeviceQBank:
    """A layer's canonical stacked bank on the device (gate/up/down x codes/scale/bias)."""

    def __init__(self, bank_np: Dict[str, Dict[str, np.ndarray]], device="cuda"):
        self.t = {p: {k: _dev(v, device) for k, v in bank_np[p].items()} for p in ("gate", "up", "down")}
        self.E = self.t["gate"]["codes"].shape[0]

    def expert_q(self, e: int) -> L.ExpertQ:
        def q(p):
            d = self.t[p]
            return L.QTensor(d["codes"][e].data_ptr(), d["scale"][e].data_ptr(), d["bias"][e].data_ptr())
        return L.ExpertQ(q("gate"), q("up"), q("down"))


class SlotPoolDev:
    """n_slots experts in the kernel layout, a slot table [E] and an occupant
    table [n_slots] (all -1 until something is packed)."""

    def __init__(self, H: int, I: int, E: int, n_slots: int, device="cuda"):
        self.H, self.I, self.E, self.n_slots = H, I, E, n_slots
        self.slot_bytes = L.e0_slot_bytes(H, I)
        self.data = torch.empty(n_slots * self.slot_bytes, dtype=torch.uint8, device=device)
        self.table = torch.full((E,), -1, dtype=torch.int32, device=device)
        self.occupant = torch.full((n_slots,), -1, dtype=torch.int32, device=device)
        self.desc = L.SlotPool(self.data.data_ptr(), self.table.data_ptr(), self.occupant.data_ptr(),
                               n_slots, H, I, E)

    def pack(self, qbank: DeviceQBank, experts: List[int], slots: List[int], set_table=True, stream=None):
        src = [qbank.expert_q(e) for e in experts]
        L.e0_pack_experts(src, self.desc, slots, experts if set_table else None, stream=stream)

    @classmethod
    def resident(cls, bank_np, H, I, device="cuda", stream=None) -> "SlotPoolDev":
        """Every expert of a layer in slot e (identity table)."""
        qb = DeviceQBank(bank_np, device)
        pool = cls(H, I, qb.E, qb.E, device)
        ids = list(range(qb.E))
        pool.pack(qb, ids, ids, stream=stream)
        del qb
        return pool


class SharedDev:
    """Shared expert (one packed slot) plus its LoRA tensors."""

    def __init__(self, shared_np: dict, H: int, I: int, device="cuda", with_lora=True):
        qb = DeviceQBank({p: {k: v[None] for k, v in shared_np["q"][p].items()} for p in ("gate", "up", "down")},
                         device)
        self.pool = SlotPoolDev(H, I, 1, 1, device)
        self.pool.pack(qb, [0], [0])
        self.lora = None
        null = None
        if with_lora and shared_np.get("lora") is not None:
            self.lora = {p: {k: _dev(v, device) for k, v in shared_np["lora"][p].items()}
                         for p in ("gate", "up", "down")}
            lo = self.lora
            self.desc = L.SharedExpert(self.pool.data.data_ptr(),
                                       lo["gate"]["A"].data_ptr(), lo["gate"]["B"].data_ptr(),
                                       lo["up"]["A"].data_ptr(), lo["up"]["B"].data_ptr(),
                                       lo["down"]["A"].data_ptr(), lo["down"]["B"].data_ptr(),
                                       int(shared_np["rank"]), float(shared_np["alpha"]))
        else:
            self.desc = L.SharedExpert(self.pool.data.data_ptr(), null, null, null, null, null, null, 0, 0.0)


class HeadDev:
    def __init__(self, head_np: dict, H: int, E: int, device="cuda"):
        self.t = {k: _dev(v, device) for k, v in head_np.items() if v is not None}
        hidden = self.t["fc1"].shape[0]
        g = lambda k: self.t[k].data_ptr() if k in self.t else None  # noqa: E731
        self.desc = L.Prerouter(g("fc1"), g("b1"), g("fc2"), g("b2"), g("lres"), H, E, hidden)
        self.hidden = hidden


class StackDev:
    """A whole decode stack on the device plus its workspace and optional trace."""

    def __init__(self, model, device="cuda", trace=False, with_lora=True):
        sh = model.shape
        s = sh.layer
        self.shape = sh
        self.H, self.I, self.E, self.K = s.H, s.I, s.E, s.K
        self.L = len(model.banks)
        self.pools = [SlotPoolDev.resident(b, s.H, s.I, device) for b in model.banks]
        self.routers = [_dev(w, device) for w in model.routers]
        self.heads = {l: HeadDev(h, s.H, s.E, device) for l, h in model.heads.items()}
        self.shared = [SharedDev(x, s.H, s.I, device, with_lora) if x is not None else None for x in model.shared]
        hidden = max([h.hidden for h in self.heads.values()], default=0)
        self._sh_descs = [C.pointer(x.desc) if x is not None else None for x in self.shared]
        self._hd_descs = {l: C.pointer(h.desc) for l, h in self.heads.items()}
        consumers = set(sh.consumers)
        layers = []
        for l in range(self.L):
            layers.append(L.StackLayer(self.pools[l].desc, self.routers[l].data_ptr(),
                                       self._sh_descs[l] if self._sh_descs[l] is not None else None,
                                       self._hd_descs.get(l), 1 if (l in consumers and (l - 1) in self.heads) else 0))
        self.layers = layers
        self.rp = L.route_params(0 if s.route == "softmax_topk" else 1, s.K, s.n_groups, s.topk_groups,
                                 s.route_scale)
        self.ws_bytes = L.e0_stack_workspace_size(self.L, s.H, s.I, s.E, s.K, hidden)
        self.ws = torch.empty(self.ws_bytes, dtype=torch.uint8, device=device)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)
        self.r_out = torch.empty(s.H, dtype=torch.float32, device=device)
        self.trace = None
        if trace:
            self.tr = {"r": torch.zeros((self.L + 1, s.H), dtype=torch.float32, device=device),
                       "inds": torch.full((self.L, s.K), -1, dtype=torch.int32, device=device),
                       "w": torch.zeros((self.L, s.K), dtype=torch.float32, device=device),
                       "head_logits": torch.zeros((self.L, s.E), dtype=torch.float32, device=device),
                       "pred_inds": torch.full((self.L, s.K), -1, dtype=torch.int32, device=device)}
            self.trace = L.StackTrace(*[self.tr[k].data_ptr() for k in ("r", "inds", "w", "head_logits",
                                                                           "pred_inds")])
        self.prepare()

    def variant(self, K: Optional[int] = None, prerouter: bool = True, device="cuda") -> "StackDev":
        """The same device weights with another routed-expert count K and/or
        without the prerouter heads (every layer then routes with its own
        router); its own workspace and status word, no trace."""
        import copy
        v = copy.copy(self)
        s = self.shape.layer
        v.K = self.K if K is None else int(K)
        consumers = set(self.shape.consumers) if prerouter else set()
        heads = self._hd_descs if prerouter else {}
        v.layers = [L.StackLayer(self.pools[l].desc, self.routers[l].data_ptr(),
                                 self._sh_descs[l] if self._sh_descs[l] is not None else None,
                                 heads.get(l), 1 if (l in consumers and (l - 1) in heads) else 0)
                    for l in range(self.L)]
        v.rp = L.route_params(0 if s.route == "softmax_topk" else 1, v.K, s.n_groups, s.topk_groups, s.route_scale)
        hidden = max([h.hidden for h in self.heads.values()], default=0) if prerouter else 0
        v.ws_bytes = L.e0_stack_workspace_size(self.L, s.H, s.I, s.E, v.K, hidden)
        v.ws = torch.empty(v.ws_bytes, dtype=torch.uint8, device=device)
        v.status = torch.zeros(1, dtype=torch.int32, device=device)
        v.r_out = torch.empty(s.H, dtype=torch.float32, device=device)
        v.trace = None
        v.prepare()
        return v

    def prepare(self, stream=None):
        L.e0_stack_prepare(self.layers, self.H, self.I, self.E, self.rp, self.ws, self.ws_bytes, stream=stream)

    def step(self, x: torch.Tensor, impl: int = 0, stream=None, out: Optional[torch.Tensor] = None):
        out = self.r_out if out is None else out
        L.e0_stack_step(x, out, self.ws, self.trace, impl, self.status, stream=stream)
        return out


class ExpertCacheDev:
    """A cross-layer cache of `capacity` expert bundles in device memory (keys
    layer * E + expert), least recently used first out."""

    def __init__(self, capacity: int, n_layers: int, H: int, I: int, E: int, device="cuda"):
        self.capacity = capacity
        sb = L.e0_slot_bytes(H, I)
        self.data = torch.empty(max(capacity, 1) * sb, dtype=torch.uint8, device=device)
        self.key = torch.full((max(capacity, 1),), -1, dtype=torch.int32, device=device)
        self.stamp = torch.zeros(max(capacity, 1), dtype=torch.int32, device=device)
        self.map = torch.full((n_layers * E,), -1, dtype=torch.int32, device=device)
        self.counters = torch.zeros(4, dtype=torch.int32, device=device)
        self.scratch = torch.zeros(4 + 4 * 32, dtype=torch.int32, device=device)
        self.desc = L.ExpertCache(self.data.data_ptr(), self.key.data_ptr(), self.stamp.data_ptr(),
                                  self.map.data_ptr(), self.counters.data_ptr(), self.scratch.data_ptr(),
                                  capacity, n_layers * E)

    def stats(self) -> dict:
        c = self.counters.cpu().tolist()
        return {"hits": c[1], "misses": c[2], "evictions": c[3]}


class StreamedStack:
    """Host-tier staged streaming on top of a StackDev (flag-carrying-word kernel).

    Each staged layer keeps its experts (kernel layout) in pinned host memory
    and only 2K slots in device memory.  A token runs as two launches, layers
    [0, split) and [split, L); the experts the prerouter predicted for the next
    token are copied host -> device by e0_stack_prefetch_experts on a second
    stream: layers below split - 1 while the second half of the token runs,
    layers from split on while the first half of the next token runs.  Layer
    split - 1, whose prediction is final only once the token has ended but
    which the next token's first half uses, stays in the resident bank, as do
    the layers that route natively.  With an ExpertCacheDev the copies first
    look in a cross-layer cache of recently used bundles in device memory.

    The decode launches leave ``free_sms`` SMs to the copy kernels, which run
    on that many blocks: a cooperative launch over every SM would wait for a
    running copy kernel instead of overlapping it.  The layers of one half
    are prefetched with one batched call (``batched=False``: one call per
    layer, the same slot contents)."""

    def __init__(self, sd: "StackDev", split: int, device="cuda", cache: Optional["ExpertCacheDev"] = None,
                 host: Optional[dict] = None, free_sms: int = 24, batched: bool = True):
        self.batched = batched
        import os
        old = os.environ.get("E0MOE_LL_FREE_SMS")
        os.environ["E0MOE_LL_FREE_SMS"] = str(int(free_sms))
        try:
            sd.prepare()
        finally:
            if old is None:
                del os.environ["E0MOE_LL_FREE_SMS"]
            else:
                os.environ["E0MOE_LL_FREE_SMS"] = old
        self.sd = sd
        self.split = split
        self.cache = cache
        consumers = [l for l in range(sd.L) if sd.layers[l].consumer]
        self.batch1 = [l for l in consumers if l <= split - 2]
        self.batch2 = [l for l in consumers if l >= split]
        self.staged = self.batch1 + self.batch2
        self.host = {}
        self.pools = {}
        n_slots = 2 * sd.K
        for l in self.staged:
            if host is not None and l in host:  # the pinned copies of an earlier run of the same stack
                self.host[l] = host[l]
            else:
                src = sd.pools[l].data
                h = torch.empty(src.shape, dtype=torch.uint8, pin_memory=True)
                h.copy_(src)
                self.host[l] = h
            self.pools[l] = SlotPoolDev(sd.H, sd.I, sd.E, n_slots, device)
        torch.cuda.synchronize()
        self.cs = torch.cuda.Stream()
        self.ps = torch.cuda.Stream()
        self.ev1 = torch.cuda.Event()
        self.ev2 = torch.cuda.Event()
        self.status = sd.status
        self.t = 0

    def copy_bytes_per_expert(self) -> int:
        return L.e0_slot_bytes(self.sd.H, self.sd.I)

    def _prefetch(self, layers, t_next, stream):
        if not self.batched:
            for l in layers:
                if self.cache is None:
                    L.e0_stack_prefetch_experts(self.sd.ws, l, t_next, self.pools[l].desc, self.host[l], self.status,
                                                stream=stream)
                else:
                    L.e0_stack_prefetch_experts_cached(self.sd.ws, l, t_next, self.pools[l].desc, self.host[l],
                                                       self.cache.desc, self.status, stream=stream)
            return
        # every layer of the batch in one copy launch and one commit launch
        pools = [self.pools[l].desc for l in layers]
        banks = [self.host[l] for l in layers]
        if self.cache is None:
            L.e0_stack_prefetch_experts_batch(self.sd.ws, layers, t_next, pools, banks, self.status, stream=stream)
        else:
            L.e0_stack_prefetch_experts_cached_batch(self.sd.ws, layers, t_next, pools, banks, self.cache.desc,
                                                     self.status, stream=stream)

    def start(self, x0: torch.Tensor, out: Optional[torch.Tensor] = None):
        """Token 0 (every layer routes natively) from the resident bank, then the
        staged layers switch to their slot pools holding the predicted experts
        of token 1."""
        sd = self.sd
        out = sd.r_out if out is None else out
        with torch.cuda.stream(self.cs):
            L.e0_stack_step_range(x0, out, sd.ws, 0, sd.L, sd.trace, self.status, stream=self.cs)
            self._prefetch(self.staged, 1, self.cs)
        self.cs.synchronize()
        layers = list(sd.layers)
        for l in self.staged:
            layers[l] = L.StackLayer(self.pools[l].desc, layers[l].W_router, layers[l].shared, layers[l].head,
                                     layers[l].consumer)
        L.e0_stack_update_layers(sd.ws, layers, stream=self.cs)
        self.layers = layers
        self.ev1.record(self.cs)
        self.ev2.record(self.cs)
        self.t = 1
        return out

    def step(self, x: torch.Tensor, out: Optional[torch.Tensor] = None, overlap: bool = True):
        """Token self.t; the copies for token self.t + 1 are issued behind it."""
        sd = self.sd
        out = sd.r_out if out is None else out
        t = self.t
        cs, ps = self.cs, (self.ps if overlap else self.cs)
        cs.wait_event(self.ev1)
        L.e0_stack_step_range(x, None, sd.ws, 0, self.split, sd.trace, self.status, stream=cs)
        ev_a = torch.cuda.Event()
        ev_a.record(cs)
        ps.wait_event(ev_a)
        self._prefetch(self.batch1, t + 1, ps)
        self.ev1.record(ps)
        cs.wait_event(self.ev2)
        L.e0_stack_step_range(None, out, sd.ws, self.split, sd.L, sd.trace, self.status, stream=cs)
        ev_b = torch.cuda.Event()
        ev_b.record(cs)
        ps.wait_event(ev_b)
        self._prefetch(self.batch2, t + 1, ps)
        self.ev2.record(ps)
        self.t = t + 1
        return out


class LinearDev:
    """A canonical int4 Q-tensor [N, K] laid out for e0_linear_forward."""

    def __init__(self, q_np: Dict[str, np.ndarray], device="cuda", stream=None):
        self.N, self.K = q_np["codes"].shape[0], q_np["codes"].shape[1] * 2
        src = {k: _dev(v, device) for k, v in q_np.items()}
        self.data = torch.empty(L.e0_linear_bytes(self.N, self.K), dtype=torch.uint8, device=device)
        L.e0_pack_linear(L.QTensor(src["codes"].data_ptr(), src["scale"].data_ptr(), src["bias"].data_ptr()),
                         self.N, self.K, self.data, stream=stream)
        torch.cuda.synchronize()  # the source tensors go


class KvCacheDev:
    """A paged 8-bit KV cache of n_layers layers for B sequences: n_blocks blocks
    a layer, one block table, one stack of free blocks (all blocks free, all
    sequences empty).  A block id means the same block of every layer."""

    def __init__(self, n_layers: int, B: int, n_blocks: int, max_blocks: int, Hkv: int, D: int, block_tokens: int = 64,
                 device="cuda"):
        self.B, self.n_blocks, self.max_blocks, self.block_tokens = B, n_blocks, max_blocks, block_tokens
        shape = (n_layers, n_blocks, Hkv, block_tokens, D)
        self.k = torch.zeros(shape, dtype=torch.uint8, device=device)
        self.v = torch.zeros(shape, dtype=torch.uint8, device=device)
        self.k_scale = torch.ones(shape[:3], device=device)
        self.v_scale = torch.ones(shape[:3], device=device)
        self.descs = [L.KvCache(self.k[l].data_ptr(), self.v[l].data_ptr(), self.k_scale[l].data_ptr(),
                                self.v_scale[l].data_ptr(), n_blocks, Hkv, block_tokens, D) for l in range(n_layers)]
        self.table = torch.full((B, max_blocks), -1, dtype=torch.int32, device=device)
        self.ctx = torch.zeros(B, dtype=torch.int32, device=device)
        self.free = torch.arange(n_blocks - 1, -1, -1, dtype=torch.int32, device=device)
        self.free_count = torch.full((1,), n_blocks, dtype=torch.int32, device=device)
        self.state = L.KvState(self.table.data_ptr(), self.ctx.data_ptr(), self.free.data_ptr(),
                               self.free_count.data_ptr(), B, max_blocks, block_tokens, n_blocks)
        torch.cuda.synchronize()  # any stream may use it from here on

    def plan(self, new_len, T_cap, cu_q, slots, positions=None, seq_ids=None, status=None, stream=None):
        """Room for new_len more tokens of each sequence; lengths and stack move in place."""
        L.e0_kv_plan(self.state, new_len, T_cap, self.ctx, self.free_count, cu_q, slots, positions, seq_ids, status,
                     stream=stream)

    def release(self, mask, status=None, stream=None):
        """Empty the sequences whose mask byte is set; their blocks are free again."""
        L.e0_kv_release(self.state, mask, self.ctx, self.free_count, status, stream=stream)


class BatchDecoder:
    """Decode steps of a batch of sequences through whole layers, attention and
    MoE, on a StackDev's weights.  For each layer:

        r += MoE of the layer before; h = norm(r) * w in 8 bits
        q, k, v = W_qkv h (fp16); edit(layer, qkv, positions); k, v into the cache
        r += W_out attention(q)
        MoE(rmsnorm(r)), with the layer's own routing (batches do not predict)

    attn: one ``synth.attention`` dict a layer.  A step takes up to T tokens, new_len[b]
    of each sequence in order, as rows of x (T <= 64, the MoE block's limit).
    edit: what a model does to queries and keys before they meet (rotary embeddings,
    norms), or None: called on the step's stream with the layer, qkv fp16 [T, (Hq + 2
    Hkv) D] (queries, keys, values; to be changed in place) and the rows' positions
    int32 [T], -1 after the last new token.  All of a step's work is on one stream and
    allocates nothing but what edit does, so a step can be captured into a CUDA graph."""

    def __init__(self, sd: StackDev, attn: List[dict], shape, cache: KvCacheDev, T: int, device="cuda",
                 edit: Optional[Callable[[int, torch.Tensor, torch.Tensor], None]] = None):
        if len(attn) != sd.L:
            raise ValueError("one attention half a layer")
        if not 1 <= T <= L.E0_MAX_T_DECODE:
            raise ValueError("T is 1..%d" % L.E0_MAX_T_DECODE)
        if len(cache.descs) < sd.L or any(c.Hkv != shape.Hkv or c.D != shape.D for c in cache.descs):
            raise ValueError("the cache has other layers or heads than the attention")
        row, back = (shape.Hq + 2 * shape.Hkv) * shape.D, shape.Hq * shape.D
        for w in attn:
            n, k = w["qkv"]["codes"].shape, w["out"]["codes"].shape
            if n != (row, sd.H // 2) or k != (sd.H, back // 2) or w["norm"].shape != (sd.H,):
                raise ValueError("an attention half of other sizes than its shape and the stack's H")
        self.sd, self.a, self.cache, self.T, self.edit = sd, shape, cache, T, edit
        self.qkv = [LinearDev(w["qkv"], device) for w in attn]
        self.out = [LinearDev(w["out"], device) for w in attn]
        self.norm = [_dev(w["norm"], device) for w in attn]
        H, a = sd.H, shape
        self.row = row

        def buf(*s, dtype=torch.float32):
            return torch.zeros(s, dtype=dtype, device=device)

        self.r, self.h, self.y = buf(T, H), buf(T, H), buf(T, H)
        self.q8, self.q8_scale = buf(T, H, dtype=torch.uint8), buf(T, -(-H // 64))
        self.x_qkv = buf(T, self.row, dtype=torch.float16)
        self.o = buf(T, a.Hq * a.D, dtype=torch.float16)
        self.cu_q = buf(cache.B + 1, dtype=torch.int32)
        self.slots, self.positions = buf(T, dtype=torch.int64), buf(T, dtype=torch.int32)
        self.inds, self.w = buf(T, sd.K, dtype=torch.int32), buf(T, sd.K)
        self.ws_bytes = L.e0_workspace_size(0, T, sd.H, sd.I, sd.E, sd.K)
        self.ws = buf(self.ws_bytes, dtype=torch.uint8)
        self.aws_bytes = L.e0_attn_workspace_size(cache.B, a.Hq, a.Hkv, a.D, T)
        self.aws = buf(self.aws_bytes, dtype=torch.uint8)
        self.status = buf(1, dtype=torch.int32)
        self.r_out = buf(T, H)
        torch.cuda.synchronize()  # any stream may take the steps

    def step(self, x: torch.Tensor, new_len: torch.Tensor, window: int = 0, stream=None) -> torch.Tensor:
        """x fp32 [T, H], new_len int32 [B] on the device; the rows of x after the
        last new token are any finite values, those of the result nothing of use.
        The result is the decoder's own buffer: the next step writes over it.  Where a
        step finds no room (E0_ST_POOL_FULL in ``status``), no token is cached."""
        sd, a, c, T, H = self.sd, self.a, self.cache, self.T, self.sd.H
        if x.dtype != torch.float32 or x.shape != (T, H) or not x.is_cuda or not x.is_contiguous():
            raise ValueError("x is contiguous fp32 [%d, %d] on the device" % (T, H))
        if new_len.dtype != torch.int32 or new_len.shape != (c.B,) or not new_len.is_cuda or not new_len.is_contiguous():
            raise ValueError("new_len is contiguous int32 [%d] on the device" % c.B)
        kw = dict(stream=stream)
        c.plan(new_len, T, self.cu_q, self.slots, self.positions, status=self.status, **kw)
        with _on(stream):
            self.o.zero_()  # attention leaves the rows after the last new token, which an earlier step may have used
        src, delta = x, None
        for l in range(sd.L):
            L.e0_rmsnorm_q8(src, delta, self.norm[l], T, H, L.E0_F32, 1e-6, H, H, self.r, None, self.q8, self.q8_scale,
                            self.status, **kw)
            p = self.qkv[l]
            L.e0_linear_forward(p.data, p.N, p.K, self.q8, L.E0_E4M3, H, self.q8_scale, T, None, 0, self.x_qkv, L.E0_F16,
                                self.row, **kw)
            if self.edit is not None:
                with _on(stream):
                    self.edit(l, self.x_qkv, self.positions)
            k = self.x_qkv.data_ptr() + 2 * a.Hq * a.D
            v = k + 2 * a.Hkv * a.D
            L.e0_kv_append(c.descs[l], k, v, L.E0_F16, self.row, self.row, self.slots, T, self.status, **kw)
            L.e0_attn_decode(c.descs[l], c.table, c.max_blocks, c.ctx, self.cu_q, c.B, T, self.x_qkv, L.E0_F16, self.row,
                             a.Hq, a.D ** -0.5, window, self.o, a.Hq * a.D, None, self.aws, self.aws_bytes, self.status,
                             **kw)
            p = self.out[l]
            L.e0_linear_forward(p.data, p.N, p.K, self.o, L.E0_F16, a.Hq * a.D, None, T, self.r, H, self.r, L.E0_F32, H,
                                **kw)
            L.e0_rmsnorm(self.r, T, H, 1e-6, self.h, **kw)
            sh = sd.shared[l].desc if sd.shared[l] is not None else None
            L.e0_moe_block_forward(self.h, T, sd.pools[l].desc, sd.routers[l], sd.rp, None, None, sh, self.y, self.inds,
                                   self.w, self.ws, self.ws_bytes, self.status, **kw)
            src, delta = self.r, self.y
        L.e0_rmsnorm_q8(self.r, self.y, None, T, H, L.E0_F32, 1e-6, H, H, self.r_out, None, None, None, self.status, **kw)
        return self.r_out
