"""Cases of the operators that a batch's step has around its attention: rotary
positions with norms of queries and keys, attention whose scores follow rules (a cap, a
bias by distance, documents, open prefixes), attention over a prefix that the batch
shares, and the next tokens from the logits.

``run`` computes each one either in plain torch operations (``own`` false) or
with libe0moe's entry points (``own`` true), on the same inputs.
"""
import math

import numpy as np
import torch

own = False

_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_CODE = {"f32": 0, "f16": 1, "bf16": 2}
_SIZE = {"f32": 4, "f16": 2, "bf16": 2}
E4M3 = 448.0    # largest e4m3 value


def listed():
    return [
        # queries and keys of a few decode tokens, as they come out of the projection
        {"name": "rope_decode", "op": "rope", "T": 8, "Hq": 16, "Hk": 2, "D": 256, "rot": 64, "axes": 1,
         "adjacent": False, "norm": True, "dtype": "f16"},
        # a long prompt with images: time, height and width
        {"name": "rope_prompt", "op": "rope", "T": 16384, "Hq": 32, "Hk": 4, "D": 128, "rot": 128, "axes": 3,
         "adjacent": False, "norm": True, "dtype": "bf16"},
        # one sequence's next token, the usual truncations
        {"name": "sample_one", "op": "sample", "T": 1, "V": 32000, "dtype": "f32", "top_k": 50, "top_p": 0.95,
         "min_p": 0.0},
        # a batch's next tokens over a large vocabulary, from the nucleus
        {"name": "sample_batch", "op": "sample", "T": 64, "V": 131071, "dtype": "f32", "top_k": 0, "top_p": 0.9,
         "min_p": 0.0},
        # nothing truncated but what is far less likely than the first
        {"name": "sample_open", "op": "sample", "T": 24, "V": 151936, "dtype": "bf16", "top_k": 0, "top_p": 1.0,
         "min_p": 0.001},
        # one decode step of short sequences whose scores lose with the distance
        {"name": "scored_short", "op": "scored", "B": 16, "Hq": 8, "Hkv": 8, "D": 64, "block": 16, "held": 500,
         "new": 1, "window": 0, "cap": 0.0, "slopes": True, "docs": 0, "open": False, "dtype": "f16"},
        # one decode step of long sequences with capped scores
        {"name": "scored_long", "op": "scored", "B": 24, "Hq": 16, "Hkv": 2, "D": 256, "block": 64, "held": 16000,
         "new": 1, "window": 0, "cap": 50.0, "slopes": False, "docs": 0, "open": False, "dtype": "bf16"},
        # a long row of documents that do not see one another
        {"name": "scored_docs", "op": "scored", "B": 1, "Hq": 32, "Hkv": 4, "D": 128, "block": 64, "held": 0,
         "new": 4096, "window": 0, "cap": 0.0, "slopes": False, "docs": 5, "open": False, "dtype": "bf16"},
        # prompts of several lengths behind what is cached, each with a part that all of it sees, capped
        {"name": "scored_open", "op": "scored", "B": 6, "Hq": 16, "Hkv": 4, "D": 128, "block": 32, "held": 900,
         "new": 1500, "window": 0, "cap": 30.0, "slopes": False, "docs": 0, "open": True, "dtype": "f16"},
        # a few short sequences behind a short prompt of all
        {"name": "shared_short", "op": "shared", "B": 8, "Hq": 8, "Hkv": 2, "D": 64, "block": 16, "prefix": 700,
         "held": 200, "new": 1, "dtype": "f16"},
        # a batch behind a prompt in common, two tokens each (one is a guess to be checked), wide heads
        {"name": "shared_wide", "op": "shared", "B": 20, "Hq": 16, "Hkv": 2, "D": 256, "block": 64, "prefix": 6000,
         "held": 900, "new": 2, "dtype": "bf16"},
        # one decode step of a large batch behind a long document
        {"name": "shared_long", "op": "shared", "B": 64, "Hq": 32, "Hkv": 4, "D": 128, "block": 64, "prefix": 16000,
         "held": 600, "new": 1, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "sample", "scored", "shared"])
    dtype = rng.choice(["f16", "bf16", "f16", "bf16", "f32"])
    if op == "rope":
        D = rng.choice([64, 80, 96, 128, 128, 192, 256])
        rot = rng.choice([D, D, D // 2])
        Hk = rng.choice([0, 1, 2, 4, 8])
        Hq = max(1, Hk) * rng.choice([1, 2, 4, 7, 8])
        most = min(16384, 16384 * 36 * 128 // ((Hq + Hk) * D * (2 if dtype == "f32" else 1)))
        return {"op": op, "T": _log(rng, 1, most), "Hq": Hq, "Hk": Hk, "D": D, "rot": rot,
                "axes": rng.choice([1, 1, 2, 3]), "adjacent": rng.random() < 0.4, "norm": rng.random() < 0.7,
                "dtype": dtype}
    if op == "sample":
        V = _log(rng, 100, 160000)
        return {"op": op, "T": _log(rng, 1, min(64, 64 * 131071 // V)), "V": V, "dtype": dtype,
                "top_k": rng.choice([0, 0, 1, 20, 100, 1000]), "top_p": rng.choice([1.0, 0.5, 0.8, 0.95, 0.99]),
                "min_p": rng.choice([0.0, 0.0, 0.02, 0.2])}
    Hkv = rng.choice([1, 2, 4])
    D = rng.choice([64, 128, 256])
    Hq = Hkv * rng.choice([1, 2, 4, 5, 8])
    block = rng.choice([16, 32, 64, 128])
    if op == "scored":
        c = {"op": op, "B": 0, "Hq": Hq, "Hkv": Hkv, "D": D, "block": block, "held": 0, "new": 1,
             "window": rng.choice([0, 0, 0, 150, 1000]), "cap": rng.choice([0.0, 0.0, 20.0, 50.0]),
             "slopes": rng.random() < 0.4, "docs": rng.choice([0, 0, 3]), "open": rng.random() < 0.3, "dtype": dtype}
        if rng.random() < 0.5:  # decode steps
            c["B"] = _log(rng, 1, 48)
            c["held"] = _log(rng, 32, min(16000, 24 * 16000 * 2 * 256 // (c["B"] * Hkv * D)))
            c["new"] = rng.choice([1, 1, 2, 4])
        else:  # prompts; fp32 queries take longer
            c["B"] = _log(rng, 1, 6)
            most = (600 if dtype == "f32" else 4000) // c["B"] + 200
            c["new"] = _log(rng, 16, most)
            c["held"] = rng.choice([0, _log(rng, 1, 1000)])
        return c
    B = _log(rng, 2, 64)
    new = rng.choice([1, 1, 1, 2, 3])
    most = max(200, min(16000, 16000 * 64 * 32 * 128 // (B * new * Hq * D)))
    if dtype == "f32":
        most = min(most, 2000)
    return {"op": op, "B": B, "Hq": Hq, "Hkv": Hkv, "D": D, "block": block, "prefix": _log(rng, 50, most),
            "held": _log(rng, 8, 600), "new": new, "dtype": dtype}


# ------------------------------------------------------------------ inputs


def _lengths(c, rng=None):
    """Tokens held before the step and tokens that join, for each request: the
    case says which lengths there are, the seed (``rng``) who has them."""
    B = c["B"]
    r = np.random.default_rng([B, c["block"], c["held"], c["new"]])
    held = r.integers(0, c["held"] + 1, B)
    if c["new"] == 1:
        new = np.ones(B, np.int64)
    elif c["new"] < 16:
        new = r.integers(0, c["new"] + 1, B)
        new[0] = c["new"]
    else:  # prompts: the longest has c["new"] tokens
        new = r.integers(c["new"] // 4, c["new"] + 1, B)
        new[0] = c["new"]
    who = np.arange(B) if rng is None else rng.permutation(B)
    return held[who], new[who]


def _starts(c, held, new):
    """The first position that each query row sees: where its document begins."""
    out = []
    for b in range(c["B"]):
        n = int(held[b] + new[b])
        r = np.random.default_rng([n, c["docs"]])
        cuts = np.concatenate([[0], np.sort(r.integers(0, n + 1, c["docs"] - 1))])
        at = np.arange(held[b], n)
        out.append(cuts[np.searchsorted(cuts, at, side="right") - 1])
    return np.concatenate(out).astype(np.int32)


def _open(held, new):
    """How many positions all queries of a request see."""
    return ((held + new) * 2 // 5).astype(np.int32)


def _axes_of(c):
    """Which axis each pair turns by: one after another, as time, height, width."""
    half = c["rot"] // 2
    return (np.arange(half) * c["axes"] // half).astype(np.uint8)


def _pow2_scale(m):
    """The smallest power of two s, at least 2^-100, with m <= 448 s (fp32)."""
    b = (m / E4M3).view(torch.int32)
    e = ((b >> 23) & 255) + ((b & 0x7FFFFF) != 0).int()
    return (e.clamp(min=27) << 23).view(torch.float32)


def prepare(case, seed):
    c = dict(case)
    rng = np.random.default_rng([int(seed), 7])
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    s = {"case": c}

    def normal(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=g, device="cuda").to(dtype)

    def dev(a):
        return torch.from_numpy(np.ascontiguousarray(a)).cuda()

    if c["op"] == "rope":
        T, heads, D = c["T"], c["Hq"] + c["Hk"], c["D"]
        dt = _DT[c["dtype"]]
        s["x"] = (normal(T, heads, D) * torch.exp(0.5 * normal(T, heads, 1))).to(dt)
        s["y"] = torch.empty_like(s["x"])
        half = c["rot"] // 2
        s["freq"] = dev((1e6 ** (-np.arange(half) / half)).astype(np.float32))
        s["axis"] = dev(_axes_of(c))
        if c["axes"] == 1 and T <= 64:  # decode tokens of sequences of any age
            pos = rng.integers(0, 200000, (1, T))
        else:
            pos = int(rng.integers(0, 5000)) + np.arange(T)[None, :].repeat(c["axes"], 0)
            for a in range(1, c["axes"]):  # rows and columns of images
                pos[a] = pos[0] - np.arange(T) + (np.arange(T) // 64 if a == 1 else np.arange(T) % 64)
        s["pos"] = dev(pos.astype(np.int32))
        s["wq"] = 1 + 0.2 * normal(D) if c["norm"] else None
        s["wk"] = 1 + 0.2 * normal(D) if c["norm"] else None
        if own:
            from int4_gathered_expert_gb300 import lib as L
            s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
            flags = (L.E0_ROPE_ADJACENT if c["adjacent"] else 0) | (L.E0_QK_NORM if c["norm"] else 0)
            s["desc"] = L.Rope(s["freq"].data_ptr(), s["axis"].data_ptr() if c["axes"] > 1 else None,
                               L.ptr(s["wq"]), L.ptr(s["wk"]), D, c["rot"], c["axes"], flags, 1e-6)
        return s
    if c["op"] == "sample":
        T, V = c["T"], c["V"]
        x = 2.0 * normal(T, V)
        some = torch.randint(0, V, (T, 40), generator=g, device="cuda")  # a few tokens stand out, more or less
        up = 4 + 4 * torch.rand((T, 40), generator=g, device="cuda")
        s["x"] = x.scatter_add(1, some, up).to(_DT[c["dtype"]])
        s["u"] = torch.rand(T, generator=g, device="cuda")
        s["temp"] = 0.6 + 0.6 * torch.rand(T, generator=g, device="cuda")
        s["k"] = torch.full((T,), c["top_k"], dtype=torch.int32, device="cuda")
        s["p"] = torch.full((T,), c["top_p"], device="cuda")
        s["mp"] = torch.full((T,), c["min_p"], device="cuda")
        s["token"] = torch.empty(T, dtype=torch.int32, device="cuda")
        s["kept"] = torch.empty(T, dtype=torch.int32, device="cuda")
        s["logp"] = torch.empty(T, device="cuda")
        if own:
            from int4_gathered_expert_gb300 import lib as L
            s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
            s["rules"] = L.Sampling(s["temp"].data_ptr(), s["k"].data_ptr() if c["top_k"] else None,
                                    s["p"].data_ptr() if c["top_p"] < 1 else None,
                                    s["mp"].data_ptr() if c["min_p"] else None)
        return s
    held, new = _lengths(c, rng)
    B, Hq, Hkv, D, bs = c["B"], c["Hq"], c["Hkv"], c["D"], c["block"]
    shared = c["prefix"] if c["op"] == "shared" else 0
    T = int(new.sum())
    # a pool of blocks in no particular order, and who has which
    need = -(-(held + new) // bs)
    front = -(-shared // bs)
    n = int((need.sum() + front) * 9 // 8 + 8)
    ids = rng.permutation(n).astype(np.int32)
    width = int(max(1, need.max()) + 2)
    table = np.full((B, width), -1, np.int32)
    at = front
    for b in range(B):
        table[b, :need[b]] = ids[at:at + need[b]]
        at += int(need[b])
    cu = np.zeros(B + 1, np.int32)
    cu[1:] = np.cumsum(new)
    s.update(T=T, n=n, width=width, max_q=int(new.max()), table=dev(table), cu=dev(cu),
             ctx=dev((held + new).astype(np.int32)), sm=1.5 / math.sqrt(D))
    for name in ("k", "v"):  # normal keys and values, their size by block and head
        size = torch.exp(0.5 * normal(n, Hkv))
        x = normal(n, Hkv, bs, D) * size[:, :, None, None]
        s[name + "s"] = _pow2_scale(x.abs().amax((2, 3)))
        s[name] = (x / s[name + "s"][:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    dt = _DT[c["dtype"]]
    s["q"] = normal(T, Hq, D, dtype=dt)
    s["o"], s["lse"] = torch.empty_like(s["q"]), torch.empty((T, Hq), device="cuda")
    if shared:
        s["ptable"], s["plen"] = dev(ids[:front]), dev(np.array([shared], np.int32))
    else:
        s["slopes"] = dev(2.0 ** (-8.0 * np.arange(1, Hq + 1) / Hq)).float() if c["slopes"] else None
        s["first"] = dev(_starts(c, held, new)) if c["docs"] else None
        s["open"] = dev(_open(held, new)) if c["open"] else None
    if own:
        from int4_gathered_expert_gb300 import lib as L
        s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        s["desc"] = L.KvCache(s["k"].data_ptr(), s["v"].data_ptr(), s["ks"].data_ptr(), s["vs"].data_ptr(), n, Hkv,
                              bs, D)
        if shared:
            s["rules"] = None
            s["ws_bytes"] = L.e0_attn_shared_workspace_size(B, T, Hq, Hkv, D, s["max_q"])
        else:
            s["rules"] = L.AttnRules(c["cap"], c["window"], L.ptr(s["slopes"]), L.ptr(s["first"]), L.ptr(s["open"]))
            s["ws_bytes"] = L.e0_attn_scored_workspace_size(B, Hq, Hkv, D, s["max_q"])
        s["ws"] = torch.empty(s["ws_bytes"], dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------ the plain forms


def _rope_plain(s):
    c = s["case"]
    x = s["x"].float()
    if c["norm"]:
        x = x / torch.sqrt((x * x).mean(2, keepdim=True) + 1e-6)
        w = torch.cat([s["wq"][None].expand(c["Hq"], -1), s["wk"][None].expand(c["Hk"], -1)])
        x = x * w[None]
    half = c["rot"] // 2
    angle = s["pos"][s["axis"].long()].double().t() * s["freq"].double()  # far positions: 64 bits
    cos, sin = torch.cos(angle).float()[:, None, :], torch.sin(angle).float()[:, None, :]
    turned, rest = x[:, :, :c["rot"]], x[:, :, c["rot"]:]
    if c["adjacent"]:
        a, b = turned[:, :, 0::2], turned[:, :, 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], 3).reshape(turned.shape)
    else:
        a, b = turned[:, :, :half], turned[:, :, half:]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], 2)
    return {"y": torch.cat([turned, rest], 2).to(s["x"].dtype)}


def _sample_plain(s):
    c = s["case"]
    T, V = c["T"], c["V"]
    x, order = torch.sort(s["x"].float(), dim=1, descending=True, stable=True)  # ties: the lower token first
    # long sums and values next to borders: 64 bits
    d = (x.double() - x[:, :1].double()) / s["temp"].double()[:, None]
    w = torch.exp(d)
    i = torch.arange(V, device=w.device)[None, :]
    n_k = torch.where(s["k"] > 0, s["k"].clamp(max=V), torch.full_like(s["k"], V)).long()[:, None]
    cum = (w * (i < n_k)).cumsum(1)
    before = torch.cat([torch.zeros_like(cum[:, :1]), cum[:, :-1]], 1)
    kept = (i < n_k) & ((before < s["p"].double()[:, None] * cum[:, -1:]) | (i == 0))
    kept = kept & (w >= s["mp"].double()[:, None])
    mask = torch.zeros((T, V), dtype=torch.bool, device=w.device).scatter(1, order, kept)
    y = torch.exp((s["x"].double() - x[:, :1].double()) / s["temp"].double()[:, None]) * mask
    run_ = y.cumsum(1)
    total = run_[:, -1:]
    token = (run_ <= s["u"].double()[:, None] * total).sum(1).clamp(max=V - 1)
    logp = torch.log(y.gather(1, token[:, None]) / total)[:, 0]
    return {"token": token.int(), "kept": kept.sum(1).int(), "logp": logp.float()}


def _rows(s):
    """For [B, max_q] query places: the row of q (its number of rows: none)."""
    cu = s["cu"].long()
    i = torch.arange(s["max_q"], device=cu.device)[None, :]
    n = (cu[1:] - cu[:-1])[:, None]
    return torch.where(i < n, cu[:-1, None] + i, torch.full_like(i, s["T"])), n, i


def _held(s, name, ids):
    """Keys or values of block ids [B, blocks] as fp32 [B, Hkv, tokens, D]."""
    x = s[name][ids].view(torch.float8_e4m3fn).float() * s[name + "s"][ids][..., None, None]
    B, n, H, bs, D = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(B, H, n * bs, D)


def _scored_plain(s):
    c = s["case"]
    B, Hq, Hkv, D, M = c["B"], c["Hq"], c["Hkv"], c["D"], s["max_q"]
    ids = s["table"][:, :s["width"] - 2].long().clamp(min=0)
    S = ids.shape[1] * c["block"]
    row, n, i = _rows(s)
    ctx = s["ctx"].long()[:, None]
    q = torch.cat([s["q"].float(), torch.zeros((1, Hq, D), device=row.device)])[row]
    q = q.view(B, M, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    x = (q @ _held(s, "k", ids).transpose(2, 3)).view(B, Hkv, Hq // Hkv, M, S) * s["sm"]
    if c["cap"]:
        x = c["cap"] * torch.tanh(x / c["cap"])
    p = (ctx - n + i)[:, :, None]
    j = torch.arange(S, device=row.device)[None, None, :]
    if s["slopes"] is not None:
        x = x - s["slopes"].view(1, Hkv, -1, 1, 1) * (p - j).abs()[:, None, None].float()
    seen = j <= p
    if s["open"] is not None:
        seen = seen | (j < s["open"].long()[:, None, None])
    seen = seen & (j < ctx[:, :, None])
    if s["first"] is not None:
        seen = seen & (j >= torch.cat([s["first"].long(), torch.zeros_like(row[0, :1])])[row][:, :, None])
    if c["window"]:
        seen = seen & (j > p - c["window"])
    x = torch.where(seen[:, None, None], x, torch.full_like(x, -torch.inf))
    m = x.amax(4, keepdim=True)
    m = torch.where(m == -torch.inf, torch.zeros_like(m), m)
    e = torch.exp(x - m)
    z = e.sum(4, keepdim=True)
    o = (e.reshape(B, Hkv, -1, S) @ _held(s, "v", ids)).view(B, Hkv, Hq // Hkv, M, D)
    o = o / torch.where(z == 0, torch.ones_like(z), z)
    return _scatter(s, row, o, (m + torch.log(z)).squeeze(4))


def _scatter(s, row, o, lse):
    """[B, Hkv, group, M, ...] back to the rows of q."""
    B, M = row.shape
    T, Hq, D = s["q"].shape
    out = torch.empty((T + 1, Hq, D), device=o.device)
    out[row] = o.permute(0, 3, 1, 2, 4).reshape(B, M, Hq, D)
    l2 = torch.empty((T + 1, Hq), device=o.device)
    l2[row] = lse.permute(0, 3, 1, 2).reshape(B, M, Hq)
    return {"o": out[:-1].to(s["q"].dtype), "lse": l2[:-1]}


def _shared_plain(s):
    c = s["case"]
    B, Hq, Hkv, D, M = c["B"], c["Hq"], c["Hkv"], c["D"], s["max_q"]
    G = Hq // Hkv
    P = c["prefix"]
    row, n, i = _rows(s)
    ctx = s["ctx"].long()[:, None]
    q = torch.cat([s["q"].float(), torch.zeros((1, Hq, D), device=row.device)])[row]
    q = q.view(B, M, Hkv, G, D).permute(0, 2, 3, 1, 4)  # B, Hkv, G, M, D
    front = s["ptable"].long()[None]
    # the prefix once, for the rows of all sequences
    k, v = _held(s, "k", front)[0, :, :P], _held(s, "v", front)[0, :, :P]
    qa = q.permute(1, 0, 2, 3, 4).reshape(Hkv, -1, D)
    xp = (qa @ k.transpose(1, 2)) * s["sm"]
    ids = s["table"][:, :s["width"] - 2].long().clamp(min=0)
    S = ids.shape[1] * c["block"]
    xo = (q.reshape(B, Hkv, -1, D) @ _held(s, "k", ids).transpose(2, 3)).view(B, Hkv, G, M, S) * s["sm"]
    j = torch.arange(S, device=row.device)[None, None, :]
    seen = j <= (ctx - n + i)[:, :, None]
    xo = torch.where(seen[:, None, None], xo, torch.full_like(xo, -torch.inf))
    mp = xp.amax(2).view(Hkv, B, G, M).transpose(0, 1)
    m = torch.maximum(mp, xo.amax(4))
    ep = torch.exp(xp - m.transpose(0, 1).reshape(Hkv, -1, 1))
    eo = torch.exp(xo - m[..., None])
    z = ep.sum(2).view(Hkv, B, G, M).transpose(0, 1) + eo.sum(4)
    o = (ep @ v).view(Hkv, B, G, M, D).transpose(0, 1)
    o = o + (eo.reshape(B, Hkv, -1, S) @ _held(s, "v", ids)).view(B, Hkv, G, M, D)
    return _scatter(s, row, o / z[..., None], m + torch.log(z))


# ------------------------------------------------------------------ the framework's calls


def _own(s):
    from int4_gathered_expert_gb300 import lib as L
    c = s["case"]
    if c["op"] == "rope":
        ld = (c["Hq"] + c["Hk"]) * c["D"]
        L.e0_qk_rope(s["x"], _CODE[c["dtype"]], ld, c["T"], c["Hq"], c["Hk"], s["desc"], s["pos"], c["T"], s["y"], ld,
                     s["status"])
        return {"y": s["y"]}
    if c["op"] == "sample":
        L.e0_sample(s["x"], _CODE[c["dtype"]], c["V"], c["T"], c["V"], s["rules"], s["u"], s["token"], s["logp"],
                    s["kept"], s["status"])
        return {"token": s["token"], "kept": s["kept"], "logp": s["logp"]}
    row = c["Hq"] * c["D"]
    if c["op"] == "scored":
        L.e0_attn_scored(s["desc"], s["table"], s["width"], s["ctx"], s["cu"], c["B"], s["max_q"], s["q"],
                         _CODE[c["dtype"]], row, c["Hq"], s["sm"], s["rules"], s["o"], row, s["lse"], s["ws"],
                         s["ws_bytes"], s["status"])
    else:
        L.e0_attn_shared(s["desc"], s["ptable"], len(s["ptable"]), s["plen"], s["table"], s["width"], s["ctx"],
                         s["cu"], c["B"], s["T"], s["max_q"], s["q"], _CODE[c["dtype"]], row, c["Hq"], s["sm"],
                         s["rules"], s["o"], row, s["lse"], s["ws"], s["ws_bytes"], s["status"])
    return {"o": s["o"], "lse": s["lse"]}


def run(state):
    if own:
        return _own(state)
    return {"rope": _rope_plain, "sample": _sample_plain, "scored": _scored_plain,
            "shared": _shared_plain}[state["case"]["op"]](state)


def work(case):
    c = case
    if c["op"] == "rope":
        n = c["T"] * (c["Hq"] + c["Hk"]) * c["D"]
        return {"bytes": 2 * n * _SIZE[c["dtype"]] + 4 * c["T"] * c["axes"] + 8 * c["D"] * c["norm"],
                "flops": n * (3 + 4 * c["norm"])}
    if c["op"] == "sample":
        return {"bytes": c["T"] * (c["V"] * _SIZE[c["dtype"]] + 32), "flops": 8 * c["T"] * c["V"]}
    held, new = _lengths(c)
    T = int(new.sum())
    row = 2 * c["Hq"] * c["D"] * _SIZE[c["dtype"]] + 4 * c["Hq"]
    if c["op"] == "shared":
        own_pairs = int(sum((held[b] + np.arange(1, new[b] + 1)).sum() for b in range(c["B"])))
        tokens = c["prefix"] + int((held + new)[new > 0].sum())
        return {"bytes": tokens * c["Hkv"] * c["D"] * 2 + T * row,
                "flops": 4 * (own_pairs + T * c["prefix"]) * c["Hq"] * c["D"]}
    pairs = tokens = at = 0
    starts = _starts(c, held, new) if c["docs"] else None
    opens = _open(held, new) if c["open"] else np.zeros(c["B"], np.int64)
    for b in range(c["B"]):
        if new[b] == 0:
            continue
        p = np.arange(held[b], held[b] + new[b])
        hi = np.maximum(p + 1, opens[b])
        lo = np.zeros_like(p) if starts is None else starts[at:at + new[b]]
        if c["window"]:
            lo = np.maximum(lo, p - c["window"] + 1)
        at += int(new[b])
        pairs += int(np.maximum(hi - lo, 0).sum())
        tokens += int(max(0, hi.max() - lo.min()))
    return {"bytes": tokens * c["Hkv"] * c["D"] * 2 + T * row, "flops": 4 * pairs * c["Hq"] * c["D"]}


# ------------------------------------------------------------------ the definitions, in 64 bits


def _exact_tokens(s, table_row, n):
    """The first n tokens of a row of block ids, [n, Hkv, D] in 64 bits."""
    bs = s["case"]["block"]
    ids = table_row[:-(-n // bs)].long()
    out = []
    for name in ("k", "v"):
        codes = s[name][ids].view(torch.float8_e4m3fn).double()
        out.append((codes * s[name + "s"][ids].double()[:, :, None, None]).transpose(1, 2).flatten(0, 1)[:n])
    return out


def exact(case, seed):
    keep, globals()["own"] = own, False
    try:
        s = prepare(case, seed)
    finally:
        globals()["own"] = keep
    c = s["case"]
    f64 = torch.float64
    if c["op"] == "rope":
        y = s["x"].to(f64).clone()
        if c["norm"]:
            y *= torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6)
            y[:, :c["Hq"]] *= s["wq"].to(f64)
            y[:, c["Hq"]:] *= s["wk"].to(f64)
        axis = _axes_of(c)
        half = c["rot"] // 2
        for i in range(half):
            a = s["pos"][int(axis[i])].to(f64) * s["freq"][i].to(f64)
            e0, e1 = (2 * i, 2 * i + 1) if c["adjacent"] else (i, i + half)
            z = torch.complex(y[:, :, e0], y[:, :, e1]) * torch.polar(torch.ones_like(a), a)[:, None]
            y[:, :, e0], y[:, :, e1] = z.real, z.imag
        return {"y": y}
    if c["op"] == "sample":
        x = s["x"].to(f64).cpu().numpy()
        logp, token, kept = np.zeros(c["T"]), np.zeros(c["T"], np.int64), np.zeros(c["T"], np.int64)
        for t in range(c["T"]):
            z = x[t] / float(s["temp"][t])
            best = np.lexsort((np.arange(c["V"]), -x[t]))
            w = np.exp(z[best] - z.max())
            if c["top_k"]:
                w = w[:c["top_k"]]
            n = 1 + int(np.searchsorted(np.cumsum(w), float(s["p"][t]) * w.sum())) if c["top_p"] < 1 else len(w)
            n = min(n, len(w), int((w >= float(s["mp"][t])).sum()))
            who = np.sort(best[:n])
            w = np.exp(z[who] - z.max())
            at = min(int(np.searchsorted(np.cumsum(w), float(s["u"][t]) * w.sum(), side="right")), n - 1)
            token[t], kept[t], logp[t] = who[at], n, math.log(w[at] / w.sum())
        return {"token": token, "kept": kept, "logp": logp}
    o = torch.zeros(s["q"].shape, dtype=f64, device="cuda")
    lse = torch.zeros(s["lse"].shape, dtype=f64, device="cuda")
    ctx, cu, Hkv = s["ctx"].tolist(), s["cu"].tolist(), c["Hkv"]
    G = c["Hq"] // Hkv
    shared = c.get("prefix", 0)
    if shared:
        front = _exact_tokens(s, s["ptable"], shared)
    for b in range(c["B"]):
        n = cu[b + 1] - cu[b]
        if n == 0:
            continue
        k, v = _exact_tokens(s, s["table"][b], ctx[b])
        if shared:
            k, v = torch.cat([front[0], k]), torch.cat([front[1], v])
        j = torch.arange(len(k), device="cuda")
        p = shared + ctx[b] - n + torch.arange(n, device="cuda")
        hidden = j[None, :] > p[:, None]
        if not shared:
            if c["open"]:
                hidden &= (j >= int(s["open"][b]))[None, :]
            if c["docs"]:
                hidden |= j[None, :] < s["first"][cu[b]:cu[b + 1], None]
            if c["window"]:
                hidden |= j[None, :] <= p[:, None] - c["window"]
        for h in range(c["Hq"]):
            x = s["q"][cu[b]:cu[b + 1], h].to(f64) @ k[:, h // G].t() * s["sm"]
            if not shared:
                if c["cap"]:
                    x = c["cap"] * torch.tanh(x / c["cap"])
                if c["slopes"]:
                    x -= float(s["slopes"][h]) * (p[:, None] - j[None, :]).abs()
            x = x.masked_fill(hidden, -math.inf)
            lse[cu[b]:cu[b + 1], h] = torch.logsumexp(x, 1)
            o[cu[b]:cu[b + 1], h] = torch.softmax(x, 1).nan_to_num(0.0) @ v[:, h // G]
    return {"o": o, "lse": lse}
