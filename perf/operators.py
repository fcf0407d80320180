"""Workloads of the rotary, query/key norm and sliding-window anchor operators.

Each case is one call (or one training step) as a user's program makes it.  `run` computes it in
plain torch operations, or through softmax_attention_sana_b200 where `own` is true; `exact` gives
the same result from the definitions in 64 bits.

Conventions: token tensors are (B, N, heads * D); a query at absolute position p of a sequence sees
the keys j < min(e, length) with j >= e - window or j < sinks, where e = (p // block + 1) * block is
the end of its own block (block = 1: causal) and window = 0 means no limit.
"""

import math

import numpy as np
import torch

own = False

EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------------- the cases

def listed():
    return [
        # one decoding step of a small batch: only the rotation of 32 query and 8 key heads; latency
        dict(name="rotary_step", op="rotary", dtype="bf16", B=8, N=1, heads=32, kv_heads=8, D=128,
             rot=128, layout="half", scaling="none", theta=500000.0, offset=8000, scattered=True),
        # the last 8191 tokens of a 131072-token context: part of the head, YaRN-scaled, fp32
        dict(name="rotary_long_f32", op="rotary", dtype="f32", B=1, N=8191, heads=16, kv_heads=4,
             D=128, rot=64, layout="interleaved", scaling="yarn", theta=10000.0, offset=122881,
             scattered=False),
        # one decoding step: norm and rotation of the new tokens' queries and keys; latency
        dict(name="qk_norm_rope_step", op="qk_norm_rope", dtype="bf16", B=16, N=1, heads=32,
             kv_heads=8, D=128, rot=128, layout="half", scaling="linear", theta=10000.0,
             offset=30000, scattered=True, T=0, H=0, W=0),
        # a 480p clip's latent grid with the 3D rotary tables of the anchors
        dict(name="qk_norm_rope_480p", op="qk_norm_rope", dtype="bf16", B=1, N=32760, heads=16,
             kv_heads=16, D=128, rot=128, layout="interleaved", scaling="none", theta=10000.0,
             offset=0, scattered=False, T=21, H=30, W=52),
        # a training step's forward and backward over two odd-length sequences
        dict(name="qk_norm_rope_train", op="qk_norm_rope_train", dtype="bf16", B=2, N=4001,
             heads=32, kv_heads=8, D=128, rot=128, layout="half", scaling="ntk", theta=10000.0,
             offset=0, scattered=False, T=0, H=0, W=0),
        # a small padded batch of short prompts
        dict(name="window_short", op="window", B=3, N=333, heads=8, kv_heads=2, window=100,
             sinks=4, block=1, ragged=True, gate=False, past=0),
        # a long prompt with a short window and four sink tokens
        dict(name="window_prompt", op="window", B=1, N=32768, heads=32, kv_heads=8, window=4096,
             sinks=4, block=1, ragged=False, gate=False, past=0),
        # twelve 480p latent frames in blocks of three, window of two blocks, first frame as sink
        dict(name="window_video", op="window", B=1, N=18720, heads=16, kv_heads=16, window=9360,
             sinks=1560, block=4680, ragged=False, gate=True, past=0),
        # a training step on a small batch with a narrow window
        dict(name="window_train_small", op="window_train", B=2, N=1023, heads=8, kv_heads=8,
             window=256, sinks=1, block=1, ragged=True, gate=True, past=0),
        # a training step on one long sequence, four query heads to a key head
        dict(name="window_train", op="window_train", B=1, N=16384, heads=16, kv_heads=4,
             window=2048, sinks=16, block=1, ragged=False, gate=False, past=0),
        # one decoding step of a few sequences over ring caches of sinks and window; latency
        dict(name="decode_step", op="window_decode", B=4, N=1, heads=32, kv_heads=8, window=1024,
             sinks=4, capacity=1028, gate=False),
        # one decoding step of a large batch over long ring caches, eight query heads to a key head
        dict(name="decode_batch", op="window_decode", B=64, N=1, heads=16, kv_heads=2, window=8192,
             sinks=128, capacity=8448, gate=True),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "qk_norm_rope", "qk_norm_rope_train", "window", "window",
                     "window_train", "window_train", "window_decode", "window_decode"])
    kv_heads = rng.choice([1, 2, 3, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 4, 5, 8])
    if op in ("rotary", "qk_norm_rope", "qk_norm_rope_train"):
        D = rng.choice([64, 128, 128, 256])
        video = op != "rotary" and rng.random() < 0.3
        c = dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), B=_log(rng, 1, 16), heads=heads,
                 kv_heads=kv_heads, D=D, theta=rng.choice([10000.0, 500000.0]))
        most = 32760 * 32 * 128 // (4 if "train" in op else 2 if c["dtype"] == "f32" else 1)
        if video:
            T, H, W = rng.randint(1, 13), rng.randint(3, 30), rng.randint(3, 40)
            while c["B"] * T * H * W * (heads + kv_heads) * D > most and c["B"] * T > 1:
                T, c["B"] = max(1, T // 2), max(1, c["B"] // 2)
            c.update(N=T * H * W, rot=D, layout="interleaved", scaling="none", offset=0,
                     theta=10000.0, scattered=False, T=T, H=H, W=W)
        else:
            most = max(1, most // (c["B"] * (heads + kv_heads) * D))
            c.update(N=_log(rng, 1, min(8192, most)), layout=rng.choice(["half", "interleaved"]),
                     scaling=rng.choice(["none", "linear", "ntk", "yarn"]),
                     rot=D if rng.random() < 0.6 else D // 2, offset=_log(rng, 1, 100000) - 1,
                     scattered=rng.random() < 0.3)
            if op != "rotary":
                c.update(T=0, H=0, W=0)
        return c
    if op == "window_decode":
        sinks = rng.choice([0, 1, 4, 64])
        N = rng.choice([1, 1, 1, 2, 4])
        window = _log(rng, 64, 8192)
        B = max(1, min(_log(rng, 1, 64), 64 * 2 * 8192 // (kv_heads * window)))
        return dict(op=op, B=B, N=N, heads=heads, kv_heads=kv_heads, window=window, sinks=sinks,
                    capacity=sinks + window + N + rng.choice([0, 3, 100]), gate=rng.random() < 0.5)
    most = 16384 if op == "window" else 6000
    N = _log(rng, 1 if op == "window" else 64, most)  # a training row that sees one key has no gradient
    B = max(1, min(_log(rng, 1, 4), 16384 // N))
    heads = heads if heads * B * N <= 16 * 16384 else kv_heads
    block = 1 if rng.random() < 0.7 else _log(rng, 2, 700)
    window = max(block, _log(rng, 1 if op == "window" else 16, 4096))
    past = 0 if op == "window_train" or rng.random() < 0.6 else _log(rng, 1, 2000)
    return dict(op=op, B=B, N=N, heads=heads, kv_heads=kv_heads, window=window,
                sinks=rng.choice([0, 1, 4, 200]), block=block, ragged=rng.random() < 0.4,
                gate=rng.random() < 0.5, past=past)


def _lengths(c):
    """Tokens of each padded sequence, or None where all are whole."""
    if not c["ragged"]:
        return None
    total = c["N"] + c["past"]
    return [max(0, total - (b * (2 * total + 1)) // (2 * c["B"])) for b in range(c["B"])]


def _held(c):
    """Tokens already in each cache: some wrapped round, some short, the last one empty."""
    return [(b + 1) * 2 * c["capacity"] // c["B"] - b if b + 1 < c["B"] or c["B"] == 1 else 0
            for b in range(c["B"])]


# ------------------------------------------------------------------------------------ the inputs

def _frequencies(c):
    """Angle per position of each rotary pair and the factor on cosine and sine, in 64 bits."""
    half = c["rot"] // 2
    k = np.arange(half, dtype=np.float64)
    inv, mul = c["theta"] ** (-k / half), 1.0
    if c["scaling"] == "linear":
        inv = inv / 4.0
    elif c["scaling"] == "ntk":
        inv = (c["theta"] * 4.0 ** (c["rot"] / (c["rot"] - 2.0))) ** (-k / half)
    elif c["scaling"] == "yarn":
        at = lambda turns: c["rot"] * math.log(16384 / (turns * 2 * math.pi)) / (2 * math.log(c["theta"]))  # noqa: E731
        lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), half - 1)
        slow = np.clip((k - lo) / max(hi - lo, 1e-3), 0.0, 1.0)
        inv, mul = inv * (1.0 - slow) + inv / 8.0 * slow, 0.1 * math.log(8.0) + 1.0
    return inv, mul


SCALING = {"none": None, "linear": ("linear", 4.0), "ntk": ("ntk", 4.0), "yarn": ("yarn", 8.0, 16384)}


def _axes(D):
    """Rotary pairs of the frame, row and column axes of a video grid."""
    side = D // 2 // 3
    return D // 2 - 2 * side, side, side


def _angles(c, positions):
    """(B or 1, N, pairs) angles in 64 bits on the GPU, and the factor."""
    if c.get("T"):
        n = torch.arange(c["N"], device="cuda")
        at = (n // (c["H"] * c["W"]), n // c["W"] % c["H"], n % c["W"])
        parts = []
        for p, pairs in zip(at, _axes(c["D"])):
            inv = c["theta"] ** (-torch.arange(pairs, device="cuda", dtype=torch.float64) / pairs)
            parts.append(p[:, None].double() * inv)
        return torch.cat(parts, dim=1)[None], 1.0
    inv, mul = _frequencies(c)
    p = positions if positions is not None else (
        torch.arange(c["N"], device="cuda")[None] + c["offset"])
    return p.double()[..., None] * torch.as_tensor(inv, device="cuda"), mul


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype=torch.bfloat16, scale=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)

    st = {"case": c}
    if c["op"] in ("rotary", "qk_norm_rope", "qk_norm_rope_train"):
        B, N, D, dt = c["B"], c["N"], c["D"], DTYPES[c["dtype"]]
        # queries, keys and values come side by side out of one projection
        qkv = normal(B, N, (c["heads"] + 2 * c["kv_heads"]) * D, dtype=dt, scale=1.5)
        st["q"], st["k"], _ = qkv.split([c["heads"] * D, c["kv_heads"] * D, c["kv_heads"] * D], dim=2)
        top = c["offset"] + N
        st["positions"] = None
        if c["scattered"]:  # every sequence of the batch is somewhere else
            start = torch.randint(0, c["offset"] + 1, (B, 1), generator=gen, device="cuda")
            st["positions"] = (start + torch.arange(N, device="cuda")[None]).int()
        if c["op"] != "rotary":
            st["wq"] = 1.0 + 0.2 * normal(D, dtype=torch.float32)
            st["wk"] = 1.0 + 0.2 * normal(D, dtype=torch.float32)
        if c["op"] == "qk_norm_rope_train":
            st["dq"] = normal(B, N, c["heads"] * D, dtype=dt)
            st["dk"] = normal(B, N, c["kv_heads"] * D, dtype=dt)
        if own:
            import softmax_attention_sana_b200 as sana
            if c.get("T"):
                st["rotary"] = sana.Rope(c["T"], c["H"], c["W"], _axes(D), theta=c["theta"])
            else:
                st["rotary"] = sana.Rotary(top, c["rot"], theta=c["theta"], layout=c["layout"],
                                           scaling=SCALING[c["scaling"]])
        else:
            ang, mul = _angles(c, st["positions"])
            st["cos"], st["sin"] = (torch.cos(ang) * mul).float(), (torch.sin(ang) * mul).float()
        return st
    B, N, D = c["B"], c["N"], 128
    st["q"] = normal(B, N, c["heads"] * D)
    if c["op"] == "window_decode":
        st["k"], st["v"] = (normal(B, N, c["kv_heads"] * D) for _ in range(2))
        st["k_cache"], st["v_cache"] = (normal(B, c["capacity"], c["kv_heads"] * D) for _ in range(2))
        st["lengths"] = torch.tensor(_held(c), dtype=torch.int32, device="cuda")
    else:
        st["k"], st["v"] = (normal(B, N + c["past"], c["kv_heads"] * D) for _ in range(2))
        held = _lengths(c)
        st["lengths"] = None if held is None else torch.tensor(held, dtype=torch.int32, device="cuda")
    st["gate"] = normal(B, N, c["heads"] * D, scale=2.0) if c["gate"] else None
    if c["op"] == "window_train":
        st["dy"] = normal(B, N, c["heads"] * D)
    return st


# --------------------------------------------------------------------------- the plain operators

def _turn(x, cos, sin, layout, back=False):
    """Rotate the first 2 * pairs elements of the last dimension (back: the transposed rotation)."""
    if back:
        sin = -sin
    R = 2 * cos.shape[-1]
    r, rest = x[..., :R], x[..., R:]
    if layout == "half":
        a, b = r[..., :R // 2], r[..., R // 2:]
        return torch.cat([a * cos - b * sin, a * sin + b * cos, rest], dim=-1)
    a, b = r[..., 0::2], r[..., 1::2]
    return torch.cat([torch.stack([a * cos - b * sin, a * sin + b * cos], dim=-1).flatten(-2), rest],
                     dim=-1)


def _split(x, D):
    return x.unflatten(2, (-1, D)).float()


def _plain_rotary(st):
    c, cos, sin = st["case"], st["cos"][:, :, None], st["sin"][:, :, None]
    return [_turn(_split(x, c["D"]), cos, sin, c["layout"]).flatten(2).to(x.dtype)
            for x in (st["q"], st["k"])]


def _plain_norm(st, train):
    c, cos, sin = st["case"], st["cos"][:, :, None], st["sin"][:, :, None]
    outs, grads, weights = [], [], []
    for x, w, dy in ((st["q"], st["wq"], st.get("dq")), (st["k"], st["wk"], st.get("dk"))):
        xf = _split(x, c["D"])
        r = torch.rsqrt((xf * xf).mean(-1, keepdim=True) + EPS)
        outs.append(_turn(xf * r * w, cos, sin, c["layout"]).flatten(2).to(x.dtype))
        if train:
            g = _turn(_split(dy, c["D"]), cos, sin, c["layout"], back=True)
            xh = xf * r
            weights.append((g * xh).sum((0, 1, 2)))
            g = g * w
            grads.append((r * (g - xh * (g * xh).mean(-1, keepdim=True))).flatten(2).to(x.dtype))
    return outs + grads + weights


def _banded(st):
    """Queries in groups of whole blocks, with the keys that any row of the group can see: index
    (groups, keys) into the keys (clamped) and which of them each row sees (B or 1, groups, rows, keys)."""
    c, dev = st["case"], st["q"].device
    N, past, P, total = c["N"], c["past"], c["block"], c["N"] + c["past"]
    W = c["window"] if c["window"] else total + P
    rows = P * max(1, 512 // P)
    groups = (past + N - 1) // rows - past // rows + 1
    first = (past // rows + torch.arange(groups, device=dev)) * rows   # position of each group's first row
    pos = first[:, None] + torch.arange(rows, device=dev)
    wide = min(W + rows - P, total + rows)
    near = first[:, None] + rows - wide + torch.arange(wide, device=dev)
    sink = torch.arange(c["sinks"], device=dev).expand(groups, -1)
    length = (torch.full((1,), total, device=dev) if st["lengths"] is None else st["lengths"])
    length = length.view(-1, 1, 1, 1)
    end = (pos // P + 1) * P
    low = end - W
    sees_near = (near[:, None] >= low[..., None]) & (near[:, None] < end[..., None]) & (near[:, None] >= 0)
    sees_sink = (sink[:, None] < low[..., None]) & (sink[:, None] < end[..., None])
    # a sink that is also within the group's near keys is taken once, as a sink, by the rows whose window it left
    keys = torch.cat([sink, near], dim=1)
    sees = torch.cat([sees_sink, sees_near], dim=2)[None]
    live = (pos >= past)[None, :, :, None] & (pos[None, :, :, None] < length)
    sees = sees & live & (keys[None, :, None, :] < length)
    return keys.clamp(0, total - 1), sees, rows, groups


def _grouped(x, st, rows, groups, heads):
    """(B, N, heads * 128) -> (B, kv_heads, groups, heads / kv_heads * rows, 128) in 32 bits."""
    c = st["case"]
    lead = c["past"] % rows
    x = torch.nn.functional.pad(x.float(), (0, 0, lead, groups * rows - lead - c["N"]))
    x = x.view(c["B"], groups, rows, c["kv_heads"], heads // c["kv_heads"], 128)
    return x.permute(0, 3, 1, 4, 2, 5).flatten(3, 4)


def _ungrouped(x, st, rows, groups, heads):
    c = st["case"]
    lead = c["past"] % rows
    x = x.unflatten(3, (heads // c["kv_heads"], rows)).permute(0, 2, 4, 1, 3, 5)
    return x.reshape(c["B"], groups * rows, heads * 128)[:, lead:lead + c["N"]]


def _plain_window(st, train):
    c = st["case"]
    heads, scale = c["heads"], 1.0 / math.sqrt(128.0)
    keys, sees, rows, groups = _banded(st)
    q = _grouped(st["q"], st, rows, groups, heads)
    kf, vf = (x.float().view(c["B"], -1, c["kv_heads"], 128).permute(0, 2, 1, 3) for x in (st["k"], st["v"]))
    k, v = (x[:, :, keys.flatten()].unflatten(2, keys.shape) for x in (kf, vf))
    g = heads // c["kv_heads"]
    sees = sees[:, None].repeat(1, 1, 1, g, 1)
    s = (q @ k.transpose(-1, -2) * scale).masked_fill_(~sees, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp_(s.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)))
    total = p.sum(-1, keepdim=True)
    p = p.div_(torch.where(total == 0, torch.ones_like(total), total))
    o = p @ v
    lse = (top + torch.log(total)).expand(-1, -1, -1, -1, 128)
    lse = _ungrouped(lse, st, rows, groups, heads)[:, :, ::128].transpose(1, 2).contiguous()
    of = _ungrouped(o, st, rows, groups, heads)
    sig = None if st["gate"] is None else torch.sigmoid(st["gate"].float())
    y = (of if sig is None else of * sig).to(st["q"].dtype)
    if not train:
        return [y]
    dy = st["dy"].float()
    do = _grouped(dy if sig is None else dy * sig, st, rows, groups, heads)
    ds = p * (do @ v.transpose(-1, -2) - (do * o).sum(-1, keepdim=True)) * scale
    dq = _ungrouped(ds @ k, st, rows, groups, heads).to(y.dtype)
    back = []
    for d in (ds.transpose(-1, -2) @ q, p.transpose(-1, -2) @ do):
        d = torch.zeros_like(kf).index_add_(2, keys.flatten(), d.flatten(2, 3))
        back.append(d.permute(0, 2, 1, 3).flatten(2).to(y.dtype))
    outs = [y, lse, dq] + back
    if sig is not None:
        # rows past a sequence's end have no output and so no gradient
        outs.append((dy * of * sig * (1.0 - sig)).to(y.dtype))
    return outs


def _plain_decode(st):
    c = st["case"]
    B, N, hk, cap, ring = c["B"], c["N"], c["kv_heads"], c["capacity"], c["capacity"] - c["sinks"]
    g, sinks, held = c["heads"] // hk, c["sinks"], st["lengths"].long()
    dev = held.device
    new = held[:, None] + torch.arange(N, device=dev)
    slot = torch.where(new < cap, new, sinks + (new - sinks) % ring)
    at = torch.arange(B, device=dev)[:, None]
    st["k_cache"][at, slot] = st["k"]
    st["v_cache"][at, slot] = st["v"]
    # the position that each slot holds: the last one that was put there
    last = (held + N - 1)[:, None]
    s = torch.arange(cap, device=dev)[None]
    pos = torch.where(s < sinks, s, last - (last - s) % ring)
    there = (pos <= last) & ((s < sinks) | (pos >= sinks))
    p = new[:, :, None]
    sees = there[:, None] & (pos[:, None] <= p) & ((pos[:, None] > p - c["window"]) | (pos[:, None] < sinks))
    sees = sees[:, None, None]  # (B, 1, 1, N, cap)
    q = st["q"].float().view(B, N, hk, g, 128).permute(0, 2, 3, 1, 4)
    k, v = (x.float().view(B, cap, hk, 1, 128).permute(0, 2, 3, 1, 4) for x in (st["k_cache"], st["v_cache"]))
    w = (q.flatten(2, 3)[:, :, None] @ k.transpose(-1, -2)).view(B, hk, g, N, cap) / math.sqrt(128.0)
    w = w.masked_fill(~sees, -math.inf)
    w = torch.exp(w - w.amax(-1, keepdim=True))
    w = w / w.sum(-1, keepdim=True)
    o = (w.view(B, hk, 1, g * N, cap) @ v).view(B, hk, g, N, 128).permute(0, 3, 1, 2, 4).reshape(B, N, -1)
    if st["gate"] is not None:
        o = o * torch.sigmoid(st["gate"].float())
    return [o.to(st["q"].dtype), st["k_cache"], st["v_cache"]]


# ----------------------------------------------------------------------- the framework's operators

def _own(st):
    import softmax_attention_sana_b200 as sana
    c = st["case"]
    h, hk = c["heads"], c["kv_heads"]
    if c["op"] in ("rotary", "qk_norm_rope", "qk_norm_rope_train"):
        at = dict(grid=(c["T"], c["H"], c["W"])) if c.get("T") else dict(
            positions=st["positions"], offset=0 if c["scattered"] else c["offset"])
        if c["op"] == "rotary":
            return list(sana.rotary_apply(st["q"], st["k"], st["rotary"], h, hk, **at))
        outs = sana.qk_norm_rope(st["q"], st["k"], st["wq"], st["wk"], st["rotary"], h, hk, eps=EPS, **at)
        if c["op"] == "qk_norm_rope":
            return list(outs)
        grads = sana.qk_norm_rope_bwd(st["dq"], st["dk"], st["q"], st["k"], st["wq"], st["wk"],
                                      st["rotary"], h, hk, eps=EPS, **at)
        return list(outs) + list(grads)
    if c["op"] == "window_decode":
        y = sana.window_anchor_decode(st["q"], st["k"], st["v"], st["gate"], st["k_cache"],
                                      st["v_cache"], st["lengths"], h, hk, window=c["window"],
                                      sinks=c["sinks"])
        return [y, st["k_cache"], st["v_cache"]]
    sees = dict(window=c["window"], sinks=c["sinks"], block=c["block"], lengths=st["lengths"])
    if c["op"] == "window":
        return [sana.window_anchor_fwd(st["q"], st["k"], st["v"], st["gate"], h, hk, **sees)]
    y, lse = sana.window_anchor_fwd(st["q"], st["k"], st["v"], st["gate"], h, hk, want_lse=True, **sees)
    grads = sana.window_anchor_bwd(st["q"], st["k"], st["v"], st["gate"], y, lse, st["dy"], h, hk, **sees)
    return [y, lse] + [x for x in grads if x is not None]


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "rotary":
        return _plain_rotary(state)
    if op in ("qk_norm_rope", "qk_norm_rope_train"):
        return _plain_norm(state, op == "qk_norm_rope_train")
    if op in ("window", "window_train"):
        return _plain_window(state, op == "window_train")
    return _plain_decode(state)


# -------------------------------------------------------------------------------- the work in them

def _pairs(c):
    """Pairs of a query and a key that it sees, over the batch (one head)."""
    total, P = c["N"] + c["past"], c["block"]
    W = c["window"] if c["window"] else total + P
    n = 0
    for length in _lengths(c) or [total] * c["B"]:
        pos = np.arange(c["past"], max(c["past"], length), dtype=np.int64)
        end = (pos // P + 1) * P
        low = np.maximum(end - W, 0)
        top = np.minimum(end, length)
        n += int((np.maximum(top - low, 0) + np.minimum(np.minimum(c["sinks"], low), top)).sum())
    return n


def work(case):
    c = case
    if c["op"] in ("rotary", "qk_norm_rope", "qk_norm_rope_train"):
        n = c["B"] * c["N"] * (c["heads"] + c["kv_heads"]) * c["D"]
        size = 2 if c["dtype"] == "bf16" else 4
        table = 4 * c["rot"] * (c["T"] + c["H"] + c["W"] if c.get("T") else
                                c["N"] * (c["B"] if c["scattered"] else 1))
        if c["op"] == "qk_norm_rope_train":  # x and dy in, y and dx out
            return {"bytes": 4 * n * size + table, "flops": 24 * n}
        return {"bytes": 2 * n * size + table, "flops": (3 if c["op"] == "rotary" else 7) * n}
    row = 2 * 128
    if c["op"] == "window_decode":
        keys = 0
        for held in _held(c):
            last = held + c["N"]
            low = max(0, held + 1 - c["window"])
            keys += (held - low) + min(c["sinks"], low) + c["N"] if last else 0
        q = c["B"] * c["N"] * c["heads"] * row * (3 if c["gate"] else 2)
        new = 4 * c["B"] * c["N"] * c["kv_heads"] * row
        return {"bytes": 2 * keys * c["kv_heads"] * row + q + new,
                "flops": 4 * 128 * keys * c["heads"] * c["N"]}
    pairs = _pairs(c) * c["heads"]
    q = c["B"] * c["N"] * c["heads"] * row
    kv = c["B"] * (c["N"] + c["past"]) * c["kv_heads"] * row
    if c["op"] == "window":
        return {"bytes": q * (3 if c["gate"] else 2) + 2 * kv, "flops": 4 * 128 * pairs}
    # the forward's two products and the backward's five: the scores again, dP, dQ, dK and dV
    return {"bytes": q * (6 if c["gate"] else 4) + 4 * kv + 4 * c["B"] * c["N"] * c["heads"],
            "flops": 14 * 128 * pairs}


# -------------------------------------------------------------------- the definitions in 64 bits

def _exact_turned(x, ang, mul, layout):
    """The rotation as a product of complex numbers."""
    R = 2 * ang.shape[-1]
    unit = torch.polar(torch.full_like(ang, mul), ang)[:, :, None]
    r = x[..., :R]
    z = (torch.complex(r[..., :R // 2].contiguous(), r[..., R // 2:].contiguous()) if layout == "half"
         else torch.view_as_complex(r.reshape(*r.shape[:-1], R // 2, 2).contiguous()))
    z = torch.view_as_real(z * unit)
    z = z.transpose(-1, -2) if layout == "half" else z
    return torch.cat([z.reshape(*r.shape), x[..., R:]], dim=-1)


def _exact_sees(pos, total, c, length):
    """(rows, keys): what the rows at these positions see of a sequence of that length."""
    j = torch.arange(total, device=pos.device)[None]
    p = pos[:, None]
    own_block_end = torch.div(p, c["block"], rounding_mode="floor") * c["block"] + c["block"]
    near = (own_block_end - j <= c["window"]) if c["window"] else torch.ones_like(j, dtype=torch.bool)
    return (near | (j < c["sinks"])) & (j < own_block_end) & (j < length) & (p < length)


def _exact_attention(q, k, v, sees):
    """(h, n, D), (hk, m, D): softmax over what each row sees; rows that see nothing give 0."""
    hk, g = k.shape[0], q.shape[0] // k.shape[0]
    s = torch.einsum("kgnd,kmd->kgnm", q.view(hk, g, *q.shape[1:]), k) / math.sqrt(128.0)
    s = s.masked_fill(~sees, -math.inf)
    some = sees.any(-1)[:, None]
    lse = torch.logsumexp(s, -1, keepdim=True)
    p = torch.where(some, torch.exp(s - torch.where(some, lse, torch.zeros_like(lse))), torch.zeros_like(s))
    return torch.einsum("kgnm,kmd->kgnd", p, v).flatten(0, 1), lse.squeeze(-1).flatten(0, 1)


def exact(case, seed):
    c = case
    st = prepare(c, seed)
    if c["op"] in ("rotary", "qk_norm_rope", "qk_norm_rope_train"):
        ang, mul = _angles(c, st["positions"])
        outs, grads, weights = [], [], []
        for x, w, dy in ((st["q"], st.get("wq"), st.get("dq")), (st["k"], st.get("wk"), st.get("dk"))):
            x = x.double().unflatten(2, (-1, c["D"])).requires_grad_(dy is not None)
            y = x
            if w is not None:
                w = w.double().requires_grad_(dy is not None)
                y = x / torch.sqrt((x ** 2).mean(-1, keepdim=True) + EPS) * w
            y = _exact_turned(y, ang, mul, c["layout"])
            if dy is not None:
                y.backward(dy.double().view_as(y))
                grads.append(x.grad.flatten(2))
                weights.append(w.grad)
            outs.append(y.detach().flatten(2))
        return outs + grads + weights
    B, N, h, hk = c["B"], c["N"], c["heads"], c["kv_heads"]
    heads_first = lambda x, n: x.double().view(x.shape[0], x.shape[1], n, 128).transpose(1, 2)  # noqa: E731
    gate = None if st["gate"] is None else torch.sigmoid(heads_first(st["gate"], h))
    if c["op"] == "window_decode":
        held, ring = st["lengths"].tolist(), c["capacity"] - c["sinks"]
        ys = []
        for b in range(B):
            for name in ("k", "v"):
                for i in range(N):
                    p = held[b] + i
                    at = p if p < c["capacity"] else c["sinks"] + (p - c["sinks"]) % ring
                    st[name + "_cache"][b, at] = st[name][b, i]
            last = held[b] + N - 1
            kept = list(range(min(c["sinks"], last + 1)))
            kept += range(max(c["sinks"], last - ring + 1), last + 1)
            p = torch.tensor(kept, device="cuda")
            at = torch.where(p < c["capacity"], p, c["sinks"] + (p - c["sinks"]) % ring)
            pos = held[b] + torch.arange(N, device="cuda")[:, None]
            sees = (p <= pos) & ((pos - p < c["window"]) | (p < c["sinks"]))
            k, v = (heads_first(st[n][b:b + 1, at], hk)[0] for n in ("k_cache", "v_cache"))
            o, _ = _exact_attention(heads_first(st["q"][b:b + 1], h)[0], k, v, sees)
            ys.append((o if gate is None else o * gate[b]).transpose(0, 1).flatten(1))
        return [torch.stack(ys), st["k_cache"], st["v_cache"]]
    total, train = N + c["past"], c["op"] == "window_train"
    if float(B) * h * N * total * (14 if train else 4) * 128 > 1e14:
        return None
    held = _lengths(c) or [total] * B
    q, k, v = heads_first(st["q"], h), heads_first(st["k"], hk), heads_first(st["v"], hk)
    y, lse = torch.zeros_like(q), torch.full(q.shape[:3], -math.inf, device="cuda", dtype=torch.float64)
    grads = [torch.zeros_like(x) for x in (q, k, v)] + ([torch.zeros_like(q)] if gate is not None else [])
    step = max(1, min(N, int(4e9 / (8 * h * total))))
    for b in range(B):
        for a in range(0, N, step):
            rows = slice(a, min(N, a + step))
            pos = c["past"] + torch.arange(rows.start, rows.stop, device="cuda")
            sees = _exact_sees(pos, total, c, held[b])
            leaves = [q[b, :, rows], k[b], v[b]]
            if gate is not None:
                leaves.append(heads_first(st["gate"][b:b + 1, rows], h)[0])
            leaves = [x.detach().clone().requires_grad_(train) for x in leaves]
            o, l = _exact_attention(*leaves[:3], sees)
            o = o if gate is None else o * torch.sigmoid(leaves[3])
            y[b, :, rows], lse[b, :, rows] = o.detach(), l.detach()
            if train:
                o.backward(heads_first(st["dy"][b:b + 1, rows], h)[0])
                grads[0][b, :, rows] = leaves[0].grad
                grads[1][b] += leaves[1].grad
                grads[2][b] += leaves[2].grad
                if gate is not None:
                    grads[3][b, :, rows] = leaves[3].grad
    flat = lambda x: x.transpose(1, 2).flatten(2)  # noqa: E731
    return [flat(y)] + ([lse] + [flat(x) for x in grads] if train else [])
