"""The attention layer's operators beside ELSAA, as cases to measure.

Four operators, each in its plain form (elementary torch operations in 32
bits) and through the framework's entry points:

  rotate  RMS norm of every query and key row and the position rotation
  window  causal sliding-window attention with sinks, forward and backward
  write   the serving form of rotate: new tokens' queries out, keys and values
          into the pages of a cache
  attend  the serving form of window: new tokens over the paged cache
"""

import math

import torch

own = False

EPS = 1e-6
BASE = 10000.0


# ---- cases -------------------------------------------------------------------

def listed():
    return [
        # a short prompt of a small model in fp32, interleaved pairs, half of the head rotated: latency
        dict(name="rotate-short-fp32", kind="rotate", B=1, H=4, Hkv=2, N=37, d=32, dtype="f32", rot=16,
             interleaved=True, layout="bhnd", grad=True),
        # the text-32k training step's queries and keys, forward and backward
        dict(name="rotate-text-32k", kind="rotate", B=2, H=12, Hkv=12, N=32768, d=64, dtype="bf16", rot=64,
             interleaved=False, layout="bhnd", grad=True),
        # a prefill that reads the heads in place from a fused [B, N, H, d] projection, odd length
        dict(name="rotate-fused-4099", kind="rotate", B=1, H=32, Hkv=8, N=4099, d=128, dtype="bf16", rot=128,
             interleaved=False, layout="bnhd", grad=False),
        # a unit-test sized fp32 step: latency of forward and backward
        dict(name="window-short-fp32", kind="window", B=1, H=4, Hkv=2, N=200, d=32, dtype="f32", window=48,
             sinks=4, ragged=False, layout="bhnd", grad=True),
        # a training step at the text-32k shape
        dict(name="window-text-32k", kind="window", B=2, H=12, Hkv=12, N=32768, d=64, dtype="bf16", window=1024,
             sinks=4, ragged=False, layout="bhnd", grad=True),
        # a long prefill with grouped heads
        dict(name="window-gqa-16k", kind="window", B=1, H=32, Hkv=8, N=16384, d=128, dtype="bf16", window=4096,
             sinks=16, ragged=False, layout="bnhd", grad=False),
        # a padded training batch of odd lengths
        dict(name="window-ragged-4001", kind="window", B=4, H=16, Hkv=4, N=4001, d=128, dtype="bf16", window=1000,
             sinks=3, ragged=True, layout="bhnd", grad=True),
        # one decoding step of 64 sequences
        dict(name="write-step-64", kind="write", S=64, new=1, context=2000, H=32, Hkv=8, d=128, dtype="bf16",
             page=16, rot=128, interleaved=False),
        # prompt chunks of five sequences
        dict(name="write-chunk", kind="write", S=5, new=701, context=1500, H=12, Hkv=12, d=64, dtype="bf16",
             page=64, rot=64, interleaved=False),
        # one sequence decoding one token: latency
        dict(name="attend-one", kind="attend", S=1, new=1, context=5001, H=12, Hkv=4, d=64, dtype="bf16",
             page=16, window=0, sinks=0),
        # a decoding step of 64 sequences of very different lengths
        dict(name="attend-step-64", kind="attend", S=64, new=1, context=16384, H=32, Hkv=8, d=128, dtype="bf16",
             page=64, window=0, sinks=0),
        # prompt chunks over long contexts, with a window and sinks
        dict(name="attend-chunk", kind="attend", S=4, new=509, context=16000, H=32, Hkv=8, d=128, dtype="bf16",
             page=16, window=4096, sinks=4),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["rotate", "window", "window", "write", "attend", "attend"])
    Hkv = rng.choice([1, 2, 4, 8, 12])
    H = Hkv * rng.choice([1, 1, 2, 3, 4, 8] if Hkv <= 4 else [1, 2, 4] if Hkv <= 8 else [1])
    f32 = rng.random() < 0.2
    c = dict(kind=kind, H=H, Hkv=Hkv, d=rng.choice([32, 64, 64, 128, 128]), dtype="f32" if f32 else "bf16")
    if kind in ("rotate", "window"):
        c["layout"] = rng.choice(["bhnd", "bnhd"])
        c["grad"] = rng.random() < 0.6
        c["B"] = rng.choice([1, 2, 3, 4])
        most = 1500 if (f32 or c["d"] == 32) and kind == "window" else (1 << 19) // (c["B"] * H)
        c["N"] = _log(rng, 1, min(most, 40000))
    else:
        c["S"] = _log(rng, 1, 100)
        c["new"] = 1 if rng.random() < 0.5 else _log(rng, 1, max(1, 2048 // c["S"]))
        slow = f32 or c["d"] == 32
        c["context"] = c["new"] + _log(rng, 1, min(20000, (20000 if slow else 1 << 19) // c["S"]))
        c["page"] = rng.choice([16, 32, 48, 64, 128, 256])
    if kind in ("rotate", "write"):
        c["interleaved"] = rng.random() < 0.4
        c["rot"] = rng.choice([c["d"], c["d"], c["d"] // 2])
    else:
        c["window"] = _log(rng, 1, 5000)
        c["sinks"] = rng.choice([0, 1, 4, 16, 130])
    if kind == "window":
        c["ragged"] = rng.random() < 0.4
        while work(c)["flops"] > 7e11:
            c["window"] //= 2
    if kind == "attend" and rng.random() < 0.5:
        c["window"] = 0
    return c


def _spread(n, lo, hi):
    """n whole numbers spread over [lo, hi], the last of them hi, in no order."""
    if n == 1:
        return [hi]
    return [lo + int((hi - lo) * ((k * 0.6180339887) % 1.0)) for k in range(1, n)] + [hi]


def _lengths(c):
    """The padded batch's lengths, one of them zero where there are three or more."""
    if not c["ragged"]:
        return [c["N"]] * c["B"]
    ls = _spread(c["B"], 1 + c["N"] // 3, c["N"])
    return ls[:1] + [0] + ls[2:] if c["B"] == 3 else ls


def _serving(c):
    """(new tokens, context with them) of every sequence."""
    new = [max(1, n) for n in _spread(c["S"], 1 + c["new"] // 2, c["new"])]
    ctx = _spread(c["S"], 1 + c["context"] // 8, c["context"])
    return new, [max(n, x) for n, x in zip(new, ctx)]


def _window_pairs(n, w, s, first=0):
    """Visible (query, key) pairs of queries first .. n - 1."""
    total = 0
    for lo, hi, per in ((0, min(w, n), None), (w, n, w)):
        lo = max(lo, first)
        if hi <= lo:
            continue
        if per is None:
            total += (lo + 1 + hi) * (hi - lo) // 2
        else:
            total += per * (hi - lo)
            # sinks outside the window: min(s, i - w + 1) of query i
            a, b = lo - w + 1, hi - w
            m = min(max(s, a - 1), b)
            total += (a + m) * (m - a + 1) // 2 + s * (b - m)
    return total


def work(case):
    c = case
    e = 4 if c["dtype"] == "f32" else 2
    heads = c["H"] + c["Hkv"]
    if c["kind"] == "rotate":
        rows = c["B"] * c["N"] * heads
        table = c["N"] * c["rot"] * 4
        return {"bytes": rows * c["d"] * e * (5 if c["grad"] else 2) + table,
                "flops": rows * c["d"] * (24 if c["grad"] else 8)}
    if c["kind"] == "window":
        ls = _lengths(c)
        pairs = sum(_window_pairs(n, c["window"], c["sinks"]) for n in ls) * c["H"]
        tok = sum(ls)
        q, k = tok * c["H"] * c["d"] * e, tok * c["Hkv"] * c["d"] * e
        lse = c["B"] * c["N"] * c["H"] * 4
        # y whole (rows behind a length are zeros); backward: dy in, dq, dk, dv whole
        whole_q, whole_k = (c["B"] * c["N"] * h * c["d"] * e for h in (c["H"], c["Hkv"]))
        return {"bytes": q + 2 * k + whole_q + lse + (q + whole_q + 2 * whole_k if c["grad"] else 0),
                "flops": pairs * c["d"] * (14 if c["grad"] else 4)}
    new, ctx = _serving(c)
    if c["kind"] == "write":
        return {"bytes": sum(new) * (c["H"] + 2 * c["Hkv"]) * c["d"] * e * 2 + sum(new) * c["rot"] * 4,
                "flops": sum(new) * heads * c["d"] * 8}
    w = c["window"] or 1 << 30
    pairs = sum(_window_pairs(x, w, c["sinks"], x - n) for n, x in zip(new, ctx)) * c["H"]
    seen = sum(min(x, n + w - 1 + c["sinks"]) for n, x in zip(new, ctx))
    return {"bytes": seen * c["Hkv"] * c["d"] * e * 2 + 2 * sum(new) * c["H"] * c["d"] * e,
            "flops": 4 * pairs * c["d"]}


# ---- inputs ------------------------------------------------------------------

def _dtype(c):
    return torch.float32 if c["dtype"] == "f32" else torch.bfloat16


def _normal(gen, shape, dt, scale=1.0, offset=0.0):
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    return (x * scale + offset).to(dt)


def _heads(c, gen, h, dt):
    """[B, h, N, d]: contiguous, or a view of a [B, N, h, d] projection."""
    if c["layout"] == "bnhd":
        return _normal(gen, (c["B"], c["N"], h, c["d"]), dt).transpose(1, 2)
    return _normal(gen, (c["B"], h, c["N"], c["d"]), dt)


def _table(rows, rot):
    """(cos, sin) of position x frequency pairs, from angles in 64 bits: [rows, rot / 2, 2] fp32."""
    freq = BASE ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(rows, dtype=torch.float64, device="cuda")[:, None] * freq
    return torch.stack([a.cos(), a.sin()], -1).float()


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = _dtype(c)
    s = {"c": c}
    if c["kind"] in ("rotate", "window"):
        s["q"], s["k"] = _heads(c, gen, c["H"], dt), _heads(c, gen, c["Hkv"], dt)
        if c["kind"] == "window":
            s["v"] = _heads(c, gen, c["Hkv"], dt)
            s["lengths"] = (torch.tensor(_lengths(c), dtype=torch.int32, device="cuda")
                            if c["ragged"] else None)
            if c["grad"]:
                s["dy"] = _heads(c, gen, c["H"], dt)
        elif c["grad"]:
            s["dqo"], s["dko"] = _heads(c, gen, c["H"], dt), _heads(c, gen, c["Hkv"], dt)
    else:
        new, ctx = _serving(c)
        T, page = sum(new), c["page"]
        need = [-(-x // page) for x in ctx]
        width, pages = max(need), sum(need) + 3
        order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
        at = torch.arange(width, device="cuda")
        off = torch.tensor([sum(need[:i]) for i in range(c["S"])], device="cuda")
        inside = at[None] < torch.tensor(need, device="cuda")[:, None]
        # entries behind a sequence's last page are not pages
        s["page_table"] = torch.where(inside, order[torch.where(inside, off[:, None] + at, 0)], -1)
        s["page_table"] = s["page_table"].to(torch.int32).contiguous()
        s["starts"] = torch.tensor([sum(new[:i]) for i in range(c["S"] + 1)], dtype=torch.int32, device="cuda")
        s["lengths"] = torch.tensor(ctx, dtype=torch.int32, device="cuda")
        s["k_pages"] = _normal(gen, (pages, c["Hkv"], page, c["d"]), dt)
        s["v_pages"] = _normal(gen, (pages, c["Hkv"], page, c["d"]), dt)
        s["q"] = _normal(gen, (T, c["H"], c["d"]), dt)
        if c["kind"] == "write":
            s["k"], s["v"] = (_normal(gen, (T, c["Hkv"], c["d"]), dt) for _ in range(2))
    if c["kind"] in ("rotate", "write"):
        rows = c["N"] if c["kind"] == "rotate" else c["context"]
        s["table"] = _table(rows, c["rot"])
        s["q_weight"] = _normal(gen, (c["d"],), torch.float32, 0.1, 1.0)
        s["k_weight"] = _normal(gen, (c["d"],), torch.float32, 0.1, 1.0)
    if own:
        _prepare_own(s)
    return s


def _prepare_own(s):
    """The problem descriptions and workspaces that a program keeps between calls."""
    from sparse_rank_hybrid_simhash_b200 import paged, rotary, window
    c = s["c"]
    if c["kind"] in ("rotate", "write"):
        B, N = (c["B"], c["N"]) if c["kind"] == "rotate" else (1, s["q"].shape[0])
        s["rp"] = rotary.RotaryParams.make(B, c["H"], c["Hkv"], N, c["d"], c["dtype"], rot_dim=c["rot"],
                                           max_pos=s["table"].shape[0], interleaved=c["interleaved"], eps=EPS)
        s["ws"] = rotary.alloc_workspace(s["rp"], s["q"].device)
    if c["kind"] == "window":
        s["p"] = window.WindowParams.make(c["B"], c["H"], c["Hkv"], c["N"], c["d"], c["dtype"],
                                          window=c["window"], sinks=c["sinks"])
        s["ws"] = window.alloc_workspace(s["p"], s["q"].device)
    elif c["kind"] in ("write", "attend"):
        pages, _, page, _ = s["k_pages"].shape
        s["p"] = paged.PagedParams.make(c["S"], s["q"].shape[0], c["H"], c["Hkv"], c["d"], c["dtype"], page, pages,
                                        s["page_table"].shape[1], window=c.get("window", 0), sinks=c.get("sinks", 0))
        s["ws"] = paged.alloc_workspace(s["p"], s["q"].device)


# ---- one pass ----------------------------------------------------------------

def run(state):
    s = state
    return {"rotate": _run_rotate, "window": _run_window, "write": _run_write, "attend": _run_attend}[s["c"]["kind"]](s)


def _run_rotate(s):
    c = s["c"]
    if own:
        from sparse_rank_hybrid_simhash_b200 import rotary
        qo, ko = rotary.forward(s["rp"], s["q"], s["k"], s["table"], s["q_weight"], s["k_weight"], ws=s["ws"])
        if not c["grad"]:
            return qo, ko
        return (qo, ko) + tuple(rotary.backward(s["rp"], s["q"], s["k"], s["table"], s["q_weight"], s["k_weight"],
                                                s["dqo"], s["dko"], ws=s["ws"]))
    cs = s["table"][None, None, :c["N"]]
    qo, ko = (_plain_norm_rotate(s[x], s[x + "_weight"], cs, c["interleaved"]) for x in "qk")
    if not c["grad"]:
        return qo, ko
    (dq, dwq), (dk, dwk) = (_plain_norm_rotate_back(s[x], s[x + "_weight"], cs, c["interleaved"], s["d%so" % x])
                            for x in "qk")
    return qo, ko, dq, dk, dwq, dwk


def _pairs(x, rot, interleaved):
    if interleaved:
        return x[..., 0:rot:2], x[..., 1:rot:2]
    return x[..., :rot // 2], x[..., rot // 2:rot]


def _turn(x, cs, interleaved, back=False):
    """The rotation by the table's angles of the first 2 x cs.shape[-2] values of every row (or its transpose)."""
    rot = 2 * cs.shape[-2]
    a, b = _pairs(x, rot, interleaved)
    cos, sin = cs[..., 0], -cs[..., 1] if back else cs[..., 1]
    u, v = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([u, v], -1).flatten(-2) if interleaved else torch.cat([u, v], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _plain_norm_rotate(x, w, cs, interleaved):
    f = x.float()
    n = f * torch.rsqrt(f.square().mean(-1, keepdim=True) + EPS)
    return _turn(n * w, cs, interleaved).to(x.dtype)


def _plain_norm_rotate_back(x, w, cs, interleaved, dy):
    f = x.float()
    r = torch.rsqrt(f.square().mean(-1, keepdim=True) + EPS)
    n = f * r
    du = _turn(dy.float(), cs, interleaved, back=True)
    dw = (du * n).double().sum((0, 1, 2)).float()
    dn = du * w
    return (r * (dn - n * (dn * n).mean(-1, keepdim=True))).to(x.dtype), dw


def _run_window(s):
    c = s["c"]
    if own:
        from sparse_rank_hybrid_simhash_b200 import window
        y, lse = window.forward(s["p"], s["q"], s["k"], s["v"], lengths=s["lengths"], ws=s["ws"])
        if not c["grad"]:
            return y, lse
        return (y, lse) + tuple(window.backward(s["p"], s["q"], s["k"], s["v"], y, lse, s["dy"],
                                                lengths=s["lengths"], ws=s["ws"]))
    return _plain_window(c, s["q"], s["k"], s["v"], s["lengths"], s.get("dy"))


def _plain_window(c, q, k, v, lengths, dy):
    """Blocks of m queries against the band of w - 1 + m keys that they see, and the sinks beside it."""
    B, H, Hkv, N, d, w = (c[x] for x in ("B", "H", "Hkv", "N", "d", "window"))
    g, dt, dev = H // Hkv, q.dtype, q.device
    w, sinks = min(w, N), min(c["sinks"], N)
    m = max(16, min(512, w))
    nb = -(-N // m)
    span = m + w - 1
    scale = 1.0 / math.sqrt(d)

    def blocks(x):      # [B, H, N, d] -> [B, Hkv, nb, g m, d]
        x = torch.nn.functional.pad(x.float(), (0, 0, 0, nb * m - N))
        return x.view(B, Hkv, g, nb, m, d).permute(0, 1, 3, 2, 4, 5).reshape(B, Hkv, nb, g * m, d)

    def band(x):        # [B, Hkv, N, d] -> [B, Hkv, nb, span, d]
        x = torch.nn.functional.pad(x.float(), (0, 0, w - 1, nb * m - N))
        return x.unfold(2, span, m).transpose(-1, -2)

    def whole(x):       # blocks() undone
        x = x.view(B, Hkv, nb, g, m, -1).permute(0, 1, 3, 2, 4, 5).reshape(B, H, nb * m, -1)
        return x[:, :, :N]

    at = torch.arange(nb * m, device=dev).view(1, 1, nb, 1, m, 1)
    to = (torch.arange(nb, device=dev).view(nb, 1) * m + torch.arange(span, device=dev) - (w - 1))
    live = at < (N if lengths is None else lengths.view(B, 1, 1, 1, 1, 1))
    key = to.view(1, 1, nb, 1, 1, span)
    see = live & (key >= 0) & (key <= at) & (key > at - w)
    far = live & (torch.arange(sinks, device=dev).view(1, 1, 1, 1, 1, sinks) <= at - w)
    see, far = (x.expand(B, 1, nb, g, m, x.shape[-1]).reshape(B, 1, nb, g * m, x.shape[-1]) for x in (see, far))
    qb, kb, vb = blocks(q), band(k), band(v)
    ks, vs = (x[:, :, None, :sinks].float() for x in (k, v))
    sb = (qb @ kb.transpose(-1, -2) * scale).masked_fill_(~see, -math.inf)
    ss = (qb @ ks.transpose(-1, -2) * scale).masked_fill_(~far, -math.inf)
    top = sb.amax(-1, keepdim=True)
    top = torch.maximum(top, ss.amax(-1, keepdim=True)) if sinks else top
    top = top.masked_fill(top == -math.inf, 0.0)
    pb, ps = sb.sub_(top).exp_(), ss.sub_(top).exp_()
    z = pb.sum(-1, keepdim=True) + ps.sum(-1, keepdim=True)
    lse = top + z.log()
    inv = torch.where(z > 0, 1.0 / z, 0.0)
    pb, ps = pb.mul_(inv), ps.mul_(inv)
    yb = pb @ vb + ps @ vs
    out = whole(yb).to(dt), whole(lse)[..., 0]
    if dy is None:
        return out
    gb = blocks(dy) * (see.any(-1, keepdim=True) | far.any(-1, keepdim=True))
    delta = (gb * yb).sum(-1, keepdim=True)

    def back(x):        # [B, Hkv, nb, span, d] -> [B, Hkv, N, d], overlapping bands added up
        full = torch.zeros(B, Hkv, w - 1 + nb * m, d, device=dev)
        return full.index_add_(2, (to + (w - 1)).reshape(-1), x.reshape(B, Hkv, nb * span, d))[:, :, w - 1:w - 1 + N]

    dv = back(pb.transpose(-1, -2) @ gb)
    dv[:, :, :sinks] += (ps.transpose(-1, -2) @ gb).sum(2)
    db = pb.mul_((gb @ vb.transpose(-1, -2)).sub_(delta)).mul_(scale)
    ds = ps * (gb @ vs.transpose(-1, -2) - delta) * scale
    dq = whole(db @ kb + ds @ ks)
    dk = back(db.transpose(-1, -2) @ qb)
    dk[:, :, :sinks] += (ds.transpose(-1, -2) @ qb).sum(2)
    return out + (dq.to(dt), dk.to(dt), dv.to(dt))


def _tokens(s):
    """The sequence and the position of every new token."""
    starts, T = s["starts"].long(), s["q"].shape[0]
    row = torch.arange(T, device=starts.device)
    seq = (row[:, None] >= starts[None, 1:]).sum(1)
    return row, seq, s["lengths"].long()[seq] - starts[1:][seq] + row


def _run_write(s):
    c = s["c"]
    if own:
        from sparse_rank_hybrid_simhash_b200 import paged
        qo = paged.write(s["p"], s["rp"], s["q"], s["k"], s["v"], s["table"], s["q_weight"], s["k_weight"],
                         s["k_pages"], s["v_pages"], s["page_table"], s["starts"], s["lengths"], ws=s["ws"])
        return qo, s["k_pages"], s["v_pages"]
    _, seq, pos = _tokens(s)
    cs = s["table"][pos][:, None]
    qo, ko = (_plain_norm_rotate(s[x], s[x + "_weight"], cs, c["interleaved"]) for x in "qk")
    page = s["page_table"].long()[seq, pos // c["page"]]
    s["k_pages"][page, :, pos % c["page"]] = ko
    s["v_pages"][page, :, pos % c["page"]] = s["v"]
    return qo, s["k_pages"], s["v_pages"]


def _run_attend(s):
    c = s["c"]
    if own:
        from sparse_rank_hybrid_simhash_b200 import paged
        return paged.attend(s["p"], s["q"], s["k_pages"], s["v_pages"], s["page_table"], s["starts"], s["lengths"],
                            ws=s["ws"])
    row, seq, pos = _tokens(s)
    S, H, Hkv, d, m = c["S"], c["H"], c["Hkv"], c["d"], c["new"]
    g = H // Hkv
    table = s["page_table"].long().clamp(min=0)
    # [S, Hkv, keys, d] and [S, Hkv, m g, d], padded to the longest
    k, v = (s[x][table].float().transpose(1, 2).reshape(S, Hkv, -1, d) for x in ("k_pages", "v_pages"))
    at = row - s["starts"].long()[seq]
    q = torch.zeros(S, m, H, d, device=s["q"].device)
    q[seq, at] = s["q"].float()
    q = q.view(S, m, Hkv, g, d).transpose(1, 2).reshape(S, Hkv, m * g, d)
    where = torch.full((S, m), -1, device=q.device)
    where[seq, at] = pos
    where = where.repeat_interleave(g, 1).view(S, 1, m * g, 1)
    key = torch.arange(k.shape[2], device=q.device)
    see = key <= where
    if c["window"]:
        see &= (key > where - c["window"]) | (key < c["sinks"])
    x = (q @ k.transpose(-1, -2) / math.sqrt(d)).masked_fill_(~see, -math.inf)
    top = x.amax(-1, keepdim=True)
    x = x.sub_(top.masked_fill(top == -math.inf, 0.0)).exp_()
    z = x.sum(-1, keepdim=True)
    y = (x @ v) / torch.where(z > 0, z, 1.0)
    y = y.view(S, Hkv, m, g, d).transpose(1, 2).reshape(S, m, H, d)
    return y[seq, at].to(s["q"].dtype)


# ---- the same in 64 bits, from the definitions -------------------------------

def exact(case, seed):
    c = case
    s = prepare({**c, "name": ""}, seed)
    with torch.no_grad():
        return {"rotate": _exact_rotate, "window": _exact_window, "write": _exact_write,
                "attend": _exact_attend}[c["kind"]](c, s)


def _exact_angles(pos, rot):
    i = torch.arange(rot // 2, dtype=torch.float64, device=pos.device)
    return pos.double()[..., None] * torch.exp(-2.0 * i / rot * math.log(BASE))


def _exact_rows(x, w, pos, c):
    """(y, dx and dw as functions of dy) of rows x [..., d] at positions pos [...]; pairs as complex numbers."""
    d, rot = c["d"], c["rot"]
    x, w = x.double(), w.double()
    ms = (x * x).sum(-1, keepdim=True) / d + EPS
    n = x / ms.sqrt()
    z = torch.polar(torch.ones((), dtype=torch.float64, device=x.device), _exact_angles(pos, rot))
    order = torch.arange(rot, device=x.device)
    order = order.view(-1, 2) if c["interleaved"] else order.view(2, -1).t()

    def rotate(u, z):
        out = u.clone()
        t = torch.view_as_complex(u[..., order].contiguous()) * z
        out[..., order] = torch.view_as_real(t)
        return out

    def grads(dy):
        du = rotate(dy.double(), z.conj())
        dn = du * w
        dx = dn / ms.sqrt() - x * (dn * x).sum(-1, keepdim=True) / (d * ms * ms.sqrt())
        return dx, (du * n).reshape(-1, d).sum(0)

    return rotate(n * w, z), grads


def _exact_rotate(c, s):
    pos = torch.arange(c["N"], device="cuda").expand(c["B"], 1, c["N"])
    (qo, qb), (ko, kb) = (_exact_rows(s[x], s[x + "_weight"], pos, c) for x in "qk")
    if not c["grad"]:
        return qo, ko
    (dq, dwq), (dk, dwk) = qb(s["dqo"]), kb(s["dko"])
    return qo, ko, dq, dk, dwq, dwk


def _exact_window(c, s):
    B, H, Hkv, N, d = (c[x] for x in ("B", "H", "Hkv", "N", "d"))
    g, w, step = H // Hkv, c["window"], 512
    y = torch.zeros(B, H, N, d, dtype=torch.float64, device="cuda")
    lse = torch.full((B, H, N), -math.inf, dtype=torch.float64, device="cuda")
    dq, dk, dv = torch.zeros_like(y), *(torch.zeros(B, Hkv, N, d, dtype=torch.float64, device="cuda") for _ in "kv")
    for b, n in enumerate(_lengths(c)):
        k, v = s["k"][b].double(), s["v"][b].double()
        q = s["q"][b].double().reshape(Hkv, g, N, d)
        for i0 in range(0, n, step):
            i1 = min(n, i0 + step)
            j0 = max(0, i0 - w + 1)
            ns = min(c["sinks"], j0)
            j = torch.cat([torch.arange(ns, device="cuda"), torch.arange(j0, i1, device="cuda")])
            i = torch.arange(i0, i1, device="cuda")[:, None]
            see = (j <= i) & ((i - j < w) | (j < c["sinks"]))
            kj, vj = k[:, None, j], v[:, None, j]
            a = torch.where(see, q[:, :, i0:i1] @ kj.transpose(-1, -2) / math.sqrt(d), -math.inf)
            l = torch.logsumexp(a, -1, keepdim=True)
            p = torch.exp(a - l)
            o = p @ vj
            y[b, :, i0:i1] = o.reshape(H, i1 - i0, d)
            lse[b, :, i0:i1] = l.reshape(H, i1 - i0)
            if c["grad"]:
                do = s["dy"][b].double().reshape(Hkv, g, N, d)[:, :, i0:i1]
                da = p * (do @ vj.transpose(-1, -2) - (do * o).sum(-1, keepdim=True)) / math.sqrt(d)
                dq[b, :, i0:i1] = (da @ kj).reshape(H, i1 - i0, d)
                dk[b, :, j] += (da.transpose(-1, -2) @ q[:, :, i0:i1]).sum(1)
                dv[b, :, j] += (p.transpose(-1, -2) @ do).sum(1)
    return (y, lse, dq, dk, dv) if c["grad"] else (y, lse)


def _exact_write(c, s):
    new, ctx = _serving(c)
    kp, vp = s["k_pages"].double(), s["v_pages"].double()
    pos = torch.cat([torch.arange(x - n, x, device="cuda") for n, x in zip(new, ctx)])
    (qo, _), (ko, _) = (_exact_rows(s[x], s[x + "_weight"], pos[:, None], c) for x in "qk")
    t0 = 0
    for b, n in enumerate(new):
        at = pos[t0:t0 + n]
        pages = s["page_table"][b, at // c["page"]].long()
        kp[pages, :, at % c["page"]] = ko[t0:t0 + n]
        vp[pages, :, at % c["page"]] = s["v"][t0:t0 + n].double()
        t0 += n
    return qo, kp, vp


def _exact_attend(c, s):
    new, ctx = _serving(c)
    H, Hkv, d = c["H"], c["Hkv"], c["d"]
    out, t0 = [], 0
    for b, (n, x) in enumerate(zip(new, ctx)):
        pages = s["page_table"][b, : -(-x // c["page"])].long()
        k, v = (s[y][pages].double().permute(1, 0, 2, 3).reshape(Hkv, 1, -1, d)[:, :, :x] for y in ("k_pages", "v_pages"))
        q = s["q"][t0:t0 + n].double().view(n, Hkv, H // Hkv, d).permute(1, 2, 0, 3)
        i = torch.arange(x - n, x, device="cuda")[:, None]
        j = torch.arange(x, device="cuda")
        see = (j <= i) & ((i - j < (c["window"] or x)) | (j < c["sinks"]))
        p = torch.softmax(torch.where(see, q @ k.transpose(-1, -2) / math.sqrt(d), -math.inf), -1)
        out.append((p @ v).permute(2, 0, 1, 3).reshape(n, H, d))
        t0 += n
    return torch.cat(out)
