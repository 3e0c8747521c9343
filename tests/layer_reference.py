"""The operators next to ELSAA from their formulas in 64 bits, each with a bound on
what a kernel's roundings can move its results by.

Rounding counts: a value kept in type t is off by at most u(t) = eps(t) / 2 of
itself; a sum of n terms in fp32 by at most n 2^-24 of the terms' absolute sum.
bf16 kernels round the probabilities and the score gradients to bf16 before a
product (u each); everything else is held in fp32.
"""

import math

import torch

F32 = 2.0 ** -24


def unit(dt):
    return torch.finfo(dt).eps / 2


def visible(n_q, n_k, first, window, sinks, device):
    """[n_q, n_k]: query first + r sees key j."""
    i = torch.arange(first, first + n_q, device=device)[:, None]
    j = torch.arange(n_k, device=device)[None]
    near = (i - j < window) if window > 0 else torch.ones_like(j <= i)
    return (j <= i) & (near | (j < sinks))


def attention(q, k, v, see, scale, dt, dy=None, few=0):
    """q [..., n, d], k, v [..., m, d] in fp64, see [..., n, m].  Values y, lse (and dq, dk, dv
    of sum(y dy)) and their bounds, as two dicts.  few: rows with up to so many keys sum
    delta = y dy over their keys (the others' has y's rounding)."""
    d, m, n = q.shape[-1], k.shape[-2], q.shape[-2]
    u = unit(dt)
    up = u if dt == torch.bfloat16 else 0.0
    s = q @ k.transpose(-1, -2) * scale
    mag = q.abs() @ k.abs().transpose(-1, -2) * scale
    s = s.masked_fill(~see, -math.inf)
    lse = torch.logsumexp(s, -1, keepdim=True)
    live = see.any(-1, keepdim=True)
    safe = torch.where(live, lse, 0.0)
    p = torch.exp(s - safe)          # masked: exp(-inf) = 0
    y = p @ v
    # a score: d products and the scaling; the exponential: its argument's
    # rounding and two units of its own
    es = torch.where(see, F32 * ((d + 4) * mag + 4 * (torch.where(see, s, 0.0).abs() + safe.abs()) + 8), 0.0)
    e_row = es.amax(-1, keepdim=True) + (m + 4) * F32
    e = es + e_row + up
    ty = (p * e) @ v.abs() + (m + 4) * F32 * (p @ v.abs()) + u * y.abs()
    val = {"y": y, "lse": lse[..., 0]}
    tol = {"y": 1.01 * ty, "lse": (e_row + 4 * F32 * safe.abs())[..., 0]}
    if dy is None:
        return val, tol
    dy = torch.where(live, dy, 0.0)
    delta = (dy * y).sum(-1, keepdim=True)
    dp = dy @ v.transpose(-1, -2)
    ds = p * (dp - delta)
    tdelta = (dy.abs() * ty).sum(-1, keepdim=True) + (d + 2) * F32 * (dy * y).abs().sum(-1, keepdim=True)
    tfew = (p * ((es + e_row + (m + 4) * F32) * dp.abs() + (d + 4) * F32 * (dy.abs() @ v.abs().transpose(-1, -2)))
            ).sum(-1, keepdim=True)
    tdelta = torch.where(see.sum(-1, keepdim=True) <= few, tfew, tdelta)
    tds = p * (e * (dp - delta).abs() + tdelta + (d + 4) * F32 * (dy.abs() @ v.abs().transpose(-1, -2))) \
        + up * ds.abs()
    val["dq"] = scale * (ds @ k)
    tol["dq"] = 1.01 * (scale * ((tds + (m + 4) * F32 * ds.abs()) @ k.abs()) + u * val["dq"].abs())
    val["dk"] = scale * (ds.transpose(-1, -2) @ q)
    tol["dk"] = 1.01 * (scale * ((tds + (n + 4) * F32 * ds.abs()).transpose(-1, -2) @ q.abs()))
    val["dv"] = p.transpose(-1, -2) @ dy
    tol["dv"] = 1.01 * ((p * (e + (n + 4) * F32)).transpose(-1, -2) @ dy.abs())
    return val, tol


def window(q, k, v, win, sinks, lengths=None, scale=0.0, dy=None, few=0):
    """[B, H, N, d] and [B, Hkv, N, d] of the kernels' dtype: (values, bounds) of y, lse, dq, dk, dv."""
    B, H, N, d = q.shape
    Hkv, g, dt = k.shape[1], H // k.shape[1], q.dtype
    scale = scale if scale > 0 else 1.0 / math.sqrt(d)
    see = visible(N, N, 0, win, sinks, q.device).expand(B, 1, 1, N, N)
    n = torch.full((B,), N, device=q.device) if lengths is None else lengths.long()
    row = torch.arange(N, device=q.device)
    ok = (row[None] < n[:, None]).view(B, 1, 1, N, 1)
    see = see & ok

    def grouped(x):
        return torch.where(ok, x.double().view(B, Hkv, g, N, d), 0.0)

    def keys(x):
        return torch.where(ok, x.double().view(B, Hkv, 1, N, d), 0.0)

    val, tol = attention(grouped(q), keys(k), keys(v), see, scale, dt, None if dy is None else grouped(dy),
                         few)
    u = unit(dt)
    for x in val:
        if x in ("dk", "dv"):   # one sum over the group's heads, one rounding
            val[x], tol[x] = val[x].sum(2), tol[x].sum(2)
            tol[x] = tol[x] + 1.01 * u * val[x].abs()
        else:
            val[x], tol[x] = (t.reshape(B, H, *t.shape[3:]) for t in (val[x], tol[x]))
    return val, tol


def paged(q, k_pages, v_pages, page_table, starts, lengths, win, sinks, scale=0.0):
    """(y, bound) of the new tokens; rows of no sequence are zeros with bound 0."""
    T, H, d = q.shape
    Hkv, page = k_pages.shape[1], k_pages.shape[2]
    g, scale = H // Hkv, scale if scale > 0 else 1.0 / math.sqrt(d)
    y, t = (torch.zeros(T, H, d, dtype=torch.float64, device=q.device) for _ in range(2))
    starts, lengths = starts.tolist(), lengths.tolist()
    for b, x in enumerate(lengths):
        r0, n = starts[b], starts[b + 1] - starts[b]
        if n == 0:
            continue
        see = visible(n, x, x - n, win, sinks, q.device)
        used = see.any(0)
        k, v = gather(k_pages, page_table[b], x, used), gather(v_pages, page_table[b], x, used)
        qq = q[r0:r0 + n].double().view(n, Hkv, g, d).permute(1, 2, 0, 3)
        val, tol = attention(qq, k[:, None], v[:, None], see, scale, q.dtype)
        y[r0:r0 + n] = val["y"].permute(2, 0, 1, 3).reshape(n, H, d)
        t[r0:r0 + n] = tol["y"].permute(2, 0, 1, 3).reshape(n, H, d)
    return y, t


def gather(pages, table, length, used):
    """[Hkv, length, d] in fp64; tokens that no query sees are zeros and their pages not looked up."""
    Hkv, page, d = pages.shape[1:]
    out = torch.zeros(Hkv, length, d, dtype=torch.float64, device=pages.device)
    j = torch.nonzero(used)[:, 0]
    at = table.long()[j // page]
    out[:, j] = pages[at, :, j % page].double().transpose(0, 1)
    return out


def rotary(x, weight, pos, table, interleaved, norm, eps, dy=None):
    """x [..., d] at positions pos [...]: y (and dx, dweight of sum(y dy)) with bounds."""
    dt, d = x.dtype, x.shape[-1]
    u = unit(dt)
    x = x.double()
    w = torch.ones(d, dtype=torch.float64, device=x.device) if weight is None else weight.double()
    r = 1.0 / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) if norm else torch.ones_like(x[..., :1])
    n = x * r
    rot = 0 if table is None else 2 * table.shape[1]
    i = torch.arange(rot, device=x.device)
    a, b = (i[0::2], i[1::2]) if interleaved else (i[:rot // 2], i[rot // 2:])
    if rot:
        cs = table.double()[pos.long()]
        c, s = cs[..., 0], cs[..., 1]

    def turn(z, back=False, absolute=False):
        out = z.clone()
        if rot:
            sn = -s if back else s
            if absolute:
                out[..., a] = z[..., a] * c.abs() + z[..., b] * s.abs()
                out[..., b] = z[..., b] * c.abs() + z[..., a] * s.abs()
            else:
                out[..., a] = z[..., a] * c - z[..., b] * sn
                out[..., b] = z[..., b] * c + z[..., a] * sn
        return out

    wv = w if norm else torch.ones_like(w)
    y = turn(n * wv)
    mag = turn((n * wv).abs(), absolute=True)
    val = {"y": y}
    # the mean of squares: d terms, halved by the root; product, weight, rotation: 8 more
    tol = {"y": 1.01 * ((d / 2 + 12) * F32 * mag + u * y.abs())}
    if dy is not None:
        g = dy.double()
        du, gm = turn(g, back=True), turn(g.abs(), back=True, absolute=True)
        if norm:
            dn, dm = du * wv, gm * wv.abs()
            dot = (dn * n).mean(-1, keepdim=True)
            val["dx"] = r * (dn - n * dot)
            size = r * (dm + n.abs() * (dm * n.abs()).mean(-1, keepdim=True))
            tol["dx"] = 1.01 * ((2 * d + 24) * F32 * size + u * val["dx"].abs())
            rows = (du * n).reshape(-1, d)
            val["dw"] = rows.sum(0)
            tol["dw"] = (rows.shape[0] + d / 2 + 16) * F32 * (gm * n.abs()).reshape(-1, d).sum(0)
        else:
            val["dx"] = du
            tol["dx"] = 1.01 * (4 * F32 * gm + u * du.abs())
    return val, tol


def angle_table(rows, rot, device, base=10000.0):
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot)
    a = torch.arange(rows, dtype=torch.float64, device=device)[:, None] * f
    return torch.stack([a.cos(), a.sin()], -1).float()


def close(got, want, tol, what=""):
    """Every value within its bound (and infinities equal)."""
    got = got.double()
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), f"{what}: infinities differ"
    d = (got - want)[~inf].abs()
    t = tol.expand_as(want)[~inf]
    assert not torch.isnan(d).any(), f"{what}: NaN"
    over = d > t + 1e-30
    assert not over.any(), (f"{what}: {int(over.sum())} of {over.numel()} values over their bound, worst "
                            f"{float((d / (t + 1e-30)).max()):.3g} times it, at |error| {float(d[over].max()):.3g}")
