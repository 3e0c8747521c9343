"""The operators next to ELSAA on the GPU against their formulas in 64 bits
(layer_reference.py), within bounds that count the kernels' roundings."""

import pytest
import torch

import layer_reference as ref
from sparse_rank_hybrid_simhash_b200 import binding as B
from sparse_rank_hybrid_simhash_b200 import paged, rotary, window

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
NAN = float("nan")


def rand(shape, dt, seed, scale=1.0, dev="cuda"):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dev).to(dt)


def heads(B_, h, N, d, dt, seed, fused=False, scale=1.0):
    """[B, h, N, d], dense or as a view of [B, N, h, d]."""
    x = rand((B_, N, h, d) if fused else (B_, h, N, d), dt, seed, scale)
    return x.transpose(1, 2) if fused else x


# ---- norm and rotation -------------------------------------------------------

ROTARY = [
    # B, H, Hkv, N, d, dtype, rot, interleaved, norm, fused
    (1, 1, 1, 1, 64, "bf16", 64, False, True, False),
    (2, 4, 2, 37, 32, "f32", 16, True, True, False),
    (1, 8, 2, 130, 128, "bf16", 128, False, True, True),
    (2, 3, 3, 33, 64, "bf16", 48, False, True, False),
    (1, 2, 1, 65, 128, "f32", 96, True, True, True),
    (3, 5, 1, 19, 32, "bf16", 32, True, False, False),
    (1, 4, 4, 50, 64, "f32", 64, False, False, True),
    (1, 4, 2, 40, 128, "bf16", 0, False, True, False),
    (2, 12, 12, 1500, 64, "bf16", 64, False, True, False),
    (1, 17, 1, 700, 32, "f32", 32, False, True, False),
]


@pytest.mark.parametrize("case", ROTARY, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("far", [False, True], ids=["token-order", "positions"])
def test_rotary(cuda_device, case, far):
    B_, H, Hkv, N, d, dt, rot, il, norm, fused = case
    dt = DT[dt]
    q, k = heads(B_, H, N, d, dt, 1, fused), heads(B_, Hkv, N, d, dt, 2, fused)
    dqo, dko = heads(B_, H, N, d, dt, 3), heads(B_, Hkv, N, d, dt, 4, fused)
    rows = 40000 if far else N
    tab = ref.angle_table(rows, rot, cuda_device) if rot else None
    pos = (torch.randint(0, rows, (B_, N), generator=torch.Generator().manual_seed(5)).int().to(cuda_device)
           if far else None)
    wq, wk = (1 + rand((d,), torch.float32, s, 0.2) for s in (6, 7)) if norm else (None, None)
    p = rotary.RotaryParams.make(B_, H, Hkv, N, d, dt, rot, rows, il, norm, 1e-5)
    ws = rotary.alloc_workspace(p, cuda_device)
    qo, ko = rotary.forward(p, q, k, tab, wq, wk, pos, ws=ws)
    got = rotary.backward(p, q, k, tab, wq, wk, dqo, dko, pos, ws=ws)
    B.check(ws)
    at = (pos if far else torch.arange(N, device=cuda_device).expand(B_, N))[:, None]
    for x, w, do, o, dx, dw in ((q, wq, dqo, qo, got[0], got[2]), (k, wk, dko, ko, got[1], got[3])):
        val, tol = ref.rotary(x, w, at.expand(x.shape[:3]), tab, il, norm, 1e-5, dy=do)
        ref.close(o, val["y"], tol["y"], "y")
        ref.close(dx, val["dx"], tol["dx"], "dx")
        if norm:
            ref.close(dw, val["dw"], tol["dw"], "dw")
        else:
            assert dw is None
    again = rotary.backward(p, q, k, tab, wq, wk, dqo, dko, pos, ws=ws)
    assert all(a is None and b is None or torch.equal(a, b) for a, b in zip(got, again))
    # in place
    a, b = q.clone(), k.clone()
    rotary.forward(p, a, b, tab, wq, wk, pos, qo=a, ko=b, ws=ws)
    assert torch.equal(a, qo) and torch.equal(b, ko)
    # queries only
    alone, none = rotary.forward(p, q, None, tab, wq, None, pos, ws=ws)
    assert none is None and torch.equal(alone, qo)


@pytest.mark.parametrize("case", [(2, 9, 3, 70, 64, "bf16"), (1, 12, 3, 900, 128, "bf16"), (3, 20, 1, 40, 32, "f32")])
def test_rotary_backward_alone_and_in_place(cuda_device, case):
    """Gradients of the queries alone, and gradients written over the incoming ones."""
    B_, H, Hkv, N, d, dt = case
    q, k, gq, gk = (rand((B_, h, N, d), DT[dt], 20 + i) for i, h in enumerate((H, Hkv, H, Hkv)))
    tab, w = rotary.angle_table(N, d, device=cuda_device), 1 + rand((d,), torch.float32, 9, 0.2)
    p = rotary.RotaryParams.make(B_, H, Hkv, N, d, dt, d, N)
    want = rotary.backward(p, q, k, tab, w, w, gq, gk)
    at = torch.arange(N, device=cuda_device).expand(B_, H, N)
    dq, dk, dwq, dwk = rotary.backward(p, q, None, tab, w, None, gq, None)
    val, tol = ref.rotary(q, w, at, tab, False, True, 1e-6, dy=gq)
    assert dk is None and dwk is None and torch.equal(dq, want[0])
    ref.close(dwq, val["dw"], tol["dw"], "dw")
    a, b = gq.clone(), gk.clone()
    got = rotary.backward(p, q, k, tab, w, w, a, b, dq=a, dk=b)
    assert all(torch.equal(x, y) for x, y in zip(got, want)) and torch.equal(a, want[0])


def test_rotary_positions_outside_the_table(cuda_device):
    p = rotary.RotaryParams.make(1, 2, 1, 5, 64, "bf16", 64, 8)
    q, k = rand((1, 2, 5, 64), torch.bfloat16, 1), rand((1, 1, 5, 64), torch.bfloat16, 2)
    tab = ref.angle_table(8, 64, cuda_device)
    ws = rotary.alloc_workspace(p, cuda_device)
    pos = torch.tensor([[0, 7, 8, -1, 3]], dtype=torch.int32, device=cuda_device)
    qo, ko = rotary.forward(p, q, k, tab, positions=pos, ws=ws)
    with pytest.raises(B.ElsaaError) as e:
        B.check(ws)
    assert e.value.code == 6
    B.check(ws)                       # read and cleared
    inside = rotary.forward(p, q, k, tab, positions=pos.clamp(0, 7), ws=ws)
    B.check(ws)
    for got, want in zip((qo, ko), inside):
        assert torch.equal(got[:, :, [0, 1, 4]], want[:, :, [0, 1, 4]])
        assert not got[:, :, 2:4].any()
    dq, dk, dwq, dwk = rotary.backward(p, q, k, tab, None, None, q, k, positions=pos, ws=ws)
    assert not dq[:, :, 2:4].any() and not dk[:, :, 2:4].any() and torch.isfinite(dwq).all()


def test_rotary_zero_rows_and_eps(cuda_device):
    p = rotary.RotaryParams.make(1, 1, 1, 4, 32, "f32", 0, 0, eps=1e-6)
    x = torch.zeros(1, 1, 4, 32, device=cuda_device)
    x[0, 0, 1, 0] = 1e-20             # its square is below fp32's range
    x[0, 0, 2] = 1e18                 # the sum of squares stays inside fp32
    y, _ = rotary.forward(p, x, x)
    val, tol = ref.rotary(x, None, None, None, False, True, 1e-6)
    ref.close(y, val["y"], tol["y"])
    assert not y[0, 0, 0].any()


def test_norm_rotate_autograd(cuda_device):
    q, k = (rand((2, h, 21, 64), torch.float32, s).requires_grad_() for h, s in ((4, 1), (2, 2)))
    wq, wk = (1 + rand((64,), torch.float32, s, 0.1) for s in (3, 4))
    wq, wk = wq.requires_grad_(), wk.requires_grad_()
    tab = rotary.angle_table(21, 32, device=cuda_device)
    qo, ko = rotary.norm_rotate(q, k, tab, wq, wk, interleaved=True)
    (qo.sum() * 2 + ko[:, :, 3].sum()).backward()       # broadcast gradients
    at = torch.arange(21, device=cuda_device).expand(2, 1, 21)
    dk = torch.zeros_like(k)
    dk[:, :, 3] = 1
    for x, w, g in ((q, wq, torch.full_like(q, 2.0)), (k, wk, dk)):
        val, tol = ref.rotary(x.detach(), w.detach(), at.expand(x.shape[:3]), tab, True, True, 1e-6, dy=g)
        ref.close(x.grad, val["dx"], tol["dx"], "dx")
        ref.close(w.grad, val["dw"], tol["dw"], "dw")


# ---- window attention ----------------------------------------------------------

WINDOW = [
    # B, H, Hkv, N, d, dtype, window, sinks, lengths, fused
    (1, 1, 1, 1, 64, "bf16", 1, 0, None, False),
    (1, 2, 1, 2, 128, "bf16", 0, 0, None, False),
    (1, 2, 2, 127, 64, "bf16", 16, 0, None, False),
    (1, 4, 2, 128, 64, "bf16", 128, 4, None, True),
    (1, 2, 1, 129, 128, "bf16", 1, 1, None, False),
    (2, 4, 2, 300, 64, "bf16", 100, 3, (300, 129), False),
    (3, 4, 1, 333, 128, "bf16", 77, 130, (0, 1, 333), True),
    (1, 6, 2, 700, 128, "bf16", 256, 16, None, False),
    (1, 3, 1, 641, 64, "bf16", 0, 0, None, False),
    (2, 2, 2, 515, 64, "bf16", 200, 300, (515, 400), False),
    (1, 2, 2, 1100, 128, "bf16", 130, 4, None, True),
    (1, 8, 1, 1030, 64, "bf16", 2000, 5, None, False),
    # several tiles a CTA, many of them empty in a row
    (4, 16, 4, 1100, 64, "bf16", 300, 3, (1100, 0, 100, 1), False),
    (5, 12, 12, 900, 128, "bf16", 0, 0, (0, 0, 1, 900, 0), False),
    (2, 4, 2, 200, 32, "f32", 48, 4, None, False),
    (1, 2, 1, 131, 64, "f32", 0, 0, (100,), True),
    (2, 3, 3, 190, 128, "f32", 1, 0, (65, 190), False),
    (1, 4, 4, 70, 128, "f32", 33, 70, None, False),
    (4, 16, 8, 520, 32, "f32", 200, 3, (520, 0, 64, 65), False),
    (1, 8, 1, 700, 128, "f32", 0, 0, (650,), False),
    (1, 8, 1, 400, 32, "bf16", 90, 20, None, True),
    (2, 4, 2, 150, 32, "bf16", 40, 2, (150, 64), False),
    # key tiles of the sinks, seen by far more queries than the others
    (2, 6, 6, 1000, 32, "f32", 10, 3, (1000, 333), False),
    (2, 12, 12, 1121, 32, "f32", 4, 1, None, False),
    (2, 24, 12, 700, 32, "bf16", 5, 130, None, False),
    (1, 4, 1, 900, 128, "f32", 20, 17, (771,), True),
]


def window_inputs(case, seed=10):
    B_, H, Hkv, N, d, dt, win, sinks, lengths, fused = case
    q, k, v, dy = (heads(B_, h, N, d, DT[dt], seed + i, fused) for i, h in enumerate((H, Hkv, Hkv, H)))
    lens = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    p = window.WindowParams.make(B_, H, Hkv, N, d, dt, win, sinks)
    return p, q, k, v, dy, lens


@pytest.mark.parametrize("case", WINDOW, ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_window(cuda_device, case):
    p, q, k, v, dy, lens = window_inputs(case)
    val, tol = ref.window(q, k, v, p.window, p.sinks, lens, dy=dy)
    if lens is not None:              # what lies behind a length is in no result
        for t in (q, k, v, dy):
            for b, n in enumerate(lens.tolist()):
                t[b, :, n:] = NAN
    ws = window.alloc_workspace(p, cuda_device)
    y, lse = window.forward(p, q, k, v, lengths=lens, ws=ws)
    B.check(ws)
    ref.close(y, val["y"], tol["y"], "y")
    ref.close(lse, val["lse"], tol["lse"], "lse")
    dq, dk, dv = window.backward(p, q, k, v, y, lse, dy, lengths=lens, ws=ws)
    B.check(ws)
    for name, g in (("dq", dq), ("dk", dk), ("dv", dv)):
        ref.close(g, val[name], tol[name], name)
    if lens is not None:
        for b, n in enumerate(lens.tolist()):
            assert not any(t[b, :, n:].any() for t in (y, dq, dk, dv))
    again = window.backward(p, q, k, v, y, lse, dy, lengths=lens, ws=ws)
    assert all(torch.equal(a, b) for a, b in zip((dq, dk, dv), again))


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("N,win,sinks", [(1, 0, 0), (2, 0, 0), (3, 9, 1), (16, 0, 0), (40, 2, 0), (150, 1, 0),
                                         (200, 7, 9), (300, 16, 0), (33, 14, 2)])
def test_window_few_keys(cuda_device, d, N, win, sinks):
    """Rows that see at most 16 keys take no part of y's rounding into their gradients."""
    for heads_, lens in (((2, 2), None), ((8, 1), (N, N // 2))):
        case = (2, *heads_, N, d, "bf16", win, sinks, lens, lens is not None)
        p, q, k, v, dy, n = window_inputs(case, seed=90)
        val, tol = ref.window(q, k, v, win, sinks, n, dy=dy, few=16)
        y, lse = window.forward(p, q, k, v, lengths=n)
        for name, g in zip(("dq", "dk", "dv"), window.backward(p, q, k, v, y, lse, dy, lengths=n)):
            ref.close(g, val[name], tol[name], name)


def test_window_large_scores(cuda_device):
    """Row maxima that grow along the keys by far more than a rescaling threshold, and that fall."""
    for flip in (False, True):
        q, k, v = (rand((1, 2, 600, 64), torch.bfloat16, s) for s in (1, 2, 3))
        k = k * torch.linspace(0, 8, 600, device=cuda_device).flip(0 if flip else []).view(1, 1, 600, 1).bfloat16()
        p = window.WindowParams.make(1, 2, 2, 600, 64, "bf16", 400, 2)
        y, lse = window.forward(p, q, k, v)
        val, tol = ref.window(q, k, v, 400, 2)
        ref.close(y, val["y"], tol["y"], "y")
        ref.close(lse, val["lse"], tol["lse"], "lse")


def test_window_scale_and_strided_outputs(cuda_device):
    q, k, v, dy = (heads(2, h, 260, 64, torch.bfloat16, s, True) for h, s in ((4, 1), (2, 2), (2, 3), (4, 4)))
    p = window.WindowParams.make(2, 4, 2, 260, 64, "bf16", 70, 1, scale=0.3)
    val, tol = ref.window(q, k, v, 70, 1, scale=0.3, dy=dy)
    wide = torch.full((2, 260, 3 * 4 * 64), 7.0, dtype=torch.bfloat16, device=cuda_device)
    y = wide[..., :256].unflatten(-1, (4, 64)).transpose(1, 2)
    dq = wide[..., 256:512].unflatten(-1, (4, 64)).transpose(1, 2)
    dk = wide[..., 512:640].unflatten(-1, (2, 64)).transpose(1, 2)
    _, lse = window.forward(p, q, k, v, y=y)
    _, _, dv = window.backward(p, q, k, v, y, lse, dy, dq=dq, dk=dk)
    for name, g in (("y", y), ("dq", dq), ("dk", dk), ("dv", dv)):
        ref.close(g, val[name], tol[name], name)
    assert (wide[..., 640:] == 7.0).all()
    with pytest.raises(ValueError):
        window.forward(p, q, k, v, y=wide[..., 1:257].unflatten(-1, (4, 64)).transpose(1, 2))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_window_attention_autograd_broadcast(cuda_device, dt):
    """A value head broadcast over the heads, and a broadcast output gradient."""
    q = rand((1, 4, 90, 64), DT[dt], 1).requires_grad_()
    k = rand((1, 2, 90, 64), DT[dt], 2).requires_grad_()
    v = rand((1, 1, 90, 64), DT[dt], 3).requires_grad_()
    y = window.window_attention(q, k, v.expand(1, 2, 90, 64), window=20, sinks=1)
    y.sum().backward()
    vv = v.detach().expand(1, 2, 90, 64)
    val, tol = ref.window(q.detach(), k.detach(), vv, 20, 1, dy=torch.ones_like(q))
    ref.close(q.grad, val["dq"], tol["dq"], "dq")
    ref.close(k.grad, val["dk"], tol["dk"], "dk")
    u = ref.unit(DT[dt])
    dv = val["dv"].sum(1, keepdim=True)          # torch adds the heads up, rounding once more
    ref.close(v.grad, dv, tol["dv"].sum(1, keepdim=True) + 2 * u * (dv.abs() + tol["dv"].sum(1, keepdim=True)), "dv")


def test_window_gradients_against_differences(cuda_device):
    q, k, v, dy = (rand((1, h, 40, 32), torch.float32, s) for h, s in ((2, 1), (1, 2), (1, 3), (2, 4)))
    p = window.WindowParams.make(1, 2, 1, 40, 32, "f32", 9, 2)
    y, lse = window.forward(p, q, k, v)
    grads = window.backward(p, q, k, v, y, lse, dy)
    h = 2.0 ** -5
    for n, (x, g) in enumerate(zip((q, k, v), grads)):
        w = rand(x.shape, torch.float32, 20 + n)
        args = [[t, t] for t in (q, k, v)]
        args[n] = [x + h * w, x - h * w]
        f = [(window.forward(p, *(a[i] for a in args))[0].double() * dy.double()).sum() for i in range(2)]
        num, ana = float(f[0] - f[1]) / (2 * h), float((g.double() * w.double()).sum())
        # the central difference is off by h^2 / 6 of the third derivative: a few of the slope's size
        assert abs(num - ana) < 2e-2 * float((g.double().abs() * w.double().abs()).sum()), (n, num, ana)


# ---- paged cache ---------------------------------------------------------------

PAGED = [
    # H, Hkv, d, dtype, page, window, sinks, (new, context) of every sequence
    (4, 4, 64, "bf16", 16, 0, 0, [(1, 1)]),
    (8, 2, 128, "bf16", 16, 0, 0, [(1, 1000), (1, 17), (1, 16), (1, 129)]),
    (12, 4, 64, "bf16", 64, 0, 0, [(1, 5000)]),
    (6, 2, 64, "bf16", 48, 0, 0, [(3, 100), (0, 50), (1, 300), (2, 2)]),
    (32, 8, 128, "bf16", 64, 0, 0, [(1, 700), (1, 64), (0, 0), (1, 65)]),
    (4, 1, 128, "bf16", 32, 100, 4, [(1, 900), (40, 300), (1, 50), (70, 70)]),
    (16, 2, 64, "bf16", 16, 64, 1, [(300, 700), (1, 800), (17, 400)]),
    (3, 3, 128, "bf16", 256, 0, 0, [(200, 600), (129, 129)]),
    (64, 1, 64, "bf16", 16, 30, 20, [(5, 300), (1, 90)]),
    (40, 8, 128, "bf16", 16, 0, 0, [(1, 400), (90, 400)]),
    (4, 2, 32, "bf16", 16, 20, 2, [(1, 100), (9, 80)]),
    (4, 2, 64, "f32", 16, 0, 0, [(1, 300), (33, 90), (0, 10)]),
    (8, 1, 128, "f32", 48, 50, 3, [(2, 400), (1, 1)]),
    (2, 2, 32, "f32", 16, 1, 0, [(4, 60)]),
    (12, 4, 128, "f32", 32, 0, 0, [(1, 3000), (1, 5)]),
    (6, 1, 32, "bf16", 64, 0, 0, [(1, 2500)]),
    (2, 2, 64, "f32", 16, 700, 5, [(100, 1500), (1, 1200)]),
    (8, 4, 32, "f32", 16, 0, 0, [(1, 1 + 53 * b) for b in range(40)]),
    (8, 8, 64, "bf16", 128, 128, 0, [(1, 1 + 37 * b) for b in range(70)]),
    # a prompt's chunk among single tokens (few rows a sequence on average)
    (8, 2, 128, "bf16", 16, 0, 0, [(1, 60 + b) for b in range(7)] + [(40, 500)] + [(1, 90)] * 9),
]


def paged_inputs(case, seed=30, spare=2, slack=3):
    H, Hkv, d, dt, page, win, sinks, seqs = case
    dt = DT[dt]
    need = [-(-x // page) for _, x in seqs]
    pages, width = sum(need) + spare, max(1, max(need))
    T = sum(n for n, _ in seqs) + slack
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).tolist()
    table = torch.full((len(seqs), width), -1, dtype=torch.int32)
    for b, n in enumerate(need):
        table[b, :n] = torch.tensor([order.pop() for _ in range(n)], dtype=torch.int32)
    starts = torch.tensor([sum(n for n, _ in seqs[:b]) for b in range(len(seqs) + 1)], dtype=torch.int32)
    lengths = torch.tensor([x for _, x in seqs], dtype=torch.int32)
    kp, vp = (torch.full((pages, Hkv, page, d), NAN, dtype=dt, device="cuda") for _ in range(2))
    for b, (_, x) in enumerate(seqs):     # what lies behind a length stays NaN
        for j0 in range(0, x, page):
            n = min(page, x - j0)
            kp[table[b, j0 // page], :, :n] = rand((Hkv, n, d), dt, seed + 7 * j0 + b)
            vp[table[b, j0 // page], :, :n] = rand((Hkv, n, d), dt, seed + 7 * j0 + b + 100000)
    q = rand((T, H, d), dt, seed + 1)
    p = paged.PagedParams.make(len(seqs), T, H, Hkv, d, dt, page, pages, width, win, sinks)
    return p, q, kp, vp, table.cuda(), starts.cuda(), lengths.cuda()


@pytest.mark.parametrize("case", PAGED, ids=lambda c: "-".join(map(str, c)).replace(" ", "")[:70])
def test_paged_attend(cuda_device, case):
    p, q, kp, vp, table, starts, lengths = paged_inputs(case)
    want, tol = ref.paged(q, kp, vp, table, starts, lengths, p.window, p.sinks)
    end = int(starts[-1])
    if p.window:      # entries that no token of the call needs are not read
        for b, (n, x) in enumerate(case[-1]):
            used = ref.visible(n, x, x - n, p.window, p.sinks, "cpu").any(0)
            for e in range(-(-x // p.page_size)):
                if not used[e * p.page_size:(e + 1) * p.page_size].any():
                    table[b, e] = p.pages + 5
    ws = paged.alloc_workspace(p, cuda_device)
    y = torch.full((p.rows, p.H, p.d), 5.0, dtype=q.dtype, device=cuda_device)
    paged.attend(p, q, kp, vp, table, starts, lengths, y=y, ws=ws)
    B.check(ws)
    ref.close(y[:end], want[:end], tol[:end], "y")
    assert (y[end:] == 5.0).all()         # rows of no sequence are left as they were
    first = y.clone()
    for _ in range(2):                    # the workspace holds the last call's partials
        paged.attend(p, q, kp, vp, table, starts, lengths, y=y, ws=ws)
    assert torch.equal(first, y)


def test_paged_other_layouts(cuda_device):
    """Pages as [pages, slot, head, d], queries as a slice of a fused projection."""
    case = (8, 2, 64, "bf16", 32, 0, 0, [(1, 100), (150, 260)])
    p, q, kp, vp, table, starts, lengths = paged_inputs(case, slack=0)
    want, tol = ref.paged(q, kp, vp, table, starts, lengths, 0, 0)
    kp, vp = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (kp, vp))
    wide = torch.zeros(p.rows, 12, 64, dtype=q.dtype, device=cuda_device)
    wide[:, :8] = q
    y = paged.attend(p, wide[:, :8], kp, vp, table, starts, lengths)
    ref.close(y, want, tol)


def test_paged_shared_pages(cuda_device):
    """Two sequences that share their first pages (a forked prefix)."""
    case = (4, 2, 128, "bf16", 16, 0, 0, [(1, 40), (1, 40)])
    p, q, kp, vp, table, starts, lengths = paged_inputs(case)
    table[1, :2] = table[0, :2]
    want, tol = ref.paged(q, kp, vp, table, starts, lengths, 0, 0)
    y = paged.attend(p, q, kp, vp, table, starts, lengths)
    ref.close(y[:2], want[:2], tol[:2])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_paged_bad_entries_are_recorded(cuda_device, dt):
    case = (4, 2, 64, dt, 16, 0, 0, [(1, 40), (1, 40), (2, 30)])
    p, q, kp, vp, table, starts, lengths = paged_inputs(case)
    good = paged.attend(p, q, kp, vp, table, starts, lengths)
    for bad in (-1, p.pages, 1 << 30):
        broken = table.clone()
        broken[1, 1] = bad
        ws = paged.alloc_workspace(p, cuda_device)
        y = paged.attend(p, q, kp, vp, broken, starts, lengths, ws=ws)
        with pytest.raises(B.ElsaaError) as e:
            B.check(ws)
        assert e.value.code == 6
        assert torch.equal(y[0], good[0]) and torch.equal(y[2:4], good[2:4])
    # a length that the page table does not hold, or that the new tokens exceed
    for bad in (p.table_width * p.page_size + 1, 0, -5):
        wrong = lengths.clone()
        wrong[1] = bad
        ws = paged.alloc_workspace(p, cuda_device)
        y = paged.attend(p, q, kp, vp, table, starts, wrong, ws=ws)
        with pytest.raises(B.ElsaaError):
            B.check(ws)
        assert torch.equal(y[0], good[0]) and torch.equal(y[2:4], good[2:4])


WRITE = [
    # H, Hkv, d, dtype, page, rot, interleaved, norm, (new, context) of every sequence
    (4, 2, 64, "bf16", 16, 64, False, True, [(1, 1)]),
    (8, 2, 128, "bf16", 16, 128, False, True, [(1, 100), (0, 30), (37, 50), (1, 16), (1, 17)]),
    (6, 3, 32, "f32", 48, 16, True, True, [(5, 60), (100, 100)]),
    (4, 4, 64, "bf16", 64, 32, True, False, [(70, 70), (3, 200)]),
    (2, 1, 128, "f32", 32, 0, False, True, [(9, 40)]),
    (4, 1, 64, "bf16", 16, 64, False, True, [(1 + b % 3, 40 + b) for b in range(90)]),
]


@pytest.mark.parametrize("case", WRITE, ids=lambda c: "-".join(map(str, c)).replace(" ", "")[:60])
def test_paged_write(cuda_device, case):
    H, Hkv, d, dt, page, rot, il, norm, seqs = case
    p, q, kp, vp, table, starts, lengths = paged_inputs((H, Hkv, d, dt, page, 0, 0, seqs))
    kp, vp = rand(kp.shape, DT[dt], 70), rand(vp.shape, DT[dt], 71)
    k, v = (rand((p.rows, Hkv, d), DT[dt], s) for s in (72, 73))
    wq, wk = (1 + rand((d,), torch.float32, s, 0.2) for s in (74, 75)) if norm else (None, None)
    most = max(x for _, x in seqs)
    tab = ref.angle_table(most, rot, cuda_device) if rot else None
    rp = rotary.RotaryParams.make(1, H, Hkv, 1, d, DT[dt], rot, most, il, norm, 1e-5)
    ws = paged.alloc_workspace(p, cuda_device)
    k0, v0 = kp.clone(), vp.clone()
    qo = torch.full_like(q, 5.0)
    paged.write(p, rp, q, k, v, tab, wq, wk, kp, vp, table, starts, lengths, qo=qo, ws=ws)
    B.check(ws)
    end = int(starts[-1])
    pos = torch.cat([torch.arange(x - n, x) for n, x in seqs]).to(cuda_device)
    seq = torch.repeat_interleave(torch.arange(len(seqs)), torch.tensor([n for n, _ in seqs])).to(cuda_device)
    for x, w, got in ((q, wq, qo[:end]),
                      (k, wk, kp[table.long()[seq, pos // page], :, pos % page])):
        x = x[:end]
        val, tol = ref.rotary(x, w, pos[:, None].expand(x.shape[:2]), tab, il, norm, 1e-5)
        ref.close(got, val["y"], tol["y"])
    assert (qo[end:] == 5.0).all()
    at = (table.long()[seq, pos // page], slice(None), pos % page)
    assert torch.equal(vp[at], v[:end])
    kp[at], vp[at] = k0[at], v0[at]       # nothing else in the pools has changed
    assert torch.equal(kp, k0) and torch.equal(vp, v0)


def test_paged_first_row_of_no_sequence(cuda_device):
    """Rows before starts[0] belong to no sequence either."""
    p, q, kp, vp, table, starts, lengths = paged_inputs((4, 2, 64, "bf16", 16, 0, 0, [(2, 20), (3, 40)]))
    starts = starts + 1
    k, v = (rand((p.rows, 2, 64), torch.bfloat16, s) for s in (1, 2))
    rp = rotary.RotaryParams.make(1, 4, 2, 1, 64, "bf16", 0)
    kw, vw = torch.zeros_like(kp), torch.zeros_like(vp)
    qo = torch.full_like(q, 5.0)
    paged.write(p, rp, q, k, v, None, None, None, kw, vw, table, starts, lengths, qo=qo)
    assert (qo[0] == 5.0).all() and (qo[6:] == 5.0).all() and (qo[1:6] != 5.0).any()
    assert int(vw.abs().sum(-1).gt(0).sum()) == 5 * 2
    y = torch.full_like(q, 5.0)
    paged.attend(p, q, kp, vp, table, starts, lengths, y=y)
    want, tol = ref.paged(q[1:], kp, vp, table, starts - 1, lengths, 0, 0)
    ref.close(y[1:6], want[:5], tol[:5])
    assert (y[0] == 5.0).all() and (y[6:] == 5.0).all()


def test_paged_write_bad_entries(cuda_device):
    p, q, kp, vp, table, starts, lengths = paged_inputs((4, 2, 64, "bf16", 16, 0, 0, [(2, 20), (3, 40)]))
    k, v = (rand((p.rows, 2, 64), torch.bfloat16, s) for s in (1, 2))
    kp, vp = torch.zeros_like(kp), torch.zeros_like(vp)
    rp = rotary.RotaryParams.make(1, 4, 2, 1, 64, "bf16", 64, 39)   # position 39 is outside the table
    tab = ref.angle_table(39, 64, cuda_device)
    ws = paged.alloc_workspace(p, cuda_device)
    table[0, 1] = p.pages
    qo = paged.write(p, rp, q, k, v, tab, None, None, kp, vp, table, starts, lengths, ws=ws)
    with pytest.raises(B.ElsaaError) as e:
        B.check(ws)
    assert e.value.code == 6
    assert not qo[4].any() and qo[2:4].any()
    assert int(vp.flatten(1).any(1).sum()) == 1      # the good sequence's page alone was written
    assert torch.equal(vp[table[1, 2], :, 5:8].transpose(0, 1), v[2:5])


# ---- together, streams, graphs, devices ------------------------------------------

@pytest.mark.parametrize("dt,d,win,sinks", [("bf16", 128, 60, 3), ("bf16", 64, 0, 0), ("f32", 64, 40, 2)])
def test_training_layer_equals_serving_layer(cuda_device, dt, d, win, sinks):
    """norm_rotate + window attention over a whole sequence, against the same tokens written and
    attended in chunks and one by one over a paged cache."""
    H, Hkv, N, page = 8, 2, 213, 16
    q, k, v = (rand((1, h, N, d), DT[dt], s) for h, s in ((H, 1), (Hkv, 2), (Hkv, 3)))
    wq, wk = (1 + rand((d,), torch.float32, s, 0.2) for s in (4, 5))
    tab = rotary.angle_table(N, d, device=cuda_device)
    qo, ko = rotary.norm_rotate(q, k, tab, wq, wk)
    whole = window.window_attention(qo, ko, v, win, sinks)[0]
    _, tol = ref.window(qo, ko, v, win, sinks)
    pages = -(-N // page)
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(9)).int().to(cuda_device)[None]
    pool = paged.PagedParams.make(1, 1, H, Hkv, d, dt, page, pages, pages)
    kp, vp = paged.alloc_pages(pool, cuda_device)
    kp.fill_(NAN), vp.fill_(NAN)
    at = 0
    for n in [100, 1, 1, 17, 64, 1, 29]:
        p = paged.PagedParams.make(1, n, H, Hkv, d, dt, page, pages, pages, win, sinks)
        rp = rotary.RotaryParams.make(1, H, Hkv, n, d, dt, d, N)
        starts = torch.tensor([0, n], dtype=torch.int32, device=cuda_device)
        length = torch.tensor([at + n], dtype=torch.int32, device=cuda_device)
        new = [t[0, :, at:at + n].transpose(0, 1) for t in (q, k, v)]
        q1 = paged.write(p, rp, *new, tab, wq, wk, kp, vp, table, starts, length)
        assert torch.equal(q1, qo[0, :, at:at + n].transpose(0, 1))
        y = paged.attend(p, q1, kp, vp, table, starts, length)
        bound = tol["y"][0, :, at:at + n].transpose(0, 1)
        ref.close(y, whole[:, at:at + n].transpose(0, 1).double(), 2 * bound, f"tokens {at}")
        at += n
    assert at == N


def test_elsaa_with_rotary(cuda_device):
    """ELSAA on normed and rotated q and k, forward and backward, in one call."""
    from sparse_rank_hybrid_simhash_b200.workloads import WORKLOADS, make_inputs, small
    w = small(WORKLOADS["text-32k"], B=1, H=2, N=1024)
    p = B.Params.from_workload(w)
    d = {n: t.to(cuda_device) for n, t in make_inputs(w).items()}
    q, k, v = (d[n].clone().requires_grad_() for n in "qkv")
    rest = [d[n] for n in ("gate_w", "gate_b", "lam", "r_sort", "r_race")]
    wq, wk = (torch.full((64,), x, device=cuda_device).requires_grad_() for x in (1.5, 0.75))
    rope = rotary.QkRotary(rotary.angle_table(1024, 64, device=cuda_device), wq, wk)
    y = B.elsaa(q, k, v, *rest, p, rotary=rope)
    y.backward(d["dy"])
    qo, ko = (t.detach().requires_grad_() for t in rope.apply(q.detach(), k.detach()))
    v2 = d["v"].clone().requires_grad_()
    y2 = B.elsaa(qo, ko, v2, *rest, p)
    y2.backward(d["dy"])
    assert torch.equal(y, y2)
    at = torch.arange(1024, device=cuda_device).expand(1, 2, 1024)
    for x, wt, g in ((q, wq, qo.grad), (k, wk, ko.grad)):
        val, tol = ref.rotary(x.detach(), wt.detach(), at, rope.table, False, True, 1e-6, dy=g)
        ref.close(x.grad, val["dx"], tol["dx"] + 1e-6, "dx")
        assert torch.isfinite(wt.grad).all() and wt.grad.any()


def test_another_stream_and_graphs(cuda_device):
    """Calls on a side stream, and two captured graphs of different shapes with a workspace each."""
    case = (2, 4, 2, 300, 64, "bf16", 100, 3, (300, 129), False)
    p, q, k, v, dy, lens = window_inputs(case)
    want = window.forward(p, q, k, v, lengths=lens)
    grads = window.backward(p, q, k, v, *want, dy, lengths=lens)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y, lse = window.forward(p, q, k, v, lengths=lens, stream=side)
    side.synchronize()
    assert torch.equal(y, want[0]) and torch.equal(lse, want[1])
    pc = (8, 2, 128, "bf16", 16, 0, 0, [(1, 1000), (1, 17), (40, 129)])
    pp, pq, kp, vp, table, starts, lengths = paged_inputs(pc)
    end = int(starts[-1])
    pwant = paged.attend(pp, pq, kp, vp, table, starts, lengths)
    bufs, graphs = [], []
    for kind in (0, 1):
        ws = window.alloc_workspace(p, cuda_device) if kind == 0 else paged.alloc_workspace(pp, cuda_device)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            if kind == 0:
                a = window.forward(p, q, k, v, lengths=lens, ws=ws)
                out = (*a, *window.backward(p, q, k, v, *a, dy, lengths=lens, ws=ws))
            else:
                out = (paged.attend(pp, pq, kp, vp, table, starts, lengths, ws=ws),)
        graphs.append(g)
        bufs.append((out, ws))
    for _ in range(2):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(bufs[0][0], (*want, *grads)))
    assert torch.equal(bufs[1][0][0][:end], pwant[:end])
    # new lengths in place: the captured launch reads them on the device
    lengths[0] = 500
    graphs[1].replay()
    y500 = paged.attend(pp, pq, kp, vp, table, starts, lengths)
    torch.cuda.synchronize()
    assert torch.equal(bufs[1][0][0][:end], y500[:end]) and not torch.equal(y500[0], pwant[0])
    for out, ws in bufs:
        B.check(ws)


@pytest.mark.parametrize("dt,d", [("bf16", 64), ("bf16", 32), ("f32", 128)])
def test_offsets_past_32_bits(cuda_device, dt, d):
    """Batches and pages whose strides put an element's offset past 2^31 values."""
    far, dtype = 2 ** 31 + 2 ** 16, DT[dt]
    room = torch.empty(far + 2 ** 20, dtype=dtype, device=cuda_device)

    def apart(x, at):      # x [2, ...] with its halves `far` values apart, at an offset
        to = room.as_strided(x.shape, (far, *x.stride()[1:]), at)
        to.copy_(x)
        return to

    p, q, k, v, dy, _ = window_inputs((2, 4, 2, 150, d, dt, 60, 2, None, False))
    want = window.forward(p, q, k, v)
    grads = window.backward(p, q, k, v, *want, dy)
    size = 4 * 150 * d
    fq, fk, fv = (apart(t, i * size) for i, t in enumerate((q, k, v)))
    y = apart(torch.zeros_like(q), 3 * size)
    _, lse = window.forward(p, fq, fk, fv, y=y)
    assert torch.equal(y, want[0]) and torch.equal(lse, want[1])
    outs = [apart(torch.zeros_like(t), (4 + i) * size) for i, t in enumerate((q, k, v))]
    window.backward(p, fq, fk, fv, y, lse, dy, dq=outs[0], dk=outs[1], dv=outs[2])
    assert all(torch.equal(a, b) for a, b in zip(outs, grads))
    table = rotary.angle_table(150, d, device=cuda_device)
    rp = rotary.RotaryParams.make(2, 4, 2, 150, d, dt, d, 150)
    rotary.forward(rp, fq, fk, table, qo=y, ko=outs[1])
    for a, b in zip((y, outs[1]), rotary.forward(rp, q, k, table)):
        assert torch.equal(a, b)
    # a pool whose page stride puts the second half of its pages there, decoding and in chunks
    for new in (1, 40):
        pp, pq, kp, vp, pages, starts, lengths = paged_inputs(
            (4, 2, d, dt, 16, 0, 0, [(new, 64), (new, 50)]), spare=0, slack=0)
        kp, vp = kp.nan_to_num(), vp.nan_to_num()
        wide = far // (pp.pages - 1) // 8 * 8 + 8      # the last page starts past 2^31
        fk, fv = (room.as_strided(kp.shape, (wide, *kp.stride()[1:]), i * 2 * 16 * d) for i in range(2))
        fk.copy_(kp), fv.copy_(vp)
        assert (pp.pages - 1) * wide > 2 ** 31
        y1 = paged.attend(pp, pq, kp, vp, pages, starts, lengths)
        assert torch.equal(paged.attend(pp, pq, fk, fv, pages, starts, lengths), y1)
        k1, v1 = (rand((pp.rows, 2, d), dtype, 60 + i) for i in range(2))
        rp = rotary.RotaryParams.make(1, 4, 2, 1, d, dt, d, 150)
        for a, b in ((kp, vp), (fk, fv)):
            paged.write(pp, rp, pq, k1, v1, table, None, None, a, b, pages, starts, lengths)
        assert torch.equal(kp, fk) and torch.equal(vp, fv)


def test_workspace_head_is_left_clear(cuda_device):
    """Error word and counters are zero after every call, whatever it shared between CTAs."""
    def clear(ws):
        torch.cuda.synchronize()
        assert not ws[:8192].any()

    for case in ((4, 16, 4, 1100, 64, "bf16", 300, 3, (1100, 0, 100, 1), False), (1, 2, 2, 90, 128, "bf16", 0, 0, None, False),
                 (2, 6, 6, 1000, 32, "f32", 10, 3, (1000, 333), False), (1, 8, 1, 700, 128, "f32", 0, 0, None, False)):
        p, q, k, v, dy, n = window_inputs(case)
        ws = window.alloc_workspace(p, cuda_device)
        y, lse = window.forward(p, q, k, v, lengths=n, ws=ws)
        clear(ws)
        window.backward(p, q, k, v, y, lse, dy, lengths=n, ws=ws)
        clear(ws)
    for case in (PAGED[6], PAGED[2], PAGED[12], PAGED[16]):
        p, *args = paged_inputs(case)
        ws = paged.alloc_workspace(p, cuda_device)
        paged.attend(p, *args, ws=ws)
        clear(ws)


def test_training_step_in_a_graph(cuda_device):
    """Forward and gradients of the training operators captured through autograd, replayed on new inputs."""
    _, q, k, v, dy, _ = window_inputs((1, 4, 2, 200, 64, "bf16", 64, 2, None, False))
    wq, wk = (1 + 0.1 * rand((64,), torch.float32, s) for s in (5, 6))
    leaves = [t.requires_grad_() for t in (q, k, v, wq, wk)]
    table = rotary.angle_table(200, 64, device=cuda_device)

    def step():
        qo, ko = rotary.norm_rotate(q, k, table, wq, wk)
        y = window.window_attention(qo, ko, v, window=64, sinks=2)
        return (y.detach(), *torch.autograd.grad(y, leaves, dy))   # (no autograd graph outlives the step)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    with torch.no_grad():
        q.copy_(q.flip(2)), v.mul_(0.5)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, step()))


def test_refusals_on_the_device(cuda_device):
    p, q, k, v, dy, _ = window_inputs((1, 2, 2, 127, 64, "bf16", 16, 0, None, False))
    with pytest.raises(TypeError):
        window.forward(p, q.float(), k, v)
    with pytest.raises(ValueError):
        window.forward(p, q[:, :1], k, v)
    with pytest.raises(ValueError):
        window.forward(p, q, k.cpu(), v)
    with pytest.raises(TypeError):
        window.forward(p, q, k, v, lengths=torch.tensor([3], device=cuda_device))
    with pytest.raises(B.ElsaaError) as e:
        window.forward(p, q, k, v, ws=torch.zeros(16, dtype=torch.uint8, device=cuda_device))
    assert e.value.code == 3
    with pytest.raises(ValueError):
        rotary.norm_rotate(q, k, rotary.angle_table(8, 64, device=cuda_device)[:, :, 0])
    with pytest.raises(ValueError):       # rows that share memory
        window.forward(p, q, k, v, y=torch.zeros(2 * 127 * 64, dtype=q.dtype, device=cuda_device)
                       .as_strided((1, 2, 127, 64), (0, 64, 64, 1)))
