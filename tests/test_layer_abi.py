"""The operators next to ELSAA without a GPU: validation, sizes, refusals."""

import ctypes

import pytest
import torch

import layer_reference as ref
from sparse_rank_hybrid_simhash_b200 import binding as B
from sparse_rank_hybrid_simhash_b200 import layer, paged, rotary, window

NULL = None
GOOD, BAD = 1 << 20, (1 << 20) + 8   # addresses that validation alone looks at


def rot(**kw):
    p = rotary.RotaryParams.make(2, 8, 2, 100, 64, "bf16", rot_dim=32, max_pos=128)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def win(**kw):
    p = window.WindowParams.make(2, 8, 2, 100, 64, "bf16", window=16, sinks=2)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def pag(**kw):
    p = paged.PagedParams.make(3, 10, 8, 2, 64, "bf16", 16, 20, 6, window=16, sinks=2)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


SHAPE = [dict(H=0), dict(Hkv=0), dict(Hkv=3), dict(d=0), dict(dtype=7), dict(H=-8), dict(H=1 << 15)]


@pytest.mark.parametrize("make,mod,bad,unsupported", [
    (rot, rotary, SHAPE + [dict(B=0), dict(N=0), dict(N=1 << 30), dict(rot_dim=8), dict(rot_dim=80),
                           dict(rot_dim=-16), dict(interleaved=2), dict(norm=2), dict(max_pos=0),
                           dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf"))], [dict(d=48)]),
    (win, window, SHAPE + [dict(B=0), dict(N=0), dict(N=1 << 30), dict(window=-1), dict(sinks=-1),
                           dict(scale=float("nan")), dict(scale=float("inf"))], [dict(d=96)]),
    (pag, paged, SHAPE + [dict(seqs=0), dict(rows=0), dict(page_size=0), dict(page_size=24), dict(pages=0),
                          dict(table_width=0), dict(window=-1), dict(sinks=-1), dict(scale=float("nan")),
                          dict(page_size=1 << 16, table_width=1 << 15), dict(seqs=1 << 20, table_width=1 << 11)],
     [dict(d=96), dict(H=130, Hkv=1)]),
])
def test_validation(make, mod, bad, unsupported):
    assert mod.validate(make()) == 0
    assert mod.workspace_bytes(make()) >= 256
    for kw in bad:
        assert mod.validate(make(**kw)) == 1, kw
        assert mod.workspace_bytes(make(**kw)) == 0, kw
    for kw in unsupported:
        assert mod.validate(make(**kw)) == 2, kw


def test_edges_that_are_valid():
    for kw in (dict(rot_dim=0, max_pos=0), dict(norm=0), dict(rot_dim=64), dict(eps=0.0), dict(d=128, rot_dim=48)):
        assert rotary.validate(rot(**kw)) == 0, kw
    for kw in (dict(window=0), dict(window=(1 << 31) - 1), dict(sinks=(1 << 31) - 1), dict(N=1), dict(Hkv=8),
               dict(scale=-1.0)):
        assert window.validate(win(**kw)) == 0, kw
    for kw in (dict(page_size=48), dict(rows=1, seqs=1), dict(H=128, Hkv=2), dict(window=0)):
        assert paged.validate(pag(**kw)) == 0, kw
    with pytest.raises(ValueError):
        rotary.alloc_workspace(rot(B=0), "cpu")


def i64(*v):
    return (ctypes.c_int64 * len(v))(*v)


def rotary_call(p, q=GOOD, strides=NULL, table=GOOD, ws=GOOD, nbytes=None, k=GOOD, ko=GOOD):
    nbytes = rotary.workspace_bytes(p) if nbytes is None else nbytes
    return B.lib().elsaa_rotary_forward(ctypes.byref(p), q, k, strides, NULL, table, NULL, NULL, GOOD, ko, ws,
                                        nbytes, NULL)


def test_rotary_refusals():
    p = rot()
    assert rotary_call(p, q=NULL) == 1 and rotary_call(p, q=BAD) == 1
    assert rotary_call(p, table=NULL) == 1 and rotary_call(p, ws=NULL) == 1 and rotary_call(p, ws=BAD) == 1
    assert rotary_call(p, ko=NULL) == 1 and rotary_call(p, k=NULL) == 1
    assert rotary_call(p, nbytes=rotary.workspace_bytes(p) - 1) == 3
    dense = (8 * 6400, 6400, 64, 2 * 6400, 6400, 64) * 2
    for at, bad in ((2, 0), (2, 68), (0, -64), (1, 32), (5, 1 << 40)):
        s = list(dense)
        s[at] = bad
        assert rotary_call(p, strides=i64(*s)) == 1, (at, bad)
    # gradients of weights without a norm
    code = B.lib().elsaa_rotary_backward(ctypes.byref(rot(norm=0)), GOOD, GOOD, NULL, NULL, GOOD, NULL, NULL, GOOD,
                                         GOOD, GOOD, GOOD, GOOD, NULL, GOOD, rotary.workspace_bytes(p), NULL)
    assert code == 1


@pytest.mark.parametrize("N,max_pos,rot_dim,code", [(100, 99, 32, 1), (8192, 4096, 64, 1), (2, 1, 16, 1)])
def test_rotary_refuses_a_table_without_a_row_for_every_token(N, max_pos, rot_dim, code):
    """Tokens in order 0 .. N - 1 (no positions) need N rows of the table, forward and backward."""
    p = rot(N=N, max_pos=max_pos, rot_dim=rot_dim)
    assert rotary.validate(p) == 0             # (with positions it is a valid problem)
    assert rotary_call(p) == code
    assert B.lib().elsaa_rotary_backward(ctypes.byref(p), GOOD, GOOD, NULL, NULL, GOOD, NULL, NULL, GOOD, GOOD, GOOD,
                                         GOOD, NULL, NULL, GOOD, rotary.workspace_bytes(p), NULL) == code


def test_window_refusals():
    p = win()
    L = B.lib()

    def fwd(q=GOOD, y=GOOD, lse=GOOD, ws=GOOD, nbytes=None, strides=NULL):
        nbytes = window.workspace_bytes(p, False) if nbytes is None else nbytes
        return L.elsaa_window_forward(ctypes.byref(p), q, GOOD, GOOD, strides, NULL, y, lse, ws, nbytes, NULL)

    for kw in (dict(q=NULL), dict(q=BAD), dict(y=NULL), dict(lse=NULL), dict(lse=GOOD + 2), dict(ws=NULL),
               dict(ws=BAD)):
        assert fwd(**kw) == 1, kw
    assert fwd(nbytes=255) == 3
    s = [8 * 6400, 6400, 64, 2 * 6400, 6400, 64, 2 * 6400, 6400, 64, 8 * 6400, 6400, 64]
    s[4] = 0                      # a broadcast key head
    assert fwd(strides=i64(*s)) == 1
    code = L.elsaa_window_backward(ctypes.byref(p), *([GOOD] * 3), NULL, NULL, *([GOOD] * 6), GOOD,
                                   window.workspace_bytes(p, True) - 1, NULL)
    assert code == 3
    code = L.elsaa_window_backward(ctypes.byref(p), *([GOOD] * 3), NULL, NULL, *([GOOD] * 5), NULL, GOOD,
                                   window.workspace_bytes(p, True), NULL)
    assert code == 1


def test_paged_refusals():
    p = pag()
    L = B.lib()

    def attend(q=GOOD, pt=GOOD, ws=GOOD, nbytes=None, ps=NULL):
        nbytes = paged.workspace_bytes(p) if nbytes is None else nbytes
        return L.elsaa_paged_attend(ctypes.byref(p), q, NULL, GOOD, GOOD, ps, pt, GOOD, GOOD, GOOD, ws, nbytes, NULL)

    for kw in (dict(q=NULL), dict(q=BAD), dict(pt=NULL), dict(pt=GOOD + 2), dict(ws=NULL), dict(ws=BAD),
               dict(ps=i64(2048, 0, 64, 2048, 1024, 64))):
        assert attend(**kw) == 1, kw
    assert attend(nbytes=paged.workspace_bytes(p) - 1) == 3
    for kw in (dict(H=4), dict(Hkv=8), dict(d=128), dict(dtype=1)):   # the norm is of another shape
        r = rot(**kw)
        code = L.elsaa_paged_write(ctypes.byref(p), ctypes.byref(r), *([GOOD] * 3), NULL, *([GOOD] * 6), NULL,
                                   *([GOOD] * 4), 1 << 20, NULL)
        assert code == 1, kw


def test_outputs_that_start_where_another_tensor_does():
    """Refused before anything is launched (each output in turn in the place of each other tensor)."""
    L, at = B.lib(), [(i + 1) << 24 for i in range(11)]
    p, w = win(), window.workspace_bytes(win(), True)
    for o, i in ((3, 0), (3, 1), (3, 2)):
        t = list(at)
        t[o] = t[i]
        assert L.elsaa_window_forward(ctypes.byref(p), *t[:3], NULL, NULL, t[3], t[4], t[5], w, NULL) == 1
    for o in (5, 6, 7):
        for i in range(o):
            t = list(at)
            t[o] = t[i]
            q, k, v, y, dy, dq, dk, dv, lse, ws = t[:10]
            assert L.elsaa_window_backward(ctypes.byref(p), q, k, v, NULL, NULL, y, lse, dy, dq, dk, dv, ws, w,
                                           NULL) == 1, (o, i)
    p, w = pag(), paged.workspace_bytes(pag())
    for i in range(3):
        q, kp, vp, pt, st, ln, y, ws = at[:8]
        y = at[i]
        assert L.elsaa_paged_attend(ctypes.byref(p), q, NULL, kp, vp, NULL, pt, st, ln, y, ws, w, NULL) == 1
    r = rot()
    for o, i in ((3, 1), (3, 2), (4, 0), (4, 1), (4, 2), (4, 3), (5, 0), (5, 1), (5, 2), (5, 3), (5, 4)):
        t = list(at)
        t[o] = t[i]
        q, k, v, qo, kp, vp, table, pt, st, ln, ws = t
        assert L.elsaa_paged_write(ctypes.byref(p), ctypes.byref(r), q, k, v, NULL, table, NULL, NULL, qo, kp, vp, NULL,
                                   pt, st, ln, ws, w, NULL) == 1, (o, i)


def test_python_checks():
    x = torch.zeros(1, 4, 8, 32)
    with pytest.raises(ValueError):          # no CPU path
        window.window_attention(x, x, x, window=4)
    with pytest.raises(TypeError):
        layer.dtype_code(torch.float16)
    for t, taken in ((x, True), (x.transpose(1, 2), True), (x[..., ::2], False), (x[..., 1:], False),
                     (x[:, :1].expand(1, 4, 8, 32), False), (x.flatten(2)[:, :, 4:], True)):
        assert layer.strided(t) == taken
    with pytest.raises(ValueError):
        layer.as_output("y", x[:, :1].expand(1, 4, 8, 32), (1, 4, 8, 32), torch.float32, x.device)
    with pytest.raises(ValueError):          # heads of one token overlap tokens of one head
        layer.as_output("y", torch.zeros(11 * 32).as_strided((1, 4, 8, 32), (0, 32, 32, 1)), (1, 4, 8, 32),
                        torch.float32, x.device)
    for t in (x, x.transpose(1, 2).contiguous().transpose(1, 2), torch.zeros(1, 4, 8, 64)[..., :32]):
        assert layer.as_output("y", t, (1, 4, 8, 32), torch.float32, x.device) is t
    y = layer.as_input("q", x[:, :1].expand(1, 4, 8, 32), (1, 4, 8, 32), torch.float32, x.device)
    assert y.is_contiguous()
    with pytest.raises(TypeError):
        layer.as_input("q", x, x.shape, torch.bfloat16, x.device)
    with pytest.raises(ValueError):
        layer.as_input("q", x, (1, 4, 8, 64), torch.float32, x.device)


def test_reference_gradients_against_differences():
    """The closed-form gradients that the kernels are held to, against autograd and against differences."""
    g = torch.Generator().manual_seed(3)
    q, k, v, dy = (torch.randn(2, h, 9, 4, generator=g, dtype=torch.float64) for h in (4, 2, 2, 4))
    n = torch.tensor([9, 6])

    def f(q, k, v):
        see = ref.visible(9, 9, 0, 3, 2, "cpu") & (torch.arange(9)[None, :, None] < n[:, None, None])[:, None]
        s = (q.view(2, 2, 2, 9, 4) @ k[:, :, None].transpose(-1, -2)) / 2.0
        s = s.masked_fill(~see[:, :, None], -1e300)
        y = torch.softmax(s, -1) @ v[:, :, None]
        return (y * (torch.arange(9)[None, :] < n[:, None]).view(2, 1, 1, 9, 1)).reshape(2, 4, 9, 4)

    leaves = [t.clone().requires_grad_() for t in (q, k, v)]
    want = torch.autograd.grad((f(*leaves) * dy).sum(), leaves)
    # (the reference takes its unit roundings from the dtype; its values are in 64 bits)
    val, _ = ref.window(q, k, v, 3, 2, lengths=n, dy=dy)
    for name, w in zip(("dq", "dk", "dv"), want):
        assert torch.allclose(val[name], w, atol=1e-12), name
    assert torch.autograd.gradcheck(f, leaves)
    x = torch.randn(5, 16, generator=g, dtype=torch.float64).requires_grad_()
    w = torch.randn(16, generator=g, dtype=torch.float64).requires_grad_()
    t, pos = ref.angle_table(9, 8, "cpu"), torch.tensor([0, 1, 8, 3, 3])
    d = torch.randn(5, 16, generator=g, dtype=torch.float64)
    for il in (False, True):
        def h(x, w):
            return ref.rotary(x, w, pos, t, il, True, 1e-3)[0]["y"]
        val, _ = ref.rotary(x.detach(), w.detach(), pos, t, il, True, 1e-3, dy=d)
        gx, gw = torch.autograd.grad((h(x, w) * d).sum(), (x, w))
        assert torch.allclose(val["dx"], gx, atol=1e-12) and torch.allclose(val["dw"], gw, atol=1e-12)
        assert torch.autograd.gradcheck(h, (x, w))
