"""Calls of the operators next to ELSAA that their documentation allows or refuses and
that test_gpu_layer.py does not make, and the code paths of larger sizes."""

import threading

import pytest
import torch

import layer_reference as ref
from sparse_rank_hybrid_simhash_b200 import binding as B
from sparse_rank_hybrid_simhash_b200 import paged, rotary, window
from test_gpu_layer import DT, heads, paged_inputs, rand, window_inputs

pytestmark = pytest.mark.gpu


# ---- sequences that do not fit ---------------------------------------------------

def starts_of(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("starts,lengths,good", [
    ((0, 3, 5, 6), (20, 1, 30), (0, 2)),           # fewer tokens than new ones
    ((0, 3, 5, 6), (20, 0, 30), (0, 2)),
    ((0, 3, 5, 6), (20, -7, 30), (0, 2)),
    ((0, 3, 5, 6), (20, 49, 30), (0, 2)),          # more than the page table holds
    ((0, 3, 5, 9), (20, 40, 30), (0, 1)),          # rows past q's
    ((0, 3, 5, 1 << 30), (20, 40, 30), (0, 1)),
    ((-2, 3, 5, 6), (20, 40, 30), (1, 2)),         # rows before q's
    ((-2, -1, 5, 6), (20, 40, 30), (2,)),
    ((0, 3, 3, 1), (20, 40, 30), (0, 1)),          # starts that fall behind a sequence without new tokens
], ids=str)
def test_sequences_that_do_not_fit_are_left_out_whole(cuda_device, dt, starts, lengths, good):
    """The write, like the attention, records such a sequence and touches nothing of it."""
    p, q, kp, vp, table, _, _ = paged_inputs((4, 2, 64, dt, 16, 0, 0, [(3, 48), (2, 48), (1, 48)]), slack=1)
    kp, vp = rand(kp.shape, DT[dt], 1), rand(vp.shape, DT[dt], 2)
    k, v = (rand((p.rows, 2, 64), DT[dt], s) for s in (3, 4))
    tab = rotary.angle_table(64, 64, device=cuda_device)
    rp = rotary.RotaryParams.make(1, 4, 2, 1, 64, dt, 64, 64)
    st, ln = starts_of(*starts), starts_of(*lengths)
    ws = paged.alloc_workspace(p, cuda_device)
    k0, v0 = kp.clone(), vp.clone()
    qo, y = torch.full_like(q, 5.0), torch.full_like(q, 5.0)
    paged.write(p, rp, q, k, v, tab, None, None, kp, vp, table, st, ln, qo=qo, ws=ws)
    with pytest.raises(B.ElsaaError) as e:
        B.check(ws)
    assert e.value.code == 6
    paged.attend(p, q, kp, vp, table, st, ln, y=y, ws=ws)
    with pytest.raises(B.ElsaaError) as e:
        B.check(ws)
    assert e.value.code == 6
    touched = torch.zeros(p.rows, dtype=torch.bool, device=cuda_device)
    for b in good:
        rows = torch.arange(starts[b], starts[b + 1], device=cuda_device)
        pos = rows + lengths[b] - starts[b + 1]
        touched[rows] = True
        at = (table.long()[b, pos // 16], slice(None), pos % 16)
        for x, got in ((q, qo[rows]), (k, kp[at])):
            val, tol = ref.rotary(x[rows], None, pos[:, None].expand(x[rows].shape[:2]), tab, False, True, 1e-6)
            ref.close(got, val["y"], tol["y"])
        assert torch.equal(vp[at], v[rows])
        kp[at], vp[at] = k0[at], v0[at]
    assert torch.equal(kp, k0) and torch.equal(vp, v0)     # nothing else in the pools has changed
    assert (qo[~touched] == 5.0).all() and (y[~touched] == 5.0).all()
    assert torch.isfinite(y).all() and (y[touched] != 5.0).any(-1).all()


# ---- positions -------------------------------------------------------------------

def test_a_short_angle_table_is_refused(cuda_device):
    """Through every entry point that takes tokens in order; a table of N rows, or positions, or no rotation serve."""
    q, k = rand((1, 2, 20, 64), torch.bfloat16, 1), rand((1, 1, 20, 64), torch.bfloat16, 2)
    short = rotary.angle_table(19, 64, device=cuda_device)
    p = rotary.RotaryParams.make(1, 2, 1, 20, 64, "bf16", 64, 19)
    for call in (lambda: rotary.norm_rotate(q, k, short), lambda: rotary.QkRotary(short).apply(q, k),
                 lambda: rotary.forward(p, q, k, short), lambda: rotary.forward(p, q, None, short),
                 lambda: rotary.backward(p, q, k, short, None, None, q, k)):
        with pytest.raises(B.ElsaaError) as e:
            call()
        assert e.value.code == 1
    pos = torch.arange(20, dtype=torch.int32, device=cuda_device).clamp(max=18)[None]
    some = rotary.norm_rotate(q, k, short, positions=pos)
    whole = rotary.norm_rotate(q, k, rotary.angle_table(20, 64, device=cuda_device))
    for a, b in zip(some, whole):
        assert torch.equal(a[:, :, :19], b[:, :, :19]) and a[:, :, 19].any()
    rotary.norm_rotate(q, k)                   # norm only


def test_records_of_the_autograd_functions_can_be_read(cuda_device):
    """With a workspace of the caller's: positions outside the table, in the forward and the backward."""
    q, k = (rand((1, h, 20, 64), torch.bfloat16, h).requires_grad_() for h in (2, 1))
    tab = rotary.angle_table(20, 64, device=cuda_device)
    ws = rotary.alloc_workspace(rotary.RotaryParams.make(1, 2, 1, 20, 64, "bf16", 64, 20), cuda_device)
    pos = torch.arange(20, dtype=torch.int32, device=cuda_device)[None]
    for at, bad in ((pos, False), (pos + 1, True), (pos - 1, True)):
        qo, ko = rotary.norm_rotate(q, k, tab, positions=at, ws=ws)
        for _ in range(2):                     # the forward's record, then the backward's
            if bad:
                with pytest.raises(B.ElsaaError) as e:
                    B.check(ws)
                assert e.value.code == 6
            B.check(ws)
            (qo.float().sum() + ko.float().sum()).backward(retain_graph=True)
        q.grad = k.grad = None
    # through ELSAA's own call, and through the attention (its error word set by hand)
    qo, ko = rotary.QkRotary(tab, positions=pos + 1, ws=ws).apply(q, k)
    with pytest.raises(B.ElsaaError):
        B.check(ws)
    ws = window.alloc_workspace(window.WindowParams.make(1, 2, 1, 20, 64, "bf16", 8), cuda_device)
    y = window.window_attention(q, k, k, window=8, ws=ws)
    want = window.window_attention(q, k, k, window=8)
    assert torch.equal(y, want)
    ws[0] = 1
    a, b = torch.autograd.grad(y.float().sum(), (q, k)), torch.autograd.grad(want.float().sum(), (q, k))
    assert all(torch.equal(s, t) for s, t in zip(a, b))
    with pytest.raises(B.ElsaaError) as e:     # the calls only ever set it
        B.check(ws)
    assert e.value.code == 5
    # one for the forward alone is too small for the backward
    small = window.alloc_workspace(window.WindowParams.make(1, 2, 1, 20, 64, "bf16", 8), cuda_device, backward=False)
    y = window.window_attention(q, k, k, window=8, ws=small)
    with pytest.raises(B.ElsaaError) as e:
        y.float().sum().backward()
    assert e.value.code == 3


# ---- masked keys --------------------------------------------------------------------

@pytest.mark.parametrize("H,Hkv,N,d,dt,win,sinks", [
    (2, 1, 260, 64, "bf16", 40, 0), (3, 3, 260, 128, "bf16", 40, 0), (4, 2, 330, 128, "bf16", 0, 0),
    (2, 2, 260, 64, "bf16", 33, 2), (2, 1, 200, 32, "bf16", 40, 0), (2, 1, 260, 64, "f32", 40, 2)])
def test_window_values_of_masked_keys_are_in_no_row(cuda_device, H, Hkv, N, d, dt, win, sinks):
    """A key that a row does not see leaves the row's bits alone, however large its value."""
    q, k, v = (rand((1, h, N, d), DT[dt], 40 + i) for i, h in enumerate((H, Hkv, Hkv)))
    p = window.WindowParams.make(1, H, Hkv, N, d, dt, win, sinks)
    y, lse = window.forward(p, q, k, v)
    for j in (2, 66, 67, 74, 107, 130, 203):    # (every eighth pair of keys takes another exponential)
        if j >= N:
            continue
        v2 = v.clone()
        v2[:, :, j] = 1e38
        y2, lse2 = window.forward(p, q, k, v2)
        blind = ~ref.visible(N, N, 0, win, sinks, cuda_device)[:, j]
        assert blind.any() and torch.equal(y[:, :, blind], y2[:, :, blind]) and torch.equal(lse, lse2)


@pytest.mark.parametrize("H,Hkv,d,dt,seqs,win", [
    (8, 2, 64, "bf16", [(60, 300), (33, 200)], 50), (8, 2, 128, "bf16", [(200, 300)], 0),
    (4, 2, 128, "bf16", [(1, 200), (4, 170)], 40), (4, 2, 32, "bf16", [(60, 300)], 50), (4, 2, 64, "f32", [(60, 300)], 50)])
def test_paged_values_of_masked_keys_are_in_no_row(cuda_device, H, Hkv, d, dt, seqs, win):
    p, q, kp, vp, table, starts, lengths = paged_inputs((H, Hkv, d, dt, 16, win, 0, seqs), slack=0)
    y = paged.attend(p, q, kp, vp, table, starts, lengths)
    n, x = seqs[0]
    for j in (106, 130, 131, 162, 234, 251):
        if j >= x:
            continue
        v2 = vp.clone()
        v2[table[0, j // 16].long(), :, j % 16] = 1e38
        y2 = paged.attend(p, q, kp, v2, table, starts, lengths)
        blind = ~ref.visible(n, x, x - n, win, 0, cuda_device)[:, j]
        assert torch.equal(y[:n][blind], y2[:n][blind]) and torch.equal(y[n:], y2[n:])


# ---- NaN is not lost ------------------------------------------------------------------

@pytest.mark.parametrize("H,Hkv,N,d,dt,win", [(2, 1, 260, 64, "bf16", 40), (3, 3, 260, 128, "bf16", 0),
                                              (2, 2, 200, 32, "bf16", 40), (2, 1, 260, 64, "f32", 40)])
def test_window_nan_stays(cuda_device, H, Hkv, N, d, dt, win):
    """Rows of a NaN query, and rows that see a NaN key, are not finite, in y, lse and the gradients."""
    q, k, v, dy = (rand((1, h, N, d), DT[dt], 50 + i) for i, h in enumerate((H, Hkv, Hkv, H)))
    p = window.WindowParams.make(1, H, Hkv, N, d, dt, win, 0)
    y0, _ = window.forward(p, q, k, v)
    rows = torch.tensor([0, 5, 130, N - 1], device=cuda_device)
    q2 = q.clone()
    q2[:, :, rows] = float("nan")
    y, lse = window.forward(p, q2, k, v)
    assert y[:, :, rows].isnan().all() and lse[:, :, rows].isnan().all()
    rest = torch.ones(N, dtype=torch.bool, device=cuda_device)
    rest[rows] = False
    assert torch.equal(y[:, :, rest], y0[:, :, rest]) and lse[:, :, rest].isfinite().all()
    dq, dk, dv = window.backward(p, q2, k, v, y, lse, dy)
    assert not dq[:, :, rows].isfinite().any() and dq[:, :, rest].isfinite().all()
    assert not dk[:, :, rows].isfinite().all(-1).any() and not dv[:, :, rows].isfinite().all(-1).any()
    for j in (3, 64, 99):
        k2 = k.clone()
        k2[:, :, j] = float("nan")
        y, lse = window.forward(p, q, k2, v)
        sees = ref.visible(N, N, 0, win, 0, cuda_device)[:, j]
        assert not y[:, :, sees].isfinite().any() and torch.equal(y[:, :, ~sees], y0[:, :, ~sees])
        dq, dk, _ = window.backward(p, q, k2, v, y, lse, dy)
        assert not dq[:, :, sees].isfinite().all(-1).any() and not dk[:, :, j].isfinite().all(-1).any()


@pytest.mark.parametrize("H,Hkv,d,dt,seqs", [
    (8, 2, 64, "bf16", [(60, 700), (33, 200)]), (4, 4, 128, "bf16", [(100, 900)]), (8, 2, 128, "bf16", [(1, 900), (2, 60)]),
    (4, 2, 32, "bf16", [(1, 2000)]), (4, 2, 64, "f32", [(60, 300), (1, 2000)])])
def test_paged_nan_stays(cuda_device, H, Hkv, d, dt, seqs):
    p, q, kp, vp, table, starts, lengths = paged_inputs((H, Hkv, d, dt, 16, 0, 0, seqs), slack=0)
    y0 = paged.attend(p, q, kp, vp, table, starts, lengths)
    assert y0.isfinite().all()
    q2 = q.clone()
    q2[0] = float("nan")
    y = paged.attend(p, q2, kp, vp, table, starts, lengths)
    assert y[0].isnan().all() and torch.equal(y[1:], y0[1:])
    n = seqs[0][0]
    k2 = kp.clone()
    k2[table[0, 1].long(), :, 7] = float("nan")
    y = paged.attend(p, q, k2, vp, table, starts, lengths)
    assert not y[:n].isfinite().any() and torch.equal(y[n:], y0[n:])


# ---- the paths of larger sizes ----------------------------------------------------------

@pytest.mark.parametrize("case", [
    # many heads a lane group, not a multiple of what is loaded together
    (2, 15, 5, 10000, 64, "bf16", 64, False, True), (1, 21, 7, 9700, 128, "bf16", 96, True, False),
    (2, 15, 5, 10000, 32, "f32", 32, False, False), (1, 18, 3, 4800, 128, "f32", 128, True, True)], ids=str)
def test_rotary_many_heads_a_group(cuda_device, case):
    B_, H, Hkv, N, d, dt, rot, il, fused = case
    q, k, gq, gk = (heads(B_, h, N, d, DT[dt], 60 + i, fused) for i, h in enumerate((H, Hkv, H, Hkv)))
    wq, wk = (1 + rand((d,), torch.float32, s, 0.2) for s in (64, 65))
    tab = rotary.angle_table(N, rot, device=cuda_device)
    p = rotary.RotaryParams.make(B_, H, Hkv, N, d, dt, rot, N, il, True, 1e-5)
    ws = rotary.alloc_workspace(p, cuda_device)
    qo, ko = rotary.forward(p, q, k, tab, wq, wk, ws=ws)
    dq, dk, dwq, dwk = rotary.backward(p, q, k, tab, wq, wk, gq, gk, ws=ws)
    B.check(ws)
    at = torch.arange(N, device=cuda_device).expand(B_, 1, N)
    for x, w, g, o, dx, dw in ((q, wq, gq, qo, dq, dwq), (k, wk, gk, ko, dk, dwk)):
        val, tol = ref.rotary(x, w, at.expand(x.shape[:3]), tab, il, True, 1e-5, dy=g)
        for name, got in (("y", o), ("dx", dx), ("dw", dw)):
            ref.close(got, val[name], tol[name], name)
    # in place, both ways
    rotary.forward(p, q, k, tab, wq, wk, qo=(a := q.clone()), ko=(b := k.clone()), ws=ws)
    assert torch.equal(a, qo) and torch.equal(b, ko)
    a, b = q.clone(), k.clone()
    rotary.forward(p, a, b, tab, wq, wk, qo=a, ko=b, ws=ws)
    assert torch.equal(a, qo) and torch.equal(b, ko)
    a, b = gq.clone(), gk.clone()
    got = rotary.backward(p, q, k, tab, wq, wk, a, b, dq=a, dk=b, ws=ws)
    assert all(torch.equal(x, y) for x, y in zip(got, (dq, dk, dwq, dwk)))


@pytest.mark.parametrize("H,Hkv,d,dt,seqs", [
    (13, 13, 128, "bf16", [(1700, 1800), (0, 5), (3300, 3301)]), (12, 6, 64, "f32", [(2600, 2600), (2500, 2501)]),
    # more sequences than a block keeps the starts of, some of them without new tokens
    (4, 2, 64, "bf16", [(b % 3, 20 + b % 40) for b in range(2500)])], ids=["heads-bf16", "heads-f32", "2500-sequences"])
def test_paged_write_of_many_rows(cuda_device, H, Hkv, d, dt, seqs):
    p, q, kp, vp, table, starts, lengths = paged_inputs((H, Hkv, d, dt, 16, 0, 0, seqs))
    kp, vp = rand(kp.shape, DT[dt], 70), rand(vp.shape, DT[dt], 71)
    k, v = (rand((p.rows, Hkv, d), DT[dt], s) for s in (72, 73))
    wq, wk = (1 + rand((d,), torch.float32, s, 0.2) for s in (74, 75))
    most = max(x for _, x in seqs)
    tab = rotary.angle_table(most, d, device=cuda_device)
    rp = rotary.RotaryParams.make(1, H, Hkv, 1, d, dt, d, most)
    ws = paged.alloc_workspace(p, cuda_device)
    k0, v0 = kp.clone(), vp.clone()
    qo = torch.full_like(q, 5.0)
    paged.write(p, rp, q, k, v, tab, wq, wk, kp, vp, table, starts, lengths, qo=qo, ws=ws)
    B.check(ws)
    end = int(starts[-1])
    pos = torch.cat([torch.arange(x - n, x) for n, x in seqs]).to(cuda_device)
    seq = torch.repeat_interleave(torch.arange(len(seqs)), torch.tensor([n for n, _ in seqs])).to(cuda_device)
    at = (table.long()[seq, pos // 16], slice(None), pos % 16)
    for x, w, got in ((q[:end], wq, qo[:end]), (k[:end], wk, kp[at])):
        val, tol = ref.rotary(x, w, pos[:, None].expand(x.shape[:2]), tab, False, True, 1e-6)
        ref.close(got, val["y"], tol["y"])
    assert (qo[end:] == 5.0).all() and torch.equal(vp[at], v[:end])
    kp[at], vp[at] = k0[at], v0[at]
    assert torch.equal(kp, k0) and torch.equal(vp, v0)


@pytest.mark.parametrize("case", [
    # more sequences than lanes for the tensor-core kernel's walk, some of them without new tokens
    (8, 2, 64, "bf16", 16, 0, 0, [(0 if b % 7 == 3 else 6 + b % 20, 30 + 11 * b) for b in range(40)]),
    (4, 1, 128, "bf16", 32, 100, 3, [(0 if b % 5 == 0 else 1 + 7 * b % 60, 60 + 5 * b) for b in range(70)]),
    (2, 2, 64, "bf16", 16, 0, 0, [(0, 9)] * 33 + [(600, 700)] + [(0, 5)] * 3),
    # the CUDA-core kernel's
    (8, 2, 64, "f32", 16, 0, 0, [(0 if b % 7 == 3 else 6 + b % 20, 30 + 11 * b) for b in range(40)]),
    # a long chunk among single tokens; as many sequences as a large server decodes
    (2, 2, 64, "bf16", 16, 0, 0, [(1, 40 + b) for b in range(63)] + [(900, 1200)]),
    (4, 2, 128, "bf16", 16, 0, 0, [(b % 2, 1 + b % 90) for b in range(2100)])],
    ids=["tc-40", "tc-70", "tc-one-of-37", "f32-40", "chunk-among-tokens", "decode-2100"])
def test_paged_attend_many_sequences(cuda_device, case):
    p, q, kp, vp, table, starts, lengths = paged_inputs(case)
    want, tol = ref.paged(q, kp, vp, table, starts, lengths, p.window, p.sinks)
    ws = paged.alloc_workspace(p, cuda_device)
    y = torch.full_like(q, 5.0)
    paged.attend(p, q, kp, vp, table, starts, lengths, y=y, ws=ws)
    B.check(ws)
    end = int(starts[-1])
    ref.close(y[:end], want[:end], tol[:end], "y")
    assert (y[end:] == 5.0).all() and not ws[:8192].any()


@pytest.mark.parametrize("case", [
    # 64-row query and key tiles in fp32
    (2, 8, 4, 500, 64, "f32", 100, 0, None, False), (2, 8, 4, 500, 128, "f32", 70, 3, (500, 321), True),
    (1, 12, 12, 600, 64, "f32", 0, 0, None, True), (1, 12, 3, 900, 128, "f32", 20, 1, (850,), False),
    (2, 12, 12, 1300, 64, "f32", 30, 5, (1300, 700), False)], ids=str)
def test_window_large_tiles_in_fp32(cuda_device, case):
    p, q, k, v, dy, lens = window_inputs(case, seed=110)
    val, tol = ref.window(q, k, v, p.window, p.sinks, lens, dy=dy)
    ws = window.alloc_workspace(p, cuda_device)
    y, lse = window.forward(p, q, k, v, lengths=lens, ws=ws)
    grads = window.backward(p, q, k, v, y, lse, dy, lengths=lens, ws=ws)
    B.check(ws)
    for name, g in zip(("y", "lse", "dq", "dk", "dv"), (y, lse, *grads)):
        ref.close(g, val[name], tol[name], name)
    assert not ws[:8192].any()


def test_calls_at_the_same_time(cuda_device):
    """Two streams with a workspace each, window steps on one and decoding on the other."""
    p, q, k, v, dy, lens = window_inputs((4, 16, 4, 1100, 64, "bf16", 300, 3, (1100, 0, 100, 1), False))
    y, lse = window.forward(p, q, k, v, lengths=lens)
    want = (y, lse, *window.backward(p, q, k, v, y, lse, dy, lengths=lens))
    pp, *args = paged_inputs((8, 2, 128, "bf16", 16, 0, 0, [(1, 900 + 13 * b) for b in range(9)]), slack=0)
    pwant = paged.attend(pp, *args)
    ws, pws = window.alloc_workspace(p, cuda_device), paged.alloc_workspace(pp, cuda_device)
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    got, pgot = [], []
    for _ in range(5):
        y, lse = window.forward(p, q, k, v, lengths=lens, ws=ws, stream=s)
        got.append((y, lse, *window.backward(p, q, k, v, y, lse, dy, lengths=lens, ws=ws, stream=s)))
        pgot += [paged.attend(pp, *args, ws=pws, stream=t) for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for g in got for a, b in zip(g, want))
    assert all(torch.equal(g, pwant) for g in pgot)
    B.check(ws), B.check(pws)


def in_a_new_thread(f):
    """f's result from a thread that has made no CUDA call."""
    got = []

    def run():
        try:
            got.append(f())
        except Exception as e:
            got.append(e)

    t = threading.Thread(target=run)
    t.start()
    t.join()
    if isinstance(got[0], Exception):
        raise got[0]
    return got[0]


def test_first_call_of_a_thread(cuda_device):
    """With every buffer the caller's, so that nothing before the call has set the thread up."""
    p, q, k, v, dy, _ = window_inputs((1, 4, 2, 200, 64, "bf16", 64, 2, None, False))
    ws = window.alloc_workspace(p, cuda_device)
    y, lse = window.forward(p, q, k, v, ws=ws)
    grads = window.backward(p, q, k, v, y, lse, dy, ws=ws)
    out = [torch.zeros_like(t) for t in (y, lse, *grads)]
    torch.cuda.synchronize()
    in_a_new_thread(lambda: window.forward(p, q, k, v, y=out[0], lse=out[1], ws=ws))
    in_a_new_thread(lambda: window.backward(p, q, k, v, y, lse, dy, dq=out[2], dk=out[3], dv=out[4], ws=ws))
    assert all(torch.equal(a, b) for a, b in zip(out, (y, lse, *grads)))
    for new in (1, 40):
        pp, *args = paged_inputs((8, 2, 128, "bf16", 16, 0, 0, [(new, 300)]), slack=0)
        ws = paged.alloc_workspace(pp, cuda_device)
        want, got = paged.attend(pp, *args, ws=ws), torch.zeros_like(args[0])
        torch.cuda.synchronize()
        in_a_new_thread(lambda: paged.attend(pp, *args, y=got, ws=ws))
        assert torch.equal(got, want)


def test_first_call_of_a_thread_elsaa(cuda_device):
    from sparse_rank_hybrid_simhash_b200.workloads import WORKLOADS, make_inputs, small
    w = small(WORKLOADS["text-32k"], B=1, H=2, N=1024)
    p = B.Params.from_workload(w)
    d = {n: t.to(cuda_device) for n, t in make_inputs(w, with_dy=True).items()}
    args = [d[n] for n in ("q", "k", "v", "r_sort", "r_race", "gate_w", "gate_b", "lam")]
    saved, ws = B.alloc_saved(p, cuda_device), B.alloc_workspace(p, cuda_device)
    y = B.forward(p, *args, saved=saved, ws=ws)
    grads = B.backward(p, *args, saved, d["dy"], ws=ws)
    torch.cuda.synchronize()
    again = in_a_new_thread(lambda: B.backward(p, *args, saved, d["dy"], ws=ws))
    assert torch.equal(in_a_new_thread(lambda: B.forward(p, *args, saved=saved, ws=ws)), y)
    assert all(torch.equal(a, b) for a, b in zip(grads, again))


def test_paged_write_in_place(cuda_device):
    """The new queries normed and rotated where they are; an output in an input's place is refused elsewhere."""
    p, q, kp, vp, table, starts, lengths = paged_inputs((12, 4, 64, "bf16", 16, 0, 0, [(30, 40), (1, 70)]), slack=0)
    k, v = (rand((p.rows, 4, 64), torch.bfloat16, s) for s in (1, 2))
    tab = rotary.angle_table(70, 64, device=cuda_device)
    rp = rotary.RotaryParams.make(1, 12, 4, 1, 64, "bf16", 64, 70)
    want = paged.write(p, rp, q, k, v, tab, None, None, kp, vp, table, starts, lengths)
    wide = torch.zeros(p.rows, 20, 64, dtype=q.dtype, device=cuda_device)
    wide[:, :12], wide[:, 12:16], wide[:, 16:] = q, k, v
    parts = wide.split([12, 4, 4], dim=1)
    paged.write(p, rp, *parts, tab, None, None, kp, vp, table, starts, lengths, qo=parts[0])
    assert torch.equal(parts[0], want) and torch.equal(parts[1], k) and torch.equal(parts[2], v)
    for call in (lambda: paged.attend(p, want, kp, vp, table, starts, lengths, y=want),
                 lambda: paged.write(p, rp, q, k, v, tab, None, None, kp, kp, table, starts, lengths)):
        with pytest.raises(B.ElsaaError) as e:
            call()
        assert e.value.code == 1


def test_rotary_refuses_gradients_it_does_not_write(cuda_device):
    """A caller's buffer is written or refused, never left as it was."""
    q, k = rand((1, 2, 9, 64), torch.float32, 1), rand((1, 1, 9, 64), torch.float32, 2)
    tab, w = rotary.angle_table(9, 64, device=cuda_device), torch.ones(64, device=cuda_device)
    plain = rotary.RotaryParams.make(1, 2, 1, 9, 64, "f32", 64, 9, norm=False)
    normed = rotary.RotaryParams.make(1, 2, 1, 9, 64, "f32", 64, 9)
    for kw in (dict(dq_weight=w), dict(dk_weight=w)):
        with pytest.raises(ValueError):
            rotary.backward(plain, q, k, tab, None, None, q, k, **kw)
    with pytest.raises(ValueError):
        rotary.backward(normed, q, None, tab, w, None, q, None, dk_weight=w)
    into = torch.full((2, 64), 7.0, device=cuda_device)
    got = rotary.backward(normed, q, k, tab, w, w, q, k, dq_weight=into[0], dk_weight=into[1])
    want = rotary.backward(normed, q, k, tab, w, w, q, k)
    assert torch.equal(into[0], want[2]) and torch.equal(into[1], want[3]) and got[2] is not None
