"""Gated linear recurrence, its reverse mode and its single step, against
float64 (GPU)."""
import numpy as np
import pytest
import torch

import learn_util as R

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.float16, torch.bfloat16]


def draw(shape, dtype, seed, scale=1.0, mean=0.0):
    rng = np.random.default_rng(seed)
    return torch.from_numpy(rng.standard_normal(shape) * scale + mean).to(dtype).cuda()


def draw_gate(shape, dtype, seed, kind):
    rng = np.random.default_rng(seed)
    g = rng.standard_normal(shape)
    if kind == "linear":
        g = 1.0 - np.exp(g - 2.0)            # decays of both signs, below 1
    elif kind == "log":
        g = -np.exp(g * 1.5 - 2.0)
    else:
        g = g * 2.0 + 2.0
    return torch.from_numpy(g).to(dtype).cuda()


def rows_of(t):
    return R.f64(t if t.dim() == 3 else t[None])


def check(gate, x, state, offsets, kind, comp, seed=0, adjoint=True, zero_state=False):
    from differentiable_cholesky_gb300 import learn
    how = dict(offsets=offsets, kind=kind, complement=comp)
    n = offsets.numel() - 1 if offsets is not None else (x.shape[0] if x.dim() == 3 else 1)
    d = x.shape[-1]
    h, last = learn.linrec_fwd(gate, x, None if zero_state else state, **how)
    s64 = np.zeros((n, d)) if zero_state else R.f64(state)
    off = None if offsets is None else offsets.cpu().tolist()
    want = R.linrec(rows_of(gate), rows_of(x), s64, off, kind, comp)
    R.within(h.view(want[0].shape), want[0], want[2], x.dtype)
    R.within(last, want[1], want[3], torch.float32)
    if not adjoint:
        return h, last
    dh = draw(tuple(x.shape), x.dtype, seed + 100)
    dlast = None if zero_state else draw((n, d), torch.float32, seed + 101)
    dg, dx, d0 = learn.linrec_adj(gate, x, h, dh, None if zero_state else state, dlast, **how)
    l64 = np.zeros((n, d)) if zero_state else R.f64(dlast)
    want = R.linrec_adj(rows_of(gate), rows_of(x), rows_of(h), rows_of(dh), s64, l64, off, kind, comp)
    R.within(dg.view(want[0].shape), want[0], want[3], x.dtype)
    R.within(dx.view(want[1].shape), want[1], want[4], x.dtype)
    R.within(d0, want[2], want[5], torch.float32)
    return h, last


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kind", ["linear", "log", "logit"])
@pytest.mark.parametrize("comp", [False, True])
@pytest.mark.parametrize("batch,time,d", [(3, 70, 40), (2, 5, 33)])
def test_every_gate(dtype, kind, comp, batch, time, d):
    gate, x = draw_gate((batch, time, d), dtype, 1, kind), draw((batch, time, d), dtype, 2)
    check(gate, x, draw((batch, d), torch.float32, 3), None, kind, comp)
    check(gate, x, None, None, kind, comp, zero_state=True)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("batch,time,d", [(1, 1, 1), (1, 1, 4096), (5, 1, 64), (1, 2, 8), (2, 3, 7),
                                          (1, 63, 64), (1, 64, 64), (1, 65, 64), (1, 127, 65),
                                          (1, 128, 128), (1, 129, 128), (2, 257, 72), (1, 1000, 136),
                                          (4, 300, 1), (1, 2049, 32), (1, 5000, 24), (33, 40, 264),
                                          (1, 640, 1001), (2, 513, 1024)])
def test_lengths_and_widths(dtype, batch, time, d):
    kind = "logit" if time % 2 else "log"
    gate, x = draw_gate((batch, time, d), dtype, 4, kind), draw((batch, time, d), dtype, 5)
    check(gate, x, draw((batch, d), torch.float32, 6), None, kind, True, seed=7)


def lengths(kind):
    if kind == "uneven":
        return [5, 0, 1, 130, 64, 0, 0, 200, 63, 1, 1, 300, 0]
    if kind == "one":
        return [777]
    if kind == "single tokens":
        return [1] * 150
    if kind == "empty first":
        return [0, 0, 40, 0]
    return [128] * 5


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("parts", ["uneven", "one", "single tokens", "empty first", "even"])
@pytest.mark.parametrize("d", [16, 70])
@pytest.mark.parametrize("comp", [False, True])
def test_packed_sequences(dtype, parts, d, comp):
    off = torch.tensor(np.concatenate([[0], np.cumsum(lengths(parts))]), dtype=torch.int64).cuda()
    t, n = int(off[-1]), off.numel() - 1
    gate, x = draw_gate((t, d), dtype, 8, "log"), draw((t, d), dtype, 9)
    check(gate, x, draw((n, d), torch.float32, 10), off, "log", comp, seed=11)
    check(gate, x, None, off, "log", comp, zero_state=True)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("sequences", [3, 40, 1500])
@pytest.mark.parametrize("d", [40, 33])
def test_packed_sequences_over_many_tiles(dtype, sequences, d):
    """A long axis, so that blocks walk several tiles: few sequences, some in
    every tile, and more than one window of boundaries (many of them empty)."""
    rng = np.random.default_rng(sequences)
    cut = np.sort(rng.integers(0, 6001, sequences - 1))
    cut[len(cut) // 2:len(cut) // 2 + sequences // 10] = cut[len(cut) // 2]  # a run of empty ones
    off = torch.from_numpy(np.concatenate([[0], np.sort(cut), [6000]])).cuda()
    gate, x = draw_gate((6000, d), dtype, 60, "log"), draw((6000, d), dtype, 61)
    check(gate, x, draw((sequences, d), torch.float32, 62), off, "log", sequences % 2 == 0, seed=63)


def test_sequences_do_not_see_one_another():
    """NaN and infinities of one packed sequence, and of its states, stay there."""
    from differentiable_cholesky_gb300 import learn
    off = torch.tensor([0, 100, 250, 251, 400], device="cuda")
    gate, x = draw_gate((400, 24), torch.float32, 12, "logit"), draw((400, 24), torch.float32, 13)
    state, dh = draw((4, 24), torch.float32, 14), draw((400, 24), torch.float32, 15)
    dlast = draw((4, 24), torch.float32, 16)
    h, last = learn.linrec_fwd(gate, x, state, off)
    adj = learn.linrec_adj(gate, x, h, dh, state, dlast, off)
    bad = [t.clone() for t in (gate, x, state, dh, dlast)]
    bad[0][120, 3] = float("nan")
    bad[1][130] = float("inf")
    bad[2][1] = float("nan")
    bad[3][240] = float("nan")
    bad[4][1] = float("inf")
    h2, last2 = learn.linrec_fwd(bad[0], bad[1], bad[2], off)
    adj2 = learn.linrec_adj(bad[0], bad[1], h2, bad[3], bad[2], bad[4], off)
    keep = torch.cat([torch.arange(100), torch.arange(250, 400)]).cuda()
    for a, b in ((h, h2), (adj[0], adj2[0]), (adj[1], adj2[1])):
        assert torch.equal(a[keep], b[keep])
    others = torch.tensor([0, 2, 3], device="cuda")
    for a, b in ((last, last2), (adj[2], adj2[2])):
        assert torch.equal(a[others], b[others])
    assert torch.isnan(h2[250 - 1]).all() and torch.isnan(adj2[2][1]).all()


@pytest.mark.parametrize("kind", ["log", "logit"])
def test_extreme_gates(kind):
    """Gates at the types' ends: a = 0 forgets, a = 1 keeps, and neither gives
    a NaN from finite values."""
    x = draw((1, 200, 16), torch.float32, 17)
    gate = draw_gate((1, 200, 16), torch.float32, 18, kind)
    low = torch.finfo(torch.float32).min
    gate[0, 50], gate[0, 120] = low, -float("inf")
    gate[0, 51:60] = 0.0 if kind == "log" else 1e30
    gate[0, 130] = 0.0 if kind == "log" else float("inf")
    from differentiable_cholesky_gb300 import learn
    state = draw((1, 16), torch.float32, 19)
    h, last = learn.linrec_fwd(gate, x, state, kind=kind)
    a, c, _, _ = R.gates(R.f64(gate), kind)
    want = R.f64(state)[0]
    hs = []
    for t in range(200):
        want = a[0, t] * want + c[0, t] * R.f64(x)[0, t]
        hs.append(want)
    assert np.abs(R.f64(h)[0] - np.stack(hs)).max() <= 1e-5
    dg, dx, d0 = learn.linrec_adj(gate, x, h, torch.ones_like(x), state, None, kind=kind)
    for t in (h, last, dg, dx, d0):
        assert torch.isfinite(t).all()
    assert not dg[0, 50].any() and not dg[0, 120].any()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [64, 50])
def test_halves_of_one_projection(dtype, d):
    """gate and x as slices of [B, T, 2 D], of [T, B, 2 D] seen as [B, T], and at
    an odd offset."""
    both = draw((3, 90, 2 * d), dtype, 20)
    both[..., :d] = draw_gate((3, 90, d), dtype, 21, "logit")
    state = draw((3, d), torch.float32, 22)
    check(both[..., :d], both[..., d:], state, None, "logit", True)
    turned = both.transpose(0, 1).contiguous().transpose(0, 1)
    check(turned[..., :d], turned[..., d:], state, None, "logit", True)
    odd = torch.zeros((3, 90, 2 * d + 1), dtype=dtype, device="cuda")
    odd[..., 1:] = both
    check(odd[..., 1:d + 1], odd[..., d + 1:], state, None, "logit", True)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kind,comp", [("linear", False), ("log", True), ("logit", True), ("logit", False)])
@pytest.mark.parametrize("batch,d", [(1, 1), (3, 40), (64, 256), (5, 33)])
def test_steps_walk_the_sequence(dtype, kind, comp, batch, d):
    """Token after token: each state to its bound, and h rounded from it."""
    from differentiable_cholesky_gb300 import learn
    time = 9
    gate, x = draw_gate((batch, time, d), dtype, 23, kind), draw((batch, time, d), dtype, 24)
    state = draw((batch, d), torch.float32, 25)
    want = R.linrec(R.f64(gate), R.f64(x), R.f64(state), None, kind, comp)
    whole, last = learn.linrec_fwd(gate, x, state, kind=kind, complement=comp)
    for t in range(time):
        h = learn.linrec_step(gate[:, t], x[:, t], state, kind=kind, complement=comp)
        R.within(h, want[0][:, t], want[2][:, t], dtype)
        assert torch.equal(h, state.to(dtype))
    R.within(state, want[1], want[3], torch.float32)


def test_gradients_agree_with_differences():
    """As for the norm: float32 gradients against central differences of the
    float64 recurrence along random directions (h = 1e-6)."""
    from differentiable_cholesky_gb300 import learn
    off = torch.tensor([0, 40, 40, 190, 200], device="cuda")
    for kind, comp in (("linear", False), ("log", True), ("logit", True)):
        gate, x = draw_gate((200, 12), torch.float32, 26, kind), draw((200, 12), torch.float32, 27)
        state = draw((4, 12), torch.float32, 28)
        dh, dl = draw((200, 12), torch.float32, 29), draw((4, 12), torch.float32, 30)
        for t in (gate, x, state):
            t.requires_grad_(True)
        h, last = learn.linrec(gate, x, state, off, kind, comp)
        ((h * dh).sum() + (last * dl).sum()).backward()

        def loss(g, xx, s):
            h, last, _, _ = R.linrec(g[None], xx[None], s, off.cpu().tolist(), kind, comp)
            return (h[0] * R.f64(dh)).sum() + (last * R.f64(dl)).sum()

        at = [R.f64(gate), R.f64(x), R.f64(state)]
        rng = np.random.default_rng(31)
        for k, t in enumerate((gate, x, state)):
            step = rng.standard_normal(at[k].shape) * 1e-6
            up, down = list(at), list(at)
            up[k], down[k] = at[k] + step, at[k] - step
            diff = (loss(*up) - loss(*down)) / 2
            got = (R.f64(t.grad) * step).sum()
            size = (np.abs(R.f64(t.grad)) * np.abs(step)).sum()
            assert abs(got - diff) <= 1000 * R.U32 * size + 1e-7 * abs(diff)


def test_autograd_with_one_output_used():
    from differentiable_cholesky_gb300 import learn
    gate = draw_gate((2, 30, 8), torch.bfloat16, 32, "logit").requires_grad_(True)
    x = draw((2, 30, 8), torch.bfloat16, 33).requires_grad_(True)
    _, last = learn.linrec(gate, x)
    last.sum().backward()
    assert torch.isfinite(x.grad).all() and gate.grad.any()
    x.grad = gate.grad = None
    h, _ = learn.linrec(gate, x)
    h[:, ::2].float().sum().backward()
    assert x.grad.any()


def test_same_bits_each_time():
    from differentiable_cholesky_gb300 import learn
    gate, x = draw_gate((2, 4000, 200), torch.bfloat16, 34, "logit"), draw((2, 4000, 200), torch.bfloat16, 35)
    state, dh = draw((2, 200), torch.float32, 36), draw((2, 4000, 200), torch.bfloat16, 37)
    h, last = learn.linrec_fwd(gate, x, state)
    adj = learn.linrec_adj(gate, x, h, dh, state, state)
    for _ in range(5):
        h2, last2 = learn.linrec_fwd(gate, x, state)
        adj2 = learn.linrec_adj(gate, x, h2, dh, state, state)
        assert torch.equal(h, h2) and torch.equal(last, last2)
        assert all(torch.equal(p, q) for p, q in zip(adj, adj2))


def test_empty_shapes():
    from differentiable_cholesky_gb300 import learn
    gate = torch.empty((2, 0, 16), device="cuda")
    state = draw((2, 16), torch.float32, 38)
    h, last = learn.linrec_fwd(gate, gate, state)
    assert h.shape == (2, 0, 16) and torch.equal(last, state)
    _, last = learn.linrec_fwd(gate, gate)
    assert not last.any()
    dg, dx, d0 = learn.linrec_adj(gate, gate, h, gate, state, state)
    assert torch.equal(d0, state) and dg.numel() == 0
    none = torch.empty((0, 5, 16), device="cuda")
    h, last = learn.linrec_fwd(none, none)
    assert h.shape == (0, 5, 16) and last.shape == (0, 16)
    off = torch.zeros(4, dtype=torch.int64, device="cuda")
    flat, s3 = torch.empty((0, 16), device="cuda"), draw((3, 16), torch.float32, 39)
    _, last = learn.linrec_fwd(flat, flat, s3, off)
    assert torch.equal(last, s3)
    h = learn.linrec_step(torch.empty((0, 16), device="cuda"), torch.empty((0, 16), device="cuda"),
                          torch.empty((0, 16), device="cuda"))
    assert h.shape == (0, 16)


def test_bidiagonal_solve_of_the_factor():
    """The recurrence is forward substitution with a bidiagonal factor: on the
    512 x 512 worked example (diagonal linspace(1, 2), sub-diagonal 0.5),
    E h = x gives h_t = -0.5 / e_t h_{t-1} + x_t / e_t."""
    from differentiable_cholesky_gb300 import learn
    from differentiable_cholesky_gb300 import workloads as W
    E = W.bidiagonal_E(512)
    rhs = np.random.default_rng(40).standard_normal((512, 6))
    want = np.linalg.solve(E, rhs)
    diag = np.diag(E)[:, None]
    gate = torch.from_numpy(np.broadcast_to(-0.5 / diag, (512, 6)).copy()).float().cuda()
    h, _ = learn.linrec_fwd(gate, torch.from_numpy(rhs / diag).float().cuda(), kind="linear",
                            complement=False)
    # |a| <= 0.5: roundings of a, x and each step add up to at most 2 * 4 units
    assert np.abs(R.f64(h) - want).max() <= 8 * R.U32 * np.abs(want).max() * 2


def test_element_offsets_beyond_32_bits():
    from differentiable_cholesky_gb300 import learn
    ts = (1 << 30) + 8
    flat = torch.zeros(2 * ts + 128, dtype=torch.bfloat16, device="cuda")
    x = flat.as_strided((1, 3, 64), (0, ts, 1))
    gate = flat[64:].as_strided((1, 3, 64), (0, ts, 1))
    x.copy_(draw((1, 3, 64), torch.bfloat16, 41))
    gate.copy_(draw_gate((1, 3, 64), torch.bfloat16, 42, "logit"))
    h, last = learn.linrec_fwd(gate, x)
    h2, last2 = learn.linrec_fwd(gate.contiguous(), x.contiguous())
    assert torch.equal(h, h2) and torch.equal(last, last2)
    adj = learn.linrec_adj(gate, x, h, x)
    adj2 = learn.linrec_adj(gate.contiguous(), x.contiguous(), h, x.contiguous())
    assert all(torch.equal(p, q) for p, q in zip(adj, adj2))


def test_a_long_axis():
    """A time axis of 2^31 / 1024 steps and a few more: element offsets of
    contiguous tensors pass 2^31.  Decays of 1/2 forget in 60 steps, so the end
    is that of the last 512 steps alone (2^-512 apart)."""
    from differentiable_cholesky_gb300 import learn
    t, d = (1 << 21) + 77, 1024
    gate = torch.zeros((t, d), dtype=torch.bfloat16, device="cuda")
    x = torch.zeros((t, d), dtype=torch.bfloat16, device="cuda")
    x[-512:] = draw((512, d), torch.bfloat16, 43)
    x[:4] = 1
    h, last = learn.linrec_fwd(gate, x)
    want = R.linrec(R.f64(gate[None, -512:]), R.f64(x[None, -512:]), np.zeros((1, d)), None, "logit", True)
    R.within(h[None, -512:], want[0], want[2], torch.bfloat16)
    R.within(last, want[1], want[3], torch.float32)
    assert torch.equal(h[:3, 0].float().cpu(), torch.tensor([0.5, 0.75, 0.875]))


@pytest.mark.parametrize("time", [1, 700])
def test_another_stream_and_graph_capture(time):
    from differentiable_cholesky_gb300 import learn
    gate, x = draw_gate((2, time, 64), torch.bfloat16, 44, "logit"), draw((2, time, 64), torch.bfloat16, 45)
    state = draw((2, 64), torch.float32, 46)
    want, last = learn.linrec_fwd(gate, x, state)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    h, l2 = learn.linrec_fwd(gate, x, state, stream=side)
    adj = learn.linrec_adj(gate, x, h, x, state, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(h, want) and torch.equal(last, l2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h3, l3 = learn.linrec_fwd(gate, x, state)
        adj3 = learn.linrec_adj(gate, x, h3, x, state)
    for seed in (47, 48):
        x.copy_(draw((2, time, 64), torch.bfloat16, seed))
        graph.replay()
        want, last = learn.linrec_fwd(gate, x, state)
        adj = learn.linrec_adj(gate, x, want, x, state)
        assert torch.equal(h3, want) and torch.equal(l3, last)
        assert all(torch.equal(p, q) for p, q in zip(adj, adj3))
