"""AdamW over many tensors, moments in 32 and in 8 bits (GPU).  Each operation
of the kernel is rounded by itself, so a float32 restatement gives the same
bits (with 8-bit moments, of the moments and of float64 parameters; others are
within 4 units of float32 of the update); the float64 formula bounds both."""
import numpy as np
import pytest
import torch

import learn_util as R

pytestmark = pytest.mark.gpu

LR, BETAS, EPS, WD = 3e-3, (0.9, 0.99), 1e-8, 0.05
COMBOS = [("float32", "float32", False), ("float32", "bfloat16", True), ("float32", "float16", True),
          ("float32", "bfloat16", False), ("bfloat16", "bfloat16", False),
          ("float16", "float16", False), ("float64", "float64", False)]
SIZES = [1, 7, 255, 256, 257, 1000, 2048, 2049, 5003, 0, 70000]


def make(sizes, ptype, gtype, bits, seed, offset=0):
    """Tensors, gradients and started moments; `offset` elements past an
    aligned address."""
    rng = np.random.default_rng(seed)
    pt, gt = getattr(torch, ptype), getattr(torch, gtype)

    def put(values, dtype):
        if dtype == torch.float8_e4m3fn:
            base = torch.zeros(values.numel() + offset, dtype=torch.uint8, device="cuda").view(dtype)
            base[offset:].view(torch.uint8).copy_(values.view(torch.uint8))
        else:
            base = torch.zeros(values.numel() + offset, dtype=dtype, device="cuda")
            base[offset:].copy_(values)
        return base[offset:]

    params, grads, m, v, ms, vs = [], [], [], [], [], []
    for n in sizes:
        params.append(put(torch.from_numpy(rng.standard_normal(n)).to(pt), pt))
        grads.append(put(torch.from_numpy(rng.standard_normal(n) * 1e-2).to(gt), gt))
        m32 = (rng.standard_normal(n) * 1e-2).astype(np.float32)
        v32 = (rng.random(n) * 1e-4).astype(np.float32)
        if n > 2:
            m32[1] = v32[1] = 0
        if bits == 32:
            m.append(put(torch.from_numpy(m32), torch.float32))
            v.append(put(torch.from_numpy(v32), torch.float32))
        else:
            for x, keep, codes, scales in ((m32, False, m, ms), (np.sqrt(v32), True, v, vs)):
                q, s = R.encode(x, keep) if n else (torch.empty(0).to(torch.float8_e4m3fn),
                                                    torch.empty(0))
                codes.append(put(q, torch.float8_e4m3fn))
                scales.append(s.cuda())
    return params, grads, m, v, ms, vs


def narrow(x, dtype):
    return torch.from_numpy(np.ascontiguousarray(x)).to(dtype)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("ptype,gtype,copied", COMBOS)
@pytest.mark.parametrize("offset", [0, 1])
def test_three_steps_bit_for_bit(bits, ptype, gtype, copied, offset):
    from differentiable_cholesky_gb300 import learn
    params, grads, m, v, ms, vs = make(SIZES, ptype, gtype, bits, 1, offset)
    state = {"step": 4, "m": m, "v": v}
    if bits == 8:
        state.update(m_scale=ms, v_scale=vs)
    decay = [WD if n != 257 else 0.0 for n in SIZES]
    copies = [torch.zeros(n, dtype=getattr(torch, gtype), device="cuda") for n in SIZES] if copied else None
    opt = learn.AdamW(params, lr=LR, betas=BETAS, eps=EPS, weight_decay=decay, state_bits=bits,
                      copies=copies, state=state)
    scale = torch.tensor(0.37, device="cuda")
    now = [(p.cpu().double().numpy() if ptype == "float64" else p.cpu().float().numpy(),
            R.decode(m[i].cpu(), ms[i].cpu()) if bits == 8 else m[i].cpu().numpy().copy(),
            R.decode(v[i].cpu(), vs[i].cpu()) if bits == 8 else v[i].cpu().numpy().copy())
           for i, p in enumerate(params)]
    for k in range(3):
        opt.step(grads, grad_scale=scale)
        for i, n in enumerate(SIZES):
            if n == 0:
                continue
            p0, m0, r0 = now[i]
            g = grads[i].cpu().float().numpy()
            p1, m1, v1, r1 = R.adamw(p0, g, m0, r0, bits, LR, *BETAS, EPS, decay[i], 5 + k,
                                     scale.item())
            if bits == 32 or ptype == "float64":
                assert torch.equal(params[i].cpu(), narrow(p1, params[i].dtype)), (k, n)
                if copied:
                    assert torch.equal(copies[i].cpu(), narrow(p1, copies[i].dtype))
            else:  # the update's units, and float32's own rounding of the difference
                upd = np.abs(p0 * np.float32(1.0 - LR * decay[i]) - p1)
                room = 4 * R.U32 * upd + R.U32 * (np.abs(p0) + upd)
                R.within(params[i], p1.astype(np.float64), room, params[i].dtype)
                if copied:
                    R.within(copies[i], p1.astype(np.float64), room, copies[i].dtype)
            p1 = params[i].cpu().double().numpy() if ptype == "float64" else params[i].cpu().float().numpy()
            if bits == 32:
                assert torch.equal(opt.m[i].cpu(), torch.from_numpy(m1))
                assert torch.equal(opt.v[i].cpu(), torch.from_numpy(v1))
                now[i] = (p1, m1, v1)
            else:
                for x, keep, q, s in ((m1, False, opt.m[i], opt.m_scale[i]),
                                      (r1, True, opt.v[i], opt.v_scale[i])):
                    want, ws = R.encode(x, keep)
                    assert torch.equal(s.cpu(), ws)
                    assert torch.equal(q.cpu().view(torch.uint8), want.view(torch.uint8))
                now[i] = (p1, R.decode(opt.m[i].cpu(), opt.m_scale[i].cpu()),
                          R.decode(opt.v[i].cpu(), opt.v_scale[i].cpu()))
    assert opt.steps == 7


@pytest.mark.parametrize("ptype", ["float32", "float64"])
def test_against_the_formula_in_64_bits(ptype):
    """Steps from zero: m and v within a few roundings of their magnitudes, the
    parameter within its own rounding and those of lr |update|."""
    from differentiable_cholesky_gb300 import learn
    params, grads, _, _, _, _ = make([3001], ptype, ptype, 32, 2)
    p64 = params[0].double().cpu().numpy()
    opt = learn.AdamW(params, lr=LR, betas=BETAS, eps=EPS, weight_decay=WD)
    m = v = mag = np.zeros(3001)
    moved = np.zeros(3001)
    for t in range(1, 6):
        g = R.f64(grads[0].float()) * (1.0 if t % 2 else -0.5)
        opt.step([(grads[0] * (1.0 if t % 2 else -0.5)).contiguous()])
        m = BETAS[0] * m + (1 - BETAS[0]) * g
        mag = BETAS[0] * mag + (1 - BETAS[0]) * np.abs(g)
        v = BETAS[1] * v + (1 - BETAS[1]) * g * g
        root = np.sqrt(v / (1 - BETAS[1] ** t)) + EPS
        p64 = p64 * (1 - LR * WD) - LR * m / (1 - BETAS[0] ** t) / root
        moved += LR * mag / (1 - BETAS[0] ** t) / root
        R.within(opt.m[0], m, 4 * t * R.U32 * mag, torch.float32)
        R.within(opt.v[0], v, 5 * t * R.U32 * v, torch.float32)
        unit = R.U32 if ptype == "float32" else 2.0 ** -53
        off = np.abs(R.f64(params[0]) - p64)
        assert np.all(off <= 3 * t * unit * (np.abs(p64) + moved) + (8 * t + 12) * R.U32 * moved)


@pytest.mark.parametrize("eps,size", [(1e-8, 1e-21), (0.0, 1e-21), (1e-30, 1e-3), (0.0, 1e-3)])
def test_small_eps_and_tiny_gradients_in_8_bits(eps, size):
    """Second moments below the normal numbers, and an eps that hides nothing:
    the same codes as one operation at a time gives."""
    from differentiable_cholesky_gb300 import learn
    rng = np.random.default_rng(8)
    n = 2048
    g = (rng.standard_normal(n) * size).astype(np.float32)
    p = torch.from_numpy(rng.standard_normal(n).astype(np.float32)).cuda()
    p0 = p.cpu().numpy()
    opt = learn.AdamW([p], lr=LR, betas=BETAS, eps=eps, weight_decay=WD, state_bits=8)
    opt.step([torch.from_numpy(g).cuda()])
    zero = np.zeros(n, np.float32)
    with np.errstate(divide="ignore", invalid="ignore"):
        p1, m1, v1, r1 = R.adamw(p0, g, zero, zero, 8, LR, *BETAS, eps, WD, 1, 1.0)
    for x, keep, q, s in ((m1, False, opt.m[0], opt.m_scale[0]), (r1, True, opt.v[0], opt.v_scale[0])):
        want, ws = R.encode(x, keep)
        assert torch.equal(s.cpu(), ws)
        assert torch.equal(q.cpu().view(torch.uint8), want.view(torch.uint8))
    upd = np.abs(p0 * np.float32(1.0 - LR * WD) - p1)
    R.within(p, p1.astype(np.float64), 4 * R.U32 * upd + R.U32 * (np.abs(p0) + upd), torch.float32)


def test_many_tensors_and_mixed_types():
    """More tensors than one launch carries, of three types; equal to one
    optimiser for each tensor."""
    from differentiable_cholesky_gb300 import learn
    rng = np.random.default_rng(3)
    sizes = [int(s) for s in rng.integers(1, 700, 800)]
    parts = [make(sizes[i::3], p, g, 8, 4 + i) for i, (p, g) in
             enumerate((("float32", "float32"), ("bfloat16", "bfloat16"), ("float64", "float64")))]
    params = sum((p[0] for p in parts), [])
    grads = sum((p[1] for p in parts), [])
    alone = [p.clone() for p in params]
    opt = learn.AdamW(params, state_bits=8)
    opt.step(grads)
    for i in range(0, len(alone), 37):
        one = learn.AdamW([alone[i]], state_bits=8)
        one.step([grads[i]])
        assert torch.equal(alone[i], params[i])
        assert torch.equal(one.m[0].view(torch.uint8), opt.m[i].view(torch.uint8))
        assert torch.equal(one.v_scale[0], opt.v_scale[i])


@pytest.mark.parametrize("bits", [32, 8])
def test_status_skips_and_missing_gradients_stay(bits):
    from differentiable_cholesky_gb300 import learn
    params, grads, m, v, ms, vs = make([500, 300], "float32", "float32", bits, 5)
    state = {"step": 0, "m": m, "v": v, "m_scale": ms, "v_scale": vs}
    opt = learn.AdamW(params, state_bits=bits, state=state)
    every = params + [t.view(torch.uint8) if bits == 8 else t for t in m + v] + ms + vs
    was = [t.clone() for t in every]
    status = torch.ones((), dtype=torch.int32, device="cuda")
    opt.step(grads, status=status)
    assert all(torch.equal(a, b) for a, b in zip(was, every))
    status.zero_()
    opt.step([None, grads[1]], status=status)
    assert torch.equal(params[0], was[0]) and not torch.equal(params[1], was[1])
    params[0].grad = grads[0]
    opt.step()
    assert not torch.equal(params[0], was[0]) and opt.steps == 3


def test_roots_above_zero_stay_above_zero_and_zero_blocks_stay_zero():
    from differentiable_cholesky_gb300 import learn
    p = torch.ones(600, device="cuda")
    g = torch.zeros(600, device="cuda")
    g[:256] = 1e-9
    g[0] = 10.0
    opt = learn.AdamW([p], state_bits=8, weight_decay=0.0)
    opt.step([g])
    root = opt.v[0].float()
    assert (root[:256] > 0).all() and not root[256:].any()
    assert torch.equal(p[256:], torch.ones(344, device="cuda"))
    assert opt.m_scale[0][1].item() == 2.0 ** -100
    before = p.clone()
    opt.step([torch.zeros_like(g)])
    # roots held at the least code: the step stays below lr times a small factor
    assert (p - before).abs().max().item() <= 1e-3 * 2


def test_nonfinite_gradients_are_seen():
    from differentiable_cholesky_gb300 import learn
    for bits in (32, 8):
        p, g = torch.ones(600, device="cuda"), torch.ones(600, device="cuda")
        g[300] = float("nan")
        opt = learn.AdamW([p], state_bits=bits)
        opt.step([g])
        assert torch.isnan(p[300]) and torch.isfinite(p[:300]).all() and torch.isfinite(p[301:]).all()
        if bits == 8:
            assert torch.isnan(opt.m_scale[0][1]) and torch.isfinite(opt.m_scale[0][[0, 2]]).all()


def test_state_round_trip_and_zero_start():
    from differentiable_cholesky_gb300 import learn
    for bits in (32, 8):
        params, grads, _, _, _, _ = make([400, 90], "float32", "float32", bits, 6)
        twin = [p.clone() for p in params]
        a = learn.AdamW(params, state_bits=bits)
        a.step(grads)
        b = learn.AdamW(twin, state_bits=bits)
        for t, p in zip(twin, params):
            t.copy_(p)
        b.load_state_dict(a.state_dict())
        a.step(grads)
        b.step(grads)
        assert all(torch.equal(x, y) for x, y in zip(params, twin)) and b.steps == 2


def test_shapes_learning_rate_and_requires_grad():
    from differentiable_cholesky_gb300 import learn
    w = torch.randn((30, 17), device="cuda", requires_grad=True)
    opt = learn.AdamW([w], lr=1.0, weight_decay=0.0)
    version = w._version
    (w * 2).sum().backward()
    before = w.detach().clone()
    opt.step(lr=0.25)
    assert torch.allclose(w.detach(), before - 0.25, atol=1e-6) and opt.m[0].shape == w.shape
    assert w._version > version  # autograd sees the change


@pytest.mark.parametrize("bits", [32, 8])
def test_element_offsets_beyond_32_bits(bits):
    """One tensor of 2^31 elements and a few: its end moves as its beginning."""
    from differentiable_cholesky_gb300 import learn
    n = (1 << 31) + 300
    p = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    values = torch.randn(300, device="cuda").to(torch.bfloat16)
    g[:300] = values
    g[-300:] = values
    opt = learn.AdamW([p], lr=1e-2, state_bits=bits)
    opt.step([g])
    assert p[:256].any() and torch.equal(p[:256], p[-300:-44])
    assert not p[300:4000].any() and not p[-5000:-300].any()
    if bits == 32:
        assert torch.equal(opt.m[0][:300], opt.m[0][-300:])


@pytest.mark.parametrize("bits", [32, 8])
def test_another_stream_and_graph_capture(bits):
    from differentiable_cholesky_gb300 import learn
    params, grads, _, _, _, _ = make([1000, 37], "bfloat16", "bfloat16", bits, 7)
    twin = [p.clone() for p in params]
    a, b = learn.AdamW(params, state_bits=bits), learn.AdamW(twin, state_bits=bits)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a.step(grads, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    b.step(grads)
    assert all(torch.equal(x, y) for x, y in zip(params, twin))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.step(grads)
    graph.replay()
    b.step(grads)
    assert all(torch.equal(x, y) for x, y in zip(params, twin))
