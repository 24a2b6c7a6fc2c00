"""Root-mean-square norm with the residual's addition, and its reverse mode,
against float64 (GPU)."""
import numpy as np
import pytest
import torch

import learn_util as R

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.float16, torch.bfloat16]
EPS = 1e-6


def draw(shape, dtype, seed, scale=1.0, mean=0.0):
    rng = np.random.default_rng(seed)
    return torch.from_numpy(rng.standard_normal(shape) * scale + mean).to(dtype).cuda()


def check_forward(x, w, res, eps=EPS):
    from differentiable_cholesky_gb300 import learn
    y, r, rstd = learn.rms_norm_fwd(x, w, res, eps=eps)
    r64, s64, y64 = R.norm(R.f64(x), R.f64(w), R.f64(res), eps)
    k = R.norm_rounds(x.shape[-1]) * R.U32
    R.within(rstd, s64, k * np.abs(s64), torch.float32)
    R.within(y, y64, k * np.abs(y64), x.dtype)
    if res is None:
        assert r is x
    else:
        R.within(r, r64, R.U32 * np.abs(r64), res.dtype)
    return y, r, rstd


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,d", [(1, 1), (1, 4096), (3, 7), (5, 64), (4, 129), (2, 1000),
                                    (7, 2048), (3, 5000), (2, 8191), (2, 16384), (1, 40000),
                                    (700, 96)])
def test_forward_sizes(dtype, rows, d):
    x, w = draw((rows, d), dtype, 1), draw((d,), dtype, 2, 0.1, 1.0)
    check_forward(x, w, None)
    check_forward(x, w, draw((rows, d), dtype, 3, 3.0))
    check_forward(x, None, draw((rows, d), torch.float32, 4, 3.0))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad", [1, 8, 24])
@pytest.mark.parametrize("d", [40, 512, 1003])
def test_slices_of_wider_rows(dtype, pad, d):
    x = draw((6, d + pad), dtype, 5)[:, :d]
    res = draw((6, d + pad), torch.float32, 6)[:, pad:]
    check_forward(x, draw((d,), dtype, 7), res)
    wide = draw((2, 3, d + pad), dtype, 8)[..., pad:]
    check_forward(wide, None, None)


def test_memory_that_is_not_vector_aligned():
    flat = draw((4 * 256 + 1,), torch.bfloat16, 9)
    check_forward(flat[1:].view(4, 256), flat[3:259], None)


def test_rows_of_zeros_large_values_and_nonfinite_rows():
    from differentiable_cholesky_gb300 import learn
    x = draw((6, 300), torch.float32, 10)
    x[0] = 0
    x[1] *= 1e18
    x[2] *= 1e-15
    x[3, 17] = float("nan")
    x[4, 299] = float("inf")
    y, _, rstd = learn.rms_norm_fwd(x, None, None, eps=EPS)
    assert not y[0].any() and torch.isnan(y[3]).all()
    assert torch.isnan(y[4, 299]) and not y[4, :299].any()
    keep = [0, 1, 2, 5]
    check_forward(x[keep].contiguous(), None, None)
    y0, _, s0 = learn.rms_norm_fwd(x[:1].contiguous(), None, None, eps=0.0)
    assert torch.isnan(y0).all() and torch.isinf(s0).all()


@pytest.mark.parametrize("kind,top", [("e4m3", 448.0), ("int8", 127.0)])
@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,d,pad", [(1, 1, 0), (3, 128, 0), (2, 5000, 120), (5, 129, 0),
                                        (4, 1000, 8), (3, 8192, 0), (2, 127, 1), (1, 33000, 0),
                                        (9, 777, 3)])
def test_eight_bit_output(kind, top, group, dtype, rows, d, pad):
    """Scales to a few roundings; codes within half a step of their number
    format, plus what the roundings before them move."""
    from differentiable_cholesky_gb300 import learn
    x = draw((rows, d + pad), dtype, 11)[:, :d]
    w, res = draw((d,), dtype, 12), draw((rows, d), dtype, 13, 2.0)
    q, scale, r, rstd = learn.rms_norm_quant(x, w, res, eps=EPS, kind=kind, group=group)
    r64, s64, y64 = R.norm(R.f64(x), R.f64(w), R.f64(res), EPS)
    k = (R.norm_rounds(d) + 8) * R.U32
    R.within(rstd, s64, k * s64, torch.float32)
    R.within(r, r64, R.U32 * np.abs(r64), dtype)
    width = group or d
    groups = -(-d // width)
    tops = np.stack([np.abs(y64[:, i * width:(i + 1) * width]).max(1) for i in range(groups)], 1)
    assert tuple(scale.shape) == (rows, groups)
    R.within(scale, tops / top, k * tops / top, torch.float32)
    step = R.f64(scale).repeat(width, axis=1)[:, :d]
    z = np.abs(y64) / step
    if kind == "e4m3":  # half of 2^-3 of its binade, down to 2^-6; subnormal steps of 2^-9
        half = np.maximum(2.0 ** np.floor(np.log2(np.maximum(z, 2.0 ** -20))), 2.0 ** -6) / 16
    else:
        half = 0.5
    got = R.f64(q.float()) * step
    assert np.all(np.abs(got - y64) <= (half * (1 + 2 * k) + 2 * k * z) * step)


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("d", [384, 301])
def test_eight_bit_zeros_and_nonfinite_values(kind, group, d):
    from differentiable_cholesky_gb300 import learn
    x = draw((4, d), torch.float32, 14)
    x[0] = 0
    x[1, 130] = float("nan")
    w = torch.ones(d, device="cuda")
    w[256:] = 0  # a group of zeros in every row
    q, scale, _, _ = learn.rms_norm_quant(x, w, None, eps=EPS, kind=kind, group=group)
    q, scale = q.float().cpu(), scale.cpu()
    assert not q[0].any() and not scale[0].any()
    if group:
        assert not q[2:, 256:].any() and not scale[2:, 2:].any()
        assert (scale[2:, :2] > 0).all()
    # a NaN makes its row's norm NaN: its scales are NaN, and so is what they stand for
    assert torch.isnan(scale[1, 0])
    # values whose scale is no normal number count as zeros
    tiny = torch.full((d,), 1e-38, device="cuda")
    q, scale, _, _ = learn.rms_norm_quant(x[2:], tiny, None, eps=EPS, kind=kind, group=group)
    assert not scale.any() and not q.float().any()


def check_adjoint(rows, d, dtype, rtype, with_w=True, with_dr=True, pad=0):
    from differentiable_cholesky_gb300 import learn
    x, w = draw((rows, d), dtype, 20), draw((d,), dtype, 21, 0.1, 1.0) if with_w else None
    res = draw((rows, d), rtype, 22, 2.0)
    _, r, rstd = learn.rms_norm_fwd(x, w, res, eps=EPS)
    dy = draw((rows, d + pad), dtype, 23)[:, pad:]
    dr = draw((rows, d), rtype, 24) if with_dr else None
    got, dw = learn.rms_norm_adj(dy, r, rstd, w, adj_r=dr)
    a, ea, b, eb = R.norm_adj(R.f64(dy), R.f64(r), R.f64(rstd), R.f64(w), R.f64(dr))
    R.within(got, a, ea, rtype)
    if with_w:
        R.within(dw, b, eb, dtype)
    else:
        assert dw is None


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,d,pad", [(1, 1, 0), (1, 4096, 0), (3, 7, 1), (5, 64, 8), (310, 129, 0),
                                        (1000, 200, 0), (7, 2048, 0), (400, 1000, 5), (2, 8191, 0),
                                        (3, 16384, 0), (1, 40000, 0), (5000, 32, 0)])
def test_adjoint_sizes(dtype, rows, d, pad):
    check_adjoint(rows, d, dtype, dtype, pad=pad)
    if dtype != torch.float32:
        check_adjoint(rows, d, dtype, torch.float32, pad=pad)


@pytest.mark.parametrize("with_w,with_dr", [(False, True), (True, False), (False, False)])
@pytest.mark.parametrize("d", [512, 333])
def test_adjoint_without_weight_or_residual_gradient(with_w, with_dr, d):
    check_adjoint(9, d, torch.bfloat16, torch.float32, with_w, with_dr)


def test_gradient_agrees_with_differences():
    """Along random directions, the kernel's gradients of a float32 input
    against central differences of the float64 norm: the difference quotient
    with h = 1e-5 is exact to 1e-9 relative, the gradient to some hundreds of U32."""
    from differentiable_cholesky_gb300 import learn
    x, w, res = draw((5, 257), torch.float32, 30), draw((257,), torch.float32, 31), \
        draw((5, 257), torch.float32, 32)
    dy, dr = draw((5, 257), torch.float32, 33), draw((5, 257), torch.float32, 34)
    for t in (x, w, res):
        t.requires_grad_(True)
    y, r = learn.rms_norm(x, w, res, EPS)
    (y * dy + r * dr).sum().backward()
    rng = np.random.default_rng(35)

    def loss(x, w, res):
        r, _, y = R.norm(x, w, res, EPS)
        return (y * R.f64(dy) + r * R.f64(dr)).sum()

    at = [R.f64(x), R.f64(w), R.f64(res)]
    for k, t in enumerate((x, w, res)):
        step = rng.standard_normal(at[k].shape) * 1e-5
        up, down = list(at), list(at)
        up[k], down[k] = at[k] + step, at[k] - step
        diff = (loss(*up) - loss(*down)) / 2
        got = (R.f64(t.grad) * step).sum()
        size = (np.abs(R.f64(t.grad)) * np.abs(step)).sum()
        assert abs(got - diff) <= 600 * R.U32 * size + 1e-8 * abs(diff)
    assert torch.equal(x.grad, res.grad)


def test_autograd_with_mixed_types_and_without_residual():
    from differentiable_cholesky_gb300 import learn
    x = draw((4, 96), torch.bfloat16, 40).requires_grad_(True)
    res = draw((4, 96), torch.float32, 41).requires_grad_(True)
    y, r = learn.rms_norm(x, None, res)
    (y.float() + r).sum().backward()
    assert x.grad.dtype == torch.bfloat16 and res.grad.dtype == torch.float32
    assert torch.equal(x.grad, res.grad.to(torch.bfloat16))
    x2 = x.detach().clone().requires_grad_(True)
    y = learn.rms_norm(x2)
    assert isinstance(y, torch.Tensor)
    y.float().sum().backward()
    assert torch.isfinite(x2.grad).all()


def test_autograd_with_one_output_used():
    from differentiable_cholesky_gb300 import learn
    x = draw((4, 96), torch.float32, 42).requires_grad_(True)
    w = draw((96,), torch.float32, 43).requires_grad_(True)
    res = draw((4, 96), torch.float32, 44).requires_grad_(True)
    _, r = learn.rms_norm(x, w, res)
    (r * 2).sum().backward()
    assert torch.equal(x.grad, torch.full_like(x, 2)) and torch.equal(res.grad, x.grad) and w.grad is None
    y, _ = learn.rms_norm(x, w, res)
    y.sum().backward()
    assert w.grad is not None
    with pytest.raises(RuntimeError):  # no second derivative
        y, _ = learn.rms_norm(x, w, res)
        g, = torch.autograd.grad(y.square().sum(), x, create_graph=True)
        g.sum().backward()


def test_same_bits_each_time_and_in_place_residual():
    from differentiable_cholesky_gb300 import binding, learn
    x, w = draw((1500, 1024), torch.bfloat16, 50), draw((1024,), torch.bfloat16, 51)
    res, dy = draw((1500, 1024), torch.float32, 52), draw((1500, 1024), torch.bfloat16, 53)
    y, r, rstd = learn.rms_norm_fwd(x, w, res)
    a, dw = learn.rms_norm_adj(dy, r, rstd, w, adj_r=res)
    for _ in range(3):
        y2, r2, s2 = learn.rms_norm_fwd(x, w, res)
        a2, dw2 = learn.rms_norm_adj(dy, r, rstd, w, adj_r=res)
        for p, q in ((y, y2), (r, r2), (rstd, s2), (a, a2), (dw, dw2)):
            assert torch.equal(p, q)
    # r over res, and the gradient over adj_r, through the C entry points
    lib, s = learn._library(), torch.cuda.current_stream().cuda_stream
    buf, out = res.clone(), torch.empty_like(x)
    assert lib.chol_rms_norm(1500, 1024, 5, 0, 5, 0, 1e-6, x.data_ptr(), 1024, buf.data_ptr(), 1024,
                             w.data_ptr(), out.data_ptr(), None, buf.data_ptr(), None, s) == 0
    assert torch.equal(buf, r) and torch.equal(out, y)
    grad, gx, gw = res.clone(), torch.empty_like(x), torch.empty_like(w)
    assert lib.chol_rms_norm_adj(1500, 1024, 5, 0, dy.data_ptr(), 1024, r.data_ptr(), 1024,
                                 w.data_ptr(), rstd.data_ptr(), grad.data_ptr(), grad.data_ptr(),
                                 gx.data_ptr(), gw.data_ptr(), None, 0, s) == 0
    assert torch.equal(grad, a) and torch.equal(gw, dw)
    assert torch.equal(gx, a.to(torch.bfloat16))
    assert binding.load_library() is lib


def test_empty_rows():
    from differentiable_cholesky_gb300 import learn
    x, w = torch.empty((0, 64), device="cuda"), torch.ones(64, device="cuda")
    y, r, rstd = learn.rms_norm_fwd(x, w, None)
    assert y.shape == (0, 64) and rstd.shape == (0,)
    a, dw = learn.rms_norm_adj(y, x, rstd, w)
    assert a.shape == (0, 64) and not dw.any()


def test_element_offsets_beyond_32_bits():
    """Rows so far apart that their offsets pass 2^31 elements."""
    from differentiable_cholesky_gb300 import learn
    ld = (1 << 30) + 8
    flat = torch.zeros(2 * ld + 512, dtype=torch.bfloat16, device="cuda")
    x = flat.as_strided((3, 512), (ld, 1))
    x.copy_(draw((3, 512), torch.bfloat16, 60))
    y, _, rstd = learn.rms_norm_fwd(x)
    y2, _, rstd2 = learn.rms_norm_fwd(x.contiguous())
    assert torch.equal(y, y2) and torch.equal(rstd, rstd2)
    a, _ = learn.rms_norm_adj(x, x, rstd)
    a2, _ = learn.rms_norm_adj(x.contiguous(), x.contiguous(), rstd)
    assert torch.equal(a, a2)


def test_another_stream():
    from differentiable_cholesky_gb300 import learn
    x, w = draw((64, 512), torch.bfloat16, 70), draw((512,), torch.bfloat16, 71)
    want = learn.rms_norm_fwd(x, w)[0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y, r, rstd = learn.rms_norm_fwd(x, w, stream=side)
    a, dw = learn.rms_norm_adj(y, r, rstd, w, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, want)
    a2, dw2 = learn.rms_norm_adj(want, x, rstd, w)
    assert torch.equal(a, a2) and torch.equal(dw, dw2)
