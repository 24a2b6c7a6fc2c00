"""Refusals of the operators for learning with the factor that need no GPU
(CPU), and of their Python entry points."""
import ctypes

import numpy as np
import pytest
import torch

from differentiable_cholesky_gb300 import learn

OK, EINVAL, EDTYPE = 0, -1, -2
F32, F64, F16, BF16, E4M3, I8 = 0, 1, 4, 5, 6, 7


@pytest.fixture(scope="module")
def lib():
    return learn._library()


def host():
    """An address in host memory, aligned to 16 bytes."""
    buf = (ctypes.c_double * 64)()
    return buf, (ctypes.addressof(buf) + 15) // 16 * 16


def test_version_and_package_names(lib):
    import differentiable_cholesky_gb300 as pkg
    assert lib.chol_learn_version() == 1 << 16
    assert pkg.AdamW is learn.AdamW and pkg.rms_norm is learn.rms_norm and pkg.linrec is learn.linrec


def test_rms_norm_arguments(lib):
    keep, p = host()

    def call(rows=2, d=4, dtype=F32, rtype=F32, ytype=F32, group=0, eps=1e-6, x=p, ldx=4, res=None,
             ldr=4, w=None, y=p, scale=None, r=None, rstd=None):
        return lib.chol_rms_norm(rows, d, dtype, rtype, ytype, group, eps, x, ldx, res, ldr, w, y,
                                 scale, r, rstd, None)

    assert call(dtype=F64) == EDTYPE and call(dtype=9) == EDTYPE
    assert call(rtype=BF16) == EDTYPE and call(dtype=F16, rtype=BF16, ytype=F16) == EDTYPE
    assert call(ytype=BF16) == EDTYPE
    assert call(rows=-1) == EINVAL and call(d=0) == EINVAL and call(d=-4) == EINVAL
    assert call(ldx=3) == EINVAL and call(res=p, ldr=3) == EINVAL and call(ldx=-4) == EINVAL
    for eps in (-1e-6, float("nan"), float("inf")):
        assert call(eps=eps) == EINVAL
    assert call(group=128) == EINVAL                      # groups go with 8-bit output
    assert call(ytype=E4M3, group=64, scale=p) == EINVAL
    assert call(ytype=E4M3) == EINVAL                     # needs scales
    assert call(scale=p) == EINVAL                        # has none
    assert call(x=None) == EINVAL and call(y=None) == EINVAL
    assert call(x=p + 2) == EINVAL and call(y=p + 2) == EINVAL and call(rstd=p + 1) == EINVAL
    assert call() == EINVAL                               # host memory
    assert call(rows=1 << 40, d=1 << 20, ldx=1 << 20) == EINVAL
    assert call(rows=0, x=None, y=None) == OK


def test_rms_norm_adj_arguments(lib):
    keep, p = host()

    def call(rows=2, d=4, dtype=F32, rtype=F32, dy=p, ldy=4, r=p, ldr=4, w=None, rstd=p, dr=None,
             out=p, dx=None, dw=None, work=None, size=0):
        return lib.chol_rms_norm_adj(rows, d, dtype, rtype, dy, ldy, r, ldr, w, rstd, dr, out, dx,
                                     dw, work, size, None)

    assert call(dtype=F64) == EDTYPE and call(rtype=F16) == EDTYPE
    assert call(rows=-1) == EINVAL and call(d=0) == EINVAL
    assert call(ldy=3) == EINVAL and call(ldr=0) == EINVAL
    assert call(dy=None) == EINVAL and call(r=None) == EINVAL and call(rstd=None) == EINVAL
    assert call() == EINVAL                               # host memory
    assert call(rows=0, dy=None, r=None, rstd=None, out=None) == OK
    assert lib.chol_rms_norm_adj_workspace(-1, 4) == EINVAL
    assert lib.chol_rms_norm_adj_workspace(1, 0) == EINVAL


def test_linrec_arguments(lib):
    keep, p = host()

    def call(batch=1, time=2, d=4, dtype=F32, gate=2, comp=1, g=p, gbs=8, gts=4, x=p, xbs=8, xts=4,
             s0=None, off=None, n=0, h=p, s1=None):
        return lib.chol_linrec(batch, time, d, dtype, gate, comp, g, gbs, gts, x, xbs, xts, s0, off,
                               n, h, s1, None)

    assert call(dtype=F64) == EDTYPE and call(dtype=E4M3) == EDTYPE
    assert call(batch=-1) == EINVAL and call(time=-1) == EINVAL and call(d=0) == EINVAL
    assert call(gate=3) == EINVAL and call(gate=-1) == EINVAL and call(comp=2) == EINVAL
    assert call(gts=3) == EINVAL and call(xts=0) == EINVAL and call(gbs=-1) == EINVAL
    assert call(off=p, n=0) == EINVAL                     # steps without a sequence
    assert call(batch=2, off=p, n=2) == EINVAL            # packed rows are one row
    assert call(batch=1 << 40, time=1 << 30) == EINVAL
    assert call() == EINVAL                               # host memory
    assert call(g=None) == EINVAL
    assert call(batch=0, g=None, x=None, h=None) == OK
    assert call(off=p, n=1 << 31) == EINVAL


def test_linrec_adj_arguments(lib):
    keep, p = host()

    def call(batch=1, time=2, d=4, dtype=F32, gate=2, comp=1, x=p, xts=4, dts=4, h=p, dh=p, dg=p, dx=p):
        return lib.chol_linrec_adj(batch, time, d, dtype, gate, comp, p, 8, 4, x, 8, xts, None, None,
                                   0, h, dh, 8, dts, None, dg, dx, None, None)

    assert call(dtype=I8) == EDTYPE and call(gate=5) == EINVAL and call(comp=-1) == EINVAL
    assert call(xts=2) == EINVAL and call(dts=2) == EINVAL
    assert call(x=None) == EINVAL and call(h=None) == EINVAL and call(dh=None) == EINVAL
    assert call(dg=None) == EINVAL and call(dx=None) == EINVAL
    assert call(batch=0) == OK


def test_adamw_arguments(lib):
    keep, p = host()

    def call(count=1, dtype=F32, gtype=F32, bits=32, lr=1e-3, b1=0.9, b2=0.999, eps=1e-8, step=1,
             tensors=True, **fields):
        t = np.zeros(1, learn._ENTRY)
        t["numel"] = 4
        for k in ("param", "grad", "m", "v"):
            t[k] = p
        for k, v in fields.items():
            t[k] = v
        return lib.chol_adamw(count, t.ctypes.data if tensors else None, dtype, gtype, bits, lr, b1,
                              b2, eps, step, None, None, None)

    for dtype, gtype in ((F16, BF16), (BF16, F32), (F64, F32), (F32, F64), (E4M3, E4M3), (9, 9)):
        assert call(dtype=dtype, gtype=gtype) == EDTYPE
    assert call(bits=16) == EINVAL and call(step=0) == EINVAL and call(count=-1) == EINVAL
    for bad in (-0.1, 1.0, float("nan")):
        assert call(b1=bad) == EINVAL and call(b2=bad) == EINVAL
    assert call(eps=-1.0) == EINVAL and call(eps=float("nan")) == EINVAL
    assert call(lr=float("inf")) == EINVAL and call(weight_decay=float("nan")) == EINVAL
    assert call(tensors=False) == EINVAL and call(numel=-1) == EINVAL
    assert call(param=0) == EINVAL and call(grad=p + 2) == EINVAL
    assert call() == EINVAL                               # host memory
    assert call(count=0, tensors=False) == OK
    assert call(numel=0, param=0, grad=0, m=0, v=0) == OK
    assert learn._ENTRY.itemsize == 72


def test_python_entries_refuse_host_tensors():
    x = torch.ones(4, 8)
    for call in (lambda: learn.rms_norm_fwd(x), lambda: learn.rms_norm_quant(x),
                 lambda: learn.rms_norm_adj(x, x, torch.ones(4)), lambda: learn.linrec_fwd(x, x),
                 lambda: learn.linrec_step(x, x, x), lambda: learn.linrec_adj(x, x, x, x),
                 lambda: learn.AdamW([x])):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ValueError):
        learn.rms_norm_quant(x, kind="int4")
    with pytest.raises(ValueError):
        learn.rms_norm_quant(x, group=64)
    with pytest.raises(ValueError):
        learn.linrec_fwd(x, x, kind="tanh")
    with pytest.raises(ValueError):
        learn.AdamW([], state_bits=16)


@pytest.mark.gpu
def test_python_entries_refuse_shapes_types_and_strides():
    dev = torch.device("cuda")
    x = torch.ones((4, 8), device=dev)
    half = x.to(torch.float16)
    bad = [
        lambda: learn.rms_norm_fwd(x.double()),
        lambda: learn.rms_norm_fwd(x.t()),
        lambda: learn.rms_norm_fwd(x, torch.ones(7, device=dev)),
        lambda: learn.rms_norm_fwd(x, half[0]),
        lambda: learn.rms_norm_fwd(half, None, x.to(torch.bfloat16)),
        lambda: learn.rms_norm_fwd(x, None, half),
        lambda: learn.rms_norm_fwd(x, None, x[:2]),
        lambda: learn.rms_norm_fwd(x[:, :0]),
        lambda: learn.rms_norm_adj(x, half, torch.ones(4, device=dev)),
        lambda: learn.rms_norm_adj(x, x, torch.ones(3, device=dev)),
        lambda: learn.rms_norm_adj(x, x, torch.ones(4, device=dev), adj_r=half),
        lambda: learn.rms_norm_adj(x, x, torch.ones(4, device=dev), adj_r=x.t().contiguous().t()),
        lambda: learn.linrec_fwd(half, x),
        lambda: learn.linrec_fwd(x[:3], x),
        lambda: learn.linrec_fwd(x.t(), x.t()),
        lambda: learn.linrec_fwd(x, x, torch.ones(8, device=dev)),
        lambda: learn.linrec_fwd(x, x, half[:1]),
        lambda: learn.linrec_fwd(x, x, None, torch.tensor([0, 4])),
        lambda: learn.linrec_fwd(x, x, None, torch.tensor([0, 4], device=dev, dtype=torch.int32)),
        lambda: learn.linrec_fwd(x[None], x[None], None, torch.tensor([0, 4], device=dev)),
        lambda: learn.linrec_fwd(x, x, torch.ones((2, 8), device=dev), torch.tensor([0, 4], device=dev)),
        lambda: learn.linrec_step(x, x, half),
        lambda: learn.linrec_step(x, x, x[:, ::2]),
        lambda: learn.linrec_step(x[0], x[0], x),
        lambda: learn.linrec_step(x, x, None),
        lambda: learn.linrec_adj(x, x, x.t().contiguous().t(), x),
        lambda: learn.linrec_adj(x, x, x, half),
        lambda: learn.linrec_adj(x, x, x, x, None, half[:1]),
        lambda: learn.AdamW([x.t()]),
        lambda: learn.AdamW([x.to(torch.int32)]),
        lambda: learn.AdamW([x], copies=[x.clone()]),
        lambda: learn.AdamW([x], weight_decay=[0.1, 0.2]),
        lambda: learn.AdamW([x], state={"step": 0, "m": [x], "v": [half]}),
        lambda: learn.AdamW([x.clone()]).step([half.double()]),
        lambda: learn.AdamW([x.clone()]).step([x[:2]]),
        lambda: learn.AdamW([half.clone()]).step([x]),
        lambda: learn.AdamW([x.clone()]).step([x, x]),
        lambda: learn.AdamW([x.clone()]).step([x], grad_scale=torch.ones(2, device=dev)),
        lambda: learn.AdamW([x.clone()]).step([x], status=torch.ones((), device=dev)),
        lambda: learn.AdamW([x.clone()], copies=[half.clone()]).step([x]),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was not refused")


@pytest.mark.gpu
def test_overlapping_outputs_are_refused():
    from differentiable_cholesky_gb300.binding import CholError
    lib = learn._library()
    buf = torch.zeros(4096, device="cuda")
    p = buf.data_ptr()
    assert lib.chol_rms_norm(4, 64, 0, 0, 0, 0, 1e-6, p, 64, None, 0, None, p, None, None, None, None) == -3
    assert lib.chol_rms_norm(4, 64, 0, 0, 0, 0, 1e-6, p, 64, None, 0, None, p + 8192, None,
                             p + 8192 + 512, None, None) == -3
    assert lib.chol_linrec(1, 4, 64, 0, 2, 1, p, 256, 64, p + 1024, 256, 64, None, None, 0, p + 512,
                           None, None) == -3
    # final states over initial ones: a single step only
    assert lib.chol_linrec(1, 2, 64, 0, 2, 1, p, 128, 64, p + 1024, 128, 64, p + 4096, None, 0,
                           p + 8192, p + 4096, None) == -3
    w = buf[:100]
    with pytest.raises(CholError):
        learn.AdamW([w, buf[50:150]]).step([buf[1000:1100], buf[2000:2100]])
    with pytest.raises(CholError):
        learn.AdamW([w]).step([w])
    with pytest.raises(CholError):
        learn.AdamW([buf[:100]], betas=(1.5, 0.9)).step([buf[200:300]])
