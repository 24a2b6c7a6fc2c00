"""The native marshalling of the operators for learning with the factor gives
what the Python one gives, and leaves to it what it does not take (GPU)."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def draw(shape, dtype, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=gen, device="cuda").to(dtype)


def calls(learn):
    """Every operator on usual and unusual arguments; the results as a list."""
    out = []
    for dtype in (torch.float32, torch.float16, torch.bfloat16):
        wide = draw((12, 300), dtype, 1)
        w, res = draw((256,), dtype, 2), draw((12, 256), torch.float32, 3)
        for x, r in ((wide[:, :256], res), (wide[:, 44:].contiguous(), None),
                     (wide[:, :256].reshape(3, 4, 256), res.view(3, 4, 256)),
                     (wide[0, :256], None), (wide[:, :256], torch.cat([res, res], 1)[:, 256:])):
            y, rr, rstd = learn.rms_norm_fwd(x, w, r, eps=1e-5)
            out += [y, rr, rstd]
            for kind in ("e4m3", "int8"):
                for group in (0, 128):
                    q, s, rq, sq = learn.rms_norm_quant(x, None, r, kind=kind, group=group)
                    out += [q.view(torch.uint8), s, rq, sq]
            out += [t for t in learn.rms_norm_adj(y, rr, rstd, w, adj_r=rr.contiguous()) if t is not None]
            out += [t for t in learn.rms_norm_adj(y, rr, rstd, w, want_weight=False) if t is not None]
        both = draw((3, 40, 96), dtype, 4)
        state = draw((3, 48), torch.float32, 5)
        off = torch.tensor([0, 13, 13, 40], device="cuda")
        for kind in ("linear", "log", "logit"):
            for g, x, s, o in ((both[..., :48] * 0.3, both[..., 48:], state, None),
                               (both[0, :, :48] * 0.3, both[0, :, 48:], state, off),
                               (both[0, :, :48] * 0.3, both[0, :, 48:], None, None)):
                h, last = learn.linrec_fwd(g, x, s, o, kind=kind, complement=kind != "linear")
                out += [h, last]
                out += list(learn.linrec_adj(g, x, h, x, s, last, o, kind=kind, complement=kind != "linear"))
            s = state.clone()
            out += [learn.linrec_step(both[:, 0, :48], both[:, 0, 48:], s, kind=kind), s]
    for ptype, gtype, bits, copied in ((torch.float32, torch.bfloat16, 32, True),
                                       (torch.bfloat16, torch.bfloat16, 8, False),
                                       (torch.float64, torch.float64, 32, False)):
        params = [draw((n,), ptype, 6 + n) for n in (5, 700)]
        grads = [draw((n,), gtype, 7 + n) for n in (5, 700)]
        copies = [torch.zeros(n, dtype=gtype, device="cuda") for n in (5, 700)] if copied else None
        opt = learn.AdamW(params, state_bits=bits, copies=copies)
        opt.step(grads)
        opt.step(grads, lr=0.5, grad_scale=torch.tensor(0.5, device="cuda"),
                 status=torch.zeros((), dtype=torch.int32, device="cuda"))
        opt.step([None, grads[1]])
        assert opt.steps == 3
        out += params + list(copies or ())
        out += [x.view(torch.uint8) if bits == 8 else x for x in opt.m + opt.v]
    return out


def test_both_ways_give_the_same_bits(monkeypatch):
    from differentiable_cholesky_gb300 import learn
    assert learn._load_native(), "the native marshalling is built with the library"
    native = calls(learn)
    monkeypatch.setattr(learn, "_native", False)
    python = calls(learn)
    assert len(native) == len(python)
    for a, b in zip(native, python):
        assert a.shape == b.shape and a.dtype == b.dtype and torch.equal(a, b)


def test_what_it_does_not_take_is_left_alone():
    from differentiable_cholesky_gb300 import learn
    m = learn._load_native()
    x, half = draw((4, 64), torch.float32, 9), draw((4, 64), torch.float16, 9)
    for call in (lambda: m.rms_norm(x.cpu(), None, None, 1e-6, 0, 0), lambda: m.rms_norm(x, 3, None, 1e-6, 0, 0),
                 lambda: m.rms_norm(x, half[0], None, 1e-6, 0, 0), lambda: m.rms_norm(x, None, None, -1.0, 0, 0),
                 lambda: m.rms_norm(x.double(), None, None, 1e-6, 0, 0), lambda: m.rms_norm(x[:0], None, None, 1e-6, 0, 0),
                 lambda: m.rms_norm(x), lambda: m.rms_norm_adj(x, half, x, None, None, True),
                 lambda: m.linrec(half, x, None, None, 2, True), lambda: m.linrec(x, x, None, None, -1, True),
                 lambda: m.linrec(x, x, x, None, 2, True), lambda: m.linrec_step(x, x, None, 2, True),
                 lambda: m.linrec_step(x, x, half, 2, True),
                 lambda: m.linrec_adj(x, x, x.t(), x, None, None, None, 2, True),
                 lambda: m.adamw([x], [half.double()], 1, -1, 32, 1e-3, 0.9, 0.9, 1e-8, 1, None, None),
                 lambda: m.adamw([x], [None], 1, -1, 32, 1e-3, 0.9, 0.9, 1e-8, 1, None, None)):
        assert call() is None
    with pytest.raises(TypeError):
        m.rms_norm(x, None, None, "a", 0, 0)
