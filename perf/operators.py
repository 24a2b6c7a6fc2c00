"""Cases that measure the operators for learning with the factor: the
root-mean-square norm with the residual's addition, the gated linear
recurrence and the AdamW step.

``run`` computes a case in its plain form (elementary torch operations in 32
bits, rounded once at the end) or, where ``own`` is true, through the calls of
``differentiable_cholesky_gb300.learn`` that a user makes.  ``exact`` gives the
same outputs from the definitions in 64 bits.

Operators (``op`` of a case):

``norm``   r = x + residual;  rstd = 1 / sqrt(mean(r^2) + eps);  y = r rstd w.
           ``mode`` "fwd" returns y and r; "quant" returns y in 8 bits with a
           scale for each ``group`` of columns (0: for each row), and r;
           "train" returns y, r and the gradients of r and w for given
           gradients of y and r.
``rec``    h_t = a_t h_{t-1} + b_t for every channel, a = exp(g) ("log") or
           1 / (1 + exp(-g)) ("logit"), b = x or (1 - a) x ("complement").
           ``mode`` "step" advances a state by one token, "fwd" runs whole
           sequences, "train" also returns the gradients of g, x and the
           initial states.  ``packed`` > 0: that many sequences of uneven
           lengths lie behind one another on one time axis.
``adamw``  one step over many tensors with first and second moments in 32
           bits, or in 8 bits (e4m3 values of m and of sqrt(v) with a scale
           for each 256 of them).
"""
import math

import numpy as np
import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "f64": torch.float64}
SIZES = {"f32": 4, "bf16": 2, "f16": 2, "f64": 8}
EPS = 1e-6
BLOCK = 256          # moments that share one scale
E4M3_MAX = 448.0
TINY = 2.0 ** -100   # the least scale: a block of zeros has it

# the optimiser's numbers, as training programs set them
LR, BETA1, BETA2, ADAM_EPS, DECAY, STEP = 3e-4, 0.9, 0.95, 1e-8, 0.1, 1000


def listed():
    return [
        # serving, one token of one sequence: the norm before a layer
        dict(name="norm_one_token", op="norm", mode="fwd", rows=1, d=4096, type="bf16", residual="bf16", group=0, pad=0),
        # a prompt or a training batch, the residual stream kept in 32 bits
        dict(name="norm_batch", op="norm", mode="fwd", rows=16384, d=4096, type="bf16", residual="f32", group=0, pad=0),
        # operands of an 8-bit product: odd row count, a last group of 8 columns, x a slice of wider rows
        dict(name="norm_e4m3_ragged", op="norm", mode="quant", rows=8191, d=5000, type="bf16", residual="bf16", group=128, pad=120),
        # a training step's norm, forward and backward, wide rows
        dict(name="norm_train", op="norm", mode="train", rows=8192, d=8192, type="bf16", residual="bf16", group=0, pad=0),
        # serving, one token for each of 64 sequences, gates and values from one projection
        dict(name="rec_one_token", op="rec", mode="step", batch=64, time=1, d=4096, type="bf16", kind="logit", complement=True, packed=0, fused=True),
        # a batch of prompts of the length that the worked example of this repository has
        dict(name="rec_prompts", op="rec", mode="fwd", batch=16, time=512, d=1024, type="bf16", kind="logit", complement=True, packed=0, fused=True),
        # one long document in training: few channels side by side, a long time axis
        dict(name="rec_train_long", op="rec", mode="train", batch=1, time=65536, d=2048, type="bf16", kind="log", complement=True, packed=0, fused=False),
        # documents of uneven lengths behind one another, 32-bit values, an odd number of channels
        dict(name="rec_train_packed", op="rec", mode="train", batch=1, time=20011, d=1001, type="f32", kind="log", complement=False, packed=37, fused=False),
        # a small model's parameters: launch latency
        dict(name="adamw_small", op="adamw", tensors=12, total=200000, type="f32", grad="f32", copy=False, bits=32),
        # mixed precision: 32-bit parameters, bf16 gradients, and a bf16 copy for the next forward pass
        dict(name="adamw_mixed", op="adamw", tensors=300, total=268435456, type="f32", grad="bf16", copy=True, bits=32),
        # moments in 8 bits, bf16 parameters
        dict(name="adamw_8bit", op="adamw", tensors=200, total=400000000, type="bf16", grad="bf16", copy=False, bits=8),
        # float64 matrices that are learned through their factors (256 of 512 x 512, and as many means)
        dict(name="adamw_f64_matrices", op="adamw", tensors=2, total=67239936, type="f64", grad="f64", copy=False, bits=32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "rec", "adamw"])
    if op == "norm":
        d = _log(rng, 64, 8192)
        d = d if rng.random() < 0.4 else max(64, d // 64 * 64)
        rows = _log(rng, 1, min(32768, 67108864 // d))
        mode = rng.choice(["fwd", "quant", "train"])
        kind = rng.choice(["bf16", "f16", "f32"])
        return dict(op="norm", mode=mode, rows=rows, d=d, type=kind, residual=rng.choice(["none", kind, "f32"]),
                    group=rng.choice([0, 128]) if mode == "quant" else 0, pad=rng.choice([0, 0, 8, 13]))
    if op == "rec":
        mode = rng.choice(["step", "fwd", "train"])
        d = _log(rng, 64, 4096)
        d = d if rng.random() < 0.4 else max(64, d // 64 * 64)
        kind = dict(type=rng.choice(["bf16", "f16", "f32"]), kind=rng.choice(["logit", "log"]), complement=rng.random() < 0.5)
        if mode == "step":
            return dict(op="rec", mode=mode, batch=_log(rng, 1, 512), time=1, d=d, packed=0, fused=rng.random() < 0.5, **kind)
        if rng.random() < 0.4:
            time = _log(rng, 64, min(65536, 67108864 // d))
            return dict(op="rec", mode=mode, batch=1, time=time, d=d, packed=_log(rng, 2, max(2, min(200, time // 8))), fused=False, **kind)
        batch = _log(rng, 1, 32)
        time = _log(rng, 2, min(65536, 67108864 // (d * batch)))
        return dict(op="rec", mode=mode, batch=batch, time=time, d=d, packed=0, fused=rng.random() < 0.5, **kind)
    kind, grad, copy = rng.choice([("f32", "f32", False), ("f32", "bf16", True), ("f32", "bf16", False), ("bf16", "bf16", False),
                                   ("f16", "f16", False), ("f32", "f16", True), ("f64", "f64", False)])
    total = _log(rng, 2000, 100000000 if kind == "f64" else 200000000)
    return dict(op="adamw", tensors=_log(rng, 1, min(400, total // 500)), total=total, type=kind, grad=grad, copy=copy, bits=rng.choice([32, 8]))


# ----------------------------------------------------------------------------
# Inputs
# ----------------------------------------------------------------------------
def _normal(gen, shape, kind, scale=1.0, mean=0.0):
    dtype = TYPES[kind]
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float64 if kind == "f64" else torch.float32)
    return x.mul_(scale).add_(mean).to(dtype)


def _tensor_sizes(case):
    """Element counts of the optimiser's tensors: matrices of uneven sizes
    with vectors between them, `total` elements in all."""
    r = np.random.RandomState(case["tensors"] * 7919 + case["total"] % 1000003)
    w = np.exp(r.uniform(0.0, math.log(300.0), case["tensors"]))
    sizes = np.maximum(1, (w / w.sum() * case["total"]).astype(np.int64))
    sizes[-1] = max(1, case["total"] - int(sizes[:-1].sum()))
    return [int(s) for s in sizes]


def _encode(x):
    """Blocks of 256 over their scales, and the scales: the largest is 448."""
    x = x.view(-1, BLOCK)
    scale = (x.abs().amax(1) * (1.0 / E4M3_MAX)).clamp(min=TINY)
    inverse = 1.0 / scale
    return x * inverse[:, None], scale


def _codes(x, kept):
    """x in e4m3; where `kept` (values above 0), not below the least e4m3 value."""
    x = x.clamp(-E4M3_MAX, E4M3_MAX)
    if kept is not None:
        x = torch.where(kept, x.clamp(min=2.0 ** -9), x)
    return x.to(torch.float8_e4m3fn)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    s = dict(case)
    if case["op"] == "norm":
        rows, d = case["rows"], case["d"]
        wide = _normal(gen, (rows, d + case["pad"]), case["type"])
        s["x"] = wide[:, :d]
        s["weight"] = _normal(gen, (d,), case["type"], 0.1, 1.0)
        s["res"] = None if case["residual"] == "none" else _normal(gen, (rows, d), case["residual"], 3.0)
        if case["mode"] == "train":
            s["dy"] = _normal(gen, (rows, d), case["type"])
            s["dr"] = _normal(gen, (rows, d), case["type"] if s["res"] is None else case["residual"])
    elif case["op"] == "rec":
        b, t, d = case["batch"], case["time"], case["d"]
        shape = (t, d) if case["packed"] else (b, d) if case["mode"] == "step" else (b, t, d)
        # one projection gives gates and values side by side, or each comes by itself
        if case["fused"]:
            both = _normal(gen, shape[:-1] + (2 * d,), case["type"])
            gate, x = both[..., :d], both[..., d:]
        else:
            gate, x = _normal(gen, shape, case["type"]), _normal(gen, shape, case["type"])
        # decays from a few tokens to some hundreds
        if case["kind"] == "logit":
            gate.mul_(1.5).add_(2.5)
        else:
            gate.copy_(-torch.nn.functional.softplus(gate.float() * 1.5 - 3.0))
        s["gate"], s["x"] = gate, x
        n = case["packed"] or b
        s["state"] = _normal(gen, (n, d), "f32")
        s["offsets"], s["longest"] = None, t
        if case["packed"]:
            # an empty document among them, and one of a single token
            r = np.random.RandomState(int(seed) % (1 << 31))
            cut = np.sort(r.randint(0, t + 1, n - 1))
            off = np.concatenate([[0], cut, [t]]).astype(np.int64)
            if n >= 4:
                off[2] = off[1]
                off[3] = min(off[2] + 1, off[4]) if n > 4 else off[3]
                off = np.maximum.accumulate(off)
                off[-1] = t
            s["offsets"], s["longest"] = torch.from_numpy(off).cuda(), int(np.diff(off).max())
        if case["mode"] == "train":
            s["dh"] = _normal(gen, shape, case["type"])
            s["dstate"] = _normal(gen, (n, d), "f32")
    else:
        sizes = _tensor_sizes(case)
        starts = np.concatenate([[0], np.cumsum([-(-n // BLOCK) * BLOCK for n in sizes])])
        total = int(starts[-1])
        real = torch.zeros(total, dtype=torch.bool, device="cuda")
        for at, n in zip(starts, sizes):
            real[int(at):int(at) + n] = True
        views = lambda flat: [flat[int(at):int(at) + n] for at, n in zip(starts, sizes)]  # noqa: E731
        # gradients of uneven size from place to place, moments of their order
        size = torch.exp(_normal(gen, (total // BLOCK,), "f32")).repeat_interleave(BLOCK) * 1e-3
        fill = lambda x: x.mul_(real)  # noqa: E731
        s["param"] = fill(_normal(gen, (total,), case["type"], 0.02))
        s["grad_flat"] = fill((_normal(gen, (total,), "f32") * size).to(TYPES[case["grad"]]))
        m = fill(_normal(gen, (total,), "f32", 0.3) * size)
        v = fill((0.25 + torch.rand(total, generator=gen, device="cuda")) * size.square_())
        del size
        s["clip"] = torch.rand((), generator=gen, device="cuda") * 0.5 + 0.5
        s["step"] = STEP - 1
        s["m_scale"] = s["v_scale"] = None
        if case["bits"] == 8:
            m, s["m_scale"] = _encode(m)
            m = _codes(m, None).view(-1)
            kept = (v > 0).view(-1, BLOCK)
            v, s["v_scale"] = _encode(v.sqrt_())
            v = _codes(v, kept).view(-1)
        s["m"], s["v"] = m, v
        s["copy_flat"] = torch.zeros(total, dtype=TYPES[case["grad"]], device="cuda") if case["copy"] else None
        if own:
            from differentiable_cholesky_gb300 import learn
            blocks = lambda flat: [flat[int(at) // BLOCK:int(at) // BLOCK - (-n // BLOCK)] for at, n in zip(starts, sizes)]  # noqa: E731
            state = dict(step=s["step"], m=views(s["m"]), v=views(s["v"]))
            if case["bits"] == 8:
                state.update(m_scale=blocks(s["m_scale"]), v_scale=blocks(s["v_scale"]))
            s["grads"] = views(s["grad_flat"])
            s["optimiser"] = learn.AdamW(views(s["param"]), lr=LR, betas=(BETA1, BETA2), eps=ADAM_EPS, weight_decay=DECAY, state_bits=case["bits"],
                                         copies=views(s["copy_flat"]) if case["copy"] else None, state=state)
    return s


# ----------------------------------------------------------------------------
# Plain forms
# ----------------------------------------------------------------------------
def _plain_norm(s):
    x = s["x"].float()
    r = x if s["res"] is None else x + s["res"].float()
    w = s["weight"].float()
    rstd = torch.rsqrt((r * r).mean(1, keepdim=True) + EPS)
    n = r * rstd
    y = n * w
    kind = TYPES[s["type"]]
    kept = None if s["res"] is None else r.to(s["res"].dtype)
    if s["mode"] == "fwd":
        return {"y": y.to(kind), "r": kept}
    if s["mode"] == "quant":
        rows, d = y.shape
        width = s["group"] or d
        groups = -(-d // width)
        full = torch.nn.functional.pad(y, (0, groups * width - d)).view(rows, groups, width)
        scale = full.abs().amax(2) * (1.0 / E4M3_MAX)
        inverse = torch.where(scale > 0, 1.0 / scale, 0.0)
        q = (full * inverse[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).view(rows, groups * width)[:, :d]
        return {"q": q.to(torch.float8_e4m3fn), "scale": scale, "r": kept}
    dy = s["dy"].float()
    u = dy * w
    dr = rstd * (u - n * (u * n).mean(1, keepdim=True)) + s["dr"].float()
    return {"y": y.to(kind), "r": kept, "dr": dr.to(s["dr"].dtype), "dw": (dy * n).sum(0).to(kind)}


def _scan(a, b, longest):
    """h_t = a_t h_{t-1} + b_t along the first axis, by doubling."""
    n = 1
    while n < longest:
        b = torch.cat([b[:n], b[n:] + a[n:] * b[:-n]])
        a = torch.cat([a[:n], a[n:] * a[:-n]])
        n *= 2
    return b


def _gates(s, g):
    if s["kind"] == "log":
        return torch.exp(g), -torch.expm1(g)
    return torch.sigmoid(g), torch.sigmoid(-g)


def _plain_rec(s):
    d, kind = s["d"], TYPES[s["type"]]
    if s["mode"] == "step":
        a, c = _gates(s, s["gate"].float())
        h = a * s["state"] + (c * s["x"].float() if s["complement"] else s["x"].float())
        s["state"].copy_(h)
        return {"h": h.to(kind), "state": s["state"]}
    shape = s["x"].shape
    g, x = s["gate"].float().reshape(-1, d), s["x"].float().reshape(-1, d)
    n, device = g.shape[0], g.device
    off = s["offsets"] if s["offsets"] is not None else torch.arange(s["batch"] + 1, device=device) * s["time"]
    at = torch.arange(n, device=device)
    seq = torch.searchsorted(off[1:].contiguous(), at, right=True)  # the sequence of each token
    first, last = (at == off[seq])[:, None], (at == off[seq + 1] - 1)[:, None]
    some = (off[1:] > off[:-1])[:, None]
    a, c = _gates(s, g)
    b = c * x if s["complement"] else x
    h = _scan(torch.where(first, 0.0, a), torch.where(first, a * s["state"][seq] + b, b), s["longest"])
    state = torch.where(some, h[(off[1:] - 1).clamp(min=0)], s["state"])
    out = {"h": h.to(kind).view(shape), "state": state}
    if s["mode"] == "fwd":
        return out
    dh = s["dh"].float().reshape(-1, d)
    # carry_t = a_t lambda_t, lambda_t = dh_t + carry_{t+1} (the final state's gradient where t is a last token)
    dh = torch.where(last, dh + s["dstate"][seq], dh)
    back = lambda v: v.flip(0)  # noqa: E731
    carry = back(_scan(back(torch.where(last, 0.0, a)), back(a * dh), s["longest"]))
    lam = torch.where(last, dh, dh + torch.cat([carry[1:], carry[:1]]))
    before = torch.where(first, s["state"][seq], torch.cat([h[:1], h[:-1]]))
    da = lam * (before - x) if s["complement"] else lam * before
    dg = da * a if s["kind"] == "log" else da * a * c
    dx = lam * c if s["complement"] else lam
    d0 = torch.where(some, carry[off[:-1].clamp(max=n - 1)], s["dstate"])
    return {**out, "dgate": dg.to(kind).view(shape), "dx": dx.to(kind).view(shape), "dstate": d0}


def _plain_adamw(s):
    s["step"] += 1
    g = s["grad_flat"].float() * s["clip"]
    if s["bits"] == 8:
        m = (s["m"].float().view(-1, BLOCK) * s["m_scale"][:, None]).view(-1)
        v = (s["v"].float().view(-1, BLOCK) * s["v_scale"][:, None]).view(-1).square()
    else:
        m, v = s["m"], s["v"]
    m = m * BETA1 + g * (1.0 - BETA1)
    v = v * BETA2 + (g * g) * (1.0 - BETA2)
    root = v.sqrt()
    step = m / (root * (1.0 / math.sqrt(1.0 - BETA2 ** s["step"])) + ADAM_EPS)
    kind = s["param"].dtype
    wide = s["param"] if kind == torch.float64 else s["param"].float()
    new = wide * (1.0 - LR * DECAY) - (step * (LR / (1.0 - BETA1 ** s["step"]))).to(wide.dtype)
    s["param"].copy_(new)
    if s["copy"]:
        s["copy_flat"].copy_(new)
    if s["bits"] == 8:
        kept = (root > 0).view(-1, BLOCK)
        m, scale = _encode(m)
        s["m_scale"].copy_(scale)
        s["m"].copy_(_codes(m, None).view(-1))
        root, scale = _encode(root)
        s["v_scale"].copy_(scale)
        s["v"].copy_(_codes(root, kept).view(-1))
    else:
        s["m"].copy_(m)
        s["v"].copy_(v)


def _adamw_outputs(s):
    return {"param": s["param"], "copy": s["copy_flat"], "m": s["m"], "v": s["v"], "m_scale": s["m_scale"], "v_scale": s["v_scale"]}


def run(s):
    if not own:
        if s["op"] == "norm":
            return _plain_norm(s)
        if s["op"] == "rec":
            return _plain_rec(s)
        _plain_adamw(s)
        return _adamw_outputs(s)
    from differentiable_cholesky_gb300 import learn
    if s["op"] == "norm":
        if s["mode"] == "quant":
            q, scale, r, _ = learn.rms_norm_quant(s["x"], s["weight"], s["res"], eps=EPS, kind="e4m3", group=s["group"])
            return {"q": q, "scale": scale, "r": r}
        y, r, rstd = learn.rms_norm_fwd(s["x"], s["weight"], s["res"], eps=EPS)
        kept = None if s["res"] is None else r
        if s["mode"] == "fwd":
            return {"y": y, "r": kept}
        dr, dw = learn.rms_norm_adj(s["dy"], r, rstd, s["weight"], adj_r=s["dr"])
        return {"y": y, "r": kept, "dr": dr, "dw": dw}
    if s["op"] == "rec":
        how = dict(kind=s["kind"], complement=s["complement"])
        if s["mode"] == "step":
            h = learn.linrec_step(s["gate"], s["x"], s["state"], **how)
            return {"h": h, "state": s["state"]}
        h, state = learn.linrec_fwd(s["gate"], s["x"], s["state"], offsets=s["offsets"], **how)
        if s["mode"] == "fwd":
            return {"h": h, "state": state}
        dg, dx, d0 = learn.linrec_adj(s["gate"], s["x"], h, s["dh"], s["state"], adj_state=s["dstate"], offsets=s["offsets"], **how)
        return {"h": h, "state": state, "dgate": dg, "dx": dx, "dstate": d0}
    s["optimiser"].step(s["grads"], grad_scale=s["clip"])
    return _adamw_outputs(s)


# ----------------------------------------------------------------------------
# What a pass cannot do without
# ----------------------------------------------------------------------------
def work(case):
    if case["op"] == "norm":
        e, n = SIZES[case["type"]], case["rows"] * case["d"]
        res = SIZES[case["residual"]] if case["residual"] != "none" else 0
        bytes_ = n * (e + 2 * res) + case["d"] * e
        if case["mode"] == "quant":
            groups = -(-case["d"] // case["group"]) if case["group"] else 1
            return {"bytes": bytes_ + n + 4 * case["rows"] * groups, "flops": 8 * n}
        if case["mode"] == "fwd":
            return {"bytes": bytes_ + n * e, "flops": 5 * n}
        return {"bytes": bytes_ + n * (2 * e + 2 * (res or e)) + case["d"] * e, "flops": 16 * n}
    if case["op"] == "rec":
        e, n = SIZES[case["type"]], case["batch"] * case["time"] * case["d"]
        states = 4 * case["d"] * (case["packed"] or case["batch"])
        if case["mode"] != "train":
            return {"bytes": 3 * e * n + 2 * states, "flops": 8 * n}
        return {"bytes": 6 * e * n + 4 * states, "flops": 22 * n}
    n = case["total"]
    moments = 16 if case["bits"] == 32 else 4 + 16 / BLOCK
    return {"bytes": n * (2 * SIZES[case["type"]] + SIZES[case["grad"]] + (SIZES[case["grad"]] if case["copy"] else 0) + moments), "flops": 16 * n}


# ----------------------------------------------------------------------------
# The definitions in 64 bits
# ----------------------------------------------------------------------------
def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "norm":
        return _exact_norm(case, s)
    return _exact_rec(case, s) if case["op"] == "rec" else _exact_adamw(case, s)


def _exact_norm(case, s):
    r = s["x"].double()
    if s["res"] is not None:
        r = r + s["res"].double()
    w, d = s["weight"].double(), case["d"]
    size = torch.sqrt(torch.einsum("ij,ij->i", r, r) / d + EPS)[:, None]
    y = r / size * w
    out = {"r": None if s["res"] is None else r}
    if case["mode"] == "quant":
        width = case["group"] or d
        parts = [y[:, i:i + width] for i in range(0, d, width)]
        tops = [p.abs().max(1, keepdim=True).values for p in parts]
        return {**out, "q": torch.cat([p / t * E4M3_MAX for p, t in zip(parts, tops)], 1), "scale": torch.cat(tops, 1) / E4M3_MAX}
    out["y"] = y
    if case["mode"] == "train":
        # y_j = r_j w_j / size, d size / d r_k = r_k / (d size)
        dy = s["dy"].double()
        along = torch.einsum("ij,ij,j->i", dy, r, w)[:, None]
        out["dr"] = dy * w / size - r * along / (d * size ** 3) + s["dr"].double()
        out["dw"] = torch.einsum("ij,ij->j", dy, r / size)
    return out


def _exact_rows(a, b, state, dh, dstate):
    """Rows [n, t, d] token after token: h, the final states, and the
    gradients of a, b and the initial states (None without dh)."""
    h, cur = torch.empty_like(b), state
    for k in range(b.shape[1]):
        cur = a[:, k] * cur + b[:, k]
        h[:, k] = cur
    if dh is None:
        return h, cur, None, None, None
    da, db, carry = torch.empty_like(b), torch.empty_like(b), dstate
    for k in reversed(range(b.shape[1])):
        lam = dh[:, k] + carry
        db[:, k] = lam
        da[:, k] = lam * (h[:, k - 1] if k else state)
        carry = a[:, k] * lam
    return h, cur, da, db, carry


def _exact_rec(case, s):
    d, shape = case["d"], s["x"].shape
    train = case["mode"] == "train"
    rows = (1, -1, d) if case["packed"] else (case["batch"], -1, d)
    g, x = s["gate"].double().reshape(rows), s["x"].double().reshape(rows)
    a = g.exp() if case["kind"] == "log" else 1.0 / (1.0 + (-g).exp())
    c = -torch.expm1(g) if case["kind"] == "log" else 1.0 / (1.0 + g.exp())
    b = c * x if case["complement"] else x
    dh = s["dh"].double().reshape(rows) if train else None
    state, dstate = s["state"].double(), s["dstate"].double() if train else None
    if not case["packed"]:
        h, last, da, db, d0 = _exact_rows(a, b, state, dh, dstate)
    else:
        off = s["offsets"].tolist()
        got = [_exact_rows(a[:, lo:hi], b[:, lo:hi], state[i:i + 1], dh[:, lo:hi] if train else None, dstate[i:i + 1] if train else None)
               for i, (lo, hi) in enumerate(zip(off, off[1:]))]
        h, last = torch.cat([q[0] for q in got], 1), torch.cat([q[1] for q in got])
        if train:
            da, db, d0 = torch.cat([q[2] for q in got], 1), torch.cat([q[3] for q in got], 1), torch.cat([q[4] for q in got])
    out = {"h": h.view(shape), "state": last}
    if not train:
        return out
    if case["complement"]:
        da = da - db * x
        db = db * c
    dg = da * a if case["kind"] == "log" else da * a * (1.0 - a)
    return {**out, "dgate": dg.view(shape), "dx": db.view(shape), "dstate": d0}


def _exact_adamw(case, s):
    g = s["grad_flat"].double() * s["clip"].double()
    m, v = s["m"].double(), s["v"].double()
    if case["bits"] == 8:
        m = m * s["m_scale"].double().repeat_interleave(BLOCK)
        v = (v * s["v_scale"].double().repeat_interleave(BLOCK)) ** 2
    m = m + (1.0 - BETA1) * (g - m)
    v = v + (1.0 - BETA2) * (g * g - v)
    del g
    first, second = m / (1.0 - BETA1 ** STEP), v / (1.0 - BETA2 ** STEP)
    p = s["param"].double()
    p = p - LR * (first / (second ** 0.5 + ADAM_EPS) + DECAY * p)
    del first, second
    out = {"param": p, "copy": p if case["copy"] else None, "m": m, "v": v, "m_scale": None, "v_scale": None}
    if case["bits"] == 8:
        for name, x in (("m", m), ("v", v ** 0.5)):
            top = x.view(-1, BLOCK).abs().max(1, keepdim=True).values
            out[name] = (x.view(-1, BLOCK) / top.clamp(min=1e-300) * E4M3_MAX).view(-1)
            out[name + "_scale"] = top.view(-1) / E4M3_MAX
    return out
