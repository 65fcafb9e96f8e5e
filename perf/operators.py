"""Cases of the training-step operators that surround the optimizer's update.

A layer is run with 8-bit operands, its model is trained against a teacher,
and the weight gradient goes to the optimizer:

* ``quantize_int8``: weights, activations or gradients to 8-bit integers with
  one scale per row, or transposed with one scale per column;
* ``int8_matmul``: the product of two such matrices (forward, input gradient,
  weight gradient);
* ``rms_norm`` / ``rms_norm_backward``: the norm in front of the product, with
  the residual's addition and an 8-bit output;
* ``distill_loss`` / ``distill_loss_backward``: the loss against a teacher's
  top logits and its gradient.

The layer sizes are those of the 8B-shaped weight set of the benchmark
(q, o 4096 x 4096; k, v 1024 x 4096; gate, up 14336 x 4096; down 4096 x
14336).  With ``own`` false, ``run`` computes in elementary torch operations;
with ``own`` true it makes the library's calls.
"""
import math

import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32
DT = {"bf16": BF16, "f32": F32}


def listed():
    return [
        # the largest weight of a layer, 8-bit again after an optimizer step
        dict(name="quant_weight", op="quant", rows=14336, cols=4096, dtype="bf16", transpose=False),
        # a layer's input, transposed for the weight gradient's product
        dict(name="quant_act_t", op="quant", rows=8192, cols=4096, dtype="bf16", transpose=True),
        # one token through the gate weight
        dict(name="mm_token", op="mm", m=1, n=14336, k=4096, dtype="bf16"),
        # a ragged batch of prompts against the key weight, odd depth
        dict(name="mm_ragged", op="mm", m=333, n=1024, k=4099, dtype="f32"),
        # the gate product of a training batch
        dict(name="mm_forward", op="mm", m=8192, n=14336, k=4096, dtype="bf16"),
        # the weight gradient of q: the depth is the tokens, fp32 for the momentum
        dict(name="mm_wgrad", op="mm", m=4096, n=4096, k=8192, dtype="f32"),
        # one token in front of an 8-bit product
        dict(name="rms_token", op="rms", rows=1, cols=4096, dtype="bf16", residual=True, int8=True),
        # a training batch, residual added, 8-bit output
        dict(name="rms_forward", op="rms", rows=16384, cols=4096, dtype="bf16", residual=True, int8=True),
        # its gradient: residual branch's gradient added, weight gradient summed
        dict(name="rms_backward", op="rms_bwd", rows=16384, cols=4096, dtype="bf16"),
        # an evaluation batch: odd vocabulary, fp32 logits, ragged teacher entries
        dict(name="distill_small", op="kd", rows=61, vocab=50001, k=20, dtype="f32", temperature=2.0),
        # a training batch over a large vocabulary: the loss, and its gradient
        dict(name="distill_forward", op="kd", rows=4096, vocab=131072, k=64, dtype="bf16", temperature=1.0),
        dict(name="distill_backward", op="kd_bwd", rows=4096, vocab=131072, k=64, dtype="bf16", temperature=1.0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quant", "mm", "mm", "rms", "rms_bwd", "kd", "kd_bwd"])
    dtype = rng.choice(["bf16", "f32"])
    if op == "quant":
        rows = _log_int(rng, 1, 16384)
        cols = _log_int(rng, 64, max(64, min(14336, 14336 * 4096 // rows)))
        return dict(op=op, rows=rows, cols=cols, dtype=dtype, transpose=rng.random() < 0.5)
    if op == "mm":
        k = _log_int(rng, 64, 14336)
        n = _log_int(rng, 16, 14336)
        m = _log_int(rng, 1, max(1, min(8192, 8192 * 14336 * 4096 // (n * k))))
        return dict(op=op, m=m, n=n, k=k, dtype=dtype)
    if op in ("rms", "rms_bwd"):
        cols = _log_int(rng, 64, 8192)
        most = 16384 * 4096 // cols // (2 if dtype == "f32" else 1)
        rows = _log_int(rng, 1, min(16384, most))
        case = dict(op=op, rows=rows, cols=cols, dtype=dtype)
        if op == "rms":
            case.update(residual=rng.random() < 0.5, int8=rng.random() < 0.5)
        return case
    vocab = _log_int(rng, 1000, 131072)
    most = 4096 * 131072 // vocab // (2 if dtype == "f32" else 1)
    return dict(op=op, rows=_log_int(rng, 1, min(4096, most)), vocab=vocab,
                k=_log_int(rng, 1, 128), dtype=dtype, temperature=rng.choice([1.0, 2.0]))


def work(case):
    op = case["op"]
    es = 2 if case["dtype"] == "bf16" else 4
    if op == "quant":
        r, c = case["rows"], case["cols"]
        # read once; 8 bits and a scale written
        return {"bytes": r * c * (es + 1) + 4 * (c if case["transpose"] else r), "flops": 3 * r * c}
    if op == "mm":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": m * k + n * k + 4 * (m + n) + es * m * n, "flops": 2 * m * n * k}
    if op == "rms":
        r, c = case["rows"], case["cols"]
        by = r * c * es + es * c + 4 * r + r * c * (1 if case["int8"] else es)
        by += (2 * r * c * es if case["residual"] else 0) + (4 * r if case["int8"] else 0)
        return {"bytes": by, "flops": 6 * r * c}
    if op == "rms_bwd":
        r, c = case["rows"], case["cols"]
        return {"bytes": 4 * r * c * es + es * c + 4 * c + 4 * r, "flops": 10 * r * c}
    t, v, k = case["rows"], case["vocab"], case["k"]
    if op == "kd":
        return {"bytes": t * v * es + t * k * 8 + 8 * t, "flops": 4 * t * v}
    return {"bytes": 2 * t * v * es + t * k * 8 + 8 * t, "flops": 4 * t * v}


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, shape, dtype, std=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype).mul_(std)


def _int8_rows(g, rows, cols):
    # rows of 8-bit integers on 16-byte boundaries, as the quantizer lays them out
    pitch = (cols + 15) // 16 * 16
    x = _randn(g, (rows, pitch), BF16, 36.0).round_().clamp_(-127, 127)
    return x.to(torch.int8)[:, :cols]


def _teacher(g, t, v, k):
    """k distinct entries of every row (an arithmetic progression modulo v),
    falling logits; a tenth of the rows has fewer entries, some have none."""
    start = torch.randint(0, v, (t, 1), generator=g, device="cuda")
    step = torch.randint(1, max(2, v // k), (t, 1), generator=g, device="cuda")
    idx = (start + step * torch.arange(k, device="cuda")) % v
    drop = torch.rand((t, k), generator=g, device="cuda").log_().neg_().mul_(0.3)
    val = 9.0 - drop.cumsum(1)
    keep = torch.randint(0, 2 * k, (t, 1), generator=g, device="cuda")
    some = torch.rand((t, 1), generator=g, device="cuda") < 0.1
    gone = some & (torch.arange(k, device="cuda") >= keep)
    return val.contiguous(), idx.masked_fill(gone, -1).to(torch.int32).contiguous()


def prepare(case, seed):
    g = _gen(seed)
    op, dt = case["op"], DT[case["dtype"]]
    s = dict(case=case)
    if op == "quant":
        r, c = case["rows"], case["cols"]
        s["x"] = _randn(g, (r, c), dt, 0.02 if r > c else 1.0)
        # where a few channels are far larger than the rest
        s["x"][:, :: 97] *= 8
        qr, qc = (c, r) if case["transpose"] else (r, c)
        s["q"] = torch.empty((qr, (qc + 15) // 16 * 16), dtype=torch.int8, device="cuda")[:, :qc]
        s["scale"] = torch.empty(qr, dtype=F32, device="cuda")
        s["values"] = torch.empty((qr, qc), dtype=BF16, device="cuda")
    elif op == "mm":
        m, n, k = case["m"], case["n"], case["k"]
        s["a"], s["b"] = _int8_rows(g, m, k), _int8_rows(g, n, k)
        s["as"] = torch.rand(m, generator=g, device="cuda").add_(0.5).mul_(0.03)
        s["bs"] = torch.rand(n, generator=g, device="cuda").add_(0.5).mul_(0.0005)
        s["d"] = torch.empty((m, n), dtype=dt, device="cuda")
    elif op == "rms":
        r, c = case["rows"], case["cols"]
        s["x"] = _randn(g, (r, c), dt)
        s["w"] = _randn(g, (c,), dt, 0.1).add_(1.0)
        s["r"] = _randn(g, (r, c), dt, 2.0) if case["residual"] else None
        s["h"] = torch.empty((r, c), dtype=dt, device="cuda") if case["residual"] else None
        s["rstd"] = torch.empty(r, dtype=F32, device="cuda")
        if case["int8"]:
            s["q"] = torch.empty((r, (c + 15) // 16 * 16), dtype=torch.int8, device="cuda")[:, :c]
            s["scale"] = torch.empty(r, dtype=F32, device="cuda")
            s["values"] = torch.empty((r, c), dtype=BF16, device="cuda")
        else:
            s["y"] = torch.empty((r, c), dtype=dt, device="cuda")
    elif op == "rms_bwd":
        r, c = case["rows"], case["cols"]
        s["h"] = _randn(g, (r, c), dt, 2.0)
        s["w"] = _randn(g, (c,), dt, 0.1).add_(1.0)
        s["dy"] = _randn(g, (r, c), dt)
        s["dh"] = _randn(g, (r, c), dt)
        s["rstd"] = torch.rsqrt(s["h"].float().square().mean(1) + 1e-6)
        s["dx"] = torch.empty((r, c), dtype=dt, device="cuda")
        s["dw"] = torch.empty(c, dtype=F32, device="cuda")
    else:
        t, v, k = case["rows"], case["vocab"], case["k"]
        s["s"] = _randn(g, (t, v), dt, 1.5)
        s["tv"], s["ti"] = _teacher(g, t, v, k)
        # a student that knows part of it
        at = s["ti"].long().clamp_min(0)
        s["s"].scatter_add_(1, at, (0.7 * s["tv"]).masked_fill_(s["ti"] < 0, 0.0).to(dt))
        s["lse"] = torch.empty(t, dtype=F32, device="cuda")
        s["loss"] = torch.empty(t, dtype=F32, device="cuda")
        if op == "kd_bwd":
            z = s["s"].float().div_(case["temperature"])
            s["lse"].copy_(torch.logsumexp(z, 1))
            s["dloss"] = torch.full((t,), 1.0 / t, device="cuda")
            s["ds"] = torch.empty((t, v), dtype=dt, device="cuda")
    return s


# ------------------------------------------------------------- plain forms


def _quantize(x):
    amax = x.abs().amax(1)
    scale = amax / 127
    q = torch.round(x * (127 / amax)[:, None]).clamp(-127, 127)
    return torch.where(amax[:, None] > 0, q, torch.zeros_like(q)), scale


def _plain_quant(s):
    x = s["x"].float()
    q, scale = _quantize(x.t() if s["case"]["transpose"] else x)
    return (q * scale[:, None]).to(BF16), scale


def _plain_mm(s):
    acc = s["a"].float() @ s["b"].float().t()
    return (acc * s["as"][:, None] * s["bs"]).to(s["d"].dtype)


def _plain_rms(s):
    x = s["x"]
    h = (x.float() + s["r"].float()).to(x.dtype) if s["r"] is not None else x
    hf = h.float()
    rstd = 1 / torch.sqrt((hf * hf).mean(1) + 1e-6)
    y = hf * rstd[:, None] * s["w"].float()
    out = [h] if s["r"] is not None else []
    if not s["case"]["int8"]:
        return out + [y.to(x.dtype), rstd]
    q, scale = _quantize(y)
    return out + [(q * scale[:, None]).to(BF16), scale, rstd]


def _plain_rms_bwd(s):
    h, dy, rstd = s["h"].float(), s["dy"].float(), s["rstd"][:, None]
    xhat = h * rstd
    gw = dy * s["w"].float()
    dx = rstd * (gw - xhat * (gw * xhat).mean(1, keepdim=True)) + s["dh"].float()
    return dx.to(s["dx"].dtype), (dy * xhat).sum(0)


def _teacher_probs(s):
    tau = s["case"]["temperature"]
    live = s["ti"] >= 0
    t = (s["tv"] / tau).masked_fill(~live, -math.inf)
    some = live.any(1, keepdim=True)
    tm = torch.where(some, t.amax(1, keepdim=True), torch.zeros_like(t[:, :1]))
    e = torch.exp(t - tm)
    z = torch.where(some, e.sum(1, keepdim=True), torch.ones_like(tm))
    logp = torch.where(live, t - tm - torch.log(z), torch.zeros_like(t))
    return e / z, logp, some[:, 0]


def _plain_kd(s):
    tau = s["case"]["temperature"]
    z = s["s"].float() / tau
    m = z.amax(1)
    lse = m + torch.log(torch.exp(z - m[:, None]).sum(1))
    p, logp, some = _teacher_probs(s)
    zt = z.gather(1, s["ti"].long().clamp_min(0))
    loss = tau * tau * (p * (logp - (zt - lse[:, None]))).sum(1)
    zero = torch.zeros_like(loss)
    return torch.where(some, loss, zero), torch.where(some, lse, zero)


def _plain_kd_bwd(s):
    tau = s["case"]["temperature"]
    q = torch.exp(s["s"].float() / tau - s["lse"][:, None])
    p, _, some = _teacher_probs(s)
    d = (q * some[:, None]).scatter_add_(1, s["ti"].long().clamp_min(0), -p)
    return (d * (tau * s["dloss"])[:, None]).to(s["ds"].dtype)


PLAIN = {"quant": _plain_quant, "mm": _plain_mm, "rms": _plain_rms, "rms_bwd": _plain_rms_bwd,
         "kd": _plain_kd, "kd_bwd": _plain_kd_bwd}


# ------------------------------------------------------- the library's calls


def _values(s):
    # what the 8-bit integers stand for
    return torch.mul(s["q"], s["scale"][:, None], out=s["values"])


def _own(s):
    import orthonormalized_update_optimizers_b200 as ouo
    case = s["case"]
    op = case["op"]
    if op == "quant":
        ouo.quantize_int8(s["x"], s["q"], s["scale"], transpose=case["transpose"])
        return _values(s), s["scale"]
    if op == "mm":
        ouo.int8_matmul(s["a"], s["as"], s["b"], s["bs"], s["d"])
        return s["d"]
    if op == "rms":
        out = [s["h"]] if s["r"] is not None else []
        if case["int8"]:
            ouo.rms_norm(s["x"], s["w"], Q=s["q"], scale=s["scale"], residual=s["r"], H=s["h"],
                         rstd=s["rstd"], eps=1e-6)
            return out + [_values(s), s["scale"], s["rstd"]]
        ouo.rms_norm(s["x"], s["w"], Y=s["y"], residual=s["r"], H=s["h"], rstd=s["rstd"], eps=1e-6)
        return out + [s["y"], s["rstd"]]
    if op == "rms_bwd":
        ouo.rms_norm_backward(s["dy"], s["h"], s["w"], s["rstd"], s["dx"], dweight=s["dw"],
                              dH=s["dh"])
        return s["dx"], s["dw"]
    if op == "kd":
        ouo.distill_loss(s["s"], s["tv"], s["ti"], s["loss"], s["lse"],
                         temperature=case["temperature"])
        return s["loss"], s["lse"]
    ouo.distill_loss_backward(s["s"], s["tv"], s["ti"], s["lse"], s["dloss"], s["ds"],
                              temperature=case["temperature"])
    return s["ds"]


def run(s):
    return _own(s) if own else PLAIN[s["case"]["op"]](s)


# ------------------------------------------------- the definition in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    d = torch.float64

    def eight_bits(v):
        # largest magnitude of the row at 127, ties to even
        step = v.abs().max(dim=1).values.div(127)
        n = v.div(step.clamp_min(torch.finfo(d).tiny).unsqueeze(1)).round()
        return n.mul(step.unsqueeze(1)), step

    if op == "quant":
        v = s["x"].to(d)
        return eight_bits(v.T if case["transpose"] else v)
    if op == "mm":
        # integers below 2^53: the sums are exact
        return torch.einsum("mk,nk->mn", s["a"].to(d), s["b"].to(d)).mul_(
            s["as"].to(d).outer(s["bs"].to(d)))
    if op == "rms":
        h = s["x"] if s["r"] is None else (s["x"].to(d) + s["r"].to(d)).to(s["x"].dtype)
        v = h.to(d)
        rstd = (v.pow(2).sum(1) / v.shape[1] + 1e-6).pow(-0.5)
        y = v * s["w"].to(d) * rstd.unsqueeze(1)
        out = [] if s["r"] is None else [s["x"].to(d) + s["r"].to(d)]
        return out + ([*eight_bits(y), rstd] if case["int8"] else [y, rstd])
    if op == "rms_bwd":
        h, dy, rs = s["h"].to(d), s["dy"].to(d), s["rstd"].to(d).unsqueeze(1)
        u = dy * s["w"].to(d)
        inner = (u * h).sum(1, keepdim=True) / h.shape[1]
        return s["dh"].to(d) + rs * u - rs.pow(3) * h * inner, (dy * h * rs).sum(0)
    tau = case["temperature"]
    keep = s["ti"].ge(0)
    t = torch.where(keep, s["tv"].to(d) / tau, torch.full((), -1e300, dtype=d, device="cuda"))
    logp = torch.log_softmax(t, 1)
    p = logp.exp() * keep
    at = s["ti"].long() * keep
    has = keep.sum(1).gt(0).to(d)
    if op == "kd":
        z = s["s"].to(d) / tau
        lse = torch.logsumexp(z, 1)
        cross = (p * (lse.unsqueeze(1) - z.gather(1, at))).sum(1)
        ent = torch.where(p > 0, p * logp, torch.zeros_like(p)).sum(1)
        return (cross + ent) * has * tau ** 2, lse * has
    z = (s["s"].to(d) / tau - s["lse"].to(d).unsqueeze(1)).exp_()
    z.mul_(has.unsqueeze(1)).scatter_add_(1, at, -p)
    return z.mul_((s["dloss"].to(d) * tau).unsqueeze(1))
