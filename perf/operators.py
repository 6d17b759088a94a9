"""Timed cases of the block operators: grouped products, 4-bit matrix-vector
products, and the norms around a block with its gate and residual scale.

Each case names an operator ("op"), its sizes and its types.  prepare() makes
what a program holds before the call, run() makes one pass, in elementary torch
operations in 32 bits or, where `own` is set, through the library, and exact()
evaluates the definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
EPS = 1e-6


def grouped(name, op, groups, rows, n, k, dtype, spread, pad=0, **more):
    return dict(name=name, op=op, groups=groups, rows=rows, n=n, k=k, dtype=dtype, spread=spread, pad=pad, **more)


def matvec(name, tokens, n, k, group, rotate, dtype, out):
    return dict(name=name, op="matvec", tokens=tokens, n=n, k=k, group=group, rotate=rotate, dtype=dtype, out=out)


def norm(name, op, tokens, width, dtype, resid, gate, post, gains):
    return dict(name=name, op=op, tokens=tokens, width=width, dtype=dtype, resid=resid, gate=gate, post=post, gains=gains)


def listed():
    return [
        # bf16 experts at a decode step of 8 sequences with 1 + 3 tokens, 6 experts each: mostly one row an expert
        grouped("grouped_decode", "grouped_mm", 256, 192, 1024, 2048, "bf16", 0.0),
        # gate/up of a prefill chunk of 2048 tokens whose routing is uneven; a padded batch, so rows lie behind the last group
        grouped("grouped_prefill", "grouped_mm", 256, 12288, 1024, 2048, "bf16", 1.0, pad=29),
        # gate/up over the largest batch, 65536 tokens: a training step's forward pass, bound by the products
        grouped("grouped_large", "grouped_mm", 256, 393216, 1024, 2048, "bf16", 0.3),
        # gradient of the rows, with sizes that no tile divides, in fp16
        grouped("grouped_dx_odd", "grouped_mm_dx", 60, 20011, 1400, 2056, "f16", 0.5, pad=5),
        # gradient of the gate/up weights over 16384 tokens, added to the fp32 sum of earlier micro-batches
        grouped("grouped_dw", "grouped_mm_dw", 256, 98304, 1024, 2048, "bf16", 0.3, grad="f32", accumulate=True),
        # one linear of one decoded token, in the rotated container format: latency
        matvec("matvec_one", 1, 2048, 2048, 128, True, "bf16", "bf16"),
        # gate and up of a dense block (width 6144) for one sequence's 1 + 3 speculative tokens
        matvec("matvec_draft", 4, 12288, 2048, 64, False, "f16", "f16"),
        # the output head over the vocabulary for 8 sequences with 1 + 3 tokens, fp32 logits
        matvec("matvec_head", 32, 150144, 2048, 128, False, "bf16", "f32"),
        # between two blocks at one decoded token: latency
        norm("norm_one", "norm", 1, 2048, "bf16", "f32", "none", False, True),
        # the same at the largest batch, with a norm behind the block and a gate for each channel
        norm("norm_large", "norm", 65536, 2048, "bf16", "f32", "channel", True, True),
        # backward of a small odd batch in fp16 with a gate for each token
        norm("norm_back_odd", "norm_back", 1001, 1000, "f16", "f16", "token", True, True),
        # backward of a training step of 16384 tokens, with the gradients of both gains and of the channel gate
        norm("norm_back", "norm_back", 16384, 2048, "bf16", "f32", "channel", True, True),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    def eights(lo, hi):
        return 8 * max(1, log(lo, hi) // 8)

    kind = rng.choice(["grouped_mm", "grouped_mm", "grouped_mm_dx", "grouped_mm_dw", "matvec", "matvec", "norm", "norm_back"])
    if kind.startswith("grouped"):
        n, k, groups = eights(64, 2048), eights(64, 2048), log(1, 256)
        rows = log(1, 200000)
        case = grouped("", kind, groups, rows, n, k, rng.choice(["bf16", "f16"]), rng.choice([0.0, 0.3, 1.0]) if rows < 20000 else 0.3, rng.randrange(0, 40))
        if kind == "grouped_mm_dw":
            case.update(grad=rng.choice(["same", "f32"]), accumulate=rng.random() < 0.5)
    elif kind == "matvec":
        group = rng.choice([32, 64, 128])
        k = 128 * log(1, 64)
        case = matvec("", log(1, 64), log(1, 40000), k, group, rng.random() < 0.5, rng.choice(["bf16", "f16"]), rng.choice(["bf16", "f16", "f32"]))
    else:
        width = eights(64, 8192)
        dtype = rng.choice(["bf16", "f16"])
        case = norm("", kind, log(1, 30000), width, dtype, rng.choice([dtype, "f32"]), rng.choice(["none", "token", "channel", "full"]), rng.random() < 0.5, rng.random() < 0.7)
    del case["name"]
    return case


# ---------------------------------------------------------------- inputs
def shares(case):
    """The probability of each group: exp(spread * z) for a fixed z, normalised."""
    z = np.random.RandomState(7).standard_normal(case["groups"])
    p = np.exp(case["spread"] * z)
    return p / p.sum()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(1000003 * (seed % 1000) + 17)

    def normal(shape, dtype, sigma=1.0, mean=0.0):
        t = torch.empty(shape, dtype=dtype, device="cuda")
        return t.normal_(mean, sigma, generator=g)

    st = {"case": case}
    if case["op"].startswith("grouped"):
        dt = DTYPES[case["dtype"]]
        e, n, k, rows = case["groups"], case["n"], case["k"], case["rows"]
        counts = np.random.RandomState(seed % 2**31).multinomial(rows, shares(case))
        st["offsets"] = torch.tensor(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32), device="cuda")
        st["most"] = int(counts.max())
        total = rows + case["pad"]
        if case["op"] != "grouped_mm_dx":
            st["x"] = normal((total, k), dt)
        if case["op"] != "grouped_mm":
            st["dy"] = normal((total, n), dt)
        if case["op"] != "grouped_mm_dw":
            st["w"] = normal((e, n, k), dt, 0.02)
        if case["op"] == "grouped_mm":
            st["y"] = torch.zeros((total, n), dtype=dt, device="cuda")
        elif case["op"] == "grouped_mm_dx":
            st["dx"] = torch.zeros((total, k), dtype=dt, device="cuda")
        else:
            grad = torch.float32 if case["grad"] == "f32" else dt
            # the sum of the earlier micro-batches' gradients, which the pass adds its own to
            st["before"] = normal((e, n, k), grad) if case["accumulate"] else None
            st["dw"] = torch.empty((e, n, k), dtype=grad, device="cuda")
    elif case["op"] == "matvec":
        m, n, k = case["tokens"], case["n"], case["k"]
        st["x"] = normal((m, k), DTYPES[case["dtype"]])
        st["codes"] = torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, device="cuda", generator=g)
        st["scales"] = (normal((n, k // case["group"]), torch.float32).abs() * 0.01).to(torch.bfloat16)
        st["y"] = torch.empty((m, n), dtype=DTYPES[case["out"]], device="cuda")
    else:
        t, h = case["tokens"], case["width"]
        dt, rt = DTYPES[case["dtype"]], DTYPES[case["resid"]]
        st["resid"] = normal((t, h), rt, 2.0)
        st["y"] = normal((t, h), dt, 0.7)
        shape = {"none": None, "token": (t,), "channel": (h,), "full": (t, h)}[case["gate"]]
        st["gate"] = None if shape is None else normal(shape, dt, 0.5)
        st["post_gain"] = normal((h,), dt, 0.1, 1.0) if case["post"] and case["gains"] else None
        st["pre_gain"] = normal((h,), dt, 0.1, 1.0) if case["gains"] else None
        st["scale"] = 0.22
        if case["op"] == "norm":
            st["resid_out"], st["x_out"] = torch.empty_like(st["resid"]), torch.empty_like(st["y"])
        else:
            st["d_resid_out"], st["d_x"] = normal((t, h), rt, 0.5), normal((t, h), dt)
            st["d_resid"], st["d_y"] = torch.empty_like(st["resid"]), torch.empty_like(st["y"])
            f32 = dict(dtype=torch.float32, device="cuda")
            st["d_gate"] = None if shape is None else torch.empty(shape, dtype=dt, device="cuda") if case["gate"] == "full" else torch.empty(shape, **f32)
            st["d_post_gain"] = torch.empty((h,), **f32) if st["post_gain"] is not None else None
            st["d_pre_gain"] = torch.empty((h,), **f32) if st["pre_gain"] is not None else None
    # scratch that a program keeps for its calls: room for a few copies of the tokens in 32 bits, or for partial column sums
    if case["op"] == "matvec":
        st["workspace"] = torch.empty((16 * case["k"] * (case["tokens"] + 16) + 65536,), dtype=torch.uint8, device="cuda")
    elif case["op"] == "norm_back":
        st["workspace"] = torch.empty((4 * 3 * 1024 * case["width"] + 65536,), dtype=torch.uint8, device="cuda")
    return st


# ---------------------------------------------------------------- one pass
def run(st):
    return run_own(st) if own else run_plain(st)


def run_own(st):
    from int4_routed_expert_amd import moe_w4 as m

    case = st["case"]
    op = case["op"]
    if op == "grouped_mm":
        m.moe_w4_grouped_mm(st["x"], st["w"], st["offsets"], st["y"])
        return st["y"]
    if op == "grouped_mm_dx":
        m.moe_w4_grouped_mm_dx(st["dy"], st["w"], st["offsets"], st["dx"])
        return st["dx"]
    if op == "grouped_mm_dw":
        m.moe_w4_grouped_mm_dw(st["x"], st["dy"], st["offsets"], st["dw"], add=st["before"])
        return st["dw"]
    if op == "matvec":
        m.moe_w4_matvec(st["x"], st["codes"], st["scales"], st["y"], st["workspace"], rotate=case["rotate"])
        return st["y"]
    kind = {"none": m.GATE_NONE, "token": m.GATE_TOKEN, "channel": m.GATE_CHANNEL, "full": m.GATE_FULL}[case["gate"]]
    if op == "norm":
        m.moe_w4_norm_residual(st["resid"], st["y"], st["resid_out"], st["x_out"], gate=st["gate"], gate_kind=kind, scale=st["scale"],
                               post_norm=case["post"], post_gain=st["post_gain"], pre_gain=st["pre_gain"], eps=EPS)
        return st["resid_out"], st["x_out"]
    m.moe_w4_norm_residual_backward(st["resid"], st["y"], st["d_resid_out"], st["d_x"], st["d_resid"], st["d_y"], st["workspace"],
                                    gate=st["gate"], gate_kind=kind, scale=st["scale"], post_norm=case["post"], post_gain=st["post_gain"],
                                    pre_gain=st["pre_gain"], d_gate=st["d_gate"], d_post_gain=st["d_post_gain"], d_pre_gain=st["d_pre_gain"], eps=EPS)
    return back_outputs(st)


def back_outputs(st):
    return {k: st[k] for k in ("d_resid", "d_y", "d_gate", "d_post_gain", "d_pre_gain")}


def by_group(rows, offsets, most):
    """[groups][most] rows of each group in 32 bits, zero behind its last."""
    at = offsets[:-1, None] + torch.arange(most, device="cuda", dtype=torch.int32)
    held = (at < offsets[1:, None]).unsqueeze(-1)
    return rows[at.clamp(max=rows.shape[0] - 1).long()].float() * held


def ungroup(out, padded, offsets, total):
    """Writes the rows of the groups back in their order; the rows behind them stay."""
    row = torch.arange(total, device="cuda", dtype=torch.int32)
    group = torch.searchsorted(offsets, row, right=True) - 1
    out[:total] = padded[group, row.long() - offsets[group].long()].to(out.dtype)


def hadamard(x):
    """Every block of 128 along the last axis times the normalised Sylvester Hadamard matrix."""
    i = torch.arange(128, device=x.device)
    v = i[:, None] & i[None, :]
    v = v ^ (v >> 4)
    v = v ^ (v >> 2)
    v = (v ^ (v >> 1)) & 1
    h = (1.0 - 2.0 * v.to(x.dtype)) / math.sqrt(128.0)
    return (x.reshape(-1, 128) @ h).reshape(x.shape)


def dequantised(codes, scales, group, dtype):
    """[n][k] weights: signed 4-bit codes, the even element in the low half of a byte, times the scale of their group."""
    both = torch.stack([codes & 15, codes >> 4], dim=-1).reshape(codes.shape[0], -1).to(torch.int8)
    return ((both ^ 8) - 8).to(dtype).reshape(codes.shape[0], -1, group).mul_(scales.to(dtype).unsqueeze(-1)).reshape(codes.shape[0], -1)


def run_plain(st):
    case = st["case"]
    op = case["op"]
    if op == "grouped_mm":
        padded = torch.bmm(by_group(st["x"], st["offsets"], st["most"]), st["w"].float().transpose(1, 2))
        ungroup(st["y"], padded, st["offsets"], case["rows"])
        return st["y"]
    if op == "grouped_mm_dx":
        padded = torch.bmm(by_group(st["dy"], st["offsets"], st["most"]), st["w"].float())
        ungroup(st["dx"], padded, st["offsets"], case["rows"])
        return st["dx"]
    if op == "grouped_mm_dw":
        dw = torch.bmm(by_group(st["dy"], st["offsets"], st["most"]).transpose(1, 2), by_group(st["x"], st["offsets"], st["most"]))
        if case["accumulate"]:
            dw = dw + st["before"]
        st["dw"].copy_(dw)
        return st["dw"]
    if op == "matvec":
        x = st["x"].float()
        if case["rotate"]:
            x = hadamard(x)
        st["y"].copy_(x @ dequantised(st["codes"], st["scales"], case["group"], torch.float32).t())
        return st["y"]
    y, resid, scale = st["y"].float(), st["resid"].float(), st["scale"]
    gate = 1.0 if st["gate"] is None else st["gate"].float()
    gate = gate.unsqueeze(1) if case["gate"] == "token" else gate
    post_gain = 1.0 if st["post_gain"] is None else st["post_gain"].float()
    pre_gain = 1.0 if st["pre_gain"] is None else st["pre_gain"].float()
    post_r = torch.rsqrt(y.square().mean(1, keepdim=True) + EPS) if case["post"] else None
    normed = y * post_r if case["post"] else y
    s = normed * post_gain
    if op == "norm":
        out = resid + scale * gate * s
        st["resid_out"].copy_(out)
        st["x_out"].copy_(out * torch.rsqrt(out.square().mean(1, keepdim=True) + EPS) * pre_gain)
        return st["resid_out"], st["x_out"]
    # backward: `resid` is the stream behind the block, as the forward pass left it
    d_x = st["d_x"].float()
    pre_r = torch.rsqrt(resid.square().mean(1, keepdim=True) + EPS)
    hat = resid * pre_r
    h = d_x * pre_gain
    d_resid = st["d_resid_out"].float() + pre_r * (h - hat * (h * hat).mean(1, keepdim=True))
    st["d_resid"].copy_(d_resid)
    if st["d_pre_gain"] is not None:
        st["d_pre_gain"].copy_((d_x * hat).sum(0))
    if st["d_gate"] is not None:
        d_gate = scale * d_resid * s
        st["d_gate"].copy_(d_gate.sum(1) if case["gate"] == "token" else d_gate.sum(0) if case["gate"] == "channel" else d_gate)
    d_s = scale * gate * d_resid
    if st["d_post_gain"] is not None:
        st["d_post_gain"].copy_((d_s * normed).sum(0))
    p = d_s * post_gain
    st["d_y"].copy_(post_r * (p - normed * (p * normed).mean(1, keepdim=True)) if case["post"] else p)
    return back_outputs(st)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    op = case["op"]
    if op.startswith("grouped"):
        n, k, rows, b = case["n"], case["k"], case["rows"], SIZE[case["dtype"]]
        flops = 2.0 * rows * n * k
        if op == "grouped_mm_dw":
            grad = 4 if case["grad"] == "f32" else b
            held = case["groups"] * n * k * grad
            return {"bytes": rows * (n + k) * b + held * (2 if case["accumulate"] else 1), "flops": flops}
        used = float(np.sum(1.0 - (1.0 - shares(case)) ** rows))   # groups with a row, expected
        return {"bytes": rows * (n + k) * b + used * n * k * b, "flops": flops}
    if op == "matvec":
        m, n, k = case["tokens"], case["n"], case["k"]
        return {"bytes": n * k / 2 + n * (k // case["group"]) * 2 + m * k * SIZE[case["dtype"]] + m * n * SIZE[case["out"]], "flops": 2.0 * m * n * k}
    t, h, b, r = case["tokens"], case["width"], SIZE[case["dtype"]], SIZE[case["resid"]]
    gate = {"none": 0, "token": t, "channel": h, "full": t * h}[case["gate"]]
    gains = h * ((1 if case["post"] else 0) + 1 if case["gains"] else 0)
    if op == "norm":
        return {"bytes": t * h * (2 * r + 2 * b) + (gate + gains) * b, "flops": 12.0 * t * h}
    back = gate * (b if case["gate"] == "full" else 4) + gains * 4
    return {"bytes": t * h * (3 * r + 3 * b) + (gate + gains) * b + back, "flops": 30.0 * t * h}


# ---------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op.startswith("grouped"):
        off = st["offsets"].tolist()
        out = {"grouped_mm": "y", "grouped_mm_dx": "dx", "grouped_mm_dw": "dw"}[op]
        out = torch.zeros(st[out].shape, dtype=torch.float64, device="cuda")
        for e, (a, b) in enumerate(zip(off[:-1], off[1:])):
            if op == "grouped_mm":
                out[a:b] = st["x"][a:b].double() @ st["w"][e].double().t()
            elif op == "grouped_mm_dx":
                out[a:b] = st["dy"][a:b].double() @ st["w"][e].double()
            else:
                out[e] = st["dy"][a:b].double().t() @ st["x"][a:b].double()
                if case["accumulate"]:
                    out[e] += st["before"][e].double()
        return out
    if op == "matvec":
        x = st["x"].double()
        if case["rotate"]:
            two = torch.tensor([[1.0, 1.0], [1.0, -1.0]], dtype=torch.float64, device="cuda")
            h = torch.ones((1, 1), dtype=torch.float64, device="cuda")
            for _ in range(7):
                h = torch.kron(two, h)
            x = torch.cat([b @ h for b in x.split(128, dim=1)], dim=1) / math.sqrt(128.0)
        y = torch.empty(st["y"].shape, dtype=torch.float64, device="cuda")
        for at in range(0, case["n"], 8192):
            c = st["codes"][at:at + 8192].to(torch.int16)
            w = torch.empty((c.shape[0], case["k"]), dtype=torch.float64, device="cuda")
            low, high = c % 16, c // 16
            w[:, 0::2] = torch.where(low > 7, low - 16, low).double()
            w[:, 1::2] = torch.where(high > 7, high - 16, high).double()
            w *= st["scales"][at:at + 8192].double().repeat_interleave(case["group"], dim=1)
            y[:, at:at + 8192] = x @ w.t()
        return y
    leaf = {k: st[k].double().requires_grad_(True) for k in ("resid", "y", "gate", "post_gain", "pre_gain") if st[k] is not None}
    s = leaf["y"]
    if case["post"]:
        s = s / torch.sqrt(s.pow(2).mean(-1, keepdim=True) + EPS)
        s = s * leaf["post_gain"] if "post_gain" in leaf else s
    if "gate" in leaf:
        s = s * (leaf["gate"][:, None] if case["gate"] == "token" else leaf["gate"])
    s = s * st["scale"]

    def before(r):
        r = r / torch.sqrt(r.pow(2).mean(-1, keepdim=True) + EPS)
        return r * leaf["pre_gain"] if "pre_gain" in leaf else r

    if op == "norm":
        out = (leaf["resid"] + s).detach()
        return out, before(out).detach()
    # the stream behind the block is given: the pre-norm's gradient meets it there, and the sum of both goes on to the block
    d_resid, = torch.autograd.grad(before(leaf["resid"]), leaf["resid"], st["d_x"].double(), retain_graph=True)
    d_resid = d_resid + st["d_resid_out"].double()
    found = {"d_resid": d_resid}
    wanted = [k for k in ("y", "gate", "post_gain") if k in leaf]
    found.update(("d_" + k, v) for k, v in zip(wanted, torch.autograd.grad(s, [leaf[k] for k in wanted], d_resid)))
    if "pre_gain" in leaf:
        found["d_pre_gain"], = torch.autograd.grad(before(leaf["resid"].detach()), leaf["pre_gain"], st["d_x"].double())
    return {k: found.get(k) for k in ("d_resid", "d_y", "d_gate", "d_post_gain", "d_pre_gain")}
