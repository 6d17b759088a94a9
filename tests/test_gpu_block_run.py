"""The block operators in a row, as a training step and a step of serving use them.

Each output is compared with the 64-bit formula of the kernels' own inputs to that
step (so that a step's bar is its own: fp32 sums of L terms, L * 2^-23 of the terms'
absolute sum, 64 * 2^-24 for a norm's chain, and half a step of the type for each
rounding); the gradients of the whole chain also with differences; a captured run
with the eager one, bit by bit, over several replays."""
import pytest
import torch

pytestmark = pytest.mark.gpu

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
EPS = 1e-6
T, H, I, E = 75, 264, 136, 5
COUNTS = [31, 0, 17, 24, 3]   # an expert without a token, one behind the last 16, all tokens in groups


@pytest.fixture(scope="module")
def m():
    from int4_routed_expert_amd import moe_w4
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return moe_w4


def near(got, ref, err, label):
    """|got - ref| <= err + half a step of what may be rounded (plus half the smallest fp16 step)."""
    bar = err + HALF_STEP[got.dtype] * (ref.abs() + err) + (2.0 ** -25 if got.dtype == torch.float16 else 0.0)
    worst = ((got.double() - ref).abs() - bar).max().item()
    assert bool(torch.isfinite(got).all()) and worst <= 0, f"{label}: {worst} over the bar"


def grouped(x, w, off):
    """y[r] = w[e] x[r] of fp64 tensors, the groups one after the other."""
    return torch.cat([x[a:b] @ w[e].T.contiguous() for e, (a, b) in enumerate(zip(off, off[1:]))])


def rms(v):
    return torch.sqrt(v.pow(2).mean(1, keepdim=True) + EPS)


class Block:
    """r, x = norm(r + s post(y0)); gate and up by experts; SwiGLU; down; r', x' = norm(r + c s' post(y))."""

    def __init__(self, m, dt, seed):
        g = torch.Generator().manual_seed(seed)

        def normal(*shape, sigma=1.0, mean=0.0, dtype=dt):
            return (torch.randn(shape, generator=g) * sigma + mean).to(dtype).cuda()

        self.m, self.dt = m, dt
        self.off = [0]
        for c in COUNTS:
            self.off.append(self.off[-1] + c)
        self.offsets = torch.tensor(self.off, dtype=torch.int32, device="cuda")
        self.p = dict(r=normal(T, H, sigma=2.0, dtype=torch.float32), y0=normal(T, H), a0=normal(H, sigma=0.2, mean=1.0),
                      b0=normal(H, sigma=0.2, mean=1.0), gu=normal(E, 2 * I, H, sigma=H ** -0.5), dn=normal(E, H, I, sigma=I ** -0.5),
                      c=normal(T, sigma=0.5), a1=normal(H, sigma=0.2, mean=1.0), b1=normal(H, sigma=0.2, mean=1.0))
        self.up = normal(T, H, dtype=torch.float32), normal(T, H)   # gradients from behind the block
        e16, e32 = (lambda *s: torch.empty(s, dtype=dt, device="cuda")), (lambda *s: torch.empty(s, device="cuda"))
        self.b = dict(r1=e32(T, H), x1=e16(T, H), gu=e16(T, 2 * I), h=e16(T, I), y=e16(T, H), r2=e32(T, H), x2=e16(T, H),
                      dr1=e32(T, H), dy=e16(T, H), dh=e16(T, I), dgu=e16(T, 2 * I), dx1=e16(T, H), dr=e32(T, H), dy0=e16(T, H))
        self.g = dict(r=self.b["dr"], y0=self.b["dy0"], a0=e32(H), b0=e32(H), gu=e32(E, 2 * I, H), dn=e32(E, H, I), c=e32(T),
                      a1=e32(H), b1=e32(H))
        self.ws = m.norm_workspace(T, H)
        self.first = dict(post_norm=True, post_gain=self.p["a0"], pre_gain=self.p["b0"], scale=0.5, eps=EPS)
        self.second = dict(gate=self.p["c"], gate_kind=m.GATE_TOKEN, post_norm=True, post_gain=self.p["a1"], pre_gain=self.p["b1"],
                           scale=0.7, eps=EPS)

    def forward(self):
        m, p, b = self.m, self.p, self.b
        m.moe_w4_norm_residual(p["r"], p["y0"], b["r1"], b["x1"], **self.first)
        m.moe_w4_grouped_mm(b["x1"], p["gu"], self.offsets, b["gu"])
        gate, up = b["gu"].float().chunk(2, 1)
        b["h"].copy_(torch.nn.functional.silu(gate) * up)
        m.moe_w4_grouped_mm(b["h"], p["dn"], self.offsets, b["y"])
        m.moe_w4_norm_residual(b["r1"], b["y"], b["r2"], b["x2"], **self.second)

    def backward(self):
        m, p, b, g = self.m, self.p, self.b, self.g
        m.moe_w4_norm_residual_backward(b["r2"], b["y"], *self.up, b["dr1"], b["dy"], self.ws, d_gate=g["c"], d_post_gain=g["a1"],
                                        d_pre_gain=g["b1"], **self.second)
        m.moe_w4_grouped_mm_dx(b["dy"], p["dn"], self.offsets, b["dh"])
        m.moe_w4_grouped_mm_dw(b["h"], b["dy"], self.offsets, g["dn"])
        gate, up = b["gu"].float().chunk(2, 1)
        dh, s = b["dh"].float(), torch.sigmoid(gate)
        b["dgu"].copy_(torch.cat([dh * up * s * (1 + gate * (1 - s)), dh * gate * s], 1))
        m.moe_w4_grouped_mm_dx(b["dgu"], p["gu"], self.offsets, b["dx1"])
        m.moe_w4_grouped_mm_dw(b["x1"], b["dgu"], self.offsets, g["gu"])
        m.moe_w4_norm_residual_backward(b["r1"], p["y0"], b["dr1"], b["dx1"], b["dr"], b["dy0"], self.ws, d_post_gain=g["a0"],
                                        d_pre_gain=g["b0"], **self.first)

    def outputs(self):
        return {**self.b, **{"grad " + k: v for k, v in self.g.items()}}


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
def test_training_step_by_step(m, dt):
    k = Block(m, dt, 5)
    k.forward()
    k.backward()
    p, b, g = ({n: t.double() for n, t in d.items()} for d in (k.p, k.b, k.g))
    eps32 = 2.0 ** -24

    def norms(r, y, out, x, a, pre, scale, gate, label):
        s = y / rms(y) * a * scale * gate
        mag = r.abs() + s.abs()
        near(k.b[out], r + s, 64 * eps32 * mag, label + " stream")
        ref = (r + s) / rms(r + s) * pre
        near(k.b[x], ref, 64 * eps32 * mag / rms(r + s) * pre.abs(), label + " norm")

    norms(p["r"], p["y0"], "r1", "x1", p["a0"], p["b0"], 0.5, 1.0, "first")
    for x, w, y, n in (("x1", "gu", "gu", H), ("h", "dn", "y", I)):
        near(k.b[y], grouped(b[x], p[w], k.off), n * 2 * eps32 * grouped(b[x].abs(), p[w].abs(), k.off), "product " + w)
    norms(b["r1"], b["y"], "r2", "x2", p["a1"], p["b1"], 0.7, p["c"][:, None], "second")

    for dy, w, dx, n in (("dy", "dn", "dh", H), ("dgu", "gu", "dx1", 2 * I)):
        wt = p[w].transpose(1, 2).contiguous()
        near(k.b[dx], grouped(b[dy], wt, k.off), n * 2 * eps32 * grouped(b[dy].abs(), wt.abs(), k.off), "dx of " + w)
    for x, dy, w in (("x1", "dgu", "gu"), ("h", "dy", "dn")):
        for e, (lo, hi) in enumerate(zip(k.off, k.off[1:])):
            xs, ds = b[x][lo:hi], b[dy][lo:hi]
            near(k.g[w][e], ds.T @ xs, (hi - lo) * 2 * eps32 * (ds.abs().T @ xs.abs()), f"dw of {w}, expert {e}")

    def back(r2, y, up, dx, dr, dy, a, pre, scale, gate, names, label):
        q = 1 / rms(r2)
        u, h = r2 * q, dx * pre
        ref = up + q * (h - u * (h * u).mean(1, keepdim=True))
        mag = up.abs() + q * (h.abs() + u.abs() * (h * u).abs().mean(1, keepdim=True))
        near(k.b[dr], ref, 64 * eps32 * mag, label + " d stream")
        pp = 1 / rms(y)
        n = y * pp
        ds, dsm = scale * gate * ref, (scale * gate * mag).abs() if torch.is_tensor(gate) else scale * mag
        kk, km = ds * a, dsm * a.abs()
        near(k.b[dy], pp * (kk - n * (kk * n).mean(1, keepdim=True)),
             64 * eps32 * pp * (km + n.abs() * (km * n.abs()).mean(1, keepdim=True)), label + " d y")
        near(k.g[names[0]], (ds * n).sum(0), (64 + T) * eps32 * (dsm * n.abs()).sum(0), label + " d post gain")
        near(k.g[names[1]], (dx * u).sum(0), (64 + T) * eps32 * (dx * u).abs().sum(0), label + " d pre gain")
        return scale * ref * n * a, scale * mag * (n * a).abs()

    up, upx = (t.double() for t in k.up)
    v, vm = back(b["r2"], b["y"], up, upx, "dr1", "dy", p["a1"], p["b1"], 0.7, p["c"][:, None], ("a1", "b1"), "second")
    near(k.g["c"], v.sum(1), (64 + H) * eps32 * vm.sum(1), "d gate")
    back(b["r1"], p["y0"], b["dr1"], b["dx1"], "dr", "dy0", p["a0"], p["b0"], 0.5, 1.0, ("a0", "b0"), "first")


def test_gradients_of_the_chain_agree_with_differences(m):
    """The chain's loss in 64 bits along each gradient d: its slope is |d|^2.

    At most ten roundings of 2^-11 lie between the inputs and a gradient, each taken
    as a relative error of a vector's norm and grown at most threefold by a product or
    norm of such well spread matrices; a step of 2^-10 of the input's norm adds 2^-9."""
    k = Block(m, torch.float16, 6)
    k.forward()
    k.backward()
    up, upx = (t.double() for t in k.up)

    def loss(p):
        r1 = p["r"] + 0.5 * p["y0"] / rms(p["y0"]) * p["a0"]
        gate, u = grouped(r1 / rms(r1) * p["b0"], p["gu"], k.off).chunk(2, 1)
        y = grouped(torch.nn.functional.silu(gate) * u, p["dn"], k.off)
        r2 = r1 + 0.7 * p["c"][:, None] * y / rms(y) * p["a1"]
        return (r2 * up).sum() + (r2 / rms(r2) * p["b1"] * upx).sum()

    p = {n: t.double() for n, t in k.p.items()}
    for n, d in k.g.items():
        d = d.double()
        step = 2.0 ** -10 * p[n].norm() / d.norm()
        slope = (loss({**p, n: p[n] + step * d}) - loss({**p, n: p[n] - step * d})) / (2 * step)
        assert abs(slope / (d * d).sum() - 1) <= 10 * 3 * 2.0 ** -11 + 2.0 ** -9, n


def test_training_captured_and_replayed(m):
    k = Block(m, torch.bfloat16, 7)
    k.forward()
    k.backward()
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        k.forward()
        k.backward()
    for i in range(3):
        k.p["r"].add_(0.25)   # inputs of a next step, and an eager run between the replays
        k.p["y0"].mul_(0.75)
        k.forward()
        k.backward()
        torch.cuda.synchronize()
        want = {n: t.clone() for n, t in k.outputs().items()}
        for t in k.outputs().values():
            t.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        for n, t in k.outputs().items():
            assert torch.equal(t, want[n]), (i, n)


@pytest.mark.parametrize("tokens", [1, 5])
def test_serving_captured_and_replayed(m, tokens):
    """Norm, 4-bit gate and up, SwiGLU, 4-bit down, norm: two layers that share a workspace."""
    h, inner, group = 512, 384, 128
    g = torch.Generator().manual_seed(8)
    layer = []
    for _ in range(2):
        layer.append([(torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, generator=g).cuda(),
                       (torch.rand((n, k // group), generator=g) * 0.02 + 0.005).bfloat16().cuda())
                      for n, k in ((2 * inner, h), (h, inner))])
    bf = dict(dtype=torch.bfloat16, device="cuda")
    r, x = torch.randn((tokens, h), generator=g).cuda(), torch.empty((tokens, h), **bf)
    ws = m.matvec_workspace(tokens, h)
    keep = [dict(gu=torch.empty((tokens, 2 * inner), **bf), a=torch.empty((tokens, inner), **bf), y=torch.empty((tokens, h), **bf),
                 r=torch.empty((tokens, h), device="cuda"), x=torch.empty((tokens, h), **bf)) for _ in layer]

    def run():
        m.moe_w4_norm_residual(r, None, None, x, eps=EPS)
        res, cur = r, x
        for (gu, dn), b in zip(layer, keep):
            m.moe_w4_matvec(cur, *gu, b["gu"], ws, rotate=True)
            gate, up = b["gu"].float().chunk(2, 1)
            b["a"].copy_(torch.nn.functional.silu(gate) * up)
            m.moe_w4_matvec(b["a"], *dn, b["y"], ws)
            m.moe_w4_norm_residual(res, b["y"], b["r"], b["x"], scale=0.5, eps=EPS)
            res, cur = b["r"], b["x"]

    run()
    # each product against 64 bits (the down products: not rotated)
    for (_, (codes, scales)), b in zip(layer, keep):
        c = torch.stack([codes & 15, codes >> 4], 2).reshape(h, inner).double()
        w = torch.where(c > 7, c - 16, c) * scales.double().repeat_interleave(group, 1)
        a = b["a"].double()
        # each group's sum starts at -24 sum(x) and adds (24 + c) x: twice 32 |x|, 128 additions, and the groups'
        err = (128 + inner // group + 1) * 2.0 ** -23 * (a.abs() @ (64 * scales.double().repeat_interleave(group, 1)).T)
        near(b["y"], a @ w.T, err, "down product")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        run()
    for i in range(3):
        r.mul_(1.25).add_(0.125)
        run()
        torch.cuda.synchronize()
        want = [{n: t.clone() for n, t in b.items()} for b in keep]
        for b in keep:
            for t in b.values():
                t.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        for b, v in zip(keep, want):
            for n in b:
                assert torch.equal(b[n], v[n]), (i, n)
