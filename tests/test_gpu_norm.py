"""The norms around a block, forward and backward, against the formulas in 64 bits.

The bar, element by element: every intermediate is fp32, the sums over a row are
trees of at most 32 steps and the formulas chain at most 32 more roundings, so
a result is off by at most 64 * 2^-24 of the same formula with every term taken
absolute, and is rounded once by half a step of its type.  Sums over rows add
T * 2^-24 of the absolute sum."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25, torch.float32: 0.0}
EPS = 1e-6


@pytest.fixture(scope="module")
def m():
    from int4_routed_expert_amd import moe_w4
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return moe_w4


def make(t, h, act, res, gate, gains, seed):
    g = torch.Generator().manual_seed(seed)

    def normal(shape, dt, sigma=1.0, mean=0.0):
        return (torch.randn(shape, generator=g) * sigma + mean).to(DT[dt]).cuda()

    d = dict(resid=normal((t, h), res, 2.0), y=normal((t, h), act), d_resid_out=normal((t, h), res), d_x=normal((t, h), act))
    shape = {"none": None, "token": (t,), "channel": (h,), "full": (t, h)}[gate]
    d["gate"] = None if shape is None else normal(shape, act, 0.5)
    d["post_gain"] = normal((h,), act, 0.2, 1.0) if gains else None
    d["pre_gain"] = normal((h,), act, 0.2, 1.0) if gains else None
    return d


def rms(v):
    return torch.sqrt(v.pow(2).mean(1, keepdim=True) + EPS)


def near(got, ref, mag, label, extra=0.0):
    got, dt = got.double().cpu(), got.dtype
    err = (64 + extra) * 2.0 ** -24 * mag.cpu()
    ref = ref.cpu()
    bar = err + HALF_STEP[dt] * (ref.abs() + err) + TINY[dt]
    worst = ((got - ref).abs() - bar).max().item() if got.numel() else 0.0
    assert bool(torch.isfinite(got).all()) and worst <= 0, f"{label}: {worst} over the bar"


def as64(t, kind=None):
    if t is None:
        return torch.ones((), dtype=torch.float64, device="cuda")
    t = t.double()
    return t[:, None] if kind == "token" else t


# widths at the edges of the kernel's forms: 8, one wave's 512, two, four, eight and sixteen waves', and odd ones between
WIDTHS = [8, 104, 512, 520, 1000, 1024, 1032, 2048, 2056, 4096, 4104, 8192]
FORMS = [("bf16", "f32", "channel", True, True), ("f16", "f16", "token", True, True), ("bf16", "bf16", "full", False, True),
         ("f32", "f32", "none", True, False), ("f16", "f32", "none", False, False)]


@pytest.mark.parametrize("act,res,gate,post,gains", FORMS)
@pytest.mark.parametrize("t,h", [(1, w) for w in WIDTHS] + [(7, w) for w in WIDTHS] + [(1100, 104), (1027, 520)])
def test_forward_and_backward(m, t, h, act, res, gate, post, gains):
    d = make(t, h, act, res, gate, gains, 31 + t + h)
    kind = {"none": m.GATE_NONE, "token": m.GATE_TOKEN, "channel": m.GATE_CHANNEL, "full": m.GATE_FULL}[gate]
    scale = 0.37
    post_gain = d["post_gain"] if post else None
    form = dict(gate=d["gate"], gate_kind=kind, scale=scale, post_norm=post, post_gain=post_gain, pre_gain=d["pre_gain"], eps=EPS)
    out, x = torch.full_like(d["resid"], 7.0), torch.full_like(d["y"], 7.0)
    m.moe_w4_norm_residual(d["resid"], d["y"], out, x, **form)
    r, y = d["resid"].double(), d["y"].double()
    g, a, b = as64(d["gate"], gate), as64(post_gain), as64(d["pre_gain"])
    p = 1 / rms(y) if post else torch.ones_like(y[:, :1])
    n = y * p
    s = n * a
    r2 = r + scale * g * s
    mag = r.abs() + (scale * g * s).abs()
    near(out, r2, mag, "resid_out")
    near(x, r2 / rms(r2) * b, mag / rms(r2) * b.abs(), "x")

    # backward: from the stream as it was written
    f32 = dict(dtype=torch.float32, device="cuda")
    dr, dy = torch.full_like(d["resid"], 7.0), torch.full_like(d["y"], 7.0)
    dg = None if gate == "none" else torch.full_like(d["gate"], 7.0, dtype=d["gate"].dtype if gate == "full" else torch.float32)
    da = torch.full((h,), 7.0, **f32) if post else None
    db = torch.full((h,), 7.0, **f32)
    ws = m.norm_workspace(t, h).fill_(0xFF)
    m.moe_w4_norm_residual_backward(out, d["y"], d["d_resid_out"], d["d_x"], dr, dy, ws, d_gate=dg, d_post_gain=da, d_pre_gain=db, **form)
    r2, dx, up = out.double(), d["d_x"].double(), d["d_resid_out"].double()
    q = 1 / rms(r2)
    u, hh = r2 * q, dx * b
    ref = up + q * (hh - u * (hh * u).mean(1, keepdim=True))
    mag = up.abs() + q * (hh.abs() + u.abs() * (hh * u).abs().mean(1, keepdim=True))
    near(dr, ref, mag, "d_resid")
    near(db, (dx * u).sum(0), (dx * u).abs().sum(0), "d_pre_gain", t)
    ds, dsm = scale * g * ref, (scale * g).abs() * mag
    if dg is not None:
        v, vm = scale * ref * s, scale * mag * s.abs()
        dim = {"token": 1, "channel": 0, "full": None}[gate]
        near(dg, v if dim is None else v.sum(dim), vm if dim is None else vm.sum(dim), "d_gate", 0 if dim is None else max(t, h))
    if post:
        near(da, (ds * n).sum(0), (dsm * n.abs()).sum(0), "d_post_gain", t)
    k, km = ds * a, dsm * a.abs()
    ref_y = p * (k - n * (k * n).mean(1, keepdim=True)) if post else k
    mag_y = p * (km + n.abs() * (km * n.abs()).mean(1, keepdim=True)) if post else km
    near(dy, ref_y, mag_y, "d_y")


def test_gradients_agree_with_differences(m):
    """d/dt of sum(out * A + x * B) along a direction, fp32 forward passes on both sides of a small step."""
    t, h = 3, 40
    d = make(t, h, "f32", "f32", "channel", True, 77)
    kw = dict(gate_kind=m.GATE_CHANNEL, scale=0.6, post_norm=True, eps=EPS)
    names = ("resid", "y", "gate", "post_gain", "pre_gain")

    def loss(v):
        out, x = torch.empty_like(v["resid"]), torch.empty_like(v["y"])
        m.moe_w4_norm_residual(v["resid"], v["y"], out, x, gate=v["gate"], post_gain=v["post_gain"], pre_gain=v["pre_gain"], **kw)
        return (out.double() * d["d_resid_out"].double() + x.double() * d["d_x"].double()).sum().item(), out

    _, out = loss(d)
    grad = {k: torch.empty_like(d[k]) for k in names}
    m.moe_w4_norm_residual_backward(out, d["y"], d["d_resid_out"], d["d_x"], grad["resid"], grad["y"], m.norm_workspace(t, h),
                                    gate=d["gate"], post_gain=d["post_gain"], pre_gain=d["pre_gain"], d_gate=grad["gate"],
                                    d_post_gain=grad["post_gain"], d_pre_gain=grad["pre_gain"], **kw)
    for i, k in enumerate(names):
        v = torch.randn(d[k].shape, generator=torch.Generator().manual_seed(i)).cuda()
        step = 2.0 ** -6
        hi, lo = ({**d, k: d[k] + sgn * step * v} for sgn in (1, -1))
        diff = (loss(hi)[0] - loss(lo)[0]) / (2 * step)
        want = (grad[k].double() * v.double()).sum().item()
        # the step's third-order term (2^-12 of the gradient's size) and fp32 sums of 240 values over 2^-5
        assert abs(diff - want) <= 2e-3 * (grad[k].double() * v.double()).abs().sum().item() + 240 * 2.0 ** -24 * 8 / step


def test_norm_alone_and_add_alone(m):
    d = make(5, 264, "bf16", "f32", "none", True, 3)
    x = torch.empty_like(d["y"])
    m.moe_w4_norm_residual(d["resid"], None, None, x, pre_gain=d["pre_gain"], eps=EPS)
    r = d["resid"].double()
    near(x, r / rms(r) * d["pre_gain"].double(), r.abs() / rms(r) * d["pre_gain"].double().abs(), "x")
    dr, db = torch.empty_like(d["resid"]), torch.empty((264,), device="cuda")
    m.moe_w4_norm_residual_backward(d["resid"], None, None, d["d_x"], dr, None, m.norm_workspace(5, 264), pre_gain=d["pre_gain"],
                                    d_pre_gain=db, eps=EPS)
    h, u = d["d_x"].double() * d["pre_gain"].double(), r / rms(r)
    ref = (h - u * (h * u).mean(1, keepdim=True)) / rms(r)
    near(dr, ref, (h.abs() + u.abs() * (h * u).abs().mean(1, keepdim=True)) / rms(r), "d_resid")
    near(db, (d["d_x"].double() * u).sum(0), (d["d_x"].double() * u).abs().sum(0), "d_pre_gain", 5)
    out = d["resid"].clone()
    m.moe_w4_norm_residual(out, d["y"], out, None, pre_norm=False, scale=2.0)       # in place, no norm at all
    near(out, r + 2 * d["y"].double(), r.abs() + 2 * d["y"].double().abs(), "resid_out")
    dy, dr = torch.empty_like(d["y"]), d["d_resid_out"].clone()
    m.moe_w4_norm_residual_backward(out, d["y"], dr, None, dr, dy, m.norm_workspace(5, 264), pre_norm=False, scale=2.0)
    assert torch.equal(dr, d["d_resid_out"]) and torch.equal(dy, (2 * d["d_resid_out"]).bfloat16())


def test_rows_of_zeros_and_of_large_values(m):
    d = make(4, 128, "bf16", "f32", "none", False, 5)
    d["resid"][0] = 0
    d["y"][0] = 0
    d["y"][1] *= 1e15
    d["resid"][2] *= 1e15
    d["y"][3] = float("nan")
    out, x = torch.empty_like(d["resid"]), torch.empty_like(d["y"])
    m.moe_w4_norm_residual(d["resid"], d["y"], out, x, post_norm=True, eps=EPS)
    assert bool((x[0] == 0).all()) and bool(torch.isfinite(x[:3]).all()) and bool(torch.isnan(x[3]).all())
    r, y = d["resid"].double()[:3], d["y"].double()[:3]
    r2 = r + y / rms(y)
    near(x[:3], r2 / rms(r2), (r.abs() + (y / rms(y)).abs()) / rms(r2), "x")


def test_no_rows(m):
    e = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    m.moe_w4_norm_residual(e, e, torch.empty_like(e), torch.empty_like(e))
    db = torch.full((64,), 7.0, device="cuda")
    m.moe_w4_norm_residual_backward(e, e, e, e, torch.empty_like(e), torch.empty_like(e), m.norm_workspace(0, 64), d_pre_gain=db)
    assert bool((db == 0).all())


def test_the_stacks_own_norm_and_add(m):
    """rmsnorm without gain and the plain residual add of moe_w4_stack_layer: the same fp32 stream, bit for bit."""
    T = 16
    w = m.generated_layer(0, 0)
    resid = torch.randn((T, m.HIDDEN), generator=torch.Generator().manual_seed(1)).cuda()
    mine, x, y = resid.clone(), torch.empty((T, m.HIDDEN), dtype=torch.bfloat16, device="cuda"), None
    xb, yb = torch.empty_like(x), torch.empty_like(x)
    m.moe_w4_stack_layer(resid, w["router_w"], w["codes"], w["scales"], w["shared_w"], xb, yb, m.workspace(T))
    m.moe_w4_norm_residual(mine, None, None, x)
    near(x, mine.double() / rms(mine.double()), (mine.double() / rms(mine.double())).abs(), "x")
    m.moe_w4_norm_residual(mine, yb, mine, x)
    assert torch.equal(mine, resid)


def test_same_bits_in_a_graph_and_on_a_side_stream(m):
    t, h = 300, 1000
    d = make(t, h, "bf16", "f32", "channel", True, 9)
    out, x, dr, dy = (torch.empty_like(v) for v in (d["resid"], d["y"], d["resid"], d["y"]))
    sums = [torch.empty((h,), device="cuda") for _ in range(3)]
    ws = m.norm_workspace(t, h)
    form = dict(gate=d["gate"], gate_kind=m.GATE_CHANNEL, scale=0.5, post_norm=True, post_gain=d["post_gain"], pre_gain=d["pre_gain"])

    def step():
        m.moe_w4_norm_residual(d["resid"], d["y"], out, x, **form)
        m.moe_w4_norm_residual_backward(out, d["y"], d["d_resid_out"], d["d_x"], dr, dy, ws, d_gate=sums[0], d_post_gain=sums[1],
                                        d_pre_gain=sums[2], **form)

    step()
    ref = [v.clone() for v in (out, x, dr, dy, *sums)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, (out, x, dr, dy, *sums)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        d["y"].copy_(torch.randn((t, h), generator=torch.Generator().manual_seed(i)))
        ws.fill_(i)
        graph.replay()
        torch.cuda.synchronize()
        got = [v.clone() for v in (out, x, dr, dy, *sums)]
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (out, x, dr, dy, *sums)))


def test_refusals(m):
    d = make(4, 64, "bf16", "f32", "channel", True, 2)
    out, x = torch.empty_like(d["resid"]), torch.empty_like(d["y"])

    def refused(status=None, **kw):
        a = dict(resid=d["resid"], y=d["y"], resid_out=out, x_out=x)
        a.update(kw)
        with pytest.raises(m.MoeW4Error) as e:
            m.moe_w4_norm_residual(a.pop("resid"), a.pop("y"), a.pop("resid_out"), a.pop("x_out"), **a)
        assert e.value.status == m.EINVAL

    refused(resid=d["resid"].cpu())
    refused(resid=d["resid"].half())
    refused(y=d["y"][:2])
    refused(y=d["y"].t().contiguous().t())
    refused(x_out=x.float())
    refused(x_out=None)
    refused(x_out=x, pre_norm=False)
    refused(gate=d["gate"])                                            # no kind
    refused(gate=d["gate"], gate_kind=m.GATE_TOKEN)                    # another kind's shape
    refused(gate_kind=m.GATE_CHANNEL)
    refused(gate=d["gate"], gate_kind=9)
    refused(post_gain=d["post_gain"])                                  # without its norm
    refused(pre_gain=d["pre_gain"], pre_norm=False, x_out=None)
    refused(pre_gain=d["pre_gain"].float())
    refused(eps=-1.0)
    refused(scale=float("nan"))
    refused(y=None)                                                    # and resid_out given
    refused(x_out=d["y"])                                              # overlaps an input
    w = m.norm_workspace(4, 64)
    with pytest.raises(m.MoeW4Error) as e:
        m.moe_w4_norm_residual_backward(out, d["y"], d["d_resid_out"], d["d_x"], out.clone(), x, w[:128])
    assert e.value.status == m.EWORKSPACE
    with pytest.raises(m.MoeW4Error):
        m.moe_w4_norm_residual_backward(out, d["y"], d["d_resid_out"], d["d_x"], out.clone(), x, w, d_post_gain=torch.empty(64, device="cuda"))
