"""Products of 4-bit weight rows against plain 64-bit products.

The bar, element by element.  A code c enters as 24 + c and 24 x is taken off
again, so a group's fp32 sum is over terms of at most (24 + c + 24) |x|: off by at
most L 2^-23 times their sum over L = K + 64 additions.  x is held as bf16 columns
that leave 2^-17 of it (two) or 2^-26 (three); rotated, its 8 fp32 steps leave
8 * 2^-24 of the block's absolute sum / sqrt(128).  The result is rounded once."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
HALF_STEP = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
TINY = {"bf16": 0.0, "f16": 2.0 ** -25, "f32": 0.0}


@pytest.fixture(scope="module")
def m():
    from int4_routed_expert_amd import moe_w4
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return moe_w4


def hadamard128():
    h = torch.ones((1, 1), dtype=torch.float64)
    for _ in range(7):
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
    return h / math.sqrt(128.0)


def make(tokens, n, k, group, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((tokens, k), generator=g).to(DT[dtype])
    codes = torch.randint(0, 256, (n, k // 2), generator=g, dtype=torch.uint8)
    scales = (torch.randn((n, k // group), generator=g) * 0.01).bfloat16()
    return x, codes, scales


def reference(x, codes, scales, group, rotate, out):
    c = torch.stack([codes & 15, codes >> 4], dim=-1).reshape(codes.shape[0], -1).double()
    c = torch.where(c > 7, c - 16, c)
    s = scales.double().repeat_interleave(group, dim=1)
    xr, k = x.double(), x.shape[1]
    rest = xr.abs() * (0.0 if x.dtype == torch.bfloat16 and not rotate else 2.0 ** -17)
    if rotate:
        b = xr.reshape(-1, 128)
        mag = (b.abs().sum(1, keepdim=True) / math.sqrt(128.0)).expand(b.shape).reshape(xr.shape)
        xr = (b @ hadamard128()).reshape(xr.shape)
        rest = xr.abs() * (2.0 ** -26 if out == "f32" else 2.0 ** -17) + 8 * 2.0 ** -24 * mag
    y = xr @ (c * s).t()
    err = (k + 64) * 2.0 ** -23 * (xr.abs() @ ((48 + c) * s.abs()).t()) + rest @ (c * s).abs().t()
    return y, err + HALF_STEP[out] * (y.abs() + err) + TINY[out]


CASES = [(t, n, k, g, r, d, o)
         for t, n, k in [(1, 1, 128), (1, 2048, 2048), (2, 17, 256), (3, 15, 384), (5, 33, 1152), (8, 64, 640),
                         (9, 100, 128), (16, 31, 2048), (17, 48, 512), (33, 16, 256), (64, 65, 1024)]
         for g, r, d, o in [(128, False, "bf16", "bf16"), (64, False, "f16", "f32"), (32, True, "bf16", "f32"),
                            (128, True, "f16", "f16"), (32, False, "bf16", "f16"), (64, True, "bf16", "bf16")]]


@pytest.mark.parametrize("tokens,n,k,group,rotate,dtype,out", CASES)
def test_matvec(m, tokens, n, k, group, rotate, dtype, out):
    x, codes, scales = make(tokens, n, k, group, dtype, 100 + tokens + n)
    y = torch.full((tokens, n), 7.0, dtype=DT[out], device="cuda")
    ws = m.matvec_workspace(tokens, k).fill_(0xFF)
    m.moe_w4_matvec(x.cuda(), codes.cuda(), scales.cuda(), y, ws, rotate=rotate)
    ref, bar = reference(x, codes, scales, group, rotate, out)
    worst = ((y.cpu().double() - ref).abs() - bar).max().item()
    assert bool(torch.isfinite(y).all()) and worst <= 0, worst


def test_wide_output(m):
    """More rows than one launch's workgroups hold at once; sampled columns."""
    x, codes, scales = make(4, 50001, 256, 128, "bf16", 9)
    y = torch.full((4, 50001), 7.0, device="cuda")
    m.moe_w4_matvec(x.cuda(), codes.cuda(), scales.cuda(), y, m.matvec_workspace(4, 256))
    ref, bar = reference(x, codes, scales, 128, False, "f32")
    assert ((y.cpu().double() - ref).abs() - bar).max().item() <= 0


def test_extreme_values(m):
    """All codes at an end of their range, x at the ends of its type, a column of infinity, a token of NaN."""
    for byte in (0x88, 0x77, 0x00):
        x, codes, scales = make(3, 20, 256, 32, "f16", 2)
        codes.fill_(byte)
        x[0] = torch.where(torch.arange(256) % 2 == 0, 65504.0, -6e-8).half()
        y = torch.empty((3, 20), device="cuda")
        m.moe_w4_matvec(x.cuda(), codes.cuda(), scales.cuda(), y, m.matvec_workspace(3, 256))
        ref, bar = reference(x, codes, scales, 32, False, "f32")
        assert ((y.cpu().double() - ref).abs() - bar - 1e-30).max().item() <= 0
    x, codes, scales = make(3, 20, 256, 32, "bf16", 2)
    x[1] = float("nan")
    y = torch.empty((3, 20), device="cuda")
    m.moe_w4_matvec(x.cuda(), codes.cuda(), scales.cuda(), y, m.matvec_workspace(3, 256))
    assert bool(torch.isnan(y[1]).all()) and bool(torch.isfinite(y[[0, 2]]).all())   # tokens do not mix


def test_reads_the_packers_rows(m):
    """Gate and up rows of a packed expert: the container's own layout and basis."""
    g = torch.Generator().manual_seed(12)
    w = (torch.randn(m.EXPERT_WEIGHTS, generator=g) * 0.05).bfloat16().cuda()
    codes = torch.empty((1, m.CODE_BYTES_PER_EXPERT), dtype=torch.uint8, device="cuda")
    scales = torch.empty((1, m.SCALES_PER_EXPERT), dtype=torch.int16, device="cuda")
    m.moe_w4_pack_experts(w, codes, scales)
    x = torch.randn((2, m.HIDDEN), generator=g).bfloat16()
    gu, sc = codes[0, :2 ** 20].view(1024, 1024), scales[0, :16384].view(1024, 16)
    y = torch.empty((2, 1024), device="cuda")
    m.moe_w4_matvec(x.cuda(), gu, sc, y, m.matvec_workspace(2, m.HIDDEN), rotate=True)
    ref, bar = reference(x, gu.cpu(), sc.view(torch.bfloat16).cpu(), 128, True, "f32")
    assert ((y.cpu().double() - ref).abs() - bar).max().item() <= 0
    full = x.double() @ w[:1024 * 2048].view(1024, 2048).cpu().double().t()
    assert ((y.cpu().double() - full).norm() / full.norm()).item() < 0.2   # the container's 4 bits, about 12%


def test_graph_and_side_stream(m):
    x, codes, scales = (t.cuda() for t in make(6, 300, 512, 64, "bf16", 21))
    y, ws = torch.empty((6, 300), dtype=torch.bfloat16, device="cuda"), m.matvec_workspace(6, 512)

    def step():
        m.moe_w4_matvec(x, codes, scales, y, ws, rotate=True)

    step()
    ref = y.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    assert torch.equal(ref, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(i)))
        ws.fill_(i)
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        step()
        torch.cuda.synchronize()
        assert torch.equal(got, y)


def test_refusals(m):
    x, codes, scales = (t.cuda() for t in make(2, 24, 256, 64, "bf16", 1))
    y, ws = torch.empty((2, 24), dtype=torch.bfloat16, device="cuda"), m.matvec_workspace(2, 256)

    def refused(status=None, **kw):
        a = dict(x=x, codes=codes, scales=scales, y=y, ws=ws)
        a.update(kw)
        with pytest.raises(m.MoeW4Error) as e:
            m.moe_w4_matvec(a["x"], a["codes"], a["scales"], a["y"], a["ws"])
        assert e.value.status == (m.EINVAL if status is None else status)

    refused(x=x.cpu())
    refused(x=x.float())
    refused(x=x[:, :128])
    refused(codes=codes.short())
    refused(codes=codes.t().contiguous().t())
    refused(codes=codes[:20])
    refused(scales=scales.float())
    refused(scales=scales[:, :3])
    refused(scales=scales[:, :2].contiguous(), codes=codes[:, :64].contiguous())
    refused(scales=scales[:, :1].contiguous())                       # a group of 256
    refused(y=y[:1])
    refused(y=y.double())
    refused(m.EWORKSPACE, ws=ws[:64])
    many = torch.zeros((65, 256), dtype=torch.bfloat16, device="cuda")
    refused(x=many, y=torch.empty((65, 24), dtype=torch.bfloat16, device="cuda"))
