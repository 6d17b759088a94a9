"""Products grouped by expert against plain 64-bit products, row by row of the groups.

The bar, element by element: products of 16-bit values are exact in fp32, a sum
of L of them is off by at most L * 2^-23 * sum|terms| (each addition rounded or
truncated, in any order), and the result is rounded once, by at most half a
step of its type (plus half the smallest fp16 step)."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
HALF_STEP = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
TINY = {"bf16": 0.0, "f16": 2.0 ** -25, "f32": 0.0}

# rows of each group: none, one, around the tile sizes, one group with all, empty ones first, last and in a row
COUNTS = {
    "ragged": [0, 1, 16, 17, 0, 0, 63, 64, 65, 3, 0],
    "tiles": [127, 128, 129, 255, 256, 257, 0, 1],
    "one": [300],
    "empty": [0, 0, 0],
    "single_rows": [1] * 37,
}
SIZES = [(8, 8), (24, 136), (64, 64), (72, 264), (264, 72), (520, 128)]


@pytest.fixture(scope="module")
def m():
    from int4_routed_expert_amd import moe_w4
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return moe_w4


def make(counts, n, k, dtype, seed, before=0, behind=0):
    g = torch.Generator().manual_seed(seed)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32) + before
    rows = int(off[-1]) + behind
    x = torch.randn((rows, k), generator=g).to(DT[dtype])
    dy = torch.randn((rows, n), generator=g).to(DT[dtype])
    w = (torch.randn((len(counts), n, k), generator=g) * 0.1).to(DT[dtype])
    return off, x, dy, w


def check(got, ref, mag, length, out, label):
    got, ref, mag = (t.double() for t in (got.cpu(), ref, mag))
    err = length * 2.0 ** -23 * mag
    bar = err + HALF_STEP[out] * (ref.abs() + err) + TINY[out]
    worst = ((got - ref).abs() - bar).max().item() if got.numel() else 0.0
    assert torch.isfinite(got).all() and worst <= 0, f"{label}: {worst} over the bar"


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("n,k", SIZES)
@pytest.mark.parametrize("counts", list(COUNTS))
def test_three_products(m, counts, n, k, dtype):
    c = COUNTS[counts]
    off, x, dy, w = make(c, n, k, dtype, 11 + n + k, before=3, behind=5)
    offsets = torch.from_numpy(off).cuda()
    xg, dyg, wg = x.cuda(), dy.cuda(), w.cuda()
    y = torch.full((x.shape[0], n), 7.0, dtype=DT[dtype], device="cuda")
    dx = torch.full((x.shape[0], k), 7.0, dtype=DT[dtype], device="cuda")
    add = torch.randn((len(c), n, k), generator=torch.Generator().manual_seed(5))
    dw = torch.full(w.shape, 7.0, dtype=DT[dtype], device="cuda")
    dwf = add.cuda()
    m.moe_w4_grouped_mm(xg, wg, offsets, y)
    m.moe_w4_grouped_mm_dx(dyg, wg, offsets, dx)
    m.moe_w4_grouped_mm_dw(xg, dyg, offsets, dw)
    m.moe_w4_grouped_mm_dw(xg, dyg, offsets, dwf, add=dwf)
    X, D, W = x.double(), dy.double(), w.double()
    for e in range(len(c)):
        a, b = int(off[e]), int(off[e + 1])
        check(y[a:b], X[a:b] @ W[e].t(), X[a:b].abs() @ W[e].abs().t(), k, dtype, f"y group {e}")
        check(dx[a:b], D[a:b] @ W[e], D[a:b].abs() @ W[e].abs(), n, dtype, f"dx group {e}")
        ref, mag = D[a:b].t() @ X[a:b], D[a:b].abs().t() @ X[a:b].abs()
        check(dw[e], ref, mag, b - a, dtype, f"dw group {e}")
        check(dwf[e], ref + add[e].double(), mag + add[e].double().abs(), b - a + 1, "f32", f"dw + add group {e}")
    for t in (y, dx):   # rows of no group
        assert bool((t[:3] == 7).all()) and bool((t[int(off[-1]):] == 7).all())


# sizes whose tiles are the largest ones of each product (many rows a group and many tiles), the ones between, and
# the smallest, each with ragged edges in every direction
@pytest.mark.parametrize("which,groups,each,n,k", [("mm", 8, 760, 2056, 264), ("mm", 20, 300, 2056, 264), ("mm", 4, 700, 1032, 136), ("mm", 6, 200, 264, 72),
                                                   ("mm", 40, 60, 648, 200), ("mm", 70, 3, 520, 264),
                                                   ("dx", 8, 760, 264, 2056), ("dx", 20, 300, 264, 2056), ("dx", 4, 700, 136, 1032), ("dx", 40, 60, 200, 648),
                                                   ("dw", 60, 90, 1400, 2056), ("dw", 5, 400, 1288, 520)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_tile_forms(m, which, groups, each, n, k, dtype):
    rng = np.random.default_rng(groups + n)
    counts = rng.multinomial(groups * each, np.ones(groups) / groups)
    counts[groups // 2] = 0
    counts[-1] = 1
    off, x, dy, w = make(counts.tolist(), n, k, dtype, 13, behind=40)
    offsets, x, dy, w = torch.from_numpy(off).cuda(), x.cuda(), dy.cuda(), w.cuda()
    src, out = (x, torch.full((x.shape[0], n), 7.0, dtype=DT[dtype], device="cuda")) if which == "mm" else \
        (dy, torch.full((x.shape[0], k), 7.0, dtype=DT[dtype], device="cuda"))
    if which == "dw":
        add = torch.randn(w.shape, device="cuda")
        out = torch.full(w.shape, 7.0, device="cuda")
        m.moe_w4_grouped_mm_dw(x, dy, offsets, out, add=add)
        half = torch.full_like(w, 7.0)
        m.moe_w4_grouped_mm_dw(x, dy, offsets, half)
    elif which == "mm":
        m.moe_w4_grouped_mm(x, w, offsets, out)
    else:
        m.moe_w4_grouped_mm_dx(dy, w, offsets, out)
    for e in range(groups):
        a, b = int(off[e]), int(off[e + 1])
        W = w[e].double()
        if which == "dw":
            ref, mag = dy[a:b].double().t() @ x[a:b].double(), dy[a:b].double().abs().t() @ x[a:b].double().abs()
            check(out[e], (ref + add[e].double()).cpu(), (mag + add[e].double().abs()).cpu(), b - a + 1, "f32", f"dw group {e}")
            check(half[e], ref.cpu(), mag.cpu(), b - a, dtype, f"16-bit dw group {e}")
            continue
        W = W.t() if which == "mm" else W
        S = src[a:b].double()
        check(out[a:b], (S @ W).cpu(), (S.abs() @ W.abs()).cpu(), W.shape[0], dtype, f"{which} group {e}")
    if which != "dw":
        assert bool((out[int(off[-1]):] == 7).all())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_dw_adds_in_its_own_type(m, dtype):
    off, x, dy, w = make([5, 0, 130], 40, 72, dtype, 3)
    offsets = torch.from_numpy(off).cuda()
    out = torch.empty_like(w, device="cuda")
    m.moe_w4_grouped_mm_dw(x.cuda(), dy.cuda(), offsets, out, add=w.cuda())
    for e in range(3):
        a, b = int(off[e]), int(off[e + 1])
        ref = dy[a:b].double().t() @ x[a:b].double() + w[e].double()
        mag = dy[a:b].double().abs().t() @ x[a:b].double().abs() + w[e].double().abs()
        check(out[e], ref, mag, b - a + 1, dtype, f"group {e}")


@pytest.mark.parametrize("counts,n,k", [([30000], 72, 136), ([9000, 0, 700, 12001], 264, 40), ([1, 0, 40000], 8, 8)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_dw_in_slices(m, counts, n, k, dtype):
    """Few groups of many rows: summed in slices that a second launch joins; with and without a workspace given."""
    off, x, dy, w = make(counts, n, k, dtype, 17, behind=9)
    offsets, x, dy = torch.from_numpy(off).cuda(), x.cuda(), dy.cuda()
    nb = m.moe_w4_grouped_mm_dw_workspace_bytes(len(counts), x.shape[0], n, k)
    assert nb > 0
    ws = torch.full((nb,), 0xFF, dtype=torch.uint8, device="cuda")
    add = torch.randn(w.shape, device="cuda")
    full, half, own = (torch.full(w.shape, 7.0, dtype=t, device="cuda") for t in (torch.float32, DT[dtype], torch.float32))
    m.moe_w4_grouped_mm_dw(x, dy, offsets, full, add=add, workspace=ws)
    m.moe_w4_grouped_mm_dw(x, dy, offsets, half, add=w.cuda(), workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    m.moe_w4_grouped_mm_dw(x, dy, offsets, own, add=add, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(own, full)
    for e in range(len(counts)):
        a, b = int(off[e]), int(off[e + 1])
        ref, mag = dy[a:b].double().t() @ x[a:b].double(), dy[a:b].double().abs().t() @ x[a:b].double().abs()
        check(full[e], (ref + add[e].double()).cpu(), (mag + add[e].double().abs()).cpu(), b - a + 1, "f32", f"group {e}")
        W = w[e].double()
        check(half[e], ref.cpu() + W, mag.cpu() + W.abs(), b - a + 1, dtype, f"16-bit group {e}")


def test_no_rows_at_all(m):
    offsets = torch.zeros(4, dtype=torch.int32, device="cuda")
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    dy = torch.empty((0, 24), dtype=torch.bfloat16, device="cuda")
    w = torch.ones((3, 24, 64), dtype=torch.bfloat16, device="cuda")
    m.moe_w4_grouped_mm(x, w, offsets, dy)
    m.moe_w4_grouped_mm_dx(dy, w, offsets, x)
    dw = torch.full((3, 24, 64), 7.0, device="cuda")
    m.moe_w4_grouped_mm_dw(x, dy, offsets, dw)
    assert bool((dw == 0).all())
    m.moe_w4_grouped_mm_dw(x, dy, offsets, dw, add=torch.ones_like(dw))
    assert bool((dw == 1).all())


def test_rows_of_no_group_reach_nothing(m):
    """NaN and infinities in the rows around the groups, and between the end of one operand's rows and a tile's."""
    off, x, dy, w = make([9, 0, 70], 72, 136, "bf16", 4, before=2, behind=150)
    bad = torch.tensor([float("nan"), float("inf"), -float("inf")])
    for t in (x, dy):
        for part in (t[:2], t[int(off[-1]):]):
            part.copy_(bad[torch.arange(part.numel()) % 3].reshape(part.shape))
    offsets = torch.from_numpy(off).cuda()
    y = torch.zeros((x.shape[0], 72), dtype=torch.bfloat16, device="cuda")
    dw = torch.empty((3, 72, 136), device="cuda")
    m.moe_w4_grouped_mm(x.cuda(), w.cuda(), offsets, y)
    m.moe_w4_grouped_mm_dw(x.cuda(), dy.cuda(), offsets, dw)
    assert bool(torch.isfinite(y).all()) and bool(torch.isfinite(dw).all()) and bool((dw[1] == 0).all())


def test_offsets_out_of_order_or_range_stay_inside(m):
    """Clamped to [0, M]; a group that would end before it begins is empty."""
    rows, n, k = 40, 24, 64
    g = torch.Generator().manual_seed(8)
    x, w = torch.randn((rows, k), generator=g).bfloat16(), torch.randn((4, n, k), generator=g).bfloat16()
    offsets = torch.tensor([-5, 10, 4, 30, 1000], dtype=torch.int32)
    y = torch.full((rows, n), 7.0, dtype=torch.bfloat16, device="cuda")
    m.moe_w4_grouped_mm(x.cuda(), w.cuda(), offsets.cuda(), y)
    dw = torch.empty((4, n, k), device="cuda")
    m.moe_w4_grouped_mm_dw(x.cuda(), x[:, :n].contiguous().cuda(), offsets.cuda(), dw)
    assert bool((dw[1] == 0).all())
    X, W = x.double(), w.double()
    for a, b, e in ((0, 4, 0), (10, 30, 2), (30, 40, 3)):   # (rows 4 .. 10 are claimed by groups 0 and 2)
        check(y[a:b], X[a:b] @ W[e].t(), X[a:b].abs() @ W[e].abs().t(), k, "bf16", f"rows {a}..{b}")


def test_same_bits_each_time_on_a_side_stream_and_in_a_graph(m):
    off, x, dy, w = make([33, 0, 200, 1], 136, 264, "bf16", 6)
    offsets = torch.from_numpy(off).cuda()
    x, dy, w = x.cuda(), dy.cuda(), w.cuda()
    y, dx = torch.empty((x.shape[0], 136), dtype=torch.bfloat16, device="cuda"), torch.empty_like(x)
    dw = torch.empty_like(w)

    def step():
        m.moe_w4_grouped_mm(x, w, offsets, y)
        m.moe_w4_grouped_mm_dx(dy, w, offsets, dx)
        m.moe_w4_grouped_mm_dw(x, dy, offsets, dw)

    step()
    ref = [t.clone() for t in (y, dx, dw)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, (y, dx, dw)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    keep = x.clone()
    for i in range(3):
        x.copy_(keep * (i + 1))
        offsets.copy_(torch.from_numpy(off).cuda())
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (y, dx, dw)]
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (y, dx, dw)))


def test_refusals(m):
    off, x, dy, w = make([4, 4], 24, 64, "bf16", 1)
    offsets, x, w = torch.from_numpy(off).cuda(), x.cuda(), w.cuda()
    y = torch.empty((8, 24), dtype=torch.bfloat16, device="cuda")

    def refused(**kw):
        a = dict(x=x, w=w, offsets=offsets, y=y)
        a.update(kw)
        with pytest.raises(m.MoeW4Error) as e:
            m.moe_w4_grouped_mm(a["x"], a["w"], a["offsets"], a["y"])
        assert e.value.status == m.EINVAL

    refused(x=x.cpu())
    refused(x=x.float())
    refused(x=x.half())
    refused(x=x[:, :32])
    refused(w=w.transpose(1, 2))
    refused(w=w[0])
    refused(offsets=offsets.long())
    refused(offsets=offsets[:2])
    refused(y=y[:4])
    refused(y=y.t().contiguous().t())
    refused(y=y.float())
    refused(w=w[:, :20].contiguous(), y=y[:, :20].contiguous())   # N no multiple of 8
