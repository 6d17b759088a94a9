"""Block operators at the edges of memory: tensors beyond 4 GiB, scales aligned to two
bytes only, a workspace taken for another stream, two calls at once.

Results far behind a tensor's start are compared, bit by bit, with those of a call on
a copy of the rows alone, where that takes the same order of sums; 4-bit products
with 64 bits (two orders of fp32 sums)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module")
def m():
    from int4_routed_expert_amd import moe_w4
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return moe_w4


@pytest.fixture(autouse=True)
def give_back():
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def normal(*shape, seed=1, dtype=BF):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def far(rows, cols, dtype=BF):
    t = torch.empty((rows, cols), dtype=dtype, device="cuda")
    assert t.numel() * t.element_size() > 2 ** 32
    return t


ROWS, WIDE, LAST = 1048576, 2112, 70


@pytest.mark.parametrize("side", ["in", "out"])
def test_grouped_rows_beyond_32_bits(m, side):
    n, k = (16, WIDE) if side == "in" else (WIDE, 16)
    w, part = normal(2, n, k, seed=2), normal(LAST, k)
    x, y = torch.empty((ROWS, k), dtype=BF, device="cuda"), torch.empty((ROWS, n), dtype=BF, device="cuda")
    x[-LAST:] = part
    ends = torch.tensor([0, 33, LAST], dtype=torch.int32, device="cuda")
    want, dx_want = torch.empty((LAST, n), dtype=BF, device="cuda"), torch.empty((LAST, k), dtype=BF, device="cuda")
    m.moe_w4_grouped_mm(part, w, ends, want)
    m.moe_w4_grouped_mm(x, w, ends + (ROWS - LAST), y)
    # (both calls take the same tiles' rows apart, and sum over k in the same order)
    err = k * 2.0 ** -23 * (part.double().abs() @ w.double().abs().amax(0).T) * 2 + 2.0 ** -7 * want.double().abs()
    assert ((y[-LAST:].double() - want.double()).abs() <= err).all()
    x_out = x   # the gradient of x, over x itself
    m.moe_w4_grouped_mm_dx(want, w, ends, dx_want)
    y[-LAST:] = want
    m.moe_w4_grouped_mm_dx(y, w, ends + (ROWS - LAST), x_out)
    err = n * 2.0 ** -23 * (want.double().abs() @ w.double().abs().amax(0)) * 2 + 2.0 ** -7 * dx_want.double().abs()
    assert ((x_out[-LAST:].double() - dx_want.double()).abs() <= err).all()
    dw, dw_want = (torch.empty((2, n, k), device="cuda") for _ in range(2))
    x_out[-LAST:] = part
    m.moe_w4_grouped_mm_dw(part, want, ends, dw_want)
    m.moe_w4_grouped_mm_dw(x_out, y, ends + (ROWS - LAST), dw)
    err = 2 * LAST * 2.0 ** -23 * (want.double().abs().T @ part.double().abs())
    assert ((dw - dw_want).double().abs() <= err).all()


def test_grouped_weights_beyond_32_bits(m):
    e, n, k = 1024, 1160, 2048
    w, dw = (far(e, n * k).view(e, n, k) for _ in range(2))
    w[-1] = normal(n, k, seed=3)
    x, dy = normal(20, k), normal(20, n)
    offsets = torch.zeros((e + 1,), dtype=torch.int32, device="cuda")
    offsets[-1] = 20   # all rows to the last expert
    one = offsets[-2:]
    y, want = (torch.empty((20, n), dtype=BF, device="cuda") for _ in range(2))
    m.moe_w4_grouped_mm(x, w, offsets, y)
    m.moe_w4_grouped_mm(x, w[-1:], one.clone(), want)
    assert ((y - want).double().abs() <= 2 * k * 2.0 ** -23 * (x.double().abs() @ w[-1].double().abs().T) + 2.0 ** -7 * want.double().abs()).all()
    dw.fill_(7.0)
    m.moe_w4_grouped_mm_dw(x, dy, offsets, dw)
    ref, mag = dy.double().T @ x.double(), dy.double().abs().T @ x.double().abs()
    err = 20 * 2.0 ** -23 * mag
    assert ((dw[-1].double() - ref).abs() <= err + 2.0 ** -8 * (ref.abs() + err)).all()
    assert not bool(dw[:-1].any())


def test_norm_beyond_32_bits(m):
    t, h, last = 262400, 8192, 3
    r, y, d = far(t, h), far(t, h), far(t, h)
    for i, v in enumerate((r, y, d)):
        v.fill_(0.5)
        v[-last:] = normal(last, h, seed=i)
    gate = torch.full((t,), 0.5, dtype=BF, device="cuda")
    form = dict(gate_kind=m.GATE_TOKEN, post_norm=True, scale=0.5)
    x = far(t, h)
    small = [v[-last:].clone() for v in (r, y, d)]
    sx, sr = torch.empty_like(small[0]), torch.empty_like(small[0])
    m.moe_w4_norm_residual(small[0], small[1], sr, sx, gate=gate[-last:].clone(), **form)
    m.moe_w4_norm_residual(r, y, r, x, gate=gate, **form)
    assert torch.equal(r[-last:], sr) and torch.equal(x[-last:], sx)
    sdr, sdy = torch.empty_like(sr), torch.empty_like(sr)
    m.moe_w4_norm_residual_backward(sr, small[1], None, small[2], sdr, sdy, m.norm_workspace(last, h), gate=gate[-last:].clone(), **form)
    dy = far(t, h)
    m.moe_w4_norm_residual_backward(r, y, None, d, x, dy, m.norm_workspace(t, h), gate=gate, **form)
    assert torch.equal(x[-last:], sdr) and torch.equal(dy[-last:], sdy)


def weights(codes, scales, group):
    c = torch.stack([codes & 15, codes >> 4], 2).flatten(1).double()
    s = scales.double().repeat_interleave(group, 1)
    return torch.where(c > 7, c - 16, c) * s, s


def bar(x, s, group):
    """Each group starts at -24 sum(x) and adds (24 + c) x, at most twice 32 |x| in size, in 128 additions and the groups'."""
    return (128 + s.shape[1] // group + 4) * 2.0 ** -23 * (x.double().abs() @ (64 * s).T)


def test_codes_beyond_32_bits(m):
    n, k, last = 270000, 32768, 40
    codes = far(n, k // 2, torch.uint8)
    scales = torch.ones((n, k // 128), dtype=BF, device="cuda")
    g = torch.Generator().manual_seed(4)
    codes[-last:] = torch.randint(0, 256, (last, k // 2), dtype=torch.uint8, generator=g).cuda()
    x, y = normal(1, k), torch.empty((1, n), device="cuda")
    m.moe_w4_matvec(x, codes, scales, y, m.matvec_workspace(1, k))
    w, s = weights(codes[-last:], scales[-last:], 128)
    assert ((y[:, -last:].double() - x.double() @ w.T).abs() <= bar(x, s, 128)).all()


@pytest.mark.parametrize("k", [256, 384, 2304])
def test_scales_aligned_to_two_bytes(m, k):
    n, g = 50, torch.Generator().manual_seed(5)
    codes = torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, generator=g).cuda()
    store = (torch.rand((n * k // 128 + 1,), generator=g) + 0.5).bfloat16().cuda()
    scales = store[1:].view(n, k // 128)
    assert scales.data_ptr() % 4 == 2
    x, y = normal(3, k), torch.empty((3, n), device="cuda")
    m.moe_w4_matvec(x, codes, scales, y, m.matvec_workspace(3, k))
    w, s = weights(codes, scales, 128)
    assert ((y.double() - x.double() @ w.T).abs() <= bar(x, s, 128)).all()


@pytest.mark.parametrize("tokens,k,group", [(1, 384, 128), (3, 640, 64), (20, 384, 32), (2, 128, 128), (40, 1664, 128), (1, 6272, 32)])
def test_runs_of_tiles_with_odd_blocks(m, tokens, k, group):
    """Several tiles of 16 rows a workgroup, whose waves' shares begin and end inside tiles of an odd number of blocks."""
    n, g = 12007, torch.Generator().manual_seed(6)
    codes = torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, generator=g).cuda()
    scales = (torch.rand((n, k // group), generator=g) + 0.5).bfloat16().cuda()
    x, y = normal(tokens, k), torch.empty((tokens, n), device="cuda")
    m.moe_w4_matvec(x, codes, scales, y, m.matvec_workspace(tokens, k))
    w, s = weights(codes, scales, group)
    assert ((y.double() - x.double() @ w.T).abs() <= bar(x, s, group)).all()


def test_dw_takes_its_workspace_from_the_calls_stream(m, monkeypatch):
    n = k = 64
    x, dy = normal(40000, k), normal(40000, n, seed=2)
    offsets = torch.tensor([0, 40000], dtype=torch.int32, device="cuda")
    assert m.moe_w4_grouped_mm_dw_workspace_bytes(1, 40000, n, k) > 0
    dw, want = (torch.empty((1, n, k), device="cuda") for _ in range(2))
    m.moe_w4_grouped_mm_dw(x, dy, offsets, want)
    torch.cuda.synchronize()
    side, seen, empty = torch.cuda.Stream(), [], torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: (seen.append(torch.cuda.current_stream().cuda_stream), empty(*a, **kw))[1])
    for stream in (side, side.cuda_stream):
        dw.fill_(7.0)
        torch.cuda.synchronize()
        m.moe_w4_grouped_mm_dw(x, dy, offsets, dw, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(dw, want)
    assert seen == [side.cuda_stream] * 2


def test_two_calls_at_once(m):
    """Two streams with buffers of their own, each call's results those of a call alone."""
    def make(seed):
        g = torch.Generator().manual_seed(seed)
        codes = torch.randint(0, 256, (4000, 512), dtype=torch.uint8, generator=g).cuda()
        scales = (torch.rand((4000, 8), generator=g) + 0.5).bfloat16().cuda()
        x, off = normal(48, 1024, seed=seed), torch.tensor([0, 20, 48], dtype=torch.int32, device="cuda")
        w = normal(2, 4000, 1024, seed=seed + 1)
        out = dict(y=torch.empty((48, 4000), device="cuda"), p=torch.empty((48, 4000), dtype=BF, device="cuda"),
                   dw=torch.empty((2, 4000, 1024), device="cuda"), d=torch.empty((48, 4000), dtype=BF, device="cuda"),
                   e=torch.empty((48, 4000), dtype=BF, device="cuda"), gain=torch.empty((4000,), device="cuda"))
        ws, wn = m.matvec_workspace(48, 1024), m.norm_workspace(48, 4000)

        def run():
            m.moe_w4_matvec(x, codes, scales, out["y"], ws)
            m.moe_w4_grouped_mm(x, w, off, out["p"])
            m.moe_w4_grouped_mm_dw(x, out["p"], off, out["dw"])
            m.moe_w4_norm_residual_backward(out["p"], out["p"], None, out["p"], out["d"], out["e"], wn, d_pre_gain=out["gain"])
        return out, run

    pairs = [make(11), make(13)]
    want = []
    for out, run in pairs:
        run()
        want.append({k: v.clone() for k, v in out.items()})
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in pairs]
    for _ in range(5):
        for (out, run), s in zip(pairs, streams):
            with torch.cuda.stream(s):
                run()
    torch.cuda.synchronize()
    for (out, _), w in zip(pairs, want):
        for k in out:
            assert torch.equal(out[k], w[k]), k
