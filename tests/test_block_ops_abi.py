"""The block operators' argument checks on the CPU: every refusal has its documented status and no call reaches the device."""
import pytest

X, W, OFF, Y, WS = 0x10000000, 0x20000000, 0x30000000, 0x40000000, 0x50000000


@pytest.fixture(scope="module")
def m():
    from int4_routed_expert_amd import moe_w4
    return moe_w4


def table(call, ok, bad):
    """`call` with the arguments of `ok` changed as each entry of `bad` says returns that entry's status."""
    for change, status in bad:
        assert call(**{**ok, **change}) == status, change


def test_limits_match_the_header(m):
    import os
    import re
    from tests.conftest import ROOT
    defines = dict(re.findall(r"#define MOE_W4_(\w+) \(?(-?\d+)\)?", open(os.path.join(ROOT, "include", "moe_w4.h")).read()))
    for n in ("F32", "BF16", "F16", "GROUPED_MAX_GROUPS", "GROUPED_MAX_ROWS", "GROUPED_MAX_DIM", "MATVEC_MAX_TOKENS", "MATVEC_MAX_K",
              "MATVEC_MAX_N", "NORM_POST", "NORM_PRE", "GATE_NONE", "GATE_TOKEN", "GATE_CHANNEL", "GATE_FULL", "NORM_MAX_ROWS",
              "NORM_MAX_WIDTH"):
        assert int(defines[n]) == getattr(m, n), n


@pytest.mark.parametrize("which", ["mm", "dx"])
def test_grouped_rows(m, which):
    f = getattr(m._lib, "moe_w4_grouped_" + ("mm" if which == "mm" else "mm_dx"))

    def call(a=X, w=W, off=OFF, e=4, M=100, N=64, K=128, dt=m.BF16, y=Y):
        return f(a, w, off, e, M, N, K, dt, y, None)

    E = m.EINVAL
    table(call, {}, [({"M": 0}, m.OK), ({"e": 0}, m.OK), ({"M": 0, "a": None, "y": None}, m.OK),
                     ({"M": -1}, E), ({"M": m.GROUPED_MAX_ROWS + 1}, E), ({"e": -1}, E), ({"e": m.GROUPED_MAX_GROUPS + 1}, E),
                     ({"N": 0}, E), ({"N": 60}, E), ({"K": 4}, E), ({"K": 130}, E), ({"N": m.GROUPED_MAX_DIM + 8}, E),
                     ({"K": m.GROUPED_MAX_DIM + 8}, E), ({"dt": m.F32}, E), ({"dt": 7}, E),
                     ({"a": None}, E), ({"w": None}, E), ({"off": None}, E), ({"y": None}, E),
                     ({"a": X + 8}, E), ({"w": W + 2}, E), ({"off": OFF + 2}, E), ({"y": Y + 8}, E),
                     ({"y": X + 1024}, E), ({"y": W + 1024}, E), ({"y": OFF}, E)])
    assert m.moe_w4_last_device_error() == 0


def test_grouped_dw(m):
    def call(x=X, dy=W, off=OFF, e=4, M=100, N=64, K=128, dt=m.F16, add=None, dw=Y, dwt=m.F32, ws=None, nb=0):
        return m._lib.moe_w4_grouped_mm_dw(x, dy, off, e, M, N, K, dt, add, dw, dwt, ws, nb, None)

    E = m.EINVAL
    big = m.moe_w4_grouped_mm_dw_workspace_bytes(1, 65536, 64, 128)
    assert big >= 2 * 64 * 128 * 4 and m.moe_w4_grouped_mm_dw_workspace_bytes(256, 65536, 1024, 2048) == 0
    assert m.moe_w4_grouped_mm_dw_workspace_bytes(1, 65536, 60, 128) == 0 and m.moe_w4_grouped_mm_dw_workspace_bytes(0, 9, 64, 128) == 0
    table(call, {"e": 1, "M": 65536}, [({"ws": WS, "nb": big - 1}, m.EWORKSPACE), ({"ws": WS + 8, "nb": big}, E), ({"ws": Y, "nb": big}, E)])
    table(call, {}, [({"e": 0}, m.OK), ({"M": -1}, E), ({"N": 4}, E), ({"dt": m.F32}, E), ({"dwt": m.BF16}, E), ({"dwt": 9}, E),
                     ({"x": None}, E), ({"dy": None}, E), ({"off": None}, E), ({"dw": None}, E), ({"M": 0, "dw": None}, E),
                     ({"x": X + 8}, E), ({"dw": Y + 4}, E), ({"add": WS + 4}, E), ({"dw": X}, E), ({"dw": W + 256}, E),
                     ({"add": Y + 1024}, E)])   # add overlaps dw without being it
    assert m.moe_w4_last_device_error() == 0


def test_matvec(m):
    nb = m.moe_w4_matvec_workspace_bytes(4, 256)
    assert nb >= 4 * 256 * 6
    assert m.moe_w4_matvec_workspace_bytes(65, 256) == 0 and m.moe_w4_matvec_workspace_bytes(4, 200) == 0
    assert m.moe_w4_matvec_workspace_bytes(-1, 256) == 0 and m.moe_w4_matvec_workspace_bytes(1, m.MATVEC_MAX_K + 128) == 0

    def call(x=X, c=W, s=OFF, M=4, N=100, K=256, g=64, rot=0, xt=m.BF16, y=Y, yt=m.F32, ws=WS, nb=nb):
        return m._lib.moe_w4_matvec(x, c, s, M, N, K, g, rot, xt, y, yt, ws, nb, None)

    E = m.EINVAL
    table(call, {}, [({"M": 0}, m.OK), ({"N": 0}, m.OK), ({"M": 65}, E), ({"M": -1}, E), ({"N": -1}, E), ({"N": m.MATVEC_MAX_N + 1}, E),
                     ({"K": 0}, E), ({"K": 192}, E), ({"K": m.MATVEC_MAX_K + 128}, E), ({"g": 16}, E), ({"g": 256}, E), ({"g": 0}, E),
                     ({"xt": m.F32}, E), ({"yt": 3}, E), ({"x": None}, E), ({"c": None}, E), ({"s": None}, E), ({"y": None}, E),
                     ({"ws": None}, E), ({"x": X + 8}, E), ({"c": W + 4}, E), ({"s": OFF + 1}, E), ({"y": Y + 4}, E), ({"ws": WS + 8}, E),
                     ({"nb": nb - 1}, m.EWORKSPACE), ({"y": X}, E), ({"y": W + 64}, E), ({"ws": Y}, E), ({"ws": X - 64}, E)])
    assert m.moe_w4_last_device_error() == 0


def test_norm(m):
    def call(r=X, y=W, gate=None, kind=0, scale=1.0, post=None, pre=None, flags=2, eps=1e-6, T=4, H=64, dt=m.BF16, rt=m.F32, out=Y, x=WS):
        return m._lib.moe_w4_norm_residual(r, y, gate, kind, scale, post, pre, flags, eps, T, H, dt, rt, out, x, None)

    E, G = m.EINVAL, 0x70000000
    table(call, {}, [({"T": 0}, m.OK), ({"T": -1}, E), ({"T": m.NORM_MAX_ROWS + 1}, E), ({"H": 0}, E), ({"H": 60}, E),
                     ({"H": m.NORM_MAX_WIDTH + 8}, E), ({"dt": 5}, E), ({"rt": m.F16}, E), ({"dt": m.F32, "rt": m.BF16}, E),
                     ({"flags": 4}, E), ({"kind": 4}, E), ({"kind": -1}, E), ({"kind": 1}, E), ({"gate": G}, E),
                     ({"eps": -1.0}, E), ({"eps": float("nan")}, E), ({"eps": float("inf")}, E), ({"scale": float("inf")}, E),
                     ({"post": G}, E), ({"pre": G, "flags": 0, "x": None}, E), ({"flags": 0}, E), ({"x": None}, E), ({"r": None}, E),
                     ({"out": None}, E), ({"y": None}, E), ({"y": None, "out": None, "flags": 0, "x": None}, E),
                     ({"y": None, "out": None, "flags": 3}, E), ({"y": None, "out": None, "gate": G, "kind": 1}, E),
                     ({"r": X + 8}, E), ({"y": W + 8}, E), ({"out": Y + 8}, E), ({"x": WS + 8}, E), ({"gate": G + 8, "kind": 2}, E),
                     ({"out": X + 16}, E), ({"x": W}, E), ({"x": Y + 16}, E), ({"x": X}, E)])
    assert m.moe_w4_last_device_error() == 0


def test_norm_backward(m):
    nb = m.moe_w4_norm_workspace_bytes(4, 64)
    assert nb >= 3 * 64 * 4 and m.moe_w4_norm_workspace_bytes(4, 60) == 0 and m.moe_w4_norm_workspace_bytes(-1, 64) == 0

    def call(r=X, y=W, gate=None, kind=0, scale=1.0, post=None, pre=None, flags=2, eps=1e-6, T=4, H=64, dt=m.BF16, rt=m.F32, up=0x60000000,
             dx=0x61000000, dr=0x62000000, dy=0x63000000, dg=None, da=None, db=None, ws=WS, nb=nb):
        return m._lib.moe_w4_norm_residual_backward(r, y, gate, kind, scale, post, pre, flags, eps, T, H, dt, rt, up, dx, dr, dy, dg, da, db,
                                                    ws, nb, None)

    E, G = m.EINVAL, 0x70000000
    table(call, {}, [({"T": -1}, E), ({"H": 12}, E), ({"dt": 5}, E), ({"rt": m.F16}, E), ({"flags": 8}, E), ({"r": None}, E),
                     ({"dx": None}, E), ({"dr": None}, E), ({"dy": None}, E), ({"y": None}, E), ({"flags": 0}, E), ({"ws": None}, E),
                     ({"da": G}, E), ({"db": G, "flags": 0, "dx": None}, E), ({"dg": G}, E), ({"nb": nb - 1}, m.EWORKSPACE),
                     ({"dr": 0x60000010}, E), ({"dy": 0x61000000}, E), ({"ws": 0x62000000}, E), ({"db": 0x62000000}, E), ({"dr": X}, E),
                     ({"db": G + 8}, E), ({"dx": 0x61000008}, E), ({"up": 0x60000004}, E)])
    assert m.moe_w4_last_device_error() == 0


def test_tensors_on_the_cpu_are_refused(m):
    import torch
    x = torch.zeros((2, 128), dtype=torch.bfloat16)
    for call in (lambda: m.moe_w4_grouped_mm(x, torch.zeros((1, 8, 128), dtype=torch.bfloat16), torch.tensor([0, 2], dtype=torch.int32), x[:, :8]),
                 lambda: m.moe_w4_grouped_mm_dw(x, x, torch.tensor([0, 2], dtype=torch.int32), torch.zeros((1, 128, 128))),
                 lambda: m.moe_w4_matvec(x, torch.zeros((8, 64), dtype=torch.uint8), torch.zeros((8, 1), dtype=torch.bfloat16), x, x),
                 lambda: m.moe_w4_norm_residual(x, x, x, x),
                 lambda: m.moe_w4_norm_residual_backward(x, x, x, x, x, x, x)):
        with pytest.raises(m.MoeW4Error) as e:
            call()
        assert e.value.status == m.EINVAL
