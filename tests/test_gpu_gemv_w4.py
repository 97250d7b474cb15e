"""moe_gemv_w4 (products of up to 16 tokens with 4-bit weights) against plain
64-bit references."""
import pytest
import torch

import mixture_experts_router_amd as moe
from mixture_experts_router_amd import device as dev
from few_helpers import Gemv, f64

pytestmark = pytest.mark.gpu

FORMATS = [("mxfp4", 0), ("nvfp4", 0), ("int4", 32), ("int4", 64), ("int4", 128)]
SIZES = [(16, 40, 8192), (16, 9000, 384), (4, 70, 33024), (1, 1, 128), (1, 16, 256), (3, 17, 384), (16, 250, 640), (5, 33, 2816), (2, 1000, 128), (8, 8, 1152),
         (1, 5000, 256), (16, 31, 16384), (7, 2, 4096)]


@pytest.mark.parametrize("fmt,group", FORMATS)
@pytest.mark.parametrize("T,N,K", SIZES)
def test_against_reference(gpu, fmt, group, T, N, K):
    g = Gemv(T, N, K, fmt, group, zeros=fmt == "int4" and N % 2 == 1, bias=N % 3 == 0, y_fp32=T % 2 == 1)
    g.check(g.run(), f"{fmt} {group} {T}x{N}x{K}")


@pytest.mark.parametrize("fmt,group", FORMATS)
@pytest.mark.parametrize("T", range(1, 17))
def test_every_token_count(gpu, fmt, group, T):
    g = Gemv(T, 100, 512, fmt, group, zeros=fmt == "int4", bias=True, y_fp32=True, seed=T)
    g.check(g.run(), f"{fmt} {group} T={T}")


@pytest.mark.parametrize("fmt,group", FORMATS)
@pytest.mark.parametrize("T,N,K", [(1, 2, 128), (4, 34, 512), (16, 630, 1408), (3, 50, 8192)])
def test_geglu(gpu, fmt, group, T, N, K):
    for bias, fp32 in ((False, False), (True, True)):
        g = Gemv(T, N, K, fmt, group, zeros=fmt == "int4" and bias, bias=bias, geglu=True, y_fp32=fp32)
        g.check(g.run(), f"geglu {fmt} {group} {T}x{N}x{K}")


@pytest.mark.parametrize("fmt,group", [("mxfp4", 0), ("nvfp4", 0), ("int4", 32)])
@pytest.mark.parametrize("K", [32, 64, 96, 160, 224, 1120, 2080])
def test_k_that_ends_inside_a_block(gpu, fmt, group, K):
    g = Gemv(3, 40, K, fmt, group, y_fp32=True)
    g.check(g.run(), f"{fmt} K={K}")


@pytest.mark.parametrize("fmt,group", [("mxfp4", 0), ("nvfp4", 0), ("int4", 64)])
def test_strided_rows(gpu, fmt, group):
    """Rows of x and y with gaps: NaN between the rows of x is not read, what
    lies between the rows of y is not written."""
    for T, N, K in ((4, 100, 384), (16, 18, 8192)):
        g = Gemv(T, N, K, fmt, group, pad_x=40, pad_y=3, bias=True)
        g.check(g.run(), f"strided {fmt}")
        g = Gemv(T, N, K, fmt, group, pad_x=8, pad_y=5, geglu=True, y_fp32=True)
        g.check(g.run(), f"strided geglu {fmt}")


@pytest.mark.parametrize("fmt,group", FORMATS)
def test_non_finite_rows_stay_apart(gpu, fmt, group):
    g = Gemv(5, 70, 256, fmt, group)
    good = g.run()
    for bad in (float("nan"), float("inf")):
        g.dx = g.x.cuda()
        g.dx[3, 100] = bad
        y = g.run()
        keep = [0, 1, 2, 4]
        assert torch.equal(y[keep], good[keep])
        assert not torch.isfinite(y[3].float()).all()


@pytest.mark.parametrize("zero", [0, 15, 200])
def test_zero_points(gpu, zero):
    """Zero points at the ends of the code range and past it: code - zero is
    what it says for any byte."""
    g = Gemv(2, 48, 256, "int4", 64, zeros=True, y_fp32=True)
    ref = f64(g.x) @ (g.values + (f64(g.zeros.float()).repeat(64, 1) - zero) * f64(g.scales).repeat(64, 1)).T
    g.zeros.fill_(zero)
    m = abs(f64(g.x)) @ ((15 + zero + 32) * abs(f64(g.scales)).repeat(64, 1)).T
    assert (abs(f64(g.run()) - ref) <= (256 / 32 + 332) * 2.0 ** -24 * m).all()


def test_repeats_and_workspace(gpu):
    """A product whose K is shared by several workgroups: the same bits every
    time, the zeroed prefix zero after every call."""
    g = Gemv(16, 200, 16384, "int4", 128, zeros=True)
    assert moe.gemv_w4_workspace_bytes(g.shape) > 0
    ws = dev.gemv_workspace(g.shape)
    first = g.run(ws)
    g.check(first, "slices")
    for _ in range(30):
        y = g.output()
        g.call(y, ws)
        assert torch.equal(y, first)
        assert not ws[:moe.FEW_ZERO_BYTES].any()


def test_graph_replays(gpu):
    a, b = Gemv(16, 200, 16384, "nvfp4", geglu=True), Gemv(1, 77, 8192, "int4", 32, y_fp32=True)
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    refs, graphs, outs = [a.run(), b.run()], [], []
    for g in (a, b):
        y = g.output()
        g.call(y, ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            g.call(y, ws)
        graphs.append(graph)
        outs.append(y)
    for _ in range(5):
        for g, y, r in zip(graphs, outs, refs):
            y.fill_(7.0)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, r)
            a.run()


def test_overlapping_calls(gpu):
    gs = [Gemv(16, 200, 16384, "int4", 64, seed=1), Gemv(2, 5000, 1024, "mxfp4", seed=2), Gemv(16, 64, 8192, "nvfp4", seed=3)]
    refs, streams = [g.run() for g in gs], [torch.cuda.Stream() for _ in gs]
    wss, outs = [dev.gemv_workspace(g.shape) for g in gs], [[g.output() for _ in range(30)] for g in gs]
    torch.cuda.synchronize()
    for i in range(30):
        for g, ws, st, o in zip(gs, wss, streams, outs):
            g.call(o[i], ws, stream=st)
    torch.cuda.synchronize()
    for o, r in zip(outs, refs):
        assert all(torch.equal(y, r) for y in o)


@pytest.mark.parametrize("fmt,group", [("mxfp4", 0), ("int4", 64)])
def test_long_rows_in_several_rounds(gpu, fmt, group):
    """Token rows that come to the LDS in windows, several rounds of units for
    each workgroup: the first, some middle and the last rows."""
    T, N, K = 16, 35_003, 5504
    gen = torch.Generator().manual_seed(7)
    codes = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device="cuda")
    x = torch.randn(T, K, generator=gen).to(torch.bfloat16)
    if fmt == "int4":
        scales = torch.rand(N, K // group, generator=gen).to(torch.bfloat16)
    else:
        scales = torch.randint(118, 124, (N, K // 32), generator=gen, dtype=torch.uint8)
    y = torch.empty(T, N, dtype=torch.float32, device="cuda")
    s = moe.w4_shape(T, N, K, fmt, group=group, y_fp32=True)
    moe.gemv_w4(s, x.cuda(), codes, scales.cuda(), None, None, y, dev.gemv_workspace(s))
    torch.cuda.synchronize()
    lut = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)
    for at in (0, 12_345, N - 64):
        c = codes[at:at + 64].cpu().long()
        c = torch.stack((c & 15, c >> 4), -1).reshape(64, K)
        if fmt == "int4":
            sc = scales[at:at + 64].double().repeat_interleave(group, 1)
            w, mag, n = sc * (c - 8), sc * (15 + 8 + 32), K / 16
        else:
            w = lut[c] * 2.0 ** (scales[at:at + 64].double().repeat_interleave(32, 1) - 127)
            mag, n = w.abs(), K / 32
        xd = x.double()
        bound = (n + 332) * 2.0 ** -24 * (xd.abs() @ mag.T)
        assert ((y[:, at:at + 64].cpu().double() - xd @ w.T).abs() <= bound).all()


def test_many_rows(gpu):
    """Weight offsets past 2^31 bytes: the last rows of a large matrix."""
    N, K = 1_100_000, 4096
    codes = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device="cuda")
    scales = torch.full((N, K // 32), 120, dtype=torch.uint8, device="cuda")
    x = torch.randn(1, K, device="cuda").to(torch.bfloat16)
    y = torch.empty(1, N, dtype=torch.float32, device="cuda")
    s = moe.w4_shape(1, N, K, "mxfp4", y_fp32=True)
    moe.gemv_w4(s, x, codes, scales, None, None, y, dev.gemv_workspace(s))
    t = moe.w4_shape(1, 64, K, "mxfp4", y_fp32=True)
    for at in (0, (1 << 31) // (K // 2) - 32, N - 64):
        part = torch.empty(1, 64, dtype=torch.float32, device="cuda")
        moe.gemv_w4(t, x, codes[at:at + 64], scales[at:at + 64], None, None, part, dev.gemv_workspace(t))
        torch.cuda.synchronize()
        lut = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)
        c = codes[at:at + 64].cpu().long()
        w = lut[torch.stack((c & 15, c >> 4), -1).reshape(64, K)] * 2.0 ** -7
        xd = x.cpu().double()[0]
        bound = (K / 32 + 332) * 2.0 ** -24 * (w.abs() @ xd.abs())
        assert ((y[0, at:at + 64].cpu().double() - w @ xd).abs() <= bound).all()
        assert ((part[0].cpu().double() - w @ xd).abs() <= bound).all()
