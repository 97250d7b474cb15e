"""moe_forward_few (the whole layer for up to 16 tokens in one launch) against
plain 64-bit references, and against the layer's other entry points."""
import numpy as np
import pytest
import torch

import mixture_experts_router_amd as moe
from mixture_experts_router_amd import device as dev
from few_helpers import Layer, Gemv, f64, BF

pytestmark = pytest.mark.gpu

FMTS = ["bf16", "mxfp4", "nvfp4"]
# odd counts, the smallest sizes, every top-k width, one expert, all experts,
# a K that ends inside a 128-wide block, rows too long for the LDS
SHAPES = {
    "one-token": dict(T=1, H=256, E=8, k=2, I=128),
    "least": dict(T=1, H=64, E=1, k=1, I=64),
    "odd-batch": dict(T=5, H=448, E=12, k=3, I=192),
    "full-batch": dict(T=16, H=512, E=24, k=4, I=128),
    "half-blocks": dict(T=3, H=320, E=6, k=2, I=448, bias=True),
    "every-expert": dict(T=7, H=128, E=6, k=6, I=64),
    "one-expert": dict(T=9, H=192, E=1, k=1, I=320, bias=True),
    "experts-100": dict(T=4, H=128, E=100, k=5, I=64),
    "experts-200": dict(T=4, H=128, E=200, k=9, I=64, bias=True),
    "experts-500": dict(T=2, H=64, E=500, k=7, I=64),
    "experts-1024": dict(T=16, H=64, E=1024, k=32, I=64),
    "mlp": dict(T=6, H=384, E=8, k=2, I=128, I_sh=320),
    "mlp-longer-than-pieces": dict(T=2, H=256, E=4, k=1, I=64, I_sh=704, bias=True),
    "mlp-shorter": dict(T=16, H=192, E=16, k=4, I=256, I_sh=64),
    "long-rows": dict(T=16, H=4160, E=4, k=2, I=64),
    "long-rows-one": dict(T=1, H=8256, E=3, k=1, I=64, I_sh=64),
    "long-rows-many-units": dict(T=16, H=3264, E=9, k=9, I=2112, I_sh=192),
    "pieces": dict(T=16, H=128, E=4, k=2, I=1600, I_sh=1984),
    "pieces-of-column-blocks": dict(T=8, H=64, E=12, k=2, I=2112, I_sh=704),
    "passes": dict(T=16, H=64, E=32, k=32, I=6400),
    "fewest-items": dict(T=16, H=64, E=2, k=2, I=64),
}


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("name", list(SHAPES))
def test_against_reference(gpu, name, fmt):
    l = Layer(**SHAPES[name], fmt=fmt)
    l.check(l.run(), f"{name} {fmt}")


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T", range(1, 17))
def test_every_token_count(gpu, fmt, T):
    l = Layer(T, 320, 10, 3, 192, I_sh=128, fmt=fmt, seed=T)
    l.check(l.run(), f"T={T} {fmt}")


@pytest.mark.parametrize("fmt", FMTS)
def test_model_width(gpu, fmt):
    """The model's rows (2816, 704, dense 2112) with fewer experts."""
    l = Layer(8, 2816, 10, 4, 704, I_sh=2112, fmt=fmt)
    l.check(l.run(), f"model width {fmt}")


@pytest.mark.parametrize("T,H", [(t, h) for t in (3, 6, 11, 16) for h in (512, 2048, 2816, 5120)])
@pytest.mark.parametrize("fmt", FMTS)
def test_every_ring(gpu, fmt, T, H):
    """Token rows that leave the rings less and less of the LDS, then none."""
    l = Layer(T, H, 4, 2, 128, fmt=fmt, seed=H)
    l.check(l.run(), f"T={T} H={H} {fmt}")


@pytest.mark.parametrize("T", [1, 4, 16])
def test_routing_is_bitwise_moe_route(gpu, T):
    """ids and weights are the bits of moe_route, also where logits tie and
    for values on no grid."""
    g = torch.Generator().manual_seed(T)
    l = Layer(T, 704, 130, 8, 64, bias=True)
    l.x = torch.randn(T, 704, generator=g).to(torch.bfloat16)
    l.wr = (0.02 * torch.randn(130, 704, generator=g)).to(torch.bfloat16)
    l.wr[40:60] = l.wr[20:40]                # twenty pairs of equal logits
    l.bias[40:60] = l.bias[20:40]
    l.upload()
    out, ids, w = l.run()
    logits = torch.empty(T, 130, device="cuda")
    rids, rw = torch.empty_like(ids), torch.empty_like(w)
    rws = torch.empty(max(1, moe.route_workspace_bytes(l.shape)), dtype=torch.uint8, device="cuda")
    moe.route(l.shape, l.dx, l.dwr, l.db, logits, rids, rw, ws=rws)
    torch.cuda.synchronize()
    assert torch.equal(ids, rids) and torch.equal(w.view(torch.int32), rw.view(torch.int32))


@pytest.mark.parametrize("fmt", FMTS)
def test_near_moe_forward(gpu, fmt):
    """moe_forward rounds each expert's row to bf16 besides: the two differ by
    at most that and their own roundings, 3 * 2^-8 in rms over many values."""
    l = Layer(8, 512, 16, 4, 192, fmt=fmt, seed=3)
    out, ids, w = l.run()
    o2, i2, w2 = l.outputs()
    moe.forward(l.shape, l.dx, l.dwr, None, l.gu.arg, l.gu.scales, l.d.arg, l.d.scales, o2, i2, w2,
                dev.workspace(l.shape))
    torch.cuda.synchronize()
    assert torch.equal(ids, i2) and torch.equal(w, w2)
    a, b = f64(out), f64(o2)
    assert np.linalg.norm(a - b) <= 3 * BF * np.linalg.norm(b)


def test_optional_outputs_and_repeats(gpu):
    """Without ids and weights; the same bits every time; the zeroed prefix of
    the workspace is zero after every call."""
    l = Layer(7, 384, 12, 4, 128, I_sh=192, fmt="mxfp4").upload()
    ws = dev.few_workspace(l.shape, I_sh=192)
    first = l.run(ws)
    for _ in range(20):
        out, ids, w = l.outputs()
        l.call(out, ids, w, ws)
        assert torch.equal(out, first[0]) and torch.equal(ids, first[1]) and torch.equal(w, first[2])
        assert not ws[:moe.FEW_ZERO_BYTES].any()
    out = l.outputs()[0]
    l.call(out, None, None, ws)
    torch.cuda.synchronize()
    assert torch.equal(out, first[0])


def test_workspace_shared_between_shapes(gpu):
    """One workspace, the largest needed, for layers of several shapes and a
    4-bit product, one after another without waiting."""
    ls = [Layer(T, H, E, k, I, I_sh, fmt).upload() for T, H, E, k, I, I_sh, fmt in
          [(16, 512, 24, 4, 128, 0, "bf16"), (1, 64, 1, 1, 64, 0, "nvfp4"), (3, 320, 40, 9, 192, 64, "mxfp4")]]
    g = Gemv(16, 300, 8192, "int4", 128)
    need = max([moe.few_workspace_bytes(l.shape, l.I_sh) for l in ls] + [moe.gemv_w4_workspace_bytes(g.shape)])
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    alone = [l.run() for l in ls]
    y = g.run()
    outs = [[l.outputs() for l in ls] for _ in range(5)]
    ys = [g.output() for _ in range(5)]
    for o, yy in zip(outs, ys):
        for l, r in zip(ls, o):
            l.call(*r, ws)
        g.call(yy, ws)
    torch.cuda.synchronize()
    for o, yy in zip(outs, ys):
        for a, r in zip(alone, o):
            assert all(torch.equal(u, v) for u, v in zip(a, r))
        assert torch.equal(yy, y)


def test_non_finite_rows_stay_apart(gpu):
    """NaN and infinities in one token's x leave the other tokens' bits alone."""
    for fmt in FMTS:
        l = Layer(6, 256, 8, 2, 128, I_sh=64, fmt=fmt).upload()
        good = l.run()
        for bad in (float("nan"), float("inf"), float("-inf")):
            l.dx = l.x.cuda()
            l.dx[2, 17] = bad
            out, ids, w = l.run()
            keep = [0, 1, 3, 4, 5]
            assert torch.equal(out[keep], good[0][keep]) and torch.equal(ids[keep], good[1][keep])
            assert not torch.isfinite(out[2].float()).any()


def test_zero_input(gpu):
    l = Layer(4, 256, 8, 3, 64).upload()
    l.dx = torch.zeros_like(l.x).cuda()
    out, ids, w = l.run()
    assert not out.any() and (ids.cpu() == torch.arange(3, dtype=torch.int32)).all()
    assert torch.allclose(w, torch.full_like(w, 1 / 3), rtol=2.0 ** -23, atol=0)


@pytest.mark.parametrize("fmt", FMTS)
def test_graph_replays(gpu, fmt):
    """Two captured calls of different shapes that share a workspace, replayed
    in turn with eager work on other streams and workspaces in between."""
    a = Layer(8, 512, 32, 4, 128, I_sh=128, fmt=fmt).upload()
    b = Layer(1, 320, 10, 3, 192, fmt=fmt).upload()
    ws = torch.zeros(max(moe.few_workspace_bytes(a.shape, 128), moe.few_workspace_bytes(b.shape)), dtype=torch.uint8,
                     device="cuda")
    ra, rb = a.run(), b.run()
    graphs, outs = [], []
    for l in (a, b):
        o = l.outputs()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            l.call(*o, ws)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            l.call(*o, ws)
        graphs.append(g)
        outs.append(o)
    for _ in range(5):
        for g, o, r in zip(graphs, outs, (ra, rb)):
            for t in o:
                t.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(u, v) for u, v in zip(o, r))
            a.run()


def test_overlapping_calls(gpu):
    """Calls on four streams at once, each with its own workspace: every one
    ends, with the bits it has alone."""
    ls = [Layer(T, 1024, 32, 4, 256, I_sh=256, fmt=f, seed=T).upload() for T, f in
          [(16, "bf16"), (1, "mxfp4"), (8, "nvfp4"), (5, "bf16")]]
    refs = [l.run() for l in ls]
    wss = [dev.few_workspace(l.shape, I_sh=256) for l in ls]
    streams = [torch.cuda.Stream() for _ in ls]
    outs = [[l.outputs() for _ in range(30)] for l in ls]
    torch.cuda.synchronize()
    for i in range(30):
        for l, ws, st, o in zip(ls, wss, streams, outs):
            l.call(*o[i], ws, stream=st)
    torch.cuda.synchronize()
    for o, r in zip(outs, refs):
        for one in o:
            assert all(torch.equal(u, v) for u, v in zip(one, r))


def test_decode_block(gpu):
    """The block's two halves as a decode step runs them: the experts by
    moe_forward_few, the dense MLP next to them by two 4-bit products, against
    the layer with the MLP inside it."""
    l = Layer(4, 512, 16, 4, 128, I_sh=320, fmt="mxfp4").upload()
    whole = l.run()[0]
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    h = torch.empty(4, 320, dtype=torch.bfloat16, device="cuda")
    y = torch.empty(4, 512, dtype=torch.float32, device="cuda")
    out = l.outputs()[0]
    moe.forward_few(l.shape, l.dx, l.dwr, None, l.gu.arg, l.gu.scales, l.d.arg, l.d.scales, out, None, None, ws)
    moe.gemv_w4(moe.w4_shape(4, 640, 512, "mxfp4", geglu=True), l.dx, l.sgu.arg, l.sgu.scales, None, None, h, ws)
    moe.gemv_w4(moe.w4_shape(4, 512, 320, "mxfp4", y_fp32=True), h, l.sd.arg, l.sd.scales, None, None, y, ws)
    both = f64(out) + f64(y)
    ref, bound, _, _ = l.reference()
    # the experts' half is rounded once more than inside the layer
    assert (np.abs(both - ref) <= bound + BF * np.abs(f64(out))).all()
    assert np.linalg.norm(both - f64(whole)) <= 2 * BF * np.linalg.norm(ref)
