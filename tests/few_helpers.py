"""Inputs and plain 64-bit references of the few-token operators
(moe_forward_few, moe_gemv_w4), with elementwise error bounds that follow from
the arithmetic.

Bounds.  A sum of K fp32 products on the matrix cores is off by at most
(K/32 + 32) 2^-24 times the sum of the products' magnitudes (one rounding per
32-wide step and at most 32 inside one; products of bf16 values are exact);
the later fp32 additions (waves, slices: at most 64 of them, experts in at most
sixteen segments each, bias) add 2^-24 of the running magnitude each.  INT4
groups are added one by one, their sums and their offsets: K/32 more.    Rounding to bf16 is off by at most
2^-8 of the value.  gelu_tanh has slope at most 1.13 and is evaluated to
within 2^-19 of |z| (exp of an argument of magnitude up to 88 carries that
argument's rounding, 88 * 2^-24 < 2^-17.5, only where the result is below
2^-120 |z|; otherwise a few fp32 ulps)."""
import math

import numpy as np
import torch

import mixture_experts_router_amd as moe
from mixture_experts_router_amd import device as dev

U = 2.0 ** -24
BF = 2.0 ** -8
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=np.float64)


def bf16(a):
    """fp64 array rounded to bf16 values."""
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16)


def f64(t):
    return t.detach().cpu().double().numpy()


def gelu(z):
    return 0.5 * z * (1 + np.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))


def pack(codes):
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def e4m3(code):
    e, m = (code.astype(np.int64) >> 3) & 15, code.astype(np.int64) & 7
    v = np.where(e == 0, m * 2.0 ** -9, np.ldexp(1 + m / 8.0, e - 7))
    return np.where(code & 0x80, -v, v)


class Weights:
    """E random matrices [E][rows][K] of a format: `arg` and `scales` are the
    device arguments, `values` the fp64 matrices."""

    def __init__(self, rng, fmt, E, rows, K):
        self.scales = None
        if fmt == "bf16":
            w = bf16(0.05 * rng.standard_normal((E, rows, K)))
            self.arg, self.values = w.cuda(), f64(w)
            return
        codes = rng.integers(0, 16, (E, rows, K), dtype=np.uint8)
        self.arg = torch.from_numpy(pack(codes)).cuda()
        if fmt == "mxfp4":
            s = rng.integers(118, 124, (E, rows, K // 32), dtype=np.uint8)
            self.scales = torch.from_numpy(s).cuda()
            f = np.ldexp(1.0, s.astype(np.int64) - 127)
            self.values = E2M1[codes] * np.repeat(f, 32, -1)
        else:
            s = rng.integers(0x20, 0x50, (E, rows, K // 16), dtype=np.uint8)   # E4M3 0.125 .. 8, both ends of it odd
            s[rng.random(s.shape) < 0.05] = 0
            m = rng.uniform(0.004, 0.02, E).astype(np.float32)
            self.scales = torch.from_numpy(moe.nvfp4_scale_buffer(m, s)).cuda()
            self.values = E2M1[codes] * np.repeat(e4m3(s), 16, -1) * m.astype(np.float64)[:, None, None]


class Layer:
    """Inputs of one layer call.  The router's operands lie on grids on which
    every fp32 sum of a logit is exact, so the ranking is unambiguous."""

    def __init__(self, T, H, E, k, I, I_sh=0, fmt="bf16", bias=False, seed=0):
        rng = np.random.default_rng([seed, T, H, E, k, I, I_sh])
        self.T, self.H, self.E, self.k, self.I, self.I_sh, self.fmt = T, H, E, k, I, I_sh, fmt
        self.x = bf16(np.round(16 * rng.standard_normal((T, H))) / 16)
        self.wr = bf16(np.round(2048 * 0.02 * rng.standard_normal((E, H))) / 2048)
        self.bias = torch.from_numpy((np.round(4096 * rng.standard_normal(E)) / 4096).astype(np.float32)) if bias else None
        self.gu, self.d = Weights(rng, fmt, E, 2 * I, H), Weights(rng, fmt, E, H, I)
        if I_sh:
            self.sgu, self.sd = Weights(rng, fmt, 1, 2 * I_sh, H), Weights(rng, fmt, 1, H, I_sh)
        self.shape = moe.shape(T, H, E, k, I, mxfp4=fmt == "mxfp4", nvfp4=fmt == "nvfp4")

    def outputs(self):
        return (torch.full((self.T, self.H), 7.0, dtype=torch.bfloat16, device="cuda"),
                torch.full((self.T, self.k), -1, dtype=torch.int32, device="cuda"),
                torch.full((self.T, self.k), 7.0, dtype=torch.float32, device="cuda"))

    def upload(self):
        self.dx, self.dwr = self.x.cuda(), self.wr.cuda()
        self.db = self.bias.cuda() if self.bias is not None else None
        return self

    def call(self, out, ids, w, ws, stream=None):
        sh = (self.sgu.arg, self.sgu.scales, self.sd.arg, self.sd.scales) if self.I_sh else (None,) * 4
        moe.forward_few(self.shape, self.dx, self.dwr, self.db, self.gu.arg, self.gu.scales, self.d.arg, self.d.scales,
                        out, ids, w, ws, self.I_sh, *sh, stream=stream)

    def run(self, ws=None):
        if not hasattr(self, "dx"):
            self.upload()
        o = self.outputs()
        self.call(*o, ws if ws is not None else dev.few_workspace(self.shape, I_sh=self.I_sh))
        torch.cuda.synchronize()
        return o

    def reference(self):
        """(out, bound of its error, ids, w) in 64 bits from the formulas."""
        x, T, k = f64(self.x), self.T, self.k
        L = x @ f64(self.wr).T + (f64(self.bias) if self.bias is not None else 0.0)
        ids = np.stack([np.lexsort((np.arange(self.E), -L[t]))[:k] for t in range(T)])
        top = np.take_along_axis(L, ids, 1)
        w = np.exp(top - top[:, :1])
        w /= w.sum(1, keepdims=True)
        out, err, mag = np.zeros((T, self.H)), np.zeros((T, self.H)), np.zeros((T, self.H))

        def mlp(t, wt, gu, d, I):
            cH, cI = (self.H / 32 + 32 + 64) * U, (I / 32 + 32 + 64) * U
            p, m = gu @ x[t], np.abs(gu) @ np.abs(x[t])
            g, u = p[:I], p[I:]
            h = gelu(g) * u
            dg = cH * m[:I] * 1.13 + 2.0 ** -19 * np.abs(g)
            dh = dg * (np.abs(u) + cH * m[I:]) + np.abs(gelu(g)) * cH * m[I:]
            dh = dh + BF * (np.abs(h) + dh) + 2.0 ** -133    # rounded to bf16 (the least subnormal's half step at the end)
            s = np.abs(d) @ np.abs(h)
            out[t] += wt * (d @ h)
            err[t] += wt * (np.abs(d) @ dh + cI * s) + 4 * U * wt * s
            mag[t] += wt * s

        for t in range(T):
            for j in range(k):
                mlp(t, w[t, j], self.gu.values[ids[t, j]], self.d.values[ids[t, j]], self.I)
            if self.I_sh:
                mlp(t, 1.0, self.sgu.values[0], self.sd.values[0], self.I_sh)
        err = err + (64 + 16 * k) * U * mag
        return out, err + BF * (np.abs(out) + err) + 2.0 ** -133, ids, w

    def check(self, got, label=""):
        out, ids, w = got
        ref, bound, rids, rw = self.reference()
        assert (ids.cpu().numpy() == rids).all(), f"{label}: ids"
        # weights: exp to a few ulps of fp32, the argument exact, k additions and a division
        assert np.abs(f64(w) - rw).max() <= (self.k + 8) * U, f"{label}: weights"
        d = np.abs(f64(out) - ref)
        n = np.linalg.norm(ref)
        rel = np.linalg.norm(d) / n if n else np.linalg.norm(d)
        print(f"{label}: rel_l2 {rel:.2e}, largest error over its bound {(d / bound).max():.3f}", flush=True)
        assert (d <= bound).all(), f"{label}: {(d / bound).max()} of the bound"
        # two roundings to bf16, each with an rms of at most 2^-8 / sqrt(3) of
        # its value: sqrt(2/3) 2^-8 = 0.82 * 2^-8 over many values
        if out.numel() >= 2048:
            assert rel <= BF, f"{label}: rel {rel}"


class Gemv:
    """Inputs of one 4-bit product; ldx and ldy pad the rows with values that
    must be neither read into a result nor written."""

    def __init__(self, T, N, K, fmt, group=0, zeros=False, bias=False, geglu=False, y_fp32=False, pad_x=0, pad_y=0,
                 seed=0):
        rng = np.random.default_rng([seed, T, N, K, group])
        self.T, self.N, self.K, self.fmt, self.geglu, self.y_fp32, self.group = T, N, K, fmt, geglu, y_fp32, group
        self.outs = N // 2 if geglu else N
        self.ldx, self.ldy = K + pad_x, self.outs + pad_y
        x = np.full((T, self.ldx), np.nan)
        x[:, :K] = rng.standard_normal((T, K))
        self.x = bf16(x)
        self.bias = torch.from_numpy(rng.standard_normal(N).astype(np.float32)) if bias else None
        self.zeros = None
        if fmt == "int4":
            codes = rng.integers(0, 16, (N, K), dtype=np.uint8)
            s = bf16(rng.uniform(0.01, 0.03, (N, K // group)) * rng.choice([-1, 1], (N, K // group)))
            z = rng.integers(0, 16, (N, K // group), dtype=np.uint8) if zeros else np.full((N, K // group), 8, np.uint8)
            self.zeros = torch.from_numpy(z).cuda() if zeros else None
            self.w, self.scales = torch.from_numpy(pack(codes)).cuda(), s.cuda()
            rs, rz = np.repeat(f64(s), group, 1), np.repeat(z.astype(np.float64), group, 1)
            self.values = (codes - rz) * rs
            self.mags = (codes + rz + 32) * np.abs(rs)     # of the terms that are added and subtracted
        else:
            w = Weights(rng, fmt, 1, N, K)
            self.w, self.scales, self.values = w.arg, w.scales, w.values[0]
            self.mags = np.abs(self.values)
        self.shape = moe.w4_shape(T, N, K, fmt, group, geglu, y_fp32, self.ldx if pad_x else 0, self.ldy if pad_y else 0)
        self.dx = self.x.cuda()[:, :K]
        self.db = self.bias.cuda() if bias else None
        self.pad_x, self.pad_y = pad_x, pad_y

    def output(self):
        return torch.full((self.T, self.ldy), 7.0, dtype=torch.float32 if self.y_fp32 else torch.bfloat16, device="cuda")

    def call(self, y, ws, stream=None):
        moe.gemv_w4(self.shape, self.dx, self.w, self.scales, self.zeros, self.db, y[:, :self.outs], ws, stream=stream)

    def run(self, ws=None):
        y = self.output()
        self.call(y, ws if ws is not None else dev.gemv_workspace(self.shape))
        torch.cuda.synchronize()
        return y

    def reference(self):
        x = f64(self.x)[:, :self.K]
        # 256 slices, eight waves, the bias
        c = (self.K / (16 if self.fmt == "int4" else 32) + 32 + 300) * U
        y, m = x @ self.values.T, np.abs(x) @ self.mags.T
        if self.bias is not None:
            y, m = y + f64(self.bias), m + np.abs(f64(self.bias))
        err = c * m
        if self.geglu:
            g, u, eg, eu = y[:, :self.outs], y[:, self.outs:], err[:, :self.outs], err[:, self.outs:]
            y = gelu(g) * u
            eg = 1.13 * eg + 2.0 ** -19 * np.abs(g)
            err = eg * (np.abs(u) + eu) + np.abs(gelu(g)) * eu
        return y, err + (U if self.y_fp32 else BF) * (np.abs(y) + err) + 2.0 ** -133

    def check(self, got, label=""):
        y = f64(got)
        assert (y[:, self.outs:] == 7.0).all(), f"{label}: wrote past the row"
        ref, bound = self.reference()
        d = np.abs(y[:, :self.outs] - ref)
        print(f"{label}: largest error over its bound {(d / bound).max():.3f}", flush=True)
        assert (d <= bound).all(), f"{label}: {(d / bound).max()} of the bound"
