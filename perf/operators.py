"""Cases of the few-token operators, with their plain forms in elementary torch operations.

Two operators of a decode step:

- "layer": the whole MoE layer for up to 16 tokens (router, top-k softmax, gate/up with GELU-tanh GEGLU,
  down, weighted sum), optionally with the block's dense GEGLU MLP added, as moe_forward_few computes it.
- "gemv": a matrix-vector product of up to 16 tokens with a 4-bit weight that has a scale per group
  (MXFP4, NVFP4 or INT4 with optional zero points), with a bias or a GEGLU epilogue, as moe_gemv_w4 computes it.

`run` computes them in fp32 from elementary operations, or (`own`) calls the library.

The router's operands lie on grids (x on multiples of 2^-4, the router weight on multiples of 2^-11, the
bias on multiples of 2^-12) on which every fp32 sum of a logit is exact in any order, so that equal and
nearly equal logits are ranked alike by every way of computing them.
"""
import math

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
WORKSPACE = 32 << 20   # one zero-filled workspace, larger than any case needs, as a serving loop keeps it


# ---------------------------------------------------------------- cases
def listed():
    layer = dict(op="layer", H=2816, E=128, k=8, I=704, I_sh=0, fmt="bf16", bias=False)
    gemv = dict(op="gemv", group=0, zeros=False, bias=False, geglu=False, y="bf16")
    return [
        # the smallest call of the layer: a short speculative step of a small model
        dict(layer, name="layer tiny", T=3, H=256, E=8, k=2, I=128),
        # one sequence decoding, expert weights in each format
        dict(layer, name="layer bf16 1", T=1),
        dict(layer, name="layer mxfp4 1", T=1, fmt="mxfp4"),
        # a decode batch of eight sequences
        dict(layer, name="layer bf16 8", T=8),
        dict(layer, name="layer mxfp4 8", T=8, fmt="mxfp4"),
        # an odd batch with a router bias
        dict(layer, name="layer nvfp4 5", T=5, fmt="nvfp4", bias=True),
        # the largest batch, with the dense MLP that every block runs next to the experts
        dict(layer, name="layer bf16 16 mlp", T=16, I_sh=2112),
        # one token through a projection back to the hidden size: the smallest product
        dict(gemv, name="gemv int4 1", T=1, N=2816, K=2112, fmt="int4", group=32),
        # one token through the dense MLP's gate/up with its activation
        dict(gemv, name="gemv mxfp4 geglu 1", T=1, N=4224, K=2816, fmt="mxfp4", geglu=True),
        # a small batch, an odd number of outputs, zero points and a bias
        dict(gemv, name="gemv int4 8 odd", T=8, N=5001, K=2816, fmt="int4", group=128, zeros=True, bias=True),
        # a wide square projection
        dict(gemv, name="gemv nvfp4 4", T=4, N=8192, K=8192, fmt="nvfp4"),
        # logits over a large vocabulary in fp32, the widest product
        dict(gemv, name="gemv int4 16 head", T=16, N=131072, K=2816, fmt="int4", group=64, y="fp32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _layer_weights(c):
    return c["E"] * 3 * c["I"] * c["H"]


def draw(rng):
    T = rng.choice((1, 1, 2, 3, 4, 5, 6, 7, 8, 9, 11, 13, 15, 16))
    if rng.random() < 0.5:
        most = 128 * 3 * 704 * 2816
        while True:
            E = _log(rng, 2, 256)
            c = dict(op="layer", T=T, H=64 * _log(rng, 2, 80), E=E, k=rng.randint(1, min(E, 10)), I=64 * _log(rng, 1, 32),
                     I_sh=rng.choice((0, 0, 64 * _log(rng, 1, 40))), fmt=rng.choice(("bf16", "mxfp4", "nvfp4")),
                     bias=rng.random() < 0.3)
            touched = c["T"] * c["k"] * 3 * c["I"] * c["H"]
            if _layer_weights(c) <= most and touched <= 16 * 8 * 3 * 704 * 2816:
                return c
    fmt = rng.choice(("mxfp4", "nvfp4", "int4", "int4"))
    group = rng.choice((32, 64, 128)) if fmt == "int4" else 0
    unit = group or 32
    while True:
        geglu = rng.random() < 0.25
        N, K = _log(rng, 1, 131072), unit * _log(rng, 1, 16384 // unit)
        N += geglu and N % 2
        if N * K <= 131072 * 2816:
            return dict(op="gemv", T=T, N=N, K=K, fmt=fmt, group=group, zeros=fmt == "int4" and rng.random() < 0.5,
                        bias=rng.random() < 0.5, geglu=geglu, y=rng.choice(("bf16", "fp32")))


# ---------------------------------------------------------------- inputs
def _normal(gen, *shape):
    return torch.randn(*shape, device="cuda", generator=gen)


def _pack(codes):
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).contiguous()


def _e2m1_codes(v):
    """Nearest E2M1 code of each value, saturating at 6."""
    edges = torch.tensor((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0), device=v.device)
    return torch.bucketize(v.abs(), edges).to(torch.uint8) | ((v < 0).to(torch.uint8) << 3)


def _quantised(w, fmt, group, zeros):
    """Codes (two a byte, the even index low), scales and zero points of fp32 rows [rows][K]; for NVFP4 the
    matrix's fp32 scale as well."""
    rows, K = w.shape
    if fmt == "mxfp4":
        b = w.reshape(rows, K // 32, 32)
        e = torch.floor(torch.log2(b.abs().amax(-1, keepdim=True).clamp_min(1e-30))) - 2
        return _pack(_e2m1_codes(b / torch.exp2(e)).reshape(rows, K)), (e[..., 0] + 127).to(torch.uint8), None, None
    if fmt == "nvfp4":
        b = w.reshape(rows, K // 16, 16)
        g = w.abs().amax() / (6 * 448)
        s = (b.abs().amax(-1, keepdim=True) / (6 * g)).to(torch.float8_e4m3fn)
        step = (s.float() * g).clamp_min(1e-30)
        return _pack(_e2m1_codes(b / step).reshape(rows, K)), s[..., 0].view(torch.uint8), None, g
    b = w.reshape(rows, K // group, group)
    if zeros:
        lo, hi = b.amin(-1, keepdim=True).clamp_max(0), b.amax(-1, keepdim=True).clamp_min(0)
        s = ((hi - lo) / 15).clamp_min(1e-30).to(torch.bfloat16)
        z = torch.round(-lo / s.float()).clamp(0, 15)
    else:
        s = (b.abs().amax(-1, keepdim=True) / 7.5).clamp_min(1e-30).to(torch.bfloat16)
        z = torch.full_like(b[..., :1], 8)
    codes = (torch.round(b / s.float()) + z).clamp(0, 15).to(torch.uint8).reshape(rows, K)
    return _pack(codes), s[..., 0].contiguous(), z[..., 0].to(torch.uint8) if zeros else None, None


def _expert_weights(gen, E, rows, K, fmt):
    """E matrices of normal weights (sigma 0.02) in the library's layout: (weights or codes, scale buffer or None)."""
    if fmt == "bf16":
        w = torch.empty(E, rows, K, dtype=torch.bfloat16, device="cuda")
        for e in range(E):
            w[e] = 0.02 * _normal(gen, rows, K)
        return w, None
    codes = torch.empty(E, rows, K // 2, dtype=torch.uint8, device="cuda")
    n = K // 32 if fmt == "mxfp4" else K // 16
    scales = torch.empty(E, rows, n, dtype=torch.uint8, device="cuda")
    matrix = torch.ones(E, dtype=torch.float32, device="cuda")
    for e in range(E):
        codes[e], scales[e], _, g = _quantised(0.02 * _normal(gen, rows, K), fmt, 0, False)
        if g is not None:
            matrix[e] = g
    return codes, (scales if fmt == "mxfp4" else _nv_buffer(matrix, scales))


def _nv_buffer(matrix, scales):
    """An NVFP4 scale argument: the fp32 matrix scales (and one unused input scale), padded to 256 bytes,
    then the E4M3 codes."""
    E = matrix.numel()
    head = torch.zeros(_nv_header(E) // 4, dtype=torch.float32, device="cuda")
    head[:E] = matrix
    head[E] = 1
    return torch.cat((head.view(torch.uint8), scales.reshape(-1)))


def _nv_header(E):
    return ((E + 1) * 4 + 255) // 256 * 256


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    c, s = case, {"case": case, "ws": torch.zeros(WORKSPACE, dtype=torch.uint8, device="cuda")}
    if c["op"] == "gemv":
        T, N, K = c["T"], c["N"], c["K"]
        s["x"] = _normal(gen, T, K).to(torch.bfloat16)
        codes = torch.empty(N, K // 2, dtype=torch.uint8, device="cuda")
        n = K // (c["group"] or {"mxfp4": 32, "nvfp4": 16}[c["fmt"]])
        scales = torch.empty(N, n, dtype=torch.bfloat16 if c["fmt"] == "int4" else torch.uint8, device="cuda")
        z = torch.empty(N, n, dtype=torch.uint8, device="cuda") if c["zeros"] else None
        # rows in runs that fit; one scale for the whole NVFP4 matrix
        for r in range(0, N, 8192):
            w = 0.02 * _normal(gen, min(8192, N - r), K)
            if c["fmt"] == "nvfp4" and r == 0:
                s["matrix"] = w.abs().amax() / (6 * 448)
            if c["fmt"] == "nvfp4":
                w = w.clamp(-6 * 448 * s["matrix"], 6 * 448 * s["matrix"])
                b = w.reshape(-1, K // 16, 16)
                e = (b.abs().amax(-1, keepdim=True) / (6 * s["matrix"])).to(torch.float8_e4m3fn)
                codes[r:r + 8192] = _pack(_e2m1_codes(b / (e.float() * s["matrix"]).clamp_min(1e-30)).reshape(-1, K))
                scales[r:r + 8192] = e[..., 0].view(torch.uint8)
                continue
            codes[r:r + 8192], scales[r:r + 8192], zr, _ = _quantised(w, c["fmt"], c["group"], c["zeros"])
            if z is not None:
                z[r:r + 8192] = zr
        s["w"], s["zeros"] = codes, z
        s["scales"] = _nv_buffer(s["matrix"].reshape(1), scales) if c["fmt"] == "nvfp4" else scales
        s["bias"] = 0.1 * _normal(gen, N) if c["bias"] else None
        s["y"] = torch.empty(T, N // 2 if c["geglu"] else N, dtype=torch.bfloat16 if c["y"] == "bf16" else torch.float32, device="cuda")
        return s
    T, H, E, k, I, I_sh, fmt = (c[n] for n in ("T", "H", "E", "k", "I", "I_sh", "fmt"))
    s["x"] = (torch.round(16 * _normal(gen, T, H)) / 16).to(torch.bfloat16)
    s["w_router"] = (torch.round(2048 * 0.02 * _normal(gen, E, H)) / 2048).to(torch.bfloat16)
    s["bias"] = torch.round(4096 * 0.5 * _normal(gen, E)) / 4096 if c["bias"] else None
    s["w_gu"], s["gu_s"] = _expert_weights(gen, E, 2 * I, H, fmt)
    s["w_d"], s["d_s"] = _expert_weights(gen, E, H, I, fmt)
    if I_sh:
        s["sh_gu"], s["sh_gu_s"] = _expert_weights(gen, 1, 2 * I_sh, H, fmt)
        s["sh_d"], s["sh_d_s"] = _expert_weights(gen, 1, H, I_sh, fmt)
    s["out"] = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    s["ids"] = torch.empty(T, k, dtype=torch.int32, device="cuda")
    s["w"] = torch.empty(T, k, dtype=torch.float32, device="cuda")
    return s


# ---------------------------------------------------------------- plain forms (fp32, elementary operations)
def _codes(packed):
    return torch.stack((packed & 15, packed >> 4), -1).reshape(*packed.shape[:-1], -1).long()


def _expert_values(s, w, buf, e, rows, K):
    """fp32 matrices [..., rows, K] of the experts `e` (an index tensor)."""
    fmt = s["case"]["fmt"]
    if fmt == "bf16":
        return w[e].float()
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device="cuda")
    v = lut[_codes(w[e])]
    if fmt == "mxfp4":
        return (v.unflatten(-1, (K // 32, 32)) * torch.exp2(buf[e].float() - 127).unsqueeze(-1)).flatten(-2)
    E = w.shape[0]
    block = buf[_nv_header(E):].view(torch.float8_e4m3fn).reshape(E, rows, K // 16)[e].float()
    matrix = buf[:4 * E].view(torch.float32)[e][..., None, None, None]
    return (v.unflatten(-1, (K // 16, 16)) * block.unsqueeze(-1) * matrix).flatten(-2)


def _gelu_tanh(z):
    return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))


def _mlp(gu, d, x):
    """(gelu_tanh(x gate^T) * (x up^T)) down^T for matrices [..., 2I, H], [..., H, I] and vectors x [..., H]."""
    g, u = torch.matmul(gu, x.unsqueeze(-1)).squeeze(-1).chunk(2, -1)
    return torch.matmul(d, (_gelu_tanh(g) * u).unsqueeze(-1)).squeeze(-1)


def _plain_layer(s):
    c = s["case"]
    H, I, I_sh, k = c["H"], c["I"], c["I_sh"], c["k"]
    x = s["x"].float()
    logits = torch.matmul(x, s["w_router"].float().t())
    if s["bias"] is not None:
        logits = logits + s["bias"]
    top, ids = torch.sort(logits, dim=-1, descending=True, stable=True)   # equal logits: the lower expert first
    top, ids = top[:, :k], ids[:, :k]
    w = torch.exp(top - top[:, :1])
    w = w / w.sum(-1, keepdim=True)
    gu = _expert_values(s, s["w_gu"], s["gu_s"], ids, 2 * I, H)
    d = _expert_values(s, s["w_d"], s["d_s"], ids, H, I)
    out = (_mlp(gu, d, x.unsqueeze(1).expand(-1, k, -1)) * w.unsqueeze(-1)).sum(1)
    if I_sh:
        one = torch.zeros(1, dtype=torch.long, device="cuda")
        gu = _expert_values(s, s["sh_gu"], s["sh_gu_s"], one, 2 * I_sh, H)
        d = _expert_values(s, s["sh_d"], s["sh_d_s"], one, H, I_sh)
        out = out + _mlp(gu, d, x)
    return out.to(torch.bfloat16), ids.to(torch.int32), w


def _gemv_values(s):
    c = s["case"]
    N, K, fmt = c["N"], c["K"], c["fmt"]
    if fmt == "int4":
        zero = s["zeros"].float().unsqueeze(-1) if s["zeros"] is not None else 8.0
        v = _codes(s["w"]).float().unflatten(-1, (K // c["group"], c["group"]))
        return ((v - zero) * s["scales"].float().unsqueeze(-1)).flatten(-2)
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device="cuda")
    v = lut[_codes(s["w"])]
    if fmt == "mxfp4":
        return (v.unflatten(-1, (K // 32, 32)) * torch.exp2(s["scales"].float() - 127).unsqueeze(-1)).flatten(-2)
    block = s["scales"][_nv_header(1):].view(torch.float8_e4m3fn).reshape(N, K // 16, 1).float()
    return (v.unflatten(-1, (K // 16, 16)) * block).flatten(-2) * s["scales"][:4].view(torch.float32)


def _plain_gemv(s):
    y = torch.matmul(s["x"].float(), _gemv_values(s).t())
    if s["bias"] is not None:
        y = y + s["bias"]
    if s["case"]["geglu"]:
        g, u = y.chunk(2, -1)
        y = _gelu_tanh(g) * u
    return y.to(s["y"].dtype)


def run(state):
    s, c = state, state["case"]
    if own:
        import mixture_experts_router_amd as moe
        if c["op"] == "gemv":
            sh = moe.w4_shape(c["T"], c["N"], c["K"], c["fmt"], group=c["group"], geglu=c["geglu"], y_fp32=c["y"] == "fp32")
            moe.gemv_w4(sh, s["x"], s["w"], s["scales"], s["zeros"], s["bias"], s["y"], s["ws"])
            return s["y"]
        sh = moe.shape(c["T"], c["H"], c["E"], c["k"], c["I"], mxfp4=c["fmt"] == "mxfp4", nvfp4=c["fmt"] == "nvfp4")
        moe.forward_few(sh, s["x"], s["w_router"], s["bias"], s["w_gu"], s["gu_s"], s["w_d"], s["d_s"], s["out"], s["ids"],
                        s["w"], s["ws"], c["I_sh"], s.get("sh_gu"), s.get("sh_gu_s"), s.get("sh_d"), s.get("sh_d_s"))
        return s["out"], s["ids"], s["w"]
    return _plain_gemv(s) if c["op"] == "gemv" else _plain_layer(s)


# ---------------------------------------------------------------- the least work
def work(case):
    c = case
    bits = {"bf16": 16, "mxfp4": 4 + 8 / 32, "nvfp4": 4 + 8 / 16}
    if c["op"] == "gemv":
        T, N, K = c["T"], c["N"], c["K"]
        b = 4 + (16 + 8 * c["zeros"]) / c["group"] if c["fmt"] == "int4" else bits[c["fmt"]]
        outs = N // 2 if c["geglu"] else N
        return {"bytes": N * K * b / 8 + 2 * T * K + 4 * N * c["bias"] + outs * T * (2 if c["y"] == "bf16" else 4),
                "flops": 2 * T * N * K}
    T, H, E, k, I, I_sh = (c[n] for n in ("T", "H", "E", "k", "I", "I_sh"))
    experts = E * (1 - (1 - k / E) ** T)   # those that T tokens of even routing touch, each read once
    weights = 3 * H * (experts * I + I_sh)
    return {"bytes": weights * bits[c["fmt"]] / 8 + 2 * E * H + 4 * T * H + 8 * T * k + 4 * E * c["bias"],
            "flops": 2 * T * (E * H + 3 * H * (k * I + I_sh))}


# ---------------------------------------------------------------- the definition in 64 bits
def _exact_matrix(codes, fmt, scales, group=0, zeros=None, matrix=None):
    """One matrix in fp64 from its stored form."""
    if fmt == "bf16":
        return codes.double()
    low, high = (codes % 16).double(), torch.div(codes, 16, rounding_mode="floor").double()
    c = torch.empty(codes.shape[0], 2 * codes.shape[1], dtype=torch.float64, device=codes.device)
    c[:, 0::2], c[:, 1::2] = low, high
    n = scales.shape[-1]
    per = c.shape[1] // n
    if fmt == "int4":
        z = zeros.double() if zeros is not None else torch.full_like(scales, 8, dtype=torch.float64)
        return (c - z.repeat_interleave(per, 1)) * scales.double().repeat_interleave(per, 1)
    sign, m = 1 - 2 * torch.floor(c / 8), c % 8
    # E2M1: magnitudes m/2 up to 3/2, then (2 + m % 2) 2^(m div 2 - 2)
    v = sign * torch.where(m < 2, m / 2, (2 + m % 2) * torch.exp2(torch.floor(m / 2) - 2))
    if fmt == "mxfp4":
        return v * torch.exp2(scales.double() - 127).repeat_interleave(per, 1)
    b = scales.double()
    ex, man = torch.floor(b / 8), b % 8   # E4M3, non-negative: 2^(ex-7) (1 + man/8), or man 2^-9 where ex is 0
    e4m3 = torch.where(ex == 0, man * 2.0 ** -9, torch.exp2(ex - 7) * (1 + man / 8))
    return v * e4m3.repeat_interleave(per, 1) * matrix.double()


def _exact_gelu(z):
    return z / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))


def _exact_expert(s, name, sname, e, rows, K):
    fmt, w, buf = s["case"]["fmt"], s[name], s[sname]
    if fmt == "nvfp4":
        E = w.shape[0]
        return _exact_matrix(w[e], fmt, buf[_nv_header(E):].reshape(E, rows, K // 16)[e], matrix=buf[:4 * E].view(torch.float32)[e])
    return _exact_matrix(w[e], fmt, None if buf is None else buf[e])


def exact(case, seed):
    s, c = prepare(case, seed), case
    x = s["x"].double()
    if c["op"] == "gemv":
        scales, matrix = s["scales"], None
        if c["fmt"] == "nvfp4":
            matrix, scales = scales[:4].view(torch.float32), scales[_nv_header(1):].reshape(c["N"], c["K"] // 16)
        rows = []
        for r in range(0, c["N"], 16384):
            z = s["zeros"][r:r + 16384] if s["zeros"] is not None else None
            m = _exact_matrix(s["w"][r:r + 16384], c["fmt"], scales[r:r + 16384], c["group"], z, matrix)
            rows.append(x @ m.T)
        y = torch.cat(rows, 1)
        if s["bias"] is not None:
            y = y + s["bias"].double()
        if c["geglu"]:
            y = _exact_gelu(y[:, :c["N"] // 2]) * y[:, c["N"] // 2:]
        return y
    T, H, E, k, I, I_sh = (c[n] for n in ("T", "H", "E", "k", "I", "I_sh"))
    logits = x @ s["w_router"].double().T
    if s["bias"] is not None:
        logits = logits + s["bias"].double()
    # rank of each expert: how many come before it (a larger logit, or an equal one of a lower index)
    a, b = logits[:, :, None], logits[:, None, :]
    lower = torch.arange(E, device="cuda")[None, :] < torch.arange(E, device="cuda")[:, None]
    rank = ((b > a) | ((b == a) & lower)).sum(-1)
    out = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    chosen = torch.where(rank < k, torch.exp(logits - logits.amax(-1, keepdim=True)), torch.zeros_like(logits))
    weight = chosen / chosen.sum(-1, keepdim=True)
    ids, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, dtype=torch.float64, device="cuda")
    for j in range(k):
        at = (rank == j).to(torch.int32).argmax(-1)
        ids[:, j], w[:, j] = at.to(torch.int32), weight.gather(1, at[:, None])[:, 0]
    for e in sorted(set(ids.flatten().tolist())):
        gu, d = _exact_expert(s, "w_gu", "gu_s", e, 2 * I, H), _exact_expert(s, "w_d", "d_s", e, H, I)
        p = x @ gu.T
        out += weight[:, e:e + 1] * ((_exact_gelu(p[:, :I]) * p[:, I:]) @ d.T)
    if I_sh:
        gu, d = _exact_expert(s, "sh_gu", "sh_gu_s", 0, 2 * I_sh, H), _exact_expert(s, "sh_d", "sh_d_s", 0, H, I_sh)
        p = x @ gu.T
        out += (_exact_gelu(p[:, :I_sh]) * p[:, I_sh:]) @ d.T
    return out, ids, w
