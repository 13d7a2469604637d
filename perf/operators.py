"""Cases and plain forms of the operators around the adapted linear layer.

Four operators: the residual addition with RMS norm (bf16 and 8-bit output), its
gradient, the adapted layer's forward with counter-based dropout, and the
matrix-vector product with a 4-bit integer weight (one scale per 16 weights).
Sizes are those of the library's own workloads (4096 and 11008 wide projections,
M = 64, 2048, 4096, 8192 tokens, ranks 8, 16, 64) and generic ones around them.
"""

import math

import numpy as np
import torch

own = False

_DEV = "cuda"
_EPS = 1e-5
_WS = []


def _q():
    import quantized_rank_fine_b200 as q
    return q


def _workspace():
    """The one workspace that a program keeps for all its calls."""
    if not _WS:
        _WS.append(_q().Workspace())
    return _WS[0]


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one decoded token: the residual stream joined and normalised straight to 8 bits
        dict(name="norm 1x4096 to 8 bits", op="norm", M=1, n=4096, res=True, y=False, block=0, p=0.0, g32=False, rstd=False),
        # training forward of one micro-batch, rstd kept for the backward
        dict(name="norm 2048x4096", op="norm", M=2048, n=4096, res=True, y=True, block=-1, p=0.0, g32=False, rstd=True),
        # the largest micro-batch, residual dropout, bf16 and blockwise 8-bit outputs
        dict(name="norm 8192x4096 dropout", op="norm", M=8192, n=4096, res=True, y=True, block=64, p=0.1, g32=True, rstd=True),
        # a ragged batch of a narrow model: the gradient with the gain's
        dict(name="norm grad 333x1032", op="norm_bwd", M=333, n=1032, res=True, p=0.0, g32=True),
        # training backward of one micro-batch
        dict(name="norm grad 2048x4096", op="norm_bwd", M=2048, n=4096, res=True, p=0.0, g32=False),
        # the largest micro-batch under residual dropout
        dict(name="norm grad 8192x4096 dropout", op="norm_bwd", M=8192, n=4096, res=True, p=0.1, g32=False),
        # the small workload's layer in training, adapter dropout without a stored mask
        dict(name="layer 256x256 M64 dropout", op="layer", M=64, K=256, N=256, r=8, p=0.05, scale=2.0),
        # an attention projection in training
        dict(name="layer 4096x4096 M2048 dropout", op="layer", M=2048, K=4096, N=4096, r=16, p=0.05, scale=2.0),
        # a narrow odd-sized layer without adapters, three tokens
        dict(name="matvec 320x192 M3", op="matvec", M=3, K=320, N=192, r=0, x8=-1),
        # one token through an attention projection
        dict(name="matvec 4096x4096 M1", op="matvec", M=1, K=4096, N=4096, r=16, x8=-1),
        # a few tokens through the down projection, 8-bit activations with block scales
        dict(name="matvec 11008x4096 M4 x8", op="matvec", M=4, K=11008, N=4096, r=16, x8=64),
        # sixteen tokens through an up projection, 8-bit activations with row scales
        dict(name="matvec 4096x11008 M16 x8", op="matvec", M=16, K=4096, N=11008, r=64, x8=0),
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of step in [lo, hi], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "layer", "matvec"])
    if op in ("norm", "norm_bwd"):
        n = _log(rng, 64, 11008, 8)
        M = _log(rng, 1, max(1, min(8192, 8192 * 4096 // n)))
        c = dict(op=op, M=M, n=n, res=rng.random() < 0.75, p=rng.choice([0.0, 0.0, 0.05, 0.1, 0.5]), g32=rng.random() < 0.5)
        if op == "norm":
            block = rng.choice([-1, 0, 64])
            if block == 64:
                c["n"] = n = max(64, n // 64 * 64)
            c.update(block=block, y=block < 0 or rng.random() < 0.5, rstd=rng.random() < 0.5)
        return c
    if op == "layer":
        return dict(op=op, M=_log(rng, 1, 2048), K=_log(rng, 64, 4096, 64), N=_log(rng, 64, 4096, 64), r=8 * rng.randint(1, 8),
                    p=rng.choice([0.05, 0.1, 0.3]), scale=rng.choice([1.0, 2.0]))
    K = _log(rng, 64, 11008, 64)
    N = _log(rng, 64, max(64, min(11008, 4096 * 11008 // K // 64 * 64)), 64)
    return dict(op=op, M=rng.randint(1, 16), K=K, N=N, r=rng.choice([0, 8 * rng.randint(1, 8)]), x8=rng.choice([-1, 0, 64]))


# ---------------------------------------------------------------- inputs

def _int16(K, N, gen):
    """A weight in symmetric 4-bit integers, one scale per 16 weights of a row: codes q + 8, two per byte, low nibble first."""
    w = torch.randn((K * N // 16, 16), generator=gen, device=_DEV) * 0.02
    s = w.abs().amax(1) / 7
    c = (torch.clamp(torch.round(w / s[:, None]), -7, 7) + 8).to(torch.uint8).view(-1, 2)
    return (c[:, 0] | (c[:, 1] << 4)).contiguous(), s.contiguous()


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=_DEV).manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=_DEV)

    s = {"case": c, "key": (int(seed) * 0x9E3779B97F4A7C15 + 1) % (1 << 64), "offset": (int(seed) % 1000) << 31}
    if c["op"] in ("norm", "norm_bwd"):
        M, n = c["M"], c["n"]
        # a residual stream: channels of different strength, a few of them far larger
        chan = torch.exp(0.5 * normal(n)) * torch.where(torch.rand(n, generator=gen, device=_DEV) < 0.004, 20.0, 1.0)
        s["gain"] = 1.0 + 0.2 * normal(n)
        if not c["g32"]:
            s["gain"] = s["gain"].to(torch.bfloat16)
        if c["op"] == "norm":
            s["x"] = normal(M, n).to(torch.bfloat16)
            s["res"] = (normal(M, n) * chan).to(torch.bfloat16) if c["res"] else None
        else:
            s["h"] = (normal(M, n) * chan).to(torch.bfloat16)
            s["rstd"] = torch.rsqrt(s["h"].float().square().mean(1) + _EPS)
            s["dy"] = (normal(M, n) * 0.1).to(torch.bfloat16)
            s["dh"] = (normal(M, n) * 0.1).to(torch.bfloat16) if c["res"] else None
        return s
    M, K, N, r = c["M"], c["K"], c["N"], c["r"]
    s["codes"], s["scales"] = _int16(K, N, gen)
    x = normal(M, K)
    if r:
        s["A"] = (normal(K, r) / math.sqrt(K)).to(torch.bfloat16)
        s["B"] = (normal(r, N) * 0.01).to(torch.bfloat16)
    if c["op"] == "matvec" and c["x8"] >= 0:
        b = x.view(M, -1, c["x8"] or K)
        sc = b.abs().amax(2) / 448
        s["xcodes"] = (b / sc[:, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(M, K).view(torch.uint8)
        s["xscales"] = sc.contiguous()
    else:
        s["x"] = x.to(torch.bfloat16)
    return s


# ---------------------------------------------------------------- the operators

def run(s):
    c = s["case"]
    return {"norm": _run_norm, "norm_bwd": _run_norm_bwd, "layer": _run_layer, "matvec": _run_matvec}[c["op"]](s, c)


def _u32(seed, offset, n):
    """Philox4x32-10: the 32-bit words of elements 0 .. n-1 (as int64)."""
    mask = 0xFFFFFFFF
    blk = torch.arange((n + 3) // 4, device=_DEV)
    x = [blk & mask, blk >> 32, torch.full_like(blk, offset & mask), torch.full_like(blk, offset >> 32)]
    k0, k1 = seed & mask, seed >> 32

    def wide(a, m):
        lo, hi = (a & 0xFFFF) * m, (a >> 16) * m
        return (hi + (lo >> 16)) >> 16, ((hi << 16) + lo) & mask

    for _ in range(10):
        h0, l0 = wide(x[0], 0xD2511F53)
        h1, l1 = wide(x[2], 0xCD9E8D57)
        x = [h1 ^ x[1] ^ k0, l1, h0 ^ x[3] ^ k1, l0]
        k0, k1 = (k0 + 0x9E3779B9) & mask, (k1 + 0xBB67AE85) & mask
    return torch.stack(x, 1).view(-1)[:n]


def _kept(t, s, p):
    """t with dropout: each element times keep times the binary32 value of 1 / (1 - p), in t's own precision."""
    if p == 0.0:
        return t
    p = float(np.float32(p))
    keep = _u32(s["key"], s["offset"], t.numel()).view(t.shape) >= round(p * 2 ** 32)
    return t * keep * float(np.float32(1.0 / (1.0 - p)))


def _bf16(t):
    """float64 to bfloat16 in one rounding (the conversion goes through binary32, whose ties are decided here)."""
    f = t.float()
    tie, up = (f.view(torch.int32) & 0xFFFF) == 0x8000, torch.full_like(f, math.inf)
    f = torch.where(tie & (t > f.double()), torch.nextafter(f, up), torch.where(tie & (t < f.double()), torch.nextafter(f, -up), f))
    return f.to(torch.bfloat16)


def _run_norm(s, c):
    if own:
        q = _q()
        d = q.Dropout(c["p"], s["key"], s["offset"]) if c["p"] else None
        o = q.qlora_rmsnorm_fwd(s["x"], s["gain"], eps=_EPS, residual=s["res"], dropout=d, want_y=c["y"],
                                quant_block=c["block"] if c["block"] >= 0 else None, save_rstd=c["rstd"])
        got = {}
        if o.H is not None:
            got["h"] = o.H
        if c["y"]:
            got["y"] = o.Y
        if c["rstd"]:
            got["rstd"] = o.rstd
        if c["block"] >= 0:
            got["q"] = o.act.codes.view(torch.float8_e4m3fn)
            got["q_scales"] = o.act.scales
        return got
    M, n = s["x"].shape
    got = {}
    h = s["x"].float()
    if s["res"] is not None or c["p"]:
        # in 64 bits: under dropout many sums lie next to the border between two bfloat16 values
        h = _kept(s["x"].double(), s, c["p"])
        got["h"] = _bf16(h + s["res"].double() if s["res"] is not None else h)
        h = got["h"].float()
    rstd = torch.rsqrt(h.square().mean(1) + _EPS)
    y = h * rstd[:, None] * s["gain"].float()
    if c["y"]:
        got["y"] = y.to(torch.bfloat16)
    if c["rstd"]:
        got["rstd"] = rstd
    if c["block"] >= 0:
        b = y.view(M, -1, c["block"] or n)
        sc = b.abs().amax(2) / 448
        v = torch.where(sc[:, :, None] > 0, b / sc[:, :, None], 0.0)
        got["q"] = v.clamp(-448, 448).to(torch.float8_e4m3fn).view(M, n)
        got["q_scales"] = sc
    return got


def _run_norm_bwd(s, c):
    if own:
        q = _q()
        d = q.Dropout(c["p"], s["key"], s["offset"]) if c["p"] else None
        dx, dr, dg = q.qlora_rmsnorm_bwd(s["dy"], s["h"], s["gain"], s["rstd"], _workspace(), dH=s["dh"], dropout=d)
        return {"dr": dr, "dx": dx, "dgain": dg} if c["p"] else {"dr": dr, "dgain": dg}
    h, dy, g = s["h"].float(), s["dy"].float(), s["gain"].float()
    rstd = s["rstd"][:, None]
    gy = dy * g
    d = rstd * (gy - h * ((gy * h).mean(1, keepdim=True) * rstd * rstd))
    if s["dh"] is not None:
        d = d + s["dh"].float()
    got = {"dr": d.to(torch.bfloat16), "dgain": (dy * h * rstd).sum(0)}
    if c["p"]:
        got["dx"] = _kept(d, s, c["p"]).to(torch.bfloat16)
    return got


def _dense(s, c):
    """w' = q scale in fp32, (K, N)."""
    b = s["codes"]
    qv = torch.stack((b & 15, b >> 4), 1).view(-1, 16).to(torch.float32) - 8.0
    return (qv * s["scales"][:, None]).view(c["K"], c["N"])


def _run_layer(s, c):
    if own:
        q = _q()
        w = q.int_weight(s["codes"], s["scales"], c["K"], c["N"])
        Y, V = q.qlora_linear_fwd(w, s["x"], s["A"], s["B"], _workspace(), adapter_scale=c["scale"],
                                  dropout=q.Dropout(c["p"], s["key"], s["offset"]))
        return {"y": Y, "v": V}
    x = s["x"].float()
    V = _kept(x @ s["A"].float() * c["scale"], s, c["p"]).to(torch.bfloat16)
    w = _dense(s, c).to(torch.bfloat16).float()   # the layer multiplies with bf16 weights
    return {"y": (x @ w + V.float() @ s["B"].float()).to(torch.bfloat16), "v": V}


def _run_matvec(s, c):
    if own:
        q = _q()
        w = q.int_weight(s["codes"], s["scales"], c["K"], c["N"])
        x = s["x"] if c["x8"] < 0 else q.Act8(s["xcodes"], s["xscales"], c["x8"])
        if not c["r"]:
            return {"y": q.qlora_matvec(w, x, _workspace())[0]}
        Y, V = q.qlora_matvec(w, x, _workspace(), s["A"], s["B"], save_V=True)
        return {"y": Y, "v": V}
    M, K = c["M"], c["K"]
    if c["x8"] < 0:
        x = s["x"].float()
    else:
        x = (s["xcodes"].view(torch.float8_e4m3fn).float().view(M, -1, c["x8"] or K) * s["xscales"][:, :, None]).view(M, K)
    y = x @ _dense(s, c)
    if not c["r"]:
        return {"y": y.to(torch.bfloat16)}
    V = (x @ s["A"].float()).to(torch.bfloat16)
    return {"y": (y + V.float() @ s["B"].float()).to(torch.bfloat16), "v": V}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    c = case
    if c["op"] == "norm":
        e, n = c["M"] * c["n"], c["n"]
        h = c["res"] or c["p"] > 0
        nbytes = 2 * e * (1 + c["res"] + h + c["y"]) + n * (4 if c["g32"] else 2) + 4 * c["M"] * c["rstd"]
        if c["block"] >= 0:
            nbytes += e + 4 * c["M"] * (n // c["block"] if c["block"] else 1)
        return {"bytes": nbytes, "flops": 6 * e}
    if c["op"] == "norm_bwd":
        e, n = c["M"] * c["n"], c["n"]
        return {"bytes": 2 * e * (3 + c["res"] + (c["p"] > 0)) + n * ((4 if c["g32"] else 2) + 4) + 4 * c["M"], "flops": 11 * e}
    M, K, N, r = c["M"], c["K"], c["N"], c["r"]
    x = 2 * M * K
    if c["op"] == "matvec" and c["x8"] >= 0:
        x = M * K + 4 * M * (K // c["x8"] if c["x8"] else 1)
    nbytes = K * N // 2 + K * N // 4 + x + 2 * M * N + 2 * r * (K + N) + 2 * M * r
    return {"bytes": nbytes, "flops": 2 * M * K * N + 2 * M * r * (K + N)}


# ---------------------------------------------------------------- the definitions in 64 bits

def _mask64(s, p, shape):
    """keep times binary32(1 / (1 - p)) as float64, the words made on the host in unsigned 64-bit arithmetic."""
    n = int(np.prod(shape))
    i = np.arange((n + 3) // 4, dtype=np.uint64)
    lo32, sh = np.uint64(0xFFFFFFFF), np.uint64(32)
    c0, c1 = i & lo32, i >> sh
    c2 = np.full_like(i, s["offset"] & 0xFFFFFFFF)
    c3 = np.full_like(i, s["offset"] >> 32)
    for t in range(10):
        ka = np.uint64(((s["key"] & 0xFFFFFFFF) + t * 0x9E3779B9) & 0xFFFFFFFF)
        kb = np.uint64(((s["key"] >> 32) + t * 0xBB67AE85) & 0xFFFFFFFF)
        pa, pb = c0 * np.uint64(0xD2511F53), c2 * np.uint64(0xCD9E8D57)
        c0, c1, c2, c3 = (pb >> sh) ^ c1 ^ ka, pb & lo32, (pa >> sh) ^ c3 ^ kb, pa & lo32
    words = np.empty((i.size, 4), dtype=np.uint32)
    for k, w in enumerate((c0, c1, c2, c3)):
        words[:, k] = w
    p64 = np.float64(np.float32(p))
    keep = words.reshape(-1)[:n] >= np.uint32(np.rint(p64 * 4294967296.0))
    return torch.from_numpy(keep.reshape(shape)).to(_DEV).double().mul_(float(np.float32(1.0 / (1.0 - p64))))


def _bf16_64(t):
    """float64 to the nearest bfloat16 (ties to even), as float64."""
    m, e = torch.frexp(t)
    return torch.ldexp(torch.round(m * 256.0), e - 8)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "norm":
        h = s["x"].double()
        if c["p"]:
            h *= _mask64(s, c["p"], h.shape)
        got = {}
        if c["res"] or c["p"]:
            if c["res"]:
                h = h + s["res"].double()
            h = got["h"] = _bf16_64(h)
        inv = 1.0 / torch.sqrt((h * h).sum(1) / c["n"] + _EPS)
        y = torch.einsum("mn,m,n->mn", h, inv, s["gain"].double())
        if c["y"]:
            got["y"] = y
        if c["rstd"]:
            got["rstd"] = inv
        if c["block"] >= 0:
            width = c["block"] or c["n"]
            top = y.abs().unflatten(1, (-1, width)).max(dim=2).values
            sc = got["q_scales"] = top / 448.0
            v = y / sc.repeat_interleave(width, dim=1)
            # the nearest value of 3 mantissa bits above 2^-6, of steps 2^-9 below
            step = torch.exp2(torch.clamp(torch.floor(torch.log2(v.abs().clamp(min=1e-30))), min=-6.0) - 3.0)
            got["q"] = torch.round(v / step) * step
        return got
    if c["op"] == "norm_bwd":
        h, g, r = s["h"].double(), s["gain"].double(), s["rstd"].double()
        dn = s["dy"].double() * g                      # gradient at the normalised row
        xh = h * r[:, None]
        d = (dn - xh * (torch.einsum("mn,mn->m", dn, xh) / c["n"])[:, None]) * r[:, None]
        if c["res"]:
            d += s["dh"].double()
        got = {"dr": d, "dgain": torch.einsum("mn,mn->n", s["dy"].double(), xh)}
        if c["p"]:
            got["dx"] = d * _mask64(s, c["p"], d.shape)
        return got
    K, N = c["K"], c["N"]
    code = torch.empty((K, N), dtype=torch.float64, device=_DEV)
    code[:, 0::2] = (s["codes"] % 16).view(K, N // 2).double()
    code[:, 1::2] = (s["codes"] // 16).view(K, N // 2).double()
    w = (code - 8.0) * s["scales"].double().view(K, N // 16).repeat_interleave(16, dim=1)
    if "x" in s:
        x = s["x"].double()
    else:
        x = s["xcodes"].view(torch.float8_e4m3fn).double() * s["xscales"].double().repeat_interleave(K // s["xscales"].shape[1], dim=1)
    if c["op"] == "layer":
        w = _bf16_64(w)
    y = torch.einsum("mk,kn->mn", x, w)
    if not c["r"]:
        return {"y": y}
    v = torch.einsum("mk,kr->mr", x, s["A"].double()) * c.get("scale", 1.0)
    if c["op"] == "layer":
        v *= _mask64(s, c["p"], v.shape)
    return {"y": y + torch.einsum("mr,rn->mn", _bf16_64(v), s["B"].double()), "v": v}
