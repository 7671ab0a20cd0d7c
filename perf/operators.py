"""What is measured of the operators around a quantized layer.

Three operators of a diffusion transformer's block, each in its plain form
(elementary torch operations in 32 bits) and as the library's calls:

* ``norm``    residual addition, RMS or layer norm, modulation, and the 8-bit
              codes and per-token scales the next layer's GEMM reads;
* ``linear``  the same norm followed by a 4-bit layer (codes with one scale per
              group), down to the layer's BF16 output;
* ``gemm``    the quantized matrix product with bias, activation, gate and
              residual in its epilogue;
* ``rope``    per-head RMS norm of queries and keys and rotary positions with
              several axes.

Every low-rank branch here is an adapter attached to a rank-0 layer: its factors
are inputs, where the singular vectors of a rank-32 layer would depend on the
solver.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
BF16 = torch.bfloat16
EPS = 1e-6


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token: the time embedding's row, or a class token; latency
        dict(name="norm 1x3072", kind="norm", M=1, K=3072, center=False, weight=True, mod=0, residual=True),
        # a FLUX.1 block at 4096 image + 512 text tokens: layer norm with adaptive scale and shift
        dict(name="norm 4608x3072", kind="norm", M=4608, K=3072, center=True, weight=False, mod=1, residual=True),
        # the same width at batch 4, RMS norm with a weight, the modulation of four prompts
        dict(name="norm 18432x3072", kind="norm", M=18432, K=3072, center=False, weight=True, mod=4, residual=True),
        # the last layer of the transformer: norm and modulation, then the projection to 64 patch values
        dict(name="linear 4608x3072-64", kind="linear", fmt="nvfp4", M=4608, K=3072, N=64, center=True,
             weight=False, mod=1, residual=False),
        # a smaller model's ragged token count and width, RMS norm in front of a projection, INT4
        dict(name="linear 1003x1216-1040", kind="linear", fmt="int4", M=1003, K=1216, N=1040, center=False,
             weight=True, mod=0, residual=True),
        # attention output projection, gated and added to the stream
        dict(name="gemm nvfp4 4608x3072-3072", kind="gemm", fmt="nvfp4", M=4608, K=3072, N=3072, gelu=False, gates=1),
        # the MLP's second layer in 8 bits, gated and added
        dict(name="gemm w8a8 4608x12288-3072", kind="gemm", fmt="w8a8", M=4608, K=12288, N=3072, gelu=False, gates=1),
        # INT4, a ragged batch of two prompts
        dict(name="gemm int4 1100x2048-1936", kind="gemm", fmt="int4", M=1100, K=2048, N=1936, gelu=False, gates=2),
        # a few tokens, activation before the addition, no gate
        dict(name="gemm nvfp4 77x512-512", kind="gemm", fmt="nvfp4", M=77, K=512, N=512, gelu=True, gates=0),
        # queries and keys of a FLUX.1 block: axes of 16, 56 and 56 values, neighbouring pairs
        dict(name="rope 4608x24x128", kind="rope", B=1, T=4608, H=24, HK=24, D=128, d0=16, d1=56, d2=56, half=False,
             norm=True, grid=64),
        # a video's latent frames: time, height, width; halves as pairs, batch 2
        dict(name="rope 2x14040x12x128", kind="rope", B=2, T=14040, H=12, HK=12, D=128, d0=44, d1=42, d2=42,
             half=True, norm=True, grid=30),
        # one short prompt, heads of 64, fewer key heads, part of each head rotated
        dict(name="rope 1x77x8x64", kind="rope", B=1, T=77, H=8, HK=2, D=64, d0=16, d1=16, d2=16, half=False,
             norm=False, grid=8),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["norm", "linear", "gemm", "rope"])
    if kind == "rope":
        half = rng.random() < 0.5
        d = [2 * rng.randint(1, 8) for _ in range(3)]
        if half:
            d[0] += (-sum(d)) % 16
        D = 8 * rng.randint((sum(d) + 7) // 8, 16)
        H = rng.randint(1, 24)
        HK = rng.choice([h for h in range(1, H + 1) if H % h == 0])
        return dict(kind=kind, B=rng.randint(1, 2), T=_log(rng, 1, 8000), H=H, HK=HK, D=D, d0=d[0], d1=d[1], d2=d[2],
                    half=half, norm=rng.random() < 0.5, grid=rng.randint(1, 64))
    M, K = _log(rng, 1, 9000), 64 * _log(rng, 2, 64)
    if kind == "gemm":
        return dict(kind=kind, fmt=rng.choice(["nvfp4", "int4", "w8a8"]), M=M, K=K, N=16 * _log(rng, 2, 160),
                    gelu=rng.random() < 0.5, gates=rng.randint(0, 3))
    c = dict(kind=kind, M=M, K=K, center=rng.random() < 0.5, weight=rng.random() < 0.5, mod=rng.randint(0, 3),
             residual=rng.random() < 0.5)
    return c if kind == "norm" else dict(c, fmt=rng.choice(["nvfp4", "int4"]), N=16 * _log(rng, 2, 80))


# ------------------------------------------------------------------ number formats and layouts

def _pad(M):
    return (M + 127) // 128 * 128


def _e4m3(t):
    return t.clamp(max=448.0).to(torch.float8_e4m3fn)


def _e2m1(q):
    """Codes 0..15 of the nearest E2M1 value, ties to the even code, saturating at 6."""
    a = q.abs()
    c = sum((a > t if i % 2 == 0 else a >= t).to(torch.uint8)
            for i, t in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)))
    return c | (torch.signbit(q).to(torch.uint8) << 3)


def _groups(v, fmt, g_exp):
    """Codes [rows, K] and scales [rows, K / group] of 32-bit values, as the library rounds them."""
    v = v.float()
    if fmt == "w8a8":
        s = v.abs().amax(1, keepdim=True) * torch.tensor(1.0 / 127.0, device=v.device)
        inv = torch.where(s == 0, s, 1.0 / s)
        return (v * inv).round().clamp(-127, 127).to(torch.int8), s
    n = 16 if fmt == "nvfp4" else 64
    g = v.view(v.shape[0], -1, n)
    a = g.abs().amax(2)
    if fmt == "nvfp4":
        c = torch.tensor(1.0 / 6.0, device=v.device) * 2.0 ** -g_exp
        s = _e4m3(a * c)
        sf = s.float()
        inv = torch.where(sf == 0, sf, 1.0 / (sf * 2.0 ** g_exp))
        return torch.where((sf == 0)[..., None], torch.zeros((), dtype=torch.uint8, device=v.device),
                           _e2m1(g * inv[..., None])).view(v.shape), s
    s = (a * torch.tensor(1.0 / 7.0, device=v.device)).to(BF16)
    sf = s.float()
    inv = torch.where(sf == 0, sf, 1.0 / sf)
    return (g * inv[..., None]).round().clamp(-7, 7).to(torch.int8).view(v.shape), s


def _values(codes, s, fmt, g_exp, dtype):
    """What codes and scales stand for, [rows, K]."""
    if fmt == "w8a8":
        return codes.to(dtype) * s.to(dtype)
    if fmt == "nvfp4":
        lut = torch.tensor(E2M1 + tuple(-x for x in E2M1), dtype=dtype, device=codes.device)
        c, n = lut[codes.long()], 16
    else:
        c, n = codes.to(dtype), 64
    v = c.view(c.shape[0], -1, n) * s.to(dtype)[..., None] * 2.0 ** g_exp
    return v.view(c.shape)


def _swizzle(dev):
    r, c = torch.arange(128, device=dev)[:, None], torch.arange(8, device=dev)[None, :]
    return r, c ^ (r & 7)


def _tile(b):
    """Rows of bytes [rows, n] in the GEMM's tiled order: blocks of 128 rows x 128 bytes, 16-byte chunks swizzled."""
    M, n = b.shape
    t = torch.zeros((_pad(M), (n + 127) // 128 * 128), dtype=b.dtype, device=b.device)
    t[:M, :n] = b
    r, c = _swizzle(b.device)
    t = t.view(_pad(M) // 128, 128, -1, 8, 16).transpose(1, 2)
    return t[:, :, r, c].contiguous()


def _untile(t, M, n):
    """The inverse of _tile: [M, n] (the swizzle is its own inverse)."""
    b = t.view(-1, (n + 127) // 128, 128, 8, 16)
    r, c = _swizzle(t.device)
    return b[:, :, r, c].transpose(1, 2).reshape(b.shape[0] * 128, -1)[:M, :n]


def _pack(c):
    c = c.view(torch.uint8) & 15
    return c[:, 0::2] | (c[:, 1::2] << 4)


def _unpack(b, fmt):
    c = torch.stack((b & 15, b >> 4), 2).view(b.shape[0], -1)
    return c if fmt == "nvfp4" else ((c ^ 8).view(torch.int8) - 8)


def _lay_out(codes, s, fmt):
    """Codes and scales in the buffers the library's GEMM reads."""
    M, K = codes.shape
    mb = _pad(M) // 128
    if fmt == "w8a8":
        sx = torch.zeros((2, _pad(M)), device=s.device)
        sx[0, :M] = s[:, 0]
        sx[1, :M] = torch.where(s == 0, s, 1.0 / s)[:, 0]
        return _tile(codes.view(torch.uint8)), sx
    if fmt == "nvfp4":
        p = torch.zeros((_pad(M), K // 16), dtype=torch.uint8, device=s.device)
        p[:M] = s.view(torch.uint8)
        return _tile(_pack(codes)), p.view(mb, 4, 32, K // 64, 4).permute(0, 3, 2, 1, 4).contiguous()
    p = torch.zeros((K // 64, _pad(M)), dtype=BF16, device=s.device)
    p[:, :M] = s.t()
    return _pack(codes).contiguous(), p


def _read_back(codes, s, fmt, M, K):
    """The inverse of _lay_out."""
    if fmt == "w8a8":
        return _untile(codes, M, K).contiguous().view(torch.int8), s[0, :M, None]
    if fmt == "nvfp4":
        sc = s.view(-1, K // 64, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, K // 16)[:M].contiguous()
        return _unpack(_untile(codes, M, K // 2), fmt), sc.view(torch.float8_e4m3fn)
    return _unpack(codes, fmt), s[:, :M].t()


# ------------------------------------------------------------------ inputs

def _exp2_ceil(x):
    m, e = math.frexp(x)
    return 0 if x <= 0 else (e - 1 if m == 0.5 else e)


def _layer(g, fmt, K, N, dev):
    """A rank-0 layer's weight, bias and calibration batch, its quantized weight, and an adapter's factors."""
    W = (torch.randn((K, N), generator=g, device=dev) / math.sqrt(K)).to(BF16)
    b = (0.14 * torch.randn(N, generator=g, device=dev)).to(BF16)
    Xc = torch.randn((64, K), generator=g, device=dev)
    Xc[:, torch.randperm(K, generator=g, device=dev)[:K // 100]] *= 20.0
    Xc = Xc.to(BF16)
    lam = Xc.float().abs().amax(0).sqrt() / W.float().abs().amax(1).sqrt()
    inv_lam = 1.0 / lam
    R = lam[:, None] * W.float()
    gw = _exp2_ceil(float(R.abs().max()) / 2688.0) if fmt == "nvfp4" else 0
    gx = _exp2_ceil(4.0 * float((Xc.float() * inv_lam).abs().max()) / 2688.0) if fmt == "nvfp4" else 0
    wq, ws = _groups(R.t().contiguous(), fmt, gw)
    A = (torch.randn((K, 32), generator=g, device=dev) / math.sqrt(K)).to(BF16)
    Bf = (0.2 * torch.randn((32, N), generator=g, device=dev)).to(BF16)
    lora = fmt != "w8a8"
    st = dict(fmt=fmt, K=K, N=N, inv_lam=inv_lam, gx=gx, gw=gw, wq=wq, wsc=ws, bias=b, A=A, B=Bf, lora=lora)
    if own:
        import w4a4_diffusion_transformer_b200 as svdq

        def bits(t):
            return t.view(torch.int16).cpu().numpy().view(np.uint16)
        L = svdq.Layer.prepare(bits(W), bits(b), bits(Xc), fmt=fmt, rank=0, device=0)
        if lora:
            L.set_lora(bits(A), bits(Bf), 1.0)
        st["layer"] = L
    else:
        # a user's program without the library keeps the weight in 32 bits
        st["w32"] = _values(wq, ws, fmt, gw, torch.float32).t().contiguous()
    return st


def _stream_in(g, M, K, dev):
    """Activations of a residual stream: a few channels much larger than the others."""
    x = torch.randn((M, K), generator=g, device=dev)
    x[:, ::97] *= 20.0
    return x.to(BF16)


def _make(case, seed, dev):
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))

    def rnd(*shape, a=1.0, b=0.0):
        return (torch.randn(shape, generator=g, device=dev) * a + b).to(BF16)
    k = case["kind"]
    if k == "rope":
        B, T, H, HK, D = (case[n] for n in ("B", "T", "H", "HK", "D"))
        qkv = rnd(B, T, (H + 2 * HK) * D)
        t = torch.arange(T, device=dev)
        side = case["grid"]
        pos = torch.stack((t // (side * side), t // side % side, t % side), 1).float()
        return dict(case=case, qkv=qkv, pos=pos.contiguous(), qw=rnd(D, a=0.1, b=1.0), kw=rnd(D, a=0.1, b=1.0),
                    q=torch.zeros((B, H, T, D), dtype=BF16, device=dev),
                    k=torch.zeros((B, HK, T, D), dtype=BF16, device=dev))
    M, K = case["M"], case["K"]
    if k == "gemm":
        fmt, N = case["fmt"], case["N"]
        st = _layer(g, fmt, K, N, dev)
        x = _stream_in(g, M, K, dev)
        codes, s = _groups(x.float() * st["inv_lam"], fmt, st["gx"])
        codes, s = _lay_out(codes, s, fmt)
        xl = None
        if st["lora"]:
            xl = torch.zeros((M, 64), dtype=BF16, device=dev)
            xl[:, 32:] = (x.float() @ st["A"].float()).to(BF16)
        gates = case["gates"]
        return dict(st, case=case, codes=codes, scales=s, xl=xl, res=rnd(M, N, a=2.0),
                    gate=rnd(gates, 6 * N, a=0.5) if gates else None, rows=-(-M // max(1, gates)),
                    y=torch.zeros((M, N), dtype=BF16, device=dev))
    fmt, N = case.get("fmt", "w8a8"), case.get("N", 16)
    st = _layer(g, fmt, K, N, dev)
    mod = case["mod"]
    st.update(case=case, x=_stream_in(g, M, K, dev), res=rnd(M, K) if case["residual"] else None,
              weight=rnd(K, a=0.2, b=1.0) if case["weight"] else None,
              mod=rnd(mod, 6 * K, a=0.3) if mod else None, rows=-(-M // max(1, mod)),
              sum=torch.zeros((M, K), dtype=BF16, device=dev) if case["residual"] else None,
              y=torch.zeros((M, N), dtype=BF16, device=dev))
    if k == "norm":
        nst = (K + 127) // 128
        st.update(codes=torch.zeros((_pad(M) // 128, nst, 128, 128), dtype=torch.int8, device=dev),
                  scales=torch.zeros((2, _pad(M)), device=dev),
                  vals=torch.zeros((_pad(M) // 128, nst, 128, 128), dtype=BF16, device=dev))
    return st


def prepare(case, seed):
    s = _make(case, seed, DEV)
    if own:
        import w4a4_diffusion_transformer_b200 as svdq
        k = case["kind"]
        if k == "rope":
            H, HK, D = case["H"], case["HK"], case["D"]
            s["rope"] = svdq.Rope(D, (case["d0"], case["d1"], case["d2"]), theta=10000.0, half=case["half"],
                                  norm=case["norm"], eps=EPS)
            w = case["norm"]
            s["hq"] = svdq.Heads(s["qkv"].view(*s["qkv"].shape[:2], -1, D)[:, :, :H], s["q"].transpose(1, 2),
                                 weight=s["qw"] if w else None)
            s["hk"] = svdq.Heads(s["qkv"].view(*s["qkv"].shape[:2], -1, D)[:, :, H:H + HK], s["k"].transpose(1, 2),
                                 weight=s["kw"] if w else None)
        elif k == "gemm":
            N = case["N"]
            s["epi"] = svdq.Residual(s["res"], gate=None if s["gate"] is None else s["gate"][:, 2 * N:3 * N],
                                     rows_per_gate=s["rows"])
        else:
            K, m = case["K"], s["mod"]
            s["norm"] = svdq.Norm(residual=s["res"], sum=s["sum"], weight=s["weight"],
                                  scale=None if m is None else m[:, K:2 * K], shift=None if m is None else m[:, :K],
                                  rows_per_mod=s["rows"], eps=EPS, center=case["center"])
            if k == "linear":
                n = s["layer"].workspace_bytes(case["M"])
                s["ws"] = torch.empty(n, dtype=torch.uint8, device=DEV)
    return s


# ------------------------------------------------------------------ the passes

def _rows(t, M, rows):
    """Row m of a tensor of shared rows is row m // rows."""
    return t[torch.arange(M, device=t.device) // rows]


def _plain_norm(s):
    """(the sum in BF16, the normalised and modulated rows in BF16)"""
    c, K = s["case"], s["K"]
    M = c["M"]
    h = s["x"] if s["res"] is None else (s["x"].float() + s["res"].float()).to(BF16)
    v = h.float()
    if c["center"]:
        v = v - v.mean(1, keepdim=True)
    v = v * torch.rsqrt(v.square().mean(1, keepdim=True) + EPS)
    if s["weight"] is not None:
        v = v * s["weight"].float()
    if s["mod"] is not None:
        m = _rows(s["mod"], M, s["rows"]).float()
        v = v * (1.0 + m[:, K:2 * K]) + m[:, :K]
    return h, v.to(BF16)


def _plain_product(s, codes, sc, xl):
    """alpha acc + bias in 32 bits."""
    x = _values(codes, sc, s["fmt"], s["gx"], torch.float32)
    y = x @ s["w32"]
    if xl is not None:
        y = y + xl.float() @ s["B"].float()
    return y + s["bias"].float()


def _plain_rope(s):
    c = s["case"]
    D, H, HK = c["D"], c["H"], c["HK"]
    dims = (c["d0"], c["d1"], c["d2"])
    ang = torch.cat([s["pos"][:, a:a + 1].double() *
                     10000.0 ** (-torch.arange(0, d, 2, device=s["pos"].device, dtype=torch.float64) / d)
                     for a, d in enumerate(dims)], 1)
    cs, sn = ang.cos().float()[None, :, None], ang.sin().float()[None, :, None]
    R = sum(dims)
    x = s["qkv"].view(*s["qkv"].shape[:2], -1, D)

    def one(t, w):
        t = t.float()
        if c["norm"]:
            t = t * torch.rsqrt(t.square().mean(3, keepdim=True) + EPS) * w.float()
        a, b = (t[..., :R // 2], t[..., R // 2:R]) if c["half"] else (t[..., 0:R:2], t[..., 1:R:2])
        u, v = a * cs - b * sn, a * sn + b * cs
        r = torch.cat((u, v), 3) if c["half"] else torch.stack((u, v), 4).flatten(3)
        return torch.cat((r, t[..., R:]), 3).to(BF16).transpose(1, 2).contiguous()
    return one(x[:, :, :H], s["qw"]), one(x[:, :, H:H + HK], s["kw"])


def run(s):
    c = s["case"]
    k = c["kind"]
    if own:
        import w4a4_diffusion_transformer_b200 as svdq
        stream = torch.cuda.current_stream()
        if k == "rope":
            svdq.rope_heads(s["rope"], s["hq"], s["hk"], s["pos"], stream)
            return {"q": s["q"], "k": s["k"]}
        L, M = s["layer"], c["M"]
        if k == "gemm":
            L.gemm_residual(s["codes"], s["scales"], s["xl"], M, s["epi"], s["y"], stream,
                            svdq.FWD_GELU if c["gelu"] else 0)
            return {"y": s["y"]}
        if k == "linear":
            L.norm_forward(s["norm"], s["x"], M, s["y"], s["ws"], s["ws"].numel(), stream)
            return {"y": s["y"], "sum": s["sum"]}
        L.norm_quantize_act(s["norm"], s["x"], M, s["codes"], s["scales"], None, stream)
        # the 8-bit codes as the values they stand for, in the GEMM's order
        torch.mul(s["codes"], s["scales"][0].view(-1, 1, 128, 1), out=s["vals"])
        return {"values": s["vals"], "sum": s["sum"]}
    if k == "rope":
        q, kk = _plain_rope(s)
        return {"q": q, "k": kk}
    if k == "gemm":
        M, K, N = c["M"], c["K"], c["N"]
        codes, sc = _read_back(s["codes"], s["scales"], s["fmt"], M, K)
        y = _plain_product(s, codes, sc, None if s["xl"] is None else s["xl"][:, 32:])
        if c["gelu"]:
            y = 0.5 * y * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (y + 0.044715 * y * y * y)))
        if s["gate"] is not None:
            y = y * _rows(s["gate"][:, 2 * N:3 * N], M, s["rows"]).float()
        return {"y": (s["res"].float() + y).to(BF16)}
    h, y = _plain_norm(s)
    codes, sc = _groups(y.float() * s["inv_lam"], s["fmt"], s["gx"])
    if k == "norm":
        return {"values": _tile(_values(codes, sc, "w8a8", 0, torch.float32).to(BF16)).view(s["vals"].shape),
                "sum": None if s["res"] is None else h}
    xl = (y.float() @ s["A"].float()).to(BF16) if s["lora"] else None
    return {"y": _plain_product(s, codes, sc, xl).to(BF16), "sum": None if s["res"] is None else h}


# ------------------------------------------------------------------ work

def work(case):
    k = case["kind"]
    if k == "rope":
        n = case["B"] * case["T"] * (case["H"] + case["HK"]) * case["D"]
        return {"bytes": 4 * n + 12 * case["T"], "flops": 10 * n}
    M, K = case["M"], case["K"]
    byte = {"w8a8": 1.0, "nvfp4": 0.5 + 1 / 16, "int4": 0.5 + 1 / 32}[case.get("fmt", "w8a8")]
    if k == "gemm":
        N, lora = case["N"], case["fmt"] != "w8a8"
        return {"bytes": byte * K * (M + N) + 4 * M * N + 2 * N * (1 + case["gates"]) + lora * 64 * (M + N),
                "flops": 2 * M * N * (K + 32 * lora)}
    read = 2 * M * K * (1 + 2 * case["residual"]) + 2 * K * (case["weight"] + 2 * case["mod"]) + 4 * K
    if k == "norm":
        return {"bytes": read + M * K + 8 * M, "flops": 12 * M * K}
    N = case["N"]
    return {"bytes": read + byte * K * N + 64 * (K + N) + 2 * M * N + 2 * N, "flops": 2 * M * (N * (K + 32) + 32 * K)}


# ------------------------------------------------------------------ 64 bits

def _round(v, to):
    """64-bit values rounded to a format's nearest value, ties to even: `to` significant bits, smallest step 2^-133."""
    m, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), torch.clamp(e - to, min=-133))
    return torch.round(v / step) * step


def _offsets8(M, cols, dev):
    """Byte offset of byte j of row r in the GEMM's tiled order, from its definition."""
    r, j = torch.arange(M, device=dev)[:, None], torch.arange(cols, device=dev)[None, :]
    nst = -(-cols // 128)
    return ((r // 128) * nst + j // 128) * 16384 + (r % 128) * 128 + (((j % 128) // 16) ^ (r % 8)) * 16 + j % 16


def _offsets_sf(M, G, dev):
    """Byte offset of the scale of group g of row r in the tensor-core order."""
    r, g = torch.arange(M, device=dev)[:, None], torch.arange(G, device=dev)[None, :]
    return ((r // 128) * (G // 4) + g // 4) * 512 + (r % 32) * 16 + (r // 32 % 4) * 4 + g % 4


def _nearest(x, grid):
    """Index of the nearest of ascending values, ties to the even index."""
    grid = torch.tensor(grid, dtype=torch.float64, device=x.device)
    mid = (grid[1:] + grid[:-1]) / 2
    lo = torch.searchsorted(mid, x.contiguous(), right=False)
    hi = torch.searchsorted(mid, x.contiguous(), right=True)
    return torch.where(lo % 2 == 0, lo, hi)


def _quant64(v, fmt, gx):
    """The values that the codes of v stand for."""
    if fmt == "w8a8":
        s = v.abs().amax(1, keepdim=True) / 127.0
        q = torch.where(s > 0, torch.round(v / torch.where(s > 0, s, 1.0)), 0.0)
        return q * s
    n = 16 if fmt == "nvfp4" else 64
    g = v.reshape(v.shape[0], -1, n)
    a = g.abs().amax(2, keepdim=True)
    if fmt == "int4":
        s = _round(a / 7.0, 8)
        q = torch.round(g / torch.where(s > 0, s, 1.0)).clamp(-7, 7) * s
        return q.reshape(v.shape)
    t = a / 6.0 * 2.0 ** -gx
    m, e = torch.frexp(t)
    step = torch.ldexp(torch.ones_like(t), torch.clamp(e - 4, min=-9))
    s = (torch.round(t / step) * step).clamp(max=448.0) * 2.0 ** gx
    i = _nearest((g / torch.where(s > 0, s, 1.0)).abs(), E2M1)
    q = torch.tensor(E2M1, dtype=torch.float64, device=v.device)[i] * torch.sign(g) * s
    return q.reshape(v.shape)


def exact(case, seed):
    keep = globals()["own"]
    globals()["own"] = False
    try:
        s = _make(case, seed, DEV)
    finally:
        globals()["own"] = keep
    k, d = case["kind"], torch.float64
    if k == "rope":
        D, H, HK = case["D"], case["H"], case["HK"]
        x = s["qkv"].to(d)
        B, T = x.shape[:2]
        out = {}
        for name, first, heads, w in (("q", 0, H, s["qw"]), ("k", H, HK, s["kw"])):
            t = x[:, :, first * D:(first + heads) * D].reshape(B, T, heads, D)
            if case["norm"]:
                t = t / torch.sqrt((t * t).sum(3, keepdim=True) / D + EPS) * w.to(d)
            y = t.clone()
            at, R = 0, case["d0"] + case["d1"] + case["d2"]
            for a, n in enumerate((case["d0"], case["d1"], case["d2"])):
                for j in range(n // 2):
                    ang = s["pos"][:, a].to(d) / 10000.0 ** (2 * j / n)
                    p = at // 2 + j
                    u, v = (p, p + R // 2) if case["half"] else (2 * p, 2 * p + 1)
                    c, z = torch.cos(ang)[None, :, None], torch.sin(ang)[None, :, None]
                    y[..., u] = t[..., u] * c - t[..., v] * z
                    y[..., v] = t[..., v] * c + t[..., u] * z
                at += n
            out[name] = y.permute(0, 2, 1, 3).contiguous()
        return out
    M, K = case["M"], case["K"]
    fmt = s["fmt"]
    if k == "gemm":
        N = case["N"]
        raw = s["codes"].reshape(-1)
        if fmt == "w8a8":
            x = raw[_offsets8(M, K, raw.device)].view(torch.int8).to(d) * s["scales"][0][:M, None].to(d)
        else:
            b = raw[_offsets8(M, K // 2, raw.device)] if fmt == "nvfp4" else raw.view(M, K // 2)
            c = torch.empty((M, K), dtype=torch.long, device=raw.device)
            c[:, 0::2], c[:, 1::2] = b.long() % 16, b.long() // 16
            if fmt == "nvfp4":
                sc = s["scales"].reshape(-1)[_offsets_sf(M, K // 16, raw.device)].view(torch.float8_e4m3fn)
                val = torch.tensor(E2M1, dtype=d, device=raw.device)[c % 8] * (1.0 - 2.0 * (c // 8))
                x = val * sc.to(d).repeat_interleave(16, 1) * 2.0 ** s["gx"]
            else:
                x = torch.where(c > 7, c - 16, c).to(d) * s["scales"][:, :M].t().to(d).repeat_interleave(64, 1)
        y = x @ s["w32"].to(d) + s["bias"].to(d)
        if s["xl"] is not None:
            y = y + s["xl"][:, 32:].to(d) @ s["B"].to(d)
        if case["gelu"]:
            u = math.sqrt(2.0 / math.pi) * (y + 0.044715 * y ** 3)
            y = y / (1.0 + torch.exp(-2.0 * u))
        if s["gate"] is not None:
            row = torch.div(torch.arange(M, device=y.device), s["rows"], rounding_mode="floor")
            y = y * s["gate"].to(d)[row, 2 * N:3 * N]
        return {"y": s["res"].to(d) + y}
    h = s["x"].to(d)
    if s["res"] is not None:
        h = _round(h + s["res"].to(d), 8)
    n = h - h.sum(1, keepdim=True) / K if case["center"] else h
    n = n / torch.sqrt((n * n).sum(1, keepdim=True) / K + EPS)
    if s["weight"] is not None:
        n = n * s["weight"].to(d)
    if s["mod"] is not None:
        row = torch.div(torch.arange(M, device=n.device), s["rows"], rounding_mode="floor")
        n = n * (1.0 + s["mod"].to(d)[row, K:2 * K]) + s["mod"].to(d)[row, :K]
    y = _round(n, 8)
    q = _quant64(y * s["inv_lam"].to(d), fmt, s["gx"])
    total = None if s["res"] is None else h
    if k == "norm":
        vals = torch.zeros(s["vals"].numel(), dtype=d, device=h.device)
        vals[_offsets8(M, K, h.device).reshape(-1)] = q.reshape(-1)
        return {"values": vals.view(s["vals"].shape), "sum": total}
    out = q @ s["w32"].to(d) + s["bias"].to(d) + _round(y @ s["A"].to(d), 8) @ s["B"].to(d)
    return {"y": out, "sum": total}
