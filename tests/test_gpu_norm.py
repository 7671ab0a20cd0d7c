"""GPU parity of the normalisation fused with the first kernel
(svdq_norm_quantize_act, svdq_norm_linear_forward).

Bar: h bit-exact (one FP32 addition, one BF16 rounding); y within half a BF16
step of the float64 formula plus the FP32 error of its sums; codes and scales
bit-exact against the oracle's quantizer on the kernel's own y (so they are
those of svdq_quantize_act on y); XL within the down projection's tolerance;
the layer's output within the tolerance every forward is held to.
"""
import numpy as np
import pytest

import synthetic as syn
from oracle import svdq_oracle as o

import w4a4_diffusion_transformer_b200 as lib
from gpu_util import assert_close_bf16, oracle_prep_from, prepare_gpu, to_numpy_f32, torch_bf16, xl_width

pytestmark = pytest.mark.gpu

EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from w4a4_diffusion_transformer_b200 import build
    build.build()
    lib.load()


def _bf(rng, *shape, a=1.0, b=0.0):
    return syn.to_bf16(rng.standard_normal(shape) * a + b)


def _inputs(seed, M, K, residual=True, weight=True, mods=0, center=False, rows_per_mod=None):
    rng = np.random.default_rng([77, seed, M, K])
    d = {"X": _bf(rng, M, K, a=2.0, b=0.3), "res": _bf(rng, M, K) if residual else None,
         "weight": _bf(rng, K, a=0.2, b=1.0) if weight else None,
         "mod": _bf(rng, mods, 6 * K, a=0.3) if mods else None, "center": center,
         "rows": (-(-M // mods) if rows_per_mod is None else rows_per_mod) if mods else 0}
    d["X"][:, ::53] *= 16.0
    return d


def reference(d):
    """h (exact BF16), y in float64, and the bound of y's error."""
    X = d["X"].astype(np.float64)
    h = o.bf16_round(X + d["res"].astype(np.float64)) if d["res"] is not None else X
    mu = h.mean(axis=1, keepdims=True) if d["center"] else 0.0
    c = h - mu
    rstd = 1.0 / np.sqrt((c * c).mean(axis=1, keepdims=True) + EPS)
    M, K = h.shape
    g = np.ones((1, K)) if d["weight"] is None else d["weight"].astype(np.float64)[None]
    sh = np.zeros((1, K))
    if d["mod"] is not None:
        row = np.arange(M) // d["rows"] if d["rows"] else np.zeros(M, dtype=int)
        g = g * (1.0 + d["mod"][row, K:2 * K].astype(np.float64))
        sh = d["mod"][row, :K].astype(np.float64)
    n = c * rstd
    y = n * g + sh
    # half a BF16 step of y, and FP32 arithmetic: a mean of K values sums at
    # most 8 + 5 + 32 terms one after the other, so each of the mean and the
    # mean square is within 46 roundings, the rest within 8 (rsqrtf: 2 ulp)
    u = 2.0 ** -24
    amp = np.abs(n * g) + np.abs(sh) + (np.abs(g) * rstd * np.abs(h).mean(axis=1, keepdims=True) if d["center"] else 0)
    return h, y, 2.0 ** -8 * np.abs(y) + 64 * u * amp + 1e-38


def _dev(a):
    return None if a is None else torch_bf16(a)


def _norm(d, x, sum_):
    m = _dev(d["mod"])
    K = d["X"].shape[1]
    return lib.Norm(residual=_dev(d["res"]), sum=sum_, weight=_dev(d["weight"]),
                    scale=None if m is None else m[:, K:2 * K], shift=None if m is None else m[:, :K],
                    rows_per_mod=d["rows"], eps=EPS, center=d["center"])


def run(L, d, alias=None, stream=None):
    import torch
    X = d["X"]
    M, K = X.shape
    extra = 5                                     # rows behind the last stay as they were
    x = torch.full((M + extra, K), 7.0, dtype=torch.bfloat16, device="cuda")
    x[:M] = torch_bf16(X)
    sum_ = torch.full((M + extra, K), -3.0, dtype=torch.bfloat16, device="cuda")
    y = torch.full((M + extra, K), -5.0, dtype=torch.bfloat16, device="cuda")
    if alias == "x":
        sum_ = x
    n = _norm(d, x, sum_)
    if alias == "res":
        n = lib.Norm(residual=n._keep[0], sum=n._keep[0], weight=n._keep[2], scale=n._keep[3], shift=n._keep[4],
                     rows_per_mod=d["rows"], eps=EPS, center=d["center"])
        sum_ = n._keep[0]
    codes = torch.full((L.act_code_bytes(M) + 64,), 0xAB, dtype=torch.uint8, device="cuda")
    scales = torch.full((L.act_scale_bytes(M) + 64,), 0xCD, dtype=torch.uint8, device="cuda")
    xl = torch.full((M + extra, xl_width(L)), float("nan"), dtype=torch.bfloat16, device="cuda")
    L.norm_quantize_act(n, x, M, codes, scales, xl, stream or torch.cuda.current_stream(), Y=y)
    torch.cuda.synchronize()
    assert bool((codes[-64:] == 0xAB).all()) and bool((scales[-64:] == 0xCD).all())
    assert bool((y[M:] == -5.0).all()) and bool(torch.isnan(xl[M:]).all())
    if alias is None:
        assert bool((sum_[M:] == -3.0).all()) and bool((x[M:] == 7.0).all())
        np.testing.assert_array_equal(to_numpy_f32(x[:M]), X)
    c, s = codes[:-64].cpu().numpy(), scales[:-64].cpu().numpy()
    return {"h": to_numpy_f32(sum_[:M]), "y": to_numpy_f32(y[:M]), "xl": to_numpy_f32(xl[:M]), "codes_dev": c,
            "scales_dev": s, "codes": L.act_codes_to_logical(c, M), "scales": L.act_scales_to_logical(s, M)}


def check(L, d, got):
    h, y, tol = reference(d)
    np.testing.assert_array_equal(got["h"], h)
    err = np.abs(got["y"].astype(np.float64) - y)
    assert np.all(err <= tol), (np.max(err / tol), np.unravel_index(np.argmax(err / tol), err.shape))


def compare_with_first_kernel(L, got, M, K):
    """The codes and scales of svdq_quantize_act on the same y, byte for byte
    (padding rows included), XL within a BF16 rounding of an FP32 sum."""
    import torch
    y = torch_bf16(got["y"])
    # the same fill as run(): bytes that neither writes (a tiled layout's K tail) compare equal
    codes = torch.full((L.act_code_bytes(M),), 0xAB, dtype=torch.uint8, device="cuda")
    scales = torch.full((L.act_scale_bytes(M),), 0xCD, dtype=torch.uint8, device="cuda")
    xl = torch.full((M, xl_width(L)), float("nan"), dtype=torch.bfloat16, device="cuda")
    L.quantize_act(y, M, codes, scales, xl, torch.cuda.current_stream(), 0)
    torch.cuda.synchronize()
    c, s = codes.cpu().numpy(), scales.cpu().numpy()
    np.testing.assert_array_equal(got["scales_dev"], s)
    np.testing.assert_array_equal(got["codes_dev"], c)
    ref = to_numpy_f32(xl)
    has = np.isfinite(ref)
    np.testing.assert_array_equal(np.isfinite(got["xl"]), has)
    # both sum K products in FP32: they differ by the sums' roundings (relative
    # to the sum of magnitudes, not known here: bounded by the column's largest
    # value times 2^-12) and by one BF16 rounding
    a, b = got["xl"][has], ref[has]
    assert np.all(np.abs(a - b) <= 2.0 ** -7 * np.abs(b) + 2.0 ** -12 * np.max(np.abs(b), initial=0.0))


RANK = {"nvfp4": 32, "int4": 32, "w8a8": 16}
CASES = [  # M, K, options
    (1, 64, dict()),
    (1, 1024, dict(center=True, mods=1)),
    (33, 128, dict(weight=False, mods=3)),
    (130, 320, dict(residual=False, center=True)),
    (200, 576, dict(weight=False, mods=2, center=True)),
    (640, 512, dict(mods=7)),                       # modulation rows change inside a tile
    (777, 1088, dict(residual=False, weight=False)),
    (1301, 256, dict(mods=2, center=True)),
]


@pytest.mark.parametrize("fmt", ["nvfp4", "int4", "w8a8"])
@pytest.mark.parametrize("M,K,opt", CASES)
def test_norm_quantize_parity(fmt, M, K, opt):
    L = prepare_gpu(syn.custom_layer(800 + K, M=8, K=K, N=64), fmt=fmt, rank=RANK[fmt])
    d = _inputs(1, M, K, **opt)
    got = run(L, d)
    check(L, d, got)
    compare_with_first_kernel(L, got, M, K)


@pytest.mark.parametrize("fmt,K", [("w8a8", 9216), ("nvfp4", 12288), ("int4", 14336), ("nvfp4", 8192)])
@pytest.mark.parametrize("M", [5, 900])
def test_norm_wide_rows(fmt, K, M):
    L = prepare_gpu(syn.custom_layer(820, M=8, K=K, N=32, calib_tokens=32), fmt=fmt, rank=RANK[fmt])
    d = _inputs(2, M, K, mods=2, center=True)
    got = run(L, d)
    check(L, d, got)
    compare_with_first_kernel(L, got, M, K)


@pytest.mark.parametrize("fmt,rank", [("nvfp4", 0), ("nvfp4", 32), ("int4", 0), ("int4", 32)])
def test_norm_with_adapter(fmt, rank):
    L = prepare_gpu(syn.custom_layer(830, M=8, K=512, N=64), fmt=fmt, rank=rank)
    rng = np.random.default_rng(31)
    L.set_lora(syn.bf16_bits(_bf(rng, 512, 20, a=0.05)), syn.bf16_bits(_bf(rng, 20, 64)), 0.5)
    for M in (37, 700):
        d = _inputs(3, M, 512, mods=1)
        got = run(L, d)
        check(L, d, got)
        compare_with_first_kernel(L, got, M, 512)


def test_norm_rank_zero_needs_no_xl():
    import torch
    L = prepare_gpu(syn.custom_layer(831, M=8, K=256, N=64), fmt="w8a8", rank=0)
    d = _inputs(4, 40, 256)
    x, s = torch_bf16(d["X"]), torch.empty((40, 256), dtype=torch.bfloat16, device="cuda")
    codes = torch.zeros(L.act_code_bytes(40), dtype=torch.uint8, device="cuda")
    scales = torch.zeros(L.act_scale_bytes(40), dtype=torch.uint8, device="cuda")
    L.norm_quantize_act(_norm(d, x, s), x, 40, codes, scales, None)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(to_numpy_f32(s), reference(d)[0])


@pytest.mark.parametrize("alias", ["x", "res"])
@pytest.mark.parametrize("M", [50, 900])
def test_sum_may_replace_an_input(alias, M):
    L = prepare_gpu(syn.custom_layer(832, M=8, K=512, N=64), fmt="w8a8", rank=16)
    d = _inputs(5, M, 512, mods=1, center=True)
    a, b = run(L, d), run(L, d, alias=alias)
    for k in ("h", "y", "codes_dev", "scales_dev", "xl"):
        np.testing.assert_array_equal(a[k], b[k])


@pytest.mark.parametrize("fmt", ["nvfp4", "int4", "w8a8"])
def test_constant_zero_huge_and_nan_rows(fmt):
    """A row of zeros or of one value (zero variance) gives finite output; large
    and tiny rows follow the formula; a NaN stays in its own row."""
    L = prepare_gpu(syn.custom_layer(833, M=8, K=256, N=64), fmt=fmt, rank=RANK[fmt])
    for center in (False, True):
        d = _inputs(6, 64, 256, residual=False, weight=True, center=center)
        d["X"][3] = 0.0
        d["X"][4] = 2.5
        d["X"][5] = syn.to_bf16(d["X"][5] * 1e15)
        d["X"][6] = syn.to_bf16(d["X"][6] * 1e-18)
        clean = run(L, d)
        check(L, d, clean)
        compare_with_first_kernel(L, clean, 64, 256)
        dirty = dict(d, X=d["X"].copy())
        dirty["X"][9, 17] = np.nan
        dirty["X"][10, 3] = np.inf
        x = torch_bf16(dirty["X"])
        import torch
        y = torch.empty((64, 256), dtype=torch.bfloat16, device="cuda")
        codes = torch.zeros(L.act_code_bytes(64), dtype=torch.uint8, device="cuda")
        scales = torch.zeros(L.act_scale_bytes(64), dtype=torch.uint8, device="cuda")
        xl = torch.zeros((64, 32), dtype=torch.bfloat16, device="cuda")
        L.norm_quantize_act(_norm(dirty, x, None), x, 64, codes, scales, xl, Y=y)
        torch.cuda.synchronize()
        keep = [r for r in range(64) if r not in (9, 10)]
        np.testing.assert_array_equal(to_numpy_f32(y)[keep], clean["y"][keep])
        np.testing.assert_array_equal(L.act_codes_to_logical(codes.cpu().numpy(), 64)[keep], clean["codes"][keep])
        assert np.all(np.isnan(to_numpy_f32(y)[9]))


@pytest.mark.parametrize("fmt,M,K,N", [("nvfp4", 77, 320, 272), ("int4", 300, 512, 144), ("w8a8", 257, 384, 512)])
def test_norm_linear_forward(fmt, M, K, N):
    import torch
    L = prepare_gpu(syn.custom_layer(840, M=8, K=K, N=N), fmt=fmt, rank=RANK[fmt])
    d = _inputs(7, M, K, mods=2, center=True)
    x = torch_bf16(d["X"])
    s = torch.empty((M, K), dtype=torch.bfloat16, device="cuda")
    y = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(L.workspace_bytes(M), dtype=torch.uint8, device="cuda")
    got = run(L, d)
    for flags, gelu in ((0, False), (lib.FWD_GELU, True)):
        L.norm_forward(_norm(d, x, s), x, M, y, ws, ws.numel(), torch.cuda.current_stream(), flags | lib.FWD_CHECK)
        ref = o.forward(oracle_prep_from(L), got["y"], gelu=gelu)["Y_bf16"]
        assert_close_bf16(to_numpy_f32(y), ref, f"{fmt} norm + layer")
        np.testing.assert_array_equal(to_numpy_f32(s), reference(d)[0])


def test_norm_captured_replayed_and_on_another_stream():
    import torch
    L = prepare_gpu(syn.custom_layer(850, M=8, K=512, N=128), fmt="nvfp4", rank=32)
    M = 700
    d, d2 = _inputs(8, M, 512, mods=1), _inputs(9, M, 512, mods=1)
    x = torch_bf16(d["X"])
    s = torch.empty((M, 512), dtype=torch.bfloat16, device="cuda")
    n = _norm(d, x, s)
    ws = torch.empty(L.workspace_bytes(M), dtype=torch.uint8, device="cuda")
    y = torch.empty((M, 128), dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        L.norm_forward(n, x, M, y, ws, ws.numel(), side)
    torch.cuda.synchronize()
    first = y.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        L.norm_forward(n, x, M, y, ws, ws.numel(), torch.cuda.current_stream())
    y.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, first)
    x.copy_(torch_bf16(d2["X"]))
    g.replay()
    torch.cuda.synchronize()
    replayed = y.clone()
    L.norm_forward(n, x, M, y, ws, ws.numel(), torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert torch.equal(y, replayed) and not torch.equal(y, first)


def test_operands_that_get_another_storage_are_followed():
    """A module's parameters keep their objects and change their storage when it is
    moved; a call reads what they hold then, and refuses host memory."""
    import torch
    L = prepare_gpu(syn.custom_layer(851, M=8, K=256, N=64), fmt="nvfp4", rank=32)
    M, d, d2 = 50, _inputs(10, 50, 256, mods=2), _inputs(11, 50, 256, mods=2)
    x, s = torch_bf16(d["X"]), torch.empty((M, 256), dtype=torch.bfloat16, device="cuda")
    made = {k: torch.nn.Parameter(torch_bf16(v), requires_grad=False)
            for k, v in (("residual", d["res"]), ("weight", d["weight"]), ("scale", d["mod"][:, 256:512]),
                         ("shift", d["mod"][:, :256]))}
    n = lib.Norm(sum=s, rows_per_mod=d["rows"], eps=EPS, **made)
    res = torch.nn.Parameter(torch.zeros((M, 64), dtype=torch.bfloat16, device="cuda"), requires_grad=False)
    epi = lib.Residual(res)
    codes = torch.empty(L.act_code_bytes(M), dtype=torch.uint8, device="cuda")
    scales = torch.empty(L.act_scale_bytes(M), dtype=torch.uint8, device="cuda")
    xl = torch.empty((M, 32), dtype=torch.bfloat16, device="cuda")
    y, out = torch.empty_like(s), torch.empty_like(res)

    def call():
        L.norm_quantize_act(n, x, M, codes, scales, xl, Y=y)
        L.gemm_residual(codes, scales, xl, M, epi, out)
        torch.cuda.synchronize()
        return to_numpy_f32(s), to_numpy_f32(y), to_numpy_f32(out)
    h, got, base = call()
    check(L, d, {"h": h, "y": got})
    for k, v in (("residual", d2["res"]), ("weight", d2["weight"]), ("scale", d2["mod"][:, 256:512]),
                 ("shift", d2["mod"][:, :256])):
        made[k].data = torch_bf16(v)
    s.zero_()
    h, got, base = call()
    check(L, dict(d2, X=d["X"]), {"h": h, "y": got})
    big = np.full((M, 64), 1024.0, np.float32)
    res.data = torch_bf16(big)
    moved = call()[2]
    # 1024 + y, rounded once: a step of 8 there
    assert np.all(np.abs(moved - 1024.0 - base) <= 4.0 + 2.0 ** -8 * np.abs(base))
    for p, name, f in ((made["weight"], "weight", call), (res, "residual", call)):
        keep = p.data
        p.data = p.data.cpu()
        with pytest.raises(ValueError, match=name):
            f()
        p.data = keep
    np.testing.assert_array_equal(call()[2], moved)
    made["weight"].untyped_storage().resize_(0)
    with pytest.raises(ValueError, match="released"):
        call()


# ------------------------------------------------------------------ every form of the kernel

def launched(fmt, M, K, nmt, sms):
    """(chunks, warps, blocks projected, unpredicated) of the kernel form that
    the launch rules choose."""
    def chunks(l):
        return -(-(K // 8) // (32 << l))

    def few(warps, l):
        return -(-M // (warps >> l)) < sms
    l, warps = 0, 8
    if nmt == 0:
        if chunks(3) > 4:
            warps = 16
        most = 4 if warps == 16 else 3
        while l < most and chunks(l) > 6:
            l += 1
        while l < most and few(warps, l):
            l += 1
        c = chunks(l)
        C = (4 if c <= 4 else 6) if warps == 16 else c if c <= 4 else 6
    else:
        while l < 3 and chunks(l) > 12:
            l += 1
        smem = (2 * 3 * 16 + 16) * 4 + 12 * K + (16 >> l) * (2 * K + 64) + 16 * nmt * 16 * 16 * 4
        C = 12
        if smem <= 232448:
            warps = 16
            while l < 3 and few(16, l):
                l += 1
            c = chunks(l)
            C = 2 if c <= 2 else 4 if c <= 4 else 6 if c <= 6 else 12
    spills = C == 12 and warps == 16 and (fmt == "w8a8" or (fmt == "int4" and nmt == 4))
    full = C >= 4 and not spills and not (nmt == 0 and warps == 16 and C == 4) and K == (256 * C) << l
    return fmt, C, warps, nmt, full


PLAIN = [  # M, K, options; rank 0, no adapter: codes and scales only
    (1, 64, dict()),
    (5, 3072, dict(center=True, mods=1)),           # few rows: eight warps to a row
    (130, 320, dict(residual=False, center=True)),
    (1201, 512, dict(mods=2, center=True)),
    (1201, 576, dict(weight=False, mods=401, rows_per_mod=3)),   # three or four modulation rows to a tile
    (1300, 128, dict(mods=1300, rows_per_mod=1, center=True)),   # ... one for each token
    (1201, 896, dict(weight=False, mods=2)),
    (1201, 1024, dict(residual=False)),             # every lane full: from four chunks on
    (1201, 1472, dict(mods=3)),
    (1201, 1536, dict(mods=2, center=True)),        # ... and one, two, four warps to a row
    (650, 3072, dict(mods=4, weight=False, center=True)),
    (300, 6144, dict(residual=False)),
    (300, 8192, dict(mods=2)),
    (5, 8256, dict(mods=2, center=True)),           # above 8192 columns: CTAs of 16 warps
    (300, 9216, dict(mods=2, center=True)),
    (301, 12288, dict(weight=False, mods=2)),
    (300, 14336, dict(center=True)),
]
PROJECT = [
    (50, 256, dict(mods=2)),
    (1201, 1920, dict(center=True)),
    (1201, 2048, dict(mods=2, center=True)),
    (1201, 576, dict(weight=False, mods=401, rows_per_mod=3)),
    (1201, 2816, dict(residual=False)),
    (1201, 3072, dict(mods=3, center=True)),
    (2401, 2944, dict(mods=2)),
    (2401, 3072, dict(mods=2, weight=False, center=True)),
    (1201, 6144, dict(residual=False, mods=1)),
    (301, 12288, dict(mods=2)),
    (300, 14336, dict(mods=2, center=True)),        # 16 rows do not fit in shared memory: CTAs of 8 warps
]
FORMS = ([(f, 0, M, K, o_) for f in ("nvfp4", "int4", "w8a8") for M, K, o_ in PLAIN]
         + [(f, n, M, K, o_) for f, n in (("w8a8", 1), ("nvfp4", 2), ("nvfp4", 4), ("int4", 2), ("int4", 4))
            for M, K, o_ in PROJECT])
_layers = {}


def _layer_of(fmt, nmt, K):
    """A layer whose norm projects nmt blocks of 16 branch columns: by its own
    rank, and with four by an adapter too."""
    key = (fmt, nmt, K)
    if key not in _layers:
        _layers.clear()                              # neighbours in FORMS differ in K
        d = syn.custom_layer(860 + K, M=8, K=K, N=64, calib_tokens=16)
        L = _layers[key] = prepare_gpu(d, fmt=fmt, rank=0 if nmt == 0 else RANK[fmt])
        if nmt == 4:
            rng = np.random.default_rng([32, K])
            L.set_lora(syn.bf16_bits(_bf(rng, K, 20, a=0.05)), syn.bf16_bits(_bf(rng, 20, 64)), 0.5)
    return _layers[key]


@pytest.mark.parametrize("fmt,nmt,M,K,opt", FORMS)
def test_every_form_of_the_kernel(fmt, nmt, M, K, opt):
    """h, y, codes, scales (byte for byte those of svdq_quantize_act on y) and XL."""
    L = _layer_of(fmt, nmt, K)
    d = _inputs(12 + nmt, M, K, **opt)
    got = run(L, d)
    check(L, d, got)
    compare_with_first_kernel(L, got, M, K)


def test_the_forms_above_are_all():
    import torch
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    reached = {launched(f, M, K, n, sms) for f, n, M, K, _ in FORMS}
    plain = [(C, 8, 0, False) for C in (1, 2, 3, 4, 6)] + [(C, 8, 0, True) for C in (4, 6)]
    plain += [(4, 16, 0, False), (6, 16, 0, False), (6, 16, 0, True)]
    want = {(f,) + v for f in ("nvfp4", "int4", "w8a8") for v in plain}
    for f, n in (("w8a8", 1), ("nvfp4", 2), ("nvfp4", 4), ("int4", 2), ("int4", 4)):
        want |= {(f, 2, 16, n, False)} | {(f, C, 16, n, full) for C in (4, 6, 12) for full in (False, True)}
        want |= {(f, 12, 8, n, full) for full in (False, True)}
    want -= {("w8a8", 12, 16, 1, True), ("int4", 12, 16, 4, True)}
    assert want == reached


@pytest.mark.parametrize("fmt,nmt,K", [("w8a8", 0, 576), ("w8a8", 1, 3072), ("nvfp4", 0, 1472), ("nvfp4", 2, 2944),
                                       ("int4", 2, 320), ("int4", 0, 14336)])
def test_rows_of_one_value_have_no_variance(fmt, nmt, K):
    """Layer norm of a row that holds one value is the shift, exactly: K equal BF16
    values (8 bits) add up without rounding (K < 2^14), and their sum divided by K
    is the value again."""
    import torch
    L = _layer_of(fmt, nmt, K)
    vals = syn.to_bf16(np.array([1000.0, -1000.0, 3.14, 1e4, 0.1, 77.7, -1e30, 2.0 ** -20], dtype=np.float32))
    M = len(vals)
    d = _inputs(30, M, K, residual=False, mods=1, center=True)
    d["X"][:] = vals[:, None]
    got = run(L, d)
    np.testing.assert_array_equal(got["y"], np.broadcast_to(d["mod"][0, :K], (M, K)))
    compare_with_first_kernel(L, got, M, K)


@pytest.mark.parametrize("fmt", ["nvfp4", "int4", "w8a8"])
@pytest.mark.parametrize("M,K", [(5, 320), (1201, 1024)])
def test_rows_too_small_for_a_reciprocal(fmt, M, K):
    """Normalised rows of 1e-36 down to BF16's smallest value: scales that are
    subnormal, or whose reciprocal is infinite, give the first kernel's codes."""
    L = _layer_of(fmt, 0, K)
    for w in (1e-36, 2e-37, 1e-38, 1e-39, 2e-40):
        d = _inputs(31, M, K)
        d["X"][0] = 0.0
        d["weight"] = syn.to_bf16(d["weight"] * np.float32(w))
        assert np.all(d["weight"][np.abs(d["weight"]) > 0] < 1e-35) and np.any(d["weight"] != 0)
        got = run(L, d)
        check(L, d, got)
        compare_with_first_kernel(L, got, M, K)


def test_an_operand_back_at_its_old_address_is_looked_at_again():
    """Storages freed and taken again by the allocator: the same address may hold
    another type or size by then."""
    import torch
    L = prepare_gpu(syn.custom_layer(852, M=8, K=1024, N=64), fmt="w8a8", rank=0)
    M, d = 20, _inputs(13, 20, 1024, residual=False)
    x, y = torch_bf16(d["X"]), torch.empty((M, 1024), dtype=torch.bfloat16, device="cuda")
    w = torch.nn.Parameter(torch_bf16(d["weight"]), requires_grad=False)
    n = lib.Norm(weight=w, eps=EPS)
    codes = torch.empty(L.act_code_bytes(M), dtype=torch.uint8, device="cuda")
    scales = torch.empty(L.act_scale_bytes(M), dtype=torch.uint8, device="cuda")

    def call():
        L.norm_quantize_act(n, x, M, codes, scales, None, Y=y)
        torch.cuda.synchronize()
        return to_numpy_f32(y)
    first = call()
    for other in (lambda t: t.float()[:512], lambda t: t.half(), lambda t: t[:512]):
        keep = w.data.cpu()
        w.data = keep                                   # the GPU's storage may be given back here ...
        w.data = other(keep).cuda()                     # ... and taken again
        with pytest.raises(ValueError, match="weight"):
            call()
        w.data = keep.cuda()
        np.testing.assert_array_equal(call(), first)
