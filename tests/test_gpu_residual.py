"""GPU parity of the residual epilogue (svdq_gemm_residual,
svdq_linear_forward_residual, svdq_mlp_block_forward), and of a whole
transformer block run through the operators around the layer.

Bar: within the tolerance every forward is held to, of the BF16 rounding of
residual + gate * layer(X) in float64; with a gate of zero the residual bit for
bit, and the plain forward's output with a residual of zero where both sum in
one order.
"""
import numpy as np
import pytest

import synthetic as syn
from oracle import svdq_oracle as o

import w4a4_diffusion_transformer_b200 as lib
from gpu_util import assert_close_bf16, oracle_prep_from, prepare_gpu, run_forward, to_numpy_f32, torch_bf16

pytestmark = pytest.mark.gpu

RANK = {"nvfp4": 32, "int4": 32, "w8a8": 16}
FORMATS = ["nvfp4", "int4", "w8a8"]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from w4a4_diffusion_transformer_b200 import build
    build.build()
    lib.load()


def _bf(rng, *shape, a=1.0):
    return syn.to_bf16(rng.standard_normal(shape) * a)


def _forward(L, X, res, gate=None, rows=0, flags=0, in_place=False, extra=3):
    """Y, and whether the rows behind the last stayed as they were."""
    import torch
    M, N = X.shape[0], L.info["N"]
    r = torch.full((M + extra, N), 4.0, dtype=torch.bfloat16, device="cuda")
    r[:M] = torch_bf16(res)
    y = r if in_place else torch.full((M + extra, N), 9.0, dtype=torch.bfloat16, device="cuda")
    g = None
    if gate is not None:
        wide = torch_bf16(np.concatenate([np.full_like(gate, np.nan), gate, np.full_like(gate, np.nan)], axis=1))
        g = wide[:, N:2 * N]                             # a column range of a wider modulation row
    ws = torch.empty(L.workspace_bytes(M), dtype=torch.uint8, device="cuda")
    epi = lib.Residual(r, gate=g, rows_per_gate=rows)
    L.forward_residual(torch_bf16(X), M, epi, y, ws, ws.numel(), torch.cuda.current_stream(), flags | lib.FWD_CHECK)
    torch.cuda.synchronize()
    assert bool((y[M:] == (4.0 if in_place else 9.0)).all())
    if not in_place:
        np.testing.assert_array_equal(to_numpy_f32(r[:M]), res)
    return to_numpy_f32(y[:M])


def _reference(L, X, res, gate=None, rows=0, gelu=False):
    y = o.forward(oracle_prep_from(L), X, gelu=gelu)["Y_act"]
    if gate is not None:
        row = np.arange(len(X)) // rows if rows else np.zeros(len(X), dtype=int)
        y = gate.astype(np.float64)[row] * y
    return o.bf16_round(res.astype(np.float64) + y)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,K,N,gates,rows", [
    (1, 64, 16, 0, 0), (77, 320, 272, 1, 0), (130, 512, 400, 2, 65), (200, 576, 528, 7, 29), (300, 256, 1040, 3, 100),
    (513, 1024, 256, 513, 1)])
@pytest.mark.parametrize("in_place", [False, True])
def test_residual_parity(fmt, M, K, N, gates, rows, in_place):
    d = syn.custom_layer(900 + M + N, M=M, K=K, N=N)
    L = prepare_gpu(d, fmt=fmt, rank=RANK[fmt])
    rng = np.random.default_rng([3, M, N])
    res, gate = _bf(rng, M, N, a=3.0), _bf(rng, gates, N) if gates else None
    y = _forward(L, d["X"], res, gate, rows, in_place=in_place)
    assert_close_bf16(y, _reference(L, d["X"], res, gate, rows), f"{fmt} residual")


@pytest.mark.parametrize("fmt", FORMATS)
def test_residual_after_gelu_and_with_adapter(fmt):
    d = syn.custom_layer(930, M=200, K=512, N=272)
    L = prepare_gpu(d, fmt=fmt, rank=RANK[fmt])
    rng = np.random.default_rng(4)
    res, gate = _bf(rng, 200, 272), _bf(rng, 1, 272)
    y = _forward(L, d["X"], res, gate, 0, flags=lib.FWD_GELU)
    assert_close_bf16(y, _reference(L, d["X"], res, gate, 0, gelu=True), f"{fmt} GELU, residual")
    if fmt != "w8a8":
        for rank in (0, 32):
            L = prepare_gpu(d, fmt=fmt, rank=rank)
            L.set_lora(syn.bf16_bits(_bf(rng, 512, 12, a=0.05)), syn.bf16_bits(_bf(rng, 12, 272, a=0.3)), 0.5)
            y = _forward(L, d["X"], res, gate, 0)
            assert_close_bf16(y, _reference(L, d["X"], res, gate, 0), f"{fmt} rank {rank} + adapter, residual")


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,K,N", [(100, 64, 256), (640, 1024, 1040), (2000, 128, 2304)])
def test_residual_of_zero_and_gate_of_zero(fmt, M, K, N):
    """A gate of zero gives the residual exactly; a residual of zero the plain
    forward: bit for bit where K is too short to be split over CTAs, otherwise
    the plain forward's bound."""
    d = syn.custom_layer(940 + K, M=M, K=K, N=N)
    L = prepare_gpu(d, fmt=fmt, rank=RANK[fmt])
    plain = run_forward(L, d["X"])
    ones = np.ones((1, N), np.float32)
    for y in (_forward(L, d["X"], np.zeros((M, N), np.float32)), _forward(L, d["X"], np.zeros((M, N), np.float32), ones)):
        if K <= 128:
            np.testing.assert_array_equal(y, plain)
        else:
            assert_close_bf16(y, plain, "residual of zero")
    res = _bf(np.random.default_rng(5), M, N)
    np.testing.assert_array_equal(_forward(L, d["X"], res, 0 * ones, in_place=True), res)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,K,N", [
    (1, 4096, 256),            # one tile, K over eight CTAs
    (77, 2048, 512), (300, 1088, 144), (513, 1600, 528),   # odd shares of K, ragged tiles
    (1100, 1024, 1936),        # 72 tiles: pairs
    (128, 3072, 3072),
    (140, 12288, 272)])        # every format over eight
def test_few_tiles_split_over_k(fmt, M, K, N):
    d = syn.custom_layer(945 + N, M=M, K=K, N=N)
    L = prepare_gpu(d, fmt=fmt, rank=RANK[fmt])
    rng = np.random.default_rng([6, M, N])
    res, gate = _bf(rng, M, N, a=3.0), _bf(rng, 3, N)
    rows = -(-M // 3)
    y = _forward(L, d["X"], res, gate, rows)
    assert_close_bf16(y, _reference(L, d["X"], res, gate, rows), f"{fmt} split, residual")
    # the partial sums are added in a fixed order
    np.testing.assert_array_equal(_forward(L, d["X"], res, gate, rows), y)
    if fmt != "w8a8":
        L.set_lora(syn.bf16_bits(_bf(rng, K, 12, a=0.05)), syn.bf16_bits(_bf(rng, 12, N, a=0.3)), 0.5)
    y = _forward(L, d["X"], res, None, 0, flags=lib.FWD_GELU, in_place=True)
    assert_close_bf16(y, _reference(L, d["X"], res, None, 0, gelu=True), f"{fmt} split, adapter, GELU, residual")


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,K,N", [(1, 2048, 272), (200, 1088, 528), (1003, 1216, 1040)])
def test_few_tiles_split_over_k_behind_a_norm(fmt, M, K, N):
    import torch
    d = syn.custom_layer(948 + N, M=M, K=K, N=N)
    L = prepare_gpu(d, fmt=fmt, rank=RANK[fmt])
    x = torch_bf16(d["X"])
    y = torch.full((M + 2, N), 9.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(L.workspace_bytes(M), dtype=torch.uint8, device="cuda")
    yn = torch.empty((M, K), dtype=torch.bfloat16, device="cuda")
    codes = torch.empty(L.act_code_bytes(M), dtype=torch.uint8, device="cuda")
    scales = torch.empty(L.act_scale_bytes(M), dtype=torch.uint8, device="cuda")
    xl = torch.empty((M, 32), dtype=torch.bfloat16, device="cuda")
    n = lib.Norm(center=True)
    L.norm_quantize_act(n, x, M, codes, scales, xl, None, yn)
    for flags, gelu in ((lib.FWD_CHECK, False), (lib.FWD_CHECK | lib.FWD_GELU, True)):
        L.norm_forward(n, x, M, y, ws, ws.numel(), None, flags)
        torch.cuda.synchronize()
        ref = o.forward(oracle_prep_from(L), to_numpy_f32(yn), gelu=gelu)["Y_bf16"]
        assert_close_bf16(to_numpy_f32(y[:M]), ref, f"{fmt} split behind a norm")
        assert bool((y[M:] == 9.0).all())


@pytest.mark.parametrize("fmt", FORMATS)
def test_split_captured_and_on_two_streams_at_once(fmt):
    """The same bytes from a replayed graph and from two streams whose clusters
    share the GPU."""
    import torch
    M, K, N = 100, 4096, 272
    d = syn.custom_layer(953, M=M, K=K, N=N)
    L = prepare_gpu(d, fmt=fmt, rank=RANK[fmt])
    x, res = torch_bf16(d["X"]), torch_bf16(_bf(np.random.default_rng(12), M, N))
    ws = [torch.empty(L.workspace_bytes(M), dtype=torch.uint8, device="cuda") for _ in range(2)]
    epi, norm = lib.Residual(res), lib.Norm(center=True)
    y, yn = torch.empty_like(res), torch.empty_like(res)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s = torch.cuda.current_stream()
        L.forward_residual(x, M, epi, y, ws[0], ws[0].numel(), s)
        L.norm_forward(norm, x, M, yn, ws[0], ws[0].numel(), s)
    graph.replay()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    out = [torch.empty_like(res) for _ in range(2)]
    for _ in range(10):
        for i in range(2):
            L.forward_residual(x, M, epi, out[i], ws[i], ws[i].numel(), streams[i])
    torch.cuda.synchronize()
    assert torch.equal(out[0], y) and torch.equal(out[1], y)
    L.norm_forward(norm, x, M, out[0], ws[0], ws[0].numel(), flags=lib.FWD_CHECK)
    torch.cuda.synchronize()
    assert torch.equal(out[0], yn)
    assert_close_bf16(to_numpy_f32(y), _reference(L, d["X"], to_numpy_f32(res), None, 0), f"{fmt} captured split")


@pytest.mark.parametrize("fmt", FORMATS)
def test_residual_over_several_waves(fmt):
    """More than two tiles per CTA: 4736 x 2560 is 370."""
    import torch
    M, K, N = 4736, 256, 2560
    d = syn.custom_layer(950, M=8, K=K, N=N)
    L = prepare_gpu(d, fmt=fmt, rank=RANK[fmt])
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((M, K), generator=g, device="cuda").to(torch.bfloat16)
    res = torch.randn((M, N), generator=g, device="cuda").to(torch.bfloat16)
    gate = torch.randn((3, N), generator=g, device="cuda").to(torch.bfloat16)
    ws = torch.empty(L.workspace_bytes(M), dtype=torch.uint8, device="cuda")
    zero, y0, y = torch.zeros_like(res), torch.empty_like(res), torch.empty_like(res)
    L.forward(x, M, y0, ws, ws.numel())
    L.forward_residual(x, M, lib.Residual(zero), y, ws, ws.numel())
    torch.cuda.synchronize()
    assert torch.equal(y, y0)
    L.forward_residual(x, M, lib.Residual(res, gate, 1600), y, ws, ws.numel(), flags=lib.FWD_CHECK)
    # gate * y rounds y to BF16 first here: half a step of |gate y| more
    row = torch.arange(M, device="cuda") // 1600
    gy = gate[row].float() * y0.float()
    ref = res.float() + gy
    assert bool(((y.float() - ref).abs() <= 2.0 ** -8 * (ref.abs() + gy.abs()) + 1e-30).all())


@pytest.mark.parametrize("fmt", FORMATS)
def test_residual_nonfinite_values_stay_where_they_are(fmt):
    d = syn.custom_layer(955, M=70, K=128, N=144)
    L = prepare_gpu(d, fmt=fmt, rank=RANK[fmt])
    res = _bf(np.random.default_rng(6), 70, 144)
    clean = _forward(L, d["X"], res)
    bad = res.copy()
    bad[11, 33], bad[69, 143], bad[40, 0] = np.nan, np.inf, -np.inf
    got = _forward(L, d["X"], bad)
    assert np.isnan(got[11, 33]) and got[69, 143] == np.inf and got[40, 0] == -np.inf
    keep = np.isfinite(bad)
    np.testing.assert_array_equal(got[keep], clean[keep])


def test_residual_captured_in_two_graphs_that_share_a_workspace():
    import torch
    d = syn.custom_layer(960, M=300, K=512, N=512)
    M = 300
    L = prepare_gpu(d)
    x = torch_bf16(d["X"])
    rng = np.random.default_rng(7)
    res = [torch_bf16(_bf(rng, M, 512)) for _ in range(2)]
    y = [torch.empty((M, 512), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    ws = torch.empty(L.workspace_bytes(M), dtype=torch.uint8, device="cuda")
    epi = [lib.Residual(r) for r in res]
    want = []
    for e, t in zip(epi, y):
        L.forward_residual(x, M, e, t, ws, ws.numel())
        torch.cuda.synchronize()
        want.append(t.clone())
    graphs = []
    for e, t in zip(epi, y):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            L.forward_residual(x, M, e, t, ws, ws.numel(), torch.cuda.current_stream())
        graphs.append(g)
    for t in y:
        t.zero_()
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(y, want))


def _mlp(K, F, seed):
    d1 = syn.custom_layer(seed, M=8, K=K, N=F)
    d2 = syn.custom_layer(seed + 1, M=8, K=F, N=K, outliers=False)
    return prepare_gpu(d1), prepare_gpu(d2)


@pytest.mark.parametrize("with_norm,with_res", [(False, False), (True, False), (False, True), (True, True)])
def test_mlp_block(with_norm, with_res):
    """Against the parts it is made of, on their own, within a BF16 rounding of
    the MLP's output."""
    import torch
    M, K, F = 333, 256, 512
    fc1, fc2 = _mlp(K, F, 970)
    rng = np.random.default_rng(8)
    x, w = torch_bf16(_bf(rng, M, K, a=2.0)), torch_bf16(syn.to_bf16(rng.standard_normal(K) * 0.2 + 1))
    gate = torch_bf16(_bf(rng, 3, K))
    wsb = lib.mlp_workspace_bytes(fc1, fc2, M, lib.FWD_GELU)
    ws = torch.empty(wsb, dtype=torch.uint8, device="cuda")
    norm = lib.Norm(weight=w, center=True) if with_norm else None
    xin = x
    if with_norm:
        xin = torch.empty_like(x)
        codes = torch.empty(fc1.act_code_bytes(M), dtype=torch.uint8, device="cuda")
        scales = torch.empty(fc1.act_scale_bytes(M), dtype=torch.uint8, device="cuda")
        fc1.norm_quantize_act(norm, x, M, codes, scales, torch.empty((M, 32), dtype=torch.bfloat16, device="cuda"),
                              Y=xin)
    y0 = torch.empty_like(x)
    lib.mlp_forward(fc1, fc2, xin, M, y0, ws, wsb, flags=lib.FWD_GELU)
    y = x.clone()                                        # the stream, updated in place
    res = lib.Residual(y, gate, 111) if with_res else None
    lib.mlp_block_forward(fc1, fc2, norm, y if with_res else x, M, res, y, ws, wsb, flags=lib.FWD_GELU | lib.FWD_CHECK)
    a, b = to_numpy_f32(y).astype(np.float64), to_numpy_f32(y0).astype(np.float64)
    if with_res:
        gy = to_numpy_f32(gate).astype(np.float64)[np.arange(M) // 111] * b
        ref = to_numpy_f32(x) + gy
        # XL sums in another order behind the fused norm: a BF16 rounding of XL,
        # like every forward's tolerance
        assert np.linalg.norm(a - ref) <= 2.0 ** -8 * (np.linalg.norm(ref) + np.linalg.norm(gy))
    elif with_norm:
        assert np.linalg.norm(a - b) <= 2e-3 * np.linalg.norm(b)
    else:
        # fc2's FP32 sums may be split over K: both sides round sums that agree to
        # F 2^-24 of their terms, so each is off by half a step, 2^-8, at most
        assert np.linalg.norm(a - b) <= 2.0 ** -8 * np.linalg.norm(b)


@pytest.mark.parametrize("fmt", FORMATS)
def test_transformer_block(fmt):
    """Norm -> QKV -> head norms and rotation -> attention -> gated projection ->
    norm -> gated MLP on a residual stream that is updated in place, modulated
    by one wide row per prompt; every stage against the oracle on its own input."""
    import torch
    B, T, H, D, F = 2, 60, 4, 64, 512
    M, K = B * T, H * D
    mk = lambda seed, k, n, out=True: prepare_gpu(  # noqa: E731
        syn.custom_layer(seed, M=8, K=k, N=n, outliers=out), fmt=fmt, rank=RANK[fmt])
    qkv, proj, fc1, fc2 = mk(980, K, 3 * K), mk(981, K, K, False), mk(982, K, F), mk(983, F, K, False)
    rng = np.random.default_rng(9)
    x0 = _bf(rng, M, K, a=2.0)
    mod = _bf(rng, B, 6 * K, a=0.3)
    wq, wk = _bf(rng, D, a=0.1) + 1.0, _bf(rng, D, a=0.1) + 1.0
    wq, wk = syn.to_bf16(wq), syn.to_bf16(wk)
    pos = rng.integers(0, 32, (T, 3)).astype(np.float32)
    x, m = torch_bf16(x0), torch_bf16(mod)
    cut = lambda i: m[:, i * K:(i + 1) * K]  # noqa: E731
    ws = torch.empty(max(L.workspace_bytes(M) for L in (qkv, proj, fc1, fc2)), dtype=torch.uint8, device="cuda")
    s = torch.cuda.current_stream()
    y = torch.empty((M, 3 * K), dtype=torch.bfloat16, device="cuda")
    n1 = lib.Norm(shift=cut(0), scale=cut(1), rows_per_mod=T, center=True)
    rope = lib.Rope(D, (16, 24, 24), norm=True)
    qkv.qkv_forward(n1, x, B, T, rope, H, H, torch.from_numpy(pos).cuda(), y, ws, ws.numel(), torch_bf16(wq),
                    torch_bf16(wk), s)
    h = y.view(B, T, 3, H, D).float()
    a = torch.softmax(torch.einsum("bthd,bshd->bhts", h[:, :, 0], h[:, :, 1]) / D ** 0.5, -1)
    att = torch.einsum("bhts,bshd->bthd", a, h[:, :, 2]).reshape(M, K).to(torch.bfloat16)
    x1 = x.clone()
    proj.forward_residual(att, M, lib.Residual(x1, cut(2), T), x1, ws, ws.numel(), s)   # in place
    u = torch.empty((M, F), dtype=torch.bfloat16, device="cuda")
    n2 = lib.Norm(shift=cut(3), scale=cut(4), rows_per_mod=T, center=True)
    fc1.norm_forward(n2, x1, M, u, ws, ws.numel(), s, lib.FWD_GELU)
    x2 = x1.clone()
    fc2.forward_residual(u, M, lib.Residual(x2, cut(5), T), x2, ws, ws.numel(), s, lib.FWD_CHECK)

    def normed(v, i):
        v = v.astype(np.float64)
        v = v - v.mean(1, keepdims=True)
        v = v / np.sqrt((v * v).mean(1, keepdims=True) + 1e-6)
        row = np.arange(M) // T
        return o.bf16_round(v * (1 + mod[row, (i + 1) * K:(i + 2) * K]) + mod[row, i * K:(i + 1) * K])

    from test_gpu_rope import reference as rotated
    ref = o.forward(oracle_prep_from(qkv), normed(x0, 0).astype(np.float32))["Y"].reshape(B, T, 3 * H, D)
    p = np.broadcast_to(pos, (B, T, 3))
    got = to_numpy_f32(y).reshape(B, T, 3 * H, D)
    for i, w in ((0, wq), (1, wk)):
        r = rotated(o.bf16_round(ref[:, :, i * H:(i + 1) * H]), p, (16, 24, 24), norm=True, w=w)[0]
        g = got[:, :, i * H:(i + 1) * H].astype(np.float64)
        # two BF16 roundings, and quantizer steps that the FP32 norm moves
        assert np.linalg.norm(g - r) <= 1e-2 * np.linalg.norm(r)
    gate = lambda i: mod[np.arange(M) // T, i * K:(i + 1) * K].astype(np.float64)  # noqa: E731
    r1 = o.bf16_round(x0 + gate(2) * o.forward(oracle_prep_from(proj), to_numpy_f32(att))["Y"])
    assert_close_bf16(to_numpy_f32(x1), r1, "projection, residual")
    ru = o.forward(oracle_prep_from(fc1), normed(to_numpy_f32(x1), 3).astype(np.float32), gelu=True)["Y_bf16"]
    assert np.linalg.norm(to_numpy_f32(u) - ru) <= 1e-2 * np.linalg.norm(ru)
    r2 = o.bf16_round(to_numpy_f32(x1) + gate(5) * o.forward(oracle_prep_from(fc2), to_numpy_f32(u))["Y"])
    assert_close_bf16(to_numpy_f32(x2), r2, "MLP, residual")
