"""GPU parity of the rotary positions with several axes (svdq_rope_heads) and of
the QKV path that applies them in place (svdq_qkv_forward).

Bar: every output within half a BF16 step of the float64 formula plus the FP32
error of the norm and the rotation.
"""
import numpy as np
import pytest

import synthetic as syn
from oracle import svdq_oracle as o

import w4a4_diffusion_transformer_b200 as lib
from gpu_util import prepare_gpu, to_numpy_f32, torch_bf16

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


def reference(x, pos, dims, theta=10000.0, half=False, span=False, norm=False, w=None):
    """x [B, T, H, D], pos [B, T, axes] -> (y, bound of its error), float64."""
    x = x.astype(np.float64)
    D, R = x.shape[-1], sum(dims)
    n = x
    if norm:
        n = x / np.sqrt((x * x).mean(-1, keepdims=True) + EPS)
        if w is not None:
            n = n * w.astype(np.float64)
    axis = np.repeat(np.arange(len(dims)), [d // 2 for d in dims])
    p = np.arange(R // 2)
    first = np.concatenate([[0], np.cumsum(dims)[:-1] // 2])[axis]
    expo = 2.0 * p / R if span else 2.0 * (p - first) / np.array(dims, dtype=np.float64)[axis]
    ang = pos.astype(np.float64)[..., axis] * theta ** -expo
    c, s = np.cos(ang)[:, :, None], np.sin(ang)[:, :, None]
    iu, iv = (p, p + R // 2) if half else (2 * p, 2 * p + 1)
    y, amp = n.copy(), np.abs(n)
    u, v = n[..., iu], n[..., iv]
    y[..., iu], y[..., iv] = u * c - v * s, v * c + u * s
    amp[..., iu] = amp[..., iv] = np.abs(u) + np.abs(v)
    # half a BF16 step; FP32: the mean square of D <= 256 values (8 + 5
    # additions in a row), rsqrtf, three products, the cosine's and sine's own
    # error (2 ulp, and an angle within 2^-24 of a turn's fraction: pi 2^-24)
    return y, 2.0 ** -8 * np.abs(y) + 32 * 2.0 ** -24 * amp + 1e-38


def assert_within(got, ref, tol):
    err = np.abs(got.astype(np.float64) - ref)
    assert np.all(err <= tol), (np.max(err / tol), np.unravel_index(np.argmax(err / tol), err.shape))


def _rand(rng, *shape, a=1.0, b=0.0):
    return syn.to_bf16(rng.standard_normal(shape) * a + b)


def _pos(rng, B, T, axes, far=False):
    return rng.integers(0, 3000000 if far else 64, (B, T, axes)).astype(np.float32)


CASES = [  # B, T, Hq, Hk, D, dims, options
    (1, 1, 1, 1, 8, (8,), dict()),
    (1, 1, 24, 24, 128, (16, 56, 56), dict(norm=True)),
    (1, 300, 24, 24, 128, (16, 56, 56), dict(norm=True)),
    (2, 77, 12, 12, 128, (44, 42, 42), dict(half=True, norm=True)),
    (2, 33, 8, 2, 64, (16, 16, 16), dict()),
    (1, 65, 5, 5, 72, (24, 24, 24), dict(norm=True)),
    (3, 17, 7, 1, 80, (16, 32, 32), dict(half=True, span=True)),
    (1, 130, 3, 3, 40, (2, 18, 20), dict(norm=True, span=True)),
    (2, 9, 4, 2, 256, (64, 96, 96), dict(half=True, norm=True)),
    (1, 12, 33, 11, 16, (2, 2, 2, 2), dict(theta=1e6)),
    (1, 5, 9, 3, 24, (16,), dict(half=True)),
    (1, 40, 2, 2, 104, (30, 6, 12), dict(half=True, norm=True)),
    (1, 7, 6, 6, 56, (2, 10, 14), dict(norm=True)),      # the span ends inside a lane's eight values
    (1, 9000, 2, 1, 64, (32, 32), dict(norm=True)),      # more tokens than warps in flight
]


@pytest.mark.parametrize("B,T,Hq,Hk,D,dims,opt", CASES)
@pytest.mark.parametrize("place", ["in", "out"])
def test_rope_parity(B, T, Hq, Hk, D, dims, opt, place):
    import torch
    rng = np.random.default_rng([5, B, T, Hq, D])
    W = (Hq + 2 * Hk) * D
    qkv = _rand(rng, B, T, W)
    pos = _pos(rng, B, T, len(dims))
    wq, wk = _rand(rng, D, a=0.2, b=1.0), _rand(rng, D, a=0.2, b=1.0)
    buf = torch_bf16(qkv)
    view = buf.view(B, T, Hq + 2 * Hk, D)
    q, k = view[:, :, :Hq], view[:, :, Hq:Hq + Hk]
    norm = opt.get("norm", False)
    rope = lib.Rope(D, dims, eps=EPS, **opt)
    tw = [torch_bf16(wq), torch_bf16(wk)]
    if place == "in":
        hq, hk = lib.Heads(q, weight=tw[0]), lib.Heads(k, weight=tw[1])
        oq, ok = q, k
    else:
        oq = torch.full((B, Hq, T, D), 9.0, dtype=torch.bfloat16, device="cuda").transpose(1, 2)
        ok = torch.full((B, T, Hk, D), 9.0, dtype=torch.bfloat16, device="cuda")
        hq, hk = lib.Heads(q, oq, tw[0]), lib.Heads(k, ok, tw[1])
    lib.rope_heads(rope, hq, hk, torch.from_numpy(pos).cuda(), torch.cuda.current_stream())
    torch.cuda.synchronize()
    x = qkv.reshape(B, T, -1, D)
    for got, src, w in ((oq, x[:, :, :Hq], wq), (ok, x[:, :, Hq:Hq + Hk], wk)):
        ref, tol = reference(src, pos, dims, w=w, **opt)
        assert_within(to_numpy_f32(got.contiguous()), ref, tol)
    # V, and out of place the input, are untouched
    after = to_numpy_f32(buf).reshape(B, T, -1, D)
    np.testing.assert_array_equal(after[:, :, Hq + Hk:], x[:, :, Hq + Hk:])
    if place == "out":
        np.testing.assert_array_equal(after, x)
    assert norm in (True, False)


def test_rope_far_fractional_and_negative_positions():
    import torch
    rng = np.random.default_rng(6)
    dims = (16, 24, 24)
    x = _rand(rng, 1, 64, 3, 64)
    for pos in (_pos(rng, 1, 64, 3, far=True), -_pos(rng, 1, 64, 3),
                (rng.standard_normal((1, 64, 3)) * 100).astype(np.float32),
                np.full((1, 64, 3), 16777216.0, dtype=np.float32)):
        out = torch.empty((1, 64, 3, 64), dtype=torch.bfloat16, device="cuda")
        lib.rope_heads(lib.Rope(64, dims), lib.Heads(torch_bf16(x), out), None, torch.from_numpy(pos).cuda())
        torch.cuda.synchronize()
        ref, tol = reference(x, pos, dims)
        assert_within(to_numpy_f32(out), ref, tol)


def test_rope_nonfinite_positions_and_values_stay_where_they_are():
    import torch
    rng = np.random.default_rng(7)
    dims = (8, 8)
    x = _rand(rng, 1, 6, 2, 32)
    x[0, 4, 1, 30] = np.nan
    pos = _pos(rng, 1, 6, 2)
    pos[0, 2, 1] = np.inf
    for norm in (False, True):
        out = torch.empty((1, 6, 2, 32), dtype=torch.bfloat16, device="cuda")
        lib.rope_heads(lib.Rope(32, dims, norm=norm), lib.Heads(torch_bf16(x), out), None,
                       torch.from_numpy(pos).cuda())
        torch.cuda.synchronize()
        bad = np.isnan(to_numpy_f32(out))
        want = np.zeros_like(bad)
        want[0, 2, :, 8:16] = True                       # the pairs of the axis with the bad position
        want[0, 4, 1, 30] = True
        if norm:
            want[0, 4, 1, :] = True                      # the head's norm
        np.testing.assert_array_equal(bad, want)


def test_rope_shared_and_own_positions():
    import torch
    rng = np.random.default_rng(8)
    x = torch_bf16(_rand(rng, 2, 20, 4, 64))
    pos = torch.from_numpy(_pos(rng, 1, 20, 2)).cuda()
    rope = lib.Rope(64, (32, 32), norm=True)
    outs = []
    for p in (pos[0], pos, torch.cat([pos, pos]).contiguous()):
        out = torch.empty_like(x)
        lib.rope_heads(rope, lib.Heads(x, out), None, p)
        outs.append(out)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_rope_captured_replayed_and_on_another_stream():
    import torch
    rng = np.random.default_rng(9)
    x = torch_bf16(_rand(rng, 1, 100, 6, 64))
    out = torch.empty_like(x)
    pos = torch.from_numpy(_pos(rng, 1, 100, 3)).cuda()
    rope, h = lib.Rope(64, (16, 24, 24), norm=True), lib.Heads(x, out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    lib.rope_heads(rope, h, None, pos, side)
    torch.cuda.synchronize()
    first = out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lib.rope_heads(rope, h, None, pos, torch.cuda.current_stream())
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first)


def test_rope_refuses_host_memory():
    import torch
    c = lib.HeadsStruct()
    host = torch.zeros((1, 1, 1, 64), dtype=torch.bfloat16).pin_memory()
    pos = torch.zeros((1, 1), device="cuda")
    import ctypes
    c.in_ = c.out = host.data_ptr()
    c.heads = 1
    rope = lib.Rope(64, (64,))
    assert lib.load().svdq_rope_heads(rope._ref, ctypes.addressof(c), None, 1, 1, pos.data_ptr(), 0, None) == lib.EINVAL


@pytest.mark.parametrize("fmt,rank", [("nvfp4", 32), ("int4", 32), ("w8a8", 16)])
@pytest.mark.parametrize("with_norm", [False, True])
def test_qkv_forward(fmt, rank, with_norm):
    import torch
    B, T, H, HK, D, K = 2, 45, 4, 2, 64, 256
    N = (H + 2 * HK) * D
    L = prepare_gpu(syn.custom_layer(870, M=8, K=K, N=N), fmt=fmt, rank=rank)
    rng = np.random.default_rng(10)
    M = B * T
    x = torch_bf16(_rand(rng, M, K, a=2.0))
    w = torch_bf16(_rand(rng, K, a=0.2, b=1.0))
    wq, wk = _rand(rng, D, a=0.2, b=1.0), _rand(rng, D, a=0.2, b=1.0)
    pos = _pos(rng, B, T, 3)
    norm = lib.Norm(weight=w) if with_norm else None
    ws = torch.empty(L.workspace_bytes(M), dtype=torch.uint8, device="cuda")
    base, y = (torch.empty((M, N), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    if with_norm:
        L.norm_forward(norm, x, M, base, ws, ws.numel())
    else:
        L.forward(x, M, base, ws, ws.numel())
    rope = lib.Rope(D, (16, 24, 24), norm=True, eps=EPS)
    L.qkv_forward(norm, x, B, T, rope, H, HK, torch.from_numpy(pos).cuda(), y, ws, ws.numel(), torch_bf16(wq),
                  torch_bf16(wk), torch.cuda.current_stream(), lib.FWD_CHECK)
    torch.cuda.synchronize()
    b, got = (to_numpy_f32(t).reshape(B, T, -1, D) for t in (base, y))
    for sl, wt in ((slice(0, H), wq), (slice(H, H + HK), wk)):
        ref, tol = reference(b[:, :, sl], pos, (16, 24, 24), norm=True, w=wt)
        assert_within(got[:, :, sl], ref, tol)
    np.testing.assert_array_equal(got[:, :, H + HK:], b[:, :, H + HK:])


def test_heads_that_get_another_storage_are_followed():
    import torch
    rng = np.random.default_rng(11)
    a, b = _rand(rng, 1, 30, 4, 64), _rand(rng, 1, 30, 4, 64)
    w = torch.nn.Parameter(torch_bf16(np.ones(64, np.float32)), requires_grad=False)
    x, out = torch_bf16(a), torch.empty((1, 30, 4, 64), dtype=torch.bfloat16, device="cuda")
    pos = _pos(rng, 1, 30, 1)
    rope, h = lib.Rope(64, (64,), norm=True, eps=EPS), lib.Heads(x, out, w)

    def call():
        lib.rope_heads(rope, h, None, torch.from_numpy(pos).cuda())
        torch.cuda.synchronize()
        return to_numpy_f32(out)
    assert_within(call(), *reference(a, pos, (64,), norm=True))
    x.data, w2 = torch_bf16(b), _rand(rng, 64, a=0.2, b=1.0)
    w.data = torch_bf16(w2)
    assert_within(call(), *reference(b, pos, (64,), norm=True, w=w2))
    out.data = torch.zeros_like(out)
    assert_within(call(), *reference(b, pos, (64,), norm=True, w=w2))
    w.data = w.data.cpu()
    with pytest.raises(ValueError, match="weight"):
        call()


@pytest.mark.parametrize("operand", ["q.in", "q.out", "q.weight", "k.in", "k.out", "k.weight", "positions"])
@pytest.mark.parametrize("pinned", [False, True])
def test_rope_refuses_host_memory_for_any_operand(operand, pinned):
    import ctypes

    import torch

    def memory(*shape, dtype=torch.bfloat16, name):
        if name != operand:
            return torch.ones(shape, dtype=dtype, device="cuda")
        t = torch.ones(shape, dtype=dtype)
        return t.pin_memory() if pinned else t
    hs, keep = [], []
    for name in ("q", "k"):
        t = [memory(1, 3, 2, 64, name=f"{name}.in"), memory(1, 3, 2, 64, name=f"{name}.out"),
             memory(64, name=f"{name}.weight")]
        h = lib.HeadsStruct()
        h.in_, h.out, h.weight = (x.data_ptr() for x in t)
        h.heads, h.in_token, h.in_head, h.out_token, h.out_head = 2, 128, 64, 128, 64
        assert all(a % 16 == 0 for a in (h.in_, h.out, h.weight))
        hs.append(h)
        keep.append(t)
    pos = memory(3, 1, dtype=torch.float32, name="positions")
    f = lib.load().svdq_rope_heads

    def call(rope):
        return f(rope._ref, ctypes.addressof(hs[0]), ctypes.addressof(hs[1]), 1, 3, pos.data_ptr(), 0, None)
    assert call(lib.Rope(64, (64,), norm=True)) == lib.EINVAL
    if operand.endswith("weight"):                      # not read without the norm
        assert call(lib.Rope(64, (64,))) == lib.OK
    torch.cuda.synchronize()
    assert bool((keep[1][1] == 1).all()) or operand.endswith("weight")


def test_positions_given_by_address_are_those_of_the_tensor():
    """Shared by all sequences, or each its own with the distance given."""
    import torch
    B, T, H, D, K = 3, 20, 2, 64, 128
    rng = np.random.default_rng(12)
    L = prepare_gpu(syn.custom_layer(871, M=8, K=K, N=3 * H * D))
    x = torch_bf16(_rand(rng, B * T, K))
    pos = torch.from_numpy(_pos(rng, B, T, 2)).cuda()
    rope = lib.Rope(D, (32, 32))
    ws = torch.empty(L.workspace_bytes(B * T), dtype=torch.uint8, device="cuda")
    q = torch_bf16(_rand(rng, B, T, H, D))
    for tensor, stride in ((pos, T * 2), (pos[0], 0)):
        a, b = (torch.empty((B * T, 3 * H * D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        c, d = torch.empty_like(q), torch.empty_like(q)
        L.qkv_forward(None, x, B, T, rope, H, H, tensor, a, ws, ws.numel())
        L.qkv_forward(None, x, B, T, rope, H, H, tensor.data_ptr(), b, ws, ws.numel(), pos_batch=stride)
        lib.rope_heads(rope, lib.Heads(q, c), None, tensor)
        lib.rope_heads(rope, lib.Heads(q, d), None, tensor.data_ptr(), pos_batch=stride)
        torch.cuda.synchronize()
        assert torch.equal(a, b) and torch.equal(c, d)
    with pytest.raises(ValueError, match="pos_batch"):
        lib.rope_heads(rope, lib.Heads(q, c), None, pos, pos_batch=T * 2)
