"""CPU tests of the refusals of the operators around the layer: the
normalisation (svdq_norm), the residual epilogue (svdq_residual) and the rotary
positions (svdq_rope, svdq_heads).  Layers are host-only and addresses made up:
every call must be answered before any of them is used -- bad arguments with
SVDQ_EINVAL, what is not built with SVDQ_EUNSUPPORTED, and a good call with
SVDQ_ESTATE for want of a device copy.
"""
import ctypes

import numpy as np
import pytest

import synthetic as syn

import w4a4_diffusion_transformer_b200 as lib

A = 1 << 30                                   # made-up 16-byte aligned addresses, a gigabyte apart
B, C, D, E, F = 2 * A, 3 * A, 4 * A, 5 * A, 6 * A


@pytest.fixture(scope="module", autouse=True)
def built():
    from w4a4_diffusion_transformer_b200 import build
    build.build()
    lib.load()


def _layer(K=256, N=128, fmt="nvfp4", rank=32):
    d = syn.custom_layer(61, M=16, K=K, N=N, calib_tokens=8)
    return lib.Layer.prepare(syn.bf16_bits(d["W"]), None, None if fmt == "w4a16" else syn.bf16_bits(d["Xc"]), fmt=fmt,
                             rank=rank if fmt != "w4a16" else 0, device=-1)


@pytest.fixture(scope="module")
def layer():
    return _layer()


def status(fn):
    try:
        fn()
    except lib.SvdqError as e:
        return e.status
    return lib.OK


# ------------------------------------------------------------------ normalisation

def norm_call(L, M=4, X=A, codes=B, scales=C, xl=D, Y=None, **kw):
    return status(lambda: L.norm_quantize_act(lib.Norm(**kw), X, M, codes, scales, xl, None, Y))


def test_norm_good_call_wants_a_device(layer):
    assert norm_call(layer) == lib.ESTATE
    assert norm_call(layer, residual=E, sum=F, weight=E, scale=E, shift=E, mod_stride=512, rows_per_mod=2,
                     center=True) == lib.ESTATE
    assert norm_call(layer, sum=A) == lib.ESTATE                       # in place of X
    assert norm_call(layer, residual=E, sum=E) == lib.ESTATE           # ... or of the residual
    assert norm_call(_layer(fmt="w8a8", rank=0), xl=None) == lib.ESTATE


@pytest.mark.parametrize("kw", [
    dict(X=None), dict(X=A + 8), dict(codes=None), dict(codes=B + 2), dict(scales=None), dict(scales=C + 4),
    dict(xl=D + 8), dict(M=0), dict(M=-3), dict(Y=F + 2),
    dict(residual=E + 8), dict(sum=E + 8), dict(weight=E + 2), dict(scale=E + 4), dict(shift=E + 8),
    dict(eps=0.0), dict(eps=-1e-6), dict(eps=float("nan")), dict(eps=float("inf")),
    dict(scale=E, mod_stride=12, rows_per_mod=2), dict(scale=E, mod_stride=-8, rows_per_mod=2),
    dict(shift=E, mod_stride=256, rows_per_mod=-1),
    dict(sum=A + 16), dict(sum=A - 256), dict(residual=E, sum=E + 32),
    dict(sum=E, weight=E + 16), dict(sum=E, shift=E - 1024, mod_stride=512, rows_per_mod=2),
    dict(Y=A), dict(Y=A + 1024), dict(residual=E, Y=E), dict(sum=E, Y=E + 2032)])
def test_norm_refuses(layer, kw):
    assert norm_call(layer, **kw) == lib.EINVAL


def test_norm_refuses_flags_missing_xl_and_null(layer):
    n = lib.Norm()
    n._c.flags = 2
    f = lib.load().svdq_norm_quantize_act
    assert f(layer._h, n._ref, A, 4, B, C, D, None, None) == lib.EINVAL
    assert f(layer._h, None, A, 4, B, C, D, None, None) == lib.EINVAL
    assert f(None, lib.Norm()._ref, A, 4, B, C, D, None, None) == lib.EINVAL
    assert f(layer._h, lib.Norm()._ref, A, 4, B, C, None, None, None) == lib.EINVAL


def test_norm_unsupported():
    assert norm_call(_layer(fmt="w4a16")) == lib.EUNSUPPORTED
    wide = _layer(K=14336 + 64, N=16, fmt="w8a8", rank=0)
    assert norm_call(wide, xl=None) == lib.EUNSUPPORTED
    assert norm_call(_layer(K=14336, N=16, fmt="w8a8", rank=0), xl=None) == lib.ESTATE


def test_norm_forward_refuses(layer):
    n, need = lib.Norm(), layer.workspace_bytes(4)

    def call(X=A, Y=E, ws=F, wsb=need, flags=0, norm=n, M=4):
        return status(lambda: layer.norm_forward(norm, X, M, Y, ws, wsb, None, flags))
    assert call() == lib.ESTATE
    assert call(flags=lib.FWD_GELU | lib.FWD_CHECK) == lib.ESTATE
    for bad in (dict(X=None), dict(Y=None), dict(Y=E + 8), dict(ws=None), dict(ws=F + 16), dict(wsb=need - 1),
                dict(Y=A), dict(Y=A + 16), dict(norm=lib.Norm(sum=E)), dict(M=0)):
        assert call(**bad) == lib.EINVAL, bad
    for flags in (lib.FWD_UNFUSED, lib.FWD_NO_BRANCH, 0x100):
        assert call(flags=flags) == lib.EUNSUPPORTED


# ------------------------------------------------------------------ residual

def test_residual_refuses(layer):
    def call(res=D, M=4, codes=A, scales=B, xl=C, Y=E, flags=0, L=layer, **kw):
        return status(lambda: L.gemm_residual(codes, scales, xl, M, lib.Residual(res, **kw), Y, None, flags))
    assert call() == lib.ESTATE
    assert call(res=E) == lib.ESTATE                                   # in place
    assert call(gate=F, gate_stride=256, rows_per_gate=2) == lib.ESTATE
    for bad in (dict(res=None), dict(res=D + 8), dict(res=E + 16), dict(res=E - 512), dict(Y=None), dict(Y=E + 2),
                dict(codes=None), dict(M=0), dict(gate=F + 8), dict(gate=F, gate_stride=4, rows_per_gate=1),
                dict(gate=F, gate_stride=-8, rows_per_gate=1), dict(gate=F, gate_stride=128, rows_per_gate=-1),
                dict(scales=B + 2), dict(xl=C + 4), dict(gate=E), dict(gate=E - 256, gate_stride=128, rows_per_gate=2)):
        assert call(**bad) == lib.EINVAL, bad
    assert call(flags=lib.FWD_UNFUSED) == lib.EUNSUPPORTED
    assert call(L=_layer(fmt="w4a16")) in (lib.EUNSUPPORTED, lib.ESTATE)
    need = layer.workspace_bytes(4)

    def fwd(X=A, Y=E, ws=F, wsb=need, flags=0, res=D):
        return status(lambda: layer.forward_residual(X, 4, lib.Residual(res), Y, ws, wsb, None, flags))
    assert fwd() == lib.ESTATE
    for bad in (dict(X=None), dict(X=A + 2), dict(Y=A), dict(Y=A + 64), dict(res=None), dict(res=E + 32)):
        assert fwd(**bad) == lib.EINVAL, bad
    for flags in (lib.FWD_UNFUSED, lib.FWD_NO_BRANCH):
        assert fwd(flags=flags) == lib.EUNSUPPORTED
    assert lib.load().svdq_gemm_residual(layer._h, A, B, C, 4, None, E, None, 0) == lib.EINVAL


def test_mlp_block_refuses():
    fc1, fc2 = _layer(K=256, N=512), _layer(K=512, N=256)
    f = lib.load().svdq_mlp_block_forward
    n, r = lib.Norm(sum=A), lib.Residual(A)

    def call(a=fc1, b=fc2, norm=n, X=A, M=4, res=r, Y=A, ws=F, wsb=1 << 28, flags=lib.FWD_GELU):
        return f(a and a._h, b and b._h, norm and norm._ref, X, M, res and res._ref, Y, ws, wsb, None, flags)
    assert call() == lib.ESTATE                                        # the stream in place throughout
    assert call(norm=None, res=None, Y=E) == lib.ESTATE
    for bad in (dict(X=None), dict(Y=None), dict(M=0), dict(b=None), dict(a=None), dict(norm=lib.Norm(eps=0.0)),
                dict(res=lib.Residual(A + 16)), dict(norm=lib.Norm(sum=A + 64))):
        assert call(**bad) == lib.EINVAL, bad


# ------------------------------------------------------------------ rotary positions

def heads(in_=A, out=B, n=2, weight=None, **strides):
    h = lib.HeadsStruct()
    h.in_, h.out, h.heads, h.weight = in_, out, n, weight
    s = dict(in_batch=4 * 128, in_token=128, in_head=64, out_batch=4 * 128, out_token=128, out_head=64)
    s.update(strides)
    for k, v in s.items():
        setattr(h, k, v)
    return h


def rope_call(rope=None, q="default", k=None, batch=2, T=4, positions=C, pos_batch=0):
    rope = lib.Rope(64, (16, 24, 24)) if rope is None else rope
    q = heads() if q == "default" else q
    return lib.load().svdq_rope_heads(rope._ref, None if q is None else ctypes.addressof(q),
                                      None if k is None else ctypes.addressof(k), batch, T, positions, pos_batch, None)


def mended(**kw):
    r = lib.Rope(64, (16, 24, 24))
    for k, v in kw.items():
        if k == "dim":
            for i, d in enumerate(v):
                r._c.dim[i] = d
        else:
            setattr(r._c, k, v)
    return r


@pytest.mark.parametrize("kw", [
    dict(axes=0), dict(axes=5), dict(axes=-1), dict(dim=(16, 0, 24)), dict(dim=(15, 24, 24)), dict(dim=(-2, 24, 24)),
    dict(dim=(16, 24, 26)), dict(head_dim=0), dict(theta=0.0), dict(theta=-1.0), dict(theta=float("nan")),
    dict(theta=float("inf")), dict(flags=8), dict(flags=lib.ROPE_NORM, eps=0.0),
    dict(flags=lib.ROPE_NORM, eps=float("nan"))])
def test_rope_refuses_its_description(kw):
    assert rope_call(mended(**kw)) == lib.EINVAL


def test_rope_unsupported_sizes():
    assert rope_call(lib.Rope(68, (16, 24, 24))) == lib.EUNSUPPORTED       # not a multiple of 8
    assert rope_call(lib.Rope(264, (16, 24, 24))) == lib.EUNSUPPORTED
    assert rope_call(lib.Rope(64, (16, 24, 20), half=True)) == lib.EUNSUPPORTED   # halves of 30 values


@pytest.mark.parametrize("q", [
    None, heads(in_=None), heads(out=None), heads(in_=A + 8), heads(out=B + 2), heads(weight=C + 4), heads(n=0),
    heads(in_token=-128), heads(out_head=60), heads(in_head=4),
    heads(out_head=0), heads(out_token=64), heads(out_batch=0), heads(out_head=56),       # outputs that meet
    heads(out=A, out_head=256, out_token=64), heads(out=A + 128), heads(out=A, out_token=256, out_batch=1024),
    heads(out=A + 16)])
def test_rope_refuses_heads(q):
    assert rope_call(q=q) == lib.EINVAL
    if q is not None:
        assert rope_call(k=q) == lib.EINVAL


@pytest.mark.parametrize("kw", [dict(batch=0), dict(T=0), dict(batch=-1), dict(batch=70000), dict(positions=None),
                                dict(positions=C + 2), dict(pos_batch=-1)])
def test_rope_refuses_calls(kw):
    assert rope_call(**kw) == lib.EINVAL
    assert lib.load().svdq_rope_heads(None, ctypes.addressof(heads()), None, 2, 4, C, 0, None) == lib.EINVAL


def test_rope_refuses_queries_that_are_keys():
    for q, k in ((heads(), heads(in_=D)),                               # both write B
                 (heads(), heads(in_=B, out=D)), (heads(in_=D, out=E), heads(in_=A, out=D))):
        assert rope_call(q=q, k=k) == lib.EINVAL


def test_rope_binding_checks_shapes():
    import torch
    x = torch.zeros((2, 4, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        lib.Heads(x)                                                    # host memory
    with pytest.raises(ValueError):
        lib.Rope(64, ())
    with pytest.raises(ValueError):
        lib.Rope(64, (8,) * 5)


def test_qkv_refuses():
    L = _layer(K=256, N=64 * 6)
    need = L.workspace_bytes(8)
    rope = lib.Rope(64, (16, 24, 24), norm=True)

    def call(norm=None, X=A, batch=2, T=4, rp=rope, hq=2, hk=2, qw=D, kw=D, pos=C, Y=E, ws=F, wsb=need, flags=0):
        return status(lambda: L.qkv_forward(norm, X, batch, T, rp, hq, hk, pos, Y, ws, wsb, qw, kw, None, flags))
    assert call() == lib.ESTATE
    assert call(norm=lib.Norm(weight=D)) == lib.ESTATE
    assert call(hk=0, qw=None, kw=None) == lib.ESTATE
    for bad in (dict(X=None), dict(Y=None), dict(batch=0), dict(T=0), dict(hq=0), dict(hk=-1), dict(hq=5, hk=2),
                dict(pos=None), dict(qw=D + 2), dict(Y=A), dict(norm=lib.Norm(eps=-1.0)), dict(rp=mended(axes=9))):
        assert call(**bad) == lib.EINVAL, bad
    assert call(flags=lib.FWD_GELU) == lib.EUNSUPPORTED


# ------------------------------------------------------------------ the binding's own checks

class FakeRows:
    """A CUDA BF16 tensor's shape and strides, no memory."""

    def __init__(self, shape, strides, dtype="torch.bfloat16", cuda=True):
        self.shape, self._s, self.is_cuda = shape, strides, cuda
        self.dtype = type("T", (), {"is_floating_point": True, "__str__": lambda s: dtype})()

    def dim(self):
        return len(self.shape)

    def stride(self, i=None):
        return self._s if i is None else self._s[i]

    def element_size(self):
        return 2

    def numel(self):
        return int(np.prod(self.shape))

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return D


def test_binding_checks_modulation_rows(layer):
    rows = lambda n, c, s=1536, **kw: FakeRows((n, c), (s, 1), **kw)  # noqa: E731
    with pytest.raises(ValueError, match="rows"):
        norm_call(layer, M=9, scale=rows(2, 256), rows_per_mod=4)      # three rows are read
    with pytest.raises(ValueError, match="columns"):
        norm_call(layer, scale=rows(2, 128), rows_per_mod=4)
    with pytest.raises(ValueError, match="BF16"):
        lib.Norm(scale=rows(1, 256, dtype="torch.float16"))
    with pytest.raises(ValueError, match="CUDA"):
        lib.Norm(shift=rows(1, 256, cuda=False))
    with pytest.raises(ValueError, match="distance"):
        lib.Norm(scale=rows(2, 256), shift=rows(2, 256, 512), rows_per_mod=4)
    with pytest.raises(ValueError, match="contiguous"):
        lib.Norm(scale=FakeRows((2, 256), (1, 2)))
    n = lib.Norm(scale=rows(3, 256), shift=rows(3, 256), rows_per_mod=4)
    assert n._c.mod_stride == 1536
    assert status(lambda: layer.norm_quantize_act(n, A, 9, B, C, E)) == lib.ESTATE
    r = lib.Residual(D, gate=rows(2, 128), rows_per_gate=4)
    assert r._c.gate_stride == 1536
    with pytest.raises(ValueError, match="rows"):
        layer.gemm_residual(A, B, C, 9, r, E)
    assert status(lambda: layer.gemm_residual(A, B, C, 8, r, E)) == lib.ESTATE


def _other_storage(t, ptr, **kw):
    """The same tensor object with another storage, as tensor.data = ... leaves it."""
    for k, v in dict(data_ptr=lambda: ptr, **kw).items():
        setattr(t, k, v)


def test_binding_follows_operands_to_another_storage(layer):
    """Addresses and placement are those at the call, not those when the object was made."""
    made = {"residual": FakeRows((4, 256), (256, 1)), "sum": FakeRows((4, 256), (256, 1)),
            "weight": FakeRows((256,), (1,)), "scale": FakeRows((2, 256), (1536, 1)),
            "shift": FakeRows((2, 256), (1536, 1))}
    for i, t in enumerate(made.values()):
        t.data_ptr = lambda i=i: (10 + i) * A
    n = lib.Norm(rows_per_mod=2, **made)
    assert status(lambda: layer.norm_quantize_act(n, A, 4, B, C, E)) == lib.ESTATE
    for i, (name, t) in enumerate(made.items()):
        assert getattr(n._c, name) == (10 + i) * A
        _other_storage(t, (20 + i) * A)
        assert status(lambda: layer.norm_quantize_act(n, A, 4, B, C, E)) == lib.ESTATE
        assert getattr(n._c, name) == (20 + i) * A
    for t in (made["scale"], made["shift"]):
        _other_storage(t, 30 * A, _s=(512, 1))          # rows another distance apart
    assert status(lambda: layer.norm_quantize_act(n, A, 4, B, C, E)) == lib.ESTATE
    assert n._c.mod_stride == 512
    for name, t in made.items():                        # moved to the host, and back
        _other_storage(t, 40 * A, is_cuda=False)
        for call in (lambda: layer.norm_quantize_act(n, A, 4, B, C, E),
                     lambda: layer.norm_forward(n, A, 4, E, F, layer.workspace_bytes(4)),
                     lambda: lib.mlp_block_forward(layer, layer, n, A, 4, None, E, F, 0)):
            with pytest.raises(ValueError, match=name):
                call()
        _other_storage(t, (50 + list(made).index(name)) * A, is_cuda=True)
    assert status(lambda: layer.norm_quantize_act(n, A, 4, B, C, E)) == lib.ESTATE
    _other_storage(made["weight"], 60 * A, shape=(128,))
    with pytest.raises(ValueError, match="weight"):
        layer.norm_quantize_act(n, A, 4, B, C, E)


def test_binding_follows_a_residual_and_a_gate(layer):
    res, gate = FakeRows((4, 128), (128, 1)), FakeRows((2, 128), (768, 1))
    res.data_ptr, gate.data_ptr = (lambda: 10 * A), (lambda: 11 * A)
    r = lib.Residual(res, gate, rows_per_gate=2)
    assert status(lambda: layer.gemm_residual(A, B, C, 4, r, E)) == lib.ESTATE
    _other_storage(res, 20 * A)
    _other_storage(gate, 21 * A, _s=(256, 1))
    assert status(lambda: layer.gemm_residual(A, B, C, 4, r, E)) == lib.ESTATE
    assert (r._c.residual, r._c.gate, r._c.gate_stride) == (20 * A, 21 * A, 256)
    _other_storage(res, E)                              # in place now
    assert status(lambda: layer.gemm_residual(A, B, C, 4, r, E)) == lib.ESTATE
    _other_storage(res, E + 64)                         # ... and over a part of Y
    assert status(lambda: layer.gemm_residual(A, B, C, 4, r, E)) == lib.EINVAL
    _other_storage(res, 22 * A)
    for t, name in ((gate, "gate"), (res, "residual")):
        _other_storage(t, 30 * A, is_cuda=False)
        for call in (lambda: layer.gemm_residual(A, B, C, 4, r, E),
                     lambda: layer.forward_residual(A, 4, r, E, F, layer.workspace_bytes(4)),
                     lambda: lib.mlp_block_forward(layer, layer, None, A, 4, r, E, F, 0)):
            with pytest.raises(ValueError, match=name):
                call()
        _other_storage(t, 31 * A, is_cuda=True)


def test_binding_follows_heads():
    def heads_of(ptr):
        t = FakeRows((2, 4, 2, 64), (512, 128, 64, 1))
        t.data_ptr, t.get_device = (lambda: ptr), (lambda: 0)
        return t
    x, out, w = heads_of(10 * A), heads_of(11 * A), FakeRows((64,), (1,))
    w.get_device = lambda: 0
    q = lib.Heads(x, out, w)
    rope, calls = lib.Rope(64, (16, 24, 20), half=True), []    # refused after the heads are taken

    def call():
        calls.append(status(lambda: lib.rope_heads(rope, q, None, C)))
        return q._c
    c = call()
    assert (c.in_, c.out, c.weight, c.out_token) == (10 * A, 11 * A, D, 128)
    _other_storage(x, 20 * A)
    _other_storage(out, 21 * A, _s=(1024, 256, 64, 1))
    _other_storage(w, 22 * A)
    c = call()
    assert (c.in_, c.out, c.weight, c.out_token) == (20 * A, 21 * A, 22 * A, 256)
    assert calls == [lib.EUNSUPPORTED] * 2
    for t, name in ((x, "x"), (out, "out"), (w, "weight")):
        _other_storage(t, 30 * A, is_cuda=False)
        with pytest.raises(ValueError, match=name):
            call()
        _other_storage(t, 31 * A, is_cuda=True)


def test_binding_asks_an_object_with_an_address_alone_each_time(layer):
    class Buffer:
        at = 10 * A

        def data_ptr(self):
            return self.at
    b = Buffer()
    n = lib.Norm(weight=b, sum=20 * A)
    assert status(lambda: layer.norm_quantize_act(n, A, 4, B, C, E)) == lib.ESTATE
    assert n._c.weight == 10 * A
    b.at = 20 * A                                       # over the sum now
    assert status(lambda: layer.norm_quantize_act(n, A, 4, B, C, E)) == lib.EINVAL


def test_binding_refuses_a_released_storage():
    import torch

    class Released(FakeRows):
        def storage_offset(self):
            return 0

        def untyped_storage(self):
            return torch.zeros(0, dtype=torch.bfloat16).untyped_storage()
    with pytest.raises(ValueError, match="released"):
        lib.Norm(weight=Released((256,), (1,)))
    with pytest.raises(ValueError, match="released"):
        lib.Residual(D, gate=Released((2, 256), (256, 1)))


def test_a_copied_rope_stands_on_its_own():
    """A copy passes its own struct, not the address of the one it was copied from."""
    import copy
    import pickle

    def passed(r):
        return bytes(ctypes.string_at(ctypes.addressof(r._ref._obj), ctypes.sizeof(r._c)))
    first = lib.Rope(64, (16, 24, 24), theta=1e4)
    copies = [copy.deepcopy(first), pickle.loads(pickle.dumps(first))]
    want = passed(first)
    first._c.head_dim, first._c.theta = -1, 0.0
    for r in copies:
        assert passed(r) == want
        assert r._ref._obj is r._c


# ------------------------------------------------------------------ outputs that meet anything else

def _near(at, n):
    """Addresses whose n bytes reach into those at `at`: from its start, its end, and from before."""
    return [at, at + n - 16, at - 16]


@pytest.mark.parametrize("name", ["residual", "weight", "scale", "shift", "sum"])
def test_norm_outputs_may_not_meet_its_operands(layer, name):
    M, K, N = 4, 256, 128
    rows = dict(mod_stride=512, rows_per_mod=2) if name in ("scale", "shift") else {}
    size = {"weight": 2 * K, "scale": 2 * (512 + K), "shift": 2 * (512 + K)}.get(name, 2 * M * K)
    kw = {name: 20 * A, **rows}
    assert norm_call(layer, Y=F, **kw) == lib.ESTATE
    for at in _near(20 * A, size):
        for out in ("Y", "codes", "scales", "xl"):
            assert norm_call(layer, **{out: at}, **kw) == lib.EINVAL, (out, at)
        assert norm_call(layer, Y=F, codes=B, **kw) == lib.ESTATE
    # ... and past its last byte, or in front of its first
    assert norm_call(layer, Y=20 * A + size, **kw) == lib.ESTATE
    assert norm_call(layer, Y=20 * A - 2 * M * K, **kw) == lib.ESTATE
    n, need = lib.Norm(**kw), layer.workspace_bytes(M)

    def fwd(Y=E, ws=F):
        return status(lambda: layer.norm_forward(n, A, M, Y, ws, need))
    assert fwd() == lib.ESTATE
    for at in _near(20 * A, size):
        assert fwd(Y=at) == lib.EINVAL
    for at in (20 * A, 20 * A - 256):
        assert fwd(ws=at) == lib.EINVAL
    assert fwd(Y=20 * A + size) == fwd(Y=20 * A - 2 * M * N) == lib.ESTATE


def test_norm_outputs_may_not_meet_each_other(layer):
    M = 4
    size = {"codes": layer.act_code_bytes(M), "scales": layer.act_scale_bytes(M), "xl": M * 64, "Y": M * 512}
    outs = dict(codes=B, scales=C, xl=D, Y=F)
    assert norm_call(layer, **outs) == lib.ESTATE
    for a in outs:
        for b in outs:
            if a != b:
                for at in _near(outs[b], size[b]):
                    assert norm_call(layer, **{**outs, a: at}) == lib.EINVAL, (a, b)
        for at in _near(A, M * 512):
            assert norm_call(layer, **{**outs, a: at}) == lib.EINVAL, a
    need = layer.workspace_bytes(M)
    for bad in (dict(ws=A), dict(ws=E), dict(Y=F + 512), dict(Y=F - 16)):
        c = {**dict(Y=E, ws=F), **bad}
        assert status(lambda: layer.norm_forward(lib.Norm(), A, M, c["Y"], c["ws"], need)) == lib.EINVAL, bad
    # rank 0 without an adapter writes no XL: what is passed for it does not count
    assert norm_call(_layer(fmt="w8a8", rank=0), xl=A) == lib.ESTATE


def test_rows_whose_last_has_no_address_are_refused(layer):
    far = (1 << 62) + 8
    assert norm_call(layer, scale=E, mod_stride=far, rows_per_mod=2) == lib.EINVAL
    assert norm_call(layer, scale=E, mod_stride=far, rows_per_mod=4) == lib.ESTATE     # one row
    for rows, want in ((2, lib.EINVAL), (4, lib.ESTATE)):
        r = lib.Residual(D, gate=F, gate_stride=far, rows_per_gate=rows)
        assert status(lambda: layer.gemm_residual(A, B, C, 4, r, E)) == want


def test_residual_outputs_may_not_meet_operands(layer):
    M, need = 4, layer.workspace_bytes(4)
    r = lib.Residual(D, gate=20 * A, gate_stride=256, rows_per_gate=2)

    def gemm(Y=E, **kw):
        c = {**dict(codes=A, scales=B, xl=C), **kw}
        return status(lambda: layer.gemm_residual(c["codes"], c["scales"], c["xl"], M, r, Y, None, c.get("flags", 0)))
    assert gemm() == lib.ESTATE
    for at, n in ((A, layer.act_code_bytes(M)), (B, layer.act_scale_bytes(M)), (C, M * 64), (20 * A, 2 * (256 + 128))):
        for y in _near(at, n):
            assert gemm(Y=y) == lib.EINVAL
        assert gemm(Y=at + n) == lib.ESTATE
    assert gemm(Y=C, flags=lib.FWD_NO_BRANCH) == lib.ESTATE            # XL is not read

    def fwd(Y=E, ws=F, X=A):
        return status(lambda: layer.forward_residual(X, M, r, Y, ws, need))
    assert fwd() == fwd(Y=D) == lib.ESTATE
    for at, n in ((A, M * 512), (D, M * 256), (E, M * 256), (20 * A, 768)):
        for ws in (at, at - 256, (at + n - 1) // 256 * 256):
            assert fwd(ws=ws) == lib.EINVAL


def test_qkv_outputs_may_not_meet_operands():
    L = _layer(K=256, N=64 * 6)
    M, need = 8, L.workspace_bytes(8)
    rope, plain = lib.Rope(64, (16, 24, 24), norm=True), lib.Rope(64, (16, 24, 24))

    def call(norm=None, qw=20 * A, kw=21 * A, pos=22 * A, Y=E, ws=F, rp=rope, hk=2):
        return status(lambda: L.qkv_forward(norm, A, 2, 4, rp, 2, hk, pos, Y, ws, need, qw, kw))
    norm = lib.Norm(sum=23 * A)
    for n in (None, norm):
        assert call(norm=n) == lib.ESTATE
        for at, size in ((20 * A, 128), (21 * A, 128), (22 * A, 48)):
            for y in _near(at, size):
                assert call(norm=n, Y=y) == lib.EINVAL
            assert call(norm=n, ws=at) == lib.EINVAL
            assert call(norm=n, Y=at + 16 * ((size + 15) // 16)) == lib.ESTATE
        assert call(norm=n, ws=E) == lib.EINVAL
        assert call(norm=n, ws=A) == lib.EINVAL
    for kw in (dict(qw=23 * A), dict(kw=23 * A + 64), dict(pos=23 * A + M * 512 - 4)):
        assert call(norm=norm, **kw) == lib.EINVAL
    assert call(Y=20 * A, rp=plain) == lib.ESTATE                      # weights are not read
    assert call(Y=21 * A, hk=0) == lib.ESTATE


def test_mlp_block_outputs_may_not_meet_operands():
    fc1, fc2 = _layer(K=256, N=512), _layer(K=512, N=256)
    M = 4
    need = 1 << 28                                                     # (host-only layers give no size)

    def call(norm=None, res=None, X=A, Y=E, ws=F):
        return status(lambda: lib.mlp_block_forward(fc1, fc2, norm, X, M, res, Y, ws, need, None, lib.FWD_GELU))
    rows = dict(mod_stride=512, rows_per_mod=2)
    stream = lib.Norm(sum=A, scale=20 * A, shift=21 * A, weight=22 * A, **rows)
    gated = lib.Residual(A, gate=24 * A, gate_stride=512, rows_per_gate=2)
    assert call(stream, gated, Y=A) == lib.ESTATE                      # the stream in place throughout
    assert call(lib.Norm(residual=23 * A, sum=B), lib.Residual(B), Y=23 * A) == lib.ESTATE
    for at in (20, 21, 22, 24):
        assert call(stream, gated, Y=at * A) == lib.EINVAL
    assert call(lib.Norm(sum=24 * A), gated) == lib.EINVAL             # the gate, read after the sum
    assert call(lib.Norm(sum=B), lib.Residual(B + 512)) == lib.EINVAL
    for at in (20, 21, 22, 24, 1):
        assert call(stream, gated, Y=A, ws=at * A) == lib.EINVAL
    assert call(None, None, ws=E) == call(None, None, ws=A) == lib.EINVAL


def _span(at, inner, terms):
    """All bytes of nested runs."""
    starts = np.array([at], dtype=np.int64)
    for stride, n in terms:
        starts = (starts[:, None] + stride * np.arange(n)[None]).reshape(-1)
    return (starts[:, None] + np.arange(inner)[None]).reshape(-1)


def _axes(h, side, heads_, B=2, T=4):
    return [(2 * getattr(h, f"{side}_{a}"), n) for a, n in (("batch", B), ("token", T), ("head", heads_))]


def test_rope_refuses_colliding_heads_and_takes_interleaved_ones():
    """q's and k's outputs against every other operand, byte by byte: heads of one
    fused buffer lie between each other, whatever their order; one value in common
    is refused."""
    rng = np.random.default_rng(20)
    B, T, D = 2, 4, 64
    rope, normed = lib.Rope(D, (16, 24, 24)), lib.Rope(D, (16, 24, 24), norm=True)
    taken = refused = 0
    for _ in range(700):
        fused = int(rng.integers(3, 8))                  # heads of a token in the fused buffer
        row = {"batch": T * fused * D, "token": fused * D, "head": D}
        if rng.random() < 0.3:                           # heads in front of tokens
            row = {"batch": T * fused * D, "head": T * D, "token": D}
        if rng.random() < 0.3:                           # room between heads
            row = {k: 2 * v for k, v in row.items()}

        def tensor(away):
            h, n = lib.HeadsStruct(), int(rng.integers(1, fused + 1))
            step = int(rng.integers(1, 3)) if n <= fused // 2 else 1
            h.heads, h.in_ = n, A + 16 * int(rng.choice([0, 8, 16, 24, 40])) * int(rng.integers(0, 3))
            for a in ("batch", "token", "head"):
                setattr(h, f"in_{a}", row[a] * (step if a == "head" else 1))
                setattr(h, f"out_{a}", row[a] * (step if a == "head" else 1))
            h.out = h.in_ + (away if rng.random() < 0.5 else 0)
            h.weight = int(rng.choice([D * A, h.out + 16 * int(rng.integers(-8, 300))])) if rng.random() < 0.3 else None
            return h
        q, k = tensor(A), tensor(int(rng.choice([A, 2 * A])))
        both = bool(rng.random() < 0.8)
        r = normed if rng.random() < 0.5 else rope
        pb = int(rng.choice([0, 12, 20]))
        pos = int(rng.choice([C * 64, q.out + 4 * int(rng.integers(-30, 1500))]))
        # each tensor by itself is taken where its outputs do not meet (checked elsewhere)
        tensors = [q, k] if both else [q]
        out = [_span(h.out, 2 * D, _axes(h, "out", h.heads)) for h in tensors]
        if any(len(np.unique(o_)) != len(o_) for o_ in out):
            continue
        bad = False
        for i, h in enumerate(tensors):
            others = [_span(pos, T * 12, [(4 * pb, B)])]
            others += [_span(g.weight, 2 * D, []) for g in tensors if r is normed and g.weight]
            if both:
                others += [_span(tensors[1 - i].in_, 2 * D, _axes(tensors[1 - i], "in", tensors[1 - i].heads)), out[1 - i]]
            bad = bad or any(len(np.intersect1d(out[i], o_)) for o_ in others)
        got = lib.load().svdq_rope_heads(r._ref, ctypes.addressof(q), ctypes.addressof(k) if both else None, B, T, pos,
                                         pb, None)
        assert (got == lib.EINVAL) == bad, ([[(f, getattr(h, f)) for f, _ in h._fields_] for h in tensors], pos, pb)
        taken, refused = taken + (not bad), refused + bad
    assert taken > 100 and refused > 100


def test_rope_takes_fused_heads_of_any_grouping():
    """Queries and keys of one buffer of grouped heads: one group's queries beside
    all groups' keys, at sizes whose elements could not be listed."""
    G, HK, D, B, T = 5, 8, 128, 300, 60000
    tok = HK * (G + 2) * D
    rope = lib.Rope(D, (32, 32, 64))

    def tensor(first, n, head):
        h = lib.HeadsStruct()
        h.in_ = h.out = A + 2 * first * D
        h.heads = n
        h.in_batch = h.out_batch = T * tok
        h.in_token = h.out_token = tok
        h.in_head = h.out_head = head
        return h

    def call(q, k):
        return lib.load().svdq_rope_heads(rope._ref, ctypes.addressof(q), ctypes.addressof(k), B, T, 1 << 50, 0, None)
    for g in range(HK):
        assert call(tensor(g * (G + 2), G, D), tensor(G, HK, (G + 2) * D)) != lib.EINVAL
        assert call(tensor(g * (G + 2) + 1, G, D), tensor(G, HK, (G + 2) * D)) == lib.EINVAL


def test_rope_refuses_sizes_that_pass_an_int():
    """Inputs of one broadcast head or token make such sizes possible; the
    kernel's indices run a step past the last."""
    for n in ((1 << 20) + 1, 2 ** 31 - 1):
        for q, k in ((heads(n=n, in_head=0, out_token=64 * n, out_batch=256 * n), None),
                     (heads(), heads(in_=D, out=1 << 45, n=n, in_head=0, out_token=64 * n, out_batch=256 * n))):
            assert rope_call(q=q, k=k) == lib.EINVAL
    assert rope_call(q=heads(in_=1 << 50, n=1 << 20, in_head=0, out_token=64 << 20, out_batch=256 << 20), batch=1,
                     positions=1 << 52) != lib.EINVAL
    one = dict(in_=1 << 50, n=1, in_token=0, out_token=64)
    assert rope_call(q=heads(**one), batch=1, T=2 ** 31 - 1, positions=1 << 52) == lib.EINVAL
    assert rope_call(q=heads(**one), batch=1, T=2 ** 31 - 5, positions=1 << 52) != lib.EINVAL


def test_binding_refuses_tensors_of_another_gpu(layer, monkeypatch):
    """The layer claims device 0 here, so that tensors of device 1 are refused before
    the library is called; the same call on device 0 reaches it."""
    monkeypatch.setattr(layer, "_device", 0)

    def on(dev, *shape, at=D):
        strides = tuple(int(np.prod(shape[i + 1:])) for i in range(len(shape)))
        t = FakeRows(shape, strides)
        t.nbytes, t.data_ptr, t.get_device = 2 * int(np.prod(shape)), (lambda: at), (lambda: dev)
        return t
    need = layer.workspace_bytes(4)
    norm, res = lib.Norm(), lib.Residual(20 * A)
    rope = lib.Rope(64, (16, 24, 24))
    act = {"X": ((4, 256), A), "codes": ((1 << 16,), B), "scales": ((1 << 16,), C), "xl": ((4, 32), D), "Y": ((4, 256), E),
           "workspace": ((need,), F), "positions": ((4, 3), 8 * A), "q_weight": ((64,), 9 * A),
           "k_weight": ((64,), 10 * A)}
    calls = {
        "norm_quantize_act": (("X", "codes", "scales", "xl", "Y"), lambda a: layer.norm_quantize_act(
            norm, a["X"], 4, a["codes"], a["scales"], a["xl"], None, a["Y"])),
        "norm_forward": (("X", "Y", "workspace"), lambda a: layer.norm_forward(
            norm, a["X"], 4, a["Y"], a["workspace"], need)),
        "gemm_residual": (("Y", "codes", "scales", "xl"), lambda a: layer.gemm_residual(
            a["codes"], a["scales"], a["xl"], 4, res, a["Y"])),
        "forward_residual": (("X", "Y", "workspace"), lambda a: layer.forward_residual(
            a["X"], 4, res, a["Y"], a["workspace"], need)),
        "qkv_forward": (("X", "Y", "workspace", "positions", "q_weight", "k_weight"), lambda a: layer.qkv_forward(
            norm, a["X"], 1, 4, rope, 1, 1, a["positions"], a["Y"], a["workspace"], need, a["q_weight"], a["k_weight"])),
        "mlp_block_forward": (("X", "Y", "workspace"), lambda a: lib.mlp_block_forward(
            layer, layer, norm, a["X"], 4, res, a["Y"], a["workspace"], need)),
    }
    for name, (operands, call) in calls.items():
        for wrong in (None,) + operands:
            a = {}
            for o_ in operands:
                shape, at = act[o_]
                a[o_] = on(1 if o_ == wrong else 0, *shape, at=at)
                if o_ == "positions":
                    a[o_].dtype = type("T", (), {"__str__": lambda s: "torch.float32"})()
            if wrong is None:
                assert status(lambda: call(a)) in (lib.ESTATE, lib.EUNSUPPORTED), name
            else:
                with pytest.raises(ValueError, match=f"{wrong}.*device 1"):
                    call(a)
    kw = {"residual": (4, 256), "sum": (4, 256), "weight": (256,), "scale": (1, 256), "shift": (1, 256)}
    for k, shape in kw.items():
        n = lib.Norm(**{k: on(1, *shape)})
        for f in (lambda: layer.norm_quantize_act(n, A, 4, B, C, E), lambda: layer.norm_forward(n, A, 4, E, F, need),
                  lambda: layer.qkv_forward(n, A, 1, 4, rope, 1, 1, C, E, F, need),
                  lambda: lib.mlp_block_forward(layer, layer, n, A, 4, None, E, F, need)):
            with pytest.raises(ValueError, match="Norm.*device 1"):
                f()
        with pytest.raises(ValueError, match="one device"):
            lib.Norm(**{**{k: on(1, *shape)}, **{("weight" if k != "weight" else "sum"): on(0, 4, 256)}})
    for r in (lib.Residual(on(1, 4, 128)), lib.Residual(B, gate=on(1, 1, 128))):
        for f in (lambda: layer.gemm_residual(A, 7 * A, C, 4, r, E), lambda: layer.forward_residual(A, 4, r, E, F, need),
                  lambda: lib.mlp_block_forward(layer, layer, None, A, 4, r, E, F, need)):
            with pytest.raises(ValueError, match="Residual.*device 1"):
                f()
    with pytest.raises(ValueError, match="one device"):
        lib.Residual(on(0, 4, 128), gate=on(1, 1, 128))
    with pytest.raises(ValueError, match="one device"):
        lib.Heads(on(0, 4, 2, 64), on(1, 4, 2, 64))


def test_binding_wants_the_stride_of_rows_given_by_address():
    """Without one every token would use row 0."""
    for kw in (dict(scale=E), dict(shift=E), dict(scale=E, shift=F)):
        with pytest.raises(ValueError, match="mod_stride"):
            lib.Norm(rows_per_mod=2, **kw)
        assert lib.Norm(**kw)._c.mod_stride == 0                       # one row for all tokens
        assert lib.Norm(rows_per_mod=2, mod_stride=512, **kw)._c.mod_stride == 512
    with pytest.raises(ValueError, match="gate_stride"):
        lib.Residual(D, gate=E, rows_per_gate=2)
    assert lib.Residual(D, gate=E)._c.gate_stride == 0
    assert lib.Residual(D, gate=E, rows_per_gate=2, gate_stride=256)._c.gate_stride == 256
    # an address beside a tensor takes the tensor's distance only if it is said
    rows = FakeRows((2, 256), (1536, 1))
    with pytest.raises(ValueError, match="mod_stride"):
        lib.Norm(scale=rows, shift=E, rows_per_mod=2)
    assert lib.Norm(scale=rows, shift=E, rows_per_mod=2, mod_stride=1536)._c.mod_stride == 1536
    with pytest.raises(ValueError, match="distance"):
        lib.Norm(scale=rows, shift=E, rows_per_mod=2, mod_stride=512)


def test_qkv_binding_wants_bf16_head_weights():
    L = _layer(K=256, N=64 * 6)
    rope = lib.Rope(64, (16, 24, 24), norm=True)

    def call(**kw):
        return status(lambda: L.qkv_forward(None, A, 2, 4, rope, 2, 2, C, E, F, L.workspace_bytes(8), **kw))
    assert call(q_weight=FakeRows((64,), (1,)), k_weight=FakeRows((64,), (1,))) == lib.ESTATE
    for name in ("q_weight", "k_weight"):
        with pytest.raises(ValueError, match=f"{name}.*BF16"):
            call(**{name: FakeRows((64,), (1,), dtype="torch.float16")})
        with pytest.raises(ValueError, match=f"{name}.*CUDA"):
            call(**{name: FakeRows((64,), (1,), cuda=False)})
