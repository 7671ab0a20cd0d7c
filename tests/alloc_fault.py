"""Run in a child process with alloc_fault.cpp preloaded: attaches an adapter
while one host allocation after the other fails.  Each failed call answers
SVDQ_ENOMEM and leaves a layer that works, with its previous adapter or with
none; on a GPU its outputs are those of such a layer, bit for bit."""
import ctypes
import sys

import numpy as np

import synthetic as syn

import w4a4_diffusion_transformer_b200 as lib

K, N, R = 256, 192, 8


def adapter(seed):
    rng = np.random.default_rng([9300, seed])
    return [syn.bf16_bits(syn.to_bf16(rng.standard_normal(s) * g)) for s, g in (((K, R), 0.05), ((R, N), 0.3))]


def held(L):
    """Which adapter the layer holds: None, or its exported factors."""
    if lib.load().svdq_tensor_bytes(L._h, lib.TENSORS["lora_A"][0]) == 0:
        return None
    return L.export("lora_A").copy(), L.export("lora_B").copy()


def outputs(L):
    import torch
    M = 40
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((M, K), generator=g, device="cuda").to(torch.bfloat16)
    y, yn = (torch.empty((M, N), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ws = torch.empty(L.workspace_bytes(M), dtype=torch.uint8, device="cuda")
    L.forward(x, M, y, ws, ws.numel(), flags=lib.FWD_CHECK)
    L.norm_forward(lib.Norm(), x, M, yn, ws, ws.numel(), flags=lib.FWD_CHECK)
    return y.cpu(), yn.cpu()


def main(device):
    fault = ctypes.CDLL(None)
    fault.fail_allocation.argtypes = [ctypes.c_long, ctypes.c_size_t]
    d = syn.custom_layer(140, M=8, K=K, N=N)
    failed = 0
    for fmt in ("nvfp4", "int4"):
        L = lib.Layer.prepare(syn.bf16_bits(d["W"]), syn.bf16_bits(d["bias"]), syn.bf16_bits(d["Xc"]), fmt=fmt,
                              rank=32, device=device)
        first, second = adapter(1), adapter(2)
        want = {}
        if device >= 0:
            for name, ab in (("none", None), ("first", first), ("second", second)):
                L.set_lora(*(ab or (None, None)))
                want[name] = outputs(L)

        def state():
            now = held(L)
            if now is None:
                return "none"
            for name, ab in (("first", first), ("second", second)):
                if all(np.array_equal(a, b) for a, b in zip(now, ab)):
                    return name
            raise AssertionError("the layer holds something else")
        for n in range(64):
            L.set_lora(*first)
            fault.fail_allocation(n, 1024)               # (the binding's own allocations are not C++'s)
            try:
                L.set_lora(*second)
                status = lib.OK
            except lib.SvdqError as e:
                status = e.status
            done = fault.allocation_fault_pending()
            s = state()
            assert (s == "second") if status == lib.OK else s in ("none", "first"), (n, status, s)
            if device >= 0:
                assert all(bool((a == b).all()) for a, b in zip(outputs(L), want[s])), (n, s)
            if done:
                assert status == lib.OK
                break
            assert status == lib.ENOMEM, (n, status)
            failed += 1
        else:
            raise AssertionError("the call never got through")
        L.close()
    print("failed", failed)


if __name__ == "__main__":
    main(int(sys.argv[1]))
