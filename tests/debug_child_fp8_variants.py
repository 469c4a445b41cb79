"""Child process of test_gpu_fp8_variants_debug_build: calls large enough for the FP8 variants that small
shapes do not reach, through ONE library file; a digest of every output saved.

    python tests/debug_child_fp8_variants.py <library.so> <out.npz>
"""
import hashlib
import os
import sys

import numpy as np

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

PROLOGUE = [(5003, 1152, 16), (10007, 1152, 32), (20001, 640, 16), (3001, 2176, 128), (4608, 2176, 32)]      # M, K, rank
GEMM = [(512, 512, 8192, 0), (300, 256, 8192, 48), (700, 2304, 640, 48), (1024, 3328, 640, 64), (2048, 2304, 384, 80)]


def main(lib_path: str, out: str) -> None:
    import torch

    from bit_w4a4_quantized_group_b200 import binding as B

    B.load(lib_path)
    g = torch.Generator(device="cuda").manual_seed(1)

    def rnd(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)

    def codes(n):
        return (torch.randint(0, 0x7F, (n,), generator=g, device="cuda", dtype=torch.int32)).to(torch.uint8)

    res = {}

    def keep(key, *tensors):
        torch.cuda.synchronize()
        h = hashlib.sha256()
        for t in tensors:
            h.update(t.view(torch.uint8).cpu().numpy().tobytes())
        res[key] = np.frombuffer(h.digest(), np.uint8)
        res[key + "_variant"] = np.array([B.svdq_last_variant()])

    for M, K, rank in PROLOGUE:
        sz = B.svdq_buffer_sizes("fp8", M, 128, K, rank)
        c, s = (torch.zeros(n, dtype=torch.uint8, device="cuda") for n in (sz.a_codes, sz.a_scales))
        Z = torch.zeros((M, rank), dtype=torch.bfloat16, device="cuda")
        lam = torch.exp(torch.randn((K,), generator=g, device="cuda"))
        B.quantize_act_lowrank_down_t("fp8", rnd(M, K), lam, 1.0, rnd(rank, K), c, s, Z)
        keep(f"prologue_{M}_{K}_{rank}", c, s, Z)
    for M, N, K, rank in GEMM:
        sz = B.svdq_buffer_sizes("fp8", M, N, K, rank)
        ac, wc = codes(sz.a_codes), codes(sz.w_codes)
        as_, ws = (torch.full((n,), 120, dtype=torch.uint8, device="cuda") for n in (sz.a_scales, sz.w_scales))
        Y = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
        B.w4a4_gemm_lowrank_up_t("fp8", M, N, K, rank, ac, as_, 1.0, wc, ws, 1.0, rnd(M, rank) if rank else None,
                                 rnd(N, rank) if rank else None, rnd(N), Y)
        keep(f"gemm_{M}_{N}_{K}_{rank}", Y)
    st, site = B.svdq_get_last_device_error(None)
    res["device_error"] = np.array([st, site])
    np.savez(out, **res)


if __name__ == "__main__":
    main(sys.argv[1], sys.argv[2])
