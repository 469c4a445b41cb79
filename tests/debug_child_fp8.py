"""Child process of test_gpu_fp8_debug_build: the FP8 operators on small odd shapes through ONE
library file (the release or the bounds-checking debug build), every output saved.

    python tests/debug_child_fp8.py <library.so> <out.npz>
"""
import os
import sys

import numpy as np

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

# (M, K, N, rank): one token, ragged token counts of every tile width, odd and even K steps, a K
# whose steps outnumber the ring, tiles that reach past N
SHAPES = [(1, 128, 128, 0), (1, 2048, 256, 16), (17, 640, 384, 0), (40, 4096, 128, 48), (100, 8192, 256, 0),
          (129, 384, 384, 16), (300, 640, 640, 48), (700, 1152, 3456, 0), (1025, 256, 3328, 16), (2048, 384, 2944, 16)]


def main(lib_path: str, out: str) -> None:
    import torch

    from bit_w4a4_quantized_group_b200 import binding as B
    from bit_w4a4_quantized_group_b200 import prepare as P
    from bit_w4a4_quantized_group_b200.layer import W4A4LowRankLinear

    B.load(lib_path)
    res = {}
    for (M, K, N, rank) in SHAPES:
        rng = np.random.default_rng(M * 7 + K + N + rank)
        X = rng.standard_normal((M, K)).astype(np.float32)
        X[:, rng.integers(0, K, 4)] *= 30.0
        prep = {"lam": rng.uniform(0.5, 4.0, K).astype(np.float32),
                "R_nk": (rng.standard_normal((N, K)) * 0.02).astype(np.float32),
                "L1_rk": (rng.standard_normal((rank, K)) * 0.05).astype(np.float32),
                "L2_nr": (rng.standard_normal((N, rank)) * 0.05).astype(np.float32), "act_gscale": 1.0}
        lin = W4A4LowRankLinear("fp8", N, K, P.pack("fp8", prep), prep["lam"], 1.0, None)
        Xd = torch.from_numpy(X).cuda().to(torch.bfloat16)
        key = f"{M}_{K}_{N}_{rank}"
        res[f"forward_{key}"] = lin.forward(Xd, check=True).view(torch.int16).cpu().numpy()
        if rank == 0:
            H = torch.empty_like(Xd)
            gamma = lin.fold_gamma(torch.ones(K))
            res[f"normed_{key}"] = lin.forward_normed(Xd, Xd, gamma, H=H).view(torch.int16).cpu().numpy()
            for act in ("silu", "gelu"):
                res[f"{act}_{key}"] = lin.forward_activated(act, Xd, H).view(torch.int16).cpu().numpy()
    # a row wider than the registers of a block: the norm's looping form
    W = 32896
    X = torch.from_numpy(np.random.default_rng(1).standard_normal((3, W)).astype(np.float32)).cuda().to(torch.bfloat16)
    sz = B.svdq_buffer_sizes("fp8", 3, 128, W, 0)
    codes = torch.zeros(sz.a_codes, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(sz.a_scales, dtype=torch.uint8, device="cuda")
    B.rmsnorm_quantize_act_t("fp8", X, X, None, 1e-6, X, codes, scales)
    res["wide_codes"], res["wide_scales"] = codes.cpu().numpy(), scales.cpu().numpy()
    torch.cuda.synchronize()
    st, site = B.svdq_get_last_device_error(None)
    res["device_error"] = np.array([st, site])
    np.savez(out, **res)


if __name__ == "__main__":
    main(sys.argv[1], sys.argv[2])
