"""A W4A4 + low-rank linear layer held on one GPU (thin wrapper over the C ABI).

``forward(X)`` makes the two device calls of include/svdq.h on the current
stream: the prologue (smooth, quantize, down-project) and the fused GEMM
(4-bit product + up-projection + bias).  Buffers are preallocated with
PyTorch; nothing here computes any part of the layer.
"""
from __future__ import annotations

from typing import Optional

import numpy as np
import torch

from . import binding as B


def _to_dev_u16_as_bf16(a: np.ndarray, device) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).to(device).view(torch.bfloat16)


class W4A4LowRankLinear:
    def __init__(self, fmt: str, N: int, K: int, packed: dict, lam: Optional[np.ndarray], act_gscale: float,
                 bias: Optional[np.ndarray] = None, device="cuda"):
        self.fmt = fmt
        self.device = torch.device(device)
        self.N, self.K = int(N), int(K)
        self.rank = packed["L1_bf16"].shape[0]
        self.w_codes = torch.from_numpy(packed["w_codes"]).to(self.device)
        self.w_scales = torch.from_numpy(packed["w_scales"]).to(self.device)
        self._dev = self.w_codes.get_device()
        self.w_gscale = float(packed["w_gscale"])
        self.act_gscale = float(act_gscale)
        self.L1 = _to_dev_u16_as_bf16(packed["L1_bf16"], self.device) if self.rank else None
        self.L2 = _to_dev_u16_as_bf16(packed["L2_bf16"], self.device) if self.rank else None
        if lam is not None:
            lam32 = np.ascontiguousarray(lam, np.float32)
            # the smoothing divide x / lambda is an IEEE divide only for finite, normal, positive
            # lambda (the C ABI's contract); anything else is rejected here, before any launch
            tiny = np.finfo(np.float32).tiny
            if lam32.shape != (self.K,) or not np.all(np.isfinite(lam32) & (lam32 >= tiny)):
                raise ValueError("lambda must hold K finite, normal, positive float32 values")
            self.lam = torch.from_numpy(lam32).to(self.device)
        else:
            self.lam = None
        self.bias = None
        if bias is not None:
            # bf16 by round-to-nearest-even (torch's conversion), like every other bf16 operand
            b32 = torch.from_numpy(np.ascontiguousarray(bias, np.float32).reshape(-1))
            self.bias = b32.to(torch.bfloat16).to(self.device)
        self._ws = {}

    def workspace(self, M: int):
        """Preallocated activation codes / scales / Z for M rows."""
        if M not in self._ws:
            sz = B.svdq_buffer_sizes(self.fmt, M, self.N, self.K, self.rank)
            self._ws[M] = {
                "a_codes": torch.empty(sz.a_codes, dtype=torch.uint8, device=self.device),
                "a_scales": torch.empty(sz.a_scales, dtype=torch.uint8, device=self.device),
                "Z": torch.empty((M, self.rank), dtype=torch.bfloat16, device=self.device) if self.rank else None,
            }
        return self._ws[M]

    def forward(self, X: torch.Tensor, Y: Optional[torch.Tensor] = None, check: bool = False) -> torch.Tensor:
        """Y = the layer applied to X (both calls on the current stream, asynchronous).

        With ``check=True`` the call also synchronizes the stream and reads the library's
        device error word: a kernel whose bounded wait ran out (for instance on a GPU that
        is time-sliced with other work) leaves Y undefined, and this raises instead of
        returning it.  Without it, callers that need the guarantee poll
        ``binding.svdq_get_last_device_error`` themselves.
        """
        M, K = self._input_rows(X), self.K
        Y = self._output(M, Y)
        ws = self.workspace(M)
        stream = torch.cuda.current_stream(self.device).cuda_stream     # one lookup for both calls
        B.quantize_act_lowrank_down_t(self.fmt, X, self.lam, self.act_gscale, self.L1,
                                      ws["a_codes"], ws["a_scales"], ws["Z"], stream)
        B.w4a4_gemm_lowrank_up_t(self.fmt, M, self.N, K, self.rank, ws["a_codes"], ws["a_scales"],
                                 self.act_gscale, self.w_codes, self.w_scales, self.w_gscale,
                                 ws["Z"], self.L2, self.bias, Y, stream)
        if check:
            self._check_device("layer forward")
        return Y

    def _check_device(self, what: str):
        st, site = B.svdq_get_last_device_error(torch.cuda.current_stream(self.device).cuda_stream)
        if st != B.SVDQ_OK:
            raise B.SvdqError(st, f"{what} (device wait site {site})")

    def _input_rows(self, X: torch.Tensor) -> int:
        """M of a prologue's input, which the library reads as dense bf16 [M, K] on the current device."""
        if X.ndim != 2 or X.shape[1] != self.K or X.dtype is not torch.bfloat16 or not X.is_contiguous():
            raise ValueError(f"X: expected contiguous bfloat16 [M, {self.K}], got {tuple(X.shape)} {X.dtype}, "
                             f"strides {X.stride()}")
        if self._dev < 0 or X.get_device() != self._dev or B._current_device() != self._dev:
            raise ValueError(f"X on {X.device}: it and the layer (on {self.w_codes.device}) have to lie on the "
                             "current CUDA device")
        return X.shape[0]

    def _output(self, M: int, Y: Optional[torch.Tensor]) -> torch.Tensor:
        """Y for M rows: a new tensor, or the caller's, which the GEMM writes as dense bf16 [M, N]."""
        if Y is None:
            return torch.empty((M, self.N), dtype=torch.bfloat16, device=self.device)
        if Y.dtype is not torch.bfloat16 or Y.nbytes < 2 * M * self.N or not Y.is_contiguous() or Y.get_device() != self._dev:
            raise ValueError(f"Y: expected contiguous bfloat16 [{M}, {self.N}] on {self.w_codes.device}, got "
                             f"{tuple(Y.shape)} {Y.dtype}, strides {Y.stride()}, on {Y.device}")
        return Y

    def _check_width(self, t: torch.Tensor, name: str):
        """The workspace is sized by this layer's K: rows of another width would be written past its end."""
        if t.ndim != 2 or t.shape[1] != self.K:
            raise ValueError(f"{name}: expected [M, {self.K}], got {tuple(t.shape)}")

    def _check_fp8_feed(self, what: str):
        if self.fmt != "fp8" or self.rank != 0:
            raise ValueError(f"{what} feeds fp8 layers without a low-rank branch (this one: {self.fmt}, rank {self.rank})")

    def fold_gamma(self, gamma: torch.Tensor) -> torch.Tensor:
        """gamma / lambda in fp32: the weight of the norm before this layer, with the layer's smoothing
        folded in.  Made once, when the model is loaded."""
        g = gamma.to(device=self.device, dtype=torch.float32)
        return (g if self.lam is None else g / self.lam).contiguous()

    def forward_normed(self, X: torch.Tensor, residual: Optional[torch.Tensor], gamma: torch.Tensor, eps: float = 1e-6,
                       H: Optional[torch.Tensor] = None, Y: Optional[torch.Tensor] = None,
                       check: bool = False) -> torch.Tensor:
        """Y = the layer applied to RMSnorm(X + residual) * gamma, in two launches: the norm writes the
        layer's quantized input directly (fp8, rank 0).  `gamma` is fp32 [K] from fold_gamma (None: all
        ones, for a layer without smoothing); H, if given, receives X + residual in bf16 (it may be
        `residual` or X itself).  Like forward(), asynchronous on the current stream unless `check`."""
        self._check_fp8_feed("forward_normed")
        if gamma is None and self.lam is not None:
            raise ValueError("a layer with smoothing factors needs gamma from fold_gamma")
        self._check_width(X, "X")
        M = X.shape[0]
        Y = self._output(M, Y)
        ws = self.workspace(M)
        B.rmsnorm_quantize_act_t(self.fmt, X, residual, gamma, eps, H, ws["a_codes"], ws["a_scales"])
        self._gemm(M, Y)
        if check:
            self._check_device("layer forward_normed")
        return Y

    def forward_activated(self, act: str, gate: torch.Tensor, up: Optional[torch.Tensor] = None,
                          Y: Optional[torch.Tensor] = None, check: bool = False) -> torch.Tensor:
        """Y = the layer applied to act(gate) [* up], in two launches: the second layer of an MLP on the
        first one's output (fp8, rank 0).  act is "silu" or "gelu" (tanh form); gate and up may be
        column slices of one GEMM output.  `check` as in forward()."""
        self._check_fp8_feed("forward_activated")
        self._check_width(gate, "gate")
        M = gate.shape[0]
        Y = self._output(M, Y)
        ws = self.workspace(M)
        B.glu_quantize_act_t(self.fmt, act, gate, up, self.lam, ws["a_codes"], ws["a_scales"])
        self._gemm(M, Y)
        if check:
            self._check_device("layer forward_activated")
        return Y

    def gemm_only(self, M: int, Y: torch.Tensor, rank: Optional[int] = None):
        """The fused GEMM alone on the current workspace (rank 0 drops the branch)."""
        if self._dev < 0 or B._current_device() != self._dev:
            raise ValueError(f"the layer (on {self.w_codes.device}) has to lie on the current CUDA device")
        self._gemm(M, self._output(M, Y), rank)

    def _gemm(self, M: int, Y: torch.Tensor, rank: Optional[int] = None):
        ws = self.workspace(M)
        r = self.rank if rank is None else rank
        B.w4a4_gemm_lowrank_up_t(self.fmt, M, self.N, self.K, r, ws["a_codes"], ws["a_scales"],
                                 self.act_gscale, self.w_codes, self.w_scales, self.w_gscale,
                                 ws["Z"] if r else None, self.L2 if r else None, self.bias, Y)

    def prologue_only(self, X: torch.Tensor, rank: Optional[int] = None):
        """The prologue alone (rank 0 quantizes without the down projection)."""
        M = self._input_rows(X)
        ws = self.workspace(M)
        r = self.rank if rank is None else rank
        B.quantize_act_lowrank_down_t(self.fmt, X, self.lam, self.act_gscale, self.L1 if r else None,
                                      ws["a_codes"], ws["a_scales"], ws["Z"] if r else None)
