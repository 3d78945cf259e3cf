"""FP8 rows and weights (E4M3 codes, one fp32 scale per block of 128) and their
product: torch buffers around ft_fp8_quant_rows, ft_fp8_pack and ft_fp8_gemm.

Codes are torch.float8_e4m3fn tensors [rows, K] whose rows start on 16 bytes
(a view of wider rows where K is not a multiple of 16); scales are fp32.
Every call is enqueued on ``stream`` (default: the current one) of the current
device, which has to be the tensors' own; the tensors that it returns are
allocated on that stream.
"""
from __future__ import annotations

from typing import Optional, Tuple

import torch

from . import _lib
from .layer import _allocating, _stream

FP8 = torch.float8_e4m3fn
_TYPES = {torch.float32: _lib.FT_F32, torch.bfloat16: _lib.FT_BF16, torch.float16: _lib.FT_F16}


def _blocks(n: int) -> int:
    return (n + 127) // 128


def _here(t: torch.Tensor) -> None:
    if t.get_device() != torch.cuda.current_device():
        raise ValueError(f"the tensors are on {t.device}, which is not the current device")


def empty_codes(rows: int, K: int, device) -> torch.Tensor:
    """float8 [rows, K] whose rows start on 16 bytes."""
    codes = torch.empty((rows, (K + 15) // 16 * 16), dtype=FP8, device=device)
    return codes if K % 16 == 0 else codes[:, :K]


def _check_codes(codes: torch.Tensor, scales: torch.Tensor, scale_rows: int, what: str) -> None:
    rows, K = codes.shape if codes.dim() == 2 else (0, 0)
    if codes.dtype != FP8 or K == 0 or (K > 1 and codes.stride(1) != 1):
        raise ValueError(f"{what}: codes must be float8_e4m3fn [rows, K] with contiguous rows")
    blocks = (K + 127) // 128
    if scales.dtype != torch.float32 or scales.shape != (scale_rows, blocks) or (blocks > 1 and scales.stride(1) != 1):
        raise ValueError(f"{what}: scales must be fp32 [{scale_rows}, {blocks}]")
    if not codes.is_cuda or codes.get_device() != scales.get_device():
        raise ValueError(f"{what}: codes and scales must be on one CUDA device")


def _pitch(t: torch.Tensor) -> int:
    """Elements between two rows (a matrix of one row may say anything)."""
    return t.stride(0) if t.shape[0] > 1 else max(t.stride(0), t.shape[1])


def _code_pitch(t: torch.Tensor) -> int:
    return t.stride(0) if t.shape[0] > 1 else (t.shape[1] + 15) // 16 * 16


def quantize_rows(x: torch.Tensor, codes: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None,
                  stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """x [M, K] (fp32, bf16 or fp16; contiguous rows) -> (codes [M, K], scales [M, ceil(K/128)])."""
    kind = _TYPES.get(x.dtype)
    if kind is None or x.dim() != 2 or not x.is_cuda or (x.shape[1] > 1 and x.stride(1) != 1):
        raise ValueError("quantize_rows: x must be a CUDA matrix of fp32, bf16 or fp16 with contiguous rows")
    _here(x)
    M, K = x.shape
    if codes is None and scales is None:     # the usual call: nothing of theirs to look up again
        pitch, blocks = (K + 15) // 16 * 16, (K + 127) // 128
        if stream is None:
            wide, scales = x.new_empty((M, pitch), dtype=FP8), x.new_empty((M, blocks), dtype=torch.float32)
        else:
            with _allocating(stream):
                wide, scales = x.new_empty((M, pitch), dtype=FP8), x.new_empty((M, blocks), dtype=torch.float32)
        _lib.fp8_quant_rows(x.data_ptr(), kind, M, K, _pitch(x), wide.data_ptr(), pitch, scales.data_ptr(), blocks,
                            _stream(stream))
        return (wide if pitch == K else wide[:, :K]), scales
    if codes is None or scales is None:
        with _allocating(stream):
            if codes is None:
                codes = empty_codes(M, K, x.device)
            if scales is None:
                scales = torch.empty((M, _blocks(K)), dtype=torch.float32, device=x.device)
    _check_codes(codes, scales, M, "quantize_rows")
    if codes.shape != (M, K) or codes.get_device() != x.get_device():
        raise ValueError("quantize_rows: codes must have x's shape and device")
    _lib.fp8_quant_rows(x.data_ptr(), kind, M, K, _pitch(x), codes.data_ptr(), _code_pitch(codes), scales.data_ptr(),
                        _pitch(scales), _stream(stream))
    return codes, scales


def pack_weight(w: torch.Tensor, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """fp32 weight [N, K] -> (codes [N, K], scales [ceil(N/128), ceil(K/128)])."""
    if w.dtype != torch.float32 or w.dim() != 2 or not w.is_cuda or not w.is_contiguous():
        raise ValueError("pack_weight: w must be a contiguous fp32 CUDA matrix")
    _here(w)
    N, K = w.shape
    with _allocating(stream):
        codes = empty_codes(N, K, w.device)
        scales = torch.empty((_blocks(N), _blocks(K)), dtype=torch.float32, device=w.device)
    _lib.fp8_pack(w.data_ptr(), N, K, codes.data_ptr(), _code_pitch(codes), scales.data_ptr(), scales.shape[1],
                  _stream(stream))
    return codes, scales


class Fp8Linear:
    """A weight [N, K] in FP8 and its product with rows: y = x W^T."""

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor):
        _check_codes(codes, scales, _blocks(codes.shape[0]), "Fp8Linear")
        self.codes, self.scales = codes, scales
        self.N, self.K = codes.shape
        self._pitches = _code_pitch(codes), _pitch(scales)

    @classmethod
    def from_weight(cls, w: torch.Tensor, stream=None) -> "Fp8Linear":
        return cls(*pack_weight(w, stream))

    def matmul(self, a: torch.Tensor, a_scales: torch.Tensor, out: Optional[torch.Tensor] = None,
               out_dtype=torch.bfloat16, stream=None) -> torch.Tensor:
        """FP8 rows (codes [M, K], scales [M, ceil(K/128)]) times the weight: [M, N] in out_dtype (bf16 or fp32)."""
        M, N = a.shape[0], self.N
        _check_codes(a, a_scales, M, "matmul")
        if a.shape[1] != self.K or a.get_device() != self.codes.get_device():
            raise ValueError("matmul: the rows must have the weight's K and device")
        _here(a)
        if out is None:
            if out_dtype not in (torch.bfloat16, torch.float32):
                raise ValueError("matmul: out_dtype must be bf16 or fp32")
            if stream is None:
                out = a.new_empty((M, N), dtype=out_dtype)
            else:
                with _allocating(stream):
                    out = a.new_empty((M, N), dtype=out_dtype)
        elif out.shape != (M, N) or out.dtype not in (torch.bfloat16, torch.float32) or \
                out.get_device() != a.get_device() or (N > 1 and out.stride(1) != 1):
            raise ValueError("matmul: out must be bf16 or fp32 [M, N] with contiguous rows, on the rows' device")
        ldb, ld_sb = self._pitches
        _lib.fp8_gemm(a.data_ptr(), _code_pitch(a), a_scales.data_ptr(), _pitch(a_scales), self.codes.data_ptr(), ldb,
                      self.scales.data_ptr(), ld_sb, M, N, self.K, out.data_ptr(), _TYPES[out.dtype], _pitch(out),
                      _stream(stream))
        return out

    def forward(self, x: torch.Tensor, out_dtype=torch.bfloat16, stream=None) -> torch.Tensor:
        """x [M, K] (fp32, bf16 or fp16) -> x W^T: its rows to FP8, then the product."""
        codes, scales = quantize_rows(x, stream=stream)
        return self.matmul(codes, scales, out_dtype=out_dtype, stream=stream)
