"""Python-side plumbing around the C ABI: device buffers (torch), streams,
the expert slot pool and the slot manager.

Every step of the layer runs in libftmoe.so; this module only allocates
memory with torch and forwards pointers (there is no fallback path).
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import Optional

import numpy as np
import torch

from . import _lib
from ._lib import FT_DOWN, FT_GATE, FT_UP


def _ptr(t: Optional[torch.Tensor]) -> int:
    return 0 if t is None else t.data_ptr()


def _stream(s: Optional[torch.cuda.Stream]) -> int:
    """The handle of s, or of the current device's current stream (without the Stream object that
    torch.cuda.current_stream() makes of it, some 5 us a call)."""
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device()) if s is None else s.cuda_stream


def _allocating(stream):
    """New tensors belong to `stream`: one of the current stream's could still be in use there."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def untile(block: np.ndarray, N: int, width: int, row_bytes: int) -> np.ndarray:
    """Stage-tiled bytes [S][N][width] -> row-major [N, row_bytes] (the first
    row_bytes of each row's S * width bytes)."""
    S = block.size // (N * width)
    return np.ascontiguousarray(block.reshape(S, N, width).transpose(1, 0, 2).reshape(N, S * width)[:, :row_bytes])


class ExpertPool:
    """A device pool of expert slots (NVFP4, or MXFP4 with fmt=FT_SCALE_MXFP4,
    FP8 with fmt=FT_SCALE_FP8), row-major or stage-tiled (tiled=True; see
    ft_tiled_slot_layout_init; not for FP8).  ``buf``: the slots' bytes, for a
    pool that is already filled."""

    def __init__(self, H: int, I: int, num_slots: int, device="cuda", fmt: int = _lib.FT_SCALE_NVFP4,
                 tiled: bool = False, buf: Optional[torch.Tensor] = None):
        self.H, self.I, self.num_slots, self.fmt, self.tiled = H, I, num_slots, fmt, tiled
        self.layout = _lib.slot_layout(H, I, num_slots, fmt, tiled)
        # the canonical row-major layout of the same format, for slots read back to the host
        self.rows_layout = _lib.slot_layout(H, I, num_slots, fmt)
        self.slot_bytes = int(self.layout.slot_bytes)
        if buf is None:
            buf = torch.zeros(num_slots * self.slot_bytes, dtype=torch.uint8, device=device)
        else:
            assert buf.is_cuda and buf.data_ptr() % 256 == 0
        assert buf.dtype == torch.uint8 and buf.is_contiguous() and buf.numel() == num_slots * self.slot_bytes
        self.buf = buf
        self._pack_ws = torch.zeros(256, dtype=torch.uint8, device=buf.device)

    @property
    def ptr(self) -> int:
        return self.buf.data_ptr()

    def shape(self, mat: int):
        return (self.I, self.H) if mat in (FT_GATE, FT_UP) else (self.H, self.I)

    def pack_into(self, slot: int, mat: int, w: torch.Tensor, stream=None) -> None:
        """Quantise fp32 weights w [N, K] (on the device) into `slot`, in the pool's format and layout."""
        N, K = self.shape(mat)
        assert w.shape == (N, K) and w.dtype == torch.float32 and w.is_cuda and w.is_contiguous()
        base = self.ptr + slot * self.slot_bytes
        if self.tiled or self.fmt == _lib.FT_SCALE_FP8:
            _lib.pack_slot(w.data_ptr(), mat, self.layout, base, self._pack_ws.data_ptr(), _stream(stream))
            return
        L = self.layout
        pack = _lib.mxfp4_pack if self.fmt == _lib.FT_SCALE_MXFP4 else _lib.nvfp4_pack
        pack(w.data_ptr(), N, K, base + L.codes_off[mat], base + L.scales_off[mat], L.ld_scale[mat],
             base + L.global_off[mat], self._pack_ws.data_ptr(), _stream(stream))

    def slot_view(self, slot: int) -> torch.Tensor:
        return self.buf[slot * self.slot_bytes:(slot + 1) * self.slot_bytes]

    def tensor_bytes(self, slot: int, mat: int):
        """(codes uint8 [N, K/2], scales uint8 [N, ld], global fp32) of one tensor, on the host, row-major;
        FP8: (codes uint8 [N, K], scales fp32 [ceil(N/128), ceil(K/128)], 1.0)."""
        N, K = self.shape(mat)
        L = self.layout
        ld = L.ld_scale[mat]
        s = self.slot_view(slot)
        if self.fmt == _lib.FT_SCALE_FP8:
            nb, kb = (N + 127) // 128, (K + 127) // 128
            codes = s[L.codes_off[mat]:L.codes_off[mat] + N * K].view(N, K).cpu().numpy()
            scales = s[L.scales_off[mat]:L.scales_off[mat] + nb * ld].cpu().numpy().view("float32").reshape(nb, ld // 4)
            return codes, np.ascontiguousarray(scales[:, :kb]), 1.0
        if self.tiled:
            S = (K + 255) // 256
            codes = untile(s[L.codes_off[mat]:L.codes_off[mat] + S * N * 128].cpu().numpy(), N, 128, K // 2)
            scales = untile(s[L.scales_off[mat]:L.scales_off[mat] + S * N * 16].cpu().numpy(), N, 16, ld)
        else:
            codes = s[L.codes_off[mat]:L.codes_off[mat] + N * K // 2].view(N, K // 2).cpu().numpy()
            scales = s[L.scales_off[mat]:L.scales_off[mat] + N * ld].view(N, ld).cpu().numpy()
        g = s[L.global_off[mat]:L.global_off[mat] + 4].cpu().numpy().view("float32")[0]
        return codes, scales, float(g)

    def export_slot(self, slot: int) -> np.ndarray:
        """The slot as a host image in the row-major layout `rows_layout`
        (what the oracle and the host banks read)."""
        if not self.tiled:
            return self.slot_view(slot).cpu().numpy()
        R = self.rows_layout
        out = np.zeros(int(R.slot_bytes), np.uint8)
        for mat in range(3):
            c, sc, g = self.tensor_bytes(slot, mat)
            out[R.codes_off[mat]:R.codes_off[mat] + c.size] = c.reshape(-1)
            out[R.scales_off[mat]:R.scales_off[mat] + sc.size] = sc.reshape(-1)
            out[R.global_off[mat]:R.global_off[mat] + 4] = np.frombuffer(np.float32(g).tobytes(), np.uint8)
        return out


class MoELayer:
    """Buffers and calls for one MoE FFN layer of fixed (T, E, k, H, I).

    ffn() and forward() take NVFP4, MXFP4 and FP8 pools.  out_dtype is the type
    of the expert outputs out_perm: torch.float32, or for FP8 pools also
    torch.bfloat16."""

    def __init__(self, T: int, E: int, k: int, H: int, I: int, mode: int = _lib.FT_ROUTE_SOFTMAX_RENORM,
                 device="cuda", fused_front: bool = False, whole: bool = False, out_dtype=torch.float32):
        assert out_dtype in (torch.float32, torch.bfloat16)
        self.T, self.E, self.k, self.H, self.I, self.mode = T, E, k, H, I, mode
        self.fused_front = fused_front   # route + permute through ft_moe_route_permute (separate calls only)
        # forward() through ft_moe_layer_nvfp4 (one launch for decode-sized batches); False: the four calls
        self.whole = whole and not fused_front
        P = T * k
        dev = torch.device(device)
        i32 = dict(dtype=torch.int32, device=dev)
        self.ids = torch.empty((T, k), **i32)
        self.w = torch.empty((T, k), dtype=torch.float32, device=dev)
        self.offsets = torch.empty(E + 1, **i32)
        self.perm_src = torch.empty(P, **i32)
        self.pair_to_row = torch.empty(P, **i32)
        self.out_perm = torch.empty((P, H), dtype=out_dtype, device=dev)
        self.y = torch.empty((T, H), dtype=torch.float32, device=dev)
        self.dev = dev
        self.perm_ws_bytes = _lib.permute_workspace_size(T, k, E)
        self.ffn_ws_bytes = _lib.ffn_workspace_size(T, H, I, E, k)
        self.layer_ws_bytes = _lib.layer_workspace_size(T, H, I, E, k)
        self.fp8_ws_bytes = _lib.ffn_fp8_workspace_size(T, H, I, E, k)
        self._perm_ws = self._ffn_ws = self._layer_ws = self._fp8_ws = None

    # workspaces, allocated on first use, on the stream of that call: the separate calls'
    # (permute, ffn) and the whole-layer call's, which is zero-filled once and left ready
    # by every call
    def _workspace(self, name: str, stream=None) -> torch.Tensor:
        ws = getattr(self, "_" + name)
        if ws is None:
            make = torch.zeros if name == "layer_ws" else torch.empty
            with _allocating(stream):
                ws = make(max(getattr(self, name + "_bytes"), 256), dtype=torch.uint8, device=self.dev)
            setattr(self, "_" + name, ws)
        return ws

    perm_ws = property(lambda self: self._workspace("perm_ws"))
    ffn_ws = property(lambda self: self._workspace("ffn_ws"))
    fp8_ws = property(lambda self: self._workspace("fp8_ws"))
    layer_ws = property(lambda self: self._workspace("layer_ws"))

    def route(self, logits: torch.Tensor, stream=None) -> None:
        _lib.route(logits.data_ptr(), self.T, self.E, self.k, self.mode, self.ids.data_ptr(), self.w.data_ptr(),
                   _stream(stream))

    def permute(self, stream=None) -> None:
        _lib.permute(self.ids.data_ptr(), self.T, self.k, self.E, self.offsets.data_ptr(), self.perm_src.data_ptr(),
                     self.pair_to_row.data_ptr(), self._workspace("perm_ws", stream).data_ptr(), self.perm_ws_bytes,
                     _stream(stream))

    def route_permute(self, logits: torch.Tensor, stream=None) -> None:
        _lib.route_permute(logits.data_ptr(), self.T, self.E, self.k, self.mode, self.ids.data_ptr(),
                           self.w.data_ptr(), self.offsets.data_ptr(), self.perm_src.data_ptr(),
                           self.pair_to_row.data_ptr(), self._workspace("perm_ws", stream).data_ptr(),
                           self.perm_ws_bytes, _stream(stream))

    def ffn(self, x: torch.Tensor, slot_table: torch.Tensor, pool: ExpertPool, stream=None) -> None:
        if pool.fmt == _lib.FT_SCALE_FP8:
            _lib.ffn_fp8(x.data_ptr(), self.T, self.H, self.I, self.E, self.k, self.perm_src.data_ptr(),
                         self.offsets.data_ptr(), slot_table.data_ptr(), pool.ptr, pool.layout,
                         self.out_perm.data_ptr(),
                         _lib.FT_F32 if self.out_perm.dtype == torch.float32 else _lib.FT_BF16,
                         self._workspace("fp8_ws", stream).data_ptr(), self.fp8_ws_bytes, _stream(stream))
            return
        assert self.out_perm.dtype == torch.float32, "bf16 expert outputs are for FP8 pools"
        _lib.ffn_nvfp4(x.data_ptr(), self.T, self.H, self.I, self.E, self.k, self.perm_src.data_ptr(),
                       self.offsets.data_ptr(), slot_table.data_ptr(), pool.ptr, pool.layout,
                       self.out_perm.data_ptr(), self._workspace("ffn_ws", stream).data_ptr(), self.ffn_ws_bytes,
                       _stream(stream))

    def combine(self, stream=None) -> None:
        combine = _lib.combine if self.out_perm.dtype == torch.float32 else _lib.combine_bf16
        combine(self.out_perm.data_ptr(), self.pair_to_row.data_ptr(), self.w.data_ptr(), self.T, self.k, self.H,
                self.y.data_ptr(), _stream(stream))

    def layer(self, x: torch.Tensor, logits: torch.Tensor, slot_table: torch.Tensor, pool: ExpertPool,
              stream=None) -> None:
        assert self.out_perm.dtype == torch.float32, "bf16 expert outputs are for FP8 pools"
        _lib.layer_nvfp4(x.data_ptr(), logits.data_ptr(), self.T, self.H, self.I, self.E, self.k, self.mode,
                         slot_table.data_ptr(), pool.ptr, pool.layout, self.ids.data_ptr(), self.w.data_ptr(),
                         self.offsets.data_ptr(), self.perm_src.data_ptr(), self.pair_to_row.data_ptr(),
                         self.out_perm.data_ptr(), self.y.data_ptr(), self._workspace("layer_ws", stream).data_ptr(),
                         self.layer_ws_bytes, _stream(stream))

    def forward(self, x: torch.Tensor, logits: torch.Tensor, slot_table: torch.Tensor, pool: ExpertPool,
                stream=None) -> torch.Tensor:
        """route -> permute -> ffn -> combine, enqueued on one stream (one ft_moe_layer_nvfp4 call, or
        the four calls when the layer was made with whole=False or the pool holds FP8 experts)."""
        assert x.dtype == torch.bfloat16 and x.shape == (self.T, self.H) and x.is_contiguous()
        assert logits.dtype == torch.float32 and logits.shape == (self.T, self.E) and logits.is_contiguous()
        assert slot_table.dtype == torch.int32 and slot_table.numel() == self.E
        if self.whole and pool.fmt != _lib.FT_SCALE_FP8:
            self.layer(x, logits, slot_table, pool, stream)
            return self.y
        if self.fused_front:
            self.route_permute(logits, stream)
        else:
            self.route(logits, stream)
            self.permute(stream)
        self.ffn(x, slot_table, pool, stream)
        self.combine(stream)
        return self.y


class SlotManager:
    """ctypes wrapper of the host LRU slot manager (ft_slot_*)."""

    def __init__(self, capacity: int, layout: _lib.SlotLayout, pool_ptr: int = 0, host_only: bool = False):
        h = ctypes.c_void_p()
        flags = _lib.FT_SLOT_HOST_ONLY if host_only else _lib.FT_SLOT_DEVICE
        _lib.check(_lib.lib().ft_slot_create(ctypes.byref(h), capacity, ctypes.byref(layout),
                                             ctypes.c_void_p(pool_ptr or None), flags))
        self.h = h
        self.layout = layout

    def register_host(self, layer: int, expert: int, src_ptr: int) -> None:
        _lib.check(_lib.lib().ft_slot_register_host(self.h, layer, expert, ctypes.c_void_p(src_ptr)))

    def acquire(self, layer: int, ids, table_ptr: int, table_len: int, compute=0, copy=0) -> None:
        arr = (ctypes.c_int32 * len(ids))(*[int(i) for i in ids])
        _lib.check(_lib.lib().ft_slot_acquire(self.h, layer, arr, len(ids), ctypes.c_void_p(table_ptr), table_len,
                                              ctypes.c_void_p(compute or None), ctypes.c_void_p(copy or None)))

    def inject_copy_failures(self, n: int) -> None:
        _lib.check(_lib.lib().ft_slot_inject_copy_failures(self.h, n))

    def stats(self) -> dict:
        s = _lib.SlotStats()
        _lib.check(_lib.lib().ft_slot_stats(self.h, ctypes.byref(s)))
        return {"hits": s.hits, "misses": s.misses, "evictions": s.evictions, "bytes_h2d": s.bytes_h2d,
                "copies": s.copies}

    def close(self) -> None:
        if self.h:
            _lib.lib().ft_slot_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
