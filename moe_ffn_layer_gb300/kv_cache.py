"""The 8-bit paged KV cache of one attention layer, held on one CUDA device: code
pools, scales and the attention's workspace.  PyTorch provides the memory and
the streams; each method is one call of a C entry point (``moe_kv_append``,
``moe_kv_attention``, ``moe_kv_evict``; their meaning, layouts and device-side
checks are documented in ``include/moe_ffn.h``).  Which pages belong to which
sequence is the caller's: ``page_table`` int32 [B, width] and ``seq_lens`` int32
[B], both on the device.
"""
from __future__ import annotations

import ctypes

import torch

from . import binding as B

# The calls are a few microseconds of kernels at decode sizes, and the host has
# to keep ahead of them: streams are taken by handle, and the C entry points are
# called with pointers at once.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _current(device_index: int) -> int:
    if _raw_stream is not None:
        return _raw_stream(device_index)
    return torch.cuda.current_stream(device_index).cuda_stream


_capturing = getattr(torch._C, "_cuda_isCurrentStreamCapturing", torch.cuda.is_current_stream_capturing)
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _call(name: str, rc: int) -> None:
    if rc != 0:
        raise B.MoEError(name, rc)


class KVCache8:
    """k, v: uint8 [num_pages, Hkv, page, D] e4m3 codes; k_scale, v_scale: fp32
    [num_pages, Hkv].  D is 64 or 128, page 16, 32, 64 or 128 tokens."""

    def __init__(self, num_pages: int, kv_heads: int, head_dim: int, page: int = 64, device="cuda"):
        shape = (num_pages, kv_heads, page, head_dim)
        self._hold(torch.zeros(shape, dtype=torch.uint8, device=device),
                   torch.zeros(shape, dtype=torch.uint8, device=device),
                   torch.zeros(shape[:2], dtype=torch.float32, device=device),
                   torch.zeros(shape[:2], dtype=torch.float32, device=device))

    @classmethod
    def from_tensors(cls, k, v, k_scale, v_scale) -> "KVCache8":
        """Over existing pools (not copied)."""
        self = cls.__new__(cls)
        self._hold(k, v, k_scale, v_scale)
        return self

    def _hold(self, k, v, k_scale, v_scale):
        self.device = k.device
        self._dev = k.get_device()
        _want("k", k, torch.uint8, 4, self.device)
        _want("v", v, torch.uint8, 4, self.device, k.shape)
        _want("k_scale", k_scale, torch.float32, 2, self.device, k.shape[:2])
        _want("v_scale", v_scale, torch.float32, 2, self.device, k.shape[:2])
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.num_pages, self.kv_heads, self.page, self.head_dim = k.shape
        self.dims = B.moe_kv_dims(self.kv_heads, self.head_dim, self.page)
        self.pool = B.moe_kv_pool(*(B.ptr(t) for t in (k, v, k_scale, v_scale)), self.num_pages)
        self._dims, self._pool = ctypes.byref(self.dims), ctypes.byref(self.pool)
        self._shape = tuple(k.shape[1:])
        self._need = (None, 0)   # the last call's sizes and the workspace bytes they need
        self._ws = {}   # by stream: calls of different streams may overlap, and replays of graphs with any

    def _on(self, stream):
        """The context of what a call on `stream` (torch's, or a handle) allocates."""
        return torch.cuda.stream(torch.cuda.ExternalStream(stream, self.device) if isinstance(stream, int) else stream)

    def _want_table(self, page_table, seq_lens, cu, cu_name):
        """Checks the sequences' tensors; returns the table's rows and width."""
        n, width = page_table.shape
        dev = self._dev
        if not (_is(page_table, torch.int32, dev, page_table.shape) and _is(seq_lens, torch.int32, dev, (n,)) and
                (cu is None or _is(cu, torch.int32, dev, (n + 1,)))):
            _want("page_table", page_table, torch.int32, 2, self.device)
            _want("seq_lens", seq_lens, torch.int32, 1, self.device, (n,))
            if cu is not None:
                _want(cu_name, cu, torch.int32, 1, self.device, (n + 1,))
        return n, width

    def append(self, k: torch.Tensor, v: torch.Tensor, page_table: torch.Tensor, seq_lens: torch.Tensor,
               cu_new: torch.Tensor, stream=None) -> None:
        """Stores the new tokens' k and v (bf16 [T, Hkv, D], rows any equal
        stride apart); seq_lens already counts them, cu_new int32 [B+1] says
        whose they are."""
        T = k.shape[0]
        shape = (T, self.kv_heads, self.head_dim)
        if not (_is_rows(k, self._dev, shape) and _is_rows(v, self._dev, shape)):
            _want("k", k, torch.bfloat16, 3, self.device, shape, rows=True)
            _want("v", v, torch.bfloat16, 3, self.device, shape, rows=True)
        stride = k.stride(0)
        if T <= 1:
            stride = self.kv_heads * self.head_dim
        elif stride != v.stride(0):
            raise ValueError(f"k and v rows lie {stride} and {v.stride(0)} elements apart")
        n, width = self._want_table(page_table, seq_lens, cu_new, "cu_new")
        seqs = B.moe_kv_seqs(page_table.data_ptr(), seq_lens.data_ptr(), n, width, min(width * self.page, 1 << 30))
        if _device() != self._dev:   # (the library works on the current device)
            with torch.cuda.device(self._dev):
                return self.append(k, v, page_table, seq_lens, cu_new, stream)
        _call("moe_kv_append", B.lib().moe_kv_append(
            self._dims, self._pool, ctypes.byref(seqs), k.data_ptr(), v.data_ptr(), stride, cu_new.data_ptr(), T,
            _current(self._dev) if stream is None else B.handle(stream)))

    def workspace(self, need: int, stream=None) -> torch.Tensor:
        """A workspace of at least `need` bytes for one call on `stream`
        (default: the current stream): the stream's own, which its calls use in
        turn.  A call that is being captured in a graph has one of its own,
        allocated and its counters zeroed in the capture: its memory is the
        graph's, whatever later calls need or other graphs are replayed."""
        if stream is not None:
            with self._on(stream):
                return self._workspace(need, B.handle(stream))
        return self._workspace(need, _current(self._dev))

    def _workspace(self, need, key):
        captured = _capturing()
        ws = None if captured else self._ws.get(key)
        if ws is None or ws.numel() < need:
            # (a stream's own has some to spare: decoding with weights asks for more every 32 tokens)
            spare = 0 if captured else min(need // 4, 64 << 20)
            ws = torch.empty(max(need + spare, 256), dtype=torch.uint8, device=self.device)
            ws[:B.KV_COUNTER_BYTES].zero_()
            if not captured:
                self._ws[key] = ws
        return ws

    def attend(self, q: torch.Tensor, page_table: torch.Tensor, seq_lens: torch.Tensor, cu_q: torch.Tensor, max_q: int,
               max_len: int, scale: float | None = None, weights: torch.Tensor | None = None,
               out: torch.Tensor | None = None, lse: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """out bf16 [T, Hq, D]: attention of the queries q (bf16 [T, Hq, D], rows
        any stride apart), the last tokens of their sequences, over the cache.
        max_q and max_len bound the queries and the length of a sequence; scale
        defaults to D ** -0.5.  lse fp32 [T, Hq], where given, takes the
        log-sum-exps; weights fp32 [B, Hkv, >= max_len], where given, gains the
        softmax weights."""
        T, Hq = q.shape[0], q.shape[1]
        dev, D = self._dev, self.head_dim
        shape = (T, Hq, D)
        if not _is_rows(q, dev, shape):
            _want("q", q, torch.bfloat16, 3, self.device, shape, rows=True)
        n, width = self._want_table(page_table, seq_lens, cu_q, "cu_q")
        seqs = B.moe_kv_seqs(page_table.data_ptr(), seq_lens.data_ptr(), n, width, max_len)
        if out is None:
            if stream is None:
                out = torch.empty(shape, dtype=torch.bfloat16, device=self.device)
            else:
                with self._on(stream):
                    out = torch.empty(shape, dtype=torch.bfloat16, device=self.device)
        if not _is(out, torch.bfloat16, dev, shape):
            _want("out", out, torch.bfloat16, 3, self.device, shape)
        if lse is not None and not _is(lse, torch.float32, dev, (T, Hq)):
            _want("lse", lse, torch.float32, 2, self.device, (T, Hq))
        w_stride = 0
        if weights is not None:
            w_stride = weights.shape[-1]
            if not _is(weights, torch.float32, dev, (n, self.kv_heads, w_stride)):
                _want("weights", weights, torch.float32, 3, self.device, (n, self.kv_heads, w_stride))
        if _device() != self._dev:
            with torch.cuda.device(self._dev):
                return self.attend(q, page_table, seq_lens, cu_q, max_q, max_len, scale, weights, out, lse, stream)
        sizes = (Hq, n, T, max_q, max_len, weights is not None)
        need = self._need   # (read once: another thread's call may put other sizes there)
        if need[0] != sizes:
            need = self._need = (sizes, B.moe_kv_attention_workspace_bytes(self.dims, *sizes))
        handle = _current(dev) if stream is None else B.handle(stream)
        ws = self._workspace(need[1], handle) if stream is None else self.workspace(need[1], stream)
        _call("moe_kv_attention", B.lib().moe_kv_attention(
            self._dims, self._pool, ctypes.byref(seqs), q.data_ptr(), q.stride(0) if T > 1 else Hq * D, Hq,
            cu_q.data_ptr(), T, max_q, D ** -0.5 if scale is None else scale, out.data_ptr(),
            None if lse is None else lse.data_ptr(), None if weights is None else weights.data_ptr(), w_stride,
            ws.data_ptr(), ws.numel(), handle))
        return out

    def evict(self, weights: torch.Tensor, page_table: torch.Tensor, seq_lens: torch.Tensor, max_len: int, budget: int,
              sink: int, recent: int, dst_table: torch.Tensor, dst: "KVCache8 | None" = None, stream=None):
        """Keeps at most `budget` tokens of each sequence and kv head (its first
        `sink`, its last `recent`, the heaviest between by `weights` fp32 [B,
        Hkv, >= max_len]), copied into the pages of dst_table int32 [B, width]
        of `dst` (default: this cache; none of them a page that is read).
        Returns (lengths int32 [B], the kept weights fp32 [B, Hkv, budget], the
        kept positions int32 [B, Hkv, budget])."""
        dst = self if dst is None else dst
        if dst._shape != self._shape:
            raise ValueError(f"dst holds pages of {dst._shape}, not {self._shape}")
        if dst._dev != self._dev:
            raise ValueError(f"dst: want pools on {self.device}, got {dst.device}")
        n, width = self._want_table(page_table, seq_lens, None, "")
        w_stride, dst_width = weights.shape[-1], dst_table.shape[-1]
        if not (_is(weights, torch.float32, self._dev, (n, self.kv_heads, w_stride)) and
                _is(dst_table, torch.int32, self._dev, (n, dst_width))):
            _want("weights", weights, torch.float32, 3, self.device, (n, self.kv_heads, w_stride))
            _want("dst_table", dst_table, torch.int32, 2, self.device, (n, dst_width))
        if _device() != self._dev:
            with torch.cuda.device(self._dev):
                return self.evict(weights, page_table, seq_lens, max_len, budget, sink, recent, dst_table, dst, stream)
        if stream is None:
            made = self._evict_outputs(n, budget)
        else:
            with self._on(stream):
                made = self._evict_outputs(n, budget)
        seqs = B.moe_kv_seqs(page_table.data_ptr(), seq_lens.data_ptr(), n, width, max_len)
        _call("moe_kv_evict", B.lib().moe_kv_evict(
            self._dims, self._pool, ctypes.byref(seqs), weights.data_ptr(), w_stride, budget, sink, recent, dst._pool,
            dst_table.data_ptr(), dst_width, made[0].data_ptr(), made[1].data_ptr(), made[2].data_ptr(),
            _current(self._dev) if stream is None else B.handle(stream)))
        return made

    def _evict_outputs(self, n, budget):
        shape = (n, self.kv_heads, max(budget, 0))
        return (torch.empty(n, dtype=torch.int32, device=self.device),
                torch.empty(shape, dtype=torch.float32, device=self.device),
                torch.empty(shape, dtype=torch.int32, device=self.device))


def _is(t, dtype, dev, shape):
    return t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous()


def _is_rows(t, dev, shape):
    """A bf16 tensor of that shape, contiguous within each row of its first axis."""
    return (t.dtype is torch.bfloat16 and t.shape == shape and t.get_device() == dev and t.stride(2) == 1 and
            t.stride(1) == shape[2])


def _want(name, t, dtype, ndim, device, shape=None, rows=False):
    """Raises ValueError unless t is a tensor of that type, shape and device,
    contiguous (rows: within each row of its first axis)."""
    if t.dtype != dtype or t.dim() != ndim or t.device != device:
        raise ValueError(f"{name}: want {ndim}-d {dtype} on {device}, got {t.dim()}-d {t.dtype} on {t.device}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: want shape {tuple(shape)}, got {tuple(t.shape)}")
    flat = t[0] if rows and t.shape[0] > 0 else t
    if not flat.is_contiguous():
        raise ValueError(f"{name}: not contiguous")
