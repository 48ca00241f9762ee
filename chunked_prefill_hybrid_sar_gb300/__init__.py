"""Hybrid-batch decoder step (chunked prefill + piggybacked decodes) on GB300.

Thin Python face of ``libsar.so``: the classes below only marshal torch
tensors (device memory and streams) and host lists into the C ABI of
``include/sar.h``; every step runs in the library's CUDA kernels.
"""

from __future__ import annotations

import ctypes

from . import _lib
from ._lib import (SAR_EPI_F32, SAR_EPI_RESIDUAL, SAR_EPI_STORE, SAR_EPI_SWIGLU, SAR_GEMM_AUTO,
                   SAR_GEMM_PAIR_N128, SAR_GEMM_PAIR_N192,
                   SAR_GEMM_PAIR_N256, SAR_GEMM_STREAM_K, SAR_GEMM_TWO_CTAS,
                   SAR_FP4_GEMM_AUTO,
                   SAR_FP4_GEMM_PAIR, SAR_FP4_GEMM_SPLIT, SAR_FP4_GEMM_TOKENS64, SAR_FP4_MX, SAR_FP4_NV,
                   SAR_GEMM_M128_N128, SAR_GEMM_M128_N256, SAR_GEMM_M256_N128, SAR_GEMM_SWAP,
                   SAR_IN_HIDDEN, SAR_IN_TOKENS, SAR_STORAGE_BF16, SAR_STORAGE_F16, KERNEL_KINDS,
                   SarError, check, lib)

__all__ = ["Model", "KVCache", "Scheduler", "Batch", "StepGraph", "SarError", "lib", "check", "gemm", "rmsnorm",
           "fp4_quantize", "fp4_dequantize", "fp4_scale_bytes", "gemm_fp4", "SAR_FP4_NV",
           "SAR_FP4_MX", "LogitControls", "logits_control", "token_state_add",
           "op_sync_status", "op_wait_check",
           "launch_count", "KERNEL_KINDS", "SAR_IN_HIDDEN", "SAR_IN_TOKENS", "SAR_STORAGE_F16",
           "SAR_STORAGE_BF16", "storage_dtype"]


def storage_dtype(storage: int):
    """torch dtype of a storage code."""
    import torch
    return torch.bfloat16 if storage == SAR_STORAGE_BF16 else torch.float16


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


def launch_count() -> int:
    return int(lib().sar_launch_count())


class Batch:
    """Owns the ctypes descriptor of one hybrid batch (chunks first, then decodes).

    ``prefill``: ``(req, start_pos, len, block_table)``, a list of such chunks
    (each of a different request, rows stacked in list order) or ``None``;
    ``decodes``: iterable of ``(req, ctx_len, block_table)``.
    """

    def __init__(self, prefill, decodes, in_kind=SAR_IN_HIDDEN):
        self._keep = []
        b = _lib.sar_batch()
        b.in_kind = in_kind
        if prefill is None:
            chunks = []
        elif isinstance(prefill, tuple):
            chunks = [prefill]
        else:
            chunks = list(prefill)
        pre = []
        for req, start, n, bt in chunks:
            arr = _lib.i32_array(bt)
            self._keep.append(arr)
            pre.append(_lib.sar_prefill(req, start, n, arr, len(bt)))
        if pre:
            b.has_prefill = 1
            b.prefill = pre[0]
        if len(pre) > 1:
            more = (_lib.sar_prefill * (len(pre) - 1))(*pre[1:])
            self._keep.append(more)
            b.n_more_prefill = len(pre) - 1
            b.more_prefill = more
        decodes = list(decodes)
        dec = (_lib.sar_decode * max(1, len(decodes)))()
        for i, (req, ctx, bt) in enumerate(decodes):
            arr = _lib.i32_array(bt)
            self._keep.append(arr)
            dec[i] = _lib.sar_decode(req, ctx, arr, len(bt))
        self._keep.append(dec)
        b.n_decode = len(decodes)
        b.decode = dec
        self.c = b
        self.chunks = chunks
        self.lp = sum(c[2] for c in chunks)
        self.bd = len(decodes)

    @property
    def rows(self) -> int:
        return self.lp + self.bd

    @property
    def logit_rows(self) -> int:
        """The last row of every chunk, then every decode row."""
        return len(self.chunks) + self.bd


class Model:
    """Weights are given in bf16; ``storage`` picks the internal 16-bit type."""

    def __init__(self, dims, max_tokens: int, max_decodes: int, storage: int = SAR_STORAGE_F16):
        self.dims = dims
        self.storage = storage
        d = _lib.sar_dims(dims.n_layers, dims.hidden, dims.n_q_heads, dims.n_kv_heads, dims.head_dim,
                          dims.ffn, dims.vocab, dims.rms_eps, dims.rope_base, max_tokens, max_decodes,
                          storage, getattr(dims, "sliding_window", 0))
        h = ctypes.c_void_p()
        check(lib().sar_model_create(ctypes.byref(d), ctypes.byref(h)))
        self.h = h

    def set_layer(self, layer: int, w: dict, stream=None) -> None:
        lw = _lib.sar_layer_weights(*[_ptr(w[n]) for n in ("wq", "wk", "wv", "wo", "wg", "wu", "wd",
                                                          "norm1", "norm2")])
        check(lib().sar_model_set_layer(self.h, layer, ctypes.byref(lw), _stream(stream)))

    def set_head(self, embed=None, final_norm=None, lm_head=None, stream=None) -> None:
        check(lib().sar_model_set_head(self.h, _ptr(embed), _ptr(final_norm), _ptr(lm_head),
                                       _stream(stream)))

    def step(self, kv: "KVCache", batch: Batch, inp, hidden_out=None, logits_out=None,
             layer_out=None, stream=None) -> None:
        check(lib().sar_step(self.h, kv.h, ctypes.byref(batch.c), _ptr(inp), _ptr(hidden_out),
                             _ptr(logits_out), _ptr(layer_out), _stream(stream)))

    def step_host(self, kv: "KVCache", batch: Batch, inp, hidden_out=None, logits_out=None,
                  stream=None) -> None:
        check(lib().sar_step_host(self.h, kv.h, ctypes.byref(batch.c), _ptr(inp), _ptr(hidden_out),
                                  _ptr(logits_out), None, _stream(stream)))

    def sample_greedy(self, logits, rows: int, out, stream=None) -> None:
        check(lib().sar_sample_greedy(self.h, _ptr(logits), rows, _ptr(out), _stream(stream)))

    def sync_status(self) -> None:
        check(lib().sar_sync_status(self.h))

    def profile(self, on: bool) -> None:
        check(lib().sar_profile_enable(self.h, 1 if on else 0))

    def set_chunk_split(self, on: bool) -> None:
        """Key-range splits of chunk-attention tiles when they leave SMs idle."""
        check(lib().sar_model_set_chunk_split(self.h, 1 if on else 0))

    def set_overlap(self, on: bool) -> None:
        """Chunk attention on a second stream, concurrent with decode attention."""
        check(lib().sar_model_set_overlap(self.h, 1 if on else 0))

    def profile_read(self) -> dict:
        n = len(KERNEL_KINDS)
        ms = (ctypes.c_double * n)()
        cnt = (ctypes.c_int64 * n)()
        check(lib().sar_profile_read(self.h, ms, cnt, n))
        return {k: (ms[i], int(cnt[i])) for i, k in enumerate(KERNEL_KINDS)}

    def debug_buffer(self, which: int) -> int:
        p = ctypes.c_void_p()
        check(lib().sar_model_debug_buffer(self.h, which, ctypes.byref(p)))
        return p.value

    def close(self) -> None:
        if self.h:
            check(lib().sar_model_destroy(self.h))
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class StepGraph:
    """One step captured as a CUDA graph (``sar_graph_*``): fixed input and
    output buffers; ``update`` re-points it at a batch whose plan has the same
    shape, ``launch`` runs it."""

    def __init__(self, model: "Model", kv: "KVCache", batch: Batch, inp, hidden_out=None, logits_out=None,
                 layer_out=None, stream=None):
        self._keep = (batch, inp, hidden_out, logits_out, layer_out)
        self._vocab = model.dims.vocab
        self._pending = self._controls = None
        self._earlier = []  # controls that an enqueued step may still read
        h = ctypes.c_void_p()
        check(lib().sar_graph_create(model.h, kv.h, ctypes.byref(batch.c), _ptr(inp), _ptr(hidden_out),
                                     _ptr(logits_out), _ptr(layer_out), _stream(stream), ctypes.byref(h)))
        self.h = h

    def update(self, batch: Batch, stream=None) -> None:
        check(lib().sar_graph_update(self.h, ctypes.byref(batch.c), _stream(stream)))
        self._keep = (batch,) + self._keep[1:]

    def launch(self, stream=None) -> None:
        check(lib().sar_graph_launch(self.h, _stream(stream)))

    def launch_host(self, inp, logits_out=None, hidden_out=None, stream=None) -> None:
        """Host input in, the captured step, host logits / hidden rows out (synchronous)."""
        check(lib().sar_graph_launch_host(self.h, _ptr(inp), _ptr(logits_out), _ptr(hidden_out), _stream(stream)))

    def launch_host_tokens(self, inp, tokens_out, stream=None) -> None:
        """Host input in, the captured step, each logits row's pick out (host
        int32 [R], synchronous): greedy, or under ``set_controls``, where -1
        stands for a row whose mask leaves no token."""
        check(lib().sar_graph_launch_host_tokens(self.h, _ptr(inp), ctypes.cast(_ptr(tokens_out), _lib.P_i32),
                                                 _stream(stream)))

    def enqueue_host_tokens(self, inp, tokens_out, stream=None) -> None:
        """As launch_host_tokens, but returns once the step is enqueued (the
        input copy on the graph's own copy stream); ``wait`` then waits for
        it.  ``inp`` must stay unchanged and ``tokens_out`` unread until then."""
        check(lib().sar_graph_enqueue_host_tokens(self.h, _ptr(inp), ctypes.cast(_ptr(tokens_out), _lib.P_i32),
                                                  _stream(stream)))
        self._pending = (inp, tokens_out)

    def set_controls(self, controls: "LogitControls | None") -> None:
        """The token launches pick under ``controls`` (a row per logits row)
        from now on; None: greedily again.  A step that is enqueued keeps the
        controls that it was enqueued under."""
        if controls is not None:
            # (the library sees strides alone: a table's columns may end before its stride does)
            if controls.rows is not None and controls.rows < self._keep[0].logit_rows:
                raise ValueError("set_controls: an array is shorter than the logits' rows")
            if controls.vocab < self._vocab:
                raise ValueError("set_controls: the token state or the mask is narrower than the vocabulary")
            logits = self._keep[3]
            if controls.device is not None and logits is not None and controls.device != logits.get_device():
                raise ValueError("set_controls: the controls are on another device than the logits")
        check(lib().sar_graph_set_controls(self.h, None if controls is None else ctypes.byref(controls.c)))
        if self._pending is not None:
            self._earlier.append(self._controls)
        self._controls = controls

    def wait(self) -> None:
        """Waits for the last enqueue_host_tokens step of this graph."""
        check(lib().sar_graph_wait(self.h))
        self._pending = None
        self._earlier.clear()

    def close(self) -> None:
        if self.h:
            check(lib().sar_graph_destroy(self.h))
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class KVCache:
    def __init__(self, model: Model, page_size: int, num_pages: int):
        h = ctypes.c_void_p()
        check(lib().sar_kv_create(model.h, page_size, num_pages, ctypes.byref(h)))
        self.h = h
        self.model = model
        self.storage = model.storage
        self.page_size = page_size
        self.num_pages = num_pages

    def layer_ptr(self, layer: int, kind: int) -> int:
        p = ctypes.c_void_p()
        check(lib().sar_kv_layer_ptr(self.h, layer, kind, ctypes.byref(p)))
        return p.value

    def close(self) -> None:
        if self.h:
            check(lib().sar_kv_destroy(self.h))
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class Scheduler:
    """Stall-free scheduler (host only)."""

    def __init__(self, tau: int, tile: int, page_size: int, num_pages: int, max_batch: int,
                 max_chunks: int = 0):
        cfg = _lib.sar_sched_cfg(tau, tile, page_size, num_pages, max_batch, max_chunks)
        h = ctypes.c_void_p()
        check(lib().sar_sched_create(ctypes.byref(cfg), ctypes.byref(h)))
        self.h = h

    def add(self, req: int, arrival: float, prompt_len: int, output_len: int, prompt_tokens=None):
        arr = _lib.i32_array(prompt_tokens) if prompt_tokens is not None else None
        check(lib().sar_sched_add(self.h, req, arrival, prompt_len, output_len, arr))

    def next(self, now: float):
        """Returns ``(chunks, decodes, tokens, c_batch)`` with Python lists copied
        out; ``chunks`` lists ``(req, start_pos, len, block_table)`` in row order."""
        b = _lib.sar_batch()
        tok = _lib.P_i32()
        check(lib().sar_sched_next(self.h, now, ctypes.byref(b), ctypes.byref(tok)))

        def chunk(p):
            return (p.req, p.start_pos, p.len, [p.block_table[i] for i in range(p.n_blocks)])

        chunks = []
        if b.has_prefill:
            chunks.append(chunk(b.prefill))
            chunks += [chunk(b.more_prefill[i]) for i in range(b.n_more_prefill)]
        decs = []
        for i in range(b.n_decode):
            dd = b.decode[i]
            decs.append((dd.req, dd.ctx_len, [dd.block_table[j] for j in range(dd.n_blocks)]))
        m = sum(c[2] for c in chunks) + len(decs)
        tokens = [tok[i] for i in range(m)] if bool(tok) else None
        return chunks, decs, tokens, b

    def commit(self, sampled) -> int:
        arr = _lib.i32_array(sampled)
        n = ctypes.c_int32()
        check(lib().sar_sched_commit(self.h, arr, len(list(sampled)), ctypes.byref(n)))
        return n.value

    def stats(self):
        v = [ctypes.c_int32() for _ in range(4)]
        check(lib().sar_sched_stats(self.h, *[ctypes.byref(x) for x in v]))
        return tuple(x.value for x in v)

    def close(self) -> None:
        if self.h:
            check(lib().sar_sched_destroy(self.h))
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


_LAYOUT = ("M", "Lp", "Bd", "R", "n_items", "n_parts", "n_tiles", "tile_rows", "o_pos", "o_slot", "o_pbt",
           "o_nkeys", "o_btoff", "o_btlen", "o_pbeg", "o_pcnt", "o_items", "o_bt", "o_rows", "o_tiles", "total",
           "n_comb", "n_cparts", "o_comb", "chunk_pairs")


def plan_inspect(dims, batch: Batch, page_size: int, num_pages: int, sms: int, max_tokens: int,
                 max_decodes: int, storage: int = SAR_STORAGE_F16, chunk_split: bool = False) -> dict:
    """The step planner on the host alone (``sar_plan_inspect``): the plan's
    sizes and array offsets, and the metadata block as a list of int32."""
    d = _lib.sar_dims(dims.n_layers, dims.hidden, dims.n_q_heads, dims.n_kv_heads, dims.head_dim,
                      dims.ffn, dims.vocab, dims.rms_eps, dims.rope_base, max_tokens, max_decodes,
                      storage, getattr(dims, "sliding_window", 0))
    lay = (ctypes.c_int32 * len(_LAYOUT))()
    n = ctypes.c_int64()
    cs = 1 if chunk_split else 0
    check(lib().sar_plan_inspect(ctypes.byref(d), page_size, num_pages, sms, cs, ctypes.byref(batch.c), lay, None,
                                 0, ctypes.byref(n)))
    meta = (ctypes.c_int32 * max(1, n.value))()
    check(lib().sar_plan_inspect(ctypes.byref(d), page_size, num_pages, sms, cs, ctypes.byref(batch.c), lay, meta,
                                 n.value, ctypes.byref(n)))
    out = dict(zip(_LAYOUT, list(lay)))
    out["meta"] = list(meta)[:n.value]
    return out


def _storage_of(t) -> int:
    import torch
    return SAR_STORAGE_BF16 if t.dtype == torch.bfloat16 else SAR_STORAGE_F16


def gemm(a, w, c, residual=None, epilogue=SAR_EPI_STORE, variant=SAR_GEMM_AUTO, stream=None) -> None:
    """C = epilogue(a . w^T); the storage type is taken from ``a`` (fp16 or bf16)."""
    M, K = a.shape
    N = w.shape[0]
    check(lib().sar_op_gemm(_ptr(a), _ptr(w), _ptr(c), _ptr(residual), M, N, K, epilogue, variant,
                            _storage_of(a), _stream(stream)))


def op_sync_status() -> None:
    """Synchronise the device and raise if a single-kernel entry point's
    kernel recorded a failure (timeout or bounds) since the last call."""
    check(lib().sar_op_sync_status())


def op_wait_check(limit_ns: int, arrivals: int, stream=None) -> None:
    """Run the bounded-wait check kernel (see ``sar_op_wait_check``)."""
    check(lib().sar_op_wait_check(int(limit_ns), int(arrivals), _stream(stream)))


def rmsnorm(x, gain, y, eps: float, stream=None) -> None:
    """y (fp16/bf16) = rmsnorm of fp32 rows x with fp32 gain."""
    check(lib().sar_op_rmsnorm(_ptr(x), _ptr(gain), _ptr(y), x.shape[0], x.shape[1], eps,
                               _storage_of(y), _stream(stream)))


# ---- 4-bit rows ----------------------------------------------------------------
#
# The checks below run in a decode loop, in front of kernels of a few
# microseconds: they read each attribute once and make no call into the library.

_ROW_TYPES: dict = {}  # torch dtype -> SAR_TYPE_*, filled at the first call


def _row_types() -> dict:
    if not _ROW_TYPES:
        import torch
        _ROW_TYPES.update({torch.float16: _lib.SAR_TYPE_F16, torch.bfloat16: _lib.SAR_TYPE_BF16,
                           torch.float32: _lib.SAR_TYPE_F32})
    return _ROW_TYPES


def _launch_stream(what: str, stream, *tensors) -> int | None:
    """Checks that every tensor is on the current device, where the library
    launches, and returns the stream's address (None: the current stream's)."""
    import torch
    dev = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:  # (-1: not on a CUDA device)
            raise ValueError(f"{what}: tensors must be on the current CUDA device")
    # (the stream's address alone: a torch.cuda.Stream object takes 3 us to make)
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream)


def _rows(what: str, t):
    """(rows, columns, row stride, SAR_TYPE_*) of a two-dimensional tensor with
    adjacent columns; a single row's stride, which means nothing, is its length."""
    kind = _ROW_TYPES.get(t.dtype) if _ROW_TYPES else _row_types().get(t.dtype)
    if kind is None:
        raise ValueError(f"{what}: rows must be float16, bfloat16 or float32")
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{what}: rows must be two-dimensional")
    rows, cols = shape
    if t.is_contiguous():
        return rows, cols, cols, kind
    ld, step = t.stride()
    if cols > 1 and step != 1:
        raise ValueError(f"{what}: a row's columns must be adjacent")
    return rows, cols, (ld if rows > 1 else cols), kind


def fp4_scale_bytes(rows: int, cols: int, format: int = SAR_FP4_NV) -> int:
    """Length in bytes of the scales of a 4-bit [rows, cols] matrix."""
    n = ctypes.c_int64()
    check(lib().sar_op_fp4_scale_bytes(rows, cols, format, ctypes.byref(n)))
    return n.value


def _fp4_check(what: str, codes, scales, rows: int, cols: int, format: int) -> None:
    import torch
    byte = torch.uint8
    if codes.dtype is not byte or scales.dtype is not byte:
        raise ValueError(f"{what}: codes and scales must be uint8")
    if codes.shape != (rows, cols >> 1) or cols & 1 or not codes.is_contiguous():
        raise ValueError(f"{what}: codes must be contiguous, two to a byte: {rows} rows of {cols}")
    # fp4_scale_bytes, for the formats and columns that the library takes
    width = 64 if format == SAR_FP4_NV else 128
    if scales.numel() < (rows + 127) // 128 * ((cols + width - 1) // width) * 512 or not scales.is_contiguous():
        raise ValueError(f"{what}: scales must be contiguous and as long as fp4_scale_bytes says")


def fp4_quantize(x, codes, scales, format: int = SAR_FP4_NV, tensor_scale: float = 1.0, stream=None) -> None:
    """codes (uint8 [rows, cols / 2]) and scales (uint8 [fp4_scale_bytes]) = the
    microscaled 4-bit form of the rows of ``x`` (fp16, bf16 or fp32, any row
    stride); see ``sar_op_fp4_quantize``."""
    rows, cols, ld, kind = _rows("fp4_quantize", x)
    _fp4_check("fp4_quantize", codes, scales, rows, cols, format)
    st = _launch_stream("fp4_quantize", stream, x, codes, scales)
    check(lib().sar_op_fp4_quantize(x.data_ptr(), ld, rows, cols, kind, format, tensor_scale, codes.data_ptr(),
                                    scales.data_ptr(), st))


def fp4_dequantize(codes, scales, y, format: int = SAR_FP4_NV, tensor_scale: float = 1.0, stream=None) -> None:
    """y (fp16, bf16 or fp32 rows, any row stride) = what 4-bit rows stand for."""
    rows, cols, ld, kind = _rows("fp4_dequantize", y)
    _fp4_check("fp4_dequantize", codes, scales, rows, cols, format)
    st = _launch_stream("fp4_dequantize", stream, codes, scales, y)
    check(lib().sar_op_fp4_dequantize(codes.data_ptr(), scales.data_ptr(), rows, cols, format, tensor_scale, y.data_ptr(),
                                      ld, kind, st))


def gemm_fp4(a, a_scales, w, w_scales, c, residual=None, alpha: float = 1.0, epilogue=SAR_EPI_STORE,
             format: int = SAR_FP4_NV, variant=SAR_FP4_GEMM_AUTO, stream=None) -> None:
    """c = epilogue(alpha * a . w^T) of 4-bit rows (codes uint8 [rows, K / 2] and
    their scales); 16-bit ``c`` for STORE and SWIGLU, fp32 for RESIDUAL and F32;
    see ``sar_op_gemm_fp4``."""
    if a.dim() != 2 or w.dim() != 2:
        raise ValueError("gemm_fp4: codes must be two-dimensional")
    M, K = a.shape
    N, K = w.shape[0], 2 * K
    _fp4_check("gemm_fp4", a, a_scales, M, K, format)
    _fp4_check("gemm_fp4", w, w_scales, N, K, format)
    rows, cols, _, kind = _rows("gemm_fp4", c)
    wide = epilogue in (SAR_EPI_F32, SAR_EPI_RESIDUAL)
    if wide != (kind == _lib.SAR_TYPE_F32):
        raise ValueError("gemm_fp4: c must be fp32 for RESIDUAL and F32, fp16 or bf16 otherwise")
    if rows != M or cols != (N // 2 if epilogue == SAR_EPI_SWIGLU else N) or not c.is_contiguous():
        raise ValueError("gemm_fp4: c has another shape, or is not contiguous")
    if (residual is None) != (epilogue != SAR_EPI_RESIDUAL):
        raise ValueError("gemm_fp4: the residual goes with the RESIDUAL epilogue")
    if residual is not None and (residual.dtype != c.dtype or residual.shape != c.shape or not residual.is_contiguous()):
        raise ValueError("gemm_fp4: residual must be contiguous fp32 of c's shape")
    st = _launch_stream("gemm_fp4", stream, a, a_scales, w, w_scales, c, residual)
    check(lib().sar_op_gemm_fp4(a.data_ptr(), a_scales.data_ptr(), w.data_ptr(), w_scales.data_ptr(), c.data_ptr(),
                                _ptr(residual), M, N, K, alpha, epilogue, format, variant, 0 if wide else kind, st))


# ---- logits controls -------------------------------------------------------------


class LogitControls:
    """What a batch's requests ask of their logits (``sar_logit_controls``): a
    handle over device tensors that the caller keeps filling; build it once.

    state       int16 [slots, >= vocab]: bit 15 the token is in the prompt, the
                low bits how often it was generated (``token_state_add``)
    slots       int32 [rows], -1 for a row without
    repetition, presence, frequency   fp32 [rows], each optional
    bias_offsets int32 [rows + 1], bias_tokens int32, bias_values fp32
    mask        int32 [masks, >= ceil(vocab / 32)], bit set = allowed
    mask_rows   int32 [rows], -1 for a row without (None: row r takes mask r)
    count_picks each pick is counted into its row's slot
    """

    def __init__(self, state=None, slots=None, repetition=None, presence=None, frequency=None, bias_offsets=None,
                 bias_tokens=None, bias_values=None, mask=None, mask_rows=None, count_picks: bool = False):
        import torch
        what = "LogitControls"

        def flat(t, dtype, name):
            if t is None:
                return None
            if t.dtype != dtype or t.dim() != 1 or not t.is_contiguous():
                raise ValueError(f"{what}: {name} must be a contiguous one-dimensional {dtype} tensor")
            return t.data_ptr()

        def table(t, dtype, name):
            if t.dtype != dtype or t.dim() != 2 or t.stride(1) != 1 or t.shape[0] < 1:
                raise ValueError(f"{what}: {name} must be a two-dimensional {dtype} tensor with adjacent columns")
            return t.data_ptr(), (t.stride(0) if t.shape[0] > 1 else t.shape[1]), t.shape[0]

        c = _lib.sar_logit_controls()
        self._keep = (state, slots, repetition, presence, frequency, bias_offsets, bias_tokens, bias_values, mask,
                      mask_rows)
        _launch_stream(what, 0, *self._keep)
        if state is not None:
            c.state, c.state_ld, c.n_slots = table(state, torch.int16, "state")
        c.slots = flat(slots, torch.int32, "slots")
        c.repetition = flat(repetition, torch.float32, "repetition")
        c.presence = flat(presence, torch.float32, "presence")
        c.frequency = flat(frequency, torch.float32, "frequency")
        c.bias_offsets = flat(bias_offsets, torch.int32, "bias_offsets")
        c.bias_tokens = flat(bias_tokens, torch.int32, "bias_tokens")
        c.bias_values = flat(bias_values, torch.float32, "bias_values")
        if len({t is None for t in (bias_offsets, bias_tokens, bias_values)}) > 1:
            raise ValueError(f"{what}: biases need offsets, tokens and values")
        if bias_tokens is not None:
            if bias_tokens.numel() != bias_values.numel():
                raise ValueError(f"{what}: bias_tokens and bias_values differ in length")
            c.n_biases = bias_tokens.numel()
            if c.n_biases == 0:  # (an empty tensor has no address)
                c.bias_offsets = c.bias_tokens = c.bias_values = None
        if mask is not None:
            c.mask, c.mask_ld, c.n_masks = table(mask, torch.int32, "mask")
        c.mask_rows = flat(mask_rows, torch.int32, "mask_rows")
        c.count_picks = 1 if count_picks else 0
        lens = [t.numel() for t in (slots, repetition, presence, frequency, mask_rows) if t is not None]
        if bias_offsets is not None:
            lens.append(bias_offsets.numel() - 1)
        if mask is not None and mask_rows is None:
            lens.append(mask.shape[0])
        self.rows = min(lens) if lens else None  # the most rows and tokens a call may have
        self.vocab = min([1 << 30] + ([] if state is None else [state.shape[1]]) + ([] if mask is None else [32 * mask.shape[1]]))
        self.device = next((t.get_device() for t in self._keep if t is not None), None)
        self.c = c


def logits_control(logits, controls: LogitControls, out=None, tokens_out=None, stream=None) -> None:
    """out (the logits' type; may be ``logits``) = the logits under ``controls``;
    tokens_out (int32 [rows]) = each row's pick, -1 where no token is left; see
    ``sar_logits_control``."""
    import torch
    rows, vocab, ld, kind = _rows("logits_control", logits)
    ld_out = 0
    if out is not None:
        out_rows, out_cols, ld_out, out_kind = _rows("logits_control", out)
        if (out_rows, out_cols, out_kind) != (rows, vocab, kind):
            raise ValueError("logits_control: out must have the logits' shape and type")
    if tokens_out is not None and (tokens_out.dtype is not torch.int32 or tokens_out.numel() < rows
                                   or not tokens_out.is_contiguous()):
        raise ValueError("logits_control: tokens_out must be contiguous int32, one per row")
    if (controls.rows is not None and controls.rows < rows) or controls.vocab < vocab:
        raise ValueError("logits_control: the controls hold fewer rows or tokens than the logits")
    st = _launch_stream("logits_control", stream, logits, out, tokens_out)
    if controls.device is not None and controls.device != logits.get_device():
        raise ValueError("logits_control: the controls are on another device")
    check(lib().sar_logits_control(logits.data_ptr(), ld, rows, vocab, kind, ctypes.byref(controls.c), _ptr(out), ld_out,
                                   _ptr(tokens_out), st))


def token_state_add(state, slots, offsets, tokens, vocab: int | None = None, prompt_lens=None, reset: bool = False,
                    stream=None) -> None:
    """Counts ``tokens[offsets[i]:offsets[i + 1]]`` into row ``slots[i]`` of the
    int16 ``state`` [slots, >= vocab], the first ``prompt_lens[i]`` of them as
    prompt tokens; ``reset``: the rows are made anew; see ``sar_token_state_add``."""
    import torch
    if state.dtype is not torch.int16 or state.dim() != 2 or (state.shape[1] > 1 and state.stride(1) != 1):
        raise ValueError("token_state_add: state must be two-dimensional int16 with adjacent columns")
    n_slots, cols = state.shape
    vocab = cols if vocab is None else vocab
    if vocab > cols:
        raise ValueError("token_state_add: state is narrower than the vocabulary")
    n = slots.numel()
    for t, least in ((slots, 0), (offsets, n + 1), (tokens, 0), (prompt_lens, n)):
        if t is not None and (t.dtype is not torch.int32 or not t.is_contiguous() or t.numel() < least):
            raise ValueError("token_state_add: index arrays must be contiguous int32 and long enough")
    st = _launch_stream("token_state_add", stream, state, slots, offsets, tokens, prompt_lens)
    check(lib().sar_token_state_add(state.data_ptr(), state.stride(0) if n_slots > 1 else cols, n_slots, vocab,
                                    slots.data_ptr(), n, offsets.data_ptr(), tokens.data_ptr(), tokens.numel(),
                                    _ptr(prompt_lens), 1 if reset else 0, st))
