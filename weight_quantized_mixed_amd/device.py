"""torch device-tensor wrapper around the C ABI (marshalling only).

PyTorch provides device memory and the stream; every computation is a
libqgemm kernel.  Non-GPU tensors are rejected: there is no host fallback.

Every call runs on the current stream, or on `stream`: outputs and workspaces made by
the call then come from that stream's memory.  Tensors passed in are the caller's to keep
until the call's work is done.
"""
from __future__ import annotations

import ctypes
import functools

import numpy as np
import torch

from . import qgemm as _q

A_DTYPE = {"i4": "f16", "u4": "f16", "f16": "f16", "i8": "i8", "i2": "i8"}
WEIGHT_BITS = {"i4": 4, "u4": 4, "f16": 16, "i8": 8, "i2": 2}
OUT_DTYPE = {"f16": ("f16", "f32"), "i8": ("i32", "i32")}


def _ptr(t):
    if t is None:
        return 0
    if not t.is_cuda:
        raise ValueError("qgemm takes device tensors only")
    if not t.is_contiguous():
        raise ValueError("qgemm takes contiguous tensors only")
    return t.data_ptr()


# the current stream's handle without building a Stream object (0.1 against 3 us a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is None:
        return torch.cuda.current_stream().cuda_stream
    return _raw_stream(torch.cuda.current_device())


def _empty(shape, dtype, device, stream=None):
    """A new tensor for work on `stream` (None: the current one).  It comes from that stream's own memory, since a
    block just freed on the current stream may still be in use there, and when freed it waits for both."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(t.device))
    return t


def _check(t, name, shape, dtype):
    """A tensor argument of this shape (a tuple) and type (None passes)."""
    if t is not None and (t.shape != shape or t.dtype != dtype):
        raise ValueError(f"{name}: {dtype} {shape} expected, got {t.dtype} {tuple(t.shape)}")
    return t


def _check_bytes(t, name, need, exact=False):
    """A tensor argument of this many bytes (or more of them), whatever its type (None passes)."""
    held = need if t is None else t.numel() * t.element_size()
    if held < need or (exact and held > need):
        raise ValueError(f"{name}: {need} bytes expected, got {held}")
    return t


def host_to_device(arr: np.ndarray, device="cuda") -> torch.Tensor:
    """Copy a numpy array to the device; uint32 words travel as int32 bits."""
    if arr is None:
        return None
    a = np.ascontiguousarray(arr)
    if a.dtype == np.uint32:
        a = a.view(np.int32)
    return torch.from_numpy(a).to(device)


def quantize_rows(A, Q=None, scales=None, stream=None):
    """Per-row symmetric int8 codes and fp32 scales of fp16 A [M, K] (one kernel)."""
    M, K = A.shape
    if Q is None:
        Q = _empty((M, K), torch.int8, A.device, stream)
    if scales is None:
        scales = _empty((M,), torch.float32, A.device, stream)
    _q.qgemm_quantize_rows(_ptr(A), M, K, _ptr(Q), _ptr(scales), _stream(stream))
    return Q, scales


class _Workspace:
    """Device scratch that grows with the calls that use it.  Outgrown buffers are kept: a
    captured graph may still replay a call that was given one."""

    def __init__(self, device):
        self.device, self.buffers, self.streams = device, [], set()

    def of(self, need, stream=None, at=None):
        """A buffer of `need` bytes for work on `stream` (None: the current one), whose handle `at` the caller may know."""
        if not need:
            return None
        if not self.buffers or self.buffers[-1].numel() < need:
            grown = max(need, 2 * self.buffers[-1].numel()) if self.buffers else need
            self.buffers.append(_empty(grown, torch.uint8, self.device, stream))
            self.streams = set()
        if at is None:
            at = _stream(stream)
        if at not in self.streams:  # freed with its object, the buffer waits for every stream that used it
            self.buffers[-1].record_stream(torch.cuda.current_stream() if stream is None else stream)
            self.streams.add(at)
        return self.buffers[-1]


class QGemm:
    """One plan: C[M,N] = A[M,K] . dequant(W) for a fixed shape and format.

    dequant_output: int8 activations with an fp16 output dequantised by per-row
    and per-column scales (run_scaled) instead of the int32 accumulator.
    Split-K (k_parts > 1) reduces with atomics, or with ordered partials when
    deterministic; split_auto lets the library pick the faster of the two.
    """

    def __init__(self, M, N, K, w_dtype, group_size=0, has_zeros=False, k_parts=1,
                 deterministic=False, device="cuda", dequant_output=False, split_auto=False):
        self.M, self.N, self.K, self.w_dtype = int(M), int(N), int(K), w_dtype
        self.a_dtype = A_DTYPE[w_dtype]
        self.out_dtype, self.accum_dtype = OUT_DTYPE[self.a_dtype]
        if dequant_output:
            if self.a_dtype != "i8":
                raise ValueError("dequant_output is for int8 activations")
            self.out_dtype = "f16"
        self.device = torch.device(device)
        flags = (_q.QGEMM_DETERMINISTIC if deterministic else 0) | (_q.QGEMM_SPLIT_AUTO if split_auto else 0)
        self.plan, self.packed_bytes, self.ws_bytes = _q.qgemm_create(
            M, N, K, self.a_dtype, w_dtype, self.out_dtype, self.accum_dtype, group_size,
            int(bool(has_zeros)), k_parts, flags)
        self.path = _q.qgemm_plan_path(self.plan)
        self._ws = _Workspace(self.device)

    def close(self):
        plan = getattr(self, "plan", None)
        if plan:
            self.plan = None
            destroy = getattr(_q, "qgemm_destroy", None)
            if callable(destroy):  # not at interpreter exit, when the module is torn down
                destroy(plan)

    __del__ = close

    def pack(self, w, s=None, z=None, out=None, stream=None):
        if out is None:
            out = _empty((self.packed_bytes,), torch.uint8, self.device, stream)
        _q.qgemm_pack_weights(self.plan, _ptr(w), _ptr(s), _ptr(z), _ptr(out), _stream(stream))
        return out

    def workspace(self, stream=None):
        return self._ws.of(self.ws_bytes, stream)

    def new_output(self, M=None, stream=None):
        dt = torch.float16 if self.out_dtype == "f16" else torch.int32
        return _empty((self.M if M is None else int(M), self.N), dt, self.device, stream)

    def run(self, A, packed, C=None, ws=None, stream=None, bias=None, M=None):
        """C = A . dequant(W) (+ bias[N]) for the plan's M rows, or M <= that."""
        if C is None:
            C = self.new_output(M, stream)
        if ws is None:
            ws = self.workspace(stream)
        wsb = 0 if ws is None else ws.numel()
        if bias is None and M is None:
            _q.qgemm_run(self.plan, _ptr(A), _ptr(packed), _ptr(C), _ptr(ws), wsb, _stream(stream))
        else:
            _q.qgemm_run_ex(self.plan, self.M if M is None else M, _ptr(A), _ptr(packed), _ptr(bias),
                            _ptr(C), _ptr(ws), wsb, _stream(stream))
        return C

    def run_scaled(self, A, packed, row_scales, col_scales, bias=None, C=None, ws=None, stream=None, M=None):
        """fp16 C = acc . row_scales[m] . col_scales[n] (+ bias) for int8 A (dequant_output plans)."""
        if C is None:
            C = self.new_output(M, stream)
        if ws is None:
            ws = self.workspace(stream)
        _q.qgemm_run_scaled(self.plan, self.M if M is None else M, _ptr(A), _ptr(packed), _ptr(row_scales),
                            _ptr(col_scales), _ptr(bias), _ptr(C), _ptr(ws),
                            0 if ws is None else ws.numel(), _stream(stream))
        return C


class QGated:
    """One gated feed-forward plan: C = act(A . dequant(Wg) + bg) * (A . dequant(Wu) + bu), N columns each.

    act: "silu" or "gelu_tanh".  int8 activations (w_dtype "i8", "i2") run through run_scaled.
    The workspaces are kept with the object: calls that may overlap in time pass their own.
    """

    def __init__(self, M, N, K, w_dtype, group_size=0, has_zeros=False, act="silu", device="cuda"):
        self.M, self.N, self.K, self.w_dtype = int(M), int(N), int(K), w_dtype
        self.a_dtype = A_DTYPE[w_dtype]
        self.device = torch.device(device)
        self.plan, self.packed_bytes, self.ws_bytes = _q.qgemm_create_gated(
            M, N, K, self.a_dtype, w_dtype, "f16", OUT_DTYPE[self.a_dtype][1], group_size, int(bool(has_zeros)), act)
        self.groups = 0 if group_size == 0 else 1 if group_size < 0 else self.K // group_size
        self.has_zeros = bool(has_zeros)
        self._ws, self._backward_ws = _Workspace(self.device), _Workspace(self.device)

    close = QGemm.close
    __del__ = close
    workspace = QGemm.workspace

    def pack(self, w_gate, w_up, s_gate=None, s_up=None, z_gate=None, z_up=None, out=None, stream=None):
        """The blob of both projections' canonical weights (scales and zero points where the plan has them)."""
        for name, w in (("w_gate", w_gate), ("w_up", w_up)):
            _check_bytes(w, name, self.N * self.K * WEIGHT_BITS[self.w_dtype] // 8, exact=True)
        tables = (("s_gate", s_gate), ("s_up", s_up)) if self.groups else ()
        for name, t in tables + ((("z_gate", z_gate), ("z_up", z_up)) if self.has_zeros else ()):
            _check(t, name, (self.N, self.groups), torch.float16)
        if out is None:
            out = _empty((self.packed_bytes,), torch.uint8, self.device, stream)
        _check_bytes(out, "out", self.packed_bytes)
        _q.qgemm_pack_gated(self.plan, _ptr(w_gate), _ptr(s_gate), _ptr(z_gate), _ptr(w_up), _ptr(s_up), _ptr(z_up),
                            _ptr(out), _stream(stream))
        return out

    def new_output(self, M=None, stream=None):
        return _empty((self.M if M is None else int(M), self.N), torch.float16, self.device, stream)

    def new_preact(self, M=None, stream=None):
        """Room for the pre-activations of M rows, which backward reads."""
        return _empty((self.M if M is None else int(M), 2 * self.N), torch.float16, self.device, stream)

    def _run(self, A, packed, rs, csg, csu, bias_gate, bias_up, preact, C, ws, stream, M):
        M = self.M if M is None else int(M)
        _check(A, "A", (M, self.K), torch.float16 if self.a_dtype == "f16" else torch.int8)
        for name, b in (("bias_gate", bias_gate), ("bias_up", bias_up)):
            _check(b, name, (self.N,), torch.float16)
        _check(preact, "preact", (M, 2 * self.N), torch.float16)
        _check_bytes(packed, "packed", self.packed_bytes)
        if C is None:
            C = self.new_output(M, stream)
        _check(C, "C", (M, self.N), torch.float16)
        if ws is None:
            ws = self.workspace(stream)
        _q.qgemm_run_gated(self.plan, M, _ptr(A), _ptr(packed), _ptr(rs), _ptr(csg), _ptr(csu), _ptr(bias_gate),
                           _ptr(bias_up), _ptr(preact), _ptr(C), _ptr(ws), 0 if ws is None else ws.numel(),
                           _stream(stream))
        return C

    def run(self, A, packed, C=None, ws=None, stream=None, bias_gate=None, bias_up=None, preact=None, M=None):
        """C for the plan's M rows (or M <= that); preact, if given, is filled for backward."""
        return self._run(A, packed, None, None, None, bias_gate, bias_up, preact, C, ws, stream, M)

    def run_scaled(self, A, packed, row_scales, col_scales_gate, col_scales_up, bias_gate=None, bias_up=None, C=None,
                   ws=None, stream=None, M=None):
        """C for int8 A with fp32 scales per row, and per column of each projection."""
        _check(row_scales, "row_scales", (self.M if M is None else int(M),), torch.float32)
        for name, s in (("col_scales_gate", col_scales_gate), ("col_scales_up", col_scales_up)):
            _check(s, name, (self.N,), torch.float32)
        return self._run(A, packed, row_scales, col_scales_gate, col_scales_up, bias_gate, bias_up, None, C, ws, stream, M)

    def backward(self, A, packed, preact, dC, input_grad=True, weight_grads=None, bias_grads=False, ws=None,
                 stream=None, M=None):
        """{"dA", "dw_gate", "dw_up", "dbias_gate", "dbias_up"} of a run that filled preact (None where not asked for).

        weight_grads: by default for fp16 weights (quantised ones are frozen).
        """
        M = self.M if M is None else int(M)
        if weight_grads is None:
            weight_grads = self.w_dtype == "f16"
        half = torch.float16
        _check(A, "A", (M, self.K), half)
        _check(preact, "preact", (M, 2 * self.N), half)
        _check_bytes(packed, "packed", self.packed_bytes)
        _check(dC, "dC", (M, self.N), half)
        new = lambda *shape: _empty(shape, half, self.device, stream)  # noqa: E731
        dA = new(M, self.K) if input_grad else None
        dw = new(2, self.N, self.K) if weight_grads else None
        db = new(2, self.N) if bias_grads else None
        need = _q.qgemm_gated_backward_workspace(self.plan, M, weight_grads or bias_grads)
        if ws is None:
            ws = self._backward_ws.of(need, stream)
        part = lambda t, i: None if t is None else t[i]  # noqa: E731
        _q.qgemm_gated_backward(self.plan, M, _ptr(A), _ptr(packed), _ptr(preact), _ptr(dC), _ptr(dA),
                                _ptr(part(dw, 0)), _ptr(part(dw, 1)), _ptr(part(db, 0)), _ptr(part(db, 1)), _ptr(ws),
                                ws.numel(), _stream(stream))
        return {"dA": dA, "dw_gate": part(dw, 0), "dw_up": part(dw, 1), "dbias_gate": part(db, 0),
                "dbias_up": part(db, 1)}


def _rows(t, name, T, width):
    """(address, values between rows) of fp16 [T, width], whose rows may be slices of wider ones.

    The step of a single row says nothing, whatever the tensor that it was cut from.
    """
    if not t.is_cuda:
        raise ValueError("qgemm takes device tensors only")
    step, one = t.stride() if t.dim() == 2 else (0, 0)
    if t.dtype != torch.float16 or t.shape != (T, width) or (one != 1 and width > 1) or (step < width and T > 1):
        raise ValueError(f"{name}: fp16 {(T, width)} with contiguous rows expected, got {t.dtype} {tuple(t.shape)}")
    return t.data_ptr(), step if T > 1 else width


def _place(t, stream):
    """(device of a tensor, handle of the stream for a call on it): a kernel runs on the device of its stream."""
    at = t.get_device()
    if at < 0:
        return at, 0  # (refused by the call, behind its other checks)
    if at != (torch.cuda.current_device() if stream is None else stream.device.index):
        raise ValueError(f"the tensors lie on device {at}, which is not that of the stream")
    if stream is not None:
        return at, stream.cuda_stream
    return at, _stream(None) if _raw_stream is None else _raw_stream(at)


# the workspace of an attention call depends on its sizes alone (the last two: window and sinks, or none of them)
_attention_workspace = functools.lru_cache(maxsize=256)(
    lambda n_pages, page_size, kv_heads, head_dim, *sizes: (
        _q.qgemm_attention_workspace if len(sizes) == 6 else _q.qgemm_attention_window_workspace)(
            _q.KVCacheDesc(4096, 4096, n_pages, page_size, kv_heads, head_dim), *sizes))


class PagedKV:
    """A paged key / value cache, k and v [n_pages, kv_heads, page_size, head_dim] in fp16 (given, or made here).

    The attention workspace is kept with the object: calls that may overlap in time pass their own.
    """

    def __init__(self, n_pages, page_size, kv_heads, head_dim, device="cuda", k=None, v=None):
        self.n_pages, self.page_size = int(n_pages), int(page_size)
        self.kv_heads, self.head_dim = int(kv_heads), int(head_dim)
        shape = (self.n_pages, self.kv_heads, self.page_size, self.head_dim)
        new = lambda: torch.zeros(shape, dtype=torch.float16, device=device)  # noqa: E731
        self.k = _check(new() if k is None else k, "k", shape, torch.float16)
        self.v = _check(new() if v is None else v, "v", shape, torch.float16)
        self.desc = _q.KVCacheDesc(_ptr(self.k), _ptr(self.v), self.n_pages, self.page_size, self.kv_heads, self.head_dim)
        self.address = ctypes.addressof(self.desc)
        self._workspace = _Workspace(self.k.device)

    def append(self, q, k, v, cos, sin, positions, slots, q_out=None, interleaved=False, stream=None, norm_eps=None,
               q_weight=None, k_weight=None):
        """Rotated queries [T, q_heads, head_dim]; the rotated keys and the values go to the cache's slots.

        q [T, q_heads * head_dim], k and v [T, kv_heads * head_dim]: rows may be slices of a wider array.
        norm_eps: every query and key head is first divided by its root mean square (this added to the mean) and
        multiplied by q_weight or k_weight (fp16 [head_dim], None: 1).
        """
        if norm_eps is not None:
            at, handle = _place(self.k, stream)
            if stream is not None and q_out is None:
                q_out = _empty((q.shape[0], q.shape[1] // self.head_dim, self.head_dim), torch.float16, q.device, stream)
            return _q.binding().append_norm(at, handle, self.address, self.kv_heads, self.head_dim, q, k, v, cos, sin, positions,
                                            q_weight, k_weight, norm_eps, interleaved, slots, q_out)
        if q_weight is not None or k_weight is not None:
            raise ValueError("q_weight and k_weight are those of norms: norm_eps is missing")
        (T, width), D = q.shape, self.head_dim
        q_heads, kv_width = width // D, self.kv_heads * D
        qp, qs = _rows(q, "q", T, q_heads * D)
        kp, ks = _rows(k, "k", T, kv_width)
        vp, vs = _rows(v, "v", T, kv_width)
        n_pos, half = cos.shape
        _check(cos, "cos", (n_pos, half), torch.float32)
        _check(sin, "sin", (n_pos, half), torch.float32)
        _check(positions, "positions", (T,), torch.int32)
        _check(slots, "slots", (T,), torch.int64)
        if q_out is None:
            q_out = _empty((T, q_heads, D), torch.float16, q.device, stream)
        _check(q_out, "q_out", (T, q_heads, D), torch.float16)
        _q.qgemm_kv_append(self.desc, T, q_heads, qp, qs, kp, ks, vp, vs, _ptr(cos), _ptr(sin), n_pos, 2 * half,
                           int(bool(interleaved)), _ptr(positions), _ptr(slots), _ptr(q_out), _stream(stream))
        return q_out

    def attend(self, q, q_starts, kv_lens, tables, max_q, max_len, prefix_table=None, prefix_len=0, scale=None,
               out=None, lse=None, ws=None, stream=None, window=None, sinks=0):
        """Causal attention of a ragged batch (q [T, q_heads, head_dim]) over its own pages and the shared prefix.

        window: of the tokens up to its own (the prefix's among them) a query sees the last `window` and the first `sinks`.
        """
        T, q_heads, D = q.shape
        if window is not None:
            at, handle = _place(self.k, stream)
            need = _attention_workspace(self.n_pages, self.page_size, self.kv_heads, self.head_dim, T, q_heads, tables.shape[0],
                                        max_q, max_len, prefix_len, window, sinks)
            if ws is None:
                ws = self._workspace.of(need, stream, handle)
            if stream is not None and out is None:
                out = _empty((T, q_heads, D), torch.float16, q.device, stream)
            return _q.binding().attend_window(at, handle, self.address, self.head_dim, q, q_starts, kv_lens, tables, max_q, max_len,
                                              prefix_table, prefix_len, scale, window, sinks, out, lse, ws)
        if sinks:
            raise ValueError("sinks are those of a window: window is missing")
        step, per_head, one = q.stride()
        if (D != self.head_dim or q.dtype != torch.float16 or not q.is_cuda or (one != 1 and D > 1)
                or (per_head != D and q_heads > 1) or (step < q_heads * D and T > 1)):
            raise ValueError(f"q: fp16 [T, q_heads, {self.head_dim}] with contiguous rows on the device expected, "
                             f"got {q.dtype} {tuple(q.shape)}")
        qp, qs = q.data_ptr(), step if T > 1 else q_heads * D
        B, width = tables.shape
        i32 = torch.int32
        _check(q_starts, "q_starts", (B + 1,), i32)
        _check(kv_lens, "kv_lens", (B,), i32)
        _check(tables, "tables", (B, width), i32)
        if prefix_len:
            if prefix_table is None or prefix_table.numel() * self.page_size < prefix_len:
                raise ValueError("prefix_table holds the pages of prefix_len tokens")
            _check(prefix_table, "prefix_table", (prefix_table.numel(),), i32)
        if out is None:
            out = _empty((T, q_heads, D), torch.float16, q.device, stream)
        _check(out, "out", (T, q_heads, D), torch.float16)
        _check(lse, "lse", (T, q_heads), torch.float32)
        need = _attention_workspace(self.n_pages, self.page_size, self.kv_heads, D, T, q_heads, B, max_q, max_len,
                                    prefix_len)
        at = _stream(stream)
        if ws is None:
            ws = self._workspace.of(need, stream, at)
        _q.qgemm_attention(self.desc, T, q_heads, qp, qs, B, _ptr(q_starts), _ptr(kv_lens), _ptr(tables), width,
                           _ptr(prefix_table) if prefix_len else 0, prefix_len, max_q, max_len,
                           D ** -0.5 if scale is None else scale, _ptr(out), _ptr(lse), _ptr(ws),
                           0 if ws is None else ws.numel(), at)
        return out


class PagePool:
    """Which pages of a cache are free, and which each of up to `sequences` sequences holds, all of it on the device.

    ring: the pool's page numbers, int32 [n_pages] (0 .. n_pages - 1 if not given); tables: int32 [sequences, table_width].
    prefix_len tokens of a shared prefix come before the sequences' own (in pages outside the pool); with a window, pages
    of tokens that no query will see again are given back, but for those of the first `sinks` tokens.
    state: int32 [2 * sequences + 2]: the sequences' lengths, their first pages that no window gave back, and of the ring
    the first free page's place and how many are free.  Each call takes the state that the one before left: calls on one
    pool follow one another, on one stream or with the caller's waits between streams.
    """

    def __init__(self, n_pages, page_size, sequences, table_width, prefix_len=0, window=None, sinks=0, device="cuda",
                 ring=None, tables=None):
        self.n_pages, self.page_size, self.B = int(n_pages), int(page_size), int(sequences)
        self.table_width, self.prefix_len = int(table_width), int(prefix_len)
        if window is not None and window < 1:
            raise ValueError("window: at least 1 expected")
        self.window, self.sinks = 0 if window is None else int(window), int(sinks)
        i32 = torch.int32
        if ring is None:
            ring = torch.arange(self.n_pages, dtype=i32, device=device)
        if tables is None:
            tables = torch.full((self.B, self.table_width), -1, dtype=i32, device=device)
        self.ring = _check(ring, "ring", (self.n_pages,), i32)
        self.tables = _check(tables, "tables", (self.B, self.table_width), i32)
        self.state = torch.zeros(2 * self.B + 2, dtype=i32, device=self.ring.device)
        self.state[-1] = self.n_pages
        self._streams = set()

    @property
    def lens(self):
        """Own tokens of each sequence, int32 [sequences]."""
        return self.state[:self.B]

    def extend(self, new_tokens, T, state_out=None, ws=None, stream=None):
        """Room for the batch's new tokens: how many each sequence gets (int32 [sequences]; -1: it ends), T rows in all.

        {"q_starts", "kv_lens", "positions", "slots", "refused"} as append and attend take them; the tables, the ring and
        the state are brought up to date.  Rows behind the last token have slot -1.  A sequence whose tokens find no room
        is marked in refused (int32 [sequences]) and keeps its length; its rows have position and slot -1.
        state_out: where the state after the call goes (by default the pool's own; else that stays as it was, and so the
        same step may be taken again).  kv_lens is a part of it: the next call that writes there changes it, behind the work
        that was put on the stream before.
        """
        at, handle = _place(self.ring, stream)
        if handle not in self._streams:  # freed with the pool, its arrays wait for every stream that used them
            for t in (self.state, self.ring, self.tables):
                if at >= 0:
                    t.record_stream(torch.cuda.current_stream() if stream is None else stream)
            self._streams.add(handle)
        made = slots = None
        if stream is not None:  # results come from the stream's memory
            B, T = self.B, int(T)
            made = _empty((2 * B + 1 + T,), torch.int32, self.ring.device, stream)
            slots = _empty((T,), torch.int64, self.ring.device, stream)
            if ws is None:
                ws = _empty((_q.qgemm_kv_extend_workspace(B, T),), torch.uint8, self.ring.device, stream)
        q_starts, kv_lens, positions, slots, refused = _q.binding().extend(
            at, handle, self.page_size, self.prefix_len, self.window, self.sinks, T, new_tokens, self.state, self.ring, self.tables,
            state_out, ws, made, slots)
        return {"q_starts": q_starts, "kv_lens": kv_lens, "positions": positions, "slots": slots, "refused": refused}


def norm_rotate(q, k, head_dim, cos, sin, positions, q_weight=None, k_weight=None, eps=1e-6, interleaved=False, q_out=None,
                k_out=None, stream=None):
    """(queries [T, q_heads, head_dim], keys [T, kv_heads, head_dim]): each head divided by its root mean square (eps added
    to the mean), multiplied by its weight (fp16 [head_dim], None: 1) and rotated by its token's angles.

    q [T, q_heads * head_dim], k [T, kv_heads * head_dim]: rows may be slices of a wider array.
    The results carry no history, whatever the inputs: norm_rotate_backward gives the gradients.
    """
    at, handle = _place(q, stream)
    if stream is not None:
        new = lambda x: _empty((x.shape[0], x.shape[1] // head_dim, head_dim), torch.float16, x.device, stream)  # noqa: E731
        q_out, k_out = new(q) if q_out is None else q_out, new(k) if k_out is None else k_out
    return _q.binding().norm_rotate(at, handle, head_dim, q, k, cos, sin, positions, q_weight, k_weight, eps, interleaved, q_out, k_out)


def norm_rotate_backward(q, k, dq_out, dk_out, cos, sin, positions, q_weight=None, k_weight=None, eps=1e-6,
                         interleaved=False, weight_grads=True, dq=None, dk=None, ws=None, stream=None):
    """{"dq", "dk", "dq_weight", "dk_weight"} of norm_rotate from the gradients of its outputs (the weights' in fp32; None
    for a weight that is None, or where not asked for).

    dq, dk: where the gradients go, shaped like q and k; rows may be slices of a wider array.
    """
    at, handle = _place(q, stream)
    dw = None
    if stream is not None:
        new = lambda shape, dtype: _empty(shape, dtype, q.device, stream)  # noqa: E731
        dq, dk = new(q.shape, torch.float16) if dq is None else dq, new(k.shape, torch.float16) if dk is None else dk
        if weight_grads:
            T, q_heads, D = dq_out.shape
            dw = new((2, D), torch.float32)
            ws = new((_q.qgemm_norm_rotate_backward_workspace(T, q_heads, dk_out.shape[1], D, True),), torch.uint8) if ws is None else ws
    dq, dk, dqw, dkw = _q.binding().norm_rotate_backward(at, handle, q, k, dq_out, dk_out, cos, sin, positions, q_weight, k_weight, eps,
                                                         interleaved, weight_grads, dq, dk, dw, ws)
    return {"dq": dq, "dk": dk, "dq_weight": dqw, "dk_weight": dkw}
