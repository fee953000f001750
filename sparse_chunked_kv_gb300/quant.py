"""Tensor-level helpers of the 8-bit chunk pool over the C ABI: argument
checks, output and workspace allocation through torch, then one call into
libpfd.  No arithmetic of the method happens here.

The pool keeps a code per value (torch.float8_e4m3fn or torch.int8) and one
power-of-two scale, as a biased exponent byte, per block of 16 slot rows and
KV head; slots start at multiples of 16 rows.

Every call runs on the device of its tensors, on that device's current stream
or on `stream` (a torch stream, or a raw cudaStream_t).  What a call allocates
(outputs that were not passed, workspace) belongs to the stream it runs on, and
what it is given is marked as in use there (Tensor.record_stream), so that a
temporary of another stream may be dropped at once; ordering the streams is the
caller's.
The calls neither copy between host and device nor wait, once a plan is made
and max_len is given, so they may be captured into a CUDA graph.  The graph keeps
addresses: the plan, the pool and the tensors given have to live as long as it.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from . import _abi

_BF16, _F32, _I32, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
_FORMATS = {torch.float8_e4m3fn: _abi.KV_E4M3, torch.int8: _abi.KV_INT8}


def _need(tensor, dtype, shape, what, device):
    """A contiguous CUDA tensor of this type, shape (a tuple) and device.  (The
    calls of a decode step are a few microseconds of kernel: what is checked per
    tensor stays this short.)"""
    if (tensor is None or tensor.dtype is not dtype or tensor.shape != shape
            or tensor.device != device or not tensor.is_contiguous()):
        _refuse(tensor, dtype, shape, what, device)


def _refuse(tensor, dtype, shape, what, device):
    if tensor is None or not tensor.is_cuda or not tensor.is_contiguous():
        raise ValueError(f"{what}: expected a contiguous CUDA tensor")
    if tensor.dtype != dtype:
        raise ValueError(f"{what}: expected {dtype}, got {tensor.dtype}")
    if tensor.device != device:
        raise ValueError(f"{what}: on {tensor.device}, the call on {device}")
    raise ValueError(f"{what}: expected shape {list(shape)}, got {list(tensor.shape)}")


def _rows(tensor, what):
    """The first extent of a tensor whose shape is checked next."""
    if tensor is None or tensor.dim() == 0:
        raise ValueError(f"{what}: expected a contiguous CUDA tensor")
    return tensor.shape[0]


def _apart(written, what, **read):
    """The entries that a call writes share no memory with those it reads."""
    if written is None or written.numel() == 0:
        return
    start = written.data_ptr()
    end = start + written.numel() * written.element_size()
    for name, t in read.items():
        if t is not None and start < t.data_ptr() + t.numel() * t.element_size() and t.data_ptr() < end:
            raise ValueError(f"{what}: may not share memory with {name}")


def _error_word(dev_err, device):
    if dev_err is None:
        return None
    _need(dev_err, _I32, (1,), "dev_err", device)
    return dev_err.data_ptr()


@contextlib.contextmanager
def _switched(device, stream, given):
    with torch.cuda.device(device):
        if stream is None:
            yield
        else:
            if isinstance(stream, int):
                stream = (torch.cuda.ExternalStream(stream, device=device) if stream
                          else torch.cuda.default_stream(device))
            if stream != torch.cuda.current_stream(device):
                for t in given:
                    if t is not None:
                        t.record_stream(stream)
            with torch.cuda.stream(stream):
                yield


def _call(device, stream, body, given):
    """Runs body() with the call's device and stream the current ones; given():
    the tensors it uses."""
    if stream is None:
        if device.index == torch.cuda.current_device():
            return body()
    elif not isinstance(stream, int) and stream.device != device:
        raise ValueError(f"stream: on {stream.device}, the call on {device}")
    with _switched(device, stream, given() if stream is not None else ()):
        return body()


def _raw_stream(device):
    """The device's current stream as a cudaStream_t.  (The public
    current_stream builds a Stream object: 2 us, a third of a small call.)"""
    return torch._C._cuda_getCurrentRawStream(device.index)


class QuantPool:
    """An 8-bit chunk pool: codes k, v [pool_rows, Hkv, D] and exponent bytes
    exp_k, exp_v [pool_rows / 16, Hkv] (torch.uint8).  Their contents may be
    changed in place; other tensors make another pool."""

    def __init__(self, k, v, exp_k, exp_v):
        if k.dtype not in _FORMATS:
            raise ValueError(f"codes: expected one of {sorted(map(str, _FORMATS))}, got {k.dtype}")
        if not k.is_cuda:
            raise ValueError("pool k: expected a contiguous CUDA tensor")
        if k.dim() != 3:
            raise ValueError(f"codes: expected [pool_rows, Hkv, D], got {list(k.shape)}")
        _need(k, k.dtype, k.shape, "pool k", k.device)
        rows, hkv, d = k.shape
        if rows % _abi.KV_BLOCK != 0 or rows == 0:
            raise ValueError(f"pool rows: expected a multiple of {_abi.KV_BLOCK}, got {rows}")
        exps = (rows // _abi.KV_BLOCK, hkv)
        _need(v, k.dtype, k.shape, "pool v", k.device)
        _need(exp_k, _U8, exps, "pool exp_k", k.device)
        _need(exp_v, _U8, exps, "pool exp_v", k.device)
        self.tensors = (k, v, exp_k, exp_v)
        self.rows, self.n_kv_heads, self.head_dim = rows, hkv, d
        self.device, self.format = k.device, _FORMATS[k.dtype]

    # Read-only: their types and shapes are checked once, when the pool is made.
    k = property(lambda self: self.tensors[0])
    v = property(lambda self: self.tensors[1])
    exp_k = property(lambda self: self.tensors[2])
    exp_v = property(lambda self: self.tensors[3])

    @property
    def pointers(self):
        """Addresses of k, v, exp_k and exp_v now."""
        k, v, exp_k, exp_v = self.tensors
        return k.data_ptr(), v.data_ptr(), exp_k.data_ptr(), exp_v.data_ptr()

    @classmethod
    def zeros(cls, pool_rows, n_kv_heads, head_dim, dtype=torch.float8_e4m3fn, device="cuda"):
        """A pool of zeros with scale 1; pool_rows is rounded up to a multiple of 16."""
        rows = -(-pool_rows // _abi.KV_BLOCK) * _abi.KV_BLOCK
        k = torch.zeros(rows, n_kv_heads, head_dim, dtype=torch.uint8, device=device).view(dtype)
        exp = torch.full((rows // _abi.KV_BLOCK, n_kv_heads), 127, dtype=torch.uint8, device=device)
        return cls(k, torch.zeros_like(k), exp, exp.clone())


def _counts(values, what):
    values = [int(x) for x in values]
    if len(values) < 2 or values[0] != 0 or any(b < a for a, b in zip(values, values[1:])):
        raise ValueError(f"{what}: expected [0, ...], not decreasing")
    return values


class _Plan:
    """Prefix sums of a step's live rows and chunks, in host and device memory."""

    def __init__(self, cu_lq, cu_chunks, n_q_heads, n_kv_heads, head_dim, device):
        cu_lq, cu_chunks = _counts(cu_lq, "cu_lq"), _counts(cu_chunks, "chunk counts")
        if len(cu_lq) != len(cu_chunks):
            raise ValueError("cu_lq and the chunk counts are of different batches")
        self.batch = len(cu_lq) - 1
        self.total_lq, self.total_chunks = cu_lq[-1], cu_chunks[-1]
        self.n_q_heads, self.n_kv_heads, self.head_dim = n_q_heads, n_kv_heads, head_dim
        self.device = torch.device("cuda" if device is None else device)
        if self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        self.cu_lq_host = (ctypes.c_int32 * len(cu_lq))(*cu_lq)
        self.cu_chunks_host = (ctypes.c_int32 * len(cu_chunks))(*cu_chunks)
        self.cu_lq = torch.tensor(cu_lq, dtype=torch.int32, device=self.device)
        self.cu_chunks = torch.tensor(cu_chunks, dtype=torch.int32, device=self.device)
        self.tensors = (self.cu_lq, self.cu_chunks)
        self.pointers = (self.cu_lq.data_ptr(), ctypes.addressof(self.cu_lq_host),
                         self.cu_chunks.data_ptr(), ctypes.addressof(self.cu_chunks_host))
        self.kv_shape = (self.total_lq, n_kv_heads, head_dim)
        self.lse_shape = (self.total_lq, n_q_heads)

    def workspace(self):
        """A new workspace for one call on the current stream (None where none
        is needed)."""
        if self.workspace_bytes == 0:
            return None
        return torch.empty(self.workspace_bytes, dtype=_U8, device=self.device)

    def given_workspace(self, given):
        if given is None:
            return None
        _need(given, _U8, (_rows(given, "workspace"),), "workspace", self.device)
        if given.shape[0] < self.workspace_bytes:
            raise ValueError(f"workspace: {given.shape[0]} bytes of {self.workspace_bytes}")
        return given


class QuantDecodePlan(_Plan):
    """What a decode step over an 8-bit pool knows beforehand: sequence b's live
    rows cu_lq[b] .. cu_lq[b+1] and selected chunks cu_k[b] .. cu_k[b+1] (host
    lists), the heads, and an upper bound of the chunks' lengths (a longer one
    is reported and skipped).  A plan holds no results and no workspace; any number of calls
    may use it at once."""

    def __init__(self, cu_lq, cu_k, n_q_heads, n_kv_heads, head_dim, max_chunk_len,
                 self_keys=True, n_splits=0, sm_scale=0.0, device=None):
        super().__init__(cu_lq, cu_k, n_q_heads, n_kv_heads, head_dim, device)
        self.max_chunk_len, self.self_keys = int(max_chunk_len), bool(self_keys)
        self.n_splits, self.sm_scale = int(n_splits), float(sm_scale)
        with torch.cuda.device(self.device):
            self.workspace_bytes = _abi.pfd_decode_quant_workspace(
                self.batch, self.cu_lq_host, self.cu_chunks_host, n_q_heads, n_kv_heads, head_dim,
                self.max_chunk_len, self.self_keys, self.n_splits)


class QuantMassPlan(_Plan):
    """The same of a chunk-mass call: sequence b's chunks are table entries
    cu_n[b] .. cu_n[b+1].  head_dim None: that of the pool of each call."""

    def __init__(self, cu_lq, cu_n, n_q_heads, n_kv_heads, head_dim=None, sm_scale=0.0, device=None):
        super().__init__(cu_lq, cu_n, n_q_heads, n_kv_heads, head_dim, device)
        self.sm_scale = float(sm_scale)
        self.complete = all(b > a for a, b in zip(self.cu_lq_host, self.cu_lq_host[1:]))
        self.workspace_bytes = _abi.pfd_chunk_mass_workspace(
            self.batch, self.cu_lq_host, self.cu_chunks_host, n_q_heads, n_kv_heads)


def _longest(table, max_len):
    if max_len is not None:
        return max(1, int(max_len))
    return max(1, int(table[:, 1].max().item())) if table.shape[0] > 0 else 1


def pool_quantize(k, v, src_table, pool, slot_row, max_len=None, table=None, dev_err=None,
                  stream=None):
    """Writes slots of an 8-bit pool from bf16 rows (pfd_pool_quantize): slot j
    gets rows src_table[j] = {row, len} of k, v [src_rows, Hkv, D] at pool row
    slot_row[j] (a multiple of 16).  max_len bounds the lengths (None reads the
    largest from the device).  Returns the pool's table [n, 2]."""
    dev, hkv, d = pool.device, pool.n_kv_heads, pool.head_dim
    shape, n = (_rows(k, "k"), hkv, d), _rows(src_table, "src_table")
    _need(k, _BF16, shape, "k", dev)
    _need(v, _BF16, shape, "v", dev)
    _need(src_table, _I32, (n, 2), "src_table", dev)
    _need(slot_row, _I32, (n,), "slot_row", dev)
    err = _error_word(dev_err, dev)
    if table is not None:
        _need(table, _I32, (n, 2), "table", dev)
        _apart(table, "table", src_table=src_table, slot_row=slot_row)

    def body():
        out = torch.empty_like(src_table) if table is None else table
        if n > 0:
            _abi._check(_abi.load().pfd_pool_quantize(
                k.data_ptr(), v.data_ptr(), shape[0], src_table.data_ptr(), n,
                _longest(src_table, max_len), hkv, d, pool.format, *pool.pointers, pool.rows,
                slot_row.data_ptr(), out.data_ptr(), err, _raw_stream(dev)))
        return out

    return _call(dev, stream, body,
                 lambda: (k, v, src_table, *pool.tensors, slot_row, table, dev_err))


def pool_dequantize(pool, table, dst_row, dst_rows=None, sel=None, max_len=None, k=None, v=None,
                    dst_table=None, dev_err=None, stream=None):
    """Reads slots of an 8-bit pool back as bf16 (pfd_pool_dequantize): the
    rows of table[sel[j]] (sel None: table[j]) go to rows dst_row[j] .. of k, v
    [dst_rows, Hkv, D], at least one row where there are slots.  Rows that no slot
    covers are left as they were, or undefined where k and v are allocated here.
    Returns (k, v, dst_table)."""
    dev, hkv, d = pool.device, pool.n_kv_heads, pool.head_dim
    table_len = _rows(table, "table")
    n = table_len if sel is None else _rows(sel, "sel")
    if (k is None) != (v is None) or (k is None and dst_rows is None):
        raise ValueError("expected k and v, or dst_rows")
    rows = _rows(k, "k") if dst_rows is None else dst_rows
    if rows < (1 if n > 0 else 0):
        raise ValueError(f"dst_rows: expected rows for {n} slots, got {rows}")
    _need(table, _I32, (table_len, 2), "table", dev)
    if sel is not None:
        _need(sel, _I32, (n,), "sel", dev)
    _need(dst_row, _I32, (n,), "dst_row", dev)
    err = _error_word(dev_err, dev)
    if k is not None:
        _need(k, _BF16, (rows, hkv, d), "k", dev)
        _need(v, _BF16, (rows, hkv, d), "v", dev)
    if dst_table is not None:
        _need(dst_table, _I32, (n, 2), "dst_table", dev)
        _apart(dst_table, "dst_table", table=table, sel=sel, dst_row=dst_row)

    def body():
        to_k, to_v, to_table = k, v, dst_table
        if to_k is None:
            to_k = torch.empty((rows, hkv, d), dtype=_BF16, device=dev)
            to_v = torch.empty_like(to_k)
        if to_table is None:
            to_table = torch.empty((n, 2), dtype=_I32, device=dev)
        if n > 0:
            _abi._check(_abi.load().pfd_pool_dequantize(
                *pool.pointers, pool.rows, table.data_ptr(), table_len,
                None if sel is None else sel.data_ptr(), n, _longest(table, max_len), hkv, d,
                pool.format, to_k.data_ptr(), to_v.data_ptr(), rows, dst_row.data_ptr(),
                to_table.data_ptr(), err, _raw_stream(dev)))
        return to_k, to_v, to_table

    return _call(dev, stream, body,
                 lambda: (*pool.tensors, table, dst_row, sel, k, v, dst_table, dev_err))


def _check_step(q, pool, plan, lse):
    dev = pool.device
    if plan.device != dev:
        raise ValueError(f"plan: on {plan.device}, the pool on {dev}")
    if plan.n_kv_heads != pool.n_kv_heads or plan.head_dim not in (None, pool.head_dim):
        raise ValueError("plan: made for other heads than the pool's")
    _need(q, _BF16, (plan.total_lq, plan.n_q_heads, pool.head_dim), "q", dev)
    if lse is not None:
        _need(lse, _F32, plan.lse_shape, "lse", dev)
    return dev


def _decode(name, q, k_self, v_self, pool, table, sel, plan, extra, out, lse, dev_err, workspace,
            stream):
    dev, table_len = _check_step(q, pool, plan, lse), _rows(table, "table")
    _need(table, _I32, (table_len, 2), "table", dev)
    _need(sel, _I32, (plan.total_chunks,), "sel", dev)
    live = (None, None)
    if plan.self_keys or k_self is not None or v_self is not None:
        _need(k_self, _BF16, plan.kv_shape, "k_self", dev)
        _need(v_self, _BF16, plan.kv_shape, "v_self", dev)
        live = (k_self.data_ptr(), v_self.data_ptr())
    err = _error_word(dev_err, dev)
    if out is not None:
        _need(out, _BF16, q.shape, "out", dev)
    space = plan.given_workspace(workspace)

    def body():
        to = torch.empty_like(q) if out is None else out
        to_lse = torch.empty(plan.lse_shape, dtype=_F32, device=dev) if lse is None else lse
        if plan.total_lq == 0:
            return to, to_lse
        ws = plan.workspace() if space is None else space
        cu_lq, cu_lq_host, cu_k, cu_k_host = plan.pointers
        _abi._check(getattr(_abi.load(), name)(
            q.data_ptr(), *live, cu_lq, cu_lq_host, pool.format, *pool.pointers, pool.rows,
            table.data_ptr(), table_len, sel.data_ptr(), cu_k, cu_k_host, plan.batch,
            plan.n_q_heads, plan.n_kv_heads, plan.head_dim, plan.max_chunk_len, plan.sm_scale, *extra,
            plan.n_splits, to.data_ptr(), to_lse.data_ptr(), err,
            None if ws is None else ws.data_ptr(), plan.workspace_bytes, _raw_stream(dev)))
        return to, to_lse

    return _call(dev, stream, body, lambda: (q, k_self, v_self, *pool.tensors, table, sel, *plan.tensors,
                                             out, lse, dev_err, space))


def decode_attention_quant(q, k_self, v_self, pool, table, sel, plan, out=None, lse=None,
                           dev_err=None, workspace=None, stream=None):
    """Static-KV decode attention of one step over an 8-bit pool
    (pfd_decode_attention_quant).  Returns (out, lse)."""
    if not plan.self_keys:
        raise ValueError("plan: made for a partial step without the live block's keys")
    return _decode("pfd_decode_attention_quant", q, k_self, v_self, pool, table, sel, plan, (), out,
                   lse, dev_err, workspace, stream)


def decode_partial_quant(q, k_self, v_self, pool, table, sel, plan, part_o=None, part_lse=None,
                         dev_err=None, workspace=None, stream=None):
    """One share of a decode step over an 8-bit pool (pfd_decode_partial_quant):
    the given chunks, plus the live block's keys when the plan has self_keys
    (else k_self and v_self may be None).  Returns (part_o, part_lse)."""
    return _decode("pfd_decode_partial_quant", q, k_self, v_self, pool, table, sel, plan,
                   (int(plan.self_keys),), part_o, part_lse, dev_err, workspace, stream)


def chunk_mass_quant(q, pool, table, lse, plan, mass=None, dev_err=None, workspace=None,
                     stream=None):
    """Attention mass of every chunk at the step's normaliser over an 8-bit
    pool's keys (pfd_chunk_mass_quant).  Entries that no sequence with live
    rows owns are left as they were (0 where mass is allocated here).  Returns
    mass [table_len]."""
    if lse is None:
        raise ValueError("lse: expected a contiguous CUDA tensor")
    dev, n = _check_step(q, pool, plan, lse), _rows(table, "table")
    _need(table, _I32, (n, 2), "table", dev)
    err = _error_word(dev_err, dev)
    if mass is not None:
        _need(mass, _F32, (n,), "mass", dev)
    space = plan.given_workspace(workspace)

    def body():
        to = mass
        if to is None:
            whole = plan.complete and plan.total_chunks == n
            to = (torch.empty if whole else torch.zeros)(n, dtype=_F32, device=dev)
        if n == 0 or plan.total_lq == 0:
            return to
        ws = plan.workspace() if space is None else space
        cu_lq, cu_lq_host, _, cu_n_host = plan.pointers
        _abi._check(_abi.load().pfd_chunk_mass_quant(
            q.data_ptr(), cu_lq, cu_lq_host, pool.format, pool.k.data_ptr(), pool.exp_k.data_ptr(),
            pool.rows, table.data_ptr(), n, cu_n_host, lse.data_ptr(), plan.batch, plan.n_q_heads,
            plan.n_kv_heads, pool.head_dim, plan.sm_scale, to.data_ptr(), err,
            None if ws is None else ws.data_ptr(), plan.workspace_bytes, _raw_stream(dev)))
        return to

    return _call(dev, stream, body, lambda: (q, pool.k, pool.exp_k, table, lse, *plan.tensors, mass,
                                             dev_err, space))
