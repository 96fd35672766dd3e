"""ctypes binding over ``libkvq.so`` (C ABI in ``include/kvq.h``).

Argument marshalling only: every step of the rotated INT4 KV path runs in the
library's CUDA kernels. Tensors are torch CUDA tensors (used for device memory
and streams); their data pointers and sizes cross the C boundary. If the
library is missing this module raises on first use -- there is no fallback.
"""

import ctypes
import math
import os

import torch

from . import build as _build

ROT_NONE, ROT_HADAMARD, ROT_QUAT, ROT_QUAT_FAST, ROT_HADAMARD_SIGNED, ROT_QUAT_MAT = \
    0, 1, 2, 3, 4, 5
FMT_INT4, FMT_MXFP4, FMT_INT2, FMT_INT3, FMT_LUT4 = 0, 1, 2, 3, 4
ERRF_PAGE, ERRF_POS, ERRF_SEQ, ERRF_LEN = 1, 2, 4, 8
STATUS = {0: "KVQ_OK", 1: "KVQ_ERR_INVALID_ARG", 2: "KVQ_ERR_UNSUPPORTED",
          3: "KVQ_ERR_MISALIGNED", 4: "KVQ_ERR_WORKSPACE", 5: "KVQ_ERR_CUDA"}

# every function the header declares, with its ctypes signature
_P, _I32, _I64, _F32, _SZ = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float,
                            ctypes.c_size_t)
SIGNATURES = {
    "kvq_quantize_append": (ctypes.c_int, [_P, _I32, _P, _P, _I64, _P, _P, _I32, _P, _I32, _P, _P,
                                           _P, _P, _P, _P]),
    "kvq_decode_workspace_bytes": (_SZ, [_P, _I32, _I32, _I32]),
    "kvq_paged_decode_attn": (ctypes.c_int, [_P, _I32, _I32, _P, _P, _I32, _P, _I32, _F32, _P, _P,
                                             _P, _P, _P, _P, _SZ, _P, _P]),
    "kvq_dequantize_pages": (ctypes.c_int, [_P, _I32, _P, _I32, _P, _I32, _P, _P, _I32, _I32, _P,
                                            _P, _P]),
    "kvq_paged_decode_attn_noalloc": (ctypes.c_int, [_P, _I32, _I32, _P, _P, _I32, _P, _I32, _F32,
                                                     _P, _P, _P, _P, _P, _P, _P]),
    "kvq_decode_step": (ctypes.c_int, [_P, _I32, _I32, _P, _P, _P, _I64, _P, _I32, _P, _I32, _F32,
                                       _P, _P, _P, _P, _P, _P, _SZ, _P, _P]),
    "kvq_prefill_workspace_bytes": (_SZ, [_P, _I32, _I32, _I32, _I32, _I32]),
    "kvq_paged_prefill_attn": (ctypes.c_int, [_P, _I32, _I32, _I32, _P, _I64, _P, _I32, _P, _I32,
                                              _P, _I32, _F32, _P, _P, _P, _P, _P, _P, _P, _SZ, _P,
                                              _P]),
    "kvq_paged_decode_attn_scored": (ctypes.c_int, [_P, _I32, _I32, _P, _P, _I32, _P, _I32, _F32,
                                                    _P, _P, _P, _P, _P, _P, _P, _SZ, _P, _P]),
    "kvq_shared_prefix_workspace_bytes": (_SZ, [_P, _I32, _I32, _I32, _I32]),
    "kvq_shared_prefix_decode_attn": (ctypes.c_int, [_P, _I32, _I32, _P, _I32, _P, _I32, _P, _I32,
                                                     _F32, _P, _P, _P, _P, _P, _P, _P, _SZ, _P,
                                                     _P]),
    "kvq_decode_fp16_workspace_bytes": (_SZ, [_P, _I32, _I32, _I32]),
    "kvq_paged_decode_attn_fp16": (ctypes.c_int, [_P, _I32, _I32, _P, _P, _I32, _P, _I32, _F32,
                                                  _P, _P, _P, _P, _SZ, _P, _P]),
    "kvq_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "kvq_version": (ctypes.c_char_p, []),
}


class KvqError(RuntimeError):
    def __init__(self, fn, status):
        super().__init__(f"{fn} returned {STATUS.get(status, status)}")
        self.status = status


class CacheDesc(ctypes.Structure):
    """Mirror of ``kvq_cache_desc``."""
    _fields_ = [("head_dim", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("num_pages", ctypes.c_int32),
                ("rot_kind", ctypes.c_int32), ("rot_block", ctypes.c_int32),
                ("quat", ctypes.c_void_p), ("rope", ctypes.c_void_p),
                ("rope_max_pos", ctypes.c_int32), ("format", ctypes.c_int32),
                ("levels", ctypes.c_void_p)]


class ScoreDesc(ctypes.Structure):
    """Mirror of ``kvq_score_desc``."""
    _fields_ = [("softcap", ctypes.c_float), ("window", ctypes.c_int32),
                ("alibi", ctypes.c_void_p), ("first_pos", ctypes.c_void_p),
                ("prefix_lens", ctypes.c_void_p)]


_lib = None


def lib_path():
    return _build.LIB


def lib():
    """Loads libkvq.so (built in-tree by ``build.build()``); raises if absent."""
    global _lib
    if _lib is None:
        path = lib_path()
        if not os.path.exists(path):
            raise RuntimeError(f"libkvq.so not built at {path}: run "
                               "bit_rotated_kv_block_b200.build.build() first")
        L = ctypes.CDLL(path)
        for name, (res, args) in SIGNATURES.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def _ptr(t):
    return None if t is None else t.data_ptr()


# the current stream's handle without building a Stream object (3 us of a
# call's host time), where this torch has it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, dev=None):
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device() if dev is None else dev)
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _ints(t, n, name, dev):
    if t.dtype is not _INT or t.numel() < n or not t.is_contiguous() or t.get_device() != dev:
        raise ValueError(f"{name} must be a contiguous int32 tensor of {n} entries on cuda:{dev}")


_U8, _INT, _HALF = torch.uint8, torch.int32, torch.float16


def _pool(t, shape, dtype, name):
    """One pool of a cache: contiguous, of the cache's shape (or that with more
    pages, or the same bytes in fewer or more dimensions)."""
    if t.dtype is dtype and t.is_contiguous():
        have = t.shape
        if have == shape or (len(have) == len(shape) and have[1:] == shape[1:]
                             and have[0] > shape[0]) \
                or (len(have) != len(shape) and t.numel() == math.prod(shape)):
            return
    raise ValueError(f"{name} must be a contiguous {dtype} tensor {list(shape)}")


def _memory(cache, kc, kp, vc, vp, workspace, err):
    """Checks of what the kernels address by the cache's geometry alone: pools of
    another type, layout or size would be misread or read past their end."""
    codes, params, cs, ps, cn, pn = cache.pool_layout
    # (the strides and size of a contiguous tensor of the shape: half the host
    # time of comparing shapes)
    if not (kc.stride() == cs and vc.stride() == cs and kp.stride() == ps and vp.stride() == ps
            and kc.nbytes == cn and vc.nbytes == cn and kp.nbytes == pn and vp.nbytes == pn
            and kc.dtype is vc.dtype is _U8 and kp.dtype is vp.dtype is _INT):
        _pool(kc, codes, torch.uint8, "k_codes")
        _pool(vc, codes, torch.uint8, "v_codes")
        _pool(kp, params, torch.int32, "k_params")
        _pool(vp, params, torch.int32, "v_params")
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    if err is not None and (err.dtype is not _INT or err.numel() < 1):
        raise ValueError("err must be an int32 tensor")


def _fit(cache, q, seqs, seq_lens, block_table, kc, kp, vc, vp, out, out_dtype, workspace, err):
    """Checks of the attention entry points with options: every tensor on the
    current device (the library launches there; call inside
    ``torch.cuda.device(...)`` for another), queries and outputs of the
    geometry, index tensors int32 and contiguous, pools of the cache's shape.
    ``seqs`` None: one per query row. Returns q's shape and the device."""
    dev = torch.cuda.current_device()
    shape = q.shape
    _memory(cache, kc, kp, vc, vp, workspace, err)
    if q.dtype is not _HALF or len(shape) != 3 or shape[2] != cache.d:
        raise ValueError(f"q must be float16 [rows][Hq][{cache.d}]")
    if seqs is None:
        seqs = shape[0]
    if out is not None and (out.dtype is not out_dtype or out.shape != shape
                            or not out.is_contiguous() or out.get_device() != dev):
        raise ValueError(f"out must be a contiguous {out_dtype} tensor of q's shape on cuda:{dev}")
    _ints(seq_lens, seqs, "seq_lens", dev)
    rows = block_table.shape
    if len(rows) != 2 or rows[0] < seqs:
        raise ValueError("block_table must have a row per sequence")
    _ints(block_table, 0, "block_table", dev)
    if not (q.get_device() == kc.get_device() == kp.get_device() == vc.get_device()
            == vp.get_device() == dev) or (workspace is not None and workspace.get_device() != dev) \
            or (err is not None and err.get_device() != dev):
        raise ValueError(f"q, pages, workspace and err must be on the current device, cuda:{dev}")
    return shape, dev


def _i32(v, name):
    """A size or position for the library (ctypes would keep its low 32 bits)."""
    v = int(v)
    if not -2147483648 <= v <= 2147483647:
        raise ValueError(f"{name} does not fit 32 bits")
    return v


def _new(shape, dtype, q, stream):
    """Output or workspace of a call on ``stream``: allocated on it, so that its
    memory is neither taken from nor given to work that the call overlaps."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=q.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=q.device)


def _check(fn, status):
    if status != 0:
        raise KvqError(fn, status)


class Cache:
    """Geometry of one paged INT4 cache plus the device quaternion table
    (kept alive here because the descriptor points at it)."""

    def __init__(self, head_dim, num_kv_heads, page_size, num_pages, rot_kind=ROT_HADAMARD,
                 rot_block=0, quat=None, device="cuda", rope=None, fmt=FMT_INT4, levels=None):
        """``rope``: optional RoPE table float32 [max_pos][d/2][2] of (cos, sin);
        ``fmt``: a kvq_format; ``levels``: the 16-entry table of FMT_LUT4."""
        self.fmt = fmt
        self.levels = None
        if levels is not None:
            self.levels = torch.as_tensor(levels, dtype=torch.float32).contiguous().to(device)
        self.d, self.H, self.P, self.NP = head_dim, num_kv_heads, page_size, num_pages
        self.rot_kind, self.rot_block = rot_kind, rot_block
        # shapes, strides and bytes of the code pools and of the parameter pools
        r = self.code_row_bytes()
        H, P = num_kv_heads, page_size
        self.pool_layout = ((num_pages, H, P, r), (num_pages, H, P), (H * P * r, P * r, r, 1),
                            (H * P, P, 1), num_pages * H * P * r, 4 * num_pages * H * P)
        self.quat = None  # the rotation's table: quaternions, or signs
        if rot_kind in (ROT_QUAT, ROT_QUAT_FAST, ROT_HADAMARD_SIGNED, ROT_QUAT_MAT):
            self.quat = torch.as_tensor(quat, dtype=torch.float32).contiguous().to(device)
        self.rope = None
        if rope is not None:
            self.rope = torch.as_tensor(rope, dtype=torch.float32).contiguous().to(device)
        self.desc = CacheDesc(head_dim, num_kv_heads, page_size, num_pages, rot_kind, rot_block,
                              None if self.quat is None else self.quat.data_ptr(),
                              None if self.rope is None else self.rope.data_ptr(),
                              0 if self.rope is None else int(self.rope.shape[0]), fmt,
                              None if self.levels is None else self.levels.data_ptr())

    def code_row_bytes(self):
        return self.d * {FMT_INT2: 2, FMT_INT3: 3}.get(self.fmt, 4) // 8

    def new_pools(self, device="cuda", fill=None):
        """(codes uint8 [NP][H][P][d * bits / 8], params int32 [NP][H][P]) for one
        of K / V; each params word is the binary16 pair (scale, minimum), scale in
        the low half (MX FP4: the four block-scale bytes)."""
        codes = torch.empty((self.NP, self.H, self.P, self.code_row_bytes()), dtype=torch.uint8,
                            device=device)
        params = torch.empty((self.NP, self.H, self.P), dtype=torch.int32, device=device)
        if fill is not None:
            codes.fill_(fill)
            params.fill_(int.from_bytes(bytes([fill] * 4), "little", signed=True))
        return codes, params


class Score:
    """Scoring options: ``softcap`` (0: none), ``window`` (0: none), ``alibi``
    float32 CUDA [num_q_heads] of slopes, ``first_pos`` int32 CUDA with one
    entry per query token, ``prefix_lens`` int32 CUDA [num_seqs] (prompt
    attention only). The tensors are kept alive here."""

    def __init__(self, softcap=0.0, window=0, alibi=None, first_pos=None, prefix_lens=None):
        for t, dt, name in ((alibi, torch.float32, "alibi"), (first_pos, torch.int32, "first_pos"),
                            (prefix_lens, torch.int32, "prefix_lens")):
            if t is not None and (t.dtype != dt or not t.is_contiguous()):
                raise ValueError(f"{name} must be a contiguous {dt} tensor")
        if not 0 <= window < 2 ** 31:
            raise ValueError("window must be in [0, 2^31)")
        # (read-only: the descriptor holds their addresses)
        self._alibi, self._first_pos, self._prefix_lens = alibi, first_pos, prefix_lens
        self.desc = ScoreDesc(softcap, window, *(None if t is None else t.data_ptr()
                                                 for t in (alibi, first_pos, prefix_lens)))
        self.held = tuple((t, n) for t, n in ((alibi, "alibi"), (first_pos, "first_pos"),
                                              (prefix_lens, "prefix_lens")) if t is not None)
        if softcap != 0.0 and self.desc.softcap == 0.0:
            raise ValueError("softcap must be 0 or a float32 number of at least 1e-6")

    alibi = property(lambda self: self._alibi)
    first_pos = property(lambda self: self._first_pos)
    prefix_lens = property(lambda self: self._prefix_lens)


def _score(score, q, seqs, shape=None):
    """The options' descriptor for queries ``q`` [rows][Hq][d] of ``seqs``
    sequences; their tensors have to fit them."""
    if score is None:
        return None
    if score.held:
        rows, heads, _ = shape or q.shape
        for t, name in score.held:
            n = heads if name == "alibi" else rows if name == "first_pos" else seqs
            if t.numel() != n or t.device != q.device:
                raise ValueError(f"{name} must hold {n} entries on {q.device}")
    return ctypes.byref(score.desc)


def quantize_append(cache, k, v, token_seq, token_pos, block_table, k_codes, k_params, v_codes,
                    v_params, err=None, stream=None, tok_stride=None):
    """k, v: float16 CUDA [T][H][d] (token stride ``tok_stride`` elements)."""
    T = int(token_seq.numel())
    if tok_stride is None:
        tok_stride = k.stride(0)
    st = lib().kvq_quantize_append(ctypes.byref(cache.desc), T, _ptr(k), _ptr(v), int(tok_stride),
                                   _ptr(token_seq), _ptr(token_pos), int(block_table.shape[0]),
                                   _ptr(block_table), int(block_table.shape[1]), _ptr(k_codes),
                                   _ptr(k_params), _ptr(v_codes), _ptr(v_params), _ptr(err),
                                   _stream(stream))
    _check("kvq_quantize_append", st)


def decode_workspace_bytes(cache, num_seqs, num_q_heads, max_seq_len):
    return int(lib().kvq_decode_workspace_bytes(ctypes.byref(cache.desc), num_seqs, num_q_heads,
                                                max_seq_len))


def paged_decode_attn(cache, q, seq_lens, max_seq_len, block_table, k_codes, k_params, v_codes,
                      v_params, out=None, workspace=None, sm_scale=None, err=None, stream=None):
    """q: float16 CUDA [S][Hq][d]; returns float32 [S][Hq][d]. The workspace
    (``decode_workspace_bytes``) needs no initialisation; without one, one is
    allocated for the call."""
    S, Hq, d = q.shape
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty((S, Hq, d), dtype=torch.float32, device=q.device)
    need = decode_workspace_bytes(cache, S, Hq, max_seq_len)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    st = lib().kvq_paged_decode_attn(ctypes.byref(cache.desc), S, Hq, _ptr(q), _ptr(seq_lens),
                                     int(max_seq_len), _ptr(block_table),
                                     int(block_table.shape[1]), float(sm_scale), _ptr(k_codes),
                                     _ptr(k_params), _ptr(v_codes), _ptr(v_params), _ptr(out),
                                     _ptr(workspace), workspace.numel() * workspace.element_size(),
                                     _ptr(err), _stream(stream))
    _check("kvq_paged_decode_attn", st)
    return out


def decode_step(cache, q, k_new, v_new, seq_lens, max_seq_len, block_table, k_codes, k_params,
                v_codes, v_params, out=None, workspace=None, sm_scale=None, err=None,
                stream=None):
    """One fused decode step: writes the new token of every sequence (k_new,
    v_new float16 CUDA [S][H][d], or row-strided views with the same row
    layout) at position seq_lens[s] - 1 and returns the attention output
    float32 [S][Hq][d] over seq_lens[s] tokens (lengths include the new
    token). Workspace as for ``paged_decode_attn``."""
    S, Hq, d = q.shape
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty((S, Hq, d), dtype=torch.float32, device=q.device)
    need = decode_workspace_bytes(cache, S, Hq, max_seq_len)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    new_stride = k_new.stride(0)
    if v_new.stride(0) != new_stride:
        raise ValueError("k_new and v_new must share the row stride")
    st = lib().kvq_decode_step(ctypes.byref(cache.desc), S, Hq, _ptr(q), _ptr(k_new), _ptr(v_new),
                               int(new_stride), _ptr(seq_lens), int(max_seq_len),
                               _ptr(block_table), int(block_table.shape[1]), float(sm_scale),
                               _ptr(k_codes), _ptr(k_params), _ptr(v_codes), _ptr(v_params),
                               _ptr(out), _ptr(workspace),
                               workspace.numel() * workspace.element_size(), _ptr(err),
                               _stream(stream))
    _check("kvq_decode_step", st)
    return out


def prefill_workspace_bytes(cache, num_seqs, num_q_heads, num_tokens, max_q_len, max_seq_len):
    return int(lib().kvq_prefill_workspace_bytes(ctypes.byref(cache.desc), num_seqs, num_q_heads,
                                                 num_tokens, _i32(max_q_len, "max_q_len"),
                                                 _i32(max_seq_len, "max_seq_len")))


def paged_prefill_attn(cache, q, q_start, max_q_len, seq_lens, max_seq_len, block_table, k_codes,
                       k_params, v_codes, v_params, out=None, workspace=None, sm_scale=None,
                       score=None, err=None, stream=None):
    """Attention of several query tokens per sequence over the cached pages
    (which already hold their K and V). q: float16 CUDA [T][Hq][d] (any token
    stride); ``q_start`` int32 [S + 1]: sequence s owns tokens
    [q_start[s], q_start[s + 1]), its last positions; returns float16
    [T][Hq][d]. ``score``: a ``Score`` (None: plain causal)."""
    S = seq_lens.numel()
    shape, dev = _fit(cache, q, S, seq_lens, block_table, k_codes, k_params, v_codes, v_params, out,
                      torch.float16, workspace, err)
    T, Hq, d = shape
    _ints(q_start, S + 1, "q_start", dev)
    if q.stride(2) != 1 or (Hq > 1 and q.stride(1) != d):
        raise ValueError("q rows of a token must be contiguous")
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(d)
    if out is None:
        out = _new((T, Hq, d), torch.float16, q, stream)
    if workspace is None:
        need = prefill_workspace_bytes(cache, S, Hq, T, max_q_len, max_seq_len)
        workspace = _new(max(need, 16), torch.uint8, q, stream)
    st = lib().kvq_paged_prefill_attn(
        ctypes.byref(cache.desc), S, Hq, T, q.data_ptr(), q.stride(0) if T > 1 else Hq * d,
        q_start.data_ptr(), _i32(max_q_len, "max_q_len"), seq_lens.data_ptr(),
        _i32(max_seq_len, "max_seq_len"), block_table.data_ptr(), int(block_table.shape[1]),
        float(sm_scale), _score(score, q, S, shape),
        k_codes.data_ptr(), k_params.data_ptr(), v_codes.data_ptr(), v_params.data_ptr(),
        out.data_ptr(), workspace.data_ptr(), workspace.nbytes, _ptr(err), _stream(stream, dev))
    _check("kvq_paged_prefill_attn", st)
    return out


def paged_decode_attn_scored(cache, q, seq_lens, max_seq_len, block_table, k_codes, k_params,
                             v_codes, v_params, score=None, out=None, workspace=None,
                             sm_scale=None, err=None, stream=None):
    """``paged_decode_attn`` with scoring options (a ``Score``; its first_pos
    has one entry per sequence); same workspace."""
    shape, dev = _fit(cache, q, None, seq_lens, block_table, k_codes, k_params, v_codes, v_params,
                      out, torch.float32, workspace, err)
    S, Hq, d = shape
    if not q.is_contiguous():
        raise ValueError("q must be contiguous")
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(d)
    if out is None:
        out = _new((S, Hq, d), torch.float32, q, stream)
    if workspace is None:
        need = decode_workspace_bytes(cache, S, Hq, max_seq_len)
        workspace = _new(max(need, 16), torch.uint8, q, stream)
    st = lib().kvq_paged_decode_attn_scored(
        ctypes.byref(cache.desc), S, Hq, q.data_ptr(), seq_lens.data_ptr(),
        _i32(max_seq_len, "max_seq_len"), block_table.data_ptr(), int(block_table.shape[1]),
        float(sm_scale), _score(score, q, S, shape),
        k_codes.data_ptr(), k_params.data_ptr(), v_codes.data_ptr(), v_params.data_ptr(),
        out.data_ptr(), workspace.data_ptr(), workspace.nbytes, _ptr(err), _stream(stream, dev))
    _check("kvq_paged_decode_attn_scored", st)
    return out


def shared_prefix_workspace_bytes(cache, num_seqs, num_q_heads, prefix_len, max_seq_len):
    return int(lib().kvq_shared_prefix_workspace_bytes(ctypes.byref(cache.desc), num_seqs,
                                                       num_q_heads, _i32(prefix_len, "prefix_len"),
                                                       _i32(max_seq_len, "max_seq_len")))


def shared_prefix_decode_attn(cache, q, prefix_len, seq_lens, max_seq_len, block_table, k_codes,
                              k_params, v_codes, v_params, score=None, out=None, workspace=None,
                              sm_scale=None, err=None, stream=None):
    """Decode attention of a batch whose sequences share their first
    ``prefix_len`` tokens (pages taken from row 0 of the table, read once for
    the batch); ``seq_lens`` are whole lengths. q: float16 CUDA [S][Hq][d];
    returns float16 [S][Hq][d]."""
    shape, dev = _fit(cache, q, None, seq_lens, block_table, k_codes, k_params, v_codes, v_params,
                      out, torch.float16, workspace, err)
    S, Hq, d = shape
    if not q.is_contiguous():
        raise ValueError("q must be contiguous")
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(d)
    if out is None:
        out = _new((S, Hq, d), torch.float16, q, stream)
    if workspace is None:
        need = shared_prefix_workspace_bytes(cache, S, Hq, prefix_len, max_seq_len)
        workspace = _new(max(need, 16), torch.uint8, q, stream)
    st = lib().kvq_shared_prefix_decode_attn(
        ctypes.byref(cache.desc), S, Hq, q.data_ptr(), _i32(prefix_len, "prefix_len"),
        seq_lens.data_ptr(), _i32(max_seq_len, "max_seq_len"), block_table.data_ptr(),
        int(block_table.shape[1]), float(sm_scale),
        _score(score, q, S, shape), k_codes.data_ptr(), k_params.data_ptr(), v_codes.data_ptr(),
        v_params.data_ptr(), out.data_ptr(), workspace.data_ptr(), workspace.nbytes, _ptr(err),
        _stream(stream, dev))
    _check("kvq_shared_prefix_decode_attn", st)
    return out


def decode_fp16_workspace_bytes(cache, num_seqs, num_q_heads, max_seq_len):
    return int(lib().kvq_decode_fp16_workspace_bytes(ctypes.byref(cache.desc), num_seqs,
                                                     num_q_heads, max_seq_len))


def paged_decode_attn_fp16(cache, q, seq_lens, max_seq_len, block_table, k_pages, v_pages,
                           out=None, workspace=None, sm_scale=None, err=None, stream=None):
    """Full-precision baseline over a binary16 paged cache ``k_pages``,
    ``v_pages`` (float16 CUDA [NP][H][P][d], unrotated); q float16 [S][Hq][d];
    returns float32 [S][Hq][d]. Workspace as for ``paged_decode_attn``."""
    S, Hq, d = q.shape
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty((S, Hq, d), dtype=torch.float32, device=q.device)
    need = decode_fp16_workspace_bytes(cache, S, Hq, max_seq_len)
    if workspace is None:
        workspace = torch.zeros(max(need, 16), dtype=torch.uint8, device=q.device)
    st = lib().kvq_paged_decode_attn_fp16(ctypes.byref(cache.desc), S, Hq, _ptr(q),
                                          _ptr(seq_lens), int(max_seq_len), _ptr(block_table),
                                          int(block_table.shape[1]), float(sm_scale),
                                          _ptr(k_pages), _ptr(v_pages), _ptr(out),
                                          _ptr(workspace),
                                          workspace.numel() * workspace.element_size(),
                                          _ptr(err), _stream(stream))
    _check("kvq_paged_decode_attn_fp16", st)
    return out


def paged_decode_attn_noalloc(cache, q, seq_lens, max_seq_len, block_table, k_codes, k_params,
                              v_codes, v_params, out=None, sm_scale=None, err=None, stream=None):
    """Decode attention whose scratch is the library's fixed device array
    (for callers that cannot allocate); q: float16 CUDA [S][Hq][d]."""
    S, Hq, d = q.shape
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty((S, Hq, d), dtype=torch.float32, device=q.device)
    st = lib().kvq_paged_decode_attn_noalloc(ctypes.byref(cache.desc), S, Hq, _ptr(q),
                                             _ptr(seq_lens), int(max_seq_len), _ptr(block_table),
                                             int(block_table.shape[1]), float(sm_scale),
                                             _ptr(k_codes), _ptr(k_params), _ptr(v_codes),
                                             _ptr(v_params), _ptr(out), _ptr(err),
                                             _stream(stream))
    _check("kvq_paged_decode_attn_noalloc", st)
    return out


def dequantize_pages(cache, seq_lens, max_seq_len, block_table, codes, params, unrotate=False,
                     out_fp32=True, out=None, err=None, stream=None):
    S = int(block_table.shape[0])
    if out is None:
        out = torch.zeros((S, max_seq_len, cache.H, cache.d),
                          dtype=torch.float32 if out_fp32 else torch.float16,
                          device=codes.device)
    st = lib().kvq_dequantize_pages(ctypes.byref(cache.desc), S, _ptr(seq_lens), int(max_seq_len),
                                    _ptr(block_table), int(block_table.shape[1]), _ptr(codes),
                                    _ptr(params), int(bool(unrotate)), int(bool(out_fp32)),
                                    _ptr(out), _ptr(err), _stream(stream))
    _check("kvq_dequantize_pages", st)
    return out


def version():
    return lib().kvq_version().decode()
