"""paged_kv_decode_gb300 -- paged-KV attention for a GB300 (sm_103a), Python binding.

Thin marshalling over the C ABI of libpkv (include/pkv.h): every step of the
path (KV append, decode attention, chunked-prefill attention) runs in the
library's CUDA kernels. torch tensors supply device memory and the current
CUDA stream. There is no CPU fallback: without the compiled library every call
raises.

Layout (see include/pkv.h): pools bf16 [num_pages, Hkv, 16, D]; q / out bf16
[rows, Hq, D]; block tables int32 [rows, max_pages]; lengths int32. The Qwen3
decoder's 16/8/128 runs the tuned kernels; append, decode, the fused append +
decode call and chunked prefill also take head_dim 64 or 128 with 1 to 8 query
heads per KV head.
"""
from __future__ import annotations

import ctypes
from typing import Optional

from . import _lib

PKV_OK = 0
PKV_STATUS_BYTES = 256
ERRORS = {
    -1: "PKV_ERR_NULL_ARG",
    -2: "PKV_ERR_BAD_SHAPE",
    -3: "PKV_ERR_UNSUPPORTED",
    -4: "PKV_ERR_WORKSPACE_TOO_SMALL",
    -5: "PKV_ERR_CUDA",
    -6: "PKV_ERR_DEVICE_TIMEOUT",
    -7: "PKV_ERR_OUT_OF_BOUNDS",
    -8: "PKV_ERR_MISALIGNED",
}
ERR_CODES = {name: code for code, name in ERRORS.items()}

__all__ = [
    "PkvError", "desc", "Workspace", "append", "decode_attn", "prefill_chunk_attn",
    "decode_workspace_bytes", "prefill_workspace_bytes", "workspace_init", "read_status", "status_string",
    "decode_attn_noalloc", "decode_append_attn", "mixed_step_attn", "mixed_workspace_bytes", "rope_cos_sin",
    "append_rope", "append_rope_fp8", "decode_attn_fp8", "expand_fp8",
]


class PkvError(RuntimeError):
    def __init__(self, code: int, what: str = ""):
        self.code = code
        super().__init__(f"{what}: {ERRORS.get(code, code)} ({status_string(code)})")


def status_string(code: int) -> str:
    return _lib.load().pkv_status_string(int(code)).decode()


def _check(code: int, what: str):
    if code != PKV_OK:
        raise PkvError(code, what)


def desc(num_pages: int, num_q_heads: int = 16, num_kv_heads: int = 8, head_dim: int = 128, page_size: int = 16):
    return _lib.CacheDesc(num_q_heads, num_kv_heads, head_dim, page_size, int(num_pages))


def _desc_of(k_pages, num_q_heads: Optional[int] = None) -> "_lib.CacheDesc":
    """Descriptor of a pool [num_pages, num_kv_heads, page_size, head_dim]; num_q_heads from the
    query tensor (default: as many as KV heads, which is all an append needs)."""
    if k_pages.dim() != 4:
        raise ValueError("pools are [num_pages, num_kv_heads, page_size, head_dim]")
    p, hkv, ps, d = k_pages.shape
    return desc(p, hkv if num_q_heads is None else int(num_q_heads), hkv, d, ps)


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream):
    import torch

    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _need(t, dtype, name, device=None):
    import torch

    if t is None:
        raise ValueError(f"{name} is required")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (the library has no CPU path)")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    return t


def workspace_init(ws, stream=None):
    _check(_lib.load().pkv_workspace_init(ctypes.c_void_p(ws.data_ptr()), ws.numel() * ws.element_size(),
                                          _stream(stream)), "pkv_workspace_init")


def read_status(ws, stream=None) -> int:
    """Status word of a workspace (synchronises the stream; tests and debugging only)."""
    return int(_lib.load().pkv_read_status(ctypes.c_void_p(ws.data_ptr()), _stream(stream)))


def decode_workspace_bytes(batch: int, max_pages: int, num_pages: int = 1, num_q_heads: int = 16,
                           num_kv_heads: int = 8, head_dim: int = 128) -> int:
    """Workspace bytes of a decode call (default geometry: the Qwen3 decoder, 16/8/128)."""
    d = desc(num_pages, num_q_heads, num_kv_heads, head_dim)
    return int(_lib.load().pkv_decode_workspace_bytes(ctypes.byref(d), int(batch), int(max_pages)))


def prefill_workspace_bytes(num_seqs: int, max_q_len: int, num_pages: int = 1, num_q_heads: int = 16,
                            num_kv_heads: int = 8, head_dim: int = 128) -> int:
    """Workspace bytes of a prefill call (default geometry: the Qwen3 decoder, 16/8/128)."""
    d = desc(num_pages, num_q_heads, num_kv_heads, head_dim)
    return int(_lib.load().pkv_prefill_workspace_bytes(ctypes.byref(d), int(num_seqs), int(max_q_len)))


class Workspace:
    """A zero-initialised device workspace (uint8 tensor) for one stream's calls."""

    def __init__(self, nbytes: int, device=None):
        import torch

        nbytes = max(int(nbytes), PKV_STATUS_BYTES)
        self.tensor = torch.empty(nbytes, dtype=torch.uint8, device=device or "cuda")
        workspace_init(self.tensor)

    @property
    def nbytes(self) -> int:
        return self.tensor.numel()

    def status(self) -> int:
        return read_status(self.tensor)

    def check(self, what: str = "device status"):
        """Read the status word (synchronises); on a device error, zero the workspace again before
        raising: a call that stopped early may have left split counters or tagged records behind,
        which the next call would take for its own."""
        code = self.status()
        if code != PKV_OK:
            workspace_init(self.tensor)
            raise PkvError(code, what)

    def ensure(self, nbytes: int):
        if nbytes > self.nbytes:
            self.__init__(nbytes, self.tensor.device)
        return self


def append(k_new, v_new, slot_mapping, k_pages, v_pages, workspace: Optional[Workspace] = None, stream=None):
    """Write rows k_new / v_new [n, 8, 128] into the pools at slot_mapping [n] (int32)."""
    import torch

    _need(k_pages, torch.bfloat16, "k_pages")
    dev = k_pages.device
    _need(v_pages, torch.bfloat16, "v_pages", dev)
    _need(k_new, torch.bfloat16, "k_new", dev)
    _need(v_new, torch.bfloat16, "v_new", dev)
    _need(slot_mapping, torch.int32, "slot_mapping", dev)
    n = slot_mapping.numel()
    if k_new.shape[0] != n or v_new.shape != k_new.shape or v_pages.shape != k_pages.shape:
        raise ValueError("shape mismatch")
    d = _desc_of(k_pages)
    ws = workspace.tensor if workspace is not None else None
    rc = _lib.load().pkv_append(_ptr(k_new), _ptr(v_new), _ptr(slot_mapping), n, _ptr(k_pages), _ptr(v_pages),
                                ctypes.byref(d), _stream(stream), _ptr(ws), 0 if ws is None else ws.numel())
    _check(rc, "pkv_append")


def decode_attn(q, k_pages, v_pages, block_table, seq_lens, out, scale: float, workspace: Workspace, stream=None):
    """Decode attention: out [B, Hq, D] from q [B, Hq, D] over the paged cache [P, Hkv, 16, D]
    (Hq / Hkv from 1 to 8 and D in 64, 128; 16/8/128 takes the tuned kernel)."""
    import torch

    _need(k_pages, torch.bfloat16, "k_pages")
    dev = k_pages.device
    _need(v_pages, torch.bfloat16, "v_pages", dev)
    _need(q, torch.bfloat16, "q", dev)
    _need(out, torch.bfloat16, "out", dev)
    _need(block_table, torch.int32, "block_table", dev)
    _need(seq_lens, torch.int32, "seq_lens", dev)
    B = q.shape[0]
    if out.shape != q.shape or block_table.dim() != 2 or block_table.shape[0] != B or seq_lens.numel() != B:
        raise ValueError("shape mismatch")
    d = _desc_of(k_pages, q.shape[1])
    ws = workspace.tensor
    rc = _lib.load().pkv_decode_attn(_ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(block_table), _ptr(seq_lens),
                                     _ptr(out), float(scale), _stream(stream), ctypes.byref(d), B,
                                     block_table.shape[1], _ptr(ws), ws.numel())
    _check(rc, "pkv_decode_attn")


EARLY_PREFETCH = 1  # PKV_DECODE_EARLY_PREFETCH


def rope_cos_sin(theta: float, max_pos: int, head_dim: int = 128, device=None, stream=None):
    """cos/sin table for decode_append_rope_attn, built on the device by pkv_rope_table: fp32
    [max_pos, head_dim], row p = cos(p w_i) for i < head_dim/2, then sin(p w_i), w_i = theta ** (-2 i /
    head_dim), angles in double rounded to float once. (RoPE theta 1e6 for the decoder on "Fun-ASR-Nano
    Native Runtime Design", "Decoder And Prompt".)"""
    import torch

    dev = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
    if dev.type != "cuda":
        raise ValueError("the table is built on a CUDA device (the library has no CPU path)")
    table = torch.empty(int(max_pos), int(head_dim), dtype=torch.float32, device=dev)
    with torch.cuda.device(dev):
        rc = _lib.load().pkv_rope_table(_ptr(table), int(max_pos), int(head_dim), float(theta), _stream(stream))
    _check(rc, "pkv_rope_table")
    return table


def decode_append_rope_attn(q, k_new, v_new, k_pages, v_pages, block_table, seq_lens, cos_sin, out, scale: float,
                            workspace: Workspace, stream=None, early_prefetch: bool = False):
    """decode_append_attn with the rotary embedding of the new token: k_new and every q row are
    rotated at position seq_lens[b] - 1 (pairs i, i + head_dim/2; cos_sin from rope_cos_sin) before
    the append and the scores (any geometry decode_append_attn takes)."""
    import torch

    _need(cos_sin, torch.float32, "cos_sin", k_pages.device)
    if cos_sin.dim() != 2 or cos_sin.shape[1] != q.shape[-1]:
        raise ValueError("cos_sin must be [max_pos, head_dim]")
    _decode_append(q, k_new, v_new, k_pages, v_pages, block_table, seq_lens, out, scale, workspace, stream,
                   early_prefetch, cos_sin)


def decode_append_attn(q, k_new, v_new, k_pages, v_pages, block_table, seq_lens, out, scale: float,
                       workspace: Workspace, stream=None, early_prefetch: bool = False):
    """One decode step of one layer in one launch: write k_new / v_new [B, Hkv, D] at position
    seq_lens[b] - 1 of each request, then decode attention over seq_lens[b] positions (any geometry
    decode_attn takes).

    early_prefetch: the previous kernel on the stream writes neither the pools nor the block
    table nor the lengths, so they may be read while it finishes (PKV_DECODE_EARLY_PREFETCH)."""
    _decode_append(q, k_new, v_new, k_pages, v_pages, block_table, seq_lens, out, scale, workspace, stream,
                   early_prefetch, None)


def _decode_append(q, k_new, v_new, k_pages, v_pages, block_table, seq_lens, out, scale, workspace, stream,
                   early_prefetch, cos_sin):
    import torch

    _need(k_pages, torch.bfloat16, "k_pages")
    dev = k_pages.device
    _need(v_pages, torch.bfloat16, "v_pages", dev)
    _need(q, torch.bfloat16, "q", dev)
    _need(k_new, torch.bfloat16, "k_new", dev)
    _need(v_new, torch.bfloat16, "v_new", dev)
    _need(out, torch.bfloat16, "out", dev)
    _need(block_table, torch.int32, "block_table", dev)
    _need(seq_lens, torch.int32, "seq_lens", dev)
    B = q.shape[0]
    if (out.shape != q.shape or block_table.dim() != 2 or block_table.shape[0] != B or seq_lens.numel() != B
            or k_new.shape[0] != B or v_new.shape != k_new.shape):
        raise ValueError("shape mismatch")
    d = _desc_of(k_pages, q.shape[1])
    ws = workspace.tensor
    flags = EARLY_PREFETCH if early_prefetch else 0
    lib = _lib.load()
    if cos_sin is None:
        rc = lib.pkv_decode_append_attn(_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_pages), _ptr(v_pages),
                                        _ptr(block_table), _ptr(seq_lens), _ptr(out), float(scale), _stream(stream),
                                        ctypes.byref(d), B, block_table.shape[1], _ptr(ws), ws.numel(), flags)
        _check(rc, "pkv_decode_append_attn")
    else:
        rc = lib.pkv_decode_append_rope_attn(_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_pages), _ptr(v_pages),
                                             _ptr(block_table), _ptr(seq_lens), _ptr(cos_sin), cos_sin.shape[0],
                                             _ptr(out), float(scale), _stream(stream), ctypes.byref(d), B,
                                             block_table.shape[1], _ptr(ws), ws.numel(), flags)
        _check(rc, "pkv_decode_append_rope_attn")


# ---------------------------------------------------------------------------- append with rotation, 8-bit cache
# (These calls' kernels are short, so the checks of the good case read each attribute once, in line; only a check that
# fails goes through the helpers that say why.)
def _refuse(dev: int, *tensors):
    """Raise for the first of the (tensor, dtype, name) triples that is not contiguous, of that type and on cuda:dev."""
    import torch

    for t, dtype, name in tensors:
        _need(t, dtype, name, torch.device("cuda", dev))
    raise ValueError("bad tensor")  # (not reached: one of them is refused)


def _device_of(pool, dtype, name: str) -> int:
    """Index of the CUDA device that a pool is on."""
    if pool is None or not pool.is_cuda:
        _need(pool, dtype, name)
    return pool.get_device()


def _good(t, dtype, dev: int) -> bool:
    return t is not None and t.dtype is dtype and t.get_device() == dev and t.is_contiguous()


def _run(what: str, dev: int, stream, fn, before, after):
    """fn(*before, stream, *after) with device `dev` current, on `stream` or the device's current one."""
    import torch

    if stream is None:
        s = torch._C._cuda_getCurrentRawStream(dev)
    else:
        if stream.device.index != dev:
            raise ValueError(f"{what}: the stream is on {stream.device}, the tensors are on cuda:{dev}")
        s = stream.cuda_stream
    if torch._C._cuda_getDevice() == dev:
        rc = fn(*before, s, *after)
    else:
        with torch.cuda.device(dev):
            rc = fn(*before, s, *after)
    if rc != PKV_OK:
        _check(rc, what)


def _ws(workspace: Optional[Workspace], dev: int):
    """(pointer, bytes) of a workspace on dev; (None, 0) without one."""
    if workspace is None:
        return None, 0
    t = workspace.tensor
    if t.get_device() != dev:
        raise ValueError(f"the workspace is on {t.device}, expected cuda:{dev}")
    return t.data_ptr(), t.numel()


def _token_rows(t, name, dev: int, n: int, heads: int, d: int) -> int:
    """Check the new tokens' rows [n, heads, d] (a token's rows contiguous, tokens any distance apart, as in a fused
    projection's output); returns the elements between tokens."""
    import torch

    if t is None:
        raise ValueError(f"{name} is required")
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name}: expected {torch.bfloat16}, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{dev}")
    if t.shape != (n, heads, d):
        raise ValueError(f"{name} must be [{n}, {heads}, {d}], got {tuple(t.shape)}")
    token, head, one = t.stride()
    if one != 1 or (head != d and heads > 1):
        raise ValueError(f"{name}: the rows of a token must be contiguous")
    return token


def _pool_shape(k_pages, v_pages):
    shape = k_pages.shape
    if len(shape) != 4 or v_pages.shape != shape:
        raise ValueError("pools are [num_pages, num_kv_heads, page_size, head_dim]")
    return shape


def _fp8_cache(k_pages, v_pages, kv_scales):
    """Check the pools and scales of an 8-bit cache; returns their device's index and the pools' shape."""
    import torch

    e4m3, e8m0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
    dev = _device_of(k_pages, e4m3, "k_pages")
    if not (_good(k_pages, e4m3, dev) and _good(v_pages, e4m3, dev) and _good(kv_scales, e8m0, dev)):
        _refuse(dev, (k_pages, e4m3, "k_pages"), (v_pages, e4m3, "v_pages"), (kv_scales, e8m0, "kv_scales"))
    shape = _pool_shape(k_pages, v_pages)
    p, h, ps, _ = shape
    if kv_scales.shape != (p, h, 2, ps):
        raise ValueError(f"kv_scales must be [{p}, {h}, 2, {ps}], got {tuple(kv_scales.shape)}")
    return dev, shape


def _append_rope(what, fn, k_new, v_new, positions, slot_mapping, cos_sin, k_pages, v_pages, kv_scales, workspace, q,
                 q_out, q_weight, k_weight, eps, stream, dev, shape):
    import torch

    i32, bf16 = torch.int32, torch.bfloat16
    num_pages, hkv, ps, d = shape
    if not _good(slot_mapping, i32, dev):
        _refuse(dev, (slot_mapping, i32, "slot_mapping"))
    n = slot_mapping.numel()
    k_stride = _token_rows(k_new, "k_new", dev, n, hkv, d)
    v_stride = _token_rows(v_new, "v_new", dev, n, hkv, d)
    hq, q_stride, q_ptr, q_out_ptr = hkv, 0, None, None
    if q is not None:
        if q_out is None:
            raise ValueError("q and q_out come together")
        if not _good(q_out, bf16, dev):
            _refuse(dev, (q_out, bf16, "q_out"))
        out_shape = q_out.shape
        hq = out_shape[1] if len(out_shape) == 3 else 0
        q_stride = _token_rows(q, "q", dev, n, hq, d)
        if out_shape != (n, hq, d):
            raise ValueError("q_out must have q's shape")
        q_ptr, q_out_ptr = q.data_ptr(), q_out.data_ptr()
        if q_out_ptr == q_ptr and not q.is_contiguous():
            raise ValueError("q_out may be q itself only where q is contiguous")
    elif q_out is not None or q_weight is not None:
        raise ValueError("q_out and q_weight come with q")
    max_pos, pos_ptr, table_ptr = 0, None, None
    if cos_sin is not None:
        if not (_good(cos_sin, torch.float32, dev) and _good(positions, i32, dev)):
            _refuse(dev, (cos_sin, torch.float32, "cos_sin"), (positions, i32, "positions"))
        table_shape = cos_sin.shape
        if len(table_shape) != 2 or table_shape[1] != d:
            raise ValueError("cos_sin must be [max_pos, head_dim]")
        if positions.numel() != n:
            raise ValueError("positions and slot_mapping differ in length")
        max_pos, pos_ptr, table_ptr = table_shape[0], positions.data_ptr(), cos_sin.data_ptr()
    for w, name in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if w is not None and not (_good(w, bf16, dev) and w.shape == (d,)):
            if w.shape != (d,):
                raise ValueError(f"{name} must be [{d}]")
            _refuse(dev, (w, bf16, name))
    ds = _lib.CacheDesc(hq, hkv, d, ps, num_pages)
    before = [q_ptr, q_stride, k_new.data_ptr(), k_stride, v_new.data_ptr(), v_stride, pos_ptr, slot_mapping.data_ptr(),
              n, table_ptr, max_pos, _ptr(q_weight), _ptr(k_weight), eps, q_out_ptr, k_pages.data_ptr(),
              v_pages.data_ptr()]
    if kv_scales is not None:
        before.append(kv_scales.data_ptr())
    before.append(ctypes.byref(ds))
    _run(what, dev, stream, fn, before, _ws(workspace, dev))


def append_rope(k_new, v_new, positions, slot_mapping, cos_sin, k_pages, v_pages,
                workspace: Optional[Workspace] = None, q=None, q_out=None, q_weight=None, k_weight=None,
                eps: float = 1e-6, stream=None):
    """append of new tokens with the rotary embedding on the way: k_new / v_new [n, Hkv, D] (tokens may lie apart, as
    in a fused projection's output) go to slots slot_mapping [n], keys rotated at positions [n] by cos_sin (from
    rope_cos_sin; None: no rotation, positions unused). With q [n, Hq, D] the query rows are rotated into q_out.
    q_weight / k_weight [D]: RMS norm of each head's row (with eps) before the rotation, as in Qwen3 decoders."""
    import torch

    bf16 = torch.bfloat16
    dev = _device_of(k_pages, bf16, "k_pages")
    if not (_good(k_pages, bf16, dev) and _good(v_pages, bf16, dev)):
        _refuse(dev, (k_pages, bf16, "k_pages"), (v_pages, bf16, "v_pages"))
    _append_rope("pkv_append_rope", _lib.load().pkv_append_rope, k_new, v_new, positions, slot_mapping, cos_sin, k_pages,
                 v_pages, None, workspace, q, q_out, q_weight, k_weight, eps, stream, dev,
                 _pool_shape(k_pages, v_pages))


def append_rope_fp8(k_new, v_new, positions, slot_mapping, cos_sin, k_pages, v_pages, kv_scales,
                    workspace: Optional[Workspace] = None, q=None, q_out=None, q_weight=None, k_weight=None,
                    eps: float = 1e-6, stream=None):
    """append_rope into the 8-bit cache: pools torch.float8_e4m3fn [P, Hkv, 16, D] and kv_scales torch.float8_e8m0fnu
    [P, Hkv, 2, 16] (a power of two per K row, then per V row). Rows are quantised from fp32 (format: include/pkv.h);
    with cos_sin None it is the plain append of the 8-bit cache."""
    dev, shape = _fp8_cache(k_pages, v_pages, kv_scales)
    _append_rope("pkv_append_rope_fp8", _lib.load().pkv_append_rope_fp8, k_new, v_new, positions, slot_mapping, cos_sin,
                 k_pages, v_pages, kv_scales, workspace, q, q_out, q_weight, k_weight, eps, stream, dev, shape)


def decode_attn_fp8(q, k_pages, v_pages, kv_scales, block_table, seq_lens, out, scale: float, workspace: Workspace,
                    stream=None, early_prefetch: bool = False):
    """decode_attn over the 8-bit cache (pools and kv_scales as for append_rope_fp8): out [B, Hq, D] from q [B, Hq, D].
    The workspace is decode_attn's (decode_workspace_bytes) and may serve both in turn.

    early_prefetch: the previous kernel on the stream writes neither the block table nor the lengths, and of the
    cache at most the rows at positions seq_lens - 1 (append_rope_fp8 of the step's tokens), so the other pages may
    be read while it finishes (PKV_DECODE_EARLY_PREFETCH)."""
    import torch

    dev, (num_pages, hkv, ps, d) = _fp8_cache(k_pages, v_pages, kv_scales)
    bf16, i32 = torch.bfloat16, torch.int32
    if not (_good(q, bf16, dev) and _good(out, bf16, dev) and _good(block_table, i32, dev)
            and _good(seq_lens, i32, dev)):
        _refuse(dev, (q, bf16, "q"), (out, bf16, "out"), (block_table, i32, "block_table"), (seq_lens, i32, "seq_lens"))
    qs, bs = q.shape, block_table.shape
    if len(qs) != 3 or qs[2] != d or out.shape != qs or len(bs) != 2 or bs[0] != qs[0] or seq_lens.numel() != qs[0]:
        raise ValueError("shape mismatch")
    ds = _lib.CacheDesc(qs[1], hkv, d, ps, num_pages)
    ws, nbytes = _ws(workspace, dev)
    _run("pkv_decode_attn_fp8", dev, stream, _lib.load().pkv_decode_attn_fp8,
         (q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), kv_scales.data_ptr(), block_table.data_ptr(),
          seq_lens.data_ptr(), out.data_ptr(), scale),
         (ctypes.byref(ds), qs[0], bs[1], ws, nbytes, EARLY_PREFETCH if early_prefetch else 0))


def expand_fp8(k_pages, v_pages, kv_scales, block_table, seq_lens, k_out, v_out, out_block_table,
               workspace: Optional[Workspace] = None, stream=None):
    """Rows before seq_lens [S] of the 8-bit pages block_table [S, max_pages] as bf16, exactly, into pages
    out_block_table [S, max_pages] of k_out / v_out [P', Hkv, 16, D] (what prefill_chunk_attn then reads)."""
    import torch

    dev, shape = _fp8_cache(k_pages, v_pages, kv_scales)
    bf16, i32 = torch.bfloat16, torch.int32
    if not (_good(k_out, bf16, dev) and _good(v_out, bf16, dev) and _good(block_table, i32, dev)
            and _good(out_block_table, i32, dev) and _good(seq_lens, i32, dev)):
        _refuse(dev, (k_out, bf16, "k_out"), (v_out, bf16, "v_out"), (block_table, i32, "block_table"),
                (out_block_table, i32, "out_block_table"), (seq_lens, i32, "seq_lens"))
    out_shape, bs = k_out.shape, block_table.shape
    if len(out_shape) != 4 or out_shape[1:] != shape[1:] or v_out.shape != out_shape:
        raise ValueError("k_out and v_out are [pages, num_kv_heads, page_size, head_dim] of the cache's geometry")
    if len(bs) != 2 or out_block_table.shape != bs or seq_lens.numel() != bs[0]:
        raise ValueError("shape mismatch")
    num_pages, hkv, ps, d = shape
    ds = _lib.CacheDesc(hkv, hkv, d, ps, num_pages)
    _run("pkv_expand_fp8", dev, stream, _lib.load().pkv_expand_fp8,
         (k_pages.data_ptr(), v_pages.data_ptr(), kv_scales.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(),
          bs[0], bs[1], k_out.data_ptr(), v_out.data_ptr(), out_block_table.data_ptr(), out_shape[0],
          ctypes.byref(ds)), _ws(workspace, dev))


def prefill_chunk_attn(q, k_pages, v_pages, block_table, prefix_lens, cu_q_lens, out, scale: float, max_q_len: int,
                       workspace: Workspace, stream=None):
    """Causal chunk attention: out [total_q, Hq, D] for chunks packed by cu_q_lens (Hq / Hkv from 1 to 8,
    D 64 or 128)."""
    import torch

    _need(k_pages, torch.bfloat16, "k_pages")
    dev = k_pages.device
    _need(v_pages, torch.bfloat16, "v_pages", dev)
    _need(q, torch.bfloat16, "q", dev)
    _need(out, torch.bfloat16, "out", dev)
    _need(block_table, torch.int32, "block_table", dev)
    _need(prefix_lens, torch.int32, "prefix_lens", dev)
    _need(cu_q_lens, torch.int32, "cu_q_lens", dev)
    S = prefix_lens.numel()
    if cu_q_lens.numel() != S + 1 or block_table.shape[0] != S or out.shape != q.shape:
        raise ValueError("shape mismatch")
    d = _desc_of(k_pages, q.shape[1])
    ws = workspace.tensor
    rc = _lib.load().pkv_prefill_chunk_attn(_ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(block_table),
                                            _ptr(prefix_lens), _ptr(cu_q_lens), S, q.shape[0], _ptr(out),
                                            float(scale), _stream(stream), ctypes.byref(d), block_table.shape[1],
                                            int(max_q_len), _ptr(ws), ws.numel())
    _check(rc, "pkv_prefill_chunk_attn")


def mixed_workspace_bytes(num_seqs: int, max_q_len: int, dec_batch: int, dec_max_pages: int,
                          num_pages: int = 1) -> int:
    """Workspace bytes of a mixed-step call (16/8/128)."""
    d = desc(num_pages)
    return int(_lib.load().pkv_mixed_workspace_bytes(ctypes.byref(d), int(num_seqs), int(max_q_len), int(dec_batch),
                                                     int(dec_max_pages)))


def mixed_step_attn(q, k_pages, v_pages, block_table, prefix_lens, cu_q_lens, out, max_q_len: int, dec_q,
                    dec_block_table, dec_seq_lens, dec_out, scale: float, workspace: Workspace, stream=None):
    """One scheduler step of chunked prefill interleaved with decode, in one launch (16/8/128): out as
    prefill_chunk_attn gives it for the chunks (q, block_table, prefix_lens, cu_q_lens; may be empty) and
    dec_out as decode_attn gives it for the decode requests (dec_q, dec_block_table, dec_seq_lens), over
    the same pools. The workspace is sized by mixed_workspace_bytes."""
    import torch

    _need(k_pages, torch.bfloat16, "k_pages")
    dev = k_pages.device
    _need(v_pages, torch.bfloat16, "v_pages", dev)
    _need(dec_q, torch.bfloat16, "dec_q", dev)
    _need(dec_out, torch.bfloat16, "dec_out", dev)
    _need(dec_block_table, torch.int32, "dec_block_table", dev)
    _need(dec_seq_lens, torch.int32, "dec_seq_lens", dev)
    B = dec_q.shape[0]
    if dec_out.shape != dec_q.shape or dec_block_table.dim() != 2 or dec_block_table.shape[0] != B \
            or dec_seq_lens.numel() != B:
        raise ValueError("shape mismatch (decode part)")
    S = 0 if prefix_lens is None else prefix_lens.numel()
    if S:
        _need(q, torch.bfloat16, "q", dev)
        _need(out, torch.bfloat16, "out", dev)
        _need(block_table, torch.int32, "block_table", dev)
        _need(prefix_lens, torch.int32, "prefix_lens", dev)
        _need(cu_q_lens, torch.int32, "cu_q_lens", dev)
        if cu_q_lens.numel() != S + 1 or block_table.shape[0] != S or out.shape != q.shape:
            raise ValueError("shape mismatch (chunk part)")
    d = _desc_of(k_pages, dec_q.shape[1])
    ws = workspace.tensor
    rc = _lib.load().pkv_mixed_step_attn(
        _ptr(q) if S else None, _ptr(k_pages), _ptr(v_pages), _ptr(block_table) if S else None,
        _ptr(prefix_lens) if S else None, _ptr(cu_q_lens) if S else None, S, q.shape[0] if S else 0,
        _ptr(out) if S else None, block_table.shape[1] if S else 1, int(max_q_len) if S else 0, _ptr(dec_q),
        _ptr(dec_block_table), _ptr(dec_seq_lens), _ptr(dec_out), B, dec_block_table.shape[1], float(scale),
        _stream(stream), ctypes.byref(d), _ptr(ws), ws.numel())
    _check(rc, "pkv_mixed_step_attn")


def decode_attn_noalloc(q, k_pages, v_pages, block_table, seq_lens, out, scale: float, stream=None):
    """decode_attn without a workspace, for callers that may not allocate device memory.

    The split-KV scratch is a fixed 2 MiB array inside the library (batch <= 256).
    Calls share that array: run them in order on one stream, never overlapping on
    the GPU. Make the first call on a device before any CUDA-graph capture.
    """
    import torch

    _need(k_pages, torch.bfloat16, "k_pages")
    dev = k_pages.device
    _need(v_pages, torch.bfloat16, "v_pages", dev)
    _need(q, torch.bfloat16, "q", dev)
    _need(out, torch.bfloat16, "out", dev)
    _need(block_table, torch.int32, "block_table", dev)
    _need(seq_lens, torch.int32, "seq_lens", dev)
    B = q.shape[0]
    if out.shape != q.shape or block_table.dim() != 2 or block_table.shape[0] != B or seq_lens.numel() != B:
        raise ValueError("shape mismatch")
    d = _desc_of(k_pages, q.shape[1])
    rc = _lib.load().pkv_decode_attn_noalloc(_ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(block_table),
                                             _ptr(seq_lens), _ptr(out), float(scale), _stream(stream),
                                             ctypes.byref(d), B, block_table.shape[1])
    _check(rc, "pkv_decode_attn_noalloc")
