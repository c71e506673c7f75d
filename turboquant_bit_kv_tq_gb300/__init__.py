"""Python binding of libtq_gb300.so, the C ABI declared in include/tq_kv.h.

Argument marshalling only: every step of the store and decode path runs in the
library's CUDA kernels.  Device buffers are torch tensors owned by the caller
(or by :class:`TQCache`, a convenience owner); PyTorch provides memory and
streams, nothing else.  The library must have been built
(``python -m turboquant_bit_kv_tq_gb300._build`` or ``__graft_entry__.build()``);
importing the functions works without it, calling them raises.
"""

import ctypes
import os

import numpy as np

__all__ = [
    "TQError", "tq_cache_config", "TQ_DTYPE_F32", "TQ_DTYPE_BF16", "TQ_OUT_ROTATED", "TQ_V_MSE", "TQ_V_G32",
    "TQ_CODEBOOK_LLOYD", "TQ_CODEBOOK_UNIFORM", "tq_make_uniform_codebook",
    "TQ_DEVERR_SLOT", "TQ_DEVERR_BLOCK", "TQ_DEVERR_SEQLEN", "TQ_DEVERR_TAIL", "TQ_DEVERR_TIMEOUT", "EXPORTED",
    "library_path", "load_library", "tq_status_string", "tq_last_cuda_error", "tq_make_codebook",
    "tq_make_rotation_signs",
    "tq_make_qjl_matrix", "tq_cache_sizes", "tq_cache_create", "tq_cache_destroy", "tq_cache_export_params",
    "tq_store", "tq_decode_attention", "tq_decode_attention_noalloc", "tq_set_profile_events",
    "tq_get_device_error", "tq_set_store_small_max", "tq_extend_attention", "TQ_DEVERR_CHUNK", "TQCache",
    "TQ_PROF_STORE", "TQ_PROF_DECODE_SPLIT", "tq_check_wait_timeout", "tq_store_decode_attention",
    "TQ_DTYPE_F16", "tq_f8_config", "tq_f8_cache_sizes", "tq_f8_cache_create", "tq_f8_cache_destroy", "tq_f8_store",
    "tq_f8_load", "tq_f8_decode_attention", "tq_f8_get_device_error", "TQF8Cache",
    "tq_prompt_config", "tq_prompt_sizes", "tq_prompt_create", "tq_prompt_destroy", "tq_prompt_attention",
    "tq_prompt_get_device_error", "TQPrompt",
]

TQ_DTYPE_F32, TQ_DTYPE_BF16, TQ_DTYPE_F16 = 0, 1, 2
TQ_OUT_ROTATED = 0x100
TQ_V_MSE, TQ_V_G32 = 0, 1
TQ_CODEBOOK_LLOYD, TQ_CODEBOOK_UNIFORM = 0, 1
TQ_DEVERR_SLOT, TQ_DEVERR_BLOCK, TQ_DEVERR_SEQLEN, TQ_DEVERR_TAIL = 1, 2, 4, 8
TQ_DEVERR_TIMEOUT, TQ_DEVERR_CHUNK = 16, 32

# every function include/tq_kv.h declares
EXPORTED = [
    "tq_status_string", "tq_make_codebook", "tq_make_rotation_signs", "tq_make_qjl_matrix", "tq_cache_sizes",
    "tq_cache_create", "tq_cache_destroy", "tq_cache_export_params", "tq_store", "tq_decode_attention",
    "tq_set_profile_events", "tq_get_device_error", "tq_decode_attention_noalloc", "tq_last_cuda_error",
    "tq_set_store_small_max", "tq_make_uniform_codebook", "tq_extend_attention", "tq_check_wait_timeout",
    "tq_store_decode_attention",
    "tq_f8_cache_sizes", "tq_f8_cache_create", "tq_f8_cache_destroy", "tq_f8_store", "tq_f8_load",
    "tq_f8_decode_attention", "tq_f8_get_device_error",
    "tq_prompt_sizes", "tq_prompt_create", "tq_prompt_destroy", "tq_prompt_attention", "tq_prompt_get_device_error",
]
TQ_PROF_STORE, TQ_PROF_DECODE_SPLIT = 0, 1


class TQError(RuntimeError):
    def __init__(self, status, what):
        self.status = status
        msg = f"{what}: {tq_status_string(status)} ({status})"
        if status == -4:
            msg += f" [{tq_last_cuda_error()}]"
        super().__init__(msg)


class tq_cache_config(ctypes.Structure):
    _fields_ = [
        ("head_dim", ctypes.c_int32),
        ("num_kv_heads", ctypes.c_int32),
        ("num_q_heads", ctypes.c_int32),
        ("block_size", ctypes.c_int32),
        ("num_blocks", ctypes.c_int64),
        ("k_bits", ctypes.c_int32),
        ("k_qjl", ctypes.c_int32),
        ("v_mode", ctypes.c_int32),
        ("v_bits", ctypes.c_int32),
        ("seed_rot", ctypes.c_uint64),
        ("seed_qjl", ctypes.c_uint64),
        ("max_batch", ctypes.c_int32),
        ("max_blocks_per_seq", ctypes.c_int32),
        ("split_blocks", ctypes.c_int32),
        ("tail_cap", ctypes.c_int32),
        ("k_codebook", ctypes.c_int32),
        ("v_codebook", ctypes.c_int32),
    ]

    def __init__(self, **kw):
        defaults = dict(block_size=16, k_qjl=1, seed_rot=2, seed_qjl=1, max_batch=1, split_blocks=32, tail_cap=0)
        defaults.update(kw)
        super().__init__(**defaults)


class tq_f8_config(ctypes.Structure):
    _fields_ = [
        ("head_dim", ctypes.c_int32),
        ("num_kv_heads", ctypes.c_int32),
        ("num_q_heads", ctypes.c_int32),
        ("block_size", ctypes.c_int32),
        ("num_blocks", ctypes.c_int64),
        ("max_batch", ctypes.c_int32),
        ("max_blocks_per_seq", ctypes.c_int32),
    ]

    def __init__(self, **kw):
        super().__init__(**{**dict(block_size=16, max_batch=1), **kw})


class tq_prompt_config(ctypes.Structure):
    _fields_ = [
        ("head_dim", ctypes.c_int32),
        ("num_kv_heads", ctypes.c_int32),
        ("num_q_heads", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("max_batch", ctypes.c_int32),
        ("max_tokens", ctypes.c_int32),
    ]

    def __init__(self, **kw):
        super().__init__(**{**dict(dtype=TQ_DTYPE_BF16, max_batch=1), **kw})


_LIB = None
_P = ctypes.c_void_p


def library_path():
    return os.path.join(os.path.dirname(os.path.abspath(__file__)), "libtq_gb300.so")


def load_library():
    """Load libtq_gb300.so (raises if it has not been built)."""
    global _LIB
    if _LIB is None:
        path = library_path()
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it first (python -m turboquant_bit_kv_tq_gb300._build)")
        lib = ctypes.CDLL(path)
        i32, i64, u64 = ctypes.c_int, ctypes.c_int64, ctypes.c_uint64
        dp = ctypes.POINTER(ctypes.c_double)
        cfgp = ctypes.POINTER(tq_cache_config)
        sz = ctypes.POINTER(ctypes.c_size_t)
        sig = {
            "tq_status_string": (ctypes.c_char_p, [i32]),
            "tq_last_cuda_error": (ctypes.c_char_p, []),
            "tq_make_codebook": (i32, [i32, i32, dp, dp, dp]),
            "tq_make_uniform_codebook": (i32, [i32, i32, dp, dp, dp]),
            "tq_make_rotation_signs": (i32, [i32, u64, ctypes.POINTER(ctypes.c_float)]),
            "tq_make_qjl_matrix": (i32, [i32, u64, ctypes.POINTER(ctypes.c_uint16)]),
            "tq_cache_sizes": (i32, [cfgp, sz, sz, sz, sz]),
            "tq_cache_create": (i32, [cfgp, _P, _P, _P, ctypes.POINTER(_P)]),
            "tq_cache_destroy": (i32, [_P]),
            "tq_cache_export_params": (i32, [_P, _P, _P, _P, _P, _P, _P]),
            "tq_store": (i32, [_P, _P, _P, i32, i64, _P, _P, _P]),
            "tq_decode_attention": (i32, [_P, _P, i32, _P, _P, _P, _P, _P, _P, ctypes.c_float, i32, _P, i32, _P]),
            "tq_set_profile_events": (i32, [_P, i32, _P, _P]),
            "tq_extend_attention": (i32, [_P, _P, i32, _P, _P, _P, _P, _P, _P, ctypes.c_float, i32, i32, _P, i32, _P]),
            "tq_decode_attention_noalloc": (
                i32, [_P, _P, i32, _P, _P, _P, _P, _P, _P, ctypes.c_float, i32, _P, i32, _P]),
            "tq_get_device_error": (i32, [_P, ctypes.POINTER(ctypes.c_uint32), _P]),
            "tq_set_store_small_max": (i32, [i64]),
            "tq_check_wait_timeout": (i32, [_P, ctypes.c_uint32, _P]),
            "tq_store_decode_attention": (
                i32, [_P, _P, _P, i32, i64, _P, _P, i32, _P, _P, _P, _P, _P, _P, ctypes.c_float, i32, _P, i32, _P]),
        }
        f8p = ctypes.POINTER(tq_f8_config)
        sig.update({
            "tq_f8_cache_sizes": (i32, [f8p, sz, sz, sz]),
            "tq_f8_cache_create": (i32, [f8p, _P, _P, ctypes.POINTER(_P)]),
            "tq_f8_cache_destroy": (i32, [_P]),
            "tq_f8_store": (i32, [_P, _P, _P, i32, i64, i64, i64, _P, _P, _P]),
            "tq_f8_load": (i32, [_P, _P, _P, _P, _P, i32, i64, _P, _P, i32, _P]),
            "tq_f8_decode_attention": (
                i32, [_P, _P, i32, i64, _P, _P, _P, ctypes.c_float, i32, _P, i32, _P]),
            "tq_f8_get_device_error": (i32, [_P, ctypes.POINTER(ctypes.c_uint32), _P]),
        })
        pcp = ctypes.POINTER(tq_prompt_config)
        sig.update({
            "tq_prompt_sizes": (i32, [pcp, sz]),
            "tq_prompt_create": (i32, [pcp, _P, _P, ctypes.POINTER(_P)]),
            "tq_prompt_destroy": (i32, [_P]),
            "tq_prompt_attention": (
                i32, [_P, _P, _P, _P, i64, i64, i64, _P, _P, i32, i32, i32, ctypes.c_float, i32, _P, _P, _P]),
            "tq_prompt_get_device_error": (i32, [_P, ctypes.POINTER(ctypes.c_uint32), _P]),
        })
        for name, (res, args) in sig.items():
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = res, args
        _LIB = lib
    return _LIB


def _check(status, what):
    if status != 0:
        raise TQError(status, what)


def tq_status_string(status):
    return load_library().tq_status_string(status).decode()


def tq_last_cuda_error():
    """The CUDA runtime message behind the last TQ_ERR_CUDA on this thread."""
    return load_library().tq_last_cuda_error().decode()


def tq_set_store_small_max(max_vectors):
    """Largest store (in token x KV-head vectors) encoded one vector per CTA;
    negative restores the default (16 x the SM count)."""
    _check(load_library().tq_set_store_small_max(int(max_vectors)), "tq_set_store_small_max")


def _dptr(a):
    return a.ctypes.data_as(ctypes.POINTER(ctypes.c_double))


def tq_make_codebook(d, bits):
    """(centroids [2^bits], boundaries [2^bits-1], per-vector mse) as float64."""
    c = np.zeros(2**bits)
    b = np.zeros(2**bits - 1)
    mse = ctypes.c_double()
    _check(load_library().tq_make_codebook(d, bits, _dptr(c), _dptr(b), ctypes.byref(mse)), "tq_make_codebook")
    return c, b, mse.value


def tq_make_uniform_codebook(d, bits):
    """Uniform-grid (centroids, boundaries, per-vector mse) as float64."""
    c = np.zeros(2**bits)
    b = np.zeros(2**bits - 1)
    mse = ctypes.c_double()
    _check(load_library().tq_make_uniform_codebook(d, bits, _dptr(c), _dptr(b), ctypes.byref(mse)),
           "tq_make_uniform_codebook")
    return c, b, mse.value


def tq_make_rotation_signs(d, seed):
    out = np.zeros(d, np.float32)
    _check(load_library().tq_make_rotation_signs(d, seed, out.ctypes.data_as(ctypes.POINTER(ctypes.c_float))),
           "tq_make_rotation_signs")
    return out


def tq_make_qjl_matrix(d, seed):
    """S as bfloat16 bit patterns, uint16 [d, d] (row j = output j)."""
    out = np.zeros((d, d), np.uint16)
    _check(load_library().tq_make_qjl_matrix(d, seed, out.ctypes.data_as(ctypes.POINTER(ctypes.c_uint16))),
           "tq_make_qjl_matrix")
    return out


def tq_cache_sizes(cfg):
    vals = [ctypes.c_size_t() for _ in range(4)]
    _check(load_library().tq_cache_sizes(ctypes.byref(cfg), *[ctypes.byref(v) for v in vals]), "tq_cache_sizes")
    return dict(zip(["page_bytes", "cache_bytes", "params_bytes", "workspace_bytes"], [v.value for v in vals]))


def _stream_ptr(stream):
    import torch

    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def tq_cache_create(cfg, params, workspace, stream=None):
    h = _P()
    _check(load_library().tq_cache_create(ctypes.byref(cfg), _P(params.data_ptr()), _P(workspace.data_ptr()),
                                          _stream_ptr(stream), ctypes.byref(h)), "tq_cache_create")
    return h


def tq_cache_destroy(handle):
    _check(load_library().tq_cache_destroy(handle), "tq_cache_destroy")


def tq_cache_export_params(handle, cfg):
    d = cfg.head_dim
    out = dict(signs=np.zeros(d, np.float32), qjl_bf16=np.zeros((d, d), np.uint16),
               k_centroids=np.zeros(2**cfg.k_bits), k_boundaries=np.zeros(2**cfg.k_bits - 1))
    if cfg.v_mode == TQ_V_MSE:
        out.update(v_centroids=np.zeros(2**cfg.v_bits), v_boundaries=np.zeros(2**cfg.v_bits - 1))
    p = lambda k: _P(out[k].ctypes.data) if k in out else _P()  # noqa: E731
    _check(load_library().tq_cache_export_params(handle, p("signs"), p("qjl_bf16"), p("k_centroids"),
                                                 p("k_boundaries"), p("v_centroids"), p("v_boundaries")),
           "tq_cache_export_params")
    return out


def _dtype_code(t):
    import torch

    if t.dtype == torch.float32:
        return TQ_DTYPE_F32
    if t.dtype == torch.bfloat16:
        return TQ_DTYPE_BF16
    raise TypeError(f"unsupported dtype {t.dtype}: float32 or bfloat16")


def _dev(t, name, dtype=None):
    if t is None:
        return _P()
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return _P(t.data_ptr())


def tq_store(handle, k, v, slot_mapping, cache, stream=None):
    """k, v [T, H_kv, d] (f32 or bf16, same dtype); slot_mapping int64 [T]."""
    import torch

    if k.dtype != v.dtype or k.shape != v.shape:
        raise ValueError("k and v must have the same shape and dtype")
    _check(load_library().tq_store(handle, _dev(k, "k"), _dev(v, "v"), _dtype_code(k), k.shape[0],
                                   _dev(slot_mapping, "slot_mapping", torch.int64), _dev(cache, "cache"),
                                   _stream_ptr(stream)), "tq_store")


def tq_decode_attention(handle, q, cache, block_table, seq_lens, out, tail_k=None, tail_v=None, tail_lens=None,
                        scale=0.0, stream=None, rotated=False):
    """q [B, H_q, d] (f32/bf16); block_table int32 [B, max_blocks_per_seq];
    seq_lens int32 [B]; out [B, H_q, d] (f32/bf16); optional bf16 tail;
    rotated: MSE values only, out in the rotated space (R out)."""
    import torch

    if tail_k is not None:
        _dev(tail_k, "tail_k", torch.bfloat16)
        _dev(tail_v, "tail_v", torch.bfloat16)
    _check(load_library().tq_decode_attention(
        handle, _dev(q, "q"), _dtype_code(q), _dev(cache, "cache"), _dev(block_table, "block_table", torch.int32),
        _dev(seq_lens, "seq_lens", torch.int32), _dev(tail_k, "tail_k"), _dev(tail_v, "tail_v"),
        _dev(tail_lens, "tail_lens", torch.int32), float(scale), q.shape[0], _dev(out, "out"),
        _dtype_code(out) | (TQ_OUT_ROTATED if rotated else 0), _stream_ptr(stream)), "tq_decode_attention")


def tq_store_decode_attention(handle, k, v, slot_mapping, q, cache, block_table, seq_lens, out, tail_k=None,
                              tail_v=None, tail_lens=None, scale=0.0, stream=None, rotated=False):
    """tq_store(k, v, slot_mapping) then tq_decode_attention(q, ...) in one
    call; k and v may have zero tokens (nothing is stored)."""
    import torch

    if k.dtype != v.dtype or k.shape != v.shape:
        raise ValueError("k and v must have the same shape and dtype")
    if tail_k is not None:
        _dev(tail_k, "tail_k", torch.bfloat16)
        _dev(tail_v, "tail_v", torch.bfloat16)
    _check(load_library().tq_store_decode_attention(
        handle, _dev(k, "k"), _dev(v, "v"), _dtype_code(k), k.shape[0],
        _dev(slot_mapping, "slot_mapping", torch.int64), _dev(q, "q"), _dtype_code(q), _dev(cache, "cache"),
        _dev(block_table, "block_table", torch.int32), _dev(seq_lens, "seq_lens", torch.int32),
        _dev(tail_k, "tail_k"), _dev(tail_v, "tail_v"), _dev(tail_lens, "tail_lens", torch.int32), float(scale),
        q.shape[0], _dev(out, "out"), _dtype_code(out) | (TQ_OUT_ROTATED if rotated else 0), _stream_ptr(stream)),
        "tq_store_decode_attention")


def tq_decode_attention_noalloc(handle, q, cache, block_table, seq_lens, out, tail_k=None, tail_v=None,
                                tail_lens=None, scale=0.0, stream=None):
    """tq_decode_attention with its scratch in the library's static device
    array instead of the handle's workspace (allocates nothing)."""
    import torch

    if tail_k is not None:
        _dev(tail_k, "tail_k", torch.bfloat16)
        _dev(tail_v, "tail_v", torch.bfloat16)
    _check(load_library().tq_decode_attention_noalloc(
        handle, _dev(q, "q"), _dtype_code(q), _dev(cache, "cache"), _dev(block_table, "block_table", torch.int32),
        _dev(seq_lens, "seq_lens", torch.int32), _dev(tail_k, "tail_k"), _dev(tail_v, "tail_v"),
        _dev(tail_lens, "tail_lens", torch.int32), float(scale), q.shape[0], _dev(out, "out"), _dtype_code(out),
        _stream_ptr(stream)), "tq_decode_attention_noalloc")


def tq_extend_attention(handle, q, cache, block_table, prefix_lens, cu_q, new_k, new_v, out, scale=0.0, stream=None,
                        rotated=False):
    """q [T, H_q, d] (f32/bf16); block_table int32 [B, max_blocks_per_seq];
    prefix_lens int32 [B]; cu_q int32 [B+1]; new_k, new_v bf16 [T, H_kv, d];
    out [T, H_q, d] (f32/bf16)."""
    import torch

    T = q.shape[0]
    if new_k.shape != new_v.shape or new_k.shape[0] != T or out.shape != q.shape:
        raise ValueError("q, new_k, new_v and out must share the token count (out shaped like q)")
    if cu_q.shape[0] != prefix_lens.shape[0] + 1 or block_table.shape[0] < prefix_lens.shape[0]:
        raise ValueError("cu_q must have batch+1 entries and block_table at least batch rows")
    _check(load_library().tq_extend_attention(
        handle, _dev(q, "q"), _dtype_code(q), _dev(cache, "cache"), _dev(block_table, "block_table", torch.int32),
        _dev(prefix_lens, "prefix_lens", torch.int32), _dev(cu_q, "cu_q", torch.int32),
        _dev(new_k, "new_k", torch.bfloat16), _dev(new_v, "new_v", torch.bfloat16), float(scale),
        prefix_lens.shape[0], q.shape[0], _dev(out, "out"), _dtype_code(out) | (TQ_OUT_ROTATED if rotated else 0),
        _stream_ptr(stream)), "tq_extend_attention")


def tq_set_profile_events(handle, kernel, start=None, stop=None):
    """Record torch.cuda.Event pairs around the store (kernel=0) or decode
    split-KV (kernel=1) launch of later calls; None switches it off."""
    ev = lambda e: _P(e.cuda_event) if e is not None else _P()  # noqa: E731
    _check(load_library().tq_set_profile_events(handle, kernel, ev(start), ev(stop)), "tq_set_profile_events")


def tq_check_wait_timeout(err_word, limit_us, stream=None):
    """Make the decode kernels' bounded mbarrier wait run out (nothing ever
    completes the phase) with a limit of limit_us microseconds; the kernel ORs
    TQ_DEVERR_TIMEOUT into err_word (a CUDA uint32/int32 tensor of one
    element) and returns."""
    if err_word.numel() < 1 or err_word.element_size() != 4:
        raise ValueError("err_word must hold one 4-byte element")
    _check(load_library().tq_check_wait_timeout(_dev(err_word, "err_word"), int(limit_us), _stream_ptr(stream)),
           "tq_check_wait_timeout")


def tq_get_device_error(handle, stream=None):
    flags = ctypes.c_uint32()
    _check(load_library().tq_get_device_error(handle, ctypes.byref(flags), _stream_ptr(stream)),
           "tq_get_device_error")
    return flags.value


class TQCache:
    """Owns the device buffers of one cache configuration (torch uint8 tensors)
    and the library handle."""

    def __init__(self, device="cuda", **cfg_kwargs):
        import torch

        self.cfg = tq_cache_config(**cfg_kwargs)
        self.sizes = tq_cache_sizes(self.cfg)
        self.device = torch.device(device)
        self.params = torch.empty(self.sizes["params_bytes"], dtype=torch.uint8, device=self.device)
        self.workspace = torch.empty(self.sizes["workspace_bytes"], dtype=torch.uint8, device=self.device)
        self.cache = torch.zeros(self.sizes["cache_bytes"], dtype=torch.uint8, device=self.device)
        self.handle = tq_cache_create(self.cfg, self.params, self.workspace)

    @property
    def page_bytes(self):
        return self.sizes["page_bytes"]

    def pages(self):
        """The cache as [num_blocks, H_kv, page_bytes]."""
        return self.cache.view(self.cfg.num_blocks, self.cfg.num_kv_heads, self.page_bytes)

    def store(self, k, v, slot_mapping, stream=None):
        tq_store(self.handle, k, v, slot_mapping, self.cache, stream)

    def decode(self, q, block_table, seq_lens, out=None, tail_k=None, tail_v=None, tail_lens=None, scale=0.0,
               stream=None, out_dtype=None, rotated=False):
        import torch

        if out is None:
            out = torch.empty(q.shape, dtype=out_dtype or torch.float32, device=q.device)
        tq_decode_attention(self.handle, q, self.cache, block_table, seq_lens, out, tail_k, tail_v, tail_lens,
                            scale, stream, rotated)
        return out

    def store_decode(self, k, v, slot_mapping, q, block_table, seq_lens, out=None, tail_k=None, tail_v=None,
                     tail_lens=None, scale=0.0, stream=None, out_dtype=None, rotated=False):
        import torch

        if out is None:
            out = torch.empty(q.shape, dtype=out_dtype or torch.float32, device=q.device)
        tq_store_decode_attention(self.handle, k, v, slot_mapping, q, self.cache, block_table, seq_lens, out,
                                  tail_k, tail_v, tail_lens, scale, stream, rotated)
        return out

    def extend(self, q, block_table, prefix_lens, cu_q, new_k, new_v, out=None, scale=0.0, stream=None,
               out_dtype=None, rotated=False):
        import torch

        if out is None:
            out = torch.empty(q.shape, dtype=out_dtype or torch.float32, device=q.device)
        tq_extend_attention(self.handle, q, self.cache, block_table, prefix_lens, cu_q, new_k, new_v, out, scale,
                            stream, rotated)
        return out

    def device_error(self, stream=None):
        return tq_get_device_error(self.handle, stream)

    def export_params(self):
        return tq_cache_export_params(self.handle, self.cfg)

    def close(self):
        if self.handle:
            tq_cache_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ------------------------------------- 8-bit cache and prompt attention
# These calls run for a few microseconds on the GPU, so their checks are kept
# short: every tensor is asked for its device index, shape and strides once.
_TORCH = None
_DTYPE_CODES = None


def _torch():
    global _TORCH, _DTYPE_CODES
    if _TORCH is None:
        import torch

        _TORCH = torch
        _DTYPE_CODES = {torch.float32: TQ_DTYPE_F32, torch.bfloat16: TQ_DTYPE_BF16, torch.float16: TQ_DTYPE_F16}
    return _TORCH


def _code(t, name):
    _torch()
    code = _DTYPE_CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name}: unsupported dtype {t.dtype}: float32, bfloat16 or float16")
    return code


def _wrong_device(t, name, dev):
    if dev is None or dev < 0 or not t.is_cuda:
        return ValueError(f"{name} must be a CUDA tensor")
    return ValueError(f"{name} is on {t.device}, not on cuda:{dev}")


def _rows(t, name, heads, d, dev):
    """Pointer and row stride of a tensor [rows, heads, d] on device `dev` whose
    rows are contiguous (they may lie apart, as in a fused projection)."""
    if t.get_device() != dev or dev < 0:
        raise _wrong_device(t, name, dev)
    shape = t.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != d:
        raise ValueError(f"{name} must be [rows, {heads}, {d}], got {tuple(shape)}")
    if shape[0] == 0:
        return t.data_ptr(), heads * d
    row, head, el = t.stride()
    if el != 1 or (head != d and heads > 1):
        raise ValueError(f"{name}: the [{heads}, {d}] part of a row must be contiguous")
    if shape[0] == 1:
        row = heads * d  # the stride of a single row says nothing
    elif row < heads * d:
        raise ValueError(f"{name}: rows overlap (row stride {row})")
    return t.data_ptr(), row


def _plain(t, name, shape, dtype, dev):
    """Pointer of a contiguous tensor of exactly this shape."""
    if t.get_device() != dev or dev < 0:
        raise _wrong_device(t, name, dev)
    if tuple(t.shape) != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous {list(shape)}, got {list(t.shape)}, strides {t.stride()}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def _index(t, name, dtype, least, dev):
    """Pointer of a contiguous index tensor of at least this many entries."""
    if t.get_device() != dev or dev < 0:
        raise _wrong_device(t, name, dev)
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.numel() < least or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous with at least {least} entries, got {list(t.shape)}")
    return t.data_ptr()


def _pages(cache, cfg):
    """Pointer of an 8-bit cache's pages."""
    need = cfg.num_blocks * cfg.num_kv_heads * (32 * cfg.head_dim + 32)
    if cache is None or not cache.is_cuda or not cache.is_contiguous() or cache.nbytes < need:
        raise ValueError(f"cache must be a contiguous CUDA tensor of at least {need} bytes")
    return cache.data_ptr()


def _table(t, batch, columns, dev):
    if t.dim() != 2 or t.shape[0] < batch or t.shape[1] != columns:
        raise ValueError(f"block_table must be [>= {batch}, {columns}], got {list(t.shape)}")
    return _index(t, "block_table", _TORCH.int32, 0, dev)


def _launch_stream(stream, dev):
    """The stream to launch on.  Calls launch on the current device, which must be the tensors'."""
    cuda = _TORCH._C
    if cuda._cuda_getDevice() != dev:
        raise ValueError(f"the current device is cuda:{cuda._cuda_getDevice()}, the tensors are on cuda:{dev}")
    if stream is None:
        return cuda._cuda_getCurrentRawStream(dev)
    if stream.device_index != dev:
        raise ValueError(f"the stream is on cuda:{stream.device_index}, the tensors on cuda:{dev}")
    return stream.cuda_stream


def _output(q, dtype, stream):
    """A tensor of q's shape for a call on `stream`, whose memory belongs to that
    stream: of another's, an earlier use might still be under way there."""
    if stream is None:
        return _TORCH.empty(q.shape, dtype=dtype, device=q.device)
    with _TORCH.cuda.stream(stream):
        return _TORCH.empty(q.shape, dtype=dtype, device=q.device)


def tq_f8_cache_sizes(cfg):
    vals = [ctypes.c_size_t() for _ in range(3)]
    _check(load_library().tq_f8_cache_sizes(ctypes.byref(cfg), *[ctypes.byref(v) for v in vals]), "tq_f8_cache_sizes")
    return dict(zip(["page_bytes", "cache_bytes", "workspace_bytes"], [v.value for v in vals]))


def tq_f8_cache_create(cfg, workspace, stream=None):
    h = _P()
    _check(load_library().tq_f8_cache_create(ctypes.byref(cfg), _P(workspace.data_ptr()), _stream_ptr(stream),
                                             ctypes.byref(h)), "tq_f8_cache_create")
    return h


def tq_f8_cache_destroy(handle):
    _check(load_library().tq_f8_cache_destroy(handle), "tq_f8_cache_destroy")


def tq_f8_store(handle, cfg, k, v, slot_mapping, cache, stream=None):
    """k, v [T, H_kv, d] (f32, bf16 or f16, same dtype; rows may lie apart);
    slot_mapping int64 [T]."""
    dt = _code(k, "k")
    if k.dtype != v.dtype or k.shape != v.shape:
        raise ValueError("k and v must have the same shape and dtype")
    dev = cache.get_device() if cache is not None else k.get_device()
    heads, d = cfg.num_kv_heads, cfg.head_dim
    kp, ks = _rows(k, "k", heads, d, dev)
    vp, vs = _rows(v, "v", heads, d, dev)
    n = k.shape[0]
    st = load_library().tq_f8_store(handle, kp, vp, dt, ks, vs, n,
                                    _index(slot_mapping, "slot_mapping", _TORCH.int64, n, dev), _pages(cache, cfg),
                                    _launch_stream(stream, dev))
    if st:
        raise TQError(st, "tq_f8_store")


def tq_f8_load(handle, cfg, cache, block_table, seq_lens, cu_out, k_out, v_out, stream=None):
    """block_table int32 [B, max_blocks_per_seq]; seq_lens int32 [B]; cu_out
    int32 [B] (or more): first row of each sequence in k_out, v_out [rows,
    H_kv, d] (f32, bf16 or f16)."""
    dt = _code(k_out, "k_out")
    if k_out.dtype != v_out.dtype or k_out.shape != v_out.shape:
        raise ValueError("k_out and v_out must have the same shape and dtype")
    dev = cache.get_device() if cache is not None else k_out.get_device()
    b, n, i32 = seq_lens.shape[0], k_out.shape[0], _TORCH.int32
    shape = (n, cfg.num_kv_heads, cfg.head_dim)
    st = load_library().tq_f8_load(
        handle, _pages(cache, cfg), _table(block_table, b, cfg.max_blocks_per_seq, dev),
        _index(seq_lens, "seq_lens", i32, b, dev), _index(cu_out, "cu_out", i32, b, dev), b, n,
        _plain(k_out, "k_out", shape, None, dev), _plain(v_out, "v_out", shape, None, dev), dt,
        _launch_stream(stream, dev))
    if st:
        raise TQError(st, "tq_f8_load")


def tq_f8_decode_attention(handle, cfg, q, cache, block_table, seq_lens, out, scale=0.0, stream=None):
    """q, out [B, H_q, d] (f32, bf16 or f16 each; q's rows may lie apart);
    block_table int32 [B, max_blocks_per_seq]; seq_lens int32 [B]."""
    qt, ot = _code(q, "q"), _code(out, "out")
    dev = cache.get_device() if cache is not None else q.get_device()
    heads, d = cfg.num_q_heads, cfg.head_dim
    qp, qs = _rows(q, "q", heads, d, dev)
    b = q.shape[0]
    st = load_library().tq_f8_decode_attention(
        handle, qp, qt, qs, _pages(cache, cfg), _table(block_table, b, cfg.max_blocks_per_seq, dev),
        _index(seq_lens, "seq_lens", _TORCH.int32, b, dev), scale, b, _plain(out, "out", (b, heads, d), None, dev), ot,
        _launch_stream(stream, dev))
    if st:
        raise TQError(st, "tq_f8_decode_attention")


def tq_f8_get_device_error(handle, stream=None):
    flags = ctypes.c_uint32()
    _check(load_library().tq_f8_get_device_error(handle, ctypes.byref(flags), _stream_ptr(stream)),
           "tq_f8_get_device_error")
    return flags.value


def _cuda_device(device):
    device = _torch().device(device)
    if device.type == "cuda" and device.index is None:
        device = _TORCH.device("cuda", _TORCH.cuda.current_device())
    return device


class TQF8Cache:
    """Owns (or adopts) the pages of an 8-bit cache, its workspace and the
    library handle.  ``cache``: an existing uint8 tensor of cache_bytes."""

    def __init__(self, device="cuda", cache=None, **cfg_kwargs):
        self.handle = None
        self.cfg = tq_f8_config(**cfg_kwargs)
        self.sizes = tq_f8_cache_sizes(self.cfg)
        self.device = _cuda_device(device)
        torch = _TORCH
        if cache is None:
            cache = torch.zeros(self.sizes["cache_bytes"], dtype=torch.uint8, device=self.device)
        elif (cache.dtype != torch.uint8 or cache.numel() != self.sizes["cache_bytes"] or not cache.is_contiguous()
              or cache.device != self.device):
            raise ValueError(f"cache must be {self.sizes['cache_bytes']} contiguous uint8 bytes on {self.device}")
        self.cache = cache
        self.workspace = torch.empty(self.sizes["workspace_bytes"], dtype=torch.uint8, device=self.device)
        with torch.cuda.device(self.device):
            self.handle = tq_f8_cache_create(self.cfg, self.workspace)

    @property
    def page_bytes(self):
        return self.sizes["page_bytes"]

    def pages(self):
        """The cache as [num_blocks, H_kv, page_bytes]."""
        return self.cache.view(self.cfg.num_blocks, self.cfg.num_kv_heads, self.page_bytes)

    def store(self, k, v, slot_mapping, stream=None):
        tq_f8_store(self.handle, self.cfg, k, v, slot_mapping, self.cache, stream)

    def load(self, block_table, seq_lens, cu_out, k_out, v_out, stream=None):
        tq_f8_load(self.handle, self.cfg, self.cache, block_table, seq_lens, cu_out, k_out, v_out, stream)
        return k_out, v_out

    def decode(self, q, block_table, seq_lens, out=None, scale=0.0, stream=None, out_dtype=None):
        if out is None:
            out = _output(q, out_dtype or q.dtype, stream)
        tq_f8_decode_attention(self.handle, self.cfg, q, self.cache, block_table, seq_lens, out, scale, stream)
        return out

    def device_error(self, stream=None):
        return tq_f8_get_device_error(self.handle, stream)

    def close(self):
        if self.handle:
            tq_f8_cache_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def tq_prompt_sizes(cfg):
    n = ctypes.c_size_t()
    _check(load_library().tq_prompt_sizes(ctypes.byref(cfg), ctypes.byref(n)), "tq_prompt_sizes")
    return dict(workspace_bytes=n.value)


def tq_prompt_create(cfg, workspace, stream=None):
    h = _P()
    _check(load_library().tq_prompt_create(ctypes.byref(cfg), _P(workspace.data_ptr()), _stream_ptr(stream),
                                           ctypes.byref(h)), "tq_prompt_create")
    return h


def tq_prompt_destroy(handle):
    _check(load_library().tq_prompt_destroy(handle), "tq_prompt_destroy")


def tq_prompt_attention(handle, cfg, q, k, v, cu_q, cu_k, out, lse=None, causal=True, scale=0.0, stream=None):
    """q, out [n_q, H_q, d], k, v [n_k, H_kv, d], all of the handle's dtype (the
    rows of q, k and v may lie apart); cu_q, cu_k int32 [B + 1]; lse f32
    [n_q, H_q] or None."""
    dt = _code(q, "q")
    if dt != cfg.dtype or k.dtype != q.dtype or v.dtype != q.dtype or out.dtype != q.dtype:
        raise TypeError(f"q, k, v and out must all have the handle's dtype (code {cfg.dtype})")
    if k.shape != v.shape:
        raise ValueError("k and v must have the same shape")
    dev = q.get_device()
    hq, hk, d, i32 = cfg.num_q_heads, cfg.num_kv_heads, cfg.head_dim, _TORCH.int32
    qp, qs = _rows(q, "q", hq, d, dev)
    kp, ks = _rows(k, "k", hk, d, dev)
    vp, vs = _rows(v, "v", hk, d, dev)
    n, b = q.shape[0], cu_q.shape[0] - 1
    if cu_k.shape[0] != b + 1:
        raise ValueError("cu_q and cu_k must both have batch + 1 entries")
    st = load_library().tq_prompt_attention(
        handle, qp, kp, vp, qs, ks, vs, _index(cu_q, "cu_q", i32, 2, dev), _index(cu_k, "cu_k", i32, 2, dev), b, n,
        k.shape[0], scale, 1 if causal else 0, _plain(out, "out", (n, hq, d), None, dev),
        None if lse is None else _plain(lse, "lse", (n, hq), _TORCH.float32, dev), _launch_stream(stream, dev))
    if st:
        raise TQError(st, "tq_prompt_attention")


def tq_prompt_get_device_error(handle, stream=None):
    flags = ctypes.c_uint32()
    _check(load_library().tq_prompt_get_device_error(handle, ctypes.byref(flags), _stream_ptr(stream)),
           "tq_prompt_get_device_error")
    return flags.value


class TQPrompt:
    """Owns the workspace and library handle of prompt attention for one head
    configuration, up to max_batch sequences and max_tokens query rows a call."""

    def __init__(self, device="cuda", dtype=None, **cfg_kwargs):
        self.handle = None
        torch = _torch()
        code = _DTYPE_CODES.get(dtype or torch.bfloat16)
        if code is None:
            raise TypeError(f"unsupported dtype {dtype}: bfloat16 or float16")
        self.cfg = tq_prompt_config(dtype=code, **cfg_kwargs)
        self.sizes = tq_prompt_sizes(self.cfg)
        self.device = _cuda_device(device)
        self.workspace = torch.empty(self.sizes["workspace_bytes"], dtype=torch.uint8, device=self.device)
        with torch.cuda.device(self.device):
            self.handle = tq_prompt_create(self.cfg, self.workspace)

    def attention(self, q, k, v, cu_q, cu_k, out=None, lse=None, causal=True, scale=0.0, stream=None):
        if q.get_device() != self.device.index:
            raise _wrong_device(q, "q", self.device.index)
        if out is None:
            out = _output(q, q.dtype, stream)
        tq_prompt_attention(self.handle, self.cfg, q, k, v, cu_q, cu_k, out, lse, causal, scale, stream)
        return out

    def device_error(self, stream=None):
        return tq_prompt_get_device_error(self.handle, stream)

    def close(self):
        if self.handle:
            tq_prompt_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
