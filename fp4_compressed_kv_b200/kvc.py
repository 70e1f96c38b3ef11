"""Thin Python binding of libkvc.so (include/kvc.h): argument marshalling only.

Every call hands raw device pointers of torch tensors and the current CUDA
stream to the C ABI; all work runs in the library's sm_100a kernels.  There
is no fallback: if ``libkvc.so`` is missing or no sm_100 device is current,
the calls raise.
"""
from __future__ import annotations

import ctypes as C
import os

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libkvc.so")

OK = 0
STATUS_NAMES = {0: "ok", 1: "invalid", 2: "capacity", 3: "cuda", 4: "unsupported", 5: "timeout",
                6: "device", 7: "workspace"}
SCALE_F32, SCALE_UE4M3 = 0, 1
FULL, REINDEX, REUSE = 0, 1, 2
F32, BF16 = 0, 1
NORM_NONE, NORM_LATENT, NORM_ROW = 0, 1, 2
ROPE_HALVES, ROPE_PAIRS = 0, 1
DEV_NONFINITE, DEV_BAD_INDEX, DEV_CAPACITY, DEV_TIMEOUT, DEV_BAD_LENGTH = 1, 2, 4, 8, 16


class KvcError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__(f"{fn}: {STATUS_NAMES.get(status, status)} ({_lib().kvc_status_string(status).decode()})")


class Config(C.Structure):
    _fields_ = [("latent_dim", C.c_int32), ("rope_dim", C.c_int32), ("group", C.c_int32),
                ("scale_fmt", C.c_int32), ("idx_dim", C.c_int32), ("topk", C.c_int32),
                ("window", C.c_int32), ("n_heads", C.c_int32), ("sm_scale", C.c_float),
                ("act_dtype", C.c_int32), ("ratio", C.c_int32), ("idx_fmt", C.c_int32)]


class CacheStruct(C.Structure):
    _fields_ = [("records", C.c_void_p), ("idx_k", C.c_void_p), ("n_entries", C.c_void_p),
                ("batch", C.c_int32), ("capacity", C.c_int32)]


_LIB = None


def _lib():
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libkvc.so not built ({LIB_PATH}); run "
                               "`python -m fp4_compressed_kv_b200.build`")
        lib = C.CDLL(LIB_PATH)
        P, I, Z = C.c_void_p, C.c_int, C.c_size_t
        S = C.c_int  # kvc_status
        sig = {
            "kvc_record_bytes": (Z, [P]),
            "kvc_idx_row_bytes": (Z, [P]),
            "kvc_bytes_resident": (Z, [P, C.c_int64, I, I]),
            "kvc_workspace_bytes": (Z, [P, I, I]),
            "kvc_pack": (S, [P, P, I, P, P, P, P, P]),
            "kvc_index_topk": (S, [P, P, P, P, P, P, Z, P, P]),
            "kvc_index_topk_noalloc": (S, [P, P, P, P, P, P, P]),
            "kvc_sparse_decode_attn": (S, [P, P, P, P, P, I, P, P, P, Z, P, P]),
            "kvc_layer_group_step": (S, [P, I, P, P, P, P, I, P, P, P, P, P, Z, P, P]),
            "kvc_workspace_bytes_hier": (Z, [P, I, I, I, I]),
            "kvc_workspace_bytes_batched": (Z, [P, I, I, I]),
            "kvc_pack_window_fp8": (S, [P, P, C.c_int64, P, P, P, P]),
            "kvc_sparse_decode_attn_fp8win": (S, [P, P, P, P, P, P, I, P, P, P, Z, P, P]),
            "kvc_index_topk_batched": (S, [P, I, P, P, P, P, Z, P, P]),
            "kvc_layer_group_step_hier": (S, [P, I, I, I, P, P, P, P, I, P, P, P, P, P, Z, P,
                                              P]),
            "kvc_unpack": (S, [P, P, P, I, I, P, P, P]),
            "kvc_unpack_window_fp8": (S, [P, P, P, C.c_int64, P, P]),
            "kvc_norm_rope": (S, [P, I, P, C.c_int64, P, I, P, P, C.c_int64, P, I, P, P, P,
                                  C.c_float, I, P, P]),
            "kvc_tree_decode_attn": (S, [P, I, P, P, P, I, P, I, P, P, P, P, P, P, P]),
            "kvc_verify_tree": (S, [I, I, I, I, P, C.c_int64, P, C.c_int64, P, P, P, P, P, P, P,
                                    P, P]),
            "kvc_e2m1_encode": (S, [P, C.c_int64, P, P]),
            "kvc_e4m3_encode": (S, [P, C.c_int64, P, P]),
            "kvc_trace_begin": (S, [I]),
            "kvc_trace_end": (S, []),
            "kvc_trace_kernel": (S, [C.c_char_p, C.POINTER(C.c_int), C.POINTER(C.c_double)]),
            "kvc_launch_count": (C.c_uint64, []),
            "kvc_debug_set_wait_limit_ns": (S, [C.c_uint64]),
            "kvc_status_string": (C.c_char_p, [I]),
            "kvc_version": (C.c_char_p, []),
        }
        for name, (res, args) in sig.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = lib
    return _LIB


def lib():
    """The loaded C library (ctypes.CDLL); raises if it is not built."""
    return _lib()


def _check(fn, rc):
    if rc != OK:
        raise KvcError(fn, rc)


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return C.c_void_p(t.data_ptr())


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return C.c_void_p(s.cuda_stream)


def _here(stream):
    """Current device and the address of `stream` on it (None: the current
    stream, without the 3 us that torch.cuda.current_stream() takes)."""
    dev = torch.cuda.current_device()
    return dev, torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _operand(name, t, dtype, shape, dev, contiguous=True):
    """Device address of an operand (None stays None), checked: type, shape,
    contiguity, and that it lives on the current device `dev` (the library's
    work and pointers belong to it)."""
    if t is None:
        return None
    if t.dtype == dtype and t.shape == shape and t.get_device() == dev and \
            (not contiguous or t.is_contiguous()):
        return t.data_ptr()
    if t.dtype != dtype or t.shape != shape:
        raise ValueError(f"{name}: expected {dtype} {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name}: expected a tensor on the current CUDA device")
    raise ValueError(f"{name}: expected a contiguous tensor")


def _records(cfg, cache, dev):
    """The C view of `cache`, checked: the kernels step through its records by
    the record size of the call's `cfg`, so they must be laid out as that says,
    and live, with the lengths, on the current device `dev`."""
    rb = _lib().kvc_record_bytes(C.byref(cfg))
    if rb == 0:  # no valid configuration, which the library says
        return cache.struct()
    own, b, cap = cache.cfg, cache.batch, cache.capacity
    if own is not cfg and (own.latent_dim != cfg.latent_dim or own.rope_dim != cfg.rope_dim or
                           own.group != cfg.group or own.scale_fmt != cfg.scale_fmt):
        raise ValueError("cache: its records are laid out for another configuration")
    return CacheStruct(_operand("cache.records", cache.records, torch.uint8, (b, cap, rb), dev),
                       cache.idx_k.data_ptr(),
                       _operand("cache.n_entries", cache.n_entries, torch.int32, (b,), dev), b, cap)


def _act(cfg: Config):
    return torch.bfloat16 if cfg.act_dtype == BF16 else torch.float32


def _status(status, dev):
    return None if status is None else _operand("status", status, torch.int32, (1,), dev)


def make_config(latent_dim, rope_dim, group, scale_fmt, idx_dim, topk, window, n_heads, sm_scale,
                act_dtype, ratio=2, idx_fmt=0) -> Config:
    """ratio: raw tokens per entry, 2 or 4; idx_fmt: indexer keys as int8 (0)
    or FP4 rows (1)."""
    return Config(latent_dim, rope_dim, group, scale_fmt, idx_dim, topk, window, n_heads,
                  float(sm_scale), act_dtype, ratio, idx_fmt)


def config_for(w) -> Config:
    """kvc_config of a synth.Workload."""
    return make_config(w.latent, w.rope, w.group, w.scale_fmt, w.idx_dim, w.topk, w.window,
                       w.heads, w.sm_scale, F32 if w.act == "f32" else BF16, w.ratio,
                       w.idx_fmt)


def record_bytes(cfg: Config) -> int:
    return int(_lib().kvc_record_bytes(C.byref(cfg)))


def idx_row_bytes(cfg: Config) -> int:
    return int(_lib().kvc_idx_row_bytes(C.byref(cfg)))


def bytes_resident(cfg: Config, entries: int, n_layers: int, padded: bool) -> int:
    return int(_lib().kvc_bytes_resident(C.byref(cfg), entries, n_layers, int(padded)))


def workspace_bytes(cfg: Config, batch: int, capacity: int) -> int:
    return int(_lib().kvc_workspace_bytes(C.byref(cfg), batch, capacity))


class Cache:
    """Device buffers of one stored cache (records, indexer keys, lengths)."""

    def __init__(self, cfg: Config, batch: int, capacity: int, device="cuda"):
        rb = record_bytes(cfg)
        if rb == 0:
            raise ValueError("invalid kvc config")
        self.cfg, self.batch, self.capacity = cfg, batch, capacity
        self.records = torch.zeros(batch, capacity, rb, dtype=torch.uint8, device=device)
        if cfg.idx_fmt == 1:  # FP4 rows of idx_dim/2 + idx_dim/16 bytes
            self.idx_k = torch.zeros(batch, capacity, idx_row_bytes(cfg), dtype=torch.uint8,
                                     device=device)
        else:
            self.idx_k = torch.zeros(batch, capacity, cfg.idx_dim, dtype=torch.int8,
                                     device=device)
        self.n_entries = torch.zeros(batch, dtype=torch.int32, device=device)

    @classmethod
    def wrap(cls, cfg: Config, records, idx_k, n_entries):
        """A cache over buffers the caller already has: records [B][cap][record
        bytes] uint8, idx_k [B][cap][indexer row bytes], n_entries [B] int32."""
        self = cls.__new__(cls)
        self.cfg, (self.batch, self.capacity) = cfg, records.shape[:2]
        self.records, self.idx_k, self.n_entries = records, idx_k, n_entries
        lead, dev = (self.batch, self.capacity), torch.cuda.current_device()
        _operand("records", records, torch.uint8, (*lead, record_bytes(cfg)), dev)
        _operand("idx_k", idx_k, torch.uint8 if cfg.idx_fmt == 1 else torch.int8,
                 (*lead, idx_row_bytes(cfg)), dev)
        _operand("n_entries", n_entries, torch.int32, (self.batch,), dev)
        return self

    def struct(self) -> CacheStruct:
        return CacheStruct(self.records.data_ptr(), self.idx_k.data_ptr(),
                           self.n_entries.data_ptr(), self.batch, self.capacity)


def workspace(cfg: Config, batch: int, capacity: int, device="cuda", hier_blocks: int = 0,
              hier_block: int = 8) -> torch.Tensor:
    """Workspace for the calls on `batch` x `capacity` (and, with hier_blocks
    > 0, for the hierarchical group step)."""
    if hier_blocks:
        n = int(_lib().kvc_workspace_bytes_hier(C.byref(cfg), batch, capacity, hier_blocks,
                                                 hier_block))
    else:
        n = workspace_bytes(cfg, batch, capacity)
    if n == 0:
        raise KvcError("invalid workspace request")
    return torch.zeros(n + 256, dtype=torch.uint8, device=device)  # zero-filled before first use


def _ws(ws):
    # 256-byte aligned view into a workspace tensor
    base = ws.data_ptr()
    off = (-base) % 256
    return C.c_void_p(base + off), ws.numel() - off


def pack_window_fp8(cfg, rows, codes, scales, status=None, stream=None):
    """rows [..][D] -> codes [..][D] uint8 (signed E4M3), scales [..] fp32."""
    n = rows.numel() // rows.shape[-1]
    _check("kvc_pack_window_fp8", _lib().kvc_pack_window_fp8(
        C.byref(cfg), _ptr(rows), n, _ptr(codes), _ptr(scales), _ptr(status), _stream(stream)))


def sparse_decode_attn_fp8win(cfg, q, cache: Cache, topk_idx, win_codes, win_scales, window_len,
                              out, ws, lse=None, status=None, stream=None):
    p, n = _ws(ws)
    cs = cache.struct()
    _check("kvc_sparse_decode_attn_fp8win", _lib().kvc_sparse_decode_attn_fp8win(
        C.byref(cfg), _ptr(q), C.byref(cs), _ptr(topk_idx), _ptr(win_codes), _ptr(win_scales),
        int(window_len), _ptr(out), _ptr(lse), p, n, _ptr(status), _stream(stream)))


def workspace_batched(cfg: Config, nq: int, batch: int, capacity: int,
                      device="cuda") -> torch.Tensor:
    """Workspace for index_topk_batched with nq queries per sequence."""
    n = int(_lib().kvc_workspace_bytes_batched(C.byref(cfg), nq, batch, capacity))
    if n == 0:
        raise KvcError("invalid batched workspace request")
    return torch.zeros(n + 256, dtype=torch.uint8, device=device)  # zero-filled before first use


def index_topk_batched(cfg, idx_q, cache: Cache, topk_out, ws, status=None, stream=None):
    """idx_q [nq][B][Di] int8 -> topk_out [nq][B][K]: every query against the
    cache in one tensor-core pass."""
    p, n = _ws(ws)
    cs = cache.struct()
    _check("kvc_index_topk_batched", _lib().kvc_index_topk_batched(
        C.byref(cfg), idx_q.shape[0], _ptr(idx_q), C.byref(cs), _ptr(topk_out), p, n,
        _ptr(status), _stream(stream)))


def pack(cfg, tokens, gate, idx_k_new, cache: Cache, status=None, stream=None):
    n_new = tokens.shape[1]
    cs = cache.struct()
    _check("kvc_pack", _lib().kvc_pack(C.byref(cfg), _ptr(tokens), n_new, _ptr(gate),
                                       _ptr(idx_k_new), C.byref(cs), _ptr(status), _stream(stream)))


def index_topk(cfg, idx_q, cache: Cache, topk_out, ws, scores=None, status=None, stream=None):
    p, n = _ws(ws)
    cs = cache.struct()
    _check("kvc_index_topk", _lib().kvc_index_topk(C.byref(cfg), _ptr(idx_q), C.byref(cs),
                                                   _ptr(topk_out), _ptr(scores), p, n,
                                                   _ptr(status), _stream(stream)))


def index_topk_noalloc(cfg, idx_q, cache: Cache, topk_out, scores=None, status=None,
                       stream=None):
    """kvc_index_topk with the library's fixed scratch (no workspace argument)."""
    cs = cache.struct()
    _check("kvc_index_topk_noalloc", _lib().kvc_index_topk_noalloc(
        C.byref(cfg), _ptr(idx_q), C.byref(cs), _ptr(topk_out), _ptr(scores), _ptr(status),
        _stream(stream)))


def sparse_decode_attn(cfg, q, cache: Cache, topk, window, window_len, out, ws, lse=None,
                       status=None, stream=None):
    p, n = _ws(ws)
    cs = cache.struct()
    _check("kvc_sparse_decode_attn", _lib().kvc_sparse_decode_attn(
        C.byref(cfg), _ptr(q), C.byref(cs), _ptr(topk), _ptr(window), int(window_len), _ptr(out),
        _ptr(lse), p, n, _ptr(status), _stream(stream)))


def layer_group_step(cfg, modes, q, idx_q, windows, window_len, cache: Cache, out, topk, ws,
                     lse=None, status=None, stream=None, hier_blocks=0, hier_block=8):
    """One decode step through a CSA2 layer group; hier_blocks > 0 turns on
    the hierarchical indexer (the workspace must have been sized for it)."""
    modes_arr = (C.c_int32 * len(modes))(*modes)
    p, n = _ws(ws)
    cs = cache.struct()
    if hier_blocks:
        _check("kvc_layer_group_step_hier", _lib().kvc_layer_group_step_hier(
            C.byref(cfg), int(hier_blocks), int(hier_block), len(modes), modes_arr, _ptr(q),
            _ptr(idx_q), _ptr(windows), int(window_len), C.byref(cs), _ptr(out), _ptr(lse),
            _ptr(topk), p, n, _ptr(status), _stream(stream)))
        return
    _check("kvc_layer_group_step", _lib().kvc_layer_group_step(
        C.byref(cfg), len(modes), modes_arr, _ptr(q), _ptr(idx_q), _ptr(windows), int(window_len),
        C.byref(cs), _ptr(out), _ptr(lse), _ptr(topk), p, n, _ptr(status), _stream(stream)))


def unpack(cfg, cache: Cache, rows, idx=None, first=0, status=None, stream=None):
    """Records read back: rows [B][n][D] act_dtype receives entries idx [B][n]
    int32 (-1: zeros), or entries first .. first + n - 1 without idx."""
    n, b = rows.shape[1], cache.batch
    d = cfg.latent_dim + cfg.rope_dim
    dev, st = _here(stream)
    cs = _records(cfg, cache, dev)
    _check("kvc_unpack", _lib().kvc_unpack(
        C.byref(cfg), C.byref(cs), _operand("idx", idx, torch.int32, (b, n), dev), int(first), n,
        _operand("rows", rows, _act(cfg), (b, n, d), dev), _status(status, dev), st))


def unpack_window_fp8(cfg, codes, scales, rows, stream=None):
    """codes [..][D] uint8 (signed E4M3) and scales [..] fp32, as
    pack_window_fp8 writes them -> rows [..][D] act_dtype."""
    d = cfg.latent_dim + cfg.rope_dim
    lead = scales.shape
    dev, st = _here(stream)
    _check("kvc_unpack_window_fp8", _lib().kvc_unpack_window_fp8(
        C.byref(cfg), _operand("codes", codes, torch.uint8, (*lead, d), dev),
        _operand("scales", scales, torch.float32, lead, dev), scales.numel(),
        _operand("rows", rows, _act(cfg), (*lead, d), dev), st))


def norm_rope(cfg, q, k, positions, inv_freq, q_out, k_out, q_gain=None, k_gain=None,
              q_norm=NORM_ROW, k_norm=NORM_LATENT, eps=1e-6, layout=ROPE_HALVES, status=None,
              stream=None):
    """Norms and position rotation of query rows q [n][H][D] and key rows k
    [n][D] (either may be None, with its output); their first dimension may be
    strided (a slice of a wider projection), the outputs are contiguous."""
    n, h, lat = positions.shape[0], cfg.n_heads, cfg.latent_dim
    d = lat + cfg.rope_dim
    act, f32 = _act(cfg), torch.float32
    width = {NORM_LATENT: lat, NORM_ROW: d}
    dev, st = _here(stream)
    qs = ks = 0
    if q is not None:
        qs, qh, qd = q.stride()
        if qd != 1 or (h > 1 and qh != d):
            raise ValueError("q: the heads of a token must be contiguous")
        if n <= 1:
            qs = h * d
        if q_out is None:
            raise ValueError("q_out: needed with q")
    if k is not None:
        ks, kd = k.stride()
        if kd != 1:
            raise ValueError("k: the channels of a row must be contiguous")
        if n <= 1:
            ks = d
        if k_out is None:
            raise ValueError("k_out: needed with k")
    _check("kvc_norm_rope", _lib().kvc_norm_rope(
        C.byref(cfg), n, _operand("q", q, act, (n, h, d), dev, False), qs,
        _operand("q_gain", q_gain, f32, (width.get(q_norm, 0),), dev), q_norm,
        _operand("q_out", q_out, act, (n, h, d), dev) if q is not None else None,
        _operand("k", k, act, (n, d), dev, False), ks,
        _operand("k_gain", k_gain, f32, (width.get(k_norm, 0),), dev), k_norm,
        _operand("k_out", k_out, act, (n, d), dev) if k is not None else None,
        _operand("positions", positions, torch.int32, (n,), dev),
        _operand("inv_freq", inv_freq, f32, (cfg.rope_dim // 2,), dev), eps, layout,
        _status(status, dev), st))


def tree_decode_attn(cfg, q, cache: Cache, topk, window, window_len, draft, parents, out, lse=None,
                     window_lens=None, status=None, stream=None):
    """Attention of T drafted tokens per sequence, each over its selected
    entries and the window of its own path: q [T][B][H][D], topk [T][B][K] or
    [B][K] (one selection for all nodes), window [B][W][D], draft [T][B][D],
    parents [T][B] -> out [T][B][H][latent] act_dtype."""
    t, b, lat = q.shape[0], cache.batch, cfg.latent_dim
    d, h, i32 = lat + cfg.rope_dim, cfg.n_heads, torch.int32
    act, shared = _act(cfg), topk.dim() == 2
    dev, st = _here(stream)
    cs = _records(cfg, cache, dev)
    _check("kvc_tree_decode_attn", _lib().kvc_tree_decode_attn(
        C.byref(cfg), t, _operand("q", q, act, (t, b, h, d), dev), C.byref(cs),
        _operand("topk", topk, i32, (b, cfg.topk) if shared else (t, b, cfg.topk), dev), shared,
        _operand("window", window, act, (b, cfg.window, d), dev), int(window_len),
        _operand("window_lens", window_lens, i32, (b,), dev),
        _operand("draft", draft, act, (t, b, d), dev),
        _operand("parents", parents, i32, (t, b), dev),
        _operand("out", out, act, (t, b, h, lat), dev),
        _operand("lse", lse, torch.float32, (t, b, h), dev), _status(status, dev), st))


def verify_tree(p, q, tokens, parents, u, v, path, n_path, next_token, status=None, stream=None):
    """Verify drafted trees: target and draft probabilities p, q [T][B][V]
    (fp32 or bf16; q None: greedy drafts; rows may be padded to equal steps),
    tokens, parents, u [T][B], v [B] -> path [B][T], n_path [B], next_token [B]."""
    t, b, vocab = p.shape
    dtype, i32, f32 = p.dtype, torch.int32, torch.float32
    dev, st = _here(stream)

    def rows(name, x):  # equally spaced rows t * B + b of contiguous entries
        st, sb, sv = x.stride()
        step = sb if b > 1 else st if t > 1 else vocab
        if (sv != 1 and vocab > 1) or (t > 1 and b > 1 and st != b * step):
            raise ValueError(f"{name}: rows must be contiguous and equally spaced")
        return _operand(name, x, dtype, (t, b, vocab), dev, False), step

    if dtype not in (f32, torch.bfloat16):
        raise ValueError("p: expected fp32 or bf16 probabilities")
    pp, ps = rows("p", p)
    qp, qs = rows("q", q) if q is not None else (None, 0)
    _check("kvc_verify_tree", _lib().kvc_verify_tree(
        b, t, vocab, F32 if dtype == f32 else BF16, pp, ps, qp, qs,
        _operand("tokens", tokens, i32, (t, b), dev),
        _operand("parents", parents, i32, (t, b), dev), _operand("u", u, f32, (t, b), dev),
        _operand("v", v, f32, (b,), dev), _operand("path", path, i32, (b, t), dev),
        _operand("n_path", n_path, i32, (b,), dev),
        _operand("next_token", next_token, i32, (b,), dev), _status(status, dev), st))


def e2m1_encode(x, codes, stream=None):
    _check("kvc_e2m1_encode", _lib().kvc_e2m1_encode(_ptr(x), x.numel(), _ptr(codes),
                                                     _stream(stream)))


def e4m3_encode(x, out, stream=None):
    _check("kvc_e4m3_encode", _lib().kvc_e4m3_encode(_ptr(x), x.numel(), _ptr(out),
                                                     _stream(stream)))


def trace_begin(max_launches: int = 4096):
    _check("kvc_trace_begin", _lib().kvc_trace_begin(max_launches))


def trace_end():
    _check("kvc_trace_end", _lib().kvc_trace_end())


def trace_kernel(name: str):
    n = C.c_int(0)
    ms = C.c_double(0.0)
    _check("kvc_trace_kernel", _lib().kvc_trace_kernel(name.encode(), C.byref(n), C.byref(ms)))
    return n.value, ms.value


def launch_count() -> int:
    return int(_lib().kvc_launch_count())


def debug_set_wait_limit_ns(ns: int):
    """Test hook: bound of every in-kernel wait of later launches (0 = one
    non-blocking poll; the library's default is 2_000_000_000)."""
    _check("kvc_debug_set_wait_limit_ns", _lib().kvc_debug_set_wait_limit_ns(int(ns)))


def version() -> str:
    return _lib().kvc_version().decode()
