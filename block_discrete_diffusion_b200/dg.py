"""Python binding of libdg.so (include/dg.h): argument marshalling only.

Every function here has the name of the C entry point it calls and passes device pointers of torch
CUDA tensors straight through.  PyTorch provides device memory and the stream; all computation runs
in the library's kernels.  There is no fallback: if libdg.so is missing or fails to load, every call
raises.
"""
from __future__ import annotations

import ctypes
import math
import os
import struct

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libdg.so")

c_int, c_float, c_void_p, c_size_t, c_uint64 = ctypes.c_int, ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_uint64
c_int64 = ctypes.c_int64

# the entry points declared in include/dg.h
ENTRY_POINTS = (
    "dg_last_error", "dg_model_create", "dg_model_destroy", "dg_kv_bytes", "dg_workspace_bytes", "dg_seqs_create",
    "dg_seqs_destroy", "dg_seqs_get_state", "dg_load_prefix", "dg_prefill", "dg_canvas_init", "dg_canvas_step",
    "dg_block_commit", "dg_decode", "dg_layer_forward", "dg_sample_workspace_bytes", "dg_sample", "dg_device_error",
    "dg_temperature", "dg_stats_reset", "dg_stats_read", "dg_sample_noalloc", "dg_sample_noalloc_max_rows",
    "dg_block_commit_last_kv", "dg_head_sample_workspace_bytes", "dg_head_sample", "dg_head_sample_error",
    "dg_kv4_pool_bytes", "dg_kv4_book_bytes", "dg_kv4_init", "dg_kv4_extend", "dg_kv4_fork", "dg_kv4_free",
    "dg_kv4_compact", "dg_kv4_append", "dg_kv4_read", "dg_kv4_attend_workspace_bytes", "dg_kv4_attend", "dg_kv4_error",
    "dg_store_prefix_kv4", "dg_load_prefix_kv4",
)

# dg_kernel_class, in order
KERNEL_CLASSES = ("embed", "rmsnorm", "qkv", "attn", "attn_merge", "oproj", "router", "topk", "bucket", "expert_up",
                  "expert_down", "combine", "head", "sampler", "misc", "dequant")
WDTYPE_BF16, WDTYPE_FP8_BLOCK128 = 0, 1
MATRICES = ("w_qkv", "w_o", "w_router", "w_gate_up", "w_down")

DG_OK, DG_ERR_INVALID_ARG, DG_ERR_CAPACITY, DG_ERR_STATE, DG_ERR_CUDA, DG_ERR_UNSUPPORTED, DG_ERR_DEVICE = range(7)


class DGError(RuntimeError):
    def __init__(self, fn, status, msg):
        super().__init__(f"{fn} -> status {status}: {msg}")
        self.status = status


class dg_model_config(ctypes.Structure):
    _fields_ = [(n, c_int) for n in ("d_model", "n_q", "n_kv", "d_head", "n_exp", "top_k", "d_ff", "n_layers",
                                     "vocab")] + [("rms_eps", c_float), ("rope_theta", c_float), ("wdtype", c_int)]


class dg_layer_weights(ctypes.Structure):
    _fields_ = [(n, c_void_p) for n in ("attn_norm", "w_qkv", "w_o", "ffn_norm", "w_router", "w_gate_up", "w_down",
                                        "s_qkv", "s_o", "s_router", "s_gate_up", "s_down")]


class dg_weights(ctypes.Structure):
    _fields_ = [("emb", c_void_p), ("final_norm", c_void_p), ("head", c_void_p),
                ("layers", ctypes.POINTER(dg_layer_weights))]


class dg_sampler_params(ctypes.Structure):
    _fields_ = [("canvas_len", c_int), ("max_steps", c_int), ("fixed_steps", c_int), ("t_start", c_float),
                ("t_end", c_float), ("entropy_bound", c_float), ("stop_mean_entropy", c_float),
                ("rerand_entropy", c_float), ("seed", c_uint64), ("eos_id", c_int), ("commit_mode", c_int),
                ("commit_rule", c_int)]


class dg_kv4_cache_t(ctypes.Structure):   # the C struct dg_kv4_cache
    _fields_ = [(n, c_int) for n in ("n_layers", "n_kv", "d_head", "n_pages", "n_seq", "max_pages")] + [
        ("d_pool", c_void_p), ("pool_bytes", c_size_t), ("d_book", c_void_p), ("book_bytes", c_size_t)]


class dg_kv4_rows(ctypes.Structure):
    _fields_ = [("k", c_void_p), ("v", c_void_p)] + [
        (n, c_int64) for n in ("k_seq", "k_row", "k_head", "v_seq", "v_row", "v_head")] + [
        ("d_rows", c_void_p), ("rows", c_int), ("dtype", c_int)]


class dg_kv4_attn(ctypes.Structure):
    _fields_ = [("q", c_void_p), ("out", c_void_p), ("lse", c_void_p), ("d_rows", c_void_p)] + [
        (n, c_int64) for n in ("q_seq", "q_row", "q_head", "o_seq", "o_row", "o_head")] + [
        (n, c_int) for n in ("n_q", "rows", "dtype", "causal")] + [("scale", c_float)]


def sampler_params(vocab, seed=0, canvas_len=256, max_steps=48, fixed_steps=0, t_start=0.8, t_end=0.4,
                   entropy_bound=0.1, stop_mean_entropy=0.005, rerand_entropy=None, eos_id=-1,
                   commit_mode=0, commit_rule=0) -> dg_sampler_params:
    if rerand_entropy is None:
        rerand_entropy = 0.5 * math.log(vocab)
    return dg_sampler_params(canvas_len, max_steps, fixed_steps, t_start, t_end, entropy_bound, stop_mean_entropy,
                             rerand_entropy, seed, eos_id, commit_mode, commit_rule)


_LIB = None


def lib():
    """Load libdg.so (raises if it is missing: there is no other implementation)."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing; build it with block_discrete_diffusion_b200.build.build()")
        L = ctypes.CDLL(LIB_PATH)
        P = ctypes.POINTER
        L.dg_last_error.restype = ctypes.c_char_p
        L.dg_model_create.argtypes = [P(dg_model_config), P(dg_weights), P(c_void_p)]
        L.dg_model_destroy.argtypes = [c_void_p]
        L.dg_model_destroy.restype = None
        L.dg_kv_bytes.argtypes = [P(dg_model_config), c_int, c_int]
        L.dg_kv_bytes.restype = c_size_t
        L.dg_workspace_bytes.argtypes = [P(dg_model_config), c_int, c_int]
        L.dg_workspace_bytes.restype = c_size_t
        L.dg_seqs_create.argtypes = [c_void_p, c_int, c_int, c_void_p, c_size_t, c_void_p, c_size_t, c_void_p,
                                     P(c_void_p)]
        L.dg_seqs_destroy.argtypes = [c_void_p]
        L.dg_seqs_destroy.restype = None
        L.dg_seqs_get_state.argtypes = [c_void_p, c_void_p, c_void_p]
        L.dg_load_prefix.argtypes = [c_void_p, c_int, c_int, c_void_p, c_void_p]
        L.dg_prefill.argtypes = [c_void_p, c_void_p, c_void_p]
        L.dg_canvas_init.argtypes = [c_void_p, P(dg_sampler_params), c_void_p, c_void_p]
        L.dg_canvas_step.argtypes = [c_void_p, P(dg_sampler_params), c_void_p, c_void_p, c_void_p, c_void_p,
                                     c_void_p, c_void_p]
        L.dg_block_commit.argtypes = [c_void_p, c_void_p]
        L.dg_block_commit_last_kv.argtypes = [c_void_p]
        L.dg_decode.argtypes = [c_void_p, P(dg_sampler_params), c_int, c_void_p, c_void_p, c_void_p]
        L.dg_layer_forward.argtypes = [c_void_p, c_int, c_int, c_int, c_void_p, c_void_p, c_void_p]
        L.dg_sample_workspace_bytes.argtypes = [c_int, c_int]
        L.dg_sample_workspace_bytes.restype = c_size_t
        L.dg_sample.argtypes = [c_void_p, c_int, c_int, P(dg_sampler_params), c_int, c_void_p, c_void_p, c_void_p,
                                c_void_p, c_void_p, c_void_p, c_size_t, c_void_p]
        L.dg_sample_noalloc.argtypes = [c_void_p, c_int, c_int, P(dg_sampler_params), c_int, c_void_p, c_void_p,
                                        c_void_p, c_void_p, c_void_p, c_void_p]
        L.dg_sample_noalloc_max_rows.argtypes = [c_int]
        L.dg_sample_noalloc_max_rows.restype = c_size_t
        L.dg_head_sample_workspace_bytes.argtypes = [c_int]
        L.dg_head_sample_workspace_bytes.restype = c_size_t
        L.dg_head_sample.argtypes = [c_void_p, c_void_p, c_int, c_int, c_int, P(dg_sampler_params), c_int, c_void_p,
                                     c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_size_t, c_void_p]
        L.dg_head_sample_error.argtypes = [c_void_p, c_void_p, P(c_int)]
        C = P(dg_kv4_cache_t)
        L.dg_kv4_pool_bytes.argtypes = [C]
        L.dg_kv4_pool_bytes.restype = c_size_t
        L.dg_kv4_book_bytes.argtypes = [C]
        L.dg_kv4_book_bytes.restype = c_size_t
        L.dg_kv4_init.argtypes = [C, c_void_p]
        L.dg_kv4_extend.argtypes = [C, c_void_p, c_void_p]
        L.dg_kv4_fork.argtypes = [C, c_void_p, c_void_p, c_int, c_void_p]
        L.dg_kv4_free.argtypes = [C, c_void_p, c_int, c_void_p]
        L.dg_kv4_compact.argtypes = [C, c_void_p]
        # (their structs: packed bytes, or ctypes.byref of the class)
        L.dg_kv4_append.argtypes = [C, c_int, c_void_p, c_void_p]
        L.dg_kv4_read.argtypes = [C, c_int, c_void_p, c_void_p]
        L.dg_kv4_attend_workspace_bytes.argtypes = [C, c_int, c_int]
        L.dg_kv4_attend_workspace_bytes.restype = c_size_t
        L.dg_kv4_attend.argtypes = [C, c_int, c_void_p, c_void_p, c_size_t, c_void_p]
        L.dg_kv4_error.argtypes = [C, c_void_p, P(c_int)]
        L.dg_store_prefix_kv4.argtypes = [c_void_p, c_int, C, c_int]
        L.dg_load_prefix_kv4.argtypes = [c_void_p, c_int, c_int, C, c_int]
        L.dg_device_error.argtypes = [c_void_p, P(c_int)]
        L.dg_stats_reset.argtypes = [c_void_p, c_int]
        L.dg_stats_read.argtypes = [c_void_p, c_void_p, c_void_p]
        L.dg_temperature.argtypes = [P(dg_sampler_params), c_int]
        L.dg_temperature.restype = c_float
        _LIB = L
    return _LIB


def _check(fn, status):
    if status != DG_OK:
        raise DGError(fn, status, lib().dg_last_error().decode())


def _ptr(t):
    if t is None:
        return None
    assert isinstance(t, torch.Tensor) and t.is_cuda and t.is_contiguous(), "expected a contiguous CUDA tensor"
    return t.data_ptr()


def _stream_handle(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def make_config(cfg) -> dg_model_config:
    return dg_model_config(cfg.d_model, cfg.n_q, cfg.n_kv, cfg.d_head, cfg.n_exp, cfg.top_k, cfg.d_ff, cfg.n_layers,
                           cfg.vocab, cfg.rms_eps, cfg.rope_theta, getattr(cfg, "wdtype", WDTYPE_BF16))


def _layer_struct(L: dict) -> "dg_layer_weights":
    """A layer dict of device tensors; in the FP8 form each matrix is {"e4m3": uint8, "scale": fp32}."""
    def mat(k):
        t = L[k]
        return (_ptr(t["e4m3"]), _ptr(t["scale"])) if isinstance(t, dict) else (_ptr(t), None)
    (q, sq), (o, so), (r, sr), (gu, sgu), (dn, sdn) = (mat(k) for k in MATRICES)
    return dg_layer_weights(_ptr(L["attn_norm"]), q, o, _ptr(L["ffn_norm"]), r, gu, dn, sq, so, sr, sgu, sdn)


# ---------------------------------------------------------------------------------------------
# thin wrappers, one per entry point
# ---------------------------------------------------------------------------------------------
class Model:
    """dg_model handle; keeps the weight tensors (borrowed by the library) alive."""

    def __init__(self, handle, cfg, weights, c_cfg):
        self.handle, self.cfg, self.weights, self.c_cfg = handle, cfg, weights, c_cfg

    def __del__(self):
        if getattr(self, "handle", None) and _LIB is not None:
            _LIB.dg_model_destroy(self.handle)
            self.handle = None


def dg_model_create(cfg, weights: dict) -> Model:
    c = make_config(cfg)
    layers = (dg_layer_weights * cfg.n_layers)()
    for i, L in enumerate(weights["layers"]):
        layers[i] = _layer_struct(L)
    w = dg_weights(_ptr(weights["emb"]), _ptr(weights["final_norm"]), _ptr(weights["head"]),
                   ctypes.cast(layers, ctypes.POINTER(dg_layer_weights)))
    h = c_void_p()
    _check("dg_model_create", lib().dg_model_create(ctypes.byref(c), ctypes.byref(w), ctypes.byref(h)))
    return Model(h, cfg, weights, c)


def dg_kv_bytes(cfg, n_seq, max_ctx) -> int:
    c = make_config(cfg)
    return int(lib().dg_kv_bytes(ctypes.byref(c), n_seq, max_ctx))


def dg_workspace_bytes(cfg, n_seq, max_ctx) -> int:
    c = make_config(cfg)
    return int(lib().dg_workspace_bytes(ctypes.byref(c), n_seq, max_ctx))


class Seqs:
    """dg_seqs handle; keeps the model, the KV cache and the workspace tensors alive."""

    def __init__(self, handle, model, n_seq, max_ctx, kv, ws, stream):
        self.handle, self.model, self.n_seq, self.max_ctx, self.kv, self.ws, self.stream = (
            handle, model, n_seq, max_ctx, kv, ws, stream)

    def __del__(self):
        if getattr(self, "handle", None) and _LIB is not None:
            _LIB.dg_seqs_destroy(self.handle)
            self.handle = None


def dg_seqs_create(model: Model, n_seq, max_ctx, kv=None, ws=None, stream=None) -> Seqs:
    """kv / ws: caller device buffers (uint8 CUDA tensors); allocated here through torch if None."""
    dev = torch.device("cuda", torch.cuda.current_device())
    if kv is None:
        kv = torch.empty(dg_kv_bytes(model.cfg, n_seq, max_ctx), dtype=torch.uint8, device=dev)
    if ws is None:
        ws = torch.empty(dg_workspace_bytes(model.cfg, n_seq, max_ctx), dtype=torch.uint8, device=dev)
    h = c_void_p()
    _check("dg_seqs_create", lib().dg_seqs_create(model.handle, n_seq, max_ctx, _ptr(kv), kv.numel(), _ptr(ws),
                                                  ws.numel(), _stream_handle(stream), ctypes.byref(h)))
    return Seqs(h, model, n_seq, max_ctx, kv, ws, stream)


def dg_seqs_get_state(seqs: Seqs):
    P = (c_int * seqs.n_seq)()
    step = c_int()
    _check("dg_seqs_get_state", lib().dg_seqs_get_state(seqs.handle, P, ctypes.byref(step)))
    return list(P), step.value


def dg_load_prefix(seqs: Seqs, seq, P, k_layers, v_layers):
    n = len(k_layers)
    ks = (c_void_p * n)(*[_ptr(k) for k in k_layers])
    vs = (c_void_p * n)(*[_ptr(v) for v in v_layers])
    _check("dg_load_prefix", lib().dg_load_prefix(seqs.handle, seq, P, ks, vs))


def dg_prefill(seqs: Seqs, ids: torch.Tensor, lens):
    lens_c = (ctypes.c_int32 * len(lens))(*lens)
    _check("dg_prefill", lib().dg_prefill(seqs.handle, _ptr(ids), lens_c))


def dg_canvas_init(seqs: Seqs, params: dg_sampler_params, ids, commit):
    _check("dg_canvas_init", lib().dg_canvas_init(seqs.handle, ctypes.byref(params), _ptr(ids), _ptr(commit)))


def dg_canvas_step(seqs: Seqs, params, ids, commit, entropy, stop, hidden=None, logits=None):
    _check("dg_canvas_step", lib().dg_canvas_step(seqs.handle, ctypes.byref(params), _ptr(ids), _ptr(commit),
                                                  _ptr(entropy), _ptr(stop), _ptr(hidden), _ptr(logits)))


def dg_block_commit(seqs: Seqs, ids):
    _check("dg_block_commit", lib().dg_block_commit(seqs.handle, _ptr(ids)))


def dg_block_commit_last_kv(seqs: Seqs):
    _check("dg_block_commit_last_kv", lib().dg_block_commit_last_kv(seqs.handle))


def dg_decode(seqs: Seqs, params, max_blocks, out):
    n_out = (ctypes.c_int32 * seqs.n_seq)()
    steps = (ctypes.c_int32 * max_blocks)()
    _check("dg_decode", lib().dg_decode(seqs.handle, ctypes.byref(params), max_blocks, _ptr(out), n_out, steps))
    return list(n_out), list(steps)


def dg_layer_forward(seqs: Seqs, layer, x, x_mid=None, router_logits=None, n_rows=256, causal=False):
    _check("dg_layer_forward", lib().dg_layer_forward(seqs.handle, layer, n_rows, int(bool(causal)), _ptr(x), _ptr(x_mid),
                                                      _ptr(router_logits)))


def dg_sample_workspace_bytes(n_rows, vocab) -> int:
    return int(lib().dg_sample_workspace_bytes(n_rows, vocab))


def dg_sample(logits, n_seq, vocab, params, step, seq_P, ids, commit, entropy, stop, ws, stream=None):
    _check("dg_sample", lib().dg_sample(_ptr(logits), n_seq, vocab, ctypes.byref(params), step, _ptr(seq_P),
                                        _ptr(ids), _ptr(commit), _ptr(entropy), _ptr(stop), _ptr(ws), ws.numel(),
                                        _stream_handle(stream)))


def dg_sample_noalloc(logits, n_seq, vocab, params, step, seq_P, ids, commit, entropy, stop, stream=None):
    """dg_sample with its scratch in the library's static device array (no workspace argument)."""
    _check("dg_sample_noalloc", lib().dg_sample_noalloc(_ptr(logits), n_seq, vocab, ctypes.byref(params), step,
                                                        _ptr(seq_P), _ptr(ids), _ptr(commit), _ptr(entropy),
                                                        _ptr(stop), _stream_handle(stream)))


def dg_sample_noalloc_max_rows(vocab) -> int:
    return int(lib().dg_sample_noalloc_max_rows(vocab))


def dg_head_sample_workspace_bytes(vocab) -> int:
    return int(lib().dg_head_sample_workspace_bytes(vocab))


def dg_head_sample(xn, head, params, step, seq_P, ids, commit, entropy, stop, ws, nv=128, logits=None, stream=None):
    """The fused vocabulary head + sampler on caller inputs (xn bf16 [256, d], head bf16 [V, d])."""
    _check("dg_head_sample", lib().dg_head_sample(_ptr(xn), _ptr(head), xn.shape[1], head.shape[0], nv,
                                                  ctypes.byref(params), step, _ptr(seq_P), _ptr(ids), _ptr(commit),
                                                  _ptr(entropy), _ptr(stop), _ptr(logits), _ptr(ws), ws.numel(),
                                                  _stream_handle(stream)))


def dg_head_sample_error(ws, stream=None) -> int:
    code = c_int()
    st = lib().dg_head_sample_error(_ptr(ws), _stream_handle(stream), ctypes.byref(code))
    if st not in (DG_OK, DG_ERR_DEVICE):
        _check("dg_head_sample_error", st)
    return code.value


# ---------------------------------------------------------------------------------------------
# the paged 4-bit cache
# ---------------------------------------------------------------------------------------------
_KV4_DTYPES = {torch.bfloat16: 0, torch.float16: 1}


class Kv4Cache:
    """A cache's shape and its two buffers (kept alive here).  lens [n_seq], refs [n_pages] and table [n_seq, max_pages]
    are int32 views of the book: read them as you like, change them through the calls below."""

    def __init__(self, c, pool, book):
        self.c, self.pool, self.book = c, pool, book
        self.ref = ctypes.byref(c)
        self.device, self.index = pool.device, pool.device.index
        self.n_seq, self.n_kv, self.d_head = c.n_seq, c.n_kv, c.d_head   # (a read of the C struct takes longer)
        pad = lambda n: (n + 3) // 4 * 4   # noqa: E731
        refs = 16 + pad(c.n_seq)
        table = refs + pad(c.n_pages)
        self.lens = book[16:16 + c.n_seq]
        self.refs = book[refs:refs + c.n_pages]
        self.table = book[table:table + c.n_seq * c.max_pages].view(c.n_seq, c.max_pages)


def dg_kv4_cache(n_layers, n_kv, d_head, n_pages, n_seq, max_pages, pool=None, book=None) -> Kv4Cache:
    """pool (uint8) and book (int32): caller device buffers, taken as they are; allocated here through torch and
    initialised (every sequence empty) if None."""
    c = dg_kv4_cache_t(n_layers, n_kv, d_head, n_pages, n_seq, max_pages, None, 0, None, 0)
    fresh = book is None
    if (pool is None) != fresh:
        raise ValueError("give both pool and book, or neither")
    if fresh:
        need = dg_kv4_pool_bytes(c)
        if not need:
            raise ValueError("dg_kv4_cache: a shape this build does not support")
        dev = torch.device("cuda", torch.cuda.current_device())
        pool = torch.empty(need, dtype=torch.uint8, device=dev)
        book = torch.empty(dg_kv4_book_bytes(c) // 4, dtype=torch.int32, device=dev)
    if pool.dtype != torch.uint8 or book.dtype != torch.int32 or book.dim() != 1 or pool.device != book.device:
        raise ValueError("pool must be uint8 and book a flat int32 tensor on one device")
    c.d_pool, c.pool_bytes, c.d_book, c.book_bytes = _ptr(pool), pool.numel(), _ptr(book), 4 * book.numel()
    if not dg_kv4_book_bytes(c) or c.book_bytes < dg_kv4_book_bytes(c):
        raise ValueError("dg_kv4_cache: a shape this build does not support, or a book too small for it")
    cache = Kv4Cache(c, pool, book)
    if fresh:
        dg_kv4_init(cache)
    return cache


def dg_kv4_pool_bytes(c) -> int:
    return int(lib().dg_kv4_pool_bytes(ctypes.byref(getattr(c, "c", c))))


def dg_kv4_book_bytes(c) -> int:
    return int(lib().dg_kv4_book_bytes(ctypes.byref(getattr(c, "c", c))))


# A small call's time is the host's, so: the current stream's handle without building a Stream object (3 us), the
# device's index without the wrapper's checks (the cache's tensors have initialised CUDA), structs packed at once.
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                              lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_pack_rows = struct.Struct("@PPqqqqqqPii")      # dg_kv4_rows
_pack_attn = struct.Struct("@PPPPqqqqqqiiiif4x")   # dg_kv4_attn
assert _pack_rows.size == ctypes.sizeof(dg_kv4_rows) and _pack_attn.size == ctypes.sizeof(dg_kv4_attn)


def _kv4_stream(cache, stream):
    """The stream's handle; the kernels run on the current device, so the cache has to lie there."""
    if cache.index != _current_device():
        raise ValueError(f"the cache lies on {cache.device}, the current device is cuda:{torch.cuda.current_device()}")
    if stream is None:
        return _current_raw_stream(cache.index)
    return stream.cuda_stream


def _kv4_ints(cache, t, n, what):
    """The address of an int32 argument of n values on the cache's device (0 for None)."""
    if t is None:
        return 0
    if t.dtype != torch.int32 or t.shape != (n,) or t.get_device() != cache.index or not t.is_contiguous():
        raise ValueError(f"{what}: expected {n} contiguous int32 values on {cache.device}")
    return t.data_ptr()


def _kv4_tensor(cache, t, shape, what, dtype=None):
    """A rows argument: its type's code and its strides; channels lie side by side."""
    own = t.dtype
    code = _KV4_DTYPES.get(own)
    if code is None or (dtype is not None and own != dtype):
        raise ValueError(f"{what}: expected bf16 or fp16, the same for every tensor of the call")
    if t.shape != shape or t.get_device() != cache.index:
        raise ValueError(f"{what}: expected shape {tuple(shape)} on {cache.device}, got {tuple(t.shape)} on {t.device}")
    s0, s1, s2, s3 = t.stride()
    if s3 != 1:
        raise ValueError(f"{what}: channels must be contiguous")
    if (s0 | s1 | s2) & 7:   # the stride of a dimension of one says nothing
        s0, s1, s2 = (0 if n == 1 else k for n, k in zip(shape, (s0, s1, s2)))
    return code, s0, s1, s2


def dg_kv4_init(cache: Kv4Cache, stream=None):
    _check("dg_kv4_init", lib().dg_kv4_init(cache.ref, _kv4_stream(cache, stream)))


def dg_kv4_extend(cache: Kv4Cache, counts, stream=None):
    """counts int32 [n_seq]: positions by which each sequence grows."""
    _check("dg_kv4_extend", lib().dg_kv4_extend(cache.ref, _kv4_ints(cache, counts, cache.n_seq, "counts"),
                                                _kv4_stream(cache, stream)))


def dg_kv4_fork(cache: Kv4Cache, src, dst, stream=None):
    n = src.numel()
    _check("dg_kv4_fork", lib().dg_kv4_fork(cache.ref, _kv4_ints(cache, src, n, "src"), _kv4_ints(cache, dst, n, "dst"),
                                            n, _kv4_stream(cache, stream)))


def dg_kv4_free(cache: Kv4Cache, slots, stream=None):
    n = slots.numel()
    _check("dg_kv4_free", lib().dg_kv4_free(cache.ref, _kv4_ints(cache, slots, n, "slots"), n,
                                            _kv4_stream(cache, stream)))


def dg_kv4_compact(cache: Kv4Cache, stream=None):
    _check("dg_kv4_compact", lib().dg_kv4_compact(cache.ref, _kv4_stream(cache, stream)))


def _kv4_rows(fn, cache, layer, k, v, rows, stream):
    shape = (cache.n_seq, k.shape[1] if k.dim() == 4 else -1, cache.n_kv, cache.d_head)
    code, k0, k1, k2 = _kv4_tensor(cache, k, shape, "k")
    _, v0, v1, v2 = _kv4_tensor(cache, v, shape, "v", k.dtype)
    r = _pack_rows.pack(k.data_ptr(), v.data_ptr(), k0, k1, k2, v0, v1, v2, _kv4_ints(cache, rows, cache.n_seq, "rows"),
                        shape[1], code)
    _check(fn, getattr(lib(), fn)(cache.ref, layer, r, _kv4_stream(cache, stream)))


def dg_kv4_append(cache: Kv4Cache, layer, k, v, rows=None, stream=None):
    """k, v [n_seq, T, n_kv, d_head] (any strides with contiguous channels) into the last positions of every sequence;
    rows int32 [n_seq]: how many of the T rows each sequence has (None: all)."""
    _kv4_rows("dg_kv4_append", cache, layer, k, v, rows, stream)


def dg_kv4_read(cache: Kv4Cache, layer, k, v, rows=None, stream=None):
    """The values of every sequence's last positions into k, v (as dg_kv4_append takes them); rows beyond a sequence's
    count are left as they were."""
    _kv4_rows("dg_kv4_read", cache, layer, k, v, rows, stream)


def dg_kv4_attend_workspace_bytes(cache: Kv4Cache, n_q, rows) -> int:
    return int(lib().dg_kv4_attend_workspace_bytes(cache.ref, n_q, rows))


def dg_kv4_attend(cache: Kv4Cache, layer, q, out, ws, rows=None, lse=None, scale=None, causal=False, stream=None):
    """q, out [n_seq, T, n_q, d_head] (any strides with contiguous channels), lse fp32 [n_seq, T, n_q]; scale defaults to
    d_head^-0.5; rows as in dg_kv4_append."""
    shape = q.shape
    if len(shape) != 4 or shape[0] != cache.n_seq or shape[3] != cache.d_head:
        raise ValueError(f"q: expected [{cache.n_seq}, T, n_q, {cache.d_head}], got {tuple(shape)}")
    code, q0, q1, q2 = _kv4_tensor(cache, q, shape, "q")
    _, o0, o1, o2 = _kv4_tensor(cache, out, shape, "out", q.dtype)
    n, T, n_q, _ = shape
    if lse is not None and (lse.dtype != torch.float32 or lse.shape != (n, T, n_q) or lse.get_device() != cache.index
                            or not lse.is_contiguous()):
        raise ValueError(f"lse: expected a contiguous fp32 tensor {(n, T, n_q)} on {cache.device}")
    if ws.get_device() != cache.index or not ws.is_contiguous():
        raise ValueError(f"ws: expected a contiguous buffer on {cache.device}")
    a = _pack_attn.pack(q.data_ptr(), out.data_ptr(), 0 if lse is None else lse.data_ptr(),
                        _kv4_ints(cache, rows, n, "rows"), q0, q1, q2, o0, o1, o2, n_q, T, code, 1 if causal else 0,
                        cache.d_head ** -0.5 if scale is None else scale)
    _check("dg_kv4_attend", lib().dg_kv4_attend(cache.ref, layer, a, ws.data_ptr(), ws.nbytes,
                                                _kv4_stream(cache, stream)))


def dg_store_prefix_kv4(seqs: Seqs, seq, cache: Kv4Cache, slot):
    """The committed prefix of sequence seq into the cache's sequence slot (grown to that length before)."""
    _kv4_stream(cache, seqs.stream)
    _check("dg_store_prefix_kv4", lib().dg_store_prefix_kv4(seqs.handle, seq, cache.ref, slot))


def dg_load_prefix_kv4(seqs: Seqs, seq, P, cache: Kv4Cache, slot):
    """The prefix of length P that the cache's sequence slot holds as sequence seq's.  Waits for the stream; a slot of
    another length changes nothing and is what dg_kv4_error and dg_device_error tell next."""
    _kv4_stream(cache, seqs.stream)
    _check("dg_load_prefix_kv4", lib().dg_load_prefix_kv4(seqs.handle, seq, P, cache.ref, slot))


def dg_kv4_error(cache: Kv4Cache, stream=None) -> int:
    code = c_int()
    st = lib().dg_kv4_error(cache.ref, _kv4_stream(cache, stream), ctypes.byref(code))
    if st not in (DG_OK, DG_ERR_DEVICE):
        _check("dg_kv4_error", st)
    return code.value


def dg_device_error(seqs: Seqs) -> int:
    code = c_int()
    st = lib().dg_device_error(seqs.handle, ctypes.byref(code))
    if st not in (DG_OK, DG_ERR_DEVICE):
        _check("dg_device_error", st)
    return code.value


def dg_temperature(params, step) -> float:
    return float(lib().dg_temperature(ctypes.byref(params), step))


def dg_stats_reset(seqs: Seqs, timing=False):
    _check("dg_stats_reset", lib().dg_stats_reset(seqs.handle, int(bool(timing))))


def dg_stats_read(seqs: Seqs):
    """{class: (launches, device ms)} accumulated since the last reset (synchronises the stream)."""
    n = len(KERNEL_CLASSES)
    launches = (ctypes.c_longlong * n)()
    ms = (ctypes.c_double * n)()
    _check("dg_stats_read", lib().dg_stats_read(seqs.handle, launches, ms))
    return {k: (int(launches[i]), float(ms[i])) for i, k in enumerate(KERNEL_CLASSES)}
