"""Python binding of libmoecache.so, the C ABI declared in include/moe_cache.h.

Argument marshalling only: every step of the MoE layer (routing, the cache
plan, miss uploads, the expert FFN and the combine) runs in the library's
CUDA kernels. PyTorch is used by callers for device memory and streams; here
it only supplies data pointers and the current stream. There is no CPU
fallback: if the library is missing or fails to load, using it raises.
"""
import ctypes
import os
import re

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoecache.so")
HEADER = os.path.join(_HERE, "..", "include", "moe_cache.h")

OK, ERR_INVALID, ERR_CAPACITY, ERR_CUDA, ERR_OOM, ERR_STATE, ERR_TIMEOUT = range(7)
FORMATS = {"bf16": 0, "q4_0": 1, "fp8_b128": 2, "nvfp4": 3}
POOL_MODES = {"per_layer": 0, "shared": 1}
UPLOAD_MODES = {"pull": 0, "memcpy": 1}
DECODE_MODES = {"auto": 0, "three_kernels": 1, "one_kernel": 2}
EVICTIONS = {"lru": 0, "lfu": 1}
PREFILL_MODES = {"read_only": 0, "page_in": 1}
STATUS_NAMES = {0: "MOE_OK", 1: "MOE_ERR_INVALID", 2: "MOE_ERR_CAPACITY", 3: "MOE_ERR_CUDA", 4: "MOE_ERR_OOM",
                5: "MOE_ERR_STATE", 6: "MOE_ERR_TIMEOUT"}

i32, i64, u64, dbl, vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64, ctypes.c_double, ctypes.c_void_p


class MoeConfig(ctypes.Structure):
    _fields_ = [("num_layers", i32), ("num_experts", i32), ("top_k", i32), ("hidden", i32), ("inter", i32),
                ("format", i32), ("has_shared", i32), ("pool_mode", i32), ("slots_per_layer", i32),
                ("upload_mode", i32), ("pool_bytes", dbl), ("norm_topk", i32), ("max_cache_tokens", i32),
                ("prefill_group", i32), ("max_tokens", i32), ("device", i32), ("split_decode", i32),
                ("multi_wave", i32), ("eviction", i32), ("speculate", i32), ("prefill_mode", i32),
                ("adapt_period", i32), ("adapt_step", i32), ("adapt_min_slots", i32), ("adapt_max_slots", i32)]


class BucketStats(ctypes.Structure):
    _fields_ = [("calls", u64), ("hits", u64), ("misses", u64), ("bytes_uploaded", u64), ("upload_ns", u64)]


class MoeStats(ctypes.Structure):
    _fields_ = [("bucket", BucketStats * 3), ("num_pools", i32), ("slots_per_pool", i32), ("slot_bytes", u64),
                ("record_bytes", u64), ("topk_fp64_rerank", u64), ("spec_prefetched", u64), ("spec_used", u64)]


class MoeInfo(ctypes.Structure):
    _fields_ = [("num_pools", i32), ("slots_per_pool", i32), ("slot_bytes", u64), ("slot_stride", u64),
                ("record_bytes", u64), ("pool_device_bytes", u64), ("store_host_bytes", u64),
                ("scratch_device_bytes", u64), ("fused_decode_calls", u64), ("split_decode_calls", u64)]


class KvConfig(ctypes.Structure):
    _fields_ = [("num_layers", i32), ("num_pages", i32), ("page_tokens", i32), ("q_heads", i32), ("kv_heads", i32),
                ("head_dim", i32), ("device", i32)]


class KvBatchArgs(ctypes.Structure):
    _fields_ = [("num_seqs", i32), ("table_stride", i32), ("cu_tokens", vp), ("kv_lens", vp), ("block_table", vp)]


class KvInfo(ctypes.Structure):
    _fields_ = [("page_bytes", u64), ("pool_device_bytes", u64), ("scratch_device_bytes", u64)]


NUM_STAGES = 7
STAGES = ["route", "copy", "gateup", "down", "prefill_topk", "prefill_plan", "layer"]


class MoeProfile(ctypes.Structure):
    _fields_ = [("ms", dbl * NUM_STAGES), ("launches", u64 * NUM_STAGES)]


_lib = None


def load():
    """Loads libmoecache.so (after torch, so both share one CUDA runtime)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run __graft_entry__.build() (nvcc, sm_103a) first")
    try:
        import torch  # noqa: F401  (loads the CUDA runtime torch uses)
    except ImportError:
        pass
    L = ctypes.CDLL(LIB_PATH)
    P = ctypes.POINTER
    sig = {
        "moe_config_default": (None, [P(MoeConfig)]),
        "moe_abi_version": (i32, []),
        "moe_last_error": (ctypes.c_char_p, [vp]),
        "moe_cache_create": (i32, [P(MoeConfig), vp, vp, P(vp)]),
        "moe_cache_load_experts": (i32, [vp, i32, i32, i32, vp]),
        "moe_cache_load_shared": (i32, [vp, i32, vp]),
        "moe_layer_forward": (i32, [vp, vp, i32, vp, vp, i32, vp, vp]),
        "moe_cache_stats": (i32, [vp, P(MoeStats)]),
        "moe_cache_info": (i32, [vp, P(MoeInfo)]),
        "moe_cache_trace_enable": (i32, [vp, i32]),
        "moe_cache_trace_read": (i32, [vp, vp, ctypes.c_int64, P(ctypes.c_int64), P(i32)]),
        "moe_cache_get_state": (i32, [vp, vp, vp, vp]),
        "moe_cache_read_slot": (i32, [vp, i32, i32, vp, i32, i32, vp, u64]),
        "moe_cache_profile_enable": (i32, [vp, i32]),
        "moe_cache_profile_read": (i32, [vp, P(MoeProfile)]),
        "moe_route_topk_noalloc": (i32, [vp, i32, vp, vp, i32, i32, i32, i32, vp, vp, vp]),
        "moe_cache_set_router": (i32, [vp, i32, vp, vp]),
        "moe_cache_pool_slots": (i32, [vp, vp]),
        "moe_kv_config_default": (None, [P(KvConfig)]),
        "moe_kv_create": (i32, [P(KvConfig), P(vp)]),
        "moe_kv_append": (i32, [vp, i32, vp, i64, vp, i64, vp, i64, i32, vp, vp, i32, vp, vp, vp]),
        "moe_kv_attend": (i32, [vp, i32, vp, i64, i32, vp, ctypes.c_float, vp, vp]),
        "moe_kv_read": (i32, [vp, i32, i32, vp, vp, vp, vp]),
        "moe_kv_info": (i32, [vp, P(KvInfo)]),
        "moe_kv_status": (i32, [vp]),
        "moe_kv_destroy": (i32, [vp]),
        "moe_attn_prompt": (i32, [vp, i64, vp, i64, vp, i64, i32, i32, i32, vp, vp, i32, i32, i32, ctypes.c_float, vp,
                                  vp]),
        "moe_cache_reset": (i32, [vp]),
        "moe_cache_destroy": (i32, [vp]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    _lib = L
    return L


def header_functions():
    """Names of the entry points include/moe_cache.h declares."""
    text = open(HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(moe_[a-z_]+)\s*\(", text)))


class MoeError(RuntimeError):
    def __init__(self, status, message):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


def _check(st, handle=None):
    if st != OK:
        msg = load().moe_last_error(handle)
        raise MoeError(st, msg.decode() if msg else "")


def make_config(L, E, k, H, I, fmt="bf16", pool_mode="per_layer", slots_per_layer=0, pool_bytes=0.0,
                has_shared=False, upload_mode="pull", norm_topk=True, max_cache_tokens=32, prefill_group=32,
                max_tokens=32, device=0, decode="auto", multi_wave=False, eviction="lru", speculate=False,
                prefill="read_only", adapt=None):
    c = MoeConfig()
    load().moe_config_default(ctypes.byref(c))
    c.num_layers, c.num_experts, c.top_k, c.hidden, c.inter = L, E, k, H, I
    c.format = FORMATS[fmt] if isinstance(fmt, str) else int(fmt)
    c.pool_mode = POOL_MODES[pool_mode] if isinstance(pool_mode, str) else int(pool_mode)
    c.slots_per_layer = slots_per_layer
    c.pool_bytes = float(pool_bytes)
    c.has_shared = 1 if has_shared else 0
    c.upload_mode = UPLOAD_MODES[upload_mode] if isinstance(upload_mode, str) else int(upload_mode)
    c.norm_topk = 1 if norm_topk else 0
    c.max_cache_tokens = max_cache_tokens
    c.prefill_group = prefill_group
    c.max_tokens = max_tokens
    c.device = device
    c.split_decode = DECODE_MODES[decode] if isinstance(decode, str) else int(decode)
    c.multi_wave = 1 if multi_wave else 0
    c.eviction = EVICTIONS[eviction] if isinstance(eviction, str) else int(eviction)
    c.speculate = 1 if speculate else 0
    c.prefill_mode = PREFILL_MODES[prefill] if isinstance(prefill, str) else int(prefill)
    if adapt is not None:  # (period, step, min slots, max slots); 0 takes the default
        c.adapt_period, c.adapt_step, c.adapt_min_slots, c.adapt_max_slots = (int(v) for v in adapt)
    return c


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if isinstance(t, np.ndarray):
        return t.ctypes.data
    return t.data_ptr()


def _refuse(msg):
    raise MoeError(ERR_INVALID, msg)


def _check_noalloc_args(hidden, router_w, ids, weights, top_k, bias):
    """Shapes, dtypes, devices and layouts of moe_route_topk_noalloc's tensors,
    checked before the C call: the kernel writes ids[t * k + j] and weights[t *
    k + j] for every token, so an undersized or mistyped output would be
    written out of bounds on the device."""
    import torch
    for name, t in (("hidden", hidden), ("router_w", router_w), ("ids", ids), ("weights", weights)):
        if not isinstance(t, torch.Tensor):
            _refuse(f"{name} must be a torch tensor")
    if hidden.dim() != 2 or router_w.dim() != 2:
        _refuse("hidden must be [T, H] and router_w [E, H]")
    T, H = hidden.shape
    E = router_w.shape[0]
    if router_w.shape[1] != H:
        _refuse(f"router_w has {router_w.shape[1]} columns, hidden has {H}")
    if hidden.element_size() != 2 or router_w.element_size() != 2:
        _refuse("hidden and router_w must hold 16-bit (bf16) values")
    if not isinstance(top_k, int) or top_k < 1:
        _refuse("top_k must be a positive int")
    if tuple(ids.shape) != (T, top_k) or ids.dtype != torch.int32:
        _refuse(f"ids must be int32 [{T}, {top_k}]")
    if tuple(weights.shape) != (T, top_k) or weights.dtype != torch.float32:
        _refuse(f"weights must be float32 [{T}, {top_k}]")
    tensors = [hidden, router_w, ids, weights]
    if bias is not None:
        if not isinstance(bias, torch.Tensor) or tuple(bias.shape) != (E,) or bias.dtype != torch.float32:
            _refuse(f"bias must be float32 [{E}]")
        tensors.append(bias)
    if not all(t.is_contiguous() for t in tensors):
        _refuse("every tensor must be contiguous")
    if not all(t.is_cuda for t in tensors):
        _refuse("every tensor must be on a CUDA device")
    dev = torch.cuda.current_device()
    if any(t.device.index != dev for t in tensors):
        _refuse(f"every tensor must be on the current CUDA device (cuda:{dev})")


def route_topk_noalloc(hidden, router_w, ids, weights, top_k, bias=None, norm_topk=True, stream=None):
    """moe_route_topk_noalloc: routing of T tokens into caller-provided ids
    [T, k] (int32) and weights [T, k] (fp32), with no allocation. The tensors
    are checked (shape, dtype, device, contiguity) before the call; a mismatch
    raises MoeError(ERR_INVALID) and launches nothing."""
    _check_noalloc_args(hidden, router_w, ids, weights, top_k, bias)
    T, H = hidden.shape
    E = router_w.shape[0]
    if stream is None:
        try:
            import torch
            stream = torch.cuda.current_stream().cuda_stream
        except Exception:
            stream = 0
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    _check(load().moe_route_topk_noalloc(_ptr(hidden), T, _ptr(router_w), _ptr(bias), E, H, top_k,
                                         1 if norm_topk else 0, _ptr(ids), _ptr(weights), stream or None))
    return ids, weights


class MoECache:
    """One handle of the C library (moe_cache_t*)."""

    def __init__(self, cfg, expert_host=None, shared_host=None):
        L = load()
        self.cfg = cfg
        h = vp()
        eh = sh = None
        if expert_host is not None:
            arr = (vp * cfg.num_layers)(*[_ptr(a) for a in expert_host])
            eh = ctypes.cast(arr, vp)
        if shared_host is not None:
            arr2 = (vp * cfg.num_layers)(*[_ptr(a) for a in shared_host])
            sh = ctypes.cast(arr2, vp)
        _check(L.moe_cache_create(ctypes.byref(cfg), eh, sh, ctypes.byref(h)))
        self.h = h.value

    def close(self):
        if getattr(self, "h", None):
            load().moe_cache_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def load_experts(self, layer, first, records):
        records = np.ascontiguousarray(records, dtype=np.uint8)
        n = records.shape[0] if records.ndim == 2 else 1
        _check(load().moe_cache_load_experts(self.h, layer, first, n, records.ctypes.data), self.h)

    def load_shared(self, layer, record):
        record = np.ascontiguousarray(record, dtype=np.uint8)
        _check(load().moe_cache_load_shared(self.h, layer, record.ctypes.data), self.h)

    def forward(self, hidden, router_w, layer, out, bias=None, stream=None, T=None):
        """hidden: device bf16 [T, H]; router_w: device bf16 [E, H]; bias:
        device fp32 [E] or None; out: device fp32 [T, H]. Pointers (ints) or
        tensors. stream: a cudaStream_t as int, a torch stream, or None for
        torch's current stream."""
        if T is None:
            T = hidden.shape[0]
        if stream is None:
            try:
                import torch
                stream = torch.cuda.current_stream().cuda_stream
            except Exception:
                stream = 0
        elif not isinstance(stream, int):
            stream = stream.cuda_stream
        _check(load().moe_layer_forward(self.h, _ptr(hidden), T, _ptr(router_w), _ptr(bias), layer, _ptr(out),
                                        stream or None), self.h)
        return out

    def set_router(self, layer, router_w, bias=None):
        """moe_cache_set_router: registers layer's router (device bf16 [E, H],
        device fp32 [E] or None) for speculative next-layer routing; the
        tensors must stay alive and unchanged while registered."""
        _check(load().moe_cache_set_router(self.h, layer, _ptr(router_w), _ptr(bias)), self.h)

    def pool_slots(self):
        """moe_cache_pool_slots: the slots each pool holds now."""
        n = self.info()["num_pools"]
        out = np.empty(n, dtype=np.int32)
        _check(load().moe_cache_pool_slots(self.h, out.ctypes.data), self.h)
        return out.tolist()

    def stats(self):
        s = MoeStats()
        _check(load().moe_cache_stats(self.h, ctypes.byref(s)), self.h)
        buckets = [{f: getattr(s.bucket[b], f) for f, _ in BucketStats._fields_} for b in range(3)]
        return {"buckets": buckets, "num_pools": s.num_pools, "slots_per_pool": s.slots_per_pool,
                "slot_bytes": s.slot_bytes, "record_bytes": s.record_bytes, "topk_fp64_rerank": s.topk_fp64_rerank,
                "spec_prefetched": s.spec_prefetched, "spec_used": s.spec_used}

    def info(self):
        s = MoeInfo()
        _check(load().moe_cache_info(self.h, ctypes.byref(s)), self.h)
        return {f: getattr(s, f) for f, _ in MoeInfo._fields_}

    def trace_enable(self, capacity):
        _check(load().moe_cache_trace_enable(self.h, capacity), self.h)

    def trace_read(self, max_words=1 << 24):
        buf = np.empty(max_words, dtype=np.int32)
        nw, nr = ctypes.c_int64(0), i32(0)
        _check(load().moe_cache_trace_read(self.h, buf.ctypes.data, max_words, ctypes.byref(nw), ctypes.byref(nr)),
               self.h)
        out, p = [], 0
        for _ in range(nr.value):
            layer, T, ni, nh, nf, nu = (int(v) for v in buf[p:p + 6])
            p += 6
            rec = {"layer": layer, "T": T, "n_hit": nh, "n_fill": nf, "n_uniq": nu}
            rec["ids"] = buf[p:p + ni].copy(); p += ni
            rec["slot_of"] = buf[p:p + ni].copy(); p += ni
            rec["hit_of"] = buf[p:p + ni].copy(); p += ni
            rec["fill_expert"] = buf[p:p + nf].copy(); p += nf
            rec["fill_slot"] = buf[p:p + nf].copy(); p += nf
            out.append(rec)
        return out

    def state(self):
        c = self.cfg
        info = self.info()
        npools, K = info["num_pools"], info["slots_per_pool"]
        sm = np.empty(c.num_layers * c.num_experts, dtype=np.int32)
        ko = np.empty(npools * K, dtype=np.int32)
        order = np.empty(npools * K, dtype=np.int32)
        _check(load().moe_cache_get_state(self.h, sm.ctypes.data, ko.ctypes.data, order.ctypes.data), self.h)
        return {"slot_map": sm.reshape(c.num_layers, c.num_experts), "key_of": ko.reshape(npools, K),
                "order": order.reshape(npools, K)}

    def read_slot(self, pool, slot, layer=-1, expert=-1, nbytes=None):
        """(slot bytes on the device, the store's bytes of (layer, expert) or None)."""
        if nbytes is None:
            nbytes = self.info()["slot_bytes"]
        dst = np.empty(nbytes, dtype=np.uint8)
        store = np.empty(nbytes, dtype=np.uint8) if layer >= 0 else None
        _check(load().moe_cache_read_slot(self.h, pool, slot, dst.ctypes.data, layer, expert,
                                          None if store is None else store.ctypes.data, nbytes), self.h)
        return dst, store

    def profile_enable(self, on=True):
        _check(load().moe_cache_profile_enable(self.h, 1 if on else 0), self.h)

    def profile_read(self):
        p = MoeProfile()
        _check(load().moe_cache_profile_read(self.h, ctypes.byref(p)), self.h)
        return {STAGES[i]: {"ms": p.ms[i], "launches": p.launches[i]} for i in range(NUM_STAGES)}

    def reset(self):
        _check(load().moe_cache_reset(self.h), self.h)


# ---------------------------------------------------------------------------
# The attention half of a decoder layer: a paged key/value cache in Q4_0
# blocks, attention over it, and attention of whole prompts.
# ---------------------------------------------------------------------------
_torch = None


def _need_torch():
    """The torch module, for the calls that take tensors (kept, so that a call
    does not pay for the import statement)."""
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    return _torch


def _rows(name, t, heads, dim, rows=None):
    """Checks t as bf16 rows [T, heads, dim] (or [T, heads * dim]) on the
    current CUDA device, dense within a row; returns its row stride."""
    torch = _need_torch()
    if not isinstance(t, torch.Tensor):
        _refuse(f"{name} must be a torch tensor")
    shape = t.shape
    if not (len(shape) == 3 and shape[1] == heads and shape[2] == dim or len(shape) == 2 and shape[1] == heads * dim):
        _refuse(f"{name} must be [T, {heads}, {dim}], got {tuple(shape)}")
    if rows is not None and shape[0] != rows:
        _refuse(f"{name} has {shape[0]} rows, not {rows}")
    if t.dtype is not torch.bfloat16:
        _refuse(f"{name} must be bfloat16")
    st = t.stride()
    if st[-1] != 1 or len(shape) == 3 and heads > 1 and st[1] != dim:
        _refuse(f"the heads and dims of a row of {name} must be contiguous")
    _on_device(name, t)
    return st[0] if shape[0] > 1 else heads * dim  # the stride of a single row means nothing


def _dense(name, t, heads, dim, rows):
    if _rows(name, t, heads, dim, rows) != heads * dim:
        _refuse(f"{name} must be contiguous")


def _on_device(name, t):
    if not t.is_cuda or t.get_device() != _torch.cuda.current_device():
        _refuse(f"{name} must be on the current CUDA device")


def _all_dense(bf16, dev, *tensors):
    """Whether every (tensor, shape) is a contiguous bf16 tensor of that shape
    on CUDA device dev: the usual call, accepted in a few hundred nanoseconds a
    tensor. Where it is false, _rows says what is wrong or finds the strides."""
    for t, shape in tensors:
        if t is not None and not (t.shape == shape and t.dtype is bf16 and t.is_contiguous() and t.get_device() == dev):
            return False
    return True


def _indexes(name, t, shape=None, dims=1):
    torch = _need_torch()
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.int32 or t.dim() != dims or not t.is_contiguous():
        _refuse(f"{name} must be a contiguous int32 tensor of {dims} dimension(s)")
    if shape is not None and tuple(t.shape) != shape:
        _refuse(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    _on_device(name, t)


def _batch(batch, device):
    if not isinstance(batch, KVBatch):
        _refuse("batch must be a KVBatch")
    if batch._device != device:
        _refuse(f"the batch is on CUDA device {batch._device}, the cache on {device}")
    return batch._ref


def _stream(stream, device):
    if stream is None:
        return _torch._C._cuda_getCurrentRawStream(device) or None
    return (stream if isinstance(stream, int) else stream.cuda_stream) or None


def make_kv_config(L, pages, q_heads, kv_heads, head_dim, page_tokens=64, device=0):
    c = KvConfig()
    load().moe_kv_config_default(ctypes.byref(c))
    c.num_layers, c.num_pages, c.page_tokens = L, pages, page_tokens
    c.q_heads, c.kv_heads, c.head_dim, c.device = q_heads, kv_heads, head_dim, device
    return c


class KVBatch:
    """moe_kv_batch_t: the packed sequences of a call. cu_tokens int32
    [B + 1], kv_lens int32 [B], block_table int32 [B, pages a sequence can
    have], all on the device and kept by the object; the tensors may be
    rewritten between calls (the kernels read them)."""

    def __init__(self, cu_tokens, kv_lens, block_table):
        _indexes("kv_lens", kv_lens)
        B = kv_lens.shape[0]
        if B < 1:
            _refuse("a batch needs at least one sequence")
        _indexes("cu_tokens", cu_tokens, (B + 1,))
        _indexes("block_table", block_table, dims=2)
        if block_table.shape[0] != B or block_table.shape[1] < 1:
            _refuse(f"block_table must have {B} rows of at least one page")
        self.cu_tokens, self.kv_lens, self.block_table = cu_tokens, kv_lens, block_table
        self.args = KvBatchArgs(B, block_table.shape[1], cu_tokens.data_ptr(), kv_lens.data_ptr(),
                                block_table.data_ptr())
        self._ref, self._device = ctypes.addressof(self.args), kv_lens.get_device()


class KVCache:
    """One handle of the C library (moe_kv_t*): keys and values of every layer
    in pages of Q4_0 blocks. Calls run on torch's current stream unless one is
    given."""

    def __init__(self, cfg):
        L = load()
        self.cfg = cfg
        self.h = None
        self._dims, self._device = (cfg.q_heads, cfg.kv_heads, cfg.head_dim), cfg.device
        _need_torch()
        h = vp()
        _check(L.moe_kv_create(ctypes.byref(cfg), ctypes.byref(h)))
        self.h = h.value

    def close(self):
        if getattr(self, "h", None):
            load().moe_kv_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def append(self, layer, q, k, v, batch, rope=None, q_out=None, k_out=None, stream=None):
        """moe_kv_append: k, v bf16 [T, kv_heads, head_dim] (views into a fused
        projection are fine) rotated by the rows of rope (fp32 [positions,
        head_dim], cosines then sines; None: no rotation) and stored; q bf16
        [T, q_heads, head_dim] rotated into q_out (None: keys and values only).
        Returns q_out."""
        hq, hkv, dim = self._dims
        torch = _torch
        if not (isinstance(k, torch.Tensor) and isinstance(v, torch.Tensor)):
            _refuse("k and v must be torch tensors")
        if q is not None and q_out is None:
            _refuse("q needs q_out")
        T = k.shape[0]
        qs, ks = hq * dim, hkv * dim
        vs = ks
        q_shape, kv_shape, dev = (T, hq, dim), (T, hkv, dim), self._device
        if not _all_dense(torch.bfloat16, dev, (k, kv_shape), (v, kv_shape), (k_out, kv_shape), (q, q_shape),
                          (q_out, q_shape)):
            ks = _rows("k", k, hkv, dim)
            vs = _rows("v", v, hkv, dim, T)
            if q is not None:
                qs = _rows("q", q, hq, dim, T)
                _dense("q_out", q_out, hq, dim, T)
            if k_out is not None:
                _dense("k_out", k_out, hkv, dim, T)
        rows = 0
        if rope is not None:
            if rope.dtype is not torch.float32 or rope.dim() != 2 or rope.shape[1] != dim \
                    or not rope.is_contiguous() or not rope.shape[0]:
                _refuse(f"rope must be contiguous float32 [positions, {dim}]")
            if rope.get_device() != dev:
                _refuse(f"rope must be on CUDA device {dev}")
            rows = rope.shape[0]
        _check(_lib.moe_kv_append(self.h, layer, None if q is None else q.data_ptr(), qs, k.data_ptr(), ks,
                                  v.data_ptr(), vs, T, _batch(batch, self._device), None if rope is None else rope.data_ptr(), rows,
                                  None if q is None else q_out.data_ptr(), None if k_out is None else k_out.data_ptr(),
                                  _stream(stream, self._device)))
        return q_out

    def attend(self, layer, q, batch, out, scale=None, stream=None):
        """moe_kv_attend: attention of the newest tokens, q bf16 [T, q_heads,
        head_dim] (rotated), into out. scale None: head_dim ** -0.5."""
        hq, hkv, dim = self._dims
        if not isinstance(q, _torch.Tensor) or not isinstance(out, _torch.Tensor):
            _refuse("q and out must be torch tensors")
        T = q.shape[0]
        qs = hq * dim
        if not _all_dense(_torch.bfloat16, self._device, (q, (T, hq, dim)), (out, (T, hq, dim))):
            qs = _rows("q", q, hq, dim)
            _dense("out", out, hq, dim, T)
        _check(_lib.moe_kv_attend(self.h, layer, q.data_ptr(), qs, T, _batch(batch, self._device),
                                  dim ** -0.5 if scale is None else scale, out.data_ptr(),
                                  _stream(stream, self._device)))
        return out

    def read(self, layer, batch, k_out, v_out, stream=None):
        """moe_kv_read: the batch's rows of the cache as bf16 into k_out, v_out
        [T, kv_heads, head_dim]."""
        hq, hkv, dim = self._dims
        if not isinstance(k_out, _torch.Tensor) or not isinstance(v_out, _torch.Tensor):
            _refuse("k_out and v_out must be torch tensors")
        T = k_out.shape[0]
        if not _all_dense(_torch.bfloat16, self._device, (k_out, (T, hkv, dim)), (v_out, (T, hkv, dim))):
            _dense("k_out", k_out, hkv, dim, T)
            _dense("v_out", v_out, hkv, dim, T)
        _check(_lib.moe_kv_read(self.h, layer, T, _batch(batch, self._device), k_out.data_ptr(), v_out.data_ptr(),
                                _stream(stream, self._device)))
        return k_out, v_out

    def info(self):
        s = KvInfo()
        _check(load().moe_kv_info(self.h, ctypes.byref(s)))
        return {f: getattr(s, f) for f, _ in KvInfo._fields_}

    def status(self):
        """moe_kv_status: synchronises; raises what the kernels found."""
        _check(load().moe_kv_status(self.h))


def attention_prompt(q, k, v, out, cu_q, cu_k=None, scale=None, stream=None):
    """moe_attn_prompt: causal attention of packed prompts, q bf16 [Tq, q_heads,
    D], k and v bf16 [Tk, kv_heads, D], out [Tq, q_heads, D]; cu_q, cu_k int32
    [B + 1] (cu_k None: cu_q). scale None: D ** -0.5. Returns out."""
    torch = _need_torch()
    T = torch.Tensor
    if not (isinstance(q, T) and isinstance(k, T) and isinstance(v, T) and isinstance(out, T)
            and q.dim() == k.dim() == v.dim() == out.dim() == 3):
        _refuse("q, k, v and out must be torch tensors [T, heads, head_dim]")
    Tq, hq, dim = q.shape
    Tk, hkv, _ = k.shape
    qs, ks = hq * dim, hkv * dim
    vs = ks
    dev = q.get_device()
    if dev < 0 or dev != torch._C._cuda_getDevice() or not _all_dense(
            torch.bfloat16, dev, (q, (Tq, hq, dim)), (out, (Tq, hq, dim)), (k, (Tk, hkv, dim)), (v, (Tk, hkv, dim))):
        qs = _rows("q", q, hq, dim)
        ks = _rows("k", k, hkv, dim)
        vs = _rows("v", v, hkv, dim, Tk)
        _dense("out", out, hq, dim, Tq)
    if cu_k is None:
        cu_k = cu_q
    for name, t in (("cu_q", cu_q), ("cu_k", cu_k)):  # the usual tensor first, as in _all_dense
        if not (isinstance(t, T) and t.dtype is torch.int32 and t.dim() == 1 and t.is_contiguous()
                and t.get_device() == dev):
            _indexes(name, t)
    B = cu_q.shape[0] - 1
    if cu_k.shape[0] != B + 1:
        _refuse(f"cu_k must have shape {(B + 1,)}, got {tuple(cu_k.shape)}")
    _check(load().moe_attn_prompt(q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, Tq, Tk, B, cu_q.data_ptr(),
                                  cu_k.data_ptr(), hq, hkv, dim, dim ** -0.5 if scale is None else scale,
                                  out.data_ptr(), _stream(stream, dev)))
    return out
