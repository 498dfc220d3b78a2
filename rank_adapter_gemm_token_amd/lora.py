"""Thin ctypes binding of liblora.so (include/lora.h), same names as the C ABI.

Argument marshalling only: tensors become device pointers, streams become raw
hipStream_t handles, non-zero status codes become LoraError.  Every step of
the computation runs in liblora.so's HIP kernels; nothing here computes, and
there is no fallback: importing this module fails if liblora.so is missing.
"""
import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "liblora.so")
if not os.path.exists(LIB_PATH):
    raise ImportError("liblora.so is not built (%s); run `python -m rank_adapter_gemm_token_amd.build` "
                      "or __graft_entry__.build()" % LIB_PATH)
_lib = ctypes.CDLL(LIB_PATH)

LORA_F32, LORA_F16, LORA_BF16 = 0, 1, 2
LORA_MODE_AUTO, LORA_MODE_FUSED, LORA_MODE_SEPARATE = 0, 1, 2
LORA_SEG_NONE, LORA_SEG_FUSED, LORA_SEG_SEPARATE = 0, 1, 2
LORA_BASE_ONLY = -1
LORA_MAX_SLOTS = 1024
LORA_MAX_RANK = 64
LORA_KV_MAX_HEADS = 256
LORA_KV_MAX_PAGE = 1024
LORA_ATTEND_MAX_TOKENS = 65536
LORA_ATTEND_MAX_PAGES = 1 << 26
LORA_VERIFY_MAX_SEQS = 65535
LORA_VERIFY_MAX_VOCAB = 1 << 21
LORA_VERIFY_MAX_DRAFTS = 63

LORA_OK = 0
LORA_EINVAL = -1
LORA_ETOKENS = -2
LORA_ESLOT_BUSY = -3
LORA_ESLOT_EMPTY = -4
LORA_ERANK = -5
LORA_EALPHA = -6
LORA_EQUOTA = -7
LORA_EMISMATCH = -8
LORA_ENOMEM = -9
LORA_EHIP = -10
LORA_ESCRATCH = -11
LORA_NOALLOC_SCRATCH_BYTES = 32 << 20

DTYPE_OF = {torch.float32: LORA_F32, torch.float16: LORA_F16, torch.bfloat16: LORA_BF16}
TORCH_DTYPE = {v: k for k, v in DTYPE_OF.items()}

# Every symbol include/lora.h declares, in declaration order.
EXPORTS = ["lora_pool_create", "lora_pool_destroy", "lora_set_tenant_quota", "lora_register",
           "lora_unregister", "lora_set_policy", "lora_get_policy", "lora_set_shrink_wait_polls", "lora_apply",
           "lora_apply_noalloc", "lora_route",
           "lora_last_routing",
           "lora_plan_create", "lora_plan_destroy", "lora_plan_route", "lora_apply_routed",
           "lora_loader_create", "lora_loader_destroy", "lora_load_async", "lora_load_poll", "lora_load_wait",
           "lora_residency_create", "lora_residency_destroy", "lora_residency_set_share",
           "lora_residency_acquire", "lora_residency_release", "lora_residency_stats_read",
           "lora_kv_create", "lora_kv_destroy", "lora_kv_write", "lora_kv_read", "lora_kv_poll_errors",
           "lora_attend_plan_create", "lora_attend_plan_destroy", "lora_attend_plan_set", "lora_attend",
           "lora_verifier_create", "lora_verifier_destroy", "lora_verify",
           "lora_pool_stats", "lora_tenant_bytes", "lora_poll_errors", "lora_profile_enable",
           "lora_profile_read", "lora_strerror", "lora_last_hip_error"]


class lora_stats(ctypes.Structure):
    _fields_ = [("d_in", ctypes.c_int32), ("d_out", ctypes.c_int32), ("max_rank", ctypes.c_int32),
                ("n_slots", ctypes.c_int32), ("max_tokens", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("active_slots", ctypes.c_int32), ("draining_slots", ctypes.c_int32),
                ("slot_bytes", ctypes.c_uint64), ("resident_bytes", ctypes.c_uint64),
                ("device_bytes", ctypes.c_uint64),
                ("last_tokens", ctypes.c_int32), ("last_adapters", ctypes.c_int32),
                ("last_fused_buckets", ctypes.c_int32), ("last_separate_buckets", ctypes.c_int32),
                ("last_base_only_tokens", ctypes.c_int32), ("last_invalid_tokens", ctypes.c_int32),
                ("last_lora_rows_padded", ctypes.c_int64), ("last_lora_rows_true", ctypes.c_int64),
                ("last_zero_pad_fraction", ctypes.c_double)]


class lora_residency_stats(ctypes.Structure):
    _fields_ = [("hits", ctypes.c_uint64), ("misses", ctypes.c_uint64), ("evictions", ctypes.c_uint64),
                ("resident", ctypes.c_int32), ("managed", ctypes.c_int32)]


class lora_profile(ctypes.Structure):
    _fields_ = [("calls", ctypes.c_int64), ("route_ms", ctypes.c_double), ("shrink_ms", ctypes.c_double),
                ("gemm_ms", ctypes.c_double), ("expand_ms", ctypes.c_double),
                ("kernel_ms", ctypes.c_double)]


class lora_attend_batch(ctypes.Structure):
    _fields_ = ([("n_seqs", ctypes.c_int32), ("n_groups", ctypes.c_int32)] +
                [(n, ctypes.c_void_p) for n in ("q_len", "kv_len", "group", "pages", "page0", "prefix_len",
                                                "prefix_pages", "prefix_page0")])


_vp = ctypes.c_void_p
_i = ctypes.c_int
_lib.lora_pool_create.argtypes = [_i, _i, _i, _i, _i, _i, ctypes.POINTER(_vp)]
_lib.lora_pool_destroy.argtypes = [_vp]
_lib.lora_set_tenant_quota.argtypes = [_vp, ctypes.c_int32, ctypes.c_uint64]
_lib.lora_register.argtypes = [_vp, _i, ctypes.c_int32, _vp, _vp, _i, ctypes.c_float, _vp]
_lib.lora_unregister.argtypes = [_vp, _i]
_lib.lora_set_policy.argtypes = [_vp, _i, _i]
_lib.lora_set_shrink_wait_polls.argtypes = [_vp, _i]
_lib.lora_get_policy.argtypes = [_vp, ctypes.POINTER(_i), ctypes.POINTER(_i)]
_lib.lora_apply.argtypes = [_vp, _vp, _vp, _vp, _i, _vp, _vp]
_lib.lora_apply_noalloc.argtypes = [_vp, _vp, _vp, _vp, _i, _vp, _vp]
_lib.lora_route.argtypes = [_vp, _vp, _i, _vp, _vp, _vp, _vp, _vp, _vp]
_lib.lora_last_routing.argtypes = [_vp, ctypes.POINTER(_i), _vp, _vp, _vp, _vp]
_lib.lora_plan_create.argtypes = [_i, _i, ctypes.POINTER(_vp)]
_lib.lora_plan_destroy.argtypes = [_vp]
_lib.lora_plan_route.argtypes = [_vp, _vp, _vp, _i, _vp]
_lib.lora_apply_routed.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp]
_lib.lora_loader_create.argtypes = [ctypes.c_uint64, ctypes.POINTER(_vp)]
_lib.lora_loader_destroy.argtypes = [_vp]
_lib.lora_load_async.argtypes = [_vp, _vp, _i, ctypes.c_int32, _vp, _vp, _i, ctypes.c_float,
                                 ctypes.POINTER(ctypes.c_uint64)]
_lib.lora_load_poll.argtypes = [_vp, ctypes.c_uint64, ctypes.POINTER(_i)]
_lib.lora_load_wait.argtypes = [_vp, ctypes.c_uint64]
_lib.lora_residency_create.argtypes = [_vp, _vp, _i, ctypes.POINTER(_vp)]
_lib.lora_residency_destroy.argtypes = [_vp]
_lib.lora_residency_set_share.argtypes = [_vp, ctypes.c_int32, _i]
_lib.lora_residency_acquire.argtypes = [_vp, ctypes.c_uint64, ctypes.c_int32, _vp, _vp, _i, ctypes.c_float,
                                        ctypes.POINTER(_i), ctypes.POINTER(ctypes.c_uint64)]
_lib.lora_residency_release.argtypes = [_vp, ctypes.c_uint64]
_lib.lora_residency_stats_read.argtypes = [_vp, ctypes.POINTER(lora_residency_stats)]
_i64 = ctypes.c_int64
_lib.lora_kv_create.argtypes = [_i, _i, _i, _i, _i, ctypes.POINTER(_vp)]
_lib.lora_kv_destroy.argtypes = [_vp]
_lib.lora_kv_write.argtypes = [_vp, _vp, _i64, _vp, _i64, _vp, _i, _vp]
_lib.lora_kv_read.argtypes = [_vp, _vp, _i, _vp, _vp, _vp]
_lib.lora_kv_poll_errors.argtypes = [_vp, ctypes.POINTER(ctypes.c_uint64)]
_lib.lora_attend_plan_create.argtypes = [_i, _i, _i, _i, _i, _i, _i, ctypes.POINTER(_vp)]
_lib.lora_attend_plan_destroy.argtypes = [_vp]
_lib.lora_attend_plan_set.argtypes = [_vp, _vp, ctypes.POINTER(lora_attend_batch), _vp]
_lib.lora_attend.argtypes = [_vp, _vp, _vp, _i64, ctypes.c_float, _vp, _vp, _vp]
_lib.lora_verifier_create.argtypes = [_i, ctypes.POINTER(_vp)]
_lib.lora_verifier_destroy.argtypes = [_vp]
_lib.lora_verify.argtypes = [_vp, _vp, _vp, _i, _i, _vp, _vp, _vp, _i, _i, _vp, _vp, _vp]
_lib.lora_pool_stats.argtypes = [_vp, ctypes.POINTER(lora_stats)]
_lib.lora_tenant_bytes.argtypes = [_vp, ctypes.c_int32, ctypes.POINTER(ctypes.c_uint64)]
_lib.lora_poll_errors.argtypes = [_vp, ctypes.POINTER(ctypes.c_uint64)]
_lib.lora_profile_enable.argtypes = [_vp, _i, _i]
_lib.lora_profile_read.argtypes = [_vp, ctypes.POINTER(lora_profile)]
_lib.lora_strerror.argtypes = [_i]
_lib.lora_strerror.restype = ctypes.c_char_p
_lib.lora_last_hip_error.argtypes = []
_lib.lora_last_hip_error.restype = ctypes.c_char_p
for _n in EXPORTS:
    if _n not in ("lora_strerror", "lora_last_hip_error"):
        getattr(_lib, _n).restype = ctypes.c_int


class LoraError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        text = lora_strerror(status)
        if status == LORA_EHIP:
            text += ": " + _lib.lora_last_hip_error().decode()
        super().__init__("%s failed: %s (%d)" % (where, text, status))


def _check(rc, where):
    if rc != LORA_OK:
        raise LoraError(rc, where)


def _ptr(t):
    """Device pointer of a contiguous CUDA tensor (or a raw int / None)."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError("expected a device tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return t.data_ptr()


def _stream(s):
    if s is None:
        # torch.cuda.current_stream() builds a Stream object: 2.8 us a call instead of 0.2.
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(s, int):
        return s
    return s.cuda_stream


def lora_strerror(status):
    return _lib.lora_strerror(int(status)).decode()


# Shapes of the pools created through this binding, so that a tensor of the
# wrong size or dtype is refused here instead of reaching a kernel.
_shapes = {}


def _need(t, numel, dtype, what):
    if isinstance(t, torch.Tensor):
        if t.dtype != dtype:
            raise ValueError("%s: expected %s, got %s" % (what, dtype, t.dtype))
        if t.numel() < numel:
            raise ValueError("%s: expected at least %d elements, got %d" % (what, numel, t.numel()))


def lora_pool_create(d_in, d_out, max_rank, n_slots, max_tokens, dtype):
    """Returns the pool handle (an int).  dtype: torch dtype or LORA_F32/F16/BF16."""
    if isinstance(dtype, torch.dtype):
        dtype = DTYPE_OF[dtype]
    h = _vp()
    _check(_lib.lora_pool_create(d_in, d_out, max_rank, n_slots, max_tokens, int(dtype), ctypes.byref(h)),
           "lora_pool_create")
    _shapes[h.value] = dict(d_in=d_in, d_out=d_out, R=max_rank, S=n_slots, max_T=max_tokens,
                            dtype=TORCH_DTYPE[int(dtype)])
    return h.value


def lora_pool_destroy(pool):
    _check(_lib.lora_pool_destroy(pool), "lora_pool_destroy")
    _shapes.pop(pool, None)


def lora_set_tenant_quota(pool, tenant, nbytes):
    _check(_lib.lora_set_tenant_quota(pool, tenant, nbytes), "lora_set_tenant_quota")


def lora_register(pool, slot, tenant, A, B, rank, alpha, stream=None):
    sh = _shapes.get(pool)
    if sh is not None and 0 < rank:
        _need(A, rank * sh["d_in"], sh["dtype"], "A")
        _need(B, sh["d_out"] * rank, sh["dtype"], "B")
    _check(_lib.lora_register(pool, slot, tenant, _ptr(A), _ptr(B), rank, float(alpha), _stream(stream)),
           "lora_register")


def lora_unregister(pool, slot):
    _check(_lib.lora_unregister(pool, slot), "lora_unregister")


def lora_set_policy(pool, mode, threshold):
    _check(_lib.lora_set_policy(pool, int(mode), int(threshold)), "lora_set_policy")


def lora_set_shrink_wait_polls(pool, polls):
    _check(_lib.lora_set_shrink_wait_polls(pool, int(polls)), "lora_set_shrink_wait_polls")


def lora_get_policy(pool):
    m, t = _i(), _i()
    _check(_lib.lora_get_policy(pool, ctypes.byref(m), ctypes.byref(t)), "lora_get_policy")
    return m.value, t.value


def lora_apply(pool, x, W_base, token_adapter_idx, n_tokens, y, stream=None):
    sh = _shapes.get(pool)
    if sh is not None and 0 < n_tokens <= sh["max_T"]:
        _need(x, n_tokens * sh["d_in"], sh["dtype"], "x")
        _need(W_base, sh["d_out"] * sh["d_in"], sh["dtype"], "W_base")
        _need(token_adapter_idx, n_tokens, torch.int32, "token_adapter_idx")
        _need(y, n_tokens * sh["d_out"], sh["dtype"], "y")
    _check(_lib.lora_apply(pool, _ptr(x), _ptr(W_base), _ptr(token_adapter_idx), int(n_tokens), _ptr(y),
                           _stream(stream)), "lora_apply")


def lora_apply_noalloc(pool, x, W_base, token_adapter_idx, n_tokens, y, stream=None):
    sh = _shapes.get(pool)
    if sh is not None and 0 < n_tokens <= sh["max_T"]:
        _need(x, n_tokens * sh["d_in"], sh["dtype"], "x")
        _need(W_base, sh["d_out"] * sh["d_in"], sh["dtype"], "W_base")
        _need(token_adapter_idx, n_tokens, torch.int32, "token_adapter_idx")
        _need(y, n_tokens * sh["d_out"], sh["dtype"], "y")
    _check(_lib.lora_apply_noalloc(pool, _ptr(x), _ptr(W_base), _ptr(token_adapter_idx), int(n_tokens), _ptr(y),
                                   _stream(stream)), "lora_apply_noalloc")


def lora_route(pool, token_adapter_idx, n_tokens, counts, offsets, perm, segs, n_seg, stream=None):
    sh = _shapes.get(pool)
    if sh is not None and 0 <= n_tokens <= sh["max_T"]:
        S = sh["S"]
        _need(token_adapter_idx, n_tokens, torch.int32, "token_adapter_idx")
        _need(counts, S + 2, torch.int32, "counts")
        _need(offsets, S + 3, torch.int32, "offsets")
        _need(perm, n_tokens, torch.int32, "perm")
        _need(segs, (S + 2) * 4, torch.int32, "segs")
        _need(n_seg, 1, torch.int32, "n_seg")
    _check(_lib.lora_route(pool, _ptr(token_adapter_idx), int(n_tokens), _ptr(counts), _ptr(offsets),
                           _ptr(perm), _ptr(segs), _ptr(n_seg), _stream(stream)), "lora_route")


def lora_last_routing(pool, perm, segs, n_seg, stream=None):
    """Copies the routing the pool's kernels last used into perm / segs / n_seg
    (device int32 tensors); returns that call's token count."""
    sh = _shapes.get(pool)
    if sh is not None:
        _need(segs, (sh["S"] + 2) * 4, torch.int32, "segs")
        _need(n_seg, 1, torch.int32, "n_seg")
        _need(perm, 0, torch.int32, "perm")  # the call's token count is known after it
    n = _i()
    _check(_lib.lora_last_routing(pool, ctypes.byref(n), _ptr(perm), _ptr(segs), _ptr(n_seg), _stream(stream)),
           "lora_last_routing")
    return n.value


# Plans created through this binding: capacity and the last routed batch size.
_plans = {}


def lora_plan_create(max_tokens, n_slots):
    """Returns the plan handle (an int)."""
    h = _vp()
    _check(_lib.lora_plan_create(int(max_tokens), int(n_slots), ctypes.byref(h)), "lora_plan_create")
    _plans[h.value] = dict(max_T=max_tokens, S=n_slots, T=None)
    return h.value


def lora_plan_destroy(plan):
    _check(_lib.lora_plan_destroy(plan), "lora_plan_destroy")
    _plans.pop(plan, None)


def lora_plan_route(plan, pool, token_adapter_idx, n_tokens, stream=None):
    pl = _plans.get(plan)
    if pl is not None and 0 <= n_tokens <= pl["max_T"]:
        _need(token_adapter_idx, n_tokens, torch.int32, "token_adapter_idx")
    _check(_lib.lora_plan_route(plan, pool, _ptr(token_adapter_idx), int(n_tokens), _stream(stream)),
           "lora_plan_route")
    if pl is not None:
        pl["T"] = int(n_tokens)


def lora_apply_routed(pool, plan, x, W_base, y, stream=None):
    sh, pl = _shapes.get(pool), _plans.get(plan)
    if sh is not None and pl is not None and pl["T"] is not None and 0 < pl["T"] <= sh["max_T"]:
        T = pl["T"]
        _need(x, T * sh["d_in"], sh["dtype"], "x")
        _need(W_base, sh["d_out"] * sh["d_in"], sh["dtype"], "W_base")
        _need(y, T * sh["d_out"], sh["dtype"], "y")
    _check(_lib.lora_apply_routed(pool, plan, _ptr(x), _ptr(W_base), _ptr(y), _stream(stream)),
           "lora_apply_routed")


def lora_loader_create(capacity_bytes):
    """Returns the loader handle (an int)."""
    h = _vp()
    _check(_lib.lora_loader_create(int(capacity_bytes), ctypes.byref(h)), "lora_loader_create")
    return h.value


def lora_loader_destroy(loader):
    _check(_lib.lora_loader_destroy(loader), "lora_loader_destroy")


def _host_ptr(t):
    """Host pointer of a contiguous CPU tensor (or a raw int)."""
    if isinstance(t, int):
        return t
    if t.is_cuda:
        raise ValueError("expected a host tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return t.data_ptr()


def lora_load_async(loader, pool, slot, tenant, A_host, B_host, rank, alpha):
    """Start loading host A [rank][d_in], B [d_out][rank] into `slot`; returns the ticket."""
    sh = _shapes.get(pool)
    if sh is not None and 0 < rank:
        _need(A_host, rank * sh["d_in"], sh["dtype"], "A")
        _need(B_host, sh["d_out"] * rank, sh["dtype"], "B")
    t = ctypes.c_uint64()
    _check(_lib.lora_load_async(loader, pool, int(slot), int(tenant), _host_ptr(A_host), _host_ptr(B_host),
                                int(rank), float(alpha), ctypes.byref(t)), "lora_load_async")
    return t.value


def lora_load_poll(loader, ticket):
    d = _i()
    _check(_lib.lora_load_poll(loader, int(ticket), ctypes.byref(d)), "lora_load_poll")
    return bool(d.value)


def lora_load_wait(loader, ticket):
    _check(_lib.lora_load_wait(loader, int(ticket)), "lora_load_wait")


def lora_residency_create(pool, loader, k=2):
    h = _vp()
    _check(_lib.lora_residency_create(pool, loader, int(k), ctypes.byref(h)), "lora_residency_create")
    return h.value


def lora_residency_destroy(res):
    _check(_lib.lora_residency_destroy(res), "lora_residency_destroy")


def lora_residency_set_share(res, tenant, max_slots):
    _check(_lib.lora_residency_set_share(res, int(tenant), int(max_slots)), "lora_residency_set_share")


def lora_residency_acquire(res, adapter_id, tenant, A_host, B_host, rank, alpha):
    """Returns (slot, ticket); ticket 0 for an adapter resident and committed."""
    s, t = _i(), ctypes.c_uint64()
    _check(_lib.lora_residency_acquire(res, int(adapter_id), int(tenant),
                                       None if A_host is None else _host_ptr(A_host),
                                       None if B_host is None else _host_ptr(B_host), int(rank), float(alpha),
                                       ctypes.byref(s), ctypes.byref(t)), "lora_residency_acquire")
    return s.value, t.value


def lora_residency_release(res, adapter_id):
    _check(_lib.lora_residency_release(res, int(adapter_id)), "lora_residency_release")


def lora_residency_stats_read(res):
    st = lora_residency_stats()
    _check(_lib.lora_residency_stats_read(res, ctypes.byref(st)), "lora_residency_stats_read")
    return {name: getattr(st, name) for name, _ in lora_residency_stats._fields_}


# Caches (heads, head_dim, dtype) and attention plans (heads, head_dim, tokens
# of the planned batch) created through this binding.
_kvs = {}
_attend_plans = {}


def lora_kv_create(n_pages, page_size, n_kv_heads, head_dim, dtype):
    """Returns the cache handle (an int).  dtype: torch dtype or LORA_F16/BF16."""
    if isinstance(dtype, torch.dtype):
        dtype = DTYPE_OF[dtype]
    h = _vp()
    _check(_lib.lora_kv_create(int(n_pages), int(page_size), int(n_kv_heads), int(head_dim), int(dtype),
                               ctypes.byref(h)), "lora_kv_create")
    _kvs[h.value] = (int(n_kv_heads), int(head_dim), TORCH_DTYPE[int(dtype)])
    return h.value


def lora_kv_destroy(kv):
    _check(_lib.lora_kv_destroy(kv), "lora_kv_destroy")
    _kvs.pop(kv, None)


def _rows(t, n, heads, dim, dtype, what):
    """Device pointer and token stride of an [n, heads, dim] tensor whose heads
    are contiguous within a token."""
    if t.dtype != dtype or not t.is_cuda:
        raise ValueError("%s: expected a device tensor of %s, got %s on %s" % (what, dtype, t.dtype, t.device))
    shape = t.shape
    if len(shape) != 3 or shape[0] < n or shape[1] != heads or shape[2] != dim:
        raise ValueError("%s: expected [%d, %d, %d], got %s" % (what, n, heads, dim, tuple(shape)))
    if t.is_contiguous():
        return t.data_ptr(), heads * dim
    st = t.stride()
    if st[2] != 1 or (heads > 1 and st[1] != dim):
        raise ValueError("%s: a token's heads must be contiguous, got strides %s" % (what, st))
    # A single row's stride says nothing.
    return t.data_ptr(), st[0] if shape[0] > 1 else heads * dim


def _flat(t, numel, dtype, what):
    """Device pointer of a contiguous device tensor of at least numel elements."""
    if t.dtype != dtype or not t.is_cuda or not t.is_contiguous() or t.numel() < numel:
        raise ValueError("%s: expected %d contiguous elements of %s on the device, got %s of %s on %s"
                         % (what, numel, dtype, tuple(t.shape), t.dtype, t.device))
    return t.data_ptr()


def lora_kv_write(kv, k, v, slots, n_tokens, stream=None):
    """k, v: [n_tokens, n_kv_heads, head_dim], strided over tokens; slots: device int32."""
    heads, dim, dtype = _kvs[kv]
    kp, ks = _rows(k, n_tokens, heads, dim, dtype, "k")
    vp, vs = _rows(v, n_tokens, heads, dim, dtype, "v")
    _check(_lib.lora_kv_write(kv, kp, ks, vp, vs, _flat(slots, n_tokens, torch.int32, "slots"), n_tokens,
                              _stream(stream)), "lora_kv_write")


def lora_kv_read(kv, slots, n_tokens, k, v, stream=None):
    heads, dim, dtype = _kvs[kv]
    n = n_tokens * heads * dim
    _check(_lib.lora_kv_read(kv, _flat(slots, n_tokens, torch.int32, "slots"), n_tokens, _flat(k, n, dtype, "k"),
                             _flat(v, n, dtype, "v"), _stream(stream)), "lora_kv_read")


def lora_kv_poll_errors(kv):
    v = ctypes.c_uint64()
    _check(_lib.lora_kv_poll_errors(kv, ctypes.byref(v)), "lora_kv_poll_errors")
    return v.value


def lora_attend_plan_create(max_seqs, max_groups, max_tokens, max_pages, n_heads, n_kv_heads, head_dim):
    """Returns the plan handle (an int)."""
    h = _vp()
    _check(_lib.lora_attend_plan_create(int(max_seqs), int(max_groups), int(max_tokens), int(max_pages),
                                        int(n_heads), int(n_kv_heads), int(head_dim), ctypes.byref(h)),
           "lora_attend_plan_create")
    _attend_plans[h.value] = [int(n_heads), int(head_dim), 0]
    return h.value


def lora_attend_plan_destroy(plan):
    _check(_lib.lora_attend_plan_destroy(plan), "lora_attend_plan_destroy")
    _attend_plans.pop(plan, None)


def lora_attend_plan_set(plan, kv, q_len, kv_len, group, pages, page0, prefix_len=None, prefix_pages=None,
                         prefix_page0=None, stream=None):
    """The batch's lists as host int32 tensors (lora_attend_batch in lora.h)."""
    def host(t, n, what):
        if t is None:
            if n > 0:
                raise ValueError("%s: expected %d elements, got none" % (what, n))
            return None
        if t.is_cuda or t.dtype != torch.int32 or not t.is_contiguous() or t.numel() < n:
            raise ValueError("%s: expected %d contiguous host int32 elements, got %s of %s on %s"
                             % (what, n, tuple(t.shape), t.dtype, t.device))
        return t.data_ptr()
    def lists(entries, first, n, what, first_what):
        """The entries, as many as their last bound says, and the n + 1 bounds
        (a longer tensor's further ones are not looked at)."""
        at = host(first, n + 1 if n else 0, first_what)
        return host(entries, int(first[n]) if n else 0, what), at
    n_seqs = q_len.numel()
    n_groups = 0 if prefix_len is None else prefix_len.numel()
    b = lora_attend_batch(n_seqs, n_groups, host(q_len, n_seqs, "q_len"), host(kv_len, n_seqs, "kv_len"),
                          host(group, n_seqs, "group"), *lists(pages, page0, n_seqs, "pages", "page0"),
                          host(prefix_len, n_groups, "prefix_len"),
                          *lists(prefix_pages, prefix_page0, n_groups, "prefix_pages", "prefix_page0"))
    _attend_plans[plan][2] = 0
    _check(_lib.lora_attend_plan_set(plan, kv, ctypes.byref(b), _stream(stream)), "lora_attend_plan_set")
    _attend_plans[plan][2] = int(q_len.sum())


def lora_attend(kv, plan, q, scale, out, lse=None, stream=None):
    """q, out: [tokens, n_heads, head_dim] of the planned batch, q strided over tokens."""
    heads, dim, tokens = _attend_plans[plan]
    dtype = _kvs[kv][2]
    qp, qs = _rows(q, tokens, heads, dim, dtype, "q")
    _check(_lib.lora_attend(kv, plan, qp, qs, scale, _flat(out, tokens * heads * dim, dtype, "out"),
                            None if lse is None else _flat(lse, tokens * heads, torch.float32, "lse"),
                            _stream(stream)), "lora_attend")


def lora_verifier_create(max_seqs):
    """Returns the verifier handle (an int)."""
    h = _vp()
    _check(_lib.lora_verifier_create(int(max_seqs), ctypes.byref(h)), "lora_verifier_create")
    return h.value


def lora_verifier_destroy(verifier):
    _check(_lib.lora_verifier_destroy(verifier), "lora_verifier_destroy")


def lora_verify(verifier, p_target, p_draft, draft, row0, u, n_seqs, n_rows, tokens, accepted, stream=None):
    """p_target: [n_rows, vocab]; p_draft: [n_rows - n_seqs, vocab] of the same dtype."""
    vocab, dtype = p_target.shape[-1], p_target.dtype
    n_drafts = max(0, n_rows - n_seqs)
    i32 = torch.int32
    if n_drafts > 0 and p_draft.shape[-1] != vocab:
        raise ValueError("p_draft: expected rows of the target's vocabulary, %d, got %s" % (vocab, tuple(p_draft.shape)))
    _check(_lib.lora_verify(verifier, _flat(p_target, n_rows * vocab, dtype, "p_target"),
                            _flat(p_draft, n_drafts * vocab, dtype, "p_draft"), DTYPE_OF[dtype], vocab,
                            _flat(draft, n_drafts, i32, "draft"), _flat(row0, n_seqs + 1, i32, "row0"),
                            _flat(u, n_rows, torch.float32, "u"), n_seqs, n_rows,
                            _flat(tokens, n_rows, i32, "tokens"), _flat(accepted, n_seqs, i32, "accepted"),
                            _stream(stream)), "lora_verify")


def lora_pool_stats(pool):
    s = lora_stats()
    _check(_lib.lora_pool_stats(pool, ctypes.byref(s)), "lora_pool_stats")
    return {name: getattr(s, name) for name, _ in lora_stats._fields_}


def lora_tenant_bytes(pool, tenant):
    v = ctypes.c_uint64()
    _check(_lib.lora_tenant_bytes(pool, tenant, ctypes.byref(v)), "lora_tenant_bytes")
    return v.value


def lora_poll_errors(pool):
    v = ctypes.c_uint64()
    _check(_lib.lora_poll_errors(pool, ctypes.byref(v)), "lora_poll_errors")
    return v.value


def lora_profile_enable(pool, enable, max_calls=1):
    _check(_lib.lora_profile_enable(pool, int(bool(enable)), int(max_calls)), "lora_profile_enable")


def lora_profile_read(pool):
    v = lora_profile()
    _check(_lib.lora_profile_read(pool, ctypes.byref(v)), "lora_profile_read")
    return {name: getattr(v, name) for name, _ in lora_profile._fields_}


def raw_lib():
    """The loaded CDLL, for tests that call the C ABI directly."""
    return _lib
