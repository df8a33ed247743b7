"""ctypes binding of libmoe_mi355x.so: argument marshalling only.

Every function here forwards to the C entry point of the same name in
include/moe.h.  Tensors are torch tensors on the GPU (torch supplies device
memory and streams); their data pointers, sizes and the current HIP stream are
passed through unchanged.  Nothing is computed in Python, and there is no
fallback: if the library is missing or a call fails, an exception is raised.
"""
from __future__ import annotations

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmoe_mi355x.so")

MOE_F32, MOE_BF16 = 0, 1
FP4, INT2, DROPPED = 0, 1, -1

c_int, c_size_t, c_void_p, c_char_p = ctypes.c_int, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_char_p


class MoeError(RuntimeError):
    def __init__(self, name, status, msg):
        super().__init__(f"{name} failed with status {status}: {msg}")
        self.status = status


class moe_layer(ctypes.Structure):
    _fields_ = [
        ("H", c_int), ("I", c_int),
        ("fp4_base", c_void_p), ("fp4_stride", c_size_t), ("num_slots", c_int),
        ("int2_base", c_void_p), ("int2_stride", c_size_t), ("num_int2", c_int),
        ("shared", c_void_p), ("flags", c_int),
    ]


MOE_LAYER_SINGLE_LAUNCH = 1


class moe_cache_desc(ctypes.Structure):
    _fields_ = [
        ("L", c_int), ("E", c_int), ("H", c_int), ("I", c_int),
        ("num_slots", c_int), ("k", c_int), ("ladder_a", c_int), ("ladder_b", c_int),
        ("max_tokens", c_int),
        ("fp4_host", c_void_p), ("int2_host", c_void_p),
        ("fp4_arena", c_void_p), ("int2_staging", c_void_p),
        ("int2_slots", c_int), ("policy", c_int), ("lfu_decay", ctypes.c_double), ("lfu_seed", c_void_p),
        ("prefetch_slots", c_int), ("poll_us", ctypes.c_longlong),
    ]


MOE_CACHE_LRU, MOE_CACHE_LFU = 0, 1


class moe_cache_stats(ctypes.Structure):
    _fields_ = [
        ("calls", ctypes.c_int64), ("hits", ctypes.c_int64), ("misses", ctypes.c_int64),
        ("int2_uses", ctypes.c_int64), ("drops", ctypes.c_int64),
        ("bytes_h2d", ctypes.c_int64), ("evictions", ctypes.c_int64), ("int2_hits", ctypes.c_int64),
        ("prefetches", ctypes.c_int64), ("ring_hits", ctypes.c_int64), ("streamed", ctypes.c_int64),
    ]


SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1
GROUP_MAX, GROUP_TOP2 = 0, 1
GATE_NONE, GATE_CHANNEL, GATE_TOKEN, GATE_FULL = 0, 1, 2, 3
GATE_LINEAR, GATE_SIGMOID = 0, 1


class moe_router(ctypes.Structure):
    _fields_ = [
        ("E", c_int), ("k", c_int), ("scoring", c_int), ("groups", c_int), ("topk_groups", c_int),
        ("group_score", c_int), ("renorm", c_int), ("scale", ctypes.c_float),
    ]


class moe_norm(ctypes.Structure):
    _dev, _tensors = None, ()  # device of the tensors it keeps, and these
    _fields_ = [
        ("H", c_int), ("eps", ctypes.c_float), ("weight_offset", ctypes.c_float), ("wt", c_int),
        ("pre_w", c_void_p), ("post_w", c_void_p), ("post_norm", c_int), ("gate", c_int), ("gate_act", c_int),
        ("alpha", ctypes.c_float),
    ]


class moe_lora(ctypes.Structure):
    _dev, _tensors = None, ()  # device of the tensors it keeps, and these
    _fields_ = [
        ("K", c_int), ("N", c_int), ("r", c_int), ("num", c_int),
        ("a", c_void_p), ("b", c_void_p), ("scale", c_void_p), ("ranks", c_void_p),
    ]


_SIGS = {
    "moe_last_error": (c_char_p, []),
    "moe_version": (c_char_p, []),
    "moe_fp4_expert_bytes": (c_size_t, [c_int, c_int]),
    "moe_int2_expert_bytes": (c_size_t, [c_int, c_int]),
    "moe_router_logits": (c_int, [c_void_p, c_int, c_void_p, c_int, c_int, c_int, c_void_p, c_void_p]),
    "moe_route": (c_int, [c_void_p, c_int, c_int, c_int, c_void_p, c_void_p, c_void_p]),
    "moe_route_groups": (c_int, [c_void_p, c_void_p, c_int, c_void_p, c_int, c_void_p, c_void_p, c_void_p]),
    "moe_norm_in": (c_int, [c_void_p, c_void_p, c_int, c_int, c_void_p, c_int, c_void_p]),
    "moe_norm_out": (c_int, [c_void_p, c_void_p, c_int, c_void_p, c_void_p, c_int, c_int, c_void_p, c_int, c_void_p,
                             c_void_p, c_int, c_void_p]),
    "moe_lora_add": (c_int, [c_void_p, c_void_p, c_int, c_int, c_void_p, c_void_p, c_void_p, c_int, c_void_p]),
    "moe_group": (c_int, [c_void_p, c_int, c_int, c_void_p, c_void_p, c_void_p, c_void_p]),
    "moe_group_scratch_bytes": (c_size_t, [c_int, c_int]),
    "moe_group_wide": (c_int, [c_void_p, c_int, c_int, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p]),
    "moe_expert_workspace_bytes": (c_size_t, [c_int, c_int, c_int, c_int, c_int]),
    "moe_expert_workspace_sync_offset": (c_size_t, [c_int, c_int, c_int, c_int, c_int]),
    "moe_expert_forward": (c_int, [ctypes.POINTER(moe_layer), c_void_p, c_int, c_int, c_int, c_void_p, c_void_p,
                                   c_void_p, c_void_p, c_int, c_void_p, c_size_t, c_void_p]),
    "moe_layer_decode": (c_int, [ctypes.POINTER(moe_layer), c_void_p, c_int, c_void_p, c_int, c_int, c_void_p,
                                 c_void_p, c_void_p, c_int, c_void_p, c_size_t, c_void_p]),
    "moe_layer_decode_noalloc": (c_int, [ctypes.POINTER(moe_layer), c_void_p, c_int, c_void_p, c_int, c_int,
                                         c_void_p, c_void_p, c_void_p, c_int, c_void_p]),
    "moe_noalloc_scratch_bytes": (c_size_t, []),
    "moe_combine": (c_int, [c_void_p, c_void_p, c_void_p, c_int, c_int, c_int, c_int, c_void_p, c_int, c_void_p]),
    "moe_debug_dequant": (c_int, [c_void_p, c_int, c_int, c_int, c_int, c_void_p, c_void_p]),
    "moe_debug_stream_read": (c_int, [c_void_p, c_size_t, c_void_p, c_void_p]),
    "moe_tp_slice": (c_int, [c_void_p, c_size_t, c_int, c_int, c_int, c_int, c_int, c_void_p, c_size_t, c_void_p]),
    "moe_quant_mxfp8": (c_int, [c_void_p, c_int, c_int, c_void_p, c_void_p, c_void_p]),
    "moe_int2_from_fp4": (c_int, [c_void_p, c_size_t, c_int, c_int, c_int, c_void_p, c_size_t, c_void_p]),
    "moe_prefill_workspace_bytes": (c_size_t, [c_int, c_int, c_int, c_int, c_int]),
    "moe_prefill_forward": (c_int, [ctypes.POINTER(moe_layer), c_void_p, c_int, c_int, c_void_p, c_void_p,
                                    c_void_p, c_void_p, c_size_t, c_void_p]),
    "moe_pinned_alloc": (c_int, [c_size_t, ctypes.POINTER(c_void_p)]),
    "moe_pinned_free": (c_int, [c_void_p]),
    "moe_cache_create": (c_int, [ctypes.POINTER(moe_cache_desc), ctypes.POINTER(c_void_p)]),
    "moe_cache_destroy": (c_int, [c_void_p]),
    "moe_cache_reset": (c_int, [c_void_p]),
    "moe_cache_plan": (c_int, [c_void_p, c_int, c_int, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p]),
    "moe_cache_ensure": (c_int, [c_void_p, c_int, c_int, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p]),
    "moe_cache_prefetch": (c_int, [c_void_p, c_int, c_int, c_void_p, c_void_p]),
    "moe_prefill_streams": (c_int, [c_int, c_int, c_int]),
    "moe_cache_stream_layer": (c_int, [c_void_p, c_int, ctypes.POINTER(c_int), c_void_p, c_void_p]),
    "moe_cache_layer_buffer": (c_int, [c_void_p, c_int, c_void_p, ctypes.POINTER(moe_layer)]),
    "moe_cache_slot_map": (c_int, [c_void_p, c_void_p]),
    "moe_cache_get_stats": (c_int, [c_void_p, ctypes.POINTER(moe_cache_stats)]),
    "moe_cache_layer": (c_int, [c_void_p, ctypes.POINTER(moe_layer)]),
    "moe_profile_begin": (c_int, [c_int]),
    "moe_profile_end": (c_int, [ctypes.POINTER(ctypes.c_double), ctypes.POINTER(c_int), c_int]),
}

_lib = None


def load():
    """Load the built library (raises if it was not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                               "(or python -m mxfp4_routed_expert_renorm_amd.build)")
        lib = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def _check(name, st):
    if st != 0:
        raise MoeError(name, st, load().moe_last_error().decode())


def _p(t):
    return None if t is None else c_void_p(t.data_ptr())


def _stream(stream):
    if stream is not None:
        return c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))
    import torch
    return c_void_p(torch.cuda.current_stream().cuda_stream)


def _dt(t):
    import torch
    if t.dtype == torch.float32:
        return MOE_F32
    if t.dtype == torch.bfloat16:
        return MOE_BF16
    raise TypeError(f"unsupported dtype {t.dtype}")


# ---------------------------------------------------------------------- sizes

def moe_version() -> str:
    return load().moe_version().decode()


def moe_fp4_expert_bytes(H, I) -> int:
    return load().moe_fp4_expert_bytes(H, I)


def moe_int2_expert_bytes(H, I) -> int:
    return load().moe_int2_expert_bytes(H, I)


def moe_expert_workspace_bytes(H, I, T, k, has_shared) -> int:
    return load().moe_expert_workspace_bytes(H, I, T, k, int(bool(has_shared)))


def moe_expert_workspace_sync_offset(H, I, T, k, has_shared) -> int:
    return load().moe_expert_workspace_sync_offset(H, I, T, k, int(bool(has_shared)))


def moe_noalloc_scratch_bytes() -> int:
    return load().moe_noalloc_scratch_bytes()


def expert_workspace(H, I, T, k, has_shared, device="cuda"):
    """A device workspace for moe_expert_forward / moe_layer_decode, zeroed
    (the single-launch batch-1 step keeps call tags in it from call to call)."""
    import torch
    return torch.zeros(moe_expert_workspace_bytes(H, I, T, k, has_shared), dtype=torch.uint8, device=device)


# -------------------------------------------------------------------- routing

def moe_router_logits(x, w_router, logits, stream=None):
    T, H = x.shape
    E = w_router.shape[0]
    _check("moe_router_logits", load().moe_router_logits(_p(x), _dt(x), _p(w_router), T, E, H, _p(logits),
                                                         _stream(stream)))
    return logits


def moe_prefill_streams(T, k, E) -> bool:
    """The prefill crossover: stream whole expert layers when T * k >= E."""
    return bool(load().moe_prefill_streams(T, k, E))


def moe_route(logits, k, ids, w, stream=None):
    T, E = logits.shape
    _check("moe_route", load().moe_route(_p(logits), T, E, k, _p(ids), _p(w), _stream(stream)))
    return ids, w


def moe_group(keys, nkeys, counts, offsets, perm, stream=None):
    n = keys.numel()
    _check("moe_group", load().moe_group(_p(keys), n, nkeys, _p(counts), _p(offsets), _p(perm), _stream(stream)))
    return counts, offsets, perm


def moe_group_scratch_bytes(n, nkeys):
    return load().moe_group_scratch_bytes(n, nkeys)


def moe_group_wide(keys, nkeys, counts, offsets, perm, scratch, stream=None):
    n = keys.numel()
    _check("moe_group_wide", load().moe_group_wide(_p(keys), n, nkeys, _p(counts), _p(offsets), _p(perm),
                                                   _p(scratch), _stream(stream)))
    return counts, offsets, perm


# --------------------------------------------------------- around the experts
#
# These calls take a descriptor made once (make_router, make_norm, make_lora) and
# tensors that are checked on every call: shape, type, density and one device,
# which must be the current one.  Next to a launch a check costs as much as the
# call itself, so a call tests its tensors in one expression and leaves it to
# _refuse to say what is wrong.

_torch_module = _type_codes = _device_now = _stream_now = None


def _types():
    """Element types of activations and their codes."""
    global _torch_module, _type_codes, _device_now, _stream_now
    if _type_codes is None:
        import torch
        _torch_module = torch
        _device_now, _stream_now = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
        _type_codes = {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16}
    return _type_codes


def _refuse(name, descriptors, tensors):
    """Raises for the first of a call's (what, tensor, shape, types) that is not a
    dense tensor of this shape and one of these types on the current device."""
    _, first, _, _ = tensors[0]
    dev = first.get_device()
    if dev < 0:
        raise ValueError(f"{name}: tensors must be on the GPU")
    if dev != _device_now():
        raise ValueError(f"{name}: the tensors are on cuda:{dev}, the current device is cuda:{_device_now()}")
    for d in descriptors:
        if d._dev is not None and d._dev != dev:
            raise ValueError(f"{name}: the descriptor's tensors are on device {d._dev}, the call's on cuda:{dev}")
    for what, t, shape, dtypes in tensors:
        if t is None:
            continue
        if t.dtype not in dtypes:
            raise TypeError(f"{name}: {what} is {t.dtype}")
        if tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name}: {what} has shape {tuple(t.shape)}, not {tuple(shape)}")
        if not t.is_contiguous():
            raise ValueError(f"{name}: {what} must be dense (row-major, contiguous)")
        if t.get_device() != dev:
            raise ValueError(f"{name}: {what} is on {t.device}, not on cuda:{dev}")
    raise ValueError(f"{name}: arguments refused")


def _plan_tensor(name, what, t, shape, dtype):
    """Checks a tensor that a descriptor keeps (on whatever device it is)."""
    if t is None:
        return None
    if t.dtype != dtype:
        raise TypeError(f"{name}: {what} is {t.dtype}, not {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: {what} has shape {tuple(t.shape)}, not {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: {what} must be dense (row-major, contiguous)")
    return t.data_ptr()


def _one_device(name, tensors):
    devs = {t.get_device() for t in tensors if t is not None}
    if len(devs) > 1:
        raise ValueError(f"{name}: tensors on different devices")
    return devs.pop() if devs else None


def make_router(E, k, scoring="sigmoid", groups=1, topk_groups=None, group_score="top2", renorm=True,
                scale=1.0) -> moe_router:
    """Settings of moe_route_groups; topk_groups None: every group stays."""
    return moe_router(E, k, {"softmax": SCORE_SOFTMAX, "sigmoid": SCORE_SIGMOID}[scoring], groups,
                      groups if topk_groups is None else topk_groups,
                      {"max": GROUP_MAX, "top2": GROUP_TOP2}[group_score], int(bool(renorm)), scale)


def moe_route_groups(router: moe_router, logits, bias, ids, w, stream=None):
    """logits [T, E] (float32 or bfloat16), bias [E] float32 or None -> ids [T, k] int32, w [T, k] float32."""
    types, shape, dev = _type_codes or _types(), logits.shape, logits.get_device()
    T, E, k, torch = shape[0], router.E, router.k, _torch_module
    code = types.get(logits.dtype)
    picks = ids.shape
    if not (code is not None and shape == (T, E) and picks == (T, k) and picks == w.shape
            and ids.dtype is torch.int32 and w.dtype is torch.float32
            and dev >= 0 and dev == _device_now() and dev == ids.get_device() and dev == w.get_device()
            and logits.is_contiguous() and ids.is_contiguous() and w.is_contiguous()
            and (bias is None or (bias.dtype is torch.float32 and bias.shape == (E,) and bias.is_contiguous()
                                  and dev == bias.get_device()))):
        _refuse("moe_route_groups", (), (("logits", logits, (T, E), types), ("bias", bias, (E,), (torch.float32,)),
                                         ("ids", ids, (T, k), (torch.int32,)), ("w", w, (T, k), (torch.float32,))))
    st = load().moe_route_groups(ctypes.addressof(router), logits.data_ptr(), code,
                                 None if bias is None else bias.data_ptr(), T, ids.data_ptr(), w.data_ptr(),
                                 _stream_now(dev) if stream is None else _stream(stream))
    if st:
        _check("moe_route_groups", st)
    return ids, w


def make_norm(H, eps=1e-6, pre=None, post=None, post_norm=None, weight_offset=0.0, gate="none", gate_act="none",
              alpha=1.0) -> moe_norm:
    """The norms around one block: pre [H] and post [H] are their weights (of
    one type, or None: all ones); post_norm: whether the block's output is
    normed (None: where post is given).  Keeps references to the weights."""
    import torch
    some = pre if pre is not None else post
    wt = torch.float32 if some is None else some.dtype
    if wt not in (torch.float32, torch.bfloat16):
        raise TypeError(f"make_norm: weights are {wt}")
    pp = _plan_tensor("make_norm", "pre", pre, (H,), wt)
    qp = _plan_tensor("make_norm", "post", post, (H,), wt)
    n = moe_norm(H, eps, weight_offset, _types()[wt], pp, qp,
                 int(post is not None if post_norm is None else bool(post_norm)),
                 {"none": GATE_NONE, "channel": GATE_CHANNEL, "token": GATE_TOKEN, "full": GATE_FULL}[gate],
                 {"none": GATE_LINEAR, "sigmoid": GATE_SIGMOID}[gate_act], alpha)
    n._tensors = (pre, post)
    n._dev = _one_device("make_norm", n._tensors)
    return n


def moe_norm_in(norm: moe_norm, x, out, stream=None):
    """out [T, H] = RMS(x [T, H]; pre)."""
    types, shape, dev = _type_codes or _types(), x.shape, x.get_device()
    xt, ot = types.get(x.dtype), types.get(out.dtype)
    if not (xt is not None and ot is not None and shape == (shape[0], norm.H) and shape == out.shape
            and dev >= 0 and dev == _device_now() and dev == out.get_device()
            and (norm._dev is None or norm._dev == dev)
            and x.is_contiguous() and out.is_contiguous()):
        want = (shape[0], norm.H)
        _refuse("moe_norm_in", (norm,), (("x", x, want, types), ("out", out, want, types)))
    st = load().moe_norm_in(ctypes.addressof(norm), x.data_ptr(), xt, shape[0], out.data_ptr(), ot,
                            _stream_now(dev) if stream is None else _stream(stream))
    if st:
        _check("moe_norm_in", st)
    return out


def moe_norm_out(norm: moe_norm, y, residual, gate, out, next=None, next_out=None, stream=None):
    """out [T, H] = residual + alpha * act(gate) * RMS(y; post) and, with next_out
    [T, H], next_out = RMS(out before its rounding; next's pre).  gate: None, [H],
    [T] or [T, H], as the norm says.  Without next_out, next is not used."""
    types, shape, dev = _type_codes or _types(), y.shape, y.get_device()
    T, H, kind = shape[0], norm.H, norm.gate
    yt, rt = types.get(y.dtype), types.get(out.dtype)
    good = (yt is not None and rt is not None and residual.dtype is out.dtype
            and shape == (T, H) and shape == residual.shape and shape == out.shape
            and dev >= 0 and dev == _device_now() and dev == residual.get_device() and dev == out.get_device()
            and (norm._dev is None or norm._dev == dev)
            and y.is_contiguous() and residual.is_contiguous() and out.is_contiguous())
    gp = gt = np_ = nt = nd = None
    if (gate is None) != (kind == GATE_NONE):
        raise ValueError("moe_norm_out: " + ("the norm has no gate" if kind == GATE_NONE
                                             else "the norm has a gate, the call has none"))
    if gate is not None:
        gt, gp = types.get(gate.dtype), gate.data_ptr()
        good = (good and gt is not None and gate.shape == ((H,) if kind == GATE_CHANNEL else (T,) if kind == GATE_TOKEN
                                                           else shape)
                and gate.is_contiguous() and dev == gate.get_device())
    if next_out is not None:
        if next is None:
            raise ValueError("moe_norm_out: next_out needs the next block's norm")
        nt, np_, nd = types.get(next_out.dtype), next_out.data_ptr(), ctypes.addressof(next)
        good = (good and nt is not None and shape == next_out.shape and next_out.is_contiguous()
                and dev == next_out.get_device() and (next._dev is None or next._dev == dev))
    if not good:
        want = (T, H)
        _refuse("moe_norm_out", (norm,) if next_out is None else (norm, next),
                (("y", y, want, types), ("residual", residual, want, types), ("out", out, want, (residual.dtype,)),
                 ("gate", gate, ((H,) if kind == GATE_CHANNEL else (T,) if kind == GATE_TOKEN else want), types),
                 ("next_out", next_out, want, types)))
    st = load().moe_norm_out(ctypes.addressof(norm), y.data_ptr(), yt, residual.data_ptr(), gp, gt or 0, T,
                             out.data_ptr(), rt, nd, np_, nt or 0,
                             _stream_now(dev) if stream is None else _stream(stream))
    if st:
        _check("moe_norm_out", st)
    return out


def make_lora(a, b, scale=None, ranks=None) -> moe_lora:
    """A bank of adapters: a [num, r, K] and b [num, N, r] bfloat16, scale [num]
    float32 or None, ranks [num] int32 or None (all r).  Keeps references."""
    import torch
    if a.dim() != 3 or b.dim() != 3:
        raise ValueError("make_lora: a is [num, r, K] and b [num, N, r]")
    num, r, K = a.shape
    N = b.shape[1]
    m = moe_lora(K, N, r, num, _plan_tensor("make_lora", "a", a, (num, r, K), torch.bfloat16),
                 _plan_tensor("make_lora", "b", b, (num, N, r), torch.bfloat16),
                 _plan_tensor("make_lora", "scale", scale, (num,), torch.float32),
                 _plan_tensor("make_lora", "ranks", ranks, (num,), torch.int32))
    m._tensors = (a, b, scale, ranks)
    m._dev = _one_device("make_lora", m._tensors)
    return m


def moe_lora_add(lora: moe_lora, x, adapter_ids, base, out, stream=None):
    """out [T, N] = base [T, N] (or zeros) + scale * B (A x [T, K]) with each token's
    adapter, adapter_ids [T] int32 (outside the bank: none)."""
    types, shape, dev = _type_codes or _types(), x.shape, x.get_device()
    T, K, N, outs = shape[0], lora.K, lora.N, out.shape
    xt, yt = types.get(x.dtype), types.get(out.dtype)
    if not (xt is not None and yt is not None and adapter_ids.dtype is _torch_module.int32
            and shape == (T, K) and outs == (T, N) and adapter_ids.shape == (T,)
            and dev >= 0 and dev == _device_now() and dev == adapter_ids.get_device() and dev == out.get_device()
            and (lora._dev is None or lora._dev == dev)
            and x.is_contiguous() and adapter_ids.is_contiguous() and out.is_contiguous()
            and (base is None or base is out or (base.dtype is out.dtype and base.shape == outs and base.is_contiguous()
                                                 and dev == base.get_device()))):
        _refuse("moe_lora_add", (lora,),
                (("x", x, (T, K), types), ("adapter_ids", adapter_ids, (T,), (_torch_module.int32,)),
                 ("out", out, (T, N), types), ("base", base, (T, N), (out.dtype,))))
    st = load().moe_lora_add(ctypes.addressof(lora), x.data_ptr(), xt, T, adapter_ids.data_ptr(),
                             None if base is None else base.data_ptr(), out.data_ptr(), yt,
                             _stream_now(dev) if stream is None else _stream(stream))
    if st:
        _check("moe_lora_add", st)
    return out


# ----------------------------------------------------------------- expert MLP

def make_layer(H, I, fp4_base=None, fp4_stride=0, num_slots=0, int2_base=None, int2_stride=0, num_int2=0,
               shared=None, flags=0) -> moe_layer:
    """A moe_layer descriptor from device tensors (uint8 records).  The
    descriptor holds raw device pointers, so it keeps references to the tensors:
    they cannot be freed (and their memory unmapped) while it is alive."""
    lay = moe_layer(H, I, _p(fp4_base), fp4_stride, num_slots, _p(int2_base), int2_stride, num_int2, _p(shared),
                    flags)
    lay._tensors = (fp4_base, int2_base, shared)
    return lay


def moe_expert_forward(layer: moe_layer, x, T, k, slot_ids, prec, w, out, workspace, stream=None):
    ot = _dt(out)
    st = load().moe_expert_forward(ctypes.byref(layer), _p(x), _dt(x), T, k, _p(slot_ids), _p(prec), _p(w),
                                   _p(out), ot, _p(workspace), workspace.numel() * workspace.element_size(),
                                   _stream(stream))
    _check("moe_expert_forward", st)
    return out


def moe_layer_decode(layer: moe_layer, logits, x, k, ids, w, out, workspace, stream=None):
    """One token: route logits [E] (or [1, E]) and run the resident layer; ids/w [k] out."""
    E = logits.shape[-1]
    st = load().moe_layer_decode(ctypes.byref(layer), _p(logits), E, _p(x), _dt(x), k, _p(ids), _p(w), _p(out),
                                 _dt(out), _p(workspace), workspace.numel() * workspace.element_size(),
                                 _stream(stream))
    _check("moe_layer_decode", st)
    return out


def moe_layer_decode_noalloc(layer: moe_layer, logits, x, k, ids, w, out, stream=None):
    """moe_layer_decode with the library's static per-device scratch as its
    workspace (no allocation in the call)."""
    E = logits.shape[-1]
    st = load().moe_layer_decode_noalloc(ctypes.byref(layer), _p(logits), E, _p(x), _dt(x), k, _p(ids), _p(w),
                                         _p(out), _dt(out), _stream(stream))
    _check("moe_layer_decode_noalloc", st)
    return out


def moe_combine(y, w, prec, T, k, H, has_shared, out, stream=None):
    st = load().moe_combine(_p(y), _p(w), _p(prec), T, k, H, int(bool(has_shared)), _p(out), _dt(out),
                            _stream(stream))
    _check("moe_combine", st)
    return out


def moe_debug_dequant(record, H, I, prec, matrix, out, stream=None):
    _check("moe_debug_dequant", load().moe_debug_dequant(_p(record), H, I, prec, matrix, _p(out), _stream(stream)))
    return out


def moe_tp_slice(src, H, I, G, g, dst, stream=None):
    """Rank g of G's share of a bank: src uint8 [n, stride] (H, I) -> dst uint8 [n, stride'] (H, I/G)."""
    def row_stride(t):  # a size-1 leading dimension may carry any stride
        return t.stride(0) if t.shape[0] > 1 else t.shape[1]
    _check("moe_tp_slice", load().moe_tp_slice(_p(src), row_stride(src), src.shape[0], H, I, G, g, _p(dst),
                                               row_stride(dst), _stream(stream)))
    return dst


def moe_int2_from_fp4(src, H, I, dst, stream=None):
    """2-bit copies of FP4 records: src uint8 [n, stride] -> dst uint8 [n, stride'] (clip search)."""
    def row_stride(t):
        return t.stride(0) if t.shape[0] > 1 else t.shape[1]
    _check("moe_int2_from_fp4", load().moe_int2_from_fp4(_p(src), row_stride(src), src.shape[0], H, I, _p(dst),
                                                         row_stride(dst), _stream(stream)))
    return dst


def moe_debug_stream_read(buf, sink, stream=None):
    """Read every byte of the uint8 device tensor `buf` once (measurement reference)."""
    _check("moe_debug_stream_read", load().moe_debug_stream_read(_p(buf), buf.numel(), _p(sink), _stream(stream)))


# -------------------------------------------------------------------- prefill

def moe_quant_mxfp8(x, codes, scales, stream=None):
    rows, K = x.shape
    _check("moe_quant_mxfp8", load().moe_quant_mxfp8(_p(x), rows, K, _p(codes), _p(scales), _stream(stream)))
    return codes, scales


def moe_prefill_workspace_bytes(H, I, T, k, has_shared) -> int:
    return load().moe_prefill_workspace_bytes(H, I, T, k, int(bool(has_shared)))


def moe_prefill_forward(layer: moe_layer, x, k, ids, w, out, workspace, stream=None):
    T = x.shape[0]
    st = load().moe_prefill_forward(ctypes.byref(layer), _p(x), T, k, _p(ids), _p(w), _p(out), _p(workspace),
                                    workspace.numel() * workspace.element_size(), _stream(stream))
    _check("moe_prefill_forward", st)
    return out


# ----------------------------------------------------------------- slot cache

class PinnedBuffer:
    """Exact-size pinned host memory from moe_pinned_alloc, viewed as uint8."""

    def __init__(self, nbytes: int):
        import numpy as np
        p = c_void_p()
        _check("moe_pinned_alloc", load().moe_pinned_alloc(nbytes, ctypes.byref(p)))
        self.ptr, self.nbytes = p.value, nbytes
        self.array = np.ctypeslib.as_array((ctypes.c_uint8 * nbytes).from_address(self.ptr))

    def free(self):
        if self.ptr:
            self.array = None
            _check("moe_pinned_free", load().moe_pinned_free(c_void_p(self.ptr)))
            self.ptr = None


def _np_p(a):
    return None if a is None else c_void_p(a.ctypes.data)


def _addr(x):
    """Address of a torch tensor, a PinnedBuffer, an int, or None."""
    if x is None:
        return None
    if isinstance(x, PinnedBuffer):
        return c_void_p(x.ptr)
    if isinstance(x, int):
        return c_void_p(x)
    return c_void_p(x.data_ptr())


class Cache:
    """moe_cache handle.  Host banks and device buffers are supplied by the
    caller; the handle keeps references to them, so they outlive it."""

    def __init__(self, L, E, H, I, num_slots, k, a, b, max_tokens=1, fp4_host=None, int2_host=None,
                 fp4_arena=None, int2_staging=None, int2_slots=0, policy="lru", lfu_decay=1.0, lfu_seed=None,
                 prefetch_slots=0, poll_us=0):
        """lfu_seed: host float32 array [L*E] of initial use counts (copied), or None.
        prefetch_slots: staging-ring entries after the slots (fp4_arena then holds
        num_slots + prefetch_slots records).  poll_us: the host's polling budget for
        each call's picks (0: the default, < 0: no poll)."""
        import numpy as np
        seed = None if lfu_seed is None else np.ascontiguousarray(lfu_seed, dtype=np.float32).reshape(-1)
        d = moe_cache_desc(L, E, H, I, num_slots, k, a, b, max_tokens, _addr(fp4_host), _addr(int2_host),
                           _addr(fp4_arena), _addr(int2_staging), int2_slots,
                           {"lru": MOE_CACHE_LRU, "lfu": MOE_CACHE_LFU}[policy], lfu_decay,
                           None if seed is None else seed.ctypes.data, prefetch_slots, poll_us)
        h = c_void_p()
        _check("moe_cache_create", load().moe_cache_create(ctypes.byref(d), ctypes.byref(h)))
        self.h, self.L, self.E, self.k = h, L, E, k
        self._buffers = (fp4_host, int2_host, fp4_arena, int2_staging)

    def destroy(self):
        if self.h:
            _check("moe_cache_destroy", load().moe_cache_destroy(self.h))
            self.h = None

    def reset(self):
        _check("moe_cache_reset", load().moe_cache_reset(self.h))

    def plan(self, layer, ids, w):
        """Host-only policy step: ids int32 [T,k], w float32 [T,k] numpy."""
        import numpy as np
        ids = np.ascontiguousarray(ids, np.int32)
        w = np.ascontiguousarray(w, np.float32)
        T = ids.shape[0]
        slots = np.empty_like(ids)
        prec = np.empty(ids.shape, np.int8)
        wo = np.empty_like(w)
        _check("moe_cache_plan", load().moe_cache_plan(self.h, layer, T, _np_p(ids), _np_p(w), _np_p(slots),
                                                       _np_p(prec), _np_p(wo)))
        return slots, prec, wo

    def ensure(self, layer, T, ids_inout, w_inout, prec_out, compute=None, copy=None):
        st = load().moe_cache_ensure(self.h, layer, T, _p(ids_inout), _p(w_inout), _p(prec_out),
                                     _stream(compute), None if copy is None else _stream(copy))
        _check("moe_cache_ensure", st)

    def prefetch(self, layer, experts, copy=None):
        """Stage predicted experts (host int sequence, most likely first) of
        `layer` into the ring; copies go on `copy` (a torch stream; None is the
        null stream, and a cache without a device arena copies nothing)."""
        import numpy as np
        e = np.ascontiguousarray(np.asarray(experts, np.int32).reshape(-1))
        st = load().moe_cache_prefetch(self.h, layer, int(e.size), _np_p(e) if e.size else None,
                                       None if copy is None else _stream(copy))
        _check("moe_cache_prefetch", st)

    def stream_layer(self, layer, compute=None, copy=None, device=True):
        """Stream every expert of `layer` into the next layer buffer; returns
        the buffer (0 or 1).  device=False: a cache without a device arena
        (policy only, no streams touched)."""
        b = c_int(-1)
        st = load().moe_cache_stream_layer(self.h, layer, ctypes.byref(b),
                                           _stream(compute) if device else None,
                                           (None if copy is None else _stream(copy)) if device else None)
        _check("moe_cache_stream_layer", st)
        return b.value

    def layer_buffer(self, layer, compute=None) -> moe_layer:
        lay = moe_layer()
        _check("moe_cache_layer_buffer", load().moe_cache_layer_buffer(self.h, layer, _stream(compute),
                                                                       ctypes.byref(lay)))
        lay._tensors = self._buffers
        return lay

    def slot_map(self):
        import numpy as np
        m = np.empty(self.L * self.E, np.int32)
        _check("moe_cache_slot_map", load().moe_cache_slot_map(self.h, _np_p(m)))
        return m

    def stats(self) -> dict:
        s = moe_cache_stats()
        _check("moe_cache_get_stats", load().moe_cache_get_stats(self.h, ctypes.byref(s)))
        return {f: getattr(s, f) for f, _ in moe_cache_stats._fields_}

    def layer(self) -> moe_layer:
        lay = moe_layer()
        _check("moe_cache_layer", load().moe_cache_layer(self.h, ctypes.byref(lay)))
        lay._tensors = self._buffers
        return lay


# --------------------------------------------------------------------- timing

PROF_KINDS = ("route", "router_logits", "gateup", "down", "combine", "group", "plan", "quant",
              "gemm_gateup", "gemm_down", "dequant", "read", "cache", "fused", "scratch", "norm", "lora")
MOE_PROF_KINDS = 24


def moe_profile_begin(max_launches: int):
    _check("moe_profile_begin", load().moe_profile_begin(max_launches))


def moe_profile_end() -> dict:
    """{kind: (total_ms, launches)} for every kind that ran."""
    tot = (ctypes.c_double * MOE_PROF_KINDS)()
    cnt = (c_int * MOE_PROF_KINDS)()
    _check("moe_profile_end", load().moe_profile_end(tot, cnt, MOE_PROF_KINDS))
    return {PROF_KINDS[i]: (tot[i], cnt[i]) for i in range(len(PROF_KINDS)) if cnt[i] > 0}
