"""Python binding of libmoe.so -- the sparse MoE block on B200 (sm_100a).

Argument marshalling only: every step of the block runs in the library's CUDA
kernels.  Tensors are CUDA torch tensors (contiguous, row-major); the calls
enqueue on the current torch stream and never synchronise.  The library is
built in-tree (``python -m sparse_moe_layer_top_b200.build``) and loaded on
first use; every call raises if it is missing -- there is no fallback.
The C ABI sees only pointers, so every call first checks its tensors' element
types and sizes against the problem and raises ValueError, before any pointer
is taken, when a buffer is of the wrong type or too small for what the call
reads or writes.  The library launches on the current CUDA device and its
current stream: every call also requires all its tensors (and a stream it is
given) to be on one device, and runs with that device current.  What a call
allocates (outputs that were not given, a workspace) belongs to the stream the
call runs on; a caller that uses an output on another stream orders the two.

Entry points mirror ``include/moe.h``: ``router_topk``, ``permute``,
``expert_ffn``, ``combine``, ``layer_forward``, ``block_forward``,
``decode_forward``, ``rmsnorm``, ``ep_expand_ids``, ``quantize_mx4``,
``dequantize_mx4``; ``quantize_experts_mx4`` turns a block's expert weights
into the 4-bit ones of w="mx4"; ``MoELayer`` keeps a layer's weights and
workspace together; ``sparse_moe_layer_top_b200.ep`` splits the experts over
several GPUs (expert parallelism).
"""
import contextlib
import ctypes
import os
import threading
import warnings

import torch

__all__ = ["MoEError", "Problem", "BlockOptions", "router_topk", "permute", "expert_ffn", "combine", "layer_forward",
           "block_forward", "decode_forward", "decode_workspace_size", "rmsnorm", "ep_expand_ids", "forward_plan",
           "quantize_mx4", "dequantize_mx4", "quantize_experts_mx4", "mx4_scale_tiles",
           "workspace_size", "stage_workspace_size", "set_path", "set_wait_limit", "device_status",
           "last_launch_count", "bounds_checked",
           "profile_enable", "profile_read",
           "MoELayer", "lib_path", "F32", "BF16", "FP8_E4M3_B128", "MXFP4_B32", "DECODE_MAX_T"]

HERE = os.path.dirname(os.path.abspath(__file__))
# MOE_CHECKS=1 loads the bounds-checking build (python -m
# sparse_moe_layer_top_b200.build --checks), whose kernels check their
# computed indices on the device (moe_bounds_checked in include/moe.h)
lib_path = os.path.join(HERE, "libmoe_checks.so" if os.environ.get("MOE_CHECKS") == "1" else "libmoe.so")

F32, BF16, FP8_E4M3_B128, MXFP4_B32 = 0, 1, 2, 3
DECODE_MAX_T = 16  # most tokens decode_forward takes
_STATUS = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED", 3: "MOE_ERR_ALIGNMENT",
           4: "MOE_ERR_WORKSPACE_TOO_SMALL", 5: "MOE_ERR_CUDA", 6: "MOE_ERR_DEVICE_CHECK", 7: "MOE_ERR_TIMEOUT"}
EXPORTS = ("moe_check_problem", "moe_workspace_size", "moe_stage_workspace_size", "moe_router_topk",
           "moe_permute", "moe_expert_ffn", "moe_combine", "moe_layer_forward", "moe_set_path",
           "moe_device_status", "moe_last_launch_count", "moe_profile_enable", "moe_profile_read",
           "moe_last_error_string", "moe_router_topk_static", "moe_block_forward", "moe_rmsnorm",
           "moe_ep_expand_ids", "moe_forward_plan", "moe_set_wait_limit", "moe_bounds_checked",
           "moe_decode_workspace_size", "moe_decode_forward", "moe_mx4_scale_bytes", "moe_mx4_quantize",
           "moe_mx4_dequantize")


class MoEError(RuntimeError):
    def __init__(self, status, msg):
        super().__init__("%s: %s" % (_STATUS.get(status, status), msg))
        self.status = status


class Problem(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("d", ctypes.c_int32), ("E", ctypes.c_int32), ("k", ctypes.c_int32),
                ("I", ctypes.c_int32), ("I_s", ctypes.c_int32), ("act_dtype", ctypes.c_int32),
                ("w_dtype", ctypes.c_int32)]

    @classmethod
    def make(cls, T, d, E, k, I, I_s, act="bf16", w="bf16"):
        codes = {"f32": F32, "bf16": BF16, "fp8": FP8_E4M3_B128, "mx4": MXFP4_B32}
        return cls(int(T), int(d), int(E), int(k), int(I), int(I_s), codes[act], codes[w])


class BlockOptions(ctypes.Structure):
    _fields_ = [("norm_weight", ctypes.c_void_p), ("norm_eps", ctypes.c_float), ("shared_gate", ctypes.c_void_p)]


_lib = None


def lib():
    global _lib
    if _lib is None:
        if not os.path.exists(lib_path):
            raise ImportError("libmoe.so is not built (run python -m sparse_moe_layer_top_b200.build)")
        L = ctypes.CDLL(lib_path)
        P, PP = ctypes.c_void_p, ctypes.POINTER(Problem)
        S = ctypes.c_int
        L.moe_check_problem.argtypes = [PP]
        L.moe_workspace_size.argtypes = [PP]
        L.moe_workspace_size.restype = ctypes.c_size_t
        L.moe_stage_workspace_size.argtypes = [PP]
        L.moe_stage_workspace_size.restype = ctypes.c_size_t
        L.moe_router_topk.argtypes = [PP, P, P, P, P, P, P, ctypes.c_size_t, P]
        L.moe_router_topk_static.argtypes = [PP, P, P, P, P, P, P]
        L.moe_permute.argtypes = [PP, P, P, P, P, P, P, P, P, P, ctypes.c_size_t, P]
        L.moe_expert_ffn.argtypes = [PP, P, P, P, P, P, P, P, P, P, P, P, ctypes.c_size_t, P]
        L.moe_combine.argtypes = [PP, P, P, P, P, P, P]
        L.moe_layer_forward.argtypes = [PP, P, P, P, P, P, P, P, P, P, P, P, P, P, P, ctypes.c_size_t, P]
        L.moe_block_forward.argtypes = [PP, ctypes.POINTER(BlockOptions), P, P, P, P, P, P, P, P, P, P, P, P, P,
                                        P, ctypes.c_size_t, P]
        L.moe_decode_workspace_size.argtypes = [PP]
        L.moe_decode_workspace_size.restype = ctypes.c_size_t
        L.moe_decode_forward.argtypes = L.moe_block_forward.argtypes
        I64 = ctypes.c_int64
        L.moe_mx4_scale_bytes.argtypes = [I64, I64, I64]
        L.moe_mx4_scale_bytes.restype = ctypes.c_size_t
        L.moe_mx4_quantize.argtypes = [P, ctypes.c_int32, I64, I64, I64, P, P, P]
        L.moe_mx4_dequantize.argtypes = [P, P, I64, I64, I64, ctypes.c_int32, P, P]
        L.moe_ep_expand_ids.argtypes = [P, ctypes.c_int32, ctypes.c_int32, ctypes.c_int64, P, P]
        I32P = ctypes.POINTER(ctypes.c_int32)
        L.moe_forward_plan.argtypes = [PP, I32P, I32P, I32P]
        L.moe_rmsnorm.argtypes = [PP, P, P, ctypes.c_float, P, P]
        L.moe_set_path.argtypes = [ctypes.c_int]
        L.moe_set_wait_limit.argtypes = [ctypes.c_int64]
        L.moe_device_status.argtypes = [ctypes.POINTER(ctypes.c_int32)]
        L.moe_last_launch_count.restype = ctypes.c_int
        L.moe_bounds_checked.restype = ctypes.c_int
        L.moe_profile_enable.argtypes = [ctypes.c_int]
        L.moe_profile_enable.restype = ctypes.c_int
        L.moe_profile_read.argtypes = [ctypes.c_int, ctypes.POINTER(ctypes.c_float),
                                       ctypes.POINTER(ctypes.c_char_p)]
        L.moe_profile_read.restype = ctypes.c_int
        L.moe_last_error_string.restype = ctypes.c_char_p
        for f in ("moe_check_problem", "moe_router_topk", "moe_router_topk_static", "moe_permute", "moe_expert_ffn", "moe_combine",
                  "moe_layer_forward", "moe_block_forward", "moe_rmsnorm", "moe_set_path", "moe_device_status",
                  "moe_set_wait_limit", "moe_decode_forward", "moe_mx4_quantize", "moe_mx4_dequantize"):
            getattr(L, f).restype = S
        _lib = L
    return _lib


def _check(status):
    if status != 0:
        raise MoEError(status, lib().moe_last_error_string().decode())


_binding = False


def _fast():
    """The binding's C++ side (csrc/binding.cpp), which makes the regular calls of
    the latency-bound entry points without the checks below; None when it is not
    built or cannot be loaded -- the calls then go through Python, with the same
    kernels and results, which a RuntimeWarning says once."""
    global _binding
    if _binding is False:
        try:
            from . import _moe_binding as m
        except ImportError as e:
            warnings.warn("the binding's C++ side is not there (python -m sparse_moe_layer_top_b200.build): small calls "
                          "take about 10 us longer on the host; %s" % e, RuntimeWarning, stacklevel=3)
            m = None
        if m is not None:
            L = lib()
            m.bind(*(ctypes.cast(getattr(L, f), ctypes.c_void_p).value for f in (
                "moe_mx4_quantize", "moe_mx4_dequantize", "moe_expert_ffn", "moe_stage_workspace_size",
                "moe_decode_workspace_size", "moe_decode_forward")))
        _binding = m
    return _binding


def _fast_call(name, *args):
    """A regular call's result, or None: this is not one (see _fast)."""
    m = _binding if _binding is not False else _fast()
    r = getattr(m, name)(*args) if m is not None else None
    if r.__class__ is int:
        _check(r)
    return r


_F32, _I32 = (torch.float32,), (torch.int32,)
_ACT_TYPES = {F32: (torch.float32,), BF16: (torch.bfloat16,)}
_W_TYPES = {F32: (torch.float32,), BF16: (torch.bfloat16,), FP8_E4M3_B128: (torch.float8_e4m3fn, torch.uint8),
            MXFP4_B32: (torch.uint8,)}


def _need(t, name, n, dtypes, row=None):
    """t (if given) holds at least n elements of one of dtypes (None: the
    problem's type code is invalid, which the library itself reports) and, if
    it has two or more dimensions, rows of `row` elements."""
    if t is None:
        return
    if dtypes is not None and t.dtype not in dtypes:
        raise ValueError("%s: element type %s, expected %s" % (name, t.dtype, " or ".join(map(str, dtypes))))
    if t.numel() < n:
        raise ValueError("%s: %d elements, the problem needs %d" % (name, t.numel(), n))
    if row is not None and t.dim() >= 2 and t.size(-1) != row:
        raise ValueError("%s: rows of %d elements, expected %d" % (name, t.shape[-1], row))


def _need_weights(prob, wg, wu, wd, s_wg, s_wu, s_wd, scales):
    d, E, I, I_s = prob.d, prob.E, prob.I, prob.I_s
    wt = _W_TYPES.get(prob.w_dtype)
    per = 2 if prob.w_dtype == MXFP4_B32 else 1  # values per tensor element
    _need(wg, "w_gate", E * I * d // per, wt, d // per)
    _need(wu, "w_up", E * I * d // per, wt, d // per)
    _need(wd, "w_down", E * d * I // per, wt, I // per)
    if I_s > 0:
        _need(s_wg, "ws_gate", I_s * d // per, wt, d // per)
        _need(s_wu, "ws_up", I_s * d // per, wt, d // per)
        _need(s_wd, "ws_down", d * I_s // per, wt, I_s // per)
    blocks = 3 * E * (I // 128) * (d // 128) + (3 * (I_s // 128) * (d // 128) if I_s > 0 else 0)
    if prob.w_dtype == FP8_E4M3_B128:
        _need(scales, "scales", blocks, _F32)
    elif prob.w_dtype == MXFP4_B32:
        _need(scales, "scales", blocks * MX4_TILE_BYTES, (torch.uint8,))


def _nbytes(t):
    return t.numel() * t.element_size()


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensor must be on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t.data_ptr()


def _device(stream=None, **tensors):
    """The one device all given tensors are on (None if none is given); a
    given stream must belong to it.  Raises ValueError naming the tensors
    otherwise -- the library would launch on the current device with
    another device's pointers."""
    first = index = None
    same = True
    for t in tensors.values():
        if t is not None:
            i = t.get_device()
            if first is None:
                first, index = t, i
            same = same and i == index and i >= 0
    if not same:  # (or not on CUDA devices)
        devs = {}
        for name, t in tensors.items():
            if t is not None:
                devs.setdefault(t.device, []).append(name)
        if len(devs) > 1:
            raise ValueError("tensors on different devices: " +
                             "; ".join("%s on %s" % (", ".join(n), d) for d, n in devs.items()))
    dev = None if first is None else first.device
    if stream is not None and dev is not None and dev.type == "cuda" and stream.device != dev:
        raise ValueError("stream on %s, tensors on %s" % (stream.device, dev))
    return dev


_NOTHING = contextlib.nullcontext()


def _current(dev):
    """A context in which `dev` is the current CUDA device (nothing to do
    for a non-CUDA device: the pointer step rejects its tensors)."""
    if dev is not None and dev.type == "cuda" and dev.index != torch.cuda.current_device():
        return torch.cuda.device(dev)
    return _NOTHING


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream=None):
    """Handle of the stream, by default torch's current one on the current device."""
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None and torch.cuda.is_initialized():  # without building a Stream object (3 us)
        return _raw_stream(torch.cuda.current_device())
    return torch.cuda.current_stream().cuda_stream


def _act(prob):
    return torch.float32 if prob.act_dtype == F32 else torch.bfloat16


def workspace_size(prob):
    return lib().moe_workspace_size(ctypes.byref(prob))


def stage_workspace_size(prob):
    return lib().moe_stage_workspace_size(ctypes.byref(prob))


def check_problem(prob):
    _check(lib().moe_check_problem(ctypes.byref(prob)))


def set_path(path):
    """0 automatic, 1 SIMT kernels only, 2 row-tiled tensor-core expert GEMMs,
    3 weight-row tensor-core expert GEMMs, 4 row-tiled on 2-CTA clusters,
    5 split: groups of 256 rows or more on 2-CTA clusters, the others in
    weight-row form (on request only), 6 on 2-CTA clusters with the tokens as
    the MMA's N (tiles of up to 256 rows, padded to 16)."""
    _check(lib().moe_set_path(int(path)))


def set_wait_limit(cycles=0):
    """Bound, in SM cycles, of the kernels' pipeline waits on the current
    device (0: the default, about 2 s).  Synchronous; call it with no library
    work in flight."""
    _check(lib().moe_set_wait_limit(int(cycles)))


def device_status():
    """(status, detail) of the device status word, which is then cleared (synchronises)."""
    d = ctypes.c_int32(0)
    s = lib().moe_device_status(ctypes.byref(d))
    return s, d.value


def bounds_checked():
    """True when the loaded library is the bounds-checking build."""
    return bool(lib().moe_bounds_checked())


def last_launch_count():
    return lib().moe_last_launch_count()


def profile_enable(mode=1):
    """1: bracket every library kernel launch of this thread with CUDA events;
    2: only the tensor-core GEMM launches; 0: off."""
    _check(lib().moe_profile_enable(int(mode)))


def profile_read(max_launches=4096):
    """[(kernel name, device ms), ...] of the launches recorded since the last
    read (waits for them), in launch order."""
    ms = (ctypes.c_float * max_launches)()
    names = (ctypes.c_char_p * max_launches)()
    n = lib().moe_profile_read(max_launches, ms, names)
    return [(names[i].decode(), float(ms[i])) for i in range(n)]


def _alloc(stream):
    """A context in which new tensors belong to `stream`, the stream that uses
    them first (nothing to do for None, the current one)."""
    return torch.cuda.stream(stream) if stream is not None else _NOTHING


def _ws(nbytes, device, ws):
    if ws is None:
        ws = torch.empty(max(int(nbytes), 1), dtype=torch.uint8, device=device)
    return ws


def router_topk(prob, x, w_router, bias=None, topk_ids=None, topk_w=None, ws=None, stream=None):
    T, k = prob.T, prob.k
    a = _ACT_TYPES.get(prob.act_dtype)
    _need(x, "x", T * prob.d, a, prob.d)
    _need(w_router, "w_router", prob.E * prob.d, a, prob.d)
    _need(bias, "router_bias", prob.E, _F32)
    _need(topk_ids, "topk_ids", T * k, _I32, k)
    _need(topk_w, "topk_w", T * k, _F32, k)
    dev = _device(stream, x=x, w_router=w_router, router_bias=bias, topk_ids=topk_ids, topk_w=topk_w, ws=ws)
    with _current(dev), _alloc(stream):
        if topk_ids is None:
            topk_ids = torch.empty((T, k), dtype=torch.int32, device=x.device)
        if topk_w is None:
            topk_w = torch.empty((T, k), dtype=torch.float32, device=x.device)
        ws = _ws(stage_workspace_size(prob), x.device, ws)
        _check(lib().moe_router_topk(ctypes.byref(prob), _ptr(x), _ptr(w_router), _ptr(bias), _ptr(topk_ids),
                                     _ptr(topk_w), _ptr(ws), _nbytes(ws), _stream(stream)))
    return topk_ids, topk_w


def rows_total(prob):
    return prob.T * prob.k + (prob.T if prob.I_s > 0 else 0)


def permute(prob, x, topk_ids, topk_w, ws=None, stream=None):
    """-> dict(x_perm, row_tok, row_w, pos, offs)."""
    _need(x, "x", prob.T * prob.d, _ACT_TYPES.get(prob.act_dtype), prob.d)
    _need(topk_ids, "topk_ids", prob.T * prob.k, _I32, prob.k)
    _need(topk_w, "topk_w", prob.T * prob.k, _F32, prob.k)
    cur = _device(stream, x=x, topk_ids=topk_ids, topk_w=topk_w, ws=ws)
    dev = x.device
    Rp = rows_total(prob)
    with _current(cur), _alloc(stream):
        out = dict(x_perm=torch.empty((Rp, prob.d), dtype=_act(prob), device=dev),
                   row_tok=torch.empty(Rp, dtype=torch.int32, device=dev),
                   row_w=torch.empty(Rp, dtype=torch.float32, device=dev),
                   pos=torch.empty((prob.T, prob.k), dtype=torch.int32, device=dev),
                   offs=torch.empty(prob.E + 2, dtype=torch.int32, device=dev))
        ws = _ws(stage_workspace_size(prob), dev, ws)
        _check(lib().moe_permute(ctypes.byref(prob), _ptr(x), _ptr(topk_ids), _ptr(topk_w), _ptr(out["x_perm"]),
                                 _ptr(out["row_tok"]), _ptr(out["row_w"]), _ptr(out["pos"]), _ptr(out["offs"]),
                                 _ptr(ws), _nbytes(ws), _stream(stream)))
    return out


def expert_ffn(prob, x_perm, offs, wg, wu, wd, s_wg=None, s_wu=None, s_wd=None, scales=None, y_perm=None,
               ws=None, stream=None):
    if stream is None:
        r = _fast_call("expert_ffn", prob, x_perm, offs, wg, wu, wd, s_wg, s_wu, s_wd, scales, y_perm, ws)
        if r is not None:
            return r
    a, Rp = _ACT_TYPES.get(prob.act_dtype), rows_total(prob)
    _need(x_perm, "x_perm", Rp * prob.d, a, prob.d)
    _need(offs, "offs", prob.E + 2, _I32)
    _need_weights(prob, wg, wu, wd, s_wg, s_wu, s_wd, scales)
    _need(y_perm, "y_perm", Rp * prob.d, a, prob.d)
    cur = _device(stream, x_perm=x_perm, offs=offs, w_gate=wg, w_up=wu, w_down=wd, ws_gate=s_wg, ws_up=s_wu,
                  ws_down=s_wd, scales=scales, y_perm=y_perm, ws=ws)
    dev = x_perm.device
    with _current(cur), _alloc(stream):
        if y_perm is None:
            y_perm = torch.empty((x_perm.shape[0], prob.d), dtype=_act(prob), device=dev)
        ws = _ws(stage_workspace_size(prob), dev, ws)
        _check(lib().moe_expert_ffn(ctypes.byref(prob), _ptr(x_perm), _ptr(offs), _ptr(wg), _ptr(wu), _ptr(wd),
                                    _ptr(s_wg), _ptr(s_wu), _ptr(s_wd), _ptr(scales), _ptr(y_perm), _ptr(ws),
                                    _nbytes(ws), _stream(stream)))
    return y_perm


def combine(prob, y_perm, pos, topk_w, offs, y=None, stream=None):
    a = _ACT_TYPES.get(prob.act_dtype)
    _need(y_perm, "y_perm", rows_total(prob) * prob.d, a, prob.d)
    _need(pos, "pos", prob.T * prob.k, _I32, prob.k)
    _need(topk_w, "topk_w", prob.T * prob.k, _F32, prob.k)
    _need(offs, "offs", prob.E + 2, _I32)
    _need(y, "y", prob.T * prob.d, a, prob.d)
    cur = _device(stream, y_perm=y_perm, pos=pos, topk_w=topk_w, offs=offs, y=y)
    with _current(cur), _alloc(stream):
        if y is None:
            y = torch.empty((prob.T, prob.d), dtype=_act(prob), device=y_perm.device)
        _check(lib().moe_combine(ctypes.byref(prob), _ptr(y_perm), _ptr(pos), _ptr(topk_w), _ptr(offs), _ptr(y),
                                 _stream(stream)))
    return y


def _need_params(prob, w_router, bias, wg, wu, wd, s_wg, s_wu, s_wd, scales, norm_weight=None, shared_gate=None):
    """The block's parameters (independent of the token count)."""
    a = _ACT_TYPES.get(prob.act_dtype)
    _need(w_router, "w_router", prob.E * prob.d, a, prob.d)
    _need(bias, "router_bias", prob.E, _F32)
    _need_weights(prob, wg, wu, wd, s_wg, s_wu, s_wd, scales)
    _need(norm_weight, "norm_weight", prob.d, a)
    _need(shared_gate, "shared_gate", prob.d, a)


def _need_tokens(prob, x, y, topk_ids, topk_w):
    """One call's token buffers."""
    T, d, k = prob.T, prob.d, prob.k
    a = _ACT_TYPES.get(prob.act_dtype)
    _need(x, "x", T * d, a, d)
    _need(y, "y", T * d, a, d)
    _need(topk_ids, "topk_ids", T * k, _I32, k)
    _need(topk_w, "topk_w", T * k, _F32, k)


def _forward(prob, x, w_router, bias, wg, wu, wd, s_wg, s_wu, s_wd, scales, norm_weight, norm_eps, shared_gate, y,
             topk_ids, topk_w, ws, stream, block):
    """The fused forward on checked arguments (moe_block_forward when `block`)."""
    cur = _device(stream, x=x, w_router=w_router, router_bias=bias, w_gate=wg, w_up=wu, w_down=wd, ws_gate=s_wg,
                  ws_up=s_wu, ws_down=s_wd, scales=scales, norm_weight=norm_weight, shared_gate=shared_gate, y=y,
                  topk_ids=topk_ids, topk_w=topk_w, ws=ws)
    with _current(cur), _alloc(stream):
        if y is None:
            y = torch.empty((prob.T, prob.d), dtype=_act(prob), device=x.device)
        ws = _ws(workspace_size(prob), x.device, ws)
        _forward_call(prob, x, w_router, bias, wg, wu, wd, s_wg, s_wu, s_wd, scales, norm_weight, norm_eps,
                      shared_gate, y, topk_ids, topk_w, ws, stream, block)
    return y


def _forward_call(prob, x, w_router, bias, wg, wu, wd, s_wg, s_wu, s_wd, scales, norm_weight, norm_eps, shared_gate,
                  y, topk_ids, topk_w, ws, stream, block):
    if block:
        opt = BlockOptions(_ptr(norm_weight), float(norm_eps), _ptr(shared_gate))
        _check(lib().moe_block_forward(ctypes.byref(prob), ctypes.byref(opt), _ptr(x), _ptr(w_router), _ptr(bias),
                                       _ptr(wg), _ptr(wu), _ptr(wd), _ptr(s_wg), _ptr(s_wu), _ptr(s_wd),
                                       _ptr(scales), _ptr(y), _ptr(topk_ids), _ptr(topk_w), _ptr(ws), _nbytes(ws),
                                       _stream(stream)))
    else:
        _check(lib().moe_layer_forward(ctypes.byref(prob), _ptr(x), _ptr(w_router), _ptr(bias), _ptr(wg), _ptr(wu),
                                       _ptr(wd), _ptr(s_wg), _ptr(s_wu), _ptr(s_wd), _ptr(scales), _ptr(y),
                                       _ptr(topk_ids), _ptr(topk_w), _ptr(ws), _nbytes(ws), _stream(stream)))


def layer_forward(prob, x, w_router, bias, wg, wu, wd, s_wg=None, s_wu=None, s_wd=None, scales=None, y=None,
                  topk_ids=None, topk_w=None, ws=None, stream=None):
    _need_params(prob, w_router, bias, wg, wu, wd, s_wg, s_wu, s_wd, scales)
    _need_tokens(prob, x, y, topk_ids, topk_w)
    return _forward(prob, x, w_router, bias, wg, wu, wd, s_wg, s_wu, s_wd, scales, None, 0.0, None, y, topk_ids,
                    topk_w, ws, stream, block=False)


def block_forward(prob, x, w_router, bias, wg, wu, wd, s_wg=None, s_wu=None, s_wd=None, scales=None,
                  norm_weight=None, norm_eps=1e-6, shared_gate=None, y=None, topk_ids=None, topk_w=None, ws=None,
                  stream=None):
    """layer_forward with the block's neighbours: zero-centred RMSNorm of x
    (norm_weight [d]) and a sigmoid gate on the shared expert (shared_gate [d])."""
    _need_params(prob, w_router, bias, wg, wu, wd, s_wg, s_wu, s_wd, scales, norm_weight, shared_gate)
    _need_tokens(prob, x, y, topk_ids, topk_w)
    return _forward(prob, x, w_router, bias, wg, wu, wd, s_wg, s_wu, s_wd, scales, norm_weight, norm_eps,
                    shared_gate, y, topk_ids, topk_w, ws, stream, block=True)


def rmsnorm(prob, x, norm_weight, eps=1e-6, out=None, stream=None):
    """Zero-centred RMSNorm of the rows of x: x / sqrt(mean x^2 + eps) * (1 + norm_weight)."""
    a = _ACT_TYPES.get(prob.act_dtype)
    _need(x, "x", prob.T * prob.d, a, prob.d)
    _need(norm_weight, "norm_weight", prob.d, a)
    _need(out, "out", prob.T * prob.d, a, prob.d)
    cur = _device(stream, x=x, norm_weight=norm_weight, out=out)
    with _current(cur), _alloc(stream):
        if out is None:
            out = torch.empty_like(x)
        _check(lib().moe_rmsnorm(ctypes.byref(prob), _ptr(x), _ptr(norm_weight), float(eps), _ptr(out),
                                 _stream(stream)))
    return out


EXPERT_FORMS = ("simt", "rows", "weight_rows", "cta_pairs", "split", "cta_pairs_tokens_n", "mx4")


def forward_plan(prob):
    """What the fused forward launches for `prob` under the current path,
    decided on the host: dict(expert_form, router_selects, gathered)."""
    f, r, g = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32()
    _check(lib().moe_forward_plan(ctypes.byref(prob), ctypes.byref(f), ctypes.byref(r), ctypes.byref(g)))
    return {"expert_form": EXPERT_FORMS[f.value], "router_selects": bool(r.value), "gathered": bool(g.value)}


def ep_expand_ids(counts, G, E_local, R, ids=None, stream=None):
    """Expert parallelism, receive side: the local expert (int32 [R]) of every
    received row, rows arriving as blocks (source s, local expert e) in that
    order with counts[s * E_local + e] rows each (int32, on the device)."""
    _need(counts, "counts", int(G) * int(E_local), _I32)
    _need(ids, "ids", int(R), _I32)
    cur = _device(stream, counts=counts, ids=ids)
    with _current(cur), _alloc(stream):
        if ids is None:
            ids = torch.empty(max(int(R), 0), dtype=torch.int32, device=counts.device)
        _check(lib().moe_ep_expand_ids(_ptr(counts), int(G), int(E_local), int(R), _ptr(ids), _stream(stream)))
    return ids


MX4_TILE_BYTES = 512  # scale bytes of 128 x 128 values
_MX4_FLOAT = {torch.float32: F32, torch.bfloat16: BF16}


def _mx4_shape(shape):
    """(batch, rows, cols) of a stack of matrices."""
    if len(shape) < 2:
        raise ValueError("x: a matrix or a stack of matrices, got %d dimension(s)" % len(shape))
    batch = 1
    for n in shape[:-2]:
        batch *= n
    return batch, shape[-2], shape[-1]


def _mx4_scale_shape(shape):
    return tuple(shape[:-2]) + ((shape[-2] + 127) // 128, (shape[-1] + 127) // 128, MX4_TILE_BYTES)


def quantize_mx4(x, codes=None, scales=None, stream=None):
    """Microscaled 4-bit codes of x [..., rows, cols] (bf16 or fp32, cols a
    multiple of 32) -> (codes uint8 [..., rows, cols / 2], scales uint8
    [..., ceil(rows / 128), ceil(cols / 128), 512]); the layouts and the
    rounding are those of moe_mx4_quantize in include/moe.h."""
    if stream is None:
        r = _fast_call("quantize", x, codes, scales)
        if r is not None:
            return r
    batch, rows, cols = _mx4_shape(x.shape)
    if x.dtype not in _MX4_FLOAT:
        raise ValueError("x: element type %s, expected torch.float32 or torch.bfloat16" % x.dtype)
    if cols <= 0 or cols % 32:
        raise ValueError("x: rows of %d elements, expected a multiple of 32" % cols)
    sshape = _mx4_scale_shape(x.shape)
    n = batch * sshape[-3] * sshape[-2] * MX4_TILE_BYTES
    _need(codes, "codes", batch * rows * cols // 2, (torch.uint8,), cols // 2)
    _need(scales, "scales", n, (torch.uint8,), MX4_TILE_BYTES)
    cur = _device(stream, x=x, codes=codes, scales=scales)
    with _current(cur), _alloc(stream):
        if codes is None:
            codes = torch.empty(tuple(x.shape[:-1]) + (cols // 2,), dtype=torch.uint8, device=x.device)
        if scales is None:
            scales = torch.empty(sshape, dtype=torch.uint8, device=x.device)
        _check(lib().moe_mx4_quantize(_ptr(x), _MX4_FLOAT[x.dtype], batch, rows, cols, _ptr(codes), _ptr(scales),
                                      _stream(stream)))
    return codes, scales


def dequantize_mx4(codes, scales, out=None, dtype=torch.bfloat16, stream=None):
    """The values codes * scale of quantize_mx4's outputs, in bf16 or fp32 (exact)."""
    if stream is None and dtype in _MX4_FLOAT:
        r = _fast_call("dequantize", codes, scales, out, dtype is torch.float32)
        if r is not None:
            return r
    if codes.dtype != torch.uint8:
        raise ValueError("codes: element type %s, expected torch.uint8" % codes.dtype)
    shape = _mx4_shape(codes.shape) and tuple(codes.shape[:-1]) + (2 * codes.shape[-1],)
    batch, rows, cols = _mx4_shape(shape)
    if cols <= 0 or cols % 32:
        raise ValueError("codes: rows of %d bytes, expected a multiple of 16" % codes.shape[-1])
    if out is not None:
        dtype = out.dtype
    if dtype not in _MX4_FLOAT:
        raise ValueError("out: element type %s, expected torch.float32 or torch.bfloat16" % dtype)
    sshape = _mx4_scale_shape(shape)
    _need(scales, "scales", batch * sshape[-3] * sshape[-2] * MX4_TILE_BYTES, (torch.uint8,))
    _need(out, "out", batch * rows * cols, (dtype,), cols)
    cur = _device(stream, codes=codes, scales=scales, out=out)
    with _current(cur), _alloc(stream):
        if out is None:
            out = torch.empty(shape, dtype=dtype, device=codes.device)
        _check(lib().moe_mx4_dequantize(_ptr(codes), _ptr(scales), batch, rows, cols, _MX4_FLOAT[dtype], _ptr(out),
                                        _stream(stream)))
    return out


def mx4_scale_tiles(scales):
    """Row-major scale bytes [..., rows, cols / 32] (how checkpoints usually
    keep them) in the tile layout of quantize_mx4; rows and cols multiples of 128."""
    if scales.dtype != torch.uint8 or scales.dim() < 2 or scales.shape[-2] % 128 or scales.shape[-1] % 4:
        raise ValueError("scales: uint8 [..., rows, cols / 32] with rows and cols multiples of 128")
    lead, n = scales.shape[:-2], scales.dim() - 2
    t = scales.reshape(lead + (scales.shape[-2] // 128, 4, 32, scales.shape[-1] // 4, 4))
    t = t.permute(tuple(range(n)) + (n, n + 3, n + 2, n + 1, n + 4))
    return t.reshape(lead + (scales.shape[-2] // 128, scales.shape[-1] // 4, MX4_TILE_BYTES)).contiguous()


def quantize_experts_mx4(wg, wu, wd, s_wg=None, s_wu=None, s_wd=None, stream=None):
    """A block's expert weights in 4 bits: the six code tensors (None where the
    shared expert's are None), then the packed scales, as layer_forward,
    decode_forward and MoELayer take them with w="mx4"."""
    codes, scales = [], []
    for w in (wg, wu, wd, s_wg, s_wu, s_wd):
        if w is None:
            codes.append(None)
            continue
        if w.shape[-1] % 128 or w.shape[-2] % 128:
            raise ValueError("expert weights %s: the block needs multiples of 128" % (tuple(w.shape),))
        q, s = quantize_mx4(w, stream=stream)
        codes.append(q)
        scales.append(s.reshape(-1))
    with _current(wg.device), _alloc(stream):
        packed = torch.cat(scales)
    return (*codes, packed)


def decode_workspace_size(prob):
    return lib().moe_decode_workspace_size(ctypes.byref(prob))


def decode_forward(prob, x, w_router, bias, wg, wu, wd, s_wg=None, s_wu=None, s_wd=None, scales=None,
                   norm_weight=None, norm_eps=1e-6, shared_gate=None, y=None, topk_ids=None, topk_w=None, ws=None,
                   stream=None):
    """block_forward for at most DECODE_MAX_T tokens in two kernels: the latency
    form.  ws: decode_workspace_size bytes."""
    if stream is None:
        r = _fast_call("decode", prob, x, w_router, bias, wg, wu, wd, s_wg, s_wu, s_wd, scales, norm_weight, norm_eps,
                       shared_gate, y, topk_ids, topk_w, ws)
        if r is not None:
            return r
    _need_params(prob, w_router, bias, wg, wu, wd, s_wg, s_wu, s_wd, scales, norm_weight, shared_gate)
    _need_tokens(prob, x, y, topk_ids, topk_w)
    return _decode(prob, x, w_router, bias, wg, wu, wd, s_wg, s_wu, s_wd, scales, norm_weight, norm_eps, shared_gate,
                   y, topk_ids, topk_w, ws, stream)


def _decode(prob, x, w_router, bias, wg, wu, wd, s_wg, s_wu, s_wd, scales, norm_weight, norm_eps, shared_gate, y,
            topk_ids, topk_w, ws, stream):
    cur = _device(stream, x=x, w_router=w_router, router_bias=bias, w_gate=wg, w_up=wu, w_down=wd, ws_gate=s_wg,
                  ws_up=s_wu, ws_down=s_wd, scales=scales, norm_weight=norm_weight, shared_gate=shared_gate, y=y,
                  topk_ids=topk_ids, topk_w=topk_w, ws=ws)
    with _current(cur), _alloc(stream):
        if y is None:
            y = torch.empty((prob.T, prob.d), dtype=_act(prob), device=x.device)
        if ws is None:
            ws = _ws(decode_workspace_size(prob), x.device, None)
        opt = BlockOptions(_ptr(norm_weight), float(norm_eps), _ptr(shared_gate))
        _check(lib().moe_decode_forward(ctypes.byref(prob), ctypes.byref(opt), _ptr(x), _ptr(w_router), _ptr(bias),
                                        _ptr(wg), _ptr(wu), _ptr(wd), _ptr(s_wg), _ptr(s_wu), _ptr(s_wd),
                                        _ptr(scales), _ptr(y), _ptr(topk_ids), _ptr(topk_w), _ptr(ws), _nbytes(ws),
                                        _stream(stream)))
    return y


class MoELayer:
    """One block's weights plus a workspace sized for up to `max_tokens` tokens.
    Calling it runs the fused forward; ``decode`` the latency form for a few
    tokens."""

    def __init__(self, d, E, k, I, I_s, w_router, wg, wu, wd, s_wg=None, s_wu=None, s_wd=None, bias=None,
                 scales=None, act="bf16", w="bf16", max_tokens=0, norm_weight=None, norm_eps=1e-6,
                 shared_gate=None):
        self.shape = (d, E, k, I, I_s, act, w)
        self.w = (w_router, bias, wg, wu, wd, s_wg, s_wu, s_wd, scales)
        self.opts = (norm_weight, norm_eps, shared_gate)
        # the parameters are checked once here; each call checks its token buffers
        _need_params(self.problem(0), w_router, bias, wg, wu, wd, s_wg, s_wu, s_wd, scales, norm_weight,
                     shared_gate)
        self.device = wg.device
        # the workspace, and the stream of the last call that used it
        self.ws = self.ws_stream = self.ws_handle = None
        self.lock = threading.Lock()
        if max_tokens:
            self._reserve(self.problem(max_tokens))

    def problem(self, T):
        d, E, k, I, I_s, act, w = self.shape
        return Problem.make(T, d, E, k, I, I_s, act, w)

    def __getstate__(self):  # a copy has its own workspace
        return {**self.__dict__, "ws": None, "ws_stream": None, "ws_handle": None, "lock": None}

    def __setstate__(self, state):
        self.__dict__.update(state, lock=threading.Lock())

    def _reserve(self, prob, stream=None):
        """The workspace of a call on `stream`.  One buffer serves the calls of every
        stream, so a call on another stream than the last one's waits for that one's
        work.  None under capture: a graph that kept the buffer would share it with
        eager calls, and outlive it when it grows; the call's own allocation comes
        from the graph's pool instead."""
        if stream is None and self.device.type == "cuda" and torch.cuda.current_device() == self.device.index:
            return self._ordered(prob, None)
        if self.device.type != "cuda" or (stream is not None and stream.device != self.device):
            return self.ws  # (the call is refused)
        with _current(self.device), _alloc(stream):
            return self._ordered(prob, stream)

    def _ordered(self, prob, stream):
        if torch.cuda.is_current_stream_capturing():
            return None
        n = workspace_size(prob)
        if self.ws is not None and _stream(stream) != self.ws_handle:
            now = torch.cuda.current_stream()
            with torch.cuda.stream(self.ws_stream):
                captured = torch.cuda.is_current_stream_capturing()
            if captured:  # (to wait for it would make this call a part of the graph)
                self.ws = None
            else:
                now.wait_stream(self.ws_stream)
                self.ws.record_stream(now)
                self.ws_stream, self.ws_handle = now, now.cuda_stream
        if self.ws is None or self.ws.numel() < n:
            self.ws = None  # (freed first: the new one may take its place)
            self.ws, self.ws_stream = torch.empty(n, dtype=torch.uint8, device=self.device), torch.cuda.current_stream()
            self.ws_handle = self.ws_stream.cuda_stream
        return self.ws

    def __call__(self, x, y=None, topk_ids=None, topk_w=None, stream=None):
        prob = self.problem(x.shape[0])
        _need_tokens(prob, x, y, topk_ids, topk_w)
        w_router, bias, wg, wu, wd, s_wg, s_wu, s_wd, scales = self.w
        norm_weight, norm_eps, shared_gate = self.opts
        block = norm_weight is not None or shared_gate is not None
        with self.lock:  # (another thread's call waits for launches, so these are queued first)
            ws = self._reserve(prob, stream)
            return _forward(prob, x, w_router, bias, wg, wu, wd, s_wg, s_wu, s_wd, scales, norm_weight, norm_eps,
                            shared_gate, y, topk_ids, topk_w, ws, stream, block)

    def decode(self, x, y=None, topk_ids=None, topk_w=None, stream=None):
        """The block on x [T, d], T <= DECODE_MAX_T, in the latency form (decode_forward):
        the faster one for bf16 and E4M3 weights; with 4-bit weights up to 8 tokens, from
        about 10 on calling the layer is as fast or faster.
        The workspace is each call's own, from the pool of its stream or,
        under capture, of its graph: calls on several streams may run at once."""
        prob = self.problem(x.shape[0])
        w_router, bias, wg, wu, wd, s_wg, s_wu, s_wd, scales = self.w
        norm_weight, norm_eps, shared_gate = self.opts
        if stream is None:
            r = _fast_call("decode", prob, x, w_router, bias, wg, wu, wd, s_wg, s_wu, s_wd, scales, norm_weight,
                           norm_eps, shared_gate, y, topk_ids, topk_w, None)
            if r is not None:
                return r
        _need_tokens(prob, x, y, topk_ids, topk_w)
        return _decode(prob, x, w_router, bias, wg, wu, wd, s_wg, s_wu, s_wd, scales, norm_weight, norm_eps,
                       shared_gate, y, topk_ids, topk_w, None, stream)

    @classmethod
    def from_inputs(cls, inp, max_tokens=0):
        return cls(inp.d, inp.E, inp.k, inp.I, inp.I_s, inp.w_r, inp.wg, inp.wu, inp.wd, inp.s_wg, inp.s_wu,
                   inp.s_wd, bias=inp.bias, scales=inp.scales, act=inp.act, w=inp.w, max_tokens=max_tokens)
