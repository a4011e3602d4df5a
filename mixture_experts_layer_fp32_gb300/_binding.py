"""ctypes binding of libmoe_gb300.so (include/moe.h).

Argument marshalling only: every step of the layer runs in the CUDA library.
Tensors are torch CUDA tensors (contiguous); the current torch stream is
passed to the library.  There is no CPU or PyTorch fallback: if the
library is missing, `lib()` raises.
"""

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libmoe_gb300.so")

SCORE = {"softmax_post": 0, "softmax_pre": 1, "sigmoid": 2, "sqrtsoftplus": 3}
DTYPE = {"f32": 0, "bf16": 1}
DROP_POLICY = {"probs": 0, "position": 1}
STATUS = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED", 3: "MOE_ERR_WORKSPACE",
          4: "MOE_ERR_CUDA", 5: "MOE_ERR_DEVICE_CHECK", 6: "MOE_ERR_TIMEOUT"}

# every function declared in include/moe.h
EXPORTS = ["moe_abi_version", "moe_status_string", "moe_last_cuda_error", "moe_capacity",
           "moe_workspace_size", "moe_max_rows", "moe_route", "moe_permute", "moe_grouped_mlp",
           "moe_grouped_fc1", "moe_grouped_fc2", "moe_combine", "moe_forward", "moe_check",
           "moe_permute_noalloc", "moe_selftest_wait_timeout", "moe_shared_expert",
           "moe_combine_shared", "moe_workspace_size_shared", "moe_forward_shared",
           "moe_probe_fp32_fma", "moe_workspace_size_host", "moe_forward_host",
           "moe_quantize_rows_e4m3", "moe_quantize_experts_e4m3", "moe_workspace_size_e4m3",
           "moe_permute_e4m3", "moe_grouped_mlp_e4m3", "moe_forward_e4m3",
           "moe_grouped_fc1_e4m3", "moe_grouped_fc2_e4m3", "moe_workspace_size_backward",
           "moe_backward", "moe_workspace_size_backward_shared", "moe_backward_shared",
           "moe_shared_expert_backward", "moe_workspace_size_host_shared",
           "moe_forward_host_shared", "moe_workspace_size_host_e4m3", "moe_forward_host_e4m3",
           "moe_permute_map", "moe_permute_map_e4m3", "moe_grouped_fc2_combine",
           "moe_grouped_fc2_f16s", "moe_combine_f16s", "moe_grouped_fc2_e4m3_f16s",
           "moe_layer_norm", "moe_workspace_size_norm_backward", "moe_layer_norm_backward",
           "moe_dropout_add", "moe_quantize_w4", "moe_pack_w4", "moe_workspace_size_linear_w4",
           "moe_linear_w4", "moe_workspace_size_experts_w4", "moe_experts_w4",
           "moe_workspace_size_w4", "moe_forward_w4"]

NORM = {"layer": 0, "rms": 1}


class MoeConfig(ctypes.Structure):
    _fields_ = [("num_tokens", ctypes.c_int32), ("hidden", ctypes.c_int32),
                ("num_experts", ctypes.c_int32), ("topk", ctypes.c_int32),
                ("ffn_hidden", ctypes.c_int32), ("score", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("drop_policy", ctypes.c_int32),
                ("capacity_factor", ctypes.c_float), ("min_capacity", ctypes.c_int32),
                ("num_groups", ctypes.c_int32), ("group_topk", ctypes.c_int32),
                ("pad_to_capacity", ctypes.c_int32)]


class NormConfig(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("dropout", ctypes.c_double),
                ("hidden", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("param_dtype", ctypes.c_int32), ("kind", ctypes.c_int32),
                ("eps", ctypes.c_float)]


class W4Pointers(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("zeros", ctypes.c_void_p)]


class MoeError(RuntimeError):
    def __init__(self, code, where, detail=""):
        self.code = code
        msg = "%s failed: %s" % (where, STATUS.get(code, code))
        if detail:
            msg += " (%s)" % detail
        super().__init__(msg)


_lib = None


def lib():
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libmoe_gb300.so is not built (expected at %s); run "
                               "mixture_experts_layer_fp32_gb300.build.build()" % LIB_PATH)
        L = ctypes.CDLL(LIB_PATH)
        vp, sz, i32, i64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32, ctypes.c_int64
        cfgp = ctypes.POINTER(MoeConfig)
        normp, w4p = ctypes.POINTER(NormConfig), ctypes.POINTER(W4Pointers)
        f64 = ctypes.c_double
        sig = {
            "moe_abi_version": ([], i32),
            "moe_status_string": ([i32], ctypes.c_char_p),
            "moe_last_cuda_error": ([], ctypes.c_char_p),
            "moe_capacity": ([cfgp, ctypes.POINTER(i64)], i32),
            "moe_workspace_size": ([cfgp, ctypes.POINTER(sz)], i32),
            "moe_max_rows": ([cfgp, ctypes.POINTER(i64)], i32),
            "moe_route": ([cfgp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp], i32),
            "moe_permute": ([cfgp, vp, vp, vp, vp, vp, vp, vp, sz, vp], i32),
            "moe_permute_map": ([cfgp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp], i32),
            "moe_permute_map_e4m3": ([cfgp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp], i32),
            "moe_grouped_mlp": ([cfgp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp], i32),
            "moe_grouped_fc1": ([cfgp, vp, vp, vp, vp, vp, vp, sz, vp], i32),
            "moe_grouped_fc2": ([cfgp, vp, vp, vp, vp, vp, sz, vp], i32),
            "moe_combine": ([cfgp, vp, vp, vp, vp, vp], i32),
            "moe_grouped_fc2_combine": ([cfgp, vp, vp, vp, vp, vp, vp, vp, sz, vp], i32),
            "moe_grouped_fc2_f16s": ([cfgp, vp, vp, vp, vp, vp, vp, sz, vp], i32),
            "moe_combine_f16s": ([cfgp, vp, vp, vp, vp, vp, vp, vp], i32),
            "moe_forward": ([cfgp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp], i32),
            "moe_check": ([vp, vp, ctypes.POINTER(i32)], i32),
            "moe_permute_noalloc": ([cfgp, vp, vp, vp, vp, vp, vp, vp], i32),
            "moe_selftest_wait_timeout": ([vp, sz, i64, vp], i32),
            "moe_shared_expert": ([cfgp, i32, vp, vp, vp, vp, vp, vp, vp, sz, vp], i32),
            "moe_combine_shared": ([cfgp, vp, vp, vp, vp, vp, vp], i32),
            "moe_workspace_size_shared": ([cfgp, i32, ctypes.POINTER(sz)], i32),
            "moe_forward_shared": ([cfgp, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                    vp, vp, sz, vp], i32),
            "moe_probe_fp32_fma": ([i64, vp, ctypes.POINTER(ctypes.c_double), vp], i32),
            "moe_workspace_size_host": ([cfgp, ctypes.POINTER(sz)], i32),
            "moe_forward_host": ([cfgp, i32, vp, sz, vp, sz, vp, vp, vp, vp, vp, vp, vp, sz, vp],
                                 i32),
            "moe_quantize_rows_e4m3": ([i64, i32, vp, vp, vp, vp], i32),
            "moe_quantize_experts_e4m3": ([cfgp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp], i32),
            "moe_workspace_size_e4m3": ([cfgp, ctypes.POINTER(sz)], i32),
            "moe_permute_e4m3": ([cfgp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp], i32),
            "moe_grouped_mlp_e4m3": ([cfgp] + [vp] * 13 + [vp, sz, vp], i32),
            "moe_forward_e4m3": ([cfgp] + [vp] * 14 + [vp, sz, vp], i32),
            "moe_grouped_fc1_e4m3": ([cfgp] + [vp] * 8 + [vp, sz, vp], i32),
            "moe_grouped_fc2_e4m3": ([cfgp] + [vp] * 7 + [vp, sz, vp], i32),
            "moe_grouped_fc2_e4m3_f16s": ([cfgp] + [vp] * 8 + [vp, sz, vp], i32),
            "moe_workspace_size_backward": ([cfgp, ctypes.POINTER(sz)], i32),
            "moe_backward": ([cfgp] + [vp] * 20 + [vp, sz, vp], i32),
            "moe_workspace_size_backward_shared": ([cfgp, i32, ctypes.POINTER(sz)], i32),
            "moe_backward_shared": ([cfgp, i32] + [vp] * 27 + [vp, sz, vp], i32),
            "moe_shared_expert_backward": ([cfgp, i32] + [vp] * 10 + [vp, sz, vp], i32),
            "moe_workspace_size_host_shared": ([cfgp, i32, ctypes.POINTER(sz)], i32),
            "moe_forward_host_shared": ([cfgp, i32, i32, vp, sz, vp, sz] + [vp] * 9 +
                                        [vp, sz, vp], i32),
            "moe_workspace_size_host_e4m3": ([cfgp, ctypes.POINTER(sz)], i32),
            "moe_forward_host_e4m3": ([cfgp, i32, vp, sz, vp, sz] + [vp] * 9 + [vp, sz, vp], i32),
            "moe_layer_norm": ([normp] + [vp] * 10, i32),
            "moe_workspace_size_norm_backward": ([normp, ctypes.POINTER(sz)], i32),
            "moe_layer_norm_backward": ([normp] + [vp] * 11 + [vp, sz, vp], i32),
            "moe_dropout_add": ([i64, i32, f64, vp, vp, vp, vp, vp], i32),
            "moe_quantize_w4": ([i32, i32, i32, i32, vp, vp, vp, vp, vp], i32),
            "moe_pack_w4": ([i32, i32, i32, vp, vp, vp], i32),
            "moe_workspace_size_linear_w4": ([i64, i32, i32, ctypes.POINTER(sz)], i32),
            "moe_linear_w4": ([i64, i32, i32, i32, vp, w4p, vp, i32, vp, sz, vp], i32),
            "moe_workspace_size_experts_w4": ([cfgp, ctypes.POINTER(sz)], i32),
            "moe_experts_w4": ([cfgp, i32, vp, vp, vp, vp, w4p, w4p, w4p, vp, vp, sz, vp], i32),
            "moe_workspace_size_w4": ([cfgp, ctypes.POINTER(sz)], i32),
            "moe_forward_w4": ([cfgp, i32, vp, vp, vp, vp, w4p, w4p, w4p, vp, vp, vp, vp, vp, sz,
                                vp], i32),
        }
        for name, (args, res) in sig.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = res
        _lib = L
    return _lib


def config(T, h, E, k, f, score="softmax_post", dtype="bf16", capacity_factor=0.0,
           min_capacity=0, drop_policy="probs", num_groups=0, group_topk=0,
           pad_to_capacity=False):
    return MoeConfig(int(T), int(h), int(E), int(k), int(f), SCORE[score], DTYPE[dtype],
                     DROP_POLICY[drop_policy], float(capacity_factor), int(min_capacity),
                     int(num_groups), int(group_topk), int(bool(pad_to_capacity)))


def _check(code, where):
    if code != 0:
        detail = lib().moe_last_cuda_error().decode() if code == 4 else ""
        raise MoeError(code, where, detail)


def _p(t):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch tensor")
    if not t.is_cuda:
        raise ValueError("tensors must live on a CUDA device (no CPU path exists)")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


def _host(t):
    """Pointer of a HOST tensor (the host-I/O entry point's batches)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch tensor")
    if t.is_cuda:
        raise ValueError("x_host / y_host must be host tensors (ideally pinned)")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


# The current stream's handle without the object around it (0.3 us, not 3); the name
# is not a public one, so a torch without it takes the public way.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream():
    if _raw_stream is None:
        return torch.cuda.current_stream().cuda_stream
    return _raw_stream(torch.cuda.current_device())


def _ws(ws):
    return _p(ws), ws.numel() * ws.element_size()


def act_dtype(cfg):
    return torch.float32 if cfg.dtype == DTYPE["f32"] else torch.bfloat16


def capacity(cfg):
    v = ctypes.c_int64()
    _check(lib().moe_capacity(ctypes.byref(cfg), ctypes.byref(v)), "moe_capacity")
    return v.value


def workspace_size(cfg):
    v = ctypes.c_size_t()
    _check(lib().moe_workspace_size(ctypes.byref(cfg), ctypes.byref(v)), "moe_workspace_size")
    return v.value


def max_rows(cfg):
    v = ctypes.c_int64()
    _check(lib().moe_max_rows(ctypes.byref(cfg), ctypes.byref(v)), "moe_max_rows")
    return v.value


def alloc_workspace(cfg, device="cuda"):
    """Zero-filled workspace of moe_workspace_size(cfg) bytes."""
    return torch.zeros(workspace_size(cfg), dtype=torch.uint8, device=device)


def route(cfg, x, Wg, gate_bias, expert_bias, topk_idx, topk_prob, keep, tokens_per_expert,
          routing_map, ws):
    w, wb = _ws(ws)
    _check(lib().moe_route(ctypes.byref(cfg), _p(x), _p(Wg), _p(gate_bias), _p(expert_bias),
                           _p(topk_idx), _p(topk_prob), _p(keep), _p(tokens_per_expert),
                           _p(routing_map), w, wb, _stream()), "moe_route")


def permute(cfg, x, topk_idx, keep, x_perm, row_map, expert_offsets, ws):
    w, wb = _ws(ws)
    _check(lib().moe_permute(ctypes.byref(cfg), _p(x), _p(topk_idx), _p(keep), _p(x_perm),
                             _p(row_map), _p(expert_offsets), w, wb, _stream()), "moe_permute")


def permute_map(cfg, x, routing_map, topk_idx, keep, x_perm, row_map, expert_offsets, ws):
    """moe_permute_map: the permutation driven by a [T,E] routing map."""
    w, wb = _ws(ws)
    _check(lib().moe_permute_map(ctypes.byref(cfg), _p(x), _p(routing_map), _p(topk_idx),
                                 _p(keep), _p(x_perm), _p(row_map), _p(expert_offsets), w, wb,
                                 _stream()), "moe_permute_map")


def permute_noalloc(cfg, x, topk_idx, keep, x_perm, row_map, expert_offsets):
    """moe_permute without a workspace (scratch in a fixed array inside the
    library; for callers that cannot provide device memory)."""
    _check(lib().moe_permute_noalloc(ctypes.byref(cfg), _p(x), _p(topk_idx), _p(keep),
                                     _p(x_perm), _p(row_map), _p(expert_offsets), _stream()),
           "moe_permute_noalloc")


def grouped_fc1(cfg, x_perm, expert_offsets, W1, W3, h_mid, ws):
    w, wb = _ws(ws)
    _check(lib().moe_grouped_fc1(ctypes.byref(cfg), _p(x_perm), _p(expert_offsets), _p(W1),
                                 _p(W3), _p(h_mid), w, wb, _stream()), "moe_grouped_fc1")


def grouped_fc2(cfg, h_mid, expert_offsets, W2, y_perm, ws):
    w, wb = _ws(ws)
    _check(lib().moe_grouped_fc2(ctypes.byref(cfg), _p(h_mid), _p(expert_offsets), _p(W2),
                                 _p(y_perm), w, wb, _stream()), "moe_grouped_fc2")


def grouped_mlp(cfg, x_perm, expert_offsets, W1, W3, W2, h_mid, y_perm, ws):
    w, wb = _ws(ws)
    _check(lib().moe_grouped_mlp(ctypes.byref(cfg), _p(x_perm), _p(expert_offsets), _p(W1),
                                 _p(W3), _p(W2), _p(h_mid), _p(y_perm), w, wb, _stream()),
           "moe_grouped_mlp")


def grouped_fc2_combine(cfg, h_mid, expert_offsets, W2, row_map, topk_prob, y, ws):
    """moe_grouped_fc2_combine: fc2 and the combine of a top-1 layer in one call."""
    w, wb = _ws(ws)
    _check(lib().moe_grouped_fc2_combine(ctypes.byref(cfg), _p(h_mid), _p(expert_offsets),
                                         _p(W2), _p(row_map), _p(topk_prob), _p(y), w, wb,
                                         _stream()), "moe_grouped_fc2_combine")


def grouped_fc2_f16s(cfg, h_mid, expert_offsets, W2, y16, y16_exp, ws):
    """moe_grouped_fc2_f16s: fc2 with y_perm as fp16 (y16, torch.float16
    [R, h]) and one power-of-two exponent per 32 columns (y16_exp, int8)."""
    w, wb = _ws(ws)
    _check(lib().moe_grouped_fc2_f16s(ctypes.byref(cfg), _p(h_mid), _p(expert_offsets), _p(W2),
                                      _p(y16), _p(y16_exp), w, wb, _stream()),
           "moe_grouped_fc2_f16s")


def combine_f16s(cfg, y16, y16_exp, row_map, topk_prob, y, y_shared=None):
    """moe_combine_f16s: the combine over that y_perm (plus the shared
    expert's fp32 output y_shared, if given)."""
    _check(lib().moe_combine_f16s(ctypes.byref(cfg), _p(y16), _p(y16_exp), _p(row_map),
                                  _p(topk_prob), _p(y_shared), _p(y), _stream()),
           "moe_combine_f16s")


def combine(cfg, y_perm, row_map, topk_prob, y):
    _check(lib().moe_combine(ctypes.byref(cfg), _p(y_perm), _p(row_map), _p(topk_prob), _p(y),
                             _stream()), "moe_combine")


def forward(cfg, x, Wg, gate_bias, expert_bias, W1, W3, W2, y, ws, topk_idx=None,
            topk_prob=None, tokens_per_expert=None):
    w, wb = _ws(ws)
    _check(lib().moe_forward(ctypes.byref(cfg), _p(x), _p(Wg), _p(gate_bias), _p(expert_bias),
                             _p(W1), _p(W3), _p(W2), _p(y), _p(topk_idx), _p(topk_prob),
                             _p(tokens_per_expert), w, wb, _stream()), "moe_forward")


def workspace_size_shared(cfg, fs):
    v = ctypes.c_size_t()
    _check(lib().moe_workspace_size_shared(ctypes.byref(cfg), int(fs), ctypes.byref(v)),
           "moe_workspace_size_shared")
    return v.value


def alloc_workspace_shared(cfg, fs, device="cuda"):
    """Zero-filled workspace for forward_shared (moe_workspace_size_shared bytes)."""
    return torch.zeros(workspace_size_shared(cfg, fs), dtype=torch.uint8, device=device)


def shared_expert(cfg, fs, x, W1s, W3s, W2s, h_mid_s, y_shared, ws):
    w, wb = _ws(ws)
    _check(lib().moe_shared_expert(ctypes.byref(cfg), int(fs), _p(x), _p(W1s), _p(W3s), _p(W2s),
                                   _p(h_mid_s), _p(y_shared), w, wb, _stream()),
           "moe_shared_expert")


def combine_shared(cfg, y_perm, row_map, topk_prob, y_shared, y):
    _check(lib().moe_combine_shared(ctypes.byref(cfg), _p(y_perm), _p(row_map), _p(topk_prob),
                                    _p(y_shared), _p(y), _stream()), "moe_combine_shared")


def forward_shared(cfg, fs, x, Wg, gate_bias, expert_bias, W1, W3, W2, W1s, W3s, W2s, y, ws,
                   topk_idx=None, topk_prob=None, tokens_per_expert=None):
    w, wb = _ws(ws)
    _check(lib().moe_forward_shared(ctypes.byref(cfg), int(fs), _p(x), _p(Wg), _p(gate_bias),
                                    _p(expert_bias), _p(W1), _p(W3), _p(W2), _p(W1s), _p(W3s),
                                    _p(W2s), _p(y), _p(topk_idx), _p(topk_prob),
                                    _p(tokens_per_expert), w, wb, _stream()),
           "moe_forward_shared")


def workspace_size_host(cfg):
    v = ctypes.c_size_t()
    _check(lib().moe_workspace_size_host(ctypes.byref(cfg), ctypes.byref(v)),
           "moe_workspace_size_host")
    return v.value


def alloc_workspace_host(cfg, device="cuda"):
    """Zero-filled workspace for forward_host (moe_workspace_size_host bytes)."""
    return torch.zeros(workspace_size_host(cfg), dtype=torch.uint8, device=device)


def forward_host(cfg, x_host, y_host, Wg, gate_bias, expert_bias, W1, W3, W2, ws,
                 num_batches=None):
    """The forward over host batches x_host [B,T,h] -> y_host [B,T,h] (or one
    [T,h] buffer reused num_batches times, stride 0), copies pipelined with
    compute on the library's copy streams.  Asynchronous on the current
    stream."""
    T, h = cfg.num_tokens, cfg.hidden
    if num_batches is None:
        num_batches = x_host.shape[0] if x_host.dim() == 3 else 1
    xs = x_host[0].numel() * x_host.element_size() if x_host.dim() == 3 else 0
    ys = y_host[0].numel() * y_host.element_size() if y_host.dim() == 3 else 0
    for t, stride in ((x_host, xs), (y_host, ys)):
        per = T * h * t.element_size()
        if (t.numel() * t.element_size()) < (per if stride == 0 else per * num_batches):
            raise ValueError("host buffer smaller than its batches")
    w, wb = _ws(ws)
    _check(lib().moe_forward_host(ctypes.byref(cfg), int(num_batches), _host(x_host), xs,
                                  _host(y_host), ys, _p(Wg), _p(gate_bias), _p(expert_bias),
                                  _p(W1), _p(W3), _p(W2), w, wb, _stream()), "moe_forward_host")


def _host_batches(cfg, x_host, y_host, num_batches):
    """Batch count and byte strides of host buffers [B,T,h] (or [T,h] reused)."""
    T, h = cfg.num_tokens, cfg.hidden
    if num_batches is None:
        num_batches = x_host.shape[0] if x_host.dim() == 3 else 1
    xs = x_host[0].numel() * x_host.element_size() if x_host.dim() == 3 else 0
    ys = y_host[0].numel() * y_host.element_size() if y_host.dim() == 3 else 0
    for t, stride in ((x_host, xs), (y_host, ys)):
        per = T * h * t.element_size()
        if (t.numel() * t.element_size()) < (per if stride == 0 else per * num_batches):
            raise ValueError("host buffer smaller than its batches")
    return num_batches, xs, ys


def workspace_size_host_shared(cfg, fs):
    v = ctypes.c_size_t()
    _check(lib().moe_workspace_size_host_shared(ctypes.byref(cfg), int(fs), ctypes.byref(v)),
           "moe_workspace_size_host_shared")
    return v.value


def alloc_workspace_host_shared(cfg, fs, device="cuda"):
    return torch.zeros(workspace_size_host_shared(cfg, fs), dtype=torch.uint8, device=device)


def forward_host_shared(cfg, fs, x_host, y_host, Wg, gate_bias, expert_bias, W1, W3, W2, W1s,
                        W3s, W2s, ws, num_batches=None):
    """forward_host with the shared expert (moe_forward_shared per batch)."""
    n, xs, ys = _host_batches(cfg, x_host, y_host, num_batches)
    w, wb = _ws(ws)
    _check(lib().moe_forward_host_shared(ctypes.byref(cfg), int(fs), int(n), _host(x_host), xs,
                                         _host(y_host), ys, _p(Wg), _p(gate_bias),
                                         _p(expert_bias), _p(W1), _p(W3), _p(W2), _p(W1s),
                                         _p(W3s), _p(W2s), w, wb, _stream()),
           "moe_forward_host_shared")


def workspace_size_host_e4m3(cfg):
    v = ctypes.c_size_t()
    _check(lib().moe_workspace_size_host_e4m3(ctypes.byref(cfg), ctypes.byref(v)),
           "moe_workspace_size_host_e4m3")
    return v.value


def alloc_workspace_host_e4m3(cfg, device="cuda"):
    return torch.zeros(workspace_size_host_e4m3(cfg), dtype=torch.uint8, device=device)


def forward_host_e4m3(cfg, x_host, y_host, Wg, gate_bias, expert_bias, q, ws, num_batches=None):
    """forward_host with E4M3 experts (moe_forward_e4m3 per batch); q: E4m3Experts."""
    n, xs, ys = _host_batches(cfg, x_host, y_host, num_batches)
    w, wb = _ws(ws)
    _check(lib().moe_forward_host_e4m3(ctypes.byref(cfg), int(n), _host(x_host), xs,
                                       _host(y_host), ys, _p(Wg), _p(gate_bias), _p(expert_bias),
                                       _p(q.W1q), _p(q.s1), _p(q.W3q), _p(q.s3), _p(q.W2q),
                                       _p(q.s2), w, wb, _stream()), "moe_forward_host_e4m3")


# ------------------------------------------------------------- E4M3 experts

def quantize_rows_e4m3(x, codes, scales):
    """x [rows, cols] bf16 -> codes [rows, cols] uint8, scales [rows] fp32."""
    rows, cols = x.shape
    _check(lib().moe_quantize_rows_e4m3(rows, cols, _p(x), _p(codes), _p(scales), _stream()),
           "moe_quantize_rows_e4m3")


class E4m3Experts:
    """The expert weights in E4M3 (device tensors): W1q/W3q [E,f,h], W2q [E,h,f]
    uint8 codes, s1/s3 [E,f] and s2 [E,h] fp32 scales."""

    def __init__(self, cfg, W1, W3, W2):
        E, h, f = cfg.num_experts, cfg.hidden, cfg.ffn_hidden
        d = W1.device
        self.W1q = torch.empty((E, f, h), dtype=torch.uint8, device=d)
        self.W3q = torch.empty((E, f, h), dtype=torch.uint8, device=d)
        self.W2q = torch.empty((E, h, f), dtype=torch.uint8, device=d)
        self.s1 = torch.empty((E, f), dtype=torch.float32, device=d)
        self.s3 = torch.empty((E, f), dtype=torch.float32, device=d)
        self.s2 = torch.empty((E, h), dtype=torch.float32, device=d)
        _check(lib().moe_quantize_experts_e4m3(ctypes.byref(cfg), _p(W1), _p(W3), _p(W2),
                                               _p(self.W1q), _p(self.W3q), _p(self.W2q),
                                               _p(self.s1), _p(self.s3), _p(self.s2), _stream()),
               "moe_quantize_experts_e4m3")


def workspace_size_e4m3(cfg):
    v = ctypes.c_size_t()
    _check(lib().moe_workspace_size_e4m3(ctypes.byref(cfg), ctypes.byref(v)),
           "moe_workspace_size_e4m3")
    return v.value


def alloc_workspace_e4m3(cfg, device="cuda"):
    return torch.zeros(workspace_size_e4m3(cfg), dtype=torch.uint8, device=device)


def permute_map_e4m3(cfg, x, routing_map, topk_idx, keep, x_perm_q, x_perm_scale, row_map,
                     expert_offsets, ws):
    """moe_permute_map_e4m3: the E4M3 permutation by the padded routing map."""
    w, wb = _ws(ws)
    _check(lib().moe_permute_map_e4m3(ctypes.byref(cfg), _p(x), _p(routing_map), _p(topk_idx),
                                      _p(keep), _p(x_perm_q), _p(x_perm_scale), _p(row_map),
                                      _p(expert_offsets), w, wb, _stream()),
           "moe_permute_map_e4m3")


def permute_e4m3(cfg, x, topk_idx, keep, x_perm_q, x_perm_scale, row_map, expert_offsets, ws):
    w, wb = _ws(ws)
    _check(lib().moe_permute_e4m3(ctypes.byref(cfg), _p(x), _p(topk_idx), _p(keep), _p(x_perm_q),
                                  _p(x_perm_scale), _p(row_map), _p(expert_offsets), w, wb,
                                  _stream()), "moe_permute_e4m3")


def grouped_mlp_e4m3(cfg, x_perm_q, x_perm_scale, expert_offsets, q, h_mid, h_q, h_scale,
                     y_perm, ws):
    w, wb = _ws(ws)
    _check(lib().moe_grouped_mlp_e4m3(ctypes.byref(cfg), _p(x_perm_q), _p(x_perm_scale),
                                      _p(expert_offsets), _p(q.W1q), _p(q.s1), _p(q.W3q),
                                      _p(q.s3), _p(q.W2q), _p(q.s2), _p(h_mid), _p(h_q),
                                      _p(h_scale), _p(y_perm), w, wb, _stream()),
           "moe_grouped_mlp_e4m3")


def grouped_fc1_e4m3(cfg, x_perm_q, x_perm_scale, expert_offsets, q, h_mid, ws):
    w, wb = _ws(ws)
    _check(lib().moe_grouped_fc1_e4m3(ctypes.byref(cfg), _p(x_perm_q), _p(x_perm_scale),
                                      _p(expert_offsets), _p(q.W1q), _p(q.s1), _p(q.W3q),
                                      _p(q.s3), _p(h_mid), w, wb, _stream()),
           "moe_grouped_fc1_e4m3")


def grouped_fc2_e4m3(cfg, h_mid, expert_offsets, q, h_q, h_scale, y_perm, ws):
    w, wb = _ws(ws)
    _check(lib().moe_grouped_fc2_e4m3(ctypes.byref(cfg), _p(h_mid), _p(expert_offsets),
                                      _p(q.W2q), _p(q.s2), _p(h_q), _p(h_scale), _p(y_perm), w,
                                      wb, _stream()), "moe_grouped_fc2_e4m3")


def grouped_fc2_e4m3_f16s(cfg, h_mid, expert_offsets, q, h_q, h_scale, y16, y16_exp, ws):
    """moe_grouped_fc2_e4m3_f16s: the E4M3 fc2 into the fp16 y_perm (a
    power-of-two scale per 32 columns), for combine_f16s."""
    w, wb = _ws(ws)
    _check(lib().moe_grouped_fc2_e4m3_f16s(ctypes.byref(cfg), _p(h_mid), _p(expert_offsets),
                                           _p(q.W2q), _p(q.s2), _p(h_q), _p(h_scale), _p(y16),
                                           _p(y16_exp), w, wb, _stream()),
           "moe_grouped_fc2_e4m3_f16s")


def forward_e4m3(cfg, x, Wg, gate_bias, expert_bias, q, y, ws, topk_idx=None, topk_prob=None,
                 tokens_per_expert=None):
    w, wb = _ws(ws)
    _check(lib().moe_forward_e4m3(ctypes.byref(cfg), _p(x), _p(Wg), _p(gate_bias),
                                  _p(expert_bias), _p(q.W1q), _p(q.s1), _p(q.W3q), _p(q.s3),
                                  _p(q.W2q), _p(q.s2), _p(y), _p(topk_idx), _p(topk_prob),
                                  _p(tokens_per_expert), w, wb, _stream()), "moe_forward_e4m3")


# ------------------------------------------------------------------ backward

def workspace_size_backward(cfg):
    v = ctypes.c_size_t()
    _check(lib().moe_workspace_size_backward(ctypes.byref(cfg), ctypes.byref(v)),
           "moe_workspace_size_backward")
    return v.value


def alloc_workspace_backward(cfg, device="cuda"):
    return torch.zeros(workspace_size_backward(cfg), dtype=torch.uint8, device=device)


class Grads:
    """Gradient buffers of one backward (dx bf16, the rest fp32)."""

    def __init__(self, cfg, device="cuda"):
        T, h, E, f = cfg.num_tokens, cfg.hidden, cfg.num_experts, cfg.ffn_hidden
        d = torch.device(device)
        self.dx = torch.empty((T, h), dtype=act_dtype(cfg), device=d)
        self.dWg = torch.empty((h, E), dtype=torch.float32, device=d)
        self.dgate_bias = torch.empty((E,), dtype=torch.float32, device=d)
        self.dW1 = torch.empty((E, h, f), dtype=torch.float32, device=d)
        self.dW3 = torch.empty((E, h, f), dtype=torch.float32, device=d)
        self.dW2 = torch.empty((E, f, h), dtype=torch.float32, device=d)


def backward(cfg, x, Wg, gate_bias, W1, W3, W2, saved, dy, g, ws):
    """saved: a Buffers object after the staged forward (topk_idx, topk_prob,
    row_map, expert_offsets, x_perm, h_mid, y_perm); g: Grads."""
    w, wb = _ws(ws)
    _check(lib().moe_backward(ctypes.byref(cfg), _p(x), _p(Wg), _p(gate_bias), _p(W1), _p(W3),
                              _p(W2), _p(saved.topk_idx), _p(saved.topk_prob), _p(saved.row_map),
                              _p(saved.expert_offsets), _p(saved.x_perm), _p(saved.h_mid),
                              _p(saved.y_perm), _p(dy), _p(g.dx), _p(g.dWg), _p(g.dgate_bias),
                              _p(g.dW1), _p(g.dW3), _p(g.dW2), w, wb, _stream()), "moe_backward")


class SharedGrads:
    """The shared expert's weight gradients (fp32): dW1s, dW3s [h,fs], dW2s [fs,h]."""

    def __init__(self, cfg, fs, device="cuda"):
        h = cfg.hidden
        d = torch.device(device)
        self.dW1s = torch.empty((h, fs), dtype=torch.float32, device=d)
        self.dW3s = torch.empty((h, fs), dtype=torch.float32, device=d)
        self.dW2s = torch.empty((fs, h), dtype=torch.float32, device=d)


def workspace_size_backward_shared(cfg, fs):
    v = ctypes.c_size_t()
    _check(lib().moe_workspace_size_backward_shared(ctypes.byref(cfg), int(fs), ctypes.byref(v)),
           "moe_workspace_size_backward_shared")
    return v.value


def alloc_workspace_backward_shared(cfg, fs, device="cuda"):
    return torch.zeros(workspace_size_backward_shared(cfg, fs), dtype=torch.uint8, device=device)


def backward_shared(cfg, fs, x, Wg, gate_bias, W1, W3, W2, W1s, W3s, W2s, saved, dy, g, gs, ws):
    """The layer backward with the shared expert: saved as for backward() plus
    h_mid_s; g: Grads (dx includes the shared path), gs: SharedGrads."""
    w, wb = _ws(ws)
    _check(lib().moe_backward_shared(
        ctypes.byref(cfg), int(fs), _p(x), _p(Wg), _p(gate_bias), _p(W1), _p(W3), _p(W2),
        _p(W1s), _p(W3s), _p(W2s), _p(saved.topk_idx), _p(saved.topk_prob), _p(saved.row_map),
        _p(saved.expert_offsets), _p(saved.x_perm), _p(saved.h_mid), _p(saved.y_perm),
        _p(saved.h_mid_s), _p(dy), _p(g.dx), _p(g.dWg), _p(g.dgate_bias), _p(g.dW1), _p(g.dW3),
        _p(g.dW2), _p(gs.dW1s), _p(gs.dW3s), _p(gs.dW2s), w, wb, _stream()),
        "moe_backward_shared")


def shared_expert_backward(cfg, fs, x, W1s, W3s, W2s, h_mid_s, dy, dx_acc, gs, ws):
    """The shared expert's backward alone: its dx is ADDED to dx_acc (fp32 [T,h])."""
    w, wb = _ws(ws)
    _check(lib().moe_shared_expert_backward(ctypes.byref(cfg), int(fs), _p(x), _p(W1s), _p(W3s),
                                            _p(W2s), _p(h_mid_s), _p(dy), _p(dx_acc),
                                            _p(gs.dW1s), _p(gs.dW3s), _p(gs.dW2s), w, wb,
                                            _stream()), "moe_shared_expert_backward")


# ------------------------------------------------- norm, dropout (the layer's block)

_DTYPE_CODE = {torch.float32: 0, torch.bfloat16: 1}


def _code(t, what):
    code = _DTYPE_CODE.get(t.dtype)
    if code is None:
        raise ValueError("%s must be float32 or bfloat16, not %s" % (what, t.dtype))
    return code


def _like(t, ref, what):
    if t is not None and (t.shape != ref.shape or t.dtype != ref.dtype):
        raise ValueError("%s must have the shape and dtype of its input" % what)
    return _p(t)


def _vec(t, n, dtype, what):
    if t is not None and (t.numel() != n or t.dtype != dtype):
        raise ValueError("%s must hold %d values of %s" % (what, n, dtype))
    return _p(t)


def _table(t, rows, cols, dtype, what):
    """A tensor [..., cols] (or flat) of rows x cols values."""
    if t is None:
        return None
    if t.dtype != dtype or t.shape != (rows, cols) and (
            t.numel() != rows * cols or (t.dim() != 1 and t.shape[-1:] != (cols,))):
        raise ValueError("%s must be [%d, %d] of %s" % (what, rows, cols, dtype))
    return _p(t)


def _rng(rng, p):
    if p > 0 and (rng is None or rng.numel() != 2 or rng.dtype not in (torch.int64,
                                                                       torch.uint64)):
        raise ValueError("rng must be a device tensor of two 64-bit integers: seed and offset")
    return _p(rng)


def _norm_config(x, weight, bias, rms, eps, p):
    if x.dim() == 0:
        raise ValueError("the normed tensor needs a last dimension")
    hidden = x.shape[-1]
    dt = _code(x, "the normed tensor")
    pt = dt
    for t, what in ((weight, "weight"), (bias, "bias")):
        if t is not None:
            pt = _code(t, what)
            if t.numel() != hidden:
                raise ValueError("%s must hold %d values" % (what, hidden))
    if weight is not None and bias is not None and weight.dtype != bias.dtype:
        raise ValueError("weight and bias must have one dtype")
    return NormConfig(x.numel() // hidden if hidden else 0, float(p), hidden, dt, pt, int(rms),
                      float(eps))


def layer_norm(x, weight, bias, eps, y, mean=None, rstd=None, rms=False, residual=None, z=None,
               p=0.0, rng=None):
    """y = norm(z) over the last dimension, z = residual + dropout(x) (or x
    without a residual); layer norm, or RMS norm with rms=True.  weight, bias:
    float32 or bfloat16, or None.  z (where given), mean and rstd (fp32, one
    value a row) are what layer_norm_backward needs.  rng: device tensor of
    two 64-bit integers, seed and offset of the dropout's mask."""
    cfg = _norm_config(x, weight, bias, rms, eps, p)
    _check(lib().moe_layer_norm(ctypes.byref(cfg), _p(x), _like(residual, x, "residual"),
                                _rng(rng, p), _p(weight), _p(bias), _like(z, x, "z"),
                                _like(y, x, "y"), _vec(mean, cfg.rows, torch.float32, "mean"),
                                _vec(rstd, cfg.rows, torch.float32, "rstd"), _stream()),
           "moe_layer_norm")


def workspace_size_norm_backward(rows, hidden):
    v = ctypes.c_size_t()
    cfg = NormConfig(int(rows), 0.0, int(hidden), 0, 0, 0, 0.0)
    _check(lib().moe_workspace_size_norm_backward(ctypes.byref(cfg), ctypes.byref(v)),
           "moe_workspace_size_norm_backward")
    return v.value


def alloc_workspace_norm_backward(rows, hidden, device="cuda"):
    return torch.zeros(workspace_size_norm_backward(rows, hidden), dtype=torch.uint8,
                       device=device)


def layer_norm_backward(dy, z, weight, mean, rstd, dx, dweight, dbias, ws, rms=False, dz=None,
                        dbranch=None, p=0.0, rng=None):
    """Backward of layer_norm: dx = the gradient of z (the norm's, plus dz) and
    so of the residual, dbranch = that of the dropout's input (p, rng as in the
    forward), dweight and dbias fp32 (each may be None)."""
    cfg = _norm_config(z, weight, None, rms, 0.0, p)
    w, wb = _ws(ws)
    n = cfg.hidden
    _check(lib().moe_layer_norm_backward(
        ctypes.byref(cfg), _like(dy, z, "dy"), _p(z), _p(weight),
        _vec(mean, cfg.rows, torch.float32, "mean"), _vec(rstd, cfg.rows, torch.float32, "rstd"),
        _like(dz, z, "dz"), _rng(rng, p if dbranch is not None else 0.0), _like(dx, z, "dx"),
        _like(dbranch, z, "dbranch"), _vec(dweight, n, torch.float32, "dweight"),
        _vec(dbias, n, torch.float32, "dbias"), w, wb, _stream()), "moe_layer_norm_backward")


def dropout_add(x, y, p, rng, residual=None):
    """y = residual + dropout(x) (or dropout(x)); on a gradient it is the
    dropout's backward (same p and rng, no residual)."""
    _check(lib().moe_dropout_add(x.numel(), _code(x, "x"), float(p), _rng(rng, p), _p(x),
                                 _like(residual, x, "residual"), _like(y, x, "y"), _stream()),
           "moe_dropout_add")


# ----------------------------------------------------------------- 4-bit weights

def w4_row_bytes(k):
    """Bytes of one row's codes: blocks of 64 bytes for 128 inputs each."""
    return -(-k // 128) * 64


class W4Weight:
    """A weight [..., N, K] in 4 bits (device tensors): codes uint8
    [..., N, w4_row_bytes(K)], scales bf16 [..., N, K/group], zeros uint8 of the
    scales' shape or None (8).  W = scales * (code - zeros).  The tensors'
    contents may change, the tensors themselves are the weight's for good; their
    addresses are read at each call."""

    def __init__(self, codes, scales, zeros=None, group=128, k=None):
        k = scales.shape[-1] * group if k is None else k
        if scales.dtype != torch.bfloat16 or codes.dtype != torch.uint8:
            raise ValueError("codes must be uint8 and scales bfloat16")
        if codes.shape[-1] != w4_row_bytes(k) or scales.shape[-1] * group != k \
                or codes.shape[:-1] != scales.shape[:-1]:
            raise ValueError("codes, scales, group and k do not fit together")
        if zeros is not None and (zeros.dtype != torch.uint8 or zeros.shape != scales.shape):
            raise ValueError("zeros must be uint8, of the scales' shape")
        self._codes, self._scales, self._zeros = codes, scales, zeros
        self._group, self._k, self._n = group, k, codes.shape[-2]
        self._form = tuple(codes.shape[:-1]), k
        self._at = None
        self._pointers()

    codes = property(lambda self: self._codes)
    scales = property(lambda self: self._scales)
    zeros = property(lambda self: self._zeros)
    group = property(lambda self: self._group)
    k = property(lambda self: self._k)
    n = property(lambda self: self._n)

    def _pointers(self):
        codes, scales, zeros = self._codes, self._scales, self._zeros
        at = (codes.data_ptr(), scales.data_ptr(), None if zeros is None else zeros.data_ptr())
        if at != self._at:  # making the structure takes longer than looking (0.3 us, not 1)
            self._ref = ctypes.byref(W4Pointers(_p(codes), _p(scales), _p(zeros)))
            self._at = at
        return self._ref


class W4Experts:
    """The experts' three weights in 4 bits: W1, W3 [E,f,h], W2 [E,h,f]."""

    def __init__(self, W1, W3, W2):
        if not W1.group == W3.group == W2.group:
            raise ValueError("the experts' weights must have one group size")
        self._weights = W1, W3, W2

    W1 = property(lambda self: self._weights[0])
    W3 = property(lambda self: self._weights[1])
    W2 = property(lambda self: self._weights[2])
    group = property(lambda self: self._weights[0].group)

    def fits(self, cfg):
        E, h, f = cfg.num_experts, cfg.hidden, cfg.ffn_hidden
        W1, W3, W2 = self._weights
        up = (E, f), h
        if W1._form != up or W3._form != up or W2._form != ((E, h), f):
            raise ValueError("the 4-bit weights do not fit the configuration")

    def _pointers(self):
        W1, W3, W2 = self._weights
        return W1._pointers(), W3._pointers(), W2._pointers()


def quantize_w4(W, group=128, zeros=False):
    """W [..., K, N] bf16 (the layout of the layer's weights) -> W4Weight of
    [..., N, K]; zeros=True: with zero points."""
    if W.dtype != torch.bfloat16:
        raise ValueError("W must be bfloat16")
    K, N = W.shape[-2:]
    lead = tuple(W.shape[:-2])
    codes = torch.empty(lead + (N, w4_row_bytes(K)), dtype=torch.uint8, device=W.device)
    if K % 128:
        codes.zero_()  # the codes past K
    scales = torch.empty(lead + (N, K // group), dtype=torch.bfloat16, device=W.device)
    z = torch.empty(scales.shape, dtype=torch.uint8, device=W.device) if zeros else None
    _check(lib().moe_quantize_w4(W.numel() // (K * N), K, N, group, _p(W), _p(codes), _p(scales),
                                 _p(z), _stream()), "moe_quantize_w4")
    return W4Weight(codes, scales, z, group=group, k=K)


def quantize_experts_w4(W1, W3, W2, group=128, zeros=False):
    """The layer's W1/W3 [E,h,f] and W2 [E,f,h] bf16 -> W4Experts."""
    return W4Experts(*(quantize_w4(W, group, zeros) for W in (W1, W3, W2)))


def pack_w4(values):
    """Codes 0..15, one byte each [..., N, K] -> the codes of a W4Weight."""
    if values.dtype != torch.uint8:
        raise ValueError("values must be uint8")
    N, K = values.shape[-2:]
    codes = torch.empty(tuple(values.shape[:-1]) + (w4_row_bytes(K),), dtype=torch.uint8,
                        device=values.device)
    _check(lib().moe_pack_w4(values.numel() // (N * K), N, K, _p(values), _p(codes), _stream()),
           "moe_pack_w4")
    return codes


def workspace_size_linear_w4(rows, w):
    v = ctypes.c_size_t()
    _check(lib().moe_workspace_size_linear_w4(int(rows), w.n, w.k, ctypes.byref(v)),
           "moe_workspace_size_linear_w4")
    return v.value


def alloc_workspace_linear_w4(rows, w, device="cuda"):
    return torch.zeros(workspace_size_linear_w4(rows, w), dtype=torch.uint8, device=device)


def linear_w4(x, w, y, ws):
    """y [..., N] (bf16 or fp32) = x [..., K] bf16 . W^T; w: W4Weight [N,K]."""
    xs, ys = x.shape, y.shape
    if x.dtype != torch.bfloat16 or not xs or xs[-1] != w.k or w.codes.dim() != 2:
        raise ValueError("x must be bfloat16 [..., K] and W [N, K]")
    if not ys or ys[-1] != w.n or ys[:-1] != xs[:-1]:
        raise ValueError("y must be [..., N]")
    b, wb = _ws(ws)
    _check(lib().moe_linear_w4(x.numel() // w.k, w.n, w.k, w.group, _p(x), w._pointers(), _p(y),
                               _code(y, "y"), b, wb, _stream()), "moe_linear_w4")


def workspace_size_experts_w4(cfg):
    v = ctypes.c_size_t()
    _check(lib().moe_workspace_size_experts_w4(ctypes.byref(cfg), ctypes.byref(v)),
           "moe_workspace_size_experts_w4")
    return v.value


def alloc_workspace_experts_w4(cfg, device="cuda"):
    return torch.zeros(workspace_size_experts_w4(cfg), dtype=torch.uint8, device=device)


def experts_w4(cfg, x, topk_idx, topk_prob, keep, q, y, ws):
    """The routed SwiGLU experts of few tokens with 4-bit weights (q: W4Experts),
    from the router's topk_idx (int32), topk_prob (fp32) and keep (one byte each,
    or None), [T,k], into y [T,h]."""
    q.fits(cfg)
    T, k, h, dt = cfg.num_tokens, cfg.topk, cfg.hidden, act_dtype(cfg)
    kept = torch.bool if keep is not None and keep.dtype == torch.bool else torch.uint8
    b, wb = _ws(ws)
    _check(lib().moe_experts_w4(ctypes.byref(cfg), q.group, _table(x, T, h, dt, "x"),
                                _table(topk_idx, T, k, torch.int32, "topk_idx"),
                                _table(topk_prob, T, k, torch.float32, "topk_prob"),
                                _table(keep, T, k, kept, "keep"), *q._pointers(),
                                _table(y, T, h, dt, "y"), b, wb, _stream()), "moe_experts_w4")


def workspace_size_w4(cfg):
    v = ctypes.c_size_t()
    _check(lib().moe_workspace_size_w4(ctypes.byref(cfg), ctypes.byref(v)),
           "moe_workspace_size_w4")
    return v.value


def alloc_workspace_w4(cfg, device="cuda"):
    return torch.zeros(workspace_size_w4(cfg), dtype=torch.uint8, device=device)


def forward_w4(cfg, x, Wg, gate_bias, expert_bias, q, y, ws, topk_idx=None, topk_prob=None,
               tokens_per_expert=None):
    """The layer forward with 4-bit experts (q: W4Experts), for decoding."""
    q.fits(cfg)
    T, k, h, E, dt = cfg.num_tokens, cfg.topk, cfg.hidden, cfg.num_experts, act_dtype(cfg)
    f32, i32 = torch.float32, torch.int32
    b, wb = _ws(ws)
    _check(lib().moe_forward_w4(ctypes.byref(cfg), q.group, _table(x, T, h, dt, "x"),
                                _table(Wg, h, E, f32, "Wg"), _vec(gate_bias, E, f32, "gate_bias"),
                                _vec(expert_bias, E, f32, "expert_bias"), *q._pointers(),
                                _table(y, T, h, dt, "y"), _table(topk_idx, T, k, i32, "topk_idx"),
                                _table(topk_prob, T, k, f32, "topk_prob"),
                                _vec(tokens_per_expert, E, i32, "tokens_per_expert"), b, wb,
                                _stream()), "moe_forward_w4")


def probe_fp32_fma(iters, out):
    """Enqueue the FP32 FMA-rate probe; returns the flops it performs (time it
    with CUDA events on the current stream).  `out`: float32 device buffer of
    4 * SM-count elements."""
    flops = ctypes.c_double()
    _check(lib().moe_probe_fp32_fma(int(iters), _p(out), ctypes.byref(flops), _stream()),
           "moe_probe_fp32_fma")
    return flops.value


def selftest_wait_timeout(ws, limit_cycles):
    """Enqueue a bounded wait that is made to run out (see include/moe.h)."""
    w, wb = _ws(ws)
    _check(lib().moe_selftest_wait_timeout(w, wb, int(limit_cycles), _stream()),
           "moe_selftest_wait_timeout")


def check(ws):
    """Synchronises the current stream and raises if a kernel flagged an error."""
    info = ctypes.c_int32(0)
    code = lib().moe_check(_p(ws), _stream(), ctypes.byref(info))
    if code != 0:
        raise MoeError(code, "device check", "info=%d" % info.value)


class Buffers:
    """Device buffers of one forward, allocated with torch (plumbing only)."""

    def __init__(self, cfg, device="cuda"):
        T, h, E, k, f = cfg.num_tokens, cfg.hidden, cfg.num_experts, cfg.topk, cfg.ffn_hidden
        R = max_rows(cfg)
        dt = act_dtype(cfg)
        d = torch.device(device)
        self.topk_idx = torch.empty((T, k), dtype=torch.int32, device=d)
        self.topk_prob = torch.empty((T, k), dtype=torch.float32, device=d)
        self.keep = torch.empty((T, k), dtype=torch.uint8, device=d)
        self.tokens_per_expert = torch.empty((E,), dtype=torch.int32, device=d)
        self.routing_map = torch.empty((T, E), dtype=torch.uint8, device=d)
        self.x_perm = torch.empty((R, h), dtype=dt, device=d)
        self.row_map = torch.empty((T, k), dtype=torch.int32, device=d)
        self.expert_offsets = torch.empty((E + 1,), dtype=torch.int32, device=d)
        self.h_mid = torch.empty((R, f), dtype=dt, device=d)
        self.y_perm = torch.empty((R, h), dtype=torch.float32, device=d)
        self.y = torch.empty((T, h), dtype=dt, device=d)
        self.ws = alloc_workspace(cfg, d)
