"""Thin ctypes binding of ``include/rl_loss.h`` (argument marshalling only).

Every function of the C ABI is exposed under its own name; ``RlLoss`` wraps a
handle and marshals torch tensors (device memory and the current stream come
from PyTorch; every step of the computation runs in the CUDA library). The
binding fails loudly when ``librl_loss.so`` is missing or a call returns an
error: there is no other code path.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
import re
import threading

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "librl_loss.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "rl_loss.h")

RL_F32, RL_BF16 = 0, 1
RL_ADV_GROUP_REWARDS, RL_ADV_PER_SEQ, RL_ADV_PER_TOKEN, RL_ADV_TEACHER_LOGP = 0, 1, 2, 3
RL_OBJ_GRPO_ICEPOP, RL_OBJ_DIS = 0, 1
RL_NORM_PER_RESPONSE, RL_NORM_PER_TOKEN = 0, 1
RL_FLAG_POP_IN_BOUNDS, RL_FLAG_CLIP_ACTIVE, RL_FLAG_MASKED, RL_FLAG_BAD_TARGET = 1, 2, 4, 8

STATUS_NAMES = {0: "RL_OK", 1: "RL_ERR_INVALID_ARG", 2: "RL_ERR_SHAPE", 3: "RL_ERR_DTYPE",
                4: "RL_ERR_ALIGNMENT", 5: "RL_ERR_CAPACITY", 6: "RL_ERR_CUDA", 7: "RL_ERR_TARGET_RANGE",
                8: "RL_ERR_NONFINITE", 9: "RL_ERR_EMPTY_SEQ", 10: "RL_ERR_TIMEOUT", 11: "RL_ERR_UNSUPPORTED",
                12: "RL_ERR_SEQLENS", 13: "RL_ERR_DEVICE", 14: "RL_ERR_INTERNAL"}
CODES = {v: k for k, v in STATUS_NAMES.items()}


class RlLossError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {STATUS_NAMES.get(code, code)}")
        self.code = code


class rl_loss_config(ctypes.Structure):
    _fields_ = [("vocab_size", ctypes.c_int32), ("group_size", ctypes.c_int32),
                ("max_tokens", ctypes.c_int32), ("max_seqs", ctypes.c_int32),
                ("eps_low", ctypes.c_float), ("eps_high", ctypes.c_float), ("beta", ctypes.c_float),
                ("adv_eps", ctypes.c_float), ("adv_mode", ctypes.c_int32), ("std_unbiased", ctypes.c_int32),
                ("pop_indicator", ctypes.c_int32), ("logits_dtype", ctypes.c_int32), ("objective", ctypes.c_int32),
                ("loss_norm", ctypes.c_int32), ("dis_stopgrad", ctypes.c_int32)]


class rl_loss_inputs(ctypes.Structure):
    _fields_ = [("num_tokens", ctypes.c_int32), ("num_seqs", ctypes.c_int32), ("ld_logits", ctypes.c_int64),
                ("logits", ctypes.c_void_p), ("targets", ctypes.c_void_p), ("logp_old", ctypes.c_void_p),
                ("logp_infer", ctypes.c_void_p), ("mask", ctypes.c_void_p), ("cu_seqlens", ctypes.c_void_p),
                ("rewards_or_adv", ctypes.c_void_p)]


class rl_loss_outputs(ctypes.Structure):
    _fields_ = [("loss", ctypes.c_void_p), ("loss_f64", ctypes.c_void_p), ("dlogits", ctypes.c_void_p),
                ("ld_dlogits", ctypes.c_int64), ("logp", ctypes.c_void_p), ("entropy", ctypes.c_void_p),
                ("flags", ctypes.c_void_p), ("seq_adv", ctypes.c_void_p), ("counts", ctypes.c_void_p),
                ("mean_entropy", ctypes.c_void_p)]


class rl_gae_config(ctypes.Structure):
    _fields_ = [("gamma", ctypes.c_double), ("lambda_", ctypes.c_double), ("skip_observations", ctypes.c_int32),
                ("cross_trajectory", ctypes.c_int32)]


class rl_topk_config(ctypes.Structure):
    _fields_ = [("k", ctypes.c_int32), ("order", ctypes.c_int32)]


RL_TOPK_BY_SCORE, RL_TOPK_BY_POSITION = 0, 1


class rl_loss_kl(ctypes.Structure):
    _fields_ = [("logp_ref", ctypes.c_void_p), ("coef", ctypes.c_float), ("estimator", ctypes.c_int32),
                ("kl", ctypes.c_void_p), ("mean_kl", ctypes.c_void_p)]


class rl_loss_distill_config(ctypes.Structure):
    _fields_ = [("logits_dtype", ctypes.c_int32), ("vocab_size", ctypes.c_int32), ("k", ctypes.c_int32),
                ("mode", ctypes.c_int32), ("reverse", ctypes.c_int32), ("loss_norm", ctypes.c_int32),
                ("temperature", ctypes.c_float), ("scale", ctypes.c_float), ("tail_floor", ctypes.c_float)]


class rl_loss_pref_config(ctypes.Structure):
    _fields_ = [("logits_dtype", ctypes.c_int32), ("vocab_size", ctypes.c_int32), ("loss_type", ctypes.c_int32),
                ("length_norm", ctypes.c_int32), ("beta", ctypes.c_float), ("margin", ctypes.c_float),
                ("label_smoothing", ctypes.c_float), ("nll_coef", ctypes.c_float)]


class rl_ln_config(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("cols", ctypes.c_int32), ("x_dtype", ctypes.c_int32),
                ("y_dtype", ctypes.c_int32), ("param_dtype", ctypes.c_int32), ("eps", ctypes.c_float)]


class rl_act8(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("ld_codes", ctypes.c_int64),
                ("ld_scales", ctypes.c_int64), ("format", ctypes.c_int32)]


class rl_loss_final_norm(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("ld_x", ctypes.c_int64), ("weight", ctypes.c_void_p), ("bias", ctypes.c_void_p),
                ("dx", ctypes.c_void_p), ("ld_dx", ctypes.c_int64), ("dweight", ctypes.c_void_p),
                ("dbias", ctypes.c_void_p)]


RL_LN_LAYER, RL_LN_RMS = 0, 1
RL_ACT8_INT8, RL_ACT8_E4M3 = 0, 1
LN_KINDS = {"layer": RL_LN_LAYER, "rms": RL_LN_RMS}
ACT8_FORMATS = {"int8": RL_ACT8_INT8, "e4m3": RL_ACT8_E4M3}
ACT8_BLOCK = 32  # columns that share a scale
RL_KL_K1, RL_KL_K2, RL_KL_K3 = 0, 1, 2
RL_DISTILL_RENORM, RL_DISTILL_TAIL = 0, 1
RL_PREF_SIGMOID, RL_PREF_HINGE, RL_PREF_IPO = 0, 1, 2
KL_ESTIMATORS = {"k1": RL_KL_K1, "k2": RL_KL_K2, "k3": RL_KL_K3}
DISTILL_MODES = {"renorm": RL_DISTILL_RENORM, "tail": RL_DISTILL_TAIL}
REVERSE_TAIL_FLOOR = 1e-9  # distill_loss's default; 1 - sum q of fp32 log-probs is known to some 1e-8
PREF_LOSSES = {"sigmoid": RL_PREF_SIGMOID, "hinge": RL_PREF_HINGE, "ipo": RL_PREF_IPO}


class rl_loss_profile(ctypes.Structure):
    _fields_ = [("num_kernels", ctypes.c_int32), ("names", (ctypes.c_char * 32) * 12),
                ("launches", ctypes.c_int64 * 12), ("total_ms", ctypes.c_double * 12)]


_lib = None


def load(path: str | None = None) -> ctypes.CDLL:
    """Load the CUDA library (raises if it has not been built). RL_LOSS_LIB in the
    environment names another build of it, such as the debug build."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or os.environ.get("RL_LOSS_LIB") or LIB_PATH
    if not os.path.exists(path):
        raise RuntimeError(f"CUDA library {path} is missing; build it with __graft_entry__.build()")
    lib = ctypes.CDLL(path)
    P = ctypes.c_void_p
    st = ctypes.c_int
    sig = {
        "rl_loss_create": ([ctypes.POINTER(rl_loss_config), ctypes.POINTER(P)], st),
        "rl_loss_destroy": ([P], st),
        "rl_loss_forward_backward": ([P, ctypes.POINTER(rl_loss_inputs), ctypes.POINTER(rl_loss_outputs), P], st),
        "rl_loss_forward_backward_from_host": ([P, ctypes.POINTER(rl_loss_inputs), ctypes.POINTER(rl_loss_inputs),
                                                ctypes.POINTER(rl_loss_outputs), ctypes.c_int32, P], st),
        "rl_loss_get_device_status": ([P, P, ctypes.POINTER(ctypes.c_uint32)], st),
        "rl_loss_status_string": ([st], ctypes.c_char_p),
        "rl_loss_profile_start": ([P, ctypes.c_int32], st),
        "rl_loss_profile_read": ([P, ctypes.POINTER(rl_loss_profile)], st),
        "rl_loss_launch_count": ([P, ctypes.POINTER(ctypes.c_int64)], st),
        "rl_loss_last_cuda_error": ([P], ctypes.c_char_p),
        "rl_loss_version": ([], ctypes.c_int32),
        "rl_loss_forward_backward_noalloc": ([ctypes.POINTER(rl_loss_config), ctypes.POINTER(rl_loss_inputs),
                                              ctypes.POINTER(rl_loss_outputs), P, P], st),
        "rl_loss_projection_setup": ([P, ctypes.c_int32, ctypes.c_int32], st),
        "rl_gae_advantages": ([ctypes.POINTER(rl_gae_config), ctypes.c_int32, ctypes.c_int32, P, P, P, P, P, P, P, P,
                               ctypes.c_size_t, P, P], st),
        "rl_gae_advantages_withheld": ([ctypes.POINTER(rl_gae_config), ctypes.c_int32, ctypes.c_int32, P, P, P, P, P, P,
                                        P, P, ctypes.c_size_t, P, P, ctypes.c_int32, ctypes.c_double], st),
        "rl_gae_workspace_bytes": ([ctypes.c_int32], ctypes.c_size_t),
        "rl_topk_max_k": ([], ctypes.c_int32),
        "rl_topk": ([ctypes.POINTER(rl_topk_config), ctypes.c_int32, P, ctypes.c_int64, P, P, P, ctypes.c_int64, P, P],
                    st),
        "rl_loss_token_logp": ([ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, P, ctypes.c_int64, P, P, P, P, P, P], st),
        "rl_loss_forward_backward_kl": ([P, ctypes.POINTER(rl_loss_inputs), ctypes.POINTER(rl_loss_kl),
                                         ctypes.POINTER(rl_loss_outputs), P], st),
        "rl_loss_distill_max_k": ([], ctypes.c_int32),
        "rl_loss_distill_workspace_bytes": ([ctypes.c_int32, ctypes.c_int32], ctypes.c_size_t),
        "rl_loss_distill": ([ctypes.POINTER(rl_loss_distill_config), ctypes.c_int32, ctypes.c_int32, P, ctypes.c_int64,
                             P, P, ctypes.c_int64, P, P, P, P, P, ctypes.c_int64, P, P, ctypes.c_size_t, P, P], st),
        "rl_loss_preference_workspace_bytes": ([ctypes.c_int32, ctypes.c_int32], ctypes.c_size_t),
        "rl_loss_preference": ([ctypes.POINTER(rl_loss_pref_config), ctypes.c_int32, ctypes.c_int32, P, ctypes.c_int64,
                                P, P, P, P, P, P, P, ctypes.c_int64, P, P, P, P, ctypes.c_size_t, P, P], st),
        "rl_loss_layer_norm_max_cols": ([], ctypes.c_int32),
        "rl_loss_layer_norm": ([ctypes.POINTER(rl_ln_config), ctypes.c_int32, P, ctypes.c_int64, P, ctypes.c_int64, P, P, P,
                                P, ctypes.c_int64, P, ctypes.c_int64, ctypes.POINTER(rl_act8), P, P, P, P], st),
        "rl_loss_layer_norm_workspace_bytes": ([ctypes.c_int32, ctypes.c_int32], ctypes.c_size_t),
        "rl_loss_layer_norm_backward": ([ctypes.POINTER(rl_ln_config), ctypes.c_int32, P, ctypes.c_int64, P, ctypes.c_int64,
                                         ctypes.POINTER(rl_act8), P, P, P, P, P, P, ctypes.c_int64, P, ctypes.c_int64, P, P,
                                         ctypes.c_int32, P, ctypes.c_int64, P, ctypes.c_size_t, P, P], st),
        "rl_loss_act8_pack": ([ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, P, ctypes.c_int64, ctypes.POINTER(rl_act8), P],
                              st),
        "rl_loss_act8_unpack": ([ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.POINTER(rl_act8), P, ctypes.c_int64,
                                 P], st),
        "rl_loss_normed_projection_workspace_bytes": ([P], ctypes.c_size_t),
        "rl_loss_normed_projection_forward_backward": ([P, ctypes.POINTER(rl_ln_config), ctypes.POINTER(rl_loss_final_norm), P,
                                                        ctypes.c_int64, ctypes.POINTER(rl_loss_inputs), P, ctypes.c_int64,
                                                        ctypes.POINTER(rl_loss_outputs), P, ctypes.c_size_t, P], st),
        "rl_loss_projection_logits": ([P, P, ctypes.c_int64, P, ctypes.c_int64, ctypes.c_int32, P, ctypes.c_int64,
                                       P], st),
        "rl_loss_fused_projection_forward_backward": ([P, P, ctypes.c_int64, P, ctypes.c_int64,
                                                       ctypes.POINTER(rl_loss_inputs), P, ctypes.c_int64, P,
                                                       ctypes.c_int64, ctypes.POINTER(rl_loss_outputs), P], st),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    _lib = lib
    return lib


def header_functions(path: str = HEADER) -> list[str]:
    """Names of every function the C header declares."""
    text = open(path).read()
    return sorted(set(re.findall(r"RL_LOSS_API\s+[\w\s\*]+?\b(rl_(?:loss_|gae_|topk)\w*)\s*\(", text)))


def _check(code: int, what: str):
    if code != 0:
        raise RlLossError(code, what)


# ------------------------------------------------------------------ the C names, one to one

def rl_loss_create(config: rl_loss_config) -> ctypes.c_void_p:
    h = ctypes.c_void_p()
    _check(load().rl_loss_create(ctypes.byref(config), ctypes.byref(h)), "rl_loss_create")
    return h


def rl_loss_destroy(handle) -> None:
    _check(load().rl_loss_destroy(handle), "rl_loss_destroy")


def rl_loss_forward_backward(handle, inputs: rl_loss_inputs, outputs: rl_loss_outputs, stream: int) -> int:
    return load().rl_loss_forward_backward(handle, ctypes.byref(inputs), ctypes.byref(outputs),
                                           ctypes.c_void_p(stream))


def rl_loss_forward_backward_from_host(handle, host: rl_loss_inputs, device: rl_loss_inputs,
                                       outputs: rl_loss_outputs, num_chunks: int, stream: int) -> int:
    return load().rl_loss_forward_backward_from_host(handle, ctypes.byref(host), ctypes.byref(device),
                                                     ctypes.byref(outputs), num_chunks, ctypes.c_void_p(stream))


def rl_loss_get_device_status(handle, stream: int) -> int:
    bits = ctypes.c_uint32(0)
    _check(load().rl_loss_get_device_status(handle, ctypes.c_void_p(stream), ctypes.byref(bits)),
           "rl_loss_get_device_status")
    return int(bits.value)


def rl_loss_status_string(code: int) -> str:
    return load().rl_loss_status_string(code).decode()


def rl_loss_profile_start(handle, max_calls: int) -> None:
    _check(load().rl_loss_profile_start(handle, max_calls), "rl_loss_profile_start")


def rl_loss_profile_read(handle) -> dict:
    prof = rl_loss_profile()
    _check(load().rl_loss_profile_read(handle, ctypes.byref(prof)), "rl_loss_profile_read")
    return {prof.names[k].value.decode(): (int(prof.launches[k]), float(prof.total_ms[k]))
            for k in range(prof.num_kernels)}


def rl_loss_launch_count(handle) -> int:
    n = ctypes.c_int64(0)
    _check(load().rl_loss_launch_count(handle, ctypes.byref(n)), "rl_loss_launch_count")
    return int(n.value)


def rl_loss_forward_backward_noalloc(config: rl_loss_config, inputs: rl_loss_inputs, outputs: rl_loss_outputs,
                                     device_status_ptr: int | None, stream: int) -> int:
    """The allocation-free entry point (no handle; static device workspace)."""
    return load().rl_loss_forward_backward_noalloc(ctypes.byref(config), ctypes.byref(inputs),
                                                   ctypes.byref(outputs), ctypes.c_void_p(device_status_ptr),
                                                   ctypes.c_void_p(stream))


def rl_loss_last_cuda_error(handle) -> str:
    return load().rl_loss_last_cuda_error(handle).decode()


def rl_loss_projection_setup(handle, hidden_dim: int, chunk_tokens: int) -> None:
    _check(load().rl_loss_projection_setup(handle, hidden_dim, chunk_tokens), "rl_loss_projection_setup")


def rl_loss_projection_logits(handle, hidden, ld_hidden, w_lm, ld_w, rows, logits, ld_logits, stream) -> int:
    return load().rl_loss_projection_logits(handle, hidden, ld_hidden, w_lm, ld_w, rows, logits, ld_logits,
                                            ctypes.c_void_p(stream))


def rl_loss_fused_projection_forward_backward(handle, hidden, ld_hidden, w_lm, ld_w, inputs, dhidden, ld_dhidden,
                                              dw_lm, ld_dw, outputs, stream) -> int:
    return load().rl_loss_fused_projection_forward_backward(handle, hidden, ld_hidden, w_lm, ld_w,
                                                            ctypes.byref(inputs), dhidden, ld_dhidden, dw_lm, ld_dw,
                                                            ctypes.byref(outputs), ctypes.c_void_p(stream))


def rl_gae_advantages(config: rl_gae_config, num_tokens, num_seqs, rewards, values, mask, cu_seqlens, rollout_ids,
                      advantages, returns, workspace, workspace_bytes, device_status, stream) -> int:
    return load().rl_gae_advantages(ctypes.byref(config), num_tokens, num_seqs, rewards, values, mask, cu_seqlens,
                                    rollout_ids, advantages, returns, workspace, workspace_bytes, device_status,
                                    ctypes.c_void_p(stream))


def rl_gae_advantages_withheld(config: rl_gae_config, num_tokens, num_seqs, rewards, values, mask, cu_seqlens,
                               rollout_ids, advantages, returns, workspace, workspace_bytes, device_status, stream,
                               withhold_chunk, wait_limit_s) -> int:
    return load().rl_gae_advantages_withheld(ctypes.byref(config), num_tokens, num_seqs, rewards, values, mask,
                                             cu_seqlens, rollout_ids, advantages, returns, workspace, workspace_bytes,
                                             device_status, ctypes.c_void_p(stream), withhold_chunk, wait_limit_s)


def rl_gae_workspace_bytes(num_tokens: int) -> int:
    return int(load().rl_gae_workspace_bytes(int(num_tokens)))


_GAE_WORKSPACE: dict = {}


def gae_workspace(num_tokens: int, device):
    """A GAE workspace for this device of at least this size, zero-filled when
    allocated and kept between calls (every completed call clears its counters
    and flags again)."""
    import torch
    dev = torch.device(device)
    if dev.index is None:
        dev = torch.device(dev.type, torch.cuda.current_device())
    need = rl_gae_workspace_bytes(num_tokens)
    ws = _GAE_WORKSPACE.get(dev)
    if ws is None or ws.numel() < need:
        ws = torch.zeros(max(need, 256), dtype=torch.uint8, device=dev)
        _GAE_WORKSPACE[dev] = ws
    return ws


def gae(rewards, values, mask, cu_seqlens, gamma: float, lam: float, skip_observations: bool = True,
        rollout_ids=None, returns=None, advantages=None, device_status=None, stream=None, workspace=None):
    """Advantages (and optionally returns) on the GPU; torch CUDA tensors in and out."""
    import torch
    T, S = int(rewards.shape[0]), int(cu_seqlens.shape[0]) - 1
    if advantages is None:
        advantages = torch.empty(T, dtype=torch.float32, device=rewards.device)
    if workspace is None:
        workspace = gae_workspace(T, rewards.device)
    cfg = rl_gae_config(gamma, lam, int(skip_observations), int(rollout_ids is not None))
    if stream is None:
        stream = torch.cuda.current_stream().cuda_stream
    _check(rl_gae_advantages(cfg, T, S, _ptr(rewards), _ptr(values), _ptr(mask), _ptr(cu_seqlens), _ptr(rollout_ids),
                             _ptr(advantages), _ptr(returns), _ptr(workspace), workspace.numel(),
                             _ptr(device_status), stream), "rl_gae_advantages")
    return advantages


def rl_topk_max_k() -> int:
    return int(load().rl_topk_max_k())


def topk(scores, k: int, lengths=None, order: str = "score", out_idx=None, out_val=None, want_values=True,
         device_status=None, stream=None):
    """Row-wise deterministic top-k on the GPU; torch CUDA tensors in and out. Returns (positions, scores)."""
    import torch
    if order not in ("score", "index"):
        raise ValueError("order is 'score' or 'index'")
    rows, ld = int(scores.shape[0]), int(scores.shape[1])
    if scores.stride(1) != 1:
        raise ValueError("scores rows must be contiguous")
    if out_idx is None:
        out_idx = torch.empty((rows, k), dtype=torch.int32, device=scores.device)
    if out_val is None and want_values:
        out_val = torch.empty((rows, k), dtype=torch.float32, device=scores.device)
    cfg = rl_topk_config(k, RL_TOPK_BY_SCORE if order == "score" else RL_TOPK_BY_POSITION)
    if stream is None:
        stream = torch.cuda.current_stream().cuda_stream
    _check(load().rl_topk(ctypes.byref(cfg), rows, _ptr(scores), int(scores.stride(0)), _ptr(lengths), _ptr(out_idx),
                          _ptr(out_val), int(out_idx.stride(0)), _ptr(device_status), ctypes.c_void_p(stream)),
           "rl_topk")
    return out_idx, out_val


# ------------------------------------------------------------------ post-training losses without a handle

def rl_loss_distill_max_k() -> int:
    return int(load().rl_loss_distill_max_k())


@functools.lru_cache(maxsize=256)
def rl_loss_distill_workspace_bytes(num_tokens: int, num_seqs: int) -> int:
    return int(load().rl_loss_distill_workspace_bytes(int(num_tokens), int(num_seqs)))


@functools.lru_cache(maxsize=256)
def rl_loss_preference_workspace_bytes(num_tokens: int, num_seqs: int) -> int:
    return int(load().rl_loss_preference_workspace_bytes(int(num_tokens), int(num_seqs)))


_POST_WORKSPACE = threading.local()


def _post_workspace(need: int, device, stream: int):
    """A workspace of this thread, device and stream, grown when a call needs more and kept between calls. (By
    thread: a call is two or three launches, between which another thread's on the same stream may go.) During a
    graph capture the caller passes its own: one allocated here would belong to the graph's memory pool."""
    import torch
    if torch._C._cuda_isCurrentStreamCapturing():
        raise ValueError("pass workspace= while a CUDA graph is captured (any torch.uint8 tensor of the size "
                         "rl_loss_*_workspace_bytes gives, kept as long as the graph)")
    kept = _POST_WORKSPACE.__dict__
    ws = kept.get((device.index, stream))
    if ws is None or ws.numel() < need:
        ws = torch.empty(max(need, 1 << 16), dtype=torch.uint8, device=device)
        kept[(device.index, stream)] = ws
    return ws


def _logits_code(logits, vocab, dlogits=None):
    """(dtype code, V) of a logits tensor, checked together with its gradient's."""
    import torch
    dt = logits.dtype
    if (dt != torch.bfloat16 and dt != torch.float32) or logits.dim() != 2 or not logits.is_cuda:
        raise ValueError("logits is a CUDA tensor [tokens, vocabulary] of torch.float32 or torch.bfloat16")
    T, W = logits.shape
    if logits.stride(1) != 1 or (dlogits is not None and (dlogits.dim() != 2 or dlogits.stride(1) != 1)):
        raise ValueError("the rows of logits and dlogits are contiguous")
    V = W if vocab is None else int(vocab)
    if V > W:
        raise ValueError("vocab is larger than the logits' rows")
    if dlogits is not None and (dlogits.dtype != dt or dlogits.shape[0] < T or dlogits.shape[1] < V
                                or dlogits.device != logits.device):
        raise ValueError("dlogits has the type of logits and at least its rows and vocabulary, on its device")
    return (RL_BF16 if dt == torch.bfloat16 else RL_F32), V


def _vector(name: str, t, n: int, dtype, device, optional: bool = False):
    """The pointer of a 1-D tensor argument after checking its type, length, place and layout."""
    if t is None:
        if optional:
            return None
        raise ValueError(f"{name} is required")
    if t.dtype is not dtype or t.numel() < n or t.get_device() != device.index or not t.is_contiguous():
        raise ValueError(f"{name} is a contiguous {dtype} tensor of at least {n} values on {device}")
    return t.data_ptr()


def _rows(name: str, t, rows: int, cols: int, dtype, device):
    """The pointer and row stride of a 2-D tensor argument after checking its type, shape, place and layout."""
    if t.dtype is dtype and t.dim() == 2 and t.get_device() == device.index:
        (have, width), (ld, step) = t.shape, t.stride()
        if have >= rows and width >= cols and step == 1:
            return t.data_ptr(), ld
    raise ValueError(f"{name} is a {dtype} tensor [at least {rows}, at least {cols}] with contiguous rows on {device}")


def _status_word(t, device):
    """The pointer of a call's optional status word, 32 bits on the device."""
    if t is None:
        return None
    if t.is_floating_point() or t.element_size() != 4 or t.numel() < 1 or t.get_device() != device.index:
        raise ValueError(f"device_status is a torch.int32 or torch.uint32 tensor of one value on {device}")
    return t.data_ptr()


def _workspace_of(t, device):
    """The pointer and bytes of a workspace that the caller passed."""
    if t.get_device() != device.index or not t.is_contiguous():
        raise ValueError(f"workspace is a contiguous tensor on {device}, of any type")
    return t.data_ptr(), t.numel() * t.element_size()


_NO_CONTEXT = contextlib.nullcontext()


def _allocations_of(stream, device):
    """The context in which a call on `stream` (None: the current one) allocates what its caller left out: the
    memory then belongs to the stream that uses it, and is not handed to another one while that still does."""
    import torch
    if stream is None or device.type != "cuda" or stream == _current_stream(device):
        return _NO_CONTEXT
    return torch.cuda.stream(torch.cuda.ExternalStream(stream, device=device))


def _gradient_of(logits, V: int, stream):
    """A gradient laid out like the logits. Calls do not write its columns past the vocabulary, which a product with
    the whole of it reads: they are 0."""
    import torch
    with _allocations_of(stream, logits.device):
        dlogits = torch.empty_strided(logits.shape, logits.stride(), dtype=logits.dtype, device=logits.device)
        if V < logits.shape[1]:
            dlogits[:, V:].zero_()
    return dlogits


def _missing(tensors: tuple, sizes: tuple, device) -> list:
    """The fp32 tensors as they were given, new ones in the place of those that were not. (An allocation takes
    1.5 us of host time; one for all of them takes 10, as a tensor is then split.)"""
    import torch
    return [torch.empty(n, dtype=torch.float32, device=device) if t is None else t for t, n in zip(tensors, sizes)]


def _current_stream(device) -> int:
    """The current stream of a CUDA device as an address, without the Stream object around it."""
    import torch
    return torch._C._cuda_getCurrentRawStream(device.index)


def token_logp(logits, targets, mask=None, *, vocab: int | None = None, logp=None, entropy=None,
               want_entropy: bool = False, device_status=None, stream=None):
    """Log-probs (and entropies) of the target tokens on the GPU, without a gradient: the pass of a reference
    or old policy. Returns (logp [T], entropy [T] or None); mask = 0 tokens get 0 and their logits are not read."""
    import torch
    code, V = _logits_code(logits, vocab)
    T, dev = logits.shape[0], logits.device
    with _allocations_of(stream, dev):
        if logp is None:
            logp = torch.empty(T, dtype=torch.float32, device=dev)
        if entropy is None and want_entropy:
            entropy = torch.empty(T, dtype=torch.float32, device=dev)
    if stream is None:
        stream = _current_stream(dev)
    f32 = torch.float32
    _check(load().rl_loss_token_logp(code, T, V, logits.data_ptr(), logits.stride(0) if T else V,
                                     _vector("targets", targets, T, torch.int32, dev),
                                     _vector("mask", mask, T, torch.uint8, dev, True), _vector("logp", logp, T, f32, dev),
                                     _vector("entropy", entropy, T, f32, dev, True), _status_word(device_status, dev),
                                     stream),
           "rl_loss_token_logp")
    return logp, entropy


def distill_loss(logits, teacher_ids, teacher_vals, mask, cu_seqlens, *, vocab: int | None = None, mode: str = "renorm",
                 direction: str = "forward", temperature: float = 1.0, scale: float = 1.0, tail_floor: float | None = None,
                 loss_norm: int = RL_NORM_PER_RESPONSE, loss=None, loss_f64=None, dlogits=None, kl=None, workspace=None,
                 device_status=None, stream=None) -> dict:
    """Distillation from a teacher's top logits, forward and backward: teacher_ids / teacher_vals [T, K] hold
    each row's entries (id -1: padding). mode "renorm" takes logits already divided by the temperature or
    log-probs, "tail" log-probs at the temperature (what they leave of the mass is one more outcome);
    direction "forward" is KL(teacher || student), "reverse" KL(student || teacher) ("tail" only). tail_floor
    bounds the teacher's remaining mass from below: 1e-9 in the reverse direction unless given, as an entry's
    log-prob of -0.0, or entries that sum to 1 in fp32, leave 0 and the divergence would be infinite; else 0. Returns
    loss [1], kl [T] and dlogits (allocated where not given; a new dlogits is 0 past the vocabulary, one that is given
    is not written there; dlogits may be logits itself). A workspace that is passed serves one call at a time:
    threads pass one each."""
    import torch
    if mode not in DISTILL_MODES or direction not in ("forward", "reverse"):
        raise ValueError("mode is 'renorm' or 'tail', direction 'forward' or 'reverse'")
    if tail_floor is None:
        tail_floor = REVERSE_TAIL_FLOOR if direction == "reverse" else 0.0
    code, V = _logits_code(logits, vocab, dlogits)
    if dlogits is None:
        dlogits = _gradient_of(logits, V, stream)
    T, S, dev, f32 = logits.shape[0], cu_seqlens.shape[0] - 1, logits.device, torch.float32
    for name, t, dt in (("teacher_ids", teacher_ids, torch.int32), ("teacher_vals", teacher_vals, f32)):
        if t.dtype != dt or t.dim() != 2 or t.shape[0] < T or t.device != dev or t.stride(1) != 1:
            raise ValueError(f"{name} is a {dt} tensor [tokens, entries] with contiguous rows on {dev}")
    if teacher_ids.shape != teacher_vals.shape or teacher_ids.stride(0) != teacher_vals.stride(0):
        raise ValueError("teacher_ids and teacher_vals have one shape and layout")
    with _allocations_of(stream, dev):
        loss, kl = _missing((loss, kl), (1, T), dev)
        if stream is None:
            stream = _current_stream(dev)
        if workspace is None:
            workspace = _post_workspace(rl_loss_distill_workspace_bytes(T, S), dev, stream)
    cfg = rl_loss_distill_config(code, V, teacher_ids.shape[1], DISTILL_MODES[mode], int(direction == "reverse"),
                                 loss_norm, temperature, scale, tail_floor)
    _check(load().rl_loss_distill(ctypes.byref(cfg), T, S, logits.data_ptr(), logits.stride(0), teacher_ids.data_ptr(),
                                  teacher_vals.data_ptr(), teacher_ids.stride(0),
                                  _vector("mask", mask, T, torch.uint8, dev),
                                  _vector("cu_seqlens", cu_seqlens, S + 1, torch.int32, dev),
                                  _vector("loss", loss, 1, f32, dev),
                                  _vector("loss_f64", loss_f64, 1, torch.float64, dev, True), dlogits.data_ptr(),
                                  dlogits.stride(0), _vector("kl", kl, T, f32, dev), *_workspace_of(workspace, dev),
                                  _status_word(device_status, dev), stream),
           "rl_loss_distill")
    return {"loss": loss, "kl": kl, "dlogits": dlogits}


def preference_loss(logits, targets, logp_ref, mask, cu_seqlens, *, vocab: int | None = None,
                    loss_type: str = "sigmoid", length_norm: bool = False, beta: float = 0.1, margin: float = 0.0,
                    label_smoothing: float = 0.0, nll_coef: float = 0.0, loss=None, loss_f64=None, dlogits=None,
                    logp=None, seq_logratio=None, pair_loss=None, workspace=None, device_status=None,
                    stream=None) -> dict:
    """Preference loss over pairs of responses (2j preferred to 2j + 1), forward and backward. logp_ref [T] are
    the reference policy's log-probs (None: no reference). Returns loss [1], logp [T], seq_logratio [S],
    pair_loss [S / 2] and dlogits (allocated where not given; a new dlogits is 0 past the vocabulary, one that is given
    is not written there; dlogits may be logits itself). A workspace that is passed serves one call at a time:
    threads pass one each."""
    import torch
    if loss_type not in PREF_LOSSES:
        raise ValueError("loss_type is 'sigmoid', 'hinge' or 'ipo'")
    code, V = _logits_code(logits, vocab, dlogits)
    if dlogits is None:
        dlogits = _gradient_of(logits, V, stream)
    T, S, dev, f32 = logits.shape[0], cu_seqlens.shape[0] - 1, logits.device, torch.float32
    with _allocations_of(stream, dev):
        P = max(S // 2, 0)
        loss, logp, seq_logratio, pair_loss = _missing((loss, logp, seq_logratio, pair_loss), (1, T, max(S, 0), P), dev)
        if stream is None:
            stream = _current_stream(dev)
        if workspace is None:
            workspace = _post_workspace(rl_loss_preference_workspace_bytes(T, S), dev, stream)
    cfg = rl_loss_pref_config(code, V, PREF_LOSSES[loss_type], int(length_norm), beta, margin, label_smoothing, nll_coef)
    _check(load().rl_loss_preference(ctypes.byref(cfg), T, S, logits.data_ptr(), logits.stride(0),
                                     _vector("targets", targets, T, torch.int32, dev),
                                     _vector("logp_ref", logp_ref, T, f32, dev, True),
                                     _vector("mask", mask, T, torch.uint8, dev),
                                     _vector("cu_seqlens", cu_seqlens, S + 1, torch.int32, dev),
                                     _vector("loss", loss, 1, f32, dev),
                                     _vector("loss_f64", loss_f64, 1, torch.float64, dev, True), dlogits.data_ptr(),
                                     dlogits.stride(0), _vector("logp", logp, T, f32, dev),
                                     _vector("seq_logratio", seq_logratio, S, f32, dev),
                                     _vector("pair_loss", pair_loss, S // 2, f32, dev), *_workspace_of(workspace, dev),
                                     _status_word(device_status, dev), stream),
           "rl_loss_preference")
    return {"loss": loss, "logp": logp, "seq_logratio": seq_logratio, "pair_loss": pair_loss, "dlogits": dlogits}


# ------------------------------------------------------------------ norms and 8-bit activation checkpoints

class Act8:
    """A matrix of activations kept in 8 bits: ``codes`` [rows, columns] and ``scales`` [rows, ceil(columns / 32)], both
    torch.uint8, in the format "int8" or "e4m3" (rl_act8 in the header says what they hold)."""

    __slots__ = ("shape", "format", "device", "_codes", "_scales", "_buffer", "_struct")

    def __init__(self, codes, scales, format: str):
        import torch
        if format not in ACT8_FORMATS:
            raise ValueError("format is 'int8' or 'e4m3'")
        if codes.dim() != 2 or not codes.is_cuda:
            raise ValueError("codes is a CUDA tensor [rows, columns]")
        rows, cols = codes.shape
        _check_sizes(rows, cols)
        blocks = (cols + ACT8_BLOCK - 1) // ACT8_BLOCK
        c, ld_codes = _like("codes", codes, rows, cols, torch.uint8, codes.device)
        s, ld_scales = _like("scales", scales, rows, blocks, torch.uint8, codes.device)
        self.shape, self.format, self.device = codes.shape, format, codes.device
        self._codes, self._scales, self._buffer = codes, scales, None
        self._struct = rl_act8(c, s, ld_codes, ld_scales, ACT8_FORMATS[format])

    @property
    def codes(self):
        if self._codes is None:
            rows, cols = self.shape
            ld = self._struct.ld_codes
            self._codes = self._buffer[:rows * ld].view(rows, ld)[:, :cols]
        return self._codes

    @property
    def scales(self):
        if self._scales is None:
            rows, first = self.shape[0], self.shape[0] * self._struct.ld_codes
            self._scales = self._buffer[first:].view(rows, self._struct.ld_scales)
        return self._scales

    @property
    def nbytes(self) -> int:
        rows, cols = self.shape
        return rows * (cols + (cols + ACT8_BLOCK - 1) // ACT8_BLOCK)


def act8_empty(rows: int, cols: int, format: str = "int8", device="cuda") -> Act8:
    """Room for rows x cols activations in 8 bits, rows of codes on 16-byte boundaries. (One allocation for both
    tensors, which are made when they are asked for: a tensor costs some 5 us of host time beside a launch.)"""
    import torch
    if format not in ACT8_FORMATS:
        raise ValueError("format is 'int8' or 'e4m3'")
    if rows < 0 or cols < 1:
        raise ValueError("an 8-bit checkpoint has a column at least")
    _check_sizes(rows, cols)
    ld, blocks = (cols + 15) & ~15, (cols + ACT8_BLOCK - 1) // ACT8_BLOCK
    a = Act8.__new__(Act8)
    a._buffer = torch.empty(rows * (ld + blocks), dtype=torch.uint8, device=device)
    a.shape, a.format, a.device, a._codes, a._scales = (rows, cols), format, a._buffer.device, None, None
    at = a._buffer.data_ptr()
    a._struct = rl_act8(at, at + rows * ld, ld, blocks, ACT8_FORMATS[format])
    return a


def _act8_struct(a: Act8, rows: int, cols: int, device) -> rl_act8:
    if not isinstance(a, Act8) or a.shape[0] != rows or a.shape[1] != cols or a.device.index != device.index:
        raise ValueError(f"an 8-bit checkpoint here is a capi.Act8 of [{rows}, {cols}] on {device}")
    return a._struct


def _float_code(name: str, dtype) -> int:
    import torch
    if dtype is torch.bfloat16:
        return RL_BF16
    if dtype is torch.float32:
        return RL_F32
    raise ValueError(f"{name} is torch.float32 or torch.bfloat16")


def _check_sizes(rows: int, cols: int) -> None:
    """The C entries take 32-bit sizes, and ctypes passes on the low 32 bits of a longer one."""
    if rows > 0x7fffffff or cols > 0x7fffffff:
        raise ValueError("a matrix has fewer than 2^31 rows and columns")


def _matrix(name: str, t):
    """(rows, cols, dtype code, pointer, row stride) of a CUDA matrix with contiguous rows."""
    if t.dim() != 2 or not t.is_cuda:
        raise ValueError(f"{name} is a CUDA tensor [rows, columns]")
    (rows, cols), (ld, step) = t.shape, t.stride()
    if (step != 1 and cols > 1) or (ld < cols and rows > 1):
        raise ValueError(f"the rows of {name} are contiguous and do not overlap")
    _check_sizes(rows, cols)
    return rows, cols, _float_code(name, t.dtype), t.data_ptr(), ld if rows > 1 else cols


def _like(name: str, t, rows: int, cols: int, dtype, device):
    """The pointer and row stride of a matrix of exactly this shape and type (None: no matrix)."""
    if t is None:
        return None, 0
    if t.dtype is dtype and t.dim() == 2 and t.get_device() == device.index:
        (have, width), (ld, step) = t.shape, t.stride()
        if have == rows and width == cols and (step == 1 or cols == 1) and (ld >= cols or rows < 2):
            return t.data_ptr(), ld if rows > 1 else cols
    raise ValueError(f"{name} is a {dtype} tensor [{rows}, {cols}] with contiguous rows that do not overlap on {device}")


def _rows_like(t, cols: int, dtype, device):
    """A new matrix with rows as those of t [rows, columns]: without gaps, or else on 32-byte boundaries."""
    import torch
    rows, ld = t.shape[0], t.stride(0)
    if ld == cols or rows < 2:
        return torch.empty((rows, cols), dtype=dtype, device=device)
    per = 8 if dtype is torch.float32 else 16
    return torch.empty((rows, (cols + per - 1) // per * per), dtype=dtype, device=device)[:, :cols]


def _params(weight, bias, cols: int, device):
    """(dtype code, pointer of weight, pointer of bias) of a norm's parameters."""
    p = weight if weight is not None else bias
    if p is None:
        return RL_F32, None, None
    code, dt = _float_code("weight", p.dtype), p.dtype
    return (code, _vector("weight", weight, cols, dt, device, True),
            _vector("bias, of the weight's type", bias, cols, dt, device, True))


def _on_device(device):
    """The context that makes a tensor's device the current one for a launch."""
    import torch
    return _NO_CONTEXT if torch._C._cuda_getDevice() == device.index else torch.cuda.device(device)


def rl_loss_layer_norm_max_cols() -> int:
    return int(load().rl_loss_layer_norm_max_cols())


@functools.lru_cache(maxsize=256)
def rl_loss_layer_norm_workspace_bytes(rows: int, cols: int) -> int:
    return int(load().rl_loss_layer_norm_workspace_bytes(int(rows), int(cols)))


def layer_norm(x, weight=None, bias=None, *, kind: str = "layer", eps: float = 1e-5, residual=None, mask=None, y=None,
               dtype=None, summed=None, checkpoint=None, mean=None, rstd=None, want_stats: bool = False,
               device_status=None, stream=None) -> dict:
    """Layer norm (or, with kind "rms", RMS norm) of the rows of x [rows, columns] on the GPU, after adding `residual`
    where there is one. Returns y (of type `dtype`, that of x unless given), summed (x + residual; None without a
    residual unless a tensor is passed), mean and rstd [rows] (with want_stats; no mean for "rms") and checkpoint: `checkpoint`
    is an Act8, or "int8" or "e4m3" for a new one, that receives the norm's input in 8 bits for layer_norm_backward. Rows whose mask
    is 0 are not read and give 0. y may be x or the residual, and so may summed. New matrices have rows like those of x:
    without gaps, or else on 32-byte boundaries."""
    import torch
    if kind not in LN_KINDS:
        raise ValueError("kind is 'layer' or 'rms'")
    rows, cols, xt, px, ldx = _matrix("x", x)
    dev, xdt, f32 = x.device, x.dtype, torch.float32
    pt, pw, pb = _params(weight, bias, cols, dev)
    with _allocations_of(stream, dev):
        if y is None:
            y = _rows_like(x, cols, dtype or xdt, dev)
            py, ldy, ydt = y.data_ptr(), y.stride(0), y.dtype
        else:
            ydt = y.dtype
            if dtype is not None and ydt is not dtype:
                raise ValueError("y has the type that dtype names")
            py, ldy = _like("y", y, rows, cols, ydt, dev)
        if summed is None and residual is not None:
            summed = _rows_like(x, cols, xdt, dev)
        if want_stats:
            if rstd is None:
                rstd = torch.empty(rows, dtype=f32, device=dev)
            if mean is None and kind == "layer":
                mean = torch.empty(rows, dtype=f32, device=dev)
        if isinstance(checkpoint, str):
            checkpoint = act8_empty(rows, cols, checkpoint, dev)
        if stream is None:
            stream = _current_stream(dev)
    pr, ldr = (None, 0) if residual is None else _like("residual", residual, rows, cols, xdt, dev)
    ps, lds = (None, 0) if summed is None else _like("summed", summed, rows, cols, xdt, dev)
    cfg = rl_ln_config(LN_KINDS[kind], cols, xt, xt if ydt is xdt else _float_code("y", ydt), pt, eps)
    with _on_device(dev):
        _check(load().rl_loss_layer_norm(cfg, rows, px, ldx, pr, ldr, pw, pb,
                                         None if mask is None else _vector("mask", mask, rows, torch.uint8, dev), py, ldy, ps, lds,
                                         None if checkpoint is None else _act8_struct(checkpoint, rows, cols, dev),
                                         None if mean is None else _vector("mean", mean, rows, f32, dev),
                                         None if rstd is None else _vector("rstd", rstd, rows, f32, dev),
                                         None if device_status is None else _status_word(device_status, dev), stream),
               "rl_loss_layer_norm")
    return {"y": y, "summed": summed, "mean": mean, "rstd": rstd, "checkpoint": checkpoint}


def layer_norm_backward(dy, weight, mean, rstd, *, x=None, checkpoint=None, kind: str = "layer", dtype=None, mask=None,
                        dsummed=None, dx=None, dweight=None, dbias=None, want_dweight: bool = True, want_dbias: bool = False,
                        accumulate: bool = False, bias=None, y=None, workspace=None, device_status=None,
                        stream=None) -> dict:
    """The backward pass of layer_norm: gradients of its input (dx, and of the residual, which is the same), weight and
    bias from dy. The input comes as x (with a residual: `summed`) or as the 8-bit `checkpoint`; mean (None for "rms") and rstd are the
    forward pass's. dsummed is the gradient that comes along the residual stream, added to dx. dx has the type of x (from a checkpoint: `dtype`, that of dy unless given). dweight (unless
    want_dweight is False) and dbias (with want_dbias, or where it is passed) are fp32; with accumulate they are
    added to. A tensor y receives the forward pass's output made again (with `bias`, if there was one). Rows whose mask is 0 are not
    read and give 0. dx may be dy, x or dsummed (a new one has rows like those of dy). A workspace that is passed serves one call at a time."""
    import torch
    if kind not in LN_KINDS:
        raise ValueError("kind is 'layer' or 'rms'")
    if (x is None) == (checkpoint is None):
        raise ValueError("the norm's input comes as x or as a checkpoint")
    rows, cols, yt, pdy, lddy = _matrix("dy", dy)
    dev, ydt, f32 = dy.device, dy.dtype, torch.float32
    if x is not None:
        if dtype is not None and dtype is not x.dtype:
            raise ValueError("dx has the type of x")
        dtype = x.dtype
    elif dtype is None:
        dtype = dx.dtype if dx is not None else ydt
    pt, pw, pb = _params(weight, bias, cols, dev)
    if accumulate and ((want_dweight and dweight is None) or (want_dbias and dbias is None)):
        raise ValueError("pass the dweight and dbias that are added to")
    with _allocations_of(stream, dev):
        if dx is None:
            dx = _rows_like(dy, cols, dtype, dev)
            pdx, lddx = dx.data_ptr(), dx.stride(0)
        else:
            pdx, lddx = _like("dx", dx, rows, cols, dtype, dev)
        if dweight is None and want_dweight:
            dweight = torch.empty(cols, dtype=f32, device=dev)
        if dbias is None and want_dbias:
            dbias = torch.empty(cols, dtype=f32, device=dev)
        if stream is None:
            stream = _current_stream(dev)
        if workspace is None and (dweight is not None or dbias is not None):
            workspace = _post_workspace(rl_loss_layer_norm_workspace_bytes(rows, cols), dev, stream)
    px, ldx = (None, 0) if x is None else _like("x", x, rows, cols, dtype, dev)
    ps, lds = (None, 0) if dsummed is None else _like("dsummed", dsummed, rows, cols, dtype, dev)
    py, ldy = (None, 0) if y is None else _like("y", y, rows, cols, ydt, dev)
    pws, ws_bytes = (None, 0) if workspace is None else _workspace_of(workspace, dev)
    cfg = rl_ln_config(LN_KINDS[kind], cols, yt if dtype is ydt else _float_code("dx", dtype), yt, pt, 0.0)
    with _on_device(dev):
        _check(load().rl_loss_layer_norm_backward(
            cfg, rows, pdy, lddy, px, ldx, None if checkpoint is None else _act8_struct(checkpoint, rows, cols, dev), pw, pb,
            None if mask is None else _vector("mask", mask, rows, torch.uint8, dev), _vector("mean", mean, rows, f32, dev, kind == "rms"),
            _vector("rstd", rstd, rows, f32, dev), ps, lds, pdx, lddx,
            None if dweight is None else _vector("dweight", dweight, cols, f32, dev),
            None if dbias is None else _vector("dbias", dbias, cols, f32, dev), int(accumulate), py, ldy, pws, ws_bytes,
            None if device_status is None else _status_word(device_status, dev), stream), "rl_loss_layer_norm_backward")
    return {"dx": dx, "dweight": dweight, "dbias": dbias, "y": y}


def act8_pack(x, *, format: str = "int8", out: Act8 | None = None, stream=None) -> Act8:
    """The activations x [rows, columns] in 8 bits, in a new Act8 or in `out`."""
    rows, cols, xt, px, ldx = _matrix("x", x)
    dev = x.device
    if out is None:
        with _allocations_of(stream, dev):
            out = act8_empty(rows, cols, format, dev)
    if stream is None:
        stream = _current_stream(dev)
    with _on_device(dev):
        _check(load().rl_loss_act8_pack(xt, rows, cols, px, ldx, _act8_struct(out, rows, cols, dev), stream),
               "rl_loss_act8_pack")
    return out


def act8_unpack(a: Act8, *, dtype=None, out=None, stream=None):
    """The activations that an Act8 stands for, as torch.bfloat16 (or `dtype`), in a new tensor or in `out`."""
    import torch
    (rows, cols), dev = a.shape, a.device
    if out is None:
        with _allocations_of(stream, dev):
            out = torch.empty((rows, cols), dtype=dtype or torch.bfloat16, device=dev)
        po, ldo = out.data_ptr(), cols
    elif dtype is not None and out.dtype is not dtype:
        raise ValueError("out has the type that dtype names")
    else:
        po, ldo = _like("out", out, rows, cols, out.dtype, dev)
    if stream is None:
        stream = _current_stream(dev)
    with _on_device(dev):
        _check(load().rl_loss_act8_unpack(_float_code("out", out.dtype), rows, cols, a._struct, po, ldo, stream),
               "rl_loss_act8_unpack")
    return out


def rl_loss_version() -> int:
    return int(load().rl_loss_version())


# ------------------------------------------------------------------ torch-facing wrapper

def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


class RlLoss:
    """One handle: fixed vocabulary, group size, hyper-parameters and capacity."""

    def __init__(self, vocab_size: int, group_size: int, max_tokens: int, max_seqs: int, logits_dtype: int,
                 eps_low: float = 0.2, eps_high: float = 0.28, beta: float = 2.0, adv_eps: float = 1e-6,
                 adv_mode: int = RL_ADV_GROUP_REWARDS, std_unbiased: bool = False, pop_indicator: bool = False,
                 objective: int = RL_OBJ_GRPO_ICEPOP, loss_norm: int = RL_NORM_PER_RESPONSE, dis_stopgrad: bool = True):
        self.config = rl_loss_config(vocab_size, group_size, max_tokens, max_seqs, eps_low, eps_high, beta,
                                     adv_eps, adv_mode, int(std_unbiased), int(pop_indicator), logits_dtype,
                                     objective, loss_norm, int(dis_stopgrad))
        self.handle = rl_loss_create(self.config)

    def close(self):
        if self.handle:
            rl_loss_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def forward_backward(self, logits, targets, logp_old, logp_infer, mask, cu_seqlens, rewards_or_adv, *,
                         loss, dlogits, loss_f64=None, logp=None, entropy=None, flags=None, seq_adv=None,
                         counts=None, mean_entropy=None, stream=None) -> None:
        """Enqueue one forward+backward on ``stream`` (default: torch's current
        stream). All tensors are caller-owned CUDA tensors."""
        import torch
        T = int(targets.shape[0])
        S = int(cu_seqlens.shape[0]) - 1
        inp = rl_loss_inputs(T, S, int(logits.stride(0)) if logits.dim() == 2 else 0, _ptr(logits), _ptr(targets),
                             _ptr(logp_old), _ptr(logp_infer), _ptr(mask), _ptr(cu_seqlens), _ptr(rewards_or_adv))
        out = rl_loss_outputs(_ptr(loss), _ptr(loss_f64), _ptr(dlogits),
                              int(dlogits.stride(0)) if dlogits.dim() == 2 else 0, _ptr(logp), _ptr(entropy),
                              _ptr(flags), _ptr(seq_adv), _ptr(counts), _ptr(mean_entropy))
        if stream is None:
            stream = torch.cuda.current_stream().cuda_stream
        code = rl_loss_forward_backward(self.handle, inp, out, stream)
        if code == CODES["RL_ERR_CUDA"]:
            raise RlLossError(code, "rl_loss_forward_backward (%s)" % rl_loss_last_cuda_error(self.handle))
        _check(code, "rl_loss_forward_backward")

    def forward_backward_from_host(self, host: dict, device: dict, *, loss, dlogits, num_chunks: int = 8,
                                   loss_f64=None, logp=None, entropy=None, flags=None, seq_adv=None, counts=None,
                                   mean_entropy=None, stream=None) -> None:
        """Enqueue one forward+backward whose inputs start in host memory: ``host`` and ``device``
        map the input names (logits, targets, logp_old, logp_infer, mask, cu_seqlens,
        rewards_or_adv) to pinned CPU tensors and to CUDA tensors of the same shapes that receive
        them. The logits go over in ``num_chunks`` row blocks, each computed as soon as it lands."""
        import torch

        def inputs(d):
            lg = d["logits"]
            return rl_loss_inputs(int(d["targets"].shape[0]), int(d["cu_seqlens"].shape[0]) - 1,
                                  int(lg.stride(0)) if lg.dim() == 2 else 0, _ptr(lg), _ptr(d["targets"]),
                                  _ptr(d["logp_old"]), _ptr(d["logp_infer"]), _ptr(d["mask"]), _ptr(d["cu_seqlens"]),
                                  _ptr(d["rewards_or_adv"]))
        out = rl_loss_outputs(_ptr(loss), _ptr(loss_f64), _ptr(dlogits),
                              int(dlogits.stride(0)) if dlogits.dim() == 2 else 0, _ptr(logp), _ptr(entropy),
                              _ptr(flags), _ptr(seq_adv), _ptr(counts), _ptr(mean_entropy))
        if stream is None:
            stream = torch.cuda.current_stream().cuda_stream
        self._raise(rl_loss_forward_backward_from_host(self.handle, inputs(host), inputs(device), out, num_chunks,
                                                       stream), "rl_loss_forward_backward_from_host")

    def forward_backward_kl(self, logits, targets, logp_old, logp_infer, mask, cu_seqlens, rewards_or_adv, logp_ref, *,
                            kl_coef: float, kl_estimator: str = "k3", loss, dlogits, loss_f64=None, logp=None,
                            entropy=None, flags=None, seq_adv=None, counts=None, mean_entropy=None, kl=None,
                            mean_kl=None, stream=None) -> None:
        """forward_backward with a KL term to a reference policy (its log-probs logp_ref [T]): kl_coef times the
        "k1", "k2" or "k3" estimate of every mask = 1 token. kl [T] and mean_kl [1] receive the estimates."""
        import torch
        if kl_estimator not in KL_ESTIMATORS:
            raise ValueError("kl_estimator is 'k1', 'k2' or 'k3'")
        if not logits.is_cuda:
            raise ValueError("logits is a CUDA tensor [tokens, vocabulary] of the handle's type")
        T, S, V = targets.numel(), cu_seqlens.numel() - 1, self.config.vocab_size
        dev, f32, i32, u8 = logits.device, torch.float32, torch.int32, torch.uint8
        dt = torch.bfloat16 if self.config.logits_dtype == RL_BF16 else f32
        z, ld = _rows("logits", logits, T, V, dt, dev)
        dz, ldd = _rows("dlogits", dlogits, T, V, dt, dev)
        inp = rl_loss_inputs(T, S, ld, z, _vector("targets", targets, T, i32, dev), _vector("logp_old", logp_old, T, f32, dev),
                             _vector("logp_infer", logp_infer, T, f32, dev), _vector("mask", mask, T, u8, dev),
                             _vector("cu_seqlens", cu_seqlens, S + 1, i32, dev),
                             _vector("rewards_or_adv", rewards_or_adv, T if self.config.adv_mode >= RL_ADV_PER_TOKEN else S,
                                     f32, dev))
        out = rl_loss_outputs(_vector("loss", loss, 1, f32, dev), _vector("loss_f64", loss_f64, 1, torch.float64, dev, True),
                              dz, ldd, _vector("logp", logp, T, f32, dev, True),
                              _vector("entropy", entropy, T, f32, dev, True), _vector("flags", flags, T, u8, dev, True),
                              _vector("seq_adv", seq_adv, S, f32, dev, True), _vector("counts", counts, 4, i32, dev, True),
                              _vector("mean_entropy", mean_entropy, 1, f32, dev, True))
        term = rl_loss_kl(_vector("logp_ref", logp_ref, T, f32, dev), kl_coef, KL_ESTIMATORS[kl_estimator],
                          _vector("kl", kl, T, f32, dev, True), _vector("mean_kl", mean_kl, 1, f32, dev, True))
        if stream is None:
            stream = _current_stream(dev)
        code = load().rl_loss_forward_backward_kl(self.handle, ctypes.byref(inp), ctypes.byref(term), ctypes.byref(out),
                                                  stream)
        if code:
            self._raise(code, "rl_loss_forward_backward_kl")

    def _raise(self, code: int, what: str):
        if code == CODES["RL_ERR_CUDA"]:
            raise RlLossError(code, "%s (%s)" % (what, rl_loss_last_cuda_error(self.handle)))
        _check(code, what)

    def projection_setup(self, hidden_dim: int, chunk_tokens: int) -> None:
        rl_loss_projection_setup(self.handle, hidden_dim, chunk_tokens)

    def projection_logits(self, hidden, w_lm, rows: int, logits, stream=None) -> None:
        """logits[:rows] (fp32) = hidden[:rows] @ w_lm^T on the tensor cores."""
        import torch
        if stream is None:
            stream = torch.cuda.current_stream().cuda_stream
        self._raise(rl_loss_projection_logits(self.handle, _ptr(hidden), hidden.stride(0), _ptr(w_lm), w_lm.stride(0),
                                              rows, _ptr(logits), logits.stride(0), stream),
                    "rl_loss_projection_logits")

    def fused_projection_forward_backward(self, hidden, w_lm, targets, logp_old, logp_infer, mask, cu_seqlens,
                                          rewards_or_adv, *, loss, dhidden, dw_lm, loss_f64=None, logp=None,
                                          entropy=None, flags=None, seq_adv=None, counts=None, mean_entropy=None,
                                          stream=None) -> None:
        import torch
        T = int(targets.shape[0])
        S = int(cu_seqlens.shape[0]) - 1
        inp = rl_loss_inputs(T, S, 0, None, _ptr(targets), _ptr(logp_old), _ptr(logp_infer), _ptr(mask),
                             _ptr(cu_seqlens), _ptr(rewards_or_adv))
        out = rl_loss_outputs(_ptr(loss), _ptr(loss_f64), None, 0, _ptr(logp), _ptr(entropy), _ptr(flags),
                              _ptr(seq_adv), _ptr(counts), _ptr(mean_entropy))
        if stream is None:
            stream = torch.cuda.current_stream().cuda_stream
        self._raise(rl_loss_fused_projection_forward_backward(
            self.handle, _ptr(hidden), hidden.stride(0), _ptr(w_lm), w_lm.stride(0), inp, _ptr(dhidden),
            dhidden.stride(0), _ptr(dw_lm), dw_lm.stride(0), out, stream), "rl_loss_fused_projection_forward_backward")

    def normed_projection_forward_backward(self, x, norm_weight, w_lm, targets, logp_old, logp_infer, mask, cu_seqlens,
                                           rewards_or_adv, *, loss, dx, dw_lm, dnorm_weight=None, norm_bias=None,
                                           dnorm_bias=None, kind: str = "rms", eps: float = 1e-5, loss_f64=None, logp=None,
                                           entropy=None, flags=None, seq_adv=None, counts=None, mean_entropy=None,
                                           workspace=None, stream=None) -> None:
        """fused_projection_forward_backward of the model's last norm of x [T, hidden size] (kind "rms" or "layer"), whose output and
        its gradient exist for one chunk of rows at a time. dx [T, hidden size] (may be x) is the gradient of x,
        dnorm_weight and dnorm_bias [hidden size] fp32 those of the norm's parameters."""
        import torch
        if kind not in LN_KINDS:
            raise ValueError("kind is 'layer' or 'rms'")
        T, cols, xt, px, ldx = _matrix("x", x)
        dev, f32, i32, u8, bf16 = x.device, torch.float32, torch.int32, torch.uint8, torch.bfloat16
        S, V = cu_seqlens.numel() - 1, self.config.vocab_size
        pt, pw, pb = _params(norm_weight, norm_bias, cols, dev)
        pdx, lddx = _like("dx", dx, T, cols, x.dtype, dev)
        w, ldw = _rows("w_lm", w_lm, V, cols, bf16, dev)
        dw, lddw = _rows("dw_lm", dw_lm, V, cols, f32, dev)
        inp = rl_loss_inputs(T, S, 0, None, _vector("targets", targets, T, i32, dev), _vector("logp_old", logp_old, T, f32, dev),
                             _vector("logp_infer", logp_infer, T, f32, dev), _vector("mask", mask, T, u8, dev),
                             _vector("cu_seqlens", cu_seqlens, S + 1, i32, dev),
                             _vector("rewards_or_adv", rewards_or_adv, T if self.config.adv_mode >= RL_ADV_PER_TOKEN else S,
                                     f32, dev))
        out = rl_loss_outputs(_vector("loss", loss, 1, f32, dev), _vector("loss_f64", loss_f64, 1, torch.float64, dev, True),
                              None, 0, _vector("logp", logp, T, f32, dev, True),
                              _vector("entropy", entropy, T, f32, dev, True), _vector("flags", flags, T, u8, dev, True),
                              _vector("seq_adv", seq_adv, S, f32, dev, True), _vector("counts", counts, 4, i32, dev, True),
                              _vector("mean_entropy", mean_entropy, 1, f32, dev, True))
        norm = rl_loss_final_norm(px, ldx, pw, pb, pdx, lddx, _vector("dnorm_weight", dnorm_weight, cols, f32, dev, True),
                                  _vector("dnorm_bias", dnorm_bias, cols, f32, dev, True))
        if stream is None:
            stream = _current_stream(dev)
        if workspace is None:
            with _allocations_of(stream, dev):
                workspace = _post_workspace(load().rl_loss_normed_projection_workspace_bytes(self.handle), dev, stream)
        cfg = rl_ln_config(LN_KINDS[kind], cols, xt, RL_BF16, pt, eps)
        code = load().rl_loss_normed_projection_forward_backward(self.handle, cfg, norm, w, ldw, inp, dw, lddw, out,
                                                                 *_workspace_of(workspace, dev), stream)
        if code:
            self._raise(code, "rl_loss_normed_projection_forward_backward")

    def device_status(self, stream=None) -> int:
        import torch
        if stream is None:
            stream = torch.cuda.current_stream().cuda_stream
        return rl_loss_get_device_status(self.handle, stream)

    def profile_start(self, max_calls: int):
        rl_loss_profile_start(self.handle, max_calls)

    def profile_read(self) -> dict:
        return rl_loss_profile_read(self.handle)

    def launch_count(self) -> int:
        return rl_loss_launch_count(self.handle)


def status_bits_to_names(bits: int) -> list[str]:
    return [STATUS_NAMES[c] for c in sorted(STATUS_NAMES) if c and bits & (1 << c)]


# ------------------------------------------------------------------ batch helpers

def handle_for_batch(batch, max_tokens: int | None = None, max_seqs: int | None = None, **overrides) -> RlLoss:
    """A handle configured for a ``synthetic.Batch`` (capacity = the batch's size)."""
    kw = dict(eps_low=batch.eps_low, eps_high=batch.eps_high, beta=batch.beta, adv_eps=batch.adv_eps,
              adv_mode=batch.adv_mode, objective=batch.objective, loss_norm=batch.loss_norm)
    kw.update(overrides)
    return RlLoss(batch.vocab, batch.group, max(1, max_tokens or batch.num_tokens), max_seqs or batch.num_seqs,
                  RL_BF16 if batch.dtype == "bf16" else RL_F32, **kw)


def alloc_outputs(batch, in_place: bool = False, ld: int | None = None) -> dict:
    """Caller-owned output tensors for one call on ``batch`` (on its device)."""
    import torch
    dev = batch.logits.device
    T, S = batch.num_tokens, batch.num_seqs
    if in_place:
        dlogits = batch.logits
    else:
        ld = ld or batch.logits.stride(0)
        dlogits = torch.empty((T, ld), dtype=batch.logits.dtype, device=dev)
    return dict(loss=torch.empty(1, dtype=torch.float32, device=dev),
                loss_f64=torch.empty(1, dtype=torch.float64, device=dev), dlogits=dlogits,
                logp=torch.empty(T, dtype=torch.float32, device=dev),
                entropy=torch.empty(T, dtype=torch.float32, device=dev),
                flags=torch.empty(T, dtype=torch.uint8, device=dev),
                seq_adv=torch.empty(S, dtype=torch.float32, device=dev),
                counts=torch.empty(4, dtype=torch.int32, device=dev),
                mean_entropy=torch.empty(1, dtype=torch.float32, device=dev))


def run_batch(rl: RlLoss, batch, outputs: dict, stream=None) -> dict:
    """One forward+backward of ``batch`` into ``outputs`` (asynchronous)."""
    adv = batch.token_adv if (batch.adv_mode >= RL_ADV_PER_TOKEN) else batch.rewards_or_adv
    rl.forward_backward(batch.logits, batch.targets, batch.logp_old, batch.logp_infer, batch.mask,
                        batch.cu_seqlens, adv, stream=stream, **outputs)
    return outputs


INPUT_NAMES = ("logits", "targets", "logp_old", "logp_infer", "mask", "cu_seqlens", "rewards_or_adv")


def batch_inputs(batch) -> dict:
    """The input tensors of ``batch`` by name (the advantage array the batch's mode reads)."""
    adv = batch.token_adv if (batch.adv_mode >= RL_ADV_PER_TOKEN) else batch.rewards_or_adv
    return {n: (adv if n == "rewards_or_adv" else getattr(batch, n)) for n in INPUT_NAMES}


def run_batch_from_host(rl: RlLoss, host: dict, device: dict, outputs: dict, num_chunks: int = 8,
                        stream=None) -> dict:
    """One forward+backward from pinned host inputs ``host`` into the device buffers ``device``."""
    rl.forward_backward_from_host(host, device, num_chunks=num_chunks, stream=stream, **outputs)
    return outputs


def projection_handle(pb, max_tokens: int | None = None, **overrides) -> RlLoss:
    """A bf16 handle with the fused projection path set up for a ``synthetic.ProjBatch``."""
    rl = handle_for_batch(pb.batch, max_tokens=max_tokens, **overrides)
    rl.projection_setup(pb.hidden_dim, pb.chunk)
    return rl


def alloc_projection_outputs(pb) -> dict:
    import torch
    b = pb.batch
    out = alloc_outputs(b, ld=8)
    del out["dlogits"]
    dev = pb.hidden.device
    out["dhidden"] = torch.empty_like(pb.hidden)
    out["dw_lm"] = torch.empty((pb.w.shape[0], pb.w.shape[1]), dtype=torch.float32, device=dev)
    return out


def run_projection(rl: RlLoss, pb, outputs: dict, stream=None) -> dict:
    b = pb.batch
    adv = b.token_adv if (b.adv_mode >= RL_ADV_PER_TOKEN) else b.rewards_or_adv
    rl.fused_projection_forward_backward(pb.hidden, pb.w, b.targets, b.logp_old, b.logp_infer, b.mask, b.cu_seqlens,
                                         adv, stream=stream, **outputs)
    return outputs
