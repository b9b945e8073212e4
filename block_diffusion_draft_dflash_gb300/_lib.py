"""ctypes binding of libdflash.so (include/dflash.h).

Argument marshalling only: every function takes torch tensors that already live on the
GPU, checks dtype / device / contiguity, and passes raw pointers plus the current CUDA
stream to the C ABI.  Nothing here computes any part of the speculative step, and there
is no fallback: if the library is missing the import fails loudly.
"""
from __future__ import annotations

import ctypes as C
import os

import torch

from . import build as _build

c_i32p = C.POINTER(C.c_int32)


class StatusError(RuntimeError):
    def __init__(self, fn, code):
        super().__init__(f"{fn} failed: {code} ({status_string(code)})")
        self.code = code


class ModelCfg(C.Structure):
    _fields_ = [("n_layers", C.c_int32), ("d_model", C.c_int32), ("n_q_heads", C.c_int32),
                ("n_kv_heads", C.c_int32), ("head_dim", C.c_int32), ("d_ff", C.c_int32), ("vocab", C.c_int32),
                ("n_feat_layers", C.c_int32), ("feat_layers", C.c_int32 * 8), ("block_size", C.c_int32),
                ("mask_id", C.c_int32), ("rms_eps", C.c_float), ("rope_theta", C.c_float),
                ("n_experts", C.c_int32), ("top_k", C.c_int32), ("d_expert", C.c_int32)]


class LayerWeights(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("attn_norm", "w_qkv", "q_norm", "k_norm", "w_o", "mlp_norm",
                                          "w_gate_up", "w_down", "w_router", "w_experts_gate_up",
                                          "w_experts_down")]


class ModelWeights(C.Structure):
    _fields_ = [("layers", C.POINTER(LayerWeights)), ("final_norm", C.c_void_p), ("embed", C.c_void_p),
                ("fc", C.c_void_p), ("fc_norm", C.c_void_p)]


class Kv4CacheStruct(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("k_codes", "k_scales", "v_codes", "v_scales")] + \
               [(n, C.c_int32) for n in ("n_layers", "b", "Hkv", "hd", "cap", "k_exp", "v_exp")]


class RowsStruct(C.Structure):
    _fields_ = [("data", C.c_void_p), ("dtype", C.c_int32), ("rows", C.c_int32), ("V", C.c_int32), ("ld", C.c_int64)]


_lib = None

_SIGS = {
    "dflash_status_string": (C.c_char_p, [C.c_int]),
    "dflash_check_device": (C.c_int, []),
    "dflash_workspace_status": (C.c_int, [C.c_void_p, C.c_void_p]),
    "dflash_trace_enable": (C.c_int, [C.c_int]),
    "dflash_trace_read": (C.c_int, [C.c_int, C.c_char_p, C.POINTER(C.c_double), C.POINTER(C.c_int)]),
    "ddtree_build_workspace_size": (C.c_size_t, [C.c_int] * 4),
    "ddtree_build": (C.c_int, [C.c_void_p, C.c_int, C.c_int, C.c_int, C.c_int] + [C.c_void_p] * 7 +
                     [C.c_size_t, C.c_void_p]),
    "ddtree_build_static": (C.c_int, [C.c_void_p, C.c_int, C.c_int, C.c_int, C.c_int] + [C.c_void_p] * 7),
    "dflash_chain_build_workspace_size": (C.c_size_t, [C.c_int, C.c_int]),
    "dflash_chain_build": (C.c_int, [C.c_void_p, C.c_int, C.c_int, C.c_int] + [C.c_void_p] * 7 +
                           [C.c_size_t, C.c_void_p]),
    "tree_verify_attention_workspace_size": (C.c_size_t, [C.c_int] * 6),
    "tree_verify_attention": (C.c_int, [C.c_int] * 5 + [C.c_void_p] * 3 + [C.c_int, C.c_void_p, C.c_void_p,
                              C.c_float, C.c_void_p, C.c_void_p, C.c_size_t, C.c_void_p]),
    "accept_and_compact_workspace_size": (C.c_size_t, [C.c_int, C.c_int]),
    "accept_and_compact": (C.c_int, [C.c_int, C.c_int] + [C.c_void_p] * 5 + [C.c_int] * 4 + [C.c_void_p] * 2 +
                           [C.c_int, C.c_void_p, C.c_int] + [C.c_void_p] * 6 + [C.c_size_t, C.c_void_p]),
    "dflash_target_tree_forward_workspace_size": (C.c_size_t, [C.c_void_p, C.c_int, C.c_int]),
    "dflash_target_tree_forward": (C.c_int, [C.c_void_p, C.c_void_p, C.c_int, C.c_int] + [C.c_void_p] * 5 +
                                   [C.c_int] + [C.c_void_p] * 4 + [C.c_size_t, C.c_void_p]),
    "dflash_target_tree_forward_sampled": (C.c_int, [C.c_void_p, C.c_void_p, C.c_int, C.c_int] + [C.c_void_p] * 5 +
                                           [C.c_int, C.c_void_p, C.c_float, C.c_ulonglong] + [C.c_void_p] * 3 +
                                           [C.c_size_t, C.c_void_p]),
    "dflash_target_tree_forward_filtered_workspace_size": (C.c_size_t, [C.c_void_p, C.c_int, C.c_int]),
    "dflash_target_tree_forward_filtered": (C.c_int, [C.c_void_p, C.c_void_p, C.c_int, C.c_int] + [C.c_void_p] * 5 +
                                            [C.c_int] + [C.c_void_p] * 5 + [C.c_ulonglong, C.c_int, C.c_float] +
                                            [C.c_void_p] * 6 + [C.c_size_t, C.c_void_p]),
    "dflash_path_rows": (C.c_int, [C.c_int] * 3 + [C.c_void_p] * 2 + [C.c_int] + [C.c_void_p] * 3),
    "dflash_target_expert_counts": (C.c_int, [C.c_void_p, C.c_int, C.c_int, C.c_void_p, C.c_size_t, C.c_void_p,
                                              C.c_void_p]),
    "dflash_linear_workspace_size": (C.c_size_t, []),
    "dflash_linear_argmax_workspace_size": (C.c_size_t, [C.c_int]),
    "dflash_linear_argmax": (C.c_int, [C.c_void_p, C.c_void_p, C.c_int, C.c_int, C.c_int, C.c_void_p,
                                       C.c_void_p, C.c_size_t, C.c_void_p]),
    "dflash_linear_sample_workspace_size": (C.c_size_t, [C.c_int]),
    "dflash_linear_sample": (C.c_int, [C.c_void_p, C.c_void_p, C.c_int, C.c_int, C.c_int, C.c_float, C.c_ulonglong,
                                       C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_size_t, C.c_void_p]),
    "dflash_linear": (C.c_int, [C.c_void_p, C.c_void_p, C.c_int, C.c_int, C.c_int, C.c_void_p, C.c_int,
                      C.c_void_p, C.c_size_t, C.c_void_p]),
    "dflash_linear_logsoftmax_workspace_size": (C.c_size_t, [C.c_int, C.c_int]),
    "dflash_linear_logsoftmax": (C.c_int, [C.c_void_p, C.c_void_p, C.c_int, C.c_int, C.c_int, C.c_void_p,
                                           C.c_void_p, C.c_size_t, C.c_void_p]),
    "dflash_workspace_configure": (C.c_int, [C.c_void_p, C.c_ulonglong, C.c_int, C.c_void_p]),
    "dflash_plant_logprobs": (C.c_int, [C.c_void_p, C.c_int, C.c_int, C.c_int, C.c_void_p, C.c_int, C.c_void_p,
                                        C.c_float, C.c_float, C.c_float, C.c_ulonglong, C.c_void_p]),
    "dflash_draft_block_workspace_size": (C.c_size_t, [C.c_void_p, C.c_int, C.c_int]),
    "dflash_draft_block": (C.c_int, [C.c_void_p, C.c_void_p, C.c_int, C.c_void_p, C.c_int] + [C.c_void_p] * 4 +
                           [C.c_int] + [C.c_void_p] * 3 + [C.c_size_t, C.c_void_p]),
    "dflash_kv4_append_workspace_size": (C.c_size_t, []),
    "dflash_kv4_append": (C.c_int, [C.c_void_p, C.c_int, C.c_void_p, C.c_void_p, C.c_int] + [C.c_void_p] * 5 +
                          [C.c_size_t, C.c_void_p]),
    "dflash_kv4_attention_workspace_size": (C.c_size_t, [C.c_void_p, C.c_int, C.c_int]),
    "dflash_kv4_attention": (C.c_int, [C.c_void_p, C.c_int, C.c_int, C.c_int] + [C.c_void_p] * 3 + [C.c_float] +
                             [C.c_void_p] * 3 + [C.c_size_t, C.c_void_p]),
    "dflash_kv4_attention_weights_workspace_size": (C.c_size_t, [C.c_void_p, C.c_int, C.c_int]),
    "dflash_kv4_attention_weights": (C.c_int, [C.c_void_p, C.c_int, C.c_int, C.c_int] + [C.c_void_p] * 5 +
                                     [C.c_int, C.c_float, C.c_float] + [C.c_void_p] * 3 + [C.c_size_t, C.c_void_p]),
    "dflash_kv4_compact_workspace_size": (C.c_size_t, []),
    "dflash_kv4_compact": (C.c_int, [C.c_void_p, C.c_void_p, C.c_int] + [C.c_void_p] * 3 + [C.c_size_t, C.c_void_p]),
    "dflash_kv4_evict_workspace_size": (C.c_size_t, [C.c_void_p, C.c_int]),
    "dflash_kv4_evict": (C.c_int, [C.c_void_p] * 3 + [C.c_int] * 3 + [C.c_void_p] * 5 + [C.c_size_t, C.c_void_p]),
    "dflash_sample_workspace_size": (C.c_size_t, [C.c_int, C.c_int]),
    "dflash_sample": (C.c_int, [C.c_void_p, C.c_int] + [C.c_void_p] * 9 + [C.c_size_t, C.c_void_p]),
    "dflash_top_logits_workspace_size": (C.c_size_t, [C.c_int, C.c_int]),
    "dflash_top_logits": (C.c_int, [C.c_void_p, C.c_int, C.c_float] + [C.c_void_p] * 4 + [C.c_size_t, C.c_void_p]),
    "dflash_distill_workspace_size": (C.c_size_t, [C.c_int, C.c_int]),
    "dflash_distill": (C.c_int, [C.c_void_p, C.c_int, C.c_int] + [C.c_void_p] * 4 + [C.c_float] + [C.c_void_p] * 4 +
                       [C.c_int64, C.c_void_p, C.c_size_t, C.c_void_p]),
    "dflash_distill_backward": (C.c_int, [C.c_void_p, C.c_int, C.c_int] + [C.c_void_p] * 4 + [C.c_float] +
                                [C.c_void_p] * 4 + [C.c_int64, C.c_void_p, C.c_size_t, C.c_void_p]),
}


def lib_path() -> str:
    return _build.LIB


def load(build_if_missing: bool = True):
    """Load libdflash.so (building it first if needed) and declare the C signatures."""
    global _lib
    if _lib is not None:
        return _lib
    if build_if_missing and not _build.up_to_date():
        _build.build()
    if not os.path.exists(_build.LIB):
        raise ImportError(f"libdflash.so not built at {_build.LIB}")
    lib = C.CDLL(_build.LIB)
    for name, (res, args) in _SIGS.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    _lib = lib
    return lib


def status_string(code: int) -> str:
    return load().dflash_status_string(code).decode()


def _p(t):
    return None if t is None else C.c_void_p(t.data_ptr())


def _stream():
    return C.c_void_p(torch.cuda.current_stream().cuda_stream)


def _check(fn, rc):
    if rc != 0:
        raise StatusError(fn, rc)


def _dev(t, dtype, name):
    if t is None:
        return
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


class Workspace:
    """A device scratch buffer for one of the calls (256-byte aligned via torch)."""

    def __init__(self, nbytes: int, device="cuda"):
        self.nbytes = int(nbytes)
        self.buf = torch.zeros(max(self.nbytes, 256), dtype=torch.uint8, device=device)

    @property
    def ptr(self):
        return C.c_void_p(self.buf.data_ptr())

    def status(self) -> int:
        return load().dflash_workspace_status(self.ptr, _stream())

    def configure(self, wait_limit_ns: int = 0, hold: bool = False):
        """Failure-path settings (see dflash_workspace_configure)."""
        _check("dflash_workspace_configure",
               load().dflash_workspace_configure(self.ptr, int(wait_limit_ns), int(hold), _stream()))


# ----------------------------------------------------------------------------- calls
def ddtree_build_workspace_size(b, D, V, B):
    return load().ddtree_build_workspace_size(b, D, V, B)


def ddtree_build(logprobs, B, out, ws: Workspace, root_tok=None):
    """logprobs [b][D][V] fp32 -> out dict of tok/parent/depth/score/anc tensors (preallocated)."""
    b, D, V = logprobs.shape
    _dev(logprobs, torch.float32, "logprobs")
    for k in ("tok", "parent", "depth"):
        _dev(out[k], torch.int32, k)
    _dev(out["score"], torch.float32, "score")
    _dev(out["anc"], torch.int32, "anc")
    _dev(root_tok, torch.int32, "root_tok")
    _check("ddtree_build", load().ddtree_build(
        _p(logprobs), b, D, V, B, _p(root_tok), _p(out["tok"]), _p(out["parent"]), _p(out["depth"]),
        _p(out["score"]), _p(out["anc"]), ws.ptr, ws.nbytes, _stream()))


def ddtree_build_static(logprobs, B, out, root_tok=None):
    """ddtree_build without a workspace (the library's fixed device scratch; see dflash.h)."""
    b, D, V = logprobs.shape
    _dev(logprobs, torch.float32, "logprobs")
    for k in ("tok", "parent", "depth"):
        _dev(out[k], torch.int32, k)
    _dev(out["score"], torch.float32, "score")
    _dev(out["anc"], torch.int32, "anc")
    _dev(root_tok, torch.int32, "root_tok")
    _check("ddtree_build_static", load().ddtree_build_static(
        _p(logprobs), b, D, V, B, _p(root_tok), _p(out["tok"]), _p(out["parent"]), _p(out["depth"]),
        _p(out["score"]), _p(out["anc"]), _stream()))


def chain_build_workspace_size(b, D):
    return load().dflash_chain_build_workspace_size(b, D)


def chain_build(logprobs, out, ws: Workspace, root_tok=None):
    """logprobs [b][D][V] fp32 -> the argmax chain in out (tok/parent/depth/score/anc, D+1 nodes)."""
    b, D, V = logprobs.shape
    _dev(logprobs, torch.float32, "logprobs")
    for k in ("tok", "parent", "depth"):
        _dev(out[k], torch.int32, k)
    _dev(out["score"], torch.float32, "score")
    _dev(out["anc"], torch.int32, "anc")
    _dev(root_tok, torch.int32, "root_tok")
    _check("dflash_chain_build", load().dflash_chain_build(
        _p(logprobs), b, D, V, _p(root_tok), _p(out["tok"]), _p(out["parent"]), _p(out["depth"]),
        _p(out["score"]), _p(out["anc"]), ws.ptr, ws.nbytes, _stream()))


def tree_verify_attention_workspace_size(b, n_tree, Hq, Hkv, hd, cap):
    return load().tree_verify_attention_workspace_size(b, n_tree, Hq, Hkv, hd, cap)


def tree_verify_attention(q, k_cache, v_cache, cache_len, anc, scale, out, ws: Workspace):
    b, T, Hq, hd = q.shape
    Hkv, cap = k_cache.shape[1], k_cache.shape[2]
    for t, n in ((q, "q"), (k_cache, "k_cache"), (v_cache, "v_cache"), (out, "out")):
        _dev(t, torch.bfloat16, n)
    _dev(cache_len, torch.int32, "cache_len")
    _dev(anc, torch.int32, "anc")
    _check("tree_verify_attention", load().tree_verify_attention(
        b, T, Hq, Hkv, hd, _p(q), _p(k_cache), _p(v_cache), cap, _p(cache_len), _p(anc), float(scale), _p(out),
        ws.ptr, ws.nbytes, _stream()))


def accept_and_compact_workspace_size(b, n_tree):
    return load().accept_and_compact_workspace_size(b, n_tree)


def accept_and_compact(choice, tok, parent, k_cache, v_cache, cache_len, tree_feat, new_feat, out, ws: Workspace,
                       cap=None):
    """k_cache [L][b][Hkv][cap][hd], v_cache [L][b][Hkv][hd][cap]; out: n_new, acc_tok, n_acc, new_bonus, src_slot.
    k_cache, v_cache None: the walk alone; cap is then the slots of the cache that kv4_compact moves."""
    b, T = choice.shape
    nl, Hkv, cap, hd = (k_cache.shape[0], k_cache.shape[2], k_cache.shape[3], k_cache.shape[4]) \
        if k_cache is not None else (0, 1, 1 if cap is None else cap, 128)
    max_new = out["acc_tok"].shape[1]
    feat_dim = tree_feat.shape[-1] if tree_feat is not None else 0
    _check("accept_and_compact", load().accept_and_compact(
        b, T, _p(choice), _p(tok), _p(parent), _p(k_cache), _p(v_cache), nl, Hkv, hd, cap, _p(cache_len),
        _p(tree_feat), feat_dim, _p(new_feat), max_new, _p(out["n_new"]), _p(out["acc_tok"]), _p(out["n_acc"]),
        _p(out["new_bonus"]), _p(out["src_slot"]), ws.ptr, ws.nbytes, _stream()))


def target_tree_forward_workspace_size(cfg: ModelCfg, b, n_tree):
    return load().dflash_target_tree_forward_workspace_size(C.byref(cfg), b, n_tree)


def target_tree_forward(cfg: ModelCfg, weights: ModelWeights, tok, depth, anc, k_cache, v_cache, cache_len, choice,
                        tree_feat, ws: Workspace, temperature: float = 0.0, seed: int = 0):
    """temperature 0: the greedy choice per node; > 0: the target's temperature draw per node
    (dflash_target_tree_forward_sampled, keyed to seed, sequence and position)."""
    b, T = tok.shape
    cap = k_cache.shape[3]
    if temperature > 0:
        _check("dflash_target_tree_forward_sampled", load().dflash_target_tree_forward_sampled(
            C.byref(cfg), C.byref(weights), b, T, _p(tok), _p(depth), _p(anc), _p(k_cache), _p(v_cache), cap,
            _p(cache_len), float(temperature), seed & 0xFFFFFFFFFFFFFFFF, _p(choice), _p(tree_feat), ws.ptr,
            ws.nbytes, _stream()))
        return
    _check("dflash_target_tree_forward", load().dflash_target_tree_forward(
        C.byref(cfg), C.byref(weights), b, T, _p(tok), _p(depth), _p(anc), _p(k_cache), _p(v_cache), cap,
        _p(cache_len), _p(choice), _p(tree_feat), ws.ptr, ws.nbytes, _stream()))


def target_tree_forward_filtered_workspace_size(cfg: ModelCfg, b, n_tree):
    return load().dflash_target_tree_forward_filtered_workspace_size(C.byref(cfg), b, n_tree)


def target_tree_forward_filtered(cfg: ModelCfg, weights: ModelWeights, tok, depth, anc, k_cache, v_cache, cache_len,
                                 choice, tree_feat, ws: Workspace, temperature=None, top_k=None, top_p=None, min_p=None,
                                 seed: int = 0, top_id=None, top_val=None, top_lse=None, top_temperature: float = 1.0):
    """The choice per node drawn under its sequence's settings (fp32 and int32 [b], or None; keyed to seed, sequence and
    position); top_id, top_val [b][n_tree][K] and top_lse [b][n_tree] (optional) take every node's first K tokens."""
    b, T = tok.shape
    for t, name in ((temperature, "temperature"), (top_p, "top_p"), (min_p, "min_p"), (top_val, "top_val"),
                    (top_lse, "top_lse")):
        _dev(t, torch.float32, name)
    for t, name in ((top_k, "top_k"), (top_id, "top_id"), (choice, "choice")):
        _dev(t, torch.int32, name)
    for t, name in ((temperature, "temperature"), (top_k, "top_k"), (top_p, "top_p"), (min_p, "min_p")):
        if t is not None and tuple(t.shape) != (b,):
            raise ValueError(f"{name} must have one entry for each of {b} sequences")
    K = 0 if top_id is None else top_id.shape[-1]
    if K and (tuple(top_id.shape) != (b, T, K) or top_val is None or tuple(top_val.shape) != (b, T, K) or
              (top_lse is not None and tuple(top_lse.shape) != (b, T))):
        raise ValueError(f"top_id and top_val must be [{b}][{T}][K], top_lse [{b}][{T}]")
    _check("dflash_target_tree_forward_filtered", load().dflash_target_tree_forward_filtered(
        C.byref(cfg), C.byref(weights), b, T, _p(tok), _p(depth), _p(anc), _p(k_cache), _p(v_cache), k_cache.shape[3],
        _p(cache_len), _p(temperature), _p(top_k), _p(top_p), _p(min_p), seed & 0xFFFFFFFFFFFFFFFF, K,
        float(top_temperature), _p(top_id), _p(top_val), _p(top_lse), _p(choice), _p(tree_feat), ws.ptr, ws.nbytes,
        _stream()))


def path_rows(n_new, src_slot, cache_len, n_tree, teacher_row):
    """teacher_row [b][D]: the nodes of the accepted path (n_new, src_slot, cache_len as accept_and_compact left them)
    whose logits stand for draft positions 1 .. D; -1 behind the path."""
    for t, name in ((n_new, "n_new"), (src_slot, "src_slot"), (cache_len, "cache_len"), (teacher_row, "teacher_row")):
        _dev(t, torch.int32, name)
    b, D = teacher_row.shape
    if n_new.shape != (b,) or cache_len.shape != (b,) or src_slot.dim() != 2 or src_slot.shape[0] != b:
        raise ValueError(f"n_new, cache_len [{b}] and src_slot [{b}][max] are wanted")
    _check("dflash_path_rows", load().dflash_path_rows(
        b, D, n_tree, _p(n_new), _p(src_slot), src_slot.shape[1], _p(cache_len), _p(teacher_row), _stream()))


def target_expert_counts(cfg: ModelCfg, b, n_tree, ws: Workspace, counts):
    """counts [n_layers][n_experts] int32 <- the last mixture-of-experts tree forward's routing."""
    _dev(counts, torch.int32, "counts")
    _check("dflash_target_expert_counts", load().dflash_target_expert_counts(
        C.byref(cfg), b, n_tree, ws.ptr, ws.nbytes, _p(counts), _stream()))


def draft_block_workspace_size(cfg: ModelCfg, b, max_new):
    return load().dflash_draft_block_workspace_size(C.byref(cfg), b, max_new)


def draft_block(cfg: ModelCfg, weights: ModelWeights, new_feat, n_new, ctx_k, ctx_v, ctx_len, bonus, logprobs,
                ws: Workspace):
    b = bonus.shape[0]
    max_new = new_feat.shape[1] if new_feat is not None else 0
    cap = ctx_k.shape[3]
    _check("dflash_draft_block", load().dflash_draft_block(
        C.byref(cfg), C.byref(weights), b, _p(new_feat), max_new, _p(n_new), _p(ctx_k), _p(ctx_v), _p(ctx_len), cap,
        _p(bonus), _p(logprobs), ws.ptr, ws.nbytes, _stream()))


def linear(X, W, out, accumulate=False, ws: Workspace = None):
    """out (+)= X W^T; X [M][K] bf16, W [N][K] bf16, out [M][N] fp32."""
    _dev(X, torch.bfloat16, "X")
    _dev(W, torch.bfloat16, "W")
    _dev(out, torch.float32, "out")
    ws = ws or Workspace(load().dflash_linear_workspace_size(), X.device)
    M, K = X.shape
    N = W.shape[0]
    _check("dflash_linear", load().dflash_linear(_p(X), _p(W), M, N, K, _p(out), int(accumulate), ws.ptr,
                                                 ws.nbytes, _stream()))
    return ws


def linear_argmax(X, W, out, ws: Workspace = None):
    """out[t] = argmax_n (X W^T)[t][n] (lowest n on ties); X [M][K] bf16, W [N][K] bf16, out [M] int32."""
    _dev(X, torch.bfloat16, "X")
    _dev(W, torch.bfloat16, "W")
    _dev(out, torch.int32, "out")
    M, K = X.shape
    N = W.shape[0]
    ws = ws or Workspace(load().dflash_linear_argmax_workspace_size(M), X.device)
    _check("dflash_linear_argmax", load().dflash_linear_argmax(_p(X), _p(W), M, N, K, _p(out), ws.ptr, ws.nbytes,
                                                               _stream()))
    return ws


def linear_sample(X, W, temperature, seed, row_seq, row_pos, out, ws: Workspace = None):
    """out[t] = the temperature draw of row t from softmax((X W^T)[t] / T), keyed to
    (seed, row_seq[t], row_pos[t]); X [M][K] bf16, W [N][K] bf16, row_seq/row_pos/out [M] int32."""
    _dev(X, torch.bfloat16, "X")
    _dev(W, torch.bfloat16, "W")
    for t, name in ((row_seq, "row_seq"), (row_pos, "row_pos"), (out, "out")):
        _dev(t, torch.int32, name)
    M, K = X.shape
    N = W.shape[0]
    ws = ws or Workspace(load().dflash_linear_sample_workspace_size(M), X.device)
    _check("dflash_linear_sample", load().dflash_linear_sample(
        _p(X), _p(W), M, N, K, float(temperature), seed & 0xFFFFFFFFFFFFFFFF, _p(row_seq), _p(row_pos), _p(out),
        ws.ptr, ws.nbytes, _stream()))
    return ws


def linear_logsoftmax(X, W, out, ws: Workspace = None):
    """out[t] = log_softmax(X W^T)[t] (fp32); X [M][K] bf16, W [N][K] bf16, out [M][N] fp32."""
    _dev(X, torch.bfloat16, "X")
    _dev(W, torch.bfloat16, "W")
    _dev(out, torch.float32, "out")
    M, K = X.shape
    N = W.shape[0]
    ws = ws or Workspace(load().dflash_linear_logsoftmax_workspace_size(M, N), X.device)
    _check("dflash_linear_logsoftmax", load().dflash_linear_logsoftmax(_p(X), _p(W), M, N, K, _p(out), ws.ptr,
                                                                       ws.nbytes, _stream()))
    return ws


# ------------------------------------------------------------------- KV cache held in 4 bits
class Kv4Cache:
    """A KV cache held in 4 bits (df_kv4_cache): four uint8 tensors and two exponents.

    k_codes, v_codes [n_layers][b][Hkv][cap][64]; k_scales, v_scales [n_layers][b][Hkv][cap][8];
    a value is 2^exp * scale (e4m3) * code (e2m1), one scale for 16 values."""

    def __init__(self, k_codes, k_scales, v_codes, v_scales, k_exp=0, v_exp=0):
        if k_codes.dim() != 5 or k_codes.shape[4] != 64:
            raise ValueError("k_codes must be [n_layers][b][Hkv][cap][64]")
        rows = k_codes.shape[:4]
        for t, last, name in ((k_codes, 64, "k_codes"), (k_scales, 8, "k_scales"), (v_codes, 64, "v_codes"),
                              (v_scales, 8, "v_scales")):
            _dev(t, torch.uint8, name)
            if t.device != k_codes.device or tuple(t.shape) != (*rows, last):
                raise ValueError(f"{name} must be [n_layers][b][Hkv][cap][{last}] on {k_codes.device}")
        self.k_codes, self.k_scales, self.v_codes, self.v_scales = k_codes, k_scales, v_codes, v_scales
        self.n_layers, self.b, self.n_kv_heads, self.cap = rows
        self.k_exp, self.v_exp = int(k_exp), int(v_exp)
        self.device, self.index = k_codes.device, k_codes.get_device()
        self.rows = tuple(rows)
        self.struct = Kv4CacheStruct(k_codes.data_ptr(), k_scales.data_ptr(), v_codes.data_ptr(), v_scales.data_ptr(),
                                     *rows[:3], 128, rows[3], self.k_exp, self.v_exp)
        self.ref = C.addressof(self.struct)

    @classmethod
    def empty(cls, n_layers, b, n_kv_heads, cap, k_exp=0, v_exp=0, device="cuda"):
        z = lambda last: torch.zeros(n_layers, b, n_kv_heads, cap, last, dtype=torch.uint8, device=device)
        return cls(z(64), z(8), z(64), z(8), k_exp, v_exp)

    def _arg(self, t, dtype, shape, name):
        """Address of an argument that lies on the cache's device (None: 0)."""
        if t is None:
            return 0
        if t.dtype is not dtype or t.get_device() != self.index or t.shape != shape or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {list(shape)} on {self.device}")
        return t.data_ptr()

    def _ws(self, ws):
        """A call's workspace and stream: the current stream of the current device, which has to be the cache's."""
        dev = self.index
        if torch._C._cuda_getDevice() != dev or ws.buf.get_device() != dev:
            raise ValueError(f"the current device and the workspace's have to be the cache's ({self.device})")
        return ws.buf.data_ptr(), ws.nbytes, torch._C._cuda_getCurrentRawStream(dev)


def kv4_append_workspace_size():
    return load().dflash_kv4_append_workspace_size()


def kv4_append(cache: Kv4Cache, layer, k, v, cache_len, ws: Workspace, n_new=None, k_held=None, v_held=None):
    """Rounds k, v [b][n][Hkv][128] bf16 into slots cache_len[s] .. of one layer (n_new [b]: rows per sequence);
    k_held, v_held (optional, like k) take the values that the cache then stands for."""
    b, n = cache.b, k.shape[1]
    shape = (b, n, cache.n_kv_heads, 128)
    arg, bf, i32 = cache._arg, torch.bfloat16, torch.int32
    _check("dflash_kv4_append", load().dflash_kv4_append(
        cache.ref, layer, arg(k, bf, shape, "k"), arg(v, bf, shape, "v"), n, arg(n_new, i32, (b,), "n_new"),
        arg(cache_len, i32, (b,), "cache_len"), arg(k_held, bf, shape, "k_held"), arg(v_held, bf, shape, "v_held"),
        *cache._ws(ws)))


def kv4_attention_workspace_size(cache: Kv4Cache, n_tree, Hq):
    return load().dflash_kv4_attention_workspace_size(cache.ref, n_tree, Hq)


def kv4_attention(cache: Kv4Cache, layer, q, cache_len, anc, scale, out, ws: Workspace, lse=None):
    """Tree attention over one layer of the cache; q, out [b][T][Hq][128] bf16, anc [b][T][ceil(T/32)] int32 or
    None (a chain), lse (optional) [b][T][Hq] fp32."""
    b, T, Hq, _ = shape = tuple(q.shape)
    arg, bf, i32 = cache._arg, torch.bfloat16, torch.int32
    if b != cache.b or shape[3] != 128:
        raise ValueError(f"q must be [{cache.b}][T][Hq][128]")
    _check("dflash_kv4_attention", load().dflash_kv4_attention(
        cache.ref, layer, T, Hq, arg(q, bf, shape, "q"), arg(cache_len, i32, (b,), "cache_len"),
        arg(anc, i32, (b, T, (T + 31) // 32), "anc"), scale, arg(out, bf, shape, "out"),
        arg(lse, torch.float32, shape[:3], "lse"), *cache._ws(ws)))


def kv4_attention_weights_workspace_size(cache: Kv4Cache, n_tree, Hq):
    return load().dflash_kv4_attention_weights_workspace_size(cache.ref, n_tree, Hq)


def kv4_attention_weights(cache: Kv4Cache, layer, q, lse, cache_len, scale, score, ws: Workspace, n_rows=None,
                          src_slot=None, decay=1.0, score_out=None):
    """score_out = decay * score + the attention weight of the rows that stayed (see dflash.h); score and score_out
    [n_layers][b][Hkv][cap] fp32, score_out None: in place.  n_rows and src_slot are accept_and_compact's n_new and
    src_slot, cache_len its new length."""
    b, T, Hq, _ = shape = tuple(q.shape)
    arg, i32, f32 = cache._arg, torch.int32, torch.float32
    if b != cache.b or shape[3] != 128:
        raise ValueError(f"q must be [{cache.b}][T][Hq][128]")
    max_src = 0 if src_slot is None else src_slot.shape[1]
    sc = arg(score, f32, cache.rows, "score")
    length, src = arg(cache_len, i32, (b,), "cache_len"), arg(src_slot, i32, (b, max_src), "src_slot")
    if src_slot is not None and max_src == 0:
        src = length        # lists without entries: not the NULL that an empty tensor's address is; never read
    _check("dflash_kv4_attention_weights", load().dflash_kv4_attention_weights(
        cache.ref, layer, T, Hq, arg(q, torch.bfloat16, shape, "q"), arg(lse, f32, shape[:3], "lse"),
        length, arg(n_rows, i32, (b,), "n_rows"), src, max_src, scale, decay, sc,
        sc if score_out is None else arg(score_out, f32, cache.rows, "score_out"), *cache._ws(ws)))


def kv4_compact_workspace_size():
    return load().dflash_kv4_compact_workspace_size()


def kv4_compact(cache: Kv4Cache, src_slot, n_acc, cache_len, ws: Workspace):
    """Moves the accepted path's rows in every layer; src_slot [b][max], n_acc, cache_len as accept_and_compact
    left them."""
    b, i32, max_src = cache.b, torch.int32, src_slot.shape[1]
    _check("dflash_kv4_compact", load().dflash_kv4_compact(
        cache.ref, cache._arg(src_slot, i32, (b, max_src), "src_slot"), max_src, cache._arg(n_acc, i32, (b,), "n_acc"),
        cache._arg(cache_len, i32, (b,), "cache_len"), *cache._ws(ws)))


def kv4_evict_workspace_size(cache: Kv4Cache, budget):
    return load().dflash_kv4_evict_workspace_size(cache.ref, budget)


def kv4_evict(cache: Kv4Cache, score, cache_len, budget, n_sink, n_recent, to: Kv4Cache, score_out, new_len, kept,
              ws: Workspace):
    """Copies the slots that stay (n_sink first, n_recent last, then the largest scores) to another cache; kept
    [n_layers][b][Hkv][budget] int32 lists them, new_len [b] may be cache_len; score_out may be None."""
    arg, i32, f32 = cache._arg, torch.int32, torch.float32
    if to.device != cache.device:
        raise ValueError("both caches have to lie on one device")
    _check("dflash_kv4_evict", load().dflash_kv4_evict(
        cache.ref, arg(score, f32, cache.rows, "score"), arg(cache_len, i32, (cache.b,), "cache_len"), budget, n_sink,
        n_recent, to.ref, arg(score_out, f32, to.rows, "score_out"), arg(new_len, i32, (cache.b,), "new_len"),
        arg(kept, i32, (*cache.rows[:3], budget), "kept"), *cache._ws(ws)))


# ------------------------------------------------------------------------- rows of logits
_ROW_TYPES = {torch.float32: 0, torch.bfloat16: 1}
_current_device, _current_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream


def _rows(t, ws, name):
    """(df_rows, device, rows, V, workspace and stream) of a call's rows [rows][V] (fp32 or bf16, any row stride), which
    have to lie on the current device, like its other arguments."""
    dtype, index = _ROW_TYPES.get(t.dtype), t.get_device()
    if dtype is None or index < 0 or t.dim() != 2:
        raise ValueError(f"{name} must be a CUDA tensor [rows][V], fp32 or bf16")
    n, V = t.shape
    ld, step = t.stride()
    if step != 1 and V > 1:
        raise ValueError(f"{name} must have a row's values next to each other")
    buf = ws.buf
    if _current_device() != index or buf.get_device() != index:
        raise ValueError(f"the current device and the workspace's have to be that of {name}")
    return (RowsStruct(t.data_ptr(), dtype, n, V, ld if n > 1 else V), index, n, V,
            (buf.data_ptr(), ws.nbytes, _current_stream(index)))


def _at(t, dtype, index, shape, name):
    """Address of an argument that lies on device `index` (None: 0)."""
    if t is None:
        return 0
    if t.dtype is not dtype or t.get_device() != index or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {list(shape)} on the rows' device")
    return t.data_ptr()


def _rows_out(t, dtype, index, n, V, name):
    """Address and row stride of an output shaped like the rows (None: 0)."""
    if t is None:
        return 0, 0
    if t.dtype is not dtype or t.get_device() != index or t.shape != (n, V):
        raise ValueError(f"{name} must be a {dtype} tensor [{n}][{V}] on the rows' device")
    ld, step = t.stride()
    if step != 1 and V > 1:
        raise ValueError(f"{name} must have a row's values next to each other")
    return t.data_ptr(), ld if n > 1 else V


def sample_workspace_size(rows, V):
    return load().dflash_sample_workspace_size(rows, V)


def sample(logits, u, token, ws: Workspace, temperature=None, top_k=None, top_p=None, min_p=None, group=1, logprob=None,
           n_kept=None):
    """token[r] = the token of row r of logits [rows][V] (fp32 or bf16) drawn with u[r] under temperature, top-k, top-p
    and min-p (see dflash.h); settings [rows / group] (row r: r / group) or None: 1, 0, 1, 0."""
    x, dev, rows, _, where = _rows(logits, ws, "logits")
    if group < 1 or rows % group:
        raise ValueError(f"{rows} rows are not groups of {group}")
    f32, i32, n, each = torch.float32, torch.int32, (rows,), (rows // group,)
    _check("dflash_sample", load().dflash_sample(
        C.addressof(x), group, _at(temperature, f32, dev, each, "temperature"), _at(top_k, i32, dev, each, "top_k"),
        _at(top_p, f32, dev, each, "top_p"), _at(min_p, f32, dev, each, "min_p"), _at(u, f32, dev, n, "u"),
        _at(token, i32, dev, n, "token"), _at(logprob, f32, dev, n, "logprob"), _at(n_kept, i32, dev, n, "n_kept"), *where))


def top_logits_workspace_size(rows, V):
    return load().dflash_top_logits_workspace_size(rows, V)


def top_logits(logits, temperature, id, val, lse, ws: Workspace):
    """The K first tokens of every row of logits [rows][V] (id, val [rows][K] int32, fp32) and, at the temperature, the
    log-sum of all of it (lse [rows] fp32, may be None)."""
    x, dev, rows, _, where = _rows(logits, ws, "logits")
    shape = (rows, id.shape[1])
    _check("dflash_top_logits", load().dflash_top_logits(
        C.addressof(x), shape[1], temperature, _at(id, torch.int32, dev, shape, "id"), _at(val, torch.float32, dev, shape, "val"),
        _at(lse, torch.float32, dev, shape[:1], "lse"), *where))


def distill_workspace_size(rows, V):
    return load().dflash_distill_workspace_size(rows, V)


def distill(student, id, val, lse, temperature, loss, stats, ws: Workspace, teacher_row=None, weight=None, grad=None):
    """loss [rows] of student rows [rows][V] (fp32 or bf16) against a teacher's lists id, val [lists][K] and lse [lists]
    (None: the lists are all there is), with stats [rows][4] for distill_backward and, where grad is given (like student, or
    student itself), the gradient of the losses' sum.  teacher_row [rows]: each row's list, -1: none."""
    x, dev, rows, V, where = _rows(student, ws, "student")
    f32, i32, n, shape = torch.float32, torch.int32, (rows,), id.shape
    _check("dflash_distill", load().dflash_distill(
        C.addressof(x), shape[1], shape[0], _at(id, i32, dev, shape, "id"), _at(val, f32, dev, shape, "val"),
        _at(lse, f32, dev, shape[:1], "lse"), _at(teacher_row, i32, dev, n, "teacher_row"), temperature,
        _at(weight, f32, dev, n, "weight"), _at(loss, f32, dev, n, "loss"), _at(stats, f32, dev, (rows, 4), "stats"),
        *_rows_out(grad, student.dtype, dev, rows, V, "grad"), *where))


def distill_backward(student, id, val, lse, temperature, stats, grad, ws: Workspace, grad_loss=None, teacher_row=None,
                     weight=None):
    """grad (like student, or student itself) = the gradient of sum grad_loss loss by the student's rows, from the arguments
    and the stats of distill."""
    x, dev, rows, V, where = _rows(student, ws, "student")
    f32, i32, n, shape = torch.float32, torch.int32, (rows,), id.shape
    _check("dflash_distill_backward", load().dflash_distill_backward(
        C.addressof(x), shape[1], shape[0], _at(id, i32, dev, shape, "id"), _at(val, f32, dev, shape, "val"),
        _at(lse, f32, dev, shape[:1], "lse"), _at(teacher_row, i32, dev, n, "teacher_row"), temperature,
        _at(weight, f32, dev, n, "weight"), _at(stats, f32, dev, (rows, 4), "stats"), _at(grad_loss, f32, dev, n, "grad_loss"),
        *_rows_out(grad, student.dtype, dev, rows, V, "grad"), *where))


def plant_logprobs(logprobs, ref, pos, rate, bias, seed, miss_bias=0.0):
    """Harness: plant agreement with reference tokens (see dflash_plant_logprobs).
    ref [b][n_pos][D] int32: tokens expected at depths 1..D of a block starting at position p."""
    _dev(logprobs, torch.float32, "logprobs")
    _dev(ref, torch.int32, "ref")
    _dev(pos, torch.int32, "pos")
    b, D, V = logprobs.shape
    assert ref.shape[0] == b and ref.shape[2] == D
    _check("dflash_plant_logprobs", load().dflash_plant_logprobs(
        _p(logprobs), b, D, V, _p(ref), ref.shape[1], _p(pos), float(rate), float(bias), float(miss_bias), int(seed),
        _stream()))


def trace_enable(on=True):
    load().dflash_trace_enable(int(on))


def trace_read(max_entries=128):
    """{tag: (total ms, launches)} since the last read (synchronises).  A tag is the kernel
    class, optionally followed by a space and the launch shape."""
    names = C.create_string_buffer(64 * max_entries)
    ms = (C.c_double * max_entries)()
    cnt = (C.c_int * max_entries)()
    n = load().dflash_trace_read(max_entries, names, ms, cnt)
    if n < 0:
        raise StatusError("dflash_trace_read", n)
    raw = names.raw
    return {raw[64 * i:64 * i + 64].split(b"\0")[0].decode(): (ms[i], cnt[i]) for i in range(n)}


def exported_symbols():
    """Names declared in include/dflash.h (used by the load/export test)."""
    return list(_SIGS)
