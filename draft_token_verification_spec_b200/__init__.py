"""Python binding of libspecverify (draft-token verification for speculative decoding).

Argument marshalling only: every step of verification runs in the CUDA library
(libspecverify.so, built in-tree for sm_100a). PyTorch supplies device memory and
streams. The functions carry the C ABI's names (include/specverify.h); each takes
torch CUDA tensors, allocates any output or workspace the caller did not pass, and
enqueues the work on the current CUDA stream (or `stream`). Calling any of them
without the built library raises; there is no fallback implementation.
"""
from __future__ import annotations

import ctypes
import os
import re

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libspecverify.so")
HEADER_PATH = os.path.join(os.path.dirname(_PKG), "include", "specverify.h")

SPEC_F32, SPEC_BF16 = 0, 1
SPEC_OK = 0
SPEC_ERR_INVALID_ARG, SPEC_ERR_UNSUPPORTED, SPEC_ERR_CUDA, SPEC_ERR_WORKSPACE = -1, -2, -3, -4
SPEC_ERR_DEVICE_TIMEOUT = -5
SPEC_MAX_VOCAB = 1 << 20
SPEC_MAX_TREE_NODES = 4096
SPEC_MAX_TOP_LOGITS = 256

_lib = None


class SpecError(RuntimeError):
    """A libspecverify call returned a non-zero spec_status."""

    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} returned {status} ({status_string(status)})")
        self.status = status


def _declare(lib):
    P, I, F, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    L = ctypes.c_int64
    sig = {
        "spec_status_string": ([I], ctypes.c_char_p),
        "spec_workspace_size": ([I, I, I], Z),
        "spec_verify_chain": ([P, P, I, I, I, I, P, P, F, I, F, P, P, P, Z, P], I),
        "spec_verify_chain_noalloc": ([P, P, I, I, I, I, P, P, F, I, F, P, P, P], I),
        "spec_verify_tree_typical": ([P, I, I, I, I, P, P, F, F, P, I, P, P, Z, P], I),
        "spec_verify_tree_greedy": ([P, I, I, I, I, P, P, P, I, P, P, P, Z, P], I),
        "spec_verify_tree_sampling": ([P, P, I, I, I, I, P, P, P, F, I, F, P, I, P, P, P, Z, P],
                                      I),
        "spec_logits_to_probs": ([P, I, I, I, F, I, F, P, P, P], I),
        "spec_residual_sample": ([P, P, I, I, P, P, P], I),
        "spec_get_device_status": ([P, P, P], I),
        "spec_linear_state_factors": ([P, P, P, P, I, I, I, I, I, P, P, P, P], I),
        "spec_lmhead_workspace_size": ([I, I, I, I, I], Z),
        "spec_verify_chain_lmhead": ([P, P, P, P, I, I, I, I, P, P, F, I, P, P, P, P, Z, P], I),
        "spec_commit_linear_state": ([P, I, I, I, I, I, P, P, P, P, P, P], I),
        "spec_sample_workspace_size": ([I, I], Z),
        "spec_sample": ([P, I, I, I, L, P, F, I, F, F, P, P, P, P, P, P, P, Z, P], I),
        "spec_top_logits_workspace_size": ([I, I, I], Z),
        "spec_top_logits": ([P, I, I, I, L, I, F, P, P, P, P, Z, P], I),
        "spec_distill_workspace_size": ([I, I], Z),
        "spec_distill_loss": ([P, I, I, I, L, P, P, P, I, F, P, P, P, Z, P], I),
        "spec_distill_grad": ([P, I, I, I, L, P, P, P, I, F, P, P, P, L, P], I),
        "spec_distill_loss_grad": ([P, I, I, I, L, P, P, P, I, F, P, P, P, L, P, Z, P], I),
        "spec_set_row_kernel_events": ([P, P], None),
        "spec_kernels_per_call": ([ctypes.c_char_p], I),
    }
    for name, (args, res) in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = res


def lib():
    """The loaded CUDA library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -c 'import __graft_entry__ as g; g.build()'`")
        l = ctypes.CDLL(LIB_PATH)
        _declare(l)
        _lib = l
    return _lib


def header_functions() -> list[str]:
    """Names of the functions declared in include/specverify.h."""
    with open(HEADER_PATH) as f:
        text = f.read()
    return sorted(set(re.findall(r"^\s*(?:const\s+)?[\w\s\*]*?\b(spec_\w+)\s*\(", text, re.M)))


def status_string(status: int) -> str:
    return lib().spec_status_string(int(status)).decode()


def _check(fn: str, status: int) -> None:
    if status != SPEC_OK:
        raise SpecError(fn, status)


def _dtype(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return SPEC_BF16
    if t.dtype == torch.float32:
        return SPEC_F32
    raise TypeError(f"logits must be bfloat16 or float32, got {t.dtype}")


def _dev(t: torch.Tensor, name: str, dtype=None) -> torch.Tensor:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _on(device):
    """Makes `device` current for the call when it is not already (launches go to the
    tensors' device); a no-op context otherwise, so the common case costs nothing."""
    import contextlib
    if device.index is None or device.index == torch.cuda.current_device():
        return contextlib.nullcontext()
    return torch.cuda.device(device)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream, device) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def spec_workspace_size(B: int, K_or_N: int, V: int) -> int:
    return int(lib().spec_workspace_size(int(B), int(K_or_N), int(V)))


def spec_verify_chain(target_logits, draft_logits, draft_tokens, uniforms, temp, top_k=0,
                      top_p=1.0, accepted_len=None, out_tokens=None, workspace=None,
                      stream=None):
    """Chain verification. target [B,K+1,V], draft [B,K,V] (None when temp == 0),
    draft_tokens int32 [B,K], uniforms float32 [B,K+1]. Returns (accepted_len [B],
    out_tokens [B,K+1]) as int32 CUDA tensors."""
    t = _dev(target_logits, "target_logits")
    B, K1, V = t.shape
    K = K1 - 1
    d = None if draft_logits is None else _dev(draft_logits, "draft_logits", t.dtype)
    if d is not None and tuple(d.shape) != (B, K, V):
        raise ValueError("draft_logits must be [B, K, V]")
    x = _dev(draft_tokens, "draft_tokens", torch.int32)
    u = _dev(uniforms, "uniforms", torch.float32)
    if tuple(x.shape) != (B, K) or tuple(u.shape) != (B, K + 1):
        raise ValueError("draft_tokens must be [B, K] and uniforms [B, K+1]")
    if accepted_len is None:
        accepted_len = torch.empty(B, dtype=torch.int32, device=t.device)
    if out_tokens is None:
        out_tokens = torch.empty((B, K + 1), dtype=torch.int32, device=t.device)
    if workspace is None:
        workspace = torch.empty(spec_workspace_size(B, K, V), dtype=torch.uint8, device=t.device)
    with _on(t.device):
        _check("spec_verify_chain", lib().spec_verify_chain(
            _ptr(t), _ptr(d), _dtype(t), B, K, V, _ptr(x), _ptr(u), float(temp), int(top_k),
            float(top_p), _ptr(accepted_len), _ptr(out_tokens), _ptr(workspace),
            workspace.numel() * workspace.element_size(), _stream(stream, t.device)))
    return accepted_len, out_tokens


def spec_verify_chain_noalloc(target_logits, draft_logits, draft_tokens, uniforms, temp,
                              top_k=0, top_p=1.0, accepted_len=None, out_tokens=None,
                              stream=None):
    """spec_verify_chain with the library's static scratch instead of a workspace (calls on
    one device must not overlap). Returns (accepted_len [B], out_tokens [B,K+1])."""
    t = _dev(target_logits, "target_logits")
    B, K1, V = t.shape
    K = K1 - 1
    d = None if draft_logits is None else _dev(draft_logits, "draft_logits", t.dtype)
    if d is not None and tuple(d.shape) != (B, K, V):
        raise ValueError("draft_logits must be [B, K, V]")
    x = _dev(draft_tokens, "draft_tokens", torch.int32)
    u = _dev(uniforms, "uniforms", torch.float32)
    if tuple(x.shape) != (B, K) or tuple(u.shape) != (B, K + 1):
        raise ValueError("draft_tokens must be [B, K] and uniforms [B, K+1]")
    if accepted_len is None:
        accepted_len = torch.empty(B, dtype=torch.int32, device=t.device)
    if out_tokens is None:
        out_tokens = torch.empty((B, K + 1), dtype=torch.int32, device=t.device)
    with _on(t.device):
        _check("spec_verify_chain_noalloc", lib().spec_verify_chain_noalloc(
            _ptr(t), _ptr(d), _dtype(t), B, K, V, _ptr(x), _ptr(u), float(temp), int(top_k),
            float(top_p), _ptr(accepted_len), _ptr(out_tokens), _stream(stream, t.device)))
    return accepted_len, out_tokens


def spec_verify_tree_typical(target_logits, node_tokens, parent_idx, eps, delta,
                             path_cap=None, best_path=None, accepted_len=None, workspace=None,
                             stream=None):
    """Typical acceptance over a candidate tree. target [B,N,V], node_tokens int32 [B,N],
    parent_idx int32 [N]. Returns (best_path [B,path_cap], accepted_len [B])."""
    t = _dev(target_logits, "target_logits")
    B, N, V = t.shape
    nt = _dev(node_tokens, "node_tokens", torch.int32)
    par = _dev(parent_idx, "parent_idx", torch.int32)
    if tuple(nt.shape) != (B, N) or tuple(par.shape) != (N,):
        raise ValueError("node_tokens must be [B, N] and parent_idx [N]")
    cap = N if path_cap is None else int(path_cap)
    if best_path is None:
        best_path = torch.empty((B, cap), dtype=torch.int32, device=t.device)
    if accepted_len is None:
        accepted_len = torch.empty(B, dtype=torch.int32, device=t.device)
    if workspace is None:
        workspace = torch.empty(spec_workspace_size(B, N, V), dtype=torch.uint8, device=t.device)
    with _on(t.device):
        _check("spec_verify_tree_typical", lib().spec_verify_tree_typical(
            _ptr(t), _dtype(t), B, N, V, _ptr(nt), _ptr(par), float(eps), float(delta),
            _ptr(best_path), cap, _ptr(accepted_len), _ptr(workspace),
            workspace.numel() * workspace.element_size(), _stream(stream, t.device)))
    return best_path, accepted_len


def spec_verify_tree_greedy(target_logits, node_tokens, parent_idx, path_cap=None,
                            best_path=None, accepted_len=None, next_token=None, workspace=None,
                            stream=None):
    """Greedy (multi-branch) verification over a candidate tree. target [B,N,V],
    node_tokens int32 [B,N], parent_idx int32 [N]. Returns (best_path [B,path_cap],
    accepted_len [B], next_token [B])."""
    t = _dev(target_logits, "target_logits")
    B, N, V = t.shape
    nt = _dev(node_tokens, "node_tokens", torch.int32)
    par = _dev(parent_idx, "parent_idx", torch.int32)
    if tuple(nt.shape) != (B, N) or tuple(par.shape) != (N,):
        raise ValueError("node_tokens must be [B, N] and parent_idx [N]")
    cap = N if path_cap is None else int(path_cap)
    if best_path is None:
        best_path = torch.empty((B, cap), dtype=torch.int32, device=t.device)
    if accepted_len is None:
        accepted_len = torch.empty(B, dtype=torch.int32, device=t.device)
    if next_token is None:
        next_token = torch.empty(B, dtype=torch.int32, device=t.device)
    if workspace is None:
        workspace = torch.empty(spec_workspace_size(B, N, V), dtype=torch.uint8, device=t.device)
    with _on(t.device):
        _check("spec_verify_tree_greedy", lib().spec_verify_tree_greedy(
            _ptr(t), _dtype(t), B, N, V, _ptr(nt), _ptr(par), _ptr(best_path), cap,
            _ptr(accepted_len), _ptr(next_token), _ptr(workspace),
            workspace.numel() * workspace.element_size(), _stream(stream, t.device)))
    return best_path, accepted_len, next_token


def spec_verify_tree_sampling(target_logits, draft_logits, node_tokens, parent_idx, uniforms,
                              temp, top_k=0, top_p=1.0, path_cap=None, best_path=None,
                              accepted_len=None, next_token=None, workspace=None, stream=None):
    """Rejection sampling over a candidate tree. target and draft [B,N,V] (draft None when
    temp == 0), node_tokens int32 [B,N], parent_idx int32 [N], uniforms float32 [B,N+1].
    Returns (best_path [B,path_cap], accepted_len [B], next_token [B])."""
    t = _dev(target_logits, "target_logits")
    B, N, V = t.shape
    d = None if draft_logits is None else _dev(draft_logits, "draft_logits", t.dtype)
    if d is not None and tuple(d.shape) != (B, N, V):
        raise ValueError("draft_logits must be [B, N, V]")
    nt = _dev(node_tokens, "node_tokens", torch.int32)
    par = _dev(parent_idx, "parent_idx", torch.int32)
    u = _dev(uniforms, "uniforms", torch.float32)
    if tuple(nt.shape) != (B, N) or tuple(par.shape) != (N,) or tuple(u.shape) != (B, N + 1):
        raise ValueError("node_tokens must be [B, N], parent_idx [N] and uniforms [B, N+1]")
    cap = N if path_cap is None else int(path_cap)
    if best_path is None:
        best_path = torch.empty((B, cap), dtype=torch.int32, device=t.device)
    if accepted_len is None:
        accepted_len = torch.empty(B, dtype=torch.int32, device=t.device)
    if next_token is None:
        next_token = torch.empty(B, dtype=torch.int32, device=t.device)
    if workspace is None:
        workspace = torch.empty(spec_workspace_size(B, N, V), dtype=torch.uint8, device=t.device)
    with _on(t.device):
        _check("spec_verify_tree_sampling", lib().spec_verify_tree_sampling(
            _ptr(t), _ptr(d), _dtype(t), B, N, V, _ptr(nt), _ptr(par), _ptr(u), float(temp),
            int(top_k), float(top_p), _ptr(best_path), cap, _ptr(accepted_len), _ptr(next_token),
            _ptr(workspace), workspace.numel() * workspace.element_size(),
            _stream(stream, t.device)))
    return best_path, accepted_len, next_token


def spec_logits_to_probs(logits, temp, top_k=0, top_p=1.0, with_entropy=True, probs=None,
                         entropy=None, stream=None):
    """Transformed distribution of each row of logits [..., V]. Returns (probs float32
    [..., V], entropy float32 [...] or None)."""
    lg = _dev(logits, "logits")
    V = lg.shape[-1]
    rows = lg.numel() // V
    if probs is None:
        probs = torch.empty(lg.shape, dtype=torch.float32, device=lg.device)
    if with_entropy and entropy is None:
        entropy = torch.empty(lg.shape[:-1], dtype=torch.float32, device=lg.device)
    with _on(lg.device):
        _check("spec_logits_to_probs", lib().spec_logits_to_probs(
            _ptr(lg), _dtype(lg), rows, V, float(temp), int(top_k), float(top_p), _ptr(probs),
            _ptr(entropy), _stream(stream, lg.device)))
    return probs, entropy


def spec_residual_sample(p, q, uniforms, tokens=None, stream=None):
    """Draw per row from norm(max(0, p - q)) (q None: from p). p, q float32 [rows, V],
    uniforms float32 [rows]. Returns int32 tokens [rows]."""
    pp = _dev(p, "p", torch.float32)
    rows, V = pp.shape
    qq = None if q is None else _dev(q, "q", torch.float32)
    if qq is not None and qq.shape != pp.shape:
        raise ValueError("q must match p")
    u = _dev(uniforms, "uniforms", torch.float32)
    if tokens is None:
        tokens = torch.empty(rows, dtype=torch.int32, device=pp.device)
    with _on(pp.device):
        _check("spec_residual_sample", lib().spec_residual_sample(
            _ptr(pp), _ptr(qq), rows, V, _ptr(u), _ptr(tokens), _stream(stream, pp.device)))
    return tokens


def spec_lmhead_workspace_size(B: int, K: int, V: int, d: int, top_k: int) -> int:
    return int(lib().spec_lmhead_workspace_size(int(B), int(K), int(V), int(d), int(top_k)))


def spec_verify_chain_lmhead(target_hidden, draft_hidden, target_weight, draft_weight,
                             draft_tokens, uniforms, temp, top_k=0, logits_out=None,
                             accepted_len=None, out_tokens=None, workspace=None, stream=None):
    """Chain verification from hidden states: target_hidden bf16 [B,K+1,d], draft_hidden
    [B,K,d] (None when temp == 0), target_weight and draft_weight bf16 [V,d] (the LM heads).
    temp == 0 (greedy) or 1 <= top_k <= 64. logits_out: None, or float32 [B*(2K+1), V] to
    receive the logits as well (target rows, then draft rows). Returns (accepted_len [B],
    out_tokens [B,K+1])."""
    ht = _dev(target_hidden, "target_hidden", torch.bfloat16)
    B, K1, d = ht.shape
    K = K1 - 1
    wt = _dev(target_weight, "target_weight", torch.bfloat16)
    V = wt.shape[0]
    greedy = float(temp) == 0.0
    hd = None if draft_hidden is None else _dev(draft_hidden, "draft_hidden", torch.bfloat16)
    wd = None if draft_weight is None else _dev(draft_weight, "draft_weight", torch.bfloat16)
    if tuple(wt.shape) != (V, d) or (hd is not None and tuple(hd.shape) != (B, K, d)) or \
            (wd is not None and tuple(wd.shape) != (V, d)):
        raise ValueError("hidden [B,K+1,d] / [B,K,d], weights [V,d]")
    x = _dev(draft_tokens, "draft_tokens", torch.int32)
    u = _dev(uniforms, "uniforms", torch.float32)
    if accepted_len is None:
        accepted_len = torch.empty(B, dtype=torch.int32, device=ht.device)
    if out_tokens is None:
        out_tokens = torch.empty((B, K + 1), dtype=torch.int32, device=ht.device)
    if logits_out is not None:
        _dev(logits_out, "logits_out", torch.float32)
    if workspace is None:
        workspace = torch.empty(spec_lmhead_workspace_size(B, K, V, d, 0 if greedy else top_k),
                                dtype=torch.uint8, device=ht.device)
    with _on(ht.device):
        _check("spec_verify_chain_lmhead", lib().spec_verify_chain_lmhead(
            _ptr(ht), _ptr(hd), _ptr(wt), _ptr(wd), B, K, V, d, _ptr(x), _ptr(u), float(temp),
            int(top_k), _ptr(accepted_len), _ptr(out_tokens), _ptr(logits_out),
            _ptr(workspace), workspace.numel() * workspace.element_size(),
            _stream(stream, ht.device)))
    return accepted_len, out_tokens


def spec_linear_state_factors(alpha, beta, keys, values, w=None, u=None, gamma=None,
                              stream=None):
    """Compact factors of every prefix of a round's S steps (gated delta rule). alpha, beta
    float32 [B,H,S]; keys [B,H,S,dk]; values [B,H,S,dv]. Returns (w [B,H,S,dk], u [B,H,S,dv],
    gamma [B,H,S])."""
    al = _dev(alpha, "alpha", torch.float32)
    be = _dev(beta, "beta", torch.float32)
    k = _dev(keys, "keys", torch.float32)
    v = _dev(values, "values", torch.float32)
    B, H, S = al.shape
    dk, dv = k.shape[3], v.shape[3]
    if tuple(be.shape) != (B, H, S) or tuple(k.shape[:3]) != (B, H, S) or \
            tuple(v.shape[:3]) != (B, H, S):
        raise ValueError("alpha, beta [B,H,S], keys [B,H,S,dk], values [B,H,S,dv]")
    if w is None:
        w = torch.empty((B, H, S, dk), dtype=torch.float32, device=k.device)
    if u is None:
        u = torch.empty((B, H, S, dv), dtype=torch.float32, device=k.device)
    if gamma is None:
        gamma = torch.empty((B, H, S), dtype=torch.float32, device=k.device)
    with _on(k.device):
        _check("spec_linear_state_factors", lib().spec_linear_state_factors(
            _ptr(al), _ptr(be), _ptr(k), _ptr(v), B, H, S, dk, dv, _ptr(w), _ptr(u),
            _ptr(gamma), _stream(stream, k.device)))
    return w, u, gamma


def spec_commit_linear_state(state, keys, w, u, gamma, steps, stream=None):
    """In place: state float32 [B,H,dk,dv] becomes the state after steps[b] steps of its
    round (keys, w [B,H,S,dk]; u [B,H,S,dv]; gamma [B,H,S]; steps int32 [B])."""
    st = _dev(state, "state", torch.float32)
    B, H, dk, dv = st.shape
    k = _dev(keys, "keys", torch.float32)
    S = k.shape[2]
    ww = _dev(w, "w", torch.float32)
    uu = _dev(u, "u", torch.float32)
    g = _dev(gamma, "gamma", torch.float32)
    n = _dev(steps, "steps", torch.int32)
    if tuple(k.shape) != (B, H, S, dk) or tuple(ww.shape) != (B, H, S, dk) or \
            tuple(uu.shape) != (B, H, S, dv) or tuple(g.shape) != (B, H, S) or \
            tuple(n.shape) != (B,):
        raise ValueError("keys, w [B,H,S,dk]; u [B,H,S,dv]; gamma [B,H,S]; steps [B]")
    with _on(st.device):
        _check("spec_commit_linear_state", lib().spec_commit_linear_state(
            _ptr(st), B, H, dk, dv, S, _ptr(k), _ptr(ww), _ptr(uu), _ptr(g), _ptr(n),
            _stream(stream, st.device)))
    return st


# ------------------------------------------------------------------ the drafter's side
# The calls take tensors' values and know nothing of autograd: a result has no graph, whether or not
# the logits require a gradient. A training step hands spec_distill_grad's (or _loss_grad's) result on
# by logits.backward(grad).
def _rows(t, name="logits"):
    """A [rows, V] CUDA tensor of bfloat16 or float32 whose rows are V adjacent entries, any
    distance (>= V) apart. Returns (tensor, dtype code, rows, V, row stride)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    code = _dtype(t)
    if t.dim() != 2:
        raise ValueError(f"{name} must be [rows, V]")
    rows, V = t.shape
    stride, step = t.stride()
    if rows <= 1:
        stride = max(stride, V)
    if (V > 1 and step != 1) or stride < V:
        raise ValueError(f"{name} must hold each row's entries next to one another, "
                         "rows apart (no transposed or expanded rows)")
    return t, code, rows, V, stride


def _like(t, name, dtype, shape, device):
    """An argument beside the logits: contiguous, of that type and shape, on their device."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.device == device
            and t.shape == shape and t.is_contiguous()):
        return t
    _dev(t, name, dtype)
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    return t


# The current stream's handle on a device, without building a Stream object for it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _here(stream, device) -> bool:
    """Whether a call may run as it is: on the current device, on its current stream."""
    return stream is None and device.index == torch.cuda.current_device()


def _there(call, stream, device, args):
    """call(*args) with the device current, and the stream (a Stream or a handle) current on it:
    what the call allocates then belongs to the stream it runs on, and is reused only after its
    work."""
    if isinstance(stream, torch.cuda.Stream) and stream.device != device:
        raise ValueError(f"stream must be one of {device}, got one of {stream.device}")
    with torch.cuda.device(device):
        if stream is None:
            return call(*args)
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(int(getattr(stream, "cuda_stream", stream)), device)
        with torch.cuda.stream(stream):
            return call(*args)


def _scratch(workspace, size, device):
    if workspace is None:
        return torch.empty(size, dtype=torch.uint8, device=device)
    _dev(workspace, "workspace")
    if workspace.device != device:
        raise ValueError(f"workspace must be on {device}, got {workspace.device}")
    return workspace


def _knob(v, name, dtype, rows, device):
    """A setting for every row (a number) or each row's own (a tensor): (scalar, pointer)."""
    if isinstance(v, torch.Tensor):
        return 0, _like(v, name, dtype, (rows,), device).data_ptr()
    return v, None


def _int32(v) -> int:
    """A count as the C ABI's int: one past its range stands for its end, not for its low bits."""
    return max(-1, min(int(v), 2**31 - 1))


def spec_sample_workspace_size(rows: int, V: int) -> int:
    return int(lib().spec_sample_workspace_size(int(rows), int(V)))


def spec_sample(logits, uniforms, temp=1.0, top_k=0, top_p=1.0, min_p=0.0, tokens=None,
                probs=None, workspace=None, stream=None):
    """Draw one token per row of logits [rows, V] (bfloat16 or float32, rows may be apart) with
    uniforms float32 [rows]. temp, top_k, top_p and min_p are numbers, or tensors [rows] on the
    logits' device (float32, top_k int32) with each row's own. Returns (tokens int32 [rows],
    probs float32 [rows]: the drawn tokens' probabilities). The verify calls test drafts against q
    under one temp, top_k and top_p a call and without min_p: draw what they are to test so."""
    t, code, rows, V, stride = _rows(logits)
    dev = t.device
    if not _here(stream, dev):
        return _there(spec_sample, stream, dev, (logits, uniforms, temp, top_k, top_p, min_p,
                                                 tokens, probs, workspace))
    _like(uniforms, "uniforms", torch.float32, (rows,), dev)
    temp, row_temp = _knob(temp, "temp", torch.float32, rows, dev)
    top_k, row_top_k = _knob(top_k, "top_k", torch.int32, rows, dev)
    top_p, row_top_p = _knob(top_p, "top_p", torch.float32, rows, dev)
    min_p, row_min_p = _knob(min_p, "min_p", torch.float32, rows, dev)
    if tokens is None:
        tokens = torch.empty(rows, dtype=torch.int32, device=dev)
    else:
        _like(tokens, "tokens", torch.int32, (rows,), dev)
    if probs is None:
        probs = torch.empty(rows, dtype=torch.float32, device=dev)
    else:
        _like(probs, "probs", torch.float32, (rows,), dev)
    l = lib()
    ws = _scratch(workspace, workspace is None and l.spec_sample_workspace_size(rows, V), dev)
    _check("spec_sample", l.spec_sample(
        t.data_ptr(), code, rows, V, stride, uniforms.data_ptr(), temp, _int32(top_k), top_p, min_p,
        row_temp, row_top_k, row_top_p, row_min_p, tokens.data_ptr(), probs.data_ptr(),
        ws.data_ptr(), ws.nbytes, _raw_stream(dev.index)))
    return tokens, probs


def spec_top_logits_workspace_size(rows: int, V: int, k: int) -> int:
    return int(lib().spec_top_logits_workspace_size(int(rows), int(V), int(k)))


def spec_top_logits(logits, k, temp=1.0, ids=None, values=None, lse=None, workspace=None,
                    stream=None):
    """The k largest logits of each row of logits [rows, V], largest first, ties by the lower id.
    Returns (ids int32 [rows, k], values float32 [rows, k], lse float32 [rows]: the log-sum-exp
    of logits / temp over the row)."""
    t, code, rows, V, stride = _rows(logits)
    dev, k = t.device, _int32(k)
    if not _here(stream, dev):
        return _there(spec_top_logits, stream, dev, (logits, k, temp, ids, values, lse, workspace))
    kept = max(0, min(k, SPEC_MAX_TOP_LOGITS))   # (the call refuses any other k)
    if ids is None:
        ids = torch.empty((rows, kept), dtype=torch.int32, device=dev)
    else:
        _like(ids, "ids", torch.int32, (rows, k), dev)
    if values is None:
        values = torch.empty((rows, kept), dtype=torch.float32, device=dev)
    else:
        _like(values, "values", torch.float32, (rows, k), dev)
    if lse is None:
        lse = torch.empty(rows, dtype=torch.float32, device=dev)
    else:
        _like(lse, "lse", torch.float32, (rows,), dev)
    l = lib()
    ws = _scratch(workspace, workspace is None and l.spec_top_logits_workspace_size(rows, V, k), dev)
    _check("spec_top_logits", l.spec_top_logits(
        t.data_ptr(), code, rows, V, stride, k, temp, ids.data_ptr(), values.data_ptr(),
        lse.data_ptr(), ws.data_ptr(), ws.nbytes, _raw_stream(dev.index)))
    return ids, values, lse


def _teacher(rows, dev, teacher_ids, teacher_logits, teacher_lse):
    """The teacher's lists: (k, ids, logits and lse as pointers)."""
    if not isinstance(teacher_ids, torch.Tensor) or teacher_ids.dim() != 2:
        raise ValueError("teacher_ids must be [rows, k]")
    k = teacher_ids.shape[1]
    _like(teacher_ids, "teacher_ids", torch.int32, (rows, k), dev)
    _like(teacher_logits, "teacher_logits", torch.float32, (rows, k), dev)
    if teacher_lse is not None:
        teacher_lse = _like(teacher_lse, "teacher_lse", torch.float32, (rows,), dev).data_ptr()
    return k, teacher_ids.data_ptr(), teacher_logits.data_ptr(), teacher_lse


def _grad_rows(grad, t):
    """The gradient's rows and their distance: the logits' type, shape and device."""
    if grad is None:
        return torch.empty(t.shape, dtype=t.dtype, device=t.device), t.shape[1]
    g, _, _, _, stride = _rows(grad, "grad")
    if g.dtype != t.dtype or g.shape != t.shape or g.device != t.device:
        raise ValueError("grad must match logits in type, shape and device")
    if not g.is_inference():
        # written behind autograd's back: a graph that kept these values (the logits', in place) is
        # to notice
        torch.autograd.graph.increment_version(g)
    return g, stride


def spec_distill_workspace_size(rows: int, V: int) -> int:
    return int(lib().spec_distill_workspace_size(int(rows), int(V)))


def spec_distill_loss(logits, teacher_ids, teacher_logits, teacher_lse=None, temp=1.0, loss=None,
                      stats=None, workspace=None, stream=None):
    """Distillation loss of each row of the student's logits [rows, V] against a teacher's top
    logits: teacher_ids int32 and teacher_logits float32 [rows, k], teacher_lse float32 [rows] or
    None (then the list is the teacher's whole distribution). Returns (loss float32 [rows], stats
    float32 [rows, 4] for spec_distill_grad), without a graph."""
    t, code, rows, V, stride = _rows(logits)
    dev = t.device
    if not _here(stream, dev):
        return _there(spec_distill_loss, stream, dev, (logits, teacher_ids, teacher_logits,
                                                       teacher_lse, temp, loss, stats, workspace))
    k, ids, values, lse = _teacher(rows, dev, teacher_ids, teacher_logits, teacher_lse)
    if loss is None:
        loss = torch.empty(rows, dtype=torch.float32, device=dev)
    else:
        _like(loss, "loss", torch.float32, (rows,), dev)
    if stats is None:
        stats = torch.empty((rows, 4), dtype=torch.float32, device=dev)
    else:
        _like(stats, "stats", torch.float32, (rows, 4), dev)
    l = lib()
    ws = _scratch(workspace, workspace is None and l.spec_distill_workspace_size(rows, V), dev)
    _check("spec_distill_loss", l.spec_distill_loss(
        t.data_ptr(), code, rows, V, stride, ids, values, lse, k, temp, loss.data_ptr(),
        stats.data_ptr(), ws.data_ptr(), ws.nbytes, _raw_stream(dev.index)))
    return loss, stats


def spec_distill_grad(logits, teacher_ids, teacher_logits, teacher_lse, temp, stats,
                      grad_loss=None, grad=None, stream=None):
    """Gradient of spec_distill_loss with respect to the logits, from the stats it returned;
    grad_loss float32 [rows] or None (1): the gradient with respect to each row's loss. grad may
    be the logits themselves. Returns grad [rows, V] in the logits' type, for logits.backward(grad)."""
    t, code, rows, V, stride = _rows(logits)
    dev = t.device
    if not _here(stream, dev):
        return _there(spec_distill_grad, stream, dev, (logits, teacher_ids, teacher_logits,
                                                       teacher_lse, temp, stats, grad_loss, grad))
    k, ids, values, lse = _teacher(rows, dev, teacher_ids, teacher_logits, teacher_lse)
    _like(stats, "stats", torch.float32, (rows, 4), dev)
    g = grad_loss
    if g is not None:
        g = _like(g, "grad_loss", torch.float32, (rows,), dev).data_ptr()
    grad, grad_stride = _grad_rows(grad, t)
    _check("spec_distill_grad", lib().spec_distill_grad(
        t.data_ptr(), code, rows, V, stride, ids, values, lse, k, temp, stats.data_ptr(), g,
        grad.data_ptr(), grad_stride, _raw_stream(dev.index)))
    return grad


def spec_distill_loss_grad(logits, teacher_ids, teacher_logits, teacher_lse=None, temp=1.0,
                           grad_loss=None, loss=None, grad=None, workspace=None, stream=None):
    """spec_distill_loss and spec_distill_grad in one call, for a training step that knows
    grad_loss beforehand (the row's weight in the mean). grad may be the logits themselves. Returns
    (loss [rows], grad [rows, V]), without a graph: logits.backward(grad) takes the step on."""
    t, code, rows, V, stride = _rows(logits)
    dev = t.device
    if not _here(stream, dev):
        return _there(spec_distill_loss_grad, stream, dev,
                      (logits, teacher_ids, teacher_logits, teacher_lse, temp, grad_loss, loss,
                       grad, workspace))
    k, ids, values, lse = _teacher(rows, dev, teacher_ids, teacher_logits, teacher_lse)
    g = grad_loss
    if g is not None:
        g = _like(g, "grad_loss", torch.float32, (rows,), dev).data_ptr()
    if loss is None:
        loss = torch.empty(rows, dtype=torch.float32, device=dev)
    else:
        _like(loss, "loss", torch.float32, (rows,), dev)
    grad, grad_stride = _grad_rows(grad, t)
    l = lib()
    ws = _scratch(workspace, workspace is None and l.spec_distill_workspace_size(rows, V), dev)
    _check("spec_distill_loss_grad", l.spec_distill_loss_grad(
        t.data_ptr(), code, rows, V, stride, ids, values, lse, k, temp, g, loss.data_ptr(),
        grad.data_ptr(), grad_stride, ws.data_ptr(), ws.nbytes, _raw_stream(dev.index)))
    return loss, grad


def spec_get_device_status(workspace, stream=None) -> int:
    out = ctypes.c_int32(0)
    with _on(workspace.device):
        _check("spec_get_device_status", lib().spec_get_device_status(
            _ptr(workspace), ctypes.byref(out), _stream(stream, workspace.device)))
    return int(out.value)


def spec_set_row_kernel_events(before=None, after=None) -> None:
    """Record torch.cuda.Event `before`/`after` around every verify call's row kernel."""
    lib().spec_set_row_kernel_events(
        None if before is None else ctypes.c_void_p(before.cuda_event),
        None if after is None else ctypes.c_void_p(after.cuda_event))


def spec_kernels_per_call(entry_point: str) -> int:
    return int(lib().spec_kernels_per_call(entry_point.encode()))
