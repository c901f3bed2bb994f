"""ctypes binding of libdllm.so: argument marshalling only.

Every function takes torch CUDA tensors (PyTorch supplies device memory and
streams), checks dtype / contiguity / device, and passes raw pointers and
sizes to the C ABI declared in ``include/dllm.h``. All arithmetic of the
denoise step runs in the library's kernels; there is no fallback path: a
missing library raises at import time.
"""

from __future__ import annotations

import array
import ctypes
import math
import os
import struct

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdllm.so")

c_int, c_float, c_size_t, c_void_p = ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.c_void_p


class DllmError(RuntimeError):
    def __init__(self, code, what):
        msg = f"{what}: {status_string(code)} (status {code})"
        if code == 4:
            name = LIB.dllm_last_cuda_error()
            if name:
                msg += f": {name.decode()}"
        super().__init__(msg)
        self.code = code


class Params(ctypes.Structure):
    _fields_ = [("tau", c_float), ("lambda_", c_float), ("kappa", c_float),
                ("hierarchical", c_int), ("hier_levels", c_int), ("smoothing", c_int),
                ("alpha", c_float), ("mask_id", c_int)]


class StepArgs(ctypes.Structure):
    _fields_ = [("q", c_void_p), ("k", c_void_p), ("v", c_void_p),
                ("attn_out", c_void_p), ("attn_out_fp32", c_int),
                ("q_off", c_void_p), ("kv_off", c_void_p),
                ("H", c_int), ("dh", c_int), ("max_q", c_int), ("max_kv", c_int),
                ("q_rows", c_int), ("kv_rows", c_int),
                ("scale", c_float),
                ("hidden", c_void_p), ("w_head", c_void_p), ("emb", c_void_p),
                ("R", c_int), ("d", c_int), ("V", c_int),
                ("argmax", c_void_p), ("conf", c_void_p), ("pe", c_void_p),
                ("row_req", c_void_p), ("row_pos", c_void_p),
                ("B", c_int), ("blk", c_int),
                ("mask", c_void_p), ("tokens", c_void_p), ("credit", c_void_p),
                ("prev_argmax", c_void_p), ("next_emb", c_void_p), ("n_commit", c_void_p),
                ("params", Params)]


# name -> (restype, argtypes); mirrors include/dllm.h
SIGNATURES = {
    "dllm_block_attn_workspace": (c_size_t, [c_int] * 5),
    "dllm_block_attn": (c_int, [c_void_p] * 4 + [c_int, c_void_p, c_void_p] + [c_int] * 7
                        + [c_float, c_void_p, c_size_t, c_void_p]),
    "dllm_head_workspace": (c_size_t, [c_int] * 4),
    "dllm_head_confidence": (c_int, [c_void_p] * 3 + [c_int] * 3 + [c_void_p] * 4
                             + [c_size_t, c_void_p]),
    "dllm_head_confidence_noalloc": (c_int, [c_void_p] * 3 + [c_int] * 3 + [c_void_p] * 4),
    "dllm_commit": (c_int, [c_void_p] * 5 + [c_int] * 3 + [c_void_p] * 5 + [c_int, c_int]
                    + [c_void_p, c_void_p, ctypes.POINTER(Params), c_void_p]),
    "dllm_denoise_step_workspace": (c_size_t, [ctypes.POINTER(StepArgs)]),
    "dllm_workspace_bytes": (c_size_t, [c_int] * 9),
    "dllm_denoise_step": (c_int, [ctypes.POINTER(StepArgs), c_void_p, c_size_t, c_void_p]),
    "dllm_status_string": (ctypes.c_char_p, [c_int]),
    "dllm_get_device_status": (c_int, [ctypes.POINTER(ctypes.c_int32), c_int]),
    "dllm_last_cuda_error": (ctypes.c_char_p, []),
    "dllm_version": (c_int, []),
    "dllm_launch_count": (ctypes.c_uint64, []),
}


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with block_decoding_gb300.build.build() "
            "(nvcc, sm_103a). There is no fallback implementation.")
    lib = ctypes.CDLL(LIB_PATH)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


LIB = _load()


def launch_count() -> int:
    """Kernels this library has enqueued since it was loaded."""
    return int(LIB.dllm_launch_count())


def status_string(code: int) -> str:
    return LIB.dllm_status_string(int(code)).decode()


def _ck(code, what):
    if code != 0:
        raise DllmError(code, what)


def device_status(clear: bool = True) -> int:
    out = ctypes.c_int32(0)
    LIB.dllm_get_device_status(ctypes.byref(out), 1 if clear else 0)
    return int(out.value)


# ---------------------------------------------------------------------------
# helpers
# ---------------------------------------------------------------------------

def _ptr(t, dtype=None, name="tensor"):
    if t is None:
        return None
    if not (isinstance(t, torch.Tensor) and t.is_cuda):
        raise TypeError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def params_struct(p: dict) -> Params:
    return Params(float(p["tau"]), float(p["lam"]), float(p["kappa"]),
                  int(p["hierarchical"]), int(p["hier_levels"]), int(p["smoothing"]),
                  float(p["alpha"]), int(p["mask_id"]))


def workspace(nbytes: int, device=None) -> torch.Tensor:
    """A caller-owned workspace buffer (torch allocations are 256-byte aligned)."""
    return torch.empty(max(int(nbytes), 1), dtype=torch.uint8, device=device or "cuda")


def _scratch(nbytes, device, stream):
    """Workspace bytes of a call on `stream` (None: the current stream). The
    memory is that stream's own: a block that the current stream's calls have
    given back, but that their kernels still use, is not handed out, and this
    one goes to no other stream's call when it is given back."""
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _alloc(shape, dtype, device, stream):
    """torch.empty, as _scratch, for what the caller gets back: kept, once the
    caller gives it up, until what the current stream then does with it is done."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(t.device))
    return t


# ---------------------------------------------------------------------------
# entry points
# ---------------------------------------------------------------------------

def block_attn_workspace(B, H, dh, max_q, max_kv) -> int:
    return int(LIB.dllm_block_attn_workspace(B, H, dh, max_q, max_kv))


def block_attn(q, k, v, q_off, kv_off, max_q, max_kv, scale=None, out=None,
               out_fp32=False, ws=None, stream=None):
    """Non-causal block attention; q [sum W][H][dh], k/v [sum L][H][dh] bf16."""
    H, dh = q.shape[1], q.shape[2]
    B = q_off.numel() - 1
    if scale is None:
        scale = 1.0 / math.sqrt(dh)
    if out is None:
        out = _alloc(q.shape, torch.float32 if out_fp32 else torch.bfloat16, q.device, stream)
    need = block_attn_workspace(B, H, dh, max_q, max_kv)
    if ws is None and need:
        ws = _scratch(need, q.device, stream)
    rc = LIB.dllm_block_attn(_ptr(q, torch.bfloat16, "q"), _ptr(k, torch.bfloat16, "k"),
                             _ptr(v, torch.bfloat16, "v"), _ptr(out, None, "out"),
                             1 if out.dtype == torch.float32 else 0,
                             _ptr(q_off, torch.int32, "q_off"), _ptr(kv_off, torch.int32, "kv_off"),
                             B, H, dh, int(max_q), int(max_kv), q.shape[0], k.shape[0], float(scale),
                             _ptr(ws, None, "ws") if ws is not None else None,
                             ws.numel() if ws is not None else 0, _stream(stream))
    _ck(rc, "dllm_block_attn")
    return out


def head_workspace(R, d, V, with_pe) -> int:
    return int(LIB.dllm_head_workspace(R, d, V, 1 if with_pe else 0))


def head_confidence(hidden, w_head, emb=None, with_pe=True, argmax=None, conf=None,
                    pe=None, ws=None, stream=None):
    """LM head + softmax stats (+ P.E); returns (argmax int32, conf f32, pe f32 or None)."""
    R, d = hidden.shape
    V = w_head.shape[0]
    dev = hidden.device
    with_pe = with_pe and emb is not None
    argmax = argmax if argmax is not None else _alloc(R, torch.int32, dev, stream)
    conf = conf if conf is not None else _alloc(R, torch.float32, dev, stream)
    if with_pe and pe is None:
        pe = _alloc((R, d), torch.float32, dev, stream)
    if not with_pe:
        pe = None
    need = head_workspace(R, d, V, with_pe)
    if ws is None:
        ws = _scratch(max(need, 1), dev, stream)
    rc = LIB.dllm_head_confidence(_ptr(hidden, torch.bfloat16, "hidden"),
                                  _ptr(w_head, torch.bfloat16, "w_head"),
                                  _ptr(emb, torch.bfloat16, "emb") if emb is not None else None,
                                  R, d, V, _ptr(argmax, torch.int32, "argmax"),
                                  _ptr(conf, torch.float32, "conf"),
                                  _ptr(pe, torch.float32, "pe") if pe is not None else None,
                                  _ptr(ws, None, "ws"), ws.numel(), _stream(stream))
    _ck(rc, "dllm_head_confidence")
    return argmax, conf, pe


def commit(argmax, conf, pe, row_req, row_pos, mask, tokens, credit, prev, emb,
           params: dict, next_emb=None, n_commit=None, stream=None):
    """Parallel-decode commit; updates mask/tokens/credit/prev in place."""
    B, blk = mask.shape
    V, d = emb.shape
    R = row_req.numel()
    dev = mask.device
    next_emb = next_emb if next_emb is not None else _alloc((B, blk, d), torch.bfloat16, dev, stream)
    n_commit = n_commit if n_commit is not None else _alloc(B, torch.int32, dev, stream)
    prm = params_struct(params)
    rc = LIB.dllm_commit(_ptr(argmax, torch.int32, "argmax"), _ptr(conf, torch.float32, "conf"),
                         _ptr(pe, torch.float32, "pe") if pe is not None else None,
                         _ptr(row_req, torch.int32, "row_req"), _ptr(row_pos, torch.int32, "row_pos"),
                         R, B, blk, _ptr(mask, torch.uint8, "mask"), _ptr(tokens, torch.int32, "tokens"),
                         _ptr(credit, torch.float32, "credit"), _ptr(prev, torch.int32, "prev"),
                         _ptr(emb, torch.bfloat16, "emb"), V, d,
                         _ptr(next_emb, torch.bfloat16, "next_emb"), _ptr(n_commit, torch.int32, "n_commit"),
                         ctypes.byref(prm), _stream(stream))
    _ck(rc, "dllm_commit")
    return next_emb, n_commit


def step_args(*, q=None, k=None, v=None, attn_out=None, q_off=None, kv_off=None,
              max_q=0, max_kv=0, scale=None, hidden, w_head, emb, argmax, conf, pe,
              row_req, row_pos, mask, tokens, credit, prev, next_emb, n_commit,
              params: dict) -> StepArgs:
    a = StepArgs()
    if attn_out is not None:
        a.q, a.k, a.v = _ptr(q, torch.bfloat16, "q"), _ptr(k, torch.bfloat16, "k"), _ptr(v, torch.bfloat16, "v")
        a.attn_out = _ptr(attn_out, None, "attn_out")
        a.attn_out_fp32 = 1 if attn_out.dtype == torch.float32 else 0
        a.q_off, a.kv_off = _ptr(q_off, torch.int32, "q_off"), _ptr(kv_off, torch.int32, "kv_off")
        a.H, a.dh = q.shape[1], q.shape[2]
        a.max_q, a.max_kv = int(max_q), int(max_kv)
        a.q_rows, a.kv_rows = q.shape[0], k.shape[0]
        a.scale = float(scale if scale is not None else 1.0 / math.sqrt(a.dh))
    a.hidden = _ptr(hidden, torch.bfloat16, "hidden")
    a.w_head = _ptr(w_head, torch.bfloat16, "w_head")
    a.emb = _ptr(emb, torch.bfloat16, "emb")
    a.R, a.d = hidden.shape
    a.V = w_head.shape[0]
    a.argmax, a.conf = _ptr(argmax, torch.int32, "argmax"), _ptr(conf, torch.float32, "conf")
    a.pe = _ptr(pe, torch.float32, "pe") if pe is not None else None
    a.row_req, a.row_pos = _ptr(row_req, torch.int32, "row_req"), _ptr(row_pos, torch.int32, "row_pos")
    a.B, a.blk = mask.shape
    a.mask = _ptr(mask, torch.uint8, "mask")
    a.tokens = _ptr(tokens, torch.int32, "tokens")
    a.credit = _ptr(credit, torch.float32, "credit")
    a.prev_argmax = _ptr(prev, torch.int32, "prev")
    a.next_emb = _ptr(next_emb, torch.bfloat16, "next_emb")
    a.n_commit = _ptr(n_commit, torch.int32, "n_commit")
    a.params = params_struct(params)
    return a


def denoise_step_workspace(args: StepArgs) -> int:
    return int(LIB.dllm_denoise_step_workspace(ctypes.byref(args)))


def denoise_step(args: StepArgs, ws, stream=None):
    rc = LIB.dllm_denoise_step(ctypes.byref(args), _ptr(ws, None, "ws"), ws.numel(), _stream(stream))
    _ck(rc, "dllm_denoise_step")


# ---------------------------------------------------------------------------
# end-to-end model (dllm_gemm_bf16, dllm_model_forward, dllm_decode_step)
# ---------------------------------------------------------------------------

class ModelDesc(ctypes.Structure):
    _fields_ = [("layers", c_int), ("d", c_int), ("H", c_int), ("dh", c_int), ("ffn", c_int), ("V", c_int),
                ("max_seq", c_int), ("rms_eps", c_float), ("rope_base", c_float),
                ("emb", c_void_p), ("w_head", c_void_p),
                ("wqkv", ctypes.POINTER(c_void_p)), ("wo", ctypes.POINTER(c_void_p)),
                ("wgu", ctypes.POINTER(c_void_p)), ("wdown", ctypes.POINTER(c_void_p))]


class DecodeState(ctypes.Structure):
    _fields_ = [("T", c_int), ("prompt_len", c_int), ("blk", c_int), ("vic", c_int),
                ("tokens", c_void_p), ("masked", c_void_p),
                ("k_cache", ctypes.POINTER(c_void_p)), ("v_cache", ctypes.POINTER(c_void_p)),
                ("bmask", c_void_p), ("btokens", c_void_p), ("bprev", c_void_p), ("bcredit", c_void_p),
                ("bnext_emb", c_void_p), ("n_commit", c_void_p), ("argmax", c_void_p), ("conf", c_void_p),
                ("pe", c_void_p), ("hidden", c_void_p), ("params", Params), ("eos_id", c_int),
                ("dual_cache", c_int)]


SIGNATURES.update({
    "dllm_gemm_bf16": (c_int, [c_void_p] * 3 + [c_int] * 4 + [c_void_p, c_void_p]),
    "dllm_model_forward_workspace": (c_size_t, [ctypes.POINTER(ModelDesc), c_int]),
    "dllm_model_forward": (c_int, [ctypes.POINTER(ModelDesc), c_void_p, c_int, c_int,
                                   ctypes.POINTER(c_void_p), ctypes.POINTER(c_void_p), c_void_p, c_void_p,
                                   c_size_t, c_void_p]),
    "dllm_decode_step_workspace": (c_size_t, [ctypes.POINTER(ModelDesc), ctypes.POINTER(DecodeState)]),
    "dllm_decode_step": (c_int, [ctypes.POINTER(ModelDesc), ctypes.POINTER(DecodeState), c_int, c_int,
                                 c_void_p, c_size_t, c_void_p]),
    "dllm_decode_graph_create": (c_int, [ctypes.POINTER(ModelDesc), ctypes.POINTER(DecodeState), c_void_p,
                                         c_size_t, ctypes.POINTER(c_void_p)]),
    "dllm_decode_graph_launch": (c_int, [c_void_p, c_void_p]),
    "dllm_decode_graph_destroy": (c_int, [c_void_p]),
})
for _name in ("dllm_gemm_bf16", "dllm_model_forward_workspace", "dllm_model_forward",
              "dllm_decode_step_workspace", "dllm_decode_step", "dllm_decode_graph_create",
              "dllm_decode_graph_launch", "dllm_decode_graph_destroy"):
    _fn = getattr(LIB, _name)
    _fn.restype, _fn.argtypes = SIGNATURES[_name]


def gemm_bf16(A, W, epilogue=0, aux=None, out=None, stream=None):
    """C = A W^T (+aux) or SwiGLU; A [M][K], W [N][K] (or [2N][K] for SwiGLU)."""
    M, K = A.shape
    N = W.shape[0] // 2 if epilogue == 2 else W.shape[0]
    out = out if out is not None else _alloc((M, N), torch.bfloat16, A.device, stream)
    rc = LIB.dllm_gemm_bf16(_ptr(A, torch.bfloat16, "A"), _ptr(W, torch.bfloat16, "W"),
                            _ptr(out, torch.bfloat16, "C"), M, N, K, int(epilogue),
                            _ptr(aux, torch.bfloat16, "aux") if aux is not None else None, _stream(stream))
    _ck(rc, "dllm_gemm_bf16")
    return out


def _ptr_array(tensors):
    arr = (c_void_p * len(tensors))(*[_ptr(t, torch.bfloat16, "weight") for t in tensors])
    return arr


def model_desc(weights: dict, max_seq: int):
    """ModelDesc over device weights: emb, w_head and per-layer lists wqkv/wo/wgu/wdown.

    Returns (desc, keepalive) -- keep the second value alive while desc is used.
    """
    L = len(weights["wqkv"])
    arrs = [_ptr_array(weights[k]) for k in ("wqkv", "wo", "wgu", "wdown")]
    d = weights["emb"].shape[1]
    desc = ModelDesc(L, d, weights["H"], d // weights["H"], weights["wgu"][0].shape[0] // 2,
                     weights["emb"].shape[0], int(max_seq), float(weights["rms_eps"]),
                     float(weights["rope_base"]), _ptr(weights["emb"], torch.bfloat16, "emb"),
                     _ptr(weights["w_head"], torch.bfloat16, "w_head"),
                     ctypes.cast(arrs[0], ctypes.POINTER(c_void_p)), ctypes.cast(arrs[1], ctypes.POINTER(c_void_p)),
                     ctypes.cast(arrs[2], ctypes.POINTER(c_void_p)), ctypes.cast(arrs[3], ctypes.POINTER(c_void_p)))
    return desc, arrs


def model_forward(desc, x_in, pos0, k_cache, v_cache, ws=None, stream=None):
    n = x_in.shape[0]
    need = int(LIB.dllm_model_forward_workspace(ctypes.byref(desc), n))
    ws = ws if ws is not None else _scratch(max(need, 1), x_in.device, stream)
    out = _alloc(x_in.shape, x_in.dtype, x_in.device, stream)
    kc, vc = _ptr_array(k_cache), _ptr_array(v_cache)
    rc = LIB.dllm_model_forward(ctypes.byref(desc), _ptr(x_in, torch.bfloat16, "x_in"), n, int(pos0),
                                ctypes.cast(kc, ctypes.POINTER(c_void_p)), ctypes.cast(vc, ctypes.POINTER(c_void_p)),
                                _ptr(out, torch.bfloat16, "hidden_out"), _ptr(ws, None, "ws"), ws.numel(),
                                _stream(stream))
    _ck(rc, "dllm_model_forward")
    return out


def decode_step_workspace(desc, state) -> int:
    return int(LIB.dllm_decode_step_workspace(ctypes.byref(desc), ctypes.byref(state)))


def decode_step(desc, state, block, refresh, ws, stream=None):
    rc = LIB.dllm_decode_step(ctypes.byref(desc), ctypes.byref(state), int(block), 1 if refresh else 0,
                              _ptr(ws, None, "ws"), ws.numel(), _stream(stream))
    _ck(rc, "dllm_decode_step")


class DecodeGraph:
    """One CUDA graph that runs the whole block decode loop on the device."""

    def __init__(self, desc, state, ws):
        h = c_void_p()
        rc = LIB.dllm_decode_graph_create(ctypes.byref(desc), ctypes.byref(state), _ptr(ws, None, "ws"),
                                          ws.numel(), ctypes.byref(h))
        _ck(rc, "dllm_decode_graph_create")
        self.handle = h

    def launch(self, stream=None):
        _ck(LIB.dllm_decode_graph_launch(self.handle, _stream(stream)), "dllm_decode_graph_launch")

    def close(self):
        if self.handle:
            LIB.dllm_decode_graph_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ---------------------------------------------------------------------------
# step-level scheduler (include/dllm_sched.h): host-only
# ---------------------------------------------------------------------------
class SchedConfig(ctypes.Structure):
    _fields_ = [("slots", c_int), ("blk", c_int), ("vic", c_int), ("quantum", c_int), ("budget_cap", c_int),
                ("max_step_rows", c_int), ("max_seq", c_int), ("policy", c_int), ("dual_cache", c_int)]


class SchedEntry(ctypes.Structure):
    _fields_ = [("slot", c_int), ("req", c_int), ("block", c_int), ("kind", c_int), ("q_pos0", c_int),
                ("q_rows", c_int), ("kv_rows", c_int), ("b0", c_int)]


_I32P = ctypes.POINTER(ctypes.c_int32)
SIGNATURES.update({
    "dllm_sched_create": (c_int, [ctypes.POINTER(SchedConfig), ctypes.POINTER(c_void_p)]),
    "dllm_sched_destroy": (None, [c_void_p]),
    "dllm_sched_submit": (c_int, [c_void_p, c_int, c_int, c_int]),
    "dllm_sched_plan": (c_int, [c_void_p, ctypes.POINTER(SchedEntry), c_int]),
    "dllm_sched_complete": (c_int, [c_void_p, _I32P, ctypes.POINTER(ctypes.c_uint8)]),
    "dllm_sched_budget": (ctypes.c_longlong, [c_void_p]),
    "dllm_sched_queued": (c_int, [c_void_p]),
    "dllm_sched_finished": (c_int, [c_void_p, _I32P, c_int]),
    "dllm_sched_pack": (c_int, [ctypes.POINTER(SchedEntry), c_int, c_int, c_int, _I32P, _I32P, _I32P, _I32P]),
})
for _name in ("dllm_sched_create", "dllm_sched_destroy", "dllm_sched_submit", "dllm_sched_plan",
              "dllm_sched_complete", "dllm_sched_budget", "dllm_sched_queued", "dllm_sched_finished",
              "dllm_sched_pack"):
    _fn = getattr(LIB, _name)
    _fn.restype, _fn.argtypes = SIGNATURES[_name]


# ---------------------------------------------------------------------------
# mixture-of-experts FFN (dllm_moe_ffn)
# ---------------------------------------------------------------------------
SIGNATURES.update({
    "dllm_moe_ffn_workspace": (c_size_t, [c_int] * 5),
    "dllm_moe_ffn": (c_int, [c_void_p] * 4 + [c_int] * 5 + [c_void_p, c_int, c_void_p, c_void_p, c_void_p,
                                                           c_size_t, c_void_p]),
})
for _name in ("dllm_moe_ffn_workspace", "dllm_moe_ffn"):
    _fn = getattr(LIB, _name)
    _fn.restype, _fn.argtypes = SIGNATURES[_name]


def moe_ffn(h, w_router, w13, w2, topk, out_fp32=True, out=None, ids=None, weights=None, ws=None, stream=None):
    """out [n][d] = top-k MoE SwiGLU FFN of h; returns (out, ids, weights).
    w13 [E][2F][d] (gate rows, then up rows per expert), w2 [E][d][F]."""
    n, d = h.shape
    E, F2, d2 = w13.shape
    F = F2 // 2
    if d2 != d or tuple(w2.shape) != (E, d, F) or tuple(w_router.shape) != (E, d):
        raise ValueError("moe_ffn: inconsistent shapes")
    dev = h.device
    if out is None:
        out = _alloc((n, d), torch.float32 if out_fp32 else torch.bfloat16, dev, stream)
    if ids is None:
        ids = _alloc((n, topk), torch.int32, dev, stream)
    if weights is None:
        weights = _alloc((n, topk), torch.float32, dev, stream)
    need = int(LIB.dllm_moe_ffn_workspace(n, d, E, F, topk))
    if need == 0 and n > 0:
        raise DllmError(2, "dllm_moe_ffn_workspace")
    if ws is None or ws.numel() < need:
        ws = _scratch(max(need, 256), dev, stream)
    rc = LIB.dllm_moe_ffn(_ptr(h, torch.bfloat16, "h"), _ptr(w_router, torch.bfloat16, "w_router"),
                          _ptr(w13, torch.bfloat16, "w13"), _ptr(w2, torch.bfloat16, "w2"), n, d, E, F, topk,
                          _ptr(out, None, "out"), 1 if out.dtype == torch.float32 else 0,
                          _ptr(ids, torch.int32, "ids"), _ptr(weights, torch.float32, "weights"),
                          _ptr(ws, None, "ws"), ws.numel(), _stream(stream))
    _ck(rc, "dllm_moe_ffn")
    return out, ids, weights


# ---------------------------------------------------------------------------
# paged K/V cache (dllm_kv_write, dllm_kv_read, dllm_paged_attn)
# ---------------------------------------------------------------------------
class KvPagesDesc(ctypes.Structure):
    _fields_ = [("k", c_void_p), ("v", c_void_p), ("k_scale", c_void_p), ("v_scale", c_void_p), ("type", c_int),
                ("num_pages", c_int), ("page_size", c_int), ("heads", c_int), ("dh", c_int)]


class PagedAttnArgs(ctypes.Structure):
    _fields_ = [("q", c_void_p), ("q_stride", ctypes.c_longlong), ("out", c_void_p), ("out_fp32", c_int),
                ("lse", c_void_p), ("q_off", c_void_p), ("kv_len", c_void_p), ("q_pos", c_void_p),
                ("page_table", c_void_p), ("max_pages", c_int), ("B", c_int), ("Hq", c_int), ("max_q", c_int),
                ("max_kv", c_int), ("q_rows", c_int), ("scale", c_float), ("left", c_int), ("right", c_int),
                ("sinks", c_int)]


_PAGES_P = ctypes.POINTER(KvPagesDesc)
SIGNATURES.update({
    "dllm_kv_write": (c_int, [_PAGES_P, c_void_p, c_void_p, ctypes.c_longlong, ctypes.c_longlong, c_int, c_void_p,
                              c_void_p, c_void_p, c_int, c_int, c_void_p]),
    "dllm_kv_read": (c_int, [_PAGES_P, c_void_p, c_void_p, c_int, c_void_p, c_void_p, c_void_p, c_int, c_int, c_void_p]),
    "dllm_paged_attn_workspace": (c_size_t, [_PAGES_P, ctypes.POINTER(PagedAttnArgs)]),
    "dllm_paged_attn": (c_int, [_PAGES_P, ctypes.POINTER(PagedAttnArgs), c_void_p, c_size_t, c_void_p]),
})
for _name in ("dllm_kv_write", "dllm_kv_read", "dllm_paged_attn_workspace", "dllm_paged_attn"):
    _fn = getattr(LIB, _name)
    _fn.restype, _fn.argtypes = SIGNATURES[_name]


_NEED = {}      # workspace bytes by shape, of pages by type and shape


class KVPages:
    """Page pools of a K/V cache: k, v [num_pages][heads][page_size][dh], bf16
    or float8_e4m3fn; the 8-bit rows with uint8 k_scale, v_scale
    [num_pages][heads][page_size] (a row stands for code * 2^(byte - 127))."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        if k.dim() != 4 or v.shape != k.shape:
            raise ValueError("k and v must be [num_pages][heads][page_size][dh]")
        if k.dtype not in (torch.bfloat16, torch.float8_e4m3fn):
            raise TypeError(f"pages must be bfloat16 or float8_e4m3fn, got {k.dtype}")
        fp8 = k.dtype == torch.float8_e4m3fn
        if fp8 != (k_scale is not None) or fp8 != (v_scale is not None):
            raise ValueError("e4m3 pages need k_scale and v_scale, bf16 pages have none")
        if fp8 and not (k_scale.shape == k.shape[:3] and v_scale.shape == k.shape[:3]):
            raise ValueError("scales must be [num_pages][heads][page_size]")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.index = dev = k.get_device()
        self.num_pages, self.heads, self.page_size, self.dh = k.shape
        self.desc = KvPagesDesc(
            _ptr_on(k, dev, k.dtype, "k"), _ptr_on(v, dev, k.dtype, "v"),
            _ptr_on(k_scale, dev, torch.uint8, "k_scale") if fp8 else None,
            _ptr_on(v_scale, dev, torch.uint8, "v_scale") if fp8 else None,
            1 if fp8 else 0, self.num_pages, self.page_size, self.heads, self.dh)
        self.device = k.device
        if len(_NEED) >= 256:
            _NEED.clear()
        self._need = _NEED.setdefault((fp8, *k.shape), {})

    @classmethod
    def empty(cls, num_pages, page_size, heads, dh, dtype=torch.bfloat16, device="cuda"):
        """Pools of uninitialised pages."""
        shape = (int(num_pages), int(heads), int(page_size), int(dh))
        k, v = (torch.empty(shape, dtype=dtype, device=device) for _ in range(2))
        if dtype != torch.float8_e4m3fn:
            return cls(k, v)
        return cls(k, v, *(torch.empty(shape[:3], dtype=torch.uint8, device=device) for _ in range(2)))


def _ptr_on(t, index, dtype, name):
    """Pointer of a contiguous `dtype` tensor on GPU `index`."""
    # one test on the way that every call goes; _ptr says what is wrong
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == index >= 0 and t.is_contiguous()):
        _ptr(t, dtype, name)
        raise ValueError(f"{name} is on {t.device}, the pages are on GPU {index}")
    return t.data_ptr()


def _rows_ptr(t, index, heads, dh, name):
    """(pointer, row stride) of bf16 rows [rows][heads][dh], dense within a row."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda):
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, the pages are on cuda:{index}")
    shape = t.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != dh:
        raise ValueError(f"{name} must be [rows][{heads}][{dh}], got {tuple(shape)}")
    n, s = shape[0], t.stride()
    if n and (s[2] != 1 or (heads > 1 and s[1] != dh)):
        raise ValueError(f"{name} must be dense within a row")
    return t.data_ptr(), s[0] if n > 1 else heads * dh


def _batch(index, off, page_table, per_request, name):
    """(B, max_pages, pointers of off, page_table and per_request) of a ragged batch."""
    po, pt = _ptr_on(off, index, torch.int32, "offsets"), _ptr_on(page_table, index, torch.int32, "page_table")
    pr = _ptr_on(per_request, index, torch.int32, name)
    B = off.numel() - 1
    shape = page_table.shape
    if B < 0 or len(shape) != 2 or shape[0] != B:
        raise ValueError("page_table must be [B][max_pages] with B = offsets - 1")
    if per_request.numel() != B:
        raise ValueError(f"{name} must have one entry per request")
    return B, shape[1], po, pt, pr


def _launch(what, index, stream, *args):
    """Call `what` with GPU `index` current, on `stream` or that GPU's current stream."""
    fn = getattr(LIB, what)
    if torch._C._cuda_getDevice() == index:
        rc = fn(*args, stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(index):
            rc = fn(*args, stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(index))
    _ck(rc, what)


def kv_write(pages: KVPages, k, v, off, pos0, page_table, stream=None):
    """Store rows k, v [rows][heads][dh] bf16 (any row stride) in the pages:
    row off[i] + t at position pos0[i] + t of request i. off int32 [B+1], pos0
    int32 [B], page_table int32 [B][max_pages]."""
    dev = pages.index
    kp, ks = _rows_ptr(k, dev, pages.heads, pages.dh, "k")
    vp, vs = _rows_ptr(v, dev, pages.heads, pages.dh, "v")
    rows = k.shape[0]
    if rows != v.shape[0]:
        raise ValueError("k and v must have the same rows")
    B, n, po, pt, pp = _batch(dev, off, page_table, pos0, "pos0")
    _launch("dllm_kv_write", dev, stream, pages.desc, kp, vp, ks, vs, rows, po, pp, pt, n, B)


def _rows_out(t, shape, pages, name, stream):
    """The bf16 rows `t`, allocated unless given, and their pointer."""
    if t is None:
        t = _alloc(shape, torch.bfloat16, pages.device, stream)
        return t, t.data_ptr()
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}")
    return t, _ptr_on(t, pages.index, torch.bfloat16, name)


def kv_read(pages: KVPages, off, pos0, page_table, rows, k=None, v=None, stream=None):
    """The cached rows of positions pos0[i] + t as bf16 rows off[i] + t of (k, v)
    [rows][heads][dh] (allocated unless given; with `stream`, order other
    streams' use of them after it)."""
    dev = pages.index
    shape = (int(rows), pages.heads, pages.dh)
    B, n, po, pt, pp = _batch(dev, off, page_table, pos0, "pos0")
    k, kp = _rows_out(k, shape, pages, "k", stream)
    v, vp = _rows_out(v, shape, pages, "v", stream)
    _launch("dllm_kv_read", dev, stream, pages.desc, kp, vp, shape[0], po, pp, pt, n, B)
    return k, v


def paged_attn_workspace(pages: KVPages, B, Hq, max_q, max_kv) -> int:
    """Workspace bytes of paged_attn for no larger B, max_q and max_kv."""
    key = (int(B), int(Hq), int(max_q), int(max_kv))
    need = pages._need.get(key)
    if need is None:
        if max(key) >= 1 << 31 or min(key) < 0:
            raise ValueError("B, Hq, max_q and max_kv must be 0 to 2^31 - 1")
        a = PagedAttnArgs(B=key[0], Hq=key[1], max_q=key[2], max_kv=key[3])
        need = int(LIB.dllm_paged_attn_workspace(ctypes.byref(pages.desc), ctypes.byref(a)))
        if len(pages._need) < 4096:
            pages._need[key] = need
    return need


_I31 = 1 << 31


def paged_attn(q, pages: KVPages, q_off, kv_len, page_table, max_q, max_kv, q_pos=None, scale=None, left=-1, right=-1,
               sinks=0, out=None, out_fp32=False, return_lse=False, lse=None, ws=None, stream=None):
    """Attention of q [rows][Hq][dh] bf16 (any row stride) over the pages.

    Row t of request i has position q_pos[i] + t (default: the last rows of
    the cache) and sees keys u < kv_len[i] with u <= position + right and
    (u >= position - left or u < sinks); negative left / right: no limit.
    Returns out [rows][Hq][dh], or (out, lse [rows][Hq]) with return_lse; with
    `stream`, order other streams' use of them after it.
    """
    return _attend("dllm_paged_attn", (), q, pages, q_off, kv_len, page_table, max_q, max_kv, q_pos, scale, left, right, sinks,
                   out, out_fp32, return_lse, lse, ws, stream)


def _attend(what, more, q, pages, q_off, kv_len, page_table, max_q, max_kv, q_pos, scale, left, right, sinks, out, out_fp32,
            return_lse, lse, ws, stream):
    """Entry point `what` with the arguments of paged_attn and `more` behind the struct."""
    # (ctypes would cut longer numbers off)
    if not (0 <= max_q < _I31 and 0 <= max_kv < _I31 and 0 <= sinks < _I31 and -_I31 <= left < _I31 and -_I31 <= right < _I31):
        raise ValueError("max_q, max_kv, left, right and sinks must fit 32 bits, and only left and right may be negative")
    dev, dh = pages.index, pages.dh
    rows, Hq = (q.shape[0], q.shape[1]) if isinstance(q, torch.Tensor) and q.dim() == 3 else (0, 0)
    qp, qs = _rows_ptr(q, dev, Hq, dh, "q")
    B, n, po, pt, pn = _batch(dev, q_off, page_table, kv_len, "kv_len")
    pp = None
    if q_pos is not None:
        pp = _ptr_on(q_pos, dev, torch.int32, "q_pos")
        if q_pos.numel() != B:
            raise ValueError("q_pos must have one entry per request")
    if out is None:
        out = _alloc((rows, Hq, dh), torch.float32 if out_fp32 else torch.bfloat16, pages.device, stream)
        op = out.data_ptr()
    elif out.shape != (rows, Hq, dh) or out.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"out must be bf16 or fp32 [{rows}][{Hq}][{dh}]")
    else:
        op = _ptr_on(out, dev, out.dtype, "out")
        out_fp32 = out.dtype is torch.float32
    lp = None
    if lse is not None:
        if lse.shape != (rows, Hq):
            raise ValueError(f"lse must be [{rows}][{Hq}]")
        lp = _ptr_on(lse, dev, torch.float32, "lse")
    elif return_lse:
        lse = _alloc((rows, Hq), torch.float32, pages.device, stream)
        lp = lse.data_ptr()
    a = PagedAttnArgs(qp, qs, op, 1 if out_fp32 else 0, lp, po, pn, pp, pt, n, B, Hq, int(max_q), int(max_kv), rows,
                      1.0 / math.sqrt(dh) if scale is None else float(scale), int(left), int(right), int(sinks))
    wp, need = None, 0
    if ws is not None:
        wp, need = _ptr_on(ws, dev, ws.dtype, "ws"), ws.numel() * ws.element_size()
    else:
        need = paged_attn_workspace(pages, B, Hq, max_q, max_kv)
        if need:
            ws = _scratch(need, pages.device, stream)
            wp = ws.data_ptr()
    _launch(what, dev, stream, pages.desc, a, *more, wp, need)
    return (out, lse) if return_lse else out


# ---------------------------------------------------------------------------
# around the paged cache: rotary positions, draft trees, eviction
# (dllm_rope_kv_write, dllm_tree_mask, dllm_tree_attn, dllm_attn_mass,
# dllm_kv_move, dllm_kv_evict)
# ---------------------------------------------------------------------------
class RopeDesc(ctypes.Structure):
    _fields_ = [("rot", c_int), ("axes", c_int), ("axis", ctypes.c_uint8 * 64), ("freq", ctypes.c_double * 64)]


_ROPE_HEAD = struct.Struct("=ii64s")


class RopeWriteArgs(ctypes.Structure):
    _fields_ = [(n, c_void_p) for n in ("pos", "q", "k", "v", "q_out")] + \
               [(n, ctypes.c_longlong) for n in ("q_stride", "k_stride", "v_stride", "q_out_stride")] + \
               [(n, c_void_p) for n in ("off", "pos0", "page_table")] + \
               [(n, c_int) for n in ("max_pages", "B", "Hq", "rows")]


class AttnMassArgs(ctypes.Structure):
    _fields_ = [("q", c_void_p), ("q_stride", ctypes.c_longlong)] + \
               [(n, c_void_p) for n in ("lse", "mass", "q_off", "kv_len", "q_pos", "fresh", "page_table")] + \
               [(n, c_int) for n in ("max_pages", "B", "Hq", "max_q", "max_kv", "q_rows")] + \
               [("scale", c_float), ("right", c_int), ("decay", c_float)]


class KvMoveArgs(ctypes.Structure):
    _fields_ = [(n, c_void_p) for n in ("src", "count", "first", "page_table", "dst_table")] + \
               [(n, c_int) for n in ("src_heads", "max_n", "max_pages", "dst_pages", "B")] + [("mass", c_void_p)]


class KvEvictArgs(ctypes.Structure):
    _fields_ = [(n, c_void_p) for n in ("mass", "kv_len", "page_table", "dst_table")] + \
               [(n, c_int) for n in ("max_pages", "dst_pages", "B", "budget", "max_kv", "sinks", "recent", "move_mass")] + \
               [("new_len", c_void_p), ("keep", c_void_p)]


_CACHE_CALLS = {
    "dllm_rope_kv_write": (c_int, [_PAGES_P, ctypes.POINTER(RopeDesc), ctypes.POINTER(RopeWriteArgs), c_void_p]),
    "dllm_tree_mask": (c_int, [c_void_p, c_void_p, c_int, c_int, c_int, c_void_p, c_int, c_void_p, c_void_p]),
    "dllm_tree_attn": (c_int, [_PAGES_P, ctypes.POINTER(PagedAttnArgs), c_void_p, c_int, c_void_p, c_size_t, c_void_p]),
    "dllm_attn_mass": (c_int, [_PAGES_P, ctypes.POINTER(AttnMassArgs), c_void_p]),
    "dllm_kv_move": (c_int, [_PAGES_P, ctypes.POINTER(KvMoveArgs), c_void_p]),
    "dllm_kv_evict": (c_int, [_PAGES_P, ctypes.POINTER(KvEvictArgs), c_void_p]),
}
SIGNATURES.update(_CACHE_CALLS)
for _name, (_res, _args) in _CACHE_CALLS.items():
    _fn = getattr(LIB, _name)
    _fn.restype, _fn.argtypes = _res, _args


class Rope:
    """Rotary frequencies of heads of `dh` elements: pair j (elements j and
    j + len(freq)) turns by position[axis[j]] * freq[j] radians; what is left of
    the head stays as it is."""

    def __init__(self, dh, axis, freq):
        n = len(freq)
        if len(axis) != n:
            raise ValueError("axis and freq must have one entry per pair")
        if n % 8 or 2 * n > dh or dh > 128:
            raise ValueError("pairs must be a multiple of 8, at most dh / 2")
        # (refuses what is negative or above 255; not an array's memory, whatever its type)
        axis = bytes(axis if isinstance(axis, (list, tuple, bytes)) else [int(a) for a in axis])
        # axes that pairs turn by, and those of the positions (standard: one per section)
        self.dh, self.used = int(dh), max(axis, default=0) + 1
        self.axes = self.used
        if self.axes > 4:
            raise ValueError("axes are numbered 0 to 3")
        # (packed at once: a tenth of the time of ctypes arrays, entry by entry)
        self.desc = RopeDesc.from_buffer_copy(_ROPE_HEAD.pack(2 * n, self.used, axis) + array.array("d", freq).tobytes() +
                                              bytes(8 * (64 - n)))

    @classmethod
    def standard(cls, dh, base=10000.0, rot=None, sections=None, interleaved=False):
        """freq[j] = base^(-2j / rot), rot = dh unless given. `sections`: the pairs
        of every axis (they add up to rot / 2; one may have none), one run after the other or, with
        `interleaved`, in turn (0, 1, 2, 0, 1, 2, ..) as long as an axis has pairs."""
        rot = dh if rot is None else rot
        if rot % 16:
            raise ValueError("rot must be a multiple of 16")
        sections = [rot // 2] if sections is None else list(sections)
        if sum(sections) != rot // 2 or min(sections) < 0:
            raise ValueError("sections must add up to rot / 2 pairs")
        if interleaved:
            left, axis = list(sections), []
            while len(axis) < rot // 2:
                for a, n in enumerate(left):
                    if n > 0:
                        axis.append(a)
                        left[a] -= 1
        else:
            axis = [a for a, n in enumerate(sections) for _ in range(n)]
        rope = cls(dh, axis, [float(base) ** (-2.0 * j / rot) for j in range(rot // 2)])
        rope.axes = max(rope.axes, len(sections))
        return rope


def rope_kv_write(pages: KVPages, rope: Rope, pos, q, k, v, off, pos0, page_table, q_out=None, stream=None):
    """Turn q [rows][Hq][dh] and k [rows][heads][dh] (bf16, any row stride) by
    their positions pos int32 [axes][rows] ([rows] with one axis; last axes that no
    pair turns by may be left out), store k and v in the pages as kv_write does, and
    return the turned q (q_out, which may be q itself; allocated unless given; with
    `stream`, order other streams' use of it after it). q None: no q, returns None."""
    dev, dh = pages.index, pages.dh
    if rope.dh != dh:
        raise ValueError(f"rope is for heads of {rope.dh}, the pages have heads of {dh}")
    kp, ks = _rows_ptr(k, dev, pages.heads, dh, "k")
    vp, vs = _rows_ptr(v, dev, pages.heads, dh, "v")
    rows = k.shape[0]
    if rows != v.shape[0]:
        raise ValueError("k and v must have the same rows")
    pp = _ptr_on(pos, dev, torch.int32, "pos")
    if not (pos.dim() == 2 and rope.used <= pos.shape[0] <= rope.axes and pos.shape[1] == rows) and \
            not (rope.used == 1 and pos.shape == (rows,)):
        raise ValueError(f"pos must be [{rope.axes}][{rows}]")
    B, n, po, pt, p0 = _batch(dev, off, page_table, pos0, "pos0")
    Hq = qp = qs = op = os_ = 0
    if q is not None:
        Hq = q.shape[1] if isinstance(q, torch.Tensor) and q.dim() == 3 else 0
        qp, qs = _rows_ptr(q, dev, Hq, dh, "q")
        if q.shape[0] != rows:
            raise ValueError("q and k must have the same rows")
        if q_out is None:
            q_out = _alloc((rows, Hq, dh), torch.bfloat16, pages.device, stream)
            op, os_ = q_out.data_ptr(), Hq * dh
        else:
            op, os_ = _rows_ptr(q_out, dev, Hq, dh, "q_out")
            if q_out.shape[0] != rows:
                raise ValueError("q_out and q must have the same rows")
    elif q_out is not None:
        raise ValueError("q_out without q")
    a = RopeWriteArgs(pp, qp, kp, vp, op, qs, ks, vs, os_, po, p0, pt, n, B, Hq, rows)
    _launch("dllm_rope_kv_write", dev, stream, pages.desc, rope.desc, a)
    return q_out


def tree_mask(parent, off, max_q, mask=None, depth=None, stream=None):
    """(mask int32 [rows][ceil(max_q / 32)], depth int32 [rows]) of the trees of
    drafted tokens parent int32 [rows] (row off[i] + t: the parent's number, less
    than t, or -1): which of its request's tokens each token descends from, itself
    included, as bits, and how many they are without itself. Rows in no request
    are left as they are. With `stream`, order other streams' use of them after it."""
    if not 0 <= max_q < _I31:       # (ctypes would cut longer numbers off)
        raise ValueError("max_q must be 0 to 2^31 - 1")
    dev = parent.get_device() if isinstance(parent, torch.Tensor) else -1
    pp, po = _ptr_on(parent, dev, torch.int32, "parent"), _ptr_on(off, dev, torch.int32, "offsets")
    rows, B, words = parent.numel(), off.numel() - 1, (int(max_q) + 31) // 32
    if B < 0:
        raise ValueError("offsets must have an entry")
    if mask is None:
        mask = _alloc((rows, words), torch.int32, parent.device, stream)
        mp = mask.data_ptr()
    elif mask.dim() != 2 or mask.shape[0] != rows or mask.shape[1] < words:
        raise ValueError(f"mask must be [{rows}][{words} or more]")
    else:
        mp, words = _ptr_on(mask, dev, torch.int32, "mask"), mask.shape[1]
    if depth is None:
        depth = _alloc((rows,), torch.int32, parent.device, stream)
        dp = depth.data_ptr()
    elif depth.shape != (rows,):
        raise ValueError(f"depth must be [{rows}]")
    else:
        dp = _ptr_on(depth, dev, torch.int32, "depth")
    _launch("dllm_tree_mask", dev, stream, pp, po, rows, int(max_q), B, mp, words, dp)
    return mask, depth


def tree_attn(q, pages: KVPages, q_off, kv_len, page_table, mask, max_q, max_kv, scale=None, out=None, out_fp32=False,
              return_lse=False, lse=None, ws=None, stream=None):
    """paged_attn of drafted tokens: the rows of request i are its last cached
    positions, and each sees all positions before them, itself, and the tokens
    whose bits are set in its row of mask int32 [rows][ceil(max_q / 32) or more]
    (tree_mask). Workspace: paged_attn_workspace of the same sizes."""
    dev = pages.index
    mp = _ptr_on(mask, dev, torch.int32, "mask")
    rows = q.shape[0] if isinstance(q, torch.Tensor) and q.dim() == 3 else 0
    if mask.dim() != 2 or mask.shape[0] != rows or 32 * mask.shape[1] < max_q:
        raise ValueError(f"mask must be [{rows}][{-(-max_q // 32)} or more]")
    return _attend("dllm_tree_attn", (mp, mask.shape[1]), q, pages, q_off, kv_len, page_table, max_q, max_kv, None, scale, -1,
                   -1, 0, out, out_fp32, return_lse, lse, ws, stream)


def _mass_ptr(mass, pages):
    """Pointer of the weights beside the pages, or None."""
    if mass is None:
        return None
    if mass.shape != pages.k.shape[:3]:
        raise ValueError("mass must be [num_pages][heads][page_size]")
    return _ptr_on(mass, pages.index, torch.float32, "mass")


def _per_request(t, B, dev, name):
    if t is None:
        return None
    if t.numel() != B:
        raise ValueError(f"{name} must have one entry per request")
    return _ptr_on(t, dev, torch.int32, name)


def attn_mass(q, lse, pages: KVPages, mass, q_off, kv_len, page_table, max_q, max_kv, q_pos=None, fresh=None, scale=None,
              right=-1, decay=1.0, stream=None):
    """Add to mass float32 [num_pages][heads][page_size] (times `decay`; times 0
    from position fresh[i] int32 [B] on) the weight that the query rows q
    [rows][Hq][dh], with lse [rows][Hq] from paged_attn, gave to every cached row
    of their requests. The rows see keys up to `right` behind their position
    (negative: all), and paged_attn has to have had the same `right` and no `left`:
    with the lse of a window or of tree_attn the keys left out there are weighed
    too. Returns mass."""
    if not (0 <= max_q < _I31 and 0 <= max_kv < _I31 and -_I31 <= right < _I31):
        raise ValueError("max_q, max_kv and right must fit 32 bits, and only right may be negative")
    dev, dh = pages.index, pages.dh
    rows, Hq = (q.shape[0], q.shape[1]) if isinstance(q, torch.Tensor) and q.dim() == 3 else (0, 0)
    qp, qs = _rows_ptr(q, dev, Hq, dh, "q")
    lp = _ptr_on(lse, dev, torch.float32, "lse")
    if lse.shape != (rows, Hq):
        raise ValueError(f"lse must be [{rows}][{Hq}]")
    B, n, po, pt, pn = _batch(dev, q_off, page_table, kv_len, "kv_len")
    a = AttnMassArgs(qp, qs, lp, _mass_ptr(mass, pages), po, pn, _per_request(q_pos, B, dev, "q_pos"),
                     _per_request(fresh, B, dev, "fresh"), pt, n, B, Hq, int(max_q), int(max_kv), rows,
                     1.0 / math.sqrt(dh) if scale is None else float(scale), int(right), float(decay))
    _launch("dllm_attn_mass", dev, stream, pages.desc, a)
    return mass


def _tables(page_table, dst_table, dev, B):
    """(pointer and pages of page_table, of dst_table): None stands for in place."""
    if page_table.dim() != 2 or page_table.shape[0] != B:
        raise ValueError("page_table must be [B][max_pages]")
    pt, n = _ptr_on(page_table, dev, torch.int32, "page_table"), page_table.shape[1]
    if dst_table is None or dst_table is page_table:
        return pt, n, None, 0
    if dst_table.dim() != 2 or dst_table.shape[0] != B:
        raise ValueError("dst_table must be [B][pages]")
    if B and not dst_table.shape[1]:        # (a null pointer, which stands for in place)
        raise ValueError("dst_table has no pages")
    return pt, n, _ptr_on(dst_table, dev, torch.int32, "dst_table"), dst_table.shape[1]


def kv_move(pages: KVPages, src, count, first, page_table, dst_table=None, mass=None, stream=None):
    """Move the cached rows at positions src int32 [B][heads or 1][n] (the first
    count[i] of them) to positions first[i] + 0, 1, .. (first None: from 0) of
    dst_table's pages, which page_table does not name, or in place: then each list
    ascends and no row moves to a later position. mass float32
    [num_pages][heads][page_size] moves with the rows."""
    dev, B = pages.index, count.numel()
    if src.dim() != 3 or src.shape[0] != B or src.shape[1] not in (1, pages.heads):
        raise ValueError(f"src must be [{B}][{pages.heads} or 1][n]")
    sp, cp, fp = _ptr_on(src, dev, torch.int32, "src"), _per_request(count, B, dev, "count"), _per_request(first, B, dev, "first")
    pt, n, dt, dn = _tables(page_table, dst_table, dev, B)
    a = KvMoveArgs(sp, cp, fp, pt, dt, src.shape[1], src.shape[2], n, dn, B, _mass_ptr(mass, pages))
    _launch("dllm_kv_move", dev, stream, pages.desc, a)


def kv_evict(pages: KVPages, mass, kv_len, page_table, budget, max_kv, sinks=0, recent=0, dst_table=None, move_mass=True,
             new_len=None, keep=None, stream=None):
    """Cut every request down to `budget` rows a cached head: the first `sinks`,
    the last `recent` and those of greatest mass float32
    [num_pages][heads][page_size] stay, in their order, at positions 0, 1, .. of
    dst_table's pages (default: in place, see kv_move). Returns (new_len int32 [B],
    which may be kv_len, keep int32 [B][heads][budget], the positions that stayed, then -1); with
    `stream`, order other streams' use of them after it."""
    if not (0 <= budget < _I31 and 0 <= max_kv < _I31 and 0 <= sinks < _I31 and 0 <= recent < _I31):
        raise ValueError("budget, max_kv, sinks and recent must be 0 to 2^31 - 1")
    dev, B = pages.index, kv_len.numel()
    kp = _ptr_on(kv_len, dev, torch.int32, "kv_len")
    pt, n, dt, dn = _tables(page_table, dst_table, dev, B)
    if new_len is None:
        new_len = _alloc((B,), torch.int32, pages.device, stream)
        np_ = new_len.data_ptr()
    else:
        np_ = _per_request(new_len, B, dev, "new_len")
    if keep is None:
        keep = _alloc((B, pages.heads, int(budget)), torch.int32, pages.device, stream)
        ep = keep.data_ptr()
    elif keep.shape != (B, pages.heads, budget):
        raise ValueError(f"keep must be [{B}][{pages.heads}][{budget}]")
    else:
        ep = _ptr_on(keep, dev, torch.int32, "keep")
    a = KvEvictArgs(_mass_ptr(mass, pages), kp, pt, dt, n, dn, B, int(budget), int(max_kv), int(sinks), int(recent),
                    1 if move_mass else 0, np_, ep)
    _launch("dllm_kv_evict", dev, stream, pages.desc, a)
    return new_len, keep
