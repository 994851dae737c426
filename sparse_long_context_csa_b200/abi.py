"""ctypes binding of libdsv4 (include/dsv4.h): argument marshalling only.

Every function here has the name of the C entry point it calls, takes torch tensors
(or None for optional NULL pointers) that already live on the GPU, passes their
device pointers, and raises ``Dsv4Error`` when the library returns a non-zero status.
No arithmetic of the method happens in Python.  The library must have been built
(``python -m sparse_long_context_csa_b200.build``); loading fails loudly otherwise.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdsv4.so")

F32, BF16 = 0, 1
STATUS = {0: "DSV4_OK", 1: "DSV4_ERR_ARG", 2: "DSV4_ERR_SHAPE", 3: "DSV4_ERR_ALIGN", 4: "DSV4_ERR_DTYPE",
          5: "DSV4_ERR_CUDA", 6: "DSV4_ERR_DEVICE_CHECK", 7: "DSV4_ERR_WORKSPACE"}

EXPORTED = ("dsv4_compress_kv", "dsv4_indexer_topk", "dsv4_sparse_mqa_attn", "dsv4_csa_layer",
            "dsv4_hca_layer", "dsv4_workspace_bytes", "dsv4_status_string", "dsv4_version",
            "dsv4_launch_count", "dsv4_indexer_topk_noalloc", "dsv4_device_check", "dsv4_indexer_scores",
            "dsv4_topk_select", "dsv4_decode_append", "dsv4_grouped_out_proj", "dsv4_set_index_checks",
            "dsv4_index_checks", "dsv4_sparse_mqa_attn_scores", "dsv4_add_rms_norm", "dsv4_route_experts",
            "dsv4_expert_mlp", "dsv4_expert_mlp_workspace_bytes")


class Dsv4Error(RuntimeError):
    def __init__(self, fn: str, status: int, msg: str):
        super().__init__(f"{fn}: {STATUS.get(status, status)} ({msg})")
        self.status = status


class Dsv4Params(ctypes.Structure):
    """Mirror of ``dsv4_params`` (field order and types must match include/dsv4.h)."""
    _fields_ = [(n, ctypes.c_int32) for n in
                ("B", "S", "Sq", "H", "D", "R", "dv", "n_win", "win_ring", "m", "overlap", "P_cap",
                 "nI", "cI", "topk")] + \
               [("scale", ctypes.c_float), ("rope_theta", ctypes.c_float)] + \
               [(n, ctypes.c_int32) for n in ("rope_q", "rotate_out", "dtype")]

    def __repr__(self):
        return "Dsv4Params(" + ", ".join(f"{n}={getattr(self, n)}" for n, _ in self._fields_) + ")"


SCORE_SOFTMAX, SCORE_SIGMOID, SCORE_SQRT_SOFTPLUS = 0, 1, 2


class Dsv4MoeParams(ctypes.Structure):
    """Mirror of ``dsv4_moe_params`` (field order and types must match include/dsv4.h)."""
    _fields_ = [(n, ctypes.c_int32) for n in
                ("T", "hidden", "inter", "E", "topk", "n_group", "topk_group", "score_fn", "renorm", "scale_pow2",
                 "dtype", "logits_dtype")] + \
               [(n, ctypes.c_float) for n in ("eps", "routed_scale", "swiglu_limit")]

    def __repr__(self):
        return "Dsv4MoeParams(" + ", ".join(f"{n}={getattr(self, n)}" for n, _ in self._fields_) + ")"


_lib = None


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libdsv4.so (once) and declare the C signatures."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with `python -m sparse_long_context_csa_b200.build`")
    lib = ctypes.CDLL(path)
    P = ctypes.POINTER(Dsv4Params)
    vp, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    lib.dsv4_compress_kv.argtypes = [P, i32, vp, vp, vp, vp, i32, vp, vp, vp]
    lib.dsv4_indexer_topk.argtypes = [P, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.dsv4_indexer_topk_noalloc.argtypes = [P, vp, vp, vp, vp, vp, vp]
    lib.dsv4_indexer_scores.argtypes = [P, vp, vp, vp, vp, vp, vp]
    lib.dsv4_topk_select.argtypes = [P, vp, vp, vp, vp]
    lib.dsv4_decode_append.argtypes = [P, i32, vp, vp, vp, vp, vp, vp, vp, vp, i32, vp, vp, vp]
    lib.dsv4_sparse_mqa_attn.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.dsv4_sparse_mqa_attn_scores.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.dsv4_csa_layer.argtypes = [P] + [vp] * 17 + [sz, vp]
    lib.dsv4_hca_layer.argtypes = [P] + [vp] * 10 + [sz, vp]
    lib.dsv4_grouped_out_proj.argtypes = [P, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp]
    M = ctypes.POINTER(Dsv4MoeParams)
    lib.dsv4_add_rms_norm.argtypes = [M] + [vp] * 8
    lib.dsv4_route_experts.argtypes = [M] + [vp] * 5
    lib.dsv4_expert_mlp.argtypes = [M] + [vp] * 8 + [sz, vp]
    lib.dsv4_expert_mlp_workspace_bytes.argtypes = [M]
    lib.dsv4_expert_mlp_workspace_bytes.restype = sz
    lib.dsv4_set_index_checks.argtypes = [i32]
    lib.dsv4_set_index_checks.restype = None
    lib.dsv4_index_checks.restype = i32
    lib.dsv4_workspace_bytes.argtypes = [P]
    lib.dsv4_workspace_bytes.restype = sz
    lib.dsv4_status_string.argtypes = [ctypes.c_int]
    lib.dsv4_status_string.restype = ctypes.c_char_p
    lib.dsv4_version.restype = i32
    lib.dsv4_launch_count.restype = ctypes.c_uint64
    lib.dsv4_device_check.argtypes = [vp]
    lib.dsv4_device_check.restype = ctypes.c_int
    for fn in ("dsv4_compress_kv", "dsv4_indexer_topk", "dsv4_sparse_mqa_attn", "dsv4_csa_layer",
               "dsv4_hca_layer", "dsv4_indexer_topk_noalloc", "dsv4_indexer_scores", "dsv4_topk_select",
               "dsv4_decode_append", "dsv4_grouped_out_proj", "dsv4_sparse_mqa_attn_scores", "dsv4_add_rms_norm",
               "dsv4_route_experts", "dsv4_expert_mlp"):
        getattr(lib, fn).restype = ctypes.c_int
    _lib = lib
    _find_calls(lib)
    return lib


# The calls without ctypes (csrc/binding.cpp): status, or None for arguments that are not for them
# (raw pointers, and what the functions below refuse); None before load() and without the module.
_norm = _route = _experts = None


def _find_calls(lib) -> None:
    global _norm, _route, _experts
    try:
        from . import _binding
    except ImportError:
        return

    def entry(name, sized=0):
        holds = sum("-ALFIQX".index(k) << 4 * i for i, k in enumerate(_HOLDS[name]))
        return _binding.entry(ctypes.cast(getattr(lib, name), ctypes.c_void_p).value, len(_HOLDS[name]), holds, sized)
    _norm = entry("dsv4_add_rms_norm")
    _route = entry("dsv4_route_experts")
    _experts = entry("dsv4_expert_mlp", 1)


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


_torch_now = None


def _now():
    """(the current CUDA device, its current stream's cudaStream_t): what torch.cuda.current_device()
    and current_stream().cuda_stream say, without a Stream object (3 us)."""
    global _torch_now
    if _torch_now is None:
        import torch
        torch.cuda.current_device()  # initialises CUDA
        _torch_now = (getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device),
                      getattr(torch._C, "_cuda_getCurrentRawStream", lambda d: torch.cuda.current_stream(d).cuda_stream))
    device = _torch_now[0]()
    return device, _torch_now[1](device)


def _stream(stream) -> int | None:
    if stream is None:
        return _now()[1]
    return stream if isinstance(stream, int) else stream.cuda_stream


def _refuse(fn: str, t, device: int):
    if t.get_device() != device:
        raise Dsv4Error(fn, 1, f"a tensor is on {t.device}, not on the current CUDA device")
    raise Dsv4Error(fn, 1, f"a tensor of strides {tuple(t.stride())} is not contiguous")


def _dense(fn: str, stream, *tensors) -> list:
    """Pointers of tensors that the kernels can read as the header's shapes say, on the current device
    (the one that the launch goes to) and contiguous; then the stream's handle."""
    first = tensors[0]
    if first is None or type(first) is int:  # raw pointers: as the C call takes them
        first = next((t for t in tensors if t is not None and type(t) is not int), None)
        if first is None:
            return [*tensors, _stream(stream)]
    if first.get_device() < 0:
        _refuse(fn, first, 0)
    device, current = _now()
    out = [t if t is None or type(t) is int else
           t.data_ptr() if t.get_device() == device and t.is_contiguous() else _refuse(fn, t, device) for t in tensors]
    out.append(current if stream is None else _stream(stream))
    return out


# What the kernels read and write of each argument: the activations' type (A) or the logits' (L), floats (F)
# and integers (I) of 32 bits, e4m3 (Q), the experts' rows (X: Q with scales, else A), whatever there is (-).
_HOLDS = {"dsv4_add_rms_norm": "AAAAAQF", "dsv4_route_experts": "LFIF", "dsv4_expert_mlp": "XFIFAAA-"}
_types = None


def _find_types() -> dict:
    global _types
    import torch
    _types = {F32: (torch.float32,), BF16: (torch.bfloat16,), "F": (torch.float32,), "I": (torch.int32,),
              "Q": (torch.float8_e4m3fn, torch.uint8)}
    return _types


def _elements(fn: str, p) -> tuple:
    """Elements that the kernels read and write of each argument."""
    rows, scales = p.T * p.hidden, p.T * -(-p.hidden // 128)
    if fn == "dsv4_add_rms_norm":
        return rows, rows, p.hidden, rows, rows, rows, scales
    if fn == "dsv4_route_experts":
        return p.T * p.E, p.E, p.T * p.topk, p.T * p.topk
    matrix = p.E * p.inter * p.hidden
    return rows, scales, p.T * p.topk, p.T * p.topk, 2 * matrix, matrix, rows, 0


def _fit(fn: str, params, *tensors) -> None:
    """The tensors hold what the kernels take them for (what torch.topk returns, int64 ids and weights of the
    logits' type, is not it), and enough of it.  Of a call without tokens nothing is looked at."""
    if params.T <= 0:
        return
    types = _types or _find_types()
    for kind, t, need in zip(_HOLDS[fn], tensors, _elements(fn, params)):
        if t is None or type(t) is int:
            continue
        if kind == "X":
            kind = "A" if tensors[1] is None else "Q"
        want = types.get(params.dtype if kind == "A" else params.logits_dtype if kind == "L" else kind)
        if want and t.dtype not in want:
            raise Dsv4Error(fn, 1, f"a tensor of type {t.dtype} instead of {want[0]}")
        if kind != "-" and t.numel() < need:
            raise Dsv4Error(fn, 1, f"a tensor of {t.numel()} elements where the call has {need}")


def _check(fn: str, st: int) -> None:
    if st != 0:
        raise Dsv4Error(fn, st, load().dsv4_status_string(st).decode())


def dsv4_device_check(stream=None) -> None:
    """Synchronise the stream and raise if a kernel reported a device-side failure."""
    _check("dsv4_device_check", load().dsv4_device_check(_stream(stream)))


def dsv4_launch_count() -> int:
    return int(load().dsv4_launch_count())


def dsv4_workspace_bytes(params: Dsv4Params) -> int:
    return int(load().dsv4_workspace_bytes(ctypes.byref(params)))


def dsv4_compress_kv(params, c, x, z, bias, pos, apply_rope, pool, x_rot, stream=None):
    _check("dsv4_compress_kv", load().dsv4_compress_kv(
        ctypes.byref(params), int(c), _ptr(x), _ptr(z), _ptr(bias), _ptr(pos), int(apply_rope), _ptr(pool),
        _ptr(x_rot), _stream(stream)))


def dsv4_indexer_topk(params, qI, wI, poolI, q_index, idx, workspace, ws_bytes=None, stream=None):
    ws_bytes = workspace.numel() * workspace.element_size() if ws_bytes is None and workspace is not None \
        else (ws_bytes or 0)
    _check("dsv4_indexer_topk", load().dsv4_indexer_topk(
        ctypes.byref(params), _ptr(qI), _ptr(wI), _ptr(poolI), _ptr(q_index), _ptr(idx), _ptr(workspace),
        ws_bytes, _stream(stream)))


def dsv4_indexer_topk_noalloc(params, qI, wI, poolI, q_index, idx, stream=None):
    """dsv4_indexer_topk without a workspace: scores go to the library's fixed device scratch."""
    _check("dsv4_indexer_topk_noalloc", load().dsv4_indexer_topk_noalloc(
        ctypes.byref(params), _ptr(qI), _ptr(wI), _ptr(poolI), _ptr(q_index), _ptr(idx), _stream(stream)))


def dsv4_indexer_scores(params, qI, wI, poolI, q_index, scores, stream=None):
    """Lightning Indexer scores only: scores[B*Sq, P_cap] f32 (entries past each row's visible count untouched)."""
    _check("dsv4_indexer_scores", load().dsv4_indexer_scores(
        ctypes.byref(params), _ptr(qI), _ptr(wI), _ptr(poolI), _ptr(q_index), _ptr(scores), _stream(stream)))


def dsv4_topk_select(params, scores, q_index, idx, stream=None):
    """Per-query top-k over given score rows: idx[B,Sq,topk] ascending entries, then -1."""
    _check("dsv4_topk_select", load().dsv4_topk_select(
        ctypes.byref(params), _ptr(scores), _ptr(q_index), _ptr(idx), _stream(stream)))


def dsv4_decode_append(params, c, x, z, bias, pos, t, buf_x, buf_z, buf_pos, apply_rope, win, pool, stream=None):
    """Append one token per sequence to the decode cache (buffer, window ring, pool)."""
    _check("dsv4_decode_append", load().dsv4_decode_append(
        ctypes.byref(params), c, _ptr(x), _ptr(z), _ptr(bias), _ptr(pos), _ptr(t), _ptr(buf_x), _ptr(buf_z),
        _ptr(buf_pos), apply_rope, _ptr(win), _ptr(pool), _stream(stream)))


def dsv4_sparse_mqa_attn(params, q, kv_win, pool, idx, sink, qpos, q_index, out, workspace=None,
                         ws_bytes=None, stream=None):
    ws_bytes = workspace.numel() * workspace.element_size() if ws_bytes is None and workspace is not None \
        else (ws_bytes or 0)
    _check("dsv4_sparse_mqa_attn", load().dsv4_sparse_mqa_attn(
        ctypes.byref(params), _ptr(q), _ptr(kv_win), _ptr(pool), _ptr(idx), _ptr(sink), _ptr(qpos),
        _ptr(q_index), _ptr(out), _ptr(workspace), ws_bytes, _stream(stream)))


def dsv4_sparse_mqa_attn_scores(params, q, kv_win, pool, scores, sink, qpos, q_index, idx, out, workspace=None,
                                ws_bytes=None, stream=None):
    ws_bytes = workspace.numel() * workspace.element_size() if ws_bytes is None and workspace is not None \
        else (ws_bytes or 0)
    _check("dsv4_sparse_mqa_attn_scores", load().dsv4_sparse_mqa_attn_scores(
        ctypes.byref(params), _ptr(q), _ptr(kv_win), _ptr(pool), _ptr(scores), _ptr(sink), _ptr(qpos),
        _ptr(q_index), _ptr(idx), _ptr(out), _ptr(workspace), ws_bytes, _stream(stream)))


def dsv4_csa_layer(params, q, kv, z, bias, qI, wI, kI, zI, biasI, sink, pos, out, pool, poolI, kv_rot, idx,
                   workspace, ws_bytes=None, stream=None):
    ws_bytes = workspace.numel() * workspace.element_size() if ws_bytes is None and workspace is not None \
        else (ws_bytes or 0)
    _check("dsv4_csa_layer", load().dsv4_csa_layer(
        ctypes.byref(params), _ptr(q), _ptr(kv), _ptr(z), _ptr(bias), _ptr(qI), _ptr(wI), _ptr(kI), _ptr(zI),
        _ptr(biasI), _ptr(sink), _ptr(pos), _ptr(out), _ptr(pool), _ptr(poolI), _ptr(kv_rot), _ptr(idx),
        _ptr(workspace), ws_bytes, _stream(stream)))


def dsv4_hca_layer(params, q, kv, z, bias, sink, pos, out, pool, kv_rot, workspace=None, ws_bytes=None,
                   stream=None):
    ws_bytes = workspace.numel() * workspace.element_size() if ws_bytes is None and workspace is not None \
        else (ws_bytes or 0)
    _check("dsv4_hca_layer", load().dsv4_hca_layer(
        ctypes.byref(params), _ptr(q), _ptr(kv), _ptr(z), _ptr(bias), _ptr(sink), _ptr(pos), _ptr(out),
        _ptr(pool), _ptr(kv_rot), _ptr(workspace), ws_bytes, _stream(stream)))


def dsv4_grouped_out_proj(params, T, groups, dg, hidden, o, wa, wb, u, y, stream=None):
    _check("dsv4_grouped_out_proj",
           load().dsv4_grouped_out_proj(ctypes.byref(params), T, groups, dg, hidden, _ptr(o), _ptr(wa), _ptr(wb),
                                        _ptr(u), _ptr(y), _stream(stream)))


def dsv4_add_rms_norm(params, x, residual, weight, res_out, y, yq=None, yscale=None, stream=None):
    """r = x + residual (res_out), y = rms_norm(r) * weight, and y in e4m3 with a scale per 128 channels."""
    if _norm is not None:
        st = _norm(params, x, residual, weight, res_out, y, yq, yscale, stream if stream is None else _stream(stream))
        if st is not None:
            return _check("dsv4_add_rms_norm", st)
    args = _dense("dsv4_add_rms_norm", stream, x, residual, weight, res_out, y, yq, yscale)
    _fit("dsv4_add_rms_norm", params, x, residual, weight, res_out, y, yq, yscale)
    _check("dsv4_add_rms_norm", load().dsv4_add_rms_norm(ctypes.byref(params), *args))


def dsv4_route_experts(params, logits, bias, ids, weights, stream=None):
    """The topk experts of each token (ids, in descending order of score + bias) and their weights."""
    if _route is not None:
        st = _route(params, logits, bias, ids, weights, stream if stream is None else _stream(stream))
        if st is not None:
            return _check("dsv4_route_experts", st)
    args = _dense("dsv4_route_experts", stream, logits, bias, ids, weights)
    _fit("dsv4_route_experts", params, logits, bias, ids, weights)
    _check("dsv4_route_experts", load().dsv4_route_experts(ctypes.byref(params), *args))


def dsv4_expert_mlp_workspace_bytes(params: Dsv4MoeParams) -> int:
    return int(load().dsv4_expert_mlp_workspace_bytes(ctypes.byref(params)))


def dsv4_expert_mlp(params, x, x_scale, ids, weights, w13, w2, out, workspace, ws_bytes=None, stream=None):
    """The weighted sum of each token's experts' clamped SwiGLU products."""
    if ws_bytes is None and _experts is not None:
        st = _experts(params, x, x_scale, ids, weights, w13, w2, out, workspace, stream if stream is None else _stream(stream))
        if st is not None:
            return _check("dsv4_expert_mlp", st)
    ws_bytes = workspace.numel() * workspace.element_size() if ws_bytes is None and workspace is not None \
        else (ws_bytes or 0)
    *ptrs, stream = _dense("dsv4_expert_mlp", stream, x, x_scale, ids, weights, w13, w2, out, workspace)
    _fit("dsv4_expert_mlp", params, x, x_scale, ids, weights, w13, w2, out, workspace)
    _check("dsv4_expert_mlp", load().dsv4_expert_mlp(ctypes.byref(params), *ptrs, ws_bytes, stream))


def dsv4_set_index_checks(on: bool) -> None:
    load().dsv4_set_index_checks(1 if on else 0)


def dsv4_index_checks() -> bool:
    return bool(load().dsv4_index_checks())
