"""MI355X-native Kimi Delta Attention (KDA) forward: Python binding of libkda.so.

The binding only marshals arguments: it checks devices, dtypes, shapes and
contiguity, allocates outputs with torch (device memory and streams are all
torch is used for) and calls the C ABI declared in ``include/kda.h``. Every step
of the computation runs in the HIP kernels. There is no CPU or PyTorch fallback:
if ``libkda.so`` is missing or a call fails, an error is raised.

Entry points (same names as the C ABI):

* ``kda_chunk_fwd(q, k, v, g, beta, scale=None, initial_state=None,
  output_final_state=True, chunk_size=64, qk_l2norm=False, beta_sigmoid=False)
  -> (o, final_state)``
* ``kda_recurrent_step(q, k, v, g, beta, state, scale=None, qk_l2norm=False,
  beta_sigmoid=False) -> o`` (updates ``state`` in place)
* ``kda_gate_fwd(x, A_log, dt_bias=None, lower_bound=None) -> g`` and
  ``kda_gate_bwd(x, A_log, dt_bias, dg, lower_bound=None) -> (dx, dA_log, ddt_bias)``:
  the decay gate that produces g, and its backward
* ``kda_chunk_fwd_gated`` / ``kda_recurrent_step_gated``: the prefill and the decode step
  with that gate applied inside the kernels (the gate's input in place of g)
* ``kda_chunk_fwd_segmented(q, k, v, g, beta, segments, ...)``: the prefill over segments
  of each sequence composed by a scan (for few heads)
* ``kda_conv_fwd`` / ``kda_conv_bwd`` / ``kda_conv_step``: the short causal convolution in front
  of the recurrence (dense batches and packed sequences), its backward, and one token on a pool
  of states
* ``kda_ssm_chunk_fwd`` / ``kda_ssm_step``: the selective state space scan with one decay per
  head, for prompts and for one token on a pool of states
* ``kda_slots_copy`` / ``kda_slots_compact``: copies, forks, clears and compaction of the slots of
  many state pools at once
* ``kda_prenorm_fwd`` / ``kda_prenorm_bwd`` and ``kda_postnorm_fwd`` / ``kda_postnorm_bwd``: the norms
  in front of and behind a block, with its gate, residual and residual scale
* ``kda_glr_fwd`` / ``kda_glr_bwd`` / ``kda_glr_step``: the gated linear recurrence with one state
  per channel, its backward, and one token on a pool of states
* ``kda_checkpoint_pack`` / ``kda_checkpoint_unpack``: activations kept in 8 bits, which these
  backward passes read as they are
* ``kda_chunk_fwd_noalloc(q, k, v, g, beta, o, final_state=None, ...)``: the prefill into
  caller-provided outputs, with the workspace taken from the library's fixed per-device
  scratch array (no device allocation anywhere in the call)

``qk_l2norm`` / ``beta_sigmoid`` ask the kernels to L2-normalise q and k and to
apply the sigmoid to beta (``kda_chunk_fwd_ex`` / ``kda_recurrent_step_ex``).
"""

import ctypes
import math
import os

import torch

__all__ = ["kda_chunk_fwd", "kda_chunk_fwd_varlen", "kda_chunk_bwd",
           "kda_chunk_bwd_varlen", "kda_recurrent_step",
           "kda_recurrent_step_slots", "kda_gate_fwd", "kda_gate_bwd",
           "kda_chunk_fwd_gated", "kda_recurrent_step_gated", "kda_chunk_fwd_segmented",
           "kda_chunk_fwd_noalloc",
           "kda_conv_fwd", "kda_conv_bwd", "kda_conv_step", "kda_slots_copy",
           "kda_slots_compact", "kda_ssm_chunk_fwd", "kda_ssm_step",
           "kda_prenorm_fwd", "kda_prenorm_bwd", "kda_postnorm_fwd", "kda_postnorm_bwd",
           "kda_checkpoint_pack", "kda_checkpoint_unpack", "kda_glr_fwd", "kda_glr_bwd", "kda_glr_step",
           "NOALLOC_SCRATCH_BYTES", "library", "library_path", "status_string",
           "KDA_OK", "KDA_ERR_INVALID", "KDA_ERR_UNSUPPORTED", "KDA_ERR_HIP", "KDA_ERR_SCRATCH",
           "KDA_FLAG_QK_L2NORM", "KDA_FLAG_BETA_SIGMOID"]

KDA_OK, KDA_ERR_INVALID, KDA_ERR_UNSUPPORTED, KDA_ERR_HIP, KDA_ERR_SCRATCH = 0, -1, -2, -3, -4
NOALLOC_SCRATCH_BYTES = 64 << 20  # KDA_NOALLOC_SCRATCH_BYTES
KDA_FLAG_QK_L2NORM, KDA_FLAG_BETA_SIGMOID = 1, 2
KDA_CONV_SILU, KDA_ZERO_REST, KDA_GLR_NORMALISE, KDA_NORM_SILU = 1, 2, 4, 1
GLR_BLOCK = 64  # tokens between the states that kda_glr_fwd keeps for kda_glr_bwd
_DTYPE = {torch.float32: 0, torch.bfloat16: 1}

library_path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libkda.so")
_lib = None


def library():
    """Load libkda.so (once) and declare its C signatures. Raises if it is not built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(library_path):
        raise RuntimeError(f"{library_path} is not built; run `python -m gated_delta_rule_67_amd.build`")
    lib = ctypes.CDLL(library_path)
    vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    lib.kda_chunk_fwd.argtypes = [vp] * 8 + [i] * 6 + [f, i, i, vp, sz, vp]
    lib.kda_chunk_fwd.restype = i
    lib.kda_chunk_fwd_ex.argtypes = [vp] * 8 + [i] * 6 + [f, i, i, vp, sz, ctypes.c_uint, vp]
    lib.kda_chunk_fwd_ex.restype = i
    lib.kda_chunk_fwd_workspace_size.argtypes = [i] * 8
    lib.kda_chunk_fwd_workspace_size.restype = sz
    lib.kda_chunk_fwd_varlen.argtypes = [vp] * 6 + [i] + [vp] * 3 + [i] * 5 + [f, i, vp, sz,
                                                                            ctypes.c_uint, vp]
    lib.kda_chunk_fwd_varlen.restype = i
    lib.kda_chunk_fwd_varlen_workspace_size.argtypes = [i] * 7
    lib.kda_chunk_fwd_varlen_workspace_size.restype = sz
    u = ctypes.c_uint
    lib.kda_chunk_bwd.argtypes = [vp] * 14 + [i] * 6 + [f, i, i, vp, sz, vp]
    lib.kda_chunk_bwd_ex.argtypes = [vp] * 14 + [i] * 6 + [f, i, i, vp, sz, u, vp]
    lib.kda_chunk_bwd_ex.restype = i
    lib.kda_chunk_bwd_workspace_size_ex.argtypes = [i] * 8 + [u]
    lib.kda_chunk_bwd_workspace_size_ex.restype = sz
    lib.kda_chunk_bwd_varlen.argtypes = [vp] * 6 + [i] + [vp] * 9 + [i] * 5 + [f, i, vp, sz, u, vp]
    lib.kda_chunk_bwd_varlen.restype = i
    lib.kda_chunk_bwd_varlen_workspace_size.argtypes = [i] * 7 + [u]
    lib.kda_chunk_bwd_varlen_workspace_size.restype = sz
    lib.kda_chunk_bwd.restype = i
    lib.kda_chunk_bwd_workspace_size.argtypes = [i] * 8
    lib.kda_chunk_bwd_workspace_size.restype = sz
    lib.kda_recurrent_step.argtypes = [vp] * 7 + [i] * 5 + [f, i, vp]
    lib.kda_recurrent_step.restype = i
    lib.kda_recurrent_step_ex.argtypes = [vp] * 7 + [i] * 5 + [f, i, ctypes.c_uint, vp]
    lib.kda_recurrent_step_ex.restype = i
    lib.kda_recurrent_step_slots.argtypes = [vp] * 7 + [i, vp] + [i] * 5 + [f, i, ctypes.c_uint, vp]
    lib.kda_recurrent_step_slots.restype = i
    lib.kda_gate_fwd.argtypes = [vp] * 4 + [i] * 4 + [f, i, vp]
    lib.kda_gate_fwd.restype = i
    lib.kda_gate_bwd_workspace_size.argtypes = [i] * 5
    lib.kda_gate_bwd_workspace_size.restype = sz
    lib.kda_gate_bwd.argtypes = [vp] * 7 + [i] * 4 + [f, i, vp, sz, vp]
    lib.kda_gate_bwd.restype = i
    lib.kda_chunk_fwd_gated.argtypes = [vp] * 6 + [f] + [vp] * 4 + [i] * 6 + [f, i, i, vp, sz,
                                                                            ctypes.c_uint, vp]
    lib.kda_chunk_fwd_gated.restype = i
    lib.kda_recurrent_step_gated.argtypes = [vp] * 6 + [f] + [vp] * 3 + [i] * 5 + [f, i,
                                                                                 ctypes.c_uint, vp]
    lib.kda_recurrent_step_gated.restype = i
    lib.kda_chunk_fwd_segmented.argtypes = [vp] * 8 + [i] * 6 + [f, i, i, vp, sz, ctypes.c_uint, vp]
    lib.kda_chunk_fwd_segmented.restype = i
    lib.kda_chunk_fwd_segmented_workspace_size.argtypes = [i] * 8
    lib.kda_chunk_fwd_segmented_workspace_size.restype = sz
    lib.kda_chunk_fwd_noalloc.argtypes = [vp] * 8 + [i] * 6 + [f, i, i, ctypes.c_uint, vp]
    lib.kda_chunk_fwd_noalloc.restype = i
    lib.kda_stream_copy.argtypes = [vp, vp, sz, vp]
    lib.kda_stream_copy.restype = i
    lib.kda_status_string.argtypes = [i]
    lib.kda_status_string.restype = ctypes.c_char_p
    i64 = ctypes.c_int64
    lib.kda_conv_fwd.argtypes = [vp, i64] + [vp] * 4 + [i] + [vp] * 2 + [i] * 5 + [vp]
    lib.kda_conv_fwd.restype = i
    lib.kda_conv_bwd_workspace_size.argtypes = [i] * 4
    lib.kda_conv_bwd_workspace_size.restype = sz
    lib.kda_conv_bwd.argtypes = ([vp, i64] + [vp] * 4 + [i, vp, i64] + [vp] * 5 + [i] * 5
                                 + [vp, sz, vp])
    lib.kda_conv_bwd.restype = i
    lib.kda_conv_step.argtypes = [vp, i64] + [vp] * 4 + [i, vp] + [i] * 5 + [vp]
    lib.kda_conv_step.restype = i
    ssm = [vp, i64, vp, i64, vp, vp, i64, vp, i64, vp, vp]
    lib.kda_ssm_chunk_fwd_workspace_size.argtypes = [i] * 8
    lib.kda_ssm_chunk_fwd_workspace_size.restype = sz
    lib.kda_ssm_chunk_fwd.argtypes = (ssm + [vp, vp, i, vp, vp] + [i] * 5
                                      + [ctypes.c_uint, i, vp, sz, vp])
    lib.kda_ssm_chunk_fwd.restype = i
    lib.kda_ssm_step.argtypes = ssm + [vp, vp, i, vp] + [i] * 6 + [vp]
    lib.kda_ssm_step.restype = i
    lib.kda_slots_copy.argtypes = [vp] * 2 + [i, i] + [vp] * 2 + [i, vp]
    lib.kda_slots_copy.restype = i
    lib.kda_slots_compact_workspace_size.argtypes = [i]
    lib.kda_slots_compact_workspace_size.restype = sz
    lib.kda_slots_compact.argtypes = [vp] * 2 + [i, i] + [vp] * 4 + [sz, vp]
    lib.kda_slots_compact.restype = i
    u = ctypes.c_uint
    rows = [i64, i, i, f]  # T, G, D, eps
    lib.kda_prenorm_fwd.argtypes = [vp, i64, vp, i64, vp, vp, vp, vp] + rows + [i, vp]
    lib.kda_postnorm_fwd.argtypes = [vp, i64, vp, vp, i64, vp, i64, vp, vp] + rows + [u, i, vp]
    lib.kda_norm_bwd_workspace_size.argtypes = [i64, i, i]
    lib.kda_norm_bwd_workspace_size.restype = sz
    kept = [vp, vp, i64]   # a tensor or codes, scales, stride
    lib.kda_prenorm_bwd.argtypes = (kept + [vp, vp, i64, vp, i64] + kept + [vp] * 5 + rows
                                    + [i, vp, sz, vp])
    lib.kda_postnorm_bwd.argtypes = (kept + [vp] + kept + [vp, i64] + [vp] * 5 + rows
                                     + [u, i, vp, sz, vp])
    lib.kda_checkpoint_pack.argtypes = [vp, i64, vp, vp, i64, i, i, vp]
    lib.kda_checkpoint_unpack.argtypes = [vp, vp, vp, i64, i, i, vp]
    lib.kda_glr_fwd_workspace_size.argtypes = [i, i]
    lib.kda_glr_fwd_workspace_size.restype = sz
    lib.kda_glr_bwd_workspace_size.argtypes = [i, i, i]
    lib.kda_glr_bwd_workspace_size.restype = sz
    lib.kda_glr_fwd.argtypes = ([vp, i64, vp, i64, vp, vp, vp, i64, vp, vp, i, vp, vp, vp, i, i, u, i]
                                + [vp, sz, vp])
    lib.kda_glr_bwd.argtypes = (kept + kept + [vp, vp] + kept + [vp, vp, i, vp, i64] + [vp] * 8
                                + [i, i, u, i, vp, sz, vp])
    lib.kda_glr_step.argtypes = [vp, i64, vp, i64, vp, vp, vp, i64, vp, vp, i, vp, i, i, u, i, vp]
    for name in ("prenorm_fwd", "prenorm_bwd", "postnorm_fwd", "postnorm_bwd", "checkpoint_pack",
                 "checkpoint_unpack", "glr_fwd", "glr_bwd", "glr_step"):
        getattr(lib, "kda_" + name).restype = i
    lib.kda_version.argtypes = []
    lib.kda_version.restype = ctypes.c_char_p
    _lib = lib
    return lib


def status_string(rc):
    return library().kda_status_string(int(rc)).decode()


def _check(rc):
    if rc != KDA_OK:
        raise RuntimeError(status_string(rc))


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _require(cond, msg):
    if not cond:
        raise ValueError(msg)


def _check_tensors(named, dtype, device):
    for name, t in named:
        _require(t.device == device, f"{name} is on {t.device}, expected {device}")
        _require(t.dtype == dtype, f"{name} has dtype {t.dtype}, expected {dtype}")
        _require(t.is_contiguous(), f"{name} must be contiguous")


def _flags(qk_l2norm, beta_sigmoid):
    return (KDA_FLAG_QK_L2NORM if qk_l2norm else 0) | (KDA_FLAG_BETA_SIGMOID if beta_sigmoid else 0)


def kda_chunk_fwd(q, k, v, g, beta, scale=None, initial_state=None, output_final_state=True,
                  chunk_size=64, qk_l2norm=False, beta_sigmoid=False):
    """Chunked KDA prefill. q, k [B,T,H,K]; v [B,T,HV,V]; g [B,T,HV,K]; beta [B,T,HV];
    initial_state [B,HV,K,V] float32 or None. Returns (o [B,T,HV,V], final_state or None).
    qk_l2norm / beta_sigmoid: apply those input transforms in the kernels."""
    _require(q.is_cuda, "inputs must be on a GPU")
    dev, dt = q.device, q.dtype
    _require(dt in _DTYPE, f"unsupported dtype {dt}")
    B, T, H, K = q.shape
    HV, V = v.shape[2], v.shape[3]
    _require(k.shape == q.shape, "k must match q")
    _require(tuple(v.shape[:2]) == (B, T), "v must be [B, T, HV, V]")
    _require(tuple(g.shape) == (B, T, HV, K), "g must be [B, T, HV, K]")
    _require(tuple(beta.shape) == (B, T, HV), "beta must be [B, T, HV]")
    _check_tensors([("q", q), ("k", k), ("v", v), ("g", g), ("beta", beta)], dt, dev)
    if initial_state is not None:
        _require(tuple(initial_state.shape) == (B, HV, K, V), "initial_state must be [B, HV, K, V]")
        _check_tensors([("initial_state", initial_state)], torch.float32, dev)
    if scale is None:
        scale = 1.0 / math.sqrt(K)
    lib = library()
    o = torch.empty((B, T, HV, V), dtype=dt, device=dev)
    final = torch.empty((B, HV, K, V), dtype=torch.float32, device=dev) if output_final_state else None
    ws_bytes = lib.kda_chunk_fwd_workspace_size(B, T, H, HV, K, V, chunk_size, _DTYPE[dt])
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev) if ws_bytes else None
    with torch.cuda.device(dev):
        stream = torch.cuda.current_stream(dev).cuda_stream
        rc = lib.kda_chunk_fwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                  _ptr(initial_state), _ptr(final), _ptr(o), B, T, H, HV, K, V,
                                  float(scale), int(chunk_size), _DTYPE[dt], _ptr(ws), ws_bytes,
                                  _flags(qk_l2norm, beta_sigmoid), ctypes.c_void_p(stream))
    _check(rc)
    return o, final


def kda_chunk_fwd_varlen(q, k, v, g, beta, cu_seqlens, scale=None, initial_state=None,
                         output_final_state=True, qk_l2norm=False, beta_sigmoid=False):
    """Packed variable-length prefill (bf16). q, k [1,T,H,K] (or [T,H,K]); v [1,T,HV,V];
    g [1,T,HV,K]; beta [1,T,HV]; cu_seqlens int32 [N+1] on the same device; initial_state
    [N,HV,K,V] float32 or None. Returns (o shaped like v, final_state [N,HV,K,V] or None)."""
    _require(q.is_cuda, "inputs must be on a GPU")
    dev, dt = q.device, q.dtype
    _require(dt in _DTYPE, f"unsupported dtype {dt}")
    squeeze = q.dim() == 3
    if not squeeze:
        _require(q.shape[0] == 1, "packed inputs have batch size 1")
        q, k, v, g, beta = q[0], k[0], v[0], g[0], beta[0]
    T, H, K = q.shape
    HV, V = v.shape[1], v.shape[2]
    _require(k.shape == q.shape, "k must match q")
    _require(v.shape[0] == T, "v must be [T, HV, V]")
    _require(tuple(g.shape) == (T, HV, K), "g must be [T, HV, K]")
    _require(tuple(beta.shape) == (T, HV), "beta must be [T, HV]")
    _check_tensors([("q", q), ("k", k), ("v", v), ("g", g), ("beta", beta)], dt, dev)
    _require(cu_seqlens.is_cuda and cu_seqlens.device == dev, "cu_seqlens must be on the same GPU")
    _require(cu_seqlens.dtype == torch.int32 and cu_seqlens.dim() == 1 and cu_seqlens.is_contiguous(),
             "cu_seqlens must be a contiguous int32 vector")
    N = cu_seqlens.numel() - 1
    _require(N >= 1, "cu_seqlens needs at least two offsets")
    if initial_state is not None:
        _require(tuple(initial_state.shape) == (N, HV, K, V), "initial_state must be [N, HV, K, V]")
        _check_tensors([("initial_state", initial_state)], torch.float32, dev)
    if scale is None:
        scale = 1.0 / math.sqrt(K)
    lib = library()
    o = torch.empty((T, HV, V), dtype=dt, device=dev)
    final = torch.empty((N, HV, K, V), dtype=torch.float32, device=dev) if output_final_state else None
    ws_bytes = lib.kda_chunk_fwd_varlen_workspace_size(N, T, H, HV, K, V, _DTYPE[dt])
    ws = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=dev)
    with torch.cuda.device(dev):
        stream = torch.cuda.current_stream(dev).cuda_stream
        rc = lib.kda_chunk_fwd_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                      _ptr(cu_seqlens), N, _ptr(initial_state), _ptr(final),
                                      _ptr(o), T, H, HV, K, V, float(scale), _DTYPE[dt], _ptr(ws),
                                      ws_bytes, _flags(qk_l2norm, beta_sigmoid),
                                      ctypes.c_void_p(stream))
    _check(rc)
    return (o if squeeze else o.unsqueeze(0)), final


def kda_chunk_bwd(q, k, v, g, beta, do, scale=None, initial_state=None, dht=None, chunk_size=64,
                  need_dh0=True, qk_l2norm=False, beta_sigmoid=False):
    """Gradients of <o, do> + <final_state, dht> for kda_chunk_fwd's inputs (bf16).
    Shapes as kda_chunk_fwd; do [B,T,HV,V]; dht [B,HV,K,V] float32 or None.
    Returns (dq, dk, dv, dg, dbeta, dh0 or None); dh0 is float32 [B,HV,K,V].
    qk_l2norm / beta_sigmoid: the forward applied those transforms; gradients are for the
    raw inputs."""
    _require(q.is_cuda, "inputs must be on a GPU")
    dev, dt = q.device, q.dtype
    _require(dt in _DTYPE, f"unsupported dtype {dt}")
    B, T, H, K = q.shape
    HV, V = v.shape[2], v.shape[3]
    _require(k.shape == q.shape, "k must match q")
    _require(tuple(v.shape[:2]) == (B, T), "v must be [B, T, HV, V]")
    _require(tuple(g.shape) == (B, T, HV, K), "g must be [B, T, HV, K]")
    _require(tuple(beta.shape) == (B, T, HV), "beta must be [B, T, HV]")
    _require(tuple(do.shape) == (B, T, HV, V), "do must be [B, T, HV, V]")
    _check_tensors([("q", q), ("k", k), ("v", v), ("g", g), ("beta", beta), ("do", do)], dt, dev)
    for name, t in (("initial_state", initial_state), ("dht", dht)):
        if t is not None:
            _require(tuple(t.shape) == (B, HV, K, V), f"{name} must be [B, HV, K, V]")
            _check_tensors([(name, t)], torch.float32, dev)
    if scale is None:
        scale = 1.0 / math.sqrt(K)
    lib = library()
    dq = torch.empty((B, T, H, K), dtype=dt, device=dev)
    dk = torch.empty((B, T, H, K), dtype=dt, device=dev)
    dv = torch.empty((B, T, HV, V), dtype=dt, device=dev)
    dg = torch.empty((B, T, HV, K), dtype=dt, device=dev)
    dbeta = torch.empty((B, T, HV), dtype=dt, device=dev)
    dh0 = torch.empty((B, HV, K, V), dtype=torch.float32, device=dev) if need_dh0 else None
    flags = _flags(qk_l2norm, beta_sigmoid)
    ws_bytes = lib.kda_chunk_bwd_workspace_size_ex(B, T, H, HV, K, V, chunk_size, _DTYPE[dt], flags)
    ws = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=dev)
    with torch.cuda.device(dev):
        stream = torch.cuda.current_stream(dev).cuda_stream
        rc = lib.kda_chunk_bwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                  _ptr(initial_state), _ptr(do), _ptr(dht), _ptr(dq), _ptr(dk),
                                  _ptr(dv), _ptr(dg), _ptr(dbeta), _ptr(dh0), B, T, H, HV, K, V,
                                  float(scale), int(chunk_size), _DTYPE[dt], _ptr(ws), ws_bytes,
                                  flags, ctypes.c_void_p(stream))
    _check(rc)
    return dq, dk, dv, dg, dbeta, dh0


def kda_chunk_bwd_varlen(q, k, v, g, beta, do, cu_seqlens, scale=None, initial_state=None,
                         dht=None, need_dh0=True, qk_l2norm=False, beta_sigmoid=False):
    """Gradients for kda_chunk_fwd_varlen's inputs (bf16, packed sequences). Token tensors
    [1,T,...] (or [T,...]); cu_seqlens int32 [N+1]; initial_state, dht [N,HV,K,V] float32 or
    None. Returns (dq, dk, dv, dg, dbeta shaped like their inputs, dh0 [N,HV,K,V] or None)."""
    _require(q.is_cuda, "inputs must be on a GPU")
    dev, dt = q.device, q.dtype
    _require(dt in _DTYPE, f"unsupported dtype {dt}")
    squeeze = q.dim() == 3
    if not squeeze:
        _require(q.shape[0] == 1, "packed inputs have batch size 1")
        q, k, v, g, beta, do = q[0], k[0], v[0], g[0], beta[0], do[0]
    T, H, K = q.shape
    HV, V = v.shape[1], v.shape[2]
    _require(k.shape == q.shape, "k must match q")
    _require(tuple(v.shape) == (T, HV, V) and tuple(do.shape) == (T, HV, V), "v, do must be [T, HV, V]")
    _require(tuple(g.shape) == (T, HV, K), "g must be [T, HV, K]")
    _require(tuple(beta.shape) == (T, HV), "beta must be [T, HV]")
    _check_tensors([("q", q), ("k", k), ("v", v), ("g", g), ("beta", beta), ("do", do)], dt, dev)
    _require(cu_seqlens.is_cuda and cu_seqlens.device == dev and cu_seqlens.dtype == torch.int32
             and cu_seqlens.dim() == 1 and cu_seqlens.is_contiguous(), "cu_seqlens must be int32 on the GPU")
    N = cu_seqlens.numel() - 1
    _require(N >= 1, "cu_seqlens needs at least two offsets")
    for name, t in (("initial_state", initial_state), ("dht", dht)):
        if t is not None:
            _require(tuple(t.shape) == (N, HV, K, V), f"{name} must be [N, HV, K, V]")
            _check_tensors([(name, t)], torch.float32, dev)
    if scale is None:
        scale = 1.0 / math.sqrt(K)
    lib = library()
    dq, dk = torch.empty_like(q), torch.empty_like(k)
    dv, dg, dbeta = torch.empty_like(v), torch.empty_like(g), torch.empty_like(beta)
    dh0 = torch.empty((N, HV, K, V), dtype=torch.float32, device=dev) if need_dh0 else None
    flags = _flags(qk_l2norm, beta_sigmoid)
    ws_bytes = lib.kda_chunk_bwd_varlen_workspace_size(N, T, H, HV, K, V, _DTYPE[dt], flags)
    ws = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=dev)
    with torch.cuda.device(dev):
        stream = torch.cuda.current_stream(dev).cuda_stream
        rc = lib.kda_chunk_bwd_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                      _ptr(cu_seqlens), N, _ptr(initial_state), _ptr(do),
                                      _ptr(dht), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dg),
                                      _ptr(dbeta), _ptr(dh0), T, H, HV, K, V, float(scale),
                                      _DTYPE[dt], _ptr(ws), ws_bytes, flags, ctypes.c_void_p(stream))
    _check(rc)
    outs = (dq, dk, dv, dg, dbeta)
    if not squeeze:
        outs = tuple(x.unsqueeze(0) for x in outs)
    return outs + (dh0,)


def kda_recurrent_step(q, k, v, g, beta, state, scale=None, qk_l2norm=False, beta_sigmoid=False):
    """One decode token. q, k [B,H,K] (or [B,1,H,K]); v [B,HV,V]; g [B,HV,K]; beta [B,HV];
    state [B,HV,K,V] float32, updated in place. Returns o [B,HV,V].
    qk_l2norm / beta_sigmoid: apply those input transforms in the kernel."""
    _require(q.is_cuda, "inputs must be on a GPU")
    dev, dt = q.device, q.dtype
    _require(dt in _DTYPE, f"unsupported dtype {dt}")
    if q.dim() == 4:
        q, k, v, g, beta = q[:, 0], k[:, 0], v[:, 0], g[:, 0], beta[:, 0]
    B, H, K = q.shape
    HV, V = v.shape[1], v.shape[2]
    _require(k.shape == q.shape, "k must match q")
    _require(tuple(g.shape) == (B, HV, K), "g must be [B, HV, K]")
    _require(tuple(beta.shape) == (B, HV), "beta must be [B, HV]")
    _require(tuple(state.shape) == (B, HV, K, V), "state must be [B, HV, K, V]")
    _check_tensors([("q", q), ("k", k), ("v", v), ("g", g), ("beta", beta)], dt, dev)
    _check_tensors([("state", state)], torch.float32, dev)
    if scale is None:
        scale = 1.0 / math.sqrt(K)
    lib = library()
    o = torch.empty((B, HV, V), dtype=dt, device=dev)
    with torch.cuda.device(dev):
        stream = torch.cuda.current_stream(dev).cuda_stream
        rc = lib.kda_recurrent_step_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                       _ptr(state), _ptr(o), B, H, HV, K, V, float(scale),
                                       _DTYPE[dt], _flags(qk_l2norm, beta_sigmoid),
                                       ctypes.c_void_p(stream))
    _check(rc)
    return o


def kda_recurrent_step_slots(q, k, v, g, beta, state_pool, slots, scale=None, qk_l2norm=False,
                             beta_sigmoid=False):
    """One decode token per request against a slot-indexed state pool. q, k [B,H,K];
    v [B,HV,V]; g [B,HV,K]; beta [B,HV]; state_pool [num_slots,HV,K,V] float32 (updated in
    place); slots int32 [B] (a slot outside [0, num_slots) gives o = 0 and no update).
    Returns o [B,HV,V]."""
    _require(q.is_cuda, "inputs must be on a GPU")
    dev, dt = q.device, q.dtype
    _require(dt in _DTYPE, f"unsupported dtype {dt}")
    if q.dim() == 4:
        q, k, v, g, beta = q[:, 0], k[:, 0], v[:, 0], g[:, 0], beta[:, 0]
    B, H, K = q.shape
    HV, V = v.shape[1], v.shape[2]
    _require(k.shape == q.shape, "k must match q")
    _require(tuple(g.shape) == (B, HV, K), "g must be [B, HV, K]")
    _require(tuple(beta.shape) == (B, HV), "beta must be [B, HV]")
    _require(state_pool.dim() == 4 and tuple(state_pool.shape[1:]) == (HV, K, V),
             "state_pool must be [num_slots, HV, K, V]")
    _check_tensors([("q", q), ("k", k), ("v", v), ("g", g), ("beta", beta)], dt, dev)
    _check_tensors([("state_pool", state_pool)], torch.float32, dev)
    _require(slots.is_cuda and slots.device == dev and slots.dtype == torch.int32
             and tuple(slots.shape) == (B,) and slots.is_contiguous(), "slots must be int32 [B] on the GPU")
    if scale is None:
        scale = 1.0 / math.sqrt(K)
    lib = library()
    o = torch.empty((B, HV, V), dtype=dt, device=dev)
    with torch.cuda.device(dev):
        stream = torch.cuda.current_stream(dev).cuda_stream
        rc = lib.kda_recurrent_step_slots(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                          _ptr(state_pool), _ptr(slots), state_pool.shape[0],
                                          _ptr(o), B, H, HV, K, V, float(scale), _DTYPE[dt],
                                          _flags(qk_l2norm, beta_sigmoid), ctypes.c_void_p(stream))
    _check(rc)
    return o


def _gate_args(x, A_log, dt_bias, lower_bound):
    _require(x.is_cuda, "inputs must be on a GPU")
    dev, dt = x.device, x.dtype
    _require(dt in _DTYPE, f"unsupported dtype {dt}")
    _require(x.dim() == 4, "x must be [B, T, HV, K]")
    B, T, HV, K = x.shape
    _check_tensors([("x", x)], dt, dev)
    _require(tuple(A_log.shape) == (HV,), "A_log must be [HV]")
    _check_tensors([("A_log", A_log)], torch.float32, dev)
    if dt_bias is not None:
        _require(dt_bias.numel() == HV * K, "dt_bias must be [HV, K]")
        _check_tensors([("dt_bias", dt_bias)], torch.float32, dev)
    lb = float("-inf") if lower_bound is None else float(lower_bound)
    return dev, dt, B, T, HV, K, lb


def kda_gate_fwd(x, A_log, dt_bias=None, lower_bound=None):
    """The KDA decay gate: g = max(lower_bound, -exp(A_log[hv]) * softplus(x + dt_bias[hv]))
    for x [B,T,HV,K] (bf16 or float32), A_log [HV] and dt_bias [HV,K] float32 (or None).
    lower_bound None is the standard gate; a number <= 0 (the pages use -5) the safe gate.
    Returns g shaped and typed like x."""
    dev, dt, B, T, HV, K, lb = _gate_args(x, A_log, dt_bias, lower_bound)
    lib = library()
    g = torch.empty_like(x)
    with torch.cuda.device(dev):
        stream = torch.cuda.current_stream(dev).cuda_stream
        rc = lib.kda_gate_fwd(_ptr(x), _ptr(A_log), _ptr(dt_bias), _ptr(g), B, T, HV, K, lb,
                              _DTYPE[dt], ctypes.c_void_p(stream))
    _check(rc)
    return g


def kda_gate_bwd(x, A_log, dt_bias, dg, lower_bound=None):
    """Backward of kda_gate_fwd for the gradient dg reaching g. Returns (dx like x,
    dA_log [HV] float32, ddt_bias [HV,K] float32)."""
    dev, dt, B, T, HV, K, lb = _gate_args(x, A_log, dt_bias, lower_bound)
    _require(dg.shape == x.shape, "dg must match x")
    _check_tensors([("dg", dg)], dt, dev)
    lib = library()
    dx = torch.empty_like(x)
    dA_log = torch.empty((HV,), dtype=torch.float32, device=dev)
    ddt_bias = torch.empty((HV, K), dtype=torch.float32, device=dev)
    ws_bytes = lib.kda_gate_bwd_workspace_size(B, T, HV, K, _DTYPE[dt])
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev) if ws_bytes else None
    with torch.cuda.device(dev):
        stream = torch.cuda.current_stream(dev).cuda_stream
        rc = lib.kda_gate_bwd(_ptr(x), _ptr(A_log), _ptr(dt_bias), _ptr(dg), _ptr(dx),
                              _ptr(dA_log), _ptr(ddt_bias), B, T, HV, K, lb, _DTYPE[dt],
                              _ptr(ws), ws_bytes, ctypes.c_void_p(stream))
    _check(rc)
    return dx, dA_log, ddt_bias


def _gate_params(A_log, dt_bias, lower_bound, HV, K, dev):
    _require(tuple(A_log.shape) == (HV,), "A_log must be [HV]")
    _check_tensors([("A_log", A_log)], torch.float32, dev)
    if dt_bias is not None:
        _require(dt_bias.numel() == HV * K, "dt_bias must be [HV, K]")
        _check_tensors([("dt_bias", dt_bias)], torch.float32, dev)
    return float("-inf") if lower_bound is None else float(lower_bound)


def kda_chunk_fwd_gated(q, k, v, gate_x, A_log, dt_bias, beta, lower_bound=-5.0, scale=None,
                        initial_state=None, output_final_state=True, chunk_size=64,
                        qk_l2norm=False, beta_sigmoid=False):
    """kda_chunk_fwd with the decay gate applied in the kernels: gate_x [B,T,HV,K] (bf16) is
    the gate's input; g = max(lower_bound, -exp(A_log) softplus(gate_x + dt_bias)), rounded
    to bf16 as kda_gate_fwd stores it. lower_bound None: the standard gate.
    Returns (o, final_state)."""
    _require(q.is_cuda, "inputs must be on a GPU")
    dev, dt = q.device, q.dtype
    _require(dt in _DTYPE, f"unsupported dtype {dt}")
    B, T, H, K = q.shape
    HV, V = v.shape[2], v.shape[3]
    _require(k.shape == q.shape, "k must match q")
    _require(tuple(v.shape[:2]) == (B, T), "v must be [B, T, HV, V]")
    _require(tuple(gate_x.shape) == (B, T, HV, K), "gate_x must be [B, T, HV, K]")
    _require(tuple(beta.shape) == (B, T, HV), "beta must be [B, T, HV]")
    _check_tensors([("q", q), ("k", k), ("v", v), ("gate_x", gate_x), ("beta", beta)], dt, dev)
    lb = _gate_params(A_log, dt_bias, lower_bound, HV, K, dev)
    if initial_state is not None:
        _require(tuple(initial_state.shape) == (B, HV, K, V), "initial_state must be [B, HV, K, V]")
        _check_tensors([("initial_state", initial_state)], torch.float32, dev)
    if scale is None:
        scale = 1.0 / math.sqrt(K)
    lib = library()
    o = torch.empty((B, T, HV, V), dtype=dt, device=dev)
    final = torch.empty((B, HV, K, V), dtype=torch.float32, device=dev) if output_final_state else None
    ws_bytes = lib.kda_chunk_fwd_workspace_size(B, T, H, HV, K, V, chunk_size, _DTYPE[dt])
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev) if ws_bytes else None
    with torch.cuda.device(dev):
        stream = torch.cuda.current_stream(dev).cuda_stream
        rc = lib.kda_chunk_fwd_gated(_ptr(q), _ptr(k), _ptr(v), _ptr(gate_x), _ptr(A_log),
                                     _ptr(dt_bias), lb, _ptr(beta), _ptr(initial_state),
                                     _ptr(final), _ptr(o), B, T, H, HV, K, V, float(scale),
                                     int(chunk_size), _DTYPE[dt], _ptr(ws), ws_bytes,
                                     _flags(qk_l2norm, beta_sigmoid), ctypes.c_void_p(stream))
    _check(rc)
    return o, final


def kda_recurrent_step_gated(q, k, v, gate_x, A_log, dt_bias, beta, state, lower_bound=-5.0,
                             scale=None, qk_l2norm=False, beta_sigmoid=False):
    """kda_recurrent_step with the decay gate applied in the kernel: gate_x [B,HV,K] is the
    gate's input (as kda_chunk_fwd_gated). Updates state in place; returns o [B,HV,V]."""
    _require(q.is_cuda, "inputs must be on a GPU")
    dev, dt = q.device, q.dtype
    _require(dt in _DTYPE, f"unsupported dtype {dt}")
    if q.dim() == 4:
        q, k, v, gate_x, beta = q[:, 0], k[:, 0], v[:, 0], gate_x[:, 0], beta[:, 0]
    B, H, K = q.shape
    HV, V = v.shape[1], v.shape[2]
    _require(k.shape == q.shape, "k must match q")
    _require(tuple(gate_x.shape) == (B, HV, K), "gate_x must be [B, HV, K]")
    _require(tuple(beta.shape) == (B, HV), "beta must be [B, HV]")
    _require(tuple(state.shape) == (B, HV, K, V), "state must be [B, HV, K, V]")
    _check_tensors([("q", q), ("k", k), ("v", v), ("gate_x", gate_x), ("beta", beta)], dt, dev)
    _check_tensors([("state", state)], torch.float32, dev)
    lb = _gate_params(A_log, dt_bias, lower_bound, HV, K, dev)
    if scale is None:
        scale = 1.0 / math.sqrt(K)
    lib = library()
    o = torch.empty((B, HV, V), dtype=dt, device=dev)
    with torch.cuda.device(dev):
        stream = torch.cuda.current_stream(dev).cuda_stream
        rc = lib.kda_recurrent_step_gated(_ptr(q), _ptr(k), _ptr(v), _ptr(gate_x), _ptr(A_log),
                                          _ptr(dt_bias), lb, _ptr(beta), _ptr(state), _ptr(o), B,
                                          H, HV, K, V, float(scale), _DTYPE[dt],
                                          _flags(qk_l2norm, beta_sigmoid), ctypes.c_void_p(stream))
    _check(rc)
    return o


def kda_chunk_fwd_segmented(q, k, v, g, beta, segments, scale=None, initial_state=None,
                            output_final_state=True, qk_l2norm=False, beta_sigmoid=False):
    """kda_chunk_fwd over `segments` equal segments of each sequence, composed by a scan of the
    segments' affine state maps (bf16; T % (64 * segments) == 0). kda_chunk_fwd takes this
    route by itself when it pays; this entry point chooses the segment count explicitly.
    Returns (o, final_state)."""
    _require(q.is_cuda, "inputs must be on a GPU")
    dev, dt = q.device, q.dtype
    _require(dt in _DTYPE, f"unsupported dtype {dt}")
    B, T, H, K = q.shape
    HV, V = v.shape[2], v.shape[3]
    _require(k.shape == q.shape, "k must match q")
    _require(tuple(v.shape[:2]) == (B, T), "v must be [B, T, HV, V]")
    _require(tuple(g.shape) == (B, T, HV, K), "g must be [B, T, HV, K]")
    _require(tuple(beta.shape) == (B, T, HV), "beta must be [B, T, HV]")
    _check_tensors([("q", q), ("k", k), ("v", v), ("g", g), ("beta", beta)], dt, dev)
    if initial_state is not None:
        _require(tuple(initial_state.shape) == (B, HV, K, V), "initial_state must be [B, HV, K, V]")
        _check_tensors([("initial_state", initial_state)], torch.float32, dev)
    if scale is None:
        scale = 1.0 / math.sqrt(K)
    lib = library()
    o = torch.empty((B, T, HV, V), dtype=dt, device=dev)
    final = torch.empty((B, HV, K, V), dtype=torch.float32, device=dev) if output_final_state else None
    ws_bytes = lib.kda_chunk_fwd_segmented_workspace_size(B, T, H, HV, K, V, int(segments), _DTYPE[dt])
    ws = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=dev)
    with torch.cuda.device(dev):
        stream = torch.cuda.current_stream(dev).cuda_stream
        rc = lib.kda_chunk_fwd_segmented(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                         _ptr(initial_state), _ptr(final), _ptr(o), B, T, H, HV,
                                         K, V, float(scale), int(segments), _DTYPE[dt], _ptr(ws),
                                         ws_bytes, _flags(qk_l2norm, beta_sigmoid),
                                         ctypes.c_void_p(stream))
    _check(rc)
    return o, final


def kda_chunk_fwd_noalloc(q, k, v, g, beta, o, final_state=None, scale=None, initial_state=None,
                          chunk_size=64, qk_l2norm=False, beta_sigmoid=False):
    """kda_chunk_fwd writing into the caller's o [B,T,HV,V] (and final_state [B,HV,K,V]
    float32, or None), with no device allocation: the library's fixed per-device scratch
    array serves as the workspace (calls overlapping on one GPU race on it). Raises on
    KDA_ERR_SCRATCH when the shape needs more than NOALLOC_SCRATCH_BYTES. Returns o."""
    _require(q.is_cuda, "inputs must be on a GPU")
    dev, dt = q.device, q.dtype
    _require(dt in _DTYPE, f"unsupported dtype {dt}")
    B, T, H, K = q.shape
    HV, V = v.shape[2], v.shape[3]
    _require(k.shape == q.shape, "k must match q")
    _require(tuple(v.shape[:2]) == (B, T), "v must be [B, T, HV, V]")
    _require(tuple(g.shape) == (B, T, HV, K), "g must be [B, T, HV, K]")
    _require(tuple(beta.shape) == (B, T, HV), "beta must be [B, T, HV]")
    _require(tuple(o.shape) == (B, T, HV, V), "o must be [B, T, HV, V]")
    _check_tensors([("q", q), ("k", k), ("v", v), ("g", g), ("beta", beta), ("o", o)], dt, dev)
    for name, st in (("initial_state", initial_state), ("final_state", final_state)):
        if st is not None:
            _require(tuple(st.shape) == (B, HV, K, V), f"{name} must be [B, HV, K, V]")
            _check_tensors([(name, st)], torch.float32, dev)
    if scale is None:
        scale = 1.0 / math.sqrt(K)
    lib = library()
    with torch.cuda.device(dev):
        stream = torch.cuda.current_stream(dev).cuda_stream
        rc = lib.kda_chunk_fwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                       _ptr(initial_state), _ptr(final_state), _ptr(o), B, T, H,
                                       HV, K, V, float(scale), int(chunk_size), _DTYPE[dt],
                                       _flags(qk_l2norm, beta_sigmoid), ctypes.c_void_p(stream))
    _check(rc)
    return o


# The entry points below are called once per layer and token, so their checks are written for few
# Python operations. Timed on a CPU: kda_ssm_step's take 5.5 us on contiguous inputs (or of one
# request), 12 us where x, b and c of several requests are slices, whose strides are walked one by one.

def _call(index, fn, *args):
    """fn(*args, stream) on the current stream of GPU `index`, with that GPU current."""
    stream = torch._C._cuda_getCurrentRawStream(index)
    if torch.cuda.current_device() == index:
        rc = fn(*args, stream)
    else:
        with torch.cuda.device(index):
            rc = fn(*args, stream)
    if rc != KDA_OK:
        _check(rc)


def _addr(t):
    return None if t is None else t.data_ptr()


def _require_ints(what, *sizes):
    """Sizes that the C ABI takes as ints (ctypes would pass on their low 32 bits)."""
    _require(max(sizes) < 1 << 31, f"{what} must be fewer than 2^31")


def _fresh(t):
    """An uninitialised contiguous tensor shaped and typed like t."""
    return torch.empty_like(t, memory_format=torch.contiguous_format)


def _dense(name, t, shape, dtype, index):
    """t (or None) must be a contiguous tensor of this shape and dtype on GPU `index`."""
    if t is not None and (t.dtype is not dtype or t.shape != shape or t.get_device() != index
                          or not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor {list(shape)} on the GPU of x")


def _token_stride(name, t, lead, width):
    """Elements between the tokens of t, whose first `lead` dimensions are tokens in order (one, or
    batch and token) and whose others, `width` elements, are dense: t may be a slice of a wider
    activation."""
    if t.is_contiguous():
        return width
    expect = 1
    for size, stride in zip(reversed(t.shape[lead:]), reversed(t.stride()[lead:])):
        _require(size == 1 or stride == expect, f"{name} must be dense in its last dimensions")
        expect *= size
    step = None
    for size, stride in zip(reversed(t.shape[:lead]), reversed(t.stride()[:lead])):
        if size > 1:
            _require(step is None or stride == step * tokens, f"{name} must hold its tokens at one stride")
            step, tokens = (stride, size) if step is None else (step, tokens * size)
    _require(step is None or step >= width, f"{name} must not overlap itself")
    return width if step is None else step


def _tokens(name, t, shape, like, index, lead, width):
    """The token stride of t, a tensor of this shape, typed like x and on its GPU."""
    if t.dtype is not like.dtype or t.shape != shape or t.get_device() != index:
        raise ValueError(f"{name} must be {list(shape)}, of the dtype and on the GPU of x")
    return _token_stride(name, t, lead, width)


def _sequences(x, cu_seqlens, dims, index):
    """(token dimensions, sequences, tokens) of x: a dense batch [B, T, ...] of `dims` dimensions
    or, with cu_seqlens, packed tokens [T, ...] or [1, T, ...]."""
    if cu_seqlens is None:
        _require(x.dim() == dims, "x must be a batch [B, T, ...] (packed sequences: give cu_seqlens)")
        N, T = x.shape[0], x.shape[0] * x.shape[1]
        _require(N >= 1 and T < 1 << 31, "x must have at least one sequence and fewer than 2^31 tokens")
        _require_ints("sequences", N)
        return 2, N, T
    _require(cu_seqlens.get_device() == index and cu_seqlens.dtype is torch.int32
             and cu_seqlens.dim() == 1 and cu_seqlens.is_contiguous() and cu_seqlens.numel() >= 2,
             "cu_seqlens must be a contiguous int32 vector of at least two offsets on the GPU of x")
    lead = x.dim() - dims + 2
    _require(lead == 1 or (lead == 2 and x.shape[0] == 1), "packed x must be [T, ...] or [1, T, ...]")
    T = x.shape[lead - 1]
    _require(T < 1 << 31, "x must have fewer than 2^31 tokens")
    _require_ints("sequences", cu_seqlens.numel() - 1)
    return lead, cu_seqlens.numel() - 1, T


def _gpu(x):
    """(GPU index, the library's dtype) of x."""
    index, code = x.get_device(), _DTYPE.get(x.dtype)
    _require(index >= 0, "inputs must be on a GPU")
    if code is None:
        raise ValueError(f"unsupported dtype {x.dtype}")
    return index, code


def _conv_flags(silu):
    return (KDA_CONV_SILU if silu else 0) | KDA_ZERO_REST


def _conv_params(x, weight, bias, index):
    _require(weight.dim() == 2, "weight must be [D, W]")
    W, D = weight.shape[1], x.shape[-1]
    _require(D >= 1, "x must have at least one channel")
    _dense("weight", weight, (D, W), torch.float32, index)
    _dense("bias", bias, (D,), torch.float32, index)
    return D, W


def kda_conv_fwd(x, weight, bias=None, initial_state=None, cu_seqlens=None, silu=True,
                 output_final_state=True):
    """Short causal depthwise convolution of each sequence, then SiLU (unless silu=False):
    y_t[d] = silu(bias[d] + sum_w weight[d, w] x_{t-(W-1)+w}[d]). x [B,T,D], or packed [T,D] /
    [1,T,D] with cu_seqlens int32 [N+1] (float32 or bf16; its rows may lie in a wider
    activation); weight [D,W] (W = 2..4) and bias [D] float32; initial_state [N,W-1,D] like x:
    the rows before each sequence (None: zeros). Returns (y shaped like x, final_state
    [N,W-1,D] or None); y rows in no packed sequence are zero."""
    index, code = _gpu(x)
    lead, N, T = _sequences(x, cu_seqlens, 3, index)
    D, W = _conv_params(x, weight, bias, index)
    _dense("initial_state", initial_state, (N, W - 1, D), x.dtype, index)
    ldx = _token_stride("x", x, lead, D)
    y = _fresh(x)
    final = x.new_empty((N, W - 1, D)) if output_final_state else None
    _call(index, library().kda_conv_fwd, x.data_ptr(), ldx, weight.data_ptr(), _addr(bias),
          _addr(initial_state), _addr(cu_seqlens), N, _addr(final), y.data_ptr(), T, D, W,
          _conv_flags(silu), code)
    return y, final


def kda_conv_bwd(x, weight, dy, bias=None, initial_state=None, dfinal_state=None, cu_seqlens=None,
                 silu=True):
    """Gradients of <y, dy> + <final_state, dfinal_state> for kda_conv_fwd's inputs. dy like y;
    dfinal_state [N,W-1,D] like x or None. Returns (dx like x, dweight [D,W] and dbias [D]
    float32, dinitial_state [N,W-1,D]); the last two are None where bias / initial_state is, and
    dx rows in no packed sequence are zero."""
    index, code = _gpu(x)
    lead, N, T = _sequences(x, cu_seqlens, 3, index)
    D, W = _conv_params(x, weight, bias, index)
    _dense("initial_state", initial_state, (N, W - 1, D), x.dtype, index)
    _dense("dfinal_state", dfinal_state, (N, W - 1, D), x.dtype, index)
    ldx = _token_stride("x", x, lead, D)
    lddy = _tokens("dy", dy, x.shape, x, index, lead, D)
    lib = library()
    dx = _fresh(x)
    dweight = torch.empty_like(weight)
    dbias = None if bias is None else torch.empty_like(bias)
    dinit = None if initial_state is None else torch.empty_like(initial_state)
    ws_bytes = lib.kda_conv_bwd_workspace_size(T, D, W, code)
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=x.device) if ws_bytes else None
    _call(index, lib.kda_conv_bwd, x.data_ptr(), ldx, weight.data_ptr(), _addr(bias),
          _addr(initial_state), _addr(cu_seqlens), N, dy.data_ptr(), lddy, _addr(dfinal_state),
          dx.data_ptr(), dweight.data_ptr(), _addr(dbias), _addr(dinit), T, D, W, _conv_flags(silu),
          code, _addr(ws), ws_bytes)
    return dx, dweight, dbias, dinit


def _slots(slots, B, num_slots, index):
    _require_ints("requests and slots", B, num_slots)
    if slots is None:
        _require(num_slots >= B, "without slots the pool needs a state per request")
        return None
    if (slots.dtype is not torch.int32 or slots.shape != (B,) or slots.get_device() != index
            or not slots.is_contiguous()):
        raise ValueError("slots must be int32 [B] on the GPU of x")
    return slots.data_ptr()


def kda_conv_step(x, weight, state_pool, bias=None, slots=None, silu=True):
    """One token of kda_conv_fwd per request. x [B,D]; state_pool [num_slots,W-1,D] like x, moved
    on by one row in place; slots int32 [B] (a slot outside [0, num_slots) gives y = 0 and no
    update), or None: request n uses slot n. Returns y [B,D]."""
    index, code = _gpu(x)
    _require(x.dim() == 2 and x.numel() > 0 and state_pool.dim() == 3,
             "x must be [B, D], state_pool [num_slots, W-1, D]")
    D, W = _conv_params(x, weight, bias, index)
    B, num_slots = x.shape[0], state_pool.shape[0]
    _dense("state_pool", state_pool, (num_slots, W - 1, D), x.dtype, index)
    at = _slots(slots, B, num_slots, index)
    ldx = _token_stride("x", x, 1, D)
    y = _fresh(x)
    _call(index, library().kda_conv_step, x.data_ptr(), ldx, weight.data_ptr(), _addr(bias),
          state_pool.data_ptr(), at, num_slots, y.data_ptr(), B, D, W, _conv_flags(silu), code)
    return y


def _ssm_args(x, dt, A_log, b, c, D, dt_bias, lead, index):
    """Checks what the scan's entry points share. Returns (H, HV, K, V, token strides of x, dt, b, c)."""
    tokens, (HV, V) = x.shape[:lead], x.shape[lead:]
    _require(b.dim() == lead + 2, "b must be [tokens, H, K]")
    H, K = b.shape[lead:]
    ldx = _token_stride("x", x, lead, HV * V)
    lddt = _tokens("dt", dt, tokens + (HV,), x, index, lead, HV)
    ldb = _tokens("b", b, tokens + (H, K), x, index, lead, H * K)
    ldc = _tokens("c", c, tokens + (H, K), x, index, lead, H * K)
    _dense("A_log", A_log, (HV,), torch.float32, index)
    _dense("D", D, (HV,), torch.float32, index)
    _dense("dt_bias", dt_bias, (HV,), torch.float32, index)
    return H, HV, K, V, ldx, lddt, ldb, ldc


def kda_ssm_chunk_fwd(x, dt, A_log, b, c, D=None, dt_bias=None, initial_state=None, cu_seqlens=None,
                      output_final_state=True):
    """Selective state space scan with a scalar decay per head: with D_t = softplus(dt_t + dt_bias),
    S_t = exp(-exp(A_log) D_t) S_{t-1} + b_t (D_t x_t)^T, y_t = S_t^T c_t + D x_t. x [B,T,HV,V], dt
    [B,T,HV], b, c [B,T,H,K] (float32 or bf16; slices of a wider activation allowed; value head hv
    reads pair hv // (HV // H)), or packed without B (or with B = 1) and cu_seqlens int32 [N+1];
    A_log, D, dt_bias [HV] float32; initial_state [N,HV,K,V] float32. Returns (y shaped like x,
    final_state [N,HV,K,V] or None); y rows in no packed sequence are zero."""
    index, code = _gpu(x)
    lead, N, T = _sequences(x, cu_seqlens, 4, index)
    H, HV, K, V, ldx, lddt, ldb, ldc = _ssm_args(x, dt, A_log, b, c, D, dt_bias, lead, index)
    _dense("initial_state", initial_state, (N, HV, K, V), torch.float32, index)
    lib = library()
    y = _fresh(x)
    final = torch.empty((N, HV, K, V), dtype=torch.float32, device=x.device) if output_final_state else None
    ws_bytes = lib.kda_ssm_chunk_fwd_workspace_size(N, T, 0 if cu_seqlens is None else 1, H, HV, K, V, code)
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=x.device) if ws_bytes else None
    _call(index, lib.kda_ssm_chunk_fwd, x.data_ptr(), ldx, dt.data_ptr(), lddt, A_log.data_ptr(),
          b.data_ptr(), ldb, c.data_ptr(), ldc, _addr(D), _addr(dt_bias), _addr(initial_state),
          _addr(cu_seqlens), N, _addr(final), y.data_ptr(), T, H, HV, K, V, KDA_ZERO_REST, code,
          _addr(ws), ws_bytes)
    return y, final


def kda_ssm_step(x, dt, A_log, b, c, state_pool, D=None, dt_bias=None, slots=None):
    """One token of kda_ssm_chunk_fwd per request. x [B,HV,V], dt [B,HV], b, c [B,H,K]; state_pool
    [num_slots,HV,K,V] float32, updated in place; slots int32 [B] (a slot outside [0, num_slots)
    gives y = 0 and no update), or None: request n uses slot n. Returns y [B,HV,V]."""
    index, code = _gpu(x)
    _require(x.dim() == 3 and x.numel() > 0, "x must be [B, HV, V]")
    H, HV, K, V, ldx, lddt, ldb, ldc = _ssm_args(x, dt, A_log, b, c, D, dt_bias, 1, index)
    B, num_slots = x.shape[0], state_pool.shape[0] if state_pool.dim() == 4 else 0
    _dense("state_pool", state_pool, (num_slots, HV, K, V), torch.float32, index)
    at = _slots(slots, B, num_slots, index)
    y = _fresh(x)
    _call(index, library().kda_ssm_step, x.data_ptr(), ldx, dt.data_ptr(), lddt, A_log.data_ptr(),
          b.data_ptr(), ldb, c.data_ptr(), ldc, _addr(D), _addr(dt_bias), state_pool.data_ptr(), at,
          num_slots, y.data_ptr(), B, H, HV, K, V, code)
    return y


def _pools(pools):
    """(GPU index, host arrays of addresses and slot sizes, count, num_slots) of one pool or several."""
    pools = [pools] if isinstance(pools, torch.Tensor) else pools
    n = len(pools)
    _require(n > 0, "at least one pool is needed")
    index, num_slots = pools[0].get_device(), pools[0].shape[0] if pools[0].dim() else 0
    _require_ints("slots", num_slots)
    _require(index >= 0, "pools must be on a GPU")
    base, size = [], []
    for p in pools:
        if p.dim() < 1 or p.shape[0] != num_slots or p.get_device() != index or not p.is_contiguous():
            raise ValueError("pools must be contiguous [num_slots, ...], with one num_slots, on one GPU")
        base.append(p.data_ptr())
        size.append(p.nbytes)
    _require(min(size) > 0, "pools must hold at least one byte a slot")
    if n > 1:
        order = sorted(zip(base, size))
        _require(all(a[0] + a[1] <= b[0] for a, b in zip(order, order[1:])), "pools must not overlap")
    return (index, (ctypes.c_void_p * n)(*base), (ctypes.c_size_t * n)(*[v // num_slots for v in size]), n,
            num_slots)


def kda_slots_copy(pools, src, dst):
    """Copies slots within every pool, in place: pair by pair, in order, slot dst[i] becomes slot
    src[i] (a fork), or zeros where src[i] < 0 (a cleared slot). pools: a tensor [num_slots, ...]
    or a list of them (a model's layers; any dtype); src, dst int32 [n] on the GPU; pairs with dst
    outside [0, num_slots) or src >= num_slots do nothing."""
    index, base, size, n, num_slots = _pools(pools)
    _require(src.dim() == 1, "src must be int32 [n] on the pools' GPU")
    for name, t in (("src", src), ("dst", dst)):
        if (t.dtype is not torch.int32 or t.shape != src.shape or t.get_device() != index
                or not t.is_contiguous()):
            raise ValueError(f"{name} must be int32 [n] on the pools' GPU")
    _call(index, library().kda_slots_copy, base, size, n, num_slots, src.data_ptr(), dst.data_ptr(),
          src.shape[0])


def kda_slots_compact(pools, live):
    """Moves the live slots of every pool to its front, in place: with c live slots, those at or
    behind slot c move, in order, into the free slots in front of it. pools: as kda_slots_copy;
    live: bool (or uint8) [num_slots] on the GPU. Returns (new_slot int32 [num_slots]: where a
    slot's state lives now, -1 for a free one; count int32 [1])."""
    index, base, size, n, num_slots = _pools(pools)
    if (live.dtype not in (torch.bool, torch.uint8) or live.shape != (num_slots,)
            or live.get_device() != index or not live.is_contiguous()):
        raise ValueError("live must be bool [num_slots] on the pools' GPU")
    lib = library()
    ws_bytes = lib.kda_slots_compact_workspace_size(num_slots)
    # the results and the workspace share one allocation; the workspace comes first (256-byte aligned)
    buf = torch.empty((ws_bytes // 4 + num_slots + 1,), dtype=torch.int32, device=live.device)
    new_slot, count = buf[ws_bytes // 4:-1], buf[-1:]
    _call(index, lib.kda_slots_compact, base, size, n, num_slots, live.data_ptr(),
          new_slot.data_ptr(), count.data_ptr(), buf.data_ptr(), ws_bytes)
    return new_slot, count


def _checkpoint(name, t, shape, index):
    """(codes, scales) must be a checkpoint, as kda_checkpoint_pack gives it, of a tensor of this shape."""
    codes, scales = t
    _require(shape[-1] % 32 == 0, f"{name}: checkpoints have a multiple of 32 channels")
    if codes.dtype is not torch.float8_e4m3fn or codes.shape != shape or codes.get_device() != index or not codes.is_contiguous():
        raise ValueError(f"{name}: codes must be a contiguous float8_e4m3fn tensor {list(shape)} on the GPU of the gradients")
    if (scales.dtype is not torch.uint8 or scales.shape != shape[:-1] + (shape[-1] // 32,)
            or scales.get_device() != index or not scales.is_contiguous()):
        raise ValueError(f"{name}: scales must be a contiguous uint8 tensor {list(shape[:-1])} + [channels / 32]")
    return codes.data_ptr(), scales.data_ptr()


def _row_layout(like, named):
    """(tokens, rows a token, {name: elements between tokens}) of the tensors (or None) in `named`,
    each shaped and typed like `like` and on its GPU: rows are their last dimension, and a tensor may
    be a slice of a wider activation, of whole rows or of the rows of a token."""
    shape, dtype, index = like.shape, like.dtype, like.get_device()
    given = [(n, t) for n, t in named if t is not None]
    dense = True
    for n, t in given:
        if t.dtype is not dtype or t.shape != shape or t.get_device() != index:
            raise ValueError(f"{n} must be {list(shape)}, {dtype}, on the GPU of the others")
        dense = dense and t.is_contiguous()
    D = shape[-1]
    rows = like.numel() // D if D else 0
    if dense:
        return rows, 1, {n: D for n, _ in given}
    lead = len(shape) - 1
    try:
        return rows, 1, {n: _token_stride(n, t, lead, D) for n, t in given}
    except ValueError:
        if lead < 2:
            raise
        G = shape[-2]
        _require_ints("rows of a token", G)
        return rows // G, G, {n: _token_stride(n, t, lead - 1, G * D) for n, t in given}


def _norm_args(x, weight, scale):
    index, code = _gpu(x)
    _require(x.dim() >= 1 and x.shape[-1] >= 1, "x must have at least one column")
    D = x.shape[-1]
    _require_ints("columns", D)
    _dense("weight", weight, (D,), torch.float32, index)
    _dense("scale", scale, (D,), torch.float32, index)
    return index, code, D


def kda_prenorm_fwd(x, weight, residual=None, scale=None, eps=1e-6):
    """The norm in front of a block, joined with the residual addition behind the block before it:
    h = residual + scale * x, y = weight * h / sqrt(mean(h^2) + eps) over the last dimension. x
    [..., D] (float32 or bf16; slices of a wider activation allowed); weight [D] float32; residual
    like x, or None: zeros; scale [D] float32, or None: ones. Returns (y, h), shaped and typed like
    x; h is x itself where neither residual nor scale is given."""
    index, code, D = _norm_args(x, weight, scale)
    T, G, ld = _row_layout(x, (("x", x), ("residual", residual)))
    y = _fresh(x)
    h = None if residual is None and scale is None else _fresh(x)
    _call(index, library().kda_prenorm_fwd, x.data_ptr(), ld["x"], _addr(residual), ld.get("residual", 0),
          weight.data_ptr(), _addr(scale), y.data_ptr(), _addr(h), T, G, D, eps, code)
    return y, x if h is None else h


def kda_postnorm_fwd(x, weight, gate=None, residual=None, scale=None, activation="sigmoid", eps=1e-6):
    """The norm behind a block, under its gate and into the residual:
    y = residual + scale * (weight * act(gate) * x / sqrt(mean(x^2) + eps)) over the last dimension,
    act the sigmoid or "silu". x, gate and residual [..., D] (gate None: no factor; residual None:
    zeros); weight, scale [D] float32 (scale None: ones). Returns y like x."""
    index, code, D = _norm_args(x, weight, scale)
    _require(activation in ("sigmoid", "silu"), "activation must be 'sigmoid' or 'silu'")
    T, G, ld = _row_layout(x, (("x", x), ("gate", gate), ("residual", residual)))
    y = _fresh(x)
    _call(index, library().kda_postnorm_fwd, x.data_ptr(), ld["x"], weight.data_ptr(), _addr(gate), ld.get("gate", 0),
          _addr(residual), ld.get("residual", 0), _addr(scale), y.data_ptr(), T, G, D, eps,
          KDA_NORM_SILU if activation == "silu" else 0, code)
    return y


def _kept(name, t, like, index):
    """(address, scales' address) of a checkpoint, or (None, None): the tensor itself is meant."""
    return _checkpoint(name, t, like.shape, index) if isinstance(t, (tuple, list)) else (None, None)


def _norm_sums(T, G, D, weight, scale):
    """Outputs and workspace of the sums over rows."""
    n = library().kda_norm_bwd_workspace_size(T, G, D)
    ws = torch.empty(n, dtype=torch.uint8, device=weight.device) if n else None
    return torch.empty_like(weight), None if scale is None else torch.empty_like(scale), ws, n


def kda_prenorm_bwd(h, weight, dy, dh=None, x=None, scale=None, eps=1e-6):
    """Gradients of <y, dy> + <h, dh> for kda_prenorm_fwd's inputs. h: as it returned it; x, needed
    where scale is given: its input; both may be checkpoints (codes, scales). dh None: zeros. Returns
    (dresidual, dx, dweight [D], dscale [D]); dx is dresidual, and dscale None, without a scale."""
    index, code, D = _norm_args(dy, weight, scale)
    _require(scale is None or x is not None, "a scale's gradient needs x")
    x = None if scale is None else x
    (hp, hs), (xp, xs) = _kept("h", h, dy, index), _kept("x", x, dy, index)
    _require(x is None or (hs is None) == (xs is None), "h and x must both be checkpoints, or neither")
    T, G, ld = _row_layout(dy, (("dy", dy), ("dh", dh), ("h", h if hs is None else None),
                                ("x", x if xs is None else None)))
    dweight, dscale, ws, n = _norm_sums(T, G, D, weight, scale)
    dres = _fresh(dy)
    dx = dres if scale is None else _fresh(dy)
    _call(index, library().kda_prenorm_bwd, hp if hs is not None else h.data_ptr(), hs, ld.get("h", 0),
          weight.data_ptr(), dy.data_ptr(), ld["dy"], _addr(dh), ld.get("dh", 0), xp if xs is not None else _addr(x), xs,
          ld.get("x", 0), _addr(scale), dres.data_ptr(), dx.data_ptr(), dweight.data_ptr(), _addr(dscale), T, G, D,
          eps, code, _addr(ws), n)
    return dres, dx, dweight, dscale


def kda_postnorm_bwd(x, weight, dy, gate=None, scale=None, activation="sigmoid", eps=1e-6):
    """Gradients of <y, dy> for kda_postnorm_fwd's inputs (the residual's is dy as it is). x and gate
    may be checkpoints (codes, scales). Returns (dx, dgate, dweight [D], dscale [D]); dgate and dscale
    are None where gate and scale are."""
    index, code, D = _norm_args(dy, weight, scale)
    _require(activation in ("sigmoid", "silu"), "activation must be 'sigmoid' or 'silu'")
    (xp, xs), (gp, gs) = _kept("x", x, dy, index), _kept("gate", gate, dy, index)
    _require(gate is None or (xs is None) == (gs is None), "x and gate must both be checkpoints, or neither")
    T, G, ld = _row_layout(dy, (("dy", dy), ("x", x if xs is None else None),
                                ("gate", gate if gs is None else None)))
    dweight, dscale, ws, n = _norm_sums(T, G, D, weight, scale)
    dx = _fresh(dy)
    dgate = None if gate is None else _fresh(dy)
    _call(index, library().kda_postnorm_bwd, xp if xs is not None else x.data_ptr(), xs, ld.get("x", 0),
          weight.data_ptr(), gp if gs is not None else _addr(gate), gs, ld.get("gate", 0), dy.data_ptr(), ld["dy"],
          _addr(scale), dx.data_ptr(), _addr(dgate), dweight.data_ptr(), _addr(dscale), T, G, D, eps,
          KDA_NORM_SILU if activation == "silu" else 0, code, _addr(ws), n)
    return dx, dgate, dweight, dscale


def kda_checkpoint_pack(x):
    """x [..., D] (float32 or bf16, D a multiple of 32; a slice of a wider activation allowed) in 8
    bits: (codes float8_e4m3fn [..., D], scales uint8 [..., D / 32]). 32 neighbours share the power of
    two 2^(scale - 127), the smallest that brings the largest finite magnitude to 448 at most."""
    index, code = _gpu(x)
    _require(x.dim() >= 1 and x.shape[-1] % 32 == 0 and x.shape[-1] > 0, "x must have a multiple of 32 channels")
    T, G, ld = _row_layout(x, (("x", x),))
    _require_ints("channels of a token", G * x.shape[-1])
    codes = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=x.device)
    scales = torch.empty(x.shape[:-1] + (x.shape[-1] // 32,), dtype=torch.uint8, device=x.device)
    _call(index, library().kda_checkpoint_pack, x.data_ptr(), ld["x"], codes.data_ptr(), scales.data_ptr(), T,
          G * x.shape[-1], code)
    return codes, scales


def kda_checkpoint_unpack(codes, scales, dtype=torch.bfloat16):
    """The values that a checkpoint of kda_checkpoint_pack stands for, as float32 or bf16 [..., D]."""
    index = codes.get_device()
    _require(index >= 0, "inputs must be on a GPU")
    _require(codes.dim() >= 1 and codes.shape[-1] > 0, "codes must have at least one channel")
    _require_ints("channels", codes.shape[-1])
    _require(dtype in _DTYPE, f"unsupported dtype {dtype}")
    _checkpoint("checkpoint", (codes, scales), codes.shape, index)
    x = torch.empty(codes.shape, dtype=dtype, device=codes.device)
    D = codes.shape[-1]
    _call(index, library().kda_checkpoint_unpack, codes.data_ptr(), scales.data_ptr(), x.data_ptr(),
          codes.numel() // D, D, _DTYPE[dtype])
    return x


def _glr_params(D, A_log, dt_bias, index):
    _require(D >= 1, "x must have at least one channel")
    _require_ints("channels", D)
    _dense("A_log", A_log, (D,), torch.float32, index)
    _dense("dt_bias", dt_bias, (D,), torch.float32, index)


def kda_glr_fwd(x, gate_x, A_log, dt_bias=None, in_gate=None, initial_state=None, cu_seqlens=None, normalise=True,
                output_final_state=True, output_block_states=False):
    """Gated linear recurrence with one state per channel: with a_t = exp(-exp(A_log) softplus(gate_x_t
    + dt_bias)), h_t = a_t h_{t-1} + w_t sigmoid(in_gate_t) x_t and y_t = h_t, where w_t is
    sqrt(1 - a_t^2), or 1 with normalise=False. x, gate_x, in_gate [B,T,D] (float32 or bf16; slices of a
    wider activation allowed; in_gate None: factor 1), or packed [T,D] / [1,T,D] with cu_seqlens int32
    [N+1]; A_log, dt_bias [D] float32; initial_state [N,D] float32. Returns (y like x, final_state [N,D]
    float32 or None); y rows in no packed sequence are zero. output_block_states: also returns the states
    [ceil(tokens / 64), D] that kda_glr_bwd takes, so that it need not compute them again. The decay is the
    library's gate, not exp(-c softplus(L) sigmoid(r)) of the published layers with this weight."""
    index, code = _gpu(x)
    lead, N, T = _sequences(x, cu_seqlens, 3, index)
    D = x.shape[-1]
    _glr_params(D, A_log, dt_bias, index)
    ldx = _token_stride("x", x, lead, D)
    ldr = _tokens("gate_x", gate_x, x.shape, x, index, lead, D)
    ldi = 0 if in_gate is None else _tokens("in_gate", in_gate, x.shape, x, index, lead, D)
    _dense("initial_state", initial_state, (N, D), torch.float32, index)
    lib = library()
    y = _fresh(x)
    final = torch.empty((N, D), dtype=torch.float32, device=x.device) if output_final_state else None
    states = (torch.empty(((T + GLR_BLOCK - 1) // GLR_BLOCK, D), dtype=torch.float32, device=x.device)
              if output_block_states else None)
    n = lib.kda_glr_fwd_workspace_size(T, D)
    ws = torch.empty(n, dtype=torch.uint8, device=x.device) if n else None
    _call(index, lib.kda_glr_fwd, x.data_ptr(), ldx, gate_x.data_ptr(), ldr, A_log.data_ptr(), _addr(dt_bias),
          _addr(in_gate), ldi, _addr(initial_state), _addr(cu_seqlens), N, _addr(final), y.data_ptr(), _addr(states), T, D,
          KDA_ZERO_REST | (KDA_GLR_NORMALISE if normalise else 0), code, _addr(ws), n)
    return (y, final, states) if output_block_states else (y, final)


def kda_glr_bwd(x, gate_x, A_log, dy, dt_bias=None, in_gate=None, initial_state=None, dfinal_state=None,
                cu_seqlens=None, normalise=True, block_states=None):
    """Gradients of <y, dy> + <final_state, dfinal_state> for kda_glr_fwd's inputs. x, gate_x and in_gate
    may be checkpoints (codes, scales), all of them or none. block_states: as kda_glr_fwd returned them for
    these inputs, or None: they are computed again. Beside checkpoints leave them None, or give those of a
    forward pass over kda_checkpoint_unpack's values: with the states of the inputs before they were packed the
    gradients would belong to neither. Returns (dx, dgate_x, din_gate, dA_log [D], ddt_bias
    [D], dinitial_state [N,D]); din_gate, ddt_bias and dinitial_state are None where their inputs are, and
    rows in no packed sequence are zero."""
    index, code = _gpu(dy)
    lead, N, T = _sequences(dy, cu_seqlens, 3, index)
    D = dy.shape[-1]
    _glr_params(D, A_log, dt_bias, index)
    args, packed = [], []
    for name, t in (("x", x), ("gate_x", gate_x), ("in_gate", in_gate)):
        if t is None:
            args.append((None, None, 0))
        elif isinstance(t, (tuple, list)):
            args.append(_checkpoint(name, t, dy.shape, index) + (D,))
            packed.append(True)
        else:
            args.append((t.data_ptr(), None, _tokens(name, t, dy.shape, dy, index, lead, D)))
            packed.append(False)
    _require(len(set(packed)) == 1, "x, gate_x and in_gate must all be checkpoints, or none of them")
    lddy = _token_stride("dy", dy, lead, D)
    _dense("initial_state", initial_state, (N, D), torch.float32, index)
    _dense("dfinal_state", dfinal_state, (N, D), torch.float32, index)
    _dense("block_states", block_states, ((T + GLR_BLOCK - 1) // GLR_BLOCK, D), torch.float32, index)
    lib = library()
    dx, dr = _fresh(dy), _fresh(dy)
    din = None if in_gate is None else _fresh(dy)
    dA = torch.empty_like(A_log)
    db = None if dt_bias is None else torch.empty_like(dt_bias)
    dinit = None if initial_state is None else torch.empty_like(initial_state)
    n = lib.kda_glr_bwd_workspace_size(T, D, 0 if block_states is None else 1)
    ws = torch.empty(n, dtype=torch.uint8, device=dy.device) if n else None
    _call(index, lib.kda_glr_bwd, *args[0], *args[1], A_log.data_ptr(), _addr(dt_bias), *args[2], _addr(initial_state),
          _addr(cu_seqlens), N, dy.data_ptr(), lddy, _addr(dfinal_state), _addr(block_states), dx.data_ptr(),
          dr.data_ptr(), _addr(din), dA.data_ptr(), _addr(db), _addr(dinit), T, D,
          KDA_ZERO_REST | (KDA_GLR_NORMALISE if normalise else 0), code, _addr(ws), n)
    return dx, dr, din, dA, db, dinit


def kda_glr_step(x, gate_x, A_log, state_pool, dt_bias=None, in_gate=None, slots=None, normalise=True):
    """One token of kda_glr_fwd per request. x, gate_x, in_gate [B,D]; state_pool [num_slots,D] float32,
    updated in place; slots int32 [B] (a slot outside [0, num_slots) gives y = 0 and no update), or
    None: request n uses slot n. Returns y [B,D]."""
    index, code = _gpu(x)
    _require(x.dim() == 2 and x.numel() > 0 and state_pool.dim() == 2, "x must be [B, D], state_pool [num_slots, D]")
    B, D = x.shape
    _glr_params(D, A_log, dt_bias, index)
    ldx = _token_stride("x", x, 1, D)
    ldr = _tokens("gate_x", gate_x, x.shape, x, index, 1, D)
    ldi = 0 if in_gate is None else _tokens("in_gate", in_gate, x.shape, x, index, 1, D)
    num_slots = state_pool.shape[0]
    _dense("state_pool", state_pool, (num_slots, D), torch.float32, index)
    at = _slots(slots, B, num_slots, index)
    y = _fresh(x)
    _call(index, library().kda_glr_step, x.data_ptr(), ldx, gate_x.data_ptr(), ldr, A_log.data_ptr(), _addr(dt_bias),
          _addr(in_gate), ldi, state_pool.data_ptr(), at, num_slots, y.data_ptr(), B, D,
          KDA_GLR_NORMALISE if normalise else 0, code)
    return y


def stream_copy(src, dst):
    """kda_stream_copy: copy the bytes of contiguous device tensor src into dst (same byte
    size, 16-byte aligned, not overlapping) with the library's streaming copy kernel. A
    measuring stick for HBM figures, not part of the operator."""
    _require(src.is_cuda and dst.is_cuda, "tensors must be on a GPU")
    _require(src.is_contiguous() and dst.is_contiguous(), "tensors must be contiguous")
    nbytes = src.numel() * src.element_size()
    _require(dst.numel() * dst.element_size() == nbytes, "src and dst must have the same byte size")
    with torch.cuda.device(src.device):
        stream = torch.cuda.current_stream(src.device).cuda_stream
        _check(library().kda_stream_copy(_ptr(src), _ptr(dst), nbytes, ctypes.c_void_p(stream)))
