"""ctypes binding for libspecverify_ops: the operators around the verification.

``hidden_norm`` (the norms before an LM head with gate and residual scale),
``quantize_fp8``, ``pack_fp8_lm_head``, ``fp8_lm_head`` and
``verify_fp8_lm_head`` (an LM head on 8-bit floats, alone and with the
verification on its logits) and ``verify_probs`` (the verification from given
probabilities).  As in ``binding``, this module checks shapes and dtypes,
allocates outputs and workspaces with torch and passes raw device pointers and
the HIP stream through the C ABI declared in ``include/specverify_ops.h``.  If
the library is not built the calls raise: there is no fallback.

8-bit values are ``torch.float8_e4m3fn`` tensors [..., D] with a
``torch.float8_e8m0fnu`` scale [..., D / 128] for each run of 128.
"""

import ctypes
import functools
import os
import threading

import torch

from . import binding
from .binding import SPECV_EINVAL, SPECV_OK, SpecVerifyError, _check

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libspecverify_ops.so")

FP8_BLOCK = 128
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
_VALUE_CODES = {torch.float32: 0, torch.bfloat16: 1}
_OUT_CODES = {**_VALUE_CODES, E4M3: 2}
_ANY_DIMS = (1, 2, 3, 4)

_lib = None
_lock = threading.Lock()


def ops_library_path():
    return _LIB_PATH


def load_ops_library():
    """Load libspecverify_ops.so and declare its C signatures (once)."""
    global _lib
    if _lib is not None:
        return _lib
    binding.load_library()
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(
                f"{_LIB_PATH} is not built; run `python -m speculative_decoding_sampling_amd.build`")
        lib = ctypes.CDLL(_LIB_PATH)
        i, f, vp, size, i64 = (ctypes.c_int, ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t,
                               ctypes.c_int64)
        lib.specv_hidden_norm.argtypes = [vp, i, vp, i, vp, vp, i, vp, i, i, i, f, f, vp, vp, i, vp,
                                          vp]
        lib.specv_hidden_norm.restype = i
        lib.specv_fp8_quantize.argtypes = [vp, i, i, i, vp, vp, vp]
        lib.specv_fp8_quantize.restype = i
        lib.specv_fp8_lm_head_packed_weight_bytes.argtypes = [i, i]
        lib.specv_fp8_lm_head_packed_weight_bytes.restype = size
        lib.specv_fp8_lm_head_pack_weight.argtypes = [vp, vp, vp, i, i, vp]
        lib.specv_fp8_lm_head_pack_weight.restype = i
        lib.specv_fp8_lm_head.argtypes = [vp, vp, vp, i, i, i, vp, i, vp]
        lib.specv_fp8_lm_head.restype = i
        lib.specv_verify_fp8_lm_head_workspace_bytes.argtypes = [i, i, i, i, i, f]
        lib.specv_verify_fp8_lm_head_workspace_bytes.restype = size
        lib.specv_verify_fp8_lm_head.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, f,
                                                 i, vp, vp, vp, vp, size, vp, vp, vp, vp, vp]
        lib.specv_verify_fp8_lm_head.restype = i
        lib.specv_verify_probs_workspace_bytes.argtypes = [i, i, i]
        lib.specv_verify_probs_workspace_bytes.restype = size
        lib.specv_verify_probs.argtypes = [vp, i64, i64, vp, i64, i64, i, vp, vp, vp, vp, i, i, i, i,
                                           vp, vp, vp, size, vp, vp, vp, vp, vp]
        lib.specv_verify_probs.restype = i
        lib.specv_ops_version.argtypes = []
        lib.specv_ops_version.restype = i
        _lib = lib
        return lib


class _Call:
    """Device and stream of one call: allocations made for it are kept from
    reuse until the stream has run it, whichever stream is current."""

    __slots__ = ("dev", "stream", "other", "ptr")

    def __init__(self, dev, stream):
        self.dev = dev
        self.ptr = torch._C._cuda_getCurrentRawStream(dev.index)
        self.other = False
        if stream is not None:
            if stream.device != dev:
                raise ValueError(f"stream is on {stream.device}, the tensors on {dev}")
            self.other = stream.cuda_stream != self.ptr
            self.ptr = stream.cuda_stream
        self.stream = stream

    def empty(self, shape, dtype):
        t = torch.empty(shape, dtype=dtype, device=self.dev)
        if self.other:
            t.record_stream(self.stream)
        return t

    def zeros(self, nbytes):
        if not self.other:
            return torch.zeros(nbytes, dtype=torch.uint8, device=self.dev)
        with torch.cuda.stream(self.stream):
            t = torch.zeros(nbytes, dtype=torch.uint8, device=self.dev)
        t.record_stream(torch.cuda.current_stream(self.dev))
        return t

    def run(self, f, *args):
        """The library call ``f`` with the tensors' device current."""
        if self.dev.index == torch._C._cuda_getDevice():
            status = f(*args)
        else:
            with torch.cuda.device(self.dev):
                status = f(*args)
        if status != SPECV_OK:
            raise SpecVerifyError(status, binding.status_string(status))


def _ptr(t):
    return None if t is None else t.data_ptr() or None


def _match(t, name, dtype, shape, dev):
    """``binding._check`` with its answer for a tensor that passes first."""
    if isinstance(t, torch.Tensor) and t.dtype == dtype and t.shape == shape and \
            t.device == dev and t.is_contiguous():
        return
    _check(t, name, dtype, shape, dev)


def _gpu(t, name, dims):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda or t.dim() not in dims:
        raise ValueError(f"{name} must be a GPU tensor of {' or '.join(map(str, dims))} dimensions")


def _value_code(t, name):
    code = _VALUE_CODES.get(getattr(t, "dtype", None))
    if code is None:
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        raise TypeError(f"{name} must be bfloat16 or float32, got {t.dtype}")
    return code


def hidden_norm(x, residual, weight, *, post_weight=None, gate=None, scale=1.0, eps=1e-6,
                dtype=torch.bfloat16, residual_out=None, out=None, out_scale=None, stream=None):
    """The norms around the target's last block with its gate and residual
    scale: r' = residual + scale * gate * N(x; post_weight), y = N(r';
    weight), N(v; w) = w * v / sqrt(mean(v^2) + eps).

    ``x`` [..., D] is the block's output, ``residual`` (same shape) the stream
    before it, ``weight`` and ``post_weight`` [D], ``gate`` [D] or [G, D] with G
    dividing the rows (consecutive rows share a gate row); each bf16 or fp32,
    the weights and the gate of one dtype.  Without ``post_weight`` x is taken
    as it is, without ``gate`` the factor is one.  Returns (r', y), y of
    ``dtype`` (bf16, fp32), or (r', y, y's scale) for float8_e4m3fn, which
    needs D a multiple of 128.  ``residual_out`` may be ``residual``.
    Asynchronous on ``stream``."""
    lib = load_ops_library()
    _gpu(x, "x", _ANY_DIMS)
    dev, shape = x.device, x.shape
    D = shape[-1]
    M = x.numel() // D if D else 0
    xc, rc, wc = _value_code(x, "x"), _value_code(residual, "residual"), _value_code(weight, "weight")
    _match(x, "x", x.dtype, shape, dev)
    _match(residual, "residual", residual.dtype, shape, dev)
    _match(weight, "weight", weight.dtype, (D,), dev)
    if post_weight is not None:
        _match(post_weight, "post_weight", weight.dtype, (D,), dev)
    rows = 1
    if gate is not None:
        _gpu(gate, "gate", (1, 2))
        if gate.dim() == 2:
            rows = gate.shape[0]
            _match(gate, "gate", weight.dtype, (rows, D), dev)
            if rows < 1 or M % rows:
                raise ValueError(f"gate has {rows} rows, which do not divide the {M} rows of x")
        else:
            _match(gate, "gate", weight.dtype, (D,), dev)
    code = _OUT_CODES.get(dtype)
    if code is None:
        raise TypeError(f"dtype must be bfloat16, float32 or float8_e4m3fn, got {dtype}")
    call = _Call(dev, stream)
    if residual_out is None:
        residual_out = call.empty(shape, residual.dtype)
    else:
        _match(residual_out, "residual_out", residual.dtype, shape, dev)
    if dtype == E4M3:
        if D % FP8_BLOCK:
            raise ValueError(f"8-bit output needs D a multiple of {FP8_BLOCK}, got {D}")
        sshape = shape[:-1] + (D // FP8_BLOCK,)
        if out_scale is None:
            out_scale = call.empty(sshape, E8M0)
        else:
            _match(out_scale, "out_scale", E8M0, sshape, dev)
    elif out_scale is not None:
        raise ValueError("out_scale goes with 8-bit output only")
    if out is None:
        out = call.empty(shape, dtype)
    else:
        _match(out, "out", dtype, shape, dev)
    call.run(lib.specv_hidden_norm, x.data_ptr(), xc, residual.data_ptr(), rc, _ptr(post_weight),
             _ptr(gate), rows, weight.data_ptr(), wc, M, D, scale, eps, residual_out.data_ptr(),
             out.data_ptr(), code, _ptr(out_scale), call.ptr)
    return (residual_out, out, out_scale) if dtype == E4M3 else (residual_out, out)


def quantize_fp8(x, *, out=None, out_scale=None, stream=None):
    """8-bit values and scales of ``x`` [..., D] (bf16 or fp32, D a multiple
    of 128): q float8_e4m3fn [..., D] and scale float8_e8m0fnu [..., D / 128],
    x ~ q * scale with the smallest power of two that brings each run's
    largest magnitude to at most 448.  Asynchronous on ``stream``."""
    lib = load_ops_library()
    _gpu(x, "x", _ANY_DIMS)
    dev, shape = x.device, x.shape
    D = shape[-1]
    code = _value_code(x, "x")
    _match(x, "x", x.dtype, shape, dev)
    if D < 1 or D % FP8_BLOCK:
        raise ValueError(f"the last dimension must be a multiple of {FP8_BLOCK}, got {D}")
    call = _Call(dev, stream)
    sshape = shape[:-1] + (D // FP8_BLOCK,)
    if out is None:
        out = call.empty(shape, E4M3)
    else:
        _match(out, "out", E4M3, shape, dev)
    if out_scale is None:
        out_scale = call.empty(sshape, E8M0)
    else:
        _match(out_scale, "out_scale", E8M0, sshape, dev)
    call.run(lib.specv_fp8_quantize, x.data_ptr(), code, x.numel() // D, D, out.data_ptr(),
             out_scale.data_ptr(), call.ptr)
    return out, out_scale


class PackedFp8LmHead:
    """An 8-bit LM-head weight [V, D] in the layout the products read
    (``specv_fp8_lm_head_pack_weight``): ``data`` is the packed device buffer."""

    def __init__(self, data, V, D):
        self.data, self.V, self.D = data, int(V), int(D)


@functools.lru_cache(maxsize=None)
def fp8_lm_head_packed_weight_bytes(V, D):
    return int(load_ops_library().specv_fp8_lm_head_packed_weight_bytes(int(V), int(D)))


def pack_fp8_lm_head(weight, scale=None, *, stream=None):
    """Lay an LM-head weight out once for ``fp8_lm_head``: ``weight`` [V, D]
    float8_e4m3fn with ``scale`` [V, D / 128] float8_e8m0fnu, or bf16 / fp32
    without a scale (quantised here, see ``quantize_fp8``).  Asynchronous on
    ``stream``."""
    lib = load_ops_library()
    _gpu(weight, "weight", (2,))
    V, D = weight.shape
    dev = weight.device
    if scale is None:
        weight, scale = quantize_fp8(weight, stream=stream)
    _match(weight, "weight", E4M3, (V, D), dev)
    nbytes = fp8_lm_head_packed_weight_bytes(V, D)
    if nbytes == 0:
        raise SpecVerifyError(SPECV_EINVAL, f"unsupported LM-head shape V={V} D={D}")
    _match(scale, "scale", E8M0, (V, D // FP8_BLOCK), dev)
    call = _Call(dev, stream)
    data = call.empty((nbytes,), torch.uint8)
    call.run(lib.specv_fp8_lm_head_pack_weight, weight.data_ptr(), scale.data_ptr(),
             data.data_ptr(), V, D, call.ptr)
    return PackedFp8LmHead(data, V, D)


def _check_hidden(hidden, hidden_scale, packed, dims):
    _gpu(hidden, "hidden", dims)
    if not isinstance(packed, PackedFp8LmHead):
        raise TypeError("packed must be a PackedFp8LmHead")
    dev, shape = hidden.device, hidden.shape
    if shape[-1] != packed.D:
        raise ValueError(f"packed weight has D={packed.D}, hidden D={shape[-1]}")
    _match(hidden, "hidden", E4M3, shape, dev)
    _match(hidden_scale, "hidden_scale", E8M0, shape[:-1] + (packed.D // FP8_BLOCK,), dev)
    _match(packed.data, "packed", torch.uint8,
           (fp8_lm_head_packed_weight_bytes(packed.V, packed.D),), dev)
    return dev, shape


def fp8_lm_head(hidden, hidden_scale, packed, *, dtype=torch.bfloat16, logits=None, stream=None):
    """Logits [..., V] (``dtype`` bf16 or fp32) of hidden states [..., D]
    float8_e4m3fn with their scales (``hidden_norm`` or ``quantize_fp8``) and a
    ``PackedFp8LmHead``; float32 accumulation.  Asynchronous on ``stream``."""
    lib = load_ops_library()
    dev, shape = _check_hidden(hidden, hidden_scale, packed, _ANY_DIMS)
    code = _VALUE_CODES.get(dtype)
    if code is None:
        raise TypeError(f"dtype must be bfloat16 or float32, got {dtype}")
    call = _Call(dev, stream)
    oshape = shape[:-1] + (packed.V,)
    if logits is None:
        logits = call.empty(oshape, dtype)
    else:
        _match(logits, "logits", dtype, oshape, dev)
    call.run(lib.specv_fp8_lm_head, hidden.data_ptr(), hidden_scale.data_ptr(),
             packed.data.data_ptr(), hidden.numel() // packed.D, packed.D, packed.V,
             logits.data_ptr(), code, call.ptr)
    return logits


def _check_round(draft_tokens, draft_len, u, u_final, B, K, dev):
    _match(draft_tokens, "draft_tokens", torch.int32, (B, K), dev)
    _match(draft_len, "draft_len", torch.int32, (B,), dev)
    _match(u, "u", torch.float32, (B, K), dev)
    _match(u_final, "u_final", torch.float32, (B,), dev)


def _outputs(call, B, K, out_tokens, n_emitted, debug):
    """The result dict and the diagnostics' addresses."""
    if out_tokens is None:
        out_tokens = call.empty((B, K + 1), torch.int32)
    else:
        _match(out_tokens, "out_tokens", torch.int32, (B, K + 1), call.dev)
    if n_emitted is None:
        n_emitted = call.empty((B,), torch.int32)
    else:
        _match(n_emitted, "n_emitted", torch.int32, (B,), call.dev)
    res = {"out_tokens": out_tokens, "n_emitted": n_emitted}
    if not debug:
        return res, (None, None, None, None)
    diag = (call.empty((B, K), torch.float32), call.empty((B,), torch.float64),
            call.empty((B,), torch.int32), call.empty((B,), torch.int32))
    res.update(zip(("accept_prob", "residual_mass", "stop_pos", "path"), diag))
    return res, tuple(_ptr(t) for t in diag)


def _space(workspace, dev):
    if not isinstance(workspace, torch.Tensor) or workspace.device != dev or \
            not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {dev}")
    return _ptr(workspace), workspace.numel() * workspace.element_size()


def verify_fp8_lm_head(hidden, hidden_scale, packed, draft_logits, draft_tokens, draft_len, u,
                       u_final, temperature=1.0, eos_id=-1, *, top_k=0, top_p=1.0,
                       target_logits=None, out_tokens=None, n_emitted=None, workspace=None,
                       debug=False, stream=None):
    """The verification step on an 8-bit LM head: ``fp8_lm_head`` of hidden
    [B, K+1, D] gives the bf16 target logits [B, K+1, V], and the verification
    runs on them.  Other arguments and the returned dict as for
    ``binding.verify_lm_head``.  Asynchronous on ``stream``."""
    lib = load_ops_library()
    dev, (B, K1, D) = _check_hidden(hidden, hidden_scale, packed, (3,))
    K, V, bf = K1 - 1, packed.V, torch.bfloat16
    _match(draft_logits, "draft_logits", bf, (B, K, V), dev)
    _check_round(draft_tokens, draft_len, u, u_final, B, K, dev)
    call = _Call(dev, stream)
    if target_logits is None:
        target_logits = call.empty((B, K1, V), bf)
    else:
        _match(target_logits, "target_logits", bf, (B, K1, V), dev)
    res, diag = _outputs(call, B, K, out_tokens, n_emitted, debug)
    res["target_logits"] = target_logits
    if workspace is None:
        nbytes = int(lib.specv_verify_fp8_lm_head_workspace_bytes(B, K, V, D, int(top_k),
                                                                  float(top_p)))
        # Path 3 keeps a call counter in its workspace.  A captured call gets
        # memory that the rest of its graph may use between two replays: the
        # graph clears it before each, so that no word of an earlier replay
        # can pass for one of this.
        if binding.path_kind(B, K, V, top_k, top_p) == 3 and \
                (call.other or torch.cuda.is_current_stream_capturing()):
            workspace = call.zeros(nbytes)
        else:
            workspace = call.empty((nbytes,), torch.uint8)
    call.run(lib.specv_verify_fp8_lm_head, _ptr(hidden), _ptr(hidden_scale), _ptr(packed.data),
             _ptr(draft_logits), _ptr(draft_tokens), _ptr(draft_len), _ptr(u), _ptr(u_final), B, K,
             V, D, float(temperature), int(top_k), float(top_p), int(eos_id), _ptr(target_logits),
             _ptr(res["out_tokens"]), _ptr(res["n_emitted"]), *_space(workspace, dev), call.ptr,
             *diag)
    return res


def _rows(t, name, shape, dev):
    """Checks a probability tensor whose rows are contiguous; its strides."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    sb, sk, sv = t.stride()
    if sv != 1 and shape[2] > 1 and t.numel():
        raise ValueError(f"the rows of {name} must be contiguous")
    return sb, sk


@functools.lru_cache(maxsize=1024)
def verify_probs_workspace_bytes(B, K, V):
    return int(load_ops_library().specv_verify_probs_workspace_bytes(int(B), int(K), int(V)))


def verify_probs(target_probs, draft_probs, draft_tokens, draft_len, u, u_final, eos_id=-1, *,
                 out_tokens=None, n_emitted=None, workspace=None, debug=False, stream=None):
    """The verification step from probabilities instead of logits.

    Shapes: target_probs [B, K+1, V] and draft_probs [B, K, V] (same dtype,
    bf16 or fp32; the rows contiguous, their strides free), draft_tokens [B, K]
    int32, draft_len [B] int32, u [B, K] fp32, u_final [B] fp32.
    ``draft_probs=None`` stands for drafts without a distribution: each was
    proposed with probability one.  Returns a dict with ``out_tokens`` [B,
    K+1] and ``n_emitted`` [B] (int32), plus ``accept_prob``,
    ``residual_mass``, ``stop_pos`` and ``path`` when ``debug`` is true, all as
    ``binding.verify`` gives them.  Asynchronous on ``stream``."""
    lib = load_ops_library()
    _gpu(target_probs, "target_probs", (3,))
    dev = target_probs.device
    B, K1, V = target_probs.shape
    K = K1 - 1
    code = _value_code(target_probs, "target_probs")
    tsb, tsk = _rows(target_probs, "target_probs", (B, K1, V), dev)
    dsb = dsk = 0
    if draft_probs is not None:
        dsb, dsk = _rows(draft_probs, "draft_probs", (B, K, V), dev)
        if draft_probs.dtype != target_probs.dtype:
            raise TypeError(f"draft_probs must be {target_probs.dtype}, got {draft_probs.dtype}")
    _check_round(draft_tokens, draft_len, u, u_final, B, K, dev)
    call = _Call(dev, stream)
    res, diag = _outputs(call, B, K, out_tokens, n_emitted, debug)
    if workspace is None:
        workspace = call.empty((verify_probs_workspace_bytes(B, K, V),), torch.uint8)
    call.run(lib.specv_verify_probs, _ptr(target_probs), tsb, tsk, _ptr(draft_probs), dsb, dsk,
             code, _ptr(draft_tokens), _ptr(draft_len), _ptr(u), _ptr(u_final), B, K, V, eos_id,
             _ptr(res["out_tokens"]), _ptr(res["n_emitted"]), *_space(workspace, dev), call.ptr,
             *diag)
    return res
