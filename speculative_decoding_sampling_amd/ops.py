"""Binding for libspecverify_ops: the operators around the verification.

``hidden_norm`` (the norms before an LM head with gate and residual scale),
``quantize_fp8``, ``pack_fp8_lm_head``, ``fp8_lm_head`` and
``verify_fp8_lm_head`` (an LM head on 8-bit floats, alone and with the
verification on its logits) and ``verify_probs`` (the verification from given
probabilities).  As in ``binding``, shapes and dtypes are checked, outputs and
workspaces allocated with torch and raw device pointers and the HIP stream
passed through the C ABI declared in ``include/specverify_ops.h``; here a native
module (``csrc/ops_ext.cpp``) does so, since these operators are often shorter
than the marshalling of a ctypes call.  If the libraries are not built the
calls raise: there is no fallback.  Nothing here records gradients.

8-bit values are ``torch.float8_e4m3fn`` tensors [..., D] with a
``torch.float8_e8m0fnu`` scale [..., D / 128] for each run of 128.
"""

import ctypes
import os
import threading

import torch

from . import binding
from .binding import SpecVerifyError

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libspecverify_ops.so")

FP8_BLOCK = 128
# None in a torch without the type: the package's other calls do without it
E4M3, E8M0 = getattr(torch, "float8_e4m3fn", None), getattr(torch, "float8_e8m0fnu", None)
_VALUE_CODES = {torch.float32: 0, torch.bfloat16: 1}
_OUT_CODES = {**_VALUE_CODES, **({E4M3: 2} if E4M3 else {})}

_lib = None
_native = None
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


def _load_native():
    """The native module, its libraries loaded first."""
    global _native
    load_ops_library()
    with _lock:
        if _native is None:
            path = os.path.join(os.path.dirname(_LIB_PATH), "_ops_native.so")
            if not os.path.exists(path):
                raise RuntimeError(
                    f"{path} is not built; run `python -m speculative_decoding_sampling_amd.build`")
            from . import _ops_native
            _native = _ops_native
    return _native


def _raw_stream(t, stream):
    """The raw handle of ``stream``, by default the current one of the tensor's
    device; 0 for a tensor that the call will refuse.  Another stream than the
    current one first waits for it: the outputs are allocated on the current
    stream, whose pending work may still use their memory."""
    index = t.get_device() if isinstance(t, torch.Tensor) else -1
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(index) if index >= 0 else 0
    if index >= 0 and stream.device != t.device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {t.device}")
    if index >= 0:
        current = torch.cuda.current_stream(t.device)
        if current != stream:
            stream.wait_stream(current)
    return stream.cuda_stream


def _done(res, stream):
    """The outputs of a native call, kept from reuse until ``stream`` has run
    it where that is not the current stream; a library error is raised."""
    if type(res) is int:
        raise SpecVerifyError(res, binding.status_string(res))
    if stream is not None:
        for t in res:
            t.record_stream(stream)
    return res


def _value_code(dtype):
    code = _VALUE_CODES.get(dtype)
    if code is None:
        raise TypeError(f"dtype must be bfloat16 or float32, got {dtype}")
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
    code = _OUT_CODES.get(dtype)
    if code is None:
        raise TypeError(f"dtype must be bfloat16, float32 or float8_e4m3fn, got {dtype}")
    return _done((_native or _load_native()).hidden_norm(
        x, residual, weight, post_weight, gate, scale, eps, code, residual_out, out, out_scale,
        _raw_stream(x, stream)), stream)


def quantize_fp8(x, *, out=None, out_scale=None, stream=None):
    """8-bit values and scales of ``x`` [..., D] (bf16 or fp32, D a multiple
    of 128): q float8_e4m3fn [..., D] and scale float8_e8m0fnu [..., D / 128],
    x ~ q * scale with the smallest power of two that brings each run's
    largest magnitude to at most 448.  Asynchronous on ``stream``."""
    return _done((_native or _load_native()).quantize_fp8(x, out, out_scale,
                                                          _raw_stream(x, stream)), stream)


class PackedFp8LmHead:
    """An 8-bit LM-head weight [V, D] in the layout the products read
    (``specv_fp8_lm_head_pack_weight``): ``data`` is the packed device buffer."""

    def __init__(self, data, V, D):
        self.data, self.V, self.D = data, int(V), int(D)


def fp8_lm_head_packed_weight_bytes(V, D):
    return int(load_ops_library().specv_fp8_lm_head_packed_weight_bytes(int(V), int(D)))


def pack_fp8_lm_head(weight, scale=None, *, stream=None):
    """Lay an LM-head weight out once for ``fp8_lm_head``: ``weight`` [V, D]
    float8_e4m3fn with ``scale`` [V, D / 128] float8_e8m0fnu, or bf16 / fp32
    without a scale (quantised here, see ``quantize_fp8``).  Asynchronous on
    ``stream``."""
    native = _native or _load_native()
    if scale is None:
        weight, scale = quantize_fp8(weight, stream=stream)
    data, = _done(native.pack_fp8_lm_head(weight, scale, _raw_stream(weight, stream)), stream)
    return PackedFp8LmHead(data, *weight.shape)


def _packed(packed):
    if not isinstance(packed, PackedFp8LmHead):
        raise TypeError("packed must be a PackedFp8LmHead")
    return packed.data, packed.V, packed.D


def fp8_lm_head(hidden, hidden_scale, packed, *, dtype=torch.bfloat16, logits=None, stream=None):
    """Logits [..., V] (``dtype`` bf16 or fp32) of hidden states [..., D]
    float8_e4m3fn with their scales (``hidden_norm`` or ``quantize_fp8``) and a
    ``PackedFp8LmHead``.  fp32 logits accumulate in float32; bf16 logits take the
    8-bit matrix product, whose sums hold fewer bits: up to 2^-10 of sum |h w|
    off before their rounding.  Asynchronous on ``stream``."""
    logits, = _done((_native or _load_native()).fp8_lm_head(
        hidden, hidden_scale, *_packed(packed), _value_code(dtype), logits,
        _raw_stream(hidden, stream)), stream)
    return logits


def _round_dict(res, names):
    """The outputs of a verification by name, the diagnostics where they were
    asked for."""
    return dict(zip(names + ("out_tokens", "n_emitted", "accept_prob", "residual_mass", "stop_pos",
                             "path"), res))


def verify_fp8_lm_head(hidden, hidden_scale, packed, draft_logits, draft_tokens, draft_len, u,
                       u_final, temperature=1.0, eos_id=-1, *, top_k=0, top_p=1.0,
                       target_logits=None, out_tokens=None, n_emitted=None, workspace=None,
                       debug=False, stream=None):
    """The verification step on an 8-bit LM head: ``fp8_lm_head`` of hidden
    [B, K+1, D] gives the bf16 target logits [B, K+1, V], and the verification
    runs on them.  Other arguments and the returned dict as for
    ``binding.verify_lm_head``.  Asynchronous on ``stream``."""
    native = _native or _load_native()
    raw = _raw_stream(hidden, stream)
    data, V, D = _packed(packed)
    if workspace is None:
        workspace = _round_workspace(hidden, V, D, top_k, top_p, stream)
    return _round_dict(_done(native.verify_fp8_lm_head(
        hidden, hidden_scale, data, V, D, draft_logits, draft_tokens, draft_len, u, u_final,
        temperature, eos_id, top_k, top_p, target_logits, out_tokens, n_emitted, workspace, debug,
        raw), stream), ("target_logits",))


def _round_workspace(hidden, V, D, top_k, top_p, stream):
    """Workspace of a fused round, allocated on the stream that will use it."""
    if not isinstance(hidden, torch.Tensor):
        raise TypeError("hidden must be a torch.Tensor")
    if hidden.dim() != 3 or not hidden.is_cuda:
        raise ValueError("hidden must be a [B, K+1, D] GPU tensor")
    B, K = hidden.shape[0], hidden.shape[1] - 1
    nbytes = int(load_ops_library().specv_verify_fp8_lm_head_workspace_bytes(
        B, K, V, D, int(top_k), float(top_p)))
    with torch.cuda.stream(stream):
        # Path 3 keeps a call counter in its workspace.  A captured call gets
        # memory that the rest of its graph may use between two replays: the
        # graph clears it before each, so that no word of an earlier replay
        # can pass for one of this.
        clear = torch.cuda.is_current_stream_capturing() and \
            binding.path_kind(B, K, V, top_k, top_p) == 3
        return (torch.zeros if clear else torch.empty)(nbytes, dtype=torch.uint8,
                                                       device=hidden.device)


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
    raw = _raw_stream(target_probs, stream)
    if stream is not None and workspace is None and isinstance(target_probs, torch.Tensor) and \
            target_probs.is_cuda and target_probs.dim() == 3:
        # allocated on the stream that uses it, the default stream (raw handle
        # 0) as well: it is given back right after
        B, K1, V = target_probs.shape
        with torch.cuda.stream(stream):
            workspace = torch.empty(verify_probs_workspace_bytes(B, K1 - 1, V), dtype=torch.uint8,
                                    device=target_probs.device)
    return _round_dict(_done((_native or _load_native()).verify_probs(
        target_probs, draft_probs, draft_tokens, draft_len, u, u_final, eos_id, out_tokens,
        n_emitted, workspace, debug, raw), stream), ())
