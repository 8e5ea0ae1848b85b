"""Binding for libspecverify_draft: the operators of a draft step.

``quantize_fp4``, ``pack_fp4_lm_head`` and ``fp4_lm_head`` (an LM head on 4-bit
floats, for hidden states in 4 or in 8 bits), ``sample_filtered`` (one token of
each row after temperature, top-k, top-p and min-p, with parameters of each
request's own) and ``filter_probs`` (those distributions themselves, with the
draw or without it, as ``verify_probs`` takes them).  As in ``ops``, a native
module (``csrc/draft_ext.cpp``) checks shapes and dtypes, allocates outputs and
workspaces and passes raw device pointers and the HIP stream through the C ABI
declared in ``include/specverify_draft.h``.  If the library is not built the calls
raise: there is no fallback.  Nothing here records gradients.

4-bit values are ``torch.float4_e2m1fn_x2`` tensors [..., D / 2] (two to an
element) with a ``torch.float8_e8m0fnu`` scale [..., D / 32] for each block of 32.
"""

import ctypes
import os
import threading

import torch

from . import binding
from .ops import _done, _raw_stream, _value_code

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libspecverify_draft.so")

FP4_BLOCK = 32
# None in a torch without the type: the package's other calls do without it
E2M1 = getattr(torch, "float4_e2m1fn_x2", None)

_lib = None
_native = None
_lock = threading.Lock()


class Filters(ctypes.Structure):
    """``specv_filters_t``."""

    _fields_ = [("temperature_array", ctypes.c_void_p), ("top_k_array", ctypes.c_void_p),
                ("top_p_array", ctypes.c_void_p), ("min_p_array", ctypes.c_void_p),
                ("temperature", ctypes.c_float), ("top_k", ctypes.c_int32),
                ("top_p", ctypes.c_float), ("min_p", ctypes.c_float)]


def draft_library_path():
    return _LIB_PATH


def load_draft_library():
    """Load libspecverify_draft.so and declare its C signatures (once)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(
                f"{_LIB_PATH} is not built; run `python -m speculative_decoding_sampling_amd.build`")
        lib = ctypes.CDLL(_LIB_PATH)
        i, vp, size, i64 = ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int64
        lib.specv_fp4_quantize.argtypes = [vp, i, i, i, vp, vp, vp]
        lib.specv_fp4_quantize.restype = i
        lib.specv_fp4_lm_head_packed_weight_bytes.argtypes = [i, i]
        lib.specv_fp4_lm_head_packed_weight_bytes.restype = size
        lib.specv_fp4_lm_head_pack_weight.argtypes = [vp, vp, vp, i, i, vp]
        lib.specv_fp4_lm_head_pack_weight.restype = i
        lib.specv_fp4_lm_head.argtypes = [vp, i, vp, vp, i, i, i, vp, i, vp]
        lib.specv_fp4_lm_head.restype = i
        lib.specv_filter_workspace_bytes.argtypes = [i, i, i, i]
        lib.specv_filter_workspace_bytes.restype = size
        lib.specv_filter.argtypes = [vp, i64, i64, i, i, i, i, ctypes.POINTER(Filters), vp, i64, i64,
                                     vp, i64, i64, vp, i64, i64, i, vp, size, vp]
        lib.specv_filter.restype = i
        lib.specv_draft_version.argtypes = []
        lib.specv_draft_version.restype = i
        _lib = lib
        return lib


def _load_native():
    """The native module, its library loaded first."""
    global _native
    binding.load_library()                          # names the status codes
    load_draft_library()
    with _lock:
        if _native is None:
            path = os.path.join(os.path.dirname(_LIB_PATH), "_draft_native.so")
            if not os.path.exists(path):
                raise RuntimeError(
                    f"{path} is not built; run `python -m speculative_decoding_sampling_amd.build`")
            from . import _draft_native
            _native = _draft_native
    return _native


def quantize_fp4(x, *, out=None, out_scale=None, stream=None):
    """4-bit values and scales of ``x`` [..., D] (bf16 or fp32, D a multiple
    of 32): q float4_e2m1fn_x2 [..., D / 2] and scale float8_e8m0fnu [..., D /
    32], x ~ q * scale with the smallest power of two that brings each block's
    largest magnitude to at most 6.  Asynchronous on ``stream``."""
    return _done((_native or _load_native()).quantize_fp4(x, out, out_scale,
                                                          _raw_stream(x, stream)), stream)


class PackedFp4LmHead:
    """A 4-bit LM-head weight [V, D] in the layout the products read
    (``specv_fp4_lm_head_pack_weight``): ``data`` is the packed device buffer."""

    def __init__(self, data, V, D):
        self.data, self.V, self.D = data, int(V), int(D)


def fp4_lm_head_packed_weight_bytes(V, D):
    return int(load_draft_library().specv_fp4_lm_head_packed_weight_bytes(int(V), int(D)))


def pack_fp4_lm_head(weight, scale=None, *, stream=None):
    """Lay an LM-head weight out once for ``fp4_lm_head``: ``weight`` [V, D / 2]
    float4_e2m1fn_x2 with ``scale`` [V, D / 32] float8_e8m0fnu, or [V, D] bf16 /
    fp32 without a scale (quantised here, see ``quantize_fp4``).  Asynchronous on
    ``stream``."""
    native = _native or _load_native()
    if scale is None:
        weight, scale = quantize_fp4(weight, stream=stream)
    data, = _done(native.pack_fp4_lm_head(weight, scale, _raw_stream(weight, stream)), stream)
    return PackedFp4LmHead(data, weight.shape[0], 2 * weight.shape[1])


def _packed(packed):
    if not isinstance(packed, PackedFp4LmHead):
        raise TypeError("packed must be a PackedFp4LmHead")
    return packed.data, packed.V, packed.D


def fp4_lm_head(hidden, hidden_scale, packed, *, dtype=torch.bfloat16, logits=None, stream=None):
    """Logits [..., V] (``dtype`` bf16 or fp32) of hidden states and a
    ``PackedFp4LmHead``.  The states are float8_e4m3fn [..., D] with a scale for
    each 128 (``hidden_norm``, ``quantize_fp8``) or float4_e2m1fn_x2 [..., D / 2]
    with a scale for each 32 (``quantize_fp4``).  Sums are float32 but for bf16
    logits of 8-bit states, which take the mixed matrix product: up to 2^-10 of
    sum |h w| off before their rounding.  Asynchronous on ``stream``."""
    logits, = _done((_native or _load_native()).fp4_lm_head(
        hidden, hidden_scale, *_packed(packed), _value_code(dtype), logits,
        _raw_stream(hidden, stream)), stream)
    return logits


def filter_workspace_bytes(B, L, V, dtype=torch.float32):
    return int(load_draft_library().specv_filter_workspace_bytes(int(B), int(L), int(V),
                                                                 _value_code(dtype)))


def _filter(logits, temperature, top_k, top_p, min_p, u, out_tokens, probs, code, workspace, stream):
    raw = _raw_stream(logits, stream)
    if stream is not None and workspace is None and isinstance(logits, torch.Tensor) and \
            logits.is_cuda and logits.dim() in (2, 3) and logits.dtype in (torch.float32,
                                                                           torch.bfloat16):
        # allocated on the stream that uses it: it is given back right after
        B, L, V = logits.shape[0], logits.shape[1] if logits.dim() == 3 else 1, logits.shape[-1]
        with torch.cuda.stream(stream):
            workspace = torch.empty(filter_workspace_bytes(B, L, V, logits.dtype),
                                    dtype=torch.uint8, device=logits.device)
    return _done((_native or _load_native()).filter(
        logits, temperature, top_k, top_p, min_p, u, out_tokens, probs, code, workspace, raw), stream)


def sample_filtered(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, *, out_tokens=None,
                    workspace=None, stream=None):
    """One token of each row of ``logits`` [B, V] or [B, L, V] (bf16 or fp32; the
    rows contiguous, their strides free) at the uniforms ``u`` [B] or [B, L].

    Each parameter is a number, or a [B] tensor (fp32; int32 for ``top_k``) with
    each request's own.  A row's distribution is softmax(z / temperature) over the
    tokens that all filters keep: the ``top_k`` largest (0: all; ties kept), of
    those the shortest prefix whose mass reaches ``top_p``, and those at least
    ``min_p`` times as probable as the most probable one.  Temperature 0 takes the
    largest logit (the lowest id of equal ones).  Returns int32 tokens, -1 for a
    row with a parameter or uniform out of range, without a finite logit, or with
    a NaN or +inf.  Asynchronous on ``stream``."""
    if u is None:
        raise TypeError("u must be a torch.Tensor")
    tokens, = _filter(logits, temperature, top_k, top_p, min_p, u, out_tokens, None, -1, workspace,
                      stream)
    return tokens


def filter_probs(logits, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, *, u=None,
                 dtype=torch.float32, probs=None, out_tokens=None, workspace=None, stream=None):
    """The filtered distributions of ``sample_filtered``: probabilities of
    ``dtype`` (bf16 or fp32) shaped like ``logits``, 0 for tokens not kept and for
    rows that would have no token.  With ``u`` returns (probs, tokens), the tokens
    drawn from them.  ``probs`` and ``out_tokens`` may be strided views, such as one
    position of the arrays that ``verify_probs`` takes.  Asynchronous on
    ``stream``."""
    res = _filter(logits, temperature, top_k, top_p, min_p, u, out_tokens, probs,
                  _value_code(dtype), workspace, stream)
    return tuple(res) if u is not None else res[0]
