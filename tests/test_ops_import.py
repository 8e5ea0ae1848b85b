"""The package imports wherever it did before the operators came (CPU only): a
torch without the 8-bit types, and a tree without the operators' libraries."""

import os
import subprocess
import sys

import pytest

pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def python(code):
    return subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)


@pytest.mark.parametrize("missing", [("float8_e8m0fnu",), ("float8_e8m0fnu", "float8_e4m3fn")])
def test_import_without_8_bit_types(missing):
    p = python(f"""
import torch
for name in {missing!r}:
    delattr(torch, name)
import speculative_decoding_sampling_amd as S
assert callable(S.verify) and callable(S.sample) and callable(S.verify_probs)
x = torch.zeros(2, 128)
for dtype in (None, torch.float16):
    try:
        S.hidden_norm(x, x, x[0], dtype=dtype)
    except TypeError as e:
        assert "dtype must be" in str(e)
    else:
        raise AssertionError(dtype)
""")
    assert p.returncode == 0, p.stderr


def test_import_without_the_operators_libraries():
    p = python("""
import os
from speculative_decoding_sampling_amd import build, ops
ops._LIB_PATH = os.path.join(os.path.dirname(build.OPS_LIB), "nowhere", "libspecverify_ops.so")
import speculative_decoding_sampling_amd as S
try:
    S.load_ops_library()
except RuntimeError as e:
    assert "is not built" in str(e)
else:
    raise AssertionError
""")
    assert p.returncode == 0, p.stderr
