"""build() of the entry module loads what it built (CPU only): the libraries and
the operators' Python module, so one that links but cannot be imported is found
there and not at the first call."""

import os

import pytest

pytest.importorskip("torch")
import __graft_entry__ as entry  # noqa: E402
from speculative_decoding_sampling_amd import build, ops  # noqa: E402


def test_build_loads_the_native_module(monkeypatch):
    monkeypatch.setattr(build, "build", lambda: build.LIB)
    loaded = []
    monkeypatch.setattr(ops, "_load_native", lambda: loaded.append(True))
    entry.build()
    assert loaded

    def broken():
        raise ImportError("undefined symbol")

    monkeypatch.setattr(ops, "_load_native", broken)
    with pytest.raises(ImportError):
        entry.build()


def test_the_built_module_has_every_operator():
    if not all(os.path.exists(p) for p in (build.LIB, build.OPS_LIB, build.OPS_EXT)):
        build.build()
    native = ops._load_native()
    assert {"hidden_norm", "quantize_fp8", "pack_fp8_lm_head", "fp8_lm_head", "verify_fp8_lm_head",
            "verify_probs"} <= set(dir(native))
