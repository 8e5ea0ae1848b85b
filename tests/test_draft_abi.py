"""The draft library builds, loads and exports what its header declares;
arguments are refused before any GPU work (CPU only)."""

import ctypes
import os
import re
import subprocess

import pytest

from tests.test_ops_abi import EINVAL, EUNSUPPORTED, EWORKSPACE, FAR, ROOT, caller


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_sampling_amd import build, draft
    if not (os.path.exists(build.DRAFT_LIB) and os.path.exists(build.DRAFT_EXT)):
        build.build_draft()
    return draft.load_draft_library()


def declared():
    with open(os.path.join(ROOT, "include", "specverify_draft.h")) as f:
        return set(re.findall(r"SPECV_DRAFT_API\s+[\w\s\*]+?\b(specv_\w+)\s*\(", f.read()))


def test_exports_are_the_declared_functions(lib):
    from speculative_decoding_sampling_amd import build
    out = subprocess.run(["nm", "-D", "--defined-only", build.DRAFT_LIB], capture_output=True,
                         text=True).stdout
    assert {l.split()[-1] for l in out.splitlines() if " T " in l} == declared()
    assert "specv_filter" in declared() and lib.specv_draft_version() == 100


def test_header_compiles_as_c(tmp_path):
    from speculative_decoding_sampling_amd.draft import Filters
    src = tmp_path / "t.c"
    src.write_text('#include "specverify_draft.h"\n#include <stdio.h>\n'
                   'int main(void) { printf("%zu", sizeof(specv_filters_t)); return 0; }\n')
    exe = tmp_path / "t"
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-D__HIP_PLATFORM_AMD__", "-I",
                    os.path.join(ROOT, "include"), "-I", "/opt/rocm/include", str(src), "-o", str(exe)],
                   check=True)
    size = subprocess.run([str(exe)], capture_output=True, text=True).stdout
    assert int(size) == ctypes.sizeof(Filters)


def test_the_built_module_has_every_operator(lib):
    from speculative_decoding_sampling_amd import draft
    assert {"quantize_fp4", "pack_fp4_lm_head", "fp4_lm_head", "filter"} <= set(dir(draft._load_native()))


def test_quantize_refuses(lib):
    call = caller(lib.specv_fp4_quantize, "x t rows D q s stream".split(),
                  dict(x=FAR[0], t=1, rows=4, D=96, q=FAR[1], s=FAR[2], stream=None))
    for kw in (dict(rows=0), dict(D=0), dict(D=48), dict(t=5), dict(x=None), dict(q=None), dict(s=None),
               dict(x=FAR[0] + 2), dict(q=FAR[1] + 2), dict(q=FAR[0]), dict(s=FAR[1] + 8),
               dict(s=FAR[0])):
        assert call(**kw) == EINVAL, kw
    assert call(D=65536 + 32) == EUNSUPPORTED
    assert call(rows=1 << 20, D=32768) == EUNSUPPORTED                 # 2^32 threads
    assert call(rows=(1 << 20) - 1, D=32768, x=None) == EINVAL


def test_packed_sizes_and_refusals(lib):
    n = lib.specv_fp4_lm_head_packed_weight_bytes
    assert n(32, 128) == 32 * 64 + 64 * 4 and n(33, 128) == 2 * n(32, 128)
    assert n(128256, 4096) == 128256 * 2048 + 128256 // 32 * 16 * 256
    assert n(32, 640) == 32 * 320 + 3 * 256                          # 10 steps: 3 words a lane
    for V, D in ((0, 128), (32, 0), (32, 96), (4194305, 128), (32, 65664), (4194304, 65536)):
        assert n(V, D) == 0
    call = caller(lib.specv_fp4_lm_head_pack_weight, "q s p V D stream".split(),
                  dict(q=FAR[0], s=FAR[1], p=FAR[2], V=100, D=256, stream=None))
    for kw in (dict(V=0), dict(D=64), dict(q=None), dict(s=None), dict(p=None), dict(q=FAR[0] + 8),
               dict(p=FAR[2] + 8), dict(p=FAR[0] + 64), dict(s=FAR[2] + 16)):
        assert call(**kw) == EINVAL, kw
    assert call(V=4194305) == EUNSUPPORTED and call(V=4194304, D=65536) == EUNSUPPORTED


def test_lm_head_refuses(lib):
    call = caller(lib.specv_fp4_lm_head, "h ht s p M D V out t stream".split(),
                  dict(h=FAR[0], ht=0, s=FAR[1], p=FAR[2], M=5, D=256, V=1000, out=FAR[3], t=1, stream=None))
    for kw in (dict(M=0), dict(D=0), dict(D=192), dict(V=0), dict(t=2), dict(ht=2), dict(ht=-1),
               dict(h=None), dict(s=None), dict(p=None), dict(out=None), dict(h=FAR[0] + 8),
               dict(p=FAR[2] + 4), dict(out=FAR[3] + 1), dict(out=FAR[2]), dict(out=FAR[0]),
               dict(out=FAR[1]), dict(out=FAR[0] + 5 * 256 - 2)):
        assert call(**kw) == EINVAL, kw
    assert call(V=4194305) == EUNSUPPORTED and call(D=65664) == EUNSUPPORTED
    assert call(M=0x7fffffff, V=4194304) == EUNSUPPORTED


FILTER = ("z zsb zsl zt B L V f u usb usl out tsb tsl p psb psl pt ws wsb stream").split()
FILTER_OK = dict(z=FAR[0], zsb=3 * 40000, zsl=40000, zt=0, B=4, L=3, V=40000, f={}, u=FAR[1], usb=3, usl=1,
                 out=FAR[2], tsb=3, tsl=1, p=FAR[3], psb=120000, psl=40000, pt=0, ws=FAR[4], wsb=1 << 28,
                 stream=None)


def call_filter(lib, **kw):
    from speculative_decoding_sampling_amd.draft import Filters
    a = dict(FILTER_OK, **kw)
    f = a["f"]
    if f is not None:
        f = ctypes.byref(Filters(**dict(dict(temperature=1.0, top_k=0, top_p=1.0, min_p=0.0), **f)))
    return lib.specv_filter(*[f if n == "f" else a[n] for n in FILTER])


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("kw", [
    dict(z=None), dict(f=None), dict(B=0), dict(L=0), dict(V=0), dict(zt=2), dict(pt=7), dict(u=None),
    dict(out=None, p=None), dict(z=FAR[0] + 2), dict(u=FAR[1] + 1), dict(out=FAR[2] + 2),
    dict(p=FAR[3] + 2), dict(zsb=-1), dict(zsl=-1), dict(usb=-1), dict(tsl=-1), dict(psb=-1),
    dict(zsb=1 << 62), dict(psl=1 << 62),
    dict(f=dict(temperature=-1.0)), dict(f=dict(temperature=NAN)), dict(f=dict(temperature=INF)),
    dict(f=dict(top_k=-1)), dict(f=dict(top_p=0.0)), dict(f=dict(top_p=1.5)), dict(f=dict(top_p=NAN)),
    dict(f=dict(min_p=-0.1)), dict(f=dict(min_p=1.5)), dict(f=dict(min_p=NAN)),
    dict(f=dict(temperature_array=FAR[9] + 2)), dict(f=dict(top_k_array=FAR[9] + 1)),
])
def test_filter_refuses(lib, kw):
    assert call_filter(lib, **kw) == EINVAL


@pytest.mark.parametrize("kw", [
    dict(p=FAR[0]), dict(p=FAR[1]), dict(out=FAR[0]), dict(out=FAR[1]), dict(out=FAR[3] + 4000),
    dict(ws=FAR[0]), dict(ws=FAR[3]), dict(ws=FAR[2]), dict(ws=FAR[1]),
    dict(f=dict(temperature_array=FAR[2])), dict(f=dict(top_p_array=FAR[3] + 16)),
    dict(f=dict(min_p_array=FAR[4])),
    dict(psl=39999), dict(psb=119999), dict(psb=0), dict(psl=0), dict(tsb=0), dict(tsl=0), dict(tsb=2),
    dict(B=1, psl=500), dict(L=1, psb=39999), dict(L=1, tsb=0),
])
def test_filter_refuses_outputs_that_overlap(lib, kw):
    assert call_filter(lib, **kw) == EINVAL


def test_filter_workspace_and_limits(lib):
    n = lib.specv_filter_workspace_bytes
    assert n(4, 3, 40000, 0) > 0 and n(1, 1, 4194304, 1) > 0
    assert n(4, 3, 1000, 0) == 0                                       # one kernel: none needed
    for a in ((0, 1, 10, 0), (1, 0, 10, 0), (1, 1, 0, 0), (1, 1, 4194305, 0), (1, 1, 10, 2)):
        assert n(*a) == 0
    for kw in (dict(ws=None), dict(ws=FAR[4] + 8), dict(wsb=16)):
        assert call_filter(lib, **kw) == EWORKSPACE, kw
    assert call_filter(lib, V=4194305) == EUNSUPPORTED
    assert call_filter(lib, B=0x7fffffff, L=2) == EUNSUPPORTED
    assert call_filter(lib, B=1 << 22) == EUNSUPPORTED                  # 2^32 threads
    # a refused probability type is not read where there are no probabilities; the
    # missing workspace is what is left to refuse
    assert call_filter(lib, p=None, pt=9, ws=None) == EWORKSPACE
    # transposed rows and rows in the gaps of others are fine: the same
    assert call_filter(lib, tsb=1, tsl=4, psb=40000, psl=160000, ws=None) == EWORKSPACE
    assert call_filter(lib, zsb=240000, zsl=80000, p=FAR[0] + 160000, psb=240000, psl=80000, ws=None) == EWORKSPACE


def test_python_calls_refuse_cpu_tensors(lib):
    torch = pytest.importorskip("torch")
    import speculative_decoding_sampling_amd as S
    x = torch.zeros(2, 128)
    for f in (lambda: S.quantize_fp4(x), lambda: S.pack_fp4_lm_head(x),
              lambda: S.fp4_lm_head(x, x, S.PackedFp4LmHead(x, 2, 128)),
              lambda: S.sample_filtered(x, x[:, 0]), lambda: S.filter_probs(x)):
        with pytest.raises(ValueError):
            f()
    for f in (lambda: S.quantize_fp4([1.0]), lambda: S.fp4_lm_head(x, x, None),
              lambda: S.sample_filtered(x, None), lambda: S.filter_probs(None),
              lambda: S.filter_probs(x, dtype=torch.float16)):
        with pytest.raises(TypeError):
            f()


def test_package_imports_without_the_4_bit_type():
    import sys
    p = subprocess.run([sys.executable, "-c", """
import torch
if hasattr(torch, "float4_e2m1fn_x2"):
    del torch.float4_e2m1fn_x2
import speculative_decoding_sampling_amd as S
assert callable(S.verify) and callable(S.fp4_lm_head) and callable(S.filter_probs)
"""], cwd=ROOT, capture_output=True, text=True)
    assert p.returncode == 0, p.stderr
