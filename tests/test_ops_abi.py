"""The companion library builds, loads and exports what its header declares;
arguments are refused before any GPU work (CPU only)."""

import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
VP, I, F, SZ, I64 = (ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t,
                     ctypes.c_int64)
EINVAL, EWORKSPACE, EUNSUPPORTED = 1, 2, 4
# never read or written: addresses that only the checks look at
A = 1 << 40
FAR = [A + (i << 36) for i in range(32)]


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_sampling_amd import build, ops
    if not (os.path.exists(build.LIB) and os.path.exists(build.OPS_LIB)):
        build.build()
    return ops.load_ops_library()


def declared():
    with open(os.path.join(ROOT, "include", "specverify_ops.h")) as f:
        return set(re.findall(r"SPECV_OPS_API\s+[\w\s\*]+?\b(specv_\w+)\s*\(", f.read()))


def test_exports_are_the_declared_functions(lib):
    import subprocess
    from speculative_decoding_sampling_amd import build
    out = subprocess.run(["nm", "-D", "--defined-only", build.OPS_LIB], capture_output=True,
                         text=True).stdout
    assert {l.split()[-1] for l in out.splitlines() if " T " in l} == declared()
    assert len(declared()) == 10 and lib.specv_ops_version() == 100


def test_header_compiles_as_c(tmp_path):
    import subprocess
    src = tmp_path / "t.c"
    src.write_text('#include "specverify_ops.h"\nint main(void) { return specv_ops_version() == 0; }\n')
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-fsyntax-only", "-D__HIP_PLATFORM_AMD__",
                    "-I", os.path.join(ROOT, "include"), "-I", "/opt/rocm/include", str(src)],
                   check=True)


def caller(f, names, base):
    def call(**kw):
        assert set(kw) <= set(names), kw
        a = dict(base, **kw)
        return f(*[a[n] for n in names])
    return call


NORM = ("x xt r rt pw gate rows w wt M D scale eps r_out out ot osc stream").split()
NORM_OK = dict(x=FAR[0], xt=1, r=FAR[1], rt=0, pw=FAR[2], gate=FAR[3], rows=2, w=FAR[4], wt=1, M=6,
               D=256, scale=1.0, eps=1e-6, r_out=FAR[5], out=FAR[6], ot=2, osc=FAR[7], stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(M=0), EINVAL), (dict(D=0), EINVAL), (dict(D=65537, ot=1), EUNSUPPORTED),
    (dict(xt=2), EINVAL), (dict(rt=7), EINVAL), (dict(wt=-1), EINVAL), (dict(ot=3), EINVAL),
    (dict(D=200), EINVAL),                         # 8-bit output: D a multiple of 128
    (dict(osc=None), EINVAL), (dict(scale=float("nan")), EINVAL), (dict(eps=0.0), EINVAL),
    (dict(eps=float("inf")), EINVAL), (dict(x=None), EINVAL), (dict(r=None), EINVAL),
    (dict(w=None), EINVAL), (dict(r_out=None), EINVAL), (dict(out=None), EINVAL),
    (dict(rows=4), EINVAL), (dict(rows=0), EINVAL), (dict(x=FAR[0] + 1), EINVAL),
    (dict(r=FAR[1] + 2), EINVAL), (dict(gate=FAR[3] + 1), EINVAL), (dict(out=FAR[6] + 4), EINVAL),
    (dict(r_out=FAR[1] + 4), EINVAL),              # shifted overlap with the residual
    (dict(r_out=FAR[0]), EINVAL),                  # over x
    (dict(out=FAR[0]), EINVAL),                    # over x of another type
    (dict(out=FAR[5]), EINVAL),                    # over residual_out
    (dict(out=FAR[4]), EINVAL), (dict(osc=FAR[6]), EINVAL),
])
def test_hidden_norm_refuses(lib, kw, want):
    assert caller(lib.specv_hidden_norm, NORM, NORM_OK)(**kw) == want


def test_quantize_refuses(lib):
    call = caller(lib.specv_fp8_quantize, "x t rows D q s stream".split(),
                  dict(x=FAR[0], t=1, rows=4, D=256, q=FAR[1], s=FAR[2], stream=None))
    for kw in (dict(rows=0), dict(D=0), dict(D=130), dict(t=5), dict(x=None), dict(q=None),
               dict(s=None), dict(x=FAR[0] + 2), dict(q=FAR[1] + 4), dict(q=FAR[0]),
               dict(s=FAR[1] + 8)):
        assert call(**kw) == EINVAL, kw
    assert call(D=65536 + 128) == EUNSUPPORTED


def test_packed_sizes_and_refusals(lib):
    n = lib.specv_fp8_lm_head_packed_weight_bytes
    assert n(32, 128) == 32 * 128 + 32 * 4 and n(33, 128) == 2 * n(32, 128)
    assert n(128256, 4096) == 128256 * 4096 + 128256 // 32 * 8 * 128
    assert n(32, 640) == 32 * 640 + 2 * 128                      # 5 runs: 2 scale words a row
    for V, D in ((0, 128), (32, 0), (32, 100), (4194305, 128), (32, 65664)):
        assert n(V, D) == 0
    call = caller(lib.specv_fp8_lm_head_pack_weight, "q s p V D stream".split(),
                  dict(q=FAR[0], s=FAR[1], p=FAR[2], V=100, D=256, stream=None))
    for kw in (dict(V=0), dict(D=64), dict(q=None), dict(s=None), dict(p=None), dict(q=FAR[0] + 8),
               dict(p=FAR[2] + 8), dict(p=FAR[0] + 64), dict(s=FAR[2] + 16)):
        assert call(**kw) == EINVAL, kw
    assert call(V=4194305) == EUNSUPPORTED


def test_lm_head_refuses(lib):
    call = caller(lib.specv_fp8_lm_head, "h s p M D V out t stream".split(),
                  dict(h=FAR[0], s=FAR[1], p=FAR[2], M=5, D=256, V=1000, out=FAR[3], t=1, stream=None))
    for kw in (dict(M=0), dict(D=0), dict(D=192), dict(V=0), dict(t=2), dict(h=None), dict(s=None),
               dict(p=None), dict(out=None), dict(h=FAR[0] + 8), dict(p=FAR[2] + 4),
               dict(out=FAR[3] + 1), dict(out=FAR[2]), dict(out=FAR[0])):
        assert call(**kw) == EINVAL, kw
    assert call(V=4194305) == EUNSUPPORTED and call(D=65664) == EUNSUPPORTED
    assert call(M=0x7fffffff, V=4194304) == EUNSUPPORTED          # more workgroups than a grid holds


FUSED = ("h s p dl tok n u uf B K V D T top_k top_p eos tl out ne ws wsb stream ap rm sp pa").split()
FUSED_OK = dict(h=FAR[0], s=FAR[1], p=FAR[2], dl=FAR[3], tok=FAR[4], n=FAR[5], u=FAR[6], uf=FAR[7],
                B=2, K=3, V=1000, D=256, T=1.0, top_k=0, top_p=1.0, eos=-1, tl=FAR[8], out=FAR[9],
                ne=FAR[10], ws=FAR[11], wsb=1 << 30, stream=None, ap=None, rm=None, sp=None, pa=None)


@pytest.mark.parametrize("kw,want", [
    (dict(B=0), EINVAL), (dict(K=65), EINVAL), (dict(K=-1), EINVAL), (dict(V=0), EINVAL),
    (dict(D=100), EINVAL), (dict(T=0.0), EINVAL), (dict(top_k=-1), EINVAL), (dict(top_p=0.0), EINVAL),
    (dict(eos=1000), EINVAL), (dict(h=None), EINVAL), (dict(p=None), EINVAL), (dict(dl=None), EINVAL),
    (dict(tok=None), EINVAL), (dict(tl=None), EINVAL), (dict(ne=None), EINVAL), (dict(u=None), EINVAL),
    (dict(dl=FAR[3] + 1), EINVAL), (dict(u=FAR[6] + 2), EINVAL), (dict(rm=FAR[12] + 4), EINVAL),
    (dict(ws=None), EWORKSPACE), (dict(ws=FAR[11] + 8), EWORKSPACE), (dict(wsb=16), EWORKSPACE),
    (dict(V=4194305), EUNSUPPORTED),
])
def test_verify_fp8_lm_head_refuses(lib, kw, want):
    assert caller(lib.specv_verify_fp8_lm_head, FUSED, FUSED_OK)(**kw) == want


def test_verify_fp8_lm_head_workspace(lib):
    from speculative_decoding_sampling_amd import binding
    n = lib.specv_verify_fp8_lm_head_workspace_bytes
    assert n(64, 4, 128256, 4096, 0, 1.0) >= binding.workspace_bytes(64, 4, 128256, 1)
    assert n(2, 4, 1000, 100, 0, 1.0) == 0 and n(0, 4, 1000, 128, 0, 1.0) == 0


PROBS = ("t tsb tsk d dsb dsk dt tok n u uf B K V eos out ne ws wsb stream ap rm sp pa").split()
PROBS_OK = dict(t=FAR[0], tsb=360000, tsk=90000, d=FAR[1], dsb=270000, dsk=90000, dt=0, tok=FAR[2],
                n=FAR[3], u=FAR[4], uf=FAR[5], B=2, K=3, V=90000, eos=-1, out=FAR[6], ne=FAR[7],
                ws=FAR[8], wsb=1 << 20, stream=None, ap=None, rm=None, sp=None, pa=None)


@pytest.mark.parametrize("kw,want", [
    (dict(B=0), EINVAL), (dict(K=65), EINVAL), (dict(K=-1), EINVAL), (dict(V=0), EINVAL),
    (dict(V=4194305), EUNSUPPORTED), (dict(B=0x7fffffff, V=4096), EUNSUPPORTED),
    (dict(dt=3), EINVAL), (dict(eos=90000), EINVAL), (dict(eos=-2), EINVAL), (dict(tsb=-1), EINVAL),
    (dict(dsk=-1), EINVAL), (dict(tsb=1 << 62), EINVAL), (dict(t=None), EINVAL),
    (dict(tok=None), EINVAL), (dict(n=None), EINVAL), (dict(u=None), EINVAL), (dict(uf=None), EINVAL),
    (dict(out=None), EINVAL), (dict(ne=None), EINVAL), (dict(t=FAR[0] + 2), EINVAL),
    (dict(d=FAR[1] + 1), EINVAL), (dict(rm=FAR[9] + 4), EINVAL), (dict(ws=None), EWORKSPACE),
    (dict(ws=FAR[8] + 4), EWORKSPACE), (dict(wsb=16), EWORKSPACE),
])
def test_verify_probs_refuses(lib, kw, want):
    assert caller(lib.specv_verify_probs, PROBS, PROBS_OK)(**kw) == want


def test_verify_probs_workspace(lib):
    n = lib.specv_verify_probs_workspace_bytes
    assert n(64, 4, 128256) == 64 * (126 * 8 + 16) and n(1, 64, 4194304) > 0
    assert n(1, 0, 1) == 0                                        # one kernel: none needed
    assert n(0, 4, 100) == 0 and n(1, 65, 100) == 0 and n(1, 1, 4194305) == 0


def test_python_calls_refuse_cpu_tensors(lib):
    torch = pytest.importorskip("torch")
    import speculative_decoding_sampling_amd as S
    x = torch.zeros(2, 128)
    for f in (lambda: S.hidden_norm(x, x, x[0]), lambda: S.quantize_fp8(x),
              lambda: S.pack_fp8_lm_head(x),
              lambda: S.fp8_lm_head(x, x, S.PackedFp8LmHead(x, 2, 128)),
              lambda: S.verify_probs(x[None], None, None, None, None, None)):
        with pytest.raises(ValueError):
            f()
    for f in (lambda: S.quantize_fp8([1.0]), lambda: S.fp8_lm_head(x, x, None),
              lambda: S.hidden_norm(x, x, x[0], dtype=torch.float16),
              lambda: S.verify_probs(None, None, None, None, None, None)):
        with pytest.raises(TypeError):
            f()
