"""Build libspecverify.so, libspecverify_ops.so and libspecverify_draft.so in-tree
with hipcc for gfx950.

Usage: ``python -m speculative_decoding_sampling_amd.build`` (or
``__graft_entry__.build()``).  Compiles every source under ``csrc/`` to an
object in ``_build/`` in parallel and links the shared libraries next to this
file, where the Python bindings load them.  libspecverify_ops calls
libspecverify's public entry points and finds it in its own folder; the Python
modules _ops_native and _draft_native (host C++, torch's headers) call
libspecverify_ops and libspecverify_draft.  ``build()`` makes the first two
libraries and their module, ``build_draft()`` the third and its own.
"""

import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libspecverify.so")
OPS_LIB = os.path.join(HERE, "libspecverify_ops.so")

ARCH = "gfx950"
SOURCES = ["specverify.hip", "row_stats.hip", "accept.hip", "sample.hip", "filter.hip",
           "filter_rows.hip", "sample_list.hip", "diagnostics.hip", "round_policy.hip",
           "lm_head.hip", "small.hip"]
OPS_SOURCES = ["ops.hip", "probs.hip", "hidden_norm.hip", "fp8_head.hip"]
# Python module of the operators, host C++ against torch's headers
OPS_EXT = os.path.join(HERE, "_ops_native.so")
OPS_EXT_SOURCE = "ops_ext.cpp"
DRAFT_LIB = os.path.join(HERE, "libspecverify_draft.so")
DRAFT_SOURCES = ["draft.hip", "fp4_head.hip", "filter_draw.hip"]
DRAFT_EXT = os.path.join(HERE, "_draft_native.so")
DRAFT_EXT_SOURCE = "draft_ext.cpp"
# Packed FP32 instructions stay off: the compiler must not form v_pk_* FP32 ops.
FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-Wall", "-fvisibility=hidden",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", INCLUDE, "-I", CSRC,
]


def _hipcc():
    for cand in (shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found (ROCm is required to build libspecverify)")


def _run(cmd):
    p = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    out = "\n".join(l for l in p.stdout.splitlines()
                    if "packed-fp32-ops" not in l and "not a recognized feature" not in l)
    if p.returncode != 0:
        raise RuntimeError("command failed: " + " ".join(cmd) + "\n" + out)
    return out


def _object(src):
    return os.path.join(BUILD, os.path.splitext(src)[0] + ".o")


def _link(hipcc, lib, sources, *extra):
    tmp = lib + ".tmp"
    out = _run([hipcc, f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp,
                *map(_object, sources), *extra])
    os.replace(tmp, lib)
    return out


def _ext_commands(source=OPS_EXT_SOURCE, libs=("-lspecverify_ops", "-lspecverify"), ext=None):
    """Compile and link command of a Python module, the operators' by default."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension

    cxx = shutil.which("g++") or "g++"
    torch_lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    inc = [INCLUDE, "/opt/rocm/include", sysconfig.get_paths()["include"],
           *cpp_extension.include_paths()]
    compile_ = [cxx, "-O2", "-std=c++17", "-fPIC", "-Wall", "-fvisibility=hidden",
                "-D__HIP_PLATFORM_AMD__", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
                *[f"-isystem{d}" for d in inc], "-c", os.path.join(CSRC, source), "-o", _object(source)]
    link = [cxx, "-shared", "-o", (ext or OPS_EXT) + ".tmp", _object(source), "-L", HERE, *libs,
            "-L", torch_lib, "-lc10", "-ltorch_cpu", "-ltorch_hip",
            "-ltorch_python", "-Wl,-rpath,$ORIGIN"]
    return compile_, link


def _build_ext():
    ext_compile, ext_link = _ext_commands()
    return _run(ext_compile), ext_link


def build(verbose=False):
    """Compile everything and link it in the order of what it needs: a library
    is in place even if something after it does not build, which is then raised."""
    hipcc = _hipcc()
    os.makedirs(BUILD, exist_ok=True)
    sources = SOURCES + OPS_SOURCES
    with ThreadPoolExecutor(max_workers=min(len(sources) + 1, os.cpu_count() or 1, 8)) as ex:
        objects = [ex.submit(_run, [hipcc, *FLAGS, "-c", os.path.join(CSRC, src), "-o", _object(src)])
                   for src in sources]
        # the only step that needs g++ and torch's headers
        module = ex.submit(_build_ext)
        outs = [f.result() for f in objects[:len(SOURCES)]]
        outs.append(_link(hipcc, LIB, SOURCES))
        outs += [f.result() for f in objects[len(SOURCES):]]
        outs.append(_link(hipcc, OPS_LIB, OPS_SOURCES, "-L", HERE, "-lspecverify",
                          "-Wl,-rpath,$ORIGIN"))
    try:
        out, ext_link = module.result()
        outs += [out, _run(ext_link)]
        os.replace(OPS_EXT + ".tmp", OPS_EXT)
    except BaseException:
        # an older module may not fit the new library
        if os.path.exists(OPS_EXT):
            os.remove(OPS_EXT)
        raise
    if verbose:
        for o in outs:
            if o.strip():
                print(o)
    return LIB


def build_draft(verbose=False):
    """The library of the draft step's operators and its Python module, in the
    same order and with the same care."""
    hipcc = _hipcc()
    os.makedirs(BUILD, exist_ok=True)

    def module():
        compile_, link = _ext_commands(DRAFT_EXT_SOURCE, ("-lspecverify_draft",), DRAFT_EXT)
        return _run(compile_), link

    with ThreadPoolExecutor(max_workers=len(DRAFT_SOURCES) + 1) as ex:
        objects = [ex.submit(_run, [hipcc, *FLAGS, "-c", os.path.join(CSRC, src), "-o", _object(src)])
                   for src in DRAFT_SOURCES]
        ext = ex.submit(module)
        outs = [f.result() for f in objects]
        outs.append(_link(hipcc, DRAFT_LIB, DRAFT_SOURCES))
    try:
        out, link = ext.result()
        outs += [out, _run(link)]
        os.replace(DRAFT_EXT + ".tmp", DRAFT_EXT)
    except BaseException:
        if os.path.exists(DRAFT_EXT):
            os.remove(DRAFT_EXT)
        raise
    if verbose:
        for o in outs:
            if o.strip():
                print(o)
    return DRAFT_LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
    print(build_draft(verbose="-v" in sys.argv))
