"""What a build leaves behind where the Python module of the operators cannot be
compiled (CPU only; the compilers are replaced by stand-ins that write their
output file): the libraries, which need neither g++ nor torch's headers, and no
older module, whose calls may not fit them."""

import os

import pytest

pytest.importorskip("torch")
from speculative_decoding_sampling_amd import build as b  # noqa: E402


@pytest.fixture
def tree(monkeypatch, tmp_path):
    for name in ("LIB", "OPS_LIB", "OPS_EXT"):
        monkeypatch.setattr(b, name, str(tmp_path / os.path.basename(getattr(b, name))))
    monkeypatch.setattr(b, "HERE", str(tmp_path))
    monkeypatch.setattr(b, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(b, "_hipcc", lambda: "hipcc")
    return tmp_path


def stand_in(monkeypatch, fails=lambda cmd: False):
    ran = []

    def run(cmd):
        ran.append(cmd)
        if fails(cmd):
            raise RuntimeError("command failed: " + " ".join(cmd))
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("new")
        return ""

    monkeypatch.setattr(b, "_run", run)
    return ran


def made(path):
    return os.path.exists(path) and open(path).read() == "new"


def test_everything_is_built(monkeypatch, tree):
    ran = stand_in(monkeypatch)
    assert b.build() == b.LIB
    assert made(b.LIB) and made(b.OPS_LIB) and made(b.OPS_EXT)
    assert len(ran) == len(b.SOURCES) + len(b.OPS_SOURCES) + 4   # the module, three links
    assert not [f for f in os.listdir(tree) if f.endswith(".tmp")]


@pytest.mark.parametrize("step", ["compile", "link"])
def test_a_module_that_does_not_build(monkeypatch, tree, step):
    # g++ fails or is missing
    open(b.OPS_EXT, "w").write("old")
    stand_in(monkeypatch, lambda cmd: cmd[0].endswith("g++") and ("-shared" in cmd) == (step == "link"))
    with pytest.raises(RuntimeError):
        b.build()
    assert made(b.LIB) and made(b.OPS_LIB) and not os.path.exists(b.OPS_EXT)


def test_no_torch_headers(monkeypatch, tree):
    stand_in(monkeypatch)

    def missing():
        raise ImportError("no module named torch")

    monkeypatch.setattr(b, "_ext_commands", missing)
    with pytest.raises(ImportError):
        b.build()
    assert made(b.LIB) and made(b.OPS_LIB) and not os.path.exists(b.OPS_EXT)


def test_a_source_of_the_operators_that_does_not_compile(monkeypatch, tree):
    for path in (b.OPS_LIB, b.OPS_EXT):
        open(path, "w").write("old")
    stand_in(monkeypatch, lambda cmd: any(c.endswith("probs.hip") for c in cmd))
    with pytest.raises(RuntimeError):
        b.build()
    # what fits together stays together
    assert made(b.LIB) and not made(b.OPS_LIB) and not made(b.OPS_EXT)
    assert os.path.exists(b.OPS_LIB) and os.path.exists(b.OPS_EXT)


def test_a_core_source_that_does_not_compile(monkeypatch, tree):
    for path in (b.LIB, b.OPS_LIB, b.OPS_EXT):
        open(path, "w").write("old")
    stand_in(monkeypatch, lambda cmd: any(c.endswith("accept.hip") for c in cmd))
    with pytest.raises(RuntimeError):
        b.build()
    assert all(open(p).read() == "old" for p in (b.LIB, b.OPS_LIB, b.OPS_EXT))
