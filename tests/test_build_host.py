"""The build's order of steps (no compiler is run)."""
import os

import pytest

from orthogonalized_momentum_optimizer_amd import build as b


def test_libraries_are_linked_where_the_binding_fails(tmp_path, monkeypatch):
    """A container without a C++ compiler or PyTorch's headers still gets libmuon.so; the error is
    raised all the same."""
    linked = []

    def run(cmd):
        out = cmd[cmd.index("-o") + 1]
        open(out, "w").close()
        if "-c" not in cmd:
            linked.append(os.path.basename(out))
        return ""

    def fails():
        raise RuntimeError("no C++ compiler found")

    for name in ("BUILD", "LIB", "PROBE_LIB"):
        monkeypatch.setattr(b, name, str(tmp_path / name))
    monkeypatch.setattr(b, "hipcc", lambda: "hipcc")
    monkeypatch.setattr(b, "_run", run)
    monkeypatch.setattr(b, "build_args", fails)
    with pytest.raises(RuntimeError, match="no C"):
        b.build()
    assert linked == ["LIB.tmp", "PROBE_LIB.tmp"]
    assert (tmp_path / "LIB").exists() and (tmp_path / "PROBE_LIB").exists()
    monkeypatch.setattr(b, "build_args", lambda: None)
    assert b.build() == str(tmp_path / "LIB")
