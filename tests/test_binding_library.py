"""A library built before an entry point was added has the same ABI version: the
binding names what it lacks."""
import subprocess

import pytest

import shared_matrix_expert_amd as em


def build(path, names):
    src = path.with_suffix(".c")
    src.write_text("".join(f"int {n}(void) {{ return 0; }}\n" for n in names))
    subprocess.run(["gcc", "-shared", "-fPIC", str(src), "-o", str(path)], check=True)
    return str(path)


def test_an_older_library_is_named(tmp_path, monkeypatch):
    new = [n for n in em.EXPORTED if "_mx_" in n or "balance" in n or "route_backward" in n]
    old = build(tmp_path / "old.so", [n for n in em.EXPORTED if n not in new])
    monkeypatch.setattr(em, "_lib", None)
    with pytest.raises(RuntimeError, match="old.so was built from other sources.*shared_matrix_expert_amd.build") as e:
        em.load(old)
    assert all(n in str(e.value) for n in new)
    assert em._lib is None


def test_a_whole_library_loads(tmp_path, monkeypatch):
    monkeypatch.setattr(em, "_lib", None)
    assert em.load(build(tmp_path / "whole.so", em.EXPORTED)) is em._lib
