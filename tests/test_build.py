"""The library's build does not hang on the Python binding's, and the binding is
made again for another torch: with stand-ins for the compilers."""

import os
import stat

import pytest


@pytest.fixture
def b(tmp_path, monkeypatch):
    from decode_attention_paged_kv_gb300 import build as m
    out = tmp_path / "out"
    for name in ("LIB", "BINDING", "BINDING_STAMP"):
        monkeypatch.setattr(m, name, str(out / os.path.basename(getattr(m, name))))
    monkeypatch.setattr(m, "BUILD", str(out))
    for tool in ("NVCC", "CXX"):
        path = tmp_path / "bin" / tool
        path.parent.mkdir(exist_ok=True)
        # writes its -o file and a line of log; fails if told to
        path.write_text(f'#!/bin/sh\necho x >> {tmp_path}/{tool}.log\n[ -e {tmp_path}/fail_{tool} ]'
                        ' && exit 1\nwhile [ "$1" != -o ]; do shift; done\necho > "$2"\n')
        path.chmod(path.stat().st_mode | stat.S_IXUSR)
        monkeypatch.setattr(m, tool, str(path))
    m.runs = lambda tool: (len((tmp_path / f"{tool}.log").read_text().split())
                           if (tmp_path / f"{tool}.log").exists() else 0)
    m.tmp = tmp_path
    yield m
    del m.runs, m.tmp


def test_library_without_binding(b):
    (b.tmp / "fail_CXX").touch()
    with pytest.raises(RuntimeError, match="binding"):
        b.build()
    assert os.path.exists(b.LIB) and not os.path.exists(b.BINDING)
    n = b.runs("NVCC")
    assert n == len(b.sources()) + 1
    # and the binding alone afterwards
    (b.tmp / "fail_CXX").unlink()
    assert b.needs_build()
    assert b.build() == b.LIB and os.path.exists(b.BINDING)
    assert b.runs("NVCC") == n and not b.needs_build()


def test_another_torch(b, monkeypatch):
    import torch
    b.build()
    n, c = b.runs("NVCC"), b.runs("CXX")
    b.build()
    assert (b.runs("NVCC"), b.runs("CXX")) == (n, c)
    monkeypatch.setattr(torch, "__version__", "0.0.0")
    assert b.needs_build()
    b.build()
    assert (b.runs("NVCC"), b.runs("CXX")) == (n, c + 2) and not b.needs_build()


def test_library_fails(b):
    (b.tmp / "fail_NVCC").touch()
    with pytest.raises(RuntimeError, match="nvcc for"):
        b.build()
    assert not os.path.exists(b.LIB) and b.needs_build()
