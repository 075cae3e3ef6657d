"""When the native binding is compiled again (its compiler and linker stand in)."""

import os

import torch

from paged_decode_attention_fp8_gb300 import build as b


def test_another_torch_rebuilds_the_binding(tmp_path, monkeypatch):
    src, out, calls = tmp_path / "csrc", tmp_path / "_build", []
    src.mkdir(), out.mkdir()
    (src / "binding.cpp").write_text("")
    monkeypatch.setattr(b, "CSRC", str(src))
    monkeypatch.setattr(b, "BUILD", str(out))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(b, "BINDING", str(tmp_path / "_binding.so"))
    (tmp_path / "lib.so").write_text("")

    def touch(path):
        with open(path, "w"):
            os.utime(path)

    monkeypatch.setattr(b, "_compile_binding", lambda s, o: (calls.append("compile"), touch(o)))
    monkeypatch.setattr(b, "_link_binding", lambda o: (calls.append("link"), touch(b.BINDING)))
    b.build()
    assert calls == ["compile", "link"]
    b.build()
    assert calls == ["compile", "link"]
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    b.build()
    assert calls == ["compile", "link"] * 2
    b.build()
    assert calls == ["compile", "link"] * 2
    # a build that stopped before the link is not taken for done
    monkeypatch.setattr(torch, "__version__", "0.0.2")
    monkeypatch.setattr(b, "_link_binding", lambda o: (_ for _ in ()).throw(RuntimeError("no linker")))
    for _ in range(2):
        try:
            b.build()
        except RuntimeError as e:
            assert "no linker" in str(e)
        else:
            raise AssertionError("built without a linker")
    assert calls == ["compile", "link"] * 2 + ["compile"] * 2
