"""The build of the C library where there is no torch (io_aware_exact_22_b200/build.py)."""
import ctypes
import sys

from io_aware_exact_22_b200 import build


def test_the_library_builds_without_torch(tmp_path, monkeypatch, capsys):
    # a source of its own, so that nothing of the tree is built anew
    src, out = tmp_path / "csrc", tmp_path / "out"
    src.mkdir()
    (src / "one.cu").write_text('extern "C" int one() { return 1; }\n')
    monkeypatch.setattr(build, "CSRC", str(src))
    monkeypatch.setattr(build, "BUILD", str(out))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(build, "EXT", str(tmp_path / "_fa_torch.so"))
    monkeypatch.setitem(sys.modules, "torch", None)  # import torch: ImportError
    assert build.build() == str(tmp_path / "lib.so")
    assert ctypes.CDLL(str(tmp_path / "lib.so")).one() == 1
    assert not (tmp_path / "_fa_torch.so").exists()
    err = capsys.readouterr().err
    assert "_fa_torch.so" in err and "torch" in err
