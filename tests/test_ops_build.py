"""The C library is built with nvcc alone: what stops the Python calls of the
training-step operators does not stop it, and is told at their first use."""
import pytest

from weight_communication_gb300 import binding, build


@pytest.fixture
def folder(tmp_path, monkeypatch):
    """A build of one small file into a folder of its own, with an older module."""
    src = tmp_path / "one.cu"
    src.write_text('extern "C" __attribute__((visibility("default"))) int one() { return 1; }\n')
    monkeypatch.setattr(build, "sources", lambda: [src])
    monkeypatch.setattr(build, "BUILD", tmp_path)
    for name, file in (("LIB", "libwc.so"), ("CALLS", "wc_calls.so"), ("CALLS_LOG", "calls.log")):
        monkeypatch.setattr(build, name, tmp_path / file, raising=False)
    build.CALLS.write_text("older")
    return tmp_path


@pytest.mark.parametrize("error", [ImportError("No module named 'torch'"),
                                   RuntimeError("the compiler failed on calls.cpp: Python.h: No such file"),
                                   FileNotFoundError("c++")], ids=lambda e: type(e).__name__)
def test_library_without_the_python_calls(folder, monkeypatch, capsys, error):
    def stopped():
        raise error
    monkeypatch.setattr(build, "_compile_calls", stopped)
    assert build.build() == build.LIB and build.LIB.exists()
    assert not build.CALLS.exists()
    assert "are not" in capsys.readouterr().err
    monkeypatch.setattr(binding, "_calls", None)
    monkeypatch.setattr(binding, "load", lambda: None)
    with pytest.raises(RuntimeError, match="wc_calls.so is missing.*stopped at") as e:
        binding.calls()
    assert str(error) in str(e.value)


def test_library_with_the_python_calls(folder, monkeypatch, capsys):
    def compiled():
        (folder / "new").write_text("new")
        return folder / "new"
    monkeypatch.setattr(build, "_compile_calls", compiled)
    build.build()
    assert build.LIB.exists() and build.CALLS.read_text() == "new"
    assert build.CALLS_LOG.read_text() == "" and capsys.readouterr().err == ""
