"""The build without a GPU: what the extension lacks does not keep the CUDA library from being built."""
import os

import pytest

from paged_mla_speculative_tree_gb300 import build


@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    """A build of one source into a directory of its own."""
    monkeypatch.setattr(build, "OUT_DIR", str(tmp_path / "lib"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "lib" / "lib.so"))
    monkeypatch.setattr(build, "BUILD_DIR", str(tmp_path / "build"))
    monkeypatch.setattr(build, "sources", lambda: [os.path.join(build.CSRC, "rope.cu")])


def test_library_is_built_without_the_extensions_headers(elsewhere, monkeypatch, capfd):
    monkeypatch.setattr(build.sysconfig, "get_paths", lambda: {"include": "/nonexistent"})
    os.makedirs(build.OUT_DIR)
    with open(build.extension_path(), "w") as f:
        f.write("of other sources")
    os.utime(build.extension_path(), (1, 1))
    assert build.build() == build.LIB and os.path.exists(build.LIB)
    assert not os.path.exists(build.extension_path())
    assert "extension was not built" in capfd.readouterr().err
    assert not build.up_to_date()
    made = os.path.getmtime(build.LIB)
    assert build.build() == build.LIB and os.path.getmtime(build.LIB) == made  # the library is not built again
    monkeypatch.undo()


def test_a_failing_library_raises(elsewhere, monkeypatch):
    monkeypatch.setattr(build.sysconfig, "get_paths", lambda: {"include": "/nonexistent"})
    with pytest.raises(RuntimeError):
        build.build(extra=["--no-such-option"])
    assert not os.path.exists(build.LIB)


def test_extension_of_another_torch_is_not_taken(monkeypatch):
    """Inline code of torch's and Python's headers is compiled into it."""
    import torch

    from paged_mla_speculative_tree_gb300 import binding
    build.build()
    assert build.up_to_date() and os.path.exists(build.extension_path())
    monkeypatch.setattr(torch, "__version__", "0.0.0+other")
    assert not build.up_to_date() and not os.path.exists(build.extension_path())
    monkeypatch.setattr(binding, "_ext", None)
    with pytest.raises(RuntimeError, match="not built"):
        binding._extension()
    monkeypatch.undo()
    monkeypatch.setattr(build.sysconfig, "get_config_var", lambda name: "cpython-399-other")
    assert not build.up_to_date() and not os.path.exists(build.extension_path())
