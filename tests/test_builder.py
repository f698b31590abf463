"""What build() makes, and when: the C library wherever nvcc is, the PyTorch
extension module for the PyTorch and Python that run.  Without a GPU; the
compilers are not called."""
import pytest
import torch

import memory_bound_normalization_rmsnorm_gb300 as gb
from memory_bound_normalization_rmsnorm_gb300 import _binding, builder


@pytest.fixture
def made(monkeypatch, tmp_path):
    """A tree of its own, and the list of what was compiled into it."""
    log = []
    for name, f in (("LIB", "libgbnorm.so"), ("TORCH_LIB", "gbnorm_torch.so"),
                    ("TORCH_STAMP", "gbnorm_torch.stamp")):
        monkeypatch.setattr(builder, name, str(tmp_path / f), raising=False)
    monkeypatch.setattr(builder, "OUT_DIR", str(tmp_path))
    monkeypatch.setattr(builder, "BUILD_DIR", str(tmp_path))

    class Done:
        returncode, stdout, stderr = 0, "", ""

    def run(cmd, **kw):
        if "-o" in cmd:
            out = cmd[cmd.index("-o") + 1]
            log.append("library" if "libgbnorm" in out else
                       "binding" if "gbnorm_torch.so" in out else "object")
            open(out, "w").close()
        return Done()

    monkeypatch.setattr(builder.subprocess, "run", run)
    return log


def test_builds_both_once(made):
    assert not builder.up_to_date()
    builder.build()
    assert made.count("library") == 1 and made.count("binding") == 1
    assert builder.up_to_date()
    made.clear()
    builder.build()
    assert not made
    builder.build(force=True)
    assert made.count("library") == 1 and made.count("binding") == 1


def test_another_torch_builds_the_extension_again(made, monkeypatch):
    builder.build()
    made.clear()
    monkeypatch.setattr(torch, "__version__", "0.0.0+other")
    assert not builder.up_to_date()
    builder.build()
    assert "library" not in made and made.count("binding") == 1
    assert builder.up_to_date()


def test_a_torch_without_cuda_gets_the_library_alone(made, monkeypatch):
    monkeypatch.setattr(torch.version, "cuda", None)
    builder.build()
    assert made.count("library") == 1 and "binding" not in made
    assert builder.up_to_date()
    made.clear()
    builder.build()
    assert not made


def test_a_failed_extension_leaves_the_library_built(made, monkeypatch):
    def fail():
        raise RuntimeError("no compiler")

    monkeypatch.setattr(builder, "_torch_compile", fail)
    with pytest.raises(RuntimeError, match="no compiler"):
        builder.build()
    assert made.count("library") == 1 and not builder.up_to_date()
    made.clear()
    with pytest.raises(RuntimeError, match="no compiler"):
        builder.build()
    assert "library" not in made  # it is not compiled again


def test_a_module_of_another_torch_is_not_loaded(monkeypatch):
    if torch.version.cuda is None:
        pytest.skip("no extension module")
    gb.lib()
    monkeypatch.setattr(_binding, "_native_module", None)
    monkeypatch.setattr(torch, "__version__", "0.0.0+other")
    with pytest.raises(RuntimeError, match="build it again"):
        gb.norm_dropout(torch.ones(8), 0.1, 1)
    monkeypatch.undo()
    with pytest.raises(ValueError):  # loaded, and refuses a CPU tensor
        gb.norm_dropout(torch.ones(8), 0.1, 1)
