"""The build's optional parts (host logic only; nothing is compiled)."""
import os

import pytest

from dynamic_shape_gemm_amd import build


class Compiler:
    """A compiler that was started."""
    args, returncode = ["g++"], 0

    def __init__(self, started):
        started.append(self)


@pytest.mark.parametrize("missing", ["all", "c10_hip", "headers", "none"])
def test_torch_without_rocm_has_no_binding(tmp_path, monkeypatch, missing):
    """A torch for the CPU alone leaves the helpers their Python form, and no module of another torch's."""
    where = tmp_path / "torch"
    (where / "include/c10/hip").mkdir(parents=True) if missing != "all" else where.mkdir()
    (where / "lib").mkdir()
    if missing in ("c10_hip", "none"):
        for h in ("HIPFunctions.h", "HIPStream.h"):
            (where / "include/c10/hip" / h).touch()
    if missing in ("headers", "none"):
        (where / "lib/libc10_hip.so").touch()
    stale = tmp_path / "_mkptorch.so"
    stale.touch()
    started = []
    monkeypatch.setattr(build, "torch_dir", lambda: str(where))
    monkeypatch.setattr(build, "DIRECT", str(stale))
    monkeypatch.setattr(build.subprocess, "Popen", lambda *a, **k: Compiler(started))
    job = build.start_torch_binding(str(tmp_path))
    if missing == "none":
        assert started == [job]
        return
    assert job is None and not started
    build.link_torch_binding(str(tmp_path), job)
    assert not os.path.exists(stale)


def test_failed_binding_is_an_error(tmp_path, monkeypatch):
    """Where the headers are there, a compile that fails does not pass silently."""
    job = Compiler([])
    job.returncode = 1
    with pytest.raises(build.subprocess.CalledProcessError):
        build.link_torch_binding(str(tmp_path), job)
