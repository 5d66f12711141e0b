"""CPU test of the build's number of compilers at a time (none is run here)."""
import pytest

from dtensor_layout_movement_amd import build as B


@pytest.mark.parametrize("given", [None, "", "0", "-3", "many", "1.5", " 2 ", "4", "100"])
def test_the_build_takes_any_max_jobs(given, monkeypatch, tmp_path):
    """A number of jobs that is none is no reason not to build."""
    if given is None:
        monkeypatch.delenv("MAX_JOBS", raising=False)
    else:
        monkeypatch.setenv("MAX_JOBS", given)
    made = []

    def run(cmd, verbose):
        made.append(cmd[cmd.index("-o") + 1])
        open(made[-1], "wb").close()

    monkeypatch.setattr(B, "hipcc", lambda: "hipcc")
    monkeypatch.setattr(B, "_run", run)
    monkeypatch.setattr(B, "LIB_PATH", str(tmp_path / "lib.so"))
    assert B.build() == str(tmp_path / "lib.so")
    assert len(made) == len(B.SOURCES) + 1 and (tmp_path / "lib.so").exists()
