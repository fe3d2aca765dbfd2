"""What the build is given: MAX_JOBS of any text, and flags for compiling and for linking."""

import pytest

from gaussian_splatting_differentiable_ewa_amd import build


@pytest.fixture
def commands(monkeypatch):
    """The commands that a build would run."""
    ran = []
    monkeypatch.setattr(build, "_run", lambda cmd, verbose: ran.append(cmd))
    monkeypatch.setattr(build.os, "replace", lambda a, b: None)
    return ran


@pytest.mark.parametrize("jobs", [None, "", "0", "1", "4", "many", "-2"])
def test_max_jobs(commands, monkeypatch, jobs):
    if jobs is None:
        monkeypatch.delenv("MAX_JOBS", raising=False)
    else:
        monkeypatch.setenv("MAX_JOBS", jobs)
    assert build.build() == build.LIB
    assert len(commands) == len(build.sources()) + 1


def test_extra_flags_reach_every_command(commands):
    build.build(extra=["-save-temps=obj", "-lm"])
    assert "-shared" in commands[-1] and not any("-shared" in c for c in commands[:-1])
    for c in commands:
        assert "-save-temps=obj" in c and "-lm" in c, c
