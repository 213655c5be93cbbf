"""bench.py's check that a committed traffic summary belongs to the kernels that run (CPU only)."""

import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import bench  # noqa: E402
from chunked_gated_delta_amd import build  # noqa: E402

MODES = list(bench.KERNEL_SRCS)


@pytest.mark.parametrize("mode", MODES)
def test_other_operators_do_not_invalidate_a_modes_traffic(mode, monkeypatch):
    """Another source in the library, and how that one is compiled, are not this mode's kernels."""
    before = bench.kernel_source_hash(mode)
    monkeypatch.setattr(build, "SOURCES", [*build.SOURCES, "another.hip"])
    monkeypatch.setitem(build.SOURCE_FLAGS, "another.hip", ["-O1"])
    assert bench.kernel_source_hash(mode) == before
    src = os.path.join(build.HERE, "build.py")
    real = open

    def changed(path, *a, **k):  # the build script with another line in it
        if os.path.abspath(str(path)) == src:
            path = os.devnull
        return real(path, *a, **k)
    monkeypatch.setattr("builtins.open", changed)
    assert bench.kernel_source_hash(mode) == before


@pytest.mark.parametrize("mode", MODES)
def test_flags_that_shape_its_kernels_do(mode, monkeypatch):
    before = bench.kernel_source_hash(mode)
    own = [f for f in bench.KERNEL_SRCS[mode] if f.endswith(".hip")][0]
    with monkeypatch.context() as m:
        m.setitem(build.SOURCE_FLAGS, own, [*build.SOURCE_FLAGS.get(own, []), "-mllvm", "-amdgpu-early-inline-all"])
        assert bench.kernel_source_hash(mode) != before
    with monkeypatch.context() as m:
        m.setattr(build, "FLAGS", [*build.FLAGS, "-ffast-math"])
        assert bench.kernel_source_hash(mode) != before
    with monkeypatch.context() as m:  # where the tree lies is no part of it
        m.setattr(build, "FLAGS", [f.replace(build.ROOT, "/elsewhere") for f in build.FLAGS])
        assert bench.kernel_source_hash(mode) == before
