"""When the build makes the C++ binding again: it is tied to torch and Python, not to its sources alone."""
import os

import pytest


@pytest.fixture
def native(monkeypatch, tmp_path):
    """The build with a fake compiler; returns the module and the list of what it was asked to make."""
    from block_circulant_layers_b200 import build
    made = []

    def run(cmd, verbose):
        out = cmd[cmd.index("-o") + 1]
        made.append(os.path.basename(out))
        with open(out, "w"):
            pass
        return ""

    monkeypatch.setattr(build, "_run", run)
    monkeypatch.setattr(build, "_nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    monkeypatch.setattr(build, "generate", lambda: None)
    for name in ("LIB", "NATIVE", "NATIVE_ABI", "EMU", "BUILD"):
        monkeypatch.setattr(build, name, str(tmp_path / os.path.basename(getattr(build, name, name))), raising=False)
    return build, made


def count(made, name):
    return sum(m.startswith(name) for m in made)


def test_the_binding_is_made_again_for_another_torch(native, monkeypatch):
    build, made = native
    build.build()
    assert count(made, "_native.so") == 1
    build.build()
    assert count(made, "_native.so") == 1                     # nothing changed
    import torch
    monkeypatch.setattr(torch, "__version__", "0.0.0+other")
    build.build()
    assert count(made, "_native.so") == 2 and count(made, "librdfft.so") == 1
    build.build()
    assert count(made, "_native.so") == 2


def test_force_makes_everything_again_once(native):
    build, made = native
    build.build()
    del made[:]
    build.build(force=True)
    assert count(made, "_native.so") == 1 and count(made, "librdfft.so") == 1
    assert count(made, "librdfft_hostemu.so") == 1
    del made[:]
    assert build.main(["--force"]) == 0
    assert count(made, "_native.so") == 1 and count(made, "librdfft.so") == 1
