"""The modules of many adapters without a GPU: what conversions and copies do to their state."""
import copy

import pytest
import torch


@pytest.fixture(scope="module")
def many():
    from block_circulant_layers_b200 import build
    build.build()
    from block_circulant_layers_b200 import many
    return many


@pytest.mark.parametrize("convert", ["bfloat16", "half", "double", "to", "to_device_and_dtype"])
def test_the_scale_keeps_its_value_in_any_dtype(many, convert):
    """alpha / r = 8 / 24 is no bf16 number: a rounded scale would change every output by up to 2^-9."""
    bank = many.LowRankAdapters(2, 64, 72, 24, alpha=8.0)
    with torch.no_grad():
        bank.scale[1] = 0.1                                   # a scale of its own for one adapter
    want = torch.tensor([8.0 / 24.0, 0.1], dtype=torch.float32)
    if convert == "to":
        bank.to(torch.bfloat16)
    elif convert == "to_device_and_dtype":
        bank.to("cpu", torch.bfloat16)
    else:
        getattr(bank, convert)()
    assert bank.a.dtype == bank.b.dtype != torch.float32
    assert bank.scale.dtype == torch.float32 and torch.equal(bank.scale, want)
    bank.float()
    assert torch.equal(bank.scale, want)
    assert torch.equal(copy.deepcopy(bank).scale, want)
    again = many.LowRankAdapters(2, 64, 72, 24)
    again.load_state_dict(bank.state_dict())
    assert torch.equal(again.scale, want)


def test_the_scale_follows_the_device(many):
    bank = many.LowRankAdapters(2, 64, 72, 24, alpha=8.0).to("meta", torch.bfloat16)
    assert bank.scale.device.type == "meta" and bank.scale.dtype == torch.float32
    bank = torch.nn.Sequential(many.LowRankAdapters(2, 64, 72, 24, alpha=8.0)).to(torch.bfloat16)
    assert bank[0].scale.dtype == torch.float32 and float(bank[0].scale[0]) == float(torch.tensor(8.0 / 24.0))


def test_the_older_calls_work_without_the_cpp_binding(many):
    """A _native module that does not load (torch has changed, say) leaves the ctypes calls usable; the
    calls that need it say what to do."""
    import subprocess
    import sys

    from conftest import ROOT
    code = """
import sys
sys.modules["block_circulant_layers_b200._native"] = None     # importing it raises ImportError
import torch, block_circulant_layers_b200 as rd
assert rd.circ_bwd_workspace_size(64, 1024, 128, torch.float32) > 0
rd.BlockCirculantLinear(128, 64)
rd.LowRankAdapters(2, 64, 64, 8)
for call in (lambda: rd.adapter_plan(torch.zeros(4, dtype=torch.int32), 2), lambda: rd.grad_norm([torch.zeros(4)])):
    try:
        call()
    except ImportError as e:
        assert "block_circulant_layers_b200.build" in str(e), e
    else:
        raise AssertionError("no error")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
