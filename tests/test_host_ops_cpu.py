"""The native host side refuses what does not fit before anything is launched (no GPU: every
tensor here is a CPU tensor, or no tensor at all, and no entry point is handed over)."""
import importlib.util
import os

import pytest
import torch

PKG = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mxfp4_block_scaled_moe_b200")


@pytest.fixture(scope="module")
def ops():
    from mxfp4_block_scaled_moe_b200 import build
    build.build()
    spec = importlib.util.spec_from_file_location("_host_ops", os.path.join(PKG, "_host_ops.so"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


ARGS = {"norm": 9, "linear": 8, "append": 7, "attention": 12, "dequantize": 4}


@pytest.mark.parametrize("name", sorted(ARGS))
def test_argument_counts_and_types(ops, name):
    f, n = getattr(ops, name), ARGS[name]
    for k in (0, n - 1, n + 1):
        with pytest.raises(TypeError, match=f"takes {n} arguments"):
            f(*[None] * k)
    with pytest.raises(TypeError, match="must be a torch.Tensor"):
        f(*[None] * n)
    with pytest.raises(TypeError, match="must be a torch.Tensor"):
        f(*["x"] * n)


@pytest.mark.parametrize("name", sorted(ARGS))
def test_cpu_tensors_are_refused(ops, name):
    t = torch.zeros(4, 64, dtype=torch.uint8)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        getattr(ops, name)(*[t] * ARGS[name])


def test_setup_wants_every_entry_point(ops):
    with pytest.raises(RuntimeError, match="no entry point"):
        ops.setup(print, {})


def test_the_binding_hands_over_the_library_s_own_entry_points():
    from mxfp4_block_scaled_moe_b200 import binding
    src = open(os.path.join(PKG, "csrc", "host_ops.cpp")).read()
    import re
    asked = re.findall(r'address\("(\w+)"\)', src)
    assert len(asked) == 6 and set(asked) <= set(binding._SIGS)
