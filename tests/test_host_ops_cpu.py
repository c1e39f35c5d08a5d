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


def _fake_cuda(*shape, dtype=torch.uint8, device="cuda:0"):
    """A tensor that says it is on a GPU and holds nothing: whatever reads its address fails."""
    from torch._subclasses.fake_tensor import FakeTensorMode
    with FakeTensorMode():
        return torch.empty(*shape, dtype=dtype, device=device)


@pytest.mark.skipif(torch.cuda.is_available(), reason="fake CUDA tensors: CPU only")
@pytest.mark.parametrize("change,match", [
    (dict(scales=(4, 1)), "scales must have 8 elements"), (dict(scales=(3, 2)), "scales must have 8 elements"),
    (dict(scales=(5, 2)), "scales must have 8 elements"), (dict(scales=(4, 2), sdt=torch.int8), "scales must be Byte"),
    (dict(out=(4, 32)), "out must have 256 elements"), (dict(out=(3, 64)), "out must have 256 elements"),
    (dict(out=(8, 64)), "out must have 256 elements"), (dict(odt=torch.bfloat16), "out must be Float"),
    (dict(odt=torch.float16), "out must be Float"), (dict(f32=False), "out must be BFloat16"),
    (dict(odev="cpu"), "out must be a CUDA tensor"), (dict(odev="cuda:1"), "out is on cuda:1"),
    (dict(sdev="cuda:1"), "scales is on cuda:1"), (dict(strided=True), "out must be contiguous")])
def test_dequantize_refuses_what_does_not_fit(ops, change, match):
    c = dict(dict(scales=(4, 2), sdt=torch.uint8, sdev="cuda:0", out=(4, 64), odt=torch.float32, odev="cuda:0", f32=True,
                  strided=False), **change)
    out = _fake_cuda(*c["out"], dtype=c["odt"], device=c["odev"])
    if c["strided"]:
        out = _fake_cuda(64, 4, dtype=c["odt"]).t()
    with pytest.raises(ValueError, match=match):
        ops.dequantize(_fake_cuda(4, 32), _fake_cuda(*c["scales"], dtype=c["sdt"], device=c["sdev"]), out, c["f32"])


def test_dequantize_knows_two_output_types():
    from mxfp4_block_scaled_moe_b200 import binding
    t = torch.zeros(4, 32, dtype=torch.uint8)
    with pytest.raises(ValueError, match="out_dtype"):
        binding.mxfp4_dequantize(t, t, torch.float16)


@pytest.mark.skipif(torch.cuda.is_available(), reason="fake CUDA tensors: CPU only")
@pytest.mark.parametrize("change,match", [
    (dict(scales=(4, 1)), "scales must have 8 elements"), (dict(scales=(5, 2)), "scales must have 8 elements"),
    (dict(sdt=torch.int8), "scales must be"), (dict(out=(4, 32)), "out must have 256 elements"),
    (dict(out=(8, 64)), "out must have 256 elements"), (dict(odt=torch.bfloat16), "out must be"),
    (dict(odev="cpu"), "out must be a CUDA tensor"), (dict(odev="cuda:1"), "out is on cuda:1"),
    (dict(sdev="cuda:1"), "scales is on cuda:1"), (dict(strided=True), "out must be contiguous")])
def test_dequantize_without_the_extension_refuses_the_same(monkeypatch, tmp_path, change, match):
    from mxfp4_block_scaled_moe_b200 import binding
    monkeypatch.setattr(binding, "_ops", None)
    monkeypatch.setattr(binding, "HOST_OPS_PATH", str(tmp_path / "none.so"))
    c = dict(dict(scales=(4, 2), sdt=torch.uint8, sdev="cuda:0", out=(4, 64), odt=torch.float32, odev="cuda:0",
                  strided=False), **change)
    out = _fake_cuda(*c["out"], dtype=c["odt"], device=c["odev"])
    if c["strided"]:
        out = _fake_cuda(64, 4, dtype=c["odt"]).t()
    with pytest.raises(ValueError, match=match):
        binding.mxfp4_dequantize(_fake_cuda(4, 32), _fake_cuda(*c["scales"], dtype=c["sdt"], device=c["sdev"]), out=out)


def test_operators_without_the_extension_say_so(monkeypatch, tmp_path):
    from mxfp4_block_scaled_moe_b200 import binding
    monkeypatch.setattr(binding, "_ops", None)
    monkeypatch.setattr(binding, "HOST_OPS_PATH", str(tmp_path / "none.so"))
    t = torch.zeros(4, 64)
    with pytest.raises(RuntimeError, match="none.so is missing"):
        binding.rmsnorm_residual(t, t[0])


def _small_library(build, monkeypatch, tmp_path):
    """build.build() into tmp_path, of one small source file."""
    src = tmp_path / "one.cu"
    src.write_text('extern "C" int one() { return 1; }\n')
    monkeypatch.setattr(build, "sources", lambda: [str(src)])
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "obj"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "lib.so"))
    return tmp_path / "lib.so"


def test_the_library_is_linked_when_the_extension_cannot_be_compiled(monkeypatch, tmp_path):
    from mxfp4_block_scaled_moe_b200 import build
    lib = _small_library(build, monkeypatch, tmp_path)

    def broken(force=False):
        raise RuntimeError("no Python.h")
    monkeypatch.setattr(build, "build_host_ops", broken)
    with pytest.raises(RuntimeError, match="no Python.h"):
        build.build(force=True)
    assert lib.exists()


def test_the_library_builds_without_torch(monkeypatch, tmp_path):
    from mxfp4_block_scaled_moe_b200 import build
    lib = _small_library(build, monkeypatch, tmp_path)
    real = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda n, *a: None if n == "torch" else real(n, *a))
    monkeypatch.setattr(build, "build_host_ops", lambda force=False: pytest.fail("built without torch"))
    assert build.build(force=True) == str(lib) and lib.exists()
    assert build.build() == str(lib)          # nothing to do


def test_the_extension_is_of_this_torch(ops, monkeypatch, tmp_path):
    """It says what it was compiled for; build_host_ops() compiles it anew for another torch, and the
    binding refuses one of another."""
    from mxfp4_block_scaled_moe_b200 import binding, build
    assert ops.built_for == build.host_ops_abi() and torch.__version__ in ops.built_for
    assert build._built_for(build.HOST_OPS, ops.built_for) and not build._built_for(build.HOST_OPS, "torch 9.9")
    runs = []

    def compiler(cmd, **kw):
        runs.append(cmd)
        raise RuntimeError("compiling")
    monkeypatch.setattr(build.subprocess, "run", compiler)
    assert build.build_host_ops() == build.HOST_OPS and not runs
    monkeypatch.setattr(torch, "__version__", torch.__version__ + ".other")
    with pytest.raises(RuntimeError, match="compiling"):
        build.build_host_ops()
    assert len(runs) == 1
    monkeypatch.setattr(binding, "_ops", None)
    monkeypatch.setattr(binding, "lib", lambda: None)
    with pytest.raises(RuntimeError, match="was built for torch"):
        binding._host_ops()
    assert binding._ops is None


@pytest.mark.skipif(torch.cuda.is_available(), reason="fake CUDA tensors: CPU only")
def test_a_stream_of_another_device_is_refused():
    """The operators run on their tensors' device; a stream of another one would not order them."""
    import types
    from mxfp4_block_scaled_moe_b200 import binding as B
    other = types.SimpleNamespace(device=torch.device("cuda", 1))
    t = _fake_cuda(4, 64)
    for call in (lambda: B.mxfp4_dequantize(t, t, stream=other), lambda: B.rmsnorm_residual(t, t, stream=other),
                 lambda: B.rmsnorm_residual_fp8(t, t, stream=other), lambda: B.fp8_linear_fused(t, t, 1.0, 1.0, stream=other),
                 lambda: B.mxfp4_kv_append(t, t, t, t, t, t, t, stream=other),
                 lambda: B.mxfp4_kv_attention(t, t, t, t, t, t, t, stream=other)):
        with pytest.raises(ValueError, match="the stream is on cuda:1, the tensors on cuda:0"):
            call()
