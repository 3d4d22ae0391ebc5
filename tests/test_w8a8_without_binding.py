"""The package without its compiled binding: it imports, with a warning, and the 8-bit calls go to the same
library by the checked way; a binding that does not compile does not stop the build.
"""
import importlib.util
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
torch = pytest.importorskip("torch")
rl = pytest.importorskip("rotated_linear_amd", reason="libparo.so not built")

WITHOUT = """
import sys, types, warnings
kind = sys.argv[1]
if kind == "missing":
    sys.modules["rotated_linear_amd._binding"] = None  # importing it raises ImportError
elif kind == "other torch":
    stale = types.ModuleType("rotated_linear_amd._binding")
    stale.torch_version = "0.1.2"
    sys.modules["rotated_linear_amd._binding"] = stale
else:
    sys.modules["rotated_linear_amd._binding"] = types.ModuleType("rotated_linear_amd._binding")  # names no version
with warnings.catch_warnings(record=True) as said:
    warnings.simplefilter("always")
    import rotated_linear_amd as rl
said = [str(w.message) for w in said if "without its compiled binding" in str(w.message)]
assert len(said) == 1 and "more host time" in said[0], said
import torch
assert len(rl.paro_rotation_encode([[[0, 1], [2, 3]] + [[2 * i, 2 * i + 1] for i in range(2, 64)]], [[0.0] * 64], [1.0] * 128))
assert rl.paro_w8a8_workspace_bytes(1, 256, 16) == 0
x, q, s = torch.zeros(2, 256, dtype=torch.float16), torch.zeros(2, 256, dtype=torch.int8), torch.zeros(2)
for call in (lambda: rl.paro_rmsnorm(x, x[0]), lambda: rl.paro_rmsnorm_q8(x, x[0]), lambda: rl.paro_quantize_q8(x),
             lambda: rl.paro_pack_weights_q8(x), lambda: rl.paro_dequantize_q8(q, s), lambda: rl.paro_w8a8_linear(q, s, q, s),
             lambda: rl.paro_w8a8_gated_linear(q, s, q, s)):
    try:
        call()
    except ValueError as e:
        assert "must live on the GPU" in str(e)
    else:
        raise AssertionError("taken on the CPU")
print("without")
"""


@pytest.mark.parametrize("kind", ["missing", "other torch", "no version"])
def test_imports_without_the_binding(kind):
    r = subprocess.run([sys.executable, "-c", WITHOUT, kind], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "without", r.stdout + r.stderr


def test_the_binding_names_the_torch_it_was_built_for():
    from rotated_linear_amd import _binding

    assert _binding.torch_version == torch.__version__.split("+")[0]


def test_a_pre_release_of_torch_keeps_the_binding():
    """Its headers name 1.2.3 where torch itself says 1.2.3.dev4+5 or 1.2.3a0."""
    run = """
import sys, warnings, torch
torch.__version__ = torch.__version__.split("+")[0] + sys.argv[1]
warnings.simplefilter("error")
import rotated_linear_amd.w8a8 as w
print(w._binding.__name__)
"""
    for tail in (".dev20300101+rocm9", "a0+git1234"):
        r = subprocess.run([sys.executable, "-c", run, tail], cwd=ROOT, capture_output=True, text=True, timeout=300)
        assert r.stdout.strip() == "rotated_linear_amd._binding", r.stdout + r.stderr


@pytest.mark.parametrize("broken", ["source", "compiler"])
def test_a_binding_that_does_not_compile_does_not_stop_the_build(broken, tmp_path, monkeypatch):
    spec = importlib.util.spec_from_file_location("build_under_test", os.path.join(ROOT, "rotated_linear_amd", "_build.py"))
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    src, out = tmp_path / "binding.cpp", tmp_path / "_binding.so"
    src.write_text("#error no\n")
    out.write_text("an older build")
    monkeypatch.setattr(b, "BINDING_SRC", str(src))
    monkeypatch.setattr(b, "BINDING", str(out))
    if broken == "compiler":
        def run(cmd, **_):
            raise FileNotFoundError(cmd[0])
        monkeypatch.setattr(b.subprocess, "run", run)
    with pytest.warns(RuntimeWarning, match="binding was not built"):
        assert b._compile_binding() is False
    assert not out.exists()


@pytest.mark.gpu
def test_the_same_results_without_the_binding(monkeypatch):
    from rotated_linear_amd import w8a8

    torch.manual_seed(5)
    x = torch.randn(40, 512, device="cuda").half()
    g = torch.ones(512, dtype=torch.float16, device="cuda")

    def run():
        w, ws = rl.paro_pack_weights_q8(x[:32].clone())
        q, s, h = rl.paro_rmsnorm_q8(x, g, residual=x)
        p, ps = rl.paro_quantize_q8(x)
        return [w, ws, q, s, h, p, ps, rl.paro_rmsnorm(x, g)[0], rl.paro_dequantize_q8(q, s), rl.paro_w8a8_linear(q, s, w, ws),
                rl.paro_w8a8_gated_linear(q, s, w, ws, torch.float32)]

    want = run()

    class Declines:
        linear = quantize = dequantize = rmsnorm = staticmethod(lambda *_: None)

    monkeypatch.setattr(w8a8, "_binding", Declines)
    for a, b in zip(run(), want):
        assert torch.equal(a, b)
    torch.cuda.synchronize()
