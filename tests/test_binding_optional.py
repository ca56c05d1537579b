"""The package without the binding's C module (built for another Python, or not
at all): the library loads, and the calls that the module speeds up are made
through ctypes."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
WITHOUT = """
import sys

class Missing:
    def find_spec(self, name, path=None, target=None):
        if name.endswith("._binding"):
            raise ImportError(name)

sys.meta_path.insert(0, Missing())
import torch
import sparse_moe_transformer_fwd_b200 as moe
"""


def _run(code):
    p = subprocess.run([sys.executable, "-c", WITHOUT + code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert p.returncode == 0 and "done" in p.stdout, p.stderr[-2000:]


def test_library_loads_and_refuses():
    _run("""
moe.lib()
assert "sparse_moe_transformer_fwd_b200._binding" not in sys.modules
assert moe.moe_workspace_size(moe.make_shape(4, 256, 8, 2, 128)) > 0
x = torch.zeros(4, 256, dtype=torch.bfloat16)
try:
    moe.moe_linear(moe.make_linear_shape(4, 256, 256), x, x, x, x, x)
except ValueError as e:
    assert "CUDA tensor" in str(e)
    print("done")
""")


@pytest.mark.gpu
def test_same_results(tmp_path):
    import torch

    import sparse_moe_transformer_fwd_b200 as moe

    code = """
g = torch.Generator("cuda").manual_seed(0)
r = lambda *s: torch.randn(*s, device="cuda", generator=g).bfloat16()
L = moe.MoELayer(r(8, 256), torch.zeros(8, device="cuda"), r(9, 256, 256) / 16, r(9, 256, 128) / 16, top_k=2)
lin = moe.Fp8Linear(r(640, 256))
x, res, gamma = r(40, 256), r(40, 640), r(256)
q, s = torch.empty(40, 256, dtype=torch.uint8, device="cuda"), torch.empty(40, 2, device="cuda")
moe.fp8_block_quant(x, 1, q, s)
outs = [lin(x, residual=res), lin.quantized(q, s), lin.forward_prenorm(x, gamma), L.forward_few(x[:3]),
        L.forward_few_prenorm(x[:3], gamma)]
assert lin.check_status(40) == 0 and L.check_status(3) == 0
"""
    here = {"moe": moe, "torch": torch}
    exec(code, here)
    path = str(tmp_path / "outs.pt")
    _run(code + "torch.save([o.cpu() for o in outs], %r)\nprint('done')\n" % path)
    for a, b in zip(torch.load(path), here["outs"]):
        assert torch.equal(a, b.cpu())
