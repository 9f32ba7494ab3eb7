"""Entry points of the operators beside the attention kernels, in a process of their own, so that one that ends the process is seen as
a failure of its own test: no call reaches a GPU."""
import os
import subprocess
import sys

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


def run(text):
    """Standard output of a Python program that has the repository and the host tests' call helpers at hand."""
    env = {**os.environ, "PYTHONPATH": os.pathsep.join([os.path.dirname(HERE), HERE]), "CUDA_VISIBLE_DEVICES": ""}
    r = subprocess.run([sys.executable, "-c", text], capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0, (r.returncode, r.stdout[-1000:], r.stderr[-2000:])
    return r.stdout


@pytest.mark.parametrize("heads", [0, -1])
def test_append_without_key_heads_is_refused(heads):
    """No key heads, whatever the queries' heads: GBATTN_ERR_DIMS (a stride's reach was divided by the number of heads)."""
    out = run("import test_operators_host as t\nimport scaled_dot_product_sdpa_gb300 as gb\n"
              "from scaled_dot_product_sdpa_gb300 import build as b\nlib = gb.load_library(b.build())\n"
              f"for more in (dict(), dict(wq=None, wk=None), dict(wq=None, wk=None, q=None, qo=None, Hq=0)):\n"
              f"    print(t.append(lib, Hkv={heads}, **more) == t.code('DIMS'))\n")
    assert out.split() == ["True"] * 3, out


@pytest.mark.parametrize("lacks", ["torch._C._cuda_getCurrentRawStream torch._C._cuda_getDevice", "torch._C._dynamo", "torch._C._dynamo.guards",
                                   "torch._C._dynamo.guards._empty_strided_cuda"])
def test_the_package_is_imported_without_torch_s_private_names(lacks):
    """A torch without CUDA, or with other private names: the package is imported, and a call says what it needs."""
    drop = "".join(f"if hasattr({n.rpartition('.')[0]}, '{n.rpartition('.')[2]}'): del {n}\n" for n in lacks.split())
    out = run(f"import torch\n{drop}"
              "import scaled_dot_product_sdpa_gb300 as gb\n"
              "q = torch.zeros(1, 2, 3, 64, dtype=torch.float16)\n"
              "try:\n    gb.attn_rope(q, None, None)\nexcept ValueError as e:\n    print(e)\n"
              "print(gb.attn_rope_frequencies(64, device='cpu')[0].shape[0])\n")
    assert "must be on a CUDA device" in out and out.split()[-1] == "32", out
