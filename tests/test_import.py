"""The binding where torch has no CUDA: what needs no device works, and the rest raises torch's error."""

import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = """
import torch
for name in [n for n in vars(torch._C) if n.startswith("_cuda_")]:
    delattr(torch._C, name)
torch.version.cuda = None
torch.backends.cuda.is_built = lambda: False
from asymmetric_kv_merging_b200 import kvs
d = kvs.make_desc(1, 8, 32, 128, 4096, kvs.BF16)
assert kvs.workspace_size(d, 32, kvs.OP_SCORE) > 0 and kvs.workspace_size(d, 0, kvs.OP_PAGES) > 0
assert kvs.plan_rounds(1000, 300, 32, 32)[-1] == 300 and kvs.page_bytes(128) == 4736
x = torch.zeros(4)
try:
    kvs.decode_attn(d, x, x, x, None, x, x, x.to(torch.uint8))
except (AssertionError, RuntimeError) as e:
    print("no device:", type(e).__name__)
"""


def test_host_functions_need_no_cuda_in_torch():
    from asymmetric_kv_merging_b200 import build
    build.build()
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")
    res = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, env=env, capture_output=True, text=True, timeout=300)
    assert res.returncode == 0 and "no device:" in res.stdout, res.stderr[-2000:]
