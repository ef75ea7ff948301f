"""GPU: block_attention over block tables whose bitmap of blocks, with the lists
kernel's own shared memory, ends just past 48 KB.  In a process of its own: a kernel
keeps the shared memory that an earlier call with a longer table asked for."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CHILD = """
import sys
import torch
from block_sparse_attention_select_gb300 import qsa

tokens, page, rows, hkv, group, D = int(sys.argv[1]), 128, 70, 2, 2, 128
g = torch.Generator(device="cuda").manual_seed(5)
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
table = (torch.arange(tokens // page, dtype=torch.int32, device="cuda") % 37)[None].contiguous()
kv = torch.randn(2, 37, page, hkv, D, generator=g, device="cuda", dtype=torch.float16)
cache = qsa.KVCache(kv[0], kv[1], table)
q = torch.randn(rows, hkv * group, D, generator=g, device="cuda", dtype=torch.float16)
sel = torch.randint(0, tokens // 128 - 1, (rows, hkv, 5), generator=g, device="cuda", dtype=torch.int32)
out = qsa.block_attention(q, sel, i32([0, rows]), i32([tokens - rows]), cache, recent=1)
assert qsa.last_launch_count() == 3 and qsa.get_device_status() == qsa.QSA_OK
for r in (0, 33, rows - 1):
    p = tokens - rows + r
    for h in range(hkv):
        blocks = sorted(set(sel[r, h].tolist()) | {p // 128})
        t = torch.cat([torch.arange(128 * c, min(128 * c + 128, p + 1), device="cuda") for c in blocks])
        k, v = (kv[i][t // page % 37, t % page, h].double() for i in (0, 1))
        for e in range(group):
            w = torch.softmax(k @ q[r, h * group + e].double() * D ** -0.5, 0)
            want, mag = w @ v, w @ v.abs()
            off = (out[r, h * group + e].double() - want).abs()
            # the output's and the weights' rounding to FP16, as in the other tests of the call
            assert torch.all(off <= 2.0 ** -11 * want.abs() + 2.0 ** -10 * mag + len(t) * 2.0 ** -25 * 6 + 2.0 ** -25)
"""


@pytest.mark.parametrize("tokens", [24117248, 24117248 + 128, 24500096, 25165824, 25165824 + 128])
def test_tables_whose_bitmap_ends_near_48_kb(tokens):
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([ROOT, os.environ.get("PYTHONPATH", "")]))
    r = subprocess.run([sys.executable, "-c", CHILD, str(tokens)], env=env, cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
