"""The waits of the weights' gradient, in processes with a limit of their own.

A limit that is shorter than the kernel and longer than any one stage. Only the last
expert's segment ends inside a K step, so the warp that writes zeros behind segments
has nothing to do for nearly all of the call: a limit on one wait must not count that
time. Rows of ones give whole numbers, which every order of fp32 additions keeps
exactly; the rows behind the segments are NaN.

A stage takes well under a microsecond of the tensor core's time and a few from a
cold start; the calls take 5 ms and more (18 TFLOP; 8 M rows through four pairs).

A limit of 1 ns. The warp that writes zeros waits for the first segment's end to come
from HBM, about a microsecond and tens of looks at the barrier: it gives up in every
call that has a segment which ends inside a K step. The kernel then sets MOE_DEV_TIMEOUT, lets copies and MMAs in flight finish,
frees its TMEM and returns, and the context stays usable."""
import json
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import json, sys
sys.path.insert(0, ROOT)
import torch
import top_routing_expert_gb300 as moe
moe.build(); moe.load_library()
lengths, K, N = CASE
off = torch.tensor([0] + lengths).cumsum(0).to(torch.int32).cuda()
rows = sum(lengths) + 5
x, g = (torch.ones(rows, n, dtype=torch.bfloat16, device="cuda") for n in (K, N))
x[rows - 5:], g[rows - 5:] = float("nan"), float("inf")
dW = torch.full((len(lengths), K, N), 7.0, device="cuda")
st = torch.zeros(1, dtype=torch.int32, device="cuda")
moe.moe_expert_wgrad(x, g, off, dW, dev_status=st)
right = [bool((dW[e] == n).all()) for e, n in enumerate(lengths)]
print(json.dumps({"status": int(st.item()), "right": right}))
"""

CASES = {
    "full_expert_before_a_cut_one": ([131072, 1001], 8192, 8192),
    "shared_tile": ([8 * 2 ** 20 + 1], 64, 64),
}


@pytest.mark.parametrize("name", CASES)
def test_limit_counts_one_stage_at_a_time(name):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    env = dict(os.environ, MOE_GB300_WAIT_TIMEOUT_NS="300000")
    code = CHILD.replace("ROOT", repr(ROOT)).replace("CASE", repr(CASES[name]))
    r = subprocess.run([sys.executable, "-c", code], env=env, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    out = json.loads(r.stdout.strip().splitlines()[-1])
    assert out["status"] == 0 and all(out["right"]), out


GIVE_UP = r"""
import json, sys
sys.path.insert(0, ROOT)
import torch
import top_routing_expert_gb300 as moe
moe.build(); moe.load_library()
seen = []
for rows, E, K, N in CASES:
    off = torch.linspace(0, rows - 3, E + 1).to(torch.int32).cuda()
    x, g = (torch.ones(rows, n, dtype=torch.bfloat16, device="cuda") for n in (K, N))
    for dt, accumulate in ((torch.float32, False), (torch.float32, True), (torch.bfloat16, False)):
        dW = torch.ones(E, K, N, dtype=dt, device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        moe.moe_expert_wgrad(x, g, off, dW, accumulate=accumulate, dev_status=st)
        seen.append(int(st.item()))
z = (torch.ones(1024, device="cuda") * 2).sum().item()
print(json.dumps({"seen": seen, "torch_op": z}))
"""

# rows, E, K, N: unsplit, down to one row; tiles shared by four pairs and by two
LIMIT_1NS = [(20000, 8, 1024, 2048), (999, 4, 512, 512), (17 * 8 + 3, 8, 512, 512), (4, 1, 64, 64),
             (20000, 1, 256, 256), (20000, 1, 1024, 1024)]


def test_waits_give_up():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    env = dict(os.environ, MOE_GB300_WAIT_TIMEOUT_NS="1")
    code = GIVE_UP.replace("ROOT", repr(ROOT)).replace("CASES", repr(LIMIT_1NS))
    r = subprocess.run([sys.executable, "-c", code], env=env, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    out = json.loads(r.stdout.strip().splitlines()[-1])
    assert out["seen"] == [8] * (3 * len(LIMIT_1NS)), out   # MOE_DEV_TIMEOUT and nothing else
    assert out["torch_op"] == 2048.0                        # the context is still usable
