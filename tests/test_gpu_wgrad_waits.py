"""The weights' gradient under a wait limit that is shorter than the kernel and
longer than any one stage. Only the last expert's segment ends inside a K step, so
the warp that writes zeros behind segments has nothing to do for nearly all of the
call: a limit on one wait must not count that time. Rows of ones give whole numbers,
which every order of fp32 additions keeps exactly; the rows behind the segments are
NaN.

A stage takes well under a microsecond of the tensor core's time and a few from a
cold start; the calls take 5 ms and more (18 TFLOP; 8 M rows through four pairs)."""
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
