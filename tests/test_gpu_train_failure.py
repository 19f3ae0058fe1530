"""Failure detection of the training products without a GPU fault: a process whose
wait limit is 1 ns. A wait looks at the clock after every 16 polls, which the
hardware may stretch, so only one of hundreds of microseconds is sure to give up:
the epilogue's for an accumulator over K = 65536. The kernel then sets
MOE_DEV_TIMEOUT, lets copies and MMAs in flight finish, frees its TMEM and returns;
the context stays usable. The weights' gradient has no wait that long: its
calls may give up or not, and have to end either way."""
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
new = lambda *n, dt=torch.bfloat16: torch.ones(n, dtype=dt, device="cuda")
seen = []
def product(rows, E, K, N, transposed):
    off = torch.linspace(0, rows - 3, E + 1).to(torch.int32).cuda()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, pre = new(rows, N), new(rows, N)
    W = new(E, N, K) if transposed else new(E, K, N)
    for epilogue in (None, "gelu", "gelu_grad"):
        moe.moe_expert_gemm(new(rows, K), off, W, out, transposed=transposed, epilogue=epilogue,
                            pre=None if epilogue is None else pre, dev_status=st)
        torch.cuda.synchronize()
    seen.append(int(st.item()))
def wgrad(rows, E, K, N):
    off = torch.linspace(0, rows - 3, E + 1).to(torch.int32).cuda()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    for dt in (torch.float32, torch.bfloat16):
        moe.moe_expert_wgrad(new(rows, K), new(rows, N), off, new(E, K, N, dt=dt), dev_status=st)
        torch.cuda.synchronize()
    seen.append(int(st.item()))
for case in CASES:
    (product if len(case) == 5 else wgrad)(*case)
z = (torch.ones(1024, device="cuda") * 2).sum().item()
print(json.dumps({"seen": seen, "torch_op": z}))
"""

CASES = {
    "product": [(300, 2, 65536, 256, False), (300, 2, 65536, 256, True), (4096, 3, 4096, 1024, False)],
    "wgrad": [(20000, 8, 1024, 2048), (1001, 4, 512, 512)],
    "wgrad_shared_tiles": [(20000, 1, 256, 256), (20000, 1, 1024, 1024)],
}


@pytest.mark.parametrize("name", CASES)
def test_wait_timeout_is_reported_and_context_survives(name):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    env = dict(os.environ, MOE_GB300_WAIT_TIMEOUT_NS="1")
    code = CHILD.replace("ROOT", repr(ROOT)).replace("CASES", repr(CASES[name]))
    r = subprocess.run([sys.executable, "-c", code], env=env, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    out = json.loads(r.stdout.strip().splitlines()[-1])
    assert all(s in (0, 8) for s in out["seen"]), out   # MOE_DEV_TIMEOUT and nothing else
    if name == "product":
        assert out["seen"][:2] == [8, 8], out
    assert out["torch_op"] == 2048.0      # the context is still usable
