"""Two host threads make a process's first calls of the operators together, each on a stream of
its own: the outputs are those of one thread."""

import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = """
import threading
import torch
import moe_expert_ffn_scan_gb300 as moe

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32
g = torch.Generator(device="cuda").manual_seed(1)
r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF16)
new = lambda *s, dt=BF16: torch.empty(*s, dtype=dt, device="cuda")
shapes = [(2048, 2560, 2048), (256, 2304, 4096), (7, 1024, 512), (600, 1031, 77)]
ops = [(r(M, K), r(N, K)) for M, N, K in shapes]
x, gain = r(700, 1024), r(1024)
logits = r(500, 61).float()
idx = torch.topk(logits, 3, dim=1).indices.to(I32)
torch.cuda.synchronize()


def calls(stream):
    out = []
    for a, b in ops:
        M, N, K = a.shape[0], b.shape[0], a.shape[1]
        y = new(M, N)
        moe.moe_linear(a, b, y, moe.alloc_workspace(moe.linear_workspace_size(M, N, K)))
        dx, dw = new(M, K), new(N, K)
        ws = moe.alloc_workspace(moe.linear_backward_workspace_size(M, N, K))
        moe.moe_linear_backward(a, b, y, ws, dx=dx, dw=dw)
        out += [y, dx, dw]
    y, rstd, dh, dg = new(700, 1024), new(700, dt=F32), new(700, 1024), new(1024, dt=F32)
    moe.moe_add_rmsnorm(x, None, gain, 1e-6, y=y, rstd=rstd)
    ws = moe.alloc_workspace(moe.add_rmsnorm_backward_workspace_size(700, 1024))
    moe.moe_add_rmsnorm_backward(y, x, gain, rstd, ws, dh=dh, dgain=dg)
    c, n, p = new(1, 61, dt=I32), new(1, dt=I32), new(1, 61, dt=F32)
    loss, dl, one = new(1, dt=F32), new(500, 61, dt=F32), torch.ones(1, device="cuda")
    ws = moe.alloc_workspace(moe.balance_loss_workspace_size(500, 61, 3))
    moe.moe_balance_loss(logits, idx, c, n, p, loss, None, ws)
    moe.moe_balance_loss_backward(logits, idx, c, n, dl, dloss=one)
    return out + [y, rstd, dh, dg, c, n, p, loss, dl]


both, got, errors = threading.Barrier(2), [None, None], []


def work(i):
    try:
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            both.wait()
            got[i] = calls(st)
        st.synchronize()
    except Exception as e:
        errors.append(e)


threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
[t.start() for t in threads]
[t.join() for t in threads]
assert not errors, errors
want = calls(None)
torch.cuda.synchronize()
for i in range(2):
    assert len(got[i]) == len(want) and all(torch.equal(a, b) for a, b in zip(got[i], want))
print("same")
"""


def test_first_calls_of_two_threads():
    r = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("same"), r.stdout + r.stderr
