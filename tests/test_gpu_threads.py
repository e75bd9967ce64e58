"""Calls from several host threads at once (ctypes lets go of the interpreter lock during a call)."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))

PRELUDE = """
import sys, threading
sys.path[:0] = [{here!r}, {root!r}]
import torch
import adapter_ref as ref
from helpers import build_lib
ql = build_lib()
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
gate, errors = threading.Barrier({threads}), []

def work(j, body):
    try:
        with torch.cuda.stream(streams[j]):
            body(j)
            streams[j].synchronize()
    except Exception as e:
        errors.append(f"{{type(e).__name__}}: {{e}}")
        gate.abort()

def at_once(body):
    torch.cuda.synchronize()
    ts = [threading.Thread(target=work, args=(j, body)) for j in range({threads})]
    [t.start() for t in ts]
    [t.join() for t in ts]
    torch.cuda.synchronize()
    assert not errors, errors
    assert ql.device_status() == ql.QLIN_OK

streams = [torch.cuda.Stream() for _ in range({threads})]
"""

def run_fresh(script, threads):
    """In a process of its own, whose first calls of a kernel are these."""
    code = PRELUDE.format(here=HERE, root=os.path.dirname(HERE), threads=threads) + script
    p = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=240)
    assert p.returncode == 0, p.stdout[-2000:] + p.stderr[-3000:]


def test_first_adapter_calls_of_eight_threads():
    """Every thread's first call of a kernel that needs more than the default shared memory, or a cluster of 16,
    at the same moment: all are launched, and give the same bits."""
    run_fresh("""
# rank 128 of few tokens (one launch), 64 scattered and consecutive tokens (two launches, 16-way split), training
for case in ((BF, 24, 4096, 1024, 2, 128, "random"), (HF, 24, 4096, 1024, 2, 128, "random"),
             (BF, 777, 8192, 512, 3, 32, "random"), (HF, 777, 8192, 512, 3, 32, "random"),
             (BF, 2000, 512, 512, 2, 64, "blocks"), (HF, 2000, 512, 512, 2, 64, "blocks")):
    d = ref.make(case)
    plan = ql.adapters_plan(d["ids"], case[4])
    got = [None] * 8

    def body(j):
        u = torch.zeros(case[1], case[5], device="cuda")
        gate.wait(60)
        out = ql.adapters_forward(d["x"], d["a"], d["b"], d["scales"], plan, base=d["base"], u=u)
        gate.wait(60)
        got[j] = (out, u, *ql.adapters_backward(d["dy"], d["a"], d["b"], d["scales"], plan, u, x=d["x"]))

    at_once(body)
    assert all(torch.equal(a, b) for g in got for a, b in zip(g, got[0]))
    ref.check_forward(d["x"], d["a"], d["b"], d["scales"], d["ids"], d["base"], got[0][0], got[0][1])
""", 8)
