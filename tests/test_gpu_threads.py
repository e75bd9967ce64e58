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

# calls in a loop without the interpreter between them: how many were refused
LOOPS = """
#include "qlin.h"
int loop_plan(int n, qlin_status (*f)(const int32_t*, int64_t, int64_t, void*, size_t, void*), const int32_t* ids,
              int64_t M, int64_t L, void* plan, size_t bytes, void* stream)
{
    int bad = 0;
    for (int i = 0; i < n; ++i)
        bad += f(ids, M, L, plan, bytes, stream) != QLIN_OK;
    return bad;
}
int loop_matmul(int n, qlin_status (*f)(const void*, qlin_dtype, int64_t, int64_t, const uint32_t*, const void*,
                                        const void*, qlin_dtype, int64_t, int, int, const void*, void*, void*, size_t,
                                        void*),
                const void* x, int64_t K, const uint32_t* codes, const void* scales, const void* biases, int64_t N, void* y,
                void* ws, size_t bytes, void* stream)
{
    int bad = 0;
    for (int i = 0; i < n; ++i)
        bad += f(x, QLIN_BF16, 1, K, codes, scales, biases, QLIN_BF16, N, 4, 64, 0, y, ws, bytes, stream) != QLIN_OK;
    return bad;
}
int loop_clip(int n, qlin_status (*f)(const void*, qlin_dtype, int64_t, int64_t, double, int8_t*, float*, void*),
              const void* w, int64_t R, int64_t C, int8_t* q, float* scale, void* stream)
{
    int bad = 0;
    for (int i = 0; i < n; ++i)
        bad += f(w, QLIN_F32, R, C, 99.0, q, scale, stream) != QLIN_OK;
    return bad;
}
"""


@pytest.fixture(scope="module")
def loops(tmp_path_factory):
    at = tmp_path_factory.mktemp("loops")
    (at / "loops.c").write_text(LOOPS)
    subprocess.run(["gcc", "-O2", "-shared", "-fPIC", "-I", os.path.join(os.path.dirname(HERE), "include"),
                    str(at / "loops.c"), "-o", str(at / "loops.so")], check=True)
    return str(at / "loops.so")


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


def test_plans_for_pools_of_different_sizes(loops):
    """Plans of 1024 adapters (131 KB of counters) beside plans of 2: no call takes another's shared memory away."""
    run_fresh(f"""
import ctypes as C
loop, f = C.CDLL({loops!r}).loop_plan, C.cast(ql.lib().qlin_adapters_plan, C.c_void_p)
gen = torch.Generator(device="cuda").manual_seed(3)
M, pools = 64, (1024, 2)
ids = [ref.make_ids("random", M, L, gen) for L in pools]
want = [ql.adapters_plan(i, L).buffer for i, L in zip(ids, pools)]

def body(j):
    L, s = pools[j % 2], streams[j]
    plan = torch.zeros_like(want[j % 2])
    for _ in range(20):
        gate.wait(60)
        bad = loop(500, f, C.c_void_p(ids[j % 2].data_ptr()), C.c_int64(M), C.c_int64(L), C.c_void_p(plan.data_ptr()),
                   C.c_size_t(plan.numel()), C.c_void_p(s.cuda_stream))
        s.synchronize()
        assert bad == 0, "calls refused: " + str(bad)
    a, b = (t.view(torch.int32) for t in (plan, want[j % 2]))
    n = 8 + 2 * ((L + 5) // 4 * 4)
    assert torch.equal(a[8:8 + L + 2], b[8:8 + L + 2]) and torch.equal(a[n:n + M], b[n:n + M])

at_once(body)
""", 4)


def test_layers_of_different_sizes(loops):
    """One decode kernel for a long and a short layer, and the clipping quantiser for long and short rows."""
    run_fresh(f"""
import ctypes as C
lib, L = C.CDLL({loops!r}), ql.lib()
P, I64 = C.c_void_p, C.c_int64
ptr = lambda t: P(t.data_ptr())
gen = torch.Generator(device="cuda").manual_seed(3)
rn = lambda *s: torch.randn(*s, generator=gen, device="cuda")
layers = [(*ql.quantize(rn(N, K) * 0.05, 4, 64), rn(1, K).to(BF)) for N, K in ((8192, 8192), (256, 512))]
rows = [rn(4, 16384), rn(4, 64)]

def matmul(j, n):
    codes, sc, bi, x = layers[j % 2]
    y = torch.empty(1, codes.shape[0], dtype=BF, device="cuda")
    ws = torch.empty(max(16, ql.workspace_size(ql.QLIN_OP_MATMUL, 1, y.shape[1], x.shape[1], 4, 64)), dtype=torch.uint8,
                     device="cuda")
    bad = lib.loop_matmul(n, C.cast(L.qlin_matmul, P), ptr(x), I64(x.shape[1]), ptr(codes), ptr(sc), ptr(bi),
                          I64(y.shape[1]), ptr(y), ptr(ws), C.c_size_t(ws.numel()), P(streams[j].cuda_stream))
    return y, bad

def clip(j, n):
    w = rows[j % 2]
    q, s = torch.empty(w.shape, dtype=torch.int8, device="cuda"), torch.empty(4, device="cuda")
    bad = lib.loop_clip(n, C.cast(L.qlin_quantize_weight_int8, P), ptr(w), I64(4), I64(w.shape[1]), ptr(q), ptr(s),
                        P(streams[j].cuda_stream))
    return q, bad

for call in (matmul, clip):
    torch.cuda.synchronize()
    want = [call(i, 1)[0] for i in (0, 1)]

    def body(j):
        for _ in range(10):
            gate.wait(60)
            got, bad = call(j, 500)
            streams[j].synchronize()
            assert bad == 0, call.__name__ + " calls refused: " + str(bad)
        assert torch.equal(got, want[j % 2])

    at_once(body)
""", 4)


@pytest.mark.parametrize("adapters", [300, 383])
def test_first_plan_of_a_pool(adapters):
    """Pools whose counters end about the shared memory that a kernel has without asking: 48 KB, less its own."""
    run_fresh(f"""
gen = torch.Generator(device="cuda").manual_seed(3)
ids = ref.make_ids("random", 500, {adapters}, gen)
plan = ql.adapters_plan(ids, {adapters})
n = 8 + 2 * (({adapters} + 5) // 4 * 4)
key = torch.where(ids < 0, {adapters}, ids.long())
assert torch.equal(plan.buffer.view(torch.int32)[n:n + 500].long(), torch.sort(key, stable=True).indices)
""", 1)
