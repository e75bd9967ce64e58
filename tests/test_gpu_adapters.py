"""Low-rank adapters of many requests: plan, forward and backward against 64 bits (adapter_ref has the bounds)."""
import ctypes as C

import pytest
import torch

import adapter_ref as ref
from helpers import build_lib

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def ql():
    return build_lib()


# dtype, tokens, K, N, adapters, rank, ids
CASES = [
    (BF, 1, 64, 64, 1, 8, "one"), (BF, 1, 4096, 512, 3, 16, "one"), (HF, 1, 72, 4096, 2, 24, "one"),
    (BF, 2, 512, 264, 2, 16, "random"), (HF, 7, 520, 1000, 5, 32, "random"), (BF, 8, 1024, 128, 1, 64, "one"),
    (BF, 9, 136, 264, 4, 40, "random"), (HF, 16, 256, 512, 16, 8, "random"), (BF, 17, 1000, 72, 3, 128, "random"),
    (BF, 61, 512, 1376, 33, 16, "random"), (BF, 64, 264, 264, 2, 48, "none"), (HF, 127, 512, 520, 1, 16, "one"),
    (BF, 128, 640, 256, 2, 32, "one"), (BF, 129, 512, 264, 4, 64, "even"), (HF, 300, 384, 776, 3, 8, "runs"),
    (BF, 300, 1032, 520, 6, 72, "outside"), (BF, 777, 512, 640, 12, 32, "random"), (HF, 1000, 640, 384, 2, 96, "runs"),
    (BF, 1531, 1024, 1288, 3, 16, "random"), (BF, 2049, 512, 512, 4, 64, "runs"), (HF, 513, 4096, 256, 40, 16, "runs"),
    (BF, 640, 256, 5000, 2, 128, "even"),
    # many steps of an adapter's tokens through the rings, the last one short: consecutive and scattered
    (BF, 2500, 256, 264, 1, 16, "one"), (BF, 2531, 512, 520, 2, 64, "blocks"), (HF, 3001, 256, 136, 2, 128, "blocks"),
    (BF, 2600, 256, 264, 1, 24, "random"), (HF, 1923, 768, 264, 1, 8, "one"),
    # ranks of 4 modulo 8: rows of b that no tensor map takes
    (BF, 300, 256, 264, 3, 12, "runs"), (HF, 5, 128, 136, 2, 4, "random"), (HF, 700, 264, 512, 4, 4, "runs"),
    (BF, 900, 512, 264, 2, 68, "blocks"),
    # one column block, many adapters, 16-way and no split of the first product, fp16 above rank 64
    (BF, 70, 8, 8, 2, 8, "random"), (BF, 1500, 64, 128, 1000, 8, "random"), (HF, 260, 8192, 136, 1, 24, "one"),
    (BF, 9000, 128, 72, 3, 16, "runs"), (HF, 333, 1016, 4104, 5, 104, "runs"), (BF, 24, 4096, 4096, 2, 128, "random"),
    # sizes that are not multiples of 8, rank 1, fp32
    (BF, 5, 100, 60, 2, 4, "random"), (HF, 33, 77, 131, 3, 1, "random"), (BF, 130, 515, 258, 2, 12, "runs"),
    (F32, 1, 256, 264, 2, 16, "one"), (F32, 65, 300, 130, 3, 5, "random"), (F32, 200, 1024, 512, 4, 64, "outside"),
    (BF, 40, 264, 64, 2, 3, "none"),
]


def name(c):
    return f"{str(c[0])[6:]}_M{c[1]}_K{c[2]}_N{c[3]}_L{c[4]}_R{c[5]}_{c[6]}"


@pytest.mark.parametrize("M,L,kind", [(1, 1, "one"), (1, 1024, "random"), (31, 2, "none"), (1000, 7, "even"),
                                      (4097, 1024, "random"), (20000, 3, "runs"), (5000, 40, "outside"),
                                      (1 << 20, 1, "one"), (300000, 1000, "random")])
def test_plan(ql, M, L, kind):
    """Every token once, by adapter and ascending inside one; every segment cut into tiles of 8 and of 128."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    ids = ref.make_ids(kind, M, L, gen)
    plan = ql.adapters_plan(ids, L)
    p = plan.buffer.view(torch.int32).cpu().long()
    up = lambda v: (v + 3) // 4 * 4  # noqa: E731
    most = lambda t: M // t + min(M, L + 1)  # noqa: E731
    head, seg = p[:8], p[8:8 + L + 2]
    perm = p[8 + 2 * up(L + 2):][:M]
    key = torch.where((ids < 0) | (ids >= L), L, ids.long()).cpu()
    want = torch.sort(key, stable=True).indices
    assert torch.equal(perm, want)
    counts = torch.bincount(key, minlength=L + 1)
    assert torch.equal(seg[1:], counts.cumsum(0)) and seg[0] == 0
    at = 8 + 2 * up(L + 2) + up(M)
    for t, n in ((8, int(head[2])), (128, int(head[3]))):
        assert n == int((counts + t - 1).div(t, rounding_mode="floor").sum()) <= most(t)
        tiles = p[at:at + 4 * n].reshape(n, 4)
        at += 4 * most(t)
        assert torch.equal(tiles[:, 1], tiles[:, 2].cumsum(0) - tiles[:, 2]) and int(tiles[:, 2].sum()) == M
        assert bool((tiles[:, 2] <= t).all()) and torch.equal(key[perm[tiles[:, 1]]], tiles[:, 0])
        first, last = perm[tiles[:, 1]], perm[tiles[:, 1] + tiles[:, 2] - 1]
        assert torch.equal(tiles[:, 3], torch.where(last - first == tiles[:, 2] - 1, first, -1))


@pytest.mark.parametrize("case", CASES, ids=name)
def test_forward(ql, case):
    d = ref.make(case)
    M, R = case[1], case[5]
    plan = ql.adapters_plan(d["ids"], case[4])
    u = torch.full((M, R), float("nan"), device="cuda")
    out = ql.adapters_forward(d["x"], d["a"], d["b"], d["scales"], plan, base=d["base"], u=u)
    assert ql.device_status() == ql.QLIN_OK
    ref.check_forward(d["x"], d["a"], d["b"], d["scales"], d["ids"], d["base"], out, u)
    none = (d["ids"] < 0) | (d["ids"] >= case[4])
    assert torch.equal(out[none], d["base"][none]) and bool((u[none] == 0).all())
    # the same in place, and without a base
    again = d["base"].clone()
    assert ql.adapters_forward(d["x"], d["a"], d["b"], d["scales"], plan, base=again, out=again) is again
    assert torch.equal(again, out)
    bare = ql.adapters_forward(d["x"], d["a"], d["b"], d["scales"], plan)
    ref.check_forward(d["x"], d["a"], d["b"], d["scales"], d["ids"], None, bare)
    assert ql.device_status() == ql.QLIN_OK


@pytest.mark.parametrize("g", [0, 64, 128, 256])
@pytest.mark.parametrize("case", CASES, ids=name)
def test_backward(ql, case, g):
    if g and case[2] % g:
        pytest.skip("K is not a multiple of the group")
    d = ref.make(case)
    x = d["x"]
    plan = ql.adapters_plan(d["ids"], case[4])
    u = torch.zeros(case[1], case[5], device="cuda")
    ql.adapters_forward(x, d["a"], d["b"], d["scales"], plan, u=u)
    args = (d["dy"], d["a"], d["b"], d["scales"], plan, u)
    kept = dict(checkpoint=(*ql.quantize_int8_groups(x, g), g)) if g else dict(x=x)
    xhat = ref.restored(*kept["checkpoint"]) if g else x.double()
    dx, da, db = ql.adapters_backward(*args, dx_base=d["dx_base"], **kept)
    assert ql.device_status() == ql.QLIN_OK
    ref.check_backward(d["dy"], d["a"], d["b"], d["scales"], d["ids"], u, xhat, d["dx_base"], dx, da, db, g > 0)
    none = (d["ids"] < 0) | (d["ids"] >= case[4])
    assert torch.equal(dx[none], d["dx_base"][none])
    again = d["dx_base"].clone()  # in place, the same bits from run to run
    dx2, da2, db2 = ql.adapters_backward(*args, dx_base=again, dx=again, **kept)
    assert dx2 is again and torch.equal(dx2, dx) and torch.equal(da2, da) and torch.equal(db2, db)
    if g in (0, 64):
        dx3, da3, db3 = ql.adapters_backward(*args, want_dx=False, **kept)
        assert dx3 is None and torch.equal(da3, da) and torch.equal(db3, db)
        dx4 = ql.adapters_backward(*args, **kept)[0]
        ref.check_backward(d["dy"], d["a"], d["b"], d["scales"], d["ids"], u, xhat, None, dx4, da, db, g > 0)


@pytest.mark.parametrize("case", [(BF, 40, 256, 264, 4, 16, "random"), (HF, 700, 512, 256, 5, 32, "random"),
                                  (BF, 700, 512, 256, 5, 64, "runs"), (F32, 70, 256, 128, 3, 8, "random")], ids=name)
def test_what_is_not_finite_stays_with_its_adapter(ql, case):
    """NaN and infinities of tokens without an adapter, and of one adapter's tokens and factors, reach nobody else."""
    d = ref.make(case)
    ids, L = d["ids"], case[4]
    d["x"][ids == -1] = float("nan")
    d["dy"][ids == -1] = float("inf")
    d["x"][ids == 1] = float("inf")
    d["dy"][ids == 1] = float("nan")
    d["a"][2], d["b"][2] = float("nan"), float("-inf")
    plan = ql.adapters_plan(ids, L)
    u = torch.empty(case[1], case[5], device="cuda")
    out = ql.adapters_forward(d["x"], d["a"], d["b"], d["scales"], plan, base=d["base"], u=u)
    assert torch.equal(out[ids == -1], d["base"][ids == -1])
    assert not out[ids == 1].isfinite().any() and not out[ids == 2].isfinite().any()
    dx, da, db = ql.adapters_backward(d["dy"], d["a"], d["b"], d["scales"], plan, u, x=d["x"], dx_base=d["dx_base"])
    assert torch.equal(dx[ids == -1], d["dx_base"][ids == -1])
    assert da[1].isnan().all() and db[1].isnan().all() and not dx[ids == 1].isfinite().any()
    fine = [i for i in range(L) if i not in (1, 2)]
    keep = torch.isin(ids, torch.tensor(fine, device="cuda"))
    sub = torch.where(keep, ids, -1)
    x, dy = (torch.where(keep[:, None], d[k], 0) for k in ("x", "dy"))
    pick = lambda t: t[keep]  # noqa: E731
    ref.check_forward(pick(x), d["a"], d["b"], d["scales"], pick(sub), pick(d["base"]), pick(out), pick(u))
    a, b = d["a"].clone(), d["b"].clone()
    a[[1, 2]], b[[1, 2]] = 0, 0
    da[[1, 2]], db[[1, 2]] = 0, 0
    ref.check_backward(pick(dy), a, b, d["scales"], pick(sub), pick(u), pick(x).double(), pick(d["dx_base"]),
                       pick(dx), da, db, False)


@pytest.mark.parametrize("dt,top", [(HF, 1e-6), (HF, 3e4), (BF, 1e-30), (BF, 1e30)], ids=str)
def test_sizes_of_the_inner_values(ql, dt, top):
    """u and v far from 1 (fp16: outside its own range) lose nothing: gradients against 64 bits."""
    case = (dt, 300, 256, 264, 2, 16, "runs")
    d = ref.make(case)
    plan = ql.adapters_plan(d["ids"], 2)
    u = torch.randn(300, 16, device="cuda") * (top if dt == BF else top * 100)
    if dt == BF:
        d["dy"] = (d["dy"].float() * min(top, 1e20)).to(dt)
        d["scales"] *= 1e-4
        u = u.clamp(-1e16, 1e16)
    else:
        d["scales"] *= 1 / (top * 100)  # db stays in range
        d["b"] = (d["b"].float() * min(top, 1.0)).to(dt)
    dx, da, db = ql.adapters_backward(d["dy"], d["a"], d["b"], d["scales"], plan, u, x=d["x"], dx_base=d["dx_base"])
    m = torch.isfinite(da).all() and torch.isfinite(db).all() and torch.isfinite(dx).all()
    if not m:  # a result outside the type's range is infinite, not wrong
        lim = torch.finfo(dt).max
        ids, sd = d["ids"], d["scales"].double()
        for i in range(2):
            r = ref.rows_of(ids, i)
            want = sd[i] * (d["dy"][r].double() @ d["b"][i].double())
            assert bool((want.T @ d["x"][r].double()).abs().max() > lim * 0.99) or da[i].isfinite().all()
        return
    ref.check_backward(d["dy"], d["a"], d["b"], d["scales"], d["ids"], u, d["x"].double(), d["dx_base"], dx, da, db,
                       False)


def test_gradients_are_differences(ql):
    """<da, A'> etc. are the slopes of sum(out * dy) along A', B' and x' (fp32, central differences)."""
    case = (F32, 30, 64, 72, 3, 8, "random")
    d = ref.make(case)
    plan = ql.adapters_plan(d["ids"], 3)
    u = torch.zeros(30, 8, device="cuda")
    ql.adapters_forward(d["x"], d["a"], d["b"], d["scales"], plan, u=u)
    dx, da, db = ql.adapters_backward(d["dy"], d["a"], d["b"], d["scales"], plan, u, x=d["x"])

    def value(x, a, b):  # in 64 bits, apart from the kernels
        out = torch.zeros(30, 72, dtype=torch.float64, device="cuda")
        for i in range(3):
            m = ref.rows_of(d["ids"], i)
            out[m] = d["scales"][i].double() * (x[m] @ a[i].T) @ b[i].T
        return (out * d["dy"].double()).sum()

    p = [d[k].double() for k in ("x", "a", "b")]
    for j, grad in enumerate((dx, da, db)):
        step = torch.randn(p[j].shape, device="cuda", dtype=torch.float64)
        h = 1e-4
        up, down = ([t + s * h * step if k == j else t for k, t in enumerate(p)] for s in (1, -1))
        slope = (value(*up) - value(*down)) / (2 * h)
        mine, size = (grad.double() * step).sum(), (grad.double() * step).abs().sum()
        # the value is of second degree along one argument at most: the difference is exact but for 64-bit
        # rounding (1e-16 / 1e-4 of the value's terms); the gradient holds 24 bits and sums of 72 + 30 + 8 terms
        assert abs(float(slope - mine)) <= ref.acc(110) * float(size) + 1e-9 * float(size) + 1e-9


@pytest.mark.parametrize("case", [(BF, 3, 512, 512, 4, 16, "random"), (BF, 300, 512, 512, 4, 16, "runs")], ids=name)
def test_graph_replays_with_new_contents(ql, case):
    """Plan, forward and backward captured once; replayed for other ids and inputs in the same buffers."""
    d, e = ref.make(case), ref.make(case, seed=9)
    M, K, N, L, R = case[1:6]
    u = torch.zeros(M, R, device="cuda")
    out, dx = torch.empty_like(d["base"]), torch.empty_like(d["dx_base"])
    plan = ql.adapters_plan(d["ids"], L)
    wf = torch.empty(ql.adapters_workspace_size(M, N, K, L, R), dtype=torch.uint8, device="cuda")
    wb = torch.empty(ql.adapters_workspace_size(M, N, K, L, R, True), dtype=torch.uint8, device="cuda")
    got = {}

    def step():
        ql.adapters_plan(d["ids"], L, out=plan)
        ql.adapters_forward(d["x"], d["a"], d["b"], d["scales"], plan, base=d["base"], out=out, u=u, workspace=wf)
        got["r"] = ql.adapters_backward(d["dy"], d["a"], d["b"], d["scales"], plan, u, x=d["x"], dx_base=d["dx_base"],
                                        dx=dx, workspace=wb)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for src in (e, ref.make(case, seed=11)):
        for k in ("x", "ids", "base", "dy", "dx_base", "a", "b", "scales"):
            d[k].copy_(src[k])
        graph.replay()
        torch.cuda.synchronize()
        ref.check_forward(d["x"], d["a"], d["b"], d["scales"], d["ids"], d["base"], out, u)
        ref.check_backward(d["dy"], d["a"], d["b"], d["scales"], d["ids"], u, d["x"].double(), d["dx_base"],
                           *got["r"], False)
    assert ql.device_status() == ql.QLIN_OK


def test_two_streams_at_once(ql):
    """Calls on two streams with workspaces of their own do not disturb one another."""
    cases = [(BF, 300, 1024, 2048, 4, 32, "runs"), (BF, 40, 2048, 1024, 4, 16, "random")]
    ds = [ref.make(c) for c in cases]
    plans = [ql.adapters_plan(d["ids"], 4) for d in ds]
    want = [ql.adapters_forward(d["x"], d["a"], d["b"], d["scales"], p, base=d["base"]) for d, p in zip(ds, plans)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [[], []]
    for _ in range(20):
        for j, s in enumerate(streams):
            with torch.cuda.stream(s):
                d = ds[j]
                outs[j].append(ql.adapters_forward(d["x"], d["a"], d["b"], d["scales"], plans[j], base=d["base"]))
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert all(torch.equal(w, t) for t in o)


def test_run_beside_a_quantized_layer(ql):
    """As they are used: a 4-bit layer with adapters, forward and the gradients of a training step from its
    input's 8-bit checkpoint, for a batch of prompts and then for single tokens."""
    K, N, L, R, g = 512, 768, 3, 16, 64
    gen = torch.Generator(device="cuda").manual_seed(5)
    w = torch.randn(N, K, generator=gen, device="cuda") * 0.05
    codes, sc, bi = ql.quantize(w, 4, 64)
    what = ql.dequantize(codes, sc, bi, K, 4, 64, torch.float32)
    for M, kind in ((200, "runs"), (4, "random")):
        d = ref.make((BF, M, K, N, L, R, kind), seed=M)
        plan = ql.adapters_plan(d["ids"], L)
        u = torch.empty(M, R, device="cuda")
        y = ql.matmul(d["x"], codes, sc, bi, 4, 64)
        base = y.clone()
        q, s = ql.quantize_int8_groups(d["x"], g)
        ql.adapters_forward(d["x"], d["a"], d["b"], d["scales"], plan, base=y, out=y, u=u)
        ref.check_forward(d["x"], d["a"], d["b"], d["scales"], d["ids"], base, y, u)
        dx_base = (d["dy"].float() @ what).to(BF)
        dx, da, db = ql.adapters_backward(d["dy"], d["a"], d["b"], d["scales"], plan, u, checkpoint=(q, s, g),
                                          dx_base=dx_base)
        ref.check_backward(d["dy"], d["a"], d["b"], d["scales"], d["ids"], u, ref.restored(q, s, g), dx_base, dx, da,
                           db, True)
    assert ql.device_status() == ql.QLIN_OK


def test_refusals(ql):
    d = ref.make((BF, 8, 64, 72, 2, 8, "random"))
    plan = ql.adapters_plan(d["ids"], 2)
    f = lambda **k: ql.adapters_forward(**{**dict(x=d["x"], a=d["a"], b=d["b"], scales=d["scales"], plan=plan), **k})  # noqa: E731
    for bad in [dict(x=d["x"][:4].contiguous()), dict(x=d["x"].t()), dict(a=d["a"][:, :4].contiguous()),
                dict(b=d["b"][:1].contiguous()), dict(scales=d["scales"][:1].contiguous()), dict(base=d["x"]),
                dict(u=torch.zeros(8, 9, device="cuda")), dict(plan=ql.adapters_plan(d["ids"], 3)),
                dict(workspace=torch.empty(1 << 20, dtype=torch.uint8))]:
        with pytest.raises(ValueError):
            f(**bad)
    for bad in [dict(a=d["a"].half()), dict(scales=d["scales"].to(BF)), dict(u=torch.zeros(8, 8, device="cuda").to(BF))]:
        with pytest.raises(TypeError):
            f(**bad)
    with pytest.raises(ql.QlinError) as e:
        f(workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.status == ql.QLIN_ERR_WORKSPACE
    with pytest.raises(ql.QlinError) as e:
        ql.adapters_plan(d["ids"], 1025)
    assert e.value.status == ql.QLIN_ERR_UNSUPPORTED
    u = torch.zeros(8, 8, device="cuda")
    with pytest.raises(ValueError):
        ql.adapters_backward(d["dy"], d["a"], d["b"], d["scales"], plan, u)
    with pytest.raises(ValueError):
        ql.adapters_backward(d["dy"], d["a"], d["b"], d["scales"], plan, u, x=d["x"], want_dx=False,
                             dx_base=d["dx_base"])
    with pytest.raises(ql.QlinError):
        ql.adapters_plan(torch.zeros(0, dtype=torch.int32, device="cuda"), 2)


@pytest.mark.parametrize("case", [(BF, 300, 256, 264, 3, 16, "runs"), (HF, 5, 128, 136, 2, 8, "random")], ids=name)
def test_tensors_aligned_to_their_elements_only(ql, case):
    """Contiguous tensors that begin one element past a 16-byte boundary take the general kernels."""
    d = ref.make(case)
    M, K, N, L, R = case[1:6]

    def shifted(t):
        flat = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        return flat[1:].view(t.shape).copy_(t)

    for k in ("x", "a", "b", "base", "dy", "dx_base"):
        d[k] = shifted(d[k])
    plan = ql.adapters_plan(d["ids"], L)
    u = shifted(torch.zeros(M, R, device="cuda"))
    out = ql.adapters_forward(d["x"], d["a"], d["b"], d["scales"], plan, base=d["base"], u=u)
    ref.check_forward(d["x"], d["a"], d["b"], d["scales"], d["ids"], d["base"], out, u)
    dx, da, db = ql.adapters_backward(d["dy"], d["a"], d["b"], d["scales"], plan, u, x=d["x"], dx_base=d["dx_base"])
    ref.check_backward(d["dy"], d["a"], d["b"], d["scales"], d["ids"], u, d["x"].double(), d["dx_base"], dx, da, db,
                       False)


def test_one_plan_serves_layers_of_other_sizes(ql):
    """A plan depends on the batch alone: projections of other sizes, ranks and types, forward and backward."""
    first = ref.make((BF, 260, 256, 512, 4, 16, "runs"))
    plan = ql.adapters_plan(first["ids"], 4)
    for case in ((BF, 260, 512, 128, 4, 32, "runs"), (HF, 260, 128, 640, 4, 8, "runs"), (F32, 260, 64, 72, 4, 3, "runs")):
        d = ref.make(case, seed=7)
        d["ids"] = first["ids"]
        u = torch.empty(260, case[5], device="cuda")
        out = ql.adapters_forward(d["x"], d["a"], d["b"], d["scales"], plan, base=d["base"], u=u)
        ref.check_forward(d["x"], d["a"], d["b"], d["scales"], d["ids"], d["base"], out, u)
        dx, da, db = ql.adapters_backward(d["dy"], d["a"], d["b"], d["scales"], plan, u, x=d["x"])
        ref.check_backward(d["dy"], d["a"], d["b"], d["scales"], d["ids"], u, d["x"].double(), None, dx, da, db, False)


def test_between_layer_calls_of_one_run(ql):
    """Layer, adapters, layer, adapters with no other operation between: the library's kernels start early behind
    one another, and each reads what the one before wrote."""
    K, N, L, R, M = 512, 512, 3, 16, 6
    gen = torch.Generator(device="cuda").manual_seed(5)
    codes, sc, bi = ql.quantize(torch.randn(N, K, generator=gen, device="cuda") * 0.05, 4, 64)
    d = ref.make((BF, M, K, N, L, R, "random"))
    plan = ql.adapters_plan(d["ids"], L)
    ws = torch.empty(ql.adapters_workspace_size(M, N, K, L, R), dtype=torch.uint8, device="cuda")
    y, z = torch.empty(M, N, dtype=BF, device="cuda"), torch.empty(M, N, dtype=BF, device="cuda")
    results = []
    for _ in range(30):
        ql.matmul(d["x"], codes, sc, bi, 4, 64, out=y)
        ql.adapters_forward(d["x"], d["a"], d["b"], d["scales"], plan, base=y, out=y, workspace=ws)
        ql.matmul(y, codes, sc, bi, 4, 64, out=z)
        ql.adapters_forward(y, d["a"], d["b"], d["scales"], plan, base=z, out=z, workspace=ws)
        results.append(z.clone())
    base = ql.matmul(d["x"], codes, sc, bi, 4, 64)
    torch.cuda.synchronize()
    mid = ql.adapters_forward(d["x"], d["a"], d["b"], d["scales"], plan, base=base)
    torch.cuda.synchronize()
    ref.check_forward(d["x"], d["a"], d["b"], d["scales"], d["ids"], base, mid)
    last = ql.matmul(mid, codes, sc, bi, 4, 64)
    torch.cuda.synchronize()
    want = ql.adapters_forward(mid, d["a"], d["b"], d["scales"], plan, base=last)
    assert all(torch.equal(r, want) for r in results)
    assert ql.device_status() == ql.QLIN_OK
