"""Low-rank adapters and 8-bit checkpoints in 64 bits, with the bounds that the tests hold the kernels to.

Bounds, per element, from the arithmetic alone:
- an fp32 sum of n products, in any order, truncating or rounding each addition: n 2^-23 of the sum
  of their absolute values;
- a factor split into two 16-bit halves: 2^-16 of its value (fp16 halves are scaled by a power of
  two first, so that values 2^-38 below the largest are still held);
- an input restored from its int8 codes and rounded to the operand type: half a step of that type;
- the one rounding of the result: half a step of its type.
"""
import torch

SPLIT = 2.0 ** -16
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}


def half(t):
    return torch.finfo(t).eps / 2


def acc(n):
    return n * 2.0 ** -23


def close(got, ref, slack, what):
    """|got - ref| <= slack + half a step of got's type at ref (+ half its smallest step)."""
    g = got.double()
    tol = slack + half(got.dtype) * (ref.abs() + slack) + TINY[got.dtype]
    bad = ~((g - ref).abs() <= tol)
    if bad.any():
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} out of bounds, first at {i}: {float(g[i])} "
                             f"for {float(ref[i])}, allowed {float(tol[i])}")


def rows_of(ids, i):
    return (ids == i).nonzero()[:, 0]


def check_forward(x, a, b, s, ids, base, out, u=None):
    L, R, K = a.shape
    xd, ad, bd, sd = x.double(), a.double(), b.double(), s.double()
    ref = torch.zeros(out.shape, dtype=torch.float64, device=out.device) if base is None else base.double()
    mag = ref.abs() * 2.0 ** -23
    uref = torch.zeros(x.shape[0], R, dtype=torch.float64, device=out.device)
    umag = torch.zeros_like(uref)
    for i in range(L):
        m = rows_of(ids, i)
        uref[m] = xd[m] @ ad[i].T
        umag[m] = xd[m].abs() @ ad[i].abs().T
        ref[m] += sd[i] * (uref[m] @ bd[i].T)
        mag[m] += (SPLIT + acc(K + R + 2)) * sd[i].abs() * (umag[m] @ bd[i].abs().T)
    close(out, ref, mag, "out")
    if u is not None:
        close(u, uref, acc(K) * umag, "u")


def check_backward(dy, a, b, s, ids, u, xhat, dx_base, dx, da, db, rounded_input):
    """xhat: the layer's input in 64 bits; rounded_input: it was restored from codes."""
    L, R, K = a.shape
    M, N = dy.shape
    yd, ad, bd, sd, ud = dy.double(), a.double(), b.double(), s.double(), u.double()
    x_off = half(dy.dtype) if rounded_input and dy.dtype != torch.float32 else 0.0
    ref = torch.zeros(M, K, dtype=torch.float64, device=dy.device) if dx_base is None else dx_base.double()
    mag = ref.abs() * 2.0 ** -23
    for i in range(L):
        m = rows_of(ids, i)
        v, vm = sd[i] * (yd[m] @ bd[i]), sd[i].abs() * (yd[m].abs() @ bd[i].abs())
        ref[m] += v @ ad[i]
        mag[m] += (SPLIT + acc(N + R + 2)) * (vm @ ad[i].abs())
        close(da[i], v.T @ xhat[m], (SPLIT + acc(N + M + 2) + x_off) * (vm.T @ xhat[m].abs()), f"da[{i}]")
        dref = sd[i] * (yd[m].T @ ud[m])
        close(db[i], dref, (SPLIT + acc(M + 2)) * sd[i].abs() * (yd[m].abs().T @ ud[m].abs()), f"db[{i}]")
    if dx is not None:
        close(dx, ref, mag, "dx")


def restored(q, scale, g):
    return torch.cat([c * s[:, None] for c, s in zip(q.double().split(g, 1), scale.double())], 1)


def make_ids(kind, M, L, gen):
    """int32 [M] on the GPU: adapter of every token."""
    if kind == "none":
        return torch.full((M,), -1, dtype=torch.int32, device="cuda")
    if kind == "one":
        return torch.full((M,), L - 1, dtype=torch.int32, device="cuda")
    if kind == "blocks":  # long runs: tiles of consecutive tokens, and some that are not
        return torch.randint(0, L, (M // 300 + 1,), generator=gen, device="cuda", dtype=torch.int32)[
            torch.arange(M, device="cuda") // 300].contiguous()
    if kind == "outside":  # what is not an adapter is none
        ids = torch.randint(-3, L + 3, (M,), generator=gen, device="cuda", dtype=torch.int32)
        ids[0] = 2 ** 31 - 1
        ids[-1] = -2 ** 31
        return ids
    ids = torch.randint(-1, L, (M,), generator=gen, device="cuda", dtype=torch.int32)
    if kind == "even":  # adapters of odd number have no tokens
        ids = torch.where(ids > 0, ids // 2 * 2, ids)
    if kind == "runs":
        ids = ids.sort().values[torch.arange(M, device="cuda") // 5 * 5 % M]
        ids = torch.roll(ids, M // 3)
    return ids.to(torch.int32).contiguous()


def make(case, seed=1):
    """Inputs of a case (dtype, M, K, N, L, R, kind of ids)."""
    dt, M, K, N, L, R, kind = case
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    t = dict(x=rn(M, K), a=rn(L, R, K) / K ** 0.5, b=rn(L, N, R) * 0.1, base=rn(M, N), dy=rn(M, N) * 0.05,
             dx_base=rn(M, K) * 0.1)
    t["x"] *= 1 + 30 * (torch.rand(K, generator=gen, device="cuda") < 0.02)
    t["dy"] *= torch.exp(2 * rn(M, 1))
    t = {k: v.to(dt) for k, v in t.items()}
    t["scales"] = rn(L) * 2
    t["ids"] = make_ids(kind, M, L, gen)
    return t
