"""Operators measured beside the quantized linear layers: low-rank adapters of many requests on a
shared projection (forward and backward) and activations kept in 8 bits for the backward pass.

Four operators, by a case's "op":

  forward     out[m] = base[m] + s_i B_i (A_i x[m]), i = the adapter of token m (-1: none)
  backward    dx, dA, dB of the same from dy, u = A_i x and x (plain or its int8 checkpoint)
  checkpoint  x -> int8 codes and one scale per token and group of inputs -> x again
  wgrad       dW = dy^T x^ and db = sum of dy, x^ the int8 checkpoint of the layer's input

Tokens are rows; A is [adapters, rank, K] and B [adapters, N, rank], as the two factors of a linear
layer's weight [N, K] are stored.  Checkpoint codes are [tokens, K] with scales [K / group, tokens].
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # one token of one request while a text is generated, on a 4096 x 4096 projection
        {"name": "forward_1_token", "op": "forward", "dtype": "bf16", "M": 1, "K": 4096, "N": 4096, "L": 8, "R": 16,
         "order": "decode", "keep_u": False},
        # one decode step of 61 requests over a pool of 32 adapters, some requests without one
        {"name": "forward_61_requests", "op": "forward", "dtype": "f16", "M": 61, "K": 4096, "N": 11008, "L": 32,
         "R": 16, "order": "decode", "keep_u": False},
        # a serving batch of prompts and single tokens on a down projection
        {"name": "forward_777_mixed", "op": "forward", "dtype": "bf16", "M": 777, "K": 11008, "N": 4096, "L": 12,
         "R": 32, "order": "mixed", "keep_u": False},
        # a training batch of four fine-tunings at once, keeping u for the backward pass
        {"name": "forward_4096_train", "op": "forward", "dtype": "bf16", "M": 4096, "K": 4096, "N": 14336, "L": 4,
         "R": 64, "order": "train", "keep_u": True},
        # a short micro-batch, rank 8, the input kept in 8 bits
        {"name": "backward_256", "op": "backward", "dtype": "f16", "M": 256, "K": 4096, "N": 4096, "L": 2, "R": 8,
         "order": "train", "g": 64},
        # a ragged batch of three adapters with the input kept as it is (g = 0)
        {"name": "backward_1531_ragged", "op": "backward", "dtype": "bf16", "M": 1531, "K": 11008, "N": 4096, "L": 3,
         "R": 16, "order": "mixed", "g": 0},
        # the training batch of forward_4096_train, the input kept in 8 bits
        {"name": "backward_4096", "op": "backward", "dtype": "bf16", "M": 4096, "K": 4096, "N": 14336, "L": 4,
         "R": 64, "order": "train", "g": 128},
        # a short sequence's layer input out to 8 bits and back
        {"name": "checkpoint_64", "op": "checkpoint", "dtype": "bf16", "M": 64, "K": 4096, "g": 64},
        # a long batch's widest activation
        {"name": "checkpoint_16384", "op": "checkpoint", "dtype": "bf16", "M": 16384, "K": 14336, "g": 128},
        # the weight gradient of a square layer from few tokens: bound by writing it
        {"name": "wgrad_129", "op": "wgrad", "dtype": "f16", "M": 129, "K": 4096, "N": 4096, "g": 64},
        # a ragged micro-batch on a down projection
        {"name": "wgrad_1000", "op": "wgrad", "dtype": "bf16", "M": 1000, "K": 11008, "N": 4096, "g": 256},
        # a training batch on an up projection: bound by the products
        {"name": "wgrad_4096", "op": "wgrad", "dtype": "bf16", "M": 4096, "K": 4096, "N": 14336, "g": 128},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["forward", "forward", "backward", "backward", "checkpoint", "wgrad"])
    m = _log(rng, 1, 4096)
    if op == "checkpoint":
        g = rng.choice([64, 128, 256])
        return {"op": op, "dtype": rng.choice(["bf16", "f16", "f32"]), "M": _log(rng, 1, 16384),
                "K": g * max(1, _log(rng, 512, 14336) // g), "g": g}
    if op == "wgrad":
        g = rng.choice([64, 128, 256])
        return {"op": op, "dtype": rng.choice(["bf16", "f16"]), "M": m, "K": g * max(1, _log(rng, 512, 8192) // g),
                "N": 8 * max(1, _log(rng, 512, 7168) // 8), "g": g}
    case = {"op": op, "dtype": rng.choice(["bf16", "bf16", "bf16", "f16", "f16", "f32"]), "M": m,
            "K": 8 * _log(rng, 64, 1024), "N": 8 * _log(rng, 64, 1024), "L": _log(rng, 1, 48),
            "R": rng.choice([4, 8, 8, 12, 16, 16, 24, 32, 32, 40, 64, 64]),
            "order": rng.choice(["mixed", "train"]) if m > 256 or op == "backward" else rng.choice(["decode", "mixed"])}
    if case["M"] * case["L"] * case["R"] > 4096 * 512:  # the plain form multiplies with every adapter
        case["L"] = max(1, 4096 * 512 // (case["M"] * case["R"]))
    if op == "forward":
        return dict(case, keep_u=rng.random() < 0.5)
    g = rng.choice([0, 64, 128])
    if g:
        case["K"] = g * max(1, case["K"] // g)
    return dict(case, g=g)


def _ids(case, gen):
    """The adapter of every token: its request's.  decode: one token a request; mixed: requests of
    one token to a few hundred; train: long sequences.  About one request in eight has none."""
    m, n = case["M"], case["L"]
    mean = {"decode": 1, "mixed": 40, "train": 512}[case["order"]]
    starts = torch.rand(m, generator=gen, device="cuda") < 1.0 / mean
    request = torch.cumsum(starts, 0)
    each = torch.randint(0, n, (m + 1,), generator=gen, device="cuda", dtype=torch.int32)
    if case["order"] != "train":
        each = torch.where(torch.rand(m + 1, generator=gen, device="cuda") < 0.125, -1, each)
    return each[request].to(torch.int32).contiguous()


def _activations(m, k, gen):
    """Layer inputs: most channels near 1, one in a hundred far larger, as in a trained model."""
    wide = 1 + 19 * (torch.rand(k, generator=gen, device="cuda") < 0.01)
    return torch.randn(m, k, generator=gen, device="cuda") * wide


def _quantized(x, g):
    """int8 codes [M, K] and scales [K / g, M]: the absmax of a token's group is 127."""
    groups = x.float().reshape(x.shape[0], -1, g)
    scale = groups.abs().amax(2)
    scale = scale / torch.full_like(scale, 127.0)
    scale = torch.where(scale == 0, 1.0, scale)
    q = (groups / scale[:, :, None]).round().clamp(-128, 127).to(torch.int8)
    return q.reshape(x.shape), scale.t().contiguous()


def _restored(q, scale, g):
    return (q.float().reshape(q.shape[0], -1, g) * scale.t()[:, :, None]).reshape(q.shape)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    t = DTYPES[case["dtype"]]
    m, k = case["M"], case["K"]
    x = _activations(m, k, gen).to(t)
    if case["op"] == "checkpoint":
        return {"case": case, "x": x}
    n = case["N"]
    # gradients differ in size from token to token
    dy = torch.randn(m, n, generator=gen, device="cuda") * 0.01
    dy = (dy * torch.exp(torch.randn(m, 1, generator=gen, device="cuda"))).to(t)
    if case["op"] == "wgrad":
        q, scale = _quantized(x, case["g"])
        return {"case": case, "dy": dy, "q": q, "scale": scale}
    adapters, r = case["L"], case["R"]
    ids = _ids(case, gen)
    a = (torch.randn(adapters, r, k, generator=gen, device="cuda") / math.sqrt(k)).to(t)
    b = (torch.randn(adapters, n, r, generator=gen, device="cuda") * 0.02).to(t)
    scales = 0.5 + 1.5 * torch.rand(adapters, generator=gen, device="cuda")
    state = {"case": case, "ids": ids, "a": a, "b": b, "scales": scales}
    if own:  # the tokens' order by adapter: made once for a batch, used by every layer of the model
        from bit_quantized_linear_qmm_b200 import qlin
        state["plan"] = qlin.adapters_plan(ids, adapters)
    if case["op"] == "forward":
        base = torch.randn(m, n, generator=gen, device="cuda").to(t)
        return dict(state, x=x, base=base)
    dx_base = (torch.randn(m, k, generator=gen, device="cuda") * 0.02).to(t)
    u = _masked(x.float() @ a.float().flatten(0, 1).t(), ids, adapters).sum(1)
    state = dict(state, dy=dy, dx_base=dx_base, u=u.contiguous())
    if case["g"]:
        state["q"], state["scale"] = _quantized(x, case["g"])
    else:
        state["x"] = x
    return state


def _masked(v, ids, adapters):
    """[M, adapters * R] -> [M, adapters, R] with zeros at the adapters that a token does not use."""
    mine = ids[:, None] == torch.arange(adapters, device=ids.device)
    return v.reshape(v.shape[0], adapters, -1) * mine[:, :, None]


def _forward(state):
    case, t = state["case"], state["x"].dtype
    a, b = state["a"].float().flatten(0, 1), state["b"].float().transpose(1, 2).flatten(0, 1)
    u = _masked(state["x"].float() @ a.t(), state["ids"], case["L"])
    out = (state["base"].float() + (u * state["scales"][:, None]).flatten(1) @ b).to(t)
    return {"out": out, "u": u.sum(1)} if case["keep_u"] else {"out": out}


def _backward(state):
    case, t = state["case"], state["dy"].dtype
    ids, adapters, s = state["ids"], case["L"], state["scales"][:, None]
    x = _restored(state["q"], state["scale"], case["g"]) if case["g"] else state["x"].float()
    a, b = state["a"].float().flatten(0, 1), state["b"].float().transpose(1, 2).flatten(0, 1)
    dy = state["dy"].float()
    v = (_masked(dy @ b.t(), ids, adapters) * s).flatten(1)
    u = (_masked(state["u"].repeat(1, adapters), ids, adapters) * s).flatten(1)
    dx = state["dx_base"].float() + v @ a
    da = (v.t() @ x).reshape(state["a"].shape)
    db = (u.t() @ dy).reshape(adapters, case["R"], case["N"]).transpose(1, 2).contiguous()
    return {"dx": dx.to(t), "da": da.to(t), "db": db.to(t)}


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        from bit_quantized_linear_qmm_b200 import qlin
        if op == "checkpoint":
            q, scale = qlin.quantize_int8_groups(state["x"], case["g"])
            return {"q": q, "scale": scale, "x": qlin.dequantize_int8_groups(q, scale, case["g"], state["x"].dtype)}
        if op == "wgrad":
            dw, db = qlin.pergroup_wgrad(state["dy"], state["q"], state["scale"], case["g"])
            return {"dw": dw, "db": db}
        if op == "forward":
            u = torch.empty(case["M"], case["R"], device="cuda") if case["keep_u"] else None
            out = qlin.adapters_forward(state["x"], state["a"], state["b"], state["scales"], state["plan"],
                                        base=state["base"], u=u)
            return {"out": out, "u": u} if case["keep_u"] else {"out": out}
        x = {"checkpoint": (state["q"], state["scale"], case["g"])} if case["g"] else {"x": state["x"]}
        dx, da, db = qlin.adapters_backward(state["dy"], state["a"], state["b"], state["scales"], state["plan"],
                                            state["u"], dx_base=state["dx_base"], **x)
        return {"dx": dx, "da": da, "db": db}
    if op == "checkpoint":
        q, scale = _quantized(state["x"], case["g"])
        return {"q": q, "scale": scale, "x": _restored(q, scale, case["g"]).to(state["x"].dtype)}
    if op == "wgrad":
        dy = state["dy"].float()
        dw = dy.t() @ _restored(state["q"], state["scale"], case["g"])
        return {"dw": dw.to(state["dy"].dtype), "db": dy.sum(0).to(state["dy"].dtype)}
    return _forward(state) if op == "forward" else _backward(state)


def work(case):
    m, k, e = case["M"], case["K"], DTYPES[case["dtype"]].itemsize
    if case["op"] == "checkpoint":
        return {"bytes": m * k * (2 * e + 1) + 4 * m * (k // case["g"]), "flops": 4 * m * k}
    n = case["N"]
    if case["op"] == "wgrad":
        return {"bytes": m * n * e + m * k + 4 * m * (k // case["g"]) + n * k * e + n * e, "flops": 2 * m * n * k}
    adapters, r = case["L"], case["R"]
    used = min(adapters, m)
    if case["op"] == "forward":
        return {"bytes": m * k * e + 2 * m * n * e + used * r * (k + n) * e + (4 * m * r if case["keep_u"] else 0),
                "flops": 2 * m * r * (k + n)}
    x = m * k + 4 * m * (k // case["g"]) if case["g"] else m * k * e
    return {"bytes": m * n * e + x + 2 * m * k * e + used * r * (k + n) * e + adapters * r * (k + n) * e + 4 * m * r,
            "flops": 4 * m * r * (k + n)}


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "checkpoint":
        x = state["x"].double()
        top = torch.stack([c.abs().max(1).values for c in x.split(case["g"], 1)])
        scale = torch.where(top > 0, top / 127, 1.0)
        kept = scale.float().double()  # the scale that is stored has 32 bits
        back = torch.cat([torch.round(c / s[:, None]) * s[:, None] for c, s in zip(x.split(case["g"], 1), kept)], 1)
        return {"q": None, "scale": scale, "x": back}
    if case["op"] != "forward" and case["g"]:
        parts = zip(state["q"].double().split(case["g"], 1), state["scale"].double())
        x = torch.cat([c * s[:, None] for c, s in parts], 1)
    else:
        x = state["x"].double()
    if case["op"] == "wgrad":
        dy = state["dy"].double()
        return {"dw": dy.t() @ x, "db": dy.sum(0)}
    a, b, s, ids = state["a"].double(), state["b"].double(), state["scales"].double(), state["ids"]
    if case["op"] == "forward":
        out = state["base"].double()
        u = torch.zeros(case["M"], case["R"], dtype=torch.float64, device=out.device)
        for i in range(case["L"]):
            rows = (ids == i).nonzero()[:, 0]
            u[rows] = x[rows] @ a[i].t()
            out[rows] += s[i] * (u[rows] @ b[i].t())
        return {"out": out, "u": u} if case["keep_u"] else {"out": out}
    dy, u, dx = state["dy"].double(), state["u"].double(), state["dx_base"].double()
    da, db = torch.zeros_like(a), torch.zeros_like(b)
    for i in range(case["L"]):
        rows = (ids == i).nonzero()[:, 0]
        v = s[i] * (dy[rows] @ b[i])
        dx[rows] += v @ a[i]
        da[i] = v.t() @ x[rows]
        db[i] = s[i] * (dy[rows].t() @ u[rows])
    return {"dx": dx, "da": da, "db": db}
