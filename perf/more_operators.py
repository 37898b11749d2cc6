"""Products whose weights differ from row to row, as a user's program calls
them, over the sizes they meet:

* ``route``   -- the choice of each token's experts from the router's logits,
                 with their weights, and the slots grouped by expert;
* ``experts`` -- the MXFP4 x MXFP4 product of grouped slots with their experts'
                 weights, plain or as a gated unit (a prefill, a batch);
* ``gemv``    -- the same weights against the f32 activations of a decode or
                 verify step;
* ``combine`` -- the weighted sum of each token's slots;
* ``lora``    -- low-rank adapters of many requests beside a shared projection.

Token t's j-th choice is slot t * top + j; every tensor of slots is in that
order.  ``run`` computes the operators in plain torch operations, in 32 bits,
or with ``own`` set through the library.  ``exact`` gives the results in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda:0"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # the router of one decode step: latency counts
        dict(name="route_decode", op="route", m=1, e=128, top=8, type="f32", renorm=True),
        # a long prefill's router, with many experts
        dict(name="route_prefill", op="route", m=8192, e=256, top=8, type="bf16", renorm=False),
        # a decode batch too large for the GEMV: a few rows for each expert, first product with its gate
        dict(name="experts_batch", op="experts", m=48, e=64, top=6, k=4096, n=2816, shared=True, glu=True, out="f32"),
        # a long prefill's first product, gated, in the type that its quantization reads
        dict(name="experts_prefill_up", op="experts", m=4096, e=64, top=8, k=4096, n=2816, shared=True, glu=True, out="bf16"),
        # an odd prefill's second product: short rows of odd scale counts
        dict(name="experts_prefill_down", op="experts", m=1999, e=16, top=4, k=1440, n=5120, shared=False, glu=False, out="f32"),
        # one token's first product
        dict(name="gemv_decode_up", op="gemv", m=1, e=64, top=8, k=4096, n=2816, shared=True, glu=True),
        # a verify batch's second product: some experts are chosen by several tokens
        dict(name="gemv_verify_down", op="gemv", m=9, e=64, top=6, k=1408, n=4096, shared=False, glu=False),
        # one token's experts summed
        dict(name="combine_decode", op="combine", m=1, top=8, n=4096, type="f32", out="f32", res=True),
        # a prefill's experts summed
        dict(name="combine_prefill", op="combine", m=4001, top=8, n=5120, type="bf16", out="bf16", res=False),
        # one token with its adapter
        dict(name="lora_decode", op="lora", m=1, requests=1, adapters=8, r=16, k=4096, n=4096, type="f32", ab="bf16"),
        # a decode batch of requests with adapters of their own beside the widest projection
        dict(name="lora_batch", op="lora", m=64, requests=64, adapters=40, r=16, k=4096, n=20480, type="f32", ab="bf16"),
        # a prefill of ragged requests, large ranks
        dict(name="lora_prefill", op="lora", m=4099, requests=7, adapters=6, r=64, k=4096, n=5152, type="f16", ab="f16"),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    most = {}
    for c in listed():
        w = work(c)
        most[c["op"]] = max(most.get(c["op"], (0, 0)), (w["bytes"] + w["flops"] / 300, w["flops"]))
    while True:
        op = rng.choice(["route", "experts", "gemv", "combine", "lora"])
        if op == "route":
            e = spread(4, 512)
            c = dict(op=op, m=spread(1, 16384), e=e, top=min(e, rng.choice([1, 2, 4, 6, 8, 10])),
                     type=rng.choice(["f32", "bf16", "f16"]), renorm=rng.random() < 0.5)
        elif op == "experts":
            e, glu = spread(2, 128), rng.random() < 0.5
            c = dict(op=op, m=spread(2, 8192), e=e, top=min(e, rng.choice([1, 2, 4, 6, 8])), k=32 * spread(8, 256),
                     n=2 * spread(48, 4096), shared=rng.random() < 0.6, glu=glu, out=rng.choice(["f32", "bf16", "f16"]))
        elif op == "gemv":
            e = spread(2, 128)
            c = dict(op=op, m=rng.randint(1, 16), e=e, top=min(e, rng.choice([1, 2, 4, 6, 8])), k=32 * spread(8, 256),
                     n=2 * spread(48, 4096), shared=rng.random() < 0.6, glu=rng.random() < 0.5)
        elif op == "combine":
            c = dict(op=op, m=spread(1, 8192), top=rng.choice([1, 2, 4, 6, 8, 10]), n=spread(256, 8192),
                     type=rng.choice(["f32", "bf16", "f16"]), out=rng.choice(["f32", "same"]), res=rng.random() < 0.5)
            if c["out"] == "same":
                c["out"] = c["type"]
        else:
            m, ab = spread(1, 8192), rng.choice(["bf16", "f16"])
            c = dict(op=op, m=m, requests=spread(1, min(m, 128)), adapters=spread(1, 64), r=rng.choice([8, 16, 32, 64, 128]),
                     k=8 * spread(32, 1280), n=spread(256, 20480), type=rng.choice(["f32", ab]), ab=ab)
        w = work(c)
        if w["bytes"] + w["flops"] / 300 <= most[op][0] and w["flops"] <= most[op][1]:
            return c


def work(case):
    """Bytes and operations of one pass: every input read once, every output written once."""
    op, m = case["op"], case["m"]
    if op == "route":
        e, top = case["e"], case["top"]
        return {"bytes": m * e * SIZE[case["type"]] + 16 * m * top + 4 * (e + 1), "flops": 5 * m * e}
    if op in ("experts", "gemv"):
        e, top, k, n = case["e"], case["top"], case["k"], case["n"]
        used = e * (1.0 - (1.0 - top / e) ** m)   # experts that some token chooses
        rows = m if case["shared"] else m * top
        out = (n // 2 if case["glu"] else n) * (SIZE[case["out"]] if op == "experts" else 4)
        x = 17 / 32 if op == "experts" else 4
        return {"bytes": used * n * k * 17 / 32 + rows * k * x + m * top * (out + 4), "flops": 2 * m * top * k * n}
    if op == "combine":
        top, n = case["top"], case["n"]
        return {"bytes": m * n * (top * SIZE[case["type"]] + SIZE[case["out"]] * (2 if case["res"] else 1)) + 4 * m * top,
                "flops": 2 * m * top * n}
    k, n, r = case["k"], case["n"], case["r"]
    used = case["adapters"] * (1.0 - (1.0 - 1.0 / case["adapters"]) ** case["requests"])
    return {"bytes": m * (k * SIZE[case["type"]] + 8 * n) + used * r * (k + n) * 2 + 4 * m, "flops": 2 * m * r * (k + n)}


# ------------------------------------------------------------------- inputs


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(shape, g, std=1.0):
    return torch.randn(shape, generator=g, device=DEV) * std


def _outliers(x, g):
    """Activations as transformers have them: about one value in a hundred ten times larger."""
    return torch.where(torch.rand(x.shape, generator=g, device=DEV) < 0.01, x * 10, x)


def _mx_random(rows, k, g, low, high):
    """Codes [rows, k/2] and scales [rows, k/32] of a quantized tensor: blocks whose largest magnitude is 4 or 6."""
    codes = torch.randint(0, 256, (rows, k // 2), generator=g, device=DEV, dtype=torch.uint8)
    codes[:, 0::16] |= 0x06
    scales = torch.randint(low, high, (rows, k // 32), generator=g, device=DEV, dtype=torch.uint8)
    return codes, scales


def _router_logits(m, e, g):
    """Some experts are liked more than others, and each token has its own taste."""
    return _normal((m, e), g, 1.5) + _normal((1, e), g, 0.5)


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    op, m = case["op"], case["m"]
    if op == "route":
        s["logits"] = _router_logits(m, case["e"], g).to(TYPES[case["type"]])
    elif op in ("experts", "gemv"):
        e, top, k, n = case["e"], case["top"], case["k"], case["n"]
        w, ws = _mx_random(e * n, k, g, 117, 121)     # weights of about 0.02
        s["w"], s["ws"] = w.view(e, n, k // 2), ws.view(e, n, k // 32)
        rows = m if case["shared"] else m * top
        if op == "experts":
            s["xq"], s["xs"] = _mx_random(rows, k, g, 125, 128)      # activations of about 1
        else:
            s["x"] = _outliers(_normal((rows, k), g), g)
        ids = torch.topk(_router_logits(m, e, g), top, 1).indices
        s["ids"] = ids.int()
        # the plan of the slots that the router's step has left
        flat = ids.reshape(-1)
        s["order"] = torch.sort(flat, stable=True).indices.int()
        s["offsets"] = torch.nn.functional.pad(torch.bincount(flat, minlength=e).cumsum(0), (1, 0)).int()
    elif op == "combine":
        s["y"] = _normal((m * case["top"], case["n"]), g).to(TYPES[case["type"]])
        s["weights"] = torch.softmax(_normal((m, case["top"]), g), 1)
        s["res"] = _normal((m, case["n"]), g, 4.0).to(TYPES[case["out"]]) if case["res"] else None
    else:
        k, n, r, count, t = case["k"], case["n"], case["r"], case["adapters"], TYPES[case["ab"]]
        s["x"] = _outliers(_normal((m, k), g), g).to(TYPES[case["type"]])
        s["a"] = _normal((count, r, k), g, 1.0 / math.sqrt(k)).to(t)
        s["b"] = _normal((count, n, r), g, 0.2).to(t)
        s["scale"] = 0.5 + torch.rand(count, generator=g, device=DEV)
        s["res"] = _normal((m, n), g)
        # ragged requests, one after another; of many one in ten has no adapter; the program that batches them knows
        # their adapters on both sides
        host = np.random.default_rng(seed)
        cuts = np.sort(host.choice(m - 1, case["requests"] - 1, replace=False) + 1) if case["requests"] > 1 else []
        lengths = np.diff(np.concatenate([[0], cuts, [m]]).astype(np.int64))
        mine = host.integers(0, count, case["requests"])
        if case["requests"] > 1:
            mine = np.where(host.random(case["requests"]) < 0.1, -1, mine)
        ids = np.repeat(mine, lengths)
        s["ids"] = torch.from_numpy(ids.astype(np.int32)).to(DEV)
        group = np.where(ids < 0, count, ids)
        s["order"] = torch.from_numpy(np.argsort(group, kind="stable").astype(np.int32)).to(DEV)
        bounds = np.concatenate([[0], np.cumsum(np.bincount(group, minlength=count + 1)[:count])])
        s["offsets"], s["bounds"] = torch.from_numpy(bounds.astype(np.int32)).to(DEV), [int(v) for v in bounds]
    s["out"] = _buffers(case)
    return s


def _buffers(c):
    """The outputs' buffers, which a program that calls the same sizes again and again keeps."""
    op, m = c["op"], c["m"]

    def new(shape, t=torch.float32):
        return torch.empty(shape, dtype=t, device=DEV)

    if op == "route":
        slots = m * c["top"]
        return {"ids": new((m, c["top"]), torch.int32), "weights": new((m, c["top"])),
                "offsets": new((c["e"] + 1,), torch.int32), "order": new((slots,), torch.int32), "workspace": None}
    if op in ("experts", "gemv"):
        return {"y": new((m * c["top"], c["n"] // 2 if c["glu"] else c["n"]), TYPES[c["out"]] if op == "experts" else torch.float32)}
    if op == "combine":
        return {"out": new((m, c["n"]), TYPES[c["out"]])}
    return {"y": new((m, c["n"])), "workspace": None}


# ---------------------------------------------------------------------- run


def run(state):
    c = state["case"]
    return (_OWN if own else _PLAIN)[c["op"]](c, state)


def _workspace(b, size):
    """The state's workspace, made at the first call."""
    if b["workspace"] is None:
        b["workspace"] = torch.empty(max(size, 1), dtype=torch.uint8, device=DEV)
    return b["workspace"]


def _own_route(c, s):
    import block_quantized_matmul_02_amd as bqm

    b = s["out"]
    ids, weights = bqm.bqm_route(s["logits"], c["top"], c["renorm"], ids=b["ids"], weights=b["weights"])
    work = _workspace(b, bqm.bqm_group_rows_workspace(ids.numel(), c["e"]))
    offsets, order = bqm.bqm_group_rows(ids, c["e"], offsets=b["offsets"], order=b["order"], workspace=work)
    return {"ids": ids, "weights": weights, "offsets": offsets, "order": order}


def _own_experts(c, s):
    import block_quantized_matmul_02_amd as bqm

    return bqm.bqm_mxfp4_grouped_gemm(s["w"], s["ws"], s["xq"], s["xs"], s["offsets"], s["order"], glu=c["glu"], y=s["out"]["y"])


def _own_gemv(c, s):
    import block_quantized_matmul_02_amd as bqm

    return bqm.bqm_mxfp4_expert_gemv(s["w"], s["ws"], s["x"], s["ids"], glu=c["glu"], y=s["out"]["y"])


def _own_combine(c, s):
    import block_quantized_matmul_02_amd as bqm

    return bqm.bqm_combine(s["y"], s["weights"], s["res"], out=s["out"]["out"])


def _own_lora(c, s):
    import block_quantized_matmul_02_amd as bqm

    b = s["out"]
    work = _workspace(b, bqm.bqm_lora_add_workspace(c["m"], c["r"]))
    return bqm.bqm_lora_add(s["x"], s["a"], s["b"], s["offsets"], s["order"], scale=s["scale"], res=s["res"], y=b["y"],
                            workspace=work)


def _plain_route(c, s):
    x = s["logits"].float()
    # the largest first, the lowest index first among equals
    chosen = torch.sort(x, dim=1, descending=True, stable=True)
    ids, top = chosen.indices[:, :c["top"]], chosen.values[:, :c["top"]]
    e = torch.exp(top - top[:, :1])
    z = e.sum(1, keepdim=True) if c["renorm"] else torch.exp(x - top[:, :1]).sum(1, keepdim=True)
    flat = ids.reshape(-1)
    order = torch.sort(flat, stable=True).indices
    experts = torch.arange(c["e"] + 1, device=x.device)
    offsets = torch.searchsorted(flat[order], experts)
    return {"ids": ids.int(), "weights": e / z, "offsets": offsets.int(), "order": order.int()}


def _decode(codes, scales):
    rows, half = codes.shape
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    both = torch.stack((codes & 15, codes >> 4), 2).view(-1).int()
    v = torch.index_select(table, 0, both).view(rows, half // 16, 32)
    return (v * torch.exp2(scales.float() - 127.0)[:, :, None]).view(rows, 2 * half)


def _gated(y):
    half = y.shape[1] // 2
    gate, up = y[:, :half], y[:, half:]
    return gate / (1.0 + torch.exp(-gate)) * up


def _plain_experts(c, s):
    x = _decode(s["xq"], s["xs"])
    order, bounds = s["order"].long(), s["offsets"].tolist()
    rows = order // c["top"] if c["shared"] else order
    y = torch.zeros_like(s["out"]["y"])
    for e in range(c["e"]):
        lo, hi = bounds[e], bounds[e + 1]
        if lo < hi:
            p = x[rows[lo:hi]] @ _decode(s["w"][e], s["ws"][e]).t()
            y[order[lo:hi]] = (_gated(p) if c["glu"] else p).to(y.dtype)
    return y


def _plain_gemv(c, s):
    order, bounds = s["order"].long(), s["offsets"].tolist()
    rows = order // c["top"] if c["shared"] else order
    y = torch.zeros_like(s["out"]["y"])
    for e in range(c["e"]):
        lo, hi = bounds[e], bounds[e + 1]
        if lo < hi:
            p = s["x"][rows[lo:hi]] @ _decode(s["w"][e], s["ws"][e]).t()
            y[order[lo:hi]] = _gated(p) if c["glu"] else p
    return y


def _plain_combine(c, s):
    m, top = s["weights"].shape
    y = (s["y"].float().view(m, top, -1) * s["weights"][:, :, None]).sum(1)
    if s["res"] is not None:
        y = y + s["res"].float()
    return y.to(TYPES[c["out"]])


def _plain_lora(c, s):
    y = s["res"].clone()
    order, bounds = s["order"].long(), s["bounds"]
    for a in range(c["adapters"]):
        lo, hi = bounds[a], bounds[a + 1]
        if lo < hi:
            rows = order[lo:hi]
            h = s["x"][rows].float() @ s["a"][a].float().t()
            y[rows] += s["scale"][a] * (h @ s["b"][a].float().t())
    return y


_OWN = {"route": _own_route, "experts": _own_experts, "gemv": _own_gemv, "combine": _own_combine, "lora": _own_lora}
_PLAIN = {"route": _plain_route, "experts": _plain_experts, "gemv": _plain_gemv, "combine": _plain_combine,
          "lora": _plain_lora}


# -------------------------------------------------------------------- exact


def _exact_values(codes, scales):
    """The values of MXFP4 codes from the format's fields: sign, two exponent bits, one mantissa bit."""
    pair = torch.stack((codes.remainder(16), codes.div(16, rounding_mode="floor")), 2).reshape(codes.shape[0], -1).double()
    sign = torch.where(pair >= 8, -1.0, 1.0).double()
    low = pair.remainder(8)
    field, bit = (low / 2).floor(), low.remainder(2)
    v = torch.where(field == 0, bit / 2, (1 + bit / 2) * torch.pow(2.0, field - 1))
    return sign * v * torch.pow(2.0, scales.double() - 127).repeat_interleave(32, 1)


def exact(case, seed):
    s = prepare(case, seed)
    op, m = case["op"], case["m"]
    if op == "route":
        x = s["logits"].double()
        p = torch.softmax(x, 1)
        # stable: of equal logits the lower index stands first
        ids = torch.argsort(-x, dim=1, stable=True)[:, :case["top"]]
        w = p.gather(1, ids)
        if case["renorm"]:
            w = torch.softmax(x.gather(1, ids), 1)
        flat = ids.reshape(-1).cpu().numpy()
        order = np.argsort(flat, kind="stable")
        offsets = np.concatenate([[0], np.cumsum(np.bincount(flat, minlength=case["e"]))])
        return {"ids": ids.int(), "weights": w, "offsets": torch.from_numpy(offsets.astype(np.int32)),
                "order": torch.from_numpy(order.astype(np.int32))}
    if op in ("experts", "gemv"):
        x = s["x"].double() if op == "gemv" else _exact_values(s["xq"], s["xs"])
        if case["shared"]:
            x = x.repeat_interleave(case["top"], 0)
        flat = s["ids"].reshape(-1)
        n = case["n"]
        y = torch.empty((x.shape[0], n), dtype=torch.float64, device=DEV)
        for e in range(case["e"]):
            at = torch.nonzero(flat == e)[:, 0]
            if len(at):
                y[at] = x[at] @ _exact_values(s["w"][e], s["ws"][e]).t().contiguous()
        if case["glu"]:
            y = torch.nn.functional.silu(y[:, :n // 2]) * y[:, n // 2:]
        return y
    if op == "combine":
        y = s["y"].double().reshape(m, case["top"], -1)
        out = sum(s["weights"][:, j, None].double() * y[:, j] for j in range(case["top"]))
        return out if s["res"] is None else out + s["res"].double()
    y = s["res"].double()
    ids = s["ids"].long()
    for a in ids.unique().tolist():
        if a >= 0:
            at = torch.nonzero(ids == a)[:, 0]
            delta = (s["x"][at].double() @ s["a"][a].double().t().contiguous()) @ s["b"][a].double().t().contiguous()
            y[at] += float(s["scale"][a]) * delta
    return y
