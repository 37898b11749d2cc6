"""The operators around the projection matmul, as a user's program calls them,
over the sizes they meet:

* ``norm``     -- root-mean-square norm with the residual's addition, written
                  as f32 / 16-bit values or straight as the 8-bit operands of
                  the library's matmuls (q8_1, block-128 e4m3);
* ``quant``    -- microscaled 4-bit quantization (MXFP4: e2m1 values, one
                  power-of-two scale for every 32), and back;
* ``gemm``     -- the MXFP4 x MXFP4 product of a prefill or a small batch;
* ``gemv``     -- the decode / verify product: MXFP4 weights, f32 activations;
* ``logprobs`` -- log probabilities of given tokens, log-sum-exp, entropy and
                  the top alternatives of rows of logits.

``run`` computes them in plain torch operations, in 32 bits, or with ``own``
set through the library.  ``exact`` gives the results in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda:0"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-6
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # the norm ahead of a projection in one decode step: one token, latency counts
        dict(name="norm_decode", op="norm", m=1, k=4096, type="f32", out="f32", res=True),
        # a ragged prefill chunk, quantized for the Q8_0 products
        dict(name="norm_q8_chunk", op="norm", m=333, k=4096, type="f32", out="q8_1", res=True),
        # a long prefill with a 16-bit residual stream, quantized for the block-128 FP8 product
        dict(name="norm_e4m3_prefill", op="norm", m=8192, k=5120, type="bf16", out="e4m3", res=True),
        # the activations of a verify batch, to 4 bits
        dict(name="quant_verify", op="quant", m=9, k=4096, type="f32"),
        # a projection's weights as they are loaded, or a long prefill's activations, to 4 bits
        dict(name="quant_prefill", op="quant", m=5120, k=17408, type="bf16"),
        # a small batch against one projection
        dict(name="gemm_batch16", op="gemm", m=16, k=4096, n=5152),
        # a prefill chunk against the widest projection
        dict(name="gemm_prefill", op="gemm", m=512, k=4096, n=20480),
        # a long, odd prefill
        dict(name="gemm_long", op="gemm", m=3001, k=5120, n=17408),
        # one decode step of a square projection
        dict(name="gemv_decode", op="gemv", m=1, k=4096, n=4096),
        # the head's rows for a verify batch
        dict(name="gemv_verify_head", op="gemv", m=9, k=4096, n=64448),
        # one sampled token with its 20 alternatives
        dict(name="logprobs_decode", op="logprobs", m=1, n=64448, type="f32", t=1, top=20),
        # a prompt's tokens scored, with 5 alternatives each
        dict(name="logprobs_prompt", op="logprobs", m=512, n=131071, type="f32", t=1, top=5),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    most = {}
    for c in listed():
        w = work(c)
        most[c["op"]] = max(most.get(c["op"], (0, 0)), (w["bytes"] + w["flops"] / 300, w["flops"]))
    while True:
        op = rng.choice(["norm", "quant", "gemm", "gemv", "logprobs"])
        if op == "norm":
            out = rng.choice(["f32", "same", "q8_1", "e4m3"])
            k = {"f32": 1, "same": 1, "q8_1": 32, "e4m3": 16}[out]
            c = dict(op=op, m=spread(1, 16384), k=k * max(1, spread(256, 20480) // k),
                     type=rng.choice(["f32", "bf16", "f16"]), out=out, res=rng.random() < 0.75)
        elif op == "quant":
            c = dict(op=op, m=spread(1, 20480), k=32 * spread(8, 544), type=rng.choice(["f32", "bf16", "f16"]))
        elif op == "gemm":
            c = dict(op=op, m=spread(1, 4096), k=32 * spread(8, 544), n=spread(64, 20480))
        elif op == "gemv":
            c = dict(op=op, m=rng.randint(1, 16), k=32 * spread(8, 544), n=spread(64, 64448))
        else:
            c = dict(op=op, m=spread(1, 2048), n=spread(2000, 262144), type=rng.choice(["f32", "bf16", "f16"]),
                     t=rng.choice([1, 1, 2, 7]), top=rng.choice([0, 1, 5, 20, 32]))
        w = work(c)
        if w["bytes"] + w["flops"] / 300 <= most[op][0] and w["flops"] <= most[op][1]:
            return c


def work(case):
    """Bytes and operations of one pass: every input read once, every output written once."""
    op, m = case["op"], case["m"]
    if op == "norm":
        k, s = case["k"], SIZE[case["type"]]
        out = {"f32": 4.0, "same": float(s), "q8_1": 1.25, "e4m3": 1.0 + 4.0 / 128}[case["out"]]
        return {"bytes": m * k * (s * (3 if case["res"] else 1) + out) + 4 * k, "flops": 5 * m * k}
    if op == "quant":
        # read the values, write codes and scales, write the values they stand for
        k, s = case["k"], SIZE[case["type"]]
        return {"bytes": m * k * (s + 2 + 17 / 32), "flops": 4 * m * k}
    if op == "gemm":
        k, n = case["k"], case["n"]
        return {"bytes": (m + n) * k * 17 / 32 + 4 * m * n, "flops": 2 * m * k * n}
    if op == "gemv":
        k, n = case["k"], case["n"]
        return {"bytes": n * k * 17 / 32 + 4 * m * (k + n), "flops": 2 * m * k * n}
    n, s = case["n"], SIZE[case["type"]]
    return {"bytes": m * n * s + m * (8 * case["t"] + 8 + 8 * case["top"]), "flops": 6 * m * n}


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


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    op, m = case["op"], case["m"]
    if op == "norm":
        k, t = case["k"], TYPES[case["type"]]
        s["x"] = _outliers(_normal((m, k), g), g).to(t)
        s["res"] = _normal((m, k), g, 4.0).to(t) if case["res"] else None
        s["gain"] = 1.0 + _normal((k,), g, 0.1)
    elif op == "quant":
        s["x"] = _outliers(_normal((m, case["k"]), g), g).to(TYPES[case["type"]])
    elif op == "gemm":
        s["w"], s["ws"] = _mx_random(case["n"], case["k"], g, 117, 121)     # weights of about 0.02
        s["xq"], s["xs"] = _mx_random(m, case["k"], g, 125, 128)            # activations of about 1
    elif op == "gemv":
        s["w"], s["ws"] = _mx_random(case["n"], case["k"], g, 117, 121)
        s["x"] = _outliers(_normal((m, case["k"]), g), g)
    else:
        n = case["n"]
        x = _normal((m, n), g, 2.5)
        # every fourth row under a grammar's mask that leaves about a tenth of the tokens
        cut = torch.rand((m, n), generator=g, device=DEV) < 0.9
        cut[torch.arange(m, device=DEV) % 4 != 3] = False
        s["logits"] = x.masked_fill_(cut, -math.inf).to(TYPES[case["type"]])
        del x, cut
        s["tokens"] = torch.randint(0, n, (m, case["t"]), generator=g, device=DEV, dtype=torch.int32)
    s["out"] = _buffers(case)
    return s


def _buffers(c):
    """The outputs' buffers, which a program that calls the same sizes again and again keeps."""
    op, m = c["op"], c["m"]

    def new(shape, t=torch.float32):
        return torch.empty(shape, dtype=t, device=DEV)

    if op == "norm":
        k, t = c["k"], TYPES[c["type"]]
        b = {"h": new((m, k), t) if c["res"] else None}
        if c["out"] == "q8_1":
            return b | {"xq": new((m, k), torch.int8), "xds": new((m, k // 32, 2))}
        if c["out"] == "e4m3":
            return b | {"xq": new((m, k), torch.uint8), "xs": new((m, -(-k // 128)))}
        return b | {"y": new((m, k), torch.float32 if c["out"] == "f32" else t)}
    if op == "quant":
        k = c["k"]
        return {"codes": new((m, k // 2), torch.uint8), "scales": new((m, k // 32), torch.uint8),
                "values": new((m, k), torch.bfloat16)}
    if op == "logprobs":
        return {"out": (new((m, c["t"])), new((m,)), new((m,)), new((m, c["top"]), torch.int32), new((m, c["top"])))}
    return {"y": new((m, c["n"]))}


# ---------------------------------------------------------------------- run


def run(state):
    c = state["case"]
    return (_OWN if own else _PLAIN)[c["op"]](c, state)


def _own_norm(c, s):
    import block_quantized_matmul_02_amd as bqm

    b = s["out"]
    if c["out"] == "q8_1":
        xq, xds, h = bqm.bqm_add_rmsnorm_q8_1(s["x"], s["res"], s["gain"], EPS, h=b["h"], xq=b["xq"], xds=b["xds"])
        return {"h": h, "q": xq.to(torch.bfloat16), "d": xds[..., 0], "s": xds[..., 1].to(torch.bfloat16)}
    if c["out"] == "e4m3":
        xq, xs, h = bqm.bqm_add_rmsnorm_e4m3_blk(s["x"], s["res"], s["gain"], EPS, h=b["h"], xq=b["xq"], xs=b["xs"])
        return {"h": h, "q": xq.view(torch.float8_e4m3fn), "d": xs}
    y, h = bqm.bqm_add_rmsnorm(s["x"], s["res"], s["gain"], EPS, h=b["h"], y=b["y"])
    return {"h": h, "y": y}


def _own_quant(c, s):
    import block_quantized_matmul_02_amd as bqm

    b = s["out"]
    codes, scales = bqm.bqm_mxfp4_quantize(s["x"], codes=b["codes"], scales=b["scales"])
    return {"values": bqm.bqm_mxfp4_dequantize(codes, scales, y=b["values"]), "scales": scales}


def _own_gemm(c, s):
    import block_quantized_matmul_02_amd as bqm

    return bqm.bqm_mxfp4_gemm(s["w"], s["ws"], s["xq"], s["xs"], y=s["out"]["y"])


def _own_gemv(c, s):
    import block_quantized_matmul_02_amd as bqm

    return bqm.bqm_mxfp4_gemv(s["w"], s["ws"], s["x"], y=s["out"]["y"])


def _own_logprobs(c, s):
    import block_quantized_matmul_02_amd as bqm

    logp, lse, entropy, ids, top = bqm.bqm_logprobs(s["logits"], s["tokens"], c["top"], out=s["out"]["out"])
    return {"logp": logp, "lse": lse, "entropy": entropy, "ids": ids, "top": top}


def _plain_norm(c, s):
    x = s["x"].float()
    h = None
    if s["res"] is not None:
        x = x + s["res"].float()
        h = x.to(s["x"].dtype)
    y = x * (1.0 / torch.sqrt((x * x).mean(1, keepdim=True) + EPS)) * s["gain"]
    m, k = y.shape
    if c["out"] == "q8_1":
        b = y.view(m, k // 32, 32)
        d = b.abs().amax(2, keepdim=True) / 127.0
        v = b / torch.where(d > 0, d, torch.ones_like(d))
        # round half away from zero: the fraction that the division left is exact
        whole = torch.trunc(v)
        q = (whole + torch.sign(v) * ((v - whole).abs() >= 0.5)).clamp(-127, 127)
        total = d[..., 0] * q.sum(2)
        return {"h": h, "q": q.view(m, k).to(torch.bfloat16), "d": d[..., 0], "s": total.to(torch.bfloat16)}
    if c["out"] == "e4m3":
        kb = -(-k // 128)
        b = torch.nn.functional.pad(y, (0, kb * 128 - k)).view(m, kb, 128)
        a = b.abs().amax(2, keepdim=True)
        mul = torch.where(a > 0, 448.0 / a, torch.zeros_like(a))
        q = (b * mul).clamp(-448, 448).view(m, kb * 128)[:, :k].to(torch.float8_e4m3fn)
        return {"h": h, "q": q, "d": a[..., 0] / 448.0}
    return {"h": h, "y": y if c["out"] == "f32" else y.to(s["x"].dtype)}


def _plain_quant(c, s):
    x = s["x"].float()
    m, k = x.shape
    b = x.view(m, k // 32, 32)
    a = b.abs().amax(2, keepdim=True)
    # floor(log2 a) - 2, from the exponent that frexp gives (a = f * 2^e, 0.5 <= f < 1)
    e = (torch.frexp(a).exponent - 3).clamp(-127, 125)
    e = torch.where(a > 0, e, torch.full_like(e, -127))
    v = torch.ldexp(b, -e).abs()
    steps = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=x.device)
    # the code is the number of midpoints below; a value on a midpoint goes to the even code
    up, low = torch.bucketize(v, steps, right=True), torch.bucketize(v, steps)
    code = torch.where(up % 2 == 0, up, low)
    r = torch.ldexp(torch.tensor(E2M1, device=x.device)[code], e)
    r = torch.copysign(r, b).view(m, k).to(torch.bfloat16)
    return {"values": r, "scales": (e[..., 0] + 127).to(torch.uint8)}


def _decode(codes, scales):
    rows, half = codes.shape
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    both = torch.stack((codes & 15, codes >> 4), 2).view(-1).int()
    v = torch.index_select(table, 0, both).view(rows, half // 16, 32)
    return (v * torch.exp2(scales.float() - 127.0)[:, :, None]).view(rows, 2 * half)


def _plain_gemm(c, s):
    return _decode(s["xq"], s["xs"]) @ _decode(s["w"], s["ws"]).t()


def _plain_gemv(c, s):
    return s["x"] @ _decode(s["w"], s["ws"]).t()


def _plain_logprobs(c, s):
    x, tokens = s["logits"].float(), s["tokens"].long()
    top = x.amax(1, keepdim=True)
    d = x - torch.where(top > -math.inf, top, torch.zeros_like(top))
    e = torch.exp(d)
    z = e.sum(1, keepdim=True)
    logz = torch.log(z)
    lse = top + logz
    entropy = logz - torch.where(e > 0, e * d, torch.zeros_like(e)).sum(1, keepdim=True) / z
    logp = d.gather(1, tokens) - logz
    # the k largest, the lowest index first among equals: one whole key for both
    n = x.shape[1]
    bits = (x + 0.0).view(torch.int32)
    order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long()
    key = (order << 32) + (n - 1 - torch.arange(n, device=x.device))
    ids = n - 1 - (torch.topk(key, c["top"], 1).values & 0xFFFFFFFF)
    return {"logp": logp, "lse": lse[:, 0], "entropy": entropy[:, 0], "ids": ids.int(), "top": d.gather(1, ids) - logz}


_OWN = {"norm": _own_norm, "quant": _own_quant, "gemm": _own_gemm, "gemv": _own_gemv, "logprobs": _own_logprobs}
_PLAIN = {"norm": _plain_norm, "quant": _plain_quant, "gemm": _plain_gemm, "gemv": _plain_gemv,
          "logprobs": _plain_logprobs}


# -------------------------------------------------------------------- exact


def _grid_round(v, mantissa, lowest):
    """Each value to the nearest with `mantissa` bits after the leading one, spacing no finer than 2^lowest; ties to even."""
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), torch.clamp(e - 1 - mantissa, min=lowest))
    return torch.round(v / step) * step


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
    if op == "norm":
        x = s["x"].double()
        h = None
        if s["res"] is not None:
            x = x + s["res"].double()
            h = x
        y = x / torch.sqrt(x.pow(2).sum(1, keepdim=True) / x.shape[1] + EPS) * s["gain"].double()
        k = y.shape[1]
        if case["out"] == "q8_1":
            b = y.reshape(m, -1, 32)
            d = b.abs().max(2, keepdim=True).values / 127
            v = b / d
            q = torch.sign(v) * torch.floor(v.abs() + 0.5)
            return {"h": h, "q": q.reshape(m, k), "d": d[..., 0], "s": (d * q).sum(2)}
        if case["out"] == "e4m3":
            edges = range(0, k, 128)
            a = torch.stack([y[:, i:i + 128].abs().max(1).values for i in edges], 1)
            v = y * (448 / a).repeat_interleave(128, 1)[:, :k]
            return {"h": h, "q": _grid_round(v, 3, -9), "d": a / 448}
        return {"h": h, "y": y}
    if op == "quant":
        x = s["x"].double().reshape(m, -1, 32)
        a = x.abs().max(2, keepdim=True).values
        e = torch.floor(torch.log2(a)) - 2
        v = _grid_round(x / torch.pow(2.0, e), 1, -1).clamp(-6, 6) * torch.pow(2.0, e)
        return {"values": v.reshape(m, -1), "scales": (e[..., 0] + 127).to(torch.uint8)}
    if op == "gemm":
        return _exact_values(s["xq"], s["xs"]) @ _exact_values(s["w"], s["ws"]).t().contiguous()
    if op == "gemv":
        return s["x"].double() @ _exact_values(s["w"], s["ws"]).t().contiguous()
    logits = s["logits"].double()
    lse = torch.logsumexp(logits, 1)
    logp = logits - lse[:, None]
    order = torch.sort(logits, dim=1, descending=True, stable=True)
    p = torch.exp(logp)
    return {"logp": logp.gather(1, s["tokens"].long()), "lse": lse,
            "entropy": -torch.nan_to_num(p * logp, nan=0.0).sum(1),
            "ids": order.indices[:, :case["top"]].int(), "top": order.values[:, :case["top"]] - lse[:, None]}
