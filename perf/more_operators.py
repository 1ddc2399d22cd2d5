"""Cases, plain forms and 64-bit forms of the operators that train adapters on an 8-bit base by
distillation: quantising to 8-bit floating point with a scale for each block of 128, the base's product and
its gradient in that form, a teacher's top logits, and the distillation loss with the gradient of its logits.

Shapes and symbols:

* 8-bit matrices: codes [rows, cols] of e4m3 or e5m2, fp32 scales [rows / b, cols / 128] (rounded up), b = 1
  for activations and gradients, 128 for weights.  Rows of codes are padded to 16 bytes.
* W is [N, K]: y = x W^T takes x [T, K], dx = dy W takes dy [T, N].
* logits: [T, V] rows of `ld` elements; a teacher's list: ids, values [T, k] and the log of the sum of
  exponentials (at the temperature) of everything that is not listed.
"""

import math
import random

import numpy as np
import torch

own = False

GROUP = 128  # columns (and rows of a weight's block) that share a scale
TINY = 2.0 ** -64  # a group whose largest value is below this holds zeros
LARGEST = {"e4m3": 448.0, "e5m2": 57344.0}
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
FLOAT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ----------------------------------------------------------------------- cases --

def _quant(name, **kw):
    c = dict(op="quantize", rows=1, cols=4096, block=1, dtype="bf16", type="e4m3", pow2=False)
    c.update(kw)
    return dict(c, name=name) if name else c


def _base(name, **kw):
    c = dict(op="base", T=1, K=4096, N=4096, back=False, out="bf16", type="e4m3")
    c.update(kw)
    return dict(c, name=name) if name else c


def _topk(name, **kw):
    c = dict(op="topk", T=16, V=32000, ld=32000, k=20, dtype="bf16", temperature=1.0)
    c.update(kw)
    return dict(c, name=name) if name else c


def _distill(name, **kw):
    c = dict(op="distill", T=16, V=32000, ld=32000, k=20, dtype="bf16", kind="forward", tail=True, temperature=1.0,
             ce=False)
    c.update(kw)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token's activations: a call whose time is launch latency
        _quant("quantize-token"),
        # gradients of a ragged batch, widths that end inside a group, scales that are powers of two
        _quant("quantize-odd-f32", rows=333, cols=1000, dtype="f32", type="e5m2", pow2=True),
        # a 13B-shaped layer's largest weight, once when the base is loaded
        _quant("quantize-weight", rows=13824, cols=5120, block=128),
        # eight requests' next tokens through one projection
        _base("base-decode", T=8),
        # a ragged batch, every size odd, logits wanted in fp32
        _base("base-odd-f32", T=333, K=1000, N=2050, out="f32"),
        # a prefill batch through a 13B-shaped MLP projection: the largest product
        _base("base-prefill", T=8192, K=5120, N=13824),
        # the gradient of a training batch's input through an MLP projection
        _base("base-backward", T=4096, K=4096, N=11008, back=True),
        # a teacher's list for one short answer, fp32 logits, softened
        _topk("topk-answer-f32", dtype="f32", temperature=2.0),
        # a teacher's lists for a training batch over a large vocabulary
        _topk("topk-batch", T=4096, V=128256, ld=128256, k=64),
        # one short answer: divergence of the student from the teacher, with the labels' cross-entropy, softened
        _distill("distill-answer-f32", T=90, V=32001, ld=32004, dtype="f32", kind="reverse", temperature=2.0, ce=True),
        # a batch over an odd vocabulary, rows on no 16-byte boundary, the symmetric divergence
        _distill("distill-odd-jsd", T=4000, V=50257, ld=50257, k=100, kind="jsd"),
        # a training batch over a large vocabulary: the largest logits
        _distill("distill-batch", T=8192, V=128256, ld=128256, k=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


WIDTHS = (328, 1000, 2056, 4096, 5120, 11008, 13824)


def _width(rng):
    return rng.choice(WIDTHS) if rng.random() < 0.5 else _log(rng, 64, 13824)


def draw(rng):
    op = rng.choice(["quantize", "base", "base", "base", "topk", "distill", "distill"])
    if op == "quantize":
        while True:
            c = _quant("", rows=_log(rng, 1, 13824), cols=_width(rng), block=rng.choice([1, 1, 128]),
                       dtype=rng.choice(["bf16", "bf16", "f32"]), type=rng.choice(["e4m3", "e4m3", "e5m2"]),
                       pow2=rng.random() < 0.3)
            if c["rows"] * c["cols"] <= 13824 * 5120:
                return c
    if op == "base":
        while True:
            c = _base("", T=_log(rng, 1, 8192), K=_width(rng), N=_width(rng), back=rng.random() < 0.4,
                      out=rng.choice(["bf16", "bf16", "f32"]), type=rng.choice(["e4m3", "e4m3", "e5m2"]))
            if c["T"] * c["K"] * c["N"] <= 8192 * 5120 * 13824:
                return c
    while True:
        T, V = _log(rng, 1, 8192), _log(rng, 200, 152064)
        if T * V <= 500e6:
            break
    kw = dict(T=T, V=V, ld=V + rng.choice([0, 0, -V % 8, 5]), dtype=rng.choice(["bf16", "bf16", "f32"]),
              k=_log(rng, 1, min(256, V // 2)), temperature=rng.choice([1.0, 1.0, 2.0, 0.7]))
    if op == "topk":
        return _topk("", **kw)
    kind = rng.choice(["forward", "reverse", "jsd"])
    return _distill("", kind=kind, tail=kind == "reverse" or rng.random() < 0.7, ce=rng.random() < 0.4, **kw)


def _out_shape(case):
    return (case["T"], case["K"] if case["back"] else case["N"])


def work(case):
    if case["op"] == "quantize":
        n = case["rows"] * case["cols"]
        scales = -(-case["rows"] // case["block"]) * -(-case["cols"] // GROUP)
        return {"bytes": n * (3 if case["dtype"] == "bf16" else 5) + 4 * scales, "flops": 3 * n}
    if case["op"] == "base":
        T, K, N = case["T"], case["K"], case["N"]
        inner = N if case["back"] else K
        read = T * inner + N * K + 4 * (T * -(-inner // GROUP) + -(-N // GROUP) * -(-K // GROUP))
        return {"bytes": read + math.prod(_out_shape(case)) * (2 if case["out"] == "bf16" else 4), "flops": 2 * T * N * K}
    b = 2 if case["dtype"] == "bf16" else 4
    n, lists = case["T"] * case["V"], 8 * case["T"] * case["k"]
    if case["op"] == "topk":
        return {"bytes": n * b + lists, "flops": 3 * n}
    return {"bytes": 2 * n * b + lists, "flops": 8 * n}


# --------------------------------------------------------------------- prepare --

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 2654435761 % (1 << 62) + 29)
    return g


def _activations(g, rows, cols, dtype):
    """Values as layers have them: rows and columns of different sizes, some entries far out, a silent group."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    x.mul_(torch.exp(torch.randn(rows, 1, generator=g, device="cuda")))
    x.mul_(torch.exp(0.5 * torch.randn(1, cols, generator=g, device="cuda")))
    x[:, 5 % cols:: 997].mul_(20.0)
    if rows > 2:
        x[rows // 2, : GROUP] = 0.0
    return x.to(dtype)


def _codes(rows, cols, type):
    """Zeroed codes, rows padded to 16 bytes."""
    return torch.zeros(rows, -(-cols // 16) * 16, dtype=torch.uint8, device="cuda").view(F8[type])[:, :cols]


def _prepare_base(case, g):
    T, K, N, back = case["T"], case["K"], case["N"], case["back"]
    inner = N if back else K
    s = {"y": torch.empty(_out_shape(case), dtype=FLOAT[case["out"]], device="cuda")}
    w = torch.randn(N, K, generator=g, device="cuda") * 0.02
    for name, x, block, type in (("x", _activations(g, T, inner, torch.float32), 1, case["type"]), ("w", w, GROUP, "e4m3")):
        codes, scales = _plain_quantize(x, block, type, False)
        padded = _codes(*x.shape, type)
        padded.view(torch.uint8).copy_(codes.view(torch.uint8))
        if block == 1:  # a group's scales of all the rows side by side
            scales = scales.t().contiguous().t()
        s[name], s[name + "s"] = padded, scales
    return s


def _distinct(T, V, k, g):
    """k entries of each row, no two alike: one in each of k stretches of the vocabulary, in any order."""
    at = torch.arange(k, device="cuda")
    lo, hi = at * V // k, (at + 1) * V // k
    ids = lo + (torch.rand(T, k, generator=g, device="cuda") * (hi - lo)).long().clamp(max=V // k - 1)
    return ids.gather(1, torch.rand(T, k, generator=g, device="cuda").argsort(1))


def _lists(case, g):
    """A teacher's list for each row: ids, values falling from the first on, and what the rest holds."""
    T, V, k, tau = case["T"], case["V"], case["k"], case["temperature"]
    ids = _distinct(T, V, k, g)
    values = 14.0 - torch.cumsum(torch.rand(T, k, generator=g, device="cuda") * (8.0 / k), 1)
    top = torch.logsumexp(values / tau, 1)
    tail = top - 0.5 - 4.0 * torch.rand(T, generator=g, device="cuda")
    return ids.to(torch.int32), values, tail


def prepare(case, seed):
    torch.cuda.set_device(0)
    g = _gen(seed)
    s = dict(case=case, err=torch.zeros(1, dtype=torch.int32, device="cuda"))
    if case["op"] == "quantize":
        s["x"] = _activations(g, case["rows"], case["cols"], FLOAT[case["dtype"]])
        s["codes"] = _codes(case["rows"], case["cols"], case["type"])
        groups, blocks = -(-case["cols"] // GROUP), -(-case["rows"] // case["block"])
        s["scales"] = torch.empty(groups, blocks, device="cuda").t() if case["block"] == 1 else torch.empty(blocks, groups, device="cuda")
    elif case["op"] == "base":
        s.update(_prepare_base(case, g))
    else:
        T, V, ld, k = case["T"], case["V"], case["ld"], case["k"]
        dtype = FLOAT[case["dtype"]]
        x = torch.randn(T, ld, generator=g, device="cuda", dtype=dtype)
        x.mul_(2.0)
        x[:, 3 % V: V: 997] = float("-inf")  # entries that the sampler forbids
        s["logits"] = x[:, :V]
        if case["op"] == "topk":
            # what the model thinks likely stands out, as it does in earnest
            likely = _distinct(T, V, 2 * k, g)
            x.scatter_(1, likely, (6.0 + 4.0 * torch.randn(T, 2 * k, generator=g, device="cuda")).to(dtype))
            s["ids"] = torch.empty(T, k, dtype=torch.int32, device="cuda")
            s["values"], s["tail"] = torch.empty(T, k, device="cuda"), torch.empty(T, device="cuda")
        else:
            ids, values, tail = _lists(case, g)
            # the student has learnt some of it
            student = values * 0.9 + 0.7 * torch.randn(T, k, generator=g, device="cuda")
            x.scatter_(1, ids.long(), student.to(dtype))
            s.update(ids=ids, values=values, tail=tail if case["tail"] else None)
            s["labels"] = ids[:, 0].clone()
            s["labels"][::7] = 1 % V
            s["labels"][::9] = -1  # the prompt's rows
            s["weight"] = (0.5 + torch.rand(T, generator=g, device="cuda")) / T
            s["loss"], s["kd"] = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
            s["grad"] = torch.zeros(T, ld, dtype=dtype, device="cuda")[:, :V]
    if own:  # the handles that a program keeps beside its buffers
        from segmented_gather_gemm_lora_gb300 import binding as B

        if case["op"] == "quantize":
            s["q"] = B.F8Matrix(s["codes"], s["scales"], block_rows=case["block"])
        elif case["op"] == "base":
            s["xq"], s["wq"] = B.F8Matrix(s["x"], s["xs"]), B.F8Matrix(s["w"], s["ws"], block_rows=GROUP)
    return s


MIX, KD_SCALE, CE_WEIGHT = 0.3, 1.0, 0.25


def _kd_weight(case):
    return KD_SCALE * case["temperature"] ** 2


# ----------------------------------------------------------------- plain forms --

def _plain_quantize(x, block, type, pow2):
    """(codes [rows, cols], scales [rows / block, cols / 128]) of x."""
    rows, cols = x.shape
    x = torch.nn.functional.pad(x.float(), (0, -cols % GROUP, 0, -rows % block))
    x = x.view(-1, block, x.shape[1] // GROUP, GROUP)
    top = x.abs().amax((1, 3))
    if pow2:  # the least power of two that the largest code reaches top with; that code is 0.875 of one too
        m, e = torch.frexp(top)
        scale = torch.ldexp(torch.ones_like(top), e - (9 if type == "e4m3" else 16) + (m > 0.875))
    else:
        scale = top / LARGEST[type]
    scale = torch.where(top < TINY, torch.zeros_like(scale), scale)
    s = scale[:, None, :, None]
    y = torch.where(s > 0, x / s, torch.zeros_like(x)).clamp(-LARGEST[type], LARGEST[type])
    y = y.view(-1, x.shape[2] * GROUP)[:rows, :cols]
    return y.to(F8[type]), scale


def _widen(codes, scales, block):
    """The fp32 values of an 8-bit matrix."""
    rows, cols = codes.shape
    s = scales.repeat_interleave(GROUP, 1)[:, :cols]
    if block > 1:
        s = s.repeat_interleave(block, 0)[:rows]
    return codes.float() * s


def _plain_base(s):
    x, w = _widen(s["x"], s["xs"], 1), _widen(s["w"], s["ws"], GROUP)
    return (x @ (w if s["case"]["back"] else w.t())).to(s["y"].dtype)


def _plain_topk(s):
    case = s["case"]
    x = s["logits"].float()
    # keys that order as the values do, then by falling index: whole numbers, no two alike
    bits = (x + 0.0).view(torch.int32)
    key = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long() * (1 << 32)
    key += torch.arange(case["V"] - 1, -1, -1, device="cuda")
    ids = torch.topk(key, case["k"], dim=1).indices
    del key, bits
    values = x.gather(1, ids)
    z = (x / case["temperature"]).scatter_(1, ids, float("-inf"))
    top = z.amax(1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    tail = top[:, 0] + torch.log(torch.exp(z - top).sum(1))
    return {"ids": ids.to(torch.int32), "values": values, "tail": tail}


def _plain_distill(s):
    case = s["case"]
    tau, k = case["temperature"], case["k"]
    x = s["logits"].float()
    ids = s["ids"].long()
    z = x / tau
    top = z.amax(1, keepdim=True)
    e = torch.exp(z - top)
    listed = e.gather(1, ids)
    e.scatter_(1, ids, 0.0)
    rest = e.sum(1, keepdim=True)  # of what is not listed: no difference of large sums
    total = rest + listed.sum(1, keepdim=True)
    logq = torch.cat([z.gather(1, ids) - top, torch.log(rest)], 1) - torch.log(total)
    tail = s["tail"][:, None] if case["tail"] else torch.full_like(rest, float("-inf"))
    logp = torch.cat([s["values"] / tau, tail], 1)
    high = logp.amax(1, keepdim=True)
    logp = logp - high - torch.log(torch.exp(logp - high).sum(1, keepdim=True))
    p, q = torch.exp(logp), torch.exp(logq)
    none = torch.zeros_like(p)
    # terms p log(p / q) - p + q: their sum is the divergence, and none of them is negative
    diverge = lambda p, q, d: torch.where(p > 0, p * d, none) - p + q  # noqa: E731
    d = logp - logq
    if case["kind"] == "forward":
        kd = diverge(p, q, d).sum(1)
        slope = -torch.expm1(d)
    elif case["kind"] == "reverse":
        kd = diverge(q, p, -d).sum(1)
        slope = -d - (q * -d).sum(1, keepdim=True)
    else:
        u = torch.log1p(MIX * torch.expm1(d))  # log of the mixture over q
        m = MIX * p + (1 - MIX) * q
        kd = (MIX * diverge(p, m, d - u) + (1 - MIX) * diverge(q, m, -u)).sum(1)
        slope = -(1 - MIX) * u
        slope = slope - (q * slope).sum(1, keepdim=True)
    on = s["labels"] >= 0
    part = slope * (_kd_weight(case) / tau)
    grad = e * (part[:, k:] / total)
    grad.scatter_(1, ids, q[:, :k] * part[:, :k])
    loss = _kd_weight(case) * kd
    if case["ce"]:
        at = s["labels"].long().clamp(min=0)[:, None]
        top = x.amax(1, keepdim=True)
        lse = top + torch.log(torch.exp(x - top).sum(1, keepdim=True))
        loss = loss + CE_WEIGHT * (lse - x.gather(1, at))[:, 0]
        grad += CE_WEIGHT * torch.exp(x - lse)
        grad.scatter_add_(1, at, torch.full_like(lse, -CE_WEIGHT))
    zero = torch.zeros_like(kd)
    grad = torch.where(on[:, None], grad * s["weight"][:, None], torch.zeros_like(grad))
    return {"loss": torch.where(on, s["weight"] * loss, zero), "kd": torch.where(on, kd, zero), "grad": grad.to(s["logits"].dtype)}


# ------------------------------------------------------------------------- run --

def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        if op == "quantize":
            codes, scales = _plain_quantize(s["x"], case["block"], case["type"], case["pow2"])
            return {"codes": codes, "scales": scales}
        return {"base": _plain_base, "topk": _plain_topk, "distill": _plain_distill}[op](s)
    from segmented_gather_gemm_lora_gb300 import binding as B

    if op == "quantize":
        B.lora_f8_quantize(s["x"], s["q"], pow2=case["pow2"], err=s["err"])
        return {"codes": s["codes"], "scales": s["scales"]}
    if op == "base":
        (B.lora_base_f8_backward if case["back"] else B.lora_base_f8)(s["xq"], s["wq"], s["y"], err=s["err"])
        return s["y"]
    if op == "topk":
        B.lora_topk_logits(s["logits"], s["ids"], s["values"], s["tail"], temperature=case["temperature"], err=s["err"])
        return {k: s[k] for k in ("ids", "values", "tail")}
    B.lora_distill_loss(s["logits"], s["ids"], s["values"], s["loss"], s["kd"], s["grad"], tail=s["tail"], labels=s["labels"],
                        weight=s["weight"], kind=getattr(B, "LORA_DISTILL_" + case["kind"].upper()), mix=MIX,
                        temperature=case["temperature"], kd_weight=_kd_weight(case), ce_weight=CE_WEIGHT if case["ce"] else 0.0,
                        err=s["err"])
    return {"loss": s["loss"], "kd": s["kd"], "grad": s["grad"]}


# --------------------------------------------------------------- 64-bit forms --

def _nearest_code(y, type):
    """The e4m3 or e5m2 value nearest to y, ties to the even code."""
    bits, low = (3, -6) if type == "e4m3" else (2, -14)
    a = y.abs().clamp(min=2.0 ** -40)
    unit = torch.exp2(torch.floor(torch.log2(a)).clamp(min=low) - bits)
    return (torch.round(y / unit) * unit).clamp(-LARGEST[type], LARGEST[type])


def _exact_quantize(s):
    case = s["case"]
    x, b = s["x"].double(), case["block"]
    rows, cols = x.shape
    scales = torch.zeros(-(-rows // b), -(-cols // GROUP), dtype=torch.float64, device="cuda")
    codes = torch.empty_like(x)
    for j in range(scales.shape[1]):
        part = x[:, j * GROUP: (j + 1) * GROUP]
        top = part.abs().max(dim=1).values
        if b > 1:
            top = torch.nn.functional.pad(top, (0, -rows % b)).view(-1, b).max(dim=1).values
        scale = top / LARGEST[case["type"]]
        if case["pow2"]:
            m, e = torch.frexp(scale)
            scale = torch.exp2(torch.where(m == 0.5, e - 1, e).double())
        # codes belong to the scale that is kept, which is fp32
        scale = torch.where(top < 2.0 ** -64, torch.zeros_like(scale), scale.float().double())
        each = scale.repeat_interleave(b)[:rows, None]
        codes[:, j * GROUP: (j + 1) * GROUP] = torch.where(
            each > 0, _nearest_code(part / torch.where(each > 0, each, torch.ones_like(each)), case["type"]), torch.zeros_like(part))
        scales[:, j] = scale
    return {"codes": codes, "scales": scales}


def _exact_base(s):
    case = s["case"]
    row = torch.arange(case["N"], device="cuda") // GROUP
    y = torch.zeros(_out_shape(case), dtype=torch.float64, device="cuda")
    inner = case["N"] if case["back"] else case["K"]
    w = s["w"].float().double()
    for a in range(0, inner, 16 * GROUP):  # some groups of the sum at a time
        b = min(inner, a + 16 * GROUP)
        col = torch.arange(a, b, device="cuda") // GROUP
        x = s["x"][:, a:b].float().double() * s["xs"].double()[:, col]
        if case["back"]:
            y += x @ (w[a:b] * s["ws"].double()[row[a:b]].repeat_interleave(GROUP, 1)[:, : case["K"]])
        else:
            y += x @ (w[:, a:b] * s["ws"].double()[row][:, col]).t()
    return y


def _exact_topk(s):
    case = s["case"]
    ids, values, tails = [], [], []
    for x in s["logits"].split(max(1, int(1e8) // case["V"])):
        v, i = torch.sort(x.double(), dim=1, descending=True, stable=True)
        ids.append(i[:, : case["k"]].to(torch.int32))
        values.append(v[:, : case["k"]])
        tails.append(torch.logsumexp(v[:, case["k"]:] / case["temperature"], 1))
    return {"ids": torch.cat(ids), "values": torch.cat(values), "tail": torch.cat(tails)}


def _exact_distill_rows(s, a, b):
    """(loss, kd, grad) of rows a to b: the loss's own derivatives with respect to the probabilities."""
    case = s["case"]
    tau, T = case["temperature"], b - a
    x = s["logits"][a:b].double()
    ids, lab = s["ids"][a:b].long(), s["labels"][a:b].long()
    q = torch.softmax(x / tau, 1)
    hidden = torch.ones_like(q, dtype=torch.bool).scatter_(1, ids, False)
    qt = (q * hidden).sum(1, keepdim=True)
    w = s["values"][a:b].double() / tau
    if case["tail"]:
        w = torch.cat([w, s["tail"][a:b, None].double()], 1)
    p = torch.softmax(w, 1)
    pt = p[:, case["k"]:] if case["tail"] else torch.zeros(T, 1, dtype=torch.float64, device="cuda")
    p = torch.cat([p[:, : case["k"]], pt], 1)
    qb = torch.cat([q.gather(1, ids), qt], 1)
    safe = lambda t: torch.where(t > 0, t, torch.ones_like(t))  # noqa: E731
    if case["kind"] == "forward":
        kd = (p * torch.log(safe(p) / qb)).sum(1)
        dq = -p / qb
    elif case["kind"] == "reverse":
        kd = (qb * torch.log(qb / p)).sum(1)
        dq = torch.log(qb / p)  # and 1, which the softmax takes away
    else:
        m = MIX * p + (1 - MIX) * qb
        kd = (MIX * p * torch.log(safe(p) / m) + (1 - MIX) * qb * torch.log(qb / m)).sum(1)
        dq = (1 - MIX) * torch.log(qb / m)
    dq = dq[:, -1:].expand(-1, case["V"]).scatter(1, ids, dq[:, : case["k"]])
    grad = _kd_weight(case) / tau * q * (dq - (q * dq).sum(1, keepdim=True))
    loss = _kd_weight(case) * kd
    if case["ce"]:
        loss = loss - CE_WEIGHT * torch.log_softmax(x, 1).gather(1, lab.clamp(min=0)[:, None])[:, 0]
        grad += CE_WEIGHT * torch.softmax(x, 1)
        grad.scatter_add_(1, lab.clamp(min=0)[:, None], torch.full((T, 1), -CE_WEIGHT, dtype=torch.float64, device="cuda"))
    on = (lab >= 0).double()
    weight = s["weight"][a:b].double() * on
    return weight * loss, on * kd, weight[:, None] * grad


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "distill":
        step = max(1, int(1e8) // case["V"])
        parts = [_exact_distill_rows(s, a, min(case["T"], a + step)) for a in range(0, case["T"], step)]
        return dict(zip(("loss", "kd", "grad"), (torch.cat(p) for p in zip(*parts))))
    return {"quantize": _exact_quantize, "base": _exact_base, "topk": _exact_topk}[case["op"]](s)
