"""Cases, plain forms and 64-bit forms of the adapter-training operators: the optimizer step
over a paged adapter pool, per-token log-probabilities, the paired preference loss and the
clipped policy loss, each with the gradient of its logits.

Shapes and symbols:

* adapters: the paged pool of the LoRA calls.  A_i is r_i rows of d_in elements, B_i r_i rows of
  d_out; a matrix's element e sits at pool[page_list[page0 + e // P] * P + e % P].  Gradients,
  fp32 weights and moments use the same positions.  Moments are fp32, or e4m3 codes with one
  bf16 scale for each 64 consecutive elements (the first moment, and the root of the second).
* logits: [T, V] rows of `ld` elements, labels [T] (negative: the row does not count).
"""

import random

import numpy as np
import torch

own = False

BLOCK = 64  # elements that share one scale of an 8-bit moment
E4M3_MAX = 448.0
TINY = 2.0 ** -100  # a block whose largest value is below this holds zeros


# ----------------------------------------------------------------------- cases --

# (d_in, d_out) of the projections of one call
SHAPES = {
    "q4096": ((4096, 4096),),
    "qkvo4096": ((4096, 4096),) * 4,
    "layer4096": ((4096, 4096),) * 4 + ((4096, 11008),) * 2 + ((11008, 4096),),
    "layer5120": ((5120, 5120),) * 4 + ((5120, 13824),) * 2 + ((13824, 5120),),
    "odd": ((1000, 2056), (2056, 328)),
}


def _adamw(name, **kw):
    c = dict(op="adamw", shapes="q4096", n=1, rank_lo=8, rank_hi=8, page=4096, state="f32", master=False,
             clip=False, zero=False, plan=1)
    c.update(kw)
    return dict(c, name=name) if name else c


def _rows(op, name, **kw):
    c = dict(op=op, T=16, V=32000, ld=32000, dtype="bf16", plan=1)
    if op == "pref":
        c.update(pairs=1, kind="sigmoid", average=False)
    c.update(kw)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one tenant's rank-8 adapter of one projection: a call whose time is launch latency
        _adamw("adamw-one-adapter"),
        # eight tenants of mixed ranks on the attention projections, fp32 weights kept, norms clipped
        _adamw("adamw-attention-clip", shapes="qkvo4096", n=8, rank_lo=8, rank_hi=64, master=True, clip=True),
        # one layer's seven projections, sixteen tenants, 8-bit moments, gradients cleared in the same pass
        _adamw("adamw-layer-8bit", shapes="layer4096", n=16, rank_lo=8, rank_hi=64, state="e4m3", clip=True, zero=True),
        # widths and ranks that end inside a page and inside a block of 64, the smallest pages
        _adamw("adamw-odd-8bit", shapes="odd", n=37, rank_lo=1, rank_hi=13, page=64, state="e4m3", zero=True),
        # many tenants on a 13B-shaped layer, fp32 moments and weights: the memory-bound end
        _adamw("adamw-13b-layer", shapes="layer5120", n=48, rank_lo=16, rank_hi=64, master=True, clip=True, zero=True),
        # the reference log-probabilities of one short answer
        _rows("logprobs", "logprobs-short"),
        # a batch of answers over a large odd vocabulary, rows on no 16-byte boundary
        _rows("logprobs", "logprobs-batch", T=4000, V=50257, ld=50257),
        # one pair of short answers
        _rows("pref", "pref-pair", T=90, pairs=1),
        # fp32 logits of an odd vocabulary, squared loss on length-normalised log ratios
        _rows("pref", "pref-odd-f32", T=700, V=32001, ld=32004, dtype="f32", pairs=3, kind="ipo", average=True),
        # a training batch of pairs
        _rows("pref", "pref-batch", T=8192, pairs=8),
        # one sampled answer with fp32 logits
        _rows("policy", "policy-answer-f32", T=200, V=32000, dtype="f32"),
        # a rollout batch over a large vocabulary: the largest logits
        _rows("policy", "policy-rollouts", T=8192, V=128256, ld=128256),
    ]


def _log(rng, lo, hi):
    return int(round(np.exp(rng.uniform(np.log(lo), np.log(hi)))))


def draw(rng):
    op = rng.choice(["adamw", "adamw", "logprobs", "pref", "policy"])
    if op == "adamw":
        state = rng.choice(["f32", "e4m3"])
        lo = rng.choice([1, 4, 8, 16])
        while True:
            c = _adamw("", shapes=rng.choice(sorted(SHAPES)), n=_log(rng, 1, 48), rank_lo=lo, rank_hi=rng.randint(lo, 64),
                       page=64 << rng.randint(0, 6), state=state, master=state == "f32" and rng.random() < 0.5,
                       clip=rng.random() < 0.6, zero=rng.random() < 0.5, plan=rng.randrange(1 << 20))
            if _elements(c) <= 130e6:
                return c
    while True:
        T, V = _log(rng, 1 if op != "pref" else 2, 8192), _log(rng, 200, 152064)
        if T * V <= 400e6:
            break
    kw = dict(T=T, V=V, ld=V + rng.choice([0, 0, -V % 8, 5]), dtype=rng.choice(["bf16", "bf16", "f32"]),
              plan=rng.randrange(1 << 20))
    if op == "pref":
        kw.update(pairs=max(1, min(T // 2, _log(rng, 1, 64))), kind=rng.choice(["sigmoid", "ipo", "hinge"]),
                  average=rng.random() < 0.3)
    return _rows(op, "", **kw)


# ---------------------------------------------------- what a case's plan fixes --

def _ranks(case):
    r = random.Random(case["plan"])
    return [r.randint(case["rank_lo"], case["rank_hi"]) for _ in range(case["n"])]


def _elements(case):
    return sum(r * (a + b) for r in _ranks(case) for a, b in SHAPES[case["shapes"]])


def _sequences(case):
    """(seq_indptr, counted rows as a list of (begin, end)): each sequence's first third is its prompt."""
    r = random.Random(case["plan"] + 1)
    n = 2 * case.get("pairs", 1)
    cuts = sorted(r.sample(range(1, case["T"]), n - 1)) if case["T"] > n else list(range(1, n))
    indptr = [0] + cuts + [case["T"]]
    return indptr, [(a + (b - a) // 3, b) for a, b in zip(indptr, indptr[1:])]


def _counted(case):
    if case["op"] == "logprobs":
        return case["T"]
    if case["op"] == "policy":
        return case["T"] - case["T"] // 8
    return sum(b - a for a, b in _sequences(case)[1])


def work(case):
    if case["op"] == "adamw":
        e = _elements(case)
        f32 = case["state"] == "f32"
        # gradient; moments in and out; weights in and out (with fp32 weights, the bf16 ones out only); cleared gradient
        per = 4 + (16 if f32 else 4) + (10 if case["master"] else 4) + (4 if case["zero"] else 0)
        return {"bytes": e * per + (0 if f32 else e / BLOCK * 8), "flops": e * 20}
    b = 2 if case["dtype"] == "bf16" else 4
    rows = _counted(case)
    read = rows * case["V"] * b
    write = 0 if case["op"] == "logprobs" else case["T"] * case["V"] * b
    return {"bytes": read + write + case["T"] * 16, "flops": rows * case["V"] * (4 if case["op"] == "logprobs" else 8)}


# --------------------------------------------------------------------- prepare --

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 2654435761 % (1 << 62) + 17)
    return g


def _prepare_adamw(case, seed):
    g = _gen(seed)
    rng = np.random.default_rng(seed)
    P, n = case["page"], case["n"]
    ranks = _ranks(case)
    n_adapters = 2 * n
    ids = rng.permutation(n_adapters)[:n].astype(np.int32)
    projs, n_pages = [], 0
    for d_in, d_out in SHAPES[case["shapes"]]:
        na = [-(-r * d_in // P) for r in ranks]
        nb = [-(-r * d_out // P) for r in ranks]
        total = sum(na) + sum(nb)
        phys = rng.permutation(total + 3).astype(np.int32)
        desc = np.zeros((n_adapters, 4), dtype=np.int32)
        at = 0
        for k, i in enumerate(ids):
            desc[i] = (ranks[k], np.float32(16.0 / ranks[k]).view(np.int32), at, at + na[k])
            at += na[k] + nb[k]
        projs.append(dict(d_in=d_in, d_out=d_out, page0=n_pages, pages=total + 3, list_host=phys[:total], desc_host=desc,
                          page_list=torch.from_numpy(phys[:total].copy()).cuda(), desc=torch.from_numpy(desc).cuda()))
        n_pages += total + 3
    # blocks of 64 in listed order: adapter, projection, A then B; `keep` marks the owned elements of each
    blocks, left, counts = [], [], []
    for k, i in enumerate(ids):
        count = 0
        for p in projs:
            for slot, d in ((int(p["desc_host"][i, 2]), p["d_in"]), (int(p["desc_host"][i, 3]), p["d_out"])):
                size = ranks[k] * d
                first = np.arange(0, size, BLOCK, dtype=np.int64)
                page = p["page0"] + p["list_host"][slot + first // P].astype(np.int64)
                blocks.append((page * P + first % P) // BLOCK)
                left.append(np.minimum(size - first, BLOCK))
                count += first.size
        counts.append(count)
    blocks, left, counts = np.concatenate(blocks), np.concatenate(left), np.array(counts)
    widest = int(counts.max())
    starts = np.concatenate([[0], np.cumsum(counts)[:-1]])
    rows = np.minimum(starts[:, None] + np.arange(widest)[None, :], blocks.size - 1)
    plan = dict(blocks=torch.from_numpy(blocks).cuda(),
                keep=torch.arange(BLOCK, device="cuda")[None, :] < torch.from_numpy(left).cuda()[:, None],
                entry=torch.repeat_interleave(torch.arange(n, device="cuda"), torch.from_numpy(counts).cuda()),
                rows=torch.from_numpy(rows).cuda(),
                has=torch.arange(widest, device="cuda")[None, :] < torch.from_numpy(counts).cuda()[:, None])
    size = n_pages * P
    w = torch.randn(size, generator=g, device="cuda") * 0.02
    # gradients and moments of one size inside a block, of many sizes between blocks
    level = torch.exp(torch.randn(size // BLOCK, 1, generator=g, device="cuda")) * 1e-3
    grad = (torch.randn(size // BLOCK, BLOCK, generator=g, device="cuda") * level).view(-1)
    m = (torch.randn(size // BLOCK, BLOCK, generator=g, device="cuda") * level * 0.3).view(-1)
    v = ((0.5 + torch.rand(size // BLOCK, BLOCK, generator=g, device="cuda")) * level).square().view(-1)
    s = dict(case=case, projs=projs, ids=torch.from_numpy(ids).cuda(), ids_host=ids, ranks=ranks, plan=plan, grad=grad,
             pool=w.to(torch.bfloat16), master=w if case["master"] else None)
    if case["state"] == "f32":
        s.update(m=m, v=v, m_scale=None, v_scale=None)
    else:
        keep = torch.ones(size // BLOCK, BLOCK, dtype=torch.bool, device="cuda")
        (mc, ms), (vc, vs) = _quantise(m.view(-1, BLOCK), keep), _quantise(v.sqrt().view(-1, BLOCK), keep, floor=True)
        s.update(m=mc.view(-1), v=vc.view(-1), m_scale=ms, v_scale=vs)
    # per adapter id: step, lr, beta1, beta2, eps, weight_decay, max_norm, grad_scale
    hyper = np.zeros((n_adapters, 8), dtype=np.float32)
    hyper[:, 1:] = (1e-4, 0.9, 0.999, 1e-8, 0.01, 0.5 if case["clip"] else 0.0, 0.5)
    hyper[:, 1] *= rng.uniform(0.5, 2.0, n_adapters).astype(np.float32)
    hyper[:, 0] = rng.integers(1, 2000, n_adapters).astype(np.int32).view(np.float32)
    s["hyper"] = torch.from_numpy(hyper).cuda()
    s["sumsq"] = torch.zeros(n_adapters, device="cuda")
    s["err"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if own:  # the handle that a program keeps beside its buffers
        from segmented_gather_gemm_lora_gb300 import binding as B

        sets = []
        for p in projs:
            a, b = p["page0"] * P, (p["page0"] + p["pages"]) * P
            cut = lambda t, q=1: None if t is None else t[a // q: b // q]  # noqa: E731
            view = B.PoolView(s["pool"][a:b].view(-1, P), p["page_list"], p["desc"], P, case["rank_hi"], p["d_in"], p["d_out"])
            sets.append(B.TrainProj(view, cut(s["grad"]), cut(s["m"]), cut(s["v"]), master=cut(s["master"]),
                                    m_scale=cut(s["m_scale"], BLOCK), v_scale=cut(s["v_scale"], BLOCK)))
        s["set"] = B.TrainSet(sets)
        s["space"] = s["set"].sumsq_workspace(n) if case["clip"] else None
    return s


def _labels(case, seed):
    rng = np.random.default_rng(seed + 99)
    lab = rng.integers(0, case["V"], case["T"]).astype(np.int32)
    if case["op"] == "pref":
        keep = np.zeros(case["T"], dtype=bool)
        for a, b in _sequences(case)[1]:
            keep[a:b] = True
        lab[~keep] = -1
    elif case["op"] == "policy":  # the prompt's rows
        lab[rng.permutation(case["T"])[: case["T"] // 8]] = -1
    return torch.from_numpy(lab).cuda()


def prepare(case, seed):
    torch.cuda.set_device(0)
    if case["op"] == "adamw":
        return _prepare_adamw(case, seed)
    g = _gen(seed)
    T, V, ld = case["T"], case["V"], case["ld"]
    dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    x = torch.randn(T, ld, generator=g, device="cuda", dtype=dtype)
    x.mul_(2.0)
    lab = _labels(case, seed)
    # the label's logit is raised, as a model that has learnt something has it
    at = lab.long().clamp(min=0)[:, None]
    x.scatter_add_(1, at, (torch.rand(T, 1, generator=g, device="cuda") * 12).to(dtype))
    x[:, 3 % V: V: 997] = float("-inf")  # entries that the sampler forbids
    x.scatter_(1, at, x.gather(1, at).clamp(min=-8.0))
    s = dict(case=case, logits=x[:, :V], labels=lab, err=torch.zeros(1, dtype=torch.int32, device="cuda"),
             logp=torch.empty(T, device="cuda"), lse=torch.empty(T, device="cuda"))
    if case["op"] == "logprobs":
        return s
    s["grad"] = torch.zeros(T, ld, dtype=dtype, device="cuda")[:, :V]
    lp = _plain_logprobs(s["logits"], lab)[0]
    near = lambda d: lp + d * torch.randn(T, generator=g, device="cuda")  # noqa: E731
    s["ref"] = near(0.3)
    s["loss"] = torch.empty(T, device="cuda")
    if case["op"] == "policy":
        s["old"] = near(0.15)
        s["adv"] = torch.randn(T, generator=g, device="cuda")
        s["weight"] = (0.5 + torch.rand(T, generator=g, device="cuda")) / T
        s["kl"] = torch.empty(T, device="cuda")
        return s
    indptr = _sequences(case)[0]
    n = 2 * case["pairs"]
    widest = max(b - a for a, b in zip(indptr, indptr[1:]))
    s["indptr"] = torch.tensor(indptr, dtype=torch.int32, device="cuda")
    i0 = s["indptr"].long()
    rows = i0[:-1, None] + torch.arange(widest, device="cuda")[None, :]
    s["rows"] = torch.where(rows < i0[1:, None], rows, torch.full_like(rows, T))
    s["seq_of"] = torch.repeat_interleave(torch.arange(n, device="cuda"), i0[1:] - i0[:-1])
    s["loss"] = torch.empty(case["pairs"], device="cuda")
    s["seq_logp"] = torch.empty(n, device="cuda")
    if own:
        from segmented_gather_gemm_lora_gb300 import binding as B

        s["space"] = B.preference_workspace(T, case["pairs"])
    return s


PREF_BETA, PREF_SMOOTH, PREF_MARGIN = 0.1, 0.1, 0.05
CLIP_LOW, CLIP_HIGH, KL_COEF = 0.2, 0.28, 0.04


# ----------------------------------------------------------------- plain forms --

def _quantise(x, keep, floor=False):
    """(e4m3 codes, bf16 scale a block) of blocks [n, 64]; floor: a positive value never becomes zero."""
    x = torch.where(keep, x, torch.zeros_like(x))
    top = x.abs().amax(1)
    scale = torch.where(top < TINY, torch.zeros_like(top), top / E4M3_MAX).to(torch.bfloat16)
    s = scale.float()[:, None]
    y = torch.where(s > 0, x / s, torch.zeros_like(x)).clamp(-E4M3_MAX, E4M3_MAX)
    if floor:
        y = torch.where((y > 0) & (y < 2.0 ** -9), torch.full_like(y, 2.0 ** -9), y)
    return y.to(torch.float8_e4m3fn), scale


def _bias(beta, step):
    return -torch.expm1(step * torch.log1p(beta - 1.0))


def _plain_adamw(s):
    case, plan = s["case"], s["plan"]
    at, keep, entry = plan["blocks"], plan["keep"], plan["entry"]
    ids = s["ids"].long()
    h = s["hyper"][ids]
    step = s["hyper"].view(torch.int32)[ids, 0].float()
    lr, b1, b2, eps, wd, most, gs = h[:, 1:].unbind(1)
    g = s["grad"].view(-1, BLOCK)[at]
    out = {}
    if case["clip"]:
        part = torch.where(keep, g * g, torch.zeros_like(g)).sum(1)
        total = torch.where(plan["has"], part[plan["rows"]], torch.zeros_like(part[:1])).sum(1)
        s["sumsq"][ids] = total
        out["sumsq"] = s["sumsq"]
        gs = gs * torch.clamp(most / (total.sqrt() * gs.abs() + 1e-6), max=1.0)
    of = lambda t: t[entry][:, None]  # noqa: E731
    g = g * of(gs)
    e4m3 = case["state"] == "e4m3"
    if e4m3:
        m, v = (s[k].view(torch.uint8).view(-1, BLOCK)[at].view(torch.float8_e4m3fn).float() for k in ("m", "v"))
        m, v = m * s["m_scale"][at].float()[:, None], v * s["v_scale"][at].float()[:, None]
        v = v * v
    else:
        m, v = s["m"].view(-1, BLOCK)[at], s["v"].view(-1, BLOCK)[at]
    m = of(b1) * m + of(1.0 - b1) * g
    v = of(b2) * v + of(1.0 - b2) * (g * g)
    size, root = lr / _bias(b1, step), torch.sqrt(_bias(b2, step))
    r = v.sqrt()
    weights = s["master"] if case["master"] else s["pool"]
    w = weights.view(-1, BLOCK)[at].float()
    w = w * of(1.0 - lr * wd) - of(size) * (m / (r / of(root) + of(eps)))

    def put(t, x):
        t = t.view(-1, BLOCK)
        t[at] = torch.where(keep, x.to(t.dtype), t[at])

    put(s["pool"], w)
    out["pool"] = s["pool"]
    if case["master"]:
        put(s["master"], w)
        out["master"] = s["master"]
    if e4m3:
        # codes move as their bytes: a store by mask of a type that few operations take
        mc, s["m_scale"][at] = _quantise(m, keep)
        vc, s["v_scale"][at] = _quantise(r, keep, floor=True)
        put(s["m"].view(torch.uint8), mc.view(torch.uint8))
        put(s["v"].view(torch.uint8), vc.view(torch.uint8))
        out.update(m_scale=s["m_scale"], v_scale=s["v_scale"])
    else:
        put(s["m"], m)
        put(s["v"], v)
    if case["zero"]:
        put(s["grad"], torch.zeros_like(g))
        out["grad"] = s["grad"]
    out.update(m=s["m"], v=s["v"])
    return out


def _plain_logprobs(logits, labels):
    """(log-probability of the label, log of the sum of exponentials) of each row, zero where it does not count."""
    x = logits.float()
    top = x.amax(1)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    lse = top + torch.log(torch.exp(x - top[:, None]).sum(1))
    at = labels.long().clamp(min=0)[:, None]
    zero = torch.zeros_like(lse)
    return (torch.where(labels >= 0, logits.gather(1, at)[:, 0].float() - lse, zero), torch.where(labels >= 0, lse, zero))


def _plain_grad(logits, labels, lse, coef):
    """coef * (one at the label - softmax), rounded once to the logits' type."""
    p = torch.exp(logits.float() - lse[:, None])
    d = -coef[:, None] * p
    at = labels.long().clamp(min=0)[:, None]
    d.scatter_add_(1, at, torch.where(labels >= 0, coef, torch.zeros_like(coef))[:, None])
    d = torch.where((labels >= 0)[:, None], d, torch.zeros_like(d))
    return d.to(logits.dtype)


def _plain_pref(s):
    case = s["case"]
    logits, lab = s["logits"], s["labels"]
    lp, lse = _plain_logprobs(logits, lab)
    none = torch.zeros(1, device="cuda")
    counts = lab >= 0
    gather = lambda t: torch.cat([t, none])[s["rows"]].sum(1)  # noqa: E731
    seq = gather(lp)
    ratio = gather(torch.where(counts, lp - s["ref"], torch.zeros_like(lp)))
    share = torch.ones_like(seq)
    if case["average"]:
        share = 1.0 / gather(counts.float()).clamp(min=1.0)
    ratio = ratio * share
    delta = ratio[0::2] - ratio[1::2]
    z = PREF_BETA * delta - PREF_MARGIN
    if case["kind"] == "sigmoid":
        up, down = torch.nn.functional.softplus(-z), torch.nn.functional.softplus(z)
        loss = (1 - PREF_SMOOTH) * up + PREF_SMOOTH * down
        slope = PREF_BETA * (PREF_SMOOTH * torch.sigmoid(z) - (1 - PREF_SMOOTH) * torch.sigmoid(-z))
    elif case["kind"] == "hinge":
        loss = torch.clamp(1 - z, min=0.0)
        slope = torch.where(z < 1, torch.full_like(z, -PREF_BETA), torch.zeros_like(z))
    else:
        off = delta - 1 / (2 * PREF_BETA)
        loss, slope = off * off, 2 * off
    slope = slope / case["pairs"]
    coef = torch.stack([slope, -slope], 1).view(-1) * share
    return {"loss": loss, "seq_logp": seq, "grad": _plain_grad(logits, lab, lse, coef[s["seq_of"]])}


def _plain_policy(s):
    logits, lab = s["logits"], s["labels"]
    lp, lse = _plain_logprobs(logits, lab)
    ratio = torch.exp(lp - s["old"])
    a, w = s["adv"], s["weight"]
    free, held = ratio * a, ratio.clamp(1 - CLIP_LOW, 1 + CLIP_HIGH) * a
    d = s["ref"] - lp
    kl = torch.expm1(d) - d
    loss = w * (KL_COEF * kl - torch.minimum(free, held))
    coef = -w * (KL_COEF * torch.expm1(d) + torch.where(free <= held, free, torch.zeros_like(free)))
    on = lab >= 0
    zero = torch.zeros_like(lp)
    return {"logp": lp, "loss": torch.where(on, loss, zero), "kl": torch.where(on, kl, zero),
            "grad": _plain_grad(logits, lab, lse, coef)}


# ------------------------------------------------------------------------- run --

def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        if op == "adamw":
            return _plain_adamw(s)
        if op == "logprobs":
            return list(_plain_logprobs(s["logits"], s["labels"]))
        return _plain_pref(s) if op == "pref" else _plain_policy(s)
    from segmented_gather_gemm_lora_gb300 import binding as B

    if op == "adamw":
        if case["clip"]:
            B.lora_grad_sumsq(s["set"], s["ids"], s["sumsq"], s["space"], err=s["err"])
        B.lora_adamw_step(s["set"], s["ids"], s["hyper"], sumsq=s["sumsq"] if case["clip"] else None,
                          zero_grad=case["zero"], err=s["err"])
        out = {k: s[k] for k in ("pool", "m", "v")}
        if case["clip"]:
            out["sumsq"] = s["sumsq"]
        if case["master"]:
            out["master"] = s["master"]
        if case["state"] == "e4m3":
            out.update(m_scale=s["m_scale"], v_scale=s["v_scale"])
        if case["zero"]:
            out["grad"] = s["grad"]
        return out
    if op == "logprobs":
        B.lora_token_logprobs(s["logits"], s["labels"], s["logp"], s["lse"], err=s["err"])
        return [s["logp"], s["lse"]]
    if op == "pref":
        B.lora_preference_loss(s["logits"], s["labels"], s["indptr"], s["loss"], s["seq_logp"], s["grad"], s["space"],
                               ref_logp=s["ref"], kind=getattr(B, "LORA_PREF_" + case["kind"].upper()), beta=PREF_BETA, label_smoothing=PREF_SMOOTH,
                               margin=PREF_MARGIN, average=case["average"], grad_scale=1.0 / case["pairs"], err=s["err"])
        return {"loss": s["loss"], "seq_logp": s["seq_logp"], "grad": s["grad"]}
    B.lora_policy_loss(s["logits"], s["labels"], s["old"], s["adv"], s["logp"], s["loss"], s["kl"], s["grad"],
                       ref_logp=s["ref"], weight=s["weight"], clip_low=CLIP_LOW, clip_high=CLIP_HIGH, kl_coef=KL_COEF,
                       err=s["err"])
    return {"logp": s["logp"], "loss": s["loss"], "kl": s["kl"], "grad": s["grad"]}


# --------------------------------------------------------------- 64-bit forms --

def _nearest_e4m3(y):
    """The e4m3 value nearest to y (ties to the even code), largest 448."""
    a = y.abs().clamp(min=2.0 ** -20)
    unit = torch.exp2(torch.floor(torch.log2(a)).clamp(min=-6.0) - 3.0)
    return (torch.round(y / unit) * unit).clamp(-448.0, 448.0)


def _codes64(x, positive):
    n = x.numel()
    x = torch.nn.functional.pad(x, (0, -n % 64)).view(-1, 64)
    top = x.abs().max(dim=1).values
    scale = torch.where(top < 2.0 ** -100, torch.zeros_like(top), top / 448.0).to(torch.bfloat16).double()
    y = _nearest_e4m3(x / torch.where(scale > 0, scale, torch.ones_like(scale))[:, None])
    if positive:
        y = torch.where((x > 0) & (y == 0), torch.full_like(y, 2.0 ** -9), y)
    return (y * (scale > 0)[:, None]).view(-1)[:n], scale


def _exact_adamw(case, seed):
    s = prepare(case, seed)
    P, e4m3 = case["page"], case["state"] == "e4m3"
    hyper = s["hyper"].double().cpu().numpy()
    steps = s["hyper"].view(torch.int32)[:, 0].cpu().numpy()
    out = {"pool": s["pool"].double(), "m": s["m"].float().double(), "v": s["v"].float().double()}
    if case["master"]:
        out["master"] = s["master"].double()
    if e4m3:
        out.update(m_scale=s["m_scale"].double(), v_scale=s["v_scale"].double())
    if case["zero"]:
        out["grad"] = s["grad"].double()
    if case["clip"]:
        out["sumsq"] = s["sumsq"].double()
    for i, r in zip(s["ids_host"].tolist(), s["ranks"]):
        places = []
        for p in s["projs"]:
            for slot, d in ((p["desc_host"][i, 2], p["d_in"]), (p["desc_host"][i, 3], p["d_out"])):
                e = torch.arange(r * d, device="cuda")
                places.append((p["page_list"].long()[int(slot) + e // P] + p["page0"]) * P + e % P)
        _, lr, b1, b2, eps, wd, most, gs = hyper[i]
        t = int(steps[i])
        if case["clip"]:
            total = sum(float(s["grad"][q].double().square().sum()) for q in places)
            out["sumsq"][i] = total
            gs *= min(1.0, most / (total ** 0.5 * abs(gs) + 1e-6))
        for q in places:
            g = s["grad"][q].double() * gs
            m, v = s["m"].view(torch.uint8 if e4m3 else torch.float32)[q], s["v"].view(torch.uint8 if e4m3 else torch.float32)[q]
            if e4m3:
                m = m.view(torch.float8_e4m3fn).float().double() * s["m_scale"].double()[q // 64]
                v = (v.view(torch.float8_e4m3fn).float().double() * s["v_scale"].double()[q // 64]) ** 2
            m = b1 * m.double() + (1 - b1) * g
            v = b2 * v.double() + (1 - b2) * g ** 2
            w = (s["master"] if case["master"] else s["pool"])[q].double()
            w = w - lr * wd * w - lr * (m / (1 - b1 ** t)) / ((v / (1 - b2 ** t)).sqrt() + eps)
            out["pool"][q] = w
            if case["master"]:
                out["master"][q] = w
            if e4m3:
                out["m"][q], out["m_scale"][q[::64] // 64] = _codes64(m, False)
                out["v"][q], out["v_scale"][q[::64] // 64] = _codes64(v.sqrt(), True)
            else:
                out["m"][q], out["v"][q] = m, v
            if case["zero"]:
                out["grad"][q] = 0.0
    return out


def exact(case, seed):
    if case["op"] == "adamw":
        return _exact_adamw(case, seed)
    s = prepare(case, seed)
    lab = s["labels"].long()
    T, op = case["T"], case["op"]
    lp, lse = torch.zeros(T, dtype=torch.float64, device="cuda"), torch.zeros(T, dtype=torch.float64, device="cuda")
    rows = torch.nonzero(lab >= 0)[:, 0]
    step = max(1, int(2e8) // case["V"])
    for part in rows.split(step):
        x = s["logits"][part].double()
        lse[part] = torch.logsumexp(x, 1)
        lp[part] = x.gather(1, lab[part, None])[:, 0] - lse[part]
    if op == "logprobs":
        return [lp, lse]
    slope = torch.zeros_like(lp)
    if op == "pref":
        indptr = _sequences(case)[0]
        seq = torch.stack([lp[a:b].sum() for a, b in zip(indptr, indptr[1:])])
        gap = torch.where(lab >= 0, lp - s["ref"].double(), torch.zeros_like(lp))
        div = [max(1, int((lab[a:b] >= 0).sum())) if case["average"] else 1 for a, b in zip(indptr, indptr[1:])]
        loss = torch.zeros(case["pairs"], dtype=torch.float64, device="cuda")
        for p in range(case["pairs"]):
            (a, b), (c, d) = indptr[2 * p: 2 * p + 2], indptr[2 * p + 1: 2 * p + 3]
            x = float(gap[a:b].sum()) / div[2 * p] - float(gap[c:d].sum()) / div[2 * p + 1]
            z = PREF_BETA * x - PREF_MARGIN
            win = 1 / (1 + np.exp(-z))
            if case["kind"] == "sigmoid":
                loss[p] = -(1 - PREF_SMOOTH) * np.log(win) - PREF_SMOOTH * np.log(1 - win)
                dx = PREF_BETA * (win - (1 - PREF_SMOOTH))
            elif case["kind"] == "hinge":
                loss[p], dx = max(0.0, 1 - z), -PREF_BETA if z < 1 else 0.0
            else:
                loss[p], dx = (x - 0.5 / PREF_BETA) ** 2, 2 * x - 1 / PREF_BETA
            slope[a:b], slope[c:d] = dx / div[2 * p] / case["pairs"], -dx / div[2 * p + 1] / case["pairs"]
        out = {"loss": loss, "seq_logp": seq}
    else:
        q = torch.exp(lp - s["old"].double())
        a, w, d = s["adv"].double(), s["weight"].double(), s["ref"].double() - lp
        first, second = q * a, torch.clip(q, 1 - CLIP_LOW, 1 + CLIP_HIGH) * a
        kl = torch.exp(d) - 1 - d
        on = (lab >= 0).double()
        slope = on * w * (KL_COEF * (1 - torch.exp(d)) - (first <= second) * first)
        out = {"logp": lp, "loss": on * w * (KL_COEF * kl - torch.minimum(first, second)), "kl": on * kl}
    grad = torch.zeros(T, case["V"], dtype=torch.float64, device="cuda")
    for part in rows.split(step):
        d = -slope[part, None] * torch.exp(s["logits"][part].double() - lse[part, None])
        d.scatter_add_(1, lab[part, None], slope[part, None])
        grad[part] = d
    return {**out, "grad": grad}
