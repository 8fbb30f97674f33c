"""Operators of a decode step whose sequences continue shared prompts, case by case: what a pass reads, computes and returns.

  shared  attention over the paged Q4_0 cache for groups of sequences that have their first positions in common (several
          continuations of one prompt, requests behind one long instruction): the common part is read once for its group;
  norm    what stands between a layer's two halves: the block's output, normed where the model norms it, times its gate and
          scale, goes into the residual stream, and the sum, normed, is the next block's input;
  sample  the next token of each row of logits: temperature, top-k, top-p and min-p, drawn with given uniform numbers from the
          kept tokens in the order of their likelihood.

`own` chooses between the plain forms (elementary torch operations) and the package's operators.
"""
import math
import random

import torch

own = False

BLOCK = 32  # values of one Q4_0 block


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # four continuations of one short prompt: latency
        dict(name="shared four", op="shared", groups=1, seqs_lo=4, seqs_hi=4, pre_lo=600, pre_hi=600, own_lo=1, own_hi=100,
             new=1, hq=32, hkv=4, dim=128, page=64, shape=1),
        # sixteen continuations of the 2451-token prompt
        dict(name="shared 2451", op="shared", groups=1, seqs_lo=16, seqs_hi=16, pre_lo=2451, pre_hi=2451, own_lo=1, own_hi=512,
             new=1, hq=32, hkv=4, dim=128, page=64, shape=2),
        # a served batch: several prompts, each continued by some sequences or by one
        dict(name="shared groups", op="shared", groups=7, seqs_lo=1, seqs_hi=15, pre_lo=0, pre_hi=6000, own_lo=0, own_hi=900,
             new=1, hq=28, hkv=4, dim=128, page=16, shape=3),
        # four drafted tokens of eight continuations checked in one pass, a head of its own for each query head
        dict(name="shared drafts", op="shared", groups=1, seqs_lo=8, seqs_hi=8, pre_lo=9001, pre_hi=9001, own_lo=4, own_hi=300,
             new=4, hq=16, hkv=16, dim=64, page=32, shape=4),
        # many requests behind one long document, the largest
        dict(name="shared large", op="shared", groups=1, seqs_lo=64, seqs_hi=64, pre_lo=32768, pre_hi=32768, own_lo=100,
             own_hi=2000, new=1, hq=64, hkv=8, dim=128, page=64, shape=5),
        # one token between attention and FFN: latency
        dict(name="norm one token", op="norm", rows=1, hidden=2048, x="fp32", y="fp32", w="bf16", post=False, gate="none"),
        # a served batch, norms on both sides of the block and a gate for each token
        dict(name="norm sandwich batch", op="norm", rows=61, hidden=4096, x="bf16", y="bf16", w="bf16", post=True, gate="token"),
        # the 2451-token prompt
        dict(name="norm prompt 2451", op="norm", rows=2451, hidden=2048, x="fp32", y="bf16", w="bf16", post=False, gate="none"),
        # packed prompts of an odd width, a learned scale for each channel, the largest
        dict(name="norm packed odd", op="norm", rows=15013, hidden=4001, x="bf16", y="fp32", w="fp32", post=True, gate="channel"),
        # one stream: latency
        dict(name="sample one", op="sample", rows=1, vocab=131072, type="bf16", top_k=50, top_p=0.95, min_p=0.0, temp=0.8,
             greedy=0.0, flat=False),
        # a served batch with settings of its own for each row
        dict(name="sample mixed batch", op="sample", rows=61, vocab=50021, type="fp32", top_k=-1, top_p=-1.0, min_p=-1.0,
             temp=-1.0, greedy=0.1, flat=False),
        # wide nuclei over a large vocabulary, the largest
        dict(name="sample wide", op="sample", rows=128, vocab=131072, type="bf16", top_k=0, top_p=0.98, min_p=0.0, temp=1.0,
             greedy=0.0, flat=True),
    ]


HEADS = [(32, 4), (32, 8), (16, 16), (64, 8), (28, 4), (8, 1), (40, 8), (12, 2), (16, 1)]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["shared", "norm", "sample"])
    if op == "norm":
        while True:
            rows, hidden = _log_int(rng, 1, 16384), _log_int(rng, 64, 8192)
            hidden = rng.choice([hidden, hidden // 8 * 8, hidden // 64 * 64])
            if rows * hidden <= 15013 * 4001:
                return dict(op=op, rows=rows, hidden=hidden, x=rng.choice(["bf16", "fp32"]), y=rng.choice(["bf16", "fp32"]),
                            w=rng.choice(["bf16", "fp32"]), post=rng.random() < 0.5,
                            gate=rng.choice(["none", "token", "channel", "full"]))
    if op == "sample":
        while True:
            rows, vocab = _log_int(rng, 1, 512), _log_int(rng, 1000, 262144)
            if rows * vocab <= 128 * 131072:
                return dict(op=op, rows=rows, vocab=vocab, type=rng.choice(["bf16", "fp32"]),
                            top_k=rng.choice([0, -1, _log_int(rng, 1, 2000)]),
                            top_p=rng.choice([1.0, -1.0, round(rng.uniform(0.3, 0.999), 3)]),
                            min_p=rng.choice([0.0, -1.0, round(rng.uniform(0.001, 0.2), 3)]),
                            temp=rng.choice([-1.0, round(rng.uniform(0.3, 1.5), 2)]), greedy=rng.choice([0.0, 0.2]),
                            flat=rng.random() < 0.3)
    while True:
        hq, hkv = rng.choice(HEADS)
        seqs, pre, own_hi = _log_int(rng, 1, 64), _log_int(rng, 16, 32768), _log_int(rng, 1, 4000)
        c = dict(op=op, groups=rng.choice([1, 1, 1, 2, 5, 16]), seqs_lo=rng.choice([1, seqs]), seqs_hi=seqs,
                 pre_lo=rng.choice([0, pre, pre]), pre_hi=pre, own_lo=rng.choice([0, own_hi // 2]), own_hi=own_hi,
                 new=rng.choice([1, 1, 1, 2, 4, 7]), hq=hq, hkv=hkv, dim=rng.choice([64, 128]), page=rng.choice([16, 32, 64, 128]),
                 shape=rng.randrange(1 << 30))
        members, P, S = _lens(c)
        T = len(S) * c["new"]
        if T <= 512 and hq * c["dim"] * c["new"] * sum(n * p for n, p in zip(members, P)) <= 64 * 128 * 64 * 32768 \
                and hkv * c["dim"] * sum(S) <= 8 * 128 * 64 * 2000:
            return c


def _lens(case):
    """Of a `shared` case: the sequences of each group, the positions each group has in common, and each sequence's own
    ones, its new tokens (always its own) among them. A part of the case, not of its inputs."""
    r = random.Random(case["shape"])
    members = [r.randint(case["seqs_lo"], case["seqs_hi"]) for _ in range(case["groups"])]
    P = [r.randint(case["pre_lo"], case["pre_hi"]) for _ in members]
    S = [r.randint(case["own_lo"], case["own_hi"]) + case["new"] for _ in range(sum(members))]
    return members, P, S


def work(case):
    if case["op"] == "norm":
        n, size = case["rows"] * case["hidden"], {"bf16": 2, "fp32": 4}
        gate = {"none": 0, "token": case["rows"], "channel": case["hidden"], "full": n}[case["gate"]]
        weights = case["hidden"] * (1 + case["post"]) + gate
        return {"bytes": n * (2 * size[case["x"]] + size[case["y"]] + 2) + weights * size[case["w"]],
                "flops": n * (10 if case["post"] else 7)}
    if case["op"] == "sample":
        n = case["rows"] * case["vocab"]
        return {"bytes": n * {"bf16": 2, "fp32": 4}[case["type"]] + 28 * case["rows"], "flops": 4 * n}
    members, P, S = _lens(case)
    hq, dim, new = case["hq"], case["dim"], case["new"]
    held = 2 * case["hkv"] * dim * 18 // BLOCK  # bytes of one token's keys and values in the cache
    seen = sum(n * new * p for n, p in zip(members, P)) + sum(sum(range(s - new + 1, s + 1)) for s in S)
    return {"bytes": held * (sum(P) + sum(S)) + 4 * len(S) * new * hq * dim, "flops": 4 * hq * dim * seen}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _shared_inputs(case, seed):
    """Queries, the common parts' keys and values (packed by group) and the sequences' own (packed by sequence): channels of
    different spread, a few of the key channels much wider, as projections of a trained model have them."""
    g = _generator(seed)
    members, P, S = _lens(case)
    hq, hkv, dim = case["hq"], case["hkv"], case["dim"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    wide = torch.exp(0.4 * normal(hkv, dim)) * (1 + 4 * (torch.rand(hkv, dim, generator=g, device="cuda") < 0.02))
    spread = torch.exp(0.3 * normal(hkv, dim))
    s = {"q": normal(len(S) * case["new"], hq, dim).bfloat16()}
    for part, rows in (("pre", sum(P)), ("own", sum(S))):
        s["k_" + part] = (normal(rows, hkv, dim) * wide).bfloat16()
        s["v_" + part] = (normal(rows, hkv, dim) * spread).bfloat16()
    s["order"] = torch.randperm(_pages(case)[-1], generator=g, device="cuda").to(torch.int32).cpu()
    return s


def _pages(case):
    """Whole pages of each group's common part, each sequence's own pages, and all of them. A page that the common part
    fills only in part is each sequence's own, with a copy of that part."""
    members, P, S = _lens(case)
    page = case["page"]
    common = [p // page for p in P]
    mine = [-(-(P[g] + S[b]) // page) - common[g] for b, g in enumerate(_group_of(members))]
    return common, mine, sum(common) + sum(mine)


def _group_of(members):
    return [g for g, n in enumerate(members) for _ in range(n)]


def _table(case, order):
    common, mine, _ = _pages(case)
    group = _group_of(_lens(case)[0])
    at, starts = 0, []
    for n in common:
        starts.append(at)
        at += n
    table = torch.zeros(len(group), max(1, max(common[g] + m for g, m in zip(group, mine))), dtype=torch.int32)
    for b, g in enumerate(group):
        table[b, : common[g]] = order[starts[g]: starts[g] + common[g]]
        table[b, common[g]: common[g] + mine[b]] = order[at: at + mine[b]]
        at += mine[b]
    return table


def _cumulative(n):
    return torch.tensor([0] + list(n), dtype=torch.int64).cumsum(0).to(torch.int32)


def _written(case, s):
    """What lies in the cache: for the groups' whole common pages, and for each sequence from there on, the packed keys and
    values, their tables and lengths."""
    members, P, S = _lens(case)
    page, group = case["page"], _group_of(members)
    cp, co = _cumulative(P).tolist(), _cumulative(S).tolist()
    common = [p // page for p in P]
    first = _cumulative(members).tolist()[:-1]  # each group's first sequence
    pre = [torch.arange(cp[g], cp[g] + common[g] * page) for g in range(len(P))]
    keys = {}
    for n in "kv":
        whole = s[n + "_pre"][torch.cat(pre).cuda()]
        rest = torch.cat([x for b, g in enumerate(group)
                          for x in (s[n + "_pre"][cp[g] + common[g] * page: cp[g + 1]], s[n + "_own"][co[b]: co[b + 1]])])
        keys[n] = (whole, rest)
    return keys, common, first, [P[g] - common[g] * page + S[b] for b, g in enumerate(group)]


def _prepare_shared(case, seed):
    s = {**case, **_shared_inputs(case, seed)}
    members, P, S = _lens(case)
    group, page = _group_of(members), case["page"]
    table = _table(case, s.pop("order"))
    lens = [P[g] + n for g, n in zip(group, S)]
    keys, common, first, rest = _written(case, s)
    for n in ("k_pre", "k_own", "v_pre", "v_own"):
        del s[n]
    s["members"], s["P"], s["S"] = members, P, S
    s["table"] = table.cuda()
    cu = torch.arange(len(S) + 1, dtype=torch.int32).cuda() * case["new"]
    kv_lens = torch.tensor(lens, dtype=torch.int32).cuda()
    if own:
        import paged_expert_cache_gb300 as pec
        s["cache"] = pec.KVCache(pec.make_kv_config(1, _pages(case)[-1], case["hq"], case["hkv"], case["dim"], page_tokens=page))
        whole_lens = torch.tensor([c * page for c in common], dtype=torch.int32)
        if sum(common):
            whole = pec.KVBatch(_cumulative(whole_lens.tolist()).cuda(), whole_lens.cuda(), s["table"][first].contiguous())
            s["cache"].append(0, None, keys["k"][0], keys["v"][0], whole)
        s["cache"].append(0, None, keys["k"][1], keys["v"][1], pec.KVBatch(_cumulative(rest).cuda(), kv_lens, s["table"]))
        torch.cuda.synchronize()
        s["batch"] = pec.KVBatch(cu, kv_lens, s["table"])
        s["common"] = pec.KVGroups(_cumulative(members).cuda(), torch.tensor(P, dtype=torch.int32).cuda())
        s["workspace"] = s["cache"].shared_workspace(s["q"].shape[0])
        s["out"] = torch.empty_like(s["q"])
        return s
    slots = _pages(case)[-1] * page
    at = torch.cat([torch.arange(common[g] * page) for g in range(len(P))])
    seq = torch.tensor([first[g] for g in range(len(P)) for _ in range(common[g] * page)], dtype=torch.int64)
    at2 = torch.cat([torch.arange(n - r, n) for n, r in zip(lens, rest)])
    seq2 = torch.tensor([b for b, r in enumerate(rest) for _ in range(r)], dtype=torch.int64)
    for n in "kv":
        s[n + "_codes"] = torch.zeros(slots, case["hkv"], case["dim"] // 2, dtype=torch.uint8, device="cuda")
        s[n + "_scale"] = torch.zeros(slots, case["hkv"], case["dim"] // BLOCK, dtype=torch.float16, device="cuda")
        for x, b, p in zip(keys[n], (seq, seq2), (at, at2)):
            if len(p):
                slot = (table[b, p // page].long() * page + p % page).cuda()
                s[n + "_codes"][slot], s[n + "_scale"][slot] = _quantise(x)
    return s


def _norm_inputs(case, seed):
    """A residual stream with a few channels far above the others, a block's output, weights around one."""
    g = _generator(seed)
    T, H = case["rows"], case["hidden"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    loud = 1 + 30 * (torch.rand(H, generator=g, device="cuda") < 0.003)
    w = TYPES[case["w"]]
    s = {"x": (2 * normal(T, H) * loud).to(TYPES[case["x"]]), "y": normal(T, H).to(TYPES[case["y"]]),
         "weight": (1 + 0.2 * normal(H)).to(w), "post": (0.5 + 0.1 * normal(H)).to(w) if case["post"] else None,
         "scale": 0.75, "eps": 1e-6}
    shape = {"none": None, "token": (T, 1), "channel": (H,), "full": (T, H)}[case["gate"]]
    s["gate"] = None if shape is None else torch.sigmoid(normal(*shape)).to(w)
    return s


def _prepare_norm(case, seed):
    s = {**case, **_norm_inputs(case, seed)}
    if own:
        s["x_out"] = torch.empty_like(s["x"])
        s["out"] = torch.empty(s["x"].shape, dtype=torch.bfloat16, device="cuda")
    return s


def _sample_inputs(case, seed):
    """Logits of a language model's shape: a broad bulk and, unless they are flat, some tokens well above it; a few tokens are
    forbidden (-inf). Settings: -1 stands for one of its own in each row."""
    g = _generator(seed)
    T, V = case["rows"], case["vocab"]

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    z = torch.randn(T, V, generator=g, device="cuda") * (1.0 if case["flat"] else 2.0) - 3.0
    if not case["flat"]:
        z += (uniform(T, V) < 64 / V) * (-3.0 * torch.log(uniform(T, V) + 1e-6))
    z[uniform(T, V) < 0.01] = -math.inf

    def setting(name, own_values):
        return own_values if case[name] < 0 else torch.full((T,), float(case[name]), device="cuda")

    def choice(*values):
        return torch.tensor(values, device="cuda")[(uniform(T) * len(values)).long().clamp(max=len(values) - 1)]

    temp = setting("temp", 0.4 + uniform(T))
    return {"logits": z.to(TYPES[case["type"]]), "uniform": uniform(T),
            "temperature": torch.where(uniform(T) < case["greedy"], 0.0, temp),
            "top_k": setting("top_k", choice(0.0, 1.0, 20.0, 200.0, 5000.0)).to(torch.int32),
            "top_p": setting("top_p", choice(1.0, 0.5, 0.9, 0.99)), "min_p": setting("min_p", choice(0.0, 0.0, 0.02, 0.1))}


def _prepare_sample(case, seed):
    s = {**case, **_sample_inputs(case, seed)}
    if own:
        s["tokens"] = torch.empty(case["rows"], dtype=torch.int32, device="cuda")
        s["logprobs"] = torch.empty(case["rows"], device="cuda")
    return s


def prepare(case, seed):
    return {"shared": _prepare_shared, "norm": _prepare_norm, "sample": _prepare_sample}[case["op"]](case, seed)


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------
def _quantise(x):
    """bf16 [T, H, D] as Q4_0 blocks: (codes [T, H, D / 2], scales fp16 [T, H, D / 32]). A block's value of largest
    magnitude takes code 0; byte i of a block holds code i and, above it, code i + 16."""
    b = x.float().unflatten(-1, (-1, BLOCK))
    hi, lo = b.amax(-1), b.amin(-1)
    d = (torch.where(hi >= -lo, hi, lo) / -8).clamp(-65504, 65504).half()
    f = d.float()[..., None]
    q = torch.where(f == 0, 8.0, ((b / f).round() + 8).clamp(0, 15)).to(torch.uint8)
    return (q[..., :16] | (q[..., 16:] << 4)).flatten(-2), d


def _values(codes, d):
    """The fp32 values of Q4_0 blocks."""
    c = codes.unflatten(-1, (-1, BLOCK // 2))
    q = torch.cat([c & 15, c >> 4], -1).float() - 8
    return (q * d.float()[..., None]).flatten(-2)


def _held(s, table, positions):
    """Keys and values in fp32 at positions of the sequences of `table`."""
    slot = table[:, positions // s["page"]].long() * s["page"] + positions % s["page"]
    return (_values(s[n + "_codes"][slot], s[n + "_scale"][slot]) for n in "kv")


def _shared_plain(s):
    """One softmax over the common part, computed once for its group, and the sequence's own part."""
    hq, hkv, dim, new = s["hq"], s["hkv"], s["dim"], s["new"]
    out, b0 = torch.empty_like(s["q"]), 0
    for n, P in zip(s["members"], s["P"]):
        own_lens = s["S"][b0:b0 + n]
        most = max(own_lens)
        table = s["table"][b0:b0 + n]
        q = s["q"][b0 * new:(b0 + n) * new].float().view(n, new, hkv, hq // hkv, dim)
        kp, vp = (x[0] for x in _held(s, table[:1], torch.arange(P, device="cuda")))
        at = P + torch.arange(most, device="cuda")
        ko, vo = _held(s, table, at.clamp(max=table.shape[1] * s["page"] - 1))
        zp = torch.einsum("bthgd,phd->bthgp", q, kp)
        zo = torch.einsum("bthgd,bphd->bthgp", q, ko)
        last = torch.tensor(own_lens, device="cuda")[:, None] - new + torch.arange(new, device="cuda")
        seen = torch.arange(most, device="cuda") <= last[..., None]
        zo = torch.where(seen[:, :, None, None], zo, -math.inf)
        z = torch.cat([zp, zo], -1) * dim ** -0.5
        e = torch.exp(z - z.amax(-1, keepdim=True))
        w = e / e.sum(-1, keepdim=True)
        o = torch.einsum("bthgp,phd->bthgd", w[..., :P], vp) + torch.einsum("bthgp,bphd->bthgd", w[..., P:], vo)
        out[b0 * new:(b0 + n) * new] = o.reshape(n * new, hq, dim).bfloat16()
        b0 += n
    return out


def _rms(x, eps):
    return x * (x.square().mean(-1, keepdim=True) + eps).rsqrt()


def _norm_plain(s):
    y = s["y"].float()
    if s["post"] is not None:
        y = _rms(y, s["eps"]) * s["post"].float()
    if s["gate"] is not None:
        y = y * s["gate"].float()
    x = s["x"].float() + s["scale"] * y
    return {"x": x.to(s["x"].dtype), "out": (_rms(x, s["eps"]) * s["weight"].float()).bfloat16()}


def _sample_plain(s):
    """In 64 bits: whether a token is in the nucleus, and which one is met, is a comparison of long sums."""
    z, V = s["logits"].double(), s["vocab"]
    t = s["temperature"].double()[:, None]
    index = torch.arange(V, device="cuda")
    top = z.amax(-1, keepdim=True)
    first = torch.where(z == top, index, V).amin(-1, keepdim=True)
    greedy = t == 0
    w = torch.exp((z - top) / torch.where(greedy, 1.0, t))
    ranked, order = torch.sort(z, stable=True, dim=-1, descending=True)
    k = s["top_k"].long()[:, None]
    keep = (index < torch.where(k <= 0, V, k)) & (ranked > -math.inf)
    mass = torch.where(keep, w.gather(1, order), 0.0)
    before = torch.cat([torch.zeros_like(top), mass.cumsum(-1)[:, :-1]], -1)
    p, m = s["top_p"].double()[:, None], s["min_p"].double()[:, None]
    keep &= (p >= 1) | (before < p * mass.sum(-1, keepdim=True))
    keep &= (m <= 0) | (ranked >= top + t * torch.log(torch.where(m <= 0, 1.0, m)))
    keep |= index == 0
    mass = torch.where(keep, mass, 0.0)
    upto = mass.cumsum(-1)  # the kept tokens from the most to the least likely: the first one past the drawn point
    met = torch.where(keep & (upto > s["uniform"].double()[:, None] * upto[:, -1:]), index, V).amin(-1, keepdim=True)
    token = torch.where(greedy, first, order.gather(1, torch.minimum(met, keep.sum(-1, keepdim=True) - 1)))
    logprob = torch.where(greedy, 0.0, (z.gather(1, token) - top) / torch.where(greedy, 1.0, t) - mass.sum(-1, keepdim=True).log())
    return {"tokens": token[:, 0].to(torch.int32), "logprobs": logprob[:, 0].float()}


def run(s):
    if not own:
        return {"shared": _shared_plain, "norm": _norm_plain, "sample": _sample_plain}[s["op"]](s)
    import paged_expert_cache_gb300 as pec
    if s["op"] == "shared":
        return s["cache"].attend_shared(0, s["q"], s["batch"], s["common"], s["out"], s["workspace"])
    if s["op"] == "norm":
        pec.residual_norm(s["x"], s["y"], s["out"], weight=s["weight"], post_weight=s["post"], gate=s["gate"],
                          scale=s["scale"], eps=s["eps"], x_out=s["x_out"])
        return {"x": s["x_out"], "out": s["out"]}
    pec.sample(s["logits"], s["tokens"], s["uniform"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
               min_p=s["min_p"], logprobs=s["logprobs"])
    return {"tokens": s["tokens"], "logprobs": s["logprobs"]}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def _held64(x):
    """What Q4_0 blocks of bf16 values stand for, fp64."""
    x = x.double()
    b = x.reshape(*x.shape[:-1], x.shape[-1] // BLOCK, BLOCK)
    most, least = b.max(-1, keepdim=True).values, b.min(-1, keepdim=True).values
    extreme = torch.where(most + least >= 0, most, least)
    d = torch.clamp(extreme * -0.125, -65504, 65504).half().double()
    steps = torch.where(d != 0, b / torch.where(d != 0, d, 1.0), 0.0)
    return (d * torch.clamp(torch.round(steps), -8, 7)).reshape(x.shape)


def _exact_shared(case, seed):
    s = _shared_inputs(case, seed)
    members, P, S = _lens(case)
    cp, co, new = _cumulative(P).tolist(), _cumulative(S).tolist(), case["new"]
    heads_a_key = case["hq"] // case["hkv"]
    out = torch.empty(*s["q"].shape, dtype=torch.float64, device="cuda")
    held = {n: _held64(s[n]) for n in ("k_pre", "v_pre", "k_own", "v_own")}
    for b, g in enumerate(_group_of(members)):
        k, v = (torch.cat([held[n + "_pre"][cp[g]:cp[g + 1]], held[n + "_own"][co[b]:co[b + 1]]]).transpose(0, 1) for n in "kv")
        q = s["q"][b * new:(b + 1) * new].double().transpose(0, 1)
        z = torch.matmul(q, k.repeat_interleave(heads_a_key, 0).transpose(1, 2)) / math.sqrt(case["dim"])
        length = P[g] + S[b]
        for i in range(new):
            z[:, i, length - new + i + 1:] = -math.inf
        out[b * new:(b + 1) * new] = torch.matmul(torch.softmax(z, -1), v.repeat_interleave(heads_a_key, 0)).transpose(0, 1)
    return out


def _exact_norm(case, seed):
    s = _norm_inputs(case, seed)
    x, y = s["x"].double(), s["y"].double()
    if case["post"]:
        y = y / torch.sqrt((y * y).sum(1, keepdim=True) / case["hidden"] + s["eps"]) * s["post"].double()
    if s["gate"] is not None:
        y = s["gate"].double() * y
    x = x + s["scale"] * y
    return {"x": x, "out": x / torch.sqrt((x * x).sum(1, keepdim=True) / case["hidden"] + s["eps"]) * s["weight"].double()}


def _exact_sample(case, seed):
    s = _sample_inputs(case, seed)
    tokens, logprobs = [], []
    settings = zip(*(s[n].double().tolist() for n in ("temperature", "top_k", "top_p", "min_p", "uniform")))
    for z, (t, k, p, m, u) in zip(s["logits"].double(), settings):
        places = torch.argsort(z, descending=True, stable=True)
        if t == 0:
            tokens.append(int(places[0]))
            logprobs.append(0.0)
            continue
        places = places[: int((z > -math.inf).sum())]
        if k >= 1:
            places = places[: int(k)]
        weight = torch.exp((z[places] - z[places[0]]) / t)
        if p < 1:
            sums = torch.cumsum(weight, 0)
            places = places[: int((sums < p * sums[-1]).sum()) + 1]
        if m > 0:
            places = places[: max(1, int((z[places] >= z[places[0]] + t * math.log(m)).sum()))]
        weight = torch.exp((z[places] - z[places[0]]) / t)
        sums = torch.cumsum(weight, 0)
        i = min(int(torch.searchsorted(sums, u * sums[-1], right=True)), len(places) - 1)
        tokens.append(int(places[i]))
        logprobs.append(float(torch.log(weight[i] / sums[-1])))
    return {"tokens": torch.tensor(tokens, dtype=torch.int32, device="cuda"),
            "logprobs": torch.tensor(logprobs, dtype=torch.float64, device="cuda")}


def exact(case, seed):
    return {"shared": _exact_shared, "norm": _exact_norm, "sample": _exact_sample}[case["op"]](case, seed)
