"""The attention operators beside the MoE layer, case by case: what a pass reads, computes and returns.

Three operators of a decoder layer's attention half:
  append  the new tokens' queries and keys are rotated at their positions, and keys and values are written into a paged cache
          held in Q4_0 blocks (32 values: one fp16 scale d and 4-bit codes q, value d * (q - 8)); the written tokens are read
          back as bf16, as a program does that goes on with a prompt over what the cache holds;
  attend  the newest tokens of each sequence (one, or a few drafted ones) attend over that cache, grouped heads;
  prompt  causal attention of packed prompts (or chunks of them with their context), grouped heads, bf16.

`own` chooses between the plain forms (elementary torch operations in 32 bits) and the package's operators.
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
        # one decode step of one stream: latency
        dict(name="append one token", op="append", seqs=1, new_lo=1, new_hi=1, ctx_lo=600, ctx_hi=600, hq=32, hkv=4,
             dim=128, page=64, shape=1),
        # one decode step of a served batch
        dict(name="append decode batch", op="append", seqs=61, new_lo=1, new_hi=1, ctx_lo=0, ctx_hi=4000, hq=32, hkv=8,
             dim=128, page=16, shape=2),
        # the 2451-token prompt of the prefill workload
        dict(name="append prompt 2451", op="append", seqs=1, new_lo=2451, new_hi=2451, ctx_lo=0, ctx_hi=0, hq=32, hkv=4,
             dim=128, page=64, shape=3),
        # chunks of many prompts at once, as a scheduler packs them
        dict(name="append packed chunks", op="append", seqs=24, new_lo=1, new_hi=1400, ctx_lo=0, ctx_hi=8000, hq=64, hkv=8,
             dim=64, page=32, shape=4),
        # one stream, short and long context
        dict(name="attend one, short", op="attend", seqs=1, new_lo=1, new_hi=1, ctx_lo=512, ctx_hi=512, hq=32, hkv=4,
             dim=128, page=64, shape=5),
        dict(name="attend one, long", op="attend", seqs=1, new_lo=1, new_hi=1, ctx_lo=100002, ctx_hi=100002, hq=32, hkv=4,
             dim=128, page=64, shape=6),
        # four drafted tokens of eight streams checked in one pass, a head of its own for each query head
        dict(name="attend drafts", op="attend", seqs=8, new_lo=4, new_hi=4, ctx_lo=1, ctx_hi=9000, hq=16, hkv=16,
             dim=64, page=32, shape=7),
        # a served batch, ragged, and the largest one
        dict(name="attend ragged batch", op="attend", seqs=32, new_lo=1, new_hi=1, ctx_lo=0, ctx_hi=4095, hq=28, hkv=4,
             dim=128, page=16, shape=8),
        dict(name="attend large batch", op="attend", seqs=64, new_lo=1, new_hi=1, ctx_lo=4000, ctx_hi=12000, hq=64, hkv=8,
             dim=128, page=64, shape=9),
        # a short prompt, the 2451-token prompt, packed prompts, a long prompt's chunk over its context
        dict(name="prompt 77", op="prompt", seqs=1, new_lo=77, new_hi=77, ctx_lo=0, ctx_hi=0, hq=32, hkv=4, dim=128, shape=10),
        dict(name="prompt packed", op="prompt", seqs=20, new_lo=1, new_hi=1500, ctx_lo=0, ctx_hi=0, hq=32, hkv=8, dim=64,
             shape=11),
        dict(name="prompt 8192", op="prompt", seqs=1, new_lo=8192, new_hi=8192, ctx_lo=0, ctx_hi=0, hq=32, hkv=4, dim=128,
             shape=12),
    ]


HEADS = [(32, 4), (32, 8), (16, 16), (64, 8), (28, 4), (8, 1), (40, 8), (12, 2), (16, 1)]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "prompt"])
    hq, hkv = rng.choice(HEADS)
    dim = rng.choice([64, 128])
    while True:
        seqs = _log_int(rng, 1, 64)
        shape = rng.randrange(1 << 30)
        if op == "append":
            hi = _log_int(rng, 1, 16384)
            c = dict(op=op, seqs=seqs, new_lo=rng.choice([1, hi]), new_hi=hi, ctx_lo=0, ctx_hi=_log_int(rng, 1, 8000),
                     hq=hq, hkv=hkv, dim=dim, page=rng.choice([16, 32, 64, 128]), shape=shape)
            most = 17000 * 64 * 64
        elif op == "attend":
            new = rng.choice([1, 1, 1, 2, 4, 7])
            hi = _log_int(rng, 1, 130000)
            c = dict(op=op, seqs=seqs, new_lo=rng.choice([1, new]), new_hi=new, ctx_lo=rng.choice([0, hi // 2]), ctx_hi=hi,
                     hq=hq, hkv=hkv, dim=dim, page=rng.choice([16, 32, 64, 128]), shape=shape)
            most = 64 * 8000 * 8 * 128
        else:
            hi = _log_int(rng, 1, 8192)
            c = dict(op=op, seqs=seqs, new_lo=rng.choice([1, hi]), new_hi=hi, ctx_lo=0,
                     ctx_hi=rng.choice([0, 0, _log_int(rng, 1, 4000)]), hq=hq, hkv=hkv, dim=dim, shape=shape)
            most = 8192 * 8192 * 32
        if _size(c) <= most:
            return c


def _lens(case):
    """(new tokens, length with them) of every sequence: a part of the case, not of its inputs."""
    r = random.Random(case["shape"])
    new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["seqs"])]
    ctx = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["seqs"])]
    return new, [c + n for c, n in zip(ctx, new)]


def _size(case):
    """A measure of what the plain form holds, to bound drawn cases."""
    new, kv = _lens(case)
    if case["op"] == "append":
        return sum(new) * case["hq"] * case["dim"]
    if case["op"] == "attend":
        return case["seqs"] * max(kv) * max(case["hkv"] * case["dim"], case["hq"] * max(new))
    return case["seqs"] * max(new) * max(kv) * case["hq"]


def work(case):
    new, kv = _lens(case)
    T, hq, hkv, dim = sum(new), case["hq"], case["hkv"], case["dim"]
    held = hkv * dim * 18 // BLOCK  # bytes of one token's keys, or values, in the cache
    if case["op"] == "append":
        # q, k, v in; q, k rotated out; the cache written, and read back as bf16
        values = T * dim * (2 * hq + 3 * hkv + 2 * hkv)
        return {"bytes": 2 * values + 4 * T * held + 4 * dim * T, "flops": 6 * T * dim * (hq + hkv)}
    seen = sum(sum(range(k - n + 1, k + 1)) for n, k in zip(new, kv))  # visible (query, key) pairs of one head
    flops = 4 * hq * dim * seen
    if case["op"] == "attend":
        return {"bytes": 2 * sum(kv) * held + 4 * T * hq * dim, "flops": flops}
    return {"bytes": 4 * T * hq * dim + 4 * sum(kv) * hkv * dim, "flops": flops}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _rope(rows, dim, device):
    """cos | sin of every position, fp32 [rows, dim]."""
    inv = 10000.0 ** (-torch.arange(0, dim, 2, dtype=torch.float64, device=device) / dim)
    a = torch.arange(rows, dtype=torch.float64, device=device)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float()


def _inputs(case, seed):
    """The tensors a pass reads, from the case and the seed: activations with channels of different spread, a few of the
    key channels much wider, as projections of a trained model have them."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    new, kv = _lens(case)
    T, hq, hkv, dim, B = sum(new), case["hq"], case["hkv"], case["dim"], case["seqs"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    wide = torch.exp(0.4 * normal(hkv, dim)) * (1 + 4 * (torch.rand(hkv, dim, generator=g, device="cuda") < 0.02))
    rows = sum(kv) if case["op"] != "append" else T
    s = {"q": (normal(T, hq, dim)).bfloat16(), "k": (normal(rows, hkv, dim) * wide).bfloat16(),
         "v": (normal(rows, hkv, dim) * torch.exp(0.3 * normal(hkv, dim))).bfloat16()}

    def cumulative(n):
        return torch.tensor([0] + n, dtype=torch.int64).cumsum(0).to(torch.int32).cuda()

    s["cu"], s["cu_kv"] = cumulative(new), cumulative(kv)
    s["kv_lens"] = torch.tensor(kv, dtype=torch.int32).cuda()
    if case["op"] != "prompt":
        page = case["page"]
        per = [-(-k // page) for k in kv]
        ids = torch.randperm(sum(per), generator=g, device="cuda").to(torch.int32)
        table = torch.zeros(B, max(per), dtype=torch.int32, device="cuda")
        at = torch.tensor([0] + per).cumsum(0).tolist()
        for b in range(B):
            table[b, : per[b]] = ids[at[b]:at[b + 1]]
        s["table"], s["pages"] = table, sum(per)
    if case["op"] == "append":
        s["rope"] = _rope(max(kv), dim, "cuda")
    return s


def prepare(case, seed):
    s = {**case, **_inputs(case, seed)}
    T, hq, hkv, dim, B = s["q"].shape[0], case["hq"], case["hkv"], case["dim"], case["seqs"]
    new, kv = _lens(case)
    s["most_new"], s["most_kv"] = max(new), max(kv)
    if own:
        import paged_expert_cache_gb300 as pec
        s["out"] = torch.empty_like(s["q"])
        if case["op"] != "prompt":
            s["cache"] = pec.KVCache(pec.make_kv_config(1, s["pages"], hq, hkv, dim, page_tokens=case["page"]))
            s["batch"] = pec.KVBatch(s["cu"], s["kv_lens"], s["table"])
        if case["op"] == "append":
            s["k_out"], s["k_held"], s["v_held"] = (torch.empty_like(s["k"]) for _ in range(3))
        if case["op"] == "attend":  # the context, as earlier calls have left it in the cache
            whole = pec.KVBatch(s["cu_kv"], s["kv_lens"], s["table"])
            s["cache"].append(0, None, s["k"], s["v"], whole)
            torch.cuda.synchronize()
            del s["k"], s["v"]
        return s
    if case["op"] != "prompt":
        slots = s["pages"] * case["page"]
        for n in "kv":
            s[n + "_codes"] = torch.zeros(slots, hkv, dim // 2, dtype=torch.uint8, device="cuda")
            s[n + "_scale"] = torch.zeros(slots, hkv, dim // BLOCK, dtype=torch.float16, device="cuda")
        if case["op"] == "attend":
            slot = _slots(s["table"], case["page"], *_places(s["cu_kv"], s["kv_lens"], sum(kv)))
            for n in "kv":
                s[n + "_codes"][slot], s[n + "_scale"][slot] = _quantise(s.pop(n))
    return s


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------
def _places(cu, kv_lens, T):
    """(sequence, position) of each of T packed tokens; a sequence's last one is at its length - 1."""
    i = torch.arange(T, device=cu.device)
    seq = torch.searchsorted(cu[1:], i, right=True)
    return seq, (kv_lens[seq] - cu[seq + 1] + i).long()


def _slots(table, page, seq, pos):
    return table[seq, pos // page].long() * page + pos % page


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


def _rotate(x, c, s):
    a, b = x.float().chunk(2, -1)
    return torch.cat([a * c - b * s, b * c + a * s], -1).bfloat16()


def _softmax(s, seen):
    s = torch.where(seen, s, -math.inf)
    m = s.amax(-1, keepdim=True)
    e = torch.where(seen, torch.exp(s - m), 0.0)
    return e / e.sum(-1, keepdim=True)


def _append_plain(s):
    seq, pos = _places(s["cu"], s["kv_lens"], s["q"].shape[0])
    c, n = s["rope"][pos][:, None].chunk(2, -1)
    q, k = _rotate(s["q"], c, n), _rotate(s["k"], c, n)
    slot = _slots(s["table"], s["page"], seq, pos)
    held = []
    for name, x in (("k", k), ("v", s["v"])):
        s[name + "_codes"][slot], s[name + "_scale"][slot] = _quantise(x)
        held.append(_values(s[name + "_codes"][slot], s[name + "_scale"][slot]).bfloat16())
    return {"q": q, "k": k, "k_held": held[0], "v_held": held[1]}


def _padded(cu, most, T):
    """Indexes [B, most] of packed rows by sequence, and which of them are a sequence's own."""
    i = torch.arange(most, device=cu.device)
    at = cu[:-1, None] + i
    return at.clamp(max=T - 1).long(), at < cu[1:, None]


def _attention(q, k, v, n, kv, scale):
    """fp32 [B, Lq, Hq, D] over [B, Lk, Hkv, D]: row i of the n sees the keys up to kv - n + i."""
    B, Lq, hq, dim = q.shape
    hkv = k.shape[2]
    i, j = torch.arange(Lq, device=q.device), torch.arange(k.shape[1], device=q.device)
    seen = j <= (kv - n)[:, None, None] + i[:, None]
    q = q.unflatten(2, (hkv, hq // hkv)).permute(0, 2, 3, 1, 4).reshape(B, hkv, -1, dim)
    s = torch.matmul(q, k.permute(0, 2, 3, 1)) * scale
    p = _softmax(s.view(B, hq, Lq, -1), seen[:, None])
    o = torch.matmul(p.view(B, hkv, -1, p.shape[-1]), v.transpose(1, 2))
    return o.view(B, hq, Lq, dim).transpose(1, 2)


def _attend_plain(s):
    T, most = s["q"].shape[0], s["most_kv"]
    pos = torch.arange(most, device="cuda")
    slot = s["table"][:, pos // s["page"]].long() * s["page"] + pos % s["page"]
    k, v = (_values(s[n + "_codes"][slot], s[n + "_scale"][slot]) for n in "kv")
    at, is_row = _padded(s["cu"], s["most_new"], T)
    n = s["cu"][1:] - s["cu"][:-1]
    o = _attention(s["q"][at].float(), k, v, n, s["kv_lens"], s["dim"] ** -0.5)
    return _packed(o, s["cu"], T)


def _packed(o, cu, T):
    i = torch.arange(T, device=cu.device)
    seq = torch.searchsorted(cu[1:], i, right=True)
    return o[seq, i - cu[seq]].bfloat16()


def _prompt_plain(s):
    T = s["q"].shape[0]
    at, _ = _padded(s["cu"], s["most_new"], T)
    ak, _ = _padded(s["cu_kv"], s["most_kv"], s["k"].shape[0])
    n = s["cu"][1:] - s["cu"][:-1]
    o = _attention(s["q"][at].float(), s["k"][ak].float(), s["v"][ak].float(), n, s["kv_lens"], s["dim"] ** -0.5)
    return _packed(o, s["cu"], T)


def run(s):
    if not own:
        return {"append": _append_plain, "attend": _attend_plain, "prompt": _prompt_plain}[s["op"]](s)
    if s["op"] == "append":
        cache, batch = s["cache"], s["batch"]
        cache.append(0, s["q"], s["k"], s["v"], batch, rope=s["rope"], q_out=s["out"], k_out=s["k_out"])
        cache.read(0, batch, s["k_held"], s["v_held"])
        return {"q": s["out"], "k": s["k_out"], "k_held": s["k_held"], "v_held": s["v_held"]}
    if s["op"] == "attend":
        return s["cache"].attend(0, s["q"], s["batch"], s["out"])
    import paged_expert_cache_gb300 as pec
    return pec.attention_prompt(s["q"], s["k"], s["v"], s["out"], s["cu"], s["cu_kv"])


# ---------------------------------------------------------------------------
# The definition in 64 bits
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


def exact(case, seed):
    s = _inputs(case, seed)
    new, kv = _lens(case)
    hq, hkv, dim = case["hq"], case["hkv"], case["dim"]
    if case["op"] == "append":
        pos = torch.cat([torch.arange(k - n, k, device="cuda") for n, k in zip(new, kv)])
        half = dim // 2
        t = s["rope"].double()[pos]
        z = torch.complex(t[:, :half], t[:, half:])[:, None]

        def turned(x):
            x = x.double()
            y = torch.complex(x[..., :half], x[..., half:]) * z
            return torch.cat([y.real, y.imag], -1)

        k = turned(s["k"])
        return {"q": turned(s["q"]), "k": k, "k_held": _held64(k.bfloat16()), "v_held": _held64(s["v"])}
    k, v = (s["k"].double(), s["v"].double()) if case["op"] == "prompt" else (_held64(s["k"]), _held64(s["v"]))
    out, at, ak = torch.empty(*s["q"].shape, dtype=torch.float64, device="cuda"), 0, 0
    group = hq // hkv
    for n, m in zip(new, kv):
        hidden = torch.arange(m, device="cuda")[None, :] > torch.arange(m - n, m, device="cuda")[:, None]
        for h in range(hkv):
            for j in range(h * group, (h + 1) * group):
                z = s["q"][at:at + n, j].double() @ k[ak:ak + m, h].T / math.sqrt(dim)
                w = torch.softmax(z.masked_fill_(hidden, -math.inf), 1)
                out[at:at + n, j] = w @ v[ak:ak + m, h]
        at, ak = at + n, ak + m
    return out
