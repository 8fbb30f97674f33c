"""Definitions of the attention operators in 64 bits, for the tests: rotation,
Q4_0 blocks, and softmax attention of packed sequences. Plain loops over
sequences and heads; no code of the package."""
import math

import torch


def held(x):
    """What Q4_0 blocks of bf16 values [..., D] stand for, fp64."""
    b = x.double().reshape(*x.shape[:-1], -1, 32)
    hi, lo = b.max(-1, keepdim=True).values, b.min(-1, keepdim=True).values
    d = (torch.where(hi >= -lo, hi, lo) * -0.125).clamp(-65504, 65504).half().double()
    q = torch.where(d != 0, torch.round(b / torch.where(d != 0, d, 1.0)), 0.0).clamp(-8, 7)
    v = torch.where(torch.isfinite(b).all(-1, keepdim=True), d * q, math.nan)
    return v.reshape(x.shape)


def rope_table(rows, dim, base=10000.0):
    inv = base ** (-torch.arange(0, dim, 2, dtype=torch.float64) / dim)
    a = torch.arange(rows, dtype=torch.float64)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float()


def rotate(x, table, pos):
    """fp64 rotation of [T, H, D] at positions pos by the fp32 table."""
    h = x.shape[-1] // 2
    t = table.double()[pos]
    c, s = t[:, None, :h], t[:, None, h:]
    x = x.double()
    return torch.cat([x[..., :h] * c - x[..., h:] * s, x[..., h:] * c + x[..., :h] * s], -1)


def attend(q, keys, values, new, scale):
    """q [T, Hq, D] packed (new[b] rows each); keys[b], values[b] [Lb, Hkv, D].
    Row i of the n of a sequence sees the keys up to L - n + i. Returns
    (out, bound): out fp64 [T, Hq, D] and, elementwise, how far a result of
    this precision may be from it:
      2^-8 |o|          rounding the output to bf16 (8 significant bits)
      2^-8 sum p |v|    rounding the probabilities to bf16, or twice to fp16
      ds   sum p |v|    scores in fp32: an error of ds in a score moves its
                        weight by a factor exp(ds); ds = 2^-20 scale sum |q k|
    """
    T, hq, D = q.shape
    out = torch.zeros(T, hq, D, dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(out)
    at = 0
    for n, k, v in zip(new, keys, values):
        L, hkv, _ = k.shape
        for i in range(n):
            seen = max(0, min(L, L - n + i + 1))
            if seen:
                kk = k[:seen].double().repeat_interleave(hq // hkv, 1)
                vv = v[:seen].double().repeat_interleave(hq // hkv, 1)
                qq = q[at + i].double()
                s = torch.einsum("hd,lhd->hl", qq, kk) * scale
                ds = torch.einsum("hd,lhd->hl", qq.abs(), kk.abs()).amax(1) * abs(scale) * 2.0 ** -20
                p = torch.softmax(s, 1)
                o = torch.einsum("hl,lhd->hd", p, vv)
                mass = torch.einsum("hl,lhd->hd", p, vv.abs())
                out[at + i] = o
                bound[at + i] = 2.0 ** -8 * o.abs() + (2.0 ** -8 + ds[:, None]) * mass + 1e-30
        at += n
    return out, bound
