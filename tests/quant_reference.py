"""Rotary positions and the 8-bit cache in 64 bits, from their definitions.
Test infrastructure: sequential code on host tensors, nothing of the library."""
import math

import torch

F64 = torch.float64
LIMIT = {torch.float8_e4m3fn: 448.0, torch.int8: 127.0}


def inverse_frequencies(r, base, scaling, factor, trained, low, high):
    """(radians per position of each pair, magnitude)"""
    if scaling == "ntk":
        base = base * factor ** (r / (r - 2)) if r > 2 else base
    out = []
    for i in range(r // 2):
        w = base ** (-2.0 * i / r)
        part = {"none": 0.0, "ntk": 0.0, "linear": 1.0}.get(scaling)
        if scaling == "yarn":
            at = lambda turns: r * math.log(trained / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
            a, b = max(0, math.floor(at(high))), min(r - 1, math.ceil(at(low)))
            part = (i - a) / max(b - a, 0.001)
        if scaling == "wavelength":
            part = 1 - (trained * w / (2 * math.pi) - low) / (high - low)
        part = min(1.0, max(0.0, part))
        out.append(w * (1 - part) + w / factor * part)
    return torch.tensor(out, dtype=F64), 0.1 * math.log(factor) + 1 if scaling == "yarn" else 1.0


def rope(x, positions, inv, magnitude, interleaved):
    """[n, heads, d] -> fp64"""
    out, r = x.to(F64).clone(), 2 * len(inv)
    angle = positions.to(F64)[:, None, None] * inv
    cos, sin = torch.cos(angle) * magnitude, torch.sin(angle) * magnitude
    i = torch.arange(r // 2)
    first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + r // 2)
    a, b = out[..., first], out[..., second]
    out[..., first], out[..., second] = a * cos - b * sin, b * cos + a * sin
    return out


def encode(x, dtype):
    """Code values of numbers that were divided by their scale."""
    if dtype == torch.int8:
        return torch.round(torch.nan_to_num(x, nan=0.0)).clamp(-127, 127)
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(2.0 ** -6, 448.0))) - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def scale_for(top, dtype):
    p = 2.0 ** -64
    while top > p * LIMIT[dtype]:
        p *= 2
    return p


def store(rows, slots, codes, scales, dtype):
    """rows fp64 [n, heads, d] into code values [blocks, bs, heads, d] fp64 and
    scales [blocks, bs / t, heads] fp64, in place."""
    bs, heads = codes.shape[1], codes.shape[2]
    t = bs // scales.shape[1]
    codes, scales = codes.view(-1, *codes.shape[2:]), scales.view(-1, heads)
    at, slots = 0, slots.tolist()
    while at < len(slots):
        end = at + 1
        if slots[at] < 0 or slots[at] >= codes.shape[0]:
            at = end
            continue
        while end < len(slots) and slots[end] == slots[end - 1] + 1 and slots[end] % t:
            end += 1
        group = slots[at] // t
        for h in range(heads):
            x = rows[at:end, h]
            finite = x[torch.isfinite(x)]
            need = scale_for(finite.abs().max().item() if finite.numel() else 0.0, dtype)
            old = scales[group, h].item()
            if slots[at] % t:
                new = max(old, need) if old == old else need
                if new != old:
                    span = codes[group * t:(group + 1) * t, h]
                    span.copy_(encode(span * (old / new if old > 0 else 0.0), dtype))
            else:
                new = need
            scales[group, h] = new
            codes[slots[at]:slots[at] + end - at, h] = encode(x / new, dtype)
        at = end


def values(codes, scales):
    """[blocks, bs, heads, d] fp64"""
    t = codes.shape[1] // scales.shape[1]
    return codes.to(F64) * scales.to(F64).repeat_interleave(t, 1)[..., None]


def tokens(values_, table, n):
    bs = values_.shape[1]
    return torch.stack([values_[table[p // bs], p % bs] for p in range(n)]) if n else values_.new_zeros((0,) + values_.shape[2:])


def decode(q, k, v, tables, lens, scale):
    """k, v: (codes, scales).  -> fp64 [b, heads, d]: the output, sum p |v|, and
    sum |code| times the largest p * scale (what a weight of 1 stands for)."""
    b, hq, d = q.shape
    bs, hkv = k[0].shape[1:3]
    out, size, unit = (torch.zeros((b, hq, d), dtype=F64) for _ in range(3))
    for i in range(b):
        n = int(lens[i])
        if not n:
            continue
        pages = tables[i, :-(-n // bs)].long()
        (kc, ks), (vc, vs) = ((c[pages].to(F64).reshape(-1, hkv, d)[:n].transpose(0, 1),
                               s[pages].to(F64).repeat_interleave(bs // s.shape[1], 1).reshape(-1, hkv)[:n].T[:, None])
                              for c, s in (k, v))
        x = q[i].to(F64).view(hkv, hq // hkv, d)
        p = torch.softmax(x @ kc.transpose(1, 2) * ks * scale, -1)
        out[i], size[i] = ((p * vs @ y).reshape(hq, d) for y in (vc, vc.abs()))
        unit[i] = ((p * vs).amax(-1, keepdim=True) * vc.abs().sum(1, keepdim=True)).reshape(hq, d)
    return out, size, unit
