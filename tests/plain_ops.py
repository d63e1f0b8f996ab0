"""Plain 64-bit forms of the routing and 4-bit operators, for their tests.

Written from the definitions in include/kmoe.h; nothing here calls the library.
"""
from __future__ import annotations

import torch

NIBBLE = [4 * (c // 2) + 16 * (c % 2) for c in range(8)]     # bit of column c in its 8-column word


def w4_words(q: torch.Tensor) -> torch.Tensor:
    """Codes 0..15 [rows, cols] as stored 32-bit words [rows, cols / 8], column by column."""
    rows, cols = q.shape
    words = torch.zeros((rows, cols // 8), dtype=torch.int64)
    for c in range(cols):
        v = c % 128 // 8
        words[:, c // 128 * 16 + 4 * (v % 4) + v // 4] |= q[:, c].long() << NIBBLE[c % 8]
    return words


def w4_bytes(q: torch.Tensor) -> torch.Tensor:
    words = w4_words(q)
    return torch.stack([(words >> (8 * b)) & 255 for b in range(4)], -1).flatten(1).to(torch.uint8)


def w4_codes(codes: torch.Tensor) -> torch.Tensor:
    """Codes 0..15 of stored bytes [..., rows, cols / 2] (int64)."""
    b = codes.long().unflatten(-1, (-1, 4))
    word = b[..., 0] | b[..., 1] << 8 | b[..., 2] << 16 | b[..., 3] << 24
    col = torch.arange(word.shape[-1] * 8, device=codes.device)
    v = col % 128 // 8
    shift = torch.tensor(NIBBLE, device=codes.device)[col % 8]
    return word[..., col // 128 * 16 + 4 * (v % 4) + v // 4] >> shift & 15


def w4_values(codes, scales, zeros=None) -> torch.Tensor:
    """FP64 values (q - z) * s of stored weights."""
    group = codes.shape[-1] * 2 // scales.shape[-1]
    z = 8.0 if zeros is None else zeros.double().repeat_interleave(group, -1)
    return (w4_codes(codes).double() - z) * scales.double().repeat_interleave(group, -1)


def quant_w4(w: torch.Tensor, group: int, zeros: bool):
    """Codes, scales and zero points of w [rows, cols] (on the CPU: IEEE FP32 throughout)."""
    b = w.float().cpu().unflatten(-1, (-1, group))
    lo, hi = b.amin(-1).clamp(max=0), b.amax(-1).clamp(min=0)
    span, steps = (hi - lo, 15.0) if zeros else (torch.maximum(-lo, hi), 7.0)
    s = (span / torch.tensor(steps)).to(torch.bfloat16)
    s[s == 0] = 1
    z = torch.round(-lo / s.float()).clamp(0, 15) if zeros else torch.full_like(lo, 8)
    q = (torch.round(b / s.float()[..., None]) + z[..., None]).clamp(0, 15)
    return q.flatten(-2).to(torch.uint8), s, (z.to(torch.uint8) if zeros else None)


def route(logits, K, bias=None, score="sigmoid", n_groups=1, topk_groups=1, group_score="top2", renormalise=True,
          scale=1.0):
    """Experts [N, K] and FP64 weights [N, K], token by token on the CPU."""
    L = logits.double().cpu()
    N, E = L.shape
    b = torch.zeros(E, dtype=torch.float64) if bias is None else bias.double().cpu()
    size = E // n_groups
    idx, w = torch.zeros((N, K), dtype=torch.int32), torch.zeros((N, K), dtype=torch.float64)
    for t in range(N):
        l = L[t].clone()
        l[torch.isnan(l)] = -float("inf")
        masked = l.isneginf() | b.isnan() | b.isneginf()
        if score == "sigmoid":
            s = 1 / (1 + torch.exp(-l))
        else:
            top = l.max()
            e = torch.zeros(E, dtype=torch.float64) if top == -float("inf") else torch.where(
                l == top, torch.ones_like(l), torch.exp(l - top).nan_to_num(0.0))
            s = e / e.sum() if e.sum() > 0 else e
        s[masked] = 0
        c = [None if masked[e] else float(s[e] + b[e]) for e in range(E)]

        def group_key(g):
            best = sorted((c[e] for e in range(g * size, (g + 1) * size) if c[e] is not None), reverse=True)
            if not best:
                return (1, 0.0, g)
            return (0, -(best[0] if group_score == "max" else sum(best[:2])), g)

        kept = set(sorted(range(n_groups), key=group_key)[:topk_groups])
        order = sorted((e for e in range(E) if e // size in kept),
                       key=lambda e: (1, 0.0, e) if c[e] is None else (0, -c[e], e))[:K]
        idx[t] = torch.tensor(order, dtype=torch.int32)
        v = s[order]
        if renormalise:
            v = v / v.sum() if v.sum() > 0 else v * 0
        w[t] = v * scale
    return idx, w
