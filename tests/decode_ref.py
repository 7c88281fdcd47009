"""Plain definitions, in 64 bits (the cache's and the 4-bit quantisers in the
fp32 steps that define them), of the decode step's operators: paged 8-bit
cache, attention over it, 4-bit group weights, token log probabilities."""

from __future__ import annotations

import numpy as np
import torch

F = np.float32
MIN_SCALE = 2.0 ** -60


def away(v: np.ndarray) -> np.ndarray:
    """Nearest whole number, halves away from zero."""
    v = v.astype(np.float64)
    return np.sign(v) * np.floor(np.abs(v) + 0.5)


def rows_of(lens, new):
    """Sequence by sequence: (first row, new rows, length)."""
    at = 0
    for n, t in zip(lens, new):
        yield at, t, n
        at += t


def append(codes, scales, x, table, lens, new):
    """In place: codes [pages, H, P, D] int8, scales [pages, H] fp32, x [T, H, D] fp32."""
    P = codes.shape[2]
    for b, (r0, t, n) in enumerate(rows_of(lens, new)):
        for p0 in range((n - t) // P * P if t else n, n, P):
            lo, hi = max(p0, n - t), min(n, p0 + P)
            page, older = table[b, p0 // P], lo - p0
            rows = x[r0 + lo - (n - t): r0 + hi - (n - t)]
            for h in range(codes.shape[1]):
                d = F(F(np.abs(rows[:, h]).max()) / F(127))
                was = scales[page, h] if older else F(0)
                d = max(d, was)
                if d < MIN_SCALE:
                    d = F(0)
                r = F(1) / d if d > 0 else F(0)
                if older and d > was:
                    codes[page, h] = away(codes[page, h].astype(F) * (was * r))
                codes[page, h, older:older + hi - lo] = np.clip(away(rows[:, h] * r), -127, 127)
                scales[page, h] = d


def attention(q, k_codes, k_scales, v_codes, v_scales, table, lens, new, scale=None, window=0):
    """(o, sum p |v|, largest sum |q k| * scale of a row's visible positions,
    sum |value code| times the value scale of the position where p vs is
    largest), all [T, Hq, D] or [T, Hq, 1] in 64 bits."""
    H, P, D = k_codes.shape[1:]
    T, Hq, _ = q.shape
    G = Hq // H
    scale = D ** -0.5 if scale is None else scale
    o, size, floor = (np.zeros((T, Hq, D)) for _ in range(3))
    mass = np.zeros((T, Hq, 1))
    k = k_codes.astype(np.float64) * k_scales.astype(np.float64)[..., None, None]
    v = v_codes.astype(np.float64) * v_scales.astype(np.float64)[..., None, None]
    for b, (r0, t, n) in enumerate(rows_of(lens, new)):
        pages = table[b, : -(-n // P)]
        kb = k[pages].transpose(1, 0, 2, 3).reshape(H, -1, D)[:, :n]
        vb = v[pages].transpose(1, 0, 2, 3).reshape(H, -1, D)[:, :n]
        cb = np.abs(v_codes[pages].astype(np.float64)).transpose(1, 0, 2, 3).reshape(H, -1, D)[:, :n]
        sb = np.repeat(np.maximum(v_scales[pages].astype(np.float64), MIN_SCALE), P, axis=0).T[:, :n]
        for i in range(t):
            pos = n - t + i
            lo = max(0, pos - window + 1) if window else 0
            if pos < lo:
                continue
            kk, vv = kb[:, lo:pos + 1], vb[:, lo:pos + 1]
            qq = q[r0 + i].astype(np.float64).reshape(H, G, D)
            s = np.einsum("hgd,hjd->hgj", qq, kk) * scale
            p = np.exp(s - s.max(-1, keepdims=True))
            p /= p.sum(-1, keepdims=True)
            o[r0 + i] = np.einsum("hgj,hjd->hgd", p, vv).reshape(Hq, D)
            size[r0 + i] = np.einsum("hgj,hjd->hgd", p, np.abs(vv)).reshape(Hq, D)
            m = np.einsum("hgd,hjd->hgj", np.abs(qq), np.abs(kk)) * abs(scale)
            mass[r0 + i] = m.max(-1).reshape(Hq, 1)
            at = (p * sb[:, None, lo:pos + 1]).argmax(-1) + lo
            floor[r0 + i] = (np.take_along_axis(sb, at, -1)[..., None]
                             * cb[:, None, lo:pos + 1].sum(2)).reshape(Hq, D)
    return o, size, mass, floor


def quantize_w4(w, group):
    """w [N, K] fp32 -> (codes [N, K] in -8..7, scales [N, K / group] fp32 of bf16 values)."""
    N, K = w.shape
    g = w.reshape(N, K // group, group)
    s = torch.from_numpy((np.abs(g).max(-1) / F(7)).astype(F)).to(torch.bfloat16).float().numpy()
    s = np.where(s < MIN_SCALE, F(0), s)
    r = np.divide(F(1), s, out=np.zeros_like(s), where=s > 0)
    return np.clip(away(g * r[..., None]), -8, 7).reshape(N, K).astype(np.int64), s


def pack_w4(codes):
    """The packed bytes [N, K / 2] of codes: weight 2i + h of a word at bits [16h + 4i, 16h + 4i + 4)."""
    N, K = codes.shape
    c = (codes + 8).astype(np.uint32).reshape(N, K // 8, 8)
    word = np.zeros((N, K // 8), dtype=np.uint32)
    for e in range(8):
        word |= c[..., e] << np.uint32(16 * (e % 2) + 4 * (e // 2))
    return word.view(np.uint8)


def logprobs(x, tokens, top):
    """(logprob, entropy, top ids, top log probabilities) of rows of fp64 values."""
    with np.errstate(divide="ignore", invalid="ignore"):
        m = x.max(-1, keepdims=True)
        e = np.exp(x - m)
        lp = x - m - np.log(e.sum(-1, keepdims=True))
        p = np.exp(lp)
        h = -np.where(p == 0, 0.0, p * lp).sum(-1)
    none = np.isneginf(m[:, 0])
    lp[none], h[none] = -np.inf, 0.0
    ids = np.argsort(-x, axis=-1, kind="stable")[:, :top]
    given = np.where(tokens < 0, 0.0, lp[np.arange(len(x)), np.maximum(tokens, 0)])
    return given, h, ids, np.take_along_axis(lp, ids, -1)
