"""What is measured of the operators around the ternary projections of a decode
step: the 8-bit paged key/value cache (writing it, attention over it), products
with 4-bit weights and group scales, and token log probabilities.

``run`` computes an operator in elementary torch operations where ``own`` is
false, and through the package's entry points where it is true; ``exact`` gives
the definition's values in 64 bits.  Both forms take the same state.

Sizes: a decoder layer of 20 query heads over 5 key/value heads of 128
(2560 -> 3840 fused projection, FFN 6912), context 4096, vocabulary 128,256,
and generic ones around them.
"""

import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one decode step of 64 running sequences writes its keys and values; most
        # pages hold older tokens, whose scale may have to grow
        {"name": "append_step", "op": "append", "batch": 64, "new_max": 1, "len_min": 1, "len_max": 4096,
         "heads": 5, "dim": 128, "page": 64, "dtype": "bf16", "mix": 1},
        # three prompts of odd lengths are written at once, one after a shared prefix
        {"name": "append_prompt", "op": "append", "batch": 3, "new_max": 2011, "len_min": 700,
         "len_max": 2700, "heads": 5, "dim": 128, "page": 64, "dtype": "bf16", "mix": 2},
        # one user, one token, a short conversation: latency
        {"name": "attend_one", "op": "attend", "batch": 1, "new_max": 1, "len_min": 701, "len_max": 701,
         "q_heads": 20, "heads": 5, "dim": 128, "page": 64, "window": 0, "dtype": "bf16", "mix": 3},
        # a serving batch at ragged lengths up to the model's context
        {"name": "attend_batch", "op": "attend", "batch": 48, "new_max": 1, "len_min": 40,
         "len_max": 4096, "q_heads": 20, "heads": 5, "dim": 128, "page": 64, "window": 0,
         "dtype": "bf16", "mix": 4},
        # two sequences far beyond the context, full precision activations, small pages
        {"name": "attend_long_f32", "op": "attend", "batch": 2, "new_max": 1, "len_min": 50021,
         "len_max": 60013, "q_heads": 20, "heads": 5, "dim": 128, "page": 32, "window": 0,
         "dtype": "f32", "mix": 5},
        # five drafted tokens of each of 16 sequences are checked at once, sliding window
        {"name": "attend_draft", "op": "attend", "batch": 16, "new_max": 5, "len_min": 900,
         "len_max": 4000, "q_heads": 16, "heads": 8, "dim": 64, "page": 16, "window": 1024,
         "dtype": "bf16", "mix": 6},
        # two prompts are read, the longer one the whole context
        {"name": "attend_prompt", "op": "attend", "batch": 2, "new_max": 4096, "len_min": 2500,
         "len_max": 4096, "q_heads": 20, "heads": 5, "dim": 128, "page": 64, "window": 0,
         "dtype": "bf16", "mix": 7},
        # one token through a square projection
        {"name": "w4_square", "op": "w4", "M": 1, "K": 2560, "N": 2560, "group": 128, "dtype": "bf16"},
        # one token through the output head
        {"name": "w4_head", "op": "w4", "M": 1, "K": 2560, "N": 128256, "group": 128, "dtype": "bf16"},
        # a batch of 23 tokens through the FFN's down projection, full precision activations
        {"name": "w4_batch_f32", "op": "w4", "M": 23, "K": 6912, "N": 2560, "group": 64, "dtype": "f32"},
        # the next token's alternatives for one sequence
        {"name": "logprobs_one", "op": "logprobs", "M": 1, "V": 128256, "top": 20, "dtype": "f32"},
        # a prompt of 701 tokens is scored
        {"name": "logprobs_prompt", "op": "logprobs", "M": 701, "V": 128256, "top": 5, "dtype": "bf16"},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "append", "attend", "attend", "attend", "attend", "w4", "w4", "logprobs",
                     "logprobs"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    mix = rng.randrange(1 << 20)
    heads = rng.choice([1, 2, 4, 5, 8])
    dim = rng.choice([64, 128])
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        batch = _spread(rng, 1, 64)
        new_max = rng.choice([1, _spread(rng, 1, max(1, 2048 // batch))])
        len_max = new_max + _spread(rng, 1, 2000)
        return {"op": op, "batch": batch, "new_max": new_max, "len_min": rng.randint(1, len_max),
                "len_max": len_max, "heads": heads, "dim": dim, "page": page, "dtype": dtype, "mix": mix}
    if op == "attend":
        q_heads = heads * rng.choice([1, 2, 3, 4, 7, 8])
        kind = rng.choice(["one", "few", "prompt"])
        if kind == "one":
            batch = _spread(rng, 1, 64)
            new_max, len_max = 1, _spread(rng, 1, 120000 // batch)
        elif kind == "few":
            batch = _spread(rng, 1, 32)
            new_max = rng.randint(2, 16)
            len_max = new_max + _spread(rng, 1, 100000 // batch)
        else:
            batch = rng.randint(1, 4)
            new_max = _spread(rng, 17, 2600 // batch)
            len_max = new_max + rng.choice([0, _spread(rng, 1, 800)])
        return {"op": op, "batch": batch, "new_max": new_max, "len_min": rng.randint(1, len_max),
                "len_max": len_max, "q_heads": min(q_heads, 24 // heads * heads), "heads": heads,
                "dim": dim, "page": page, "window": rng.choice([0, 0, _spread(rng, 1, 2 * len_max)]),
                "dtype": dtype, "mix": mix}
    if op == "w4":
        group = rng.choice([32, 64, 128])
        M = rng.choice([1, _spread(rng, 1, 64)])
        K = group * _spread(rng, 1, 8192 // group)
        return {"op": op, "M": M, "K": K, "N": _spread(rng, 1, 100000000 // K // max(1, M // 8)),
                "group": group, "dtype": dtype}
    M = rng.choice([1, _spread(rng, 1, 600)])
    V = _spread(rng, 1000, min(260000, 60000000 // M))
    return {"op": op, "M": M, "V": V, "top": rng.choice([0, 1, rng.randint(2, 32)]), "dtype": dtype}


# ---------------------------------------------------------------- the cases' own shape
def _lengths(case):
    """Cached tokens (the new ones among them) and new tokens of each sequence:
    the case alone decides them.  The first sequence has the most of both."""
    r = random.Random(case["mix"])
    lens = [case["len_max"]] + [r.randint(case["len_min"], case["len_max"]) for _ in range(case["batch"] - 1)]
    new = [min(case["new_max"], lens[0])]
    for n in lens[1:]:
        new.append(min(n, case["new_max"] if case["new_max"] <= 16 else r.randint(1, case["new_max"])))
    return lens, new


def _visible(case):
    """Query-key pairs that the causal mask and the window leave, per query head."""
    lens, new = _lengths(case)
    w = case["window"] or 1 << 40
    total = 0
    for n, t in zip(lens, new):
        pos = np.arange(n - t, n, dtype=np.int64)
        total += int(np.minimum(pos + 1, w).sum())
    return total


def _reach(case):
    """Cached tokens that some query of their sequence sees."""
    lens, new = _lengths(case)
    w = case["window"] or 1 << 40
    return sum(min(n, t - 1 + w) for n, t in zip(lens, new))


def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "append":
        lens, new = _lengths(case)
        row = case["heads"] * case["dim"]
        P = case["page"]
        pages = sum((n - 1) // P - (n - t) // P + 1 for n, t in zip(lens, new))
        # new rows in, their codes and the pages' scales out, and the touched pages' values
        return {"bytes": sum(new) * row * 2 * (size + 1) + pages * case["heads"] * 2 * (4 + P * case["dim"] * 4),
                "flops": sum(new) * row * 2 * 4}
    if case["op"] == "attend":
        lens, new = _lengths(case)
        reach = _reach(case)
        return {"bytes": reach * case["heads"] * case["dim"] * 2 + reach // case["page"] * case["heads"] * 8
                + 2 * sum(new) * case["q_heads"] * case["dim"] * size,
                "flops": 4 * _visible(case) * case["q_heads"] * case["dim"]}
    if case["op"] == "w4":
        M, K, N = case["M"], case["K"], case["N"]
        return {"bytes": N * K // 2 + N * (K // case["group"]) * 2 + M * (K + N) * size,
                "flops": 2 * M * K * N}
    M, V = case["M"], case["V"]
    return {"bytes": M * V * size + M * (16 + 12 * case["top"]), "flops": 6 * M * V}


# ---------------------------------------------------------------- inputs
def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _codes(x):
    """8-bit codes and scales, one scale for the last two dimensions."""
    d = x.abs().amax(dim=(-1, -2)) / 127
    return torch.round(x / d[..., None, None]).clamp(-127, 127).to(torch.int8), d


def _rows(g, T, H, D):
    """Rows of keys or values: a few channels of a head are larger than the others."""
    return _randn(g, T, H, D) * (1 + 4 * (torch.rand(1, H, D, generator=g, device=DEV) < 0.03))


def _paged(case, g, seed):
    """Page table, lengths and offsets; pages lie in any order."""
    lens, new = _lengths(case)
    P = case["page"]
    held = [-(-n // P) for n in lens]
    if case["op"] == "append":  # only the pages that the new tokens fall into are kept: [first, last]
        first = [(n - t) // P for n, t in zip(lens, new)]
    else:
        first = [0] * len(lens)
    total = sum(h - f for h, f in zip(held, first)) + 3
    order = np.random.RandomState(seed % (1 << 31)).permutation(total)
    table = np.zeros((len(lens), max(held)), dtype=np.int32)
    at = 0
    for b, (h, f) in enumerate(zip(held, first)):
        table[b, f:h] = order[at:at + h - f]
        at += h - f
    to = lambda v: torch.tensor(np.asarray(v, dtype=np.int32), device=DEV)  # noqa: E731
    offsets = np.concatenate([[0], np.cumsum(new)])
    return total, {"pages": to(table), "lens": to(lens), "offsets": to(offsets), "T": sum(new),
                   "seq": to(np.repeat(np.arange(len(new)), new)).long(), "one": max(new) == 1}


def prepare(case, seed):
    g = _generator(seed)
    dtype = DTYPES[case["dtype"]]
    state = {"case": case}
    if case["op"] in ("append", "attend"):
        total, s = _paged(case, g, seed)
        state |= s
        shape = (total, case["heads"], case["page"], case["dim"])
        channel = 1 + 4 * (torch.rand(1, shape[1], 1, shape[3], generator=g, device=DEV) < 0.03)
        state["k_codes"], state["k_scales"] = _codes(_randn(g, *shape) * channel)
        state["v_codes"], state["v_scales"] = _codes(_randn(g, *shape))
        if case["op"] == "append":
            H, D = case["heads"], case["dim"]
            # keys and values are columns of the fused projection's output
            rows = torch.cat([_rows(g, s["T"], H, D), _rows(g, s["T"], H, D)], dim=1).to(dtype)
            state["rows"] = rows
            state["k"], state["v"] = rows[:, :H], rows[:, H:]
        else:
            state["q"] = (1.5 * _randn(g, s["T"], case["q_heads"], case["dim"])).to(dtype)
        if own:
            import ternary_weight_linear_token_b200 as bl
            state["cache"] = bl.KVCache.from_tensors(state["k_codes"], state["v_codes"], state["k_scales"],
                                                     state["v_scales"])
    elif case["op"] == "w4":
        M, K, N, G = case["M"], case["K"], case["N"], case["group"]
        # weights of N(0, 0.02), their group's largest at code 7, stored as the library packs them: a
        # 32-bit word holds 8 consecutive weights, weight 2i + h at bits [16h + 4i, 16h + 4i + 4)
        w = (0.02 * torch.randn(N, K // G, G, generator=g, device=DEV, dtype=torch.float16)).float()
        s = (w.abs().amax(-1) / 7).to(torch.bfloat16)
        c = torch.round(w / s.float()[..., None]).clamp(-8, 7).to(torch.int32) + 8
        del w
        c = c.view(N, K // 8, 4, 2)
        shift = torch.tensor([[0, 16], [4, 20], [8, 24], [12, 28]], device=DEV, dtype=torch.int32)
        state["packed"] = (c << shift).sum((-1, -2), dtype=torch.int32).view(torch.uint8)  # [N, K / 2]
        state["scales"] = s
        state["x"] = _randn(g, M, K).to(dtype)
    else:
        M, V = case["M"], case["V"]
        x = 3 * _randn(g, M, V)
        x[:, ::97] += 6
        state["logits"] = x.to(dtype)
        state["tokens"] = torch.randint(0, V, (M,), generator=g, device=DEV)
        top = state["logits"].argmax(-1)
        state["tokens"] = torch.where(torch.arange(M, device=DEV) % 2 == 0, top, state["tokens"])
    return state


# ---------------------------------------------------------------- plain forms
def _away(v):
    """Nearest whole number, halves away from zero (the sum in 64 bits: 0.49999997 + 0.5 is below one)."""
    return torch.copysign(torch.floor(v.double().abs() + 0.5), v.double()).float()


def _append_plain(s, x, codes, scales):
    P = s["case"]["page"]
    pages, lens, offsets, seq = s["pages"].long(), s["lens"].long(), s["offsets"].long(), s["seq"]
    B = lens.numel()
    x = x.float()
    first = lens - (offsets[1:] - offsets[:-1])                       # [B] first new position
    pos = first[seq] + torch.arange(x.shape[0], device=x.device) - offsets[seq]
    page = pages[seq, pos // P]                                       # [T]
    # largest new value of each page and head
    peak = torch.zeros_like(scales).index_reduce_(0, page, x.abs().amax(-1), "amax", include_self=True)
    # older rows of the page in which a sequence's first new token falls
    at = pages[torch.arange(B, device=x.device), first.clamp(max=pages.shape[1] * P - 1) // P]
    older = torch.zeros(scales.shape[0], dtype=torch.long, device=x.device).index_put_((at,), first % P)
    touched = torch.zeros(scales.shape[0], dtype=torch.bool, device=x.device)
    touched[page] = True
    was = torch.where((older > 0)[:, None], scales, torch.zeros_like(scales))
    # (a tensor of 127s: torch multiplies by the rounded inverse of a plain number)
    now = torch.where(touched[:, None], torch.maximum(was, peak / torch.full_like(peak, 127)), scales)
    now = torch.where(touched[:, None] & (now < 2.0 ** -60), torch.zeros_like(now), now)
    inv = torch.where(now > 0, 1 / now, torch.zeros_like(now))
    grown = (now > scales) & (older > 0)[:, None] & touched[:, None]
    kept = torch.where(grown, was * inv, torch.ones_like(now))
    codes.copy_(_away(codes.float() * kept[..., None, None]))
    codes[page, :, pos % P] = _away(x * inv[page][..., None]).clamp(-127, 127).to(torch.int8)
    scales.copy_(now)


def _attend_plain(s):
    case = s["case"]
    H, D, G = case["heads"], case["dim"], case["q_heads"] // case["heads"]
    lens, offsets = s["lens"].long(), s["offsets"].long()
    B, n = lens.numel(), min(case["new_max"], case["len_max"])
    pages = s["pages"].long()
    L = pages.shape[1] * case["page"]

    def dense(codes, scales):  # [B, H, L, D]
        return (codes[pages].float() * scales[pages][..., None, None]).transpose(1, 2).reshape(B, H, L, D)

    new = offsets[1:] - offsets[:-1]
    i = torch.arange(n, device=lens.device)
    row = (offsets[:-1, None] + i).clamp(max=s["T"] - 1)              # [B, n]
    q = s["q"].float()[row].view(B, n, H, G, D).permute(0, 2, 3, 1, 4).reshape(B, H, G * n, D)
    scores = (q @ dense(s["k_codes"], s["k_scales"]).transpose(-1, -2)).view(B, H, G, n, L) / math.sqrt(D)
    at = (lens - new)[:, None] + i                                    # [B, n] positions
    j = torch.arange(L, device=lens.device)
    seen = (j <= at[..., None]) & (j < lens[:, None, None])
    if case["window"]:
        seen &= j > at[..., None] - case["window"]
    scores.masked_fill_(~seen[:, None, None], float("-inf"))
    scores -= scores.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    p = scores.exp_()
    total = p.sum(-1, keepdim=True)
    p /= torch.where(total > 0, total, torch.ones_like(total))
    o = p.view(B, H, G * n, L) @ dense(s["v_codes"], s["v_scales"])
    o = o.view(B, H, G, n, D).permute(0, 3, 1, 2, 4).reshape(B, n, H * G, D)
    return o[s["seq"], torch.arange(s["T"], device=lens.device) - offsets[s["seq"]]].to(s["q"].dtype)


def _w4_plain(s):
    K, G = s["case"]["K"], s["case"]["group"]
    word = s["packed"].view(torch.int32)                              # [N, K / 8]
    shift = torch.tensor([0, 16, 4, 20, 8, 24, 12, 28], device=word.device, dtype=torch.int32)
    w = ((word[..., None] >> shift) & 15).view(-1, K // G, G).float() - 8
    w = (w * s["scales"].float()[..., None]).view(-1, K)
    return (s["x"].float() @ w.T).to(s["x"].dtype)


def _logprobs_plain(s):
    top = s["case"]["top"]
    x = s["logits"].float()
    m = x.amax(-1, keepdim=True)
    e = (x - m).exp()
    total = e.sum(-1, keepdim=True)
    lp = x - m - total.log()
    out = {"logprob": lp.gather(-1, s["tokens"][:, None])[:, 0],
           "entropy": -(e * lp).sum(-1) / total[:, 0]}
    if top:
        at = torch.sort(x, dim=-1, descending=True, stable=True).indices[:, :top]
        out |= {"top_ids": at, "top_logprobs": lp.gather(-1, at)}
    return out


def run(state):
    op = state["case"]["op"]
    if own:
        import ternary_weight_linear_token_b200 as bl
        if op == "w4":
            return bl.bitnet_w4a16_matmul(state["x"], state["packed"], state["scales"], out_dtype=state["x"].dtype,
                                          weights_static=True)
        if op == "logprobs":
            lp, h, ids, top = bl.bitnet_token_logprobs(state["logits"], state["tokens"], top=state["case"]["top"])
            out = {"logprob": lp, "entropy": h}
            return out | {"top_ids": ids, "top_logprobs": top} if state["case"]["top"] else out
        offsets = None if state["one"] else state["offsets"]
        if op == "attend":
            return bl.bitnet_kv_attention(state["cache"], state["q"], state["pages"], state["lens"], offsets=offsets,
                                          max_new=min(state["case"]["new_max"], state["case"]["len_max"]),
                                          window=state["case"]["window"])
        bl.bitnet_kv_append(state["cache"], state["k"], state["v"], state["pages"], state["lens"], offsets=offsets,
                            max_new=min(state["case"]["new_max"], state["case"]["len_max"]))
    elif op == "w4":
        return _w4_plain(state)
    elif op == "logprobs":
        return _logprobs_plain(state)
    elif op == "attend":
        return _attend_plain(state)
    else:
        _append_plain(state, state["k"], state["k_codes"], state["k_scales"])
        _append_plain(state, state["v"], state["v_codes"], state["v_scales"])
    # the cache after the append, as the values that it stands for
    return {"k_scales": state["k_scales"], "v_scales": state["v_scales"],
            "k": state["k_codes"] * state["k_scales"][..., None, None],
            "v": state["v_codes"] * state["v_scales"][..., None, None]}


# ---------------------------------------------------------------- 64 bits
def _append_exact(case, x, codes, scales, table, lens, new):
    """Sequence by sequence, page by page, on the host; the definition rounds the scale, its inverse and
    the products to 32 bits, everything else is exact."""
    P, f = case["page"], np.float32

    def nearest(v):
        v = v.astype(np.float64)
        return np.sign(v) * np.floor(np.abs(v) + 0.5)
    at = 0
    for b, (n, t) in enumerate(zip(lens, new)):
        p = n - t
        while p < n:
            end = min(n, (p // P + 1) * P)
            rows = x[at:at + end - p]                                 # [r, H, D] float32
            page, lo = table[b, p // P], p % P
            for h in range(case["heads"]):
                d = f(np.abs(rows[:, h]).max()) / f(127)
                if lo:
                    before = scales[page, h]
                    d = max(d, before)
                if d < 2.0 ** -60:
                    d = f(0)
                inv = f(1) / d if d > 0 else f(0)
                if lo and d > before:
                    codes[page, h] = nearest(codes[page, h].astype(f) * (before * inv))
                codes[page, h, lo:lo + end - p] = np.clip(nearest(rows[:, h] * inv), -127, 127)
                scales[page, h] = d
            at += end - p
            p = end
    return codes.astype(np.float64) * scales.astype(np.float64)[..., None, None]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        lens, new = _lengths(case)
        host = lambda t: t.cpu().numpy()  # noqa: E731
        table = host(s["pages"])
        out = {}
        for name in ("k", "v"):
            scales = host(s[name + "_scales"]).copy()
            out[name] = torch.from_numpy(_append_exact(case, host(s[name].float()), host(s[name + "_codes"]).copy(),
                                                       scales, table, lens, new))
            out[name + "_scales"] = torch.from_numpy(scales.astype(np.float64))
        return out
    if case["op"] == "attend":
        lens, new = _lengths(case)
        P, G = case["page"], case["q_heads"] // case["heads"]
        out, at = [], 0
        for b, (n, t) in enumerate(zip(lens, new)):
            j = torch.arange(n, device=DEV)
            page, row = s["pages"][b, j // P].long(), j % P
            pos = torch.arange(n - t, n, device=DEV)
            hidden = j[None] > pos[:, None]
            if case["window"]:
                hidden |= j[None] + case["window"] <= pos[:, None]
            o = torch.empty(t, case["q_heads"], case["dim"], dtype=torch.float64, device=DEV)
            for h in range(case["heads"]):
                k = s["k_codes"][page, h, row].double() * s["k_scales"][page, h].double()[:, None]
                v = s["v_codes"][page, h, row].double() * s["v_scales"][page, h].double()[:, None]
                for i in range(h * G, h * G + G):
                    z = torch.einsum("td,jd->tj", s["q"][at:at + t, i].double(), k) * case["dim"] ** -0.5
                    o[:, i] = torch.softmax(z.masked_fill(hidden, -math.inf), -1) @ v
            out.append(o)
            at += t
        return torch.cat(out)
    if case["op"] == "w4":
        K, G, N = case["K"], case["group"], case["N"]
        y = torch.empty(case["M"], N, dtype=torch.float64, device=DEV)
        x = s["x"].double()
        for lo in range(0, N, 8192):  # rows of the weights at a time
            b = s["packed"][lo:lo + 8192].view(-1, K // 8, 4).to(torch.int16)
            w = torch.empty(b.shape[0], K // 8, 8, dtype=torch.float64, device=DEV)
            for i in range(8):  # weight i of a word: half i % 2, nibble i // 2 of that half
                byte = b[..., 2 * (i % 2) + i // 4]
                w[..., i] = (byte // 16 if i // 2 % 2 else byte % 16) - 8
            w = w.view(-1, K // G, G) * s["scales"][lo:lo + 8192].double()[..., None]
            y[:, lo:lo + 8192] = torch.einsum("mk,nk->mn", x, w.reshape(-1, K))
        return y
    out = {"logprob": [], "entropy": [], "top_logprobs": []}
    for x, t in zip(s["logits"], s["tokens"]):
        lp = torch.log_softmax(x.double(), -1)
        out["logprob"].append(lp[t])
        out["entropy"].append(-(lp.exp() * lp).sum())
        out["top_logprobs"].append(torch.topk(lp, case["top"]).values)
    out = {k: torch.stack(v) for k, v in out.items()}
    return out | {"top_ids": None} if case["top"] else {k: out[k] for k in ("logprob", "entropy")}
