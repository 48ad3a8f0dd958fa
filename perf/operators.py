"""The attention operators of the FP8 KV cache: what a pass of each is, its inputs, and its plain form.

  attend  new query tokens (a decode step or a chunk of a prompt) against the paged FP8 cache, if asked with
          the attention weight that every cached position has received so far
  evict   the positions to keep by that weight, and the cache rows and weights moved together into other pages
  prompt  causal attention of whole packed prompts over their bf16 states, before they are in a cache

`own` chooses between elementary torch operations in 32 bits and the library's calls.
"""

import math
import random

import torch

own = False

LLAMA8B = {"heads": 32, "kv_heads": 8, "head_dim": 128}   # the attention shape of the KV-cache workload


def listed():
    return [
        # one user, a short conversation: latency of a decode step
        {"name": "decode_b1_ctx500", "op": "attend", "batch": 1, "ctx": 500, "chunk": 1, "ragged": False, **LLAMA8B,
         "fmt": "e4m3", "scale": "channel", "block": 16, "weights": False},
        # the KV-cache workload: 32 sequences at 8k tokens, one step
        {"name": "decode_b32_ctx8k", "op": "attend", "batch": 32, "ctx": 8192, "chunk": 1, "ragged": False, **LLAMA8B,
         "fmt": "e4m3", "scale": "channel", "block": 16, "weights": False},
        # one very long document: the split over the cached positions carries it
        {"name": "decode_b1_ctx128k", "op": "attend", "batch": 1, "ctx": 131071, "chunk": 1, "ragged": False, **LLAMA8B,
         "fmt": "e5m2", "scale": "head", "block": 64, "weights": False},
        # a mixed batch whose weights are collected for a later eviction
        {"name": "decode_b24_weights", "op": "attend", "batch": 24, "ctx": 5003, "chunk": 1, "ragged": True,
         "heads": 28, "kv_heads": 4, "head_dim": 128, "fmt": "e4m3", "scale": "head", "block": 16, "weights": True},
        # verification of five drafted tokens a sequence, small heads
        {"name": "verify_b16_q5", "op": "attend", "batch": 16, "ctx": 2777, "chunk": 5, "ragged": True,
         "heads": 16, "kv_heads": 8, "head_dim": 64, "fmt": "e4m3", "scale": "tensor", "block": 32, "weights": False},
        # a chunk of a long prompt behind what is cached of it already
        {"name": "chunk_b2_q512_ctx8k", "op": "attend", "batch": 2, "ctx": 8192, "chunk": 512, "ragged": False, **LLAMA8B,
         "fmt": "e4m3", "scale": "channel", "block": 16, "weights": False},
        # chunks of different lengths with the weights collected
        {"name": "chunk_b6_q300_weights", "op": "attend", "batch": 6, "ctx": 3001, "chunk": 301, "ragged": True, **LLAMA8B,
         "fmt": "e4m3", "scale": "channel", "block": 16, "weights": True},
        # one conversation cut to a third
        {"name": "evict_b1_ctx1500", "op": "evict", "batch": 1, "ctx": 1500, "keep": 500, "ragged": False, "kv_heads": 8,
         "head_dim": 128, "block": 16, "first": 4, "recent": 64},
        # the KV-cache workload's batch cut to a half
        {"name": "evict_b32_ctx8k", "op": "evict", "batch": 32, "ctx": 8192, "keep": 4000, "ragged": True, "kv_heads": 8,
         "head_dim": 128, "block": 16, "first": 4, "recent": 256},
        # a few short requests that arrived together
        {"name": "prompt_b4_len200", "op": "prompt", "batch": 4, "len": 200, "ragged": True, **LLAMA8B},
        # a packed batch of chat prompts
        {"name": "prompt_b12_len1900", "op": "prompt", "batch": 12, "len": 1900, "ragged": True, **LLAMA8B},
        # two prompts as long as the workload's context
        {"name": "prompt_b2_len8k", "op": "prompt", "batch": 2, "len": 8192, "ragged": False, **LLAMA8B},
    ]


def _log_between(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    kv_heads, head_dim = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 128, 256])
    heads = kv_heads * rng.choice([1, 2, 3, 4, 7, 8])
    shape = {"heads": heads, "kv_heads": kv_heads, "head_dim": head_dim}
    op = rng.choice(["decode", "decode", "chunk", "chunk", "evict", "prompt", "prompt"])
    if op == "prompt":
        length = _log_between(rng, 16, 6000)
        batch = min(_log_between(rng, 1, 24), max(1, (1 << 29) // (heads * length * length)))
        return {"op": "prompt", "batch": batch, "len": length, "ragged": rng.random() < 0.7, **shape}
    ctx = _log_between(rng, 64, 32768)
    block = rng.choice([1, 16, 16, 32, 64, 128])
    batch = min(_log_between(rng, 1, 48), max(1, (1 << 18) // ctx), max(1, (1 << 28) // (ctx * kv_heads * head_dim)))
    if op == "evict":
        keep = max(1, int(ctx * rng.uniform(0.1, 0.9)))
        first = min(keep // 4, rng.randrange(0, 9))
        return {"op": "evict", "batch": batch, "ctx": ctx, "keep": keep, "ragged": rng.random() < 0.7,
                "kv_heads": kv_heads, "head_dim": head_dim, "block": block, "first": first,
                "recent": rng.randrange(0, keep // 2 + 1)}
    chunk = 1 if op == "decode" else min(ctx, _log_between(rng, 2, 1024), max(2, (1 << 28) // (batch * heads * ctx)))
    return {"op": "attend", "batch": batch, "ctx": ctx, "chunk": chunk, "ragged": rng.random() < 0.7, **shape,
            "fmt": rng.choice(["e4m3", "e4m3", "e5m2"]), "scale": rng.choice(["tensor", "head", "channel"]),
            "block": block, "weights": rng.random() < 0.35}


def _lengths(n, top, ragged, low=1):
    """n lengths up to top (the first is top), by the case alone."""
    rng = random.Random(n * 1000003 + top)
    return [top if not ragged or i == 0 else rng.randint(min(low, top), top) for i in range(n)]


def _attend_lengths(case):
    ctx = _lengths(case["batch"], case["ctx"], case["ragged"], max(1, case["ctx"] // 8))
    new = _lengths(case["batch"], case["chunk"], case["ragged"])
    return [min(a, b) for a, b in zip(new, ctx)], ctx


def work(case):
    if case["op"] == "prompt":
        lens, h, d = _lengths(case["batch"], case["len"], case["ragged"]), case["heads"], case["head_dim"]
        pairs = sum(n * (n + 1) // 2 for n in lens)
        return {"bytes": sum(lens) * (2 * d * (2 * h + 2 * case["kv_heads"]) + 4 * h), "flops": 4 * pairs * h * d}
    row = case["kv_heads"] * case["head_dim"]
    if case["op"] == "evict":
        lens = _lengths(case["batch"], case["ctx"], case["ragged"], case["ctx"] // 2)
        kept = sum(min(n, case["keep"]) for n in lens)
        return {"bytes": 4 * case["kv_heads"] * (sum(lens) + kept) + 4 * row * kept + 8 * kept, "flops": 0}
    new, ctx = _attend_lengths(case)
    pairs = sum(n * c - n * (n - 1) // 2 for n, c in zip(new, ctx))
    per_token = case["heads"] * (4 * case["head_dim"] + 4)
    return {"bytes": 2 * row * sum(ctx) + per_token * sum(new) + (8 * case["kv_heads"] * sum(ctx) if case["weights"] else 0),
            "flops": 4 * pairs * case["heads"] * case["head_dim"]}


# ---- inputs ---------------------------------------------------------------------

def _starts(lens):
    s = [0]
    for n in lens:
        s.append(s[-1] + n)
    return torch.tensor(s, dtype=torch.int64, device="cuda")


def _pool(g, slots, kv_heads, head_dim, fmt, scale):
    """Codes of a whole pool (also of slots no sequence holds: earlier requests' tokens) and their static scales:
    states N(0, sigma^2) with 1/64 of the channels at sigma 20, scales of sigma / 56 for a channel, or the largest."""
    sigma = torch.ones(kv_heads, head_dim, device="cuda")
    sigma.view(-1)[torch.randperm(kv_heads * head_dim, generator=g, device="cuda")[:max(1, kv_heads * head_dim // 64)]] = 20.0
    s = {"channel": sigma, "head": sigma.amax(1, keepdim=True), "tensor": sigma.amax().view(1, 1)}[scale] / 56
    f8, top = (torch.float8_e4m3fn, 448.0) if fmt == "e4m3" else (torch.float8_e5m2, 57344.0)
    codes = torch.empty(slots, kv_heads, head_dim, dtype=torch.uint8, device="cuda")
    for at in range(0, slots, 1 << 16):
        part = codes[at:at + (1 << 16)]
        x = torch.randn(part.shape, generator=g, device="cuda") * sigma / s
        part.copy_(x.clamp_(-top, top).to(f8).view(torch.uint8))
    return codes, s.reshape(-1).contiguous()


def _pages(g, batch, top, block, extra=0):
    """A block table of random pages for `batch` sequences of up to `top` positions, and the pool's slots."""
    per = -(-top // block)
    blocks = batch * per + batch * per // 4 + 1
    table = torch.randperm(blocks, generator=g, device="cuda")[:batch * per].view(batch, per).contiguous()
    return table, (blocks + extra) * block, blocks


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    if case["op"] == "prompt":
        lens = _lengths(case["batch"], case["len"], case["ragged"])
        h, hk, d, n = case["heads"], case["kv_heads"], case["head_dim"], sum(lens)
        # the output of one fused projection: queries, keys and values side by side in a row
        qkv = torch.randn(n, (h + 2 * hk) * d, generator=g, device="cuda").to(torch.bfloat16)
        s["q"] = qkv[:, :h * d].view(n, h, d)
        s["k"] = qkv[:, h * d:(h + hk) * d].view(n, hk, d)
        s["v"] = qkv[:, (h + hk) * d:].view(n, hk, d)
        s["starts"] = _starts(lens)
        return s
    hk, d, block = case["kv_heads"], case["head_dim"], case["block"]
    if case["op"] == "evict":
        lens = _lengths(case["batch"], case["ctx"], case["ragged"], case["ctx"] // 2)
        per = -(-case["keep"] // block)
        s["table"], slots, first = _pages(g, case["batch"], case["ctx"], block, case["batch"] * per)
        s["to"] = torch.arange(first, first + case["batch"] * per, device="cuda").view(case["batch"], per)
        s["new"] = slice(first * block, slots)       # the destination's slots: free pages at the pool's end
        s["k"], _ = _pool(g, slots, hk, d, "e4m3", "channel")
        s["v"], _ = _pool(g, slots, hk, d, "e4m3", "channel")
        s["k"][s["new"]] = 0
        s["v"][s["new"]] = 0
        s["lens"] = torch.tensor(lens, dtype=torch.int64, device="cuda")
        # accumulated softmax weights: a heavy tail
        s["weights"] = torch.exp(2 * torch.randn(case["batch"], hk, case["ctx"], generator=g, device="cuda") - 4)
        s["weights_to"] = torch.zeros(case["batch"], hk, case["keep"], device="cuda")
        return s
    new, ctx = _attend_lengths(case)
    s["table"], slots, _ = _pages(g, case["batch"], case["ctx"], block)
    s["k"], s["ks"] = _pool(g, slots, hk, d, case["fmt"], case["scale"])
    s["v"], s["vs"] = _pool(g, slots, hk, d, case["fmt"], case["scale"])
    s["q"] = torch.randn(sum(new), case["heads"], d, generator=g, device="cuda").to(torch.bfloat16)
    s["starts"] = _starts(new)
    s["lens"] = torch.tensor(ctx, dtype=torch.int64, device="cuda")
    if case["weights"]:
        s["weights"] = torch.zeros(case["batch"], hk, case["ctx"], device="cuda")
        s["weights_to"] = torch.zeros_like(s["weights"])
        seen = torch.rand(case["batch"], hk, case["ctx"], generator=g, device="cuda")
        live = torch.arange(case["ctx"], device="cuda") < (s["lens"] - s["starts"].diff()).view(-1, 1, 1)
        s["weights"].copy_(torch.where(live, seen, 0))
    return s


# ---- the plain forms ------------------------------------------------------------

def _values(codes, fmt):
    return codes.view(torch.float8_e4m3fn if fmt == "e4m3" else torch.float8_e5m2).to(torch.float32)


def _spread(scales, hk, d):
    return scales.view(1, 1) if scales.numel() == 1 else scales.view(hk, -1).expand(hk, d)


def _slots(table, block, top):
    at = torch.arange(top, device="cuda")
    return table[:, at // block] * block + at % block


def _padded(x, starts, top):
    """Packed rows [tokens, ...] as [batch, top, ...], the last row again behind each sequence."""
    at = starts[:-1, None] + torch.arange(top, device="cuda")
    return x[at.clamp(max=x.shape[0] - 1)]


def _packed(x, starts, tokens):
    """The inverse of _padded."""
    at = torch.arange(tokens, device="cuda")
    b = torch.bucketize(at, starts[1:], right=True)
    return x[b, at - starts[b]]


def _softmax_attention(q, k, v, limit):
    """q [B, Q, H, D] against k, v [B, L, Hk, D]: position j is seen by token i of a sequence where j < limit[b, i].
    Outputs [B, Q, H, D], log sums [B, Q, H] and probabilities [B, Hk, G, Q, L]."""
    B, Q, H, D = q.shape
    L, Hk = k.shape[1], k.shape[2]
    q = q.view(B, Q, Hk, H // Hk, D).permute(0, 2, 3, 1, 4).reshape(B, Hk, -1, D)
    s = torch.matmul(q, k.permute(0, 2, 3, 1).contiguous()).view(B, Hk, H // Hk, Q, L)
    s.mul_(D ** -0.5)
    s.masked_fill_((torch.arange(L, device="cuda") >= limit[..., None]).view(B, 1, 1, Q, L), -math.inf)
    m = s.amax(-1, keepdim=True)
    p = s.sub_(m.clamp(min=-1e30)).exp_()
    l = p.sum(-1, keepdim=True)
    p = p.div_(l.clamp(min=1e-30))
    o = torch.matmul(p.view(B, Hk, -1, L), v.permute(0, 2, 1, 3).contiguous()).view(B, Hk, H // Hk, Q, D)
    lse = (m + torch.log(l)).squeeze(-1)
    return o.permute(0, 3, 1, 2, 4).reshape(B, Q, H, D), lse.permute(0, 3, 1, 2).reshape(B, Q, H), p


def _plain_attend(s):
    case = s["case"]
    hk, d, Q, L = case["kv_heads"], case["head_dim"], case["chunk"], case["ctx"]
    at = _slots(s["table"], case["block"], L)
    k = _values(s["k"][at], case["fmt"]).mul_(_spread(s["ks"], hk, d))
    v = _values(s["v"][at], case["fmt"]).mul_(_spread(s["vs"], hk, d))
    new, i = s["starts"].diff(), torch.arange(Q, device="cuda")
    limit = s["lens"][:, None] - new[:, None] + i + 1
    o, lse, p = _softmax_attention(_padded(s["q"], s["starts"], Q).float(), k, v, limit.minimum(s["lens"][:, None]))
    n = s["q"].shape[0]
    out = [_packed(o, s["starts"], n).to(torch.bfloat16), _packed(lse, s["starts"], n)]
    if case["weights"]:
        p.mul_((i < new[:, None]).view(-1, 1, 1, Q, 1))
        out.append(s["weights"] + p.sum((2, 3)))
    return out


def _plain_evict(s):
    case = s["case"]
    L, keep = case["ctx"], case["keep"]
    lens, at = s["lens"][:, None], torch.arange(L, device="cuda")
    score = s["weights"].double().sum(1).float()         # one order of the heads or another: the same after rounding
    score = torch.where((at < case["first"]) | (at >= lens - case["recent"]), math.inf, score)
    score = torch.where(at < lens, score, -1.0)
    order = torch.sort(score, dim=1, descending=True, stable=True).indices[:, :keep]
    kept = torch.where(order < lens, order, L).sort(1).values
    have = kept < L
    count = have.sum(1)
    src = _slots(s["table"], case["block"], L).gather(1, kept.clamp(max=L - 1))[have]
    dst = _slots(s["to"], case["block"], keep)[have]
    s["k"][dst] = s["k"][src]
    s["v"][dst] = s["v"][src]
    moved = s["weights"].gather(2, kept.clamp(max=L - 1)[:, None].expand(-1, case["kv_heads"], -1))
    f8 = torch.float8_e4m3fn
    return [torch.where(have, kept, -1), count, s["k"][s["new"]].view(f8), s["v"][s["new"]].view(f8),
            torch.where(have[:, None], moved, 0.0)]


def _plain_prompt(s):
    case = s["case"]
    L = case["len"]
    limit = (torch.arange(L, device="cuda") + 1).expand(case["batch"], L)
    o, lse, _ = _softmax_attention(*(_padded(s[x], s["starts"], L).float() for x in "qkv"), limit)
    n = s["q"].shape[0]
    return [_packed(o, s["starts"], n).to(torch.bfloat16), _packed(lse, s["starts"], n)]


# ---- the library's calls --------------------------------------------------------

def _own_attend(s):
    import block_scaled_precision_x128_amd as fb
    case = s["case"]
    fmt = fb.E4M3 if case["fmt"] == "e4m3" else fb.E5M2
    kind = {"tensor": fb.KV_SCALE_TENSOR, "head": fb.KV_SCALE_HEAD, "channel": fb.KV_SCALE_CHANNEL}[case["scale"]]
    out, lse = fb.fp8_kv_attention(s["q"], s["k"], s["v"], s["table"], case["block"], s["starts"], s["lens"],
                                   s["ks"], s["vs"], fmt, kind, max_q=case["chunk"], max_kv=case["ctx"],
                                   weights_in=s.get("weights"), weights_out=s.get("weights_to"))
    return [out, lse] + ([s["weights_to"]] if case["weights"] else [])


def _own_evict(s):
    import block_scaled_precision_x128_amd as fb
    case = s["case"]
    kept, count = fb.fp8_kv_evict_select(s["weights"], s["lens"], case["keep"], first=case["first"],
                                         recent=case["recent"])
    fb.fp8_kv_compact(s["k"], s["v"], s["table"], s["to"], case["block"], kept, count, weights_in=s["weights"],
                      weights_out=s["weights_to"])
    f8 = torch.float8_e4m3fn
    return [kept, count, s["k"][s["new"]].view(f8), s["v"][s["new"]].view(f8), s["weights_to"]]


def _own_prompt(s):
    import block_scaled_precision_x128_amd as fb
    out, lse = fb.fp8_prompt_attention(s["q"], s["k"], s["v"], s["starts"], max_len=s["case"]["len"])
    return [out, lse]


def run(state):
    op = state["case"]["op"]
    if own:
        return {"attend": _own_attend, "evict": _own_evict, "prompt": _own_prompt}[op](state)
    return {"attend": _plain_attend, "evict": _plain_evict, "prompt": _plain_prompt}[op](state)


# ---- the definition in 64 bits --------------------------------------------------

def _exact_sequence(q, k, v):
    """One sequence in float64: q [n, H, D] are the last n of the positions of k, v [L, Hk, D]."""
    n, H, D = q.shape
    L, Hk = k.shape[:2]
    out, lse, received = torch.empty_like(q), torch.empty(n, H, dtype=q.dtype, device=q.device), []
    hidden = torch.ones(n, L, dtype=torch.bool, device=q.device).triu(L - n + 1)
    for kh in range(Hk):
        total = 0
        for h in range(kh * (H // Hk), (kh + 1) * (H // Hk)):
            s = (q[:, h] @ k[:, kh].T.contiguous()) / math.sqrt(D)
            s[hidden] = -math.inf
            lse[:, h] = torch.logsumexp(s, 1)
            p = torch.exp(s - lse[:, h, None])
            out[:, h] = p @ v[:, kh]
            total = total + p.sum(0)
        received.append(total)
    return out, lse, torch.stack(received)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "evict":
        L, keep, got = case["ctx"], case["keep"], []
        for b, n in enumerate(s["lens"].tolist()):
            score = [float(x) for x in s["weights"][b, :, :n].double().sum(0).float().tolist()]
            forced = [j for j in range(n) if j < case["first"] or j >= n - case["recent"]]
            rest = sorted(set(range(n)) - set(forced), key=lambda j: (-score[j], j))
            got.append(sorted((forced + rest)[:keep]) if n > keep else list(range(n)))
        kept = torch.tensor([x + [-1] * (keep - len(x)) for x in got])
        moved = torch.zeros(case["batch"], case["kv_heads"], keep, dtype=torch.float64)
        for b, x in enumerate(got):
            moved[b, :, :len(x)] = s["weights"][b].double().cpu()[:, x]
        return [kept, torch.tensor([len(x) for x in got]), None, None, moved]
    starts = s["starts"].tolist()
    if case["op"] == "prompt":
        parts = [_exact_sequence(*(s[x][a:b].double() for x in "qkv")) for a, b in zip(starts, starts[1:])]
        return [torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts])]
    hk, d = case["kv_heads"], case["head_dim"]
    f8 = torch.float8_e4m3fn if case["fmt"] == "e4m3" else torch.float8_e5m2
    fold = {"tensor": lambda x: x.view(1, 1), "head": lambda x: x.view(hk, 1), "channel": lambda x: x.view(hk, d)}[case["scale"]]
    ks, vs = fold(s["ks"]).double(), fold(s["vs"]).double()
    outs, lses, weights = [], [], s["weights"].double() if case["weights"] else None
    for b, n in enumerate(s["lens"].tolist()):
        pages = s["table"][b, :-(-n // case["block"])]
        rows = (pages[:, None] * case["block"] + torch.arange(case["block"], device="cuda")).view(-1)[:n]
        o, lse, received = _exact_sequence(s["q"][starts[b]:starts[b + 1]].double(),
                                           s["k"][rows].view(f8).double() * ks, s["v"][rows].view(f8).double() * vs)
        outs.append(o)
        lses.append(lse)
        if weights is not None:
            weights[b, :, :n] += received
    return [torch.cat(outs), torch.cat(lses)] + ([weights] if weights is not None else [])
