"""What is measured of the operators that bring a prompt into a cache of bounded size.

A server that bounds the keys it keeps of each request attends over the prompt's
own projections, sums up how much attention every key received, chooses the keys
that stay, and closes the gaps in the paged cache:

  packed   attention over whole prompts, packed one behind the other: grouped heads,
           causal or not, with capped scores and a window
  weigh    the attention weight that each key of the paged cache received from the
           call's queries, added to what it had ("step" cases: single tokens;
           others: a prompt's last tokens, or all of them)
  select   the keys of each request and kv head that stay: the first ones, the
           latest ones, and those of the largest weight
  compact  their rows moved into the slots that became free below the new length

A case is a dict of plain values.  The lengths of its requests follow from the
case alone (its "lens" number), the values from the seed of prepare().
"""
import math
import random

import numpy as np
import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp8": torch.float8_e4m3fn}
_SIZES = {"bf16": 2, "fp16": 2, "fp8": 1}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one long prompt: the rate of the products counts
        dict(name="packed_16k", op="packed", requests=1, new=16384, past=0, lens=1, heads=32, kv_heads=8, dim=128,
             dtype="bf16", causal=True, cap=0.0, window=0),
        # a batch of ragged prompts whose model caps its scores and sees a window
        dict(name="packed_cap_window_b16", op="packed", requests=16, new=2500, past=0, lens=2, heads=32, kv_heads=8,
             dim=128, dtype="bf16", causal=True, cap=50.0, window=1024),
        # a few short texts to embed, every token sees all of its own, seven heads to a kv head: latency
        dict(name="packed_short_fp16", op="packed", requests=3, new=77, past=0, lens=3, heads=28, kv_heads=4, dim=64,
             dtype="fp16", causal=False, cap=0.0, window=0),
        # a decode step of 64 requests, the new weights added to those before
        dict(name="weigh_step_b64", op="weigh", requests=64, new=1, keys=4096, lens=4, heads=32, kv_heads=8, dim=128,
             page=16, dtype="bf16", cap=0.0, window=0, last=0, prior=True, decay=1.0),
        # a decode step on a few long contexts in an fp8 cache, the weights fading
        dict(name="weigh_step_fp8_long", op="weigh", requests=4, new=1, keys=131072, lens=5, heads=64, kv_heads=8,
             dim=128, page=64, dtype="fp8", cap=0.0, window=0, last=0, prior=True, decay=0.95),
        # what the last 64 tokens of a 32768-token prompt look at
        dict(name="weigh_last_32k", op="weigh", requests=1, new=64, keys=32768, lens=6, heads=32, kv_heads=8, dim=128,
             page=16, dtype="bf16", cap=0.0, window=0, last=64, prior=False, decay=1.0),
        # what all tokens of a 16384-token prompt looked at
        dict(name="weigh_prompt_16k", op="weigh", requests=1, new=16384, keys=16384, lens=7, heads=32, kv_heads=8,
             dim=128, page=16, dtype="bf16", cap=0.0, window=0, last=0, prior=False, decay=1.0),
        # after the prompts of a batch: each down to at most 1024 keys
        dict(name="select_b64", op="select", requests=64, keys=4096, even=False, lens=8, kv_heads=8, budget=1024,
             sinks=4, recent=64, pool=7, moved=False),
        # a few long contexts down to 8192 keys
        dict(name="select_long", op="select", requests=4, keys=131072, even=False, lens=9, kv_heads=8, budget=8192,
             sinks=4, recent=256, pool=1, moved=False),
        # one user while decoding, keys out of order by earlier evictions: latency
        dict(name="select_step_b1", op="select", requests=1, keys=1088, even=True, lens=10, kv_heads=8, budget=1024,
             sinks=4, recent=128, pool=1, moved=True),
        # 32768-token prompts down to 4096 keys
        dict(name="compact_prompt_32k", op="compact", requests=4, keys=32768, even=False, lens=11, kv_heads=8, dim=128,
             page=16, dtype="bf16", budget=4096, moved=False),
        # 64 requests while decoding, 64 of 1088 keys leave
        dict(name="compact_step_b64", op="compact", requests=64, keys=1088, even=True, lens=12, kv_heads=8, dim=128,
             page=16, dtype="bf16", budget=1024, moved=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["packed", "step", "prompt", "select", "compact"])
    dim = rng.choice([64, 128, 128])
    kv = rng.choice([1, 2, 4, 8, 8])
    group = rng.choice([1, 2, 4, 7, 8])
    page = rng.choice([16, 32, 48, 64])
    lens = rng.randrange(1 << 30)
    cap = rng.choice([0.0, 0.0, 30.0, 50.0])
    if op == "packed":
        new = _log(rng, 1, 6000)
        return dict(op="packed", requests=rng.randint(1, max(1, min(12, 8192 // new))), new=new,
                    past=rng.choice([0, 0, _log(rng, 1, 2048)]), lens=lens, heads=kv * group, kv_heads=kv, dim=dim,
                    dtype=rng.choice(["bf16", "fp16"]), causal=rng.random() < 0.8, cap=cap,
                    window=rng.choice([0, 0, _log(rng, 1, 4096)]))
    dtype = rng.choice(["bf16", "fp16"] if dim == 64 else ["bf16", "bf16", "fp16", "fp8"])
    prior = rng.random() < 0.6
    if op == "step":
        requests = _log(rng, 1, 128)
        return dict(op="weigh", requests=requests, new=rng.choice([1, 1, 1, 3]),
                    keys=_log(rng, 3, min(32768, 262144 // requests)), lens=lens, heads=kv * group,
                    kv_heads=kv, dim=dim, page=page, dtype=dtype, cap=cap, window=rng.choice([0, 0, 500]), last=0,
                    prior=prior, decay=rng.choice([1.0, 0.9]))
    if op == "prompt":
        new = _log(rng, 8, 8192)
        return dict(op="weigh", requests=rng.randint(1, max(1, min(8, 8192 // new))), new=new,
                    keys=new + rng.choice([0, 0, _log(rng, 1, 8192)]), lens=lens, heads=kv * group, kv_heads=kv,
                    dim=dim, page=page, dtype=dtype, cap=cap, window=rng.choice([0, 0, _log(rng, 16, 4096)]),
                    last=rng.choice([0, 16, 32, 100]), prior=prior, decay=rng.choice([1.0, 0.9]))
    requests = _log(rng, 1, 128)
    keys = _log(rng, 16, max(16, min(131072 if op == "select" else 16384, 4000000 // (requests * kv))))
    budget = max(8, int(keys * rng.choice([0.05, 0.3, 0.6, 0.95])))
    moved = rng.random() < 0.4
    if op == "select":
        sinks = rng.randint(0, min(8, budget // 4))
        return dict(op="select", requests=requests, keys=keys, even=rng.random() < 0.4, lens=lens, kv_heads=kv,
                    budget=budget, sinks=sinks, recent=rng.randint(0, min(256, budget // 2)),
                    pool=1 if moved else rng.choice([1, 5, 7]), moved=moved)
    return dict(op="compact", requests=requests, keys=keys, even=rng.random() < 0.4, lens=lens, kv_heads=kv, dim=dim,
                page=page, dtype=dtype, budget=budget, moved=moved)


def _lengths(c):
    """Per request: the new tokens (none of select and compact), and all its keys with them."""
    r = random.Random(c["lens"])
    B = c["requests"]
    if "budget" in c:
        least = c["keys"] if c["even"] or B == 1 else max(1, c["keys"] // 4)
        return [0] * B, [r.randint(least, c["keys"]) for _ in range(B)]
    steps = c["op"] == "weigh" and c["new"] <= 3
    new = [c["new"] if steps or B == 1 else r.randint(max(1, c["new"] // 4), c["new"]) for _ in range(B)]
    most = c["past"] if c["op"] == "packed" else c["keys"] - c["new"]
    return new, [n + (most if B == 1 or most <= 0 else r.randint(most // 8, most)) for n in new]


def _seen(c, pos, L):
    """Keys [lo, hi) that a token at position `pos` of a request of L keys sees (tensors or numbers of numpy)."""
    hi = pos + 1 if c.get("causal", True) else L + 0 * pos
    lo = pos - (c["window"] - 1) if c["window"] else 0 * pos
    return lo, hi


def _weighers(c, n):
    """How many of a request's n tokens weigh its keys."""
    return min(n, c["last"]) if c["last"] else n


def work(case):
    c = case
    H = c["kv_heads"]
    new, keys = _lengths(c)
    if c["op"] == "select":
        return {"bytes": sum(H * 4 * (L + min(L, c["budget"])) for L in keys), "flops": sum(H * L for L in keys)}
    if c["op"] == "compact":
        # each row below the new length is kept with the chance budget / L: the others receive one
        n = c["budget"]
        rows = sum(H * n * (1 - n / L) for L in keys if L > n)
        each = 2 * c["dim"] * _SIZES[c["dtype"]] + 4 + (4 if c["moved"] else 0)
        return {"bytes": int(rows * 2 * each) + sum(H * 4 * n for L in keys if L > n) + 4 * len(keys), "flops": 0}
    D, Hq, elt = c["dim"], c["heads"], _SIZES[c["dtype"]]
    pairs = tokens = 0
    for n, L in zip(new, keys):
        m = n if c["op"] == "packed" else _weighers(c, n)
        lo, hi = _seen(c, np.arange(L - m, L), L)
        pairs += int(np.maximum(np.minimum(hi, L) - np.maximum(lo, 0), 0).sum())
        tokens += m
    if c["op"] == "packed":
        return {"bytes": tokens * Hq * (2 * D * elt + 4) + sum(keys) * H * 2 * D * elt, "flops": 4 * D * Hq * pairs}
    return {"bytes": tokens * Hq * (D * elt + 4) + sum(keys) * H * (D * elt + 4 + (4 if c["prior"] else 0)),
            "flops": 2 * D * Hq * pairs}


# ------------------------------------------------------------------ the inputs
def _quantise(x):
    """Values in e4m3 with the scale that takes the largest to 448."""
    scale = float(x.abs().amax().float()) / 448.0
    return (x.float() / scale).clamp(-448.0, 448.0).to(torch.float8_e4m3fn), scale


def _values(gen, shape, dtype, spread=1.0):
    """(normal values, their scale)"""
    if dtype != "fp8":
        return (spread * torch.randn(shape, device="cuda", generator=gen, dtype=torch.float32)).to(_TYPES[dtype]), 1.0
    return _quantise(spread * torch.randn(shape, device="cuda", generator=gen, dtype=torch.float16))


def _bits(x):
    return x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x


def _tables(gen, lens, page):
    """Block tables of requests with these lengths, their pages scattered over a pool, and the pool's pages."""
    counts = [-(-n // page) for n in lens]
    pages = sum(counts) + 3
    order = torch.randperm(pages, device="cuda", generator=gen).to(torch.int32)
    width, rows, at = max(counts), [], 0
    for n in counts:
        rows.append(torch.nn.functional.pad(order[at:at + n], (0, width - n)))
        at += n
    return torch.stack(rows).contiguous(), pages


def _ints(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _received(gen, shape):
    """Attention weight received: spread over orders of magnitude, nothing at all for some keys."""
    x = torch.exp(2.0 * torch.randn(shape, device="cuda", generator=gen))
    return x * (torch.rand(shape, device="cuda", generator=gen) > 0.3)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    H = c["kv_heads"]
    new, keys = _lengths(c)
    s = {"case": c, "lens": _ints(keys), "longest": max(keys)}
    if "budget" in c:
        B, S = c["requests"], max(keys)
        if c["op"] == "compact":
            s["table"], pages = _tables(gen, keys, c["page"])
            S = s["table"].shape[1] * c["page"]
            k, _ = _values(gen, (pages, H, c["page"], 2 * c["dim"]), c["dtype"])
            s["cache"] = k
            # what a selection answers: the n largest of random weights, rising, and how many
            x = _received(gen, (B, H, S)).masked_fill_(torch.arange(S, device="cuda") >= s["lens"][:, None, None], -1.0)
            n = torch.minimum(s["lens"], torch.tensor(c["budget"], device="cuda")).int()
            first = min(c["budget"], S)
            kept = x.sort(dim=-1, descending=True, stable=True)[1][..., :first]
            kept = kept.masked_fill(torch.arange(first, device="cuda") >= n[:, None, None], S).sort(-1)[0]
            kept = torch.nn.functional.pad(kept, (0, c["budget"] - first), value=S)
            s["kept"], s["kept_lens"] = kept.masked_fill(kept == S, -1).int().contiguous(), n
        s["weights"] = _received(gen, (B, H, S))
        # after earlier evictions the keys lie in any order, with gaps between their positions
        if c["moved"]:
            s["context"] = _ints([2 * S + 5] * B)
            order = torch.rand((B, H, 2 * S + 5), device="cuda", generator=gen).argsort(-1)
            s["positions"] = order[..., :S].int().contiguous()
        return s
    D, Hq = c["dim"], c["heads"]
    s["scale"] = D ** -0.5
    s["starts"] = _ints(np.concatenate([[0], np.cumsum(new)]))
    s["most"] = max(new)
    # scores with a spread of 3
    s["q"], s["q_scale"] = _values(gen, (sum(new), Hq, D), c["dtype"], 3.0)
    if c["op"] == "packed":
        s["key_starts"] = _ints(np.concatenate([[0], np.cumsum(keys)])) if keys != new else None
        # the fused projection of a layer: keys and values are strided views of one tensor
        kv, _ = _values(gen, (sum(keys), 2 * H, D), c["dtype"])
        s["k"], s["v"] = kv[:, :H], kv[:, H:]
        return s
    s["table"], pages = _tables(gen, keys, c["page"])
    k, s["k_scale"] = _values(gen, (pages, H, c["page"], D), c["dtype"])
    v, _ = _values(gen, (pages, H, c["page"], D), c["dtype"])
    s["cache"] = torch.cat([_bits(k), _bits(v)], -1).view(k.dtype)
    S = s["table"].shape[1] * c["page"]
    # what the tokens' attention left in hand: the logarithm of each row's sum
    s["lse"] = torch.zeros((sum(new), Hq), device="cuda")
    for x, token, real in _scores(s, _queries(s, 0), _gathered(s)):
        s["lse"][token[real]] = x.flatten(1, 2).transpose(1, 2).logsumexp(-1)[real]
    s["prior"] = _received(gen, (c["requests"], H, S)) if c["prior"] else None
    s["out"] = torch.zeros((c["requests"], H, S), device="cuda")
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    return {"packed": _packed, "weigh": _weigh, "select": _select, "compact": _compact}[state["case"]["op"]](state)


def _queries(s, last):
    """The (last) tokens of each request, padded: token [B, n], whether it is one, its position, keys [lo, hi)."""
    c, L = s["case"], s["lens"].long()
    new = (s["starts"][1:] - s["starts"][:-1]).long()
    n = min(s["most"], last) if last else s["most"]
    i = torch.arange(n, device="cuda")
    if last:
        i = i + (new - n).clamp(min=0)[:, None]
    real = (i < new[:, None]).expand(len(L), n)
    token = (s["starts"][:-1].long()[:, None] + i).clamp(max=s["q"].shape[0] - 1)
    lo, hi = _seen(c, L[:, None] - new[:, None] + i, L[:, None])
    return token, real, lo.expand_as(real), torch.minimum(hi, L[:, None]).expand_as(real)


def _gathered(s):
    """The keys of each row of the block table in 32 bits: [B, longest, kv heads, D]."""
    t, P = torch.arange(s["longest"], device="cuda"), s["case"]["page"]
    rows = _bits(s["cache"])[..., :s["cache"].shape[-1] // 2][s["table"][:, t // P].long(), :, t % P]
    return rows.contiguous().view(s["cache"].dtype).float() * s["k_scale"]


def _scores(s, queries, k):
    """The masked scores [B, kv heads, G, tokens, keys] of some tokens at a time (4 GB), with those tokens."""
    c = s["case"]
    token, real, lo, hi = queries
    B, S, H, D = k.shape
    t = torch.arange(S, device="cuda")
    for at in torch.arange(token.shape[1], device="cuda").split(max(1, (1 << 30) // (B * S * c["heads"]))):
        q = (s["q"][token[:, at]].float() * s["q_scale"]).view(B, len(at), H, -1, D).permute(0, 2, 3, 1, 4)
        x = torch.matmul(q.reshape(B, H, -1, D), k.permute(0, 2, 3, 1)).mul_(s["scale"]).view(B, H, -1, len(at), S)
        if c["cap"]:
            x = x.div_(c["cap"]).tanh_().mul_(c["cap"])
        seen = (t >= lo[:, at, None]) & (t < hi[:, at, None]) & real[:, at, None]
        yield x.masked_fill_(~seen[:, None, None], -math.inf), token[:, at], real[:, at]


def _packed(s):
    c = s["case"]
    if own:
        import paged_kv_decode_15_gb300 as pkd
        return dict(zip(("out", "lse"), pkd.packed_attention(
            s["q"], s["k"], s["v"], s["starts"], s["scale"], key_start=s["key_starts"], causal=c["causal"],
            window=c["window"], softcap=c["cap"], max_query_len=s["most"], max_kv_len=s["longest"])))
    s = {**s, "q_scale": 1.0}
    starts = s["starts"] if s["key_starts"] is None else s["key_starts"]
    row = (starts[:-1, None].long() + torch.arange(s["longest"], device="cuda")).clamp(max=s["k"].shape[0] - 1)
    v = s["v"][row].float().transpose(1, 2)
    out = torch.empty(s["q"].shape, device="cuda", dtype=s["q"].dtype)
    lse = torch.empty(s["q"].shape[:2], device="cuda")
    for x, token, real in _scores(s, _queries(s, 0), s["k"][row].float()):
        B, H, G, n, S = x.shape
        top = x.amax(-1, keepdim=True)
        x = x.sub_(top.masked_fill(top == -math.inf, 0.0)).exp_()
        total = x.sum(-1, keepdim=True)
        o = torch.matmul(x.view(B, H, G * n, S), v).view(B, H, G, n, -1) / total.masked_fill(total == 0, 1.0)
        out[token[real]] = o.permute(0, 3, 1, 2, 4).flatten(2, 3)[real].to(out.dtype)
        lse[token[real]] = (top + total.log())[..., 0].permute(0, 3, 1, 2).flatten(2, 3)[real]
    return {"out": out, "lse": lse}


def _weigh(s):
    c = s["case"]
    if own:
        import paged_kv_decode_15_gb300 as pkd
        return pkd.key_weights(s["q"], s["cache"], s["table"], s["lens"], s["starts"], s["lse"], s["scale"],
                               weights=s["prior"], decay=c["decay"], window=c["window"], softcap=c["cap"],
                               last_queries=c["last"], max_query_len=s["most"], max_kv_len=s["longest"],
                               q_scale=s["q_scale"], k_scale=s["k_scale"], out=s["out"])
    B, H, L = c["requests"], c["kv_heads"], s["longest"]
    t = torch.arange(L, device="cuda")
    got = torch.zeros((B, H, L), device="cuda")
    for x, token, _ in _scores(s, _queries(s, c["last"]), _gathered(s)):
        lse = s["lse"][token].view(B, -1, H, x.shape[2]).permute(0, 2, 3, 1)[..., None]
        got += x.sub_(lse.masked_fill(lse == -math.inf, math.inf)).exp_().sum((2, 3))
    if s["prior"] is not None:
        new = s["starts"][1:] - s["starts"][:-1]
        got += torch.where(t < (s["lens"] - new)[:, None, None], s["prior"][..., :L] * c["decay"], 0.0)
    s["out"][..., :L] = torch.where(t < s["lens"][:, None, None], got, s["out"][..., :L])
    return s["out"]


def _select(s):
    c = s["case"]
    if own:
        import paged_kv_decode_15_gb300 as pkd
        return dict(zip(("kept", "kept_lens"), pkd.evict_select(
            s["weights"], s["lens"], c["budget"], sinks=c["sinks"], recent=c["recent"], pool=c["pool"],
            positions=s.get("positions"), context_lens=s.get("context"))))
    B, H, S = s["weights"].shape
    L = s["lens"].long()[:, None, None]
    t = torch.arange(S, device="cuda").expand(B, H, S)
    pos, context = (s["positions"].long(), s["context"].long()[:, None, None]) if c["moved"] else (t, L)
    always = (pos < c["sinks"]) | (pos >= context - c["recent"])
    x = s["weights"].masked_fill(always | (t >= L), -math.inf)
    side = c["pool"] // 2
    x = torch.nn.functional.pad(x, (side, side), value=-math.inf).unfold(-1, c["pool"], 1).amax(-1)
    x = x.masked_fill(always, math.inf).masked_fill(t >= L, -math.inf)
    n = L.clamp(max=c["budget"])
    first = min(S, c["budget"])
    kept = x.sort(dim=-1, descending=True, stable=True)[1][..., :first]
    kept = kept.masked_fill(torch.arange(first, device="cuda") >= n, S).sort(-1)[0]
    kept = torch.nn.functional.pad(kept, (0, c["budget"] - first), value=S)
    return {"kept": kept.masked_fill(kept == S, -1).int(), "kept_lens": n[:, 0, 0].int()}


def _compact(s):
    c = s["case"]
    if own:
        import paged_kv_decode_15_gb300 as pkd
        pkd.cache_compact(s["cache"], s["table"], s["kept"], s["kept_lens"], weights=s["weights"],
                          positions=s.get("positions"))
        return {k: s[k] for k in ("cache", "weights", "positions") if k in s}
    n = s["kept_lens"].long()[:, None, None]
    i = torch.arange(c["budget"], device="cuda")
    kept = s["kept"].long().masked_fill(i >= n, -1)
    # of each request and kv head as many slots are free below n as kept rows lie behind them
    taken = torch.zeros((*kept.shape[:2], c["budget"] + 1), device="cuda", dtype=torch.bool)
    taken.scatter_(2, kept.masked_fill((kept >= n) | (kept < 0), c["budget"]), True)
    b, h, to = torch.nonzero(~taken[..., :-1] & (i < n), as_tuple=True)
    source = kept[kept >= n]
    P, cache = c["page"], _bits(s["cache"])
    page, origin = s["table"][b, to // P].long(), s["table"][b, source // P].long()
    cache[page, h, to % P] = cache[origin, h, source % P]
    s["weights"][b, h, to] = s["weights"][b, h, source]
    if c["moved"]:
        s["positions"][b, h, to] = s["positions"][b, h, source]
    return {k: s[k] for k in ("cache", "weights", "positions") if k in s}


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    c = case
    if work(c)["flops"] > 3e12:
        return None
    s = prepare(c, seed)
    H, B = c["kv_heads"], c["requests"]
    new, keys = _lengths(c)
    if c["op"] == "select":
        weights = s["weights"].double().cpu().numpy()
        kept = np.full((B, H, c["budget"]), -1, np.int32)
        for b, L in enumerate(keys):
            for h in range(H):
                at = np.arange(L)
                pos = s["positions"][b, h, :L].cpu().numpy() if c["moved"] else at
                context = int(s["context"][b]) if c["moved"] else L
                free = at[(pos >= c["sinks"]) & (pos < context - c["recent"])]
                value = np.full(L, np.inf)
                value[free] = -np.inf
                for d in range(-(c["pool"] // 2), c["pool"] // 2 + 1):
                    near = free[np.isin(free + d, free)]
                    value[near] = np.maximum(value[near], weights[b, h, near + d])
                best = np.lexsort((at, -value))[:c["budget"]]
                kept[b, h, :len(best)] = np.sort(best)
        return {"kept": kept, "kept_lens": np.minimum(keys, c["budget"]).astype(np.int32)}
    if c["op"] == "compact":
        P, parts = c["page"], {k: s[k].clone() for k in ("weights", "positions") if k in s}
        cache = s["cache"].double()
        for b in range(B):
            n, table = int(s["kept_lens"][b]), s["table"][b].cpu().numpy()
            for h in range(H):
                mine = s["kept"][b, h, :n].cpu().numpy()
                source, to = mine[mine >= n], np.setdiff1d(np.arange(n), mine)
                cache[table[to // P], h, to % P] = cache[table[source // P], h, source % P]
                for x in parts.values():
                    x[b, h, to] = x[b, h, source]
        return {"cache": cache, **{k: x.double() if k == "weights" else x for k, x in parts.items()}}

    G, D = c["heads"] // H, c["dim"]

    def probabilities(q, k, b, at, lse=None):
        """[heads, tokens, keys] of the tokens `at` of request b, and the logarithms of their sums."""
        x = torch.einsum("nhd,shd->hns", q.double() * s["q_scale"], k.repeat_interleave(G, 1)) * s["scale"]
        if c["cap"]:
            x = c["cap"] * torch.tanh(x / c["cap"])
        pos, t = (keys[b] - new[b] + at)[:, None], torch.arange(keys[b], device="cuda")
        seen = torch.ones((len(at), keys[b]), dtype=torch.bool, device="cuda")
        if c.get("causal", True):
            seen &= t <= pos
        if c["window"]:
            seen &= t > pos - c["window"]
        x = torch.where(seen, x, -math.inf)
        lse = torch.logsumexp(x, -1) if lse is None else lse.double().t()
        return torch.exp(x - torch.where(lse == -math.inf, math.inf, lse)[..., None]), lse.t()

    outs, lses, weights = [], [], None if c["op"] == "packed" else s["out"].double()
    q0 = k0 = 0
    for b, (n, L) in enumerate(zip(new, keys)):
        tokens = torch.arange(n, device="cuda")
        if c["op"] == "packed":
            k, v = s["k"][k0:k0 + L].double(), s["v"][k0:k0 + L].double()
        else:
            pages = s["table"][b, :-(-L // c["page"])].long()
            rows = _bits(s["cache"])[pages].view(s["cache"].dtype)[..., :D].double() * s["k_scale"]
            k = rows.transpose(1, 2).reshape(-1, H, D)[:L]
            tokens = tokens[n - _weighers(c, n):]
            total = torch.zeros((H, L), device="cuda", dtype=torch.float64)
        for at in tokens.split(max(1, (1 << 28) // (L * c["heads"]))):
            if c["op"] == "packed":
                p, lse = probabilities(s["q"][q0 + at], k, b, at)
                outs.append(torch.einsum("hns,shd->nhd", p, v.repeat_interleave(G, 1)))
                lses.append(lse)
            else:
                p, _ = probabilities(s["q"][q0 + at], k, b, at, s["lse"][q0 + at])
                total += p.view(H, -1, L).sum(1)
        if c["op"] == "weigh":
            if c["prior"]:
                total[:, :L - n] += c["decay"] * s["prior"][b, :, :L - n].double()
            weights[b, :, :L] = total
        q0, k0 = q0 + n, k0 + L
    return weights if c["op"] == "weigh" else {"out": torch.cat(outs), "lse": torch.cat(lses)}
