"""What is measured of the serving operators around the paged KV cache.

Three operators, each in the forms a server calls it in:

  rope    the rotary step of a layer: queries rotated, keys rotated and appended
          to the paged cache with their values
  attend  attention of ragged query tokens over the paged cache, with capped
          scores, a distance bias, window, prefix and document masks; "step"
          cases are single tokens (or a few), "prompt" cases whole prompts
  shared  a decode step of requests that share the pages of a long prefix

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
        # one layer of a 64-request decode step: what counts is the latency of a small launch
        dict(name="rope_step_b64", op="rope", tokens=64, heads=32, kv_heads=8, dim=128, rotary=128, page=16,
             dtype="bf16", cache="bf16", q8=False, interleaved=False),
        # prompts of 32768 tokens into an fp8 cache, queries quantised for it
        dict(name="rope_prompt_fp8", op="rope", tokens=32768, heads=32, kv_heads=8, dim=128, rotary=128, page=16,
             dtype="bf16", cache="fp8", q8=True, interleaved=False),
        # an odd number of tokens, seven heads to a kv head, half of each head rotated, pairs side by side
        dict(name="rope_odd_fp16", op="rope", tokens=4099, heads=28, kv_heads=4, dim=128, rotary=64, page=32,
             dtype="fp16", cache="fp16", q8=False, interleaved=True),
        # a decode step of 64 requests whose model caps its scores
        dict(name="step_cap_b64", op="attend", requests=64, new=1, keys=4096, lens=1, heads=32, kv_heads=8, dim=128,
             page=16, dtype="bf16", cap=50.0, bias=False, window=0, prefix=0, docs=0),
        # long contexts in an fp8 cache with a distance bias
        dict(name="step_bias_fp8_long", op="attend", requests=4, new=1, keys=131072, lens=2, heads=64, kv_heads=8,
             dim=128, page=64, dtype="fp8", cap=0.0, bias=True, window=0, prefix=0, docs=0),
        # one user with a short context: latency
        dict(name="step_cap_b1", op="attend", requests=1, new=1, keys=611, lens=3, heads=32, kv_heads=8, dim=128,
             page=16, dtype="bf16", cap=30.0, bias=False, window=0, prefix=0, docs=0),
        # a batch of ragged prompts, capped scores, a sliding window
        dict(name="prompt_cap_window_b8", op="attend", requests=8, new=2500, keys=2500, lens=4, heads=32, kv_heads=8,
             dim=128, page=16, dtype="bf16", cap=50.0, bias=False, window=1024, prefix=0, docs=0),
        # one long document, its first 1024 tokens seen by all (a prefix mask)
        dict(name="prompt_32k", op="attend", requests=1, new=32768, keys=32768, lens=5, heads=32, kv_heads=8, dim=128,
             page=16, dtype="bf16", cap=0.0, bias=False, window=0, prefix=1024, docs=0),
        # the last chunk of packed documents, smaller heads
        dict(name="chunk_docs_fp16", op="attend", requests=2, new=4096, keys=14000, lens=6, heads=16, kv_heads=16,
             dim=64, page=64, dtype="fp16", cap=0.0, bias=False, window=0, prefix=0, docs=9),
        # 64 requests after one common prompt of 16384 tokens
        dict(name="shared_b64_16k", op="shared", groups=1, requests=64, new=1, shared=16384, keys=1024, lens=7,
             heads=32, kv_heads=8, dim=128, page=16, dtype="bf16", cap=0.0, causal=False),
        # three tenants with prompts of their own, fp8 cache
        dict(name="shared_groups_fp8", op="shared", groups=3, requests=100, new=1, shared=8192, keys=700, lens=8,
             heads=64, kv_heads=8, dim=128, page=64, dtype="fp8", cap=0.0, causal=False),
        # a few requests verifying drafts of four tokens after a short prompt
        dict(name="shared_drafts_b5", op="shared", groups=1, requests=5, new=4, shared=1000, keys=77, lens=9, heads=8,
             kv_heads=2, dim=64, page=16, dtype="fp16", cap=30.0, causal=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    dim = rng.choice([64, 128, 128])
    kv = rng.choice([1, 2, 4, 8, 8])
    op = rng.choice(["rope", "step", "prompt", "shared"])
    page = rng.choice([16, 32, 48, 64])
    if op == "rope":
        dtype = rng.choice(["bf16", "fp16"])
        cache = rng.choice([dtype, "fp8"])
        return dict(op="rope", tokens=_log(rng, 1, 32768), heads=kv * rng.choice([1, 2, 3, 4]), kv_heads=kv, dim=dim,
                    rotary=rng.choice([32, dim, dim]), page=page, dtype=dtype, cache=cache,
                    q8=cache == "fp8" and rng.random() < 0.7, interleaved=rng.random() < 0.5)
    dtype = rng.choice(["bf16", "fp16"] if dim == 64 else ["bf16", "bf16", "fp16", "fp8"])
    cap = rng.choice([0.0, 30.0, 50.0])
    lens = rng.randrange(1 << 30)
    group = rng.choice([1, 2, 4, 7, 8])
    if op == "step":
        requests = _log(rng, 1, 128)
        return dict(op="attend", requests=requests, new=rng.choice([1, 1, 2]), lens=lens,
                    keys=_log(rng, 2, min(32768, 262144 // requests)), heads=kv * group, kv_heads=kv, dim=dim,
                    page=page, dtype=dtype, cap=cap, bias=rng.random() < 0.4, window=rng.choice([0, 0, 500]), prefix=0,
                    docs=0)
    if op == "prompt":
        new = _log(rng, 20, 8192)
        return dict(op="attend", requests=rng.randint(1, max(1, min(12, 16384 // new))), new=new, lens=lens,
                    keys=new + rng.choice([0, 0, _log(rng, 1, 8192)]), heads=kv * group, kv_heads=kv, dim=dim,
                    page=page, dtype=dtype, cap=cap, bias=rng.random() < 0.3,
                    window=rng.choice([0, 0, _log(rng, 16, 4096)]), prefix=rng.choice([0, 0, _log(rng, 1, new)]),
                    docs=rng.choice([0, 0, 5]))
    requests = _log(rng, 1, 200)
    return dict(op="shared", groups=rng.randint(1, min(4, requests)), requests=requests, new=rng.choice([1, 1, 2]),
                shared=_log(rng, 16, 16384), keys=_log(rng, 1, 1024), lens=lens, heads=kv * group, kv_heads=kv,
                dim=dim, page=page, dtype=dtype, cap=cap, causal=rng.random() < 0.5)


def _lengths(c):
    """Per request: the new tokens, and all its keys with them (its own keys where a prefix is shared)."""
    r = random.Random(c["lens"])
    new, keys = [], []
    for b in range(c["requests"]):
        if c["op"] == "shared" or c["new"] <= 2:
            n = c["new"]  # steps: every request brings as many
        else:
            n = c["new"] if c["requests"] == 1 else r.randint(max(1, c["new"] // 4), c["new"])
        most = c["keys"] - c["new"]
        past = most if c["requests"] == 1 else r.randint(most // 8, most) if most > 0 else 0
        new.append(n)
        keys.append(n + max(0, past))
    return new, keys


def _prefixes(c):
    """Of the shared prefixes: the first request of each group (and the number of all), and their lengths."""
    r = random.Random(c["lens"] + 1)
    cuts = sorted(r.sample(range(1, c["requests"]), c["groups"] - 1))
    return [0] + cuts + [c["requests"]], [c["shared"] - (r.randint(0, c["shared"] // 2) if g else 0)
                                          for g in range(c["groups"])]


def _ranges(c):
    """Per query token of an attend case: its request, its position, and the keys [lo, hi) that it sees."""
    new, keys = _lengths(c)
    r = random.Random(c["lens"] + 2)
    req, pos, lo, hi, doc = [], [], [], [], []
    for b, (n, L) in enumerate(zip(new, keys)):
        p = np.arange(L - n, L)
        starts = np.array(sorted([0] + [r.randrange(L) for _ in range(c["docs"])]))
        d = starts[np.searchsorted(starts, p, side="right") - 1]
        req.append(np.full(n, b))
        pos.append(p)
        doc.append(d)
        lo.append(np.maximum(d, p - (c["window"] - 1) if c["window"] else 0))
        hi.append(np.minimum(np.maximum(p + 1, c["prefix"]), L))
    return [np.concatenate(x) for x in (req, pos, lo, hi, doc)]


def work(case):
    c = case
    D, Hq, Hkv = c["dim"], c["heads"], c["kv_heads"]
    if c["op"] == "rope":
        read = c["tokens"] * ((Hq + 2 * Hkv) * D * 2 + c["rotary"] * 4 + 16)
        wrote = c["tokens"] * D * (Hq * (1 if c["q8"] else 2) + 2 * Hkv * _SIZES[c["cache"]])
        return {"bytes": read + wrote, "flops": 3 * c["tokens"] * (Hq + Hkv) * c["rotary"]}
    elt = _SIZES[c["dtype"]]
    if c["op"] == "attend":
        req, _, lo, hi, _ = _ranges(c)
        tokens, pairs, cached = len(req), int(np.maximum(hi - lo, 0).sum()), 0
        for b in range(c["requests"]):
            mine = (req == b) & (hi > lo)
            cached += int(hi[mine].max() - lo[mine].min()) if mine.any() else 0
    else:
        _, keys = _lengths(c)
        first, plens = _prefixes(c)
        tokens = c["requests"] * c["new"]
        cached = sum(keys) + sum(plens)
        pairs = sum(keys) * c["new"] + sum(p * (b - a) * c["new"] for a, b, p in zip(first, first[1:], plens))
        if c["causal"]:
            pairs -= c["requests"] * c["new"] * (c["new"] - 1) // 2
    return {"bytes": tokens * Hq * D * (elt + 2) + tokens * Hq * 4 + cached * Hkv * 2 * D * elt,
            "flops": 4 * D * Hq * pairs}


# ------------------------------------------------------------------ the inputs
def _quantise(x):
    """Values in e4m3 with the scale that takes the largest to 448."""
    scale = float(x.abs().amax().float()) / 448.0
    return (x.float() / scale).clamp(-448.0, 448.0).to(torch.float8_e4m3fn), scale


def _cache(gen, pages, c, dtype):
    """A pool of pages [pages, kv heads, page, K | V] of normal values; (pool, k scale, v scale)."""
    D = c["dim"]
    pool = torch.randn((pages, c["kv_heads"], c["page"], 2 * D), device="cuda", generator=gen, dtype=torch.float16)
    if dtype != "fp8":
        return pool.to(_TYPES[dtype]), 1.0, 1.0
    k, ks = _quantise(pool[..., :D])
    v, vs = _quantise(pool[..., D:])
    return torch.cat([k.view(torch.uint8), v.view(torch.uint8)], -1).view(torch.float8_e4m3fn), ks, vs


def _tables(gen, lens, page, spare):
    """Block tables of requests with these lengths, their pages scattered over a pool, and the pool's pages."""
    counts = [-(-n // page) for n in lens]
    pages = sum(counts) + spare
    order = torch.randperm(pages, device="cuda", generator=gen).to(torch.int32)
    width, rows, at = max(max(counts), 1), [], 0
    for n in counts:
        rows.append(torch.nn.functional.pad(order[at:at + n], (0, width - n)))
        at += n
    return torch.stack(rows).contiguous(), pages


def _queries(gen, shape, dtype):
    x = 3.0 * torch.randn(shape, device="cuda", generator=gen, dtype=torch.float32)  # scores with a spread of 3
    if dtype == "fp8":
        return _quantise(x)
    return x.to(_TYPES[dtype]), 1.0


def _ints(x, dtype=torch.int32):
    return torch.as_tensor(np.asarray(x), dtype=dtype, device="cuda")


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    D, Hq, Hkv = c["dim"], c["heads"], c["kv_heads"]
    s = {"case": c, "scale": D ** -0.5}
    if c["op"] == "rope":
        T, P, rd = c["tokens"], c["page"], c["rotary"]
        # the fused projection of a layer, its parts strided views of one tensor
        qkv = torch.randn((T, Hq + 2 * Hkv, D), device="cuda", generator=gen, dtype=torch.float32).to(_TYPES[c["dtype"]])
        pages = -(-T // P) + 4
        far = 40960
        angle = torch.arange(far, device="cuda", dtype=torch.float64)[:, None] * \
            10000.0 ** (-torch.arange(0, rd, 2, device="cuda", dtype=torch.float64) / rd)
        s |= {"q": qkv[:, :Hq], "k": qkv[:, Hq:Hq + Hkv], "v": qkv[:, Hq + Hkv:],
              "positions": torch.randint(0, far, (T,), device="cuda", generator=gen, dtype=torch.int64),
              "table": torch.cat([angle.cos(), angle.sin()], -1).float(),
              "slots": torch.randperm(pages * P, device="cuda", generator=gen)[:T].contiguous()}
        s["cache"] = torch.zeros((pages, Hkv, P, 2 * D), device="cuda", dtype=_TYPES[c["cache"]])
        s["k_scale"], s["v_scale"] = (5.5 / 448, 4.5 / 448) if c["cache"] == "fp8" else (1.0, 1.0)
        s["q_scale"] = 6.0 / 448 if c["q8"] else 1.0
        s["q_type"] = torch.float8_e4m3fn if c["q8"] else _TYPES[c["dtype"]]
        return s
    new, keys = _lengths(c)
    if c["op"] == "attend":
        req, pos, lo, hi, doc = _ranges(c)
        s["table"], pages = _tables(gen, keys, c["page"], 3)
        s["q"], s["q_scale"] = _queries(gen, (len(req), Hq, D), c["dtype"])
        s["starts"] = _ints(np.concatenate([[0], np.cumsum(new)]))
        s["docs"] = _ints(doc) if c["docs"] else None
        s["prefix"] = _ints(np.full(c["requests"], c["prefix"])) if c["prefix"] else None
        slopes = 2.0 ** (-8.0 * (torch.arange(Hq, device="cuda", dtype=torch.float32) + 1) / Hq)
        s["slopes"] = slopes if c["bias"] else None
        s["max_new"] = max(new)
    else:
        first, plens = _prefixes(c)
        both, pages = _tables(gen, plens + keys, c["page"], 3)
        wide = -(-max(plens) // c["page"])
        s["prefix_table"] = both[:c["groups"], :wide].contiguous()
        s["table"] = both[c["groups"]:, :max(1, -(-max(keys) // c["page"]))].contiguous()
        s["prefix_lens"], s["group_start"] = _ints(plens), _ints(first)
        s["q"], s["q_scale"] = _queries(gen, (c["requests"], c["new"], Hq, D), c["dtype"])
    s["lens"], s["longest"] = _ints(keys), max(keys)
    s["cache"], s["k_scale"], s["v_scale"] = _cache(gen, pages, c, c["dtype"])
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    return {"rope": _rope, "attend": _attend, "shared": _shared}[state["case"]["op"]](state)


def _rope(s):
    if own:
        import paged_kv_decode_15_gb300 as pkd
        q = pkd.rope_cache_write(s["q"], s["k"], s["v"], s["positions"], s["table"], s["slots"], s["cache"],
                                 interleaved=s["case"]["interleaved"], q_out_dtype=s["q_type"], q_scale=s["q_scale"],
                                 k_scale=s["k_scale"], v_scale=s["v_scale"])
        return {"q": q, "cache": s["cache"]}
    c, D, P = s["case"], s["case"]["dim"], s["case"]["page"]
    half = c["rotary"] // 2
    cs = s["table"][s["positions"]][:, None]
    cos, sin = cs[..., :half], cs[..., half:]

    def turned(x):
        x = x.float()
        r, rest = x[..., :c["rotary"]], x[..., c["rotary"]:]
        a, b = (r[..., 0::2], r[..., 1::2]) if c["interleaved"] else (r[..., :half], r[..., half:])
        p, q = a * cos - b * sin, b * cos + a * sin
        r = torch.stack([p, q], -1).flatten(-2) if c["interleaved"] else torch.cat([p, q], -1)
        return torch.cat([r, rest], -1)

    def stored(x, scale, dtype):
        return (x / scale).clamp(-448.0, 448.0).to(dtype) if dtype == torch.float8_e4m3fn else x.to(dtype)

    dtype = s["cache"].dtype
    bits = torch.uint8 if dtype == torch.float8_e4m3fn else torch.int16
    kv = torch.cat([stored(turned(s["k"]), s["k_scale"], dtype).view(bits),
                    stored(s["v"].float(), s["v_scale"], dtype).view(bits)], -1)
    page, at = s["slots"] // P, s["slots"] % P
    s["cache"].view(bits)[page, :, at] = kv
    return {"q": stored(turned(s["q"]), s["q_scale"], s["q_type"]), "cache": s["cache"]}


def _softmax_values(q, k, v, lo, hi, pos, scale, cap, slopes):
    """out, lse of q [N, n, H, D] over k, v [N, S, Hkv, D]; the token (N, n) sees keys [lo, hi)."""
    N, n, H, D = q.shape
    S, Hkv = k.shape[1], k.shape[2]
    t = torch.arange(S, device=q.device)
    seen = ((t >= lo[..., None]) & (t < hi[..., None]))[:, None, None]  # [N, 1, 1, n, S]
    x = q.view(N, n, Hkv, H // Hkv, D).permute(0, 2, 3, 1, 4)
    x = torch.matmul(x.reshape(N, Hkv, -1, D), k.permute(0, 2, 3, 1)).view(N, Hkv, H // Hkv, n, S).mul_(scale)
    if cap:
        x = x.div_(cap).tanh_().mul_(cap)
    if slopes is not None:
        x = x - slopes.view(Hkv, -1, 1, 1) * (pos[..., None] - t).abs()[:, None, None].float()
    x = x.masked_fill_(~seen, -math.inf)
    top = x.amax(-1, keepdim=True)
    x = x.sub_(top.masked_fill(top == -math.inf, 0.0)).exp_()
    total = x.sum(-1, keepdim=True)
    out = torch.matmul(x.view(N, Hkv, -1, S), v.transpose(1, 2)).view(N, Hkv, H // Hkv, n, D)
    out = out / total.masked_fill(total == 0, 1.0)
    return out.permute(0, 3, 1, 2, 4).reshape(N, n, H, D), (top + total.log())[..., 0].permute(0, 3, 1, 2).reshape(N, n, H)


def _gathered(s, table, longest):
    """The keys and values of each row of a block table in 32 bits: [rows, longest, kv heads, D]."""
    D, P = s["case"]["dim"], s["case"]["page"]
    t = torch.arange(longest, device="cuda")
    bits = s["cache"].view(torch.uint8) if s["cache"].dtype == torch.float8_e4m3fn else s["cache"]
    rows = bits[table[:, t // P].long(), :, t % P]
    rows = rows.view(s["cache"].dtype).float()
    return rows[..., :D] * s["k_scale"], rows[..., D:] * s["v_scale"]


def _in_blocks(q, k, v, lo, hi, pos, scale, cap, slopes):
    """_softmax_values in blocks of requests, kv heads and query tokens that keep the scores under 4 GB."""
    N, n, H, D = q.shape
    S, Hkv = k.shape[1], k.shape[2]
    out, lse = torch.empty_like(q), torch.empty((N, n, H), device=q.device)
    most = 1 << 30
    heads = max(1, min(Hkv, most // max(1, n * S * (H // Hkv))))
    rows = max(1, min(n, most // max(1, S * (H // Hkv) * heads)))
    reqs = max(1, min(N, most // max(1, n * S * H)))
    G = H // Hkv
    for a in range(0, N, reqs):
        for h in range(0, Hkv, heads):
            for i in range(0, n, rows):
                at = (slice(a, a + reqs), slice(i, i + rows), slice(h * G, (h + heads) * G))
                kv = (slice(a, a + reqs), slice(None), slice(h, h + heads))
                out[at], lse[at] = _softmax_values(
                    q[at], k[kv], v[kv], lo[at[:2]], hi[at[:2]], pos[at[:2]], scale, cap,
                    None if slopes is None else slopes[at[2]])
    return out, lse


def _attend(s):
    c = s["case"]
    if own:
        import paged_kv_decode_15_gb300 as pkd
        return dict(zip(("out", "lse"), pkd.paged_attention(
            s["q"], s["cache"], s["table"], s["lens"], s["starts"], s["scale"], causal=True, window=c["window"],
            softcap=c["cap"], alibi_slopes=s["slopes"], prefix_lens=s["prefix"], doc_start=s["docs"],
            max_query_len=s["max_new"], q_scale=s["q_scale"], k_scale=s["k_scale"], v_scale=s["v_scale"])))
    T, Hq, D = s["q"].shape
    starts, lens, n = s["starts"].long(), s["lens"].long(), s["max_new"]
    new = starts[1:] - starts[:-1]
    i = torch.arange(n, device="cuda")
    real = i < new[:, None]                                  # [B, n]: the requests' tokens, padded
    token = (starts[:-1, None] + i).clamp(max=T - 1)
    pos = lens[:, None] - new[:, None] + i
    lo = torch.zeros_like(pos) if s["docs"] is None else s["docs"].long()[token]
    if c["window"]:
        lo = torch.maximum(lo, pos - (c["window"] - 1))
    hi = pos + 1 if s["prefix"] is None else torch.maximum(pos + 1, s["prefix"].long()[:, None])
    hi = torch.minimum(hi, lens[:, None])
    k, v = _gathered(s, s["table"], s["longest"])
    out, lse = _in_blocks(s["q"].float()[token] * s["q_scale"], k, v, lo, hi, pos, s["scale"], c["cap"], s["slopes"])
    kind = torch.bfloat16 if c["dtype"] == "fp8" else s["q"].dtype
    return {"out": out[real].to(kind), "lse": lse[real]}


def _shared(s):
    c = s["case"]
    if own:
        import paged_kv_decode_15_gb300 as pkd
        return dict(zip(("out", "lse"), pkd.prefix_decode(
            s["q"], s["cache"], s["prefix_table"], s["prefix_lens"], s["table"], s["lens"], s["scale"],
            group_start=s["group_start"], causal=c["causal"], softcap=c["cap"], q_scale=s["q_scale"],
            k_scale=s["k_scale"], v_scale=s["v_scale"])))
    B, sq, Hq, D = s["q"].shape
    q = s["q"].float() * s["q_scale"]
    i = torch.arange(sq, device="cuda")
    # the prefix, once a group: the rows of all its requests against its keys
    member = torch.arange(B, device="cuda")
    group = torch.searchsorted(s["group_start"][1:].long(), member, right=True)
    rank = member - s["group_start"].long()[group]
    most = B if c["groups"] == 1 else int(max(b - a for a, b in zip(_prefixes(c)[0], _prefixes(c)[0][1:])))
    padded = torch.zeros((c["groups"], most, sq, Hq, D), device="cuda")
    padded[group, rank] = q
    k, v = _gathered(s, s["prefix_table"], c["shared"])
    hi = s["prefix_lens"].long()[:, None].expand(-1, most * sq)
    zero = torch.zeros_like(hi)
    o1, l1 = _in_blocks(padded.view(c["groups"], most * sq, Hq, D), k, v, zero, hi, zero, s["scale"], c["cap"], None)
    o1 = o1.view(c["groups"], most, sq, Hq, D)[group, rank]
    l1 = l1.view(c["groups"], most, sq, Hq)[group, rank]
    # each request's own keys, and the join of the two
    L = s["lens"].long()[:, None]
    pos = L - sq + i
    hi = pos + 1 if c["causal"] else L.expand(-1, sq)
    k, v = _gathered(s, s["table"], s["longest"])
    o2, l2 = _in_blocks(q, k, v, torch.zeros_like(pos), hi, pos, s["scale"], c["cap"], None)
    lse = torch.logaddexp(l1, l2)
    out = o1 * (l1 - lse).exp()[..., None] + o2 * (l2 - lse).exp()[..., None]
    return {"out": out.to(torch.bfloat16 if c["dtype"] == "fp8" else s["q"].dtype), "lse": lse}


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    c = case
    if work(c)["flops"] > 1.5e12:
        return None
    s = prepare(c, seed)
    D = c["dim"]
    if c["op"] == "rope":
        rd = c["rotary"]
        first = torch.arange(0, rd, 2) if c["interleaved"] else torch.arange(rd // 2)
        second = first + (1 if c["interleaved"] else rd // 2)
        # as one complex product per pair, by the table's own 32-bit entries
        turn = torch.complex(s["table"][:, :rd // 2].double(), s["table"][:, rd // 2:].double())[s["positions"]][:, None]

        def rotate(x):
            y = x.double().clone()
            z = torch.complex(y[..., first], y[..., second]) * turn
            y[..., first], y[..., second] = z.real, z.imag
            return y

        cache = s["cache"].double()
        rows = torch.cat([rotate(s["k"]) / s["k_scale"], s["v"].double() / s["v_scale"]], -1)
        if c["cache"] == "fp8":
            rows = rows.clamp(-448, 448)
        flat = cache.transpose(1, 2).reshape(-1, c["kv_heads"], 2 * D)
        flat[s["slots"]] = rows
        q = rotate(s["q"]) / s["q_scale"]
        cache = flat.view(cache.shape[0], c["page"], c["kv_heads"], 2 * D).transpose(1, 2).contiguous()
        return {"q": q.clamp(-448, 448) if c["q8"] else q, "cache": cache}

    G, P = c["heads"] // c["kv_heads"], c["page"]
    new, keys = _lengths(c)

    def rows_of(table, length):
        """K and V [kv heads, length, D] of one request, page by page."""
        pages = table[:-(-length // P)].long()
        kv = s["cache"].view(torch.uint8)[pages].view(s["cache"].dtype).double() if c["dtype"] == "fp8" else s["cache"][pages].double()
        kv = kv.transpose(0, 1).reshape(c["kv_heads"], -1, 2 * D)[:, :length]
        return kv[..., :D] * s["k_scale"], kv[..., D:] * s["v_scale"]

    def attention(q, k, v, seen, bias):
        """q [n, Hq, D], seen [n, S], bias [Hq, n, S] or None."""
        k, v = k.repeat_interleave(G, 0), v.repeat_interleave(G, 0)
        x = torch.einsum("nhd,hsd->hns", q.double() * s["q_scale"], k) * s["scale"]
        if c["cap"]:
            x = c["cap"] * torch.tanh(x / c["cap"])
        if bias is not None:
            x = x + bias
        x = torch.where(seen, x, -math.inf)
        lse = torch.logsumexp(x, -1)
        p = torch.exp(x - torch.where(lse == -math.inf, 0.0, lse)[..., None])
        return torch.einsum("hns,hsd->nhd", p, v), lse.t()

    outs, lses = [], []
    if c["op"] == "attend":
        req, pos, lo, hi, _ = (torch.as_tensor(x, device="cuda") for x in _ranges(c))
        for b in range(c["requests"]):
            k, v = rows_of(s["table"][b], keys[b])
            t = torch.arange(keys[b], device="cuda")
            mine = torch.nonzero(req == b)[:, 0]
            for at in mine.split(max(1, (1 << 28) // (keys[b] * c["heads"]))):
                seen = (t >= lo[at, None]) & (t < hi[at, None])
                bias = None
                if s["slopes"] is not None:
                    bias = -s["slopes"].double()[:, None, None] * (pos[at, None] - t).abs()
                o, l = attention(s["q"][at], k, v, seen, bias)
                outs.append(o)
                lses.append(l)
        return {"out": torch.cat(outs), "lse": torch.cat(lses)}
    first, plens = _prefixes(c)
    for g in range(c["groups"]):
        pk, pv = rows_of(s["prefix_table"][g], plens[g])
        for b in range(first[g], first[g + 1]):
            k, v = rows_of(s["table"][b], keys[b])
            t = torch.arange(plens[g] + keys[b], device="cuda") - plens[g]
            last = keys[b] - c["new"] + torch.arange(c["new"], device="cuda") if c["causal"] else \
                torch.full((c["new"],), keys[b], device="cuda")
            o, l = attention(s["q"][b], torch.cat([pk, k], 1), torch.cat([pv, v], 1), t <= last[:, None], None)
            outs.append(o)
            lses.append(l)
    return {"out": torch.stack(outs), "lse": torch.stack(lses)}
