"""The operators that bound a paged cache, against a plain 64-bit reference: weights that
keys receive, choice of the keys that stay, compaction, and a run of them together."""
import numpy as np
import pytest
import torch

import paged_kv_decode_15_gb300 as pkd
from tests import eviction_ref as ref
from tests import ragged_ref

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp8": torch.float8_e4m3fn}


def dev(x):
    return torch.as_tensor(np.ascontiguousarray(x)).cuda()


def stored(x, dtype):
    """A CPU tensor of fp32 values rounded to the type, and those values in fp64."""
    t = x.to(TYPES[dtype])
    return t, t.float().double().numpy()


def problem(seed, *, new, lens, heads, kv, dim, page, dtype, spread=1.5, spare=2, columns=None):
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + spare
    order = torch.randperm(pages, generator=g).numpy().astype(np.int32)
    table = np.full((len(lens), columns or max(max(need), 1)), -7, np.int32)
    at = 0
    for b, c in enumerate(need):
        table[b, :c] = order[at:at + c]
        at += c
    q, qv = stored(spread * torch.randn((sum(new), heads, dim), generator=g), dtype)
    cache, cv = stored(torch.randn((pages, kv, page, 2 * dim), generator=g), dtype)
    starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    return dict(q=q, qv=qv, cache=cache, cv=cv, table=table, lens=np.array(lens, np.int32), starts=starts, scale=dim ** -0.5,
                g=g, page=page, kv=kv)


def weigh_both(p, *, prior=None, lse=None, in_place=False, out=None, q_scale=1.0, k_scale=1.0, last=0, **opt):
    """(library's, reference's, bound) of one key_weights call."""
    mask = {k: opt[k] for k in ("causal", "window", "softcap") if k in opt}
    if lse is None:
        _, lse, _, _ = ragged_ref.attention(p["qv"], p["cv"], p["table"], p["lens"], p["starts"], p["scale"],
                                            q_scale=q_scale, k_scale=k_scale, **mask)
        lse = lse.astype(np.float32)
    want, err = ref.key_weights(p["qv"], p["cv"], p["table"], p["lens"], p["starts"], lse.astype(np.float64), p["scale"],
                                prior=prior, decay=opt.get("decay", 1.0), last=last, q_scale=q_scale, k_scale=k_scale,
                                **mask)
    w = dev(prior.astype(np.float32)) if prior is not None else None
    q = p.get("dev_q")
    got = pkd.key_weights(p["q"].cuda() if q is None else q, p["cache"].cuda(), dev(p["table"]), dev(p["lens"]),
                          dev(p["starts"]), dev(lse), p["scale"], weights=w, out=w if in_place else out, q_scale=q_scale,
                          k_scale=k_scale, last_queries=last, **opt)
    return got, want, err


def close(got, want, err, lens):
    got = got.double().cpu().numpy()
    for b, L in enumerate(lens):
        d = np.abs(got[b, :, :L] - want[b, :, :L])
        assert np.isfinite(got[b, :, :L]).all()
        assert (d <= err[b, :, :L] + 1e-30).all(), (b, float(np.max(d / (err[b, :, :L] + 1e-30))))


@pytest.mark.parametrize("dtype,dim", [("bf16", 128), ("fp16", 128), ("fp8", 128), ("bf16", 64), ("fp16", 64)])
@pytest.mark.parametrize("heads,kv", [(4, 4), (8, 2), (14, 2), (16, 1), (40, 2)])
@pytest.mark.parametrize("page", [16, 48])
def test_weights_of_a_step(dtype, dim, heads, kv, page):
    """One new token per request, lengths from none to several chunks, the last page partly filled."""
    p = problem(1, new=[1, 1, 1, 1, 0, 1], lens=[1, 17, 333, 64, 40, 0], heads=heads, kv=kv, dim=dim, page=page, dtype=dtype)
    prior = np.random.default_rng(2).random((6, kv, p["table"].shape[1] * page)).astype(np.float32).astype(np.float64)
    got, want, err = weigh_both(p, prior=prior, decay=0.75, max_query_len=1, q_scale=0.5, k_scale=0.7)
    close(got, want, err, p["lens"])
    # each request's new weights sum up to its heads
    got, want, err = weigh_both(p, max_query_len=1)
    close(got, want, err, p["lens"])
    assert np.allclose(got.double().cpu().numpy()[:4].sum((1, 2)), heads, rtol=1e-4)


@pytest.mark.parametrize("opt", [dict(), dict(window=37), dict(window=1), dict(causal=False), dict(softcap=5.0),
                                 dict(softcap=20.0, window=100), dict(last=9), dict(last=1, window=20),
                                 dict(last=1000, causal=False, window=60)])
@pytest.mark.parametrize("dtype,dim,heads,kv", [("bf16", 128, 8, 2), ("fp16", 64, 7, 1), ("fp8", 128, 16, 4)])
def test_weights_of_prompts(dtype, dim, heads, kv, opt):
    p = problem(3, new=[150, 1, 60, 33], lens=[150, 77, 201, 33], heads=heads, kv=kv, dim=dim, page=16, dtype=dtype)
    prior = np.random.default_rng(4).random((4, kv, p["table"].shape[1] * 16)).astype(np.float32).astype(np.float64)
    got, want, err = weigh_both(p, prior=prior, max_query_len=150, **opt)
    close(got, want, err, p["lens"])


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("new,L", [(64, 1500), (300, 900), (700, 700)])
def test_weights_of_long_prompts(dtype, new, L):
    p = problem(5, new=[new], lens=[L], heads=8, kv=2, dim=128, page=32, dtype=dtype)
    got, want, err = weigh_both(p)
    close(got, want, err, p["lens"])


def test_weights_in_place_leave_what_lies_behind():
    p = problem(6, new=[1, 1, 2], lens=[40, 7, 90], heads=8, kv=2, dim=128, page=16, dtype="bf16")
    S = 120
    store = torch.full((3, 2, 2, S), 3.5, device="cuda")  # rows of a larger pool: strides
    view = store[:, 1]
    prior = view.double().cpu().numpy()
    want, err = ref.key_weights(p["qv"], p["cv"], p["table"], p["lens"], p["starts"],
                                lse := ragged_ref.attention(p["qv"], p["cv"], p["table"], p["lens"], p["starts"],
                                                            p["scale"])[1].astype(np.float32), p["scale"], prior=prior)
    got = pkd.key_weights(p["q"].cuda(), p["cache"].cuda(), dev(p["table"]), dev(p["lens"]), dev(p["starts"]), dev(lse),
                          p["scale"], weights=view, out=view, max_query_len=2)
    assert got is view
    close(got, want, err, p["lens"])
    for b, L in enumerate(p["lens"]):
        assert (view[b, :, L:] == 3.5).all()
    assert (store[:, 0] == 3.5).all()


def test_weights_of_rows_that_see_nothing_and_of_hidden_values():
    """LSEs of -inf weigh nothing; keys that no token sees get 0 whatever they hold, and NaN
    behind the length or outside the window reaches nothing."""
    p = problem(7, new=[2, 3], lens=[100, 61], heads=4, kv=2, dim=128, page=16, dtype="bf16")
    cache = p["cache"].clone()
    for b, L in enumerate((100, 61)):
        for t in list(range(0, L - 3 - 20)) + list(range(L, -(-L // 16) * 16)):
            cache[p["table"][b, t // 16], :, t % 16, :128] = float("nan")
    cache[..., 128:] = float("nan")  # V is not read
    lse = ragged_ref.attention(p["qv"], p["cv"], p["table"], p["lens"], p["starts"], p["scale"], window=21)[1]
    lse = lse.astype(np.float32)
    lse[1, 2] = lse[3] = -np.inf
    want, err = ref.key_weights(p["qv"], p["cv"], p["table"], p["lens"], p["starts"], lse.astype(np.float64), p["scale"],
                                window=21)
    p["cache"] = cache
    got = pkd.key_weights(p["q"].cuda(), cache.cuda(), dev(p["table"]), dev(p["lens"]), dev(p["starts"]), dev(lse), p["scale"],
                          window=21, max_query_len=3)
    close(got, want, err, p["lens"])
    assert (got[0, :, :100 - 3 - 20] == 0).all()


def test_weights_of_strided_queries_and_wide_tables():
    p = problem(8, new=[1] * 5, lens=[20, 40, 1, 16, 99], heads=8, kv=2, dim=64, page=16, dtype="fp16", columns=9)
    wide = torch.zeros((5, 3, 8, 64), dtype=torch.float16, device="cuda")
    wide[:, 1] = p["q"].cuda()
    p["dev_q"] = wide[:, 1]
    got, want, err = weigh_both(p, max_query_len=1, max_kv_len=99)
    close(got, want, err, p["lens"])


def test_weights_of_bad_pages_and_lengths():
    p = problem(9, new=[1, 1], lens=[64, 64], heads=4, kv=2, dim=128, page=16, dtype="bf16")
    lse = ragged_ref.attention(p["qv"], p["cv"], p["table"], p["lens"], p["starts"], p["scale"])[1].astype(np.float32)
    table = p["table"].copy()
    table[0, 1], table[1, 3] = 10 ** 6, -1
    lens = np.array([64, 900], np.int32)
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    got = pkd.key_weights(p["q"].cuda(), p["cache"].cuda(), dev(table), dev(lens), dev(p["starts"]), dev(lse), p["scale"],
                          max_query_len=1, workspace=ws)
    assert pkd.workspace_check(ws) == pkd.EDEVICE_BOUNDS and pkd.workspace_check(ws) == pkd.OK
    want, err = ref.key_weights(p["qv"], p["cv"], table, p["lens"], p["starts"], lse.astype(np.float64), p["scale"])
    close(got, want, err, p["lens"])
    assert (got[0, :, 16:32] == 0).all() and (got[1, :, 48:64] == 0).all()


def test_weights_without_tokens_fade():
    """A call of no tokens: what was there times decay."""
    p = problem(10, new=[0, 0], lens=[30, 5], heads=4, kv=2, dim=128, page=16, dtype="bf16")
    prior = torch.rand((2, 2, 32), device="cuda")
    got = pkd.key_weights(p["q"].cuda(), p["cache"].cuda(), dev(p["table"]), dev(p["lens"]), dev(p["starts"]),
                          torch.zeros((0, 4), device="cuda"), p["scale"], weights=prior, decay=0.5)
    assert torch.equal(got[0, :, :30], prior[0, :, :30] * 0.5) and torch.equal(got[1, :, :5], prior[1, :, :5] * 0.5)
    assert (got[1, :, 5:] == 0).all()


def test_weights_repeat_bit_for_bit():
    p = problem(11, new=[200, 90, 1], lens=[500, 90, 300], heads=16, kv=4, dim=128, page=16, dtype="bf16")
    a, _, _ = weigh_both(p, max_query_len=200)
    for _ in range(3):
        assert torch.equal(a, weigh_both(p, max_query_len=200)[0])


@pytest.mark.parametrize("softcap", [0.0, 5.0])
def test_weights_do_not_depend_on_what_ran_before(softcap):
    """Keys behind the length and columns without a row hold what an earlier call left in shared
    memory: large values there change no bit."""
    p = problem(12, new=[90, 41], lens=[150, 41], heads=14, kv=2, dim=128, page=16, dtype="bf16")
    big = problem(13, new=[300], lens=[900], heads=14, kv=2, dim=128, page=16, dtype="bf16", spread=30.0)
    lse = torch.full((131, 14), 3.0, device="cuda")
    args = (p["q"].cuda(), p["cache"].cuda(), dev(p["table"]), dev(p["lens"]), dev(p["starts"]), lse, p["scale"])
    good = pkd.key_weights(*args, softcap=softcap, max_query_len=90)
    for huge in (1.0, 50.0):
        cache = (big["cache"].float() * huge).to(torch.bfloat16).cuda()
        for _ in range(2):
            pkd.key_weights(big["q"].cuda(), cache, dev(big["table"]), dev(big["lens"]), dev(big["starts"]),
                            torch.zeros((300, 14), device="cuda"), big["scale"], max_query_len=300)
        assert torch.equal(pkd.key_weights(*args, softcap=softcap, max_query_len=90), good)


def test_a_timeout_of_weights_is_reported_and_recovered_from():
    p = problem(14, new=[1500, 700], lens=[1500, 700], heads=16, kv=8, dim=128, page=16, dtype="bf16")
    lse = torch.full((2200, 16), 5.0, device="cuda")
    args = (p["q"].cuda(), p["cache"].cuda(), dev(p["table"]), dev(p["lens"]), dev(p["starts"]), lse, p["scale"])
    ws = torch.zeros(1 << 26, dtype=torch.uint8, device="cuda")
    good = pkd.key_weights(*args, max_query_len=1500, workspace=ws)
    assert pkd.workspace_check(ws) == pkd.OK
    pkd.key_weights(*args, max_query_len=1500, workspace=ws, test_timeout=True)
    assert pkd.workspace_check(ws) == pkd.ETIMEOUT
    pkd.workspace_init(ws)
    again = pkd.key_weights(*args, max_query_len=1500, workspace=ws)
    assert pkd.workspace_check(ws) == pkd.OK and torch.equal(again, good)
    pkd.key_weights(*args, max_query_len=1500, test_timeout=True)
    assert pkd.workspace_check() == pkd.ETIMEOUT
    assert torch.equal(pkd.key_weights(*args, max_query_len=1500), good)


@pytest.mark.parametrize("window,softcap", [(0, 0.0), (40, 0.0), (40, 5.0)])
def test_weights_of_many_short_items(window, softcap):
    """More items than SMs, of one to four query tiles, on blocks of one key tile and of two in turn:
    every call has the same bits, and none runs into a wait's limit."""
    lens = [150, 140, 67, 300, 149, 390, 81, 260]
    p = problem(16, new=[150, 140, 67, 120, 149, 150, 81, 130], lens=lens, heads=128, kv=2, dim=64, page=16, dtype="bf16")
    _, lse, _, _ = ragged_ref.attention(p["qv"], p["cv"], p["table"], p["lens"], p["starts"], p["scale"], window=window,
                                        softcap=softcap)
    lse = lse.astype(np.float32)
    opt = dict(window=window, softcap=softcap)
    got, want, err = weigh_both(p, lse=lse, max_query_len=150, **opt)
    close(got, want, err, lens)
    ws = torch.zeros(1 << 26, dtype=torch.uint8, device="cuda")
    args = (p["q"].cuda(), p["cache"].cuda(), dev(p["table"]), dev(p["lens"]), dev(p["starts"]), dev(lse), p["scale"])
    for _ in range(60):
        ws[256 + 4 * 65536:] = 255  # parts that are read before they are written show as NaN
        again = pkd.key_weights(*args, max_query_len=150, workspace=ws, **opt)
        assert torch.equal(again, got)
    assert pkd.workspace_check(ws) == pkd.OK
    assert not ws[256:256 + 4 * 65536].any()


def test_weights_of_a_batch_whose_rows_stay():
    """Few rows of many requests: runs of key blocks, some behind the last key, one unseen by a window."""
    lens = [2000, 10, 700, 1300, 0, 257, 256]
    p = problem(15, new=[12, 5, 9, 12, 0, 1, 12], lens=lens, heads=8, kv=2, dim=64, page=16, dtype="fp16")
    got, want, err = weigh_both(p, max_query_len=12)
    close(got, want, err, lens)
    got, want, err = weigh_both(p, max_query_len=12, window=300, last=7)
    close(got, want, err, lens)


# ------------------------------------------------------------------ choice of the keys
def select_both(weights, lens, budget, **opt):
    pos, ctx = opt.pop("positions", None), opt.pop("context", None)
    want = ref.evict_select(weights, lens, budget, positions=pos, context=ctx, **opt)
    got = pkd.evict_select(dev(weights.astype(np.float32)), dev(np.asarray(lens, np.int32)), budget,
                           positions=None if pos is None else dev(pos.astype(np.int32)),
                           context_lens=None if ctx is None else dev(np.asarray(ctx, np.int32)), **opt)
    return [x.cpu().numpy() for x in got], want


@pytest.mark.parametrize("S,budget", [(1, 1), (5, 5), (40, 8), (513, 512), (700, 1), (1500, 333), (5000, 4000)])
@pytest.mark.parametrize("pool", [1, 5, 7, 33])
def test_select(S, budget, pool):
    rng = np.random.default_rng(S + budget)
    lens = [S, S // 2, min(S, budget), min(S, budget + 1), 0]
    w = np.exp(3 * rng.standard_normal((5, 3, S))).astype(np.float32)
    w[rng.random(w.shape) < 0.3] = 0.0
    s, r = (min(4, budget // 4), budget // 3)
    got, want = select_both(w, lens, budget, sinks=s, recent=r, pool=pool)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])


@pytest.mark.parametrize("values", [[0.0], [1.0, 2.0], [-0.0, 0.0], [float("nan"), 0.5, -1.0], [float("inf"), 3e38, 1e-42],
                                    [-float("inf"), float("nan"), -5.0], [1.0, float(np.nextafter(np.float32(1), np.float32(2)))]])
def test_select_ties_and_special_values(values):
    rng = np.random.default_rng(1)
    w = np.array(values, np.float32)[rng.integers(0, len(values), (2, 2, 300))]
    for pool in (1, 3):
        got, want = select_both(w, [300, 123], 77, sinks=2, recent=5, pool=pool)
        assert np.array_equal(got[0], want[0])


def test_select_out_of_order():
    """Positions of keys that compactions have put out of order."""
    rng = np.random.default_rng(2)
    S = 260
    pos = np.stack([[rng.permutation(400)[:S] for _ in range(2)] for _ in range(3)])
    w = rng.random((3, 2, S)).astype(np.float32)
    got, want = select_both(w, [260, 150, 90], 100, sinks=6, recent=40, positions=pos, context=[400, 400, 401])
    assert np.array_equal(got[0], want[0])


def test_select_clamps_lengths_and_takes_strides():
    store = torch.rand((2, 4, 3, 90), device="cuda")
    view = store[:, 2]
    lens = torch.tensor([-5, 1000], dtype=torch.int32, device="cuda")
    kept, n = pkd.evict_select(view, lens, 30, recent=4)
    want = ref.evict_select(view.cpu().numpy(), [-5, 1000], 30, recent=4)
    assert np.array_equal(kept.cpu().numpy(), want[0]) and n.tolist() == [0, 30]


@pytest.mark.parametrize("S,budget", [(10000, 164), (70000, 3000), (130001, 128), (200001, 150000)])
def test_select_long(S, budget):
    g = torch.Generator(device="cuda").manual_seed(S)
    w = torch.exp(2 * torch.randn((2, 2, S), device="cuda", generator=g))
    w[torch.rand(w.shape, device="cuda", generator=g) < 0.4] = 0
    lens = torch.tensor([S, S - 4321], dtype=torch.int32, device="cuda")
    kept, n = pkd.evict_select(w, lens, budget, sinks=3, recent=100)
    for b, L in enumerate(lens.tolist()):
        x = w[b, :, :L].clone()
        x[:, :3] = x[:, L - 100:] = torch.inf
        want = x.sort(dim=-1, descending=True, stable=True)[1][:, :budget].sort(-1)[0]
        assert torch.equal(kept[b].long(), want)


@pytest.mark.parametrize("S,pool", [(9000, 255), (20000, 7), (140000, 5)])
def test_select_pooled_over_several_ctas(S, pool):
    """Neighbours across the CTAs of a row, and rows that are read again."""
    g = torch.Generator(device="cuda").manual_seed(S)
    w = torch.exp(2 * torch.randn((1, 2, S), device="cuda", generator=g))
    lens = torch.tensor([S - 77], dtype=torch.int32, device="cuda")
    kept, _ = pkd.evict_select(w, lens, 500, sinks=2, recent=30, pool=pool)
    L, side = S - 77, pool // 2
    x = w[..., :L].clone()
    x[..., :2] = x[..., L - 30:] = -torch.inf
    x = torch.nn.functional.pad(x, (side, side), value=-torch.inf).unfold(-1, pool, 1).amax(-1)
    x[..., :2] = x[..., L - 30:] = torch.inf
    assert torch.equal(kept[0].long(), x[0].sort(dim=-1, descending=True, stable=True)[1][:, :500].sort(-1)[0])


# ------------------------------------------------------------------ compaction
@pytest.mark.parametrize("dtype,dim,page", [("bf16", 128, 16), ("fp16", 64, 48), ("fp8", 128, 64), ("fp8", 64, 16)])
@pytest.mark.parametrize("S,budget", [(40, 40), (300, 1), (300, 17), (900, 512), (900, 899)])
def test_compact(dtype, dim, page, S, budget):
    rng = np.random.default_rng(S + budget)
    H, lens = 3, [S, max(1, S // 2), 1]
    p = problem(20, new=[1] * 3, lens=lens, heads=H, kv=H, dim=dim, page=page, dtype=dtype)
    keys = p["table"].shape[1] * page
    w, x = rng.random((3, H, keys)).astype(np.float32), rng.integers(0, 10 ** 6, (3, H, keys)).astype(np.int32)
    kept, n = ref.evict_select(rng.random((3, H, S)), lens, budget)
    bits = p["cache"].view(torch.uint8)
    cache, dw, dx = bits.cuda().view(p["cache"].dtype), dev(w), dev(x)
    assert pkd.cache_compact(cache, dev(p["table"]), dev(kept), dev(n), weights=dw, positions=dx) is cache
    want = bits.numpy().copy()
    ref.cache_compact(want, p["table"], kept, n, (w, x))
    assert np.array_equal(cache.view(torch.uint8).cpu().numpy(), want)
    assert np.array_equal(dw.cpu().numpy(), w) and np.array_equal(dx.cpu().numpy(), x)


@pytest.mark.parametrize("budget", [10240, 11000])
def test_compact_long_lists(budget):
    """Lists that fill shared memory, and such as are searched where they are."""
    rng = np.random.default_rng(budget)
    p = problem(22, new=[1], lens=[12000], heads=2, kv=2, dim=64, page=16, dtype="fp16")
    kept, n = ref.evict_select(rng.random((1, 2, 12000)), [12000], budget)
    cache = p["cache"].cuda()
    pkd.cache_compact(cache, dev(p["table"]), dev(kept), dev(n))
    want = p["cache"].view(torch.int16).numpy().copy()
    ref.cache_compact(want, p["table"], kept, n)
    assert np.array_equal(cache.view(torch.int16).cpu().numpy(), want)


@pytest.mark.parametrize("name,dtype", [("weights", torch.float32), ("positions", torch.int32)])
def test_compact_refuses_arrays_without_keys(name, dtype):
    p = problem(23, new=[1], lens=[40], heads=2, kv=2, dim=64, page=16, dtype="bf16")
    kept, n = ref.evict_select(np.arange(80.).reshape(1, 2, 40), [40], 8)
    cache = p["cache"].cuda()
    with pytest.raises(ValueError, match="must have keys"):
        pkd.cache_compact(cache, dev(p["table"]), dev(kept), dev(n), **{name: torch.empty((1, 2, 0), dtype=dtype, device="cuda")})
    assert torch.equal(cache.cpu().view(torch.int16), p["cache"].view(torch.int16))


def test_compact_bad_pages_and_indexes_move_nothing():
    rng = np.random.default_rng(21)
    p = problem(21, new=[1] * 2, lens=[200, 200], heads=2, kv=2, dim=128, page=16, dtype="bf16")
    kept, n = ref.evict_select(rng.random((2, 2, 200)), [200, 200], 60)
    kept[1, 0, -1] = 10 ** 8  # behind the table: does not move
    table = p["table"].copy()
    table[0, 0], table[0, 9] = -1, 10 ** 7
    bits = p["cache"].view(torch.int16)
    cache = p["cache"].cuda()
    w = rng.random((2, 2, 208)).astype(np.float32)
    dw = dev(w)
    pkd.cache_compact(cache, dev(table), dev(kept), dev(n), weights=dw)
    want = bits.numpy().copy()
    for b in range(2):
        for h in range(2):
            stay = kept[b, h]
            free = sorted(set(range(60)) - set(int(s) for s in stay))
            for s, t in zip([s for s in stay if s >= 60], free):
                if s >= 208 or not 0 <= table[b, s // 16] < len(want) or not 0 <= table[b, t // 16] < len(want):
                    continue
                want[table[b, t // 16], h, t % 16] = want[table[b, s // 16], h, s % 16]
                w[b, h, t] = w[b, h, s]
    assert np.array_equal(cache.view(torch.int16).cpu().numpy(), want)
    assert np.array_equal(dw.cpu().numpy(), w)


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("dtype,tol", [("bf16", 2.0 ** -8), ("fp16", 2.0 ** -11)])
def test_prompt_to_bounded_cache_and_on(dtype, tol):
    """A prompt is attended to, its last tokens weigh its keys, the cache goes down to a budget, and
    a decode step attends to what stayed, weighs it, and goes down again: against 64 bits."""
    heads, kv, dim, page, budget = 8, 2, 128, 16, 96
    lens = [300, 90, 180]
    p = problem(30, new=lens, lens=lens, heads=heads, kv=kv, dim=dim, page=page, dtype=dtype, columns=20)
    cache, table, q = p["cache"].cuda(), dev(np.maximum(p["table"], 0)), p["q"].cuda()
    starts = dev(p["starts"])
    seq = dev(p["lens"])
    _, lse = pkd.paged_attention(q, cache, table, seq, starts, p["scale"], max_query_len=300)
    w = pkd.key_weights(q, cache, table, seq, starts, lse, p["scale"], last_queries=16, max_query_len=300)
    kept, n = pkd.evict_select(w, seq, budget, sinks=2, recent=16, pool=5)
    want, _ = ref.evict_select(w.cpu().numpy(), lens, budget, sinks=2, recent=16, pool=5)
    assert np.array_equal(kept.cpu().numpy(), want)
    pos = torch.arange(w.shape[2], dtype=torch.int32, device="cuda").expand(3, kv, -1).contiguous()
    pkd.cache_compact(cache, table, kept, n, weights=w, positions=pos)
    # the positions tell which key lies where
    for b in range(3):
        for h in range(kv):
            assert sorted(pos[b, h, :n[b]].tolist()) == want[b, h, :int(n[b])].tolist()
    g = torch.Generator().manual_seed(31)
    context = [L for L in lens]
    for step in range(2):
        k, v = (torch.randn((3, kv, dim), generator=g).to(TYPES[dtype]).cuda() for _ in range(2))
        qs = (1.5 * torch.randn((3, 1, heads, dim), generator=g)).to(TYPES[dtype]).cuda()
        at = n.long()
        slots = table[torch.arange(3, device="cuda"), at // page].long() * page + at % page
        pkd.cache_write(k, v, slots, cache)
        for b in range(3):
            pos[b, :, int(n[b])] = context[b]
            context[b] += 1
        n = n + 1
        out, lse = pkd.paged_decode(qs, cache, table, n, p["scale"])
        old = w.double().cpu().numpy()
        ones = torch.arange(4, dtype=torch.int32, device="cuda")
        w = pkd.key_weights(qs[:, 0], cache, table, n, ones, lse[:, 0], p["scale"], weights=w, out=w, max_query_len=1)
        cv, qv = cache.float().double().cpu().numpy(), qs[:, 0].float().double().cpu().numpy()
        tb, ln, st = table.cpu().numpy(), n.cpu().numpy(), np.arange(4)
        o, l, mag, _ = ragged_ref.attention(qv, cv, tb, ln, st, p["scale"])
        # a rounding of the weights and one of the result, and the fp32 sums
        assert (np.abs(out[:, 0].double().cpu().numpy() - o) <= tol * (mag + np.abs(o)) + 2.0 ** -12 * mag).all()
        want, err = ref.key_weights(qv, cv, tb, ln, st, lse[:, 0].double().cpu().numpy(), p["scale"], prior=old)
        close(w, want, err, ln)
        kept, m = pkd.evict_select(w, n, budget, sinks=2, recent=16, positions=pos,
                                   context_lens=torch.tensor(context, dtype=torch.int32, device="cuda"))
        want, _ = ref.evict_select(w.cpu().numpy(), ln, budget, sinks=2, recent=16, positions=pos.cpu().numpy(),
                                   context=context)
        assert np.array_equal(kept.cpu().numpy(), want)
        bits = cache.view(torch.int16).cpu().numpy()
        ref.cache_compact(bits, tb, want, m.cpu().numpy())
        pkd.cache_compact(cache, table, kept, m, weights=w, positions=pos)
        assert np.array_equal(cache.view(torch.int16).cpu().numpy(), bits)
        n = m


@pytest.mark.parametrize("side", [False, True])
def test_a_captured_step_of_eviction(side):
    """Weights, choice and compaction captured into a graph and replayed, on another stream too."""
    p = problem(40, new=[1] * 4, lens=[140, 130, 129, 128], heads=8, kv=2, dim=128, page=16, dtype="bf16")
    lse = dev(ragged_ref.attention(p["qv"], p["cv"], p["table"], p["lens"], p["starts"], p["scale"])[1].astype(np.float32))
    args = (p["q"].cuda(), p["cache"].cuda(), dev(p["table"]), dev(p["lens"]), dev(p["starts"]), lse, p["scale"])
    start = p["cache"].cuda()

    def step():
        w = pkd.key_weights(*args, max_query_len=1)
        kept, n = pkd.evict_select(w, args[3], 128, recent=8)
        pkd.cache_compact(args[1], args[2], kept, n, weights=w)
        return w, kept, n

    w, kept, n = step()
    moved = args[1].clone()
    args[1].copy_(start)
    stream = torch.cuda.Stream() if side else torch.cuda.current_stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(torch.cuda.Stream()):
        step()  # warm up, and undo
        args[1].copy_(start)
        torch.cuda.synchronize()
    with torch.cuda.graph(g):
        w2, kept2, n2 = step()
    args[1].copy_(start)
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(args[1], moved) and torch.equal(kept, kept2) and torch.equal(n, n2)


def test_calls_on_two_streams_and_graphs_at_once():
    """Weights on two streams, each with the workspace kept for it, and in two graphs that are
    replayed side by side: split tokens, so that counters and parts are in use."""
    p = problem(41, new=[700], lens=[900], heads=16, kv=2, dim=128, page=16, dtype="bf16")
    lse = torch.full((700, 16), 6.0, device="cuda")
    args = (p["q"].cuda(), p["cache"].cuda(), dev(p["table"]), dev(p["lens"]), dev(p["starts"]), lse, p["scale"])
    good = pkd.key_weights(*args)
    streams = [torch.cuda.Stream() for _ in range(2)]
    graphs, outs = [], []
    for _ in streams:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(pkd.key_weights(*args))
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(10):
        got = []
        for s in streams:
            with torch.cuda.stream(s):
                got.append(pkd.key_weights(*args))
        torch.cuda.synchronize()
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, good) for x in got + outs)
    assert pkd.workspace_check(stream=streams[0]) == pkd.workspace_check(stream=streams[1]) == pkd.OK
