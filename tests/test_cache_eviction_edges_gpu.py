"""Choice and compaction where they can go wrong: results beside their inputs, rows that cannot move,
long lists of keys out of order, many lists."""
import numpy as np
import pytest
import torch

import paged_kv_decode_15_gb300 as pkd
from tests import eviction_ref as ref
from tests.test_cache_eviction_gpu import dev, problem, select_both

pytestmark = pytest.mark.gpu


def test_select_writes_right_beside_its_inputs():
    """One allocation: kept_lens, lengths, weights, kept, with nothing between them; and a refusal of
    lengths as kept_lens leaves them as they were."""
    rng = np.random.default_rng(1)
    S, budget = 90, 30
    w = rng.random((2, 3, S)).astype(np.float32)
    want = ref.evict_select(w, [90, 41], budget, sinks=2, recent=4)
    store = torch.full((2 + 2 + 6 * S + 6 * budget,), 7, dtype=torch.int32, device="cuda")
    n, lens, at, kept = store[:2], store[2:4], store[4:4 + 6 * S].view(torch.float32).view(2, 3, S), store[4 + 6 * S:].view(2, 3, budget)
    lens.copy_(torch.tensor([90, 41]))
    at.copy_(torch.as_tensor(w))
    got = pkd.evict_select(at, lens, budget, sinks=2, recent=4, kept=kept, kept_lens=n)
    assert got[0] is kept and got[1] is n
    assert np.array_equal(kept.cpu().numpy(), want[0]) and np.array_equal(n.cpu().numpy(), want[1])
    assert np.array_equal(at.cpu().numpy(), w) and lens.tolist() == [90, 41]
    with pytest.raises(pkd.PkdError, match="overlaps"):
        pkd.evict_select(at, lens, budget, sinks=2, recent=4, kept_lens=lens)
    assert lens.tolist() == [90, 41]


def status(call, **kw):
    """Results of a call, and the status that it leaves in a workspace of its own and in the kept one."""
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    got = call(workspace=ws, **kw)
    own = pkd.workspace_check(ws)
    assert pkd.workspace_check(ws) == pkd.OK
    pkd.workspace_check()
    call(**kw)
    assert pkd.workspace_check() == own and pkd.workspace_check() == pkd.OK
    return got, own


@pytest.mark.parametrize("S", [90, 9000])
@pytest.mark.parametrize("lens,code", [([5, 90], pkd.OK), ([0, 30], pkd.OK), ([91, 3], pkd.EDEVICE_BOUNDS), ([3, -1], pkd.EDEVICE_BOUNDS)])
def test_select_reports_lengths_out_of_range(S, lens, code):
    """Alone and by clusters; the lengths are clamped, as before."""
    rng = np.random.default_rng(2)
    lens = [n if n <= 90 and S == 90 else n - 90 + S if n > 90 else n for n in lens]
    w = rng.random((2, 2, S)).astype(np.float32)
    (kept, n), got = status(lambda **kw: pkd.evict_select(dev(w), dev(np.array(lens, np.int32)), 30, recent=4, **kw))
    want = ref.evict_select(w, lens, 30, recent=4)
    assert got == code and np.array_equal(kept.cpu().numpy(), want[0]) and np.array_equal(n.cpu().numpy(), want[1])


@pytest.mark.parametrize("what,code", [("none", pkd.OK), ("narrow weights", pkd.EDEVICE_BOUNDS), ("narrow positions", pkd.EDEVICE_BOUNDS),
                                       ("just wide enough", pkd.OK), ("source page", pkd.EDEVICE_BOUNDS),
                                       ("target page", pkd.EDEVICE_BOUNDS), ("behind the table", pkd.EDEVICE_BOUNDS),
                                       ("kept_lens", pkd.EDEVICE_BOUNDS), ("page of no way", pkd.OK)])
def test_compact_reports_rows_that_do_not_move(what, code):
    """A row moves with its weight and position or not at all, and the status says when one did not."""
    p = problem(3, new=[1, 1], lens=[200, 200], heads=2, kv=2, dim=64, page=16, dtype="bf16")
    rng = np.random.default_rng(4)
    x = rng.random((2, 2, 200))
    x[..., 185:] = 2  # keys 185 to 199 stay, and move
    x[..., :20] = np.where(np.arange(20) % 2, 3, -1)  # of the first twenty every other stays
    if what == "page of no way":
        x[..., 176:192] = -1
    kept, n = ref.evict_select(x, [200, 200], 60)
    table, keys = p["table"].copy(), p["table"].shape[1] * 16
    w, pos = rng.random((2, 2, keys)).astype(np.float32), rng.integers(0, 9999, (2, 2, keys)).astype(np.int32)
    limit = keys
    if what == "narrow weights":
        w, limit = np.ascontiguousarray(w[..., :190]), 190
    if what == "narrow positions":
        pos, limit = np.ascontiguousarray(pos[..., :199]), 199
    if what == "just wide enough":
        w, pos = np.ascontiguousarray(w[..., :200]), np.ascontiguousarray(pos[..., :200])
    if what == "source page":
        table[1, 12] = -1
    if what == "target page":
        table[0, 0] = len(p["cache"])
    if what == "behind the table":
        kept[0, 1, -1] = keys
    if what == "kept_lens":
        n[1] = 61
    if what == "page of no way":
        table[0, 11] = table[1, 11] = 10 ** 6  # (no key of it stays)
    want, rows = p["cache"].view(torch.int16).numpy().copy(), [w.copy(), pos.copy()]
    for b in range(2):
        m = min(int(n[b]), 60)
        for h in range(2):
            stay = [int(s) for s in kept[b, h, :m]]
            for s, t in zip([s for s in stay if s >= m], sorted(set(range(m)) - set(stay))):
                if s >= limit or not 0 <= table[b, s // 16] < len(want) or not 0 <= table[b, t // 16] < len(want):
                    continue
                want[table[b, t // 16], h, t % 16] = want[table[b, s // 16], h, s % 16]
                for r in rows:
                    r[b, h, t] = r[b, h, s]

    def call(**kw):
        cache, dw, dx = p["cache"].cuda(), dev(w), dev(pos)
        pkd.cache_compact(cache, dev(table), dev(kept), dev(n), weights=dw, positions=dx, **kw)
        return cache, dw, dx

    (cache, dw, dx), got = status(call)
    assert got == code
    assert np.array_equal(cache.view(torch.int16).cpu().numpy(), want)
    assert np.array_equal(dw.cpu().numpy(), rows[0]) and np.array_equal(dx.cpu().numpy(), rows[1])


def test_captured_choice_and_compaction_report_to_a_workspace_given():
    p = problem(5, new=[1], lens=[100], heads=2, kv=2, dim=64, page=16, dtype="fp16")
    w, lens, table = torch.rand((1, 2, 100), device="cuda"), dev(np.array([100], np.int32)), dev(p["table"])
    cache, ws = p["cache"].cuda(), torch.zeros(256, dtype=torch.uint8, device="cuda")
    pkd.workspace_check()

    def step(**kw):
        kept, n = pkd.evict_select(w, lens, 50, **kw)
        pkd.cache_compact(cache, table, kept, n, **kw)

    with torch.cuda.stream(torch.cuda.Stream()):
        step()
        torch.cuda.synchronize()
    for kw in (dict(), dict(workspace=ws)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(**kw)
        for bad in (False, True):
            lens.fill_(101 if bad else 100)
            g.replay()
            torch.cuda.synchronize()
            assert pkd.workspace_check(ws) == (pkd.EDEVICE_BOUNDS if kw and bad else pkd.OK)
    assert pkd.workspace_check() == pkd.OK


@pytest.mark.parametrize("B,S,budget", [(40, 3000, 900), (12, 9000, 1000), (1, 16000, 15000), (1, 70000, 4096), (1, 140001, 3000)])
def test_select_of_long_rows_out_of_order(B, S, budget):
    """Positions in every tier: a CTA to a row, clusters, and rows that are read again; ties of weight
    and of nothing received, lengths around the budget."""
    H = 2
    g = torch.Generator(device="cuda").manual_seed(S)
    w = torch.exp(2 * torch.randn((B, H, S), device="cuda", generator=g))
    w[torch.rand(w.shape, device="cuda", generator=g) < 0.4] = 0
    w = (w * 64).round() / 64
    context = [S + 500 + 7 * b for b in range(B)]
    pos = torch.stack([torch.rand((H, context[b]), device="cuda", generator=g).argsort(-1)[:, :S] for b in range(B)]).int()
    lens = [S, budget, budget + 1, S - 3][:B] + [S - 31 * b for b in range(4, B)]
    sinks, recent = 5, min(700, budget // 2)
    kept, n = pkd.evict_select(w, dev(np.array(lens, np.int32)), budget, sinks=sinks, recent=recent, positions=pos,
                               context_lens=dev(np.array(context, np.int32)))
    assert n.tolist() == [min(L, budget) for L in lens]
    for b, L in enumerate(lens):
        x, at, m = w[b, :, :L].clone(), pos[b, :, :L], min(L, budget)
        x[(at < sinks) | (at >= context[b] - recent)] = torch.inf
        want = x.sort(dim=-1, descending=True, stable=True)[1][:, :m].sort(-1)[0]
        assert torch.equal(kept[b, :, :m].long(), want) and (kept[b, :, m:] == -1).all()


@pytest.mark.parametrize("dtype,dim", [("fp8", 64), ("bf16", 64), ("fp16", 128)])
def test_compact_of_many_lists_with_many_moves(dtype, dim):
    """More moves than the one CTA of a list takes at a time: rows of 128, 256 and 512 bytes, with
    weights and positions."""
    B, H, S, budget = 40, 16, 1500, 700
    rng = np.random.default_rng(6)
    need, order = -(-S // 16), rng.permutation(B * -(-S // 16)).astype(np.int32)
    table = order.reshape(B, need)
    bits = rng.integers(0, 256, (B * need, H, 16, 2 * dim * (1 if dtype == "fp8" else 2)), dtype=np.uint8)
    lens = [S - 3 * b for b in range(B)]
    kept = np.stack([np.stack([np.sort(rng.permutation(L)[:budget]) for _ in range(H)]) for L in lens]).astype(np.int32)
    n = np.full(B, budget, np.int32)
    w, x = rng.random((B, H, need * 16)).astype(np.float32), rng.integers(0, 9999, (B, H, need * 16)).astype(np.int32)
    cache, dw, dx = dev(bits), dev(w), dev(x)
    view = cache.view({"fp8": torch.float8_e4m3fn, "bf16": torch.bfloat16, "fp16": torch.float16}[dtype])
    pkd.cache_compact(view, dev(table), dev(kept), dev(n), weights=dw, positions=dx)
    assert min((kept[b, h] >= budget).sum() for b in range(B) for h in range(H)) > 256
    ref.cache_compact(bits, table, kept, n, (w, x))
    assert np.array_equal(cache.cpu().numpy(), bits)
    assert np.array_equal(dw.cpu().numpy(), w) and np.array_equal(dx.cpu().numpy(), x)


@pytest.mark.parametrize("S", [300, 3000, 20000])
@pytest.mark.parametrize("pool", [3, 7, 9, 11, 255])
def test_select_with_windows_in_registers_and_looped_over(S, pool):
    """Both sides of the rule; neighbours across threads and CTAs, at both ends, beside sinks and the recent."""
    g = torch.Generator(device="cuda").manual_seed(S + pool)
    w = torch.exp(2 * torch.randn((2, 2, S), device="cuda", generator=g))
    w[torch.rand(w.shape, device="cuda", generator=g) < 0.3] = 0
    lens, side = [S, S - 101], pool // 2
    for sinks, recent in ((0, 0), (3, 20)):
        kept, _ = pkd.evict_select(w, dev(np.array(lens, np.int32)), 100, sinks=sinks, recent=recent, pool=pool)
        for b, L in enumerate(lens):
            x = w[b, :, :L].clone()
            x[:, :sinks] = x[:, L - recent:] = -torch.inf
            x = torch.nn.functional.pad(x, (side, side), value=-torch.inf).unfold(-1, pool, 1).amax(-1)
            x[:, :sinks] = x[:, L - recent:] = torch.inf
            assert torch.equal(kept[b].long(), x.sort(dim=-1, descending=True, stable=True)[1][:, :100].sort(-1)[0])
