"""Weights of keys where they can go wrong, on each plan of the kernels: the step grid, query
tiles that stay, query tiles that stream past (their tokens split)."""
import numpy as np
import pytest
import torch

import paged_kv_decode_15_gb300 as pkd
from tests import eviction_ref as ref
from tests import ragged_ref
from tests.test_cache_eviction_gpu import close, dev, problem, weigh_both

pytestmark = pytest.mark.gpu

# tokens of two requests; 4 heads to a kv head
PLANS = {"step": (3, 2), "stay": (40, 33), "stream": (700, 90)}


def plan(name, seed, *, lens=None, dtype="bf16", dim=128):
    new = PLANS[name]
    return problem(seed, new=list(new), lens=lens or [max(new[0], 300), 210], heads=8, kv=2, dim=dim, page=16, dtype=dtype)


def lses(p, **mask):
    return ragged_ref.attention(p["qv"], p["cv"], p["table"], p["lens"], p["starts"], p["scale"], **mask)[1].astype(np.float32)


def call(p, lse, *, cache=None, table=None, lens=None, **opt):
    n = np.diff(p["starts"]).max()
    return pkd.key_weights(p["q"].cuda(), (p["cache"] if cache is None else cache).cuda(),
                           dev(p["table"] if table is None else table), dev(p["lens"] if lens is None else lens),
                           dev(p["starts"]), dev(lse), p["scale"], max_query_len=int(n), **opt)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("opt", [dict(), dict(softcap=5.0), dict(window=50), dict(causal=False, softcap=5.0)])
@pytest.mark.parametrize("name", PLANS)
def test_tokens_of_no_lse_weigh_nothing_whatever_they_hold(name, opt, bad):
    """A padding token: LSE -inf, q not finite; of one head of a token too.  The last key is seen by
    such a token alone (causal), and holds NaN."""
    p = plan(name, 1)
    lse = lses(p, **opt)
    n = int(p["starts"][1])
    q, cache = p["q"].clone(), p["cache"].clone()
    for t in {0, n // 2 if n > 3 else 0, n - 1}:
        q[t] = bad
        lse[t] = -np.inf
    q[n + 1, 3] = bad
    lse[n + 1, 3] = -np.inf
    if opt.get("causal", True):
        t = int(p["lens"][0]) - 1
        cache[p["table"][0, t // 16], :, t % 16] = float("nan")
    want, err = ref.key_weights(p["qv"], p["cv"], p["table"], p["lens"], p["starts"], lse.astype(np.float64), p["scale"], **opt)
    p["q"] = q
    close(call(p, lse, cache=cache, **opt), want, err, p["lens"])


def test_parts_of_split_tokens_are_joined_from_what_other_ctas_wrote():
    """Six parts of a block's tokens, whose place in the workspace holds NaN before every call: the
    same bits each time, and the workspace ready for the next call."""
    p = problem(13, new=[700], lens=[1000], heads=8, kv=2, dim=64, page=16, dtype="bf16")
    lse = lses(p)
    want, err = ref.key_weights(p["qv"], p["cv"], p["table"], p["lens"], p["starts"], lse.astype(np.float64), p["scale"])
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    args = (p["q"].cuda(), p["cache"].cuda(), dev(p["table"]), dev(p["lens"]), dev(p["starts"]), dev(lse), p["scale"])
    good = pkd.key_weights(*args, workspace=ws)
    close(good, want, err, p["lens"])
    for _ in range(200):
        ws[256 + 4 * 65536:] = 255
        assert torch.equal(pkd.key_weights(*args, workspace=ws), good)
    assert pkd.workspace_check(ws) == pkd.OK and not ws[256:256 + 4 * 65536].any()


@pytest.mark.parametrize("softcap", [0.0, 5.0])
@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("name", PLANS)
def test_bad_pages_and_lengths_on_every_plan(name, dtype, softcap):
    """Keys on a page outside the pool receive nothing (their earlier weights stay), a length
    behind the table is clamped, and the status says so; in place."""
    p = plan(name, 2, dtype=dtype)
    lse = lses(p, softcap=softcap)
    table, lens = p["table"].copy(), p["lens"].copy()
    columns = table.shape[1]
    table[0, 1], table[0, 12], table[1, 13], table[1, 0] = 10 ** 6, p["cache"].shape[0], -1, -2 ** 31
    table[1, 14:] = p["table"][0, 14:]  # (the clamped length reaches them)
    lens[1] = columns * 16 + 900
    prior = np.random.default_rng(3).random((2, 2, columns * 16)).astype(np.float32)
    want, err = ref.key_weights(p["qv"], p["cv"], table, np.minimum(lens, columns * 16), p["starts"], lse.astype(np.float64),
                                p["scale"], prior=prior.astype(np.float64), decay=0.5, softcap=softcap)
    ws, w = torch.zeros(1 << 24, dtype=torch.uint8, device="cuda"), dev(prior)
    got = call(p, lse, table=table, lens=lens, weights=w, out=w, decay=0.5, softcap=softcap, workspace=ws)
    assert got is w
    assert pkd.workspace_check(ws) == pkd.EDEVICE_BOUNDS and pkd.workspace_check(ws) == pkd.OK
    close(got, want, err, np.minimum(lens, columns * 16))
    for b, x in ((0, 1), (0, 12), (1, 13), (1, 0)):  # (none of the call's own tokens' keys, but for the last plan's)
        keys = np.arange(16 * x, 16 * x + 16)
        old = keys < min(lens[b], columns * 16) - int(p["starts"][b + 1] - p["starts"][b])
        bits = np.where(old, prior[b][:, keys] * np.float32(0.5), np.float32(0))
        assert np.array_equal(got[b][:, keys].cpu().numpy(), bits)
    # the same workspace and no bad entry: no status, and the counters were left ready
    want, err = ref.key_weights(p["qv"], p["cv"], p["table"], p["lens"], p["starts"], lse.astype(np.float64), p["scale"],
                                softcap=softcap)
    close(call(p, lse, softcap=softcap, workspace=ws), want, err, p["lens"])
    assert pkd.workspace_check(ws) == pkd.OK


@pytest.mark.parametrize("name", PLANS)
def test_capped_weights_beside_a_bad_page_do_not_depend_on_what_ran_before(name):
    """Rows of keys that were not loaded hold what an earlier call left in shared memory: large
    values there change no bit of the other keys' weights."""
    p = plan(name, 4)
    lse = lses(p, softcap=5.0)
    table = p["table"].copy()
    table[0, 1], table[1, 5] = -1, 10 ** 6
    big = problem(5, new=[700], lens=[1400], heads=8, kv=2, dim=128, page=16, dtype="bf16", spread=30.0)
    good = None
    for huge in (0.0, 1.0, 50.0):
        cache = (big["cache"].float() * huge).to(torch.bfloat16).cuda()
        for _ in range(2):
            pkd.key_weights(big["q"].cuda(), cache, dev(big["table"]), dev(big["lens"]), dev(big["starts"]),
                            torch.zeros((700, 8), device="cuda"), big["scale"])
        got = call(p, lse, table=table, softcap=5.0)
        good = got if good is None else good
        assert torch.equal(got, good)


@pytest.mark.parametrize("window,softcap", [(60, 0.0), (60, 5.0), (0, 0.0)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("name", PLANS)
def test_hidden_values_on_every_plan(name, dtype, window, softcap):
    """NaN in V, in K of keys that no token sees and behind the length reaches nothing; those keys get 0."""
    p = plan(name, 6, dtype=dtype)
    lse = lses(p, window=window, softcap=softcap)
    want, err = ref.key_weights(p["qv"], p["cv"], p["table"], p["lens"], p["starts"], lse.astype(np.float64), p["scale"],
                                window=window, softcap=softcap)
    cache = p["cache"].clone()
    cache[..., 128:] = float("nan")
    for b, L in enumerate(p["lens"]):
        n = int(p["starts"][b + 1] - p["starts"][b])
        unseen = range(0, max(0, L - n - window + 1)) if window else ()
        for t in [*unseen, *range(L, -(-L // 16) * 16)]:
            cache[p["table"][b, t // 16], :, t % 16, :128] = float("nan")
    cache[list(set(range(len(cache))) - set(p["table"].ravel()))] = float("nan")
    got = call(p, lse, cache=cache, window=window, softcap=softcap)
    close(got, want, err, p["lens"])
    for b, L in enumerate(p["lens"]):
        n = int(p["starts"][b + 1] - p["starts"][b])
        if window:
            assert (got[b, :, :max(0, L - n - window + 1)] == 0).all()


@pytest.mark.parametrize("name", PLANS)
def test_weights_in_place_on_every_plan(name):
    """The earlier weights' own memory, rows of a larger pool: what lies behind the lengths and
    beside the rows stays."""
    p = plan(name, 7)
    S = p["table"].shape[1] * 16 + 5
    store = torch.full((2, 3, 2, S), 3.5, device="cuda")
    view = store[:, 1]
    view.copy_(torch.as_tensor(np.random.default_rng(8).random((2, 2, S)).astype(np.float32)))
    prior = view.cpu()
    lse = lses(p)
    want, err = ref.key_weights(p["qv"], p["cv"], p["table"], p["lens"], p["starts"], lse.astype(np.float64), p["scale"],
                                prior=prior.double().numpy(), decay=0.75)
    assert call(p, lse, weights=view, out=view, decay=0.75) is view
    close(view, want, err, p["lens"])
    for b, L in enumerate(p["lens"]):
        assert torch.equal(view[b, :, L:].cpu(), prior[b, :, L:])
    assert (store[:, 0] == 3.5).all() and (store[:, 2] == 3.5).all()


def wide(seed, *, most, lens, new, heads, kv, dim, dtype):
    """A problem whose lengths may be up to `most` (the step grid's chunk follows from it)."""
    return problem(seed, new=new, lens=lens, heads=heads, kv=kv, dim=dim, page=64, dtype=dtype, columns=-(-most // 64))


# kv heads, requests and the longest length: chunks of 512, 896 and 2048 keys a CTA
CHUNKS = {512: (8, 64, 4096), 896: (8, 4, 131072), 2048: (8, 8, 160000)}


@pytest.mark.parametrize("dtype,dim,group", [("bf16", 128, 1), ("bf16", 128, 4), ("fp16", 64, 7), ("fp8", 128, 8),
                                             ("fp8", 128, 16), ("bf16", 64, 12)])
@pytest.mark.parametrize("opt", [dict(), dict(softcap=5.0), dict(window=700)])
@pytest.mark.parametrize("chunk", CHUNKS)
def test_steps_of_long_chunks(chunk, opt, dtype, dim, group):
    """Many steps of a warp through its ring: pages far down a lane's share, earlier weights steps
    ahead, chunks that end between two warps' keys."""
    kv, B, most = CHUNKS[chunk]
    ends = [2 * chunk + 777, chunk + 1, 1, 3 * chunk - 17, chunk - 1, chunk, 0, 65]
    lens = [min(ends[b], most) if b < len(ends) else (b * 37) % 130 for b in range(B)]
    p = wide(9, most=most, lens=lens, new=[int(n > 0) for n in lens], heads=kv * group, kv=kv, dim=dim, dtype=dtype)
    lse = lses(p, **opt)
    prior = np.random.default_rng(10).random((B, kv, most)).astype(np.float32)
    ref_prior = np.zeros((B, kv, p["table"].shape[1] * 64))
    ref_prior[..., :most] = prior
    got, want, err = weigh_both(p, prior=None, lse=lse, max_query_len=1, max_kv_len=most, **opt)
    close(got, want, err, lens)
    want, err = ref.key_weights(p["qv"], p["cv"], p["table"], p["lens"], p["starts"], lse.astype(np.float64), p["scale"],
                                prior=ref_prior, decay=0.75, **opt)
    w = dev(prior)
    call(p, lse, weights=w, out=w, decay=0.75, max_kv_len=most, **opt)
    close(w, want, err, lens)
    for b, L in enumerate(lens):
        assert np.array_equal(w[b, :, L:].cpu().numpy(), prior[b, :, L:])


@pytest.mark.parametrize("dtype,dim,heads,kv", [("bf16", 128, 8, 2), ("fp16", 128, 4, 4), ("fp8", 128, 16, 4), ("bf16", 64, 10, 2),
                                                ("fp16", 64, 3, 1)])
@pytest.mark.parametrize("opt", [dict(softcap=5.0), dict(softcap=50.0, window=40), dict(causal=False), dict(causal=False, softcap=20.0),
                                 dict(causal=False, window=33)])
def test_steps_capped_and_not_causal(dtype, dim, heads, kv, opt):
    p = problem(11, new=[3, 1, 2, 3, 0], lens=[333, 1, 90, 2, 50], heads=heads, kv=kv, dim=dim, page=16, dtype=dtype, spread=4.0)
    prior = np.random.default_rng(12).random((5, kv, p["table"].shape[1] * 16)).astype(np.float32).astype(np.float64)
    got, want, err = weigh_both(p, prior=prior, decay=0.9, max_query_len=3, **opt)
    close(got, want, err, p["lens"])


def test_parts_of_a_wider_table_are_not_read_past_their_columns(monkeypatch):
    """Columns of a larger table, whose last row ends with the memory: max_kv_len for the larger one
    reaches the library as what the columns hold, and the weights are right."""
    p = problem(14, new=[1, 1, 1], lens=[60, 33, 64], heads=4, kv=2, dim=64, page=16, dtype="bf16")
    store = torch.full((3 * 8,), -5, dtype=torch.int32, device="cuda")
    table = store.as_strided((3, 4), (8, 1), 4)  # the last four columns of eight
    table.copy_(torch.as_tensor(p["table"]))
    lse = lses(p)
    args = (p["q"].cuda(), p["cache"].cuda(), table, dev(p["lens"]), dev(p["starts"]), dev(lse), p["scale"])
    lib, asked = pkd.load_library(), []

    class Recorder:
        def __getattr__(self, name):
            return (lambda *a: asked.append(a) or 0) if name == "pkd_key_weights" else getattr(lib, name)

    monkeypatch.setattr(pkd, "_lib", Recorder())
    pkd.key_weights(*args, max_query_len=1, max_kv_len=128)
    monkeypatch.undo()
    assert asked[0][18] == 64 and asked[0][7] == 8  # max_kv_len, the table's stride
    want, err = ref.key_weights(p["qv"], p["cv"], p["table"], p["lens"], p["starts"], lse.astype(np.float64), p["scale"])
    got = pkd.key_weights(*args, max_query_len=1, max_kv_len=128)
    assert got.shape == (3, 2, 128)
    close(got, want, err, p["lens"])
    with pytest.raises(pkd.PkdError, match="stride"):  # a table that does not have the columns
        pkd.key_weights(*args, max_query_len=1, max_kv_len=256)


def test_more_requests_than_runs_of_key_blocks():
    """Few rows of many short requests: runs end with a request's blocks."""
    rng = np.random.default_rng(15)
    new = rng.integers(0, 10, 180).tolist()
    lens = [n + int(rng.integers(0, 60)) for n in new]
    lens[7], lens[90] = 700, 300
    p = problem(16, new=new, lens=lens, heads=16, kv=8, dim=64, page=16, dtype="bf16")
    lse = lses(p)
    want, err = ref.key_weights(p["qv"], p["cv"], p["table"], p["lens"], p["starts"], lse.astype(np.float64), p["scale"])
    args = (p["q"].cuda(), p["cache"].cuda(), dev(p["table"]), dev(p["lens"]), dev(p["starts"]), dev(lse), p["scale"])
    got = pkd.key_weights(*args, max_query_len=9)
    close(got, want, err, lens)
    for most in (700, 704):  # the table's columns hold no more
        assert torch.equal(pkd.key_weights(*args, max_query_len=9, max_kv_len=most)[..., :700], got[..., :700])
