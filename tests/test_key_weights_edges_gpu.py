"""Weights of keys where they can go wrong, on each plan of the kernels: the step grid, query
tiles that stay, query tiles that stream past (their tokens split)."""
import numpy as np
import pytest
import torch

import paged_kv_decode_15_gb300 as pkd
from tests import eviction_ref as ref
from tests import ragged_ref
from tests.test_cache_eviction_gpu import close, dev, problem

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
