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
