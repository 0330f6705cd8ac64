"""The status of calls without a workspace outlives the workspace kept for them, which grows."""
import numpy as np
import pytest
import torch

import paged_kv_decode_15_gb300 as pkd
from tests.test_cache_eviction_gpu import dev, problem

pytestmark = pytest.mark.gpu


def call(p, table=None, **kw):
    """Weights of keys; a workspace that grows with the tokens and kv heads."""
    T, Hq = p["q"].shape[:2]
    return pkd.key_weights(p["q"].cuda(), p["cache"].cuda(), dev(p["table"] if table is None else table), dev(p["lens"]),
                           dev(p["starts"]), torch.zeros((T, Hq), device="cuda"), p["scale"], **kw)


def test_a_status_is_reported_after_the_workspace_has_grown():
    small = problem(1, new=[1], lens=[40], heads=4, kv=2, dim=64, page=16, dtype="bf16")
    more = problem(2, new=[700], lens=[900], heads=8, kv=2, dim=64, page=16, dtype="bf16")
    most = problem(3, new=[1500], lens=[1500], heads=32, kv=8, dim=64, page=16, dtype="bf16")
    bad = np.full_like(small["table"], -1)
    with torch.cuda.stream(torch.cuda.Stream()):
        torch.cuda.synchronize()
        call(small, bad, max_query_len=1)
        call(more)
        call(most)
        assert pkd.workspace_check() == pkd.EDEVICE_BOUNDS and pkd.workspace_check() == pkd.OK
        call(most)
        assert pkd.workspace_check() == pkd.OK
    with torch.cuda.stream(torch.cuda.Stream()):  # the later of two that grew out of use
        call(small, max_query_len=1)
        bad = more["table"].copy()
        bad[0, 3] = 10 ** 6
        call(more, bad)
        call(most)
        assert pkd.workspace_check() == pkd.EDEVICE_BOUNDS and pkd.workspace_check() == pkd.OK
        call(more, bad)
        pkd.release_workspaces()
        assert pkd.workspace_check() == pkd.OK
