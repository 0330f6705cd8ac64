"""More refusals of the operators that bound a paged cache, without a GPU: calls that were taken
and gave wrong results or lost rows."""
import ctypes

import pytest

import paged_kv_decode_15_gb300 as pkd
from tests.test_eviction_boundary import compact, lib, select, weigh  # noqa: F401  (lib: a fixture)


def at(address):
    return ctypes.c_void_p(address)


# one call's arrays, far apart: 2 requests, 2 kv heads, 100 keys in rows of 200 and 100 values, budget 50
APART = dict(weights=at(1 << 20), lens=at(2 << 20), kept=at(3 << 20), kept_lens=at(4 << 20))
MOVED = dict(APART, positions=at(5 << 20), context=at(6 << 20))


@pytest.mark.parametrize("base,over,needle", [
    (APART, dict(kept_lens=at(2 << 20)), "overlaps weights, positions, seq_lens"),       # lengths that change under the readers
    (APART, dict(kept_lens=at((2 << 20) + 4)), "overlaps"), (APART, dict(kept_lens=at((2 << 20) - 4)), "overlaps"),
    (APART, dict(kept=at(1 << 20)), "overlaps"), (APART, dict(kept=at((1 << 20) + 4 * 399)), "overlaps"),
    (APART, dict(kept=at((1 << 20) - 4 * 199)), "overlaps"), (APART, dict(kept_lens=at((1 << 20) + 4 * 150)), "overlaps"),
    (APART, dict(kept=at((2 << 20) - 4 * 199)), "overlaps"), (APART, dict(kept_lens=at((3 << 20) + 4 * 199)), "kept overlaps kept_lens"),
    (MOVED, dict(kept=at(5 << 20)), "overlaps"), (MOVED, dict(kept_lens=at(6 << 20)), "overlaps")])
def test_select_refuses_results_that_lie_in_its_inputs(lib, base, over, needle):
    assert select(lib, **{**base, **over}) == pkd.EINVAL
    assert needle in lib.pkd_last_error().decode()


WRAP = (1 << 63) // 7 + 1  # seven such head strides are past 2^63, where a batch stride of 0 seemed to be enough


@pytest.mark.parametrize("call,over", [
    (weigh, dict(Hq=8, Hkv=8, q_stride=1024, wh=WRAP, wb=0)), (weigh, dict(wb=1 << 41)), (weigh, dict(wh=1 << 41, wb=1 << 42)),
    (weigh, dict(prior=at(1 << 20), pb=1 << 62)), (weigh, dict(prior=at(1 << 20), ph=(1 << 40) + 1)),
    (compact, dict(H=8, weights=at(1 << 20), wh=WRAP, wb=0)), (compact, dict(positions=at(1 << 20), pb=1 << 41)),
    (select, dict(APART, wb=1 << 41)), (select, dict(MOVED, ph=1 << 62))])
def test_strides_whose_sums_could_wrap_are_refused(lib, call, over):
    assert call(lib, **over) == pkd.EUNSUPPORTED
    assert "2^40" in lib.pkd_last_error().decode()


@pytest.mark.parametrize("over", [dict(weights=at(1 << 20), wkeys=0), dict(positions=at(1 << 20), pkeys=0),
                                  dict(weights=at(1 << 20), positions=at(2 << 20), pkeys=0)])
def test_compact_refuses_arrays_without_keys(lib, over):
    """No row could move with its values, and kept_lens would count rows that were not there."""
    assert compact(lib, **over) == pkd.EINVAL
    assert "must have keys" in lib.pkd_last_error().decode()


@pytest.mark.parametrize("ws,size", [(at((1 << 20) + 128), 1 << 20), (at(1 << 20), 255)])
def test_workspaces_of_choice_and_compaction_are_checked(lib, ws, size):
    a = dict(weights=at(1 << 20), wb=200, wh=100, keys=100, lens=at(2 << 20), B=2, H=2, budget=50, sinks=4, recent=16, pool=1,
             positions=None, pb=200, ph=100, context=None, kept=at(3 << 20), kept_lens=at(4 << 20), ws=ws, size=size, stream=None)
    assert lib.pkd_evict_select_checked(*a.values()) == pkd.EINVAL and "workspace" in lib.pkd_last_error().decode()
    a = dict(cache=at(1 << 20), kv_dt=pkd.BF16, num_pages=8, table=at(2 << 20), stride=8, columns=8, kept=at(3 << 20),
             kept_lens=at(4 << 20), B=2, H=2, D=128, P=16, budget=50, weights=None, wb=256, wh=128, wkeys=128, positions=None,
             pb=256, ph=128, pkeys=128, ws=ws, size=size, stream=None)
    assert lib.pkd_cache_compact_checked(*a.values()) == pkd.EINVAL and "workspace" in lib.pkd_last_error().decode()
