"""The workspaces that the binding keeps for calls without one: their status can be
read, and a timeout does not spoil the calls after it."""
import threading

import pytest
import torch

from tests import ragged_ref as ref
from tests.test_attention_timeouts_gpu import CASES, until_timeout
from tests.test_paged_attention_gpu import dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.fail("a CUDA GPU is required for -m gpu tests")
    import paged_kv_decode_15_gb300 as pkd
    pkd.build()
    pkd.load_library()


def call_of(pkd, c):
    args = [dev(x) for x in (c.q, c.cache, c.table, c.lens, c.starts)]
    return lambda **kw: pkd.paged_attention(*args, c.scale, max_query_len=int(c.news.max()), **c.scales(), **kw)


def test_no_call_no_status():
    import paged_kv_decode_15_gb300 as pkd
    assert pkd.workspace_check(stream=torch.cuda.Stream()) == pkd.OK


@pytest.mark.parametrize("news", [[1, 1], [70, 40]])
def test_a_bad_page_is_reported_without_a_workspace(news):
    import paged_kv_decode_15_gb300 as pkd
    good = ref.Paged(lens=[100, 90], news=news, Hq=4, Hkv=2, D=128, seed=11)
    bad = ref.Paged(lens=[100, 90], news=news, Hq=4, Hkv=2, D=128, seed=11)
    bad.table[0, 2] = -1
    pkd.workspace_check()
    call_of(pkd, good)()
    assert pkd.workspace_check() == pkd.OK
    call_of(pkd, bad)()
    assert pkd.workspace_check() == pkd.EDEVICE_BOUNDS
    assert pkd.workspace_check() == pkd.OK, "read once, cleared"
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call_of(pkd, bad)(stream=side)
    assert pkd.workspace_check() == pkd.OK, "each stream has its own"
    assert pkd.workspace_check(stream=side) == pkd.EDEVICE_BOUNDS
    seen = []
    worker = threading.Thread(target=lambda: (call_of(pkd, bad)(), seen.append(pkd.workspace_check())))
    worker.start()
    worker.join()
    assert seen == [pkd.EDEVICE_BOUNDS] and pkd.workspace_check() == pkd.OK, "and each thread"


def test_a_bad_page_of_shared_prefix_decode_is_reported():
    import paged_kv_decode_15_gb300 as pkd
    c = ref.Paged(lens=[64, 20, 30], news=[0, 1, 1], Hq=4, Hkv=2, D=128, seed=12)
    table = c.table.copy()
    table[0, 1] = c.num_pages
    pkd.workspace_check()
    pkd.prefix_decode(dev(c.q).view(2, 1, 4, 128), dev(c.cache), dev(table[:1]), dev(c.lens[:1]), dev(table[1:]),
                      dev(c.lens[1:]), c.scale)
    assert pkd.workspace_check() == pkd.EDEVICE_BOUNDS


@pytest.mark.parametrize("name", ["step", "prompts", "split"])
def test_calls_after_a_timeout_are_right(name):
    import paged_kv_decode_15_gb300 as pkd
    c = ref.Paged(seed=53, **CASES[name])
    call = call_of(pkd, c)
    pkd.workspace_check()
    until_timeout(pkd, None, lambda: call(test_timeout=True))
    want = c.reference()
    for _ in range(2):
        out, lse = call()
        ref.check(out.cpu(), lse.cpu(), want, c.dtype)
    assert pkd.workspace_check() == pkd.OK


def test_kept_workspaces_are_freed():
    """One a stream and thread while the thread lives, and none afterwards."""
    import paged_kv_decode_15_gb300 as pkd
    c = ref.Paged(lens=[4000, 3000], news=[30, 28], Hq=8, Hkv=1, D=64, seed=54)   # split keys: partial results
    call = call_of(pkd, c)
    streams = [torch.cuda.Stream() for _ in range(4)]
    want = call()
    torch.cuda.synchronize()

    def work():
        for s in streams:
            call(stream=s)
        torch.cuda.synchronize()

    work()
    pkd.release_workspaces()
    before = torch.cuda.memory_allocated()
    for _ in range(5):
        worker = threading.Thread(target=work)
        worker.start()
        worker.join()
    assert torch.cuda.memory_allocated() == before, "workspaces outlived their threads"
    call()
    assert torch.cuda.memory_allocated() > before, "a call keeps its workspace"
    pkd.release_workspaces()
    assert torch.cuda.memory_allocated() == before
    again = call()
    assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])


def test_a_workspace_released_while_its_calls_are_queued():
    """Its memory is used again in the order of its stream only."""
    import paged_kv_decode_15_gb300 as pkd
    c = ref.Paged(lens=[4000, 3000], news=[30, 28], Hq=8, Hkv=1, D=64, seed=55)
    call = call_of(pkd, c)
    want = call()
    got = []
    for _ in range(20):
        got.append(call())
        pkd.release_workspaces()
        torch.empty(1 << 22, dtype=torch.uint8, device="cuda").fill_(255)
    for g in got:
        assert torch.equal(g[0], want[0]) and torch.equal(g[1], want[1])
