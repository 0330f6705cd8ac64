"""The timeout path of ragged attention and shared-prefix decode: with the diagnostic
flag every wait on a copy tests its barrier once, so copies still in flight count as
lost.  No copy is withheld and no wait is without a limit: the kernels let every copy
land, report PKD_ETIMEOUT through the status word and return."""
import numpy as np
import pytest
import torch

from tests import ragged_ref as ref
from tests.test_paged_attention_gpu import dev, slopes_of
from tests.test_prefix_decode_gpu import Shared

pytestmark = pytest.mark.gpu

HEAD = 256 + 4 * 65536  # PKD_ATTENTION_WORKSPACE_HEAD


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.fail("a CUDA GPU is required for -m gpu tests")
    import paged_kv_decode_15_gb300 as pkd
    pkd.build()
    pkd.load_library()


def until_timeout(pkd, ws, call):
    """A copy that lands before its first test is no timeout: a few tries, each with a
    cold L2 (256 MB written over it)."""
    for _ in range(8):
        torch.empty(1 << 28, dtype=torch.uint8, device="cuda").zero_()
        call()
        status = pkd.workspace_check(ws)
        if status != pkd.OK:
            break
    assert status == pkd.ETIMEOUT


CASES = {
    # steps; unsplit prompts; few rows whose keys are split and joined; with other types and masks
    "step": dict(lens=[3000, 700, 4000], news=[1, 1, 1], Hq=8, Hkv=2, D=128),
    "step fp8": dict(lens=[3000, 700, 4000], news=[2, 2, 1], Hq=8, Hkv=2, D=128, dtype="fp8"),
    "prompts": dict(lens=[210, 300], news=[210, 130], Hq=64, Hkv=32, D=64, dtype="fp16"),
    "split": dict(lens=[4000, 1024, 40], news=[20, 5, 40], Hq=8, Hkv=1, D=128),
    "split fp8": dict(lens=[4000, 1024, 40], news=[20, 5, 40], Hq=8, Hkv=2, D=128, dtype="fp8"),
    "split, two row tiles": dict(lens=[4000, 3000], news=[30, 28], Hq=8, Hkv=1, D=64),
}


@pytest.mark.parametrize("name", CASES)
@pytest.mark.parametrize("mod", ["plain", "cap+bias"])
def test_attention_reports_a_timeout_and_recovers(name, mod):
    import paged_kv_decode_15_gb300 as pkd
    c = ref.Paged(seed=51, **CASES[name])
    slopes = slopes_of(c.Hq) if mod != "plain" else None
    kw = dict(max_query_len=int(c.news.max()), softcap=0.0 if mod == "plain" else 20.0, alibi_slopes=dev(slopes, torch.float32),
              **c.scales())
    args = [dev(x) for x in (c.q, c.cache, c.table, c.lens, c.starts)]
    ws = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    pkd.workspace_init(ws)
    until_timeout(pkd, ws, lambda: pkd.paged_attention(*args, c.scale, workspace=ws, test_timeout=True, **kw))
    assert not ws[64:192].any(), "the item queues are at their start again"
    pkd.workspace_init(ws[:HEAD])   # as the header asks; the rest is written before it is read
    want = c.reference(softcap=kw["softcap"], slopes=slopes)
    for _ in range(2):
        out, lse = pkd.paged_attention(*args, c.scale, workspace=ws, **kw)
        assert pkd.workspace_check(ws) == pkd.OK
        ref.check(out.cpu(), lse.cpu(), want, c.dtype)


@pytest.mark.parametrize("sq,dtype", [(1, "bf16"), (6, "fp16"), (2, "fp8")])
def test_prefix_decode_reports_a_timeout_and_recovers(sq, dtype):
    import paged_kv_decode_15_gb300 as pkd
    s = Shared(prefixes=[1500, 300], group_start=[0, 4, 7], own=[100, 20, 300, 7, 64, 900, 33], sq=sq, Hq=8, Hkv=2, D=128,
               dtype=dtype, seed=52)
    c, P = s.c, s.c.P
    wide = -(-max(s.prefixes) // P), -(-int(s.own.max()) // P)
    args = [dev(c.q).view(s.B, sq, c.Hq, c.D), dev(c.cache), dev(c.table[:2, :wide[0]].copy()),
            dev(np.asarray(s.prefixes, np.int32)), dev(c.table[2:, :wide[1]].copy()), dev(s.own)]
    kw = dict(group_start=dev(s.group_start), **c.scales())
    ws = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    pkd.workspace_init(ws)
    until_timeout(pkd, ws, lambda: pkd.prefix_decode(*args, c.scale, workspace=ws, test_timeout=True, **kw))
    assert not ws[64:192].any(), "the item queues are at their start again"
    pkd.workspace_init(ws[:HEAD])
    want = s.reference()
    for _ in range(2):
        out, lse = pkd.prefix_decode(*args, c.scale, workspace=ws, **kw)
        assert pkd.workspace_check(ws) == pkd.OK
        ref.check(out.cpu().view(-1, c.Hq, c.D), lse.cpu().view(-1, c.Hq), want, dtype)
