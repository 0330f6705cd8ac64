"""Tables without columns: no prefix, no own keys, no keys at all."""
import numpy as np
import pytest
import torch

from tests import ragged_ref as ref
from tests.test_paged_attention_gpu import dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.fail("a CUDA GPU is required for -m gpu tests")
    import paged_kv_decode_15_gb300 as pkd
    pkd.build()
    pkd.load_library()


def none(rows):
    return torch.empty((rows, 0), dtype=torch.int32, device="cuda"), torch.zeros(rows, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("sq", [1, 9])
def test_shared_prefix_decode_with_one_part_empty(sq, dtype):
    import paged_kv_decode_15_gb300 as pkd
    c = ref.Paged(lens=[300, 40, 25, 60], news=[0, sq, sq, sq], Hq=8, Hkv=2, D=128, dtype=dtype, seed=71)
    q, cache, table, lens = dev(c.q).view(3, sq, 8, 128), dev(c.cache), dev(c.table), dev(c.lens)
    flat = lambda r: (r[0].cpu().view(-1, 8, 128), r[1].cpu().view(-1, 8))
    starts = np.arange(4) * sq

    def want(rows, lens, causal):
        return ref.attention(ref.values(c.q), np.nan_to_num(ref.values(c.cache)), c.table[rows], lens, starts, c.scale,
                             causal=causal, **c.scales())

    pkd.workspace_check()
    empty, zero = none(3)
    got = pkd.prefix_decode(q, cache, table[:1], lens[:1], empty, zero, c.scale, **c.scales())
    ref.check(*flat(got), want([0, 0, 0], [300] * 3, False), dtype, what="prefix alone")
    got = pkd.prefix_decode(q, cache, *none(1), table[1:], lens[1:], c.scale, causal=True, **c.scales())
    ref.check(*flat(got), want([1, 2, 3], c.lens[1:], True), dtype, what="own keys alone")
    out, lse = pkd.prefix_decode(q, cache, *none(1), empty, zero, c.scale, **c.scales())
    assert not out.any() and torch.isneginf(lse).all()
    assert pkd.workspace_check() == pkd.OK


@pytest.mark.parametrize("news", [[1, 2], [40, 30]])
def test_attention_over_no_keys_at_all(news):
    import paged_kv_decode_15_gb300 as pkd
    c = ref.Paged(lens=[40, 30], news=news, Hq=8, Hkv=2, D=64, seed=72)
    empty, zero = none(2)
    pkd.workspace_check()
    out, lse = pkd.paged_attention(dev(c.q), dev(c.cache), empty, zero, dev(c.starts), c.scale, max_query_len=max(news))
    assert not out.any() and torch.isneginf(lse).all() and pkd.workspace_check() == pkd.OK
    # a length that says otherwise is reported, and no table is read
    out, lse = pkd.paged_attention(dev(c.q), dev(c.cache), empty, zero + 5, dev(c.starts), c.scale, max_query_len=max(news))
    assert not out.any() and torch.isneginf(lse).all() and pkd.workspace_check() == pkd.EDEVICE_BOUNDS
