"""The operators that bound a paged cache at their largest: pages and rows past 32 bits of offset, and
the most requests that a call takes."""
import numpy as np
import pytest
import torch

import paged_kv_decode_15_gb300 as pkd
from tests import eviction_ref as ref
from tests.test_cache_eviction_gpu import close, dev, problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def far():
    """Two requests' weights 2^31 values apart, in one allocation."""
    store = torch.zeros(2 ** 31 + 4 * 2048, device="cuda")
    yield store.as_strided((2, 4, 2048), (2 ** 31, 2048, 1))
    del store
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("new", [(1, 1), (40, 33), (300, 90)])
def test_pages_and_weights_past_32_bits(far, new, dtype):
    """The same bits as from a small cache and weights side by side: the steps of a server, one after the other."""
    p = problem(1, new=list(new), lens=[900, 650], heads=8, kv=4, dim=128, page=16, dtype=dtype)
    small, table = p["cache"].cuda(), dev(np.maximum(p["table"], 0))
    first = 2 ** 32 // (4 * 16 * 256) // small.element_size() + 5  # pages before 4 GiB
    cache = torch.zeros((first + len(small), *small.shape[1:]), dtype=torch.uint8 if dtype == "fp8" else small.dtype, device="cuda")
    cache[first:] = small.view(cache.dtype)
    cache = cache.view(small.dtype)
    q, lens, starts = p["q"].cuda(), dev(p["lens"]), dev(p["starts"])
    lse = torch.full(q.shape[:2], 5.0, device="cuda")
    prior = torch.rand((2, 4, 2048), device="cuda", generator=torch.Generator(device="cuda").manual_seed(2))
    far.copy_(prior)
    opt = dict(max_query_len=max(new), decay=0.5)
    near = prior.clone()
    pkd.key_weights(q, small, table, lens, starts, lse, p["scale"], weights=near, out=near, **opt)
    pkd.key_weights(q, cache, table + first, lens, starts, lse, p["scale"], weights=far, out=far, **opt)
    assert torch.equal(far, near)
    pos = torch.arange(2048, dtype=torch.int32, device="cuda").expand(2, 4, -1).contiguous()
    pos2 = pos.clone()
    kept, n = pkd.evict_select(near, lens, 500, sinks=2, recent=9, pool=3)
    got = pkd.evict_select(far, lens, 500, sinks=2, recent=9, pool=3)
    assert torch.equal(got[0], kept) and torch.equal(got[1], n)
    pkd.cache_compact(small, table, kept, n, weights=near, positions=pos)
    pkd.cache_compact(cache, table + first, kept, n, weights=far, positions=pos2)
    assert torch.equal(cache[first:].view(torch.uint8), small.view(torch.uint8))
    assert torch.equal(far, near) and torch.equal(pos, pos2)
    assert not cache[:first].view(torch.uint8).any()


def test_weights_of_the_most_requests():
    """2048 requests of more than 16 rows, and of one token each; one more is refused."""
    B = 2048
    rng = np.random.default_rng(3)
    lens = rng.integers(3, 40, B).tolist()
    lens[2047] = 300
    for new in (3, 1):
        p = problem(4, new=[new] * B, lens=lens, heads=8, kv=1, dim=64, page=16, dtype="bf16")
        lse = np.full((new * B, 8), 2.0, np.float32)
        want, err = ref.key_weights(p["qv"], p["cv"], p["table"], p["lens"], p["starts"], lse.astype(np.float64), p["scale"])
        args = [p["q"].cuda(), p["cache"].cuda(), dev(p["table"]), dev(p["lens"]), dev(p["starts"]), dev(lse), p["scale"]]
        close(pkd.key_weights(*args, max_query_len=new), want, err, lens)
    for i in (2, 3):
        args[i] = torch.cat([args[i], args[i][-1:]])
    args[4] = torch.cat([args[4], args[4][-1:]])
    with pytest.raises(pkd.PkdError, match="2049"):
        pkd.key_weights(*args, max_query_len=1)


def test_choice_and_compaction_of_the_most_requests():
    B, S, budget = 65535, 20, 12
    rng = np.random.default_rng(5)
    w = rng.random((B, 1, S)).astype(np.float32)
    lens = rng.integers(0, S + 1, B).astype(np.int32)
    kept, n = pkd.evict_select(dev(w), dev(lens), budget, recent=2)
    want = ref.evict_select(w, lens, budget, recent=2)
    assert np.array_equal(kept.cpu().numpy(), want[0]) and np.array_equal(n.cpu().numpy(), want[1])
    table = rng.permutation(2 * B).astype(np.int32).reshape(B, 2)
    bits = rng.integers(0, 256, (2 * B, 1, 16, 128), dtype=np.uint8)
    cache, dw = dev(bits), dev(w)
    pkd.cache_compact(cache, dev(table), kept, n, weights=dw)
    ref.cache_compact(bits, table, want[0], want[1], (w,))
    assert np.array_equal(cache.cpu().numpy(), bits) and np.array_equal(dw.cpu().numpy(), w)
    with pytest.raises(pkd.PkdError, match="65535"):
        pkd.evict_select(torch.zeros((65536, 1, 1), device="cuda"), torch.zeros(65536, dtype=torch.int32, device="cuda"), 1)


def test_choice_of_rows_past_32_bits():
    """130 rows of 2^24 keys, read again in every pass: the first rows and the last."""
    B, S, budget = 130, 1 << 24, 1000
    g = torch.Generator(device="cuda").manual_seed(6)
    w = torch.empty((B, 1, S), device="cuda").uniform_(generator=g)
    lens = torch.full((B,), S, dtype=torch.int32, device="cuda")
    lens[B - 1] = S - 12345
    kept, _ = pkd.evict_select(w, lens, budget, sinks=1, recent=3)
    for b in (0, 1, 127, 128, B - 1):
        L = int(lens[b])
        x = w[b, 0, :L].clone()
        x[0] = x[L - 3:] = torch.inf
        top = x.sort(descending=True, stable=True)[1][:budget].sort()[0]
        assert torch.equal(kept[b, 0].long(), top)
    del w
    torch.cuda.empty_cache()
