"""Uses of the serving operators in forms of their own: a distance bias over keys behind
the position, the rotary append captured, on other streams and into a cache whose slots
pass 31 bits."""
import numpy as np
import pytest
import torch

from tests import ragged_ref as ref
from tests.test_paged_attention_gpu import dev, slopes_of, verify
from tests.test_rope_cache_write_gpu import problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.fail("a CUDA GPU is required for -m gpu tests")
    import paged_kv_decode_15_gb300 as pkd
    pkd.build()
    pkd.load_library()


# ------------------------------------- a distance bias over keys behind the position
@pytest.mark.parametrize("dtype,Hq,Hkv,D", [("bf16", 8, 2, 128), ("fp16", 4, 4, 64), ("fp8", 8, 2, 128)])
@pytest.mark.parametrize("cap", [0.0, 5.0])
@pytest.mark.parametrize("kind", ["dense", "dense window", "prefix", "documents"])
def test_a_bias_behind_the_position(dtype, Hq, Hkv, D, cap, kind):
    lens = [333, 200, 17, 400]
    for news in ([2, 1, 2, 1], [300, 130, 17, 257]):
        if D == 64:
            news = [2 * n if n < 3 else n for n in news]
        c = ref.Paged(lens=lens, news=news, Hq=Hq, Hkv=Hkv, D=D, dtype=dtype, seed=81)
        kw = dict(slopes=4 * slopes_of(Hq), softcap=cap)
        if kind.startswith("dense"):
            kw["causal"] = False
        if kind == "dense window":
            kw["window"] = 50
        if kind == "prefix":
            kw["prefix_lens"] = [320, 90, 17, 399]
        if kind == "documents":
            kw.update(causal=False, doc_start=np.random.default_rng(82).integers(0, 300, c.T))
        verify(c, f"{kind} {news}", **kw)


def test_a_bias_behind_the_position_in_split_keys():
    c = ref.Paged(lens=[3000, 1024, 40], news=[20, 5, 40], Hq=8, Hkv=1, D=128, seed=83)
    verify(c, "prefix", prefix_lens=[2995, 1000, 11], slopes=slopes_of(8))
    verify(c, "dense", causal=False, slopes=slopes_of(8), softcap=20.0)


# ------------------------------------------------------------- the rotary append
def parts(qkv):
    return qkv[:, :4], qkv[:, 4:6], qkv[:, 6:]


def test_rotary_append_on_other_streams():
    import paged_kv_decode_15_gb300 as pkd
    qkv, table, pos, slots, pages, _ = problem(130, 4, 2, 128, 16, 128, "bf16", 84)
    d, rest = qkv.cuda(), [x.cuda() for x in (pos, table, slots)]
    pools = [torch.zeros(pages, 2, 16, 256, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    want = pkd.rope_cache_write(*parts(d), *rest, pools[0])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    given = pkd.rope_cache_write(*parts(d), *rest, pools[1], stream=side)
    with torch.cuda.stream(torch.cuda.Stream()):
        current = pkd.rope_cache_write(*parts(d), *rest, pools[2])
    torch.cuda.synchronize()
    for q, pool in ((given, pools[1]), (current, pools[2])):
        assert torch.equal(q, want) and torch.equal(pool, pools[0])


def test_rotary_append_captured_and_replayed():
    """Replayed on new tokens, positions and slots; tokens of no slot leave the cache alone."""
    import paged_kv_decode_15_gb300 as pkd
    qkv, table, pos, slots, pages, rng = problem(64, 4, 2, 128, 16, 64, "fp16", 85)
    other, _, pos2, _, _, _ = problem(64, 4, 2, 128, 16, 64, "fp16", 86)
    slots2 = torch.from_numpy(rng.permutation(pages * 16)[:64].astype(np.int64))
    slots2[::5] = -1
    empty = lambda: torch.zeros(pages, 2, 16, 256, dtype=torch.float8_e4m3fn, device="cuda")
    kw = dict(k_scale=0.02, v_scale=0.01, interleaved=True)
    expected = []
    for x, p, s in ((qkv, pos, slots), (other, pos2, slots2)):
        pool = empty()
        expected.append((pkd.rope_cache_write(*parts(x.cuda()), p.cuda(), table.cuda(), s.cuda(), pool, **kw), pool))
    d, p, t, s, pool = qkv.cuda(), pos.cuda(), table.cuda(), slots.cuda(), empty()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q = pkd.rope_cache_write(*parts(d), p, t, s, pool, **kw)
    for x, new in ((0, (qkv, pos, slots)), (1, (other, pos2, slots2))):
        for dst, src in zip((d, p, s), new):
            dst.copy_(src)
        pool.zero_()
        q.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(q, expected[x][0]) and torch.equal(pool.view(torch.uint8), expected[x][1].view(torch.uint8))


@pytest.mark.parametrize("P", [16, 48])
def test_rotary_append_to_a_cache_of_more_slots_than_31_bits(P):
    """The slot's page is found by a 64-bit division there.  The cache is said to have the
    slots; those used lie in its first pages, the only ones that there are."""
    import paged_kv_decode_15_gb300 as pkd
    qkv, table, pos, slots, pages, _ = problem(100, 4, 2, 64, P, 64, "bf16", 87)
    d, p, t, s = qkv.cuda(), pos.cuda(), table.cuda(), slots.cuda()
    a, b = (torch.zeros(pages, 2, P, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    want = pkd.rope_cache_write(*parts(d), p, t, s, a)
    got = torch.empty_like(want)
    many = 2 ** 31 // P + 1
    row = 8 * 64
    status = pkd.load_library().pkd_rope_cache_write(
        d.data_ptr(), row, d[:, 4:].data_ptr(), row, d[:, 6:].data_ptr(), row, pkd.BF16, p.data_ptr(), t.data_ptr(),
        t.shape[0], 64, 0, s.data_ptr(), 100, 4, 2, 64, P, many, b.data_ptr(), pkd.BF16, 1.0, 1.0, got.data_ptr(), 4 * 64,
        pkd.BF16, 1.0, torch.cuda.current_stream().cuda_stream)
    assert status == pkd.OK
    assert torch.equal(got, want) and torch.equal(a, b) and a.any()
