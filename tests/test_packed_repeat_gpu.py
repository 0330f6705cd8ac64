"""Attention over packed prompts repeats itself bit for bit: whichever CTA takes an item, whatever
ran before, on two streams at once and in a graph."""
import numpy as np
import pytest
import torch

import paged_kv_decode_15_gb300 as pkd

pytestmark = pytest.mark.gpu


def prompts(seed, new, keys, Hq, Hkv, D, dtype, spread=3.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    starts = [torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device="cuda") for n in (new, keys)]
    q = (spread * torch.randn((sum(new), Hq, D), device="cuda", generator=g)).to(dtype)
    kv = torch.randn((sum(keys), 2 * Hkv, D), device="cuda", generator=g).to(dtype)
    return dict(q=q, k=kv[:, :Hkv], v=kv[:, Hkv:], query_start=starts[0], key_start=starts[1], scale=D ** -0.5,
                max_query_len=max(new), max_kv_len=max(keys))


CASES = {
    "many items": (dict(new=[700, 3, 511, 129, 640, 1, 257, 384], keys=[700, 3, 511, 129, 640, 1, 257, 384], Hq=32, Hkv=8, D=128,
                        dtype=torch.bfloat16), dict()),
    "capped, window": (dict(new=[700, 90, 511, 129], keys=[900, 90, 1511, 129], Hq=16, Hkv=2, D=128, dtype=torch.bfloat16),
                       dict(softcap=20.0, window=200)),
    "split keys": (dict(new=[60, 2], keys=[9000, 5000], Hq=8, Hkv=2, D=64, dtype=torch.float16), dict()),
    "not causal": (dict(new=[300, 77], keys=[300, 1077], Hq=28, Hkv=4, D=64, dtype=torch.float16), dict(causal=False)),
}


@pytest.mark.parametrize("name", CASES)
def test_packed_attention_repeats_bit_for_bit(name):
    shape, opt = CASES[name]
    p = prompts(1, **shape)
    big = prompts(2, new=[900], keys=[2000], Hq=16, Hkv=2, D=shape["D"], dtype=shape["dtype"], spread=100.0)
    good = pkd.packed_attention(**p, **opt)

    def same(got):
        assert torch.equal(got[0], good[0]) and torch.equal(got[1], good[1])

    for _ in range(10):
        pkd.packed_attention(**big)  # (large values stay in shared memory)
        same(pkd.packed_attention(**p, **opt))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured = pkd.packed_attention(**p, **opt)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [pkd.packed_attention(**p, **opt, stream=s) for s in streams]
        with torch.cuda.stream(streams[0]):
            g.replay()
        torch.cuda.synchronize()
        for x in (*got, captured):
            same(x)
    assert all(pkd.workspace_check(stream=s) == pkd.OK for s in streams)
