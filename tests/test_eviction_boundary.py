"""Refusals of the operators that bound a paged cache, without a GPU: status codes and
messages come before any CUDA call."""
import ctypes

import pytest
import torch

import paged_kv_decode_15_gb300 as pkd

FAKE = ctypes.c_void_p(0x10000)  # aligned, never read: every call here is refused first
FAR = ctypes.c_void_p(1 << 40)
ODD = ctypes.c_void_p(0x10002)


@pytest.fixture(scope="module")
def lib():
    pkd.build()
    return pkd.load_library()


def packed(lib, **over):
    a = dict(q=FAKE, qs=512, k=FAKE, ks=256, v=FAKE, vs=256, dt=pkd.BF16, starts=FAKE, key_start=None, B=2, T=20, Tk=20, max_q=16,
             max_kv=16, Hq=4, Hkv=2, D=128, scale=0.1, softcap=0.0, window=0, out=FAR, out_dt=pkd.BF16, lse=None, ws=FAKE,
             ws_bytes=1 << 40, flags=pkd.FLAG_CAUSAL, stream=None)
    a.update(over)
    return lib.pkd_packed_attention(*a.values())


@pytest.mark.parametrize("over,code,needle", [
    (dict(Hq=5), pkd.EUNSUPPORTED, "multiple of num_kv_heads"), (dict(D=96), pkd.EUNSUPPORTED, "head_dim"),
    (dict(dt=pkd.FP8_E4M3), pkd.EUNSUPPORTED, "dtype"), (dict(dt=pkd.FP32), pkd.EUNSUPPORTED, "dtype"),
    (dict(Tk=21), pkd.EINVAL, "key_start"), (dict(Tk=-1), pkd.EINVAL, "total_keys"), (dict(Tk=(1 << 29) + 1), pkd.EINVAL, "total_keys"),
    (dict(q=None), pkd.EINVAL, "null"), (dict(k=None), pkd.EINVAL, "null"), (dict(v=None), pkd.EINVAL, "null"),
    (dict(v=ODD), pkd.EINVAL, "misaligned"), (dict(ks=252), pkd.EINVAL, "k_stride"), (dict(vs=260), pkd.EINVAL, "v_stride"),
    (dict(vs=1 << 39), pkd.EINVAL, "2^38"), (dict(qs=511), pkd.EINVAL, "q_stride"), (dict(starts=None), pkd.EINVAL, "query_start"),
    (dict(key_start=ODD), pkd.EINVAL, "misaligned"), (dict(max_q=0), pkd.EINVAL, "max_query_len"),
    (dict(max_kv=-1), pkd.EINVAL, "max_kv_len"), (dict(out=FAKE), pkd.EINVAL, "overlaps q"),
    (dict(out=FAKE, q=FAR), pkd.EINVAL, "overlaps k"), (dict(out=FAKE, q=FAR, k=FAR), pkd.EINVAL, "overlaps v"),
    (dict(softcap=-1.0), pkd.EINVAL, "softcap"), (dict(scale=-1.0), pkd.EINVAL, "scale"), (dict(ws_bytes=100), pkd.EINVAL, "workspace"),
    (dict(out_dt=pkd.FP8_E4M3), pkd.EUNSUPPORTED, "out dtype"), (dict(flags=8), pkd.EUNSUPPORTED, "PKD_FLAG_CAUSAL")])
def test_packed_refusals(lib, over, code, needle):
    assert packed(lib, **over) == code
    assert needle in lib.pkd_last_error().decode()


def test_packed_calls_without_rows_are_ok(lib):
    assert packed(lib, B=0) == pkd.OK
    assert packed(lib, T=0, Tk=0, max_q=0, q=None, k=None, v=None) == pkd.OK


def weigh(lib, **over):
    a = dict(q=FAKE, q_dt=pkd.BF16, q_stride=512, cache=FAKE, kv_dt=pkd.BF16, num_pages=8, table=FAKE, stride=8, lens=FAKE,
             starts=FAKE, B=2, T=20, max_q=16, last=0, Hq=4, Hkv=2, D=128, P=16, max_kv=100, scale=0.1, qs=1.0, ks=1.0,
             softcap=0.0, window=0, lse=FAKE, prior=None, pb=200, ph=100, decay=1.0, weights=FAR, wb=200, wh=100, ws=FAKE,
             ws_bytes=1 << 40, flags=pkd.FLAG_CAUSAL, stream=None)
    a.update(over)
    return lib.pkd_key_weights(*a.values())


@pytest.mark.parametrize("over,code,needle", [
    (dict(Hq=5), pkd.EUNSUPPORTED, "multiple of num_kv_heads"), (dict(D=96), pkd.EUNSUPPORTED, "head_dim"),
    (dict(P=8), pkd.EUNSUPPORTED, "page_size"), (dict(kv_dt=pkd.FP32), pkd.EUNSUPPORTED, "kv dtype"),
    (dict(q_dt=pkd.FP16), pkd.EUNSUPPORTED, "q dtype"), (dict(q=None), pkd.EINVAL, "null"),
    (dict(weights=None), pkd.EINVAL, "null"), (dict(lse=None), pkd.EINVAL, "null"), (dict(starts=None), pkd.EINVAL, "query_start"),
    (dict(weights=ODD), pkd.EINVAL, "4-byte"), (dict(last=-1), pkd.EINVAL, "last_queries"),
    (dict(decay=float("nan")), pkd.EINVAL, "decay"), (dict(decay=float("inf")), pkd.EINVAL, "decay"),
    (dict(wh=99), pkd.EINVAL, "overlap"), (dict(wb=150), pkd.EINVAL, "overlap"), (dict(wh=-100), pkd.EINVAL, "overlap"),
    (dict(prior=FAKE, ph=-1), pkd.EINVAL, "negative"), (dict(prior=ctypes.c_void_p((1 << 40) + 4)), pkd.EINVAL, "overlaps prior"),
    (dict(prior=FAR, ph=101), pkd.EINVAL, "overlaps prior"), (dict(softcap=-1.0), pkd.EINVAL, "softcap"),
    (dict(scale=0.0), pkd.EINVAL, "scale"), (dict(stride=6), pkd.EINVAL, "stride"), (dict(ws_bytes=100), pkd.EINVAL, "workspace"),
    (dict(q_stride=511), pkd.EINVAL, "q_stride"), (dict(max_q=0), pkd.EINVAL, "max_query_len"),
    (dict(flags=2), pkd.EUNSUPPORTED, "PKD_FLAG_CAUSAL"), (dict(max_kv=(1 << 29) + 1), pkd.EUNSUPPORTED, "2^29")])
def test_weigh_refusals(lib, over, code, needle):
    assert weigh(lib, **over) == code
    assert needle in lib.pkd_last_error().decode()


def test_empty_weigh_calls_are_ok(lib):
    assert weigh(lib, B=0) == pkd.OK
    assert weigh(lib, max_kv=0) == pkd.OK


def select(lib, **over):
    a = dict(weights=FAKE, wb=200, wh=100, keys=100, lens=FAKE, B=2, H=2, budget=50, sinks=4, recent=16, pool=1, positions=None,
             pb=200, ph=100, context=None, kept=FAKE, kept_lens=FAKE, stream=None)
    a.update(over)
    return lib.pkd_evict_select(*a.values())


@pytest.mark.parametrize("over,code,needle", [
    (dict(budget=0), pkd.EINVAL, "budget"), (dict(sinks=40), pkd.EINVAL, "within the budget"), (dict(sinks=-1), pkd.EINVAL, "sinks"),
    (dict(recent=(1 << 31) - 1, sinks=10), pkd.EINVAL, "within the budget"), (dict(pool=2), pkd.EINVAL, "pool"),
    (dict(pool=0), pkd.EINVAL, "pool"), (dict(pool=257), pkd.EINVAL, "pool"), (dict(positions=FAKE), pkd.EINVAL, "together"),
    (dict(context=FAKE), pkd.EINVAL, "together"), (dict(positions=FAKE, context=FAKE, pool=3), pkd.EUNSUPPORTED, "pool"),
    (dict(weights=None), pkd.EINVAL, "null"), (dict(kept=None), pkd.EINVAL, "null"), (dict(lens=None), pkd.EINVAL, "null"),
    (dict(weights=ODD), pkd.EINVAL, "4-byte"), (dict(kept=ODD), pkd.EINVAL, "misaligned"), (dict(wh=-1), pkd.EINVAL, "strides"),
    (dict(keys=(1 << 29) + 1), pkd.EUNSUPPORTED, "2^29"), (dict(B=70000), pkd.EUNSUPPORTED, "65535"), (dict(B=-1), pkd.EINVAL, "shape")])
def test_select_refusals(lib, over, code, needle):
    assert select(lib, **over) == code
    assert needle in lib.pkd_last_error().decode()


def compact(lib, **over):
    a = dict(cache=FAKE, kv_dt=pkd.BF16, num_pages=8, table=FAKE, stride=8, columns=8, kept=FAKE, kept_lens=FAKE, B=2, H=2, D=128,
             P=16, budget=50, weights=None, wb=256, wh=128, wkeys=128, positions=None, pb=256, ph=128, pkeys=128, stream=None)
    a.update(over)
    return lib.pkd_cache_compact(*a.values())


@pytest.mark.parametrize("over,code,needle", [
    (dict(budget=0), pkd.EINVAL, "budget"), (dict(D=96), pkd.EUNSUPPORTED, "head_dim"), (dict(kv_dt=pkd.FP32), pkd.EUNSUPPORTED, "kv dtype"),
    (dict(P=0), pkd.EINVAL, "page_size"), (dict(num_pages=0), pkd.EINVAL, "num_pages"), (dict(columns=-1), pkd.EINVAL, "columns"),
    (dict(cache=None), pkd.EINVAL, "null"), (dict(kept=None), pkd.EINVAL, "null"), (dict(table=None), pkd.EINVAL, "null"),
    (dict(cache=ODD), pkd.EINVAL, "misaligned"), (dict(stride=7), pkd.EINVAL, "stride"),
    (dict(num_pages=1 << 40), pkd.EUNSUPPORTED, "2^31"), (dict(weights=FAKE, wh=100), pkd.EINVAL, "weights strides"),
    (dict(positions=FAKE, pb=0), pkd.EINVAL, "positions strides"), (dict(weights=ODD), pkd.EINVAL, "4-byte"),
    (dict(weights=FAKE, wkeys=-1), pkd.EINVAL, "negative")])
def test_compact_refusals(lib, over, code, needle):
    assert compact(lib, **over) == code
    assert needle in lib.pkd_last_error().decode()


def test_calls_of_no_requests_are_ok(lib):
    assert select(lib, B=0, weights=None, lens=None, kept=None, kept_lens=None) == pkd.OK
    assert compact(lib, B=0, cache=None, kept=None, kept_lens=None) == pkd.OK


def test_the_binding_wants_cuda_tensors():
    w, n = torch.zeros(1, 1, 4), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        pkd.evict_select(w, n, 2)
    with pytest.raises(ValueError, match="CUDA"):
        pkd.cache_compact(torch.zeros(1, 1, 16, 128), torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, 1, 2), n)
    with pytest.raises(ValueError, match="CUDA"):
        pkd.key_weights(torch.zeros(1, 1, 64), torch.zeros(1, 1, 16, 128), torch.zeros(1, 1, dtype=torch.int32), n,
                        torch.zeros(2, dtype=torch.int32), torch.zeros(1, 1), 1.0)
