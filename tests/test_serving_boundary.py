"""Refusals and plans of the serving operators, without a GPU: status codes and
messages come before any CUDA call."""
import ctypes

import pytest

import paged_kv_decode_15_gb300 as pkd

FAKE = ctypes.c_void_p(0x10000)  # aligned, never read: every call here is refused first


@pytest.fixture(scope="module")
def lib():
    pkd.build()
    return pkd.load_library()


def rope(lib, **over):
    a = dict(q=FAKE, q_stride=512, key=FAKE, key_stride=256, value=FAKE, value_stride=256, in_dtype=pkd.BF16,
             positions=FAKE, cos_sin=FAKE, max_position=64, rotary_dim=128, interleaved=0, slots=FAKE, T=4, Hq=4, Hkv=2,
             D=128, P=16, num_pages=8, cache=FAKE, kv_dtype=pkd.BF16, k_scale=1.0, v_scale=1.0,
             q_out=ctypes.c_void_p(0x20000), q_out_stride=512, q_dt=pkd.BF16, q_scale=1.0, stream=None)
    a.update(over)
    return lib.pkd_rope_cache_write(*a.values())


@pytest.mark.parametrize("over,code,needle", [
    (dict(D=96), pkd.EUNSUPPORTED, "head_dim"), (dict(rotary_dim=24), pkd.EUNSUPPORTED, "rotary_dim"),
    (dict(rotary_dim=144), pkd.EUNSUPPORTED, "rotary_dim"), (dict(in_dtype=pkd.FP32), pkd.EUNSUPPORTED, "dtype"),
    (dict(kv_dtype=pkd.FP16), pkd.EUNSUPPORTED, "cache dtype"), (dict(q_dt=pkd.FP16), pkd.EUNSUPPORTED, "q_out dtype"),
    (dict(q_stride=511), pkd.EINVAL, "stride"), (dict(key_stride=260), pkd.EINVAL, "stride"),
    (dict(kv_dtype=pkd.FP8_E4M3, k_scale=0.0), pkd.EINVAL, "scale"),
    (dict(q_dt=pkd.FP8_E4M3, q_scale=float("nan")), pkd.EINVAL, "q_scale"), (dict(key=None), pkd.EINVAL, "null"),
    (dict(q_out=None), pkd.EINVAL, "null"), (dict(cos_sin=ctypes.c_void_p(0x10004)), pkd.EINVAL, "aligned"),
    (dict(T=-1), pkd.EINVAL, "shape"), (dict(q_out=FAKE, q_dt=pkd.FP8_E4M3), pkd.EINVAL, "q itself"),
    (dict(q_out=FAKE, q_out_stride=1024), pkd.EINVAL, "q itself")])
def test_rope_refusals(lib, over, code, needle):
    assert rope(lib, **over) == code
    assert needle in lib.pkd_last_error().decode()


def test_rope_of_no_tokens_is_ok(lib):
    assert rope(lib, T=0, q=None, key=None, value=None, positions=None, slots=None, cache=None, q_out=None) == pkd.OK


def attend(lib, opt=None, **over):
    a = dict(q=FAKE, q_dt=pkd.BF16, q_stride=512, cache=FAKE, kv_dt=pkd.BF16, num_pages=8, table=FAKE, stride=8, lens=FAKE,
             starts=FAKE, B=2, T=20, max_q=16, Hq=4, Hkv=2, D=128, P=16, max_kv=100, scale=0.1, qs=1.0, ks=1.0, vs=1.0,
             opt=None, out=FAKE, out_dt=pkd.BF16, lse=None, ws=FAKE, ws_bytes=1 << 40, flags=pkd.FLAG_CAUSAL, stream=None)
    a.update(over)
    a["opt"] = opt
    return lib.pkd_paged_attention(*a.values())


@pytest.mark.parametrize("over,code,needle", [
    (dict(Hq=5), pkd.EUNSUPPORTED, "multiple of num_kv_heads"), (dict(D=96), pkd.EUNSUPPORTED, "head_dim"),
    (dict(P=8), pkd.EUNSUPPORTED, "page_size"), (dict(kv_dt=pkd.FP32), pkd.EUNSUPPORTED, "kv dtype"),
    (dict(kv_dt=pkd.FP8_E4M3, q_dt=pkd.FP8_E4M3, D=64), pkd.EUNSUPPORTED, "head_dim 128"),
    (dict(q_dt=pkd.FP16), pkd.EUNSUPPORTED, "q dtype"), (dict(out_dt=pkd.FP8_E4M3), pkd.EUNSUPPORTED, "out dtype"),
    (dict(B=5000), pkd.EUNSUPPORTED, "batch"), (dict(Hq=260, Hkv=2), pkd.EUNSUPPORTED, "num_heads/num_kv_heads"),
    (dict(max_q=0), pkd.EINVAL, "max_query_len"), (dict(q_stride=500), pkd.EINVAL, "q_stride"),
    (dict(q_stride=513), pkd.EINVAL, "q_stride"), (dict(stride=6), pkd.EINVAL, "stride"),
    (dict(ws_bytes=1000), pkd.EINVAL, "workspace"), (dict(scale=0.0), pkd.EINVAL, "scale"),
    (dict(scale=-1.0), pkd.EINVAL, "scale"), (dict(scale=float("nan")), pkd.EINVAL, "scale"),
    (dict(flags=pkd.FLAG_HOST_IO), pkd.EUNSUPPORTED, "FLAG_CAUSAL"), (dict(starts=None), pkd.EINVAL, "query_start"),
    (dict(num_pages=1 << 40), pkd.EUNSUPPORTED, "cache too large"), (dict(T=1 << 40), pkd.EUNSUPPORTED, "2^31"),
    (dict(max_kv=(1 << 29) + 1, stride=1 << 30), pkd.EUNSUPPORTED, "2^29"),
    (dict(lens=None), pkd.EINVAL, "null"), (dict(q=ctypes.c_void_p(0x10008)), pkd.EINVAL, "misaligned")])
def test_paged_attention_refusals(lib, over, code, needle):
    assert attend(lib, **over) == code
    assert needle in lib.pkd_last_error().decode()


@pytest.mark.parametrize("opt,flags,needle", [
    (pkd.ScoreOptions(-1.0, None, 0, None, None), pkd.FLAG_CAUSAL, "softcap"),
    (pkd.ScoreOptions(float("inf"), None, 0, None, None), pkd.FLAG_CAUSAL, "softcap"),
    (pkd.ScoreOptions(float("nan"), None, 0, None, None), pkd.FLAG_CAUSAL, "softcap"),
    (pkd.ScoreOptions(1e-30, None, 0, None, None), pkd.FLAG_CAUSAL, "softcap"),
    (pkd.ScoreOptions(0.0, 0x10002, 0, None, None), pkd.FLAG_CAUSAL, "aligned"),
    (pkd.ScoreOptions(0.0, None, 0, 0x10000, None), 0, "prefix_lens")])
def test_option_refusals(lib, opt, flags, needle):
    assert attend(lib, opt, flags=flags) == pkd.EINVAL
    assert needle in lib.pkd_last_error().decode()


def test_cap_and_scale_whose_quotient_overflows(lib):
    small = pkd.ScoreOptions(1e-20, None, 0, None, None)
    assert attend(lib, small, scale=1e20) == pkd.EINVAL and "softcap too small" in lib.pkd_last_error().decode()
    assert attend(lib, scale=3e38) == pkd.EINVAL and "scale" in lib.pkd_last_error().decode()
    assert prefix(lib, cap=1e-20, scale=1e20) == pkd.EINVAL and "softcap too small" in lib.pkd_last_error().decode()


def test_results_over_the_queries_are_refused(lib):
    assert attend(lib) == pkd.EINVAL and "overlaps" in lib.pkd_last_error().decode()
    last = ctypes.c_void_p(0x10000 + 2 * (19 * 512 + 512) - 16)  # the last 16 bytes of q
    assert attend(lib, out=last) == pkd.EINVAL and "overlaps" in lib.pkd_last_error().decode()
    assert prefix(lib) == pkd.EINVAL and "overlaps" in lib.pkd_last_error().decode()


def test_attention_of_nothing_is_ok(lib):
    assert attend(lib, B=0, q=None, cache=None) == pkd.OK
    assert attend(lib, T=0, q=None, cache=None) == pkd.OK


def test_plans_and_kernel_choice(lib):
    name = lambda *a: lib.pkd_paged_attention_kernel_name(*a).decode()
    size = lib.pkd_paged_attention_workspace_size
    # at most 16 rows (tokens x heads of a kv head): the step grid, for every cache type
    assert "step" in name(64, 64, 1, 32, 8, 128, 16, 4096, pkd.BF16, None)
    assert "step" in name(64, 128, 2, 64, 8, 128, 16, 4096, pkd.FP8_E4M3, None)
    assert "tcgen05" in name(64, 320, 5, 32, 8, 128, 16, 4096, pkd.BF16, None)
    # a window bounds the keys a step can span, and with them the chunks; prefix keys lift the bound
    whole = size(4, 4, 1, 32, 8, 128, 16, 131072, pkd.BF16, None)
    assert size(4, 4, 1, 32, 8, 128, 16, 131072, pkd.BF16, pkd.ScoreOptions(0.0, None, 512, None, None)) < whole
    assert size(4, 4, 1, 32, 8, 128, 16, 131072, pkd.BF16, pkd.ScoreOptions(0.0, None, 512, 0x10000, None)) == whole
    # prompts that fill the GPU are not split: no partial results
    base = 256 + 4 * 65536
    assert size(8, 20000, 4000, 32, 8, 128, 16, 8192, pkd.BF16, None) == base
    assert size(1, 64, 64, 8, 1, 128, 16, 65536, pkd.BF16, None) > base


def prefix(lib, **over):
    a = dict(q=FAKE, q_dt=pkd.BF16, cache=FAKE, kv_dt=pkd.BF16, num_pages=8, ptable=FAKE, pstride=8, plens=FAKE,
             gstart=FAKE, groups=1, max_prefix=100, table=FAKE, stride=8, lens=FAKE, B=2, sq=1, Hq=4, Hkv=2, D=128, P=16,
             max_kv=100, scale=0.1, qs=1.0, ks=1.0, vs=1.0, cap=0.0, out=FAKE, out_dt=pkd.BF16, lse=None, ws=FAKE,
             ws_bytes=1 << 40, flags=0, stream=None)
    a.update(over)
    return lib.pkd_prefix_decode(*a.values())


@pytest.mark.parametrize("over,code,needle", [
    (dict(groups=0), pkd.EINVAL, "groups"), (dict(groups=5000), pkd.EUNSUPPORTED, "groups"),
    (dict(sq=0), pkd.EINVAL, "sq"), (dict(max_prefix=(1 << 29) + 1, pstride=1 << 30), pkd.EUNSUPPORTED, "2^29"), (dict(cap=-1.0), pkd.EINVAL, "softcap"), (dict(pstride=6), pkd.EINVAL, "prefix_table"),
    (dict(gstart=None, groups=2), pkd.EINVAL, "group_start"), (dict(plens=None), pkd.EINVAL, "null"),
    (dict(ws_bytes=1000), pkd.EINVAL, "workspace"), (dict(flags=pkd.FLAG_GRID), pkd.EUNSUPPORTED, "FLAG_CAUSAL"),
    (dict(Hq=6, Hkv=4), pkd.EUNSUPPORTED, "multiple"), (dict(max_prefix=-1), pkd.EINVAL, "max_prefix_len")])
def test_prefix_decode_refusals(lib, over, code, needle):
    assert prefix(lib, **over) == code
    assert needle in lib.pkd_last_error().decode()


def test_prefix_decode_of_nothing_is_ok(lib):
    assert prefix(lib, B=0, q=None, cache=None, out=None, ws=None) == pkd.OK
