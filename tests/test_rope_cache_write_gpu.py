"""Rotary cache append on the GPU against the plain 64-bit formula."""
import numpy as np
import pytest
import torch

from tests import ragged_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.fail("a CUDA GPU is required for -m gpu tests")
    import paged_kv_decode_15_gb300 as pkd
    pkd.build()
    pkd.load_library()


def rotated(x, cs, rd, interleaved):
    """x [T, H, D] fp64 and each token's table row cs [T, rd]."""
    y = x.copy()
    for j in range(rd // 2):
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + rd // 2)
        c, s = cs[:, None, j], cs[:, None, rd // 2 + j]
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def close(got, want, kind, size):
    """Rounded once from an fp32 value that is off by 4 fp32 half steps of the
    pair's size at most (two products, their sum, the scaling)."""
    g = ref.values(got)
    if kind == "fp8":
        want = np.clip(want, -448, 448)
    near = 4 * ref.HALF_STEP["fp32"] * size
    # below the type's normal range the step is absolute
    tiny = {"bf16": 0.0, "fp16": 2.0 ** -25, "fp8": 2.0 ** -10}[kind]
    tol = ref.HALF_STEP[kind] * (np.abs(want) + near) + near + tiny
    bad = int((np.abs(g - want) > tol).sum())
    assert bad == 0, f"{bad} values off, by up to {np.abs(g - want).max()}"


def problem(T, Hq, Hkv, D, P, rd, dt, seed):
    rng = np.random.default_rng(seed)
    qkv = torch.from_numpy(rng.standard_normal((T, Hq + 2 * Hkv, D)).astype(np.float32)).to(ref.TORCH[dt])
    qkv[rng.random(qkv.shape) < 0.002] = 900.0   # saturates e4m3
    far = 5000
    angle = np.arange(far)[:, None] * 10000.0 ** (-np.arange(0, rd, 2) / rd)
    table = torch.from_numpy(np.concatenate([np.cos(angle), np.sin(angle)], -1)).float()
    pages = -(-T // P) + 2
    slots = rng.permutation(pages * P)[:T].astype(np.int64)
    return qkv, table, torch.from_numpy(rng.integers(0, far, T)), torch.from_numpy(slots), pages, rng


@pytest.mark.parametrize("T", [1, 3, 130])
@pytest.mark.parametrize("Hq,Hkv,D,P,rd,dt,cache,q8,inter", [
    (8, 2, 128, 16, 128, "bf16", "bf16", False, False), (8, 2, 128, 16, 128, "bf16", "fp8", True, False),
    (28, 4, 128, 32, 64, "fp16", "fp16", False, True), (3, 1, 64, 48, 16, "bf16", "fp8", False, True),
    (64, 8, 64, 16, 32, "fp16", "fp8", True, False), (5, 5, 128, 16, 112, "bf16", "bf16", True, False),
    (1, 1, 64, 64, 48, "fp16", "fp16", True, True), (56, 8, 128, 16, 128, "bf16", "bf16", False, True)])
def test_rotates_and_appends(T, Hq, Hkv, D, P, rd, dt, cache, q8, inter):
    import paged_kv_decode_15_gb300 as pkd
    qkv, table, pos, slots, pages, rng = problem(T, Hq, Hkv, D, P, rd, dt, T + Hq + rd)
    if T > 100:
        slots[[5, 77]] = -1
        slots[9] = pages * P + 3
    before = torch.from_numpy(rng.standard_normal((pages, Hkv, P, 2 * D)).astype(np.float32)).to(ref.TORCH[cache])
    pool, d = before.cuda(), qkv.cuda()
    ks, vs, qs = (0.0137, 1.0 / 64, 0.021) if cache == "fp8" else (1.0, 1.0, 0.021 if q8 else 1.0)
    out = pkd.rope_cache_write(d[:, :Hq], d[:, Hq:Hq + Hkv], d[:, Hq + Hkv:], pos.cuda(), table.cuda(), slots.cuda(), pool,
                               interleaved=inter, q_out_dtype=ref.TORCH["fp8"] if q8 else None, q_scale=qs, k_scale=ks,
                               v_scale=vs)
    x, cs = ref.values(qkv), ref.values(table)[pos.numpy()]
    turned = rotated(x, cs, rd, inter)
    size = np.sqrt(2) * np.abs(x).max(-1, keepdims=True)
    sq = qs if q8 else 1.0   # q_scale is that of e4m3 queries
    close(out.cpu(), turned[:, :Hq] / sq, "fp8" if q8 else dt, size[:, :Hq] / sq)
    got, old = pool.cpu(), ref.values(before)
    written = np.zeros((pages, P), bool)
    for t in range(T):
        s = int(slots[t])
        if not 0 <= s < pages * P:
            continue
        row = got[s // P, :, s % P]
        written[s // P, s % P] = True
        close(row[:, :D], turned[t, Hq:Hq + Hkv] / ks, cache, size[t, Hq:Hq + Hkv] / ks)
        close(row[:, D:], x[t, Hq + Hkv:] / vs, cache, size[t, Hq + Hkv:] / vs)
        if cache != "fp8":   # values keep their bits
            assert torch.equal(row[:, D:], qkv[t, Hq + Hkv:])
    keep = ~written[:, None, :, None].repeat(Hkv, 1).repeat(2 * D, 3)
    assert np.array_equal(ref.values(got)[keep], old[keep])


def test_in_place_queries_strided_outputs_and_unknown_positions():
    import paged_kv_decode_15_gb300 as pkd
    qkv, table, pos, slots, pages, _ = problem(40, 4, 2, 128, 16, 128, "bf16", 5)
    pos[3], pos[4] = -1, 5000
    want = pkd.rope_cache_write(*(qkv.cuda()[:, a:b] for a, b in ((0, 4), (4, 6), (6, 8))), pos.cuda(), table.cuda(),
                                slots.cuda(), torch.zeros(pages, 2, 16, 256, dtype=torch.bfloat16, device="cuda"),
                                q_out=torch.full((40, 4, 128), 3.0, dtype=torch.bfloat16, device="cuda"))
    assert (want[3:5] == 3).all()
    d = qkv.cuda()
    pool = torch.zeros(pages, 2, 16, 256, dtype=torch.bfloat16, device="cuda")
    got = pkd.rope_cache_write(d[:, :4], d[:, 4:6], d[:, 6:], pos.cuda(), table.cuda(), slots.cuda(), pool, q_out=d[:, :4])
    assert got.data_ptr() == d.data_ptr()
    rows = [t for t in range(40) if t not in (3, 4)]
    assert torch.equal(d[rows, :4], want[rows]) and torch.equal(d[3:5, :4].cpu(), qkv[3:5, :4])
    for t in (3, 4):
        assert (pool[int(slots[t]) // 16, :, int(slots[t]) % 16] == 0).all()


def test_keys_only_and_no_tokens():
    import paged_kv_decode_15_gb300 as pkd
    qkv, table, pos, slots, pages, _ = problem(7, 4, 2, 64, 16, 64, "fp16", 6)
    a, b = (torch.zeros(pages, 2, 16, 128, dtype=torch.float16, device="cuda") for _ in range(2))
    d = qkv.cuda()
    parts = (d[:, 4:6], d[:, 6:], pos.cuda(), table.cuda(), slots.cuda())
    pkd.rope_cache_write(d[:, :4], *parts, a)
    assert pkd.rope_cache_write(None, *parts, b) is None
    assert torch.equal(a, b) and a.any()
    out = pkd.rope_cache_write(d[:0, :4], d[:0, 4:6], d[:0, 6:], pos[:0].cuda(), table.cuda(), slots[:0].cuda(), b)
    assert out.shape == (0, 4, 64) and torch.equal(a, b)


def test_zero_angle_is_the_plain_cache_write():
    """Position 0 turns nothing: the same bytes as cache_write, for every cache type."""
    import paged_kv_decode_15_gb300 as pkd
    qkv, table, _, slots, pages, _ = problem(65, 4, 4, 128, 16, 128, "bf16", 7)
    d, pos = qkv.cuda(), torch.zeros(65, dtype=torch.int64, device="cuda")
    for dtype, scales in ((torch.bfloat16, {}), (torch.float8_e4m3fn, dict(k_scale=0.0137, v_scale=0.25))):
        a, b = (torch.zeros((pages, 4, 16, 256), dtype=dtype, device="cuda") for _ in range(2))
        q = pkd.rope_cache_write(d[:, :4], d[:, 4:8], d[:, 8:], pos, table.cuda(), slots.cuda(), a, **scales)
        pkd.cache_write(d[:, 4:8], d[:, 8:], slots.cuda(), b, **scales)
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)) and torch.equal(q, d[:, :4])


def test_every_16_bit_value_is_divided_as_by_the_plain_cache_write():
    """All bit patterns of both types, scales of every kind: powers of two, ordinary
    ones, a significand of all ones, and far ones (the IEEE division)."""
    import paged_kv_decode_15_gb300 as pkd
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16)
    table = torch.cat([torch.ones(1, 64), torch.zeros(1, 64)], -1).cuda()
    pos, slots = torch.zeros(256, dtype=torch.int64, device="cuda"), torch.arange(256, device="cuda")
    odd = float(np.float32(2.0) - np.float32(2.0 ** -23)) / 64
    for dtype in (torch.bfloat16, torch.float16):
        x = bits.view(dtype).view(256, 2, 128).cuda()
        for ks, vs in ((0.0137, 1.0 / 64), (odd, 3.3e-7), (41.7, 2.0 ** -70), (2.0 ** 66 * 1.1, 1.0)):
            a, b = (torch.zeros((16, 2, 16, 256), dtype=torch.uint8, device="cuda") for _ in range(2))
            pkd.rope_cache_write(None, x, x, pos, table, slots, a, k_scale=ks, v_scale=vs)
            pkd.cache_write(x, x, slots, b, k_scale=ks, v_scale=vs)
            # values: the same bytes.  Keys went through x1 * 1 - x2 * 0: an infinity of the pair becomes NaN,
            # and -0 - (-0) = +0 for x1 = -0, x2 < 0; so finite pairs are compared as numbers
            f8 = [t.view(torch.float8_e4m3fn).float()[..., :128] for t in (a, b)]
            fine = torch.stack([x.float()[..., :64], x.float()[..., 64:]], -1).isfinite().all(-1).repeat(1, 1, 2)
            fine = fine.view(16, 16, 2, 128).transpose(1, 2)
            values, keys = int((a != b)[..., 128:].sum()), int((f8[0] != f8[1])[fine].sum())
            assert (values, keys) == (0, 0), (dtype, ks, vs, values, keys)
