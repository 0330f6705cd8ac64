"""Long sums of ragged attention and shared-prefix decode: prompts over tens and
hundreds of thousands of keys against a 64-bit reference."""
import numpy as np
import pytest
import torch

from tests import ragged_ref as ref

pytestmark = pytest.mark.gpu

HEAD = 256 + 4 * 65536  # PKD_ATTENTION_WORKSPACE_HEAD


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.fail("a CUDA GPU is required for -m gpu tests")
    import paged_kv_decode_15_gb300 as pkd
    pkd.build()
    pkd.load_library()


class Long:
    """One request of n keys whose T last ones bring queries, all tokens alike, so that the
    reference is one pass over the keys.  Dim 0 of the keys is `profile` (times 8), dim 0 of
    a head's query its gap, the scale 1/8: gap * profile is added to scores that are alike
    but for a spread of 0.05 or so."""

    def __init__(self, n, T, G, Hkv, D, dtype, profile, gaps, seed=61, size=1.0):
        rng = np.random.default_rng(seed)
        self.n, self.T, self.G, self.Hkv, self.D, self.dtype, self.scale, self.gaps = n, T, G, Hkv, D, dtype, 0.125, gaps
        k = rng.standard_normal((n, Hkv, D)).astype(np.float32)
        k[:, :, 0] = 8.0 * profile[:, None]
        v = 1.0 + 0.25 * rng.standard_normal((n, Hkv, D)).astype(np.float32)
        v[profile == profile.max()] = -1.0
        v *= size
        q = 0.05 * rng.standard_normal((Hkv, len(gaps), D)).astype(np.float32)
        q[:, :, 0] = gaps
        t, P = ref.TORCH[dtype], 64
        self.k, self.v, self.q = (torch.from_numpy(x).to(t) for x in (k, v, q))
        order = rng.permutation(n // P)
        assert n % P == 0
        kv = torch.cat([self.k, self.v], -1).float().view(n // P, P, Hkv, 2 * D).transpose(1, 2)
        cache = torch.empty_like(kv)
        cache[torch.from_numpy(order)] = kv
        self.cache = cache.to(t).contiguous().cuda()
        self.table = torch.from_numpy(order.astype(np.int32))[None].cuda()
        self.lens = torch.tensor([n], dtype=torch.int32, device="cuda")
        self.starts = torch.tensor([0, T], dtype=torch.int32, device="cuda")
        self.level = np.arange(G) % len(gaps)
        one = self.q.float()[:, self.level].reshape(Hkv * G, D)
        self.queries = one[None].expand(T, -1, -1).to(t).contiguous().cuda()

    def check(self, out, lse, causal=False, slope=0.0):
        """out [T, Hq, D] fp32, lse [T, Hq].  The bounds, with mag = sum of w |v|:

        A score is off by ds = 1e-5 (1 + S) (S: the sum of its absolute products and of
        its bias), so a weight by 2 ds relative; a weight is rounded to its type for the
        product; the products' sum is cut off to fp32 every 16 keys, at most 2048 times a
        sum: 2048 * 2^-23 = 2^-12; the sum of the weights is rounded to fp32 every 128
        keys: n / 128 half steps of 2^-24; and small fp16 weights may lose 2^-13 of the
        sum together (below 2^-14 a weight is off by 2^-25 at most where the largest is
        at least 2^(log2 n - 12))."""
        T, L = self.T, len(self.gaps)
        k, v, q = ref.values(self.k), ref.values(self.v), ref.values(self.q)
        operand = ref.HALF_STEP["fp16" if self.dtype == "fp8" else self.dtype]
        adds, lost = self.n / 128 * 2.0 ** -24, 0.0 if self.dtype == "bf16" else 2.0 ** -13
        for h in range(self.Hkv):
            s = (k[:, h] @ q[h].T) * self.scale                       # [n, levels]
            # a distance bias -slope (pos - key): the same for all tokens but for -slope pos
            s += slope * np.arange(self.n)[:, None]
            size = (np.abs(k[:, h]) @ np.abs(q[h]).T).max(0) * self.scale + slope * self.n
            top = s.max(0)
            w = np.exp(s - top)
            first, last = self.n - T, slice(self.n - T, self.n)
            sums = []
            for x in (v[:, h], np.abs(v[:, h]), np.ones((self.n, 1))):
                base = w[:first].T @ x[:first]                         # [levels, D]
                tail = np.cumsum(w[last][:, :, None] * x[last][:, None, :], 0)
                sums.append(base[None] + (tail if causal else np.broadcast_to(tail[-1:], tail.shape)))
            want, mag = sums[0] / sums[2], sums[1] / sums[2]           # [T, levels, D]
            want_lse = top + np.log(sums[2][..., 0]) - slope * np.arange(first, self.n)[:, None]
            ds = 1e-5 * (1 + size)
            tol = (operand + 2 * ds + 1e-5 + 2.0 ** -12 + adds)[None, :, None] * mag + lost * np.abs(v[:, h]).max()
            rows = slice(h * self.G, (h + 1) * self.G)
            worst = np.abs(ref.values(out[:, rows].cpu()) - want[:, self.level]) / tol[:, self.level]
            worst = {g: round(float(worst[:, self.level == i].max()), 3) for i, g in enumerate(self.gaps)}
            assert max(worst.values()) <= 1, worst
            off = np.abs(ref.values(lse[:, rows].cpu()) - want_lse[:, self.level])
            lim = (ds + adds)[None] + 1e-6 * np.abs(want_lse) + 2e-6
            assert (off <= lim[:, self.level]).all(), off.max()


def flat(n):
    """Keys alike, but for the first."""
    return (np.arange(n) == 0).astype(np.float32)


def ramp(n):
    return np.floor(np.arange(n) / n * 16).astype(np.float32) / 16


@pytest.mark.parametrize("n", [32768, 32832, 96000, 524288])
@pytest.mark.parametrize("causal", [False, True])
def test_many_keys_of_alike_weight(n, causal):
    import paged_kv_decode_15_gb300 as pkd
    c = Long(n, 304, 128, 1, 64, "fp16", flat(n), [0.0, 0.5])
    out, lse = pkd.paged_attention(c.queries, c.cache, c.table, c.lens, c.starts, c.scale, causal=causal, out_dtype=torch.float32)
    c.check(out, lse, causal)


@pytest.mark.parametrize("dtype,D", [("fp16", 64), ("bf16", 128), ("fp8", 128), ("fp16", 128), ("bf16", 64)])
@pytest.mark.parametrize("mod", ["plain", "cap", "bias", "cap+bias"])
def test_long_sums_whose_references_move(dtype, D, mod):
    """Scores that rise by up to 24 along the keys.  (A cap c = 1e5 moves a score s by
    s^3 / (3 c^2), within ds.)"""
    import paged_kv_decode_15_gb300 as pkd
    c = Long(96000, 152, 128, 2, D, dtype, ramp(96000), [0.0, 1.0, 10.0, 24.0])
    slope = 2.0 ** -14 if "bias" in mod else 0.0
    out, lse = pkd.paged_attention(c.queries, c.cache, c.table, c.lens, c.starts, c.scale, causal=True,
                                   softcap=1e5 if "cap" in mod else 0.0, out_dtype=torch.float32,
                                   alibi_slopes=torch.full((256,), slope, device="cuda") if slope else None)
    c.check(out, lse, True, slope)


@pytest.mark.parametrize("dtype,D", [("fp16", 64), ("fp8", 128)])
def test_a_long_prefix_and_long_own_keys(dtype, D):
    """Both passes fold, each in its own part of the workspace, while they may overlap."""
    import paged_kv_decode_15_gb300 as pkd
    n, T, cut = 80000, 152, 600
    c = Long(n, T, 128, 2, D, dtype, ramp(n), [0.0, 1.0, 10.0, 24.0])
    lens = torch.tensor([cut * 64], dtype=torch.int32, device="cuda")
    out, lse = pkd.prefix_decode(c.queries.view(1, T, 256, D), c.cache, c.table[:, :cut].contiguous(), lens,
                                 c.table[:, cut:].contiguous(), c.lens - lens, c.scale, causal=True, out_dtype=torch.float32)
    c.check(out.view(T, 256, D), lse.view(T, 256), True)


SINK = [0.0, 6.0, 10.0, 13.0, 16.0, 18.0, 20.0, 24.0]


def one_key(n, at):
    return (np.arange(n) == at).astype(np.float32)


@pytest.mark.parametrize("dtype,D", [("fp16", 64), ("fp16", 128), ("fp8", 128), ("bf16", 128)])
@pytest.mark.parametrize("at", [0, 70000])
@pytest.mark.parametrize("cap", [0.0, 1e5])
def test_a_large_score_beside_many_small_ones(dtype, D, at, cap):
    """131072 weights of e^-18, 2^-9 of the sum together, are not lost beside one of 1."""
    import paged_kv_decode_15_gb300 as pkd
    n = 131072
    c = Long(n, 152, 128, 2, D, dtype, one_key(n, at), SINK)
    out, lse = pkd.paged_attention(c.queries, c.cache, c.table, c.lens, c.starts, c.scale, causal=False, softcap=cap,
                                   out_dtype=torch.float32)
    c.check(out, lse)


@pytest.mark.parametrize("dtype,D", [("fp16", 64), ("fp8", 128)])
@pytest.mark.parametrize("T", [1, 24])
def test_a_large_score_in_split_keys(dtype, D, T):
    """Steps and few rows: each chunk has a reference of its own."""
    import paged_kv_decode_15_gb300 as pkd
    n = 131072
    c = Long(n, T, 8, 2, D, dtype, one_key(n, 99), SINK)
    out, lse = pkd.paged_attention(c.queries, c.cache, c.table, c.lens, c.starts, c.scale, causal=False,
                                   out_dtype=torch.float32)
    c.check(out, lse)


@pytest.mark.parametrize("dtype,D", [("fp16", 128), ("fp8", 128)])
def test_a_large_score_in_a_shared_prefix(dtype, D):
    import paged_kv_decode_15_gb300 as pkd
    n, B = 131072, 150
    c = Long(n, B, 128, 2, D, dtype, one_key(n, 5000), SINK)
    own = torch.zeros(B, dtype=torch.int32, device="cuda")
    out, lse = pkd.prefix_decode(c.queries.view(B, 1, 256, D), c.cache, c.table, c.lens,
                                 c.table[:, :1].expand(B, 1).contiguous(), own, c.scale, out_dtype=torch.float32)
    c.check(out.view(B, 256, D), lse.view(B, 256))


@pytest.mark.parametrize("dtype,D", [("fp16", 64), ("fp8", 128)])
def test_long_chunks_of_split_keys(dtype, D):
    import paged_kv_decode_15_gb300 as pkd
    n = 524288
    c = Long(n, 40, 128, 2, D, dtype, ramp(n), [0.0, 1.0, 10.0, 24.0])
    need = pkd.load_library().pkd_paged_attention_workspace_size(1, 40, 40, 256, 2, D, 64, n, pkd.FP16, None)
    assert need > HEAD + 2 * 40 * 256 * D * 4, "split"
    for _ in range(2):
        out, lse = pkd.paged_attention(c.queries, c.cache, c.table, c.lens, c.starts, c.scale, causal=True, out_dtype=torch.float32)
        c.check(out, lse, True)


@pytest.mark.parametrize("dtype,D", [("fp16", 64), ("bf16", 128)])
def test_a_long_prefix_of_many_requests(dtype, D):
    import paged_kv_decode_15_gb300 as pkd
    n, B = 131072, 150
    c = Long(n, B, 128, 2, D, dtype, ramp(n), [0.0, 1.0, 10.0, 24.0])
    own = torch.zeros(B, dtype=torch.int32, device="cuda")
    out, lse = pkd.prefix_decode(c.queries.view(B, 1, 256, D), c.cache, c.table, c.lens,
                                 c.table[:, :1].expand(B, 1).contiguous(), own, c.scale, out_dtype=torch.float32)
    c.check(out.view(B, 256, D), lse.view(B, 256))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("n,size", [(2048, 3e34), (2048, 1e-30), (40000, 3e33)])
@pytest.mark.parametrize("mod", ["plain", "cap", "bias"])
def test_values_of_any_size(dtype, n, size, mod):
    """Scores that rise by 24, 2^34.6, along the keys: the weights on the way must not take
    large values out of fp32's range, nor small ones (fp16: of its own range)."""
    import paged_kv_decode_15_gb300 as pkd
    if dtype == "fp16":
        size = {3e34: 2e4, 3e33: 2e4, 1e-30: 1e-3}[size]
    c = Long(n, 152, 128, 2, 64, dtype, ramp(n), [0.0, 1.0, 10.0, 24.0], size=size)
    slope = 2.0 ** -14 if mod == "bias" else 0.0
    out, lse = pkd.paged_attention(c.queries, c.cache, c.table, c.lens, c.starts, c.scale, causal=True,
                                   softcap=1e5 if mod == "cap" else 0.0, out_dtype=torch.float32,
                                   alibi_slopes=torch.full((256,), slope, device="cuda") if slope else None)
    c.check(out, lse, True, slope)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("exponent", [22, 24, 25, 26, 27, 28])
def test_logits_so_large_that_fp32_has_few_digits_left(dtype, exponent):
    """Logits of 2^exponent (log2 units) that rise by 16 here and there: the largest weight
    is one whatever the rest, so the result lies among the values."""
    import paged_kv_decode_15_gb300 as pkd
    n, T, half = 1024, 304, exponent // 2
    k = torch.zeros(n, 128)
    k[:, 0] = 2.0 ** (exponent - half)
    k[:, 1] = 2.0 * torch.tensor([0, 1, 2, 3, 3, 4, 4, 2]).repeat_interleave(128)  # times 8: key tiles that rise by 16 or not
    k[:, 64:] = torch.from_numpy(np.random.default_rng(88).uniform(1, 2, (n, 64)).astype(np.float32))
    q = torch.zeros(T, 128, 64)
    q[..., 0], q[..., 1] = 2.0 ** half, 8.0
    t = ref.TORCH[dtype]
    cache = k.to(t).view(n // 64, 1, 64, 128).contiguous().cuda()
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    out, lse = pkd.paged_attention(q.to(t).cuda(), cache, ints([list(range(n // 64))]), ints([n]), ints([0, T]), float(np.log(2.0)),
                                   causal=False, out_dtype=torch.float32)
    assert torch.isfinite(out).all() and out.min() >= 1 - 2.0 ** -7 and out.max() <= 2 + 2.0 ** -6
    top = np.log(2.0) * (2.0 ** exponent + 64)
    assert (lse.double().cpu() - top).abs().max() <= 1e-6 * top + np.log(n)


@pytest.mark.parametrize("T", [2, 40])
def test_large_values_in_split_keys_and_shared_prefixes(T):
    import paged_kv_decode_15_gb300 as pkd
    c = Long(2048, T, 8, 2, 128, "bf16", ramp(2048), [0.0, 1.0, 10.0, 24.0], size=3e34)
    out, lse = pkd.paged_attention(c.queries, c.cache, c.table, c.lens, c.starts, c.scale, causal=False,
                                   out_dtype=torch.float32)
    c.check(out, lse)
    own = torch.zeros(T, dtype=torch.int32, device="cuda")
    out, lse = pkd.prefix_decode(c.queries.view(T, 1, 16, 128), c.cache, c.table, c.lens,
                                 c.table[:, :1].expand(T, 1).contiguous(), own, c.scale, out_dtype=torch.float32)
    c.check(out.view(T, 16, 128), lse.view(T, 16))
