"""Attention over packed prompts on the GPU against the plain 64-bit reference: types, head
layouts, lengths from none to many tiles, masks, strides, bounds, and the prompt's way
into a bounded cache."""
import numpy as np
import pytest
import torch

import paged_kv_decode_15_gb300 as pkd
from tests import eviction_ref
from tests import ragged_ref as ref

pytestmark = pytest.mark.gpu


def dev(x):
    return torch.as_tensor(x).cuda()


class Packed:
    """A packed problem: the rows of a paged one's keys and values, side by side in one
    projection, NaN in rows of no prompt."""

    def __init__(self, lens, news=None, *, extra=3, **kw):
        self.c = c = ref.Paged(lens=lens, news=lens if news is None else news, extra_tokens=extra, **kw)
        k, v = [], []
        for b, L in enumerate(c.lens):
            t = np.arange(int(L))
            rows = c.cache[c.table[b, t // c.P].astype(np.int64), :, t % c.P]
            k.append(rows[..., :c.D])
            v.append(rows[..., c.D:])
        pad = torch.full((extra, c.Hkv, c.D), float("nan"), dtype=c.q.dtype)
        self.kv = torch.cat([torch.cat(k + [pad]), torch.cat(v + [pad])], 1).cuda()  # [Tk, 2 Hkv, D]
        self.q = c.q.cuda()
        self.starts = dev(c.starts)
        ends = np.concatenate([[0], np.cumsum(c.lens)]).astype(np.int32)
        self.key_start = dev(ends) if news is not None else None

    @property
    def k(self):
        return self.kv[:, :self.c.Hkv]

    @property
    def v(self):
        return self.kv[:, self.c.Hkv:]

    def run(self, **kw):
        kw.setdefault("max_query_len", max(1, int(self.c.news.max(initial=1))))
        kw.setdefault("max_kv_len", int(self.c.lens.max(initial=0)))
        ws = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
        pkd.workspace_init(ws)
        out, lse = pkd.packed_attention(self.q, self.k, self.v, self.starts, self.c.scale, key_start=self.key_start,
                                        workspace=ws, **kw)
        assert pkd.workspace_check(ws) == pkd.OK
        return out.cpu(), lse.cpu()

    def verify(self, what="", out_dtype=None, **kw):
        out, lse = self.run(out_dtype=out_dtype, **kw)
        name = {torch.float32: "fp32", torch.float16: "fp16", torch.bfloat16: "bf16", None: None}[out_dtype]
        ref.check(out, lse, self.c.reference(**kw), self.c.dtype, name, what)


@pytest.mark.parametrize("dtype,Hq,Hkv,D", [("bf16", 4, 1, 128), ("fp16", 2, 2, 64), ("bf16", 7, 1, 64), ("fp16", 8, 1, 128),
                                            ("bf16", 1, 1, 128), ("fp16", 14, 2, 128)])
@pytest.mark.parametrize("mod", ["plain", "cap", "window", "dense", "dense+window+cap"])
def test_prompts(dtype, Hq, Hkv, D, mod):
    kw = {}
    if "cap" in mod:
        kw["softcap"] = 5.0
    if "window" in mod:
        kw["window"] = 41
    if "dense" in mod:
        kw["causal"] = False
    Packed([1, 17, 129, 0, 200, 333], Hq=Hq, Hkv=Hkv, D=D, dtype=dtype, seed=Hq * D).verify(mod, **kw)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("fp16", 64)])
def test_keys_of_other_lengths(dtype, D, causal):
    """More keys than tokens (the tokens are the last ones), fewer (early tokens see none), none."""
    p = Packed([300, 20, 0, 140, 64], [30, 50, 4, 140, 1], Hq=6, Hkv=2, D=D, dtype=dtype, seed=5)
    p.verify("lengths", causal=causal)
    p.verify("lengths, window", causal=causal, window=25)


def test_split_keys():
    """Few rows over many keys: split, and joined."""
    p = Packed([3000, 700], [20, 9], Hq=8, Hkv=2, D=128, dtype="bf16", seed=6)
    p.verify("split")
    p.verify("split, capped", softcap=20.0)


@pytest.mark.parametrize("D", [64, 128])
def test_many_tiles(D):
    Packed([1400, 515], Hq=4, Hkv=2, D=D, dtype="bf16", seed=7).verify("tiles")


def test_hundreds_of_prompts():
    rng = np.random.default_rng(8)
    Packed(rng.integers(0, 40, 300), Hq=2, Hkv=1, D=64, dtype="fp16", seed=9).verify("many")


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_output_types(out_dtype):
    Packed([50, 20], Hq=4, Hkv=2, D=128, dtype="fp16", seed=1).verify("types", out_dtype)


@pytest.mark.parametrize("bad", ["nan", "inf", "1e4"])
@pytest.mark.parametrize("softcap", [0.0, 5.0])
def test_other_prompts_do_not_enter(bad, softcap):
    """A prompt's values reach its own tokens only, also inside a key tile that holds both."""
    p = Packed([70, 50, 90], Hq=4, Hkv=2, D=128, dtype="bf16", seed=10, extra=0)
    good, lse = p.run(softcap=softcap)
    p.kv[70:120] = float(bad)
    out, lse2 = p.run(softcap=softcap)
    for a, b in ((good, out), (lse, lse2)):
        assert torch.equal(a[:70], b[:70]) and torch.equal(a[120:210], b[120:210])


def test_rows_of_no_prompt_and_no_keys():
    p = Packed([40, 30], Hq=4, Hkv=2, D=64, dtype="fp16", seed=11, extra=5)
    p.q[70:] = float("nan")
    out, lse = torch.full((75, 4, 64), 7.0, dtype=torch.float16, device="cuda"), torch.full((75, 4), 7.0, device="cuda")
    pkd.packed_attention(p.q, p.k, p.v, p.starts, p.c.scale, out=out, lse=lse, max_query_len=40)
    assert (out[70:] == 7).all() and (lse[70:] == 7).all() and torch.isfinite(out[:70]).all()
    none = torch.zeros(3, dtype=torch.int32, device="cuda")
    out, lse = pkd.packed_attention(p.q[:70], p.k[:0], p.v[:0], p.starts, p.c.scale, key_start=none, max_query_len=40)
    assert (out == 0).all() and (lse == -torch.inf).all()
    out, lse = pkd.packed_attention(p.q[:0], p.k, p.v, none, p.c.scale, key_start=p.starts)
    assert out.shape == (0, 4, 64)


def test_bad_starts_are_clamped():
    p = Packed([40, 30], Hq=4, Hkv=2, D=64, dtype="fp16", seed=12, extra=0)
    ws = torch.zeros(1 << 24, dtype=torch.uint8, device="cuda")
    good, _ = pkd.packed_attention(p.q, p.k, p.v, p.starts, p.c.scale, max_query_len=40, workspace=ws)
    assert pkd.workspace_check(ws) == pkd.OK
    for starts, keys in (([0, 40, 900], [0, 40, 70]), ([0, 40, 70], [0, 40, 10 ** 9]), ([0, 40, 70], [-3, 40, 70])):
        out, _ = pkd.packed_attention(p.q, p.k, p.v, dev(np.array(starts, np.int32)), p.c.scale,
                                      key_start=dev(np.array(keys, np.int32)), max_query_len=40, max_kv_len=40, workspace=ws)
        assert pkd.workspace_check(ws) == pkd.EDEVICE_BOUNDS
        assert torch.equal(out, good)
    out, _ = pkd.packed_attention(p.q, p.k, p.v, p.starts, p.c.scale, max_query_len=40, max_kv_len=35, workspace=ws)
    assert pkd.workspace_check(ws) == pkd.EDEVICE_BOUNDS and torch.equal(out[40:], good[40:])
    pkd.packed_attention(p.q, p.k, p.v, p.starts, p.c.scale, max_query_len=40, workspace=ws)
    assert pkd.workspace_check(ws) == pkd.OK


def test_captured_and_on_another_stream():
    p = Packed([400, 90], Hq=8, Hkv=2, D=128, dtype="bf16", seed=13, extra=0)
    good = p.run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, lse = pkd.packed_attention(p.q, p.k, p.v, p.starts, p.c.scale, max_query_len=400, stream=side)
    side.synchronize()
    assert torch.equal(out.cpu(), good[0]) and torch.equal(lse.cpu(), good[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = pkd.packed_attention(p.q, p.k, p.v, p.starts, p.c.scale, max_query_len=400)
    for _ in range(2):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.cpu(), good[0]) and torch.equal(lse.cpu(), good[1])


def test_a_timeout_is_reported_and_recovered_from():
    p = Packed([2000, 1500], Hq=16, Hkv=8, D=128, dtype="bf16", seed=14, extra=0)
    good = p.run()
    ws = torch.zeros(1 << 26, dtype=torch.uint8, device="cuda")
    args = (p.q, p.k, p.v, p.starts, p.c.scale)
    pkd.packed_attention(*args, max_query_len=2000, workspace=ws, test_timeout=True)
    assert pkd.workspace_check(ws) == pkd.ETIMEOUT
    pkd.workspace_init(ws)
    out, lse = pkd.packed_attention(*args, max_query_len=2000, workspace=ws)
    assert pkd.workspace_check(ws) == pkd.OK
    assert torch.equal(out.cpu(), good[0]) and torch.equal(lse.cpu(), good[1])


@pytest.mark.parametrize("wrong,error", [(dict(key_start=torch.zeros(5, dtype=torch.int32)), ValueError),
                                         (dict(max_query_len=0), pkd.PkdError), (dict(softcap=-1.0), pkd.PkdError)])
def test_refusals(wrong, error):
    p = Packed([40, 30], Hq=4, Hkv=2, D=64, dtype="fp16", seed=15, extra=0)
    wrong = {k: dev(v) if isinstance(v, torch.Tensor) else v for k, v in wrong.items()}
    with pytest.raises(error):
        pkd.packed_attention(p.q, p.k, p.v, p.starts, p.c.scale, **wrong)
    with pytest.raises(ValueError):
        pkd.packed_attention(p.q, p.k, p.v[:, :, :32], p.starts, p.c.scale)
    with pytest.raises(pkd.PkdError, match="overlaps"):
        pkd.packed_attention(p.q, p.q, p.q, p.starts, p.c.scale, out=p.q)


def test_from_a_prompt_to_a_bounded_cache():
    """A layer of a prompt: packed attention, its keys written to the cache, weighed by its last
    tokens with the LSE in hand, the cache bounded, a step attends to what stayed."""
    p = Packed([260, 45, 150], Hq=8, Hkv=2, D=128, dtype="bf16", seed=16, extra=0)
    c = p.c
    _, lse = pkd.packed_attention(p.q, p.k, p.v, p.starts, c.scale, max_query_len=260)
    cache = torch.zeros((40, 2, 16, 256), dtype=torch.bfloat16, device="cuda")
    table = torch.randperm(40, device="cuda")[:39].view(3, 13).to(torch.int32)
    table = torch.cat([table, torch.full((3, 4), -1, dtype=torch.int32, device="cuda")], 1)
    at = torch.cat([torch.arange(n, device="cuda") for n in (208, 45, 150)])
    req = torch.repeat_interleave(torch.arange(3, device="cuda"), torch.tensor([208, 45, 150], device="cuda"))
    # (the first prompt's pages hold 208 keys: it comes as two chunks, the second one's keys not cached here)
    rows = torch.cat([torch.arange(208), torch.arange(260, 455)]).cuda()
    slots = table[req, at // 16].long() * 16 + at % 16
    pkd.cache_write(p.k[rows], p.v[rows], slots, cache)
    lens = torch.tensor([208, 45, 150], dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, 208, 253, 403], dtype=torch.int32, device="cuda")
    q, some = p.q[rows].contiguous(), lse[rows].contiguous()
    w = pkd.key_weights(q, cache, table, lens, starts, some, c.scale, last_queries=8, max_query_len=208, max_kv_len=208)
    qv, cv = q.float().double().cpu().numpy(), cache.float().double().cpu().numpy()
    tb, ln = table.cpu().numpy(), lens.cpu().numpy()
    want, err = eviction_ref.key_weights(qv, cv, tb, ln, starts.cpu().numpy(), some.double().cpu().numpy(), c.scale, last=8)
    for b in range(3):
        assert (np.abs(w.double().cpu().numpy()[b, :, :ln[b]] - want[b, :, :ln[b]]) <= err[b, :, :ln[b]] + 1e-30).all()
    kept, n = pkd.evict_select(w, lens, 64, sinks=4, recent=8)
    assert np.array_equal(kept.cpu().numpy(), eviction_ref.evict_select(w.cpu().numpy(), ln, 64, sinks=4, recent=8)[0])
    pkd.cache_compact(cache, table, kept, n, weights=w)
    step = torch.randn((3, 1, 8, 128), device="cuda").to(torch.bfloat16)
    out, lse2 = pkd.paged_decode(step, cache, table, n, c.scale, max_kv_len=208)
    # the kept keys themselves, in their old order
    for b in range(3):
        for h in range(8):
            keep = kept[b, h // 4, :int(n[b])].long()
            row = (int(p.starts[b]) + keep)
            k, v = p.k[row, h // 4].double(), p.v[row, h // 4].double()
            s = (k @ step[b, 0, h].double()) * c.scale
            prob = torch.softmax(s, 0)
            mag = prob @ v.abs()
            assert ((out[b, 0, h].double() - prob @ v).abs() <= 2.0 ** -8 * (mag + (prob @ v).abs()) + 2.0 ** -12 * mag).all()
            assert abs(float(lse2[b, 0, h]) - float(torch.logsumexp(s, 0))) < 1e-4
