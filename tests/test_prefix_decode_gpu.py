"""Shared-prefix decode on the GPU against the plain 64-bit reference over each
request's prefix and own keys, and a server's round of all the operators."""
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


class Shared:
    """Groups of requests: the prefixes and the own keys are rows of one pool."""

    def __init__(self, *, prefixes, group_start, own, sq, seed=0, **kw):
        self.prefixes, self.group_start = list(prefixes), np.asarray(group_start, np.int32)
        self.own, self.sq, self.B = np.asarray(own, np.int32), sq, len(own)
        g = len(self.prefixes)
        self.c = ref.Paged(lens=self.prefixes + list(own), news=[0] * g + [sq] * self.B, seed=seed, **kw)
        self.g = g

    def call(self, **kw):
        import paged_kv_decode_15_gb300 as pkd
        c, g, P = self.c, self.g, self.c.P
        wide = max(1, -(-max(self.prefixes) // P)), max(1, -(-int(self.own.max(initial=1)) // P))
        kw.setdefault("group_start", dev(self.group_start))
        ws = torch.empty(1 << 29, dtype=torch.uint8, device="cuda")
        pkd.workspace_init(ws)
        out, lse = pkd.prefix_decode(
            dev(c.q).view(self.B, self.sq, c.Hq, c.D), dev(c.cache), dev(c.table[:g, :wide[0]].copy()),
            dev(np.asarray(self.prefixes, np.int32)), dev(c.table[g:, :wide[1]].copy()), dev(self.own), c.scale,
            workspace=ws, **c.scales(), **kw)
        return out.cpu(), lse.cpu(), pkd.workspace_check(ws)

    def reference(self, causal=False, softcap=0.0):
        """As ordinary attention over a cache in which each request's keys are its prefix, then its own."""
        c = self.c
        cache = np.nan_to_num(ref.values(c.cache))
        Hkv, D, sq = c.Hkv, c.D, self.sq
        parts = [[], [], [], []]
        for b in range(self.B):
            rows = []
            for g in range(self.g):
                if self.group_start[g] <= b < self.group_start[g + 1]:
                    rows.append((g, self.prefixes[g]))
            rows.append((self.g + b, int(self.own[b])))
            kv = np.concatenate([cache[c.table[r][np.arange(n) // c.P], :, np.arange(n) % c.P] for r, n in rows])
            n, plen = len(kv), len(kv) - int(self.own[b])
            pages = max(1, -(-n // 16))
            own = np.zeros((pages * 16, Hkv, 2 * D))
            own[:n] = kv
            own = own.reshape(pages, 16, Hkv, 2 * D).transpose(0, 2, 1, 3)
            # with a causal mask a token behind the own keys still sees the whole prefix
            r = ref.attention(ref.values(c.q)[b * sq:(b + 1) * sq], own, np.arange(pages)[None], [n], [0, sq], c.scale,
                              causal=causal, prefix_lens=[plen], softcap=softcap, **c.scales())
            for p, x in zip(parts, r):
                p.append(x)
        return [np.concatenate(p) for p in parts]

    def verify(self, **kw):
        import paged_kv_decode_15_gb300 as pkd
        out, lse, status = self.call(**kw)
        assert status == pkd.OK
        kw.pop("group_start", None)
        kind = kw.pop("out_dtype", None)
        c = self.c
        # two parts joined in fp32: each part's own bound, and the join's roundings inside it
        ref.check(out.view(-1, c.Hq, c.D), lse.view(-1, c.Hq), self.reference(**kw), c.dtype,
                  {torch.float32: "fp32", torch.float16: "fp16", None: None}[kind])


@pytest.mark.parametrize("dtype,Hq,Hkv,D,P,sq", [("bf16", 8, 2, 128, 16, 1), ("fp16", 4, 4, 64, 32, 2),
                                                 ("bf16", 14, 2, 64, 48, 1), ("fp16", 16, 2, 128, 16, 4),
                                                 ("fp8", 8, 2, 128, 64, 1), ("fp8", 16, 2, 128, 16, 3)])
@pytest.mark.parametrize("causal,cap", [(False, 0.0), (True, 8.0)])
def test_groups(dtype, Hq, Hkv, D, P, sq, causal, cap):
    s = Shared(prefixes=[700, 1, 130], group_start=[0, 5, 6, 9], own=[sq, 70, 33, 5, 200, 17, 4, 16, 90], sq=sq, Hq=Hq,
               Hkv=Hkv, D=D, P=P, dtype=dtype, seed=D + P)
    s.verify(causal=causal, softcap=cap)


def test_empty_prefixes_empty_requests_and_requests_of_no_group():
    s = Shared(prefixes=[0, 65, 300], group_start=[1, 3, 3, 6], own=[40, 0, 7, 0, 12, 1, 0, 20], sq=1, Hq=4, Hkv=2, D=128,
               seed=3)
    s.verify()
    s.verify(causal=True)


def test_one_group_by_default_and_many_requests():
    rng = np.random.default_rng(4)
    s = Shared(prefixes=[2600], group_start=[0, 150], own=rng.integers(0, 40, 150), sq=1, Hq=4, Hkv=1, D=64, dtype="fp16",
               seed=4)
    a = s.call()
    b = s.call(group_start=None)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    s.verify()


def test_same_as_decode_over_the_whole_context():
    """A request's result does not depend on whether its prefix is shared (beyond rounding)."""
    import paged_kv_decode_15_gb300 as pkd
    c = ref.Paged(lens=[1600, 1600, 1600], news=[1, 1, 1], Hq=8, Hkv=2, D=128, seed=5)
    table = dev(c.table)
    table[1:, :64] = table[0, :64]   # 1024 common keys
    q, cache, lens = dev(c.q), dev(c.cache), dev(c.lens)
    whole = pkd.paged_decode(q.view(3, 1, 8, 128), cache, table, lens, c.scale)
    split = pkd.prefix_decode(q.view(3, 1, 8, 128), cache, table[:1, :64].contiguous(),
                              torch.tensor([1024], dtype=torch.int32, device="cuda"), table[:, 64:].contiguous(),
                              lens - 1024, c.scale)
    # both round weights and outputs to bf16: two half steps of weights of values up to 5, one step of the output
    assert (whole[0].float() - split[0].float()).abs().max() <= 2 * 2.0 ** -8 * 5.0
    assert (whole[1] - split[1]).abs().max() <= 1e-4


def test_a_round_of_serving():
    """A common prompt and own prompts appended and attended, then steps on the shared prefix."""
    import paged_kv_decode_15_gb300 as pkd
    rng = np.random.default_rng(6)
    Hq, Hkv, D, P, n0, own = 8, 2, 128, 16, 96, [20, 33, 1]
    B, scale = len(own), D ** -0.5
    angle = np.arange(300)[:, None] * 10000.0 ** (-np.arange(0, D, 2) / D)
    table_cs = torch.from_numpy(np.concatenate([np.cos(angle), np.sin(angle)], -1)).float().cuda()
    cache = torch.zeros((40, Hkv, P, 2 * D), dtype=torch.bfloat16, device="cuda")
    pages = rng.permutation(40)
    pre, rows = pages[:n0 // P], pages[n0 // P:n0 // P + 4 * B].reshape(B, 4)

    def layer(slots, positions):
        n = len(slots)
        x = torch.from_numpy(rng.standard_normal((n, Hq + 2 * Hkv, D)).astype(np.float32)).bfloat16().cuda()
        q = pkd.rope_cache_write(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], dev(positions), table_cs, dev(slots), cache)
        return q

    def slot(row, t):
        return row[t // P].astype(np.int64) * P + t % P

    # the common prompt
    t = np.arange(n0)
    q = layer(slot(pre, t), t)
    one = dev(np.array([0, n0], np.int32))
    out, lse = pkd.paged_attention(q, cache, dev(pre[None].astype(np.int32)), dev(np.array([n0], np.int32)), one, scale,
                                   softcap=30.0, max_query_len=n0)
    r = ref.attention(ref.values(q.cpu()), ref.values(cache.cpu()), pre[None], [n0], [0, n0], scale, softcap=30.0)
    ref.check(out.cpu(), lse.cpu(), r, "bf16", what="prompt")
    # the own prompts behind it, chunked on the whole context
    both = np.concatenate([np.tile(pre, (B, 1)), rows], 1).astype(np.int32)
    starts = np.concatenate([[0], np.cumsum(own)]).astype(np.int32)
    q = layer(np.concatenate([slot(rows[b], np.arange(own[b])) for b in range(B)]),
              np.concatenate([n0 + np.arange(own[b]) for b in range(B)]))
    lens = np.array([n0 + n for n in own], np.int32)
    out, lse = pkd.paged_attention(q, cache, dev(both), dev(lens), dev(starts), scale, softcap=30.0, max_query_len=max(own))
    r = ref.attention(ref.values(q.cpu()), ref.values(cache.cpu()), both, lens, starts, scale, softcap=30.0)
    ref.check(out.cpu(), lse.cpu(), r, "bf16", what="chunk")
    # a step: appended, then decoded with the prefix shared
    q = layer(np.array([slot(rows[b], np.array([own[b]]))[0] for b in range(B)]), n0 + np.array(own))
    out, lse = pkd.prefix_decode(q.view(B, 1, Hq, D), cache, dev(pre[None].astype(np.int32)), dev(np.array([n0], np.int32)),
                                 dev(rows.astype(np.int32)), dev(np.array(own, np.int32) + 1), scale, softcap=30.0)
    r = ref.attention(ref.values(q.cpu()), ref.values(cache.cpu()), both, lens + 1, np.arange(B + 1), scale, softcap=30.0)
    ref.check(out.view(B, Hq, D).cpu(), lse.view(B, Hq).cpu(), r, "bf16", what="step")


def test_captured_and_replayed():
    import paged_kv_decode_15_gb300 as pkd
    s = Shared(prefixes=[900], group_start=[0, 4], own=[10, 20, 300, 1], sq=1, Hq=8, Hkv=2, D=128, seed=8)
    c = s.c
    args = [dev(c.q).view(4, 1, 8, 128), dev(c.cache), dev(c.table[:1].copy()), dev(np.array([900], np.int32)),
            dev(c.table[1:].copy()), dev(s.own)]
    eager = pkd.prefix_decode(*args, c.scale)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o = pkd.prefix_decode(*args, c.scale)
    for _ in range(3):
        o[0].zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o[0], eager[0]) and torch.equal(o[1], eager[1])
    args[3].fill_(333)
    g.replay()
    torch.cuda.synchronize()
    s.prefixes = [333]
    ref.check(o[0].view(4, 8, 128).cpu(), o[1].view(4, 8).cpu(), s.reference(), "bf16")


@pytest.mark.parametrize("kind", [torch.float32, torch.float16])
def test_output_types(kind):
    Shared(prefixes=[300], group_start=[0, 3], own=[5, 60, 0], sq=1, Hq=4, Hkv=2, D=128, seed=9).verify(out_dtype=kind)


def test_two_threads_on_one_stream():
    import threading

    import paged_kv_decode_15_gb300 as pkd
    calls = []
    for i in range(2):
        s = Shared(prefixes=[900], group_start=[0, 4], own=[10, 20, 300, 1], sq=1, Hq=8, Hkv=2, D=128, seed=30 + i)
        c = s.c
        calls.append(([dev(c.q).view(4, 1, 8, 128), dev(c.cache), dev(c.table[:1].copy()), dev(np.array([900], np.int32)),
                       dev(c.table[1:].copy()), dev(s.own)], c.scale))
    want = [pkd.prefix_decode(*a, scale) for a, scale in calls]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        for _ in range(50):
            o = pkd.prefix_decode(*calls[i][0], calls[i][1])
            if not (torch.equal(o[0], want[i][0]) and torch.equal(o[1], want[i][1])):
                wrong.append(i)

    ts = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    [t.start() for t in ts]
    [t.join() for t in ts]
    assert not wrong
