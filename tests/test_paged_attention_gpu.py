"""Ragged paged attention on the GPU against the plain 64-bit reference: steps and
prompts, every mask and score modification, ragged and odd sizes, rows without
keys, strides, streams, graphs, bad pages."""
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


def dev(x, dtype=None):
    return None if x is None else torch.as_tensor(x, dtype=dtype).cuda()


def run(c, *, slopes=None, prefix_lens=None, doc_start=None, **kw):
    import paged_kv_decode_15_gb300 as pkd
    kw.setdefault("max_query_len", max(1, int(c.news.max(initial=1))))
    ws = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    pkd.workspace_init(ws)
    out, lse = pkd.paged_attention(
        dev(c.q), dev(c.cache), dev(c.table), dev(c.lens), dev(c.starts), c.scale, alibi_slopes=dev(slopes, torch.float32),
        prefix_lens=dev(prefix_lens, torch.int32), doc_start=dev(doc_start, torch.int32), workspace=ws, **c.scales(), **kw)
    status = pkd.workspace_check(ws)
    return out.cpu(), lse.cpu(), status


def verify(c, what="", out_dtype=None, **kw):
    import paged_kv_decode_15_gb300 as pkd
    call = dict(kw)
    if out_dtype:
        call["out_dtype"] = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}[out_dtype]
    out, lse, status = run(c, **call)
    assert status == pkd.OK
    kw.pop("max_query_len", None)
    kw.pop("max_kv_len", None)
    ref.check(out, lse, c.reference(**kw), c.dtype, out_dtype, what)


def slopes_of(Hq):
    return 2.0 ** (-8.0 * (np.arange(Hq) + 1) / Hq)


# ---------------------------------------------------------------- steps
@pytest.mark.parametrize("dtype,Hq,Hkv,D,P", [("bf16", 8, 2, 128, 16), ("fp16", 4, 4, 64, 32), ("fp8", 16, 2, 128, 64),
                                              ("bf16", 14, 2, 64, 48), ("fp8", 7, 1, 128, 16), ("fp16", 16, 1, 128, 16)])
@pytest.mark.parametrize("mod", ["plain", "cap", "bias", "cap+bias", "window"])
def test_steps(dtype, Hq, Hkv, D, P, mod):
    lens = [1, 2, 15, 16, 17, 63, 64, 65, 300, 1037]
    c = ref.Paged(lens=lens, news=[1] * len(lens), Hq=Hq, Hkv=Hkv, D=D, P=P, dtype=dtype, seed=Hq * D + P)
    kw = {}
    if "cap" in mod:
        kw["softcap"] = 5.0
    if "bias" in mod:
        kw["slopes"] = slopes_of(Hq)
    if mod == "window":
        kw["window"] = 37
    verify(c, mod, **kw)


def test_steps_of_several_tokens_with_masks():
    c = ref.Paged(lens=[5, 40, 0, 133, 700, 3], news=[3, 1, 0, 4, 2, 4], Hq=8, Hkv=2, D=128, seed=3, extra_tokens=2)
    doc = np.array([0, 4, 2, 7, 100, 140, 0, 130, 690, 699, 0, 0, 0, 1, 0, 0])  # token 5: behind its position
    verify(c, "docs", doc_start=doc)
    verify(c, "prefix", prefix_lens=[5, 40, 9, 131, 2, 0], window=20)
    verify(c, "dense", causal=False)
    verify(c, "dense window", causal=False, window=9)


@pytest.mark.parametrize("dtype,D,Hkv", [("bf16", 128, 8), ("fp8", 128, 8), ("fp16", 64, 2)])
def test_steps_with_split_keys(dtype, D, Hkv):
    """Long requests, one short and one empty: several chunks merged by LSE."""
    c = ref.Paged(lens=[6000, 1, 0, 2777], news=[1, 1, 0, 2], Hq=2 * Hkv, Hkv=Hkv, D=D, dtype=dtype, seed=9)
    verify(c, "split", softcap=30.0, slopes=slopes_of(2 * Hkv))


# --------------------------------------------------------------- prompts
@pytest.mark.parametrize("dtype,Hq,Hkv,D,P", [("bf16", 4, 1, 128, 16), ("fp16", 2, 2, 64, 64), ("bf16", 7, 1, 64, 48),
                                              ("fp16", 8, 1, 128, 32), ("bf16", 1, 1, 128, 16), ("fp8", 4, 2, 128, 32),
                                              ("fp8", 9, 1, 128, 16)])
@pytest.mark.parametrize("mod", ["plain", "cap", "bias", "cap+bias", "window", "dense"])
def test_prompts(dtype, Hq, Hkv, D, P, mod):
    lens = [1, 17, 129, 200, 333]
    c = ref.Paged(lens=lens, news=[1, 17, 128, 150, 333], Hq=Hq, Hkv=Hkv, D=D, P=P, dtype=dtype, seed=Hq * D + P)
    kw = {}
    if "cap" in mod:
        kw["softcap"] = 5.0
    if "bias" in mod:
        kw["slopes"] = slopes_of(Hq)
    if mod == "window":
        kw["window"] = 41
    if mod == "dense":
        kw["causal"] = False
    verify(c, mod, **kw)


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_prompts_with_prefix_and_document_masks(dtype):
    c = ref.Paged(lens=[300, 0, 260, 90], news=[290, 0, 40, 90], Hq=8, Hkv=2, D=128, dtype=dtype, seed=5, extra_tokens=3)
    verify(c, "prefix", prefix_lens=[100, 3, 250, 0])
    verify(c, "prefix+window", prefix_lens=[100, 3, 250, 60], window=30)
    rng = np.random.default_rng(1)
    doc = np.zeros(c.T, np.int64)
    doc[:290] = np.repeat([0, 57, 130, 131, 260], [67, 73, 1, 129, 20])
    doc[290:330] = 250          # before 250: no key at all
    doc[330:420] = rng.integers(0, 90, 90)
    verify(c, "docs", doc_start=doc)
    verify(c, "docs+cap", doc_start=doc, softcap=20.0)


@pytest.mark.parametrize("slopes", [False, True])
@pytest.mark.parametrize("dtype,D,Hq,Hkv", [("bf16", 128, 4, 4), ("fp16", 64, 3, 1), ("fp8", 128, 4, 4)])
def test_documents_that_end_inside_a_row_tile(dtype, D, Hq, Hkv, slopes):
    """Many key tiles that some rows of a warp see whole and the others not at all; a key
    that is not finite reaches the tokens of its own document only."""
    c = ref.Paged(lens=[1500, 700], news=[700, 500], Hq=Hq, Hkv=Hkv, D=D, dtype=dtype, seed=24, spread=3.0)
    first, second = np.arange(800, 1500), np.arange(200, 700)
    doc = np.concatenate([np.select([first < 811, first < 1203], [0, 811], 1203),
                          np.select([second < 443, second < 460], [0, 443], 460)])
    kw = dict(slopes=slopes_of(Hq)) if slopes else {}
    verify(c, "documents", doc_start=doc, **kw)
    good, lse, _ = run(c, doc_start=doc, **kw)
    c.cache[c.table[0, 500 // c.P], :, 500 % c.P, :D] = float("nan" if dtype == "fp8" else "inf")
    out, lse2, _ = run(c, doc_start=doc, **kw)
    assert torch.equal(out[11:], good[11:]) and torch.equal(lse2[11:], lse[11:])


@pytest.mark.parametrize("dtype,D,Hq,Hkv", [("bf16", 128, 8, 1), ("bf16", 64, 12, 2), ("fp8", 128, 8, 2)])
def test_few_rows_over_many_keys_split(dtype, D, Hq, Hkv):
    """A small chunk of queries on a long context: the keys are split and merged."""
    c = ref.Paged(lens=[3000, 1024, 40], news=[20, 5, 40], Hq=Hq, Hkv=Hkv, D=D, dtype=dtype, seed=2)
    import paged_kv_decode_15_gb300 as pkd
    need = pkd.load_library().pkd_paged_attention_workspace_size(3, c.T, 40, Hq, Hkv, D, 16, 3008, pkd.BF16, None)
    assert need > 256 + 4 * 65536 + c.T * Hq * D * 4  # partial results are planned
    verify(c, "split")
    verify(c, "split window", window=1500)
    verify(c, "split prefix", prefix_lens=[2995, 0, 11], softcap=15.0)


@pytest.mark.parametrize("window", [1030, 900, 2 ** 31 - 1])
def test_unsplit_prompts_whose_keys_start_late(window):
    """Enough row tiles to leave the keys unsplit, first keys past 1024."""
    c = ref.Paged(lens=[2500], news=[40], Hq=1024, Hkv=8, D=64, dtype="fp16", seed=16)
    import paged_kv_decode_15_gb300 as pkd
    need = pkd.load_library().pkd_paged_attention_workspace_size(1, 40, 40, 1024, 8, 64, 16, 2512, pkd.FP16, None)
    assert need == 256 + 4 * 65536
    verify(c, "late", window=window)


def test_large_scores_move_the_reference_maximum():
    """Scores that grow by hundreds along the keys: accumulators are rescaled."""
    c = ref.Paged(lens=[700], news=[300], Hq=2, Hkv=1, D=64, dtype="fp16", seed=4)
    kv = c.cache.float()
    order = torch.from_numpy(c.table[0].astype(np.int64))
    for t in range(700):
        kv[order[t // 16], 0, t % 16, :64] *= 0.02 * (1 + t % 350)
    c.cache = kv.to(torch.float16)
    verify(c, "growing")
    verify(c, "growing, capped", softcap=50.0)


def test_hundreds_of_requests():
    rng = np.random.default_rng(8)
    news = rng.integers(0, 4, 700)
    news[rng.integers(0, 700, 8)] = 33
    c = ref.Paged(lens=news + rng.integers(0, 9, 700), news=news, Hq=2, Hkv=1, D=64, seed=6)
    verify(c, "many")


@pytest.mark.parametrize("out_dtype", ["fp32", "bf16", "fp16"])
def test_output_types(out_dtype):
    verify(ref.Paged(lens=[50, 20], news=[1, 1], Hq=4, Hkv=2, D=128, dtype="fp16", seed=1), "step", out_dtype)
    verify(ref.Paged(lens=[50, 20], news=[44, 20], Hq=4, Hkv=2, D=128, dtype="fp16", seed=1), "prompt", out_dtype)


# ------------------------------------------- what a caller may do around it
@pytest.mark.parametrize("news", [[1, 2, 0], [30, 50, 0]])
def test_padding_tokens_and_strided_queries(news):
    """q as a slice of a fused projection; rows of no request keep their contents."""
    import paged_kv_decode_15_gb300 as pkd
    c = ref.Paged(lens=[60, 55, 20], news=news, Hq=4, Hkv=2, D=128, seed=7, extra_tokens=5)
    c.q[c.starts[-1]:] = float("nan")
    fused = torch.randn(c.T, 8, 128).to(torch.bfloat16)
    fused[:, 2:6] = c.q
    out = torch.full((c.T, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((c.T, 4), 7.0, device="cuda")
    pkd.paged_attention(dev(fused)[:, 2:6], dev(c.cache), dev(c.table), dev(c.lens), dev(c.starts), c.scale,
                        max_query_len=max(news), out=out, lse=lse)
    n = int(c.starts[-1])
    assert (out[n:] == 7).all() and (lse[n:] == 7).all()
    r = c.reference()
    ref.check(out[:n].cpu(), lse[:n].cpu(), [x[:n] for x in r], "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("news", [[1, 1], [70, 40]])
def test_bad_pages_are_skipped_and_reported(news, dtype):
    import paged_kv_decode_15_gb300 as pkd
    c = ref.Paged(lens=[100, 90], news=news, Hq=4, Hkv=2, D=128, dtype=dtype, seed=11)
    c.table[0, 2] = -1
    c.table[1, 0] = c.num_pages
    out, lse, status = run(c)
    assert status == pkd.EDEVICE_BOUNDS
    ref.check(out, lse, c.reference(), dtype)


def test_bad_lengths_and_starts_are_clamped_and_reported():
    import paged_kv_decode_15_gb300 as pkd
    for news in ([1, 1], [30, 30]):
        c = ref.Paged(lens=[64, 64], news=news, Hq=4, Hkv=2, D=128, seed=12)
        good, lse, _ = run(c)
        starts, lens = c.starts.copy(), c.lens.copy()
        c.lens = np.array([64, 65], np.int32)   # beyond max_kv_len: as 64
        out, _, status = run(c, max_kv_len=64)
        assert status == pkd.EDEVICE_BOUNDS and torch.equal(out, good)
        c.lens, c.starts = lens, starts.copy()
        c.starts[2] += 100                      # past the tokens: as T
        out, _, status = run(c)
        assert status == pkd.EDEVICE_BOUNDS and torch.equal(out, good)


@pytest.mark.parametrize("dtype,Hq,D", [("bf16", 14, 128), ("fp16", 6, 64), ("fp8", 10, 128)])
@pytest.mark.parametrize("cap", [0.0, 4.0])
def test_results_do_not_depend_on_the_schedule(dtype, Hq, D, cap):
    """Row tiles with lanes to spare and key tiles that end early, hundreds of items in any
    order, after calls that leave large queries and keys on the SMs: the same bits every time."""
    import paged_kv_decode_15_gb300 as pkd
    rng = np.random.default_rng(25)
    news = rng.integers(20, 400, 24)
    c = ref.Paged(lens=news + rng.integers(0, 300, 24), news=news, Hq=Hq, Hkv=2, D=D, dtype=dtype, seed=26, spread=4.0)
    args = [dev(x) for x in (c.q, c.cache, c.table, c.lens, c.starts)]
    call = lambda: pkd.paged_attention(*args, c.scale, softcap=cap, max_query_len=400, **c.scales())
    big = ref.Paged(lens=[400] * 40, news=[200] * 40, Hq=16, Hkv=2, D=D, dtype=dtype, seed=27, spread=50.0)
    loud = [dev(x) for x in (big.q, big.cache, big.table, big.lens, big.starts)]
    small = ref.Paged(lens=[400] * 40, news=[200] * 40, Hq=16, Hkv=2, D=D, dtype=dtype, seed=27, spread=0.0)
    quiet = [dev(small.q)] + loud[1:]
    out, lse = call()
    for i in range(10):
        pkd.paged_attention(*(loud if i % 2 else quiet), 1.0, softcap=cap, max_query_len=200)
        again = call()
        assert torch.equal(again[0], out) and torch.equal(again[1], lse)


def test_requests_that_overlap_stay_inside_the_plan():
    """A query_start that falls 299 times: every second request is all 256 tokens, 38400
    row-tile pairs for a plan of at most 728; all requests alike, so the first's rows are right."""
    import paged_kv_decode_15_gb300 as pkd
    c = ref.Paged(lens=[2000], news=[256], Hq=128, Hkv=1, D=64, seed=23)
    good, lse, status = run(c)
    assert status == pkd.OK
    q, cache = dev(c.q), dev(c.cache)
    table, lens = dev(c.table).expand(600, -1).contiguous(), dev(c.lens).expand(600).contiguous()
    starts = torch.tensor([0, 256] * 300 + [0], dtype=torch.int32, device="cuda")
    ws = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    pkd.workspace_init(ws)
    got = pkd.paged_attention(q, cache, table, lens, starts, c.scale, max_query_len=256, workspace=ws)
    assert pkd.workspace_check(ws) == pkd.EDEVICE_BOUNDS
    assert torch.equal(got[0].cpu(), good) and torch.equal(got[1].cpu(), lse)
    assert not ws[256:256 + 4 * 65536].any(), "arrival counters are zero again"
    again = pkd.paged_attention(q, cache, table[:1], lens[:1], dev(c.starts), c.scale, workspace=ws)
    assert torch.equal(again[0].cpu(), good) and torch.equal(again[1].cpu(), lse)


@pytest.mark.parametrize("news", [[1, 1, 1], [100, 37, 64]])
def test_captured_and_replayed_on_another_stream(news):
    """Captured once, replayed on new lengths; two graphs in turn on two streams."""
    import paged_kv_decode_15_gb300 as pkd
    c = ref.Paged(lens=[2000, 300, 64], news=news, Hq=4, Hkv=1, D=128, seed=13)
    args = [dev(c.q), dev(c.cache), dev(c.table), dev(c.lens), dev(c.starts)]
    kw = dict(max_query_len=max(news), softcap=30.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        eager = [x.clone() for x in pkd.paged_attention(*args, c.scale, **kw)]
    side.synchronize()
    ref.check(eager[0].cpu(), eager[1].cpu(), c.reference(softcap=30.0), "bf16")
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = pkd.paged_attention(*args, c.scale, **kw)
        graphs.append((g, o))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        for (g, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for _, o in graphs:
        assert torch.equal(o[0], eager[0]) and torch.equal(o[1], eager[1])
    shorter = np.array([max(n, L - 40) for n, L in zip(news, c.lens)], np.int32)
    args[3].copy_(torch.from_numpy(shorter))
    graphs[0][0].replay()
    torch.cuda.synchronize()
    c.lens = shorter
    ref.check(graphs[0][1][0].cpu(), graphs[0][1][1].cpu(), c.reference(softcap=30.0), "bf16")


def test_one_workspace_serves_any_plan_and_results_repeat():
    import paged_kv_decode_15_gb300 as pkd
    ws = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    pkd.workspace_init(ws)
    cases = [ref.Paged(lens=[3000, 700], news=n, Hq=8, Hkv=1, D=128, seed=14) for n in ([1, 1], [40, 30], [700, 700], [2, 1])]
    first = []
    for _ in range(3):
        for i, c in enumerate(cases):
            o = pkd.paged_attention(dev(c.q), dev(c.cache), dev(c.table), dev(c.lens), dev(c.starts), c.scale,
                                    max_query_len=int(c.news.max()), workspace=ws)
            if len(first) == i:
                first.append(o)
            else:
                assert torch.equal(o[0], first[i][0]) and torch.equal(o[1], first[i][1])
    assert pkd.workspace_check(ws) == pkd.OK


def test_key_offsets_past_32_bits():
    """A cache of more than 4 GB: the last pages, by bytes and by elements."""
    c = ref.Paged(lens=[200, 130], news=[100, 130], Hq=4, Hkv=8 // 2, D=128, P=64, seed=15)
    big = 2 ** 33 // (4 * 64 * 256 * 2) + 8   # pages: 8 GB of bf16
    import paged_kv_decode_15_gb300 as pkd
    cache = torch.empty((big, 4, 64, 256), dtype=torch.bfloat16, device="cuda")
    cache[-c.num_pages:] = dev(c.cache)
    table = dev(c.table) + (big - c.num_pages)
    for news in ([100, 130], [1, 1]):
        starts = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
        c.news, c.starts, T = np.array(news), starts, int(starts[-1])
        out, lse = pkd.paged_attention(dev(c.q)[:T], cache, table, dev(c.lens), dev(starts), c.scale, max_query_len=max(news))
        q = c.q
        c.q = c.q[:T]
        c.T = T
        ref.check(out.cpu(), lse.cpu(), c.reference(), "bf16")
        c.q = q


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("cap", [1e-3, 0.5, 1000.0, 1e6])
def test_caps_of_any_size(cap, dtype):
    """A cap far below the scores (all of them at its ends) and far above (no effect)."""
    verify(ref.Paged(lens=[300, 40], news=[1, 1], Hq=4, Hkv=2, D=128, dtype=dtype, seed=17), "step", softcap=cap)
    verify(ref.Paged(lens=[300, 140], news=[270, 140], Hq=4, Hkv=2, D=128, dtype=dtype, seed=17), "prompt", softcap=cap)


@pytest.mark.parametrize("docs", [False, True])
@pytest.mark.parametrize("slopes", [False, True])
def test_many_row_tiles_of_unlike_weight(docs, slopes):
    """Enough row tiles to be ordered by their keys, of several requests, some empty."""
    c = ref.Paged(lens=[900, 0, 60, 300, 1, 33], news=[37, 0, 30, 20, 1, 33], Hq=256, Hkv=4, D=64, seed=18, extra_tokens=1)
    doc = np.zeros(c.T, np.int64)
    doc[:37] = np.repeat([0, 640, 880, 899], [11, 7, 18, 1])
    doc[37:67] = 31
    kw = dict(slopes=slopes_of(256)) if slopes else {}
    verify(c, "ordered", window=700, **(dict(doc_start=doc) if docs else {}), **kw)


@pytest.mark.parametrize("news", [[3, 1], [60, 10]])
def test_more_tokens_than_announced_are_cut_and_reported(news):
    import paged_kv_decode_15_gb300 as pkd
    c = ref.Paged(lens=[100, 90], news=news, Hq=4, Hkv=2, D=64, seed=19)
    out, lse, status = run(c, max_query_len=news[0] - 1)
    assert status == pkd.EDEVICE_BOUNDS
    # the request's first tokens, as the last ones of its keys
    cut = ref.Paged(lens=[100, 90], news=news, Hq=4, Hkv=2, D=64, seed=19)
    starts = np.array([0, news[0] - 1], np.int32)
    want = ref.attention(ref.values(cut.q), np.nan_to_num(ref.values(cut.cache)), cut.table[:1], cut.lens[:1], starts, cut.scale)
    n = news[0] - 1
    ref.check(out[:n], lse[:n], [x[:n] for x in want], "bf16")


def test_calls_on_streams_of_their_own_and_from_two_threads():
    import threading

    import paged_kv_decode_15_gb300 as pkd
    cases = [ref.Paged(lens=[3000, 500], news=n, Hq=8, Hkv=1, D=128, seed=20 + i) for i, n in enumerate(([1, 1], [33, 20]))]
    args = [[dev(x) for x in (c.q, c.cache, c.table, c.lens, c.starts)] for c in cases]
    want = [pkd.paged_attention(*a, c.scale, max_query_len=int(c.news.max())) for a, c in zip(args, cases)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in cases], {}

    def work(i, stream):
        for _ in range(20):
            got[i] = pkd.paged_attention(*args[i], cases[i].scale, max_query_len=int(cases[i].news.max()), stream=stream)

    for use in (streams, [None, None]):   # a stream each, then both on the default one
        ts = [threading.Thread(target=work, args=(i, s)) for i, s in enumerate(use)]
        [t.start() for t in ts]
        [t.join() for t in ts]
        torch.cuda.synchronize()
        for i, w in enumerate(want):
            assert torch.equal(got[i][0], w[0]) and torch.equal(got[i][1], w[1])


def test_refusals_of_the_binding():
    import paged_kv_decode_15_gb300 as pkd
    c = ref.Paged(lens=[40], news=[4], Hq=4, Hkv=2, D=64, seed=22)
    q, cache, table, lens, starts = (dev(x) for x in (c.q, c.cache, c.table, c.lens, c.starts))
    call = lambda **kw: pkd.paged_attention(*[kw.pop(n, x) for n, x in zip(("q", "cache", "table", "lens", "starts"),
                                                                          (q, cache, table, lens, starts))], c.scale, **kw)
    for kw, error in ((dict(q=c.q), ValueError), (dict(q=q.transpose(0, 1)), ValueError), (dict(cache=cache[:, :, :, :64]), ValueError),
                      (dict(table=table.long()), TypeError), (dict(lens=lens.expand(2)), ValueError), (dict(starts=starts[:1]), ValueError),
                      (dict(prefix_lens=lens.long()), ValueError), (dict(doc_start=lens), ValueError),
                      (dict(alibi_slopes=torch.ones(3, device="cuda")), ValueError),
                      (dict(out=torch.empty(4, 4, 32, device="cuda")), ValueError), (dict(softcap=-1.0), pkd.PkdError),
                      (dict(q=q.half()), pkd.PkdError), (dict(max_query_len=0), pkd.PkdError),
                      (dict(window=(1 << 32) + 5), ValueError), (dict(window=-1), ValueError),
                      (dict(max_kv_len=1 << 32), ValueError), (dict(max_query_len=(1 << 32) + 4), ValueError)):
        with pytest.raises(error):
            call(**kw)
    assert pkd.paged_attention(q[:0], cache, table, lens, torch.zeros_like(starts), c.scale)[0].shape == (0, 4, 64)
