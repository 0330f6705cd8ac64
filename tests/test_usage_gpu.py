"""The usage that the README shows of a cache of bounded size, run as it stands there."""
import os

import numpy as np
import pytest
import torch

import paged_kv_decode_15_gb300 as pkd
from tests.test_cache_eviction_gpu import dev, problem

pytestmark = pytest.mark.gpu
README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def usage():
    """Its lines for a prompt, and those for a step."""
    with open(README) as f:
        text = f.read()
    block = text.split("    # a cache that keeps at most 1024 keys", 1)[1].split("    # lengths, pages, starts", 1)[0]
    prompt, step = ("#" + block).split("    # a step of decoding", 1)
    return ["\n".join(line[4:] if line.startswith("    ") else line for line in part.splitlines()) for part in (prompt, "#" + step)]


def test_the_first_and_the_latest_keys_stay_through_prompt_and_steps():
    lens, budget, H, Hq, D = [1500, 1024, 1101, 30], 1024, 2, 8, 64
    p = problem(1, new=lens, lens=lens, heads=Hq, kv=H, dim=D, page=16, dtype="bf16", columns=100)
    rows = torch.cat([p["cache"][p["table"][b, np.arange(L) // 16], :, np.arange(L) % 16] for b, L in enumerate(lens)]).cuda()
    table = p["table"].copy()
    free = sorted(set(range(len(p["cache"]))) - set(table.ravel().tolist()))
    table[1, 64], table[3, 2] = free[:2]  # (the requests that grow into a new page)
    x = dict(pkd=pkd, torch=torch, q=p["q"].cuda(), key=rows[..., :D].contiguous(), value=rows[..., D:].contiguous(), longest=1500,
             kv_cache=p["cache"].cuda(), block_table=dev(table), seq_lens=dev(p["lens"]), query_start=dev(p["starts"]),
             scale=p["scale"], page_size=16, requests=torch.arange(4, device="cuda"))
    prompt, step = usage()
    pkd.workspace_check()
    exec(prompt, x)
    assert x["kept_lens"].tolist() == [1024, 1024, 1024, 30]
    g = torch.Generator(device="cuda").manual_seed(2)
    x["query_start"] = torch.arange(5, dtype=torch.int32, device="cuda")
    for i in range(4):
        if i:
            exec_step(x, step, g, H, Hq, D)
        for b, L in enumerate(lens):
            n, context = int(x["kept_lens"][b]), L + i
            for h in range(H):
                there = sorted(x["positions"][b, h, :n].tolist())
                assert n == min(budget, context) and len(set(there)) == n
                assert there[:4] == [0, 1, 2, 3] and there[-min(64, n):] == list(range(context - min(64, n), context))
    assert pkd.workspace_check() == pkd.OK


def exec_step(x, step, g, H, Hq, D):
    new = [torch.randn((4, h, D), device="cuda", generator=g).bfloat16() for h in (Hq, H, H)]
    x.update(q=new[0][:, None], key=new[1], value=new[2])
    exec(step, x)
