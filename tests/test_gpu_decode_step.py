"""The decoding step as the README shows it, in a pool that runs out of pages:
every beam's cache holds its own tokens, whoever found no room."""

import os
import re

import numpy as np
import pytest
import torch

import int8_quantized_matmul_amd as i8
from decode_util import ints
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _step():
    blocks = re.findall(r"```python\n(.*?)```", open(os.path.join(ROOT, "README.md")).read(), re.S)
    return compile(next(b for b in blocks if "cache_append" in b), "README.md", "exec")


@pytest.mark.parametrize("pages", [7, 9, 40])
def test_beams_keep_their_tokens_when_pages_run_out(pages):
    g = torch.Generator(device=DEV).manual_seed(pages)
    kv, page, d, n, vocab, prompt = 2, 16, 16, 4, 50, 20
    shape = (pages, kv, page, d)
    K, V = (torch.zeros(shape, dtype=torch.float16, device=DEV) for _ in range(2))
    say(f"  launch: the README's step in {pages} pages")
    none = ints(np.full((0, 5), -1)), ints([]), ints(np.zeros(pages))
    tables, lens, refs, _ = i8.cache_fork(*none, page, parents=ints([-1]), grow=ints([prompt]))
    first = torch.randn((prompt, kv * d), generator=g, device=DEV).half()
    i8.cache_append(first, first, K, V, tables, ints(range(prompt)), ints([0] * prompt))
    tables, lens, refs, _ = i8.cache_fork(tables, lens, refs, page, parents=ints([0] * n), grow=ints([1] * n), pools=[K, V])
    assert lens.tolist() == [prompt + 1] * n
    s = dict(i8=i8, torch=torch, K_pages=K, V_pages=V, tables=tables, lens=lens, refs=refs, page=page, pos=lens - 1,
             scores=torch.zeros((1, n), device=DEV), one_each=ints([1] * n),
             history=torch.zeros((n, 0), dtype=torch.int32, device=DEV))
    texts, short = [list(first) for _ in range(n)], 0
    for _ in range(45):
        s["k"], s["q"] = (torch.randn((n, kv * d), generator=g, device=DEV).half() for _ in range(2))
        s["v"], s["logits"] = s["k"], 3 * torch.randn((n, vocab), generator=g, device=DEV)
        for j in range(n):
            if s["pos"][j] >= 0:
                texts[j].append(s["k"][j])
        exec(_step(), s)
        texts = [list(texts[p]) for p in s["parents"].view(-1).tolist()]
        short += int(s["state"][2])
        for j, row in enumerate(s["tables"].tolist()):
            assert int(s["lens"][j]) - int(s["pos"][j] >= 0) == len(texts[j])
            for pool in (K, V):
                held = torch.stack([pool[row[t // page], :, t % page].reshape(-1) for t in range(len(texts[j]))])
                assert torch.equal(held, torch.stack(texts[j]))
    # 5 pages a sequence end the longest run; fewer pages end it earlier
    assert short > 0 if pages < 40 else len(texts[0]) == prompt + 45
