"""A beam search as a user runs it: layer norm, the fused int8 projection with adapters, its rows into a paged cache,
attention over it, the logits, the selection, and the cache following the chosen beams, with compactions in between.

Every call is checked against its definition on the inputs that it had (the integers exactly, the attention within
decode_util.attention_bounds). Keys and values depend on a token and its position alone here, so at the end every
beam's cache must hold, bit for bit, what its own history of tokens gives."""

import numpy as np
import pytest
import torch

import int8_quantized_matmul_amd as i8
from adapt_util import near, wide
from decode_util import attention_bounds, ints
from gpu_util import DEV, say
from oracle import decode

pytestmark = pytest.mark.gpu

H, HEADS, KV, D, PAGE, VOCAB = 256, 4, 4, 64, 16, 640


class _Layer:
    def __init__(self, seed):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.embed = torch.randn((VOCAB, H), generator=g, device=DEV).half()
        self.places = torch.randn((256, H), generator=g, device=DEV).half()
        W = (0.08 * torch.randn((H, 3 * HEADS * D), generator=g, device=DEV)).half()
        self.W, (self.Wq, self.c_w) = W, i8.quantize_colwise_weights(W)
        self.A = (torch.randn((2, 4, H), generator=g, device=DEV) / 16).half()
        self.B = (0.1 * torch.randn((2, 4, 3 * HEADS * D), generator=g, device=DEV)).half()
        self.scale = torch.tensor([1.0, 0.5], device=DEV)
        self.w, self.b = torch.ones(H, device=DEV), torch.zeros(H, device=DEV)
        self.head = i8.pack_fp16_weights((torch.randn((HEADS * D, VOCAB), generator=g, device=DEV) * 0.3).half())

    def rows(self, tokens, positions, ids):
        """The fused projection's rows of each token, one after another (so that a row does not depend on its neighbours)."""
        x = self.embed[tokens.long()] + self.places[positions.long()]
        n, _, _ = i8.layer_norm(x, self.w, self.b)
        out = []
        for i in range(len(n)):
            c = i8.forward(n[i:i + 1].contiguous(), self.Wq, self.c_w, self.W)
            out.append(i8.lora_forward(n[i:i + 1], self.A, self.B, ids[i:i + 1], self.scale, base=c, Y=c)[0])
        return torch.cat(out)


@pytest.mark.parametrize("requests,beams,seed", [(2, 3, 0), (1, 5, 1), (3, 1, 2)])
def test_beam_search(requests, beams, seed):
    rng = np.random.default_rng(seed)
    layer, n = _Layer(seed), requests * beams
    M, P = 6, requests * 5 + n * 4
    prompts = [list(rng.integers(0, VOCAB, size=int(k))) for k in rng.integers(3, 40, size=requests)]
    store = torch.full((P, 2, KV * PAGE * D), float("nan"), dtype=torch.float16, device=DEV)     # keys and values of a page
    K, V = (store[:, i].unflatten(1, (KV, PAGE, D)) for i in range(2))
    ids = ints(np.arange(n) // beams % 3 - 1)
    slopes = torch.tensor([0.5, 0.25, 0.125, 0.0625], device=DEV)
    # the prompts: one sequence a request, grown from nothing
    none = ints(np.full((0, M), -1)), ints([]), ints(np.zeros(P))
    say(f"  launch: beam search, {requests} requests of {beams} beams")
    tables, lens, refs, state = i8.cache_fork(*none, PAGE, parents=ints([-1] * requests), grow=ints([len(p) for p in prompts]))
    assert lens.tolist() == [len(p) for p in prompts] and state.tolist()[1:] == [0, 0, 0]
    pos = ints([t for p in prompts for t in range(len(p))])
    seq = ints([i for i, p in enumerate(prompts) for _ in p])
    width = HEADS * D
    rows = layer.rows(ints([t for p in prompts for t in p]), pos, ids.view(requests, beams)[:, 0].contiguous()[seq.long()])
    i8.cache_append(rows[:, width:2 * width], rows[:, 2 * width:], K, V, tables, pos, seq)
    # the last prompt token's row asks; then one row a beam does
    history = [list(p) for p in prompts]
    last = np.cumsum([len(p) for p in prompts]) - 1
    q, here, scores = rows[torch.as_tensor(last, device=DEV)][:, :width], requests, torch.zeros((requests, 1), device=DEV)
    for step in range(24):
        t, l = tables.cpu().numpy(), lens.cpu().numpy()
        out, lse = i8.decode_attention(q, K, V, tables, lens, slopes=slopes, beams=here // requests)
        ro, rl = decode.attention(wide(q), wide(K), wide(V), t, l, D ** -0.5, wide(slopes))
        bo, bl = attention_bounds(q, K, V, t, l, D ** -0.5, wide(slopes), torch.float16)
        near(out, ro, bo, "out")
        assert (np.abs(wide(lse) - rl) <= bl).all()
        logits = i8.fp16_gemm(out, layer.head)
        total, parents, tokens, _ = i8.beam_select(logits, scores, beams)
        s, p, v, _ = decode.select(wide(logits), wide(scores), beams)
        assert np.abs(wide(total) - s).max() <= 2.0 ** -20 + 2.0 ** -23 * np.abs(s).max()
        chosen = list(zip(parents.view(-1).tolist(), tokens.view(-1).tolist()))
        assert sorted(chosen) == sorted(zip(p.reshape(-1).tolist(), v.reshape(-1).tolist()))
        old = tables.cpu().numpy(), lens.cpu().numpy(), refs.cpu().numpy()
        host = [store.cpu().numpy().copy()]
        grow = np.ones(n, np.int32)
        want = decode.fork(*old, PAGE, parents.view(-1).cpu().numpy(), grow, host)
        tables, lens, refs, state = i8.cache_fork(tables, lens, refs, PAGE, parents=parents.view(-1), grow=ints(grow), pools=[store])
        for a, b in zip((tables, lens, refs, state), want):
            assert np.array_equal(a.cpu().numpy(), b)
        assert np.array_equal(store.cpu().numpy().view(np.int16), host[0].view(np.int16)) and state.tolist()[2] == 0
        if step % 7 == 5:
            want = decode.compact(tables.cpu().numpy(), refs.cpu().numpy(), host)
            tables, refs, _, _ = i8.cache_compact(tables, refs, pools=[store])
            assert np.array_equal(tables.cpu().numpy(), want[0]) and np.array_equal(refs.cpu().numpy(), want[1])
            assert np.array_equal(store.cpu().numpy().view(np.int16), host[0].view(np.int16))
        history = [history[a] + [b] for a, b in chosen]
        scores, here = total, n
        rows = layer.rows(tokens.view(-1), lens - 1, ids)
        i8.cache_append(rows[:, width:2 * width], rows[:, 2 * width:], K, V, tables, lens - 1)
        q = rows[:, :width]
    # what each beam's pages hold is what its own tokens give
    t = tables.cpu().numpy()
    for j, tokens in enumerate(history):
        assert int(lens[j]) == len(tokens)
        who = ids[j:j + 1].expand(len(tokens)).contiguous()
        rows = layer.rows(ints(tokens), ints(np.arange(len(tokens))), who).view(len(tokens), 3, KV, D)
        for pages, part in ((K, rows[:, 1]), (V, rows[:, 2])):
            held = torch.stack([pages[int(t[j, i // PAGE]), :, i % PAGE] for i in range(len(tokens))])
            assert torch.equal(held, part)
