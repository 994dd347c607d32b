"""The decoding kernels' paths that only large calls take: several runs a block and pages beyond 2^32 elements in the
attention, more than 16 columns of queries, more rows of an append than a launch has blocks for."""

import numpy as np
import pytest
import torch

import int8_quantized_matmul_amd as i8
from adapt_util import near, randn, wide
from decode_util import attention_bounds, ints, paged, pool
from gpu_util import DEV, say
from oracle import decode

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16


def _against(out, lse, q, K, V, tables, lens, heads, few, beams=1):
    """The query heads of the key-value heads `few` against the definition."""
    kv, d = K.shape[1], K.shape[3]
    group = heads // kv
    mine = [h * group + j for h in few for j in range(group)]
    pages = np.unique(tables[tables >= 0])
    small = np.full(tables.shape, -1, np.int32)
    small[tables >= 0] = np.searchsorted(pages, tables[tables >= 0])
    at = torch.as_tensor(pages, device=DEV).long()
    Ks, Vs = (torch.stack([p[:, h][at] for h in few], 1) for p in (K, V))
    qs = q.view(len(lens), heads, d)[:, mine].reshape(len(lens), -1)
    ro, rl = decode.attention(wide(qs), wide(Ks), wide(Vs), small, lens, d ** -0.5)
    bo, bl = attention_bounds(qs, Ks, Vs, small, lens, d ** -0.5, None, q.dtype)
    near(out.view(len(lens), heads, d)[:, mine].reshape(len(lens), -1), ro, bo, "out")
    got = wide(lse)[:, mine]
    some = np.isfinite(rl)
    assert np.array_equal(np.isneginf(got), ~some) and (np.abs(got[some] - rl[some]) <= bl[some]).all()


def _values(g, shape, dtype):
    return torch.randn(shape, generator=g, device=DEV).to(dtype)


@pytest.mark.parametrize("n,heads,kv,d,most,beams,dtype", [(40, 16, 16, 256, 5000, 1, F16), (70, 32, 32, 128, 4100, 1, BF16),
                                                           (90, 60, 60, 64, 2100, 1, F16), (40, 256, 16, 256, 5000, 1, BF16),
                                                           (88, 32, 16, 256, 5000, 4, F16)])
def test_several_runs_a_block(n, heads, kv, d, most, beams, dtype):
    """More tiles than 24 for every block that is resident at once, of sequences from nothing to `most` tokens."""
    rng = np.random.default_rng(d + heads)
    g = torch.Generator(device=DEV).manual_seed(d)
    page = 64
    lens = [int(x) for x in rng.integers(most // 4, most, size=n)]
    lens[3], lens[5], lens[-1] = 0, 1, most
    tables, pages = paged(rng, lens, page)
    tiles = [-(-x // 128) for x in lens]
    for i in range(0, n, beams) if beams > 1 else ():     # a group's beams share what half of its shortest has
        k = min(lens[i:i + beams]) // page // 2
        tables[i:i + beams, :k] = tables[i, :k]
        tiles[i:i + beams] = [t - k * page // 128 for t in tiles[i:i + beams]]
    K, V = (_values(g, (pages, kv, page, d), dtype) for _ in range(2))
    q = _values(g, (n, heads * d), dtype)
    blocks = 256 if d > 128 else 512 if d > 64 else 1024
    assert sum(tiles) * kv >= 2 * 24 * blocks
    say(f"  launch: decode_attention, {n} sequences, {heads} heads on {kv} of {d}")
    out, lse = i8.decode_attention(q, K, V, ints(tables), ints(lens), beams=beams)
    torch.cuda.synchronize()
    _against(out, lse, q, K, V, tables, lens, heads, (0, kv // 2, kv - 1) if heads < 100 else (kv - 1,))


@pytest.mark.parametrize("beams", [1, 2])
def test_far_pages_split_and_joined(beams):
    """Pages behind the 2^32nd element, in a table of more positions than a block takes whole."""
    rng = np.random.default_rng(10)
    heads, page, d = 64, 64, 128
    pages = 2 ** 32 // (heads * page * d) + 9
    K, V = (torch.empty((pages, heads, page, d), dtype=F16, device=DEV) for _ in range(2))
    lens, tables = [130, 70], np.full((2, 20), -1, np.int32)
    tables[0, :3], tables[1, :2] = [pages - 1, 3, pages - 2], [pages // 2 + 1, 0]
    for p in (K, V):
        for id in tables[tables >= 0]:
            p[int(id)] = randn(rng, (heads, page, d), F16)
    q = randn(rng, (2, heads * d), F16)
    say("  launch: decode_attention over 2 x 8.6 GB, split")
    out, lse = i8.decode_attention(q, K, V, ints(tables), ints(lens), beams=beams)
    torch.cuda.synchronize()
    _against(out, lse, q, K, V, tables, lens, heads, (0, 31, 63))


@pytest.mark.parametrize("heads,kv,d,beams", [(32, 1, 64, 4), (24, 1, 128, 4), (34, 2, 128, 3), (40, 2, 256, 2), (17, 1, 64, 64)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_beams_of_more_than_16_heads_a_key_value_head(heads, kv, d, beams, dtype):
    rng = np.random.default_rng(heads + beams)
    page, n = 16, 2 * beams
    lens = [int(x) for x in rng.integers(90, 400, size=n)]
    lens[0] = 0
    tables, pages = paged(rng, lens, page, width=40)
    for i in range(n):
        k = min(lens[i], lens[i - i % beams + 1]) // page
        tables[i, :k] = tables[i - i % beams + 1, :k]
    K, V = (torch.nan_to_num(pool(rng, tables, lens, pages, kv, page, d, dtype)) for _ in range(2))
    q = randn(rng, (n, heads * d), dtype)
    say(f"  launch: decode_attention, {beams} beams of {heads} heads on {kv}")
    out, lse = i8.decode_attention(q, K, V, ints(tables), ints(lens), beams=beams)
    alone = i8.decode_attention(q, K, V, ints(tables), ints(lens))
    torch.cuda.synchronize()
    _against(out, lse, q, K, V, tables, lens, heads, range(kv))
    _against(*alone, q, K, V, tables, lens, heads, range(kv))


def test_append_of_more_rows_than_blocks():
    """9300 rows of 32 heads: 9.5 million pieces of 16 bytes, where a launch has blocks for 8.4 million."""
    rng = np.random.default_rng(4)
    g = torch.Generator(device=DEV).manual_seed(4)
    s, heads, d, page, n = 9300, 32, 128, 32, 3
    room = [4000, 3300, 2000]
    tables, pages = paged(rng, room, page)
    seq = np.repeat(np.arange(n), room)[:s]
    pos = np.concatenate([np.arange(k) for k in room])[:s]
    order = rng.permutation(s)
    K, V = (torch.randint(-30000, 30000, (s, heads * d), generator=g, device=DEV, dtype=torch.int16).view(F16) for _ in range(2))
    Kp, Vp = (torch.zeros((pages, heads, page, d), dtype=F16, device=DEV) for _ in range(2))
    say("  launch: cache_append, 9300 rows of 32 heads")
    i8.cache_append(K, V, Kp, Vp, ints(tables), ints(pos[order]), ints(seq[order]))
    torch.cuda.synchronize()
    ids = torch.as_tensor(tables[seq[order], pos[order] // page], device=DEV).long()
    slot = torch.as_tensor(pos[order] % page, device=DEV).long()
    for rows, pool_ in ((K, Kp), (V, Vp)):
        bits = pool_.view(torch.int16)
        assert torch.equal(bits[ids, :, slot].reshape(s, -1), rows.view(torch.int16))
        bits[ids, :, slot] = 0
        assert not bits.any()
