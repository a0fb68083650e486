"""Attention outputs of the serving calls against the fp64 oracle, within a bound
that does not grow with the length where nothing is lost (serving_bounds), and
prompts as long as the measured ones."""
import numpy as np
import pytest
import torch

from oracle import serving_oracle as SO
from serving_bounds import check, score_error
from test_gpu_serving import (D, DECODE, DEV, DTYPES, PACKED, SCALE, SENTINEL, _built, f64, make_cache,  # noqa: F401
                              make_packed, rnd, rows_of)

pytestmark = pytest.mark.gpu

rtp = pytest.importorskip("long_context_hybrid_b200")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", PACKED, ids=lambda c: f"{c[0][:12]}w{c[3]}")
def test_packed_outputs(case, dtype):
    lens, Hq, Hkv, window, heads, lead, tail, pad = case
    (q, k, v), cu, cu_d = make_packed(lens, Hq, Hkv, dtype, 111 + sum(lens), lead, tail, pad)
    v += 0.5                                     # values with a mean, so that a gain shows
    o = torch.full_like(q, SENTINEL)
    rtp.attn_packed(q, k, v, o, heads, cu_d, window=window)
    og, qn, kn, vn = f64(o), f64(q), f64(k), f64(v)
    for i, n in enumerate(lens[:12]):
        rows = slice(cu[i], cu[i + 1])
        for h in heads if n else []:
            g = h // (Hq // Hkv)
            ref, _, pv, size = SO.packed_head(qn[rows, h], kn[rows, g], vn[rows, g], window or n, SCALE)
            sum_v = SO.attended(n, window or n) @ np.abs(vn[rows, g])
            check(og[rows, h], ref, pv, size, dtype, sum_v, f"sequence {i} head {h}")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,window,Hq,Hkv", [(32768, None, 8, 2), (32767, 5000, 8, 1), (20011, 300, 4, 2),
                                             (9001, None, 2, 2)])
def test_packed_outputs_of_long_prompts(n, window, Hq, Hkv, dtype):
    """Sampled rows of prompts as long as the measured ones, a short prompt behind
    them: the first and last rows of tiles, of window turns and of the prompt."""
    lens = [n, 130]
    (q, k, v), cu, cu_d = make_packed(lens, Hq, Hkv, dtype, 121)
    v += 0.5
    o, lse = torch.zeros_like(q), torch.zeros(Hq, n + 130, device=DEV)
    rtp.attn_packed(q, k, v, o, list(range(Hq)), cu_d, window=window, lse=lse)
    rng = np.random.default_rng(n)
    t = np.unique(np.concatenate([[0, 1, 127, 128, 255, 256, n - 257, n - 256, n - 129, n - 128, n - 2, n - 1],
                                  rng.integers(0, n, 24)]))
    qn, kn, vn, og, lg = f64(q), f64(k), f64(v), f64(o), f64(lse)
    for h in range(Hq):
        g = h // (Hq // Hkv)
        for row in t:
            slots = np.arange(max(0, row + 1 - (window or n)), row + 1)
            ref, rl, _, pv, size = SO.decode_head(qn[row, h], kn[:n, g], vn[:n, g], slots, SCALE)
            check(og[row, h], ref, pv, size, dtype, np.abs(vn[slots, g]).sum(0), f"row {row} head {h}")
            assert abs(lg[h, row] - rl) <= score_error(size) + 2.0 ** -21 * (1 + abs(rl))
        last = slice(n, n + 130)
        ref, _, pv, size = SO.packed_head(qn[last, h], kn[last, g], vn[last, g], window or 130, SCALE)
        check(og[last, h], ref, pv, size, dtype, SO.attended(130, window or 130) @ np.abs(vn[last, g]), f"behind, {h}")


@pytest.mark.parametrize("dtype,head_major", [(torch.bfloat16, True), (torch.float16, False), (torch.float16, True)])
@pytest.mark.parametrize("case", DECODE, ids=lambda c: f"{c[0][:5]}p{c[3]}w{c[4]}s{c[5]}")
def test_decode_outputs(case, dtype, head_major):
    lens, Hq, Hkv, page, window, sink, heads = case
    cache, gen = make_cache(lens, Hkv, page, dtype, 131 + sum(lens), head_major=head_major)
    cache.v.add_(0.5)
    B, G = len(lens), Hq // Hkv
    q = rnd((B, Hq, D), dtype, gen, 1.5).to(DEV)
    o = torch.full((B, Hq, D), SENTINEL, dtype=dtype, device=DEV)
    rtp.paged_attn_decode(q, cache, torch.tensor(lens, dtype=torch.int32, device=DEV), o, heads, window=window,
                          sink=sink)
    qn, og, kc, vc = f64(q), f64(o), cache.k.cpu(), cache.v.cpu()
    for b, n in enumerate(lens):
        kn, vn = f64(rows_of(cache, kc, b, n)), f64(rows_of(cache, vc, b, n))
        slots = SO.decode_slots(n, window or max(n, 1), sink)
        for h in heads:
            g = h // G
            ref, _, _, pv, size = SO.decode_head(qn[b, h], kn[:, g], vn[:, g], slots, SCALE)
            check(og[b, h], ref, pv, np.float64(size), dtype, np.abs(vn[slots, g]).sum(0), f"sequence {b} head {h}")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [700, 5000])
def test_decode_splits_agree(n, dtype):
    """One sequence alone (a cluster shares its segments, or the list is cut),
    within a batch of many (few cuts), and under a table far wider than its
    length: every split is within the bound, and the parts that no split cuts
    differently are the same bits twice."""
    Hq, Hkv, page, others = 16, 2, 64, [64, 1, 333] * 50
    cache, gen = make_cache([n] + others, Hkv, page, dtype, 141)
    q = rnd((1 + len(others), Hq, D), dtype, gen, 1.5).to(DEV)
    wide = torch.full((1, 4096), -1, dtype=torch.int32, device=DEV)
    wide[:, :cache.table.shape[1]] = cache.table[:1]
    alone = rtp.PagedCache(cache.k, cache.v, cache.table[:1])
    outs = []
    for c, lens in ((alone, [n]), (rtp.PagedCache(cache.k, cache.v, wide), [n]), (cache, [n] + others)):
        lens_d = torch.tensor(lens, dtype=torch.int32, device=DEV)
        pair = []
        for _ in range(2):
            o = torch.zeros(len(lens), Hq, D, dtype=dtype, device=DEV)
            rtp.paged_attn_decode(q[:len(lens)], c, lens_d, o, list(range(Hq)))
            pair.append(o)
        assert torch.equal(*pair)
        outs.append(f64(pair[0][0]))
    kn, vn = (f64(rows_of(cache, x.cpu(), 0, n)) for x in (cache.k, cache.v))
    for h in range(Hq):
        g = h // 8
        ref, _, _, pv, size = SO.decode_head(f64(q)[0, h], kn[:, g], vn[:, g], np.arange(n), SCALE)
        for o in outs:
            check(o[h], ref, pv, np.float64(size), dtype, np.abs(vn[:, g]).sum(0), f"head {h}")
