"""The serving calls on the GPU against the fp64 oracle.

Tolerances are bounds, element by element, from the roundings that the calls
document. Let u = half the spacing of the 16-bit type (finfo.eps / 2) and

* ds: how far a score can be off. It is an fp32 sum of D = 128 exact products:
  at most D roundings of 2^-24 (doubled for an accumulator that truncates) of
  scale * sum |q||k|, plus the roundings of scale * log2(e) and of the scaled
  score, 2^-22 of that sum;
* a softmax numerator is then off by a factor within e^(+-ds), times 1 + 2^-21
  (exponential unit, difference with the running maximum), and so is the
  denominator: dp = 2 (e^ds - 1) + 2^-19 together, the fp32 sums included;
* rounded once to 16 bits it is off by u more, the output by another u:
  |o - exact| <= (dp + u) sum p|v| (1 + u) + u |exact|. Numerators below the
  type's smallest normal number lose absolute precision instead: 2^-25 (fp16),
  relative to a largest numerator of at least 2^-8, for each of n keys;
* lse: ds, plus 2^-21 (1 + |lse|) for the logarithm and the conversion of bases;
* a key's weight is a sum of positive terms e^x: each is off by e^(ds + |x| 2^-21),
  with |x| below |score| + |lse|, the sum of n by n 2^-24.
"""
import itertools
import math

import numpy as np
import pytest
import torch

from oracle import serving_oracle as SO

pytestmark = pytest.mark.gpu

rtp = pytest.importorskip("long_context_hybrid_b200")
DEV = "cuda"
D = 128
SCALE = 1 / math.sqrt(D)
DTYPES = [torch.bfloat16, torch.float16]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from long_context_hybrid_b200 import build
    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    rtp.lib()


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def ds_of(size):
    return size * (2 * D * 2.0 ** -24 + 2.0 ** -22)


def check_o(got, ref, pv, size, dtype, n, what):
    u = torch.finfo(dtype).eps / 2
    ds = np.asarray(ds_of(size))
    dp = 2 * np.expm1(ds) + 2.0 ** -19
    tol = (dp[..., None] + u) * pv * (1 + u) + u * np.abs(ref) + 1e-30
    if dtype == torch.float16:
        tol = tol + n * 2.0 ** -17 * pv.max() + 2.0 ** -25
    err = np.abs(got - ref)
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size}, worst {np.nanmax(err / tol):.2f} of the bound"


def check_lse(got, ref, size, what):
    tol = ds_of(size) + 2.0 ** -21 * (1 + np.abs(ref))
    assert np.all(np.abs(got - ref) <= tol), f"{what}: {np.nanmax(np.abs(got - ref) / tol):.2f} of the bound"


def rnd(shape, dtype, gen, scale=1.0):
    return (torch.randn(*shape, generator=gen) * scale).to(dtype)


def make_packed(lens, Hq, Hkv, dtype, seed, lead=0, tail=0, pad=0):
    """Packed q, k, v on the GPU, `lead` rows before the first sequence and
    `tail` behind the last, both NaN; with `pad` the rows are spaced out."""
    gen = torch.Generator().manual_seed(seed)
    T = lead + sum(lens) + tail
    cu = np.concatenate([[0], np.cumsum(lens)]) + lead
    out = []
    for H, s in ((Hq, 1.5), (Hkv, 1.0), (Hkv, 1.0)):
        x = rnd((T, H, D), dtype, gen, s)
        x[:lead] = float("nan")
        x[T - tail:] = float("nan") if tail else x[T - tail:]
        room = torch.full((T, H, D + pad), float("nan"), dtype=dtype)
        room[..., :D] = x
        out.append(room.to(DEV)[..., :D])
    return out, cu.astype(np.int64), torch.tensor(cu, dtype=torch.int32, device=DEV)


SENTINEL = 7.0

PACKED = [
    # lens, Hq, Hkv, window, heads, lead, tail, pad
    ([1], 1, 1, None, [0], 0, 0, 0),
    ([2, 0, 1, 0, 3], 4, 2, None, [3, 0, 1], 0, 5, 8),
    ([127, 128, 129], 8, 2, None, [0, 5, 7], 3, 0, 0),
    ([255, 256, 257, 1], 4, 4, None, [1, 2], 0, 1, 0),
    ([700, 65], 4, 1, 1, [0, 3], 0, 0, 0),
    ([513, 64, 400], 6, 2, 100, [0, 2, 5], 0, 70, 16),
    ([1000], 2, 1, 129, [0, 1], 9, 9, 0),
    ([640, 300], 4, 2, 128, [1, 3], 0, 0, 0),
    ([1500, 1, 64], 16, 1, None, [0, 15], 0, 0, 0),
    # many heads, or several prompts of a few tiles
    ([700, 65, 0, 300, 1, 129], 32, 4, None, list(range(32)), 0, 3, 0),
    ([700, 65, 0, 300, 1, 129], 32, 4, 100, list(range(32)), 1, 0, 0),
    ([600, 300, 500], 8, 2, None, list(range(8)), 0, 0, 8),
    ([600, 300, 500], 8, 2, 129, list(range(8)), 0, 0, 0),
    # few units of many keys: three CTAs share a unit's keys, and two
    ([900, 1500, 700], 2, 1, None, [1, 0], 2, 5, 0),
    ([900, 1500, 700], 4, 1, None, list(range(4)), 0, 0, 8),
    ([900, 1500, 700], 4, 2, 700, list(range(4)), 0, 0, 0),
    # short prompts and many tiles: one query tile a CTA; long ones: two
    ([1, 513, 0, 128, 2, 127, 256, 129, 16, 1], 32, 8, None, list(range(1, 32, 2)), 2, 200, 8),
    ([1, 513, 0, 128, 2, 127, 256, 129, 16, 1], 32, 8, 70, list(range(32)), 0, 0, 0),
    ([9] * 90, 4, 1, None, [0, 3], 0, 1, 0),
    ([1900, 5], 8, 1, 300, list(range(8)), 0, 0, 0),
    ([1900, 5], 8, 1, 600, list(range(8)), 0, 0, 0),
    ([1200, 1300], 20, 4, None, list(range(20)), 5, 0, 0),
    ([1200, 1300], 20, 4, 550, list(range(20)), 0, 0, 0),
    # several units a CTA, of one query tile and of two
    ([70, 3, 200, 0, 129, 40] * 40, 16, 4, None, list(range(16)), 0, 0, 0),
    ([70, 3, 200, 0, 129, 40] * 40, 16, 4, 50, list(range(16)), 1, 1, 0),
    ([700, 1300, 2, 900], 32, 4, None, list(range(32)), 0, 0, 0),
    ([700, 1300, 2, 900], 32, 4, 600, list(range(32)), 0, 4, 0),
]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", PACKED, ids=lambda c: f"{c[0][:12]}w{c[3]}")
def test_attn_packed(case, dtype):
    lens, Hq, Hkv, window, heads, lead, tail, pad = case
    (q, k, v), cu, cu_d = make_packed(lens, Hq, Hkv, dtype, 11 + sum(lens), lead, tail, pad)
    T = q.shape[0]
    o = torch.full((T, Hq, D + pad), SENTINEL, dtype=dtype, device=DEV)[..., :D]
    lse = torch.full((len(heads), T), SENTINEL, device=DEV)
    ws = torch.full((256,), 255, dtype=torch.uint8, device=DEV)
    rtp.attn_packed(q, k, v, o, heads, cu_d, window=window, lse=lse, ws=ws)
    assert rtp.workspace_status(ws) == 0
    og, lg = f64(o), f64(lse)
    qn, kn, vn = f64(q), f64(k), f64(v)
    for i, n in enumerate(lens):
        rows = slice(cu[i], cu[i + 1])
        for j, h in enumerate(heads if n else []):
            g = h // (Hq // Hkv)
            ref, rl, pv, size = SO.packed_head(qn[rows, h], kn[rows, g], vn[rows, g], window or n, SCALE)
            check_o(og[rows, h], ref, pv, size, dtype, n, f"sequence {i} head {h}")
            check_lse(lg[j, rows], rl, size, f"lse of sequence {i} head {h}")
    outside = np.ones(T, bool)
    outside[cu[0]:cu[-1]] = False
    assert (og[outside] == SENTINEL).all() and (lg[:, outside] == SENTINEL).all(), "rows of no sequence written"
    unlisted = [h for h in range(Hq) if h not in heads]
    assert (og[:, unlisted] == SENTINEL).all(), "unlisted head written"


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("window", [None, 40, 200, 600])
@pytest.mark.parametrize("Hq", [4, 12, 32, 64])
def test_attn_packed_unattended_values_do_not_matter(dtype, window, Hq):
    """NaN and infinities in keys and values reach exactly the rows that attend
    them: not the neighbour sequence, not earlier rows, not rows whose window
    has passed."""
    lens = [150, 1300 if window == 600 else 300, 90]
    end = 150 + lens[1]
    (q, k, v), cu, cu_d = make_packed(lens, Hq, 2, dtype, 5)
    heads = list(range(Hq))
    G = Hq // 2

    def run():
        o = torch.zeros_like(q)
        rtp.attn_packed(q, k, v, o, heads, cu_d, window=window)
        return o.float().cpu()

    clean = run()
    at = {150 + 140: float("nan"), end - 1: float("inf"), 150 + 3: float("-inf")}   # all in sequence 1
    for row, bad in at.items():
        v[row, 0, 17] = bad
    k[150 + 250, 1] = float("nan")
    got = run()
    T = q.shape[0]
    t = torch.arange(T)[:, None]
    reach = lambda row: ((t >= row) & (t < (min(end, row + window) if window else end))).squeeze(1)  # noqa: E731
    hit_v = torch.zeros(T, dtype=torch.bool)
    for row in at:
        hit_v |= reach(row)
    fin = torch.isfinite(got)
    fine = torch.ones(T, Hq, D, dtype=torch.bool)
    fine[hit_v, :G, 17] = False
    fine[reach(400), G:] = False
    assert torch.equal(fin, fine)
    assert torch.equal(got[fin], clean[fin])
    only_inf = reach(end - 1) & ~reach(290) & ~reach(153)
    assert (got[only_inf][:, :G, 17] == float("inf")).all()


def test_attn_packed_many_empty_prompts():
    """Far more tile numbers than tiles: nothing runs out, and what is there is right."""
    lens = [0] * 50000 + [5] + [0] * 40000 + [300, 0, 1] + [0] * 30000
    Hq, Hkv = 8, 2
    (q, k, v), cu, cu_d = make_packed(lens, Hq, Hkv, torch.bfloat16, 77)
    o = torch.full_like(q, SENTINEL)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    rtp.attn_packed(q, k, v, o, list(range(Hq)), cu_d, ws=ws)
    assert rtp.workspace_status(ws) == 0
    og, qn, kn, vn = f64(o), f64(q), f64(k), f64(v)
    for i, n in enumerate(lens):
        if n == 0:
            continue
        rows = slice(cu[i], cu[i + 1])
        for h in range(Hq):
            g = h // (Hq // Hkv)
            ref, _, pv, size = SO.packed_head(qn[rows, h], kn[rows, g], vn[rows, g], n, SCALE)
            check_o(og[rows, h], ref, pv, size, torch.bfloat16, n, f"sequence {i} head {h}")


def test_attn_packed_long_prompt_sampled_rows():
    """A prompt long enough for many ring turns, sampled rows against fp64."""
    n, Hq, Hkv = 5003, 8, 2
    (q, k, v), cu, cu_d = make_packed([n], Hq, Hkv, torch.bfloat16, 77)
    o, lse = torch.zeros_like(q), torch.zeros(Hq, n, device=DEV)
    rtp.attn_packed(q, k, v, o, list(range(Hq)), cu_d, lse=lse)
    rows = np.array([0, 1, 255, 256, 1023, 2500, 4863, 4864, 5001, 5002])
    qn, kn, vn, og, lg = f64(q), f64(k), f64(v), f64(o), f64(lse)
    for h in range(Hq):
        g = h // 4
        for t in rows:
            slots = np.arange(t + 1)
            ref, rl, _, pv, size = SO.decode_head(qn[t, h], kn[:, g], vn[:, g], slots, SCALE)
            check_o(og[t, h], ref, pv, size, torch.bfloat16, t + 1, f"row {t} head {h}")
            check_lse(lg[h, t], rl, size, f"lse {t}")


def test_attn_packed_growing_scores_rescale():
    """Scores that rise along the keys by far more than the lazy threshold, so
    that O and the first half's P are rescaled; and rows that fall."""
    n = 600
    gen = torch.Generator().manual_seed(3)
    direction = torch.nn.functional.normalize(torch.randn(D, generator=gen), dim=0)
    ramp = torch.linspace(-30, 30, n)[:, None]
    k = (direction * ramp + 0.1 * torch.randn(n, D, generator=gen)).to(torch.bfloat16)[:, None].to(DEV)
    sign = torch.where(torch.arange(n) % 2 == 0, 1.0, -1.0)[:, None]
    q = (direction * 12 * sign).to(torch.bfloat16)[:, None].to(DEV)
    v = torch.randn(n, 1, D, generator=gen).to(torch.bfloat16).to(DEV)
    o, lse = torch.zeros_like(q), torch.zeros(1, n, device=DEV)
    rtp.attn_packed(q, k, v, o, [0], torch.tensor([0, n], dtype=torch.int32, device=DEV), lse=lse)
    ref, rl, pv, size = SO.packed_head(f64(q)[:, 0], f64(k)[:, 0], f64(v)[:, 0], n, SCALE)
    check_o(f64(o)[:, 0], ref, pv, size, torch.bfloat16, n, "ramp")
    check_lse(f64(lse)[0], rl, size, "ramp lse")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", [
    ([1], 1, 1, None, None, [0]),
    ([2, 0, 1, 300], 4, 2, None, None, [3, 0, 2]),
    ([127, 128, 129, 700], 8, 2, None, 64, [0, 1, 2, 5]),
    ([513, 64, 400], 6, 2, 100, 130, [0, 2, 1]),
    ([1000, 3], 4, 1, 129, None, [0, 1, 2, 3]),
    ([900], 2, 2, 1, 5, [0, 1]),
    ([2100], 16, 1, None, 1, list(range(16))),
    ([700, 64, 1, 0, 65, 1500], 16, 2, None, 64, list(range(16))),
    ([300, 900, 40], 8, 2, 200, 100, [0, 1, 2, 3, 5, 6]),
    ([60] * 300, 2, 2, None, 17, [0, 1]),
], ids=lambda c: f"{c[0][:5]}w{c[3]}o{c[4]}")
def test_attn_key_weights(case, dtype):
    lens, Hq, Hkv, window, n_obs, heads = case
    (q, k, v), cu, cu_d = make_packed(lens, Hq, Hkv, dtype, 23 + sum(lens), 2, 130, 8)
    T, G = q.shape[0], Hq // Hkv
    qn, kn, vn = f64(q), f64(k), f64(v)
    # the statistics of the observed rows only: nothing else may be read
    lse = np.full((len(heads), T), np.nan, np.float32)
    for i, n in enumerate(lens):
        rows = slice(cu[i], cu[i + 1])
        for j, h in enumerate(heads if n else []):
            x = SO.packed_head(qn[rows, h], kn[rows, h // G], vn[rows, h // G], window or n, SCALE)[1]
            first = max(0, n - (n_obs or n))
            lse[j, cu[i] + first:cu[i + 1]] = x[first:]
    w = torch.full((Hkv, T), SENTINEL, device=DEV)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    rtp.attn_key_weights(q, k, torch.from_numpy(lse).to(DEV), w, heads, cu_d, n_obs=n_obs, window=window, ws=ws)
    assert rtp.workspace_status(ws) == 0
    got = f64(w)
    groups = sorted({h // G for h in heads})
    for g in groups:
        for i, n in enumerate(lens):
            if n == 0:
                continue
            rows = slice(cu[i], cu[i + 1])
            ref, tol, terms = np.zeros(n), np.zeros(n), np.zeros(n)
            for j, h in enumerate(heads):
                if h // G != g:
                    continue
                x, size_x, size, count = SO.key_weights_head(qn[rows, h], kn[rows, g],
                                                             lse[j, rows].astype(np.float64), n_obs or n, window or n,
                                                             SCALE)
                ref += x
                tol += x * np.expm1(ds_of(size) + size_x * 2.0 ** -21 + 2.0 ** -21)
                terms += count
            tol += ref * terms * 2.0 ** -24 + 1e-37
            err = np.abs(got[g, rows] - ref)
            assert np.all(err <= tol), f"KV head {g} sequence {i}: {np.nanmax(err / tol):.2f} of the bound"
    outside = np.ones(T, bool)
    outside[cu[0]:cu[-1]] = False
    assert (got[:, outside] == SENTINEL).all()
    assert (got[[g for g in range(Hkv) if g not in groups]] == SENTINEL).all()


# ---------------------------------------------------------------------------
# The paged cache
# ---------------------------------------------------------------------------
def make_cache(lens, Hkv, page, dtype, seed, spare=3, head_major=False, weights=True, extra_cols=1):
    """A cache whose pages lie in random order, every row behind a sequence's
    end and every spare page NaN, unused table entries -1."""
    gen = torch.Generator().manual_seed(seed)
    need = [(n + page - 1) // page for n in lens]
    total = sum(need) + spare
    order = torch.randperm(total, generator=gen)
    table = torch.full((len(lens), max(1, max(need)) + extra_cols), -1, dtype=torch.int32)
    pools, at = [], 0
    for b, m in enumerate(need):
        table[b, :m] = order[at:at + m]
        at += m
    for _ in range(2):
        x = torch.full((total, page, Hkv, D), float("nan"), dtype=dtype)
        for b, n in enumerate(lens):
            for j in range(need[b]):
                m = min(page, n - j * page)
                x[table[b, j].item(), :m] = rnd((m, Hkv, D), dtype, gen)
        x = x.to(DEV)
        if head_major:                         # stored [pages, Hkv, page, D]
            x = x.transpose(1, 2).contiguous().transpose(1, 2)
        pools.append(x)
    w = None
    if weights:
        w = torch.rand(total, Hkv, page, generator=gen)
        w[torch.rand(total, Hkv, page, generator=gen) < 0.2] = 0.0
        w = w.to(DEV)
    return rtp.PagedCache(pools[0], pools[1], table.to(DEV), w), gen


def rows_of(cache, x, b, n):
    """[n, ...] rows of sequence b in order, from a pool [pages, page, ...]."""
    t = cache.table[b].cpu().long()
    s = torch.arange(n)
    return x[t[s // cache.page_size], s % cache.page_size]


DECODE = [
    # lens, Hq, Hkv, page, window, sink, heads
    ([1], 1, 1, 1, None, 0, [0]),
    ([0, 1, 0, 2], 4, 2, 16, None, 0, [0, 1, 2, 3]),
    ([0], 2, 1, 16, None, 0, [1]),
    ([63, 64, 65, 200], 8, 2, 32, None, 0, [7, 0, 3, 4]),
    ([1000, 17, 333], 6, 3, 64, 100, 4, [0, 1, 2, 3, 4, 5]),
    ([500, 40], 16, 1, 16, 64, 100, list(range(16))),
    ([777, 3], 4, 4, 128, 1, 1, [1, 3]),
    ([2050, 0, 1, 129], 32, 4, 256, None, 0, list(range(32))),
    ([9000], 8, 1, 64, None, 0, list(range(8))),
    ([6000, 0, 100], 16, 1, 64, None, 0, list(range(16))),
    ([3000, 129, 0, 64], 24, 2, 32, None, 0, [0, 5, 11, 12, 13, 14, 15, 16, 17, 18, 19, 20, 21, 22]),
    ([200] * 70, 8, 4, 16, None, 0, list(range(8))),
    ([70] * 150, 2, 2, 16, None, 0, [0, 1]),
    ([64] * 40 + [3000] + [0] * 130 + [5], 4, 4, 2, 1000, 3, [0, 1, 2, 3]),
]


@pytest.mark.parametrize("dtype,head_major", [(torch.bfloat16, False), (torch.float16, True)])
@pytest.mark.parametrize("case", DECODE, ids=lambda c: f"{c[0][:5]}p{c[3]}w{c[4]}s{c[5]}")
def test_paged_attn_decode(case, dtype, head_major):
    lens, Hq, Hkv, page, window, sink, heads = case
    cache, gen = make_cache(lens, Hkv, page, dtype, 31 + sum(lens), head_major=head_major)
    B, G = len(lens), Hq // Hkv
    q = rnd((B, Hq, D), dtype, gen, 1.5).to(DEV)
    o = torch.full((B, Hq, D), SENTINEL, dtype=dtype, device=DEV)
    lse = torch.full((B, len(heads)), SENTINEL, device=DEV)
    lens_d = torch.tensor(lens, dtype=torch.int32, device=DEV)
    w_out = torch.full_like(cache.weights, SENTINEL)
    before = [cache.k.clone(), cache.v.clone(), cache.weights.clone()]
    rtp.paged_attn_decode(q, cache, lens_d, o, heads, window=window, sink=sink, lse=lse, weights_out=w_out)
    plain = torch.full_like(o, SENTINEL)
    rtp.paged_attn_decode(q, cache, lens_d, plain, heads, window=window, sink=sink)
    assert torch.equal(o, plain), "the weights change the output"
    for x, y in zip(before, (cache.k, cache.v, cache.weights)):
        assert torch.equal(torch.nan_to_num(x.float()), torch.nan_to_num(y.float()))
    qn, og, lg = f64(q), f64(o), f64(lse)
    kc, vc, wc, wo = cache.k.cpu(), cache.v.cpu(), cache.weights.cpu(), w_out.cpu()
    expect_w = torch.full_like(wo, SENTINEL).double()
    tol_w = torch.zeros_like(wo).double()
    for b, n in enumerate(lens):
        kn, vn = f64(rows_of(cache, kc, b, n)), f64(rows_of(cache, vc, b, n))
        slots = SO.decode_slots(n, window or max(n, 1), sink)
        table = cache.table[b].cpu().long()
        s = torch.arange(n)
        pg, off = table[s // page], s % page
        for g in sorted({h // G for h in heads}):
            expect_w[pg, g, off] = wc[pg, g, off].double()
        for j, h in enumerate(heads):
            g = h // G
            ref, rl, p, pv, size = SO.decode_head(qn[b, h], kn[:, g], vn[:, g], slots, SCALE)
            check_o(og[b, h], ref, pv, size, dtype, n, f"sequence {b} head {h}")
            if n == 0:
                assert lg[b, j] == -np.inf
                continue
            check_lse(lg[b, j], rl, size, f"lse {b} {h}")
            ps, os_ = pg[slots], off[slots]
            expect_w[ps, g, os_] += torch.from_numpy(p)
            # the exponent's roundings: |score| + |lse| within size + |lse|
            rel = math.expm1(2 * ds_of(size) + (size + abs(rl)) * 2.0 ** -21 + 2.0 ** -20)
            tol_w[ps, g, os_] += torch.from_numpy(p * rel)
    tol_w += expect_w.abs() * (G + 1) * 2.0 ** -23
    assert ((wo.double() - expect_w).abs() <= tol_w).all()
    unlisted = [h for h in range(Hq) if h not in heads]
    assert (og[:, unlisted] == SENTINEL).all()


def test_paged_attn_decode_missing_pages_hold_no_token():
    """Page ids outside the pool (inside a sequence's length) are skipped."""
    lens = [300, 130]
    cache, gen = make_cache(lens, 2, 32, torch.bfloat16, 8)
    for b, j, bad in ((0, 2, -1), (0, 9, 10 ** 6), (1, 0, cache.num_pages), (1, 4, -2 ** 31)):
        cache.table[b, j] = bad
    q = rnd((2, 4, D), torch.bfloat16, gen).to(DEV)
    o = torch.zeros_like(q)
    w_out = torch.full_like(cache.weights, SENTINEL)
    rtp.paged_attn_decode(q, cache, torch.tensor(lens, dtype=torch.int32, device=DEV), o, [0, 1, 2, 3],
                          weights_out=w_out)
    table = cache.table.cpu().long()
    kc, vc = cache.k.cpu(), cache.v.cpu()
    for b, n in enumerate(lens):
        s = torch.arange(n)
        pg = table[b][s // 32]
        slots = s[(pg >= 0) & (pg < cache.num_pages)]
        kn, vn = f64(kc[table[b][slots // 32], slots % 32]), f64(vc[table[b][slots // 32], slots % 32])
        for h in range(4):
            ref, _, _, pv, size = SO.decode_head(f64(q)[b, h], kn[:, h // 2], vn[:, h // 2], np.arange(len(slots)),
                                                 SCALE)
            check_o(f64(o)[b, h], ref, pv, size, torch.bfloat16, n, f"{b} {h}")


def test_paged_attn_decode_lengths_are_clamped():
    """Lengths beyond max_len, and negative ones, stay within the call's limits."""
    lens = [100, 100, 100]
    cache, gen = make_cache(lens, 1, 16, torch.bfloat16, 9, extra_cols=0)
    q = rnd((3, 2, D), torch.bfloat16, gen).to(DEV)
    o, ref = torch.zeros_like(q), torch.zeros_like(q)
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    rtp.paged_attn_decode(q, cache, dev([2 ** 31 - 1, -5, 64]), o, [0, 1], max_len=64)
    rtp.paged_attn_decode(q, cache, dev([64, 0, 64]), ref, [0, 1], max_len=64)
    assert torch.equal(o, ref) and (o[1] == 0).all()


def test_paged_attn_decode_is_repeatable_and_splits_agree():
    """The same call twice gives the same bits; the split over more CTAs (a
    longer batch around the same sequence) stays within the bound."""
    cache, gen = make_cache([5000], 2, 64, torch.bfloat16, 10)
    q = rnd((1, 16, D), torch.bfloat16, gen).to(DEV)
    lens = torch.tensor([5000], dtype=torch.int32, device=DEV)
    outs = []
    for _ in range(3):
        o, w = torch.zeros_like(q), torch.zeros_like(cache.weights)
        rtp.paged_attn_decode(q, cache, lens, o, list(range(16)), weights_out=w)
        outs.append((o, w))
    for o, w in outs[1:]:
        assert torch.equal(o, outs[0][0]) and torch.equal(w, outs[0][1])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lens,pos,Hkv,page,weights", [
    ([1], [0], 1, 1, True), ([0, 5, 1, 70], [3, 0, 15, 16], 2, 16, True), ([1] * 40, list(range(40)), 4, 32, False),
    ([300, 1000], [7, 0], 3, 128, True), ([3, 40], [90, 2], 2, 16, False)])
def test_paged_append(lens, pos, Hkv, page, weights, dtype):
    ends = [p + n for p, n in zip(pos, lens)]
    cache, gen = make_cache(ends, Hkv, page, dtype, 41 + sum(lens), extra_cols=0)
    capacity = cache.capacity
    if lens == [3, 40]:
        pos = [capacity - 2, -1]                # rows past the capacity and before slot 0 are dropped
    (_, k, v), cu, cu_d = make_packed(lens, 1, Hkv, dtype, 43, 1, 2, 8)
    T = k.shape[0]
    w = torch.rand(Hkv, T, generator=gen).to(DEV) if weights else None
    table = cache.table.cpu().numpy()
    old = [torch.nan_to_num(x.float(), nan=-9.0).cpu().numpy() for x in (cache.k, cache.v)]
    old_w = cache.weights.cpu().numpy()
    rtp.paged_append(cache, k, v, cu_d, torch.tensor(pos, dtype=torch.int32, device=DEV), weights=w)
    for got, before, rows in zip((cache.k, cache.v), old, (k, v)):
        want = SO.append(before, torch.nan_to_num(rows.float(), nan=-9.0).cpu().numpy(), cu, pos, table, page)
        assert np.array_equal(torch.nan_to_num(got.float(), nan=-9.0).cpu().numpy(), want)
    rows = w.t().cpu().numpy() if weights else np.zeros((T, Hkv), np.float32)
    want = SO.append(old_w.transpose(0, 2, 1), rows, cu, pos, table, page).transpose(0, 2, 1)
    assert np.array_equal(cache.weights.cpu().numpy(), want)


EVICT = [
    # lens, Hkv, page, budget, sink, recent
    ([1, 0, 5], 2, 16, 8, 1, 2),
    ([9], 1, 1, 8, 1, 2),
    ([100, 64, 65], 2, 16, 64, 4, 20),
    ([100, 300], 3, 32, 50, 0, 0),
    ([500, 20], 2, 64, 40, 10, 30),             # nothing left to choose
    ([3000, 1], 2, 16, 700, 4, 64),
    ([12000, 9000, 100], 1, 64, 2000, 1, 500),
    ([30000], 1, 256, 5000, 3, 100),
]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("case", EVICT, ids=lambda c: f"{c[0]}b{c[3]}")
def test_cache_evict(case, in_place):
    lens, Hkv, page, budget, sink, recent = case
    dtype = torch.bfloat16
    cache, gen = make_cache(lens, Hkv, page, dtype, 51 + sum(lens))
    cache.weights[(cache.weights > 0.5) & (cache.weights < 0.6)] = 0.55      # many equal weights
    cache.weights[(cache.weights > 0.6) & (cache.weights < 0.601)] = float("nan")
    cache.weights[(cache.weights > 0.3) & (cache.weights < 0.301)] = -0.0
    cache.weights[(cache.weights > 0.2) & (cache.weights < 0.21)] = 1e-41    # subnormal
    B = len(lens)
    olds = [x.cpu() for x in (cache.k, cache.v)]
    old_w = cache.weights.cpu()
    table = cache.table.cpu().long()
    if in_place:
        out = cache
    else:
        kept = [min(n, budget) for n in lens]
        out, _ = make_cache(kept, Hkv, 2 * page, dtype, 61)
        out.k.fill_(SENTINEL); out.v.fill_(SENTINEL); out.weights.fill_(SENTINEL)
    lens_d = torch.tensor(lens, dtype=torch.int32, device=DEV)
    idx, new_lens = rtp.cache_evict(cache, lens_d, budget, sink, recent, out=None if in_place else out)
    assert new_lens.tolist() == [min(n, budget) for n in lens]
    idx = idx.cpu().numpy()
    to = out.table.cpu().long()
    touched = torch.zeros(out.num_pages, Hkv, out.page_size, dtype=torch.bool)
    for b, n in enumerate(lens):
        keep = min(n, budget)
        for g in range(Hkv):
            s = torch.arange(n)
            w = old_w[table[b][s // page], g, s % page].numpy()
            want = SO.evict_slots(w, n, budget, sink, recent)
            assert np.array_equal(idx[b, g, :keep], want), f"sequence {b} head {g}"
            assert (idx[b, g, keep:] == -1).all()
            src, dst = torch.from_numpy(want), torch.arange(keep)
            sp, so = table[b][src // page], src % page
            dp, do = to[b][dst // out.page_size], dst % out.page_size
            for new, old in zip((out.k, out.v), olds):
                assert torch.equal(new.cpu()[dp, do, g], old[sp, so, g])
            assert np.array_equal(out.weights.cpu()[dp, g, do].numpy(), old_w[sp, g, so].numpy(), equal_nan=True)
            touched[dp, g, do] = True
    if in_place:
        same = ~touched
        assert np.array_equal(cache.weights.cpu()[same].numpy(), old_w[same].numpy(), equal_nan=True)
        k_new, k_old = cache.k.cpu().transpose(1, 2)[same].float(), olds[0].transpose(1, 2)[same].float()
        assert np.array_equal(k_new.numpy(), k_old.numpy(), equal_nan=True)
    else:
        assert (out.weights.cpu()[~touched] == SENTINEL).all()
        assert (out.k.cpu().transpose(1, 2)[~touched] == SENTINEL).all()


def test_cache_evict_keys_beyond_shared_memory():
    """More candidates than the cluster's shared memory holds: the rest is read again."""
    n, page, budget = 400_000, 256, 1000
    pages = (n + page - 1) // page
    gen = torch.Generator().manual_seed(4)
    k = torch.zeros(pages, page, 1, D, dtype=torch.bfloat16, device=DEV)
    k[..., 0, 0] = (torch.arange(pages * page) % 251).view(pages, page).to(torch.bfloat16).to(DEV)
    w = torch.rand(pages, 1, page, generator=gen).round(decimals=3).to(DEV)
    table = torch.randperm(pages, generator=gen).to(torch.int32)[None].to(DEV)
    cache = rtp.PagedCache(k, k.clone(), table, w)
    to = rtp.PagedCache(torch.zeros(4, page, 1, D, dtype=torch.bfloat16, device=DEV),
                        torch.zeros(4, page, 1, D, dtype=torch.bfloat16, device=DEV),
                        torch.arange(4, dtype=torch.int32, device=DEV)[None], torch.zeros(4, 1, page, device=DEV))
    idx, _ = rtp.cache_evict(cache, torch.tensor([n], dtype=torch.int32, device=DEV), budget, 2, 100, out=to)
    flat = w.cpu()[table[0].cpu().long(), 0].flatten()[:n].numpy()
    want = SO.evict_slots(flat, n, budget, 2, 100)
    assert np.array_equal(idx.cpu().numpy()[0, 0], want)


# ---------------------------------------------------------------------------
# Together, as a serving loop uses them
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", DTYPES)
def test_serving_loop(dtype):
    """Prompts -> cache with weights -> decode steps -> eviction -> decode, all
    of it against the oracle carried along on the host."""
    lens, Hq, Hkv, page, steps = [150, 1, 333], 8, 2, 16, 5
    streaming, window, sink, n_obs, budget, recent = [1, 2, 5], 60, 4, 32, 100, 20
    G, B = Hq // Hkv, len(lens)
    (q, k, v), cu, cu_d = make_packed(lens, Hq, Hkv, dtype, 91)
    most = (max(lens) + steps + 1 + page - 1) // page
    cache = rtp.PagedCache(torch.zeros(B * most, page, Hkv, D, dtype=dtype, device=DEV),
                           torch.zeros(B * most, page, Hkv, D, dtype=dtype, device=DEV),
                           torch.randperm(B * most, generator=torch.Generator().manual_seed(1)).to(torch.int32)
                           .view(B, most).to(DEV), torch.zeros(B * most, Hkv, page, device=DEV))
    layer = rtp.PagedLayer(cache, Hq, streaming, window, sink, n_obs)
    o = torch.zeros_like(q)
    layer.prefill(q, k, v, o, cu_d)
    qn, kn, vn = f64(q), f64(k), f64(v)
    keys = [[kn[cu[b]:cu[b + 1], g] for g in range(Hkv)] for b in range(B)]
    vals = [[vn[cu[b]:cu[b + 1], g] for g in range(Hkv)] for b in range(B)]
    wts = [[np.zeros(n) for _ in range(Hkv)] for n in lens]
    for b, n in enumerate(lens):
        for h in range(Hq):
            win = window if h in streaming else n
            ref, lse, pv, size = SO.packed_head(qn[cu[b]:cu[b + 1], h], keys[b][h // G], vals[b][h // G], win, SCALE)
            check_o(f64(o)[cu[b]:cu[b + 1], h], ref, pv, size, dtype, n, f"prompt {b} {h}")
            wts[b][h // G] += SO.key_weights_head(qn[cu[b]:cu[b + 1], h], keys[b][h // G], lse, n_obs, win, SCALE)[0]
    assert layer.lens.tolist() == lens

    def decode(seed):
        gen = torch.Generator().manual_seed(seed)
        qd, kd, vd = (rnd((B, H, D), dtype, gen, 1.2).to(DEV) for H in (Hq, Hkv, Hkv))
        od = torch.zeros_like(qd)
        layer.decode(qd, kd, vd, od)
        for b in range(B):
            for g in range(Hkv):
                keys[b][g] = np.concatenate([keys[b][g], f64(kd)[b, g][None]])
                vals[b][g] = np.concatenate([vals[b][g], f64(vd)[b, g][None]])
                wts[b][g] = np.append(wts[b][g], 0.0)
            for h in range(Hq):
                g, n = h // G, len(keys[b][h // G])
                slots = SO.decode_slots(n, window, sink) if h in streaming else np.arange(n)
                ref, _, p, pv, size = SO.decode_head(f64(qd)[b, h], keys[b][g], vals[b][g], slots, SCALE)
                check_o(f64(od)[b, h], ref, pv, size, dtype, n, f"step {seed} {b} {h}")
                wts[b][g][slots] += p

    def check_weights():
        for b in range(B):
            n = len(keys[b][0])
            got = f64(rows_of(cache, cache.weights.cpu().transpose(1, 2), b, n))
            for g in range(Hkv):
                # sums of at most 8 heads x 40 rows of terms, each within the bounds above (scores below 20)
                assert np.allclose(got[:, g], wts[b][g], rtol=2e-4, atol=1e-30)

    for s in range(steps):
        decode(100 + s)
    check_weights()
    idx = layer.evict(budget, recent).cpu().numpy()
    for b in range(B):
        for g in range(Hkv):
            n = len(keys[b][g])
            kept = idx[b, g][idx[b, g] >= 0]
            # the oracle's weights carry their own rounding: the choice is checked on the device's
            assert len(kept) == min(n, budget) and (np.diff(kept) > 0).all()
            keys[b][g], vals[b][g], wts[b][g] = keys[b][g][kept], vals[b][g][kept], wts[b][g][kept]
    assert layer.lens.tolist() == [min(n + steps, budget) for n in lens]
    check_weights()
    decode(200)
    check_weights()


def test_captured_step_follows_lengths_and_tables():
    """A captured append + decode + eviction replays with the lengths, tables and
    rows that the buffers hold at the replay."""
    B, Hq, Hkv, page, cap = 2, 4, 2, 16, 256
    gen = torch.Generator().manual_seed(6)
    P = B * cap // page
    mk = lambda: rnd((P, page, Hkv, D), torch.bfloat16, gen).to(DEV)  # noqa: E731
    table = torch.arange(P, dtype=torch.int32).view(B, -1).to(DEV)
    cache = rtp.PagedCache(mk(), mk(), table, torch.rand(P, Hkv, page, generator=gen).to(DEV))
    layer = rtp.PagedLayer(cache, Hq)
    q, k, v = (rnd((B, H, D), torch.bfloat16, gen).to(DEV) for H in (Hq, Hkv, Hkv))
    o = torch.zeros_like(q)
    layer.lens.copy_(torch.tensor([10, 0], dtype=torch.int32))
    layer.decode(q, k, v, o)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer.decode(q, k, v, o)
    for lens in ([3, 100], [200, 0], [255, 17]):
        table.copy_(torch.randperm(P, generator=gen).to(torch.int32).view(B, -1))
        q.copy_(rnd((B, Hq, D), torch.bfloat16, gen))
        k.copy_(rnd((B, Hkv, D), torch.bfloat16, gen))
        layer.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        saved = [x.clone() for x in (cache.k, cache.v, cache.weights)]
        g.replay()
        got = [x.clone() for x in (o, cache.k, cache.weights, layer.lens)]
        for x, y in zip((cache.k, cache.v, cache.weights), saved):
            x.copy_(y)
        layer.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        o.zero_()
        layer.decode(q, k, v, o)
        for x, y in zip(got, (o, cache.k, cache.weights, layer.lens)):
            assert torch.equal(x, y)
        assert layer.lens.tolist() == [n + 1 for n in lens]


def test_calls_on_two_streams():
    """Two calls in flight at once, each on a stream and workspace of its own."""
    lens = [[3000, 100], [900, 2500]]
    streams = [torch.cuda.Stream() for _ in lens]
    jobs = []
    for i, ls in enumerate(lens):
        cache, gen = make_cache(ls, 2, 32, torch.bfloat16, 71 + i)
        q = rnd((2, 8, D), torch.bfloat16, gen).to(DEV)
        (pq, pk, pv), _, cu = make_packed([700, 41], 4, 2, torch.bfloat16, 73 + i)
        jobs.append((cache, q, torch.tensor(ls, dtype=torch.int32, device=DEV), pq, pk, pv, cu))

    def run(stream):
        outs = []
        for s, (cache, q, ln, pq, pk, pv, cu) in zip(streams, jobs):
            o, w, po = torch.zeros_like(q), torch.zeros_like(cache.weights), torch.zeros_like(pq)
            torch.cuda.synchronize()
            st = s if stream else None
            for _ in range(5):
                rtp.paged_attn_decode(q, cache, ln, o, list(range(8)), weights_out=w, stream=st)
                rtp.attn_packed(pq, pk, pv, po, [0, 1, 2, 3], cu, stream=st)
            outs += [o, w, po]
        torch.cuda.synchronize()
        return outs

    for a, b in zip(run(True), run(False)):
        assert torch.equal(a, b)


def test_kernels_of_every_kind_beside_each_other():
    """Calls whose CTAs stay for many units, next to the other tensor-core
    kernels, each on a stream of its own: the results of one after the other."""
    dt = torch.bfloat16
    (q1, k1, v1), _, cu1 = make_packed([100] * 200, 16, 4, dt, 81)
    (q2, k2, v2), _, cu2 = make_packed([1500, 900, 1700, 1100], 16, 4, dt, 82)
    gen = torch.Generator().manual_seed(83)
    q3, k3, v3 = (rnd((1, 2048, h, D), dt, gen).to(DEV) for h in (8, 2, 2))
    qt, kt = (rnd((1, h, 4096, 16), dt, gen).to(DEV) for h in (4, 2))
    streams = [torch.cuda.Stream() for _ in range(5)]
    ws = [torch.zeros(1 << 20, dtype=torch.uint8, device=DEV) for _ in streams]
    lse = torch.zeros(16, q2.shape[0], device=DEV)
    rtp.attn_packed(q2, k2, v2, torch.zeros_like(q2), list(range(16)), cu2, lse=lse)

    def run(apart):
        o1, o2, o3 = torch.zeros_like(q1), torch.zeros_like(q2), torch.zeros_like(q3)
        w = torch.zeros(4, q2.shape[0], device=DEV)
        blocks = torch.zeros(1, 4, 64, 16, dtype=torch.int32, device=DEV)
        counts = torch.zeros(1, 4, 64, dtype=torch.int32, device=DEV)
        calls = [lambda st, b: rtp.attn_packed(q1, k1, v1, o1, list(range(16)), cu1, ws=b, stream=st),
                 lambda st, b: rtp.attn_packed(q2, k2, v2, o2, list(range(16)), cu2, ws=b, stream=st),
                 lambda st, b: rtp.attn_key_weights(q2, k2, lse, w, list(range(16)), cu2, ws=b, stream=st),
                 lambda st, b: rtp.swa(q3, k3, v3, o3, list(range(8)), 512, ws=b, stream=st),
                 lambda st, b: rtp.select_prefill(qt, kt, [0, 0, 1, 1], 16, blocks, counts, ws=b, stream=st)]
        torch.cuda.synchronize()
        for _ in range(10):
            for call, stream, b in zip(calls, streams, ws):
                call(stream if apart else None, b)
                if not apart:
                    torch.cuda.synchronize()
        torch.cuda.synchronize()
        assert all(rtp.workspace_status(b) == 0 for b in ws)
        return o1, o2, o3, w, blocks, counts

    for x, y in zip(run(False), run(True)):
        assert torch.equal(x, y)


def test_long_cache_offsets_pass_32_bits():
    """Page offsets beyond 2^31 elements (and 2^32 bytes) are addressed in 64 bits."""
    page, Hkv, pages = 256, 1, 70_000                       # 2.3e9 elements of k, as many of v
    k = torch.zeros(pages, page, Hkv, D, dtype=torch.bfloat16, device=DEV)
    v = torch.zeros(pages, page, Hkv, D, dtype=torch.bfloat16, device=DEV)
    gen = torch.Generator().manual_seed(2)
    table = torch.tensor([[pages - 1, 0, pages - 2]], dtype=torch.int32, device=DEV)
    cache = rtp.PagedCache(k, v, table)
    n = 600
    (_, kk, vv), cu, cu_d = make_packed([n], 1, Hkv, torch.bfloat16, 3)
    rtp.paged_append(cache, kk, vv, cu_d, torch.zeros(1, dtype=torch.int32, device=DEV))
    assert torch.equal(k[pages - 1, :, 0], kk[:256, 0]) and torch.equal(v[pages - 2, :88, 0], vv[512:, 0])
    q = rnd((1, 2, D), torch.bfloat16, gen).to(DEV)
    o = torch.zeros_like(q)
    rtp.paged_attn_decode(q, cache, torch.tensor([n], dtype=torch.int32, device=DEV), o, [0, 1])
    for h in range(2):
        ref, _, _, pv, size = SO.decode_head(f64(q)[0, h], f64(kk)[:, 0], f64(vv)[:, 0], np.arange(n), SCALE)
        check_o(f64(o)[0, h], ref, pv, size, torch.bfloat16, n, f"head {h}")


@pytest.mark.parametrize("cu", [[0, 300, 100, 400], [500, -5, 10 ** 9, 20], [-10, -10, -10, -10], [400, 300, 200, 0],
                                [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1, 17], [390, 390, 400, 1000]])
def test_bad_offsets_stay_inside_the_tensors(cu):
    """Offsets that decrease or leave [0, T]: nothing outside the tensors is
    touched (guard rows around every output), and the calls end."""
    T, guard, Hq, Hkv = 400, 64, 4, 2
    gen = torch.Generator().manual_seed(12)
    room = lambda H: rnd((T + 2 * guard, H, D), torch.bfloat16, gen).to(DEV)  # noqa: E731
    inner = slice(guard, guard + T)
    q, k, v = room(Hq)[inner], room(Hkv)[inner], room(Hkv)[inner]
    o_room = torch.full((T + 2 * guard, Hq, D), SENTINEL, dtype=torch.bfloat16, device=DEV)
    lse_room = torch.full((Hq * T + 2 * guard,), SENTINEL, device=DEV)
    w_room = torch.full((Hkv * T + 2 * guard,), SENTINEL, device=DEV)
    lse, w = lse_room[guard:-guard].view(Hq, T), w_room[guard:-guard].view(Hkv, T)
    cu_d = torch.tensor(cu, dtype=torch.int64).to(torch.int32).to(DEV)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    rtp.attn_packed(q, k, v, o_room[inner], [0, 1, 2, 3], cu_d, lse=lse, ws=ws)
    assert rtp.workspace_status(ws) == 0
    for n_obs in (None, 20):
        rtp.attn_key_weights(q, k, lse, w, [0, 1, 2, 3], cu_d, n_obs=n_obs, ws=ws)
        assert rtp.workspace_status(ws) == 0
    cache, _ = make_cache([T] * 3, Hkv, 16, torch.bfloat16, 13)
    rtp.paged_append(cache, k, v, cu_d, torch.tensor([0, 2 ** 31 - 1, -2 ** 31], dtype=torch.int64).to(torch.int32)
                     .to(DEV))
    torch.cuda.synchronize()
    for x in (o_room[:guard], o_room[-guard:], lse_room[:guard], lse_room[-guard:], w_room[:guard], w_room[-guard:]):
        assert (x == SENTINEL).all()


def test_cache_is_bound_to_its_tensors():
    cache, _ = make_cache([5], 1, 16, torch.bfloat16, 14)
    for name in ("k", "v", "table", "weights"):
        with pytest.raises(AttributeError):
            setattr(cache, name, None)
