"""CPU checks of the serving calls: refusals before any launch, and pins of
their oracle."""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import serving_oracle as SO

INVALID, UNSUP, WS = 1, 2, 5
FAKE = 0x10000                                  # never dereferenced: validation fails first
F = ctypes.c_float


@pytest.fixture(scope="module")
def rtp():
    from long_context_hybrid_b200 import build
    build.build()
    import long_context_hybrid_b200 as rtp
    rtp.lib()
    return rtp


def heads(*h):
    return (ctypes.c_int32 * len(h))(*h)


def packed(rtp, **kw):
    S = rtp.Strides
    a = dict(q=FAKE, qs=S(0, 1024, 128), k=FAKE, ks=S(0, 256, 128), v=FAKE, vs=S(0, 256, 128), o=FAKE,
             os=S(0, 1024, 128), dtype=0, T=100, Hq=8, Hkv=2, heads=heads(0, 3), n=2, cu=FAKE, S=3, window=10,
             scale=F(0.1), lse=None, ws=FAKE, ws_bytes=256, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return rtp.lib().rtp_attn_packed(*a.values())


def weights(rtp, **kw):
    S = rtp.Strides
    a = dict(q=FAKE, qs=S(0, 1024, 128), k=FAKE, ks=S(0, 256, 128), dtype=0, T=100, Hq=8, Hkv=2, heads=heads(0, 3),
             n=2, cu=FAKE, S=3, lse=FAKE, n_obs=5, window=10, scale=F(0.1), w=FAKE, ws=FAKE, ws_bytes=256,
             stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return rtp.lib().rtp_attn_key_weights(*a.values())


def cache(rtp, **kw):
    from long_context_hybrid_b200.serving import _CacheStruct
    S = rtp.Strides
    a = dict(k=FAKE, v=FAKE, ks=S(16 * 256, 256, 128), vs=S(16 * 256, 256, 128), weights=FAKE, table=FAKE,
             table_stride=8, num_pages=10, page_size=16, max_pages=8, Hkv=2)
    assert set(kw) <= set(a)
    a.update(kw)
    return _CacheStruct(*a.values())


def append(rtp, c=None, **kw):
    S = rtp.Strides
    a = dict(c=c or cache(rtp), k=FAKE, ks=S(0, 256, 128), v=FAKE, vs=S(0, 256, 128), w=None, T=5, cu=FAKE, S=2,
             pos=FAKE, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return rtp.lib().rtp_paged_append(*a.values())


def decode(rtp, c=None, **kw):
    S = rtp.Strides
    a = dict(q=FAKE, qs=S(1024, 0, 128), c=c or cache(rtp), lens=FAKE, max_len=128, o=FAKE, os=S(1024, 0, 128),
             dtype=0, B=2, Hq=8, heads=heads(0, 3), n=2, window=10, sink=1, scale=F(0.1), lse=None, w=None, ws=FAKE,
             ws_bytes=1 << 30, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return rtp.lib().rtp_paged_attn_decode(*a.values())


def evict(rtp, src=None, dst=None, **kw):
    src = src or cache(rtp)
    a = dict(src=src, dst=dst or src, B=2, lens=FAKE, max_len=128, budget=64, sink=4, recent=10, idx=FAKE,
             new=FAKE + 64, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return rtp.lib().rtp_cache_evict(*a.values())


@pytest.mark.parametrize("call", [packed, weights])
def test_packed_calls_refuse(rtp, call):
    S = rtp.Strides
    for name in ("q", "k", "cu", "heads"):
        assert call(rtp, **{name: None}) == INVALID, name
    for kw in (dict(q=FAKE + 2), dict(k=FAKE + 8), dict(qs=S(0, 1020, 128)), dict(ks=S(0, 0, 128)),
               dict(ks=S(0, 256, 64)), dict(qs=S(0, -1024, 128)), dict(T=-1), dict(S=0), dict(Hkv=3), dict(Hq=0),
               dict(dtype=1), dict(dtype=7), dict(window=0), dict(scale=F(0.0)), dict(scale=F(float("nan"))),
               dict(n=0), dict(n=129), dict(heads=heads(0, 8)), dict(heads=heads(-1, 0)), dict(heads=heads(3, 3))):
        assert call(rtp, **kw) == INVALID, kw
    assert call(rtp, Hq=512, Hkv=2, heads=heads(0), n=1) == UNSUP
    assert call(rtp, T=(1 << 30) + 1) == UNSUP
    assert call(rtp, S=1 << 30, heads=heads(0, 1, 2), n=3) == UNSUP
    for kw in (dict(ws=None), dict(ws_bytes=255), dict(ws=FAKE + 16)):
        assert call(rtp, **kw) == WS, kw


def test_packed_calls_refuse_what_is_theirs(rtp):
    assert packed(rtp, v=None) == INVALID
    assert packed(rtp, o=None) == INVALID
    assert packed(rtp, os=rtp.Strides(0, 0, 128)) == INVALID
    assert packed(rtp, vs=rtp.Strides(0, 256, 0)) == INVALID
    assert weights(rtp, lse=None) == INVALID
    assert weights(rtp, w=None) == INVALID
    assert weights(rtp, n_obs=0) == INVALID


@pytest.mark.parametrize("call", [append, decode, evict])
def test_caches_are_checked(rtp, call):
    S = rtp.Strides
    for kw in (dict(k=None), dict(v=None), dict(table=None), dict(num_pages=0), dict(page_size=0), dict(max_pages=0),
               dict(Hkv=0), dict(table_stride=7), dict(k=FAKE + 8), dict(ks=S(16 * 256, 252, 128)),
               dict(vs=S(0, 256, 128)), dict(vs=S(16 * 256, 256, 64))):
        assert call(rtp, cache(rtp, **kw)) == INVALID, kw
    for kw in (dict(page_size=24), dict(page_size=1 << 17), dict(Hkv=129),
               dict(page_size=65536, max_pages=1 << 15, table_stride=1 << 15)):
        assert call(rtp, cache(rtp, **kw)) == UNSUP, kw


def test_paged_calls_refuse(rtp):
    S = rtp.Strides
    assert rtp.lib().rtp_paged_append(None, FAKE, S(0, 256, 128), FAKE, S(0, 256, 128), None, 5, FAKE, 2, FAKE,
                                      None) == INVALID
    for kw in (dict(k=None), dict(v=None), dict(cu=None), dict(pos=None), dict(T=-1), dict(S=0), dict(k=FAKE + 2),
               dict(ks=S(0, 0, 128)), dict(vs=S(0, 256, 100))):
        assert append(rtp, **kw) == INVALID, kw
    assert append(rtp, cache(rtp, weights=None), w=FAKE) == INVALID
    for kw in (dict(q=None), dict(o=None), dict(lens=None), dict(dtype=1), dict(B=0), dict(Hq=7), dict(max_len=0),
               dict(max_len=129), dict(window=0), dict(sink=-1), dict(scale=F(-1.0)), dict(heads=None),
               dict(heads=heads(0, 8)), dict(q=FAKE + 4), dict(qs=S(0, 0, 128)), dict(os=S(1024, 0, 8))):
        assert decode(rtp, **kw) == INVALID, kw
    assert decode(rtp, cache(rtp, weights=None), w=FAKE) == INVALID
    assert decode(rtp, Hq=34, heads=heads(0), n=1) == UNSUP
    assert decode(rtp, B=65536) == UNSUP
    need = rtp.lib().rtp_workspace_size_paged_attn_decode(2, 128, 2, 10, 1, 1)
    for kw in (dict(ws=None), dict(ws=FAKE + 8), dict(ws_bytes=255), dict(w=FAKE, ws_bytes=need - 1)):
        assert decode(rtp, **kw) == WS, kw


def test_evict_refuses(rtp):
    for kw in (dict(lens=None), dict(idx=None), dict(new=None), dict(new=FAKE), dict(B=0), dict(max_len=0),
               dict(max_len=129), dict(budget=0), dict(sink=-1), dict(recent=-1), dict(sink=60),
               dict(sink=2 ** 31 - 1, recent=2 ** 31 - 1)):
        assert evict(rtp, **kw) == INVALID, kw
    assert evict(rtp, cache(rtp, weights=None)) == INVALID
    other = dict(k=FAKE * 2, v=FAKE * 3, weights=FAKE * 4, table=FAKE * 5)
    assert evict(rtp, dst=cache(rtp, **{**other, "Hkv": 1})) == INVALID
    assert evict(rtp, dst=cache(rtp, **{**other, "max_pages": 3})) == INVALID          # 48 slots for 64 tokens
    for shared in ("k", "v", "weights"):                                               # one buffer, one table
        assert evict(rtp, dst=cache(rtp, **{x: y for x, y in other.items() if x not in (shared, "table")})) == INVALID
    assert evict(rtp, dst=cache(rtp, page_size=32)) == INVALID                         # in place with another page size
    assert evict(rtp, cache(rtp, Hkv=128), B=512) == UNSUP


def test_decode_workspace_follows_what_is_attended(rtp):
    size = rtp.lib().rtp_workspace_size_paged_attn_decode
    assert size(8, 131072, 32, 131072, 0, 0) == size(8, 64, 32, 64, 0, 0)      # partials: by CTAs, not by lengths
    assert size(8, 131072, 32, 131072, 0, 1) - size(8, 131072, 32, 131072, 0, 0) >= 8 * 32 * 131072 * 4
    scores = lambda window, sink: size(8, 131072, 32, window, sink, 1) - size(8, 131072, 32, window, sink, 0)  # noqa: E731
    assert scores(1000, 4) < scores(131072, 0) / 50


def test_binding_refuses_before_the_call(rtp):
    """What the C side cannot see: dtypes, shapes, layouts, devices."""
    E = rtp.RtpError
    bf = dict(dtype=torch.bfloat16)
    k = torch.zeros(4, 16, 2, 128, **bf)
    table = torch.zeros(2, 3, dtype=torch.int32)
    for bad in ((k.float(), k.float(), table), (k, k.half(), table), (k, k[:3], table), (k[..., :64], k[..., :64], table),
                (k, k, table.long()), (k, k, table[0]), (k, k.transpose(2, 3), table), (k, k, table.t())):
        with pytest.raises(E):
            rtp.PagedCache(*bad)
    with pytest.raises(E):
        rtp.PagedCache(k, k, table)                              # not on a GPU
    q, kv = torch.zeros(5, 4, 128, **bf), torch.zeros(5, 2, 128, **bf)
    with pytest.raises(E):
        rtp.attn_packed(q, kv, kv, q.clone(), [0], torch.zeros(2, dtype=torch.int32))
    with pytest.raises(E):
        rtp.attn_key_weights(q, kv, torch.zeros(1, 5), torch.zeros(2, 5), [0], torch.zeros(2, dtype=torch.int32))


# ---------------------------------------------------------------------------
# Pins of the oracle
# ---------------------------------------------------------------------------
def test_oracle_packed_head_is_masked_softmax_attention():
    rng = np.random.default_rng(0)
    q, k, v = (rng.standard_normal((9, 16)) for _ in range(3))
    for window in (1, 3, 9, 100):
        mask = torch.tensor([[u <= t and t - u < window for u in range(9)] for t in range(9)])
        ref = torch.nn.functional.scaled_dot_product_attention(
            torch.from_numpy(q)[None], torch.from_numpy(k)[None], torch.from_numpy(v)[None], attn_mask=mask[None],
            scale=0.3)[0].numpy()
        o, lse, _, _ = SO.packed_head(q, k, v, window, 0.3)
        assert np.allclose(o, ref, atol=1e-12)
        t = 5
        assert math.isclose(lse[t], math.log(sum(math.exp(0.3 * q[t] @ k[u]) for u in range(9) if mask[t, u])))


def test_oracle_key_weights_sum_to_the_observed_rows():
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((12, 16)), rng.standard_normal((12, 16))
    for window, n_obs in ((12, 12), (4, 12), (12, 1), (5, 3)):
        lse = SO.packed_head(q, k, k, window, 0.2)[1]
        w = SO.key_weights_head(q, k, lse, n_obs, window, 0.2)[0]
        assert math.isclose(w.sum(), n_obs)                       # every row's weights sum to 1
    assert np.count_nonzero(SO.key_weights_head(q, k, lse, 3, 5, 0.2)[0]) == 7     # rows 9..11 with 5 keys each


def test_oracle_decode_and_packed_agree_on_the_last_row():
    rng = np.random.default_rng(2)
    q, k, v = (rng.standard_normal((20, 16)) for _ in range(3))
    assert np.array_equal(SO.decode_slots(20, 6, 0), np.arange(14, 20))
    assert np.array_equal(SO.decode_slots(5, 6, 2), np.arange(5))
    assert np.array_equal(SO.decode_slots(10, 3, 2), [0, 1, 7, 8, 9])
    o, lse, p, _, _ = SO.decode_head(q[19], k, v, SO.decode_slots(20, 6, 0), 0.25)
    ref, rl, _, _ = SO.packed_head(q, k, v, 6, 0.25)
    assert np.allclose(o, ref[19]) and math.isclose(lse, rl[19]) and math.isclose(p.sum(), 1)


def test_oracle_eviction_by_hand():
    w = np.array([9, 1, 5, 5, np.nan, 0.0, -0.0, 5, 2, 3], np.float32)
    keep = lambda *a: SO.evict_slots(w, 10, *a).tolist()  # noqa: E731
    assert keep(3, 0, 0) == [0, 2, 4]                 # NaN first, then 9, then the lowest 5
    assert keep(4, 0, 0) == [0, 2, 3, 4]
    assert keep(4, 1, 2) == [0, 4, 8, 9]
    assert keep(9, 0, 0) == [0, 1, 2, 3, 4, 5, 7, 8, 9]    # 0.0 and -0.0 tie
    assert keep(10, 0, 0) == list(range(10))
    assert SO.evict_slots(w, 4, 5, 1, 1).tolist() == [0, 1, 2, 3]


def test_oracle_append_drops_what_has_no_slot():
    pages = np.zeros((3, 2, 1))
    table = np.array([[2, 0], [1, 7]])
    rows = np.arange(1, 8, dtype=float)[:, None]
    got = SO.append(pages, rows, [1, 4, 7], [1, 0], table, 2)
    # sequence 0: rows 1..3 to slots 1, 2, 3; sequence 1: rows 4, 5 to page 1, row 6 to a page that is not there
    assert got[:, :, 0].tolist() == [[3, 4], [5, 6], [0, 2]]
