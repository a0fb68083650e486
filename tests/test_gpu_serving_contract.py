"""What the serving calls promise beside their results: concurrent host threads,
graphs, streams, empty batches, statuses and full caches, on the GPU."""
import ctypes
import threading

import numpy as np
import pytest
import torch

from oracle import serving_oracle as SO
from test_gpu_serving import D, DEV, _built, make_cache  # noqa: F401  (_built: the module's fixture)

pytestmark = pytest.mark.gpu

rtp = pytest.importorskip("long_context_hybrid_b200")


def _struct(cache):
    """The cache as the C ABI takes it."""
    from long_context_hybrid_b200.serving import _CacheStruct
    S = rtp.Strides
    k, v, t = cache.k, cache.v, cache.table
    return _CacheStruct(k.data_ptr(), v.data_ptr(), S(*k.stride()[:3]), S(*v.stride()[:3]), cache.weights.data_ptr(),
                        t.data_ptr(), t.stride(0), k.shape[0], k.shape[1], t.shape[1], k.shape[2])


def test_evictions_of_two_host_threads():
    """Calls are reentrant: a small and a large eviction, issued side by side by
    two host threads (the C calls run without the interpreter's lock), are each
    accepted and each give what they give alone."""
    jobs = []
    for n, budget, seed in ((300, 100, 1), (400_000, 1000, 2)):
        page = 256
        pages = (n + page - 1) // page
        gen = torch.Generator().manual_seed(seed)
        k = torch.zeros(pages, page, 1, D, dtype=torch.bfloat16, device=DEV)
        w = torch.rand(pages, 1, page, generator=gen).to(DEV)
        table = torch.randperm(pages, generator=gen).to(torch.int32)[None].to(DEV)
        src = rtp.PagedCache(k, k.clone(), table, w)
        kept = (budget + page - 1) // page
        dst = rtp.PagedCache(*(torch.zeros(kept, page, 1, D, dtype=torch.bfloat16, device=DEV) for _ in range(2)),
                             torch.arange(kept, dtype=torch.int32, device=DEV)[None],
                             torch.zeros(kept, 1, page, device=DEV))
        flat = w.cpu()[table[0].cpu().long(), 0].flatten()[:n].numpy()
        jobs.append(dict(src=src, dst=dst, n=n, budget=budget, lens=torch.tensor([n], dtype=torch.int32, device=DEV),
                         idx=torch.zeros(1, 1, budget, dtype=torch.int32, device=DEV),
                         new=torch.zeros(1, dtype=torch.int32, device=DEV), stream=torch.cuda.Stream(),
                         want=SO.evict_slots(flat, n, budget, 2, 10), bad=[]))
    torch.cuda.synchronize()
    call, gate = rtp.lib().rtp_cache_evict, threading.Barrier(len(jobs))

    def work(j):
        a, b = _struct(j["src"]), _struct(j["dst"])
        gate.wait()
        for _ in range(4000):
            s = call(ctypes.byref(a), ctypes.byref(b), 1, j["lens"].data_ptr(), j["n"], j["budget"], 2, 10,
                     j["idx"].data_ptr(), j["new"].data_ptr(), j["stream"].cuda_stream)
            if s != 0:
                j["bad"].append(s)

    threads = [threading.Thread(target=work, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for j in jobs:
        assert not j["bad"], f"{len(j['bad'])} calls refused, status {set(j['bad'])}"
        assert np.array_equal(j["idx"].cpu().numpy()[0, 0], j["want"])
        assert j["new"].tolist() == [j["budget"]]


def make_layer(B, capacity, Hq=4, Hkv=2, page=16, seed=0, **kw):
    """A layer over zeroed pages in random order."""
    gen = torch.Generator().manual_seed(seed)
    pages = B * capacity // page
    cache = rtp.PagedCache(*(torch.zeros(pages, page, Hkv, D, dtype=torch.bfloat16, device=DEV) for _ in range(2)),
                           torch.randperm(pages, generator=gen).to(torch.int32).view(B, -1).to(DEV),
                           torch.zeros(pages, Hkv, page, device=DEV))
    return rtp.PagedLayer(cache, Hq, **kw), gen


def rows(gen, n, H, scale=1.0):
    return (torch.randn(n, H, D, generator=gen) * scale).to(torch.bfloat16).to(DEV)


def test_empty_prompts():
    """A batch of empty prompts: nothing is attended, weighed or cached, and
    decoding goes on from length 0."""
    B = 3
    layer, gen = make_layer(B, 32)
    layer.lens.fill_(5)
    q, kv = rows(gen, 0, 4), rows(gen, 0, 2)
    cu = torch.zeros(B + 1, dtype=torch.int32, device=DEV)
    layer.prefill(q, kv, kv, torch.zeros_like(q), cu)
    assert layer.lens.tolist() == [0] * B and not layer.cache.weights.any()
    q1, k1, v1 = rows(gen, B, 4), rows(gen, B, 2), rows(gen, B, 2)
    o1 = torch.zeros_like(q1)
    layer.decode(q1, k1, v1, o1)
    assert torch.equal(o1, v1.repeat_interleave(2, dim=1))     # one key: its value
    assert layer.lens.tolist() == [1] * B


@pytest.mark.parametrize("late", [0, 1, 2, 3])
def test_a_prefills_status_survives_its_later_calls(monkeypatch, late):
    """A prefill of full and streaming heads makes four tensor-core calls. A
    status that one of them leaves (planted here) is still there at the end, and
    gone after the next prefill."""
    from long_context_hybrid_b200 import serving
    layer, gen = make_layer(2, 64, streaming=[1], window=8, sink=1)
    lens = [20, 7]
    q, k, v = rows(gen, 27, 4), rows(gen, 27, 2), rows(gen, 27, 2)
    cu = torch.tensor([0, 20, 27], dtype=torch.int32, device=DEV)
    made = []

    def planting(call):
        def wrapped(*args):
            call(*args)
            if len(made) == late:
                args[-1].view(torch.int32)[0] = 4
            made.append(call)
        return wrapped

    o = torch.zeros_like(q)
    with monkeypatch.context() as m:
        for name in ("attn_packed", "attn_key_weights"):
            m.setattr(serving, name, planting(getattr(serving, name)))
        layer.prefill(q, k, v, o, cu)
    assert len(made) == 4
    assert layer.device_status() == 4 and layer.device_status(torch.cuda.Stream()) == 4
    layer.decode(rows(gen, 2, 4), rows(gen, 2, 2), rows(gen, 2, 2), rows(gen, 2, 4))
    assert layer.device_status() == 4
    layer.prefill(q, k, v, o, cu)
    assert layer.device_status() == 0 and layer.lens.tolist() == lens


def test_tokens_beyond_the_capacity_are_reported():
    """A full sequence: what finds no slot is dropped and counted, in prompts and
    in decoding, before and after an eviction; nobody else's pages change."""
    B, cap = 3, 32
    layer, gen = make_layer(B, cap)
    lens = [40, 31, 3]
    q, k, v = (rows(gen, sum(lens), h) for h in (4, 2, 2))
    cu = torch.tensor([0, 40, 71, 74], dtype=torch.int32, device=DEV)
    layer.prefill(q, k, v, torch.zeros_like(q), cu)
    assert layer.dropped().tolist() == [8, 0, 0]
    cached = lambda b, n: layer.cache.k[layer.cache.table[b].long()].flatten(0, 1)[:n]  # noqa: E731
    for b, n in enumerate([32, 31, 3]):
        assert torch.equal(cached(b, n), k[cu[b]:cu[b] + n])
    new = []
    for step in range(3):
        q1, k1, v1 = (rows(gen, B, h) for h in (4, 2, 2))
        new.append(k1)
        layer.decode(q1, k1, v1, torch.zeros_like(q1))
    assert layer.dropped().tolist() == [11, 2, 0]
    assert torch.equal(cached(0, 32), k[:32])
    assert torch.equal(cached(1, 32), torch.cat([k[40:71], new[0][1:2]]))
    assert torch.equal(cached(2, 6), torch.cat([k[71:74]] + [x[2:3] for x in new]))
    layer.evict(20, 10)
    assert layer.lens.tolist() == [20, 20, 6] and layer.dropped().tolist() == [11, 2, 0]
    layer.decode(q1, k1, v1, torch.zeros_like(q1))
    assert layer.lens.tolist() == [21, 21, 7] and layer.dropped().tolist() == [11, 2, 0]
    layer.prefill(q, k, v, torch.zeros_like(q), cu)
    assert layer.dropped().tolist() == [8, 0, 0]


def test_a_layers_buffers_are_ready_on_every_stream():
    """A layer made on a stream that is still busy, used on another at once."""
    busy, other = torch.cuda.Stream(), torch.cuda.Stream()
    ready, gen = make_layer(2, 32)
    q, k, v = (rows(gen, 2, h) for h in (4, 2, 2))
    o = torch.zeros_like(q)
    ready.decode(q, k, v, o, stream=other)       # every kernel is loaded before the sleep
    ready.cache.k.zero_(), ready.cache.v.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(busy):
        torch.cuda._sleep(400_000_000)           # about a fifth of a second
        layer = rtp.PagedLayer(ready.cache, 4)
    layer.decode(q, k, v, o, stream=other)
    torch.cuda.synchronize()
    assert layer.lens.tolist() == [1, 1] and layer.cu_decode.tolist() == [0, 1, 2]
    assert torch.equal(o, v.repeat_interleave(2, dim=1))


@pytest.mark.parametrize("in_place", [False, True])
def test_eviction_around_missing_pages(in_place):
    """Slots whose page is missing rank behind every token, move nothing and
    leave their new slot as it was; all the others move as ever."""
    lens, page, budget, sink, recent, Hkv = [300, 90], 16, 64, 20, 20, 2
    cache, gen = make_cache(lens, Hkv, page, torch.bfloat16, 15)
    for b, j, bad in ((0, 1, -1), (0, 7, 10 ** 6), (1, 0, -2 ** 31), (1, 3, cache.num_pages), (0, 18, -1)):
        cache.table[b, j] = bad                  # in the sink, among the candidates, at the end
    table = cache.table.cpu().long()
    there = (table >= 0) & (table < cache.num_pages)
    old = [x.cpu() for x in (cache.k, cache.v)]
    old_w = cache.weights.cpu()
    out = cache
    if not in_place:
        out, _ = make_cache([budget] * 2, Hkv, 32, torch.bfloat16, 16)
        for x in (out.k, out.v, out.weights):
            x.fill_(7.0)
    before = [x.cpu() for x in (out.k, out.v)]
    before_w = out.weights.cpu()
    idx, new = rtp.cache_evict(cache, torch.tensor(lens, dtype=torch.int32, device=DEV), budget, sink, recent,
                               out=None if in_place else out)
    assert new.tolist() == [budget, budget]
    to = out.table.cpu().long()
    there_to = (to >= 0) & (to < out.num_pages)
    for b, n in enumerate(lens):
        s = torch.arange(n)
        real = there[b][s // page]
        for g in range(Hkv):
            w = torch.where(real, old_w[table[b][s // page].clamp(0, cache.num_pages - 1), g, s % page], -torch.inf)
            want = SO.evict_slots(w.numpy(), n, budget, sink, recent)
            assert np.array_equal(idx[b, g].cpu().numpy(), want)
            for j, slot in enumerate(want):
                dp, do = to[b, j // out.page_size], j % out.page_size
                if not there_to[b, j // out.page_size]:
                    continue
                sp, so = table[b, slot // page], slot % page
                moved = bool(real[slot])
                for x, o, was in zip((out.k, out.v), old, before):
                    assert torch.equal(x[dp, do, g].cpu(), o[sp, so, g] if moved else was[dp, do, g])
                assert out.weights[dp, g, do] == (old_w[sp, g, so] if moved else before_w[dp, g, do])


def test_calls_in_the_order_that_the_readme_shows():
    """The calls one by one, the new token appended before it attends, give what
    PagedLayer gives: prompts, an eviction, a token."""
    B, Hq, Hkv, cap, lens = 2, 4, 2, 128, [100, 37]
    layer, gen = make_layer(B, cap, seed=3, n_obs=16, sink=2)
    twin, _ = make_layer(B, cap, seed=3)
    cache, heads = twin.cache, list(range(Hq))
    q, k, v = (rows(gen, sum(lens), h) for h in (Hq, Hkv, Hkv))
    q1, k1, v1 = (rows(gen, B, h) for h in (Hq, Hkv, Hkv))
    cu = torch.tensor([0, 100, 137], dtype=torch.int32, device=DEV)
    o, o1 = torch.zeros_like(q), torch.zeros_like(q1)
    layer.prefill(q, k, v, o, cu)
    kept = layer.evict(50, 10)
    layer.decode(q1, k1, v1, o1)

    mine, mine1 = torch.zeros_like(q), torch.zeros_like(q1)
    lse, w = torch.zeros(Hq, sum(lens), device=DEV), torch.zeros(Hkv, sum(lens), device=DEV)
    pos, cu1 = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([0, 0], [0, 1, 2]))
    lens_d = torch.tensor(lens, dtype=torch.int32, device=DEV)
    rtp.attn_packed(q, k, v, mine, heads, cu, lse=lse)
    rtp.attn_key_weights(q, k, lse, w, heads, cu, n_obs=16)
    rtp.paged_append(cache, k, v, cu, pos, weights=w)
    idx, lens_d = rtp.cache_evict(cache, lens_d, 50, sink=2, recent=10)
    rtp.paged_append(cache, k1, v1, cu1, lens_d)
    lens_d += 1
    rtp.paged_attn_decode(q1, cache, lens_d, mine1, heads, weights_out=cache.weights)
    for a, b in ((o, mine), (kept, idx), (o1, mine1), (layer.lens, lens_d), (layer.cache.k, cache.k),
                 (layer.cache.v, cache.v), (layer.cache.weights, cache.weights)):
        assert torch.equal(a, b)


def test_captured_eviction_follows_lengths_tables_and_weights():
    """A captured eviction and the step behind it replay with the lengths, tables,
    rows and weights that the buffers hold at the replay."""
    B, Hq, Hkv, cap, budget = 2, 4, 2, 256, 40
    layer, gen = make_layer(B, cap, Hq, Hkv, sink=3)
    cache = layer.cache
    for x in (cache.k, cache.v):
        x.copy_(torch.randn(x.shape, generator=gen).to(x))
    q1, k1, v1 = (rows(gen, B, h) for h in (Hq, Hkv, Hkv))
    o = torch.zeros_like(q1)

    def step():
        idx = layer.evict(budget, 11)
        layer.decode(q1, k1, v1, o)
        return idx

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        idx = step()
    for lens in ([256, 41], [40, 200], [0, 256], [39, 1]):
        cache.table.copy_(torch.randperm(cache.num_pages, generator=gen).to(torch.int32).view(B, -1))
        cache.weights.copy_(torch.rand(cache.weights.shape, generator=gen))
        layer.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        saved = [x.clone() for x in (cache.k, cache.v, cache.weights, layer.lens)]
        graph.replay()
        got = [x.clone() for x in (idx, o, cache.k, cache.v, cache.weights, layer.lens)]
        for b, n in enumerate(lens):
            s = torch.arange(n)
            for g in range(Hkv):
                w = saved[2].cpu()[cache.table[b].cpu().long()[s // 16], g, s % 16].numpy()
                want = SO.evict_slots(w, n, budget, 3, 11)
                assert np.array_equal(got[0][b, g].cpu().numpy()[:len(want)], want)
        for x, y in zip((cache.k, cache.v, cache.weights, layer.lens), saved):
            x.copy_(y)
        o.zero_()
        again = step()
        for x, y in zip(got, (again, o, cache.k, cache.v, cache.weights, layer.lens)):
            assert torch.equal(x, y)
        assert layer.lens.tolist() == [min(n, budget) + 1 for n in lens]


@pytest.mark.parametrize("budget,sink,recent", [(100, 4, 20), (64, 0, 0), (30, 10, 20)])
def test_a_loops_eviction_keeps_what_its_weights_say(budget, sink, recent):
    """After prompts and steps, the layer's choice is the oracle's on the weights
    that the cache holds."""
    lens, Hq, Hkv = [150, 1, 333], 8, 2
    layer, gen = make_layer(3, 512, Hq, Hkv, seed=9, sink=sink, n_obs=32)
    q, k, v = (rows(gen, sum(lens), h, 1.3) for h in (Hq, Hkv, Hkv))
    cu = torch.tensor([0, 150, 151, 484], dtype=torch.int32, device=DEV)
    layer.prefill(q, k, v, torch.zeros_like(q), cu)
    for _ in range(4):
        q1, k1, v1 = (rows(gen, 3, h, 1.3) for h in (Hq, Hkv, Hkv))
        layer.decode(q1, k1, v1, torch.zeros_like(q1))
    w, table = layer.cache.weights.cpu(), layer.cache.table.cpu().long()
    idx = layer.evict(budget, recent).cpu().numpy()
    for b, n in enumerate(x + 4 for x in lens):
        s = torch.arange(n)
        for g in range(Hkv):
            want = SO.evict_slots(w[table[b][s // 16], g, s % 16].numpy(), n, budget, sink, recent)
            assert np.array_equal(idx[b, g][:len(want)], want) and (idx[b, g][len(want):] == -1).all()


@pytest.mark.parametrize("cu", [[0, 300, 100, 400], [500, -5, 10 ** 9, 20], [-10, -10, -10, -10], [400, 300, 200, 0],
                                [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1, 17], [390, 390, 400, 1000]])
def test_bad_offsets_of_an_append_stay_inside_the_pages(cu):
    """Offsets that decrease or leave [0, T] and positions out of range: the pages
    in front of and behind the pool, and the weights there, are left alone."""
    T, Hkv, page, n, guard = 400, 2, 16, 80, 8
    gen = torch.Generator().manual_seed(17)
    pools = [torch.full((n + 2 * guard, page, Hkv, D), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    weights = torch.full((n + 2 * guard, Hkv, page), 7.0, device=DEV)
    inner = slice(guard, guard + n)
    table = torch.randperm(n, generator=gen).to(torch.int32)[:75].view(3, 25).to(DEV)
    cache = rtp.PagedCache(pools[0][inner], pools[1][inner], table, weights[inner])
    k, v = rows(gen, T, Hkv), rows(gen, T, Hkv)
    cu_d = torch.tensor(cu, dtype=torch.int64).to(torch.int32).to(DEV)
    for pos in ([0, 2 ** 31 - 1, -2 ** 31], [-100, 399, 5], [400, -1, 0]):
        rtp.paged_append(cache, k, v, cu_d, torch.tensor(pos, dtype=torch.int64).to(torch.int32).to(DEV),
                         weights=torch.rand(Hkv, T, device=DEV))
    for x in (*pools, weights):
        assert (x[:guard] == 7.0).all() and (x[guard + n:] == 7.0).all()
