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
