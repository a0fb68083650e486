"""Calls from other host threads than the one that loaded the library, one after
the other and side by side (the C calls run without the interpreter's lock)."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

rtp = pytest.importorskip("long_context_hybrid_b200")
DEV = "cuda"
D, R = 128, 16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from long_context_hybrid_b200 import build
    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    rtp.lib()


def rnd(gen, *shape):
    return torch.randn(*shape, generator=gen).to(torch.bfloat16).to(DEV)


@pytest.mark.parametrize("name", ["attn_packed", "attn_key_weights", "swa", "select_prefill", "triangle_prefill"])
def test_the_first_cuda_call_of_a_host_thread(name):
    """A thread that has made no CUDA call yet has no current context: a call that
    encodes tensor maps gives there what it gives elsewhere."""
    gen = torch.Generator().manual_seed(5)
    T, Hq, Hkv = 512, 4, 2
    q, k, v = (rnd(gen, 1, T, h, D) for h in (Hq, Hkv, Hkv))
    qt, kt = rnd(gen, 1, 2, T, R), rnd(gen, 1, 2, T, R)
    cu = torch.tensor([0, 300, T], dtype=torch.int32, device=DEV)
    heads = list(range(Hq))
    lse = torch.zeros(Hq, T, device=DEV)
    rtp.attn_packed(q[0], k[0], v[0], torch.zeros_like(q[0]), heads, cu, lse=lse)
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device=DEV)
    stream = torch.cuda.current_stream()
    outs = {n: torch.zeros_like(q) for n in ("attn_packed", "swa", "triangle_prefill")}
    outs["attn_key_weights"] = torch.zeros(Hkv, T, device=DEV)
    outs["select_prefill"] = torch.zeros(1, 2, T // 64, 4, dtype=torch.int32, device=DEV)
    counts = torch.zeros(1, 2, T // 64, dtype=torch.int32, device=DEV)
    out = outs[name]
    calls = {
        "attn_packed": lambda: rtp.attn_packed(q[0], k[0], v[0], out[0], heads, cu, ws=ws, stream=stream),
        "attn_key_weights": lambda: rtp.attn_key_weights(q[0], k[0], lse, out, heads, cu, ws=ws, stream=stream),
        "swa": lambda: rtp.swa(q, k, v, out, heads, 100, ws=ws, stream=stream),
        "select_prefill": lambda: rtp.select_prefill(qt, kt, [0, 1], 4, out, counts, ws=ws, stream=stream),
        "triangle_prefill": lambda: rtp.triangle_prefill(q, k, v, out, heads, 1, 2, 64, ws=ws, stream=stream),
    }
    calls[name]()
    torch.cuda.synchronize()
    want = out.clone()
    out.zero_()
    raised = []

    def work():
        try:
            calls[name]()
        except Exception as e:                   # noqa: BLE001 (shown by the assertion)
            raised.append(e)

    torch.cuda.synchronize()
    t = threading.Thread(target=work)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not raised, raised
    assert torch.equal(out, want)


def side_by_side(jobs, repeats):
    """Each job (C function, its arguments before the stream, its output) in a host
    thread and on a stream of its own: every call is accepted, and the outputs are
    those of the job alone."""
    bad = [[] for _ in jobs]
    outs = []
    for call, args, out in jobs:
        assert call(*args, torch.cuda.current_stream().cuda_stream) == 0
        torch.cuda.synchronize()
        outs.append(out.clone())
        out.zero_()
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    gate = threading.Barrier(len(jobs))

    def work(i):
        call, args, _ = jobs[i]
        gate.wait()
        for _ in range(repeats):
            s = call(*args, streams[i].cuda_stream)
            if s != 0:
                bad[i].append(s)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not any(bad), f"refused: {[len(b) for b in bad]} of {repeats} each, status {set(sum(bad, []))}"
    for (_, _, out), want in zip(jobs, outs):
        assert torch.equal(out, want)


def ws_of(n):
    return torch.zeros(n, dtype=torch.uint8, device=DEV)


def test_select_prefill():
    jobs, keep = [], []
    for N in (1024, 16384):
        gen = torch.Generator().manual_seed(N)
        qt, kt = (torch.randn(1, 1, N, R, generator=gen).to(torch.bfloat16).to(DEV) for _ in range(2))
        blocks = torch.zeros(1, 1, N // 64, 8, dtype=torch.int32, device=DEV)
        counts = torch.zeros(1, 1, N // 64, dtype=torch.int32, device=DEV)
        n = rtp.lib().rtp_workspace_size_select_prefill(1, N, 1, 8)
        ws = ws_of(n)
        keep.append((qt, kt, counts, ws))
        jobs.append((rtp.lib().rtp_select_prefill,
                     (qt.data_ptr(), kt.data_ptr(), N, 1, N, 1, 1, R, rtp._i32([0]), 8, blocks.data_ptr(),
                      counts.data_ptr(), ws.data_ptr(), n), blocks))
    side_by_side(jobs, 3000)


def test_sparse_attn_prefill():
    jobs, keep = [], []
    for N, topk in ((1024, 1), (16384, 64)):
        gen = torch.Generator().manual_seed(N)
        q, k, v = (torch.randn(1, N, 1, D, generator=gen).to(torch.bfloat16).to(DEV) for _ in range(3))
        o = torch.zeros_like(q)
        qt, kt = (torch.randn(1, 1, N, R, generator=gen).to(torch.bfloat16).to(DEV) for _ in range(2))
        blocks, counts = rtp.select_prefill(qt, kt, [0], topk)
        n = rtp.lib().rtp_workspace_size_sparse_attn_prefill(1, N, 1, topk)
        ws = ws_of(n)
        keep.append((q, k, v, o, blocks, counts, ws))
        s = rtp._strides4
        jobs.append((rtp.lib().rtp_sparse_attn_prefill,
                     (q.data_ptr(), s(q), k.data_ptr(), s(k), v.data_ptr(), s(v), o.data_ptr(), s(o), 1, N, 1, 1,
                      rtp._i32([0]), 1, blocks.data_ptr(), counts.data_ptr(), topk, 2, 1, D ** -0.5, ws.data_ptr(), n),
                     o))
    side_by_side(jobs, 2000)


@pytest.mark.parametrize("heads", [(3, 4), (5, 16)])
def test_select_decode(heads):
    L, topk = 4096, 64
    jobs, keep = [], []
    for Hr in heads:
        gen = torch.Generator().manual_seed(Hr)
        qt = torch.randn(1, Hr, R, generator=gen).to(DEV)
        kt = torch.randn(1, 1, L, R, generator=gen).to(torch.bfloat16).to(DEV)
        idx = torch.zeros(1, Hr, topk, dtype=torch.int32, device=DEV)
        n = rtp.lib().rtp_workspace_size_select_decode(1, L, Hr, topk)
        ws = ws_of(n)
        keep.append((qt, kt, ws))
        jobs.append((rtp.lib().rtp_select_decode,
                     (qt.data_ptr(), kt.data_ptr(), L, 1, L, Hr, 1, R, rtp._i32([0] * Hr), topk, idx.data_ptr(),
                      ws.data_ptr(), n), idx))
    side_by_side(jobs, 3000)
