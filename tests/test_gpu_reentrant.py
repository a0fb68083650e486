"""Calls from other host threads than the one that loaded the library."""
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
