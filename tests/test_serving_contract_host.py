"""CPU checks of what the serving calls promise: argument marshalling seen
through stand-in tensors (nothing here reaches a device)."""
import ctypes

import numpy as np
import pytest
import torch

from long_context_hybrid_b200 import serving
from oracle import serving_oracle as SO
from serving_bounds import D, o_bound

FAKE = 0x10000                                  # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def rtp():
    from long_context_hybrid_b200 import build
    build.build()
    import long_context_hybrid_b200 as rtp
    rtp.lib()
    return rtp


class OnGpu:
    """A CPU tensor's layout under a device number and an address."""

    def __init__(self, t, address=FAKE):
        self.t, self.address, self.dtype, self.shape = t, address, t.dtype, t.shape

    def stride(self):
        return self.t.stride()

    def data_ptr(self):
        return self.address

    def get_device(self):
        return 0


@pytest.fixture
def native(rtp, monkeypatch):
    """The native module with device 0 current, whatever the machine has."""
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(serving, "_native", None)
    yield serving._marshal()
    monkeypatch.undo()
    serving._native = None                       # set up again at the next call


def test_tensors_without_rows_are_contiguous(rtp, native):
    """T = 0 with several listed heads: the empty lse and weights are taken as
    they are, and the call goes on to the C checks (a misaligned workspace ends
    it there)."""
    q, k = (OnGpu(torch.zeros(0, h, 128, dtype=torch.bfloat16)) for h in (4, 2))
    cu = OnGpu(torch.zeros(4, dtype=torch.int32))
    lse, w = OnGpu(torch.zeros(3, 0)), OnGpu(torch.zeros(2, 0))
    ws = OnGpu(torch.zeros(256, dtype=torch.uint8), FAKE + 16)
    heads = serving._head_bytes((0, 1, 3))
    with pytest.raises(rtp.RtpError, match="RTP_ERR_WORKSPACE"):
        native.attn_packed(q, k, k, q, heads, cu, None, None, lse, ws, 0)
    with pytest.raises(rtp.RtpError, match="RTP_ERR_WORKSPACE"):
        native.attn_key_weights(q, k, lse, w, heads, cu, None, None, None, ws, 0)
    with pytest.raises(rtp.RtpError, match="contiguous"):         # the shape is still checked
        native.attn_packed(q, k, k, q, heads, cu, None, None, OnGpu(torch.zeros(2, 0)), ws, 0)
    strided = OnGpu(torch.zeros(3, 8)[:, ::2])
    q5, k5 = (OnGpu(torch.zeros(4, h, 128, dtype=torch.bfloat16)) for h in (4, 2))
    with pytest.raises(rtp.RtpError, match="contiguous"):         # and so is the layout of what has rows
        native.attn_packed(q5, k5, k5, q5, heads, cu, None, None, strided, ws, 0)


def test_decode_refuses_what_its_split_cannot_count(rtp):
    """The split counts the 64-slot chunks of up to 128 sequences in 32 bits:
    128 sequences of 2^30 attended slots are refused before the workspace is
    looked at, 127 of them or a window that bounds them are not."""
    S = rtp.Strides
    c = serving._CacheStruct(FAKE, FAKE, S(65536 * 128, 128, 128), S(65536 * 128, 128, 128), FAKE, FAKE, 1 << 14, 10,
                             65536, 1 << 14, 1)
    heads = (ctypes.c_int32 * 1)(0)

    def decode(B, max_len=1 << 30, window=2 ** 31 - 1, sink=0, ws=None):
        return rtp.lib().rtp_paged_attn_decode(FAKE, S(128, 0, 128), c, FAKE, max_len, FAKE, S(128, 0, 128), 0, B, 1,
                                               heads, 1, window, sink, ctypes.c_float(0.1), None, None, ws, 1 << 40,
                                               None)

    unsupported, workspace = 2, 5
    for B in (128, 129, 65535):
        assert decode(B) == unsupported, B
        assert decode(B, window=1 << 29, sink=1 << 29) == unsupported, B
        assert decode(B, window=1 << 20) == workspace, B
        assert decode(B, max_len=1 << 29) == workspace, B
    assert decode(127) == workspace


@pytest.fixture
def small_build(tmp_path, monkeypatch):
    """The build over one small source, into a folder of its own."""
    from long_context_hybrid_b200 import build
    src = tmp_path / "one.cu"
    src.write_text('extern "C" __attribute__((visibility("default"))) int one() { return 1; }\n')
    for name, value in (("OUT", tmp_path / "librtp.so"), ("MARSHAL", tmp_path / "_marshal.so"),
                        ("BUILD_DIR", tmp_path / "_build")):
        monkeypatch.setattr(build, name, str(value))
    monkeypatch.setattr(build, "sources", lambda: [str(src)])
    return build


def test_library_builds_without_python_headers(small_build, tmp_path, monkeypatch):
    real = small_build.sysconfig.get_paths()
    monkeypatch.setattr(small_build.sysconfig, "get_paths", lambda: {**real, "include": str(tmp_path / "none")})
    (tmp_path / "_marshal.so").write_text("of an earlier library")
    with pytest.warns(UserWarning, match="Python.h"):
        small_build.build(force=True)
    assert ctypes.CDLL(small_build.OUT).one() == 1 and not (tmp_path / "_marshal.so").exists()
    assert small_build.up_to_date()


def test_library_is_there_although_the_module_fails(small_build, tmp_path, monkeypatch):
    monkeypatch.setattr(small_build, "cxx", lambda: "false")
    with pytest.raises(RuntimeError, match="marshal.cpp"):
        small_build.build()
    assert ctypes.CDLL(small_build.OUT).one() == 1
    assert not small_build.up_to_date()                          # the module is still to be built


# ---------------------------------------------------------------------------
# The bound that the GPU tests use
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n", [64, 1500, 9000])
def test_bound_rejects_what_is_lost(n, dtype):
    """An output of zeros and one that leaves out 64 keys in the middle are off by
    more than the bound at many places (where 64 keys weigh 8 u or more); so is one with a gain of 8 steps of the
    type where values share a sign (8 steps are 16 u |ref|, the bound is a little
    over 2 u |ref| there; values about 0 leave |ref| below u sum p|v| / 16 u on
    long rows, and no bound on roundings can tell). The exact one rounded to the
    type is within it everywhere."""
    rng = np.random.default_rng(n)
    q, k, v = (rng.standard_normal(s) for s in ((8, D), (n, D), (n, D)))
    q *= 1.5
    for row in q:
        ref, _, p, pv, size = SO.decode_head(row, k, v, np.arange(n), D ** -0.5)
        tol = o_bound(ref, pv, size, dtype, np.abs(v).sum(0))
        rounded = torch.from_numpy(ref).to(dtype).double().numpy()
        assert (np.abs(rounded - ref) <= tol).all()
        assert np.mean(np.abs(ref) > tol) > 0.75     # 9000 bf16 keys: a deviation of 0.026, a bound of 0.0035
        if 64 < n <= 64 / (4 * torch.finfo(dtype).eps):          # 64 keys weigh at least 8 u (bf16: up to 2048 keys)
            cut = np.r_[0:n // 2, n // 2 + 64:n]
            less = p[cut] @ v[cut] / p[cut].sum()
            assert np.mean(np.abs(less - ref) > tol) > 0.1
        ref, _, p, pv, size = SO.decode_head(row, k, np.abs(v), np.arange(n), D ** -0.5)
        tol = o_bound(ref, pv, size, dtype, np.abs(v).sum(0))
        assert np.mean(np.abs(8 * torch.finfo(dtype).eps * ref) > tol) > 0.9
