"""Refusals of the scalar-gate delta rule's and the state cache's entry points, without a GPU: every
call below fails its checks before a pointer is used or a kernel launched."""
import ctypes

import pytest
import torch

FAKE = 0x100000  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    from gated_delta_rule_83_b200 import build, kda
    build.build()
    return kda.load_library()


def fwd(lib, q=FAKE, la=FAKE, out=FAKE, cu=None, n=0, B=1, T=64, H=2, Hk=2, dk=128, dv=128, dt=0, ws=FAKE, size=1 << 40):
    return lib.kda_gdn_chunk_fwd(q, FAKE, FAKE, la, FAKE, None, cu, n, out, None, B, T, H, Hk, dk, dv, dt, ws, size, None)


def bwd(lib, dout=FAKE, dq=FAKE, dla=FAKE, cu=None, n=0, B=1, T=64, H=2, Hk=2, dk=128, dv=128, dt=0, ws=FAKE,
        size=1 << 40):
    return lib.kda_gdn_chunk_bwd(FAKE, FAKE, FAKE, FAKE, FAKE, None, cu, n, dout, None, dq, FAKE, FAKE, dla, FAKE, None,
                                 B, T, H, Hk, dk, dv, dt, ws, size, None)


@pytest.mark.parametrize("call", [fwd, bwd])
@pytest.mark.parametrize("kw,want", [
    (dict(Hk=0), 1), (dict(Hk=-1), 1), (dict(H=3, Hk=2), 1), (dict(H=2, Hk=4), 1), (dict(H=0, Hk=1), 1),
    (dict(dt=2), 1), (dict(T=-1), 1), (dict(B=0), 1),
    (dict(dk=96), 2), (dict(dv=256), 2), (dict(H=70000, Hk=70000), 2),
    (dict(cu=FAKE, n=0), 1), (dict(cu=FAKE, n=2, B=2), 1), (dict(cu=FAKE + 2, n=1), 1),
    (dict(ws=None), 5), (dict(ws=FAKE + 16), 5), (dict(size=64), 5),
])
def test_chunk_calls_refuse(lib, call, kw, want):
    assert call(lib, **kw) == want


def test_chunk_calls_refuse_missing_and_misaligned_tensors(lib):
    assert fwd(lib, q=None) == 1 and fwd(lib, q=FAKE + 8) == 1 and fwd(lib, la=FAKE + 2) == 1 and fwd(lib, out=None) == 1
    assert bwd(lib, dout=None) == 1 and bwd(lib, dq=FAKE + 4) == 1 and bwd(lib, dla=None) == 1 and bwd(lib, dla=FAKE + 1) == 1


def test_workspace_sizes_grow_with_the_problem(lib):
    n = ctypes.c_size_t(0)

    def size(fn, *a):
        assert getattr(lib, fn)(*a, ctypes.byref(n)) == 0
        return n.value

    f, b = "kda_gdn_chunk_fwd_workspace_size", "kda_gdn_chunk_bwd_workspace_size"
    for dt in (0, 1):
        assert 0 < size(f, 1, 0, 2, 128, 128, 0, 0, dt) < size(f, 1, 64, 2, 128, 128, 0, 0, dt) \
            < size(f, 1, 640, 2, 128, 128, 0, 0, dt)
        assert 0 < size(b, 1, 0, 2, 1, 128, 128, 0, 0, dt) < size(b, 1, 640, 2, 1, 128, 128, 0, 0, dt)
    assert size(f, 1, 640, 2, 128, 128, 1, 9, 0) >= size(f, 1, 640, 2, 128, 128, 1, 1, 0)
    assert lib.kda_gdn_chunk_bwd_workspace_size(1, 64, 3, 2, 128, 128, 0, 0, 0, ctypes.byref(n)) == 1
    assert lib.kda_gdn_chunk_fwd_workspace_size(1, 64, 2, 32, 128, 0, 0, 0, ctypes.byref(n)) == 2
    assert lib.kda_gdn_chunk_fwd_workspace_size(1, 64, 2, 128, 128, 0, 0, 0, None) == 1


def test_decode_refuses(lib):
    def step(q=FAKE, S=FAKE, N=2, H=4, Hk=2, dk=128, dv=128, dt=0):
        return lib.kda_gdn_decode_step(q, FAKE, FAKE, FAKE, FAKE, S, FAKE, N, H, Hk, dk, dv, dt, None)

    assert step(q=None) == 1 and step(S=FAKE + 4) == 1 and step(Hk=3) == 1 and step(Hk=0) == 1 and step(dt=9) == 1
    assert step(N=-1) == 1 and step(dk=48) == 2
    assert step(q=None, N=0) == 0  # no sequences: nothing is touched


def test_state_cache_refuses(lib):
    def write(S=FAKE, cache=FAKE, scale=FAKE, slots=FAKE, N=2, num=4, H=2, dk=128, dv=128):
        return lib.kda_state_cache_write(S, cache, scale, slots, N, num, H, dk, dv, None)

    def read(S=FAKE, cache=FAKE, scale=FAKE, slots=FAKE, N=2, num=4, H=2, dk=128, dv=128):
        return lib.kda_state_cache_read(cache, scale, slots, S, N, num, H, dk, dv, None)

    for call in (write, read):
        assert call(S=None) == 1 and call(cache=None) == 1 and call(scale=None) == 1 and call(slots=None) == 1
        assert call(S=FAKE + 8) == 1 and call(cache=FAKE + 4) == 1 and call(slots=FAKE + 2) == 1
        assert call(N=-1) == 1 and call(num=-1) == 1 and call(H=0) == 1 and call(dv=32) == 2 and call(H=1 << 20) == 2
        assert call(S=None, slots=None, N=0) == 0


def test_binding_refuses_host_tensors_and_wrong_kinds():
    import gated_delta_rule_83_b200 as kda
    x = torch.zeros(1, 4, 2, 64)
    b = torch.zeros(1, 4, 2)
    with pytest.raises(ValueError, match="CUDA tensor"):
        kda.gdn_chunk_fwd(x, x, x, b, b)
    with pytest.raises(ValueError, match="CUDA tensor"):
        kda.gdn_chunk_bwd(x, x, x, b, b, x)
    with pytest.raises(TypeError, match="must be a torch.Tensor"):
        kda.gdn_decode_step(None, x, x, b, b, x)
    c, s, i = torch.zeros(2, 2, 64, 64, dtype=torch.int8), torch.zeros(2, 2, 64), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        kda.state_cache_write(torch.zeros(1, 2, 64, 64), c, s, i)
    with pytest.raises(ValueError, match="CUDA tensor"):
        kda.state_cache_read(c, s, i)
