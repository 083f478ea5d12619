"""The 8-bit state cache on the GPU.  Codes and scales are functions of the values alone (two IEEE fp32
divisions and a rounding), so they are held to equality with the same two divisions in numpy."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


def kda():
    import gated_delta_rule_83_b200 as m
    return m


def reference(S):
    """Codes and scales of fp32 states [.., dv]; rows with an infinity or NaN: codes 0, scale NaN."""
    S = S.astype(np.float32)
    with np.errstate(all="ignore"):
        scale = (np.abs(S).max(-1) / np.float32(127.0)).astype(np.float32)
        ok = np.isfinite(S).all(-1)
        step = np.where(ok & (scale > 0), scale, np.float32(1.0))[..., None].astype(np.float32)
        code = np.clip(np.rint((S / step).astype(np.float32)), -127, 127)
        code = np.where((ok & (scale > 0))[..., None], code, 0)
    return code.astype(np.int8), np.where(ok, scale, np.float32(np.nan)).astype(np.float32)


def states(seed, N, H, dk, dv):
    g = torch.Generator().manual_seed(seed)
    S = torch.randn(N, H, dk, dv, generator=g) * torch.exp(2 * torch.randn(N, H, dk, 1, generator=g))
    S[0, 0, 0] = 0.0                       # a row of zeros
    S[0, 0, 1] = 0.0
    S[0, 0, 1, 3] = -2.5                   # one value alone
    S[0, 0, 2] *= 1e-42 / S[0, 0, 2].abs().max()   # denormal values: the scale itself is denormal or zero
    S[0, 0, 3] = torch.where(torch.arange(dv) % 2 == 0, 127.0, 0.5)  # ties
    S[0, 0, 4] *= 3e38 / S[0, 0, 4].abs().max()    # near the largest finite value, or past it
    return S


@pytest.mark.parametrize("N,num,H,dk,dv", [(1, 1, 1, 64, 64), (3, 5, 2, 64, 128), (2, 2, 5, 128, 64), (7, 40, 3, 128, 128)])
def test_write_then_read(N, num, H, dk, dv):
    m = kda()
    S = states(1, N, H, dk, dv)
    code, sc = reference(S.numpy())
    cache = torch.full((num, H, dk, dv), 99, dtype=torch.int8, device=DEV)
    scale = torch.full((num, H, dk), 5.0, device=DEV)
    at = torch.randperm(num, generator=torch.Generator().manual_seed(2))[:N].to(torch.int32)
    m.state_cache_write(S.to(DEV), cache, scale, at.to(DEV))
    m.check()
    assert np.array_equal(cache.cpu().numpy()[at.numpy()], code)
    assert np.array_equal(scale.cpu().numpy()[at.numpy()], sc, equal_nan=True)
    rest = np.setdiff1d(np.arange(num), at.numpy())
    assert (cache.cpu().numpy()[rest] == 99).all() and (scale.cpu().numpy()[rest] == 5.0).all()
    back = m.state_cache_read(cache, scale, at.to(DEV))
    m.check()
    want = code.astype(np.float32) * sc[..., None]
    assert np.array_equal(back.cpu().numpy(), want, equal_nan=True)
    # a value of a normal scale comes back within half a step; the products' roundings add 2^-22 of the row's largest
    err = np.abs(want.astype(np.float64) - S.numpy())
    normal = sc > 1e-36
    assert (err <= (0.5 + 127 * 2.0 ** -22) * sc[..., None])[normal].all()


def test_infinite_and_nan_rows_read_back_as_nan():
    m = kda()
    S = states(3, 2, 2, 64, 64)
    S[1, 1, 7, 9] = float("inf")
    S[1, 0, 8, 1] = float("nan")
    S[1, 0, 9, 0] = -float("inf")
    S[1, 0, 9, 1] = float("nan")
    cache = torch.zeros(2, 2, 64, 64, dtype=torch.int8, device=DEV)
    scale = torch.zeros(2, 2, 64, device=DEV)
    at = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    m.state_cache_write(S.to(DEV), cache, scale, at)
    code, sc = reference(S.numpy())
    assert np.array_equal(cache.cpu().numpy(), code) and np.array_equal(scale.cpu().numpy(), sc, equal_nan=True)
    back = m.state_cache_read(cache, scale, at).cpu()
    for h, r in ((1, 7), (0, 8), (0, 9)):
        assert torch.isnan(back[1, h, r]).all()
    assert torch.isfinite(back[0]).all()


def test_slots_none_past_the_end_and_twice():
    m = kda()
    S = states(4, 6, 2, 128, 128)
    cache = torch.full((4, 2, 128, 128), 9, dtype=torch.int8, device=DEV)
    scale = torch.full((4, 2, 128), 3.0, device=DEV)
    at = torch.tensor([2, -1, 0, 2, 4, 2], dtype=torch.int32, device=DEV)
    m.state_cache_write(S.to(DEV), cache, scale, at)
    with pytest.raises(m.KdaError) as e:
        m.check()  # slot 4 of 4
    assert e.value.code == 1
    code, sc = reference(S.numpy())
    assert np.array_equal(cache.cpu().numpy()[2], code[5]) and np.array_equal(scale.cpu().numpy()[2], sc[5])
    assert np.array_equal(cache.cpu().numpy()[0], code[2])
    assert (cache[1] == 9).all() and (cache[3] == 9).all() and (scale[3] == 3.0).all()
    out = torch.full((4, 2, 128, 128), 7.0, device=DEV)
    got = m.state_cache_read(cache, scale, torch.tensor([0, -1, 7, 0], dtype=torch.int32, device=DEV), out=out)
    assert got is out
    with pytest.raises(m.KdaError):
        m.check()
    assert torch.equal(out[0], out[3]) and (out[1] == 0).all() and (out[2] == 0).all()
    assert np.array_equal(out[0].cpu().numpy(), code[2].astype(np.float32) * sc[2][..., None])


def test_nothing_to_do_and_refusals():
    m = kda()
    cache = torch.zeros(2, 2, 64, 128, dtype=torch.int8, device=DEV)
    scale = torch.zeros(2, 2, 64, device=DEV)
    none = torch.zeros(0, dtype=torch.int32, device=DEV)
    m.state_cache_write(torch.zeros(0, 2, 64, 128, device=DEV), cache, scale, none)
    assert m.state_cache_read(cache, scale, none).shape == (0, 2, 64, 128)
    one = torch.zeros(1, dtype=torch.int32, device=DEV)
    S = torch.zeros(1, 2, 64, 128, device=DEV)
    for args, err in (((S.bfloat16(), cache, scale, one), TypeError), ((S, cache.float(), scale, one), TypeError),
                      ((S, cache, scale[:1].contiguous(), one), ValueError), ((S, cache, scale, one.long()), TypeError),
                      ((S[:, :1].contiguous(), cache, scale, one), ValueError),
                      ((S, cache, scale, torch.zeros(2, dtype=torch.int32, device=DEV)), ValueError),
                      ((S, cache.transpose(2, 3), scale, one), ValueError)):
        with pytest.raises(err):
            m.state_cache_write(*args)
    m.check()


@pytest.mark.parametrize("kind", ["head", "channel"])
def test_a_request_put_aside_and_resumed(kind):
    """Prefill, store, restore, decode and prefill again, for both gate forms: the outputs after the
    restore are those of the run on the values that the cache stands for, bit for bit."""
    m = kda()
    g = torch.Generator().manual_seed(6)
    N, T, H, d = 3, 90, 2, 128
    unit = torch.nn.functional.normalize

    def tokens(*lead):
        gate = (*lead, H) if kind == "head" else (*lead, H, d)
        x = dict(q=unit(torch.randn(*lead, H, d, generator=g), dim=-1).bfloat16(),
                 k=unit(torch.randn(*lead, H, d, generator=g), dim=-1).bfloat16(),
                 v=torch.randn(*lead, H, d, generator=g).bfloat16(),
                 log_alpha=torch.nn.functional.logsigmoid(torch.randn(gate, generator=g) + 3),
                 beta=torch.sigmoid(torch.randn(*lead, H, generator=g)))
        return {k: v.to(DEV) for k, v in x.items()}

    fwd = m.gdn_chunk_fwd if kind == "head" else m.chunk_fwd
    step = m.gdn_decode_step if kind == "head" else m.decode_step
    _, S = fwd(**tokens(N, T))
    cache = torch.zeros(8, H, d, d, dtype=torch.int8, device=DEV)
    scale = torch.zeros(8, H, d, device=DEV)
    at = torch.tensor([5, 0, 3], dtype=torch.int32, device=DEV)
    m.state_cache_write(S, cache, scale, at)
    code, sc = reference(S.cpu().numpy())
    held = torch.from_numpy(code.astype(np.float32) * sc[..., None]).to(DEV)
    one, more = tokens(N), tokens(N, T)
    want = held.clone()
    o1 = step(*one.values(), want)
    o2, want = fwd(**more, S0=want)
    got = m.state_cache_read(cache, scale, at)
    p1 = step(*one.values(), got)
    p2, got = fwd(**more, S0=got)
    m.check()
    assert torch.equal(o1, p1) and torch.equal(o2, p2) and torch.equal(want, got)
