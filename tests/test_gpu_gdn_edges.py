"""Edges of the scalar-gate delta rule on the GPU, against the fp64 oracle of the recurrence.  Inputs, reference
and tolerances (2^-15 of a result's norm for fp32 inputs, 2^-13 for bf16 ones, 2^-8 more for a result in bf16) are
those of test_gpu_gdn."""
import pytest
import torch

from tests.test_gpu_gdn import DEV, check, kda, make, ref_bwd, ref_fwd, rel, run_bwd, run_fwd

pytestmark = pytest.mark.gpu
BOTH = [torch.bfloat16, torch.float32]
GRADS = ("dq", "dk", "dv", "dlog_alpha", "dbeta", "dS0")


@pytest.mark.parametrize("dt,dk,dv", [(torch.bfloat16, 128, 128), (torch.float32, 128, 128), (torch.float32, 64, 128)])
@pytest.mark.parametrize("every", [2, 3, 4])
@pytest.mark.parametrize("gate", [-100.0, float("-inf")])
def test_resets_through_a_chunk(dt, dk, dv, every, gate):
    """A token that forgets all every few tokens, as in short documents packed into one sequence: the cumulative gate
    reaches thousands, and the decays e^-0.02 between the tokens in between are small differences of it.  Keys are
    alike, so that these decays carry the results, and the last eight tokens of the chunks, where the sums are
    largest, are held to the tolerance by themselves."""
    d = make(43, dt, 2, 1, dk, dv, T=192, corr=1.0)
    d["log_alpha"].fill_(-0.02)
    d["log_alpha"][:, ::every] = gate
    late = torch.arange(192, device=DEV).view(-1, 64)[:, 56:].flatten()
    (out, S), (o_ref, s_ref) = run_fwd(d), ref_fwd(d)
    check(S, s_ref, dt, "S")
    check(out, o_ref, dt, "out")
    at = late.cpu().numpy()
    check(out[:, late], o_ref[:, at], dt, "out, late tokens")
    g, ref = run_bwd(d), ref_bwd(d)
    for x in GRADS:
        check(g[x], ref[x], dt, x)
    for x in GRADS[:-1]:
        check(g[x][:, late], ref[x][:, at], dt, x + ", late tokens")


@pytest.mark.parametrize("dt", BOTH)
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 128)])
@pytest.mark.parametrize("kw", [dict(T=2, B=3), dict(T=64, B=2), dict(T=130, B=2), dict(lens=[2, 0, 64, 1, 130, 65])])
def test_the_first_gate_has_no_gradient_without_a_start_state(dt, dk, dv, kw):
    """It multiplies zeros, whatever follows: exactly zero; the other gates' gradients are right."""
    d = make(44, dt, 4, 2, dk, dv, s0=False, **kw)
    g, ref = run_bwd(d), ref_bwd(d)
    check(g["dlog_alpha"], ref["dlog_alpha"], dt, "dlog_alpha")
    if "lens" in kw:
        first = [int(t) for t, n in zip(d["cu"][:-1].tolist(), kw["lens"]) if n]
    else:
        first = [0]
    assert not g["dlog_alpha"][:, first].any()
    if d["q"].shape[1] > 2:
        assert g["dlog_alpha"].any()


def _untouched(call, like):
    """A call with malformed offsets and all gradients given: none is written and the fault is reported."""
    m = kda()
    mine = {x: torch.full_like(y, 3.0) for x, y in like.items()}
    call(mine)
    with pytest.raises(m.KdaError) as e:
        m.check()
    assert e.value.code == 6
    for x, y in mine.items():
        assert (y == 3.0).all(), x


@pytest.mark.parametrize("dt", BOTH)
@pytest.mark.parametrize("dk", [64, 128])
def test_bad_offsets_leave_every_gradient(dt, dk):
    d = make(41, dt, 4, 2, dk, dk, lens=[30, 30, 40])
    d["cu"] = torch.tensor([0, 50, 40, 100], dtype=torch.int32, device=DEV)
    _untouched(lambda mine: kda().gdn_chunk_bwd(d["q"], d["k"], d["v"], d["log_alpha"], d["beta"], d["dout"],
                                                S0=d["S0"], cu_seqlens=d["cu"], grads=mine),
               {"dq": d["q"], "dk": d["k"], "dv": d["v"], "dlog_alpha": d["log_alpha"], "dbeta": d["beta"],
                "dS0": d["S0"]})


@pytest.mark.parametrize("dt", BOTH)
@pytest.mark.parametrize("prologue", [0, "all"])
def test_bad_offsets_leave_every_gradient_of_channel_gates(dt, prologue):
    """The form with a gate a key channel: shared heads and the input prologue add passes behind the chunks'."""
    m = kda()
    d = make(42, dt, 4, 2, 128, 128, lens=[30, 30, 40])
    la = torch.randn(1, 100, 4, 128, device=DEV, generator=torch.Generator(DEV).manual_seed(1))
    pro = 0
    if prologue:
        pro = m.PROLOGUE_L2NORM_QK | m.PROLOGUE_GATE_LOGITS | m.PROLOGUE_BETA_LOGITS
    d["cu"] = torch.tensor([0, 50, 40, 100], dtype=torch.int32, device=DEV)
    _untouched(lambda mine: m.chunk_bwd(d["q"], d["k"], d["v"], la if prologue else -la.abs(), d["beta"], d["dout"],
                                        S0=d["S0"], cu_seqlens=d["cu"], grads=mine, prologue=pro),
               {"dq": d["q"], "dk": d["k"], "dv": d["v"], "dlog_alpha": la, "dbeta": d["beta"], "dS0": d["S0"]})


@pytest.mark.parametrize("dt", BOTH)
def test_scalars_may_start_at_any_element(dt):
    """log_alpha, beta and their gradients lie one element into a buffer, as a slice of a larger tensor does."""
    d = make(40, dt, 3, 1, 64, 128, lens=[70, 1, 20])
    want = (run_fwd(d), run_bwd(d))

    def behind(x):
        y = torch.empty(x.numel() + 1, device=DEV)[1:].view(x.shape)
        return y.copy_(x)

    e = dict(d, log_alpha=behind(d["log_alpha"]), beta=behind(d["beta"]))
    mine = {x: behind(torch.zeros_like(d["beta"])) for x in ("dlog_alpha", "dbeta")}
    out, S = run_fwd(e)
    g = run_bwd(e, grads=mine)
    assert torch.equal(out, want[0][0]) and torch.equal(S, want[0][1])
    assert g["dbeta"] is mine["dbeta"] and g["dlog_alpha"] is mine["dlog_alpha"]
    assert all(torch.equal(g[x], want[1][x]) for x in GRADS)


def launched(call):
    """The call's result and the names of the kernels it launched."""
    m = kda()
    m.profile_begin()
    try:
        got = call()
    finally:
        names = set(m.profile_end())
    m.check()
    return got, names


# lengths, heads, q/k heads, dk, dv, start state
CUT = [
    dict(lens=[6000, 10, 0, 3000, 0], H=1, Hk=1, dk=128, dv=128),
    dict(lens=[0, 6000, 0, 70, 5100, 1], H=2, Hk=1, dk=128, dv=128),
    dict(lens=[2049, 64, 0, 5000], H=2, Hk=2, dk=64, dv=128, s0=False),
    dict(lens=[63] * 14 + [0] * 10 + [50000] + [1] * 8 + [46000, 130], H=1, Hk=1, dk=64, dv=64),
    dict(lens=[5000], H=2, Hk=2, dk=128, dv=64),
    dict(T=3300, B=2, H=2, Hk=1, dk=128, dv=128),
    dict(T=4097, B=3, H=1, Hk=1, dk=64, dv=64, s0=False),
    dict(T=2900, B=2, H=1, Hk=1, dk=64, dv=128),
]


@pytest.mark.parametrize("case", CUT, ids=[",".join(f"{k}={v}" for k, v in c.items())[:90] for c in CUT])
def test_sequences_cut_into_segments(case):
    """Packed sequences and batches that are cut, forward and backward; the state passed in place too.  Each call's
    launches show that it was: the ends of the segments and the join are kernels of their own.

    Gates of 1e-4 a token and small beta, so that a segment's start state still weighs e^-0.5 at its end: a token takes
    beta / dk off the state, at beta = 0.1 and dk = 128 a chunk 0.05 and the gates 0.01, a memory of 1 / 0.06 = 17
    chunks.  The errors of so many chunks may add where their parts of the result add as squares: sqrt(17) < 2^2.1 of
    the tolerance of one chunk, 2^-13, so 2^-10.9."""
    c = dict(case)
    d = make(45, torch.bfloat16, c.pop("H"), c.pop("Hk"), c.pop("dk"), c.pop("dv"), gate=9.0, **c)
    d["beta"] *= 0.2

    def check(got, want, name):
        tol = 2.0 ** -10.9 + (2.0 ** -8 if got.dtype == torch.bfloat16 else 0.0)
        assert rel(got, want) <= tol, f"{name}: {rel(got, want):.3e} > {tol:.3e}"

    (out, S), names = launched(lambda: run_fwd(d))
    assert {"gdn_ends", "gdn_join", "gdn_chain"} <= names
    o_ref, s_ref = ref_fwd(d)
    check(out, o_ref, "out")
    check(S, s_ref, "S")
    if d["S0"] is not None:
        mine = d["S0"].clone()
        m = kda()
        out2, S2 = m.gdn_chunk_fwd(d["q"], d["k"], d["v"], d["log_alpha"], d["beta"], S0=mine, S_final=mine,
                                   cu_seqlens=d["cu"])
        m.check()
        assert S2 is mine and torch.equal(out, out2) and torch.equal(S, mine)
    g, names = launched(lambda: run_bwd(d))
    assert {"gdn_bwd_ends", "gdn_join", "gdn_bwd_chains"} <= names
    ref = ref_bwd(d)
    for x in GRADS:
        check(g[x], ref[x], x)
    # each sequence's own state and its cotangent, as the norm over all hides a short one
    for n in range(S.shape[0]):
        check(S[n], s_ref[n], f"S[{n}]")
        check(g["dS0"][n], ref["dS0"][n], f"dS0[{n}]")
