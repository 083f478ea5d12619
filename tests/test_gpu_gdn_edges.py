"""Edges of the scalar-gate delta rule on the GPU, against the fp64 oracle of the recurrence.  Inputs, reference
and tolerances (2^-15 of a result's norm for fp32 inputs, 2^-13 for bf16 ones, 2^-8 more for a result in bf16) are
those of test_gpu_gdn."""
import pytest
import torch

from tests.test_gpu_gdn import DEV, check, make, ref_bwd, ref_fwd, run_bwd, run_fwd

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
