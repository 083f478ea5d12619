"""GPU parity of the scalar-gate delta rule against the fp64 oracle of the recurrence, whose gate for each
key channel is given the head's gate in every channel.

Tolerances.  An output rounded to bf16 is off by at most 2^-8 of its value; one in fp32 carries the
products' error alone.  With fp32 inputs that is the rounding of sums of up to 128 terms, at most
128 * 2^-24 = 2^-17 of the operands' norms for each of four dependent products in a chunk: 2^-15 of the
result's norm.  With bf16 inputs the tensor-core products split each fp32 operand into two bf16 parts:
the split leaves 2^-17 of each operand and the dropped low-by-low product 2^-16, so at most 2^-15 a
product and 2^-13 for four.  (Chunks further back weigh less by the gates' decay.)  The reference is
evaluated on the very inputs."""
import numpy as np
import pytest
import torch

import oracle
from tests.kda_testutil import np64

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32_TOL = {torch.float32: 2.0 ** -15, torch.bfloat16: 2.0 ** -13}


def kda():
    import gated_delta_rule_83_b200 as m
    return m


def make(seed, dtype, H, Hk, dk, dv, T=None, B=1, lens=None, s0=True, gate=3.0, corr=0.0, qk_scale=1.0):
    """Inputs on the GPU: q/k of unit length, gates log sigmoid(N(gate, 1)), beta sigmoid(N(0, 1))."""
    g = torch.Generator().manual_seed(seed)
    cu = None
    if lens is not None:
        B, T = 1, sum(lens)
        cu = torch.tensor(np.cumsum([0] + list(lens)), dtype=torch.int32, device=DEV)
    N = B if lens is None else len(lens)

    def rnd(*s):
        return torch.randn(s, generator=g)

    d = {"q": torch.nn.functional.normalize(rnd(B, T, Hk, dk) + corr, dim=-1) * qk_scale,
         "k": torch.nn.functional.normalize(rnd(B, T, Hk, dk) + corr, dim=-1) * qk_scale, "v": rnd(B, T, H, dv),
         "dout": rnd(B, T, H, dv)}
    d = {x: y.to(dtype).to(DEV) for x, y in d.items()}
    d["log_alpha"] = torch.nn.functional.logsigmoid(rnd(B, T, H) + gate).to(DEV)
    d["beta"] = torch.sigmoid(rnd(B, T, H)).to(DEV)
    d["S0"] = (rnd(N, H, dk, dv) * 0.2).to(DEV) if s0 else None
    d["dS_final"] = (rnd(N, H, dk, dv) * 0.3).to(DEV)
    d["cu"] = cu
    return d


def _oracle_args(d):
    H, dk = d["v"].shape[2], d["q"].shape[-1]
    q, k, v, b = (np64(d[x]) for x in ("q", "k", "v", "beta"))
    G = H // q.shape[2]
    la = np.repeat(np64(d["log_alpha"])[..., None], dk, axis=-1)
    args = [np.repeat(q, G, axis=2), np.repeat(k, G, axis=2), v, la, b]
    S0 = None if d["S0"] is None else np64(d["S0"])
    if d["cu"] is not None:
        return [a[0] for a in args], S0, d["cu"].cpu().numpy().astype(np.int64)
    return args, S0, None


def ref_fwd(d):
    args, S0, cu = _oracle_args(d)
    kw = {} if cu is None else {"cu_seqlens": cu}
    out, S = oracle.seq(*args, S0=S0, **kw)
    return (out if cu is None else out[None]), S


def ref_bwd(d, dsf=True):
    args, S0, cu = _oracle_args(d)
    do = np64(d["dout"])
    kw = {} if cu is None else {"cu_seqlens": cu}
    g = oracle.bwd(*args, do if cu is None else do[0], S0=S0, dS_final=np64(d["dS_final"]) if dsf else None, **kw)
    if cu is not None:
        for x in ("dq", "dk", "dv", "dlog_alpha", "dbeta"):
            g[x] = g[x][None]
    g["dlog_alpha"] = g["dlog_alpha"].sum(-1)
    Hk, H = d["q"].shape[2], d["v"].shape[2]
    for x in ("dq", "dk"):
        g[x] = g[x].reshape(*g[x].shape[:2], Hk, H // Hk, -1).sum(3)
    return g


def rel(a, b):
    b = np.asarray(b, np.float64)
    return float(np.linalg.norm(np64(a) - b) / max(np.linalg.norm(b), 1e-30))


def check(got, want, dtype, name):
    """A tensor in fp32: the products' error.  One in bf16: its rounding on top."""
    tol = F32_TOL[dtype] + (2.0 ** -8 if got.dtype == torch.bfloat16 else 0.0)
    assert tuple(got.shape) == tuple(want.shape), name
    assert rel(got, want) <= tol, f"{name}: {rel(got, want):.3e} > {tol:.3e}"


def run_fwd(d, **kw):
    m = kda()
    out, S = m.gdn_chunk_fwd(d["q"], d["k"], d["v"], d["log_alpha"], d["beta"], S0=d["S0"], cu_seqlens=d["cu"], **kw)
    m.check()
    return out, S


def run_bwd(d, dsf=True, **kw):
    m = kda()
    g = m.gdn_chunk_bwd(d["q"], d["k"], d["v"], d["log_alpha"], d["beta"], d["dout"], S0=d["S0"],
                        dS_final=d["dS_final"] if dsf else None, cu_seqlens=d["cu"], **kw)
    m.check()
    return g


# dtype, H, Hk, dk, dv, extra
SHAPES = [
    ("bf16", 2, 2, 128, 128, dict(T=200)),
    ("bf16", 2, 2, 128, 128, dict(T=64, s0=False)),
    ("bf16", 3, 1, 128, 128, dict(T=1, B=2)),
    ("bf16", 4, 2, 128, 128, dict(T=129, B=3)),
    ("bf16", 1, 1, 128, 128, dict(T=1500)),
    ("bf16", 4, 2, 128, 128, dict(lens=[1, 0, 64, 65, 190, 63])),
    ("bf16", 2, 2, 128, 128, dict(lens=[0, 0, 3], s0=False)),
    ("bf16", 2, 1, 128, 128, dict(T=300, gate=0.0)),
    ("bf16", 2, 2, 128, 128, dict(T=300, gate=9.0)),
    ("bf16", 2, 2, 128, 128, dict(T=260, corr=0.3)),
    ("bf16", 1, 1, 128, 128, dict(lens=[700, 0, 1333, 64, 1, 2100])),
    ("bf16", 2, 1, 64, 128, dict(lens=[900, 30, 1500])),
    ("bf16", 3, 3, 128, 64, dict(T=2065)),
    ("bf16", 2, 2, 64, 64, dict(T=700, B=2, s0=False)),
    ("fp32", 2, 2, 128, 128, dict(T=200)),
    ("fp32", 2, 1, 64, 64, dict(T=256)),
    ("fp32", 2, 2, 64, 128, dict(lens=[70, 0, 1, 128])),
    ("bf16", 2, 1, 64, 64, dict(T=130, B=2)),
    ("bf16", 2, 2, 128, 64, dict(T=65)),
    ("bf16", 2, 2, 64, 128, dict(T=127, s0=False)),
]
IDS = [f"{a[0]}-H{a[1]}/{a[2]}-{a[3]}x{a[4]}-" + ",".join(f"{k}={v}" for k, v in a[5].items()) for a in SHAPES]


def dtype_of(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_prefill_matches_the_recurrence(shape):
    dt = dtype_of(shape[0])
    d = make(1, dt, *shape[1:5], **shape[5])
    out, S = run_fwd(d)
    o_ref, s_ref = ref_fwd(d)
    check(out, o_ref, dt, "out")
    check(S, s_ref, dt, "S_final")


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_backward_matches_the_derivative(shape):
    dt = dtype_of(shape[0])
    d = make(2, dt, *shape[1:5], **shape[5])
    g, ref = run_bwd(d), ref_bwd(d)
    for x in ("dq", "dk", "dv", "dlog_alpha", "dbeta", "dS0"):
        check(g[x], ref[x], dt, x)


def test_backward_options():
    """No cotangent of the final state, no dS0 wanted, gradients into the caller's tensors."""
    d = make(3, torch.bfloat16, 2, 2, 128, 128, T=100)
    ref = ref_bwd(d, dsf=False)
    mine = {"dq": torch.full_like(d["q"], 7.0), "dlog_alpha": torch.full_like(d["log_alpha"], 7.0)}
    g = run_bwd(d, dsf=False, want_dS0=False, grads=mine)
    assert g["dS0"] is None and g["dq"].data_ptr() == mine["dq"].data_ptr()
    for x in ("dq", "dk", "dv", "dlog_alpha", "dbeta"):
        check(g[x], ref[x], torch.bfloat16, x)


@pytest.mark.parametrize("dt,dk", [(torch.bfloat16, 128), (torch.float32, 64)])
def test_backward_against_differences(dt, dk):
    """dlog_alpha, dbeta and dS0 against central differences of the library's own forward, whose fp32
    loss terms are summed in 64 bits.  With a step of h the difference carries the forward's error / h
    (2^-8 outputs rounded to bf16 average out over the 2 * 96 * dv terms) and h^2 of the third derivative;
    both stay under 2 % of the directional derivative at h = 0.05 along a direction of unit size."""
    d = make(4, dt, 2, 1, dk, dk, T=96, corr=0.1)
    g = run_bwd(d)

    def loss(**over):
        e = dict(d, **over)
        out, S = run_fwd(e)
        return float((out.double() * d["dout"].double()).sum() + (S.double() * d["dS_final"].double()).sum())

    for x, key in (("log_alpha", "dlog_alpha"), ("beta", "dbeta"), ("S0", "dS0")):
        # along the gradient itself, so that the derivative is as large as it can be
        u = g[key] / g[key].norm()
        h = 0.05
        num = (loss(**{x: d[x] + h * u}) - loss(**{x: d[x] - h * u})) / (2 * h)
        ana = float(g[key].double().norm())
        assert abs(num - ana) <= 0.02 * abs(ana), (x, num, ana)


@pytest.mark.parametrize("dt,H,Hk,dk,dv,N", [(torch.bfloat16, 4, 2, 128, 128, 3), (torch.float32, 3, 3, 64, 128, 5),
                                             (torch.bfloat16, 5, 1, 64, 64, 1), (torch.float32, 2, 1, 128, 64, 2)])
def test_decode_matches_the_recurrence(dt, H, Hk, dk, dv, N):
    """Eight steps: the decode step is fp32 whatever the inputs' type, so its state has fp32 rounding alone
    (8 steps of sums of dk <= 128 terms: 2^-14 at worst)."""
    m = kda()
    d = make(6, dt, H, Hk, dk, dv, T=8, B=N)
    o_ref, s_ref = ref_fwd(d)
    S = d["S0"].clone()
    outs = [m.gdn_decode_step(*(d[x][:, t].contiguous() for x in ("q", "k", "v", "log_alpha", "beta")), S)
            for t in range(8)]
    m.check()
    out = torch.stack(outs, 1)
    assert rel(S, s_ref) <= 2.0 ** -14
    assert rel(out, o_ref) <= 2.0 ** -14 + (2.0 ** -8 if dt == torch.bfloat16 else 0.0)


@pytest.mark.parametrize("dt,d_", [(torch.bfloat16, 128), (torch.float32, 64)])
def test_prefill_in_pieces_then_decode(dt, d_):
    """A prompt in two calls with the state passed in place, then single tokens: the run of a server."""
    m = kda()
    d = make(7, dt, 4, 2, d_, d_, T=150, B=2)
    o_ref, s_ref = ref_fwd(d)
    S = d["S0"].clone()
    outs = []
    for a, b in ((0, 100), (100, 140)):
        part = {x: d[x][:, a:b].contiguous() for x in ("q", "k", "v", "log_alpha", "beta")}
        out, S1 = m.gdn_chunk_fwd(**part, S0=S, S_final=S)
        assert S1 is S
        outs.append(out)
    for t in range(140, 150):
        outs.append(m.gdn_decode_step(*(d[x][:, t].contiguous() for x in ("q", "k", "v", "log_alpha", "beta")),
                                      S)[:, None])
    m.check()
    check(torch.cat(outs, 1), o_ref, dt, "out")
    check(S, s_ref, dt, "S")


@pytest.mark.parametrize("dt,d_", [(torch.bfloat16, 128), (torch.float32, 64)])
def test_no_tokens(dt, d_):
    """T = 0: the state passes through, gradients of the state too."""
    d = make(8, dt, 2, 2, d_, d_, T=0, B=2)
    out, S = run_fwd(d)
    assert out.numel() == 0 and torch.equal(S, d["S0"])
    g = run_bwd(d)
    assert torch.equal(g["dS0"], d["dS_final"]) and g["dq"].numel() == 0
    m = kda()
    z = torch.zeros(0, 2, d_, device=DEV, dtype=dt)
    zs = torch.zeros(0, 2, device=DEV)
    assert m.gdn_decode_step(z, z, z, zs, zs, torch.zeros(0, 2, d_, d_, device=DEV)).shape == (0, 2, d_)


@pytest.mark.parametrize("dt,d_", [(torch.bfloat16, 128), (torch.float32, 64)])
def test_gate_extremes(dt, d_):
    """beta = 0 (the state only decays), beta = 1 with alpha = 1 (an overwrite) and log alpha = -40 a step
    (all before is forgotten): finite and right in forward and backward."""
    d = make(9, dt, 4, 4, d_, d_, T=140)
    d["beta"][:, :, 0] = 0.0
    d["beta"][:, :, 1] = 1.0
    d["log_alpha"][:, :, 1] = 0.0
    d["log_alpha"][:, :, 2] = -40.0
    out, S = run_fwd(d)
    o_ref, s_ref = ref_fwd(d)
    check(out, o_ref, dt, "out")
    check(S, s_ref, dt, "S")
    g, ref = run_bwd(d), ref_bwd(d)
    for x in ("dq", "dk", "dv", "dlog_alpha", "dbeta", "dS0"):
        assert torch.isfinite(g[x]).all(), x
        check(g[x], ref[x], dt, x)


@pytest.mark.parametrize("dt,d_", [(torch.bfloat16, 128), (torch.float32, 64)])
@pytest.mark.parametrize("gate", [-30.0, -100.0, float("-inf")])
def test_tokens_that_forget_all(dt, d_, gate):
    """A gate that is zero or nearly so inside a chunk, at its border and twice in one: what lies before has no
    weight, and the decays between the tokens behind keep their digits."""
    d = make(13, dt, 2, 2, d_, d_, T=300, gate=4.0)
    for t in (0, 5, 64, 70, 71, 191, 299):
        d["log_alpha"][:, t, 0] = gate
    out, S = run_fwd(d)
    o_ref, s_ref = ref_fwd(d)
    check(out, o_ref, dt, "out")
    check(S, s_ref, dt, "S")
    g, ref = run_bwd(d), ref_bwd(d)
    for x in ("dq", "dk", "dv", "dlog_alpha", "dbeta", "dS0"):
        check(g[x], ref[x], dt, x)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dk,dv,kw", [(128, 128, dict(lens=[1, 1, 0, 1, 1])), (64, 128, dict(T=1, B=3))])
def test_a_gate_on_a_zero_state_has_no_gradient(dt, dk, dv, kw):
    """Sequences of one token and no start state: log_alpha multiplies zeros, so its gradient is exactly
    zero; with a start state it is alpha <(I - beta k k^T) S0, dS> alone, small where S0 is."""
    d = make(31, dt, 4, 2, dk, dv, s0=False, **kw)
    assert not run_bwd(d)["dlog_alpha"].any()
    d = make(32, dt, 4, 2, dk, dv, **kw)
    d["S0"] *= 2.0 ** -7
    check(run_bwd(d)["dlog_alpha"], ref_bwd(d)["dlog_alpha"], dt, "dlog_alpha")


def test_sequences_do_not_see_their_neighbours():
    """Packed input in which one sequence holds NaN and infinities throughout, cotangents too: the others get
    the very numbers they get without it."""
    lens = [70, 100, 1, 63, 200]
    d = make(14, torch.bfloat16, 2, 1, 128, 128, lens=lens)
    a = (run_fwd(d), run_bwd(d))
    lo, hi = 70, 170
    for x, bad in (("q", float("nan")), ("k", float("inf")), ("v", float("nan")), ("dout", float("inf")),
                   ("log_alpha", float("nan")), ("beta", float("nan"))):
        d[x][:, lo:hi] = bad
    d["S0"][1] = float("nan")
    d["dS_final"][1] = float("inf")
    b = (run_fwd(d), run_bwd(d))
    rows = torch.cat([torch.arange(lo), torch.arange(hi, sum(lens))]).to(DEV)
    seqs = torch.tensor([0, 2, 3, 4], device=DEV)
    assert torch.equal(a[0][0][:, rows], b[0][0][:, rows]) and torch.equal(a[0][1][seqs], b[0][1][seqs])
    for x in ("dq", "dk", "dv", "dlog_alpha", "dbeta"):
        assert torch.equal(a[1][x][:, rows], b[1][x][:, rows]), x
    assert torch.equal(a[1]["dS0"][seqs], b[1]["dS0"][seqs])


@pytest.mark.parametrize("kw", [dict(T=4000, B=1), dict(lens=[3000, 10, 0, 1500])])
def test_long_sequences_in_place(kw):
    """Sequences long enough to be cut into segments, the state passed in place: as with a state of its own."""
    d = make(15, torch.bfloat16, 1, 1, 128, 128, **kw)
    out, S = run_fwd(d)
    mine = d["S0"].clone()
    m = kda()
    out2, S2 = m.gdn_chunk_fwd(d["q"], d["k"], d["v"], d["log_alpha"], d["beta"], S0=mine, S_final=mine,
                               cu_seqlens=d["cu"])
    m.check()
    assert S2 is mine and torch.equal(out, out2) and torch.equal(S, mine)
    o_ref, s_ref = ref_fwd(d)
    check(out, o_ref, torch.bfloat16, "out")
    check(S, s_ref, torch.bfloat16, "S")


def test_calls_repeat_bit_for_bit_and_leave_inputs():
    d = make(10, torch.bfloat16, 4, 2, 128, 128, lens=[100, 300, 7])
    before = {x: y.clone() for x, y in d.items() if y is not None}
    a, b = run_fwd(d), run_fwd(d)
    g, h = run_bwd(d), run_bwd(d)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert all(torch.equal(g[x], h[x]) for x in g)
    assert all(torch.equal(d[x], before[x]) for x in before)


def test_two_streams_and_a_captured_graph():
    """Calls on two streams at once and a replayed capture give what a lone call gives."""
    m = kda()
    d = [make(20 + i, torch.bfloat16, 4, 2, 128, 128, T=500) for i in range(2)]
    want = [(run_fwd(x), run_bwd(x)) for x in d]
    streams = [torch.cuda.Stream() for _ in d]
    got = []
    for x, s in zip(d, streams):
        s.wait_stream(torch.cuda.current_stream())
        got.append((m.gdn_chunk_fwd(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], S0=x["S0"], stream=s),
                    m.gdn_chunk_bwd(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], x["dout"], S0=x["S0"],
                                    dS_final=x["dS_final"], stream=s)))
    torch.cuda.synchronize()
    m.check()
    for (f, g), (f0, g0) in zip(got, want):
        assert torch.equal(f[0], f0[0]) and torch.equal(f[1], f0[1]) and all(torch.equal(g[k], g0[k]) for k in g)
    graphs, held = [], []
    static = {k: v.clone() for k, v in d[0].items() if v is not None}
    for _ in range(2):  # two graphs of the same calls: no buffer is shared between them
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            f = m.gdn_chunk_fwd(static["q"], static["k"], static["v"], static["log_alpha"], static["beta"],
                                S0=static["S0"])
            g = m.gdn_chunk_bwd(static["q"], static["k"], static["v"], static["log_alpha"], static["beta"],
                                static["dout"], S0=static["S0"], dS_final=static["dS_final"])
        graphs.append(graph)
        held.append((f, g))
    for k in static:
        static[k].copy_(d[1][k])
    for graph in graphs:
        graph.replay()
    torch.cuda.synchronize()
    m.check()
    for f, g in held:
        assert torch.equal(f[0], want[1][0][0]) and torch.equal(f[1], want[1][0][1])
        assert all(torch.equal(g[k], want[1][1][k]) for k in g)


@pytest.mark.parametrize("bad", [[0, 50, 40, 100], [1, 50, 80, 100], [0, 50, 80, 99]])
def test_bad_offsets_are_reported_and_nothing_is_written(bad):
    m = kda()
    d = make(11, torch.bfloat16, 2, 2, 128, 128, lens=[30, 30, 40])
    d["cu"] = torch.tensor(bad, dtype=torch.int32, device=DEV)
    out = torch.full_like(d["v"], 3.0)
    S = torch.full_like(d["S0"], 3.0)
    m.gdn_chunk_fwd(d["q"], d["k"], d["v"], d["log_alpha"], d["beta"], S0=d["S0"], cu_seqlens=d["cu"], out=out,
                    S_final=S)
    with pytest.raises(m.KdaError) as e:
        m.check()
    assert e.value.code == 6
    assert (out == 3.0).all() and (S == 3.0).all()


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_bad_offsets_leave_the_gradients(dt):
    m = kda()
    d = make(12, dt, 2, 1, 128, 128, lens=[30, 30, 40])
    d["cu"] = torch.tensor([0, 50, 40, 100], dtype=torch.int32, device=DEV)
    mine = {x: torch.full_like(d[y], 3.0) for x, y in (("dq", "q"), ("dk", "k"), ("dv", "v"), ("dS0", "S0"),
                                                       ("dlog_alpha", "log_alpha"), ("dbeta", "beta"))}
    m.gdn_chunk_bwd(d["q"], d["k"], d["v"], d["log_alpha"], d["beta"], d["dout"], S0=d["S0"], cu_seqlens=d["cu"],
                    grads=mine)
    with pytest.raises(m.KdaError) as e:
        m.check()
    assert e.value.code == 6
    for x in ("dv", "dS0", "dlog_alpha", "dbeta") + (("dq", "dk") if dt == torch.bfloat16 else ()):
        assert (mine[x] == 3.0).all(), x  # (in fp32 the sum over shared heads writes dq and dk)


def test_binding_refuses():
    m = kda()
    d = make(12, torch.bfloat16, 4, 2, 128, 128, T=8)
    a = [d[x] for x in ("q", "k", "v", "log_alpha", "beta")]

    def swap(i, t):
        return [*a[:i], t, *a[i + 1:]]

    for args, err in ((swap(0, a[0].half()), TypeError), (swap(1, a[1].float()), TypeError),
                      (swap(2, a[2][:, :, :3].contiguous()), ValueError), (swap(3, a[3].bfloat16()), TypeError),
                      (swap(3, a[3][..., None].expand(1, 8, 4, 128).contiguous()), ValueError),
                      (swap(4, a[4][:, :7].contiguous()), ValueError), (swap(1, a[1].transpose(1, 2)), ValueError)):
        with pytest.raises(err):
            m.gdn_chunk_fwd(*args)
    for kw, err in ((dict(S0=d["S0"].bfloat16()), TypeError), (dict(S0=d["S0"][:, :2].contiguous()), ValueError),
                    (dict(cu_seqlens=torch.tensor([0, 8], device=DEV)), TypeError),
                    (dict(out=torch.empty_like(a[0])), ValueError),
                    (dict(workspace=torch.empty(512, dtype=torch.uint8, device=DEV)), m.KdaError)):
        with pytest.raises(err):
            m.gdn_chunk_fwd(*a, **kw)
    with pytest.raises(ValueError):
        m.gdn_chunk_bwd(*a, d["dout"][:, :4].contiguous())
    with pytest.raises(ValueError):
        m.gdn_decode_step(a[0][0], a[1][0], a[2][0], a[3][0], a[4][0], torch.zeros(8, 4, 64, 128, device=DEV))
