"""Cases, plain forms and exact values of the gated delta rule's operators.

With one forget gate a head (log alpha a scalar for each token and head), a state S [dk, dv] evolves as

    S_t = alpha_t S_{t-1} + beta_t k_t (v_t - alpha_t S_{t-1}^T k_t)^T,     o_t = S_t^T q_t.

Operators, by the case's "op":

    prefill   the chunked form over whole prompts: out and the final states
    backward  its gradients, for the cotangents of out and of the final states
    decode    one token for each sequence, the fp32 states updated in place
    store     states written into slots of an 8-bit cache and read back (a request put aside and resumed)
    restore   states read back from slots of such a cache (requests that resume from a shared prefix)

The cache holds int8 codes with one fp32 scale for each row (slot, head, key channel):
scale = max |row| / 127, code = row / scale rounded to the nearest, ties to even, both quotients in 32 bits.
"""
import random

import torch

own = False

CHUNK = 64


# ---------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------
def _seq(op, name, dtype, H, Hk, dk, dv, lens, packed, s0):
    return {"name": name, "op": op, "dtype": dtype, "H": H, "Hk": Hk, "dk": dk, "dv": dv,
            "lens": ",".join(map(str, lens)), "packed": packed, "s0": s0}


def _dec(name, dtype, N, H, Hk, dk, dv):
    return {"name": name, "op": "decode", "dtype": dtype, "N": N, "H": H, "Hk": Hk, "dk": dk, "dv": dv}


def _cache(op, name, N, slots, H, dk, dv):
    return {"name": name, "op": op, "N": N, "slots": slots, "H": H, "dk": dk, "dv": dv}


def listed():
    return [
        # one long prompt, the size of this repository's headline workload
        _seq("prefill", "prefill_32k", "bf16", 32, 32, 128, 128, [32768], False, True),
        # a ragged batch of packed prompts, q/k heads shared by two value heads, an empty one among them
        _seq("prefill", "prefill_packed", "bf16", 32, 16, 128, 128, [4099, 1, 8191, 0, 63, 2050, 65, 1027], True, False),
        # a padded batch of prompts of a small model
        _seq("prefill", "prefill_batch", "bf16", 16, 16, 128, 128, [1000] * 8, False, True),
        # the smallest configuration: fp32 throughout, d = 64, where the launches count
        _seq("prefill", "prefill_tiny_fp32", "fp32", 2, 2, 64, 64, [256], False, False),
        # a training step on one long sequence
        _seq("backward", "backward_32k", "bf16", 32, 32, 128, 128, [32768], False, True),
        # a training step on packed documents with shared q/k heads
        _seq("backward", "backward_packed", "bf16", 16, 8, 128, 128, [2049, 511, 1, 4096, 130, 1405], True, True),
        # the smallest training step, fp32 throughout
        _seq("backward", "backward_tiny_fp32", "fp32", 2, 2, 64, 64, [256], False, False),
        # a serving batch, the size of this repository's decode workload
        _dec("decode_256", "bf16", 256, 32, 32, 128, 128),
        # one user
        _dec("decode_1", "bf16", 1, 32, 16, 128, 128),
        # a batch of preempted requests put aside and resumed
        _cache("store", "store_64", 64, 96, 32, 128, 128),
        # a few requests of a smaller layer
        _cache("store", "store_3", 3, 8, 16, 64, 128),
        # many requests that resume from a few shared prefixes
        _cache("restore", "restore_192", 192, 24, 32, 128, 128),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(lo * (hi / lo) ** rng.random())))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "prefill", "backward", "backward", "decode", "decode", "store", "restore"])
    dk, dv = rng.choice([(128, 128)] * 5 + [(64, 64), (64, 128), (128, 64)])
    if op in ("store", "restore"):
        return {k: v for k, v in _cache(op, "", _log(rng, 1, 192 if op == "restore" else 64), rng.randint(64, 96),
                                        rng.choice([2, 7, 16, 32]), dk, dv).items() if k != "name"}
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    Hk = rng.choice([1, 2, 4, 5, 8, 16])
    H = Hk * rng.choice([1, 1, 2, 4] if Hk <= 8 else [1, 2])
    if op == "decode":
        c = _dec("", dtype, _log(rng, 1, 256), H, Hk, dk, dv)
    else:
        small = dtype == "fp32" or (dk, dv) != (128, 128)
        total = _log(rng, 1, (4096 if small else 32768) * 32 // max(H, 8) // (2 if small else 1))
        total = min(total, 32768)
        packed = rng.random() < 0.6
        if packed:
            n = rng.randint(1, 12)
            cuts = sorted(rng.randint(0, total) for _ in range(n - 1))
            lens = [b - a for a, b in zip([0] + cuts, cuts + [total])]
        else:
            n = rng.choice([1, 1, 2, 3, 8])
            lens = [max(1, total // n)] * n
        c = _seq(op, "", dtype, H, Hk, dk, dv, lens, packed, rng.random() < 0.5)
    del c["name"]
    return c


# ---------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------
def _lens(case):
    return [int(x) for x in case["lens"].split(",")]


def _unit(x):
    return x / x.norm(dim=-1, keepdim=True)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    H, dk, dv = case["H"], case["dk"], case["dv"]

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=g, device="cuda") * std

    s = {"op": case["op"]}
    if case["op"] in ("store", "restore"):
        N, slots = case["N"], case["slots"]
        r = random.Random(seed)
        # states whose rows differ in size, as key channels do, some of them never written
        S = normal(N if case["op"] == "store" else slots, H, dk, dv) * torch.exp(normal(1, H, dk, 1))
        S[:, :, 5] = 0.0
        if case["op"] == "store":
            s["S"] = S
            s["cache"] = torch.zeros(slots, H, dk, dv, dtype=torch.int8, device="cuda")
            s["scale"] = torch.zeros(slots, H, dk, device="cuda")
            ids = r.sample(range(slots), N)
        else:
            s["cache"], s["scale"] = _quantise(S)
            ids = [r.randrange(slots) for _ in range(N)]
        s["slots"] = torch.tensor(ids, dtype=torch.int32, device="cuda")
        return s

    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    Hk = case["Hk"]
    if case["op"] == "decode":
        lead = (case["N"],)
        N = case["N"]
    else:
        lens = _lens(case)
        N = len(lens)
        lead = (1, sum(lens)) if case["packed"] else (N, lens[0])
        s["cu"] = None
        if case["packed"]:
            cu = [0]
            for x in lens:
                cu.append(cu[-1] + x)
            s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        s["lens"] = lens
    s["q"] = _unit(normal(*lead, Hk, dk)).to(dt)
    s["k"] = _unit(normal(*lead, Hk, dk)).to(dt)
    s["v"] = normal(*lead, H, dv).to(dt)
    s["log_alpha"] = torch.nn.functional.logsigmoid(normal(*lead, H) + 3.0)
    s["beta"] = torch.sigmoid(normal(*lead, H))
    if case["op"] == "decode":
        s["S"] = normal(N, H, dk, dv, std=0.02)
        return s
    s["S0"] = normal(N, H, dk, dv, std=0.02) if case["s0"] else None
    if case["op"] == "backward":
        s["dout"] = normal(*lead, H, dv).to(dt)
        s["dS_final"] = normal(N, H, dk, dv, std=0.1)
    return s


# ---------------------------------------------------------------------------------------------------
# plain forms: chunks of 64 tokens, all sequences and heads at once, 32 bits
# ---------------------------------------------------------------------------------------------------
def _rows(s):
    """[N, Tp] row numbers of the flattened tokens, Tp a multiple of 64; one past the last for padding."""
    lens = s["lens"]
    longest = max(lens)
    Tp = max(CHUNK, (longest + CHUNK - 1) // CHUNK * CHUNK)
    n = torch.tensor(lens, device="cuda")
    start = n.cumsum(0) - n
    t = torch.arange(Tp, device="cuda")
    return torch.where(t < n[:, None], start[:, None] + t, sum(lens))


def _chunks(x, rows, group=1):
    """[B, T, h, ...] -> [N h*group, chunks, 64, ...] in 32 bits, zeros behind each sequence's end."""
    x = x.reshape(-1, *x.shape[2:]).float()
    x = torch.cat([x, x.new_zeros(1, *x.shape[1:])])[rows]
    if group > 1:
        x = x.repeat_interleave(group, dim=2)
    N, Tp, h = x.shape[:3]
    return x.transpose(1, 2).reshape(N * h, Tp // CHUNK, CHUNK, *x.shape[3:])


def _tokens(x, like, rows, H):
    """[N H, chunks, 64, ...] -> the tokens' layout of `like`, with H heads, in its type."""
    N, Tp = rows.shape
    x = x.reshape(N, H, Tp, *x.shape[3:]).transpose(1, 2)
    T = like.shape[0] * like.shape[1]
    return x[rows < T].reshape(*like.shape[:2], *x.shape[2:]).to(like.dtype)


def _intra(s):
    """What no state enters, for all chunks: decays, the system's inverse and the causal scores."""
    H = s["v"].shape[2]
    group = H // s["q"].shape[2]
    rows = _rows(s)
    c = {"rows": rows, "H": H, "group": group}
    c["q"], c["k"], c["v"] = _chunks(s["q"], rows, group), _chunks(s["k"], rows, group), _chunks(s["v"], rows)
    c["b"] = _chunks(s["beta"], rows)
    c["g"] = _chunks(s["log_alpha"], rows).cumsum(-1)
    c["D"] = torch.exp((c["g"][..., :, None] - c["g"][..., None, :]).tril()).tril()
    c["KK"] = c["k"] @ c["k"].mT
    c["A"] = (c["b"][..., :, None] * c["KK"] * c["D"]).tril(-1)
    eye = torch.eye(CHUNK, device="cuda")
    c["X"] = torch.linalg.solve_triangular(eye + c["A"], eye.expand_as(c["A"]), upper=False, unitriangular=True)
    c["P"] = c["q"] @ c["k"].mT * c["D"]
    c["eg"] = torch.exp(c["g"])[..., None]
    c["w"] = torch.exp(c["g"][..., -1:] - c["g"])[..., None]
    c["last"] = torch.exp(c["g"][..., -1])[..., None, None]
    return c


def _start(s, c):
    dk, dv = s["k"].shape[-1], s["v"].shape[-1]
    n = c["v"].shape[0]
    if s["S0"] is None:
        return torch.zeros(n, dk, dv, device="cuda")
    return s["S0"].reshape(n, dk, dv)


def _plain_prefill(s):
    c = _intra(s)
    S = _start(s, c)
    out = []
    for i in range(c["v"].shape[1]):
        k, eg = c["k"][:, i], c["eg"][:, i]
        U = c["X"][:, i] @ (c["b"][:, i, :, None] * (c["v"][:, i] - eg * (k @ S)))
        out.append(eg * (c["q"][:, i] @ S) + c["P"][:, i] @ U)
        S = c["last"][:, i] * S + k.mT @ (c["w"][:, i] * U)
    N, H = len(s["lens"]), c["H"]
    return {"out": _tokens(torch.stack(out, 1), s["v"], c["rows"], H), "S_final": S.reshape(N, H, *S.shape[1:])}


def _plain_backward(s):
    c = _intra(s)
    n, nc = c["v"].shape[:2]
    do = _chunks(s["dout"], c["rows"])
    S, before, R, U = _start(s, c), [], [], []
    for i in range(nc):
        before.append(S)
        R.append(c["v"][:, i] - c["eg"][:, i] * (c["k"][:, i] @ S))
        U.append(c["X"][:, i] @ (c["b"][:, i, :, None] * R[i]))
        S = c["last"][:, i] * S + c["k"][:, i].mT @ (c["w"][:, i] * U[i])
    dS = s["dS_final"].reshape(S.shape)
    grads = []
    for i in reversed(range(nc)):
        q, k, d, D = c["q"][:, i], c["k"][:, i], do[:, i], c["D"][:, i]
        eg, w, b, last = c["eg"][:, i], c["w"][:, i], c["b"][:, i, :, None], c["last"][:, i]
        S = before[i]
        dU = c["P"][:, i].mT @ d + w * (k @ dS)
        dR = c["X"][:, i].mT @ dU
        dP, dA = (d @ U[i].mT).tril(), -(dR @ U[i].mT).tril(-1)
        dq_S, dk_S, dk_w = eg * (d @ S.mT), -eg * b * (dR @ S.mT), w * (U[i] @ dS.mT)
        PD, G = dP * D, dA * b * D
        E = dP * c["P"][:, i] + dA * c["A"][:, i]
        db = (dR * R[i]).sum(-1) + (dA * D * c["KK"][:, i]).sum(-1)
        kw = (k * dk_w).sum(-1)
        dg = (q * dq_S).sum(-1) + (k * dk_S).sum(-1) - kw + E.sum(-1) - E.sum(-2)
        dg[:, -1] += kw.sum(-1) + (last * S * dS).sum((-1, -2))
        grads.append((dq_S + PD @ k, dk_S + dk_w + PD.mT @ q + (G + G.mT) @ k, b * dR,
                      dg.flip(-1).cumsum(-1).flip(-1), db))
        dS = last * dS + q.mT @ (eg * d) - k.mT @ (eg * b * dR)
    dq, dk, dv, dla, db = (torch.stack(x[::-1], 1) for x in zip(*grads))
    rows, H, group = c["rows"], c["H"], c["group"]

    def heads(x):  # the value heads that share a q/k head, summed
        x = x.reshape(len(s["lens"]), H // group, group, nc, CHUNK, -1).sum(2)
        return x.reshape(-1, nc, CHUNK, x.shape[-1])

    return {"dq": _tokens(heads(dq), s["q"], rows, H // group), "dk": _tokens(heads(dk), s["k"], rows, H // group),
            "dv": _tokens(dv, s["v"], rows, H), "dlog_alpha": _tokens(dla, s["log_alpha"], rows, H),
            "dbeta": _tokens(db, s["beta"], rows, H), "dS0": dS.reshape(len(s["lens"]), H, *dS.shape[1:])}


def _plain_decode(s):
    H = s["v"].shape[1]
    group = H // s["q"].shape[1]
    q, k = (s[x].float().repeat_interleave(group, dim=1) for x in ("q", "k"))
    S = s["S"]
    S *= torch.exp(s["log_alpha"])[..., None, None]
    u = s["beta"][..., None] * (s["v"].float() - (k[..., None, :] @ S).squeeze(-2))
    S += k[..., :, None] * u[..., None, :]
    return {"out": (q[..., None, :] @ S).squeeze(-2).to(s["v"].dtype), "S": S}


def _quantise(S):
    scale = S.abs().amax(-1)
    scale = scale / torch.full_like(scale, 127.0)  # by a tensor: a division, not a product with 1/127
    step = torch.where(scale > 0, scale, torch.ones_like(scale))
    return torch.round(S / step[..., None]).clamp(-127, 127).to(torch.int8), scale


def _plain_store(s):
    at = s["slots"].long()
    s["cache"][at], s["scale"][at] = _quantise(s["S"])
    return _plain_restore(s)


def _plain_restore(s):
    at = s["slots"].long()
    return {"S": s["cache"][at].float() * s["scale"][at][..., None]}


def _kernels(s):
    import gated_delta_rule_83_b200 as kda
    if s["op"] == "prefill":
        out, S = kda.gdn_chunk_fwd(s["q"], s["k"], s["v"], s["log_alpha"], s["beta"], S0=s["S0"], cu_seqlens=s["cu"])
        return {"out": out, "S_final": S}
    if s["op"] == "backward":
        return kda.gdn_chunk_bwd(s["q"], s["k"], s["v"], s["log_alpha"], s["beta"], s["dout"], S0=s["S0"],
                                 dS_final=s["dS_final"], cu_seqlens=s["cu"])
    if s["op"] == "decode":
        return {"out": kda.gdn_decode_step(s["q"], s["k"], s["v"], s["log_alpha"], s["beta"], s["S"]), "S": s["S"]}
    if s["op"] == "store":
        kda.state_cache_write(s["S"], s["cache"], s["scale"], s["slots"])
    return {"S": kda.state_cache_read(s["cache"], s["scale"], s["slots"])}


def run(state):
    if own:
        return _kernels(state)
    return {"prefill": _plain_prefill, "backward": _plain_backward, "decode": _plain_decode, "store": _plain_store,
            "restore": _plain_restore}[state["op"]](state)


# ---------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------------
def work(case):
    H, dk, dv = case["H"], case["dk"], case["dv"]
    if case["op"] in ("store", "restore"):
        f32, i8 = 4 * H * dk * dv, H * dk * dv + 4 * H * dk
        if case["op"] == "store":
            return {"bytes": case["N"] * (2 * f32 + 2 * i8 + 4), "flops": 4 * case["N"] * H * dk * dv}
        return {"bytes": case["N"] * (f32 + 4) + min(case["N"], case["slots"]) * i8, "flops": case["N"] * H * dk * dv}
    e = 2 if case["dtype"] == "bf16" else 4
    Hk = case["Hk"]
    token = e * (2 * Hk * dk + H * dv) + 8 * H  # q, k, v, log alpha, beta
    if case["op"] == "decode":
        return {"bytes": case["N"] * (token + e * H * dv + 8 * H * dk * dv), "flops": 7 * case["N"] * H * dk * dv}
    lens = _lens(case)
    T, state = sum(lens), 4 * len(lens) * H * dk * dv
    if case["op"] == "prefill":
        return {"bytes": T * (token + e * H * dv) + state * (2 if case["s0"] else 1), "flops": 7 * T * H * dk * dv}
    return {"bytes": T * (2 * token + e * H * dv) + state * (3 if case["s0"] else 2), "flops": 20 * T * H * dk * dv}


# ---------------------------------------------------------------------------------------------------
# exact values: token by token, 64 bits
# ---------------------------------------------------------------------------------------------------
def _token_major(x, lens, group=1):
    """[B, T, h, ...] -> [T, N, h*group, ...] in 64 bits."""
    x = x.reshape(-1, *x.shape[2:]).double()
    y = x.new_zeros(max(lens), len(lens), *x.shape[1:])
    at = 0
    for n, L in enumerate(lens):
        y[:L, n] = x[at:at + L]
        at += L
    return y.repeat_interleave(group, dim=2) if group > 1 else y


def _packed(y, lens, like):
    y = torch.cat([y[:L, n] for n, L in enumerate(lens)])
    return y.reshape(*like.shape[:2], *y.shape[1:])


def _step(S, k, v, a, b):
    """The decayed state, the value's error and the new state."""
    Sd = a[..., None, None] * S
    e = v - torch.einsum("nhk,nhkv->nhv", k, Sd)
    return Sd, e, Sd + k[..., :, None] * (b[..., None] * e)[..., None, :]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "store":
        # the definition rounds the scale and the quotient to 32 bits; both roundings are made here from 64
        x = s["S"].double()
        scale = (x.abs().amax(-1, keepdim=True) / 127.0).float().double()
        code = torch.where(scale > 0, x / torch.where(scale > 0, scale, 1.0), 0.0).float().round().double()
        return {"S": (code * scale).float()}
    if op == "restore":
        rows = [s["cache"][int(i)].double() * s["scale"][int(i)].double()[..., None] for i in s["slots"].tolist()]
        return {"S": torch.stack(rows).float()}
    H = case["H"]
    group = H // case["Hk"]
    if op == "decode":
        q, k = (s[x].double().repeat_interleave(group, dim=1) for x in ("q", "k"))
        S = _step(s["S"].double(), k, s["v"].double(), s["log_alpha"].double().exp(), s["beta"].double())[2]
        return {"out": torch.einsum("nhk,nhkv->nhv", q, S), "S": S}
    lens = _lens(case)
    T, N = max(lens), len(lens)
    dk, dv = case["dk"], case["dv"]
    bytes_a_step = 8 * N * H * dk * dv * (14 if op == "prefill" else 50)
    if T * ((10 if op == "prefill" else 50) * 8e-6 + bytes_a_step / 4e12) > 15:
        return None
    q, k = (_token_major(s[x], lens, group) for x in ("q", "k"))
    v, a, b = _token_major(s["v"], lens), _token_major(s["log_alpha"], lens).exp(), _token_major(s["beta"], lens)
    S = s["S0"].double() if s["S0"] is not None else v.new_zeros(N, H, dk, dv)
    if op == "prefill":
        out = torch.zeros_like(v)
        for t in range(T):
            S = _step(S, k[t], v[t], a[t], b[t])[2]
            out[t] = torch.einsum("nhk,nhkv->nhv", q[t], S)
        return {"out": _packed(out, lens, s["v"]), "S_final": S}
    do = _token_major(s["dout"], lens)
    every = 128
    kept = []
    for t in range(T):
        if t % every == 0:
            kept.append(S)
        S = _step(S, k[t], v[t], a[t], b[t])[2]
    dS = s["dS_final"].double()
    dq, dk_, dv_, da, db = (torch.zeros_like(x) for x in (q, k, v, a, b))
    for first in reversed(range(0, T, every)):
        S, steps = kept.pop(), []
        for t in range(first, min(T, first + every)):
            Sd, e, S1 = _step(S, k[t], v[t], a[t], b[t])
            steps.append((S, e))
            S = S1
        for t in reversed(range(first, min(T, first + every))):
            S, e = steps.pop()
            Sd = a[t][..., None, None] * S
            u = b[t][..., None] * e
            S1 = Sd + k[t][..., :, None] * u[..., None, :]
            dq[t] = torch.einsum("nhkv,nhv->nhk", S1, do[t])
            dS = dS + q[t][..., :, None] * do[t][..., None, :]
            du = torch.einsum("nhk,nhkv->nhv", k[t], dS)
            de = b[t][..., None] * du
            db[t] = (du * e).sum(-1)
            dk_[t] = torch.einsum("nhkv,nhv->nhk", dS, u) - torch.einsum("nhkv,nhv->nhk", Sd, de)
            dv_[t] = de
            dS = dS - k[t][..., :, None] * de[..., None, :]
            da[t] = (dS * Sd).sum((-1, -2))  # times alpha: with respect to log alpha
            dS = a[t][..., None, None] * dS

    def heads(x):
        return x.unflatten(2, (H // group, group)).sum(3)

    return {"dq": _packed(heads(dq), lens, s["q"]), "dk": _packed(heads(dk_), lens, s["k"]),
            "dv": _packed(dv_, lens, s["v"]), "dlog_alpha": _packed(da, lens, s["log_alpha"]),
            "dbeta": _packed(db, lens, s["beta"]), "dS0": dS}

