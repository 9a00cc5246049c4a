"""Cases, plain forms and 64-bit values of the gated delta rule's operators and of the state pool's copies.

Per sequence b and value head h, with a d x e state S (rows: key features, columns: value features),

    S_t = exp(g_t) (I - beta_t k_t k_t^T) S_{t-1} + beta_t k_t v_t^T,    o_t = S_t^T q_t.

Four operators: "fwd" (whole sequences), "bwd" (its gradients), "decode" (one token per sequence over a pool of
states) and "copy" (pool slots forked, moved and cleared).  q and k have Hk heads, v, g and beta have H heads,
and value head h reads key head h // (H / Hk).
"""
import torch

own = False

_CHUNK = 64


# ---------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one short prompt on 16 narrow heads, answered at once: latency of a prefill, with the state kept for decoding
        {"name": "fwd_prompt", "op": "fwd", "B": 1, "Hk": 16, "H": 16, "T": 77, "d": 64, "e": 64, "dtype": "bf16",
         "out": "bf16", "layout": "bthd", "final": True, "init": False, "ragged": False},
        # training forward of the 400M-shaped layer (8 x 2048 tokens, 16 heads of 64)
        {"name": "fwd_400m", "op": "fwd", "B": 8, "Hk": 16, "H": 16, "T": 2048, "d": 64, "e": 64, "dtype": "bf16",
         "out": "bf16", "layout": "bhtd", "final": False, "init": False, "ragged": False},
        # training forward of the 15B-shaped layer (2 x 6144 tokens, 40 heads of 128)
        {"name": "fwd_15b", "op": "fwd", "B": 2, "Hk": 40, "H": 40, "T": 6144, "d": 128, "e": 128, "dtype": "bf16",
         "out": "bf16", "layout": "bhtd", "final": False, "init": False, "ragged": False},
        # a batch of prompts of different lengths that continue earlier states, two value heads per key head
        {"name": "fwd_ragged", "op": "fwd", "B": 8, "Hk": 16, "H": 32, "T": 4099, "d": 128, "e": 128, "dtype": "bf16",
         "out": "bf16", "layout": "bthd", "final": True, "init": True, "ragged": True},
        # one long document on 16 heads: few sequences, a long axis
        {"name": "fwd_long", "op": "fwd", "B": 1, "Hk": 16, "H": 16, "T": 65536, "d": 128, "e": 128, "dtype": "bf16",
         "out": "bf16", "layout": "bhtd", "final": True, "init": False, "ragged": False},
        # fp32 training in pieces: small, with states on both sides and ragged lengths
        {"name": "bwd_f32_piece", "op": "bwd", "B": 2, "Hk": 1, "H": 2, "T": 517, "d": 64, "e": 64, "dtype": "f32",
         "out": "f32", "layout": "bhtd", "final": True, "init": True, "ragged": True},
        # training backward of the 400M-shaped layer
        {"name": "bwd_400m", "op": "bwd", "B": 8, "Hk": 16, "H": 16, "T": 2048, "d": 64, "e": 64, "dtype": "bf16",
         "out": "bf16", "layout": "bhtd", "final": False, "init": False, "ragged": False},
        # training backward of the 15B-shaped layer
        {"name": "bwd_15b", "op": "bwd", "B": 2, "Hk": 40, "H": 40, "T": 6144, "d": 128, "e": 128, "dtype": "bf16",
         "out": "bf16", "layout": "bhtd", "final": False, "init": False, "ragged": False},
        # one token of an interactive session: latency of the recurrent step
        {"name": "decode_one", "op": "decode", "B": 1, "Hk": 16, "H": 16, "slots": 1, "d": 64, "e": 64,
         "dtype": "bf16"},
        # one token of each of 64 sequences out of a pool of 96 slots, 40 heads of 128
        {"name": "decode_64", "op": "decode", "B": 64, "Hk": 40, "H": 40, "slots": 96, "d": 128, "e": 128,
         "dtype": "bf16"},
        # four sequences forked eight ways before sampling continues on each branch
        {"name": "copy_fork", "op": "copy", "n": 32, "slots": 48, "H": 40, "d": 128, "e": 128, "kind": "fork"},
        # a pool with holes packed to its front, the freed slots cleared: sources are themselves overwritten
        {"name": "copy_compact", "op": "copy", "n": 100, "slots": 257, "H": 16, "d": 64, "e": 64, "kind": "compact"},
    ]


def _log(rng, lo, hi):
    import math
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "bwd", "bwd", "decode", "copy"])
    if op in ("fwd", "bwd"):
        f32 = rng.random() < 0.3
        if f32:
            d, e = rng.randint(1, 128), rng.randint(1, 128)
        else:
            d, e = rng.choice([64, 128]), rng.choice([64, 128])
        Hk = rng.randint(1, 16)
        H = Hk * rng.choice([1, 1, 2, 3])
        B = _log(rng, 1, 8)
        most = (1 << 19) // (4 if f32 else 1)
        T = _log(rng, 1, max(1, min(16384, most // (B * H))))
        return {"op": op, "B": B, "Hk": Hk, "H": H, "T": T, "d": d, "e": e, "dtype": "f32" if f32 else "bf16",
                "out": "f32" if f32 else "bf16", "layout": rng.choice(["bhtd", "bthd"]),
                "final": rng.random() < 0.5, "init": rng.random() < 0.5, "ragged": rng.random() < 0.4}
    d, e = rng.randint(1, 128), rng.randint(1, 128)
    if rng.random() < 0.7:
        d, e = rng.choice([64, 128]), rng.choice([64, 128])
    if op == "decode":
        B, Hk = _log(rng, 1, 128), rng.randint(1, 20)
        return {"op": op, "B": B, "Hk": Hk, "H": Hk * rng.choice([1, 2]), "slots": B + rng.randint(0, 32), "d": d,
                "e": e, "dtype": rng.choice(["bf16", "bf16", "f32"])}
    n = _log(rng, 1, 100)
    return {"op": op, "n": n, "slots": 2 * n + rng.randint(0, 20), "H": rng.randint(1, 16), "d": d, "e": e,
            "kind": rng.choice(["fork", "compact"])}


# ---------------------------------------------------------------------------------------------- inputs

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _lengths(case, gen):
    """Ragged lengths: uniform over 0 .. T, with one sequence at T."""
    n = torch.randint(0, case["T"] + 1, (case["B"],), generator=gen, device="cuda", dtype=torch.int32)
    n[0] = case["T"]
    return n


def _gates(shape, gen, heads_dim):
    """Log-gates -A softplus(x - 4) with A in 1 .. 16 per head (most tokens keep 0.7 .. 0.99 of the state, a few drop
    it) and write strengths sigmoid(x), as a gated layer's projections produce them."""
    a_shape = [1] * len(shape)
    a_shape[heads_dim] = shape[heads_dim]
    A = 1 + 15 * torch.rand(a_shape, generator=gen, device="cuda")
    x = torch.randn(shape, generator=gen, device="cuda") - 4
    g = -A * torch.log1p(torch.exp(x))
    beta = torch.sigmoid(torch.randn(shape, generator=gen, device="cuda"))
    return g, beta


def _unit(x):
    """silu and division by the length: keys of a delta-rule layer have length 1 and lean to one side."""
    x = x * torch.sigmoid(x)
    return x / (x.square().sum(-1, keepdim=True) + 1e-6).sqrt()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    rn = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    if case["op"] == "copy":
        n, slots = case["n"], case["slots"]
        states = rn(slots, case["H"], case["d"], case["e"])
        order = torch.randperm(slots, generator=gen, device="cuda").to(torch.int32)
        if case["kind"] == "fork":  # an eighth of the pairs' number of sources, destinations outside of them
            few = max(1, n // 8)
            src = order[:few].repeat(-(-n // few))[:n].contiguous()
            dst = order[few:few + n].contiguous()
        else:  # slots at even places of a row move one place down it, every fourth is cleared
            dst = order[:n].contiguous()
            src = order[1:n + 1].clone()
            src[3::4] = -1
        return {"case": case, "states": states, "src": src, "dst": dst}
    dt = _TYPES[case["dtype"]]
    B, Hk, H, d, e = (case[n] for n in ("B", "Hk", "H", "d", "e"))
    if case["op"] == "decode":
        q = (_unit(rn(B, Hk, d)) * d ** -0.5).to(dt)
        k = _unit(rn(B, Hk, d)).to(dt)
        g, beta = _gates((B, H), gen, 1)
        states = 0.3 * rn(case["slots"], H, d, e)
        slots = torch.randperm(case["slots"], generator=gen, device="cuda")[:B].to(torch.int32)
        return {"case": case, "q": q, "k": k, "v": rn(B, H, e).to(dt), "g": g, "beta": beta, "states": states,
                "slots": slots}
    T = case["T"]
    shape = (lambda h, w: (B, h, T, w)) if case["layout"] == "bhtd" else (lambda h, w: (B, T, h, w))
    g, beta = _gates((B, H, T) if case["layout"] == "bhtd" else (B, T, H), gen, 1 if case["layout"] == "bhtd" else 2)
    s = {"case": case, "q": (_unit(rn(*shape(Hk, d))) * d ** -0.5).to(dt), "k": _unit(rn(*shape(Hk, d))).to(dt),
         "v": rn(*shape(H, e)).to(dt), "g": g, "beta": beta}
    s["init"] = 0.3 * rn(B, H, d, e) if case["init"] else None
    s["lens"] = _lengths(case, gen) if case["ragged"] else None
    if case["op"] == "bwd":
        s["do"] = rn(*shape(H, e)).to(dt)
        s["dfinal"] = 0.3 * rn(B, H, d, e) if case["final"] else None
    elif case["ragged"]:  # rows behind a sequence's end stay as they are in the caller's buffer
        s["o"] = torch.zeros(shape(H, e), dtype=_TYPES[case["out"]], device="cuda")
    return s


# ---------------------------------------------------------------------------------------------- plain forms

def _seqs(x, layout, rep=1):
    """[B, h, T, ...] or [B, T, h, ...] as [B * h * rep, T, ...] in 32 bits."""
    x = x if layout == "bhtd" else x.transpose(1, 2)
    x = x.float()
    if rep > 1:
        x = x.repeat_interleave(rep, dim=1)
    return x.reshape(x.shape[0] * x.shape[1], *x.shape[2:])


def _back(x, B, layout, dtype):
    """[B * h, T, ...] in the call's layout, rounded once."""
    x = x.reshape(B, x.shape[0] // B, *x.shape[1:]).to(dtype)
    return (x if layout == "bhtd" else x.transpose(1, 2)).contiguous()


def _cut(x):
    """[N, T, ...] as [N, chunks, 64, ...], zeros behind T."""
    T = x.shape[1]
    n = -(-T // _CHUNK)
    y = x.new_zeros(x.shape[0], n * _CHUNK, *x.shape[2:])
    y[:, :T] = x
    return y.reshape(x.shape[0], n, _CHUNK, *x.shape[2:])


def _unit_lower_inverse(L):
    """Inverse of unit lower triangular [..., 64, 64] matrices: blocks of 1, 2, .. 32 joined two by two."""
    n = L.shape[-1]
    X = torch.eye(n, device=L.device, dtype=L.dtype).expand_as(L).clone()
    m = 1
    while m < n:
        Lb = L.reshape(*L.shape[:-2], n // (2 * m), 2 * m, n // (2 * m), 2 * m)
        Xb = X.reshape(*L.shape[:-2], n // (2 * m), 2 * m, n // (2 * m), 2 * m)
        i = torch.arange(n // (2 * m), device=L.device)
        low = Lb[..., i, m:, i, :m]          # [pairs, ..., m, m]
        top, bot = Xb[..., i, :m, i, :m], Xb[..., i, m:, i, m:]
        Xb[..., i, m:, i, :m] = -(bot @ low @ top)
        m *= 2
    return X


def _chunks(s):
    """What both directions share, in 32 bits: chunked inputs, cumulative gates, the masked matrices."""
    c = s["case"]
    rep = c["H"] // c["Hk"]
    q, k = _seqs(s["q"], c["layout"], rep), _seqs(s["k"], c["layout"], rep)
    v, g, b = (_seqs(s[n], c["layout"]) for n in ("v", "g", "beta"))
    N, T = g.shape
    if s["lens"] is None:
        live = torch.ones(N, T, dtype=torch.bool, device=g.device)
    else:
        live = torch.arange(T, device=g.device) < s["lens"].repeat_interleave(c["H"])[:, None]
    g, b = g * live, b * live
    q, k, v, g, b = (_cut(x) for x in (q, k, v, g, b))
    G = g.double().cumsum(-1)
    low = torch.ones(_CHUNK, _CHUNK, dtype=torch.bool, device=g.device).tril()
    M = (G[..., :, None] - G[..., None, :]).masked_fill(~low, -torch.inf).exp().float()
    eG, eC, rest = G.exp().float(), G[..., -1].exp().float(), (G[..., -1:] - G).exp().float()
    A = (k @ k.transpose(-1, -2) * M).tril(-1)
    inv = _unit_lower_inverse(torch.eye(_CHUNK, device=g.device) + A * b[..., :, None])
    return {"q": q, "k": k, "v": v, "b": b, "M": M, "eG": eG, "eC": eC, "rest": rest, "A": A, "inv": inv,
            "live": live, "T": T, "N": N}


def _states(s, x):
    """The state that enters each chunk, and the last one."""
    c = s["case"]
    Uv = x["inv"] @ (x["b"][..., None] * x["v"])
    Uk = x["inv"] @ ((x["b"] * x["eG"])[..., None] * x["k"])
    S = x["v"].new_zeros(x["N"], c["d"], c["e"]) if s["init"] is None else s["init"].reshape(x["N"], c["d"], c["e"])
    at, U = [], []
    for i in range(Uv.shape[1]):
        at.append(S)
        U.append(Uv[:, i] - Uk[:, i] @ S)
        S = x["eC"][:, i, None, None] * S + (x["rest"][:, i, :, None] * x["k"][:, i]).transpose(-1, -2) @ U[-1]
    return torch.stack(at, 1), torch.stack(U, 1), S


def _plain_fwd(s):
    c, x = s["case"], _chunks(s)
    S0, U, last = _states(s, x)
    o = x["eG"][..., None] * (x["q"] @ S0) + (x["q"] @ x["k"].transpose(-1, -2) * x["M"]) @ U
    o = o.reshape(x["N"], -1, c["e"])[:, :x["T"]] * x["live"][..., None]
    out = {"o": _back(o, c["B"], c["layout"], _TYPES[c["out"]])}
    if c["final"]:
        out["state"] = last.reshape(c["B"], c["H"], c["d"], c["e"]).contiguous()
    return out


def _plain_bwd(s):
    c, x = s["case"], _chunks(s)
    N, rep = x["N"], c["H"] // c["Hk"]
    q, k, v, b, M = x["q"], x["k"], x["v"], x["b"], x["M"]
    do = _cut(_seqs(s["do"], c["layout"]) * x["live"][..., None])
    S0, U, last = _states(s, x)
    # u = beta w; w itself, since beta may be 0
    W = v - x["eG"][..., None] * (k @ S0) - x["A"] @ U
    P = q @ k.transpose(-1, -2) * M
    PdO, QdO = P.transpose(-1, -2) @ do, q.transpose(-1, -2) @ (x["eG"][..., None] * do)
    invT = x["inv"].transpose(-1, -2)
    dS = S0.new_zeros(N, c["d"], c["e"]) if s["dfinal"] is None else s["dfinal"].reshape(N, c["d"], c["e"])
    at, X = [None] * S0.shape[1], [None] * S0.shape[1]
    for i in range(S0.shape[1] - 1, -1, -1):
        at[i] = dS
        dU = PdO[:, i] + x["rest"][:, i, :, None] * (k[:, i] @ dS)
        X[i] = invT[:, i] @ dU
        dS = x["eC"][:, i, None, None] * dS + QdO[:, i] - \
            ((b * x["eG"])[:, i, :, None] * k[:, i]).transpose(-1, -2) @ X[i]
    dS1, X = torch.stack(at, 1), torch.stack(X, 1)
    dv, dbeta = b[..., None] * X, (X * W).sum(-1)
    dP = M * (do @ U.transpose(-1, -2))
    E = -(X @ U.transpose(-1, -2) * M).tril(-1) * b[..., :, None]
    dq = x["eG"][..., None] * (do @ S0.transpose(-1, -2)) + dP @ k
    row = E @ k - (b * x["eG"])[..., None] * (X @ S0.transpose(-1, -2))
    col = E.transpose(-1, -2) @ k + dP.transpose(-1, -2) @ q + x["rest"][..., None] * (U @ dS1.transpose(-1, -2))
    dG = ((q * dq).double().sum(-1) + (k * row).double().sum(-1) - (k * col).double().sum(-1))
    S1 = torch.cat([S0[:, 1:], last[:, None]], 1)
    dG[..., -1] += (dS1.double() * S1.double()).sum((-1, -2))
    dg = dG.flip(-1).cumsum(-1).flip(-1).float()
    flat = lambda t: t.reshape(N, -1, *t.shape[3:])[:, :x["T"]]  # noqa: E731
    live = x["live"]
    dq, dk, dv = (flat(t) * live[..., None] for t in (dq, row + col, dv))
    dq, dk = (t.reshape(c["B"] * c["Hk"], rep, *t.shape[1:]).sum(1) for t in (dq, dk))
    dg, dbeta = flat(dg) * live, flat(dbeta) * live
    dt = _TYPES[c["out"]]
    out = {"dq": _back(dq, c["B"], c["layout"], dt), "dk": _back(dk, c["B"], c["layout"], dt),
           "dv": _back(dv, c["B"], c["layout"], dt), "dg": _back(dg, c["B"], c["layout"], torch.float32),
           "dbeta": _back(dbeta, c["B"], c["layout"], torch.float32)}
    if c["init"]:
        out["dinit"] = dS.reshape(c["B"], c["H"], c["d"], c["e"]).contiguous()
    return out


def _plain_decode(s):
    c = s["case"]
    rep = c["H"] // c["Hk"]
    q, k = (s[n].float().repeat_interleave(rep, dim=1)[..., None] for n in ("q", "k"))
    at = s["slots"].long()
    S = s["g"].exp()[..., None, None] * s["states"][at]
    u = s["beta"][..., None] * (s["v"].float() - (k * S).sum(-2))
    S = S + k * u[..., None, :]
    s["states"][at] = S
    return {"o": (q * S).sum(-2), "states": s["states"]}


def _plain_copy(s):
    src = s["src"].long()
    moved = s["states"][src.clamp(min=0)] * (src >= 0)[:, None, None, None]
    s["states"][s["dst"].long()] = moved
    return {"states": s["states"]}


# ---------------------------------------------------------------------------------------------- one pass

def run(state):
    s, c = state, state["case"]
    if not own:
        return {"fwd": _plain_fwd, "bwd": _plain_bwd, "decode": _plain_decode, "copy": _plain_copy}[c["op"]](s)
    from causal_linear_attention_la2_b200 import la2
    if c["op"] == "fwd":
        r = la2.la2_gdr_fwd(s["q"], s["k"], s["v"], s["g"], s["beta"], layout=c["layout"], init_state=s["init"],
                            seq_lens=s["lens"], out=s.get("o"), want_final=c["final"], out_dtype=_TYPES[c["out"]])
        return {"o": r[0], "state": r[1]} if c["final"] else {"o": r}
    if c["op"] == "bwd":
        r = la2.la2_gdr_bwd(s["q"], s["k"], s["v"], s["g"], s["beta"], s["do"], layout=c["layout"],
                            init_state=s["init"], d_final_state=s["dfinal"], seq_lens=s["lens"],
                            want_d_init=c["init"], out_dtype=_TYPES[c["out"]])
        return dict(zip(("dq", "dk", "dv", "dg", "dbeta", "dinit"), r))
    if c["op"] == "decode":
        o = la2.la2_gdr_decode(s["q"], s["k"], s["v"], s["g"], s["beta"], s["states"], slots=s["slots"])
        return {"o": o, "states": s["states"]}
    la2.la2_state_copy(s["states"], s["src"], s["dst"])
    return {"states": s["states"]}


# ---------------------------------------------------------------------------------------------- 64 bits

def _exact_sequences(case, s):
    """The recurrence token by token in 64 bits, forward and, for "bwd", back again; states are kept every 64 tokens
    and the ones between them made again."""
    c = case
    rep, T = c["H"] // c["Hk"], c["T"]
    as64 = lambda t: (t if c["layout"] == "bhtd" else t.transpose(1, 2)).double()  # noqa: E731
    q, k = (as64(s[n]).repeat_interleave(rep, dim=1) for n in ("q", "k"))
    v, g, b = (as64(s[n]) for n in ("v", "g", "beta"))
    B, H, d, e = c["B"], c["H"], c["d"], c["e"]
    length = torch.full((B,), T, device=g.device) if s["lens"] is None else s["lens"].long()
    live = (torch.arange(T, device=g.device)[None] < length[:, None])[:, None].double()  # [B, 1, T]
    g, b = g * live, b * live
    a = g.exp()
    S = torch.zeros(B, H, d, e, dtype=torch.float64, device=g.device) if s["init"] is None else s["init"].double()

    def step(S, t):
        decayed = a[:, :, t, None, None] * S
        w = v[:, :, t] - torch.einsum("bhde,bhd->bhe", decayed, k[:, :, t])
        u = b[:, :, t, None] * w
        return decayed, w, u, decayed + k[:, :, t, :, None] * u[:, :, None, :]

    o, kept = torch.zeros_like(v), []
    for t in range(T):
        if t % 64 == 0:
            kept.append(S)
        S = step(S, t)[3]
        if c["op"] == "fwd":
            o[:, :, t] = torch.einsum("bhde,bhd->bhe", S, q[:, :, t])
    undo = lambda t: (t if c["layout"] == "bhtd" else t.transpose(1, 2)).contiguous()  # noqa: E731
    if c["op"] == "fwd":
        out = {"o": undo(o * live[..., None])}
        if c["final"]:
            out["state"] = S
        return out
    do = as64(s["do"]) * live[..., None]
    dq, dk, dv, dg, db = (torch.zeros_like(x) for x in (q, k, v, g, b))
    dS = torch.zeros_like(S) if s["dfinal"] is None else s["dfinal"].double()
    for c0 in range((T - 1) // 64 * 64, -1, -64):
        S, steps = kept.pop(), []
        for t in range(c0, min(T, c0 + 64)):
            decayed, w, u, S = step(S, t)
            steps.append((w, u, S, decayed))
        for t in range(min(T, c0 + 64) - 1, c0 - 1, -1):
            w, u, S, decayed = steps.pop()
            dq[:, :, t] = torch.einsum("bhde,bhe->bhd", S, do[:, :, t])
            dS = dS + q[:, :, t, :, None] * do[:, :, t, None, :]
            du = torch.einsum("bhde,bhd->bhe", dS, k[:, :, t])
            dw = b[:, :, t, None] * du
            db[:, :, t] = (du * w).sum(-1)
            dv[:, :, t] = dw
            # S = decayed + k u^T and w = v - decayed^T k
            dk[:, :, t] = torch.einsum("bhde,bhe->bhd", dS, u) - torch.einsum("bhde,bhe->bhd", decayed, dw)
            dS = dS - k[:, :, t, :, None] * dw[:, :, None, :]
            dg[:, :, t] = (dS * decayed).sum((-1, -2))
            dS = a[:, :, t, None, None] * dS
    group = lambda x: x.reshape(B, c["Hk"], rep, T, d).sum(2)  # noqa: E731
    l4 = live[..., None]
    out = {"dq": undo(group(dq * l4)), "dk": undo(group(dk * l4)), "dv": undo(dv * l4), "dg": undo(dg * live),
           "dbeta": undo(db * live)}
    if c["init"]:
        out["dinit"] = dS
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("fwd", "bwd"):
        return _exact_sequences(case, s)
    if case["op"] == "copy":
        old, new = s["states"].double(), s["states"].double()
        for i, j in zip(s["src"].tolist(), s["dst"].tolist()):
            new[j] = old[i] if i >= 0 else 0.0
        return {"states": new}
    states, rep = s["states"].double(), case["H"] // case["Hk"]
    o = torch.zeros(case["B"], case["H"], case["e"], dtype=torch.float64, device="cuda")
    for i, slot in enumerate(s["slots"].tolist()):
        k, q = (s[n][i].double().repeat_interleave(rep, dim=0) for n in ("k", "q"))
        S = torch.exp(s["g"][i].double())[:, None, None] * states[slot]
        u = s["beta"][i].double()[:, None] * (s["v"][i].double() - torch.einsum("hde,hd->he", S, k))
        S = S + torch.einsum("hd,he->hde", k, u)
        states[slot], o[i] = S, torch.einsum("hde,hd->he", S, q)
    return {"o": o, "states": states}


# ---------------------------------------------------------------------------------------------- work

def work(case):
    """Inputs read once, outputs written once; the recurrence's products (8 d e flops a token forward: decay, k S, the
    update, q S; 22 d e back: the state again, and the products of its gradient)."""
    if case["op"] == "copy":
        page = 4.0 * case["H"] * case["d"] * case["e"]
        reads = max(1, case["n"] // 8) if case["kind"] == "fork" else case["n"] - case["n"] // 4
        return {"bytes": page * (reads + case["n"]), "flops": 0.0}
    B, Hk, H, d, e = (case[n] for n in ("B", "Hk", "H", "d", "e"))
    w = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "decode":
        return {"bytes": B * (2.0 * 4 * H * d * e + 2 * w * Hk * d + (w + 4) * H * e), "flops": 8.0 * B * H * d * e}
    T, ow = case["T"], 2 if case["out"] == "bf16" else 4
    rows = B * T * (0.55 if case["ragged"] else 1.0)
    state = 4.0 * B * H * d * e
    if case["op"] == "fwd":
        return {"bytes": rows * (w * (2 * Hk * d + H * e) + 8 * H + ow * H * e) +
                state * (case["init"] + case["final"]), "flops": 8.0 * rows * H * d * e}
    return {"bytes": rows * (w * (2 * Hk * d + 2 * H * e) + 16 * H + ow * (2 * Hk * d + H * e)) +
            state * (2 * case["init"] + case["final"]), "flops": 22.0 * rows * H * d * e}
