"""The gated delta rule token by token in 64 bits on the CPU, forward and backward, from its definition, and the
inputs the tests draw.  Tensors are [B, H, T, .] here; `lens` are the rows of each sequence."""
import torch


def make(B, Hk, H, T, d, e, dtype, seed, gate=True, init=False, final=False, lens=None, scale=1.0):
    """Inputs in the call's types ([B, heads, T, .]): keys of length 1, gates between 0.2 and 1, beta in (0, 1)."""
    r = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=r)  # noqa: E731
    unit = lambda x: x / (x.norm(dim=-1, keepdim=True) + 1e-6)  # noqa: E731
    x = {"q": (unit(rn(B, Hk, T, d)) * scale).to(dtype), "k": unit(rn(B, Hk, T, d)).to(dtype),
         "v": rn(B, H, T, e).to(dtype), "do": rn(B, H, T, e).to(dtype),
         "g": -rn(B, H, T).abs() * 0.3 if gate else None, "beta": torch.sigmoid(rn(B, H, T)),
         "init": 0.5 * rn(B, H, d, e) if init else None, "dfinal": 0.5 * rn(B, H, d, e) if final else None,
         "lens": None if lens is None else torch.tensor(lens, dtype=torch.int32)}
    return x


def _prepared(x):
    q, k, v, do, b = (x[n].double() for n in ("q", "k", "v", "do", "beta"))
    B, H, T, e = v.shape
    Hk, d = q.shape[1], q.shape[3]
    rep = H // Hk
    q, k = q.repeat_interleave(rep, 1), k.repeat_interleave(rep, 1)
    g = torch.zeros_like(b) if x["g"] is None else x["g"].double()
    n = torch.full((B,), T) if x["lens"] is None else x["lens"].long().clamp(0, T)
    live = (torch.arange(T)[None] < n[:, None])[:, None]  # [B, 1, T]
    zero = torch.zeros((), dtype=torch.float64)
    # rows behind the end: read nothing, whatever is there
    g, b = torch.where(live, g, zero), torch.where(live, b, zero)
    q, k, v, do = (torch.where(live[..., None], t, zero) for t in (q, k, v, do))
    S = torch.zeros(B, H, d, e, dtype=torch.float64) if x["init"] is None else x["init"].double()
    return q, k, v, do, g, b, S, live, rep


def forward(x):
    """(o, final state); o is zero behind a sequence's end."""
    q, k, v, _, g, b, S, live, _ = _prepared(x)
    o = torch.zeros_like(v)
    for t in range(v.shape[2]):
        S = g[:, :, t].exp()[..., None, None] * S
        u = b[:, :, t, None] * (v[:, :, t] - (S * k[:, :, t, :, None]).sum(-2))
        S = S + k[:, :, t, :, None] * u[:, :, None]
        o[:, :, t] = (S * q[:, :, t, :, None]).sum(-2)
    return o, S


def backward(x):
    """{dq, dk, dv, dg, dbeta, dinit}; `mag` is the size of the terms that dg is the difference of."""
    q, k, v, do, g, b, S, live, rep = _prepared(x)
    B, H, T, e = v.shape
    d = q.shape[3]
    steps = []
    for t in range(T):
        D = g[:, :, t].exp()[..., None, None] * S
        w = v[:, :, t] - (D * k[:, :, t, :, None]).sum(-2)
        S = D + k[:, :, t, :, None] * (b[:, :, t, None] * w)[:, :, None]
        steps.append((D, w, S))
    dS = torch.zeros_like(S) if x["dfinal"] is None else x["dfinal"].double()
    dq, dk, dv, dg, db = (torch.zeros_like(t) for t in (q, k, v, g, b))
    mag = torch.zeros_like(g)
    for t in range(T - 1, -1, -1):
        D, w, S1 = steps[t]
        mag[:, :, t] = (dS * S1).sum((-1, -2)).abs()
        dq[:, :, t] = (S1 * do[:, :, t, None]).sum(-1)
        dS = dS + q[:, :, t, :, None] * do[:, :, t, None]
        du = (dS * k[:, :, t, :, None]).sum(-2)
        dw = b[:, :, t, None] * du
        db[:, :, t] = (du * w).sum(-1)
        dv[:, :, t] = dw
        put = (dS * (b[:, :, t, None] * w)[:, :, None]).sum(-1)
        got = -(D * dw[:, :, None]).sum(-1)
        dk[:, :, t] = put + got
        mag[:, :, t] += sum((a * c).sum(-1).abs() for a, c in ((q[:, :, t], dq[:, :, t]), (k[:, :, t], put),
                                                               (k[:, :, t], got)))
        dS = dS - k[:, :, t, :, None] * dw[:, :, None]
        dg[:, :, t] = (dS * D).sum((-1, -2))
        dS = g[:, :, t].exp()[..., None, None] * dS
    dg, db, mag = (t * live for t in (dg, db, mag))
    group = lambda y: y.reshape(B, H // rep, rep, T, d).sum(2)  # noqa: E731
    return {"dq": group(dq), "dk": group(dk), "dv": dv, "dg": dg, "dbeta": db, "dinit": dS, "mag": mag}


def decode(q, k, v, g, b, S):
    """One step from states S [B, H, d, e]: (o, new states)."""
    rep = v.shape[1] // q.shape[1]
    q, k = (t.double().repeat_interleave(rep, 1) for t in (q, k))
    a = torch.ones_like(b).double() if g is None else g.double().exp()
    S = a[..., None, None] * S.double()
    u = b.double()[..., None] * (v.double() - (S * k[..., None]).sum(-2))
    S = S + k[..., None] * u[:, :, None]
    return (S * q[..., None]).sum(-2), S
