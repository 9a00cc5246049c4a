"""The gated delta rule (la2_gdr_fwd, la2_gdr_bwd, la2_gdr_decode) and the state pool's copies (la2_state_copy).

CPU: the 64-bit reference against autograd, differences and special cases; refusals.  GPU: every call against the
reference.

Tolerances.  With fp32 outputs |err| <= TOL rms(exact) + OWN |exact|, element by element.  fp32 inputs: TOL = 1e-5, the
library's contract, and OWN = 0: a result is a sum of at most 128 + 128 products whose roundings (2^-24 each) add up
like a random walk, sqrt(256) 2^-24 = 1e-6 of the sum's size, and the largest element of a few 10^4 is some 5 sigma
out.  bf16 inputs: an operand x that the kernels form is split into two bf16 numbers, the first off by at most 2^-8 |x|,
their sum by 2^-8 2^-8 |x| = 2^-16 |x|; a product of two such operands drops that of the two low parts, 2^-16 more: off
by at most 3 2^-16 of itself.  Where one product makes an element (its own row's, say, which a sum over others cannot
average), that is what it is off by, twice where an operand came out of such a product: OWN = 6 2^-16; the sums of many
average it, and TOL = 5e-5 covers them.  A bf16 output adds its one rounding, 2^-8 |x|.
dg is a difference of terms larger than itself (`mag` in the reference, summed over a chunk of 64 rows): its
error is measured against rms(dg) + 8 rms(mag), 8 = sqrt(64)."""
import numpy as np
import pytest
import torch

import gdr_ref as R
from causal_linear_attention_la2_b200 import la2 as L

TOL = {torch.float32: 1e-5, torch.bfloat16: 5e-5}
OWN = {1e-5: 0.0, 5e-5: 6 * 2.0 ** -16}
BF16, F32 = torch.bfloat16, torch.float32


# ------------------------------------------------------------------------------------------------ CPU: reference

def _leaves(x):
    return {n: x[n].double().requires_grad_() for n in ("q", "k", "v", "g", "beta", "init")}


@pytest.mark.parametrize("T,lens", [(1, None), (7, None), (9, [9, 4, 0])])
def test_reference_gradients_are_autograds(T, lens):
    x = R.make(3, 2, 4, T, 5, 6, F32, 1, init=True, final=True, lens=lens)
    y = dict(x, **_leaves(x))
    o, S = R.forward(y)
    ((o * x["do"].double()).sum() + (S * x["dfinal"].double()).sum()).backward()
    r = R.backward(x)
    for n, m in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("g", "dg"), ("beta", "dbeta"), ("init", "dinit")):
        assert torch.allclose(y[n].grad, r[m], rtol=1e-11, atol=1e-12), n


def test_reference_gradients_are_differences():
    x = R.make(1, 1, 2, 6, 4, 3, F32, 2, init=True, final=True)
    x = {n: t.double() if t is not None and t.is_floating_point() else t for n, t in x.items()}

    def loss(y):
        o, S = R.forward(y)
        return float((o * x["do"]).sum() + (S * x["dfinal"]).sum())

    r, h = R.backward(x), 1e-4
    gen = torch.Generator().manual_seed(0)
    for n, m in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("g", "dg"), ("beta", "dbeta"), ("init", "dinit")):
        z = torch.randn(x[n].shape, generator=gen, dtype=torch.float64)
        f = lambda s: loss(dict(x, **{n: x[n] + s * z}))  # noqa: E731,B023
        diff = (8 * (f(h) - f(-h)) - (f(2 * h) - f(-2 * h))) / (12 * h)  # error O(h^4) = 1e-16, roundings 1e-16 / h
        assert abs(diff - float((r[m] * z).sum())) <= 1e-9, n


def test_reference_without_overlap_is_linear_attention():
    """Orthonormal keys with beta = 1 never correct one another: o_t = sum_s e^{G_t - G_s} (q_t . k_s) v_s."""
    x = R.make(1, 1, 1, 8, 8, 5, F32, 3)
    x["k"] = torch.linalg.qr(torch.randn(8, 8, dtype=torch.float64, generator=torch.Generator().manual_seed(1)))[0][None, None]
    x["beta"] = torch.ones(1, 1, 8)
    o, _ = R.forward(x)
    G = x["g"].double().cumsum(-1)[0, 0]
    M = (G[:, None] - G[None]).exp().tril()
    want = (x["q"][0, 0].double() @ x["k"][0, 0].T * M) @ x["v"][0, 0].double()
    assert torch.allclose(o[0, 0], want, rtol=1e-12, atol=1e-13)


# ------------------------------------------------------------------------------------------------ CPU: refusals

FAKE = 1 << 20


@pytest.fixture(scope="module")
def lib():
    from causal_linear_attention_la2_b200 import build
    build.build()
    return L.load()


def _raw_fwd(**kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, beta=FAKE, out=FAKE, init=0, fin=0, lens=0, B=1, Hk=1, H=2, T=64, d=64, e=64,
             dtype=1, out_dtype=1, layout=0, ws=FAKE, n=1 << 40)
    a.update(kw)
    return L.la2_gdr_fwd_raw(*a.values())


def _raw_bwd(**kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, beta=FAKE, dout=FAKE, init=0, dfinal=0, dq=FAKE, dk=FAKE, dv=FAKE, dg=FAKE,
             dbeta=FAKE, dinit=0, lens=0, B=1, Hk=1, H=2, T=64, d=64, e=64, dtype=1, out_dtype=1, layout=0, ws=FAKE,
             n=1 << 40)
    a.update(kw)
    return L.la2_gdr_bwd_raw(*a.values())


def _raw_decode(**kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, beta=FAKE, states=FAKE, slots=0, n_slots=4, out=FAKE, B=1, Hk=1, H=2, d=64,
             e=64, dtype=1)
    a.update(kw)
    return L.la2_gdr_decode_raw(*a.values())


def _raw_copy(**kw):
    a = dict(states=FAKE, src=FAKE, dst=FAKE, n=2, n_slots=4, elems=64)
    a.update(kw)
    return L.la2_state_copy_raw(*a.values())


SIZES = [dict(B=-1), dict(Hk=-1), dict(H=-2), dict(Hk=0), dict(H=3, Hk=2), dict(d=0), dict(e=0), dict(dtype=5)]


@pytest.mark.parametrize("kw", SIZES + [dict(T=-1), dict(out_dtype=3), dict(layout=2), dict(layout=-1)])
def test_sequence_calls_refuse_sizes(lib, kw):
    assert _raw_fwd(**kw) == L.LA2_ERR_INVALID_ARG
    assert _raw_bwd(**kw) == L.LA2_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", SIZES + [dict(n_slots=-1)])
def test_decode_refuses_sizes(lib, kw):
    assert _raw_decode(**kw) == L.LA2_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(d=129), dict(e=200)])
def test_wide_heads_are_unsupported(lib, kw):
    for call in (_raw_fwd, _raw_bwd, _raw_decode):
        assert call(**kw) == L.LA2_ERR_UNSUPPORTED
    assert _raw_fwd(dtype=0) == L.LA2_ERR_UNSUPPORTED  # bf16 outputs of fp32 inputs
    assert _raw_bwd(dtype=0) == L.LA2_ERR_UNSUPPORTED


def test_more_rows_than_a_grid_holds_are_unsupported(lib):
    assert _raw_fwd(B=1 << 14, H=1 << 13, T=1 << 20) == L.LA2_ERR_UNSUPPORTED
    assert L.la2_gdr_workspace_bytes(1 << 14, 1, 1 << 13, 1 << 20, 64, 64, 1, 1) == (1 << 64) - 1


@pytest.mark.parametrize("T", [2 ** 31 - 1, 2 ** 31 - 63])
@pytest.mark.parametrize("d,dtype", [(1, 1), (1, 0), (64, 1)])
def test_rows_whose_numbers_pass_32_bits_are_unsupported(lib, T, d, dtype):
    """The kernels step 16, 32 or 64 rows past a sequence's last one, in 32 bits."""
    kw = dict(B=1, Hk=1, H=1, T=T, d=d, e=d, dtype=dtype, out_dtype=0)
    assert _raw_fwd(**kw) == L.LA2_ERR_UNSUPPORTED
    assert _raw_bwd(**kw) == L.LA2_ERR_UNSUPPORTED
    assert L.la2_gdr_workspace_bytes(1, 1, 1, T, d, d, dtype, 1) == (1 << 64) - 1
    assert L.la2_gdr_workspace_bytes(1, 1, 1, 2 ** 31 - 64, d, d, dtype, 1) < 1 << 62


@pytest.mark.parametrize("name", ["q", "k", "v", "beta", "out"])
def test_forward_refuses_null_and_misaligned(lib, name):
    assert _raw_fwd(**{name: 0}) == L.LA2_ERR_INVALID_ARG
    assert _raw_fwd(**{name: FAKE + (2 if name == "beta" else 8)}) == L.LA2_ERR_INVALID_ARG


@pytest.mark.parametrize("name", ["q", "k", "v", "beta", "dout", "dq", "dk", "dv", "dbeta"])
def test_backward_refuses_null_and_misaligned(lib, name):
    assert _raw_bwd(**{name: 0}) == L.LA2_ERR_INVALID_ARG
    assert _raw_bwd(**{name: FAKE + (2 if name in ("beta", "dbeta") else 8)}) == L.LA2_ERR_INVALID_ARG


@pytest.mark.parametrize("name", ["init", "lens", "g"])
def test_optional_pointers_refuse_misalignment(lib, name):
    for call in (_raw_fwd, _raw_bwd):
        assert call(**{name: FAKE + 2}) == L.LA2_ERR_INVALID_ARG


def test_gate_gradient_needs_a_gate(lib):
    assert _raw_bwd(g=0) == L.LA2_ERR_INVALID_ARG


def test_workspace_is_checked(lib):
    need = L.la2_gdr_workspace_bytes(1, 1, 2, 64, 64, 64, 1, 1)
    assert need > 0
    assert _raw_bwd(ws=0, n=0) == L.LA2_ERR_WORKSPACE
    assert _raw_bwd(n=need - 1) == L.LA2_ERR_WORKSPACE
    assert _raw_bwd(ws=FAKE + 16) == L.LA2_ERR_INVALID_ARG


def test_empty_problems(lib):
    for kw in (dict(B=0), dict(H=0), dict(H=0, Hk=0), dict(T=0)):
        assert _raw_fwd(**{n: 0 for n in ("q", "k", "v", "g", "beta", "out")}, **kw) == L.LA2_OK
        assert _raw_bwd(**{n: 0 for n in ("q", "k", "v", "g", "beta", "dout", "dq", "dk", "dv", "dg", "dbeta")},
                        **kw) == L.LA2_OK
    assert _raw_decode(B=0, q=0, states=0) == L.LA2_OK
    assert _raw_copy(n=0, states=0, src=0, dst=0) == L.LA2_OK
    assert _raw_copy(n_slots=0, states=0) == L.LA2_OK


@pytest.mark.parametrize("name", ["q", "k", "v", "beta", "out", "states"])
def test_decode_refuses_null_and_misaligned(lib, name):
    assert _raw_decode(**{name: 0}) == L.LA2_ERR_INVALID_ARG
    assert _raw_decode(**{name: FAKE + 1}) == L.LA2_ERR_INVALID_ARG


def test_copy_refuses(lib):
    for kw in (dict(n=-1), dict(n_slots=-1), dict(elems=-1), dict(states=0), dict(src=0), dict(dst=0),
               dict(states=FAKE + 2), dict(src=FAKE + 1), dict(dst=FAKE + 2)):
        assert _raw_copy(**kw) == L.LA2_ERR_INVALID_ARG
    assert _raw_copy(n=4097) == L.LA2_ERR_UNSUPPORTED


def test_the_binding_refuses_cpu_tensors():
    z = torch.zeros(1, 1, 4, 8)
    with pytest.raises(ValueError):
        L.la2_gdr_fwd(z, z, z, None, z[..., 0])
    with pytest.raises(ValueError):
        L.la2_gdr_bwd(z, z, z, None, z[..., 0], z)
    with pytest.raises(ValueError):
        L.la2_gdr_decode(z[0], z[0], z[0], None, z[0, ..., 0], z)
    with pytest.raises(ValueError):
        L.la2_state_copy(z, torch.zeros(1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))


# ------------------------------------------------------------------------------------------------ GPU

@pytest.fixture(scope="module")
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from causal_linear_attention_la2_b200 import build
    build.build()
    L.load()
    return torch.device("cuda")


def _put(x, layout, dev):
    """The call's tensors on the device; NaN behind each sequence's end."""
    y = {}
    for n, t in x.items():
        if t is None:
            y[n] = None
            continue
        if n in ("q", "k", "v", "do", "g", "beta"):
            if x["lens"] is not None:
                t = t.clone()
                for b, m in enumerate(x["lens"].tolist()):
                    t[b, :, max(0, m):] = float("nan")
            if layout == "bthd":
                t = t.transpose(1, 2)
        y[n] = t.contiguous().to(dev)
    return y


def _back(t, layout):
    t = t.detach().double().cpu()
    return t.transpose(1, 2) if layout == "bthd" else t


def _close(got, want, tol, extra=0.0, name=""):
    """|err| <= tol (rms(want) + extra) + OWN |want|, one bf16 rounding more where `got` is bf16."""
    assert torch.isfinite(got).all(), name
    if not want.numel():
        return
    rms = _rms(want) + extra
    near = tol * rms + OWN[tol] * want.abs()
    if name.endswith("bf16"):  # one rounding of a value that is this near
        near = near * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs()
    over = float(((got - want).abs() - near).max())
    assert over <= 1e-30, f"{name}: {over:.3e} over, rms {rms:.3e}, largest error {float((got - want).abs().max()):.3e}"


def _rms(t):
    return float(t.square().mean().sqrt())


def _check_fwd(dev, x, layout="bhtd", out_dtype=None, cancel=0.0):
    """`cancel`: how many times rms(exact) the terms' roundings come to where large terms cancel."""
    y = _put(x, layout, dev)
    o, S = L.la2_gdr_fwd(y["q"], y["k"], y["v"], y["g"], y["beta"], layout=layout, init_state=y["init"],
                         seq_lens=y["lens"], want_final=True, out_dtype=out_dtype)
    ro, rS = R.forward(x)
    tol = TOL[x["q"].dtype]
    _close(_back(o, layout), ro, tol, cancel * _rms(ro), name="o" + ("bf16" if out_dtype == BF16 else ""))
    _close(S.double().cpu(), rS, tol, cancel * _rms(rS), name="state")


def _check_bwd(dev, x, layout="bhtd", out_dtype=None, cancel=0.0):
    y = _put(x, layout, dev)
    got = L.la2_gdr_bwd(y["q"], y["k"], y["v"], y["g"], y["beta"], y["do"], layout=layout, init_state=y["init"],
                        d_final_state=y["dfinal"], seq_lens=y["lens"], want_d_init=True, out_dtype=out_dtype)
    r = R.backward(x)
    tol = TOL[x["q"].dtype]
    for n, t in zip(("dq", "dk", "dv", "dg", "dbeta", "dinit"), got):
        if t is None:
            assert n == "dg" and x["g"] is None
            continue
        extra = 8 * _rms(r["mag"]) if n == "dg" else cancel * _rms(r[n])
        half = out_dtype == BF16 and n in ("dq", "dk", "dv")
        _close(t.double().cpu() if n == "dinit" else _back(t, layout), r[n], tol, extra, n + ("bf16" if half else ""))


LENGTHS = [1, 2, 15, 16, 17, 33, 63, 64, 65, 127, 128, 130, 200]


@pytest.mark.gpu
@pytest.mark.parametrize("T", LENGTHS)
@pytest.mark.parametrize("dtype,d,e", [(BF16, 64, 64), (BF16, 128, 128), (F32, 64, 64), (F32, 33, 20)])
def test_lengths(gpu, dtype, d, e, T):
    x = R.make(2, 1, 2, T, d, e, dtype, T + d, init=T % 2 == 0, final=T % 3 == 0)
    _check_fwd(gpu, x)
    _check_bwd(gpu, x)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d,e", [(BF16, 64, 128), (BF16, 128, 64), (BF16, 1, 1), (BF16, 72, 100), (BF16, 128, 17),
                                       (F32, 1, 1), (F32, 128, 128), (F32, 3, 128), (F32, 127, 5), (F32, 128, 16)])
@pytest.mark.parametrize("layout", ["bhtd", "bthd"])
def test_widths_and_layouts(gpu, dtype, d, e, layout):
    x = R.make(2, 2, 4, 77, d, e, dtype, d * 3 + e, init=True, final=True)
    _check_fwd(gpu, x, layout)
    _check_bwd(gpu, x, layout)


@pytest.mark.gpu
@pytest.mark.parametrize("out_dtype", [F32, BF16])
@pytest.mark.parametrize("layout", ["bhtd", "bthd"])
@pytest.mark.parametrize("d,e", [(64, 64), (128, 128), (64, 128), (40, 24)])
def test_output_types(gpu, d, e, layout, out_dtype):
    x = R.make(1, 2, 2, 100, d, e, BF16, 5, init=True, final=True)
    _check_fwd(gpu, x, layout, out_dtype)
    _check_bwd(gpu, x, layout, out_dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("Hk,H", [(1, 1), (1, 4), (3, 3), (2, 6), (5, 5)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_heads(gpu, dtype, Hk, H):
    x = R.make(3, Hk, H, 70, 64, 64, dtype, H, final=True)
    _check_fwd(gpu, x)
    _check_bwd(gpu, x)


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["bhtd", "bthd"])
@pytest.mark.parametrize("dtype,d,e", [(BF16, 64, 64), (BF16, 128, 128), (F32, 24, 40)])
def test_ragged_batches_leave_rows_behind_the_end(gpu, dtype, d, e, layout):
    """Lengths of 0, 1, chunk borders and beyond T; NaN in the inputs and a mark in the outputs behind each end."""
    lens = [0, 1, 64, 65, 131, 32, -3, 1000]
    T = 131
    x = R.make(len(lens), 1, 2, T, d, e, dtype, 9, init=True, final=True, lens=lens)
    _check_fwd(gpu, x, layout)
    _check_bwd(gpu, x, layout)
    y = _put(x, layout, gpu)
    mark = 7.0
    for odt in {F32, dtype}:
        like = lambda t, dt=odt: torch.full(t.shape, mark, dtype=dt, device=gpu)  # noqa: E731,B023
        o = like(y["v"])
        L.la2_gdr_fwd(y["q"], y["k"], y["v"], y["g"], y["beta"], layout=layout, seq_lens=y["lens"], out=o, out_dtype=odt)
        outs = dict(dq=like(y["q"]), dk=like(y["k"]), dv=like(y["v"]), dg=like(y["g"], F32), dbeta=like(y["beta"], F32))
        L.la2_gdr_bwd(y["q"], y["k"], y["v"], y["g"], y["beta"], y["do"], layout=layout, seq_lens=y["lens"],
                      out_dtype=odt, **outs)
        _marked(dict(outs, o=o), layout, lens, T, mark)


def _marked(outs, layout, lens, T, mark):
    for name, t in outs.items():
        t = t.transpose(1, 2) if layout == "bthd" else t
        for b, m in enumerate(lens):
            m = min(max(m, 0), T)
            assert (t[b, :, m:] == mark).all(), name
            assert torch.isfinite(t[b, :, :m]).all(), name


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d", [(BF16, 64), (BF16, 128), (F32, 48)])
def test_without_a_gate(gpu, dtype, d):
    x = R.make(2, 2, 2, 150, d, d, dtype, 4, gate=False, init=True, final=True)
    _check_fwd(gpu, x)
    _check_bwd(gpu, x)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d", [(BF16, 64), (BF16, 128), (F32, 48)])
def test_extreme_gates_and_strengths(gpu, dtype, d):
    """Gates of -inf, -1e30 and 0 (forget all, keep all), beta of 0 and 1, repeated and zero keys."""
    x = R.make(2, 1, 2, 140, d, d, dtype, 8, init=True, final=True)
    x["g"][:, :, 3] = -float("inf")
    x["g"][:, :, 64] = -1e30
    x["g"][:, :, 66:75] = -300.0
    x["g"][:, :, 100:] = 0.0
    x["beta"][:, :, 5:9] = 0.0
    x["beta"][:, :, 20:40] = 1.0
    x["beta"][:, :, 63] = 0.0
    x["k"][:, :, 20:36] = x["k"][:, :, 20:21]
    x["k"][:, :, 50] = 0.0
    _check_fwd(gpu, x)
    # the reference's product exp(-inf) * S is 0 and its gradients are finite
    _check_bwd(gpu, x)


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["bhtd", "bthd"])
@pytest.mark.parametrize("dtype,d,e,T,at", [(BF16, 64, 64, 150, 70), (BF16, 128, 128, 150, 70), (BF16, 128, 64, 150, 149),
                                            (BF16, 64, 128, 150, 0), (BF16, 72, 100, 150, 70), (F32, 64, 64, 150, 70),
                                            (F32, 128, 20, 40, 39), (BF16, 128, 128, 2200, 1000)])
def test_a_nan_gate_is_seen(gpu, dtype, d, e, T, at, layout):
    """One gate that is NaN: every row from it on, the final state and the gradients that depend on it are NaN; what does
    not depend on it is, bit by bit, what it is without (by chunks of 64 rows, the other rows of its chunk aside)."""
    x = R.make(3, 1, 2, T, d, e, dtype, 60, init=True, final=True)
    runs = []
    for bad in (False, True):
        z = dict(x)
        if bad:
            z["g"] = x["g"].clone()
            z["g"][1, 0, at] = float("nan")
        y = _put(z, layout, gpu)
        a = (y["q"], y["k"], y["v"], y["g"], y["beta"])
        o, S = L.la2_gdr_fwd(*a, layout=layout, init_state=y["init"], want_final=True)
        gr = L.la2_gdr_bwd(*a, y["do"], layout=layout, init_state=y["init"], d_final_state=y["dfinal"], want_d_init=True)
        runs.append([_back(o, layout), S.double().cpu(), *(_back(t, layout) for t in gr[:5]), gr[5].double().cpu()])
    first = at // 64 * 64  # first row of the chunk
    for name, c, n in zip(("o", "S", "dq", "dk", "dv", "dg", "dbeta", "dinit"), *runs):
        assert torch.isfinite(c).all(), name
        others = [0, 2]
        assert torch.equal(n[others], c[others]), name
        if name in ("dq", "dk"):  # sums over the two value heads
            continue
        assert torch.equal(n[1, 1], c[1, 1]), name
    o, S, dq, dk, dv, dg, db, dinit = runs[1]
    assert torch.isnan(o[1, 0, at:]).all() and torch.equal(o[1, 0, :first], runs[0][0][1, 0, :first])
    assert torch.isnan(S[1, 0]).all() and torch.isnan(dinit[1, 0]).all()
    assert torch.isnan(dq[1, 0, at:]).all()
    for t in (dk[1, 0], dv[1, 0], db[1, 0], dg[1, 0]):
        assert torch.isnan(t[:at]).all()
    assert torch.isnan(dg[1, 0, at]) and torch.isnan(db[1, 0, at])
    assert torch.equal(dv[1, 0, first + 64:], runs[0][4][1, 0, first + 64:])


@pytest.mark.gpu
@pytest.mark.parametrize("B", [3, 200])
def test_a_nan_gate_is_seen_by_a_step(gpu, B):
    x = R.make(B, 1, 2, 1, 64, 64, F32, 61)
    one = {n: x[n][:, :, 0].contiguous().to(gpu) for n in ("q", "k", "v", "g", "beta")}
    one["g"][1, 0] = float("nan")
    pool = torch.randn(B, 2, 64, 64, device=gpu)
    o = L.la2_gdr_decode(one["q"], one["k"], one["v"], one["g"], one["beta"], pool)
    for t in (o, pool):
        assert torch.isnan(t[1, 0]).all()
        t[1, 0] = 0.0
        assert torch.isfinite(t).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d,e", [(BF16, 64, 64), (BF16, 128, 64), (BF16, 64, 128), (BF16, 128, 128), (F32, 48, 48)])
def test_gate_gradient_where_the_gate_closes(gpu, dtype, d, e):
    """One row that forgets the state before it, whose product with the gradient is all that the row wrote: dg is
    c - c = 0 with c = k . dS1 u.

    Both c are sums of the same d products of k_i and (dS1 u)_i, one of them over up to 64 partial sums in another order:
    64 roundings of at most 2^-24 (2^-24 / sqrt(3) on average) of a partial sum no larger than c as a rule add up to
    sqrt(64) 2^-24 = 4.8e-7 of c on average over many heads.  A c from operands of two bf16 parts would be off by
    2e-6."""
    x = R.make(4, 1, 64, 1, d, e, dtype, 21, init=True, final=True)
    x["g"][:] = -60.0
    x["do"][:] = 0.0
    y = _put(x, "bhtd", gpu)
    got = L.la2_gdr_bwd(y["q"], y["k"], y["v"], y["g"], y["beta"], y["do"], init_state=y["init"], d_final_state=y["dfinal"])
    u = x["beta"].double()[..., None] * x["v"].double()  # [B, H, 1, e]
    c = torch.einsum("bhi,bhij,bhj->bh", x["k"].double().expand(4, 64, 1, d)[:, :, 0], x["dfinal"].double(), u[:, :, 0])
    assert _rms(got[3].double().cpu()) <= 4.8e-7 * _rms(c)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_correlated_keys(gpu, dtype):
    """Keys close to one another with beta near 1: every position corrects nearly all of the ones before it.

    u_t is then about v_t - v_{t-1}, sqrt(2) times v_t's size, and an output or gradient the telescoping sum of up to 64
    such terms of one chunk (earlier chunks come as a state that is one), no larger than one of them: their roundings
    add up to sqrt(64) sqrt(2) = 11 times those of one."""
    x = R.make(1, 1, 2, 192, 64, 64, dtype, 11, gate=False)
    base = torch.randn(1, 1, 1, 64, generator=torch.Generator().manual_seed(3))
    k = base / base.norm() + 0.1 * x["k"].float()
    x["k"] = (k / k.norm(dim=-1, keepdim=True)).to(dtype)
    x["beta"] = torch.full_like(x["beta"], 0.98)
    _check_fwd(gpu, x, cancel=11.0)
    _check_bwd(gpu, x, cancel=11.0)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d,cut", [(BF16, 128, 64), (BF16, 64, 37), (F32, 50, 37)])
def test_pieces_are_the_whole(gpu, dtype, d, cut):
    """Forward and backward over two pieces with handed-on states against the reference over the whole."""
    T = 150
    x = R.make(2, 1, 2, T, d, d, dtype, 13, init=True, final=True)
    y = _put(x, "bhtd", gpu)
    part = lambda a, b: {n: (t[:, :, a:b].contiguous() if n in ("q", "k", "v", "do", "g", "beta") else t)  # noqa: E731
                         for n, t in y.items()}
    p, q = part(0, cut), part(cut, T)
    o1, S1 = L.la2_gdr_fwd(p["q"], p["k"], p["v"], p["g"], p["beta"], init_state=y["init"], want_final=True)
    o2, S2 = L.la2_gdr_fwd(q["q"], q["k"], q["v"], q["g"], q["beta"], init_state=S1, want_final=True)
    g2 = L.la2_gdr_bwd(q["q"], q["k"], q["v"], q["g"], q["beta"], q["do"], init_state=S1, d_final_state=y["dfinal"],
                       want_d_init=True)
    g1 = L.la2_gdr_bwd(p["q"], p["k"], p["v"], p["g"], p["beta"], p["do"], init_state=y["init"], d_final_state=g2[5],
                       want_d_init=True)
    ro, rS = R.forward(x)
    r, tol = R.backward(x), TOL[dtype]
    _close(torch.cat([o1, o2], 2).double().cpu(), ro, tol, name="o")
    _close(S2.double().cpu(), rS, tol, name="state")
    for i, n in enumerate(("dq", "dk", "dv", "dg", "dbeta")):
        extra = 8 * _rms(r["mag"]) if n == "dg" else 0.0
        _close(torch.cat([g1[i], g2[i]], 2).double().cpu(), r[n], tol, extra, n)
    _close(g1[5].double().cpu(), r["dinit"], tol, name="dinit")


@pytest.mark.gpu
@pytest.mark.parametrize("B,Hk,H,T,d,lens", [(1, 1, 1, 2100, 128, None), (1, 1, 2, 1030, 64, None),
                                             (3, 1, 2, 1500, 128, [1500, 0, 700])])
def test_long_sequences_in_segments(gpu, B, Hk, H, T, d, lens):
    """Few long sequences, which the forward walks in segments: ragged ends, an empty sequence, carried states."""
    x = R.make(B, Hk, H, T, d, 128, BF16, 23, init=True, lens=lens)
    x["g"] *= 0.1  # states that last over many chunks
    _check_fwd(gpu, x)


def _segments(B, H, T, d):
    """Segments of the forward walk, from the states that the workspace holds for them (e = 64 is not cut)."""
    need = [L.la2_gdr_workspace_bytes(B, 1, H, T, d, e, L.LA2_DTYPE_BF16, 0) for e in (128, 64)]
    return 1 + (need[0] - need[1]) // (B * H * 3 * d * 128 * 4)


def _on(dev, f, x):
    """A function of gdr_ref in 64 bits on the device."""
    with torch.device(dev):
        r = f({n: t if t is None else t.to(dev) for n, t in x.items()})
    return {n: t.cpu() for n, t in r.items()} if isinstance(r, dict) else [t.cpu() for t in r]


@pytest.mark.gpu
@pytest.mark.parametrize("d,B,H,T,lens,final", [
    (64, 1, 1, 2100, None, True), (128, 1, 2, 2112, None, False), (128, 1, 1, 19195, None, True), (64, 1, 1, 9000, None, True),
    (64, 6, 1, 2100, [2100, 0, 1, 576, 577, 1190], True), (128, 6, 1, 2100, [575, 0, 2100, 1152, 640, 1], True),
    (128, 2, 2, 2100, [64, 1700], False), (64, 2, 3, 2100, [0, 0], True)])
def test_segments_of_long_sequences(gpu, d, B, H, T, lens, final):
    """Batches that the plan does cut: lengths of 0, 1, a segment's border (9 chunks) and beside it, ends inside a segment
    and segments behind an end, states in and out, both layouts and output types."""
    assert _segments(B, H, T, d) > 3
    x = R.make(B, 1, H, T, d, 128, BF16, 24, init=True, lens=lens)
    x["g"] *= 0.1  # states that last over many chunks
    ro, rS = _on(gpu, R.forward, x)
    for layout in ("bhtd", "bthd"):
        y = _put(x, layout, gpu)
        for odt in (F32, BF16):
            o = L.la2_gdr_fwd(y["q"], y["k"], y["v"], y["g"], y["beta"], layout=layout, init_state=y["init"],
                              seq_lens=y["lens"], want_final=final, out_dtype=odt)
            if final:
                o, S = o
                _close(S.double().cpu(), rS, TOL[BF16], name="state")
            _close(_back(o, layout), ro, TOL[BF16], name="o" + ("bf16" if odt == BF16 else ""))


def _check_all(dev, x, layout):
    """Forward and backward of many elements against the reference on the device: rms(err) <= 1.1e-5 rms(exact) over the
    rows that exist.

    An operand of two bf16 parts is off by at most 2^-17 of itself (half a step of the second part) and by 2^-17 / sqrt(3)
    on average, a product of two of them by 6.2e-6, an element that is three such products deep (a state, the rows w or x,
    a gradient) by sqrt(3) 6.2e-6 = 1.1e-5 of its size on average.  (The largest error has no such bound: the terms are
    products of normal numbers, some elements the difference of two large ones.)  One element in 10^6 that is off by 2% of
    rms would show."""
    y = _put(x, layout, dev)
    a = (y["q"], y["k"], y["v"], y["g"], y["beta"])
    lens = [x["v"].shape[2]] * len(x["v"]) if x["lens"] is None else x["lens"].tolist()
    live = lambda t: torch.cat([t[b, :, :n].flatten() for b, n in enumerate(lens)])  # noqa: E731

    def near(t, want, name, extra=0.0):
        err, size = _rms(t - want), _rms(want) + extra
        assert err <= 1.1e-5 * size, f"{name}: {err:.3e} of {size:.3e}"

    def rows(t, want, name, extra=0.0):
        t = _back(t, layout)
        for b, n in enumerate(lens):
            assert not t[b, :, n:].any(), name
        near(live(t), live(want), name, extra)

    ro, rS = _on(dev, R.forward, x)
    o, S = L.la2_gdr_fwd(*a, layout=layout, init_state=y["init"], seq_lens=y["lens"], want_final=True)
    rows(o, ro, "o")
    near(S.double().cpu(), rS, "state")
    r = _on(dev, R.backward, x)
    got = L.la2_gdr_bwd(*a, y["do"], layout=layout, init_state=y["init"], d_final_state=y["dfinal"], seq_lens=y["lens"],
                        want_d_init=True)
    for n, t in zip(("dq", "dk", "dv", "dg", "dbeta"), got):
        rows(t, r[n], n, 8 * _rms(live(r["mag"])) if n == "dg" else 0.0)
    near(got[5].double().cpu(), r["dinit"], "dinit")


@pytest.mark.gpu
@pytest.mark.parametrize("lens", [None, [600, 0, 65, 130, 599, 320]])
@pytest.mark.parametrize("H", [4, 12])
@pytest.mark.parametrize("d,e,layout", [(64, 64, "bhtd"), (128, 64, "bthd"), (64, 128, "bhtd"), (128, 128, "bthd")])
def test_more_chunks_than_sms(gpu, d, e, layout, H, lens):
    """240 chunks of key heads, so that CTAs of the gradients take a second one, chunks behind an end passed over."""
    _check_all(gpu, R.make(6, 4, H, 600, d, e, BF16, 25, init=True, final=True, lens=lens), layout)


@pytest.mark.gpu
@pytest.mark.parametrize("d,e,layout", [(64, 64, "bthd"), (128, 64, "bhtd"), (64, 128, "bthd"), (128, 128, "bhtd")])
def test_many_ragged_ends(gpu, d, e, layout):
    """800 chunks of key heads of short sequences: a CTA of the gradients meets several that end inside a chunk."""
    lens = torch.randint(0, 101, (50,), generator=torch.Generator().manual_seed(5)).tolist()
    _check_all(gpu, R.make(50, 8, 8, 100, d, e, BF16, 26, init=True, final=True, lens=lens), layout)


@pytest.mark.gpu
@pytest.mark.parametrize("d,e,lens", [(128, 128, None), (64, 64, [1400, 1337]), (64, 128, [1281, 1400]), (128, 64, None)])
def test_sequences_of_many_chunks(gpu, d, e, lens):
    """22 chunks a sequence, forward and backward; gates near 0, so that states last over many of them."""
    x = R.make(2, 4, 4, 1400, d, e, BF16, 27, init=True, final=True, lens=lens)
    x["g"] *= 0.1
    _check_all(gpu, x, "bhtd")


@pytest.mark.gpu
@pytest.mark.parametrize("d,e", [(64, 64), (128, 64), (64, 128), (128, 128)])
def test_gate_gradient_of_a_first_row_without_a_state(gpu, d, e):
    """The first gate of a sequence that starts from nothing multiplies zeros: dg is 0, the difference of sums over the
    rows t of q_t . dq_t, k_t . row_t and k_t . col_t (what the row reads and what it writes), in which every pair of rows
    appears twice.

    The two appearances are made of the same operands, so what differs are the roundings of sums in fp32: an element of a
    row is a sum over 64 rows, a term one over up to 128 elements, dg one over 64 rows: 256 roundings of at most 2^-24,
    sqrt(256) 2^-24 = 9.5e-7 of a term, random between the 3 x 64 terms, so 9.5e-7 sqrt(sum of their squares), for which
    `mag` (the sum of a row's terms) stands.  Keys are all the same, where the pairs' terms are largest: from operands of
    their own, each of two bf16 parts, the 2016 pairs would be off by 1e-6 sqrt(2016) of one each, 5e-6 of that root."""
    T = 64
    x = R.make(4, 1, 32, T, d, e, BF16, 28)
    x["k"] = x["k"][:, :, :1].expand(4, 1, T, d).contiguous()
    x["g"] *= 0.1
    y = _put(x, "bhtd", gpu)
    dg = L.la2_gdr_bwd(y["q"], y["k"], y["v"], y["g"], y["beta"], y["do"])[3]
    r = _on(gpu, R.backward, x)
    assert float(r["dg"][:, :, 0].abs().max()) <= 1e-12
    terms = float(r["mag"].square().sum(-1).mean().sqrt())
    assert _rms(dg[:, :, 0].double().cpu()) <= 9.5e-7 * terms


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d,e", [(F32, 8, 8), (BF16, 64, 64), (BF16, 128, 128), (BF16, 64, 128)])
def test_empty_sequences_hand_states_on(gpu, dtype, d, e):
    s = torch.randn(2, 2, d, e, device=gpu)
    z, v = (torch.zeros(2, 2, 0, n, device=gpu, dtype=dtype) for n in (d, e))
    g = torch.zeros(2, 2, 0, device=gpu)
    o, S = L.la2_gdr_fwd(z, z, v, g, g, init_state=s, want_final=True)
    assert o.numel() == 0 and torch.equal(S, s)
    assert torch.equal(L.la2_gdr_bwd(z, z, v, g, g, v, d_final_state=s, want_d_init=True)[5], s)
    S = L.la2_gdr_fwd(z, z, v, None, g, want_final=True)[1]
    assert not S.any()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d", [(BF16, 128), (BF16, 64), (F32, 30)])
def test_runs_are_bitwise_repeatable(gpu, dtype, d):
    x = R.make(2, 2, 4, 260, d, d, dtype, 17, init=True, final=True)
    y = _put(x, "bhtd", gpu)
    a, b = ([*L.la2_gdr_fwd(y["q"], y["k"], y["v"], y["g"], y["beta"], want_final=True),
             *L.la2_gdr_bwd(y["q"], y["k"], y["v"], y["g"], y["beta"], y["do"], want_d_init=True)] for _ in range(2))
    for s, t in zip(a, b):
        assert torch.equal(s, t)


# ---- decode

@pytest.mark.gpu
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("dtype,d,e,Hk,H", [(BF16, 128, 128, 2, 4), (BF16, 64, 64, 3, 3), (F32, 64, 64, 1, 2),
                                            (F32, 1, 1, 1, 1), (F32, 100, 72, 2, 2), (BF16, 128, 7, 1, 3),
                                            (F32, 5, 127, 1, 1), (F32, 128, 4, 1, 1), (BF16, 127, 126, 1, 1)])
def test_decode_step(gpu, dtype, d, e, Hk, H, gate):
    B, N = 5, 9
    x = R.make(B, Hk, H, 1, d, e, dtype, d + e, gate=gate)
    one = {n: (x[n][:, :, 0].contiguous() if x[n] is not None else None) for n in ("q", "k", "v", "g", "beta")}
    pool = torch.randn(N, H, d, e, generator=torch.Generator().manual_seed(1))
    slots = torch.tensor([7, -1, 2, 9, 0], dtype=torch.int32)
    dp = pool.to(gpu)
    dev = {n: (t.to(gpu) if t is not None else None) for n, t in one.items()}
    o = L.la2_gdr_decode(dev["q"], dev["k"], dev["v"], dev["g"], dev["beta"], dp, slots=slots.to(gpu))
    live = [0, 2, 4]
    at = slots[live].long()
    ro, rS = R.decode(*(None if one[n] is None else one[n][live] for n in ("q", "k", "v", "g", "beta")), pool[at])
    # fp32 arithmetic whatever the inputs' type
    _close(o[live].double().cpu(), ro, 1e-5, name="o")
    _close(dp[at].double().cpu(), rS, 1e-5, name="state")
    rest = [i for i in range(N) if i not in at.tolist()]
    assert torch.equal(dp[rest].cpu(), pool[rest])
    assert not o[[1, 3]].any()


@pytest.mark.gpu
@pytest.mark.parametrize("B,Hk,H,d,e,dtype", [(40, 20, 20, 128, 128, BF16), (75, 4, 8, 64, 64, F32), (43, 7, 14, 100, 44, BF16),
                                              (150, 4, 4, 128, 36, F32), (300, 1, 2, 34, 120, BF16), (150, 2, 2, 64, 128, F32),
                                              (700, 1, 1, 128, 32, BF16), (1400, 1, 1, 16, 4, F32), (101, 3, 3, 1, 128, F32),
                                              (99, 3, 3, 128, 12, F32), (74, 4, 4, 33, 124, F32)])
def test_decode_of_many_states(gpu, B, Hk, H, d, e, dtype):
    """More states than the GPU holds at a time, padded and repeated slots among them."""
    N = B + 3
    x = R.make(B, Hk, H, 1, d, e, dtype, 3)
    one = {n: x[n][:, :, 0].contiguous() for n in ("q", "k", "v", "g", "beta")}
    pool = torch.randn(N, H, d, e, generator=torch.Generator().manual_seed(1))
    slots = torch.randperm(N, generator=torch.Generator().manual_seed(2))[:B].to(torch.int32)
    slots[3], slots[B // 2], slots[B - 1], slots[B - 2] = -1, slots[1], N, slots[B - 4]
    dead = [3, B // 2, B - 1, B - 2]
    live = [i for i in range(B) if i not in dead]
    dp, dev = pool.to(gpu), {n: t.to(gpu) for n, t in one.items()}
    o = L.la2_gdr_decode(dev["q"], dev["k"], dev["v"], dev["g"], dev["beta"], dp, slots=slots.to(gpu))
    at = slots[live].long()
    ro, rS = R.decode(*(one[n][live] for n in ("q", "k", "v", "g", "beta")), pool[at])
    _close(o[live].double().cpu(), ro, 1e-5, name="o")
    _close(dp[at].double().cpu(), rS, 1e-5, name="state")
    rest = [i for i in range(N) if i not in set(at.tolist())]
    assert torch.equal(dp[rest].cpu(), pool[rest]) and not o[dead].any()


@pytest.mark.gpu
def test_decode_same_slot_twice(gpu):
    """The first row that names a slot has it; later ones give zeros."""
    x = R.make(4, 1, 2, 1, 64, 64, F32, 2)
    one = {n: x[n][:, :, 0].contiguous() for n in ("q", "k", "v", "g", "beta")}
    pool = torch.randn(3, 2, 64, 64)
    dp, dev = pool.to(gpu), {n: t.to(gpu) for n, t in one.items()}
    slots = torch.tensor([1, 1, 0, 1], dtype=torch.int32, device=gpu)
    o = L.la2_gdr_decode(dev["q"], dev["k"], dev["v"], dev["g"], dev["beta"], dp, slots=slots)
    ro, rS = R.decode(*(one[n][[0, 2]] for n in ("q", "k", "v", "g", "beta")), pool[[1, 0]])
    _close(o[[0, 2]].double().cpu(), ro, 1e-5, name="o")
    _close(dp[[1, 0]].double().cpu(), rS, 1e-5, name="state")
    assert not o[[1, 3]].any() and torch.equal(dp[2].cpu(), pool[2])


@pytest.mark.gpu
def test_decode_without_slots_and_unaligned_pool(gpu):
    x = R.make(3, 2, 2, 1, 16, 20, F32, 2)
    one = {n: x[n][:, :, 0].contiguous().to(gpu) for n in ("q", "k", "v", "g", "beta")}
    flat = torch.randn(1 + 4 * 2 * 16 * 20, device=gpu)
    pool = flat[1:].view(4, 2, 16, 20)  # 4-byte aligned
    before = pool.clone()
    o = L.la2_gdr_decode(one["q"], one["k"], one["v"], one["g"], one["beta"], pool)
    ro, rS = R.decode(*(x[n][:, :, 0] for n in ("q", "k", "v", "g", "beta")), before[:3].cpu())
    _close(o.double().cpu(), ro, 1e-5, name="o")
    _close(pool[:3].double().cpu(), rS, 1e-5, name="state")
    assert torch.equal(pool[3], before[3])
    with pytest.raises(ValueError):
        L.la2_gdr_decode(one["q"], one["k"], one["v"], one["g"], one["beta"], pool[:2])


# ---- the state pool

def _copied(pool, src, dst):
    want = pool.clone()
    for s, t in zip(src, dst):
        if 0 <= t < len(pool) and s < len(pool):
            want[t] = pool[s] if s >= 0 else 0.0
    return want


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(2, 16, 16), (1, 1, 1), (3, 5, 7), (1, 128, 128), (40, 64, 64)])
@pytest.mark.parametrize("n", [1, 3, 17, 60])
def test_state_copy(gpu, shape, n):
    """Random pairs: chains, cycles, forks, clears, slots out of range and repeated destinations."""
    N = 41
    rng = np.random.RandomState(n)
    src = rng.randint(-2, N + 1, n).tolist()
    dst = rng.randint(-1, N + 1, n).tolist()
    pool = torch.randn(N, *shape, device=gpu)
    want = _copied(pool.cpu(), src, dst)
    i32 = dict(dtype=torch.int32, device=gpu)
    assert L.la2_state_copy(pool, torch.tensor(src, **i32), torch.tensor(dst, **i32)) is pool
    assert torch.equal(pool.cpu(), want)


@pytest.mark.gpu
@pytest.mark.parametrize("spare", [0, 5000])
@pytest.mark.parametrize("n,elems", [(257, 3), (1000, 16), (4096, 40), (4096, 9)])
def test_state_copy_of_many_pairs(gpu, n, elems, spare):
    """A rotation of the first n slots, then one destination for all pairs; pools with and without a table of slots."""
    N = n + spare
    flat = torch.randn(N * elems + 1, device=gpu)
    for pool in (flat[:N * elems].view(N, elems), flat[1:].view(N, elems)):
        i = torch.arange(n, dtype=torch.int32, device=gpu)
        before = pool.clone()
        L.la2_state_copy(pool, i, torch.roll(i, 1).contiguous())
        assert torch.equal(pool[torch.roll(i, 1).long()], before[:n]) and torch.equal(pool[n:], before[n:])
        before = pool.clone()
        L.la2_state_copy(pool, i, torch.full_like(i, 5))
        before[5] = before[n - 1]
        assert torch.equal(pool, before)


# ---- together, and how a program runs them

@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d", [(BF16, 128), (BF16, 64), (F32, 32)])
def test_prefill_fork_and_decode(gpu, dtype, d):
    """Two ragged prompts into slots, each forked, every branch continued token by token; against the reference over
    prompt and continuation."""
    B, H, P, G = 2, 2, 70, 5
    lens = [70, 33]
    x = R.make(B, 1, H, P, d, d, dtype, 21, lens=lens)
    y = _put(x, "bthd", gpu)
    _, S = L.la2_gdr_fwd(y["q"], y["k"], y["v"], y["g"], y["beta"], layout="bthd", seq_lens=y["lens"], want_final=True)
    pool = torch.full((6, H, d, d), float("nan"), device=gpu)
    pool[1], pool[4] = S[0], S[1]
    i32 = dict(dtype=torch.int32, device=gpu)
    L.la2_state_copy(pool, torch.tensor([1, 4, -1], **i32), torch.tensor([0, 5, 3], **i32))
    more = [R.make(4, 1, H, 1, d, d, dtype, 30 + i) for i in range(G)]
    slots = torch.tensor([1, 0, 4, 5], **i32)
    outs = []
    for m in more:
        t = {n: m[n][:, :, 0].contiguous().to(gpu) for n in ("q", "k", "v", "g", "beta")}
        outs.append(L.la2_gdr_decode(t["q"], t["k"], t["v"], t["g"], t["beta"], pool, slots=slots))
    for row, src in enumerate((0, 0, 1, 1)):
        n = lens[src]
        z = {m: torch.cat([x[m][src:src + 1, :, :n]] + [s[m][row:row + 1] for s in more], 2)
             for m in ("q", "k", "v", "do", "g", "beta")}
        ro, rS = R.forward(dict(z, init=None, lens=None))
        got = torch.stack([o[row] for o in outs], 1).double().cpu()
        _close(got, ro[0, :, n:], TOL[dtype], name="o")
        _close(pool[int(slots[row])].double().cpu(), rS[0], TOL[dtype], name="state")
    assert not pool[3].any() and torch.isnan(pool[2]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d", [(BF16, 128), (BF16, 64), (F32, 32)])
def test_calls_on_a_given_stream(gpu, dtype, d):
    """A stream argument: what the call allocates and clears is ordered on that stream."""
    x = R.make(3, 1, 2, 90, d, d, dtype, 50, final=True, lens=[90, 3, 0])
    y = _put(x, "bhtd", gpu)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    torch.cuda._sleep(20_000_000)  # the current stream is behind: work that lands on it comes too late
    o, S = L.la2_gdr_fwd(y["q"], y["k"], y["v"], y["g"], y["beta"], seq_lens=y["lens"], want_final=True, stream=side)
    dq = L.la2_gdr_bwd(y["q"], y["k"], y["v"], y["g"], y["beta"], y["do"], d_final_state=y["dfinal"],
                       seq_lens=y["lens"], stream=side)[0]
    side.synchronize()
    ro, rS = R.forward(x)
    _close(o.double().cpu(), ro, TOL[dtype], name="o")
    _close(S.double().cpu(), rS, TOL[dtype], name="state")
    _close(dq.double().cpu(), R.backward(x)["dq"], TOL[dtype], name="dq")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d", [(BF16, 128), (F32, 32)])
def test_two_streams_and_a_captured_step(gpu, dtype, d):
    """A forward and backward captured into a graph and replayed on new inputs, with other calls on another stream."""
    x = [R.make(2, 1, 2, 200, d, d, dtype, 40 + i, init=True, final=True) for i in range(2)]
    y = [_put(t, "bhtd", gpu) for t in x]

    def step(t):
        o, S = L.la2_gdr_fwd(t["q"], t["k"], t["v"], t["g"], t["beta"], init_state=t["init"], want_final=True)
        return [o, S, *L.la2_gdr_bwd(t["q"], t["k"], t["v"], t["g"], t["beta"], t["do"], init_state=t["init"],
                                     d_final_state=t["dfinal"], want_d_init=True)]

    want = [step(t) for t in y]
    torch.cuda.synchronize()
    held = {n: (t.clone() if t is not None else None) for n, t in y[0].items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(held)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for i in (1, 0):
        for n, t in held.items():
            if t is not None:
                t.copy_(y[i][n])
        graph.replay()
        with torch.cuda.stream(side):
            other = step(y[1 - i])
        torch.cuda.synchronize()
        for a, b in zip(got, want[i]):
            assert torch.equal(a, b)
        for a, b in zip(other, want[1 - i]):
            assert torch.equal(a, b)


@pytest.mark.gpu
def test_the_binding_refuses(gpu):
    x = _put(R.make(2, 1, 2, 8, 16, 16, F32, 1), "bhtd", gpu)
    a = (x["q"], x["k"], x["v"], x["g"], x["beta"])
    with pytest.raises(ValueError):
        L.la2_gdr_fwd(x["q"], x["k"][:, :, :4], *a[2:])
    with pytest.raises(ValueError):
        L.la2_gdr_fwd(x["q"], x["k"], x["v"], x["g"], x["beta"].transpose(1, 2))
    with pytest.raises(ValueError):
        L.la2_gdr_fwd(*a, layout="tbhd")
    with pytest.raises(TypeError):
        L.la2_gdr_fwd(x["q"].half(), *a[1:])
    with pytest.raises(TypeError):
        L.la2_gdr_fwd(x["q"], x["k"].bfloat16(), *a[2:])
    with pytest.raises(TypeError):
        L.la2_gdr_fwd(*a, seq_lens=torch.tensor([8, 8], device=gpu))
    with pytest.raises(L.LA2Error):
        L.la2_gdr_fwd(*a, out_dtype=BF16)  # fp32 inputs
    with pytest.raises(ValueError):
        L.la2_gdr_bwd(*a, x["v"][:1])
    with pytest.raises(ValueError):
        L.la2_gdr_bwd(x["q"], x["k"], x["v"], None, x["beta"], x["do"], dg=torch.empty_like(x["beta"]))
    with pytest.raises(ValueError):
        L.la2_gdr_bwd(*a, x["do"], workspace=torch.empty(16, dtype=torch.uint8, device=gpu))
    with pytest.raises(TypeError):
        L.la2_state_copy(x["v"], torch.zeros(1, dtype=torch.int64, device=gpu), torch.zeros(1, dtype=torch.int64, device=gpu))
