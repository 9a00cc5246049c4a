"""The bounded waits of the gated delta rule's kernels, made to run out without faulting, trapping or hanging the GPU.

la2_gdr_selftest_timeout launches a kernel with one copy that is announced and never issued.  The wait for it runs out:
the kernel records LA2_ERR_TIMEOUT with the wait's site, waits for its copies and products in flight and ends, and the
calls that follow give, bit by bit, what they gave before.
"""
import pytest
import torch

import gdr_ref as R
from causal_linear_attention_la2_b200 import la2 as L

KERNELS = {"decode": L.LA2_GDR_KERNEL_DECODE, "gradients": L.LA2_GDR_KERNEL_GRAD, "walk": L.LA2_GDR_KERNEL_WALK,
           "walks": L.LA2_GDR_KERNEL_WALKS}
BARRIERS = set(range(200, 230))  # 200 + the barrier that the first role gave up on
SITES = {"decode": {230}, "gradients": BARRIERS, "walk": BARRIERS, "walks": BARRIERS}
FAKE = 1 << 20


def test_bad_arguments_are_refused():
    from causal_linear_attention_la2_b200 import build
    build.build()
    n = L.LA2_GDR_SELFTEST_BYTES
    for kernel in (-1, 4):
        assert L.la2_gdr_selftest_timeout_raw(kernel, FAKE, n) == L.LA2_ERR_INVALID_ARG
    for kernel in KERNELS.values():
        assert L.la2_gdr_selftest_timeout_raw(kernel, 0, n) == L.LA2_ERR_WORKSPACE
        assert L.la2_gdr_selftest_timeout_raw(kernel, FAKE, n - 1) == L.LA2_ERR_WORKSPACE
        assert L.la2_gdr_selftest_timeout_raw(kernel, FAKE + 16, n) == L.LA2_ERR_INVALID_ARG


def _ordinary(dev):
    """The calls whose kernels the self-test holds."""
    x = R.make(2, 1, 2, 200, 128, 128, torch.bfloat16, 70, init=True, final=True, lens=[100, 200])
    y = {n: t.to(dev) for n, t in x.items()}
    a = (y["q"], y["k"], y["v"], y["g"], y["beta"])
    o, S = L.la2_gdr_fwd(*a, init_state=y["init"], seq_lens=y["lens"], want_final=True)
    grads = L.la2_gdr_bwd(*a, y["do"], init_state=y["init"], d_final_state=y["dfinal"], seq_lens=y["lens"])
    z = R.make(300, 1, 2, 1, 128, 128, torch.bfloat16, 71)
    z = {n: z[n][:, :, 0].contiguous().to(dev) for n in ("q", "k", "v", "g", "beta")}
    pool = torch.ones(300, 2, 128, 128, device=dev)
    return [o, S, *grads, L.la2_gdr_decode(*z.values(), pool), pool]


@pytest.mark.gpu
@pytest.mark.parametrize("kernel", KERNELS)
def test_a_wait_runs_out_and_the_gpu_keeps_working(kernel):
    dev = torch.device("cuda")
    assert L.la2_device_status(reset=True) == 0
    before = _ordinary(dev)
    space = torch.empty(L.LA2_GDR_SELFTEST_BYTES, dtype=torch.uint8, device=dev)
    stream = torch.cuda.current_stream().cuda_stream
    st = L.la2_gdr_selftest_timeout_raw(KERNELS[kernel], space.data_ptr(), space.numel(), stream)
    assert st == L.LA2_OK, L.la2_status_str(st)
    torch.cuda.synchronize()
    code = L.la2_device_status(reset=True)
    assert code & 0xFF == L.LA2_ERR_TIMEOUT, hex(code)
    assert code >> 8 in SITES[kernel], code >> 8
    after = _ordinary(dev)
    torch.cuda.synchronize()
    assert L.la2_device_status(reset=True) == 0
    for a, b in zip(before, after):
        assert torch.equal(a, b)
