"""Bounded waits of the cross-attention's tensor-core kernels that run out.

With the limit at 1 ns the first wait that has to spin gives up: the call is
accepted, the device records the timeout, every CTA ends, and the next call in
the same process is right again.  What the timed-out calls write is undefined.
"""

import pytest
import torch

from block_ops_ref import assert_within, cross_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    torch.cuda.init()


@pytest.mark.parametrize("d", [64, 128])
def test_short_wait_limit_then_context_stays_usable(lib, d):
    gen = torch.Generator(device="cuda").manual_seed(90)

    def x(L, h=8):
        return torch.randn(1, h, L, d, device="cuda", generator=gen).bfloat16()

    q, k, v, g = x(8192), x(700), x(700), x(8192)  # thousands of waits
    out, lse = lib.cross_attn_fwd(q, k, v, return_lse=True)
    torch.cuda.synchronize()
    assert lib.device_status() == lib.PISA_OK
    try:
        lib.set_wait_limit(1)
        for name, run in (("forward", lambda: lib.cross_attn_fwd(q, k, v)),
                          ("backward", lambda: lib.cross_attn_bwd(g, q, k, v, out, lse))):
            run()
            torch.cuda.synchronize()
            assert lib.device_status(reset=True) == lib.PISA_ERR_TIMEOUT, name
    finally:
        lib.set_wait_limit(0)
    assert lib.device_status() == lib.PISA_OK
    q, g = q[:, :, :300].contiguous(), g[:, :, :300].contiguous()
    ref = cross_ref(q, k, v, dout=g)
    out, lse = lib.cross_attn_fwd(q, k, v, return_lse=True)
    assert_within(out, ref["out"], "out")
    for name, y in zip(("dq", "dk", "dv"), lib.cross_attn_bwd(g, q, k, v, out, lse)):
        assert_within(y, ref[name], name)
    assert lib.device_status() == lib.PISA_OK
