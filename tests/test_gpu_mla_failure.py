"""A bounded wait of the dense-attention kernels that runs out: reported, and the context recovers.

As in the other failure tests, the test build's MMA warp of the kernel's first CTA waits on an mbarrier
that no thread arrives on, for 20 ms at most.  The launch must end with DSA_ERR_TIMEOUT in the status
word, and the next calls, of the test build and of the product, must give what they give alone.
"""
import pytest
import torch

import dsa_sparse_attention_li_gb300 as dsa
from test_mla import make_decode, make_prefill, run_decode, run_prefill, verify_decode, verify_prefill

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("what", ["decode_bf16", "decode_fp8", "prefill"])
def test_timed_out_wait_is_reported_and_the_context_recovers(cuda_lib, monkeypatch, what):
    if what == "prefill":
        c, run, verify, kernel = make_prefill([700, 300], [900, 300], 4), run_prefill, verify_prefill, 4
    else:
        c, run, verify, kernel = make_decode([9000, 700], [1, 2], 64, what == "decode_fp8"), run_decode, verify_decode, 3
    hooks = dsa.load_testhooks()
    with monkeypatch.context() as m:
        m.setattr(dsa, "_lib", hooks)
        hooks.dsa_test_inject_stall(kernel)
        try:
            assert run(c)[2] == dsa.DSA_ERR_TIMEOUT
        finally:
            hooks.dsa_test_inject_stall(0)
        out, lse, status = run(c)
        assert status == 0
        verify(c, out, lse)
    out, lse, status = run(c)
    assert status == 0
    verify(c, out, lse)
