"""A bounded wait of dsa_matmul_fp8 that runs out: reported, and the context recovers.

As in the other failure tests, the test build's first CTA waits on an mbarrier that no thread arrives on (10),
or leaves a load out (11), for 20 ms at most.  The launch must end with DSA_ERR_TIMEOUT in the status word, and the
next calls, of the test build and of the product, must give what they give alone.
"""
import pytest
import torch

import dsa_sparse_attention_li_gb300 as dsa
from test_matmul_fp8 import definition, gen, whole

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("stall", [10, 11])
@pytest.mark.parametrize("m,n,k,plan", [(2300, 2560, 896, 0), (9, 2112, 7168, 128 * 16 + 8), (200, 8192, 1024, 128 * 16 + 1)])
def test_timed_out_wait_is_reported_and_the_context_recovers(cuda_lib, monkeypatch, m, n, k, plan, stall):
    case = whole(m, n, k, gen(m))
    want = definition(*case)[0].float().bfloat16()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    hooks = dsa.load_testhooks()
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert hooks.dsa_test_matmul_plan(m, n, k, sms) // 16 == plan // 16   # (wide, or the width)
    with monkeypatch.context() as mp:
        mp.setattr(dsa, "_lib", hooks)
        hooks.dsa_test_inject_stall(stall)
        try:
            dsa.matmul_fp8(*case, status=status)
            torch.cuda.synchronize()
        finally:
            hooks.dsa_test_inject_stall(0)
        assert int(status) == dsa.DSA_ERR_TIMEOUT
        status.zero_()
        assert torch.equal(dsa.matmul_fp8(*case, status=status), want) and int(status) == 0
    assert torch.equal(dsa.matmul_fp8(*case, status=status), want) and int(status) == 0
