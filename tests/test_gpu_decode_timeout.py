"""The few-token kernel's grid barriers running out (the bound set far below them,
as in test_gpu_timeout.py): one or eight CTAs compute the gate/up product of a very
wide block while the others wait for them.  Those record the timeout, wait for
their own copies and return; with 4-bit weights the late CTAs then run out at the
second barrier, where the others never arrive.  The same workspace then gives the
same bits."""
import pytest
import torch

import sparse_moe_layer_top_b200 as moe

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("w,I", [("bf16", 16), ("fp8", 128), ("mx4", 128)])
def test_barriers_that_run_out_report_timeout_and_the_workspace_stays_usable(w, I):
    T, d, E, k = 2, 131072, 2, 1
    g = torch.Generator(device="cuda").manual_seed(17)
    r = lambda *s: (torch.randn(s, generator=g, device="cuda") * 0.05).to(torch.bfloat16)
    W, scales = [r(E, I, d), r(E, I, d), r(E, d, I)], None
    if w == "mx4":
        *W, scales = moe.quantize_experts_mx4(*W)
        W = W[:3]
    elif w == "fp8":
        W = [t.to(torch.float8_e4m3fn) for t in W]
        scales = torch.ones(3 * E * (d // 128) * (I // 128), device="cuda")
    x, w_router = r(T, d), r(E, d)
    bias = torch.tensor([40.0, -40.0], device="cuda")  # one expert for every token
    prob = moe.Problem.make(T, d, E, k, I, 0, "bf16", w)
    ws = torch.empty(moe.decode_workspace_size(prob), dtype=torch.uint8, device="cuda")
    call = lambda: moe.decode_forward(prob, x, w_router, bias, *W, scales=scales, ws=ws)
    want = call()
    torch.cuda.synchronize()
    assert moe.device_status()[0] == 0
    moe.set_wait_limit(100)
    try:
        call()
        s, detail = moe.device_status()
        assert s == 7 and (detail >> 8) & 0xff == 4 and detail & 0xff in (1, 2), (s, hex(detail))
    finally:
        moe.set_wait_limit(0)
    assert torch.equal(call(), want)
    assert moe.device_status()[0] == 0
