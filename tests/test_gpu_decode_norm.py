"""The normalised input of the few-token forward is the 64-bit one rounded to bf16.

Seen through the routing weights: an expert whose router row is one column of the
identity has that column of the normalised x as its logit, exactly, and with as
many experts as are taken the weights are the softmax of 16 columns.  They are
compared with that of the 64-bit values' roundings: equal inputs leave the
softmax's own error, 2^-20; a column rounded the other way shows as a step of its
bf16, 2^-9 of it or more."""
import pytest
import torch

import sparse_moe_layer_top_b200 as moe

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,d,std", [(1, 4096, 1.0), (5, 1000, 30.0), (16, 2048, 1.0), (16, 2048, 0.01)])
def test_the_normalised_input_is_the_64_bit_one_rounded(T, d, std):
    E = 16
    g = torch.Generator().manual_seed(T + d)
    x = (torch.randn(T, d, generator=g) * std).to(torch.bfloat16)
    gamma = (torch.randn(d, generator=g) * 0.1).to(torch.bfloat16)
    x64 = x.double()
    xn = (x64 / torch.sqrt(x64.pow(2).mean(1, keepdim=True) + 1e-6) * (1 + gamma.double())).to(torch.bfloat16).double()
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")
    W = z(E, 8, d), z(E, 8, d), z(E, d, 8)
    prob = moe.Problem.make(T, d, E, E, 8, 0, "bf16", "bf16")
    xd, gd = x.cuda(), gamma.cuda()
    ids = torch.empty((T, E), dtype=torch.int32, device="cuda")
    worst = 0.0
    for c in range(0, d - E + 1, E):
        wr = z(E, d)
        wr[torch.arange(E), c + torch.arange(E)] = 1
        tw = torch.empty((T, E), dtype=torch.float32, device="cuda")
        moe.decode_forward(prob, xd, wr, None, *W, norm_weight=gd, norm_eps=1e-6, topk_ids=ids, topk_w=tw)
        got = torch.zeros((T, E), dtype=torch.float64).scatter(1, ids.cpu().long(), tw.double().cpu())
        want = torch.softmax(xn[:, c:c + E], 1)
        worst = max(worst, ((got - want).abs() / want).max().item())
    assert worst <= 2.0 ** -20


@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_rows_of_zeros_infinities_and_extremes_are_the_stage_calls(eps):
    """Where the sum of squares is 0, infinite or NaN the normalised row is
    moe.rmsnorm's: zeros, NaN, or zeros beside the NaN of the infinity itself."""
    d, E, k = 264, 6, 2
    g = torch.Generator().manual_seed(3)
    x = torch.randn(7, d, generator=g)
    x[0] = 0
    x[1, 9] = float("inf")
    x[2, 9] = float("nan")
    x[3] *= 1e30  # squares past fp32
    x[4] *= 1e-30  # and below it
    x[5, 1:] = 0
    r = lambda *s: (torch.randn(*s, generator=g) * 0.1).to(torch.bfloat16).cuda()
    x, wr, gamma = x.to(torch.bfloat16).cuda(), r(E, d), r(d)
    W = r(E, 16, d), r(E, 16, d), r(E, d, 16)
    prob = moe.Problem.make(7, d, E, k, 16, 0, "bf16", "bf16")
    out = []
    for xi, kw in ((x, dict(norm_weight=gamma, norm_eps=eps)), (moe.rmsnorm(prob, x, gamma, eps), {})):
        ids = torch.empty((7, k), dtype=torch.int32, device="cuda")
        out.append((moe.decode_forward(prob, xi, wr, None, *W, topk_ids=ids, **kw), ids))
    assert torch.equal(out[0][1], out[1][1])
    # (finite rows: a step of bf16 of x and of y apart at most, 2^-6 of the row's largest)
    a, b = out[0][0].float(), out[1][0].float()
    assert torch.equal(a.isnan(), b.isnan()) and torch.equal(a.isinf(), b.isinf())
    a, b = a.nan_to_num(0, 0, 0), b.nan_to_num(0, 0, 0)
    assert ((a - b).abs() <= 2.0 ** -6 * b.abs().amax(1, keepdim=True)).all()
