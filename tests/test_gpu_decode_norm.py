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
