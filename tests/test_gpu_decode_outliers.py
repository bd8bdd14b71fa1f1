"""The few-token forward on E4M3 weights where one channel in 128 is thousands of
times the others: those keep the precision of a bf16 (x) and of an f16 (h).

The bound is the one of test_gpu_decode.py for values held as f16 under a power of
two per 128 columns: half of f16's smallest spacing, 2^-25, where the largest of
the 128 is at least 2^14, and 2^-11 relative for h; x, a bf16, is exact above that
floor.  The far channels meet zero weights, so what they cost the others is all
that could pass the bound: a value held to 2^-18 of the largest of its 128 columns
would be off by 2^-18 * 3000 = 1 %, against 0.4 % for y's rounding."""
import pytest
import torch

import sparse_moe_layer_top_b200 as moe
import test_gpu_decode as few

pytestmark = pytest.mark.gpu


def _bound_of_f16(kw):
    p = kw["prob"]  # (the problem only picks the operands' rounding there)
    return {**kw, "prob": moe.Problem.make(p.T, p.d, p.E, p.k, p.I, p.I_s, "bf16", "mx4")}


def _zero_columns(kw, ref, names, at):
    for n in names:
        i = ("wg", "wu", "wd", "s_wg", "s_wu", "s_wd").index(n)
        if kw[n] is not None:
            kw[n].view(torch.uint8)[..., at] = 0
            ref[i][..., at] = 0


@pytest.mark.parametrize("T,d,I,I_s", [(1, 512, 256, 0), (4, 256, 128, 128), (8, 1024, 128, 384), (9, 384, 256, 128),
                                       (16, 256, 384, 0)])
def test_a_far_channel_of_x(T, d, I, I_s):
    kw, ref = few._make(T, d, 8, 3, I, I_s, "fp8", seed=T)
    at = slice(5, None, 128)
    kw["x"][:, at] = (kw["x"][:, at].float() * 3000).to(torch.bfloat16)
    kw["w_router"][:, at] = 0
    _zero_columns(kw, ref, ("wg", "wu", "s_wg", "s_wu"), at)
    out = few._run(kw)
    few._check(out, few._reference(_bound_of_f16(kw), ref, out=out))


@pytest.mark.parametrize("T,d,I,I_s", [(1, 256, 256, 0), (8, 384, 128, 256), (16, 256, 128, 0)])
def test_a_far_feature_of_h(T, d, I, I_s):
    kw, ref = few._make(T, d, 6, 2, I, I_s, "fp8", seed=30 + T)
    for n, i in (("wu", 1), ("s_wu", 4)):  # the up rows but one in 128, 2^-12 times as large
        if kw[n] is None:
            continue
        q = kw[n].cpu().float()
        scale = torch.where(q == 0, torch.zeros_like(ref[i]), ref[i] / q.double())
        # (one scale a block of 128 columns: that of any code in it that is not 0)
        scale = scale.unflatten(-1, (-1, 128)).amax(-1).repeat_interleave(128, -1)
        keep = torch.arange(q.shape[-2]) % 128 == 7
        small = (q * 2.0 ** -12).to(torch.float8_e4m3fn)
        new = torch.where(keep[:, None], q, small.float())
        kw[n] = new.to(torch.float8_e4m3fn).cuda()
        ref[i] = new.double() * scale
    _zero_columns(kw, ref, ("wd", "s_wd"), slice(7, None, 128))
    out = few._run(kw)
    few._check(out, few._reference(_bound_of_f16(kw), ref, out=out))


def test_an_infinite_down_weight_gives_infinities():
    T, E, k = 9, 12, 3
    kw, ref = few._make(T, 256, E, k, 136, 72, "bf16", seed=60)
    e = int(few._run(kw)[1][0, 0])
    kw["wd"][e, 5, 7] = float("inf")
    y, ids, _ = few._run(kw)
    hit = (ids == e).any(1).cpu()
    x, wg, wu = kw["x"].double().cpu(), ref[0][e, 7], ref[1][e, 7]
    h = x @ wg * torch.sigmoid(x @ wg) * (x @ wu)
    assert hit.any() and (y[~hit.cuda()].isfinite()).all()
    assert torch.equal(y[hit.cuda(), 5].cpu().double(), torch.copysign(torch.full_like(h, float("inf")), h)[hit])
    y[:, 5] = 0
    assert y.isfinite().all()
