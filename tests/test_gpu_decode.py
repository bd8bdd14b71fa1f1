"""The few-token forward against a plain 64-bit computation,
element by element, with the error bound the kernel's roundings give.

The bound, per element of y (u32 = 2^-24, u16 = 2^-8: half a step of fp32 and
bf16, relative):
  a product sum of n exact products in fp32, in any order, is off by at most
  n * 2 * u32 times the sum of the products' magnitudes (the tensor core may
  truncate where a scalar addition rounds: one step, 2 * u32, each);
  h = w * silu(g) * u inherits g's and u's (|silu'| <= 1.1), the fast exponential
  and the divisions (2^-18 together), the routing weight's own error, and with
  bf16 weights one rounding to bf16; y its sum's, plus one rounding to bf16.
With E4M3 weights the bound allows x and h two E4M3 terms under one scale per 128
columns: off by at most half of the second term's smallest spacing, 2^-10, where
the largest of the 128 is above 224, or 2^-8 relative (a term's half step,
twice).  (They are held closer, as with 4-bit weights: test_gpu_decode_outliers.py.)
With 4-bit weights they are f16 under such a scale: half of its smallest
spacing, 2^-25, where the largest is at least 2^14, or 2^-11 relative.  x, a
bf16, is held exactly where that relative error is the larger.
The routing weight: a logit's error moves a softmax weight by at most twice
that, relatively; expf and the division add 2^-20."""
import numpy as np
import pytest
import torch

import mx4_ref
import moe_inputs
import sparse_moe_layer_top_b200 as moe

pytestmark = pytest.mark.gpu
U32, U16 = 2.0 ** -24, 2.0 ** -8


def _make(T, d, E, k, I, I_s, w, seed, bias=None, wstd=0.05):
    """-> kwargs of decode_forward on the GPU, and the float64 weights (CPU)."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)
    x, wr = r(T, d).to(torch.bfloat16), (r(E, d) * d ** -0.5).to(torch.bfloat16)
    shapes = [(E, I, d), (E, I, d), (E, d, I)] + ([(I_s, d), (I_s, d), (d, I_s)] if I_s else [])
    dev, ref, sc = [], [], []
    for s in shapes:
        t = (r(*s) * wstd).to(torch.bfloat16)
        if w == "bf16":
            dev.append(t)
            ref.append(t.double())
        elif w == "fp8":
            q, s_ = moe_inputs.quantize_e4m3_blocks(t)
            dev.append(q)
            sc.append(s_.reshape(-1))
            ref.append(q.double() * s_.double().repeat_interleave(128, -2).repeat_interleave(128, -1))
        else:
            # block sizes from 2^-12 to 2^3 of the usual: scales on both sides of 2
            e = torch.randint(-12, 4, s[:-1] + (s[-1] // 32,), generator=g).float()
            c, b, v = mx4_ref.weights(t.float() * torch.exp2(e).repeat_interleave(32, -1))
            dev.append(c)
            sc.append(b)
            ref.append(v)
    if not I_s:
        dev += [None] * 3
        ref += [None] * 3
    names = ("wg", "wu", "wd", "s_wg", "s_wu", "s_wd")
    kw = dict(prob=moe.Problem.make(T, d, E, k, I, I_s, "bf16", w), x=x.cuda(), w_router=wr.cuda(),
              bias=None if bias is None else bias.cuda(), scales=torch.cat(sc).cuda() if sc else None)
    kw.update({n: None if t is None else t.cuda() for n, t in zip(names, dev)})
    return kw, ref


def _reference(kw, ref, gate=None, out=None):
    """(y, bound, ids, w, w_bound) in float64 from the block's (normalised) input
    kw["x"].  Where the k-th and the next logit are closer than their error
    bounds either set is right: there the set of `out` (the kernel's outputs) is
    taken, after checking that it is one of the right ones."""
    p = kw["prob"]
    x, wr = kw["x"].double().cpu(), kw["w_router"].double().cpu()
    l = x @ wr.T + (0 if kw["bias"] is None else kw["bias"].double().cpu())
    order = torch.sort(l, dim=1, descending=True, stable=True)
    ids = order.indices[:, :p.k]
    w = torch.softmax(l.gather(1, ids), 1)
    dl = (p.d + 8) * 2 * U32 * (x.abs() @ wr.abs().T + l.abs().nan_to_num(posinf=0)).max(1).values
    if out is not None:
        got = out[1].cpu().long()
        lg = l.gather(1, got)
        left = l.scatter(1, got, float("-inf"))
        assert all(len(set(r)) == p.k for r in got.tolist())
        # descending, and nothing left out that is larger, to within the two logits' errors
        assert (lg[:, 1:] <= lg[:, :-1] + 2 * dl[:, None]).all()
        assert p.k == p.E or (left.max(1).values <= lg.min(1).values + 2 * dl).all()
        near = (got != ids).any(1)
        ids = torch.where(near[:, None], got, ids)
        w = torch.softmax(l.gather(1, ids), 1)
    w_rel = 2 * dl + 2.0 ** -20

    def terms(v):
        if p.w_dtype == 1:  # bf16 weights: v itself
            return torch.zeros_like(v)
        top = v.abs().unflatten(0, (-1, 128)).amax(1).repeat_interleave(128)
        return top * (2.0 ** -10 / 224 if p.w_dtype == 2 else 2.0 ** -39)

    def expert(xt, f, wt, wrel):
        wg, wu, wd = f
        g, u = wg @ xt, wu @ xt
        dx = (p.d + 8) * 2 * U32 * xt.abs() + terms(xt)
        dg, du = wg.abs() @ dx, wu.abs() @ dx
        s = g * torch.sigmoid(g)
        h = wt * s * u
        dh = wt * (1.1 * dg * u.abs() + (s.abs() + 1.1 * dg) * du)
        dh = dh + (h.abs() + dh) * ((2.0 ** -11 if p.w_dtype == 3 else U16) + 2.0 ** -18 + wrel)
        dh = dh + terms(h.abs() + dh)
        return wd @ h, wd.abs() @ dh, wd.abs() @ h.abs()

    y = torch.zeros_like(x)
    b, m = torch.zeros_like(x), torch.zeros_like(x)
    for t in range(p.T):
        for j in range(p.k):
            e = int(ids[t, j])
            o = expert(x[t], (ref[0][e], ref[1][e], ref[2][e]), w[t, j], w_rel[t])
            y[t], b[t], m[t] = y[t] + o[0], b[t] + o[1], m[t] + o[2]
        if p.I_s:
            gt = 1.0 if gate is None else torch.sigmoid(x[t] @ gate)
            grel = 0.0 if gate is None else (p.d + 8) * 2 * U32 * (x[t].abs() @ gate.abs()) + 2.0 ** -20
            o = expert(x[t], ref[3:], gt, grel)
            y[t], b[t], m[t] = y[t] + o[0], b[t] + o[1], m[t] + o[2]
    n = p.k * p.I + p.I_s + 32
    b = b + n * 2 * U32 * (m + b)
    b = b + U16 * (y.abs() + b) + 1e-30
    return y, b, ids, w, w * (w_rel[:, None]) + 1e-30


def _run(kw, **opt):
    p = kw["prob"]
    ids = torch.empty((p.T, p.k), dtype=torch.int32, device="cuda")
    tw = torch.empty((p.T, p.k), dtype=torch.float32, device="cuda")
    y = moe.decode_forward(**kw, **opt, topk_ids=ids, topk_w=tw)
    torch.cuda.synchronize()
    s, detail = moe.device_status()
    assert s == 0, hex(detail)
    return y, ids, tw


def _check(out, want):
    y, ids, tw = out
    yr, b, ir, wr, wb = want
    assert torch.equal(ids.cpu().long(), ir)
    assert ((tw.double().cpu() - wr).abs() <= wb).all()
    err = (y.double().cpu() - yr).abs()
    assert (err <= b).all(), "worst %.3g of the bound" % (err / b).max()


CASES = [
    # T, d, E, k, I, I_s, weights
    (1, 8, 1, 1, 8, 0, "bf16"),
    (1, 2048, 256, 8, 512, 512, "bf16"),
    (2, 24, 3, 2, 16, 40, "bf16"),
    (3, 1000, 24, 3, 328, 200, "bf16"),
    (7, 136, 5, 5, 72, 0, "bf16"),
    (8, 264, 130, 6, 136, 24, "bf16"),
    (9, 256, 20, 4, 192, 128, "bf16"),
    (16, 520, 512, 16, 40, 64, "bf16"),
    (16, 4104, 4, 2, 48, 8, "bf16"),
    (1, 128, 4, 1, 128, 0, "fp8"),
    (5, 384, 12, 3, 256, 128, "fp8"),
    (8, 1024, 40, 10, 128, 384, "fp8"),
    (16, 256, 17, 16, 384, 0, "fp8"),
    (1, 128, 4, 1, 128, 0, "mx4"),
    (1, 2048, 32, 8, 512, 512, "mx4"),
    (6, 384, 12, 3, 256, 128, "mx4"),
    (8, 1152, 9, 2, 128, 384, "mx4"),
    (13, 256, 40, 10, 384, 0, "mx4"),
    (16, 640, 6, 6, 256, 128, "mx4"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_matches_the_64_bit_block(case):
    kw, ref = _make(*case, seed=sum(case[:6]))
    out = _run(kw)
    _check(out, _reference(kw, ref, out=out))


@pytest.mark.parametrize("w,T,d,I,I_s", [("bf16", 5, 264, 136, 72), ("fp8", 16, 256, 128, 256), ("mx4", 3, 256, 128, 128)])
def test_bias_norm_and_shared_gate(w, T, d, I, I_s):
    E, k = 12, 3
    g = torch.Generator().manual_seed(2)
    bias = torch.randn(E, generator=g)
    bias[4] = float("-inf")  # an expert nobody may take
    kw, ref = _make(T, d, E, k, I, I_s, w, seed=5, bias=bias)
    gamma = (torch.randn(d, generator=g) * 0.2).to(torch.bfloat16)
    gate = (torch.randn(d, generator=g) * 0.1).to(torch.bfloat16)
    out = _run(kw, norm_weight=gamma.cuda(), norm_eps=1e-6, shared_gate=gate.cuda())
    assert not (out[1] == 4).any()
    kn = dict(kw)
    kn["x"] = moe.rmsnorm(kw["prob"], kw["x"], gamma.cuda(), 1e-6)  # the stage call, tested by itself
    _check(out, _reference(kn, ref, gate.double(), out))
    out = _run(kn, shared_gate=gate.cuda())
    _check(out, _reference(kn, ref, gate.double(), out))


def test_equal_logits_go_to_the_lowest_experts():
    kw, ref = _make(4, 64, 70, 5, 32, 0, "bf16", seed=1)
    kw["w_router"].zero_()
    out = _run(kw)
    assert (out[1].cpu() == torch.arange(5)).all() and (out[2] == 0.2).all()
    _check(out, _reference(kw, ref))


@pytest.mark.parametrize("w", ["bf16", "fp8", "mx4"])
def test_bad_weights_reach_only_their_own_tokens(w):
    """An infinity or NaN in an expert's weights leaves every token not routed
    to it as it was, bit for bit."""
    kw, _ = _make(8, 256, 16, 2, 128, 128, w, seed=3)
    y0, ids, _ = _run(kw)
    e = int(ids[0, 0])
    hit = (ids == e).any(1)
    assert hit.any() and not hit.all()
    for name in ("wg", "wu", "wd"):
        k2 = dict(kw)
        k2[name] = kw[name].clone()
        if w == "bf16":
            k2[name][e, 5, 7] = float("inf")
            k2[name][e, 6, 9] = float("nan")
        elif w == "fp8":
            k2[name].view(torch.uint8)[e, 5, 7] = 0x7f
            k2[name].view(torch.uint8)[e, 77, 200 % k2[name].shape[2]] = 0xff
        else:
            k2["scales"] = kw["scales"].clone()
            i = ("wg", "wu", "wd").index(name)
            per = 16 * 128 * 256 // 32
            k2["scales"][i * per + e * per // 16 + 3] = 255
        y, _, _ = _run(k2)
        assert torch.equal(y[~hit], y0[~hit])
        assert torch.isnan(y[hit]).any()


def test_infinite_and_nan_tokens_stay_their_own():
    kw, _ = _make(9, 264, 16, 3, 136, 72, "bf16", seed=4)
    y0, ids0, _ = _run(kw)
    kw["x"][2, 11] = float("nan")
    kw["x"][5, 100] = float("inf")
    y, ids, _ = _run(kw)
    keep = [t for t in range(9) if t not in (2, 5)]
    assert torch.equal(y[keep], y0[keep]) and torch.equal(ids[keep], ids0[keep])
    assert torch.isnan(y[2]).all()
    assert ((ids >= 0) & (ids < 16)).all()
    assert all(len(set(r)) == 3 for r in ids.tolist())


def test_large_activations_do_not_overflow():
    """Hidden activations far above the 16-bit float range (bf16 holds them)."""
    kw, ref = _make(3, 256, 8, 2, 128, 128, "mx4", seed=6)
    kw["x"] = (kw["x"].float() * 4096).to(torch.bfloat16)
    kw["w_router"] = (kw["w_router"].float() / 4096).to(torch.bfloat16)
    out = _run(kw)
    want = _reference(kw, ref, out=out)
    assert want[0].abs().max() > 1e5
    _check(out, want)


def test_scale_extremes():
    """Scale bytes at the ends of their range (2^-127 and 2^60)."""
    kw, ref = _make(2, 128, 2, 1, 128, 0, "mx4", seed=7)
    per = 128 * 128 // 32
    for i, (byte, shift) in enumerate(((0, None), (187, None))):  # expert 0: tiny up weights; expert 1: huge down weights
        m = 1 if i == 0 else 2
        kw["scales"][(m * 2 + i) * per:(m * 2 + i + 1) * per] = byte
    for i, m, byte in ((0, 1, 0), (1, 2, 187)):
        q, _ = kw[("wg", "wu", "wd")[m]][i].cpu().numpy(), None
        ref[m][i] = torch.from_numpy(mx4_ref.values(q, np.full((128, 4), byte, np.uint8)))
    out = _run(kw)
    want = _reference(kw, ref, out=out)
    # a product with 2^-127 weights may leave fp32's range at the bottom: sums below
    # 2^-100 count as zero here
    y, b = out[0].double().cpu(), want[1] + 2.0 ** -100
    assert torch.isfinite(y).all()
    assert ((y - want[0]).abs() <= b).all()


def test_rows_behind_the_last_token_are_left_alone_and_runs_repeat():
    kw, _ = _make(5, 264, 16, 3, 136, 72, "bf16", seed=8)
    y0, _, _ = _run(kw)
    y = torch.full((9, 264), 7.0, dtype=torch.bfloat16, device="cuda")
    x = torch.cat([kw["x"], torch.full((4, 264), float("nan"), device="cuda", dtype=torch.bfloat16)])
    moe.decode_forward(**{**kw, "x": x}, y=y)
    assert torch.equal(y[:5], y0) and (y[5:] == 7).all()
    for _ in range(20):
        assert torch.equal(moe.decode_forward(**kw), y0)


@pytest.mark.parametrize("w,norm", [("bf16", False), ("bf16", True), ("mx4", False)])
def test_replays_from_a_cuda_graph(w, norm):
    kw, _ = _make(4, 256, 16, 3, 128, 128, w, seed=9)
    p = kw["prob"]
    opt = dict(norm_weight=torch.full((256,), 0.1, dtype=torch.bfloat16, device="cuda")) if norm else {}
    x2 = kw["x"].flip(0).contiguous()
    want = [moe.decode_forward(**kw, **opt), moe.decode_forward(**{**kw, "x": x2}, **opt)]
    x, y = kw["x"].clone(), torch.empty_like(kw["x"])
    ws = torch.empty(moe.decode_workspace_size(p), dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        moe.decode_forward(**{**kw, "x": x}, **opt, y=y, ws=ws, stream=s)
    for xi, yi in ((kw["x"], want[0]), (x2, want[1]), (kw["x"], want[0])):
        x.copy_(xi)
        ws.fill_(255)  # nothing is kept in the workspace between replays
        g.replay()
        assert torch.equal(y, yi)
    assert moe.device_status()[0] == 0


def test_two_streams_at_once():
    """Two calls in flight on two streams, each in its own workspace."""
    a, _ = _make(3, 512, 16, 3, 256, 128, "bf16", seed=10)
    b, _ = _make(11, 384, 12, 2, 256, 128, "fp8", seed=11)
    ya, yb = moe.decode_forward(**a), moe.decode_forward(**b)
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for _ in range(20):
        outs.append((moe.decode_forward(**a, stream=sa), moe.decode_forward(**b, stream=sb)))
    torch.cuda.synchronize()
    assert all(torch.equal(p, ya) and torch.equal(q, yb) for p, q in outs)
    assert moe.device_status()[0] == 0


def test_layer_object_quantise_and_decode_together():
    """A block's weights quantised on the GPU, then one token, a few tokens and a
    batch through one MoELayer: the few-token form agrees with the fused forward
    to the rounding both do (two bf16 roundings of h and of each slot row)."""
    inp = moe_inputs.make_inputs(64, 512, 16, 4, 256, 128, seed=12, device="cuda")
    *codes, scales = moe.quantize_experts_mx4(inp.wg, inp.wu, inp.wd, inp.s_wg, inp.s_wu, inp.s_wd)
    layer = moe.MoELayer(512, 16, 4, 256, 128, inp.w_r, *codes, scales=scales, w="mx4", max_tokens=64)
    y = layer(inp.x)
    dense = [moe.dequantize_mx4(*moe.quantize_mx4(t)) for t in (inp.wg, inp.wu, inp.wd, inp.s_wg, inp.s_wu, inp.s_wd)]
    ref = moe.MoELayer(512, 16, 4, 256, 128, inp.w_r, *dense, max_tokens=64)
    for lo, hi in ((0, 1), (1, 9), (9, 25)):
        got, want = layer.decode(inp.x[lo:hi]), ref.decode(inp.x[lo:hi])
        # the dequantised block in bf16 holds the same values: the same products, summed in another K order
        assert torch.allclose(got.float(), want.float(), rtol=2 * 2.0 ** -7, atol=1e-3)
        assert (got.float() - y[lo:hi].float()).norm() <= 1e-2 * y[lo:hi].float().norm()
    with pytest.raises(moe.MoEError, match="moe_layer_forward"):
        layer.decode(inp.x[:17])


@pytest.mark.parametrize("w,T", [("fp8", 6), ("mx4", 6), ("fp8", 12), ("mx4", 12)])
def test_infinite_and_nan_tokens_stay_their_own_with_scaled_weights(w, T):
    kw, _ = _make(T, 256, 16, 3, 128, 128, w, seed=13)
    y0, ids0, _ = _run(kw)
    kw["x"][2, 11] = float("nan")
    kw["x"][5, 100] = float("inf")
    y, ids, _ = _run(kw)
    keep = [t for t in range(T) if t not in (2, 5)]
    assert torch.equal(y[keep], y0[keep]) and torch.equal(ids[keep], ids0[keep])
    assert torch.isnan(y[2]).all() and not torch.isfinite(y[5]).any()


@pytest.mark.parametrize("w", ["bf16", "fp8", "mx4"])
@pytest.mark.parametrize("T", [8, 9, 16])
def test_every_token_at_one_expert(w, T):
    """The bias sends all tokens to the same experts: full column blocks, and a
    second one from nine tokens on."""
    E, k = 20, 2
    bias = torch.full((E,), -50.0)
    bias[[3, 17]] = 50.0
    kw, ref = _make(T, 384, E, k, 256, 0, w, seed=14 + T, bias=bias)
    out = _run(kw)
    assert (out[1].cpu().sort(1).values == torch.tensor([3, 17])).all()
    _check(out, _reference(kw, ref, out=out))
