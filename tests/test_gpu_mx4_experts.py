"""The expert GEMMs on microscaled 4-bit weights against a plain 64-bit
computation, element by element, and the whole block against the oracle.

Error bound of an element (u32 = 2^-24, u16 = 2^-8, half a step relative):
  a value x enters the tensor core as two E4M3 terms that hold it to
  2^-21 of the largest value of its 32 (half a step of the second term's
  smallest spacing, 2^-9 / 16, against a largest value above 224);
  a sum of n products: n * 2 * u32 of the products' magnitudes;
  the activation h is rounded once, to bf16 or to two such terms (2^-4 twice;
  its exponential and division are good to 2^-18), the result once."""
import numpy as np
import pytest
import torch

import moe_inputs
import mx4_ref
import oracle
import sparse_moe_layer_top_b200 as moe
from parity import check_routing, rel_l2

pytestmark = pytest.mark.gpu
U32, U16 = 2.0 ** -24, 2.0 ** -8


@pytest.fixture(autouse=True)
def _automatic_path_after_each_test():
    yield
    moe.set_path(0)


def _weights(E, d, I, I_s, seed, spread=True):
    g = torch.Generator().manual_seed(seed)
    dev, ref, sc = [], [], []
    for s in [(E, I, d), (E, I, d), (E, d, I)] + ([(I_s, d), (I_s, d), (d, I_s)] if I_s else []):
        t = torch.randn(s, generator=g) * 0.05
        if spread:
            t = t * torch.exp2(torch.randint(-6, 3, s[:-1] + (s[-1] // 32,), generator=g).float()).repeat_interleave(32, -1)
        c, b, v = mx4_ref.weights(t)
        dev.append(c.cuda())
        sc.append(b)
        ref.append(v)
    if not I_s:
        dev += [None] * 3
        ref += [None] * 3
    return dev, torch.cat(sc).cuda(), ref


def _blockmax(x):
    return x.abs().unflatten(-1, (-1, 32)).amax(-1).repeat_interleave(32, -1)


def _group(x, f):
    """(y, bound) of one expert's rows x (float64)."""
    wg, wu, wd = f
    d, I = wg.shape[1], wg.shape[0]
    g, u = x @ wg.T, x @ wu.T
    dx = (d + 8) * 2 * U32 * x.abs() + 2.0 ** -21 * _blockmax(x)
    dg, du = dx @ wg.abs().T, dx @ wu.abs().T
    s = g * torch.sigmoid(g)
    h = s * u
    dh = 1.1 * dg * u.abs() + (s.abs() + 1.1 * dg) * du
    dh = dh + (h.abs() + dh) * (U16 + 2.0 ** -18)
    dh = dh + (I + 8) * 2 * U32 * (h.abs() + dh) + 2.0 ** -21 * _blockmax(h.abs() + dh)
    y, b = h @ wd.T, dh @ wd.abs().T
    return y, b + U16 * (y.abs() + b) + 1e-30


def _ffn(prob, x, offs, dev, scales, **kw):
    y = moe.expert_ffn(prob, x, offs, *dev, scales=scales, **kw)
    torch.cuda.synchronize()
    s, detail = moe.device_status()
    assert s == 0, hex(detail)
    return y


# T, d, E, k, I, I_s, group sizes (routed; they sum to T * k)
CASES = [
    (1, 128, 1, 1, 128, 0, [1]),
    (3, 128, 2, 1, 128, 128, [0, 3]),
    (20, 256, 5, 2, 128, 256, [17, 0, 1, 16, 6]),
    (16, 256, 5, 2, 256, 128, [17, 0, 1, 14, 0]),
    (10, 384, 8, 8, 128, 0, [0, 80] + [0] * 6),  # more rows of one group than tokens
    (100, 384, 6, 2, 256, 128, [64, 65, 0, 7, 63, 1]),
    (150, 512, 3, 2, 640, 0, [128, 129, 43]),
    (300, 640, 4, 3, 384, 384, [700, 200, 0, 0]),
    (64, 1152, 40, 4, 128, 128, None),
]


@pytest.mark.parametrize("path", [0, 1])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c[:6])))
def test_expert_ffn_matches_64_bit(case, path):
    T, d, E, k, I, I_s, sizes = case
    if sizes is None:
        sizes = [(7 * e) % 13 for e in range(E)]
        sizes[0] += T * k - sum(sizes)
        assert sizes[0] >= 0
    assert sum(sizes) == T * k
    dev, scales, ref = _weights(E, d, I, I_s, seed=T)
    rows = T * k + (T if I_s else 0)
    offs = moe_inputs.random_groups(E, sizes + [T if I_s else 0], device="cuda")
    g = torch.Generator().manual_seed(d)
    x = torch.randn(rows, d, generator=g) * torch.exp2(torch.randint(-9, 10, (rows, 1), generator=g).float())
    x[:, 5] *= 300  # an outlier channel
    x = x.to(torch.bfloat16)
    moe.set_path(path)
    y = _ffn(moe.Problem.make(T, d, E, k, I, I_s, "bf16", "mx4"), x.cuda(), offs, dev, scales).double().cpu()
    r = 0
    for e, n in enumerate(sizes + [T if I_s else 0]):
        if n:
            f = [ref[i][e] for i in range(3)] if e < E else ref[3:]
            want, b = _group(x[r:r + n].double(), f)
            err = (y[r:r + n] - want).abs()
            assert (err <= b).all(), "group %d: %.3g of the bound" % (e, (err / b).max())
        r += n


def test_rows_outside_the_groups_are_left_alone():
    """The expert-parallel call: only the last T of 2T rows belong to a group."""
    T, d, E, I, I_s = 70, 256, 3, 128, 128
    dev, scales, ref = _weights(E, d, I, I_s, seed=1)
    x = torch.randn(2 * T, d, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    x[:T] = float("nan")
    offs = torch.tensor([T] * (E + 1) + [2 * T], dtype=torch.int32, device="cuda")
    y = torch.full((2 * T + 5, d), 7.0, dtype=torch.bfloat16, device="cuda")
    _ffn(moe.Problem.make(T, d, E, 1, I, I_s, "bf16", "mx4"), x.cuda(), offs, dev, scales, y_perm=y)
    want, b = _group(x[T:].double(), ref[3:])
    assert (y[:T] == 7).all() and (y[2 * T:] == 7).all()
    assert ((y[T:2 * T].double().cpu() - want).abs() <= b).all()


def test_bad_values_stay_in_their_rows_and_experts():
    T, d, E, I = 40, 256, 4, 128
    dev, scales, _ = _weights(E, d, I, 0, seed=3)
    sizes = [20, 12, 0, 8]
    offs = moe_inputs.random_groups(E, sizes + [0], device="cuda")
    prob = moe.Problem.make(T, d, E, 1, I, 0, "bf16", "mx4")
    x = torch.randn(T, d, generator=torch.Generator().manual_seed(4)).to(torch.bfloat16).cuda()
    y0 = _ffn(prob, x, offs, dev, scales)
    x2 = x.clone()
    x2[3, 9], x2[25, 200], x2[39, 0] = float("nan"), float("inf"), float("-inf")
    y = _ffn(prob, x2, offs, dev, scales)
    bad = torch.tensor([3, 25, 39])
    keep = torch.tensor([i for i in range(T) if i not in bad.tolist()])
    assert torch.equal(y[keep], y0[keep]) and torch.isnan(y[bad]).all()
    s2 = scales.clone()
    per = I * d // 32
    s2[(E + 1) * per + 7] = 255  # a NaN block in expert 1's up matrix
    y = _ffn(prob, x, offs, dev, s2)
    assert torch.isnan(y[20:32]).any()
    assert torch.equal(y[:20], y0[:20]) and torch.equal(y[32:], y0[32:])


def test_extreme_scales_and_magnitudes():
    """Weight scales near 2^-100 against activations near 2^60, and zero rows."""
    T, d, E, I = 30, 256, 2, 128
    dev, scales, ref = _weights(E, d, I, 0, seed=5, spread=False)
    per = I * d // 32
    b = scales.reshape(3 * E, per)
    b[0:2] -= 60  # gate, both experts
    b[2:4] -= 60  # up
    for i in (0, 1):
        ref[i] = ref[i] * 2.0 ** -60
    offs = moe_inputs.random_groups(E, [13, 17, 0], device="cuda")
    x = torch.randn(T, d, generator=torch.Generator().manual_seed(6)) * 2.0 ** 60
    x[4], x[20] = 0, 0
    x = x.to(torch.bfloat16)
    y = _ffn(moe.Problem.make(T, d, E, 1, I, 0, "bf16", "mx4"), x.cuda(), offs, dev, scales).double().cpu()
    for e, (lo, hi) in enumerate(((0, 13), (13, 30))):
        want, bd = _group(x[lo:hi].double(), [ref[i][e] for i in range(3)])
        assert ((y[lo:hi] - want).abs() <= bd).all()
    assert (y[4] == 0).all() and (y[20] == 0).all()


@pytest.mark.parametrize("path", [0, 1, 2, 3, 4, 5, 6])
@pytest.mark.parametrize("case", [(1, 256, 8, 2, 128, 128, None), (300, 384, 12, 3, 256, 128, None),
                                  (700, 256, 6, 2, 384, 0, "zipf"), (2100, 128, 24, 4, 128, 128, "zipf")],
                         ids=lambda c: "-".join(map(str, c)))
def test_forward_matches_oracle(case, path):
    T, d, E, k, I, I_s, bias = case
    inp = moe_inputs.make_inputs(T, d, E, k, I, I_s, bias=bias, seed=T)
    ws = [getattr(inp, n) for n in ("wg", "wu", "wd", "s_wg", "s_wu", "s_wd")]
    dev = [t if t is None else t.cuda() for t in ws]
    *codes, scales = moe.quantize_experts_mx4(*dev)
    # the 4-bit values are bf16 values: the oracle reads them as such
    dense = [None if t is None else moe.dequantize_mx4(*moe.quantize_mx4(t)).cpu() for t in dev]
    moe.set_path(path)
    prob = moe.Problem.make(T, d, E, k, I, I_s, "bf16", "mx4")
    ids = torch.empty((T, k), dtype=torch.int32, device="cuda")
    tw = torch.empty((T, k), dtype=torch.float32, device="cuda")
    b = None if inp.bias is None else inp.bias.cuda()
    y = moe.layer_forward(prob, inp.x.cuda(), inp.w_r.cuda(), b, *codes, scales=scales, topk_ids=ids, topk_w=tw)
    torch.cuda.synchronize()
    s, detail = moe.device_status()
    assert s == 0, hex(detail)
    args = (inp.x, inp.w_r, *dense, k)
    y_or, ids_or, _, probs = oracle.moe_forward(*args, bias=inp.bias)
    use, differ = check_routing(ids.cpu().numpy(), tw.cpu().numpy(), probs, ids_or, 1e-3)
    if differ:
        y_or, *_ = oracle.moe_forward(*args, bias=inp.bias, force_ids=use)
    assert rel_l2(y.float().cpu().numpy(), y_or) <= 1e-2
    assert moe.forward_plan(prob)["expert_form"] == ("simt" if path == 1 else "mx4")


def test_forward_with_norm_gate_and_replay():
    T, d, E, k, I, I_s = 200, 256, 16, 3, 128, 128
    inp = moe_inputs.make_inputs(T, d, E, k, I, I_s, seed=9, device="cuda")
    *codes, scales = moe.quantize_experts_mx4(inp.wg, inp.wu, inp.wd, inp.s_wg, inp.s_wu, inp.s_wd)
    g = torch.Generator().manual_seed(1)
    gamma = (torch.randn(d, generator=g) * 0.2).to(torch.bfloat16).cuda()
    gate = (torch.randn(d, generator=g) * 0.1).to(torch.bfloat16).cuda()
    layer = moe.MoELayer(d, E, k, I, I_s, inp.w_r, *codes, scales=scales, w="mx4", max_tokens=T, norm_weight=gamma,
                         shared_gate=gate)
    y0 = layer(inp.x)
    moe.set_path(1)
    simt = layer(inp.x)
    moe.set_path(0)
    assert rel_l2(y0.float().cpu().numpy(), simt.float().cpu().numpy()) <= 1e-2
    x, y = inp.x.clone(), torch.empty_like(y0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        layer(x, y, stream=s)
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr, stream=s):
        layer(x, y, stream=s)
    for xi in (inp.x, inp.x.flip(0).contiguous(), inp.x):
        want = layer(xi)
        x.copy_(xi)
        layer.ws.fill_(255)
        gr.replay()
        assert torch.equal(y, want)
    assert moe.device_status()[0] == 0


def test_expert_parallel_ranks_with_4_bit_weights():
    """Two emulated ranks (their steps run in turn) equal one device."""
    from sparse_moe_layer_top_b200 import ep
    T, d, E, k, I, I_s, G = 60, 256, 8, 2, 128, 128, 2
    inp = moe_inputs.make_inputs(T, d, E, k, I, I_s, seed=10, device="cuda")
    *codes, scales = moe.quantize_experts_mx4(inp.wg, inp.wu, inp.wd, inp.s_wg, inp.s_wu, inp.s_wd)
    layers, states = [], []
    for r in range(G):
        layers.append(ep.EPMoELayer(r, G, d, E, k, I, I_s, inp.w_r, *ep.split_experts(r, G, *codes[:3]), *codes[3:],
                                    w="mx4", scales=ep.split_scales(r, G, E, d, I, I_s, scales)))
        states.append(layers[r].dispatch(inp.x[r * 30:(r + 1) * 30]))
    for r, (l, st) in enumerate(zip(layers, states)):
        l.set_received(st, [c for s in states for c in s.send_counts[r * 4:(r + 1) * 4]])
    back = []
    for r, l in enumerate(layers):
        parts = []
        for s in states:
            lo = sum(s.send_rows[:r])
            parts.append(s.x_perm[lo:lo + s.send_rows[r]])
        back.append(l.experts(states[r], torch.cat(parts)))
    for r, (l, st) in enumerate(zip(layers, states)):
        l.shared(st)
        lo = 0
        for dst in range(G):
            o = sum(states[q].send_rows[dst] for q in range(r))
            n = st.send_rows[dst]
            st.y_full[lo:lo + n] = back[dst][o:o + n]
            lo += n
    y = torch.cat([l.combine(st) for l, st in zip(layers, states)])
    prob = moe.Problem.make(T, d, E, k, I, I_s, "bf16", "mx4")
    want = moe.layer_forward(prob, inp.x, inp.w_r, None, *codes, scales=scales)
    assert rel_l2(y.float().cpu().numpy(), want.float().cpu().numpy()) <= 1e-2
    with pytest.raises(ValueError, match="4-bit weights need"):
        ep.EPMoELayer(0, G, d, E, k, I, I_s, inp.w_r, *ep.split_experts(0, G, *codes[:3]), *codes[3:], w="mx4",
                      scales=scales)


def test_misaligned_weights_are_refused():
    T, d, E, k, I = 4, 128, 2, 1, 128
    buf = torch.zeros(E * I * d // 2 + 32, dtype=torch.uint8, device="cuda")
    off = 16 + (-buf.data_ptr()) % 32
    w = buf[off:off + E * I * d // 2].view(E, I, d // 2)
    good = torch.zeros(E, d, I // 2, dtype=torch.uint8, device="cuda")
    scales = torch.full((3 * E * 512,), 127, dtype=torch.uint8, device="cuda")
    x = torch.zeros(T, d, dtype=torch.bfloat16, device="cuda")
    prob = moe.Problem.make(T, d, E, k, I, 0, "bf16", "mx4")
    offs = torch.tensor([0, 4, 4, 4], dtype=torch.int32, device="cuda")
    with pytest.raises(moe.MoEError, match="32-byte"):
        moe.expert_ffn(prob, x, offs, w, good.view(E, I, d // 2), good, scales=scales)


def test_waits_that_run_out_report_timeout_and_the_device_stays_usable():
    """The bound set far below the kernel's longer waits: the call comes back, the
    status names the kernel, and the same call then gives the same bits."""
    T, d, E, I = 200, 8192, 4, 256
    g = torch.Generator(device="cuda").manual_seed(15)
    r = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=torch.float32) * 0.05
    *codes, scales = moe.quantize_experts_mx4(r(E, I, d), r(E, I, d), r(E, d, I))
    offs = torch.tensor([0, 60, 70, 70, T, T], dtype=torch.int32, device="cuda")
    x = r(T, d).to(torch.bfloat16)
    prob = moe.Problem.make(T, d, E, 1, I, 0, "bf16", "mx4")
    want = moe.expert_ffn(prob, x, offs, *codes, scales=scales)
    torch.cuda.synchronize()
    assert moe.device_status()[0] == 0
    moe.set_wait_limit(100)
    try:
        moe.expert_ffn(prob, x, offs, *codes, scales=scales)
        s, detail = moe.device_status()
        assert s == 7 and (detail >> 8) & 0xff == 5 and 1 <= detail & 0xff <= 6, (s, hex(detail))
    finally:
        moe.set_wait_limit(0)
    y = moe.expert_ffn(prob, x, offs, *codes, scales=scales)
    assert moe.device_status()[0] == 0 and torch.equal(y, want)
