"""Microscaled 4-bit weights and the few-token forward without a GPU: the
reference's own pins, the scale layout helper, and every refusal (none of the
calls below reaches a launch)."""
import ctypes

import numpy as np
import pytest
import torch

import mx4_ref
import sparse_moe_layer_top_b200 as moe

ON_DEVICE = "must be on a CUDA device"


def test_reference_rounds_to_the_even_code_at_each_middle():
    x = torch.zeros(1, 32)
    x[0, :10] = torch.tensor([4.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -5.0])
    c, b = mx4_ref.quantize(x)
    assert b.tolist() == [[127]]  # floor(log2 5) - 2 = 0
    assert mx4_ref.values(c, b)[0, :10].tolist() == [4, 0, 1, 1, 2, 2, 4, 4, 0, -4]
    x = torch.tensor([[7.9] + [1.0] * 31])
    c, b = mx4_ref.quantize(x)
    assert b.tolist() == [[127]] and mx4_ref.values(c, b)[0, 0] == 6  # saturates


def test_reference_errors_are_within_the_format():
    x = torch.randn(40, 96, dtype=torch.float64)
    c, b = mx4_ref.quantize(x)
    v = mx4_ref.values(c, b)
    s = np.repeat(2.0 ** (b.astype(np.float64) - 127), 32, 1)
    a = np.abs(x.numpy()) / s
    # half the spacing of the magnitudes (0.5 below 2, 1 below 4, 2 above), or the saturated part
    bound = np.where(a < 2, 0.25, np.where(a < 4, 0.5, np.maximum(1.0, a - 6)))
    assert (np.abs(v - x.numpy()) <= bound * s).all()


def test_scale_tiles_helper_matches_the_byte_formula():
    b = torch.randint(0, 256, (3, 256, 12), dtype=torch.uint8)
    t = moe.mx4_scale_tiles(b)
    assert t.shape == (3, 2, 3, 512)
    assert np.array_equal(t.numpy(), mx4_ref.tiles(b.numpy()))
    for bad in (b.float(), b[:, :100], b[..., :3]):
        with pytest.raises(ValueError, match="scales"):
            moe.mx4_scale_tiles(bad)


def test_scale_bytes():
    L = moe.lib()
    assert L.moe_mx4_scale_bytes(1, 128, 128) == 512
    assert L.moe_mx4_scale_bytes(3, 129, 160) == 3 * 2 * 2 * 512
    assert L.moe_mx4_scale_bytes(0, 5, 32) == 0
    assert L.moe_mx4_scale_bytes(1, 5, 33) == 0


def test_quantize_rejected_before_any_launch():
    L = moe.lib()
    v = ctypes.c_void_p
    q = lambda x=16, dt=1, b=2, r=5, c=64, codes=16, sc=16: L.moe_mx4_quantize(
        None if x is None else v(x), dt, b, r, c, None if codes is None else v(codes), None if sc is None else v(sc),
        None)
    d = lambda codes=16, sc=16, b=2, r=5, c=64, dt=1, out=16: L.moe_mx4_dequantize(
        None if codes is None else v(codes), None if sc is None else v(sc), b, r, c, dt, None if out is None else v(out),
        None)
    for f in (q, d):
        assert f(b=-1) == 1 and f(r=-1) == 1 and f(c=0) == 1 and f(c=48) == 1
        assert f(dt=2) == 1 and f(dt=7) == 1
        assert f(codes=None) == 1 and f(sc=None) == 1
        assert f(codes=8) == 3 and f(sc=0x1008) == 3
        assert f(b=1 << 32) == 2 and f(r=1 << 32) == 2
        assert f(b=1 << 20, r=1 << 20, c=128) == 2  # more than 2^31 - 1 tiles
        assert f(b=0) == 0 and f(r=0) == 0
    assert q(x=None) == 1 and q(x=4) == 3
    assert d(out=None) == 1 and d(out=4) == 3


def test_quantize_binding_checks_name_the_argument():
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="x: a matrix"):
        moe.quantize_mx4(torch.zeros(64))
    with pytest.raises(ValueError, match="x: element type"):
        moe.quantize_mx4(x.double())
    with pytest.raises(ValueError, match="x: rows of 40"):
        moe.quantize_mx4(torch.zeros(4, 40))
    with pytest.raises(ValueError, match="codes: 64 elements"):
        moe.quantize_mx4(x, codes=torch.zeros(2, 32, dtype=torch.uint8))
    with pytest.raises(ValueError, match="scales: element type"):
        moe.quantize_mx4(x, scales=torch.zeros(512))
    with pytest.raises(ValueError, match=ON_DEVICE):
        moe.quantize_mx4(x)
    c, s = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(1, 1, 512, dtype=torch.uint8)
    with pytest.raises(ValueError, match="codes: element type"):
        moe.dequantize_mx4(c.float(), s)
    with pytest.raises(ValueError, match="codes: rows of 20"):
        moe.dequantize_mx4(torch.zeros(4, 20, dtype=torch.uint8), s)
    with pytest.raises(ValueError, match="scales: 512 elements"):
        moe.dequantize_mx4(torch.zeros(200, 32, dtype=torch.uint8), s)
    with pytest.raises(ValueError, match="out: element type"):
        moe.dequantize_mx4(c, s, dtype=torch.float16)
    with pytest.raises(ValueError, match=ON_DEVICE):
        moe.dequantize_mx4(c, s)
    with pytest.raises(ValueError, match="multiples of 128"):
        moe.quantize_experts_mx4(torch.zeros(2, 64, 128), torch.zeros(2, 64, 128), torch.zeros(2, 128, 64))


def P(**kw):
    base = dict(T=4, d=256, E=8, k=2, I=128, I_s=128, act="bf16", w="mx4")
    base.update(kw)
    return moe.Problem.make(**base)


@pytest.mark.parametrize("kw,status", [(dict(), 0), (dict(I_s=0), 0), (dict(d=192), 1), (dict(I=64), 1),
                                       (dict(I_s=64), 1), (dict(act="f32"), 2)])
def test_check_problem_with_4_bit_weights(kw, status):
    assert moe.lib().moe_check_problem(ctypes.byref(P(**kw))) == status


def _mx4_args(E=8, d=256, I=128, I_s=128, T=4, k=2):
    z = lambda *s: torch.zeros(s, dtype=torch.uint8)
    blocks = 3 * E * (I // 128) * (d // 128) + 3 * (I_s // 128) * (d // 128)
    return dict(prob=P(), x=torch.zeros(T, d, dtype=torch.bfloat16), w_router=torch.zeros(E, d, dtype=torch.bfloat16),
                bias=None, wg=z(E, I, d // 2), wu=z(E, I, d // 2), wd=z(E, d, I // 2), s_wg=z(I_s, d // 2),
                s_wu=z(I_s, d // 2), s_wd=z(d, I_s // 2), scales=z(blocks * 512))


def test_4_bit_weights_binding_checks():
    for f in (moe.layer_forward, moe.decode_forward):
        with pytest.raises(ValueError, match=ON_DEVICE):
            f(**_mx4_args())
        for name, bad, msg in (("wg", lambda t: t.to(torch.bfloat16), "w_gate: element type"),
                               ("wu", lambda t: t[:7], "w_up:"), ("wd", lambda t: t.reshape(8, 128, 128), "w_down: rows"),
                               ("s_wd", lambda t: t[:100], "ws_down:"), ("scales", lambda t: t[:-1], "scales:"),
                               ("scales", lambda t: t.float(), "scales: element type")):
            a = _mx4_args()
            a[name] = bad(a[name])
            with pytest.raises(ValueError, match=msg):
                f(**a)


def _call_decode(prob, x=16, wr=16, y=16, ws=16, ws_bytes=None, wg=16, sc=16, opt=None, sg=16):
    L = moe.lib()
    v = lambda a: None if a is None else ctypes.c_void_p(a)
    n = moe.decode_workspace_size(prob) if ws_bytes is None else ws_bytes
    return L.moe_decode_forward(ctypes.byref(prob), ctypes.byref(opt) if opt else None, v(x), v(wr), None, v(wg), v(16),
                                v(16), v(sg), v(16), v(16), v(sc), v(y), None, None, v(ws), n, None)


def test_decode_rejected_before_any_launch():
    p = P(w="bf16")
    assert _call_decode(p, x=None) == 1 and _call_decode(p, wr=None) == 1 and _call_decode(p, wg=None) == 1
    assert _call_decode(p, y=0x1008) == 3 and _call_decode(p, sg=None) == 1
    assert _call_decode(p, ws=None) == 1
    assert _call_decode(p, ws_bytes=moe.decode_workspace_size(p) - 1) == 4
    assert _call_decode(P(w="mx4"), sc=None) == 1 and _call_decode(P(w="fp8"), sc=None) == 1
    assert _call_decode(P(T=17)) == 2 and b"moe_layer_forward" in moe.lib().moe_last_error_string()
    assert _call_decode(P(act="f32", w="f32")) == 2
    assert _call_decode(P(k=9)) == 1
    assert _call_decode(p, opt=moe.BlockOptions(16, -1.0, None)) == 1
    assert _call_decode(p, opt=moe.BlockOptions(0x1008, 1e-6, None)) == 3
    assert _call_decode(P(T=0), x=None) == 0
    assert moe.decode_workspace_size(P(T=17)) == 0
    assert 0 < moe.decode_workspace_size(P(T=1)) <= moe.decode_workspace_size(P(T=16))


def test_decode_binding_checks():
    a = _mx4_args()
    a["prob"] = P(T=5)
    with pytest.raises(ValueError, match="x: 1024 elements"):
        moe.decode_forward(**a)
    a = _mx4_args()
    with pytest.raises(ValueError, match="norm_weight"):
        moe.decode_forward(**a, norm_weight=torch.zeros(255, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="topk_ids"):
        moe.decode_forward(**a, topk_ids=torch.zeros(4, 2))


def test_split_scales_takes_scale_tiles():
    from sparse_moe_layer_top_b200 import ep
    E, d, I, I_s, G = 4, 256, 128, 128, 2
    per = (I // 128) * (d // 128) * 512
    s = torch.arange(3 * E * per + 3 * per, dtype=torch.int64)
    tag = (s // per % 251).to(torch.uint8)  # one tag per matrix
    out = [ep.split_scales(r, G, E, d, I, I_s, tag) for r in range(G)]
    m = tag.reshape(-1, per)[:, 0].tolist()
    for r in range(G):
        lo = r * 2
        want = [m[i] for b in range(3) for i in range(b * E + lo, b * E + lo + 2)] + m[3 * E:]
        assert out[r].reshape(-1, per)[:, 0].tolist() == want
        assert (out[r].reshape(-1, per) == out[r].reshape(-1, per)[:, :1]).all()
    with pytest.raises(ValueError, match="scales hold"):
        ep.split_scales(0, G, E, d, I, I_s, tag[:-1])


def test_decode_of_a_layer_makes_the_calls_decode_forward_makes(monkeypatch):
    """The regular call in C++, with the same arguments as decode_forward's."""
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    W = [z(4, 128, 128), z(4, 128, 128), z(4, 128, 128), z(128, 128), z(128, 128), z(128, 128)]
    bias, gamma, gate = torch.zeros(4), z(128), z(128)
    layer = moe.MoELayer(128, 4, 2, 128, 128, z(4, 128), *W, bias=bias, norm_weight=gamma, norm_eps=1e-5,
                         shared_gate=gate)
    calls = []
    monkeypatch.setattr(moe, "_fast_call", lambda *a: calls.append(a) or "y")
    x, y = z(3, 128), z(3, 128)
    ids, tw = torch.zeros((3, 2), dtype=torch.int32), torch.zeros((3, 2))
    assert layer.decode(x, y, ids, tw) == "y"
    assert moe.decode_forward(layer.problem(3), x, layer.w[0], bias, *W, norm_weight=gamma, norm_eps=1e-5,
                              shared_gate=gate, y=y, topk_ids=ids, topk_w=tw) == "y"
    (a, b) = calls
    assert bytes(a[1]) == bytes(b[1]) and len(a) == len(b)
    assert all(p is q for p, q in zip(a[:1] + a[2:], b[:1] + b[2:]))


def test_a_missing_cpp_side_is_reported_once(monkeypatch):
    import sys
    import warnings
    monkeypatch.setitem(sys.modules, "sparse_moe_layer_top_b200._moe_binding", None)
    monkeypatch.delattr(moe, "_moe_binding", raising=False)
    monkeypatch.setattr(moe, "_binding", False)
    with pytest.warns(RuntimeWarning, match="C\\+\\+ side"):
        assert moe._fast() is None
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        assert moe._fast() is None
        with pytest.raises(ValueError, match=ON_DEVICE):
            moe.quantize_mx4(torch.zeros(4, 64))


def test_profile_case_refuses_4_bit_weights_for_a_named_workload(capsys):
    from sparse_moe_layer_top_b200 import profile_case
    with pytest.raises(SystemExit):
        profile_case.main(["--config", "qwen38max_decode_bf16", "--w", "mx4"])
    assert "--w mx4" in capsys.readouterr().err
