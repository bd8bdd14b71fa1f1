"""The C++ side of the binding: a regular call gives what the Python side gives,
bit for bit; anything else is left to the Python side, which says why."""
import pytest
import torch

import moe_inputs
import sparse_moe_layer_top_b200 as moe

pytestmark = pytest.mark.gpu


@pytest.fixture
def python_side(monkeypatch):
    """-> a function that runs f without the C++ side."""
    def run(f):
        monkeypatch.setattr(moe, "_binding", None)
        try:
            return f()
        finally:
            monkeypatch.undo()
    return run


def _weights(w, E=6, d=256, I=128, I_s=128):
    inp = moe_inputs.make_inputs(12, d, E, 2, I, I_s, seed=3, device="cuda")
    ws = [inp.wg, inp.wu, inp.wd, inp.s_wg, inp.s_wu, inp.s_wd]
    if w == "bf16":
        return inp, ws, None
    if w == "mx4":
        *codes, scales = moe.quantize_experts_mx4(*ws)
        return inp, codes, scales
    q = [moe_inputs.quantize_e4m3_blocks(t.cpu()) for t in ws]
    return inp, [a.cuda() for a, _ in q], torch.cat([s.reshape(-1) for _, s in q]).cuda()


def test_the_cpp_side_is_there():
    assert moe._fast() is not None


@pytest.mark.parametrize("shape,dtype", [((5, 64), torch.float32), ((2, 130, 96), torch.bfloat16),
                                         ((2, 1, 3, 256), torch.bfloat16), ((0, 8, 32), torch.float32)])
def test_quantise_and_read_back(shape, dtype, python_side):
    x = torch.randn(shape, device="cuda").to(dtype)
    got = moe.quantize_mx4(x)
    want = python_side(lambda: moe.quantize_mx4(x))
    for a, b in zip(got, want):
        assert a.dtype == b.dtype and a.shape == b.shape and a.device == b.device and torch.equal(a, b)
    for out_type in (torch.bfloat16, torch.float32):
        a = moe.dequantize_mx4(*got, dtype=out_type)
        b = python_side(lambda: moe.dequantize_mx4(*got, dtype=out_type))
        assert a.dtype == out_type and a.shape == x.shape and torch.equal(a, b)
    out = torch.empty(shape, dtype=torch.float32, device="cuda")
    assert moe.dequantize_mx4(*got, out=out) is out and torch.equal(out, moe.dequantize_mx4(*got, dtype=torch.float32))
    c, s = torch.empty_like(got[0]), torch.empty_like(got[1])
    r = moe.quantize_mx4(x, c, s)
    assert r[0] is c and r[1] is s and torch.equal(c, got[0]) and torch.equal(s, got[1])


@pytest.mark.parametrize("w", ["bf16", "fp8", "mx4"])
def test_few_tokens_and_expert_stage(w, python_side):
    inp, ws, scales = _weights(w)
    prob = moe.Problem.make(12, 256, 6, 2, 128, 128, "bf16", w)
    gamma = torch.full((256,), 0.1, dtype=torch.bfloat16, device="cuda")

    def few(**kw):
        return moe.decode_forward(prob, inp.x, inp.w_r, None, *ws, scales=scales, norm_weight=gamma, norm_eps=1e-5, **kw)

    want = python_side(few)
    assert torch.equal(few(), want)
    y = torch.empty_like(inp.x)
    ids = torch.empty((12, 2), dtype=torch.int32, device="cuda")
    assert few(y=y, topk_ids=ids) is y and torch.equal(y, want)
    offs = torch.tensor([0, 5, 5, 9, 12, 20, 24, 36], dtype=torch.int32, device="cuda")
    rows = torch.randn(36, 256, device="cuda").to(torch.bfloat16)

    def experts(**kw):
        return moe.expert_ffn(prob, rows, offs, *ws, scales=scales, **kw)

    want = python_side(experts)
    assert torch.equal(experts(), want)
    y = torch.empty_like(rows)
    assert experts(y_perm=y, ws=torch.empty(moe.stage_workspace_size(prob), dtype=torch.uint8, device="cuda")) is y
    assert torch.equal(y, want)


def test_irregular_calls_are_refused_in_the_python_sides_words():
    inp, ws, scales = _weights("mx4")
    prob = moe.Problem.make(12, 256, 6, 2, 128, 128, "bf16", "mx4")
    few = lambda x=inp.x, w=ws, s=scales, p=prob, **kw: moe.decode_forward(p, x, inp.w_r, None, *w, scales=s, **kw)
    with pytest.raises(ValueError, match="x: element type"):
        few(x=inp.x.float())
    with pytest.raises(ValueError, match="x: .* elements, the problem needs"):
        few(x=inp.x[:11])
    with pytest.raises(ValueError, match="w_down: rows of"):
        few(w=ws[:2] + [ws[2].reshape(6, 128, -1)] + ws[3:])
    with pytest.raises(ValueError, match="scales"):
        few(s=scales[:-1])
    with pytest.raises(ValueError, match="contiguous"):
        few(x=torch.randn(24, 256, device="cuda").to(torch.bfloat16)[::2])
    with pytest.raises(ValueError, match="different devices"):
        few(x=inp.x.cpu())
    with pytest.raises(ValueError, match="topk_ids"):
        few(topk_ids=torch.empty((12, 2), dtype=torch.int64, device="cuda"))
    with pytest.raises(moe.MoEError, match="17 > 16"):
        few(x=inp.x.repeat(2, 1), p=moe.Problem.make(17, 256, 6, 2, 128, 128, "bf16", "mx4"))
    with pytest.raises(moe.MoEError, match="workspace"):
        few(ws=torch.empty(64, dtype=torch.uint8, device="cuda"))
    x = torch.randn(4, 64, device="cuda")
    for bad, what in ((x.half(), "element type"), (x[:, :40], "multiple of 32"), (x[::2], "contiguous"), (x[0], "matrix")):
        with pytest.raises(ValueError, match=what):
            moe.quantize_mx4(bad)
    c, s = moe.quantize_mx4(x)
    with pytest.raises(ValueError, match="codes"):
        moe.quantize_mx4(x, codes=c[:2])
    with pytest.raises(ValueError, match="scales"):
        moe.dequantize_mx4(c, s.reshape(-1)[:100])
    with pytest.raises(ValueError, match="out"):
        moe.dequantize_mx4(c, s, out=torch.empty(4, 64, dtype=torch.int32, device="cuda"))


def test_the_current_stream_is_used():
    """Work queued on a side stream before the call is done before it."""
    s = torch.cuda.Stream()
    x = torch.zeros(64, 4096, device="cuda")
    big = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        for _ in range(4):
            big = big @ big * 1e-3
        x.fill_(3.0)
        c, sc = moe.quantize_mx4(x)
        v = moe.dequantize_mx4(c, sc)
    s.synchronize()
    assert (v == 3).all()


def test_a_call_gives_up_the_interpreters_lock():
    """In the place of the library's entry points a function that says whether its
    thread holds the lock: 0 (the status of success) when it does not."""
    import ctypes
    inp, ws, scales = _weights("mx4")
    prob = moe.Problem.make(12, 256, 6, 2, 128, 128, "bf16", "mx4")
    rows, offs = torch.zeros(36, 256, dtype=torch.bfloat16, device="cuda"), torch.zeros(8, dtype=torch.int32, device="cuda")
    x = torch.zeros(8, 64, device="cuda")
    codes, tiles = moe.quantize_mx4(x)
    stage, few = (torch.empty(f(prob), dtype=torch.uint8, device="cuda")
                  for f in (moe.stage_workspace_size, moe.decode_workspace_size))
    m = moe._fast()
    names = ("moe_mx4_quantize", "moe_mx4_dequantize", "moe_expert_ffn", "moe_stage_workspace_size",
             "moe_decode_workspace_size", "moe_decode_forward")
    real = [ctypes.cast(getattr(moe.lib(), n), ctypes.c_void_p).value for n in names]
    held = ctypes.cast(ctypes.pythonapi.PyGILState_Check, ctypes.c_void_p).value
    m.bind(*[r if n.endswith("_size") else held for n, r in zip(names, real)])
    try:
        got = [m.quantize(x, None, None), m.dequantize(codes, tiles, None, True),
               m.expert_ffn(prob, rows, offs, *ws, scales, None, stage),
               m.decode(prob, inp.x, inp.w_r, None, *ws, scales, None, 1e-6, None, None, None, None, few)]
    finally:
        m.bind(*real)
    assert not any(isinstance(g, int) or g is None for g in got), got
