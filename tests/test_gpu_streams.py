"""Calls on a stream that is not torch's current one: nothing that the current
stream allocates and writes while they run reaches their workspace or outputs."""
import pytest
import torch

import moe_inputs
import sparse_moe_layer_top_b200 as moe

pytestmark = pytest.mark.gpu

T, D, E, K, I, I_S = 200, 1024, 16, 4, 512, 256


def _inputs(w, T=T):
    inp = moe_inputs.make_inputs(T, D, E, K, I, I_S, seed=21, device="cuda")
    W, scales = [inp.wg, inp.wu, inp.wd, inp.s_wg, inp.s_wu, inp.s_wd], None
    if w == "mx4":
        *W, scales = moe.quantize_experts_mx4(*W)
    return inp, W, scales


def _overwrite(nbytes):
    """What a program does next on the current stream: buffers of a workspace's
    and of an output's size, written at once."""
    for n in (nbytes, nbytes // 2, 2 * T * (K + 1) * D, 2 * T * D):
        torch.empty(max(n, 1), dtype=torch.uint8, device="cuda").fill_(255)


@pytest.mark.parametrize("w", ["bf16", "mx4"])
def test_calls_without_a_workspace_on_a_side_stream(w):
    inp, W, scales = _inputs(w)
    prob = moe.Problem.make(T, D, E, K, I, I_S, "bf16", w)
    few = moe.Problem.make(9, D, E, K, I, I_S, "bf16", w)
    ids, tw = moe.router_topk(prob, inp.x, inp.w_r)
    perm = moe.permute(prob, inp.x, ids, tw)
    s = torch.cuda.Stream()
    calls = [
        (lambda **kw: moe.expert_ffn(prob, perm["x_perm"], perm["offs"], *W, scales=scales, **kw),
         moe.stage_workspace_size(prob)),
        (lambda **kw: moe.layer_forward(prob, inp.x, inp.w_r, None, *W, scales=scales, **kw),
         moe.workspace_size(prob)),
        (lambda **kw: moe.decode_forward(few, inp.x[:9], inp.w_r, None, *W, scales=scales, **kw),
         moe.decode_workspace_size(few)),
    ]
    for call, nbytes in calls:
        want = call()
        torch.cuda.synchronize()
        for _ in range(5):
            got = call(stream=s)
            _overwrite(nbytes)
            torch.cuda.synchronize()
            assert torch.equal(got, want)
    assert moe.device_status()[0] == 0


@pytest.mark.parametrize("w", ["bf16", "mx4"])
def test_one_layers_decode_on_two_streams_and_in_a_graph_at_once(w):
    inp, W, scales = _inputs(w)
    layer = moe.MoELayer(D, E, K, I, I_S, inp.w_r, *W, scales=scales, w=w)
    xs = [inp.x[:1], inp.x[1:12], inp.x[12:15].clone()]
    want = [layer.decode(x) for x in xs]
    torch.cuda.synchronize()
    sa, sb, sc = (torch.cuda.Stream() for _ in range(3))
    y = torch.empty_like(want[2])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=sc):
        layer.decode(xs[2], y, stream=sc)
    for _ in range(20):
        y.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(sc):
            g.replay()
        a, b = layer.decode(xs[0], stream=sa), layer.decode(xs[1], stream=sb)
        _overwrite(moe.decode_workspace_size(layer.problem(16)))
        torch.cuda.synchronize()
        assert torch.equal(a, want[0]) and torch.equal(b, want[1]) and torch.equal(y, want[2])
    assert moe.device_status()[0] == 0


@pytest.mark.parametrize("w", ["bf16", "mx4"])
def test_a_layers_forward_on_side_streams_and_in_a_graph(w):
    """One layer: a first call on a side stream, calls on two streams in turn, and
    a captured one that stays right after the layer's workspace has grown."""
    inp, W, scales = _inputs(w)
    layer = moe.MoELayer(D, E, K, I, I_S, inp.w_r, *W, scales=scales, w=w)
    small = inp.x[:40].clone()
    ref = moe.MoELayer(D, E, K, I, I_S, inp.w_r, *W, scales=scales, w=w, max_tokens=T)
    want, want_small = ref(inp.x), ref(small)
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    got = layer(small, stream=sa)
    _overwrite(moe.workspace_size(layer.problem(40)))
    torch.cuda.synchronize()
    assert torch.equal(got, want_small)
    y = torch.empty_like(small)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=sa):
        layer(small, y, stream=sa)
    big = layer(inp.x)  # the workspace grows
    _overwrite(moe.workspace_size(layer.problem(40)))
    y.zero_()
    torch.cuda.synchronize()
    g.replay()
    outs = [layer(inp.x, stream=s) for s in (sa, sb, sa, sb)]
    torch.cuda.synchronize()
    assert torch.equal(big, want) and torch.equal(y, want_small)
    assert all(torch.equal(o, want) for o in outs)
    assert moe.device_status()[0] == 0


@pytest.mark.parametrize("method", ["forward", "decode"])
def test_one_layer_from_two_threads(method):
    import threading
    inp, W, scales = _inputs("mx4")
    layer = moe.MoELayer(D, E, K, I, I_S, inp.w_r, *W, scales=scales, w="mx4", max_tokens=T)
    xs = [inp.x, inp.x[:70].clone()] if method == "forward" else [inp.x[:3].clone(), inp.x[5:16].clone()]
    call = layer if method == "forward" else layer.decode
    want = [call(x) for x in xs]
    torch.cuda.synchronize()
    bad, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]

    def work(i):
        try:
            with torch.cuda.stream(streams[i]):
                for _ in range(40):
                    if not torch.equal(call(xs[i]), want[i]):
                        bad.append(i)
        except Exception as e:
            bad.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad and moe.device_status()[0] == 0
