"""What the binding allocates for a call belongs to the stream the call runs on.

The caching allocator hands a freed block out again on the stream that it was
allocated on, at once: a workspace from another stream's pool may still be used
by work queued there, and goes back there while the call's own kernels run.
Here, without a GPU, torch.cuda.stream and the library's launches are replaced
by recorders; the calls themselves are the binding's."""
import contextlib

import pytest
import torch

import sparse_moe_layer_top_b200 as moe

T, D, E, K, I = 12, 128, 4, 2, 128
ROWS = T * (K + 1)


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle
        self.device = torch.device("cpu")


@pytest.fixture
def recorded(monkeypatch):
    """-> (list of the stream in effect at each allocation, list of (entry point, stream) launches)."""
    allocs, launches, stack = [], [], []

    @contextlib.contextmanager
    def use(stream):
        stack.append(stream)
        try:
            yield
        finally:
            stack.pop()

    class Lib:
        def __getattr__(self, name):
            if name.endswith("_size") or name.endswith("_bytes"):
                return getattr(real, name)
            return lambda *a: launches.append((name, a[-1])) or 0

    real, empty, empty_like = moe.lib(), torch.empty, torch.empty_like
    monkeypatch.setattr(moe, "_lib", Lib())
    monkeypatch.setattr(moe, "_ptr", lambda t: None if t is None else t.data_ptr())
    monkeypatch.setattr(torch.cuda, "stream", use)
    for name, f in (("empty", empty), ("empty_like", empty_like)):
        monkeypatch.setattr(torch, name,
                            lambda *a, f=f, **kw: allocs.append(stack[-1] if stack else None) or f(*a, **kw))
    return allocs, launches


def _block():
    bf = torch.bfloat16
    z = lambda *s, t=bf: torch.zeros(s, dtype=t)
    return dict(x=z(T, D), w_router=z(E, D), wg=z(E, I, D), wu=z(E, I, D), wd=z(E, D, I), s_wg=z(I, D), s_wu=z(I, D),
                s_wd=z(D, I))


def _calls():
    p = moe.Problem.make(T, D, E, K, I, I, "bf16", "bf16")
    b = _block()
    x = b["x"]
    rows = torch.zeros((ROWS, D), dtype=torch.bfloat16)
    ids, tw = torch.zeros((T, K), dtype=torch.int32), torch.zeros((T, K))
    offs = torch.zeros(E + 2, dtype=torch.int32)
    W = [b[n] for n in ("wg", "wu", "wd", "s_wg", "s_wu", "s_wd")]
    codes = [torch.zeros(t.shape[:-1] + (t.shape[-1] // 2,), dtype=torch.uint8) for t in W]
    scales = torch.full((sum(t.numel() // 32 for t in W),), 127, dtype=torch.uint8)
    p4 = moe.Problem.make(T, D, E, K, I, I, "bf16", "mx4")
    return {
        "router_topk": lambda s: moe.router_topk(p, x, b["w_router"], stream=s),
        "permute": lambda s: moe.permute(p, x, ids, tw, stream=s),
        "expert_ffn": lambda s: moe.expert_ffn(p, rows, offs, *W, stream=s),
        "expert_ffn, 4-bit": lambda s: moe.expert_ffn(p4, rows, offs, *codes, scales=scales, stream=s),
        "combine": lambda s: moe.combine(p, rows, ids, tw, offs, stream=s),
        "layer_forward": lambda s: moe.layer_forward(p, x, b["w_router"], None, *W, stream=s),
        "block_forward": lambda s: moe.block_forward(p, x, b["w_router"], None, *W, stream=s),
        "decode_forward": lambda s: moe.decode_forward(p, x, b["w_router"], None, *W, stream=s),
        "rmsnorm": lambda s: moe.rmsnorm(p, x, torch.zeros(D, dtype=torch.bfloat16), stream=s),
        "ep_expand_ids": lambda s: moe.ep_expand_ids(torch.zeros(E, dtype=torch.int32), 1, E, 5, stream=s),
        "quantize_mx4": lambda s: moe.quantize_mx4(x, stream=s),
        "dequantize_mx4": lambda s: moe.dequantize_mx4(codes[0], scales[:E * I * D // 32], stream=s),
    }


@pytest.mark.parametrize("name", list(_calls()))
def test_a_call_allocates_on_the_stream_it_runs_on(name, recorded):
    allocs, launches = recorded
    s = Stream(41)
    calls = _calls()
    allocs.clear()
    calls[name](s)
    assert allocs and all(a is s for a in allocs), allocs
    assert len(launches) == 1 and launches[0][1] == 41, launches


def _layer(**kw):
    b = _block()
    return moe.MoELayer(D, E, K, I, I, *[b[n] for n in ("w_router", "wg", "wu", "wd", "s_wg", "s_wu", "s_wd")], **kw)


def test_decode_of_a_layer_has_a_workspace_of_its_own_on_every_stream(recorded):
    allocs, launches = recorded
    layer = _layer()
    x, y = torch.zeros((3, D), dtype=torch.bfloat16), torch.zeros((3, D), dtype=torch.bfloat16)
    s1, s2 = Stream(41), Stream(42)
    allocs.clear()
    for s in (s1, s2, s1):
        layer.decode(x, y, stream=s)
    assert allocs == [s1, s2, s1]
    assert [l[1] for l in launches] == [41, 42, 41]


def test_a_layers_workspace_is_ordered_between_streams_and_never_a_graphs(recorded, monkeypatch):
    """One buffer, and a call on another stream waits for the last one's; a
    captured call allocates for itself, so that a later growth takes nothing
    from its graph."""
    allocs, launches = recorded
    waits, state = [], {"capturing": None}

    class S(Stream):
        def wait_stream(self, other):
            waits.append((self.cuda_stream, other.cuda_stream))

    home, s1, s2 = S(40), S(41), S(42)
    for s in (home, s1, s2):
        s.device = torch.device("cuda", 0)
    enter = torch.cuda.stream
    stack = [home]

    @contextlib.contextmanager
    def use(stream):
        stack.append(stream)
        with enter(stream):
            yield
        stack.pop()

    monkeypatch.setattr(torch.cuda, "stream", use)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: stack[-1])
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: stack[-1] is state["capturing"])
    monkeypatch.setattr(moe, "_stream", lambda stream=None: (stream or stack[-1]).cuda_stream)
    monkeypatch.setattr(moe, "_device", lambda *a, **kw: torch.device("cuda", 0))
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: None)
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **kw: empty(*a, **kw))
    layer = _layer()
    layer.device = torch.device("cuda", 0)
    layer._reserve(layer.problem(T))
    ws = layer.ws
    x, y = torch.zeros((T, D), dtype=torch.bfloat16), torch.zeros((T, D), dtype=torch.bfloat16)
    used = []
    monkeypatch.setattr(moe, "_forward_call", lambda *a: used.append((a[17], a[18])))
    layer(x, y)
    layer(x, y, stream=s1)
    layer(x, y, stream=s1)
    layer(x, y, stream=s2)
    assert [u[0] is ws for u in used] == [True] * 4 and [u[1] for u in used] == [None, s1, s1, s2]
    assert waits == [(41, 40), (42, 41)]
    used.clear()
    state["capturing"] = s1
    allocs.clear()
    layer(x, y, stream=s1)
    assert used[0][0] is not ws and allocs == [s1] and layer.ws is ws and waits[2:] == []
    state["capturing"] = None
    x = torch.zeros((4 * T, D), dtype=torch.bfloat16)
    layer(x, torch.zeros_like(x), stream=s1)  # grows on the stream that uses it
    assert layer.ws is not ws and allocs[1:] == [s1] and layer.ws_stream is s1 and waits[2:] == [(41, 42)]
    state["capturing"], ws = s1, layer.ws
    layer(x, torch.zeros_like(x), stream=s2)  # a wait for s1 would join its capture
    assert layer.ws is not ws and allocs[2:] == [s2] and layer.ws_stream is s2 and waits[3:] == []


def test_a_layer_queues_one_call_at_a_time_and_can_be_copied(recorded, monkeypatch):
    import copy
    import pickle
    layer = _layer()
    x, y = torch.zeros((T, D), dtype=torch.bfloat16), torch.zeros((T, D), dtype=torch.bfloat16)
    held = []
    monkeypatch.setattr(moe, "_forward_call", lambda *a: held.append(layer.lock.locked()))
    layer(x, y)
    assert held == [True] and not layer.lock.locked()
    for other in (copy.copy(layer), copy.deepcopy(layer), pickle.loads(pickle.dumps(layer))):
        assert other.ws is None and other.lock is not layer.lock and not other.lock.locked()
        assert torch.equal(other.w[2], layer.w[2]) and other.shape == layer.shape
