"""The layer's calls allocate on the stream that they are given, and run on their
tensors' device (CPU only: the library, the switch and the tensors' place are
stood in for)."""
import pytest
import torch

from sparse_mixture_experts_noisy_b200 import moe


class Switch:
    depth = 0

    def __enter__(self):
        Switch.depth += 1

    def __exit__(self, *a):
        Switch.depth -= 1


class Lib:
    def __init__(self, calls):
        self.calls = calls

    def __getattr__(self, name):
        def f(*a):
            if name.endswith("_size"):
                return 1024
            if name == "moe_gathered_rows":
                return 128
            self.calls.append((name, Switch.depth))
            return 0
        return f


class Tensor(torch.Tensor):
    is_cuda = True


def fake(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(Tensor)


I32 = torch.int32
N, D, E, F, K, R = 4, 8, 3, 16, 2, 128


def arguments():
    x, topk, gates = fake(N, D), fake(N, K, dtype=I32), fake(N, K)
    xg, off, cnt, up, dn = fake(R, D), fake(E + 1, dtype=I32), fake(E, dtype=I32), fake(E, F, D), fake(E, D, F)
    H, Wg, ws = fake(R, F), fake(E, D), fake(4096, dtype=torch.uint8)
    return {
        "moe_route": (x, Wg, K), "moe_dispatch": (topk, x, E, None), "moe_dispatch_noalloc": (topk, x, E, None),
        "moe_shard_count": (topk, E, ws), "moe_shard_base": (fake(2, K, E, dtype=I32), 0),
        "moe_shard_dispatch": (topk, x, E, 4, fake(K, E, dtype=I32), fake(K, E, dtype=I32), ws),
        "moe_expert_ffn": (xg, off, cnt, up, dn), "moe_expert_ffn_train": (xg, off, cnt, up, dn),
        "moe_backward": (x, Wg, up, dn, K, topk, gates, topk, off, cnt, xg, H, xg, x),
        "moe_combine": (xg, topk, topk, off, gates), "moe_load_stats": (topk, E, None),
        "moe_forward": (x, Wg, up, dn, K, None),
    }


@pytest.fixture
def calls(monkeypatch):
    seen, allocated = [], []
    lib = Lib(seen)
    Switch.depth = 0
    monkeypatch.setattr(moe, "load_library", lambda *a: lib)
    monkeypatch.setattr(moe, "_elsewhere", lambda t, stream: None if stream is None else Switch())
    monkeypatch.setattr(moe, "_stream", lambda stream: "current" if stream is None else stream)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    empty = torch.empty

    def note(*a, **k):
        allocated.append(Switch.depth)
        return empty(*a, **k)
    monkeypatch.setattr(torch, "empty", note)
    return seen, allocated


@pytest.mark.parametrize("name", sorted(arguments()))
def test_a_given_stream_is_current_for_allocations_and_kernels(calls, name):
    seen, allocated = calls
    args = arguments()[name]
    f = getattr(moe, name)
    f(*args, stream="side")
    launches = [c for c in seen if c[0].startswith("moe_")]
    assert launches and allocated and all(d == 1 for _, d in launches) and all(d == 1 for d in allocated)
    assert Switch.depth == 0
    seen.clear(), allocated.clear()
    f(*args)
    assert seen and all(d == 0 for _, d in seen) and all(d == 0 for d in allocated)


def test_a_stream_by_position(calls):
    seen, allocated = calls
    moe.moe_combine(*arguments()["moe_combine"], "side")
    assert all(d == 1 for _, d in seen) and all(d == 1 for d in allocated)


def test_the_layer(calls):
    seen, allocated = calls
    a = arguments()["moe_forward"]
    layer = moe.MoELayer(a[1], a[2], a[3], K, None)
    layer(a[0], stream="side")
    assert seen and all(d >= 1 for _, d in seen) and all(d >= 1 for d in allocated)


class OneRank:
    def __init__(self, seen):
        self.seen = seen

    def world(self):
        return 1

    def rank(self):
        return 0

    def all_gather(self, t):
        self.seen.append(("all_gather", Switch.depth))
        return torch.zeros_like(t).unsqueeze(0)

    def all_to_all(self, out, given):
        self.seen.append(("all_to_all", Switch.depth))


def test_collectives_follow_the_kernels(calls, monkeypatch):
    """The exchanges read what the kernels wrote: they belong on the same stream."""
    from sparse_mixture_experts_noisy_b200 import ep, shard
    seen, allocated = calls
    monkeypatch.setattr(moe, "_cuda", lambda t, name: None)   # what torch.empty gives here is on the host
    x, Wg, up, dn, _, _ = arguments()["moe_forward"]
    ep.expert_parallel_forward(x, Wg, up, dn, K, None, N, comm=OneRank(seen), stream="side")
    names = {n for n, _ in seen}
    assert {"all_gather", "all_to_all", "moe_shard_dispatch", "moe_combine"} <= names
    assert all(d >= 1 for _, d in seen) and all(d >= 1 for d in allocated)
    seen.clear(), allocated.clear()
    monkeypatch.setattr(shard.dist, "get_rank", lambda group: 0)
    monkeypatch.setattr(shard, "exchange_counts", lambda t, group: OneRank(seen).all_gather(t))
    shard.sharded_forward(x, Wg, up, dn, K, None, N, stream="side")
    assert "all_gather" in {n for n, _ in seen}
    assert all(d >= 1 for _, d in seen) and all(d >= 1 for d in allocated)
    assert Switch.depth == 0


def test_a_capture_is_on_the_inputs_device(calls, monkeypatch):
    """GraphedForward switches to its input's device for the warm-up and the capture."""
    inside = []

    class On:
        def __init__(self, device=None):
            self.device = device

        def __enter__(self):
            inside.append(self)

        def __exit__(self, *a):
            inside.pop()

        def wait_stream(self, other):
            assert inside

    seen = []
    monkeypatch.setattr(torch.cuda, "device", On)
    monkeypatch.setattr(torch.cuda, "Stream", lambda device=None: seen.append(bool(inside)) or On())
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: seen.append(bool(inside)) or On())
    monkeypatch.setattr(torch.cuda, "stream", lambda s: On())
    monkeypatch.setattr(torch.cuda, "graph", lambda g, stream: On())
    monkeypatch.setattr(torch.cuda, "CUDAGraph", On)
    monkeypatch.setattr(torch.cuda, "synchronize", lambda device=None: None)

    class Layer:
        def _reserve(self, n, dtype):
            seen.append(bool(inside))

        def __call__(self, x, noise=None, y=None):
            seen.append(len(inside) >= 2)   # the device, then the stream or the capture

    moe.GraphedForward(Layer(), fake(N, D))
    assert len(seen) == 6 and all(seen) and not inside
