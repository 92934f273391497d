"""Captured graphs of the operators replayed at once on several streams, beside eager calls: each answers as it does
alone.  The routed layer's CTAs wait for one another and want the whole GPU, so two of its launches may not share it
half and half."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def sot():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import sinkhorn_point_cloud_gb300 as s
    from sinkhorn_point_cloud_gb300 import build
    build.build()
    return s


def layer(seed, T, H, E, F, dtype):
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = lambda *n: (torch.randn(*n, generator=g, device="cuda") * n[-1] ** -0.5).to(dtype)  # noqa: E731
    return H ** 0.5 * w(T, H), w(E, H), w(E, 2 * F, H), w(E, H, F)


def test_graphs_at_once(sot):
    layers = [(layer(1, 3, 1024, 16, 256, torch.bfloat16), 4), (layer(2, 40, 512, 24, 320, torch.float16), 2),
              (layer(3, 128, 256, 8, 128, torch.bfloat16), 2)]
    g = torch.Generator(device="cuda").manual_seed(0)
    logits, grad = torch.randn(12, 60000, generator=g, device="cuda"), torch.randn(5000, 64, generator=g, device="cuda")
    ids = torch.randint(0, 700, (5000,), generator=g, device="cuda")
    calls = [lambda a=a, k=k: sot.sot_routed_layer(*a, k) for a, k in layers]
    calls += [lambda: sot.sot_token_topk(logits, 200)[1:], lambda: (sot.sot_embed_grad(grad, ids, 700),)]
    alone = [c() for c in calls]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for c in calls:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append([c() for _ in range(3)])
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(20):
        eager = []
        for s, graph, c in zip(streams, graphs, calls):
            with torch.cuda.stream(s):
                graph.replay()
                eager.append(c())
                graph.replay()
        torch.cuda.synchronize()
        sot.sot_async_status()  # no wait has run out
        for out, e, ref in zip(outs, eager, alone):
            for got in (*out, e):
                for a, b in zip(got, ref):
                    assert torch.equal(a, b)
