"""The decoding example runs: tokens with their scores, entropies and alternatives; and the routed layer answers
the same beside calls on another stream."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def sot():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import sinkhorn_point_cloud_gb300 as s
    from sinkhorn_point_cloud_gb300 import build
    build.build()
    return s


def test_decoding_example_runs(sot):
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import routed_lm_decode as d
    said, logps, entropies, best, counts = d.decode(tokens=6, sequences=3, alternatives=5)
    assert tuple(said.shape) == tuple(logps.shape) == tuple(entropies.shape) == (6, 3) and tuple(best.shape) == (6, 3, 5)
    assert ((said >= 0) & (said < d.VOCAB)).all() and (logps <= 0).all() and (entropies > 0).all()
    assert all(int(c.sum()) == 6 * 3 * d.CHOICES for c in counts)


def test_training_example_with_entropy_bonus(sot):
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import routed_lm_step
    h = routed_lm_step.train(steps=3, report=False, bonus=0.01)
    assert len(h) == 3 and all(v == v for step in h for v in step.values())


def test_lookup_gradient_matches_indexing(sot):
    """The example's embedding against torch's indexing: values and gradients."""
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    from routed_lm_step import Lookup
    g = torch.Generator(device="cuda").manual_seed(0)
    table = torch.randn(50, 24, generator=g, device="cuda", requires_grad=True)
    tokens = torch.randint(0, 50, (700,), generator=g, device="cuda")
    w = torch.randn(700, 24, generator=g, device="cuda")
    a, = torch.autograd.grad((Lookup.apply(table, tokens) * w).sum(), table)
    b, = torch.autograd.grad((table.double()[tokens] * w.double()).sum(), table)
    size, = torch.autograd.grad((table.double()[tokens] * w.double().abs()).sum(), table)
    assert torch.equal(Lookup.apply(table, tokens), table[tokens])
    # up to 700 additions of 2^-24 of the terms' size each
    assert ((a - b).abs() <= 700 * 2.0 ** -24 * size).all()


def test_routed_layers_on_two_streams(sot):
    """Calls of two streams under way at once, each of which wants the whole GPU: each answers as it does alone."""
    def inputs(seed, T, H, E, F):
        g = torch.Generator(device="cuda").manual_seed(seed)
        w = lambda *n: (torch.randn(*n, generator=g, device="cuda") * n[-1] ** -0.5).bfloat16()  # noqa: E731
        return H ** 0.5 * w(T, H), w(E, H), w(E, 2 * F, H), w(E, H, F)
    args = [inputs(1, 3, 256, 8, 128), inputs(2, 40, 512, 16, 192)]
    alone = [sot.sot_routed_layer(*a, 2) for a in args]
    streams = [torch.cuda.Stream() for _ in args]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(30):
        for i, s in enumerate(streams):
            got[i].append(sot.sot_routed_layer(*args[i], 2, stream=s))
    torch.cuda.synchronize()
    sot.sot_async_status()
    for i in (0, 1):
        for out in got[i]:
            for a, b in zip(out, alone[i]):
                assert torch.equal(a, b)


def test_routed_layer_of_many_tokens_and_few_stages(sot):
    """128 tokens that all choose the same experts: the widest token side, the fewest places in the ring."""
    import numpy as np

    import lm_operators_ref as R
    rng = np.random.default_rng(3)
    f = lambda *n, s=1.0: torch.from_numpy((s * rng.standard_normal(n)).astype(np.float32)).bfloat16().cuda()  # noqa: E731
    T, H, E, F = 128, 1536, 6, 320
    x, router, gu, dn = f(T, H), f(E, H, s=H ** -0.5), f(E, 2 * F, H, s=H ** -0.5), f(E, H, F, s=F ** -0.5)
    bias = torch.tensor([0.0, 60.0, 0.0, 50.0, 0.0, 0.0]).cuda()
    out, logits, ids, w = sot.sot_routed_layer(x, router, gu, dn, 2, bias=bias)
    assert (ids.cpu().numpy() == [1, 3]).all()
    h = lambda t: t.double().cpu().numpy()  # noqa: E731
    ro, _, _, rw, size = R.routed(h(x), h(router), h(gu), h(dn), 2, h(bias), True, 1.0)
    # bf16: half an ulp of the output and of each term's h, and the sums' 2^-16
    assert (np.abs(h(out) - ro) <= 2.0 ** -8 * np.abs(ro) + (2.0 ** -8 + 2.0 ** -15) * size).all()
    again = sot.sot_routed_layer(x, router, gu, dn, 2, bias=bias)[0]
    assert torch.equal(out, again)
