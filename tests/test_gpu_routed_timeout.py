"""The bounded waits of the routed layer's tensor-core kernel give up cleanly: a call whose wait runs out has an output
of NaN and SOT_ERR_TIMEOUT, and the next call is right.  The failure is made by a testing hook: one CTA withholds
its arrival at a meeting of all CTAs, or its weights from some unit of work on, with a limit of 1 ms; nothing faults, nothing
hangs."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

LIMIT_NS = 1_000_000  # 1 ms


@pytest.fixture(scope="module")
def sot():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import sinkhorn_point_cloud_gb300 as s
    from sinkhorn_point_cloud_gb300 import build
    build.build()
    return s


@pytest.fixture(autouse=True)
def hook_off(sot):
    yield
    sot.sot_test_hold_routed(-1)
    torch.cuda.synchronize()
    try:
        sot.sot_async_status()
    except sot.SotError:
        pass


def inputs(T, H, E, F, dtype):
    g = torch.Generator(device="cuda").manual_seed(T)
    w = lambda *n: (torch.randn(*n, generator=g, device="cuda") * n[-1] ** -0.5).to(dtype)  # noqa: E731
    return H ** 0.5 * w(T, H), w(E, H), w(E, 2 * F, H), w(E, H, F)


def dirty():
    """Memory that a call's outputs are taken from holds what no expert's number is."""
    keep = [torch.full((n,), 0x7f7f7f7f, dtype=torch.int32, device="cuda") for n in (8, 32, 64, 128, 256, 512, 1024, 4096, 16384)]
    torch.cuda.synchronize()
    del keep


# meetings 0, 2 and, where a call has them, 1 and 3; units of the first and of the second product
CASES = [(1, 2, w) for w in (0, 2, 4, 5)] + [(8, 2, w) for w in (0, 2, 4)] + [(8, 4, 1)] + \
    [(40, 4, w) for w in (0, 1, 2, 3, 4, 5, 7)] + [(128, 8, w) for w in (1, 3, 4, 6)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,K,what", CASES)
def test_timeout_reported(sot, T, K, what, dtype):
    args = inputs(T, 1024, 16, 512, dtype)
    good = sot.sot_routed_layer(*args, K)
    sot.sot_async_status()
    sot.sot_test_hold_routed(what, LIMIT_NS)
    dirty()
    bad = sot.sot_routed_layer(*args, K)
    with pytest.raises(sot.SotError) as ei:
        sot.sot_async_status()
    assert ei.value.status == sot.SOT_ERR_TIMEOUT
    assert torch.isnan(bad[0]).all()
    for a, b in zip(bad[1:], good[1:]):
        assert torch.equal(a, b)  # scores, choices and weights do not depend on what was waited for
    sot.sot_async_status()  # cleared by the previous read
    sot.sot_test_hold_routed(-1)
    for a, b in zip(sot.sot_routed_layer(*args, K), good):
        assert torch.equal(a, b)
    sot.sot_async_status()


def test_many_timeouts_in_a_row(sot):
    """With every kind of wait running out, one call behind another."""
    args = inputs(33, 512, 8, 256, torch.bfloat16)
    good = sot.sot_routed_layer(*args, 2)
    for _ in range(6):
        for what in (0, 1, 2, 3, 4, 5):
            sot.sot_test_hold_routed(what, LIMIT_NS // 2)
            assert torch.isnan(sot.sot_routed_layer(*args, 2)[0]).all()
    sot.sot_test_hold_routed(-1)
    with pytest.raises(sot.SotError):
        sot.sot_async_status()
    assert torch.equal(sot.sot_routed_layer(*args, 2)[0], good[0])
    sot.sot_async_status()


def test_nothing_withheld(sot):
    """A unit that the CTA does not have, and another limit: nothing changes."""
    args = inputs(40, 1024, 16, 512, torch.bfloat16)
    good = sot.sot_routed_layer(*args, 4)
    sot.sot_test_hold_routed(4 + (1 << 20), 1_000_000_000)
    for a, b in zip(sot.sot_routed_layer(*args, 4), good):
        assert torch.equal(a, b)
    sot.sot_async_status()
