"""What the routed layer's tensor-core form keeps of silu(gate x) * (up x) between its two products: the digits of
32-bit sums and, in fp16, their range.

Tolerances.  A sum of n products of 16-bit values in 32 bits, added in steps of 16, in up to 153 pieces and a tree over
them: under n / 16 + 8 roundings of 2^-23 each (the accumulators may cut off instead of rounding) of the sum of the absolute
terms; written here for gate, up and the second product.  silu is 1.1-Lipschitz.  h in two parts is good to 2^-17 of itself
(bf16; fp16 2^-22), the exponential, the quotient and the products to 2^-21 together, the softmax weight to
2^-20; the output is rounded once, half an ulp.  One part alone would be off by 2^-9 (bf16) or 2^-12 of h."""
import numpy as np
import pytest

import lm_operators_ref as R

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

HALF_ULP = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f16": 2.0 ** -25, "bf16": 2.0 ** -126}
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
PART = {"f16": 2.0 ** -22, "bf16": 2.0 ** -17}


@pytest.fixture(scope="module")
def sot():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import sinkhorn_point_cloud_gb300 as s
    from sinkhorn_point_cloud_gb300 import build
    build.build()
    return s


def inputs(T, H, E, F, dtype, seed, x=1.0, gu=1.0, dn=1.0):
    rng = np.random.default_rng(seed)
    f = lambda *n, s=1.0: (s * torch.from_numpy(rng.standard_normal(n))).to(TYPES[dtype]).cuda()  # noqa: E731
    return [f(T, H, s=x), f(E, H, s=H ** -0.5 / max(x, 1.0)), f(E, 2 * F, H, s=gu * H ** -0.5), f(E, H, F, s=dn * F ** -0.5)]


def bounds(x, gate_up, down, ids, w, dtype):
    """Size of the error of each output before its own rounding."""
    (T, H), F = x.shape, down.shape[2]
    step1, step2 = (H / 16 + 8) * 2.0 ** -23, (F / 16 + 8) * 2.0 ** -23
    err = np.zeros(x.shape)
    for t in range(T):
        for e, s in zip(ids[t], w[t]):
            if e < 0:
                continue
            a, mass = gate_up[e] @ x[t], np.abs(gate_up[e]) @ np.abs(x[t])
            g, u, mg, mu = a[:F], a[F:], mass[:F], mass[F:]
            with np.errstate(over="ignore"):
                h = np.abs(g / (1 + np.exp(-g)) * u)
            dh = step1 * (1.1 * mg * (np.abs(u) + step1 * mu) + np.abs(g) * mu) + (PART[dtype] + 2.0 ** -21) * h
            err[t] += abs(s) * (np.abs(down[e]) @ (dh + (step2 + 2.0 ** -20) * h))
    return err


def check(sot, args, K, dtype, renorm=True):
    x, router, gu, dn = (t.double().cpu().numpy() for t in args)
    with np.errstate(over="ignore"):
        ref, _, ids, w, _ = R.routed(x, router, gu, dn, K, None, renorm, 1.0)
    out, _, got, _ = sot.sot_routed_layer(*args, K, renorm=renorm)
    assert np.array_equal(got.cpu().numpy(), ids)
    out = out.double().cpu().numpy()
    assert np.isfinite(ref).all() and np.abs(ref).max() < 6e4 and np.isfinite(out).all()
    over = np.abs(out - ref) - HALF_ULP[dtype] * np.abs(ref) - bounds(x, gu, dn, ids, w, dtype) - TINY[dtype]
    assert over.max() <= 0, over.max()
    return out


SHAPES = [(1, 128, 6, 16, 2), (4, 256, 9, 24, 4), (40, 256, 8, 64, 4), (96, 128, 2, 200, 2), (20, 1032, 3, 72, 1)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("T,H,E,F,K", SHAPES)
def test_digits_between_the_products(sot, T, H, E, F, K, dtype):
    check(sot, inputs(T, H, E, F, dtype, T), K, dtype)
    check(sot, inputs(T, H, E, F, dtype, T + 1), K, dtype, renorm=False)


@pytest.mark.parametrize("T,H,E,F,K", SHAPES)
@pytest.mark.parametrize("gu,dn", [(600.0, 1e-3), (6e3, 1e-4), (3e-3, 1e2), (3e-4, 3e3)])
def test_half_precision_keeps_its_range(sot, T, H, E, F, K, gu, dn):
    """gate and up of some hundreds to thousands, whose product lies beyond 65504, or of 2^-9 to 2^-12, whose product lies below
    the type's smallest number; the outputs are ordinary ones."""
    args = inputs(T, H, E, F, "f16", T, gu=gu, dn=dn)
    out = check(sot, args, K, "f16")
    a = args[2].double() @ args[0].double().T  # [E, 2 F, T]
    most = (torch.nn.functional.silu(a[:, :F]) * a[:, F:]).abs().amax()
    assert (most > 65504 if gu > 1 else most < 2.0 ** -12) and np.abs(out).max() > 1e-4


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("T", [3, 33])
def test_tokens_of_all_sizes_beside_each_other(sot, T, dtype):
    """Tokens 2^-8 to 2^8 as large as others of the same expert, one of them zeros."""
    args = inputs(T, 192, 4, 40, dtype, 5, gu=4.0, dn=2.0 ** -8)
    args[0].mul_((2.0 ** ((torch.arange(T) * 5) % 17 - 8.0)).cuda()[:, None].to(args[0].dtype))
    args[0][1] = 0
    args[1].zero_()  # (all tokens to the first experts)
    check(sot, args, 2, dtype)


@pytest.mark.parametrize("T", [2, 40])
def test_both_forms_agree_beyond_the_range(sot, T):
    """The same call with x at an address that the tensor cores' copies do not take."""
    args = inputs(T, 128, 6, 64, "f16", 7, gu=600.0, dn=1e-3)
    wide = torch.zeros(T, 130, dtype=torch.float16, device="cuda")
    wide[:, 1:129] = args[0]
    a, b = sot.sot_routed_layer(*args, 2)[0], sot.sot_routed_layer(wide[:, 1:129], *args[1:], 2)[0]
    assert torch.isfinite(a).all() and torch.isfinite(b).all()
    size = b.float().abs().amax(1, keepdim=True)
    assert ((a.float() - b.float()).abs() <= 2 * HALF_ULP["f16"] * b.float().abs() + 2.0 ** -13 * size).all()


@pytest.mark.parametrize("T", [2, 40])
def test_infinite_between_the_products(sot, T):
    """An h beyond 32 bits' range, and NaN among the weights, reach the tokens of that expert and no others."""
    args = inputs(T, 64, 4, 24, "bf16", 9)
    args[1].zero_()
    args[1][:2, 0], args[0][:, 0] = torch.tensor([1.0, -1.0], device="cuda").bfloat16(), 1.0
    args[0][1::2, 0] = -1.0  # odd tokens to expert 1, even ones to expert 0
    clean = sot.sot_routed_layer(*args, 1)
    assert torch.equal(clean[2][:, 0].long().cpu(), torch.arange(T) % 2)
    args[2][1] *= 2.0 ** 66
    out = sot.sot_routed_layer(*args, 1)[0]
    assert torch.equal(out[::2], clean[0][::2]) and not torch.isfinite(out[1::2]).any()
    args[2][1, 3, 5] = float("nan")
    out = sot.sot_routed_layer(*args, 1)[0]
    assert torch.equal(out[::2], clean[0][::2]) and torch.isnan(out[1::2]).all()
