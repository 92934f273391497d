"""The language-model losses at their edges: values that are not finite, calls from several host threads, in captured
graphs, in place and under other default types.  Tolerances are those of test_gpu_lm_losses.py unless a test derives
its own; values that are not finite have to be the same ones."""
import threading

import numpy as np
import pytest

import lm_ref as R
from test_gpu_lm_losses import (ATOL, GTOL, RTOL, SIZES, TYPES, close_grad, host, policy_inputs, rows, sot,  # noqa: F401
                                targets)

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

INF, NAN = float("inf"), float("nan")


def f32(v):
    return torch.from_numpy(np.asarray(v, np.float32)).cuda()


def alike(got, ref, bound):
    """Within `bound` where the reference is finite, the same infinity or NaN where it is not."""
    got, ref = host(got), np.asarray(ref, np.float64)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), (got, ref)
    ends = np.isinf(got) | np.isinf(ref)
    assert np.array_equal(got[ends], ref[ends]), (got, ref)
    ok = np.isfinite(ref)
    over = np.abs(got[ok] - ref[ok]) - np.broadcast_to(bound, ref.shape)[ok]
    assert over.size == 0 or over.max() <= 0, over.max()


@pytest.mark.parametrize("default", [torch.bfloat16, torch.float16, torch.float64])
def test_outputs_are_float32_under_any_default_type(sot, default):
    """torch's default type says nothing about the outputs: they are float32, and the same bits."""
    T, V = 700, 50
    x, tg, old, adv, ref, w = policy_inputs(T, V, "bf16", 0, 1.0, 3)
    ids = torch.arange(5, dtype=torch.int32).expand(T, 5).contiguous().cuda()
    z = torch.randn(T, 5, generator=torch.Generator().manual_seed(1)).cuda()
    off = torch.arange(0, T + 1, 2).cuda()
    off = off[:off.numel() // 2 * 2 - 1].contiguous()
    pts, eps = torch.rand(1, 40, 3, generator=torch.Generator().manual_seed(2)).cuda(), 0.1

    def calls():
        out = list(sot.sot_token_logprob(x, tg))
        out.append(sot.sot_token_logprob_grad(x, tg, out[1], adv))
        out += sot.sot_distill_topk(x, ids, z, weight=w)
        out += sot.sot_policy_loss(x, tg, old, adv, ref, w, kl_coef=0.1)
        out += sot.sot_preference_loss(out[0], off)
        out += sot.sot_balance_loss(x, ids, z_coef=0.1)
        f, g = sot.sot_potentials(pts, pts, eps=eps, iters=10)
        got = sot.sot_plan_coo_operands(pts, pts, None, None, f, g, eps)
        return out + [got[k] for k in ("xc", "lwx", "yc", "lwy", "Mr", "Mc")]
    want = calls()
    before = torch.get_default_dtype()
    torch.set_default_dtype(default)
    try:
        got = calls()
    finally:
        torch.set_default_dtype(before)
    for a, b in zip(got, want):
        assert a.dtype == b.dtype and torch.equal(a, b)
