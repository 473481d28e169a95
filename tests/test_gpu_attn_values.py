"""Dense-stage attention over the whole range of caps and score sizes, and at values that are not finite.

Bounds beside those of ``tests._attn``, u = finfo(dtype).eps / 2: where one key (or n of the same score) takes a row whole,
every other score being lower by more than 200, o is the mean of those keys' values, off by the rounding of the
probabilities and of the result, (2 u + 2^-14) times the mean of their magnitudes."""

from __future__ import annotations

import math

import pytest
import torch

from tests import _attn as A
from tests.test_gpu_attn import mods, spans

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def lh(cuda_device):
    from hierarchical_sparse_attention_avg_b200 import lh as mod

    return mod


def _all(lh, P, q, k, v, dout, m, **kw):
    o, lse = lh.lh_attn_forward(P, q, k, v, **m, **kw)
    g = lh.lh_attn_backward(P, q, k, v, o, lse, dout, **m)
    return dict(o=o, lse=lse, dq=g[0], dk=g[1], dv=g[2], **({"dtable": g[3]} if P.buckets else {}))


@pytest.mark.parametrize("cap", [1e3, 1e4, 1e5, 1e6, 1e7, 1e12])
@pytest.mark.parametrize("Sq,Skv,d,dtype,more", [
    (1, 500, 64, BF, {}), (1, 3000, 128, FP, {}), (7, 500, 128, BF, dict(slopes=True)), (30, 300, 64, FP, {}),
    (60, 400, 64, BF, {}), (200, 200, 128, BF, {}), (200, 200, 64, FP, dict(slopes=True)),
])
def test_large_caps_leave_the_scores(lh, cuda_device, cap, Sq, Skv, d, dtype, more):
    """A cap far above the scores: their error does not grow with it, in any form of the kernels."""
    P = lh.AttnParams(1, 4, 2, Sq, Skv, d, dtype=dtype, softcap=cap)
    x = A.make(P, 13, cuda_device, grad=True)
    m = mods(P, cuda_device, **more)
    ref = A.reference(P, *x[:3], dout=x[3], **m)
    for n, g in _all(lh, P, *x, m).items():
        A.check(n, g, ref)


@pytest.mark.parametrize("cap", [20.0, 1e3, 1e5, 1e7])
@pytest.mark.parametrize("Sq,d,dtype", [(1, 64, BF), (5, 128, BF), (200, 64, BF), (200, 128, BF), (7, 128, FP), (150, 64, FP)])
def test_small_scores_beside_some_beyond_the_cap(lh, cuda_device, cap, Sq, d, dtype):
    """Rows with scores beyond the cap between rows with scores of a few units, in the same tiles."""
    P = lh.AttnParams(1, 4, 1, Sq, 300, d, dtype=dtype, softcap=cap)
    q, k, v, dout = A.make(P, 14, cuda_device, grad=True)
    f = math.sqrt(cap / 2)
    beyond = (torch.arange(4)[:, None] + torch.arange(Sq)[None] + 1).to(cuda_device) % 4 == 2
    q, k = torch.where(beyond[None, :, :, None], q * f, q / f), k * f
    ref = A.reference(P, q, k, v, dout=dout)
    raw = (q.double() @ k.double().transpose(2, 3)).abs() * d ** -0.5
    assert raw[:, beyond].max() > cap and raw[:, ~beyond].max() < 100
    for n, g in _all(lh, P, q, k, v, dout, {}).items():
        A.check(n, g, ref)


@pytest.mark.parametrize("cap", [1e-42, 1.2e-38, 1e-30, 1e24, 1e30, 2e38, 3.4e38])
@pytest.mark.parametrize("Sq", [1, 130])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_caps_at_the_ends_of_the_type(lh, cuda_device, cap, Sq, dtype):
    P = lh.AttnParams(1, 4, 2, Sq, 300, 64, dtype=dtype, softcap=cap)
    x = A.make(P, 15, cuda_device, grad=True)
    x[0][:, 0] = 0.0  # scores of nothing too
    ref = A.reference(P, *x[:3], dout=x[3])
    for n, g in _all(lh, P, *x, {}).items():
        A.check(n, g, ref)
