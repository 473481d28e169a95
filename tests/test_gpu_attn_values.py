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


def _peaks(P, dev, size, tie):
    """Rows whose scores are whole multiples of `size` (exact in fp32), one key (or `tie` of them) the largest."""
    g = torch.Generator().manual_seed(16)
    q, k, v, dout = A.make(P, 16, dev, grad=True)
    q.zero_(), k.zero_()
    q[..., 0] = 2.0 ** math.ceil(math.log2(size) / 2)
    step = size / float(q.flatten()[0])
    order = torch.stack([torch.randperm(P.Skv, generator=g) for _ in range(P.B * P.Hkv)]).view(P.B, P.Hkv, P.Skv)
    level = torch.where(order < tie, torch.full_like(order, 3), order % 3).to(dev)  # 3 for the winners, 0 .. 2 elsewhere
    k[..., 0] = (step * level).to(P.dtype)
    win = (level == 3)[:, :, None, :].repeat_interleave(P.Hq // P.Hkv, 1).double()  # [B, Hq, 1, Skv]
    return q, k, v, dout, win / win.sum(3, keepdim=True), 3.0 * size


# (a bias parts equal scores: ties without one only)
PEAKS = [(Sq, Skv, d, "", tie) for Sq, Skv, d in ((1, 500, 64), (1, 9000, 128), (9, 500, 128), (60, 700, 64), (300, 700, 64),
                                                  (520, 520, 128)) for tie in (1, 2)]
PEAKS += [(300, 300, 64, "slopes", 1), (300, 300, 128, "table", 1), (1, 500, 128, "table", 1)]


@pytest.mark.parametrize("dtype,size", [(BF, 2.0 ** e) for e in (10, 20, 24, 27, 30, 36, 60)] +
                         [(FP, 2.0 ** e) for e in (10, 20, 24, 26, 27)])
@pytest.mark.parametrize("Sq,Skv,d,bias,tie", PEAKS)
def test_large_scores_are_a_choice_of_keys(lh, cuda_device, size, dtype, Sq, Skv, d, bias, tie):
    """Finite scores of any size: nothing overflows, and the softmax is the choice of the largest key (or of two)."""
    f = dict(buckets=32, max_distance=128) if bias == "table" else {}
    P = lh.AttnParams(1, 4, 2, Sq, Skv, d, dtype=dtype, causal=False, scale=1.0, **f)
    q, k, v, dout, p, top = _peaks(P, cuda_device, size, tie)
    m = mods(P, cuda_device, slopes=bias == "slopes")  # (biases of at most 75: far below the steps)
    o, lse = lh.lh_attn_forward(P, q, k, v, **m)
    V, u = v.double().repeat_interleave(2, 1), A.half_step(P)
    want, mean = ((p @ x).expand(1, 4, Sq, d) for x in (V, V.abs()))
    assert torch.isfinite(o).all() and ((o.double() - want).abs() <= (2 * u + 2.0 ** -14) * mean + 1e-7).all()
    # lse: four roundings of numbers up to log2(e) times the top score, the bias or the logarithm of the tie
    assert ((lse.double() - top).abs() <= 8 * 2.0 ** -24 * top + (75.0 if bias else math.log(tie) + 1e-3)).all()


@pytest.mark.parametrize("dtype,size", [(BF, 2.0 ** e) for e in (10, 20, 24, 27, 30, 36, 60)] +
                         [(FP, 2.0 ** e) for e in (10, 20, 24, 26, 27)])
@pytest.mark.parametrize("Sq,Skv,d,bias,tie", PEAKS)
def test_gradients_of_large_scores(lh, cuda_device, size, dtype, Sq, Skv, d, bias, tie):
    """The same scores: finite gradients, of probabilities that are at most 1."""
    f = dict(buckets=32, max_distance=128) if bias == "table" else {}
    P = lh.AttnParams(1, 4, 2, Sq, Skv, d, dtype=dtype, causal=False, scale=1.0, **f)
    q, k, v, dout, p, top = _peaks(P, cuda_device, size, tie)
    m, u = mods(P, cuda_device, slopes=bias == "slopes"), A.half_step(P)
    o, lse = lh.lh_attn_forward(P, q, k, v, **m)
    grads = lh.lh_attn_backward(P, q, k, v, o, lse, dout, **m)
    # what P <= 1 allows: |dZ| = |dP - D| at the keys chosen, with D of a rounded o; beyond the type's largest number
    # a gradient is infinite, and nowhere is it NaN
    heads = lambda a: a.view(1, 2, 2, Skv, d).sum(2)  # noqa: E731
    V, W, win = v.double().repeat_interleave(2, 1), dout.double(), (p > 0).expand(1, 4, Sq, Skv)
    dP = W @ V.transpose(2, 3)
    Z = ((dP - (dP * p).sum(3, keepdim=True)).abs() + 4 * u * (W.abs() @ V.abs().transpose(2, 3))) * win
    most = (Z @ k.double().abs().repeat_interleave(2, 1), heads(Z.transpose(2, 3) @ q.double().abs()),
            heads(win.double().transpose(2, 3) @ W.abs()), torch.zeros(()))
    for g, b in zip(grads, most):
        if g is not None:
            assert not torch.isnan(g).any() and (torch.isfinite(g) | (b > 0.9 * torch.finfo(dtype).max).to(g.device)).all()
    if not bias:
        # P = exp(z - lse) is a factor exp(error of lse) off, of at most 1: dv by as much of its own sum
        mass = lambda a: (p.expand(1, 4, Sq, Skv).transpose(2, 3) @ a).view(1, 2, 2, Skv, d).sum(2)  # noqa: E731
        off = math.expm1(min(12 * 2.0 ** -24 * top, 0.5)) if size < 2.0 ** 19 else 1.0
        got, W = grads[2].double(), mass(dout.double())
        assert ((got - W).abs() <= (off + 2 * u + 2.0 ** -14) * mass(dout.double().abs()) + 1e-6).all()


@pytest.mark.parametrize("junk", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("d,dtype", [(64, BF), (128, FP)])
def test_values_that_are_not_finite_under_vanished_probabilities(lh, cuda_device, junk, d, dtype):
    """A key so low that every row's probability of it is nothing, its value not finite: the rows of both query tiles of a
    block that share it come out one way, call after call."""
    P = lh.AttnParams(1, 8, 4, 512, 512, d, dtype=dtype)
    q, k, v = A.make(P, 17, cuda_device)
    q[..., 0], k[..., 0] = 64.0, 0.0
    at = [10, 70, 127, 300]
    k[:, :, at, 0] = -64.0  # scores lower by 360 and more
    v[:, :, at, 5] = junk
    first = lh.lh_attn_forward(P, q, k, v)
    for i in range(60):
        o, lse = lh.lh_attn_forward(P, q, k, v)
        assert torch.equal(lse, first[1])
        assert torch.equal(o.view(torch.int16), first[0].view(torch.int16)), i
    sees = torch.arange(512, device=cuda_device) >= 10
    assert not torch.isfinite(o[:, :, sees, 5]).any() and torch.isfinite(o[:, :, ~sees]).all()
    keep = torch.arange(d, device=cuda_device) != 5
    ref = A.reference(P, q, k, v.nan_to_num(0.0, 0.0, 0.0))
    A.check("o", o[..., keep], {n: ref[n][..., keep] for n in ("o", "e_o")})


@pytest.mark.parametrize("junk", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("d,dtype", [(64, BF), (64, FP), (128, BF), (128, FP)])
def test_both_query_tiles_take_a_value_that_is_not_finite_the_same_way(lh, cuda_device, junk, d, dtype):
    """The first query tile sees a key tile whole, the second one part of it (documents): a value that is not finite, under
    a probability of nothing, is what comes out of either."""
    P = lh.AttnParams(1, 2, 2, 256, 256, d, dtype=dtype, causal=False)
    q, k, v = A.make(P, 18, cuda_device)
    m = mods(P, cuda_device, docs=[spans(256, 192, 64)])
    q[..., 0], k[..., 0] = 64.0, 0.0
    k[:, :, 20, 0] = -64.0
    v[:, :, 20, d - 1] = junk
    for _ in range(20):
        o, _ = lh.lh_attn_forward(P, q, k, v, **m)
        hit = o[:, :, :192, d - 1].float()
        assert (torch.isnan(hit) if junk != junk else hit == junk).all()
        assert torch.isfinite(o[:, :, 192:]).all() and torch.isfinite(o[..., :d - 1]).all()
