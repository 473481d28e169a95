"""Dense-stage attention (``lh_attn_forward``) against its definition in float64, at the sizes, masks and layouts where
it can go wrong."""

from __future__ import annotations

import pytest
import torch

from tests import _attn as A

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def lh(cuda_device):
    from hierarchical_sparse_attention_avg_b200 import lh as mod

    return mod


def mods(P, dev, seed=5, slopes=False, docs=None, prefix=None, kv_len=None):
    g = torch.Generator().manual_seed(seed)
    m = {}
    if slopes:
        m["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / P.Hq) for h in range(P.Hq)], device=dev)
    if P.buckets:
        m["table"] = torch.randn(P.Hq, P.buckets, generator=g).to(P.dtype).to(dev)
    if docs is not None:
        m["docs"] = torch.tensor(docs, dtype=torch.int32, device=dev)
    if prefix is not None:
        m["prefix"] = torch.tensor(prefix, dtype=torch.int32, device=dev)
    if kv_len is not None:
        m["kv_len"] = torch.tensor(kv_len, dtype=torch.int32, device=dev)
    return m


def spans(S, *lengths):
    """Ids 0, 1, ... over the given lengths, -1 up to S."""
    ids = [n for n, c in enumerate(lengths) for _ in range(c)]
    return ids + [-1] * (S - len(ids))


# (params, mods): lengths around the tiles (1, 127..129, 255..257), both dtypes and widths, every mask and bias
FORWARD = {
    "one_key": (dict(B=1, Hq=1, Hkv=1, Sq=1, Skv=1, d=64), {}),
    "one_token": (dict(B=2, Hq=4, Hkv=4, Sq=1, Skv=300, d=128), dict(kv_len=[300, 1])),
    "empty_entry": (dict(B=3, Hq=2, Hkv=1, Sq=2, Skv=130, d=64), dict(kv_len=[0, 1, 130])),
    "short": (dict(B=1, Hq=2, Hkv=2, Sq=127, Skv=127, d=64, dtype=FP), {}),
    "tile": (dict(B=1, Hq=2, Hkv=2, Sq=128, Skv=128, d=128), {}),
    "tile1": (dict(B=2, Hq=2, Hkv=1, Sq=129, Skv=129, d=128, softcap=20.0), {}),
    "pair1": (dict(B=1, Hq=3, Hkv=3, Sq=257, Skv=257, d=64), dict(slopes=True)),
    "all": (dict(B=1, Hq=2, Hkv=2, Sq=300, Skv=300, d=64, causal=False), {}),
    "all_slopes": (dict(B=1, Hq=2, Hkv=2, Sq=300, Skv=300, d=128, causal=False, dtype=FP), dict(slopes=True)),
    "cross": (dict(B=1, Hq=2, Hkv=2, Sq=40, Skv=700, d=64, causal=False, softcap=5.0), dict(slopes=True)),
    "more_rows": (dict(B=2, Hq=2, Hkv=2, Sq=300, Skv=200, d=64), dict(kv_len=[200, 90])),
    "prefix": (dict(B=3, Hq=2, Hkv=2, Sq=391, Skv=391, d=64), dict(prefix=[0, 150, 391])),
    "prefix_bias": (dict(B=2, Hq=2, Hkv=2, Sq=391, Skv=391, d=128, buckets=32, max_distance=128, bidirectional=True),
                    dict(prefix=[129, 1000])),
    "docs": (dict(B=2, Hq=2, Hkv=2, Sq=700, Skv=700, d=128),
             dict(docs=[spans(700, 1, 127, 300, 200), spans(700, 700)])),
    "docs_mixed": (dict(B=1, Hq=2, Hkv=1, Sq=600, Skv=600, d=64, causal=False, softcap=30.0),
                   dict(docs=[[(i * 7) % 5 - 1 for i in range(600)]])),
    "docs_none": (dict(B=1, Hq=2, Hkv=2, Sq=200, Skv=200, d=64), dict(docs=[[-1] * 200])),
    "docs_cache": (dict(B=1, Hq=8, Hkv=2, Sq=3, Skv=900, d=128), dict(docs=[spans(900, 400, 500)], kv_len=[880])),
    "slopes_cap": (dict(B=1, Hq=4, Hkv=2, Sq=513, Skv=513, d=128, softcap=50.0), dict(slopes=True)),
    "bias": (dict(B=1, Hq=4, Hkv=4, Sq=513, Skv=513, d=64, buckets=32, max_distance=128), {}),
    "bias_cap": (dict(B=1, Hq=2, Hkv=2, Sq=400, Skv=400, d=128, buckets=16, max_distance=100, softcap=20.0), {}),
    "bias_both": (dict(B=2, Hq=2, Hkv=2, Sq=509, Skv=509, d=64, buckets=32, max_distance=128, bidirectional=True,
                       causal=False), dict(docs=[spans(509, 509), spans(509, 300)])),
    "bias_far": (dict(B=1, Hq=7, Hkv=1, Sq=5, Skv=3000, d=64, buckets=64, max_distance=2000, dtype=FP), {}),
    "bias_two": (dict(B=1, Hq=2, Hkv=2, Sq=260, Skv=260, d=64, buckets=2, max_distance=2), {}),
    "bias_most": (dict(B=1, Hq=2, Hkv=2, Sq=300, Skv=300, d=64, buckets=128, max_distance=1000000), {}),
    "group7": (dict(B=2, Hq=14, Hkv=2, Sq=3, Skv=1000, d=128), dict(kv_len=[1000, 517])),
    "group32": (dict(B=1, Hq=32, Hkv=1, Sq=1, Skv=5000, d=64), dict(slopes=True)),
    "group17": (dict(B=1, Hq=17, Hkv=1, Sq=2, Skv=500, d=64), {}),
    "group5_chunk": (dict(B=1, Hq=10, Hkv=2, Sq=60, Skv=2000, d=128, softcap=50.0), dict(kv_len=[1999])),
    "chunk": (dict(B=2, Hq=4, Hkv=2, Sq=257, Skv=4000, d=128, softcap=50.0), dict(kv_len=[4000, 300])),
    "long_cache": (dict(B=1, Hq=4, Hkv=2, Sq=1, Skv=70001, d=128), {}),
    "bias_one": (dict(B=2, Hq=2, Hkv=1, Sq=1, Skv=1, d=64, buckets=32, max_distance=128), {}),
    "group16_full": (dict(B=1, Hq=16, Hkv=1, Sq=8, Skv=700, d=128, buckets=32, max_distance=128, dtype=FP), {}),
    "group16_two": (dict(B=1, Hq=16, Hkv=1, Sq=9, Skv=700, d=128, buckets=64, max_distance=500, softcap=20.0), {}),
    "group16_copies": (dict(B=2, Hq=16, Hkv=1, Sq=2, Skv=900, d=128, buckets=32, max_distance=128), dict(kv_len=[900, 1])),
    "group48": (dict(B=1, Hq=48, Hkv=1, Sq=1, Skv=300, d=64), dict(slopes=True)),
    "few_rows_docs": (dict(B=2, Hq=4, Hkv=2, Sq=30, Skv=260, d=64, softcap=30.0),
                      dict(docs=[spans(260, 100, 140), [3] * 60 + [1] * 200], kv_len=[250, 255])),
    "wide_grid": (dict(B=40, Hq=8, Hkv=4, Sq=1, Skv=400, d=64), dict(kv_len=[10 * i for i in range(40)])),
}


BACKWARD = {n: FORWARD[n] for n in FORWARD if n not in ("long_cache", "wide_grid")}
BACKWARD.update({
    "group8": (dict(B=1, Hq=8, Hkv=1, Sq=700, Skv=700, d=128, softcap=50.0), dict(docs=[spans(700, 300, 350)])),
    "longer": (dict(B=1, Hq=2, Hkv=2, Sq=2100, Skv=2100, d=64, dtype=FP), {}),
    "bias_longer": (dict(B=2, Hq=2, Hkv=1, Sq=1500, Skv=1500, d=128, buckets=32, max_distance=128), {}),
    "bias_wide": (dict(B=1, Hq=2, Hkv=2, Sq=1500, Skv=1500, d=64, buckets=48, max_distance=1000, bidirectional=True,
                       causal=False, dtype=FP), {}),
})


@pytest.mark.parametrize("name", FORWARD)
def test_forward(lh, cuda_device, name):
    p, m = FORWARD[name]
    P = lh.AttnParams(**p)
    q, k, v = A.make(P, 3, cuda_device)
    m = mods(P, cuda_device, **m)
    o, lse = lh.lh_attn_forward(P, q, k, v, **m)
    assert lh.lh_get_status() == lh.LH_OK
    ref = A.reference(P, q, k, v, **m)
    A.check("lse", lse, ref)
    A.check("o", o, ref)
    o2, lse2 = lh.lh_attn_forward(P, q, k, v, **m)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)  # no order left open


@pytest.mark.parametrize("exact", [False, True], ids=["o", "o_low"])
@pytest.mark.parametrize("name", BACKWARD)
def test_backward(lh, cuda_device, name, exact):
    p, m = BACKWARD[name]
    P = lh.AttnParams(**p)
    q, k, v, dout = A.make(P, 3, cuda_device, grad=True)
    m = mods(P, cuda_device, **m)
    low = torch.empty_like(q) if exact else None
    o, lse = lh.lh_attn_forward(P, q, k, v, low=low, **m)
    m["low"] = low
    grads = lh.lh_attn_backward(P, q, k, v, o, lse, dout, **m)
    assert lh.lh_get_status() == lh.LH_OK
    ref = A.reference(P, q, k, v, dout=dout, **m)
    if exact:  # low is a second rounding's remainder
        assert ((o.double() + low.double() - ref["o"]).abs() <= ref["e_o"] - A.half_step(P) * ref["o"].abs() * 0.99 + 1e-7).all()
    names = ("dq", "dk", "dv") + (("dtable",) if P.buckets else ())
    assert len(grads) == 4 and (P.buckets or grads[3] is None)
    for n, g in zip(names, grads):
        A.check(n, g, ref)
    again = lh.lh_attn_backward(P, q, k, v, o, lse, dout, **m)
    for n, g, g2 in zip(names[1:], grads[1:], again[1:]):  # (dq's fp32 sums have no fixed order)
        assert torch.equal(g, g2), n
