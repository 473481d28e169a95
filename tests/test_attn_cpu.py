"""Dense-stage attention without a GPU: what the library accepts and refuses (before any CUDA call), the buckets' borders,
and the test's own definition of the gradients against differences."""

from __future__ import annotations

import ctypes
import struct

import pytest
import torch

from hierarchical_sparse_attention_avg_b200 import lh
from tests import _attn as A

OK = dict(B=2, Hq=4, Hkv=2, Sq=16, Skv=64, d=64)


@pytest.mark.parametrize("change,code", [
    (dict(), 0), (dict(d=128, dtype=torch.float16), 0), (dict(Sq=100, Skv=3), 0), (dict(softcap=30.0), 0),
    (dict(buckets=2, max_distance=2), 0), (dict(buckets=128, max_distance=65, bidirectional=True), 0),
    (dict(B=0), 1), (dict(Hq=0), 1), (dict(Hkv=0), 1), (dict(Sq=0), 1), (dict(Skv=0), 1), (dict(d=0), 1), (dict(Sq=-1), 1),
    (dict(Hq=5), 1), (dict(scale=0.0), 1), (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1),
    (dict(scale=float("inf")), 1), (dict(softcap=-1.0), 1), (dict(softcap=float("nan")), 1), (dict(softcap=float("inf")), 1),
    (dict(buckets=1, max_distance=10), 1), (dict(buckets=130, max_distance=1000), 1), (dict(buckets=-2), 1),
    (dict(buckets=32, max_distance=16), 1), (dict(buckets=7, max_distance=100, bidirectional=True), 1),
    (dict(buckets=2, max_distance=100, bidirectional=True), 1),
    (dict(d=96), 2), (dict(d=256), 2), (dict(B=65536), 2), (dict(Skv=(1 << 20) + 1), 2), (dict(B=60000, Hq=1, Hkv=1, Sq=40000), 2),
])
def test_validation_codes(change, code):
    P = lh.AttnParams(**{**OK, **change})
    assert lh.lh_attn_validate(P) == code
    assert (lh.lh_attn_workspace_bytes(P) > 0) == (code == 0)
    if code:
        for call in (lambda: lh.new_attn_workspace(P, "cpu"), lambda: lh.lh_attn_forward(P, None, None, None)):
            with pytest.raises(lh.LighthouseError) as e:
                call()
            assert e.value.status == code


def test_other_dtypes_are_refused():
    with pytest.raises(ValueError):
        lh.AttnParams(**OK, dtype=torch.float32)


@pytest.mark.parametrize("both", [False, True])
@pytest.mark.parametrize("buckets,distance", [(32, 128), (64, 500), (16, 100), (64, 2000), (128, 10**6), (4, 3), (32, 17),
                                              (128, 2**31 - 1), (20, 160)])
def test_bucket_borders(buckets, distance, both):
    """The first distance of each bucket, against the definition in whole numbers on both of its sides."""
    P = lh.AttnParams(**OK, buckets=buckets, max_distance=distance, bidirectional=both)
    if lh.lh_attn_validate(P):
        pytest.skip("not a valid table")
    n = buckets // 2 if both else buckets
    e = n // 2
    starts = lh.lh_attn_bucket_starts(P)
    assert len(starts) == n and starts[:e] == list(range(e))
    for b in range(e, n):
        reaches = lambda x: x ** (n - e) * e ** (b - e) >= distance ** (b - e) * e ** (n - e)  # noqa: E731
        assert reaches(starts[b]) and not reaches(starts[b] - 1), b
    far = torch.arange(-300, 301)
    idx = A.bucket_index(far, buckets, distance, both)
    size = far.abs() if both else far.clamp(min=0)
    want = sum((size >= s).long() for s in starts) - 1 + (n * (far < 0) if both else 0)
    assert torch.equal(idx, want)


def test_no_table_has_no_starts():
    with pytest.raises(lh.LighthouseError):
        lh.lh_attn_bucket_starts(lh.AttnParams(**OK))


def _c_args(P, **change):
    """Arguments of the C entry points with plausible device addresses that nothing dereferences."""
    row = lambda S, H: struct.pack("4q", 4096, S * H * P.d, S * P.d, P.d)  # noqa: E731
    a = dict(q=row(P.Sq, P.Hq), k=row(P.Skv, P.Hkv), v=row(P.Skv, P.Hkv), o=row(P.Sq, P.Hq), low=None, lse=4096,
             dout=row(P.Sq, P.Hq), dq=row(P.Sq, P.Hq), dk=row(P.Skv, P.Hkv), dv=row(P.Skv, P.Hkv), dtable=0, mods=bytes(40),
             ws=4096, ws_bytes=1 << 40)
    a.update(change)
    return a


def _calls(P, a):
    lib = lh.library()
    f = lib.lh_attn_forward(P._ref, a["mods"], a["q"], a["k"], a["v"], a["o"], a["low"], a["lse"], a["ws"], a["ws_bytes"], None)
    b = lib.lh_attn_backward(P._ref, a["mods"], a["q"], a["k"], a["v"], a["o"], a["low"], a["lse"], a["dout"], a["dq"], a["dk"],
                             a["dv"], a["dtable"], a["ws"], a["ws_bytes"], None)
    return f, b


def _row(P, ptr=4096, sb=None, sh=None, ss=None):
    S, H = P.Sq, P.Hq
    return struct.pack("4q", ptr, S * H * P.d if sb is None else sb, S * P.d if sh is None else sh, P.d if ss is None else ss)


def _mods(slopes=0, table=0, docs=0, prefix=0, kv_len=0):
    return struct.pack("5Q", slopes, table, docs, prefix, kv_len)


def test_c_entries_refuse_before_any_cuda_call():
    P = lh.AttnParams(**OK)
    T = lh.AttnParams(**OK, buckets=32, max_distance=128)
    N = lh.AttnParams(**OK, causal=False)
    bad = lh.LH_ERR_INVALID_ARG
    both = [
        (P, dict(q=None)), (P, dict(q=_row(P, ptr=0))), (P, dict(q=_row(P, ptr=4104))), (P, dict(o=_row(P, ptr=4098))),
        (P, dict(q=_row(P, sh=0))), (P, dict(q=_row(P, ss=-64))), (P, dict(q=_row(P, sb=1001))), (P, dict(o=_row(P, ss=60))),
        (P, dict(low=_row(P, ptr=4100))), (P, dict(k=None)), (P, dict(v=None)), (P, dict(o=None)), (P, dict(lse=0)),
        (P, dict(lse=4098)), (P, dict(q=_row(P, sb=1 << 50))),
        (P, dict(mods=_mods(table=4096))), (T, dict(mods=_mods())), (T, dict(mods=_mods(table=4096, slopes=4096))),
        (T, dict(mods=_mods(table=4097))), (N, dict(mods=_mods(prefix=4096))), (P, dict(mods=_mods(docs=4098))),
        (P, dict(mods=_mods(kv_len=4097))), (P, dict(ws=0)), (P, dict(ws=4097)),
    ]
    for params, change in both:
        f, b = _calls(params, _c_args(params, **change))
        want = lh.LH_ERR_WORKSPACE if change.get("ws") else bad
        assert (f, b) == (want, want), change
    only_backward = [(P, dict(dout=None)), (P, dict(dq=None)), (P, dict(dk=_row(P, ptr=1))), (P, dict(dv=None)),
                     (T, dict(mods=_mods(table=4096)))]
    for params, change in only_backward:
        assert _calls(params, _c_args(params, **change))[1] == bad, change
    need = lh.lh_attn_workspace_bytes(P, True)
    assert _calls(P, _c_args(P, ws_bytes=need - 1))[1] == lh.LH_ERR_WORKSPACE
    assert lh.library().lh_attn_validate(None) == bad
    assert lh.library().lh_attn_forward(None, None, None, None, None, None, None, None, None, 0, None) == bad


def test_dimensions_of_one_may_have_any_stride():
    P = lh.AttnParams(1, 1, 1, 1, 64, 64)
    a = _c_args(P, q=struct.pack("4q", 4096, 0, 3, -1), ws_bytes=0)
    assert _calls(P, a)[0] == lh.LH_ERR_WORKSPACE  # past the tensors' checks


def test_python_refusals():
    P = lh.AttnParams(**OK)
    t = lambda S, H: torch.zeros(P.B, H, S, P.d, dtype=torch.bfloat16)  # noqa: E731
    with pytest.raises(ValueError):  # host tensors
        lh.lh_attn_forward(P, t(P.Sq, P.Hq), t(P.Skv, P.Hkv), t(P.Skv, P.Hkv))
    dev = torch.device("cpu")
    good = t(P.Sq, P.Hq)
    ok = lambda x: lh._rows(x, P._qs, P.dtype, dev, "q")  # noqa: E731
    assert len(ok(good)) == 32 and ok(torch.zeros(P.B, P.Sq, P.Hq, P.d, dtype=P.dtype).transpose(1, 2))
    for x in (good.float(), good[:1], good.transpose(2, 3).contiguous().transpose(2, 3), good[:, :1].expand(P._qs),
              torch.zeros(P.B, P.Hq, P.Sq, P.d + 4, dtype=P.dtype)[..., :P.d]):
        with pytest.raises(ValueError):
            ok(x)
    with pytest.raises(ValueError):
        lh._vec(torch.zeros(P.B, dtype=torch.int64), (P.B,), torch.int32, dev, "kv_len")
    with pytest.raises(ValueError):
        lh._vec(torch.zeros(2 * P.B, dtype=torch.int32)[::2], (P.B,), torch.int32, dev, "kv_len")


@pytest.mark.parametrize("kind", ["cap_slopes", "table", "table_both"])
def test_reference_gradients_against_differences(kind):
    """The formulas that the GPU tests hold the kernels to, against central differences in float64."""
    torch.manual_seed(1)
    p = dict(B=1, Hq=2, Hkv=1, Sq=9, Skv=9, d=8, dtype=torch.bfloat16)
    m = dict(docs=torch.tensor([[0] * 5 + [1] * 3 + [-1]], dtype=torch.int32))
    if kind == "cap_slopes":
        p["softcap"], m["slopes"] = 2.0, torch.tensor([0.5, 0.25])
    else:
        p.update(buckets=8, max_distance=6, bidirectional=kind == "table_both", causal=kind == "table")
    P = lh.AttnParams(**p)
    x = [torch.randn(1, h, 9, 8, dtype=torch.float64) for h in (2, 1, 1)]
    table = torch.randn(2, 8, dtype=torch.float64) if P.buckets else None
    dout = torch.randn(1, 2, 9, 8, dtype=torch.float64)

    def loss(q, k, v, t):
        return (A.reference(P, q, k, v, table=t, **m)["o"] * dout).sum()

    g = A.reference(P, *x, table=table, dout=dout, **m)
    leaves = dict(dq=0, dk=1, dv=2)
    for name, i in list(leaves.items()) + ([("dtable", 3)] if P.buckets else []):
        args = x + [table]
        for at in torch.randperm(args[i].numel())[:12]:
            hi, lo = [a.clone() if a is not None else None for a in args], [a.clone() if a is not None else None for a in args]
            hi[i].view(-1)[at] += 1e-5
            lo[i].view(-1)[at] -= 1e-5
            slope = (loss(*hi) - loss(*lo)) / 2e-5
            assert abs(slope - g[name].reshape(-1)[at]) <= 1e-6 * (1 + abs(slope)), (name, int(at))
