"""Dense-stage attention as programs use it: masked places holding anything, strided and preallocated tensors, streams,
graphs, shared workspaces, a training step followed by decoding from its cache, and the wait limit."""

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


@pytest.mark.parametrize("name,p,m", [
    ("pad", dict(B=2, Hq=4, Hkv=2, Sq=333, Skv=333, d=128, softcap=30.0), dict(docs=[spans(333, 200, 50), spans(333, 1)])),
    ("pad_all", dict(B=2, Hq=2, Hkv=2, Sq=200, Skv=200, d=64, causal=False, dtype=FP, buckets=32, max_distance=128,
                     bidirectional=True), dict(docs=[spans(200, 150), [-1, -1] + [0] * 198])),
    ("lengths", dict(B=3, Hq=4, Hkv=1, Sq=150, Skv=400, d=64), dict(kv_len=[400, 131, 20], slopes=True)),
    ("token", dict(B=3, Hq=8, Hkv=2, Sq=1, Skv=400, d=128), dict(kv_len=[400, 131, 0])),
    ("short", dict(B=2, Hq=8, Hkv=2, Sq=20, Skv=300, d=64), dict(kv_len=[290, 5])),
])
@pytest.mark.parametrize("junk", [math.nan, math.inf])
def test_dead_positions_hold_anything(lh, cuda_device, name, p, m, junk):
    P = lh.AttnParams(**p)
    q, k, v, dout = A.make(P, 7, cuda_device, grad=True)
    m = mods(P, cuda_device, **m)
    ref = A.reference(P, q, k, v, dout=dout, **m)
    x, seen = A.visible(P.B, P.Sq, P.Skv, P.causal, **{n: m.get(n) for n in ("docs", "prefix", "kv_len")})
    dead_q, dead_k = ~seen.any(2).to(cuda_device), ~seen.any(1).to(cuda_device)
    assert dead_q.any() or dead_k.any()
    for t, dead in ((q, dead_q), (dout, dead_q), (k, dead_k), (v, dead_k)):
        t.masked_fill_(dead[:, None, :, None], junk)
    got = _all(lh, P, q, k, v, dout, m)
    for n, g in got.items():
        A.check(n, g, ref)
    assert lh.lh_get_status() == lh.LH_OK


@pytest.mark.parametrize("ban", [-math.inf, torch.finfo(BF).min])
@pytest.mark.parametrize("name,p,m,which", [
    ("self", dict(B=2, Hq=4, Hkv=2, Sq=300, Skv=300, d=64), dict(docs=[spans(300, 100, 7, 193), spans(300, 300)]), [0]),
    ("far", dict(B=1, Hq=2, Hkv=1, Sq=700, Skv=700, d=128, softcap=20.0), {}, [31, 20]),
    ("all", dict(B=1, Hq=2, Hkv=2, Sq=150, Skv=150, d=64), {}, list(range(32))),
    ("both", dict(B=2, Hq=4, Hkv=4, Sq=200, Skv=200, d=64, causal=False, bidirectional=True),
     dict(docs=[spans(200, 150), spans(200, 200)]), [0, 15, 20]),
    ("token", dict(B=3, Hq=8, Hkv=2, Sq=1, Skv=900, d=128), dict(kv_len=[900, 131, 1]), [31, 0]),
    ("split", dict(B=1, Hq=4, Hkv=2, Sq=5, Skv=6000, d=64), {}, [31]),
])
def test_table_entries_that_mask_their_bucket(lh, cuda_device, name, p, m, which, ban):
    P = lh.AttnParams(**p, buckets=32, max_distance=128)
    q, k, v, dout = A.make(P, 3, cuda_device, grad=True)
    m = mods(P, cuda_device, **m)
    m["table"][:, which] = ban
    ref = A.reference(P, q, k, v, dout=dout, **m)
    for n, g in _all(lh, P, q, k, v, dout, m).items():
        A.check(n, g, ref)


@pytest.mark.parametrize("junk", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("p", [dict(d=128), dict(d=64, softcap=20.0), dict(d=64, dtype=FP, buckets=32, max_distance=128)])
def test_masked_values_reach_no_row(lh, cuda_device, p, junk):
    """A key or value that is not finite reaches the rows that see it, and no other (causal and documents)."""
    P = lh.AttnParams(B=1, Hq=2, Hkv=1, Sq=500, Skv=500, **p)
    q, k, v = A.make(P, 8, cuda_device)
    m = mods(P, cuda_device, docs=[spans(500, 140, 360)])
    ref = A.reference(P, q, k, v, **m)
    _, seen = A.visible(1, 500, 500, True, docs=m["docs"])
    for bad in ([100], [139, 141, 300]):
        for which in ("k", "v"):
            kk, vv = k.clone(), v.clone()
            (kk if which == "k" else vv)[:, :, bad, 3] = junk
            o, lse = lh.lh_attn_forward(P, q, kk, vv, **m)
            touched = seen[0][:, bad].any(1).to(cuda_device)
            clean = {n: r[:, :, ~touched] for n, r in ref.items() if n != "p"}
            A.check("o", o[:, :, ~touched], clean)
            A.check("lse", lse[:, :, ~touched], clean)
            if which == "v":
                hit = o[:, :, touched, 3].float()
                assert not torch.isfinite(hit).any() and (torch.isnan(hit) if junk != junk else hit == junk).all()
                other = torch.arange(P.d, device=cuda_device) != 3  # the other features as if nothing was there
                A.check("o", o[:, :, touched][..., other], {n: ref[n][:, :, touched][..., other] for n in ("o", "e_o")})


def test_strided_inputs_and_outputs_inside_larger_buffers(lh, cuda_device):
    B, S, H, d = 2, 300, 4, 64
    P = lh.AttnParams(B, H, H, S, S, d, softcap=30.0)
    g = torch.Generator().manual_seed(2)
    qkv = torch.randn(B, S, 3, H, d, generator=g).to(BF).to(cuda_device)
    q, k, v = (qkv[:, :, i].transpose(1, 2) for i in range(3))
    dout = torch.randn(B, S, H, d, generator=g).to(BF).to(cuda_device).transpose(1, 2)
    big = torch.full((5, B, S + 3, H + 1, d + 8), 7.0, dtype=BF, device=cuda_device)
    o, low, dq, dk, dv = (b[:, 1:S + 1, :H, 8:].transpose(1, 2) for b in big)
    lse = torch.empty(B, H, S, device=cuda_device)
    lh.lh_attn_forward(P, q, k, v, o=o, low=low, lse=lse)
    lh.lh_attn_backward(P, q, k, v, o, lse, dout, low=low, dq=dq, dk=dk, dv=dv)
    ref = A.reference(P, q, k, v, dout=dout, low=low)
    for n, t in (("o", o), ("lse", lse), ("dq", dq), ("dk", dk), ("dv", dv)):
        A.check(n, t, ref)
    rest = torch.ones_like(big, dtype=torch.bool)
    rest[:, :, 1:S + 1, :H, 8:] = False
    assert (big[rest] == 7.0).all()  # nothing beside the tensors was written


def test_default_outputs_follow_their_inputs(lh, cuda_device):
    P = lh.AttnParams(2, 4, 2, 30, 50, 64)
    q, k, v, dout = A.make(P, 3, cuda_device, grad=True, head_rows=False)
    o, lse = lh.lh_attn_forward(P, q, k, v)
    dq, dk, dv, none = lh.lh_attn_backward(P, q, k, v, o, lse, dout)
    assert o.shape == q.shape == dq.shape and dk.shape == k.shape and none is None
    ref = A.reference(P, q, k, v, dout=dout)
    for n, t in (("o", o), ("dq", dq), ("dk", dk), ("dv", dv)):
        A.check(n, t, ref)


@pytest.mark.parametrize("Sq", [1, 200])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_many_small_probabilities_beside_a_large_one(lh, cuda_device, dtype, Sq):
    """One key 18 (natural) above 20,000 others: what they have in common must not round away."""
    S = 20200
    P = lh.AttnParams(1, 2, 1, Sq, S, 64, dtype=dtype, causal=False, scale=1.0)
    q, k, v = (torch.zeros(1, h, n, 64, dtype=dtype, device=cuda_device) for h, n in ((2, Sq), (1, S), (1, S)))
    q[..., 0], k[:, :, 7, 0] = 1.0, 18.0
    v[:] = 1.0
    v[:, :, 7] = 0.0
    ref = A.reference(P, q, k, v)
    o, lse = lh.lh_attn_forward(P, q, k, v)
    A.check("o", o, ref, tiny=0.0)  # 3e-4 everywhere
    A.check("lse", lse, ref)


def test_many_documents_beyond_the_own_ranges(lh, cuda_device):
    S = 4500  # more key tiles than a block classes by itself
    P = lh.AttnParams(1, 2, 1, S, S, 64, softcap=50.0)
    q, k, v, dout = A.make(P, 4, cuda_device, grad=True)
    m = mods(P, cuda_device, docs=[spans(S, 1, 700, 128, 1500, 77, 2000)])
    ref = A.reference(P, q, k, v, dout=dout, **m)
    for n, t in _all(lh, P, q, k, v, dout, m).items():
        A.check(n, t, ref)


def test_extreme_ids_lengths_and_prefixes(lh, cuda_device):
    """Ids at both ends of the type, lengths outside [0, Skv], prefixes below 0 and beyond the length."""
    lo, hi = -2 ** 31, 2 ** 31 - 1
    P = lh.AttnParams(4, 4, 2, 300, 300, 64)
    ids = [[hi] * 100 + [0] * 80 + [lo] * 20 + [hi - 1] * 100, [lo] * 300, [hi] * 300, [0, hi] * 150]
    m = mods(P, cuda_device, docs=ids, kv_len=[hi, 250, lo, 299], prefix=[lo, 10, hi, hi])
    q, k, v, dout = A.make(P, 8, cuda_device, grad=True)
    ref = A.reference(P, q, k, v, dout=dout, **m)
    for n, g in _all(lh, P, q, k, v, dout, m).items():
        A.check(n, g, ref)


def test_largest_batch(lh, cuda_device):
    P = lh.AttnParams(4095, 16, 16, 1, 5, 64)  # B Hq = 65,520
    q, k, v, dout = A.make(P, 6, cuda_device, grad=True)
    ref = A.reference(P, q, k, v, dout=dout)
    for n, t in _all(lh, P, q, k, v, dout, {}).items():
        A.check(n, t, ref)


@pytest.mark.parametrize("slopes", [False, True])
def test_more_query_tiles_than_the_heads_first_grid_takes(lh, cuda_device, slopes):
    """131,328 rows in documents of 128: the same as so many entries of 128 rows."""
    n, w, d = 1026, 128, 64
    P, E = lh.AttnParams(1, 1, 1, n * w, n * w, d), lh.AttnParams(n, 1, 1, w, w, d)
    x = A.make(P, 9, cuda_device, grad=True)
    m = mods(P, cuda_device, slopes=slopes)
    docs = (torch.arange(n * w, device=cuda_device) // w).to(torch.int32)[None]
    got = _all(lh, P, *x, dict(m, docs=docs))
    short = [t.view(1, n, w, d).transpose(0, 1) for t in x]
    ref = A.reference(E, *short[:3], dout=short[3], **m)
    for name, t in got.items():
        A.check(name, t.view(1, n, w, *t.shape[3:]).transpose(0, 1), ref)


def test_offsets_beyond_32_bits(lh, cuda_device):
    """A cache of 18 heads of 2^20 keys: 2.4e9 elements each of keys and values."""
    H, S, d = 18, 1 << 20, 128
    P = lh.AttnParams(1, H, H, 1, S, d)
    g = torch.Generator(cuda_device).manual_seed(1)
    k, v = (torch.randn(1, H, S, d, generator=g, device=cuda_device, dtype=BF) for _ in range(2))
    q = torch.randn(1, H, 1, d, generator=g, device=cuda_device, dtype=BF)
    kv_len = torch.tensor([S - 3], dtype=torch.int32, device=cuda_device)
    k[:, :, S - 3:], v[:, :, S - 3:] = math.nan, math.nan
    o, lse = lh.lh_attn_forward(P, q, k, v, kv_len=kv_len)
    one = lh.AttnParams(1, 1, 1, 1, S, d)
    for h in (0, H - 1):
        ref = A.reference(one, q[:, h:h + 1], k[:, h:h + 1], v[:, h:h + 1], kv_len=kv_len)
        A.check("o", o[:, h:h + 1], ref)
        A.check("lse", lse[:, h:h + 1], ref)


def test_workspaces(lh, cuda_device):
    P = lh.AttnParams(1, 4, 2, 1, 3000, 128)
    q, k, v = A.make(P, 5, cuda_device)
    with pytest.raises(lh.LighthouseError) as e:
        lh.lh_attn_forward(P, q, k, v, ws=torch.empty(16, dtype=torch.uint8, device=cuda_device))
    assert e.value.status == lh.LH_ERR_WORKSPACE
    with pytest.raises(ValueError):
        lh.lh_attn_forward(P, q, k, v, ws=torch.empty(1 << 20, device=cuda_device))
    # leftovers of another call in it change nothing
    want = lh.lh_attn_forward(P, q, k, v)
    ws = torch.full((lh.lh_attn_workspace_bytes(P, True),), 0xFF, dtype=torch.uint8, device=cuda_device)
    for _ in range(2):
        got = lh.lh_attn_forward(P, q, k, v, ws=ws)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    dout = torch.randn_like(q)
    first = lh.lh_attn_backward(P, q, k, v, *want, dout, ws=ws)
    ws.fill_(0xFF)
    again = lh.lh_attn_backward(P, q, k, v, *want, dout, ws=ws)
    assert torch.equal(first[1], again[1]) and torch.equal(first[2], again[2])


def test_two_streams_at_once(lh, cuda_device):
    P = lh.AttnParams(1, 8, 8, 700, 700, 64, buckets=32, max_distance=128)
    sets = [A.make(P, 10 + i, cuda_device, grad=True) for i in range(2)]
    m = mods(P, cuda_device)
    want = [_all(lh, P, *s, m) for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = _all(lh, P, *sets[i], m)
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        for n in w:
            if n != "dq":
                assert torch.equal(w[n], g[n]), n


@pytest.mark.parametrize("dtype", [BF, FP])
def test_captured_step_replays_on_new_contents(lh, cuda_device, dtype):
    P = lh.AttnParams(2, 4, 2, 200, 500, 64, dtype=dtype, buckets=16, max_distance=100)
    q, k, v, dout = A.make(P, 20, cuda_device, grad=True)
    m = mods(P, cuda_device, kv_len=[500, 300])
    ws = lh.new_attn_workspace(P, cuda_device, backward=True)
    low = torch.empty_like(q)

    def step():
        o, lse = lh.lh_attn_forward(P, q, k, v, low=low, ws=ws, **m)
        return (o, lse) + lh.lh_attn_backward(P, q, k, v, o, lse, dout, low=low, ws=ws, **m)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in (21, 22):
        for t, n in zip((q, k, v, dout), A.make(P, seed, cuda_device, grad=True)):
            t.copy_(n)
        m["kv_len"].copy_(torch.tensor([seed, 499], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        ref = A.reference(P, q, k, v, dout=dout, low=low, **m)
        for n, t in zip(("o", "lse", "dq", "dk", "dv", "dtable"), out):
            A.check(n, t, ref)
    assert lh.lh_get_status() == lh.LH_OK


@pytest.mark.parametrize("kind", ["slopes_cap", "table"])
def test_train_then_decode_from_the_cache(lh, cuda_device, kind):
    """A training step over whole sequences, then the same tokens one by one (and in a chunk) from a growing cache: the
    same rows come out."""
    B, Hq, Hkv, S, d = 2, 8, 2, 270, 128
    f = dict(softcap=30.0) if kind == "slopes_cap" else dict(buckets=32, max_distance=128)
    P = lh.AttnParams(B, Hq, Hkv, S, S, d, **f)
    q, k, v, dout = A.make(P, 30, cuda_device, grad=True)
    m = mods(P, cuda_device, slopes=kind == "slopes_cap")
    ref = A.reference(P, q, k, v, dout=dout, **m)
    for n, t in _all(lh, P, q, k, v, dout, m).items():
        A.check(n, t, ref)
    cap = 320
    kc, vc = (torch.full((B, Hkv, cap, d), math.nan, dtype=BF, device=cuda_device) for _ in range(2))  # not yet written
    n0 = 200
    kc[:, :, :n0], vc[:, :, :n0] = k[:, :, :n0], v[:, :, :n0]
    kv_len = torch.full((B,), n0, dtype=torch.int32, device=cuda_device)
    part = lambda a, b: {n: r[:, :, a:b] for n, r in ref.items() if n in ("o", "e_o", "lse", "e_lse")}  # noqa: E731
    chunk = lh.AttnParams(B, Hq, Hkv, 50, cap, d, **f)
    o, lse = lh.lh_attn_forward(chunk, q[:, :, n0 - 50:n0], kc, vc, kv_len=kv_len, **m)
    A.check("o", o, part(n0 - 50, n0))
    A.check("lse", lse, part(n0 - 50, n0))
    one = lh.AttnParams(B, Hq, Hkv, 1, cap, d, **f)
    ws = lh.new_attn_workspace(one, cuda_device)
    for t in range(n0, S, 13):
        kc[:, :, :t + 1], vc[:, :, :t + 1] = k[:, :, :t + 1], v[:, :, :t + 1]
        kv_len.fill_(t + 1)
        o, lse = lh.lh_attn_forward(one, q[:, :, t:t + 1], kc, vc, kv_len=kv_len, ws=ws, **m)
        A.check("o", o, part(t, t + 1))
        A.check("lse", lse, part(t, t + 1))


@pytest.mark.parametrize("p", [dict(Sq=900, Skv=900, d=128), dict(Sq=700, Skv=700, d=64, buckets=32, max_distance=128),
                               dict(Sq=1, Skv=3000, d=128), dict(Sq=60, Skv=2000, d=64, softcap=20.0)])
def test_wait_limit_is_reported_and_the_next_call_is_clean(lh, cuda_device, p):
    P = lh.AttnParams(B=1, Hq=4, Hkv=2, **p)
    q, k, v, dout = A.make(P, 40, cuda_device, grad=True)
    m = mods(P, cuda_device)
    ref = A.reference(P, q, k, v, dout=dout, **m)
    _all(lh, P, q, k, v, dout, m)
    assert lh.lh_get_status() == lh.LH_OK
    for ns in (1, 2000, 8000):
        lh.lh_set_wait_limit_ns(ns)
        try:
            _all(lh, P, q, k, v, dout, m)
            status = lh.lh_get_status()
        finally:
            lh.lh_set_wait_limit_ns(0)
        assert status == lh.LH_ERR_TIMEOUT if ns == 1 else status in (lh.LH_OK, lh.LH_ERR_TIMEOUT)
    for n, t in _all(lh, P, q, k, v, dout, m).items():
        A.check(n, t, ref)
    assert lh.lh_get_status() == lh.LH_OK


def test_traced_kernels(lh, cuda_device):
    P = lh.AttnParams(1, 4, 2, 300, 300, 64, buckets=32, max_distance=128)
    q, k, v, dout = A.make(P, 50, cuda_device, grad=True)
    m = mods(P, cuda_device)
    lh.lh_profile_enable(True)
    _all(lh, P, q, k, v, dout, m)
    names = lh.lh_profile_read()
    lh.lh_profile_enable(False)
    assert set(names) == {"dense_fwd", "dense_bwd_prep", "dense_bwd", "dense_bwd_out"}
    assert all(n == 1 and ms > 0 for n, ms in names.values())
