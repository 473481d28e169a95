"""Dense-stage attention in workspaces that hold other calls' leftovers and on two streams at once, every result held to the
definition (dq too, whose fp32 accumulator lies in the workspace), and plain causal attention over 98,304 positions."""

from __future__ import annotations

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


CASES = {
    "fp16_table_group": (dict(B=2, Hq=8, Hkv=2, Sq=300, Skv=500, d=64, dtype=FP, buckets=32, max_distance=128), dict(kv_len=[500, 333])),
    "fp16_docs_cap": (dict(B=1, Hq=4, Hkv=4, Sq=700, Skv=700, d=128, dtype=FP, softcap=20.0), dict(docs=[spans(700, 100, 500)])),
    "bf16_group_docs": (dict(B=1, Hq=8, Hkv=1, Sq=600, Skv=600, d=128), dict(docs=[spans(600, 250, 300)])),
    "bf16_slopes": (dict(B=3, Hq=2, Hkv=2, Sq=257, Skv=257, d=64), dict(slopes=True)),
    "bf16_table_both": (dict(B=2, Hq=4, Hkv=2, Sq=400, Skv=400, d=128, buckets=16, max_distance=100, bidirectional=True, causal=False), {}),
    "bf16_split": (dict(B=1, Hq=4, Hkv=2, Sq=9, Skv=6000, d=64), {}),
}


def _step(lh, P, x, m, ws):
    low = torch.empty_like(x[0])
    o, lse = lh.lh_attn_forward(P, *x[:3], low=low, ws=ws, **m)
    g = lh.lh_attn_backward(P, *x[:3], o, lse, x[3], low=low, ws=ws, **m)
    return dict(o=o, lse=lse, dq=g[0], dk=g[1], dv=g[2], **({"dtable": g[3]} if P.buckets else {}))


@pytest.mark.parametrize("name", CASES)
def test_a_used_workspace_changes_nothing(lh, cuda_device, name):
    p, m = CASES[name]
    P = lh.AttnParams(**p)
    x, m = A.make(P, 23, cuda_device, grad=True), mods(P, cuda_device, **m)
    ref = A.reference(P, *x[:3], dout=x[3], low=x[0], **m)  # (low: any tensor, for the bounds)
    ws = lh.new_attn_workspace(P, cuda_device, backward=True)
    for fill in (0xFF, 0x7F, 0x3C, None):  # NaN, large and ordinary numbers, then the last call's own
        if fill is not None:
            ws.fill_(fill)
        for n, t in _step(lh, P, x, m, ws).items():
            A.check(n, t, ref)
    assert lh.lh_get_status() == lh.LH_OK


@pytest.mark.parametrize("name", CASES)
def test_two_streams_at_once_give_their_own_results(lh, cuda_device, name):
    p, m = CASES[name]
    P = lh.AttnParams(**p)
    m = mods(P, cuda_device, **m)
    sets = [A.make(P, 24 + i, cuda_device, grad=True) for i in range(2)]
    refs = [A.reference(P, *x[:3], dout=x[3], low=x[0], **m) for x in sets]
    spaces = [lh.new_attn_workspace(P, cuda_device, backward=True) for _ in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(8):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = _step(lh, P, sets[i], m, spaces[i])
    torch.cuda.synchronize()
    for g, r in zip(got, refs):
        for n, t in g.items():
            A.check(n, t, r)


@pytest.mark.parametrize("d,dtype", [(128, BF), (64, FP)])
def test_plain_causal_training_over_98304_positions(lh, cuda_device, d, dtype):
    """One key head and two query heads; dq of some rows, dk and dv of some keys, o and lse of every row."""
    S, H = 98304, 2
    P = lh.AttnParams(1, H, 1, S, S, d, dtype=dtype)
    q, k, v, dout = A.make(P, 25, cuda_device, grad=True)
    low = torch.empty_like(q)
    o, lse = lh.lh_attn_forward(P, q, k, v, low=low)
    dq, dk, dv, _ = lh.lh_attn_backward(P, q, k, v, o, lse, dout, low=low)
    assert lh.lh_get_status() == lh.LH_OK
    u, eps, scale = A.half_step(P), 2.0 ** -14, d ** -0.5
    K, V = k[0, 0].double(), v[0, 0].double()
    g = torch.Generator().manual_seed(26)
    some = torch.cat([torch.tensor([0, 1, 127, 128, S // 2, S - 129, S - 128, S - 1]), torch.randint(0, S, (56,), generator=g)])
    some = some.unique().to(cuda_device)
    j = torch.arange(S, device=cuda_device)
    sums = torch.zeros(4, len(some), d, dtype=A.F8, device=cuda_device)  # dk, its bound, dv, its bound
    for h in range(H):
        for r0 in range(0, S, 2048):
            rows, n = j[r0:r0 + 2048, None], r0 + 2048  # (no row sees a key beyond n)
            Q, W = q[0, h, r0:n].double(), dout[0, h, r0:n].double()
            z = (Q @ K[:n].T) * scale
            z.masked_fill_(j[:n] > rows, -float("inf"))
            L = torch.logsumexp(z, 1, keepdim=True)
            ez = Q.norm(dim=1, keepdim=True) * K.norm(dim=1).max() * (scale * d * 2.0 ** -24)
            ez = ez + (1 + z.masked_fill(j[:n] > rows, 0).abs().amax(1, keepdim=True)) * 2.0 ** -18
            p = torch.exp(z - L)
            del z
            O, pv = p @ V[:n], p @ V[:n].abs()
            D, wpv = (W * O).sum(1, keepdim=True), (W.abs() * pv).sum(1, keepdim=True)
            eD, ep = (u + u * u + eps) * wpv, 2.0 ** -16 + 2 * ez

            def gradients(p, V):  # dS and its error, of these pairs
                dp = W[:len(p)] @ V.T
                dz = p * (dp - D[:len(p)])
                e = p * eD[:len(p)] + ep[:len(p)] * p * (dp.abs() + wpv[:len(p)])
                return dz, u * dz.abs() + e + p * (2.0 ** -17 * W[:len(p)].norm(dim=1, keepdim=True) * V.norm(dim=1))

            part = dict(lse=L[:, 0], e_lse=(ez + 2.0 ** -18 * (1 + L.abs()))[:, 0], o=O, e_o=u * O.abs() + (u + eps + ez) * pv)
            A.check("lse", lse[0, h, r0:n], part)
            A.check("o", o[0, h, r0:n], part)
            here = some[some < n]
            ds, e = gradients(p[:, here], V[here])
            sums[0, :len(here)] += scale * (ds.T @ Q)
            sums[1, :len(here)] += scale * (e.T @ Q.abs())
            sums[2, :len(here)] += p[:, here].T @ W
            sums[3, :len(here)] += (u + eps + ez.max()) * (p[:, here].T @ W.abs())
            mine = some[(some >= r0) & (some < n)] - r0
            if len(mine):
                pm = p[mine]
                del p
                W, D, wpv, eD, ep = (t[mine] for t in (W, D, wpv, eD, ep))
                ds, e = gradients(pm, V[:n])
                want = scale * (ds @ K[:n])
                A.check("dq", dq[0, h, r0 + mine], dict(dq=want, e_dq=u * want.abs() + scale * (e @ K[:n].abs())))
    A.check("dk", dk[0, 0, some], dict(dk=sums[0], e_dk=u * sums[0].abs() + sums[1]))
    A.check("dv", dv[0, 0, some], dict(dv=sums[2], e_dv=u * sums[2].abs() + sums[3]))
