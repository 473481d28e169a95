"""The dense-stage attention's definition in float64 (any device), its input makers and elementwise error bounds.

Bounds count the roundings of the kernels' number formats, u = finfo(dtype).eps / 2 relative each, and leave a little for
the 32-bit sums and exponentials (EPS32):
  o: the probabilities are rounded once before P V, the result once:      u |o| + (u + EPS32) P|V|
  dV: P rounded, the result rounded:                                      u |dV| + (u + EPS32) P^T|dO|
  dZ: D = <dO, O> uses O of rounded probabilities (u), rounded (u, or u^2 with `low`): eD = (2 u + EPS32) |dO|.(P|V|), P eD
  dK: dS rounded, D's error, the result rounded:                          u |dK| + scale ((u + EPS32) |dS| + P eD)^T |Q|
  dQ: likewise over the keys.   dtable: sums of dZ in 32 bits, D's error, the result rounded.
EPS32: scores are fp32 sums of d <= 128 products (d 2^-24 of |q||k| scale, measured there as `ez`), exponentials 2^-22."""

from __future__ import annotations

import math

import torch

F8 = torch.float64


def half_step(P) -> float:
    return torch.finfo(P.dtype).eps / 2


def bucket_index(far: torch.Tensor, buckets: int, distance: int, both: bool) -> torch.Tensor:
    """Bucket of each distance, from the definition in whole numbers."""
    n = buckets // 2 if both else buckets
    e = n // 2
    size = far.abs() if both else far.clamp(min=0)
    out = size.clamp(max=e - 1)
    for b in range(e, n):
        x = max(1, int(e * (distance / e) ** ((b - e) / (n - e))) - 2)
        while x ** (n - e) * e ** (b - e) < distance ** (b - e) * e ** (n - e):
            x += 1
        out = torch.where(size >= x, torch.full_like(out, b), out)
    return out + n * (far < 0) if both else out


def visible(B, Sq, Skv, causal, docs=None, prefix=None, kv_len=None):
    """(positions of the rows [B, Sq], mask [B, Sq, Skv]) on the CPU."""
    n = kv_len.cpu().long().clamp(0, Skv) if kv_len is not None else torch.full((B,), Skv)
    x = n[:, None] - Sq + torch.arange(Sq)
    j = torch.arange(Skv)
    m = (x >= 0)[:, :, None] & (j[None] < n[:, None])[:, None]
    if causal:
        p = prefix.cpu().long() if prefix is not None else torch.zeros(B, dtype=torch.long)
        m = m & ((j[None, None] <= x[:, :, None]) | (j[None] < p[:, None])[:, None])
    if docs is not None:
        ids = docs.cpu().long()
        mine = ids.gather(1, x.clamp(0, Skv - 1))
        m = m & (mine[:, :, None] == ids[:, None]) & (ids >= 0)[:, None]
    return x, m


def reference(P, q, k, v, slopes=None, table=None, docs=None, prefix=None, kv_len=None, low=None, dout=None):
    """dict of o, lse (and dq, dk, dv, dtable) in float64, each with its bound e_*."""
    dev, G = q.device, P.Hq // P.Hkv
    u, eps = torch.finfo(P.dtype).eps / 2, 2.0 ** -14
    scale = P.d ** -0.5 if P.scale is None else P.scale
    x, m = visible(P.B, P.Sq, P.Skv, P.causal, docs, prefix, kv_len)
    far = (x[:, :, None] - torch.arange(P.Skv)).to(dev)
    m = m.to(dev)
    dead_q, dead_k = ~m.any(2), ~m.any(1)
    clean = lambda t, dead: t.to(F8).masked_fill(dead[:, None, :, None], 0.0)  # noqa: E731
    Q = clean(q, dead_q)
    K, V = (clean(t, dead_k).repeat_interleave(G, 1) for t in (k, v))
    raw = Q @ K.transpose(2, 3) * scale
    t = torch.tanh(raw / P.softcap) if P.softcap else None
    z = P.softcap * t if P.softcap else raw
    if slopes is not None:
        z = z - slopes.to(F8)[None, :, None, None] * far.abs()[:, None]
    if table is not None:
        idx = bucket_index(far, P.buckets, P.max_distance, P.bidirectional)
        z = z + table.to(F8)[:, idx].transpose(0, 1)
    mm = m[:, None].expand_as(z) & (z > -1e38)  # a table's -inf or lowest value masks its bucket
    zmax = torch.where(mm, z.abs(), torch.zeros_like(z)).amax(3)
    z = z.masked_fill(~mm, -math.inf)
    lse = torch.logsumexp(z, 3)
    p = torch.where(mm, torch.exp(z - lse[..., None]), torch.zeros_like(z)).nan_to_num(0.0)
    ez = (Q.norm(dim=3) * K.norm(dim=3).amax(2, keepdim=True)) * (scale * P.d * 2.0 ** -24) + (1 + zmax) * 2.0 ** -18
    o, pv = p @ V, p @ V.abs()
    r = dict(lse=lse, e_lse=ez + 2.0 ** -18 * (1 + lse.abs().nan_to_num(0, 0, 0)), o=o,
             e_o=u * o.abs() + (u + eps + ez[..., None]) * pv, p=p)
    if dout is None:
        return r
    W = clean(dout, dead_q)
    heads = lambda a: a.view(P.B, P.Hkv, G, P.Skv, P.d).sum(2)  # noqa: E731
    dv, e_dv = p.transpose(2, 3) @ W, p.transpose(2, 3) @ W.abs()
    dp = W @ V.transpose(2, 3)
    dz = p * (dp - (W * o).sum(3, keepdim=True))
    eD = (((u + u * u if low is not None else 2 * u) + eps) * (W.abs() * pv).sum(3, keepdim=True))
    ep = (2.0 ** -16 + 2 * ez[..., None])  # relative error of p, and of dP against its products' size
    e_dz = p * eD + ep * p * (dp.abs() + (W.abs() * pv).sum(3, keepdim=True)) + p * (
        2.0 ** -17 * W.norm(dim=3)[..., None] * V.norm(dim=3)[:, :, None])
    ds = dz * (1 - t * t) if P.softcap else dz
    e_ds = u * ds.abs() + e_dz
    dq, e_dq = scale * (ds @ K), scale * (e_ds @ K.abs())
    dk, e_dk = scale * (ds.transpose(2, 3) @ Q), scale * (e_ds.transpose(2, 3) @ Q.abs())
    r.update(dq=dq, e_dq=u * dq.abs() + e_dq)
    r.update(dk=heads(dk), dv=heads(dv))
    r.update(e_dk=u * r["dk"].abs() + heads(e_dk), e_dv=u * r["dv"].abs() + (u + eps + ez.max()) * heads(e_dv))
    if table is not None:
        hot = lambda a: torch.stack([(a * (idx == b)[:, None]).sum((0, 2, 3)) for b in range(P.buckets)], 1)  # noqa: E731
        r["dtable"] = hot(dz)
        r["e_dtable"] = u * r["dtable"].abs() + hot(e_dz) + 2.0 ** -18 * hot(dz.abs())
    return r


def make(P, seed, device, grad=False, head_rows=True):
    """q, k, v (and dout): [B, H, S, d], views of [B, S, H, d] unless head_rows."""
    g = torch.Generator().manual_seed(seed)

    def rows(S, H):
        z = torch.randn(P.B, S, H, P.d, generator=g) * torch.exp(0.5 * torch.randn(P.B, S, H, 1, generator=g))
        z = z.to(P.dtype).to(device).transpose(1, 2)
        return z.contiguous() if head_rows else z

    out = [rows(P.Sq, P.Hq), rows(P.Skv, P.Hkv), rows(P.Skv, P.Hkv)]
    return out + [rows(P.Sq, P.Hq)] if grad else out


def check(name, got, ref, tiny=1e-7):
    """Elementwise |got - ref| <= bound; the same infinities."""
    want, bound = ref[name], ref["e_" + name]
    g = got.to(F8)
    assert g.shape == want.shape, (name, g.shape, want.shape)
    fin = torch.isfinite(want)
    assert torch.equal(torch.isfinite(g), fin), f"{name}: not finite at other places"
    assert torch.equal(g[~fin], want[~fin]), name
    over = ((g - want).abs() - bound)[fin] - tiny
    if over.numel() and over.max() > 0:
        i = int(over.argmax())
        raise AssertionError(f"{name}: {int((over > 0).sum())} of {over.numel()} outside; worst got {g[fin][i]:.6g}, "
                             f"want {want[fin][i]:.6g}, bound {bound[fin][i]:.3g}")
