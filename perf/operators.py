"""The operators of the dense stage that are measured: attention with capped scores, distance biases (fixed slopes, or
a learned table by buckets), document and prefix masks, over whole sequences and over a cache, and its gradients.

For row i of a batch entry, at position x = kv_len - Sq + i, and key j (GQA: query head h reads key head h // G):

    z = cap * tanh(scale * <q_i, k_j> / cap)  (or scale * <q_i, k_j> without a cap)
    z += -slope[h] * |x - j|   or   z += table[h, bucket(x - j)]
    visible: x >= 0, j < kv_len, doc[x] == doc[j] >= 0, and (not causal, or j <= x, or j < prefix)
    o_i = sum_j softmax(z)_ij v_j,   lse_i = log sum_j exp z_ij      (no visible key: o = 0, lse = -inf)

`run` computes that in elementary operations (`own` false) or through the library's entry points (`own` true)."""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _case(name, kind, B, Hq, Hkv, Sq, Skv, d, dtype="bf16", causal=True, cap=0.0, slopes=False, buckets=0, distance=0,
          both=False, docs=0, pad=False, prefix=False, ragged=False):
    c = dict(name=name, kind=kind, B=B, Hq=Hq, Hkv=Hkv, Sq=Sq, Skv=Skv, d=d, dtype=dtype, causal=causal, cap=cap,
             slopes=slopes, buckets=buckets, distance=distance, both=both, docs=docs, pad=pad, prefix=prefix,
             ragged=ragged)
    return c


def listed():
    return [
        # one token of one sequence over a short cache: what a single user waits for, all latency
        _case("token_short", "forward", 1, 16, 16, 1, 512, 64, cap=30.0, ragged=True),
        # one token for each sequence of a serving batch of uneven lengths, shared key heads
        _case("token_batch", "forward", 16, 32, 8, 1, 8192, 128, slopes=True, ragged=True),
        # one token of one very long sequence: the keys are split over the whole card
        _case("token_long", "forward", 1, 16, 4, 1, 200001, 128, cap=50.0),
        # one token with the learned bias, one key head a query head
        _case("token_bias", "forward", 8, 16, 16, 1, 4096, 64, dtype="fp16", buckets=32, distance=128, ragged=True),
        # a prompt taken in chunks: some hundred rows behind a long cache
        _case("chunk", "forward", 2, 16, 4, 257, 16384, 128, cap=50.0, ragged=True),
        # a packed prompt of several documents
        _case("prompt_docs", "forward", 1, 16, 16, 8192, 8192, 128, slopes=True, docs=6),
        # prompts whose first part is seen both ways
        _case("prompt_prefix", "forward", 4, 16, 16, 1531, 1531, 64, dtype="fp16", prefix=True),
        # the smallest training step
        _case("train_small", "train", 1, 2, 2, 200, 200, 64, cap=30.0, docs=3, pad=True),
        # a packed training row, capped scores, shared key heads
        _case("train_docs", "train", 1, 16, 4, 8192, 8192, 128, cap=50.0, docs=5, pad=True),
        # the largest: one long document with slopes
        _case("train_long", "train", 1, 8, 8, 16384, 16384, 128, slopes=True),
        # an encoder's batch, padded, bias both ways
        _case("train_encoder", "train", 8, 16, 16, 509, 509, 64, causal=False, buckets=32, distance=128, both=True,
              docs=1, pad=True),
        # a decoder's training step with the learned bias
        _case("train_bias", "train", 2, 16, 16, 4001, 4001, 128, dtype="fp16", buckets=32, distance=128),
    ]


def draw(rng):
    size = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))  # noqa: E731
    kind = rng.choice(["token", "chunk", "prompt", "train", "train"])
    d = rng.choice([64, 128])
    G = rng.choice([1, 1, 2, 4, 7, 8])
    c = dict(d=d, dtype=rng.choice(["bf16", "fp16"]), cap=rng.choice([0.0, 0.0, 20.0, 50.0]))
    bias = rng.choice(["none", "slopes", "table", "table"])
    c["slopes"] = bias == "slopes"
    if bias == "table":
        c.update(buckets=rng.choice([16, 32, 32, 64]), distance=rng.choice([100, 128, 500, 2000]))
    if kind in ("token", "chunk"):
        Hkv = rng.choice([1, 2, 4, 8])
        Sq = 1 if kind == "token" else size(2, 400)
        B = size(1, 24 if kind == "token" else 4)
        Skv = Sq + size(100, max(200, 600000 // (B * Hkv)) if kind == "token" else 16000)
        return {k: v for k, v in _case("", "forward", B, Hkv * G, Hkv, Sq, Skv, ragged=rng.random() < 0.7, **c).items()
                if k != "name"}
    S = size(150, 9000)
    Hkv = rng.choice([1, 2, 4])
    while Hkv * G > 16 or Hkv * G * S * S > 8 * 16384 * 16384:
        Hkv, G = max(1, Hkv // 2), max(1, G // 2)
    B = max(1, min(size(1, 8), 8 * 16384 * 16384 // (Hkv * G * S * S)))
    mask = rng.choice(["causal", "docs", "docs", "prefix", "all"])
    c.update(causal=mask != "all", prefix=mask == "prefix", both=bias == "table" and mask in ("prefix", "all"))
    if mask in ("docs", "all"):
        c.update(docs=rng.choice([1, 2, 5, 9]), pad=rng.random() < 0.5)
    return {k: v for k, v in _case("", "train" if kind == "train" else "forward", B, Hkv * G, Hkv, S, S, **c).items()
            if k != "name"}


def _layout(case, seed):
    """Lengths of a batch: valid keys, prefix lengths, and the documents' starts (the last entry: where padding begins)."""
    r = random.Random(seed * 7919 + 13)
    B, Sq, Skv = case["B"], case["Sq"], case["Skv"]
    lens = [r.randint(max(Sq, Skv // 4), Skv) if case["ragged"] else Skv for b in range(B)]
    prefix = [r.randint(1, max(1, Skv // 2)) if case["prefix"] else 0 for b in range(B)]
    ends = [r.randint(Skv // 2, Skv) if case["pad"] else Skv for b in range(B)]
    cuts = [sorted(r.sample(range(1, e), min(e - 1, max(0, case["docs"] - 1)))) for e in ends]
    docs = [[0] + c + [e] for c, e in zip(cuts, ends)]
    return lens, prefix, docs


def _slopes(H):
    return [2.0 ** (-8.0 * (h + 1) / H) for h in range(H)]


def prepare(case, seed):
    B, Hq, Hkv, Sq, Skv, d = (case[k] for k in ("B", "Hq", "Hkv", "Sq", "Skv", "d"))
    dt, dev = DTYPES[case["dtype"]], torch.device("cuda")
    g = torch.Generator(dev).manual_seed(seed)

    def rows(b, s, h):  # token rows of uneven size, as projections give them
        z = torch.randn(b, s, h, d, generator=g, device=dev)
        z *= torch.exp(0.5 * torch.randn(b, s, h, 1, generator=g, device=dev))
        return z.to(dt)

    lens, prefix, docs = _layout(case, seed)
    s = dict(case=case, q=rows(B, Sq, Hq).transpose(1, 2))  # [B, H, S, d] views of [B, S, H, d]
    s["k"], s["v"] = rows(B, Skv, Hkv).transpose(1, 2), rows(B, Skv, Hkv).transpose(1, 2)
    if case["Sq"] < case["Skv"]:  # a cache keeps each head's rows together
        s["k"], s["v"] = s["k"].contiguous(), s["v"].contiguous()
    if case["kind"] == "train":
        s["dout"] = (0.1 * torch.randn(B, Sq, Hq, d, generator=g, device=dev)).to(dt).transpose(1, 2)
    s["slopes"] = torch.tensor(_slopes(Hq), dtype=torch.float32, device=dev) if case["slopes"] else None
    s["table"] = torch.randn(Hq, case["buckets"], generator=g, device=dev).to(dt) if case["buckets"] else None
    s["kv_len"] = torch.tensor(lens, dtype=torch.int32, device=dev) if case["ragged"] else None
    s["prefix"] = torch.tensor(prefix, dtype=torch.int32, device=dev) if case["prefix"] else None
    s["docs"] = None
    if case["docs"]:
        ids = np.full((B, Skv), -1, dtype=np.int32)
        for b, starts in enumerate(docs):
            for n in range(len(starts) - 1):
                ids[b, starts[n]:starts[n + 1]] = n
        s["docs"] = torch.from_numpy(ids).to(dev)
    if own:  # the sizes and the workspace that a program keeps for calls of this shape
        from hierarchical_sparse_attention_avg_b200 import lh

        P = lh.AttnParams(B, Hq, Hkv, Sq, Skv, d, dtype=dt, causal=case["causal"], softcap=case["cap"],
                          buckets=case["buckets"], max_distance=case["distance"], bidirectional=case["both"])
        s["lh"], s["P"] = lh, P
        s["ws"] = lh.new_attn_workspace(P, dev, backward=case["kind"] == "train")
        if case["kind"] == "train":  # both calls get the buffer for what the output's rounding drops
            from functools import partial
            from types import SimpleNamespace

            low = torch.empty(B, Hq, Sq, d, dtype=dt, device=dev)
            s["lh"] = SimpleNamespace(lh_attn_forward=partial(lh.lh_attn_forward, low=low),
                                      lh_attn_backward=partial(lh.lh_attn_backward, low=low))
    return s


def _starts(n, distance):
    """First distance of each of n buckets: n // 2 single distances, then logarithmic ones up to `distance`."""
    e = max(1, n // 2)

    def first(b):  # the least x with (x / e) ** (n - e) >= (distance / e) ** (b - e), in whole numbers
        x = int(e * (distance / e) ** ((b - e) / (n - e)))
        ok = lambda y: y ** (n - e) * e ** (b - e) >= distance ** (b - e) * e ** (n - e)  # noqa: E731
        return next(y for y in range(max(1, x - 1), x + 3) if ok(y))

    return list(range(e)) + [first(b) for b in range(e, n)]


def _bias(s):
    """The buckets [Sq, Skv, B] of each pair, or None, and the distances' sizes."""
    case, dev = s["case"], s["q"].device
    B, Sq, Skv = case["B"], case["Sq"], case["Skv"]
    kv_len = s["kv_len"].long() if s["kv_len"] is not None else torch.full((B,), Skv, device=dev)
    x = kv_len[:, None] - Sq + torch.arange(Sq, device=dev)  # [B, Sq]
    delta = x[:, :, None] - torch.arange(Skv, device=dev)  # [B, Sq, Skv]
    if not case["buckets"]:
        return kv_len, x, delta, None
    n = case["buckets"] // 2 if case["both"] else case["buckets"]
    far = torch.arange(-(Skv + Sq), Skv + Sq + 1, device=dev)
    size = far.abs() if case["both"] else far.clamp(min=0)
    which = (size[:, None] >= torch.tensor(_starts(n, case["distance"]), device=dev)).sum(1) - 1
    which = which + n * (far < 0) if case["both"] else which
    return kv_len, x, delta, which[delta + (Skv + Sq)]


def _plain(s):
    case = s["case"]
    B, Hq, Hkv, Sq, Skv, d = (case[k] for k in ("B", "Hq", "Hkv", "Sq", "Skv", "d"))
    G, scale, cap = Hq // Hkv, 1.0 / math.sqrt(case["d"]), case["cap"]
    dt, dev = s["q"].dtype, s["q"].device
    kv_len, x, delta, bucket = _bias(s)
    j = torch.arange(Skv, device=dev)
    seen = (j < kv_len[:, None])[:, None, :] & (x >= 0)[:, :, None]
    if case["causal"]:
        p = s["prefix"] if s["prefix"] is not None else torch.zeros(B, device=dev)
        seen = seen & ((delta >= 0) | (j < p[:, None])[:, None, :])
    if s["docs"] is not None:
        ids = s["docs"]
        mine = ids.gather(1, x.clamp(min=0))
        seen = seen & (mine[:, :, None] == ids[:, None, :]) & (ids >= 0)[:, None, :]
    seen = seen[:, None, None]  # [B, 1, 1, Sq, Skv]
    q = s["q"].float().reshape(B, Hkv, G * Sq, d)
    k, v = s["k"].float(), s["v"].float()
    z = (q @ k.transpose(2, 3)).mul_(scale).view(B, Hkv, G, Sq, Skv)
    t = torch.tanh(z / cap) if cap else None
    z = t * cap if cap else z
    if s["slopes"] is not None:
        z = z - s["slopes"].view(1, Hkv, G, 1, 1) * delta.abs()[:, None, None]
    if bucket is not None:
        z = z + s["table"].float()[:, bucket].transpose(0, 1).view(B, Hkv, G, Sq, Skv)
    z = z.masked_fill_(~seen, -math.inf)
    top = z.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
    e = torch.exp(z - top)
    del z
    total = e.sum(-1, keepdim=True)
    lse = (top + torch.log(total)).view(B, Hq, Sq)
    p = e.div_(torch.where(total > 0, total, torch.ones_like(total)))
    o32 = p.view(B, Hkv, G * Sq, Skv) @ v
    o = o32.view(B, Hq, Sq, d).to(dt)
    if case["kind"] != "train":
        return o, lse
    do = s["dout"].float().reshape(B, Hkv, G * Sq, d)
    dv = p.view(B, Hkv, G * Sq, Skv).transpose(2, 3) @ do
    dz = (do @ v.transpose(2, 3)).sub_((do * o32).sum(-1, keepdim=True)).view(B, Hkv, G, Sq, Skv).mul_(p)
    del p
    dtable = None
    if bucket is not None:  # the batch (distances are the same in each entry), then each row's buckets, then the rows
        hot = (bucket[0, :, :, None] == torch.arange(case["buckets"], device=dev)).float()  # [Sq, Skv, buckets]
        rows = dz.view(B, Hq, Sq, Skv).sum(0).transpose(0, 1) @ hot
        dtable = rows.double().sum(0).to(dt)
        del hot, rows
    if cap:
        dz = dz.mul_(1 - t * t)
    dz = dz.view(B, Hkv, G * Sq, Skv)
    dq, dk = (dz @ k).mul_(scale), (dz.transpose(2, 3) @ q).mul_(scale)
    out = (o, lse, dq.view(B, Hq, Sq, d).to(dt), dk.to(dt), dv.to(dt))
    return out if dtable is None else out + (dtable,)


def run(state):
    if not own:
        return _plain(state)
    lh, P, s = state["lh"], state["P"], state
    mods = dict(slopes=s["slopes"], table=s["table"], docs=s["docs"], prefix=s["prefix"], kv_len=s["kv_len"])
    o, lse = lh.lh_attn_forward(P, s["q"], s["k"], s["v"], ws=s["ws"], **mods)
    if s["case"]["kind"] != "train":
        return o, lse
    grads = lh.lh_attn_backward(P, s["q"], s["k"], s["v"], o, lse, s["dout"], ws=s["ws"], **mods)
    return (o, lse) + tuple(g for g in grads if g is not None)


def work(case):
    """Each visible pair: two products of length d forward and five backward; tensors moved once (the valid keys)."""
    lens, prefix, docs = _layout(case, 0)
    pairs, keys = 0, 0
    for b in range(case["B"]):
        spans = zip(docs[b][:-1], docs[b][1:]) if case["docs"] else [(0, lens[b])]
        for lo, hi in spans:
            x = np.arange(max(lo, lens[b] - case["Sq"]), hi, dtype=np.int64)
            last = np.minimum(np.maximum(x, prefix[b] - 1), hi - 1) if case["causal"] else np.full_like(x, hi - 1)
            pairs += int(np.maximum(last - lo + 1, 0).sum())
            keys += hi - lo
    d, Hq, Hkv, rows = case["d"], case["Hq"], case["Hkv"], case["B"] * case["Sq"]
    flops = 4 * pairs * Hq * d
    nbytes = 2 * d * (2 * rows * Hq + 2 * keys * Hkv) + 4 * rows * Hq
    if case["kind"] == "train":
        flops += 10 * pairs * Hq * d
        nbytes += 2 * d * (2 * rows * Hq + 2 * keys * Hkv)
    return {"bytes": nbytes, "flops": flops}


def exact(case, seed):
    """The definition in 64 bits, one head of one batch entry at a time."""
    s = prepare(case, seed)
    dev, f8 = s["q"].device, torch.float64
    B, Hq, Hkv, Sq, Skv, d = (case[k] for k in ("B", "Hq", "Hkv", "Sq", "Skv", "d"))
    G, scale, cap, train = Hq // Hkv, 1.0 / math.sqrt(d), case["cap"], case["kind"] == "train"
    if B * Hq * Sq * Skv * (d if train else 1) > 1 << 42:
        return None
    lens, prefix, docs = _layout(case, seed)
    o = torch.zeros(B, Hq, Sq, d, dtype=f8, device=dev)
    lse = torch.full((B, Hq, Sq), -math.inf, dtype=f8, device=dev)
    dq, dk, dv = torch.zeros_like(o), torch.zeros(B, Hkv, Skv, d, dtype=f8, device=dev), None
    dv, dtable = torch.zeros_like(dk), torch.zeros(Hq, max(1, case["buckets"]), dtype=f8, device=dev)
    for b in range(B):
        x0 = lens[b] - Sq
        spans = list(zip(docs[b][:-1], docs[b][1:])) if case["docs"] else [(0, lens[b])]
        for lo, hi in spans:  # rows and keys of one document see nothing outside it
            r0, r1 = max(lo, x0), hi
            if r1 <= r0 or hi <= lo:
                continue
            x = torch.arange(r0, r1, device=dev)[:, None]
            j = torch.arange(lo, hi, device=dev)[None]
            hidden = ((j > x) & (j >= prefix[b])) if case["causal"] else torch.zeros_like(j > x)
            far = x - j
            if case["buckets"]:
                n = case["buckets"] // 2 if case["both"] else case["buckets"]
                away = far.abs() if case["both"] else far.clamp(min=0)
                bucket = torch.zeros_like(far)
                for first in _starts(n, case["distance"])[1:]:
                    bucket += away >= first
                if case["both"]:
                    bucket[far < 0] += n
            for h in range(Hq):
                a = h // G
                q, k, v = s["q"][b, h, r0 - x0:r1 - x0].to(f8), s["k"][b, a, lo:hi].to(f8), s["v"][b, a, lo:hi].to(f8)
                z = scale * (q @ k.T)
                slope = None
                if cap:
                    slope = torch.cosh(z / cap) ** -2
                    z = cap * torch.tanh(z / cap)
                if case["slopes"]:  # the operator takes the slopes in 32 bits
                    z = z - float(np.float32(_slopes(Hq)[h])) * far.abs()
                if case["buckets"]:
                    z = z + s["table"][h].to(f8)[bucket]
                z[hidden] = -math.inf
                L = torch.logsumexp(z, 1)
                P = torch.exp(z - L[:, None])
                y = P @ v
                lse[b, h, r0 - x0:r1 - x0], o[b, h, r0 - x0:r1 - x0] = L, y
                if train:
                    w = s["dout"][b, h, r0 - x0:r1 - x0].to(f8)
                    dv[b, a, lo:hi] += P.T @ w
                    D = P * (w @ v.T - (w * y).sum(1, keepdim=True))
                    if case["buckets"]:  # sums of equal distance first: row i of the flipped D starts i columns later
                        R, C = D.shape
                        shifted = torch.nn.functional.pad(D.flip(1), (0, R)).reshape(-1)[:R * (C + R - 1)]
                        wide = torch.arange(C + R - 1, device=dev) + (r0 - lo) - (C - 1)
                        away = wide.abs() if case["both"] else wide.clamp(min=0)
                        at = (away[:, None] >= torch.tensor(_starts(n, case["distance"]), device=dev)).sum(1) - 1
                        at = at + n * (wide < 0) if case["both"] else at
                        dtable[h].index_add_(0, at, shifted.view(R, C + R - 1).sum(0))
                    D = D * slope if slope is not None else D
                    dq[b, h, r0 - x0:r1 - x0] = scale * (D @ k)
                    dk[b, a, lo:hi] += scale * (D.T @ q)
    if not train:
        return o, lse
    return (o, lse, dq, dk, dv) + ((dtable,) if case["buckets"] else ())
