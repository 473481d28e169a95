"""``AttnParams`` as an ordinary value: copied, pickled, replaced and out of range."""

from __future__ import annotations

import copy
import ctypes
import dataclasses
import gc
import pickle

import pytest
import torch

from hierarchical_sparse_attention_avg_b200 import lh

OK = dict(B=2, Hq=4, Hkv=2, Sq=16, Skv=64, d=64)
TABLE = dict(OK, dtype=torch.float16, causal=False, scale=0.3, softcap=20.0, buckets=32, max_distance=128, bidirectional=True)


@pytest.mark.parametrize("fields", [OK, TABLE])
@pytest.mark.parametrize("again", [copy.copy, copy.deepcopy, lambda p: pickle.loads(pickle.dumps(p)), dataclasses.replace,
                                   lambda p: copy.deepcopy({"attn": [p]})["attn"][0]],
                         ids=["copy", "deepcopy", "pickle", "replace", "nested"])
def test_copies_hold_their_own_sizes(fields, again):
    P = lh.AttnParams(**fields)
    want = (lh.lh_attn_validate(P), lh.lh_attn_workspace_bytes(P), lh.lh_attn_workspace_bytes(P, True))
    Q = again(P)
    assert Q == P and hash(Q) == hash(P) and Q is not P
    # the address that the calls pass is that of the copy's own struct (checked before anything reads through it)
    assert Q._ref == ctypes.addressof(Q._c) and (Q._c is not P._c)
    assert bytes(Q._c) == bytes(P._c)
    del P
    gc.collect()
    others = [lh.AttnParams(B=1, Hq=1, Hkv=1, Sq=1, Skv=1, d=96) for _ in range(64)]  # what the freed memory may hold now
    assert (lh.lh_attn_validate(Q), lh.lh_attn_workspace_bytes(Q), lh.lh_attn_workspace_bytes(Q, True)) == want
    assert len(others) == 64


def test_the_struct_that_calls_read_is_not_handed_out():
    P = lh.AttnParams(**OK)
    P.c().d = 128
    assert P.c().d == P._c.d == 64


@pytest.mark.parametrize("change", [dict(max_distance=2 ** 32 + 128), dict(B=2 ** 32 + 1), dict(Sq=2 ** 31), dict(Skv=-2 ** 32 + 64),
                                    dict(buckets=2 ** 32), dict(Hq=2 ** 32 + 4), dict(d=2 ** 32 + 64)])
def test_sizes_beyond_32_bits_are_refused(change):
    """The library's sizes are 32-bit: a larger one is not cut down to another one."""
    with pytest.raises(ValueError):
        lh.AttnParams(**{**TABLE, **change})
    assert lh.lh_attn_validate(lh.AttnParams(**dict(TABLE, max_distance=2 ** 31 - 1))) == lh.LH_OK


@pytest.mark.parametrize("given", [False, True])
def test_backward_without_its_table_is_refused(given):
    P = lh.AttnParams(**TABLE)
    q, k = (torch.zeros(P.B, h, s, P.d, dtype=P.dtype) for h, s in ((P.Hq, P.Sq), (P.Hkv, P.Skv)))
    dtable = torch.zeros(P.Hq, P.buckets, dtype=P.dtype) if given else None
    with pytest.raises(lh.LighthouseError) as e:
        lh.lh_attn_backward(P, q, k, k, q, torch.zeros(P.B, P.Hq, P.Sq), q, dtable=dtable)
    assert e.value.status == lh.LH_ERR_INVALID_ARG


def test_workspace_of_the_longest_queries():
    """Rows near 2^31 over 2^20 keys: the span of distances, their sum, stays positive."""
    size = lambda Sq: lh.lh_attn_workspace_bytes(lh.AttnParams(B=1, Hq=1, Hkv=1, Sq=Sq, Skv=1 << 20, d=64, buckets=32,  # noqa: E731
                                                               max_distance=2 ** 31 - 1), True)
    sizes = [size(Sq) for Sq in (2 ** 30, 2 ** 31 - 2 ** 21, 2 ** 31 - 2 ** 19, 2 ** 31 - 1)]
    assert sizes == sorted(sizes)
    # at least the fp32 accumulator of dq and the bias of each distance up to the last bucket's first one
    near = min(lh.lh_attn_bucket_starts(lh.AttnParams(B=1, Hq=1, Hkv=1, Sq=1, Skv=1, d=64, buckets=32, max_distance=2 ** 31 - 1))[-1],
               2 ** 31 - 1 + 2 ** 20)
    assert sizes[-1] >= (2 ** 31 - 1) * 64 * 4 + 2 * near * 5
