"""Host-side checks of the prompt, scored and shared-prefix attention entry
points: bad arguments return before any CUDA call (fake pointers, no GPU)."""

import ctypes
import os
import re

import pytest

from bit_rotated_kv_block_b200 import build, kvq

OK, INV, UNS, MIS, WSP = 0, 1, 2, 3, 4
GOOD = 1 << 20
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def L():
    build.build()
    return kvq.lib()


def desc(**kw):
    base = dict(head_dim=128, num_kv_heads=8, page_size=16, num_pages=16, rot_kind=1,
                rot_block=128, quat=None)
    base.update(kw)
    return kvq.CacheDesc(**base)


def score(**kw):
    base = dict(softcap=0.0, window=0, alibi=None, first_pos=None, prefix_lens=None)
    base.update(kw)
    return kvq.ScoreDesc(**base)


def prefill(L, d=None, S=2, Hq=32, T=10, q=GOOD, stride=4096, qs=GOOD, mq=5, lens=GOOD, mx=100,
            bt=GOOD, bts=8, sm=0.1, sc=None, pool=GOOD, out=GOOD, ws=GOOD, wsb=1 << 40):
    d = desc() if d is None else d
    return L.kvq_paged_prefill_attn(
        ctypes.byref(d), S, Hq, T, P(q), stride, P(qs), mq, P(lens), mx, P(bt), bts, sm,
        None if sc is None else ctypes.byref(sc), P(pool), P(GOOD), P(GOOD), P(GOOD), P(out), P(ws),
        wsb, None, None)


def scored(L, d=None, S=2, Hq=32, q=GOOD, lens=GOOD, mx=100, bt=GOOD, bts=8, sm=0.1, sc=None,
           pool=GOOD, out=GOOD, ws=GOOD, wsb=0):
    d = desc() if d is None else d
    return L.kvq_paged_decode_attn_scored(
        ctypes.byref(d), S, Hq, P(q), P(lens), mx, P(bt), bts, sm,
        None if sc is None else ctypes.byref(sc), P(pool), P(GOOD), P(GOOD), P(GOOD), P(out), P(ws),
        wsb, None, None)


def shared(L, d=None, S=2, Hq=32, q=GOOD, pre=64, lens=GOOD, mx=100, bt=GOOD, bts=8, sm=0.1,
           sc=None, pool=GOOD, out=GOOD, ws=GOOD, wsb=0):
    d = desc() if d is None else d
    return L.kvq_shared_prefix_decode_attn(
        ctypes.byref(d), S, Hq, P(q), pre, P(lens), mx, P(bt), bts, sm,
        None if sc is None else ctypes.byref(sc), P(pool), P(GOOD), P(GOOD), P(GOOD), P(out), P(ws),
        wsb, None, None)


def test_prefill_refusals(L):
    assert prefill(L, T=0) == OK                    # no query token: nothing is launched
    assert prefill(L, T=-1) == INV
    assert prefill(L, S=0) == INV
    assert prefill(L, mq=0) == INV
    assert prefill(L, mx=-1) == INV
    assert prefill(L, bts=0) == INV
    assert prefill(L, sm=float("nan")) == INV
    assert prefill(L, sm=float("inf")) == INV
    assert prefill(L, Hq=30) == INV
    for k in ("q", "qs", "lens", "bt", "pool", "out"):
        assert prefill(L, **{k: 0}) == INV, k
    assert prefill(L, stride=4088) == INV
    assert prefill(L, stride=4100) == MIS
    assert prefill(L, q=GOOD + 8) == MIS
    assert prefill(L, out=GOOD + 4) == MIS
    assert prefill(L, qs=GOOD + 2) == MIS
    assert prefill(L, ws=GOOD + 8) == MIS
    assert prefill(L, desc(head_dim=64, rot_block=64)) == UNS
    assert prefill(L, desc(format=kvq.FMT_MXFP4)) == UNS
    assert prefill(L, desc(format=kvq.FMT_INT3)) == UNS
    assert prefill(L, desc(page_size=24)) == UNS
    assert prefill(L, mx=2**31 - 1) == UNS          # positions stay 32-bit sums
    assert prefill(L, T=2**30, mq=2**30, wsb=1 << 50) == UNS
    # few tokens over a long cache are split: the workspace is then needed
    assert prefill(L, mx=1 << 16, bts=1 << 12, wsb=64) == WSP
    assert prefill(L, mx=1 << 16, bts=1 << 12, ws=0) == WSP


def test_prefill_workspace_size(L):
    d = ctypes.byref(desc())
    assert L.kvq_prefill_workspace_bytes(d, 2, 32, 10, 5, 1 << 16) > 0
    assert L.kvq_prefill_workspace_bytes(d, 2, 30, 10, 5, 1 << 16) == 0
    assert L.kvq_prefill_workspace_bytes(d, 0, 32, 10, 5, 1 << 16) == 0
    assert L.kvq_prefill_workspace_bytes(d, 2, 32, 10, 0, 1 << 16) == 0
    assert L.kvq_prefill_workspace_bytes(d, 64, 32, 1 << 16, 1024, 1024) == 0   # enough rows


@pytest.mark.parametrize("call", [prefill, scored, shared])
def test_score_options_are_checked(L, call):
    for bad in (score(softcap=-1.0), score(softcap=float("nan")), score(softcap=float("inf")),
                score(softcap=1e-9), score(window=-1)):
        assert call(L, sc=bad) == INV
    for bad in (score(alibi=GOOD + 2), score(first_pos=GOOD + 1)):
        assert call(L, sc=bad) == MIS


@pytest.mark.parametrize("call", [scored, shared])
def test_decode_forms_refusals(L, call):
    assert call(L, sc=score(prefix_lens=GOOD)) == INV   # a prompt option
    assert call(L, S=0) == INV
    assert call(L, Hq=30) == INV
    assert call(L, Hq=8 * 9) == UNS
    assert call(L, desc(head_dim=256), Hq=40) == UNS
    assert call(L, desc(head_dim=64, rot_block=64)) == UNS
    assert call(L, desc(format=kvq.FMT_INT2)) == UNS
    assert call(L, mx=2**31 - 1) == UNS
    assert call(L, sm=float("nan")) == INV
    for k in ("q", "lens", "bt", "pool", "out"):
        assert call(L, **{k: 0}) == INV, k
    assert call(L, q=GOOD + 4) == MIS
    assert call(L, ws=GOOD + 8) == MIS


def test_shared_prefix_refusals(L):
    assert shared(L, pre=-1) == INV
    assert shared(L, pre=8 * 16 + 1) == INV        # does not fit in a table row
    assert shared(L, bts=1, pre=17) == INV
    d = ctypes.byref(desc())
    assert L.kvq_shared_prefix_workspace_bytes(d, 2, 32, -1, 100) == 0
    assert L.kvq_shared_prefix_workspace_bytes(d, 2, 31, 64, 100) == 0


def test_score_desc_mirrors_the_header_struct():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(root, "include", "kvq.h")).read(), flags=re.S)
    heads = text[:text.index("} kvq_score_desc")]
    body = heads[heads.rindex("typedef struct"):].split("{", 1)[1]
    names = [f.replace("*", " ").split()[-1] for f in body.split(";") if f.strip()]
    assert names == [n for n, _ in kvq.ScoreDesc._fields_]
    assert ctypes.sizeof(kvq.ScoreDesc) == 32 and kvq.ScoreDesc.alibi.offset == 8


def test_score_object_checks_its_tensors():
    import torch
    with pytest.raises(ValueError):
        kvq.Score(alibi=torch.zeros(8, dtype=torch.float64))
    with pytest.raises(ValueError):
        kvq.Score(first_pos=torch.zeros((4, 2), dtype=torch.int32)[:, 0])
    with pytest.raises(ValueError):
        kvq.Score(prefix_lens=torch.zeros(4, dtype=torch.int64))


def test_score_tensors_have_to_fit_the_call():
    import torch
    q = torch.zeros((3, 8, 128))
    assert kvq._score(None, q, 2) is None
    kvq._score(kvq.Score(alibi=torch.zeros(8), first_pos=torch.zeros(3, dtype=torch.int32),
                         prefix_lens=torch.zeros(2, dtype=torch.int32)), q, 2)
    for bad in (kvq.Score(alibi=torch.zeros(7)), kvq.Score(first_pos=torch.zeros(2, dtype=torch.int32)),
                kvq.Score(prefix_lens=torch.zeros(3, dtype=torch.int32)),
                kvq.Score(alibi=torch.zeros(8, device="meta"))):
        with pytest.raises(ValueError):
            kvq._score(bad, q, 2)


def test_score_window_range_and_read_only_tensors():
    import torch
    for w in (-1, 2 ** 31, 2 ** 32 + 5):
        with pytest.raises(ValueError):
            kvq.Score(window=w)
    sc = kvq.Score(alibi=torch.zeros(8))
    with pytest.raises(AttributeError):
        sc.alibi = torch.ones(8)     # the descriptor would go on holding the old address
