"""Decode attention with scoring options (kvq_paged_decode_attn_scored) and
behind a shared prefix (kvq_shared_prefix_decode_attn) against plain float64
attention over the same pages."""

import math

import pytest
import torch

from attn_plain import attention, float_tolerance, half_tolerance, rows, seen_mask
from bit_rotated_kv_block_b200 import kvq
from test_gpu_prefill import Batch

pytestmark = pytest.mark.gpu


def reference(b, s, L, q, cap=0.0, window=0, slopes=None, first=None, sm=None, skip_pages=()):
    pages = b.table[s, :-(-L // b.P)].clamp(0, b.cache.NP - 1).long()  # (bad ones are masked)
    k, v = rows(b.kc, b.kp, pages, b.d)[:L], rows(b.vc, b.vp, pages, b.d)[:L]
    pos = torch.tensor([L - 1], device="cuda")
    bad = torch.zeros(len(pages), dtype=torch.bool, device="cuda")
    for pg in skip_pages:
        bad[pg] = True
    seen = seen_mask(L, pos, window, None if first is None else first[s:s + 1], 0,
                     bad.repeat_interleave(b.P)[:L])
    sm = 1.0 / math.sqrt(b.d) if sm is None else sm
    ref, A, S = attention(q[s:s + 1], k, v, pos, b.G, sm, b.R, cap, slopes, seen, b.rope)
    vis = v[seen[0]]
    return ref[0], A[0], S[0], float(vis.abs().max()) if len(vis) else 0.0


def scored(b, q, cap=0.0, window=0, slopes=None, first=None, lens=None, max_len=None, **kw):
    lens = b.lens if lens is None else lens
    out = kvq.paged_decode_attn_scored(
        b.cache, q, b.i32(lens), max(lens) if max_len is None else max_len, b.table, b.kc, b.kp,
        b.vc, b.vp, score=kvq.Score(cap, window, slopes, first), err=b.err, **kw)
    torch.cuda.synchronize()
    return out


def check(b, out, q, half=False, **kw):
    slopes = kw.get("slopes")
    for s, L in enumerate(b.lens):
        if L == 0:
            assert bool((out[s] == 0).all())
            continue
        ref, A, S, vmax = reference(b, s, L, q, **kw)
        bias = 0.0 if slopes is None else float(slopes.abs().max()) * L
        cap = kw.get("cap", 0.0)
        tol = half_tolerance(ref, A, S, L, vmax, cap, bias) if half else \
            float_tolerance(A, S, L, cap, bias)
        off = (out[s].double() - ref).norm(dim=-1)
        assert bool((off <= tol).all()), (s, L, float((off / tol).max()))


def batch(lens, **kw):
    b = Batch(lens, [1 if n else 0 for n in lens], **kw)
    g = torch.Generator().manual_seed(77)
    return b, torch.randn((len(lens), b.H * b.G, b.d), generator=g).half().cuda()


SHAPES = [(128, 4, 16, 1, 64), (128, 8, 32, 1, 128), (128, 1, 64, 1, 16), (128, 5, 16, 2, 0),
          (128, 3, 32, 0, 0), (256, 4, 16, 1, 256), (256, 2, 32, 1, 64), (256, 1, 64, 5, 0)]
OPTS = [dict(), dict(cap=50.0), dict(cap=3.0), dict(window=1), dict(window=100), dict(slopes=1),
        dict(first=1), dict(cap=30.0, window=333, slopes=1, first=1)]


def options(opt, b):
    kw = dict(opt)
    if "slopes" in kw:
        n = b.H * b.G
        kw["slopes"] = torch.tensor([2.0 ** (-1 - 7 * i / n) for i in range(n)], device="cuda")
    if "first" in kw:
        kw["first"] = b.i32([n // 3 for n in b.lens])
    return kw


@pytest.mark.parametrize("d,G,P,kind,block", SHAPES)
def test_scored_shapes(d, G, P, kind, block):
    b, q = batch([1, 700, 16, 333, 0, 2050], d=d, G=G, P=P, kind=kind, block=block, wide=10.0)
    for opt in (OPTS[1], OPTS[-1]):
        kw = options(opt, b)
        check(b, scored(b, q, **kw), q, **kw)
    assert int(b.err.item()) == 0


@pytest.mark.parametrize("opt", OPTS, ids=lambda o: "-".join(o) or "plain")
@pytest.mark.parametrize("d,G", [(128, 4), (128, 8), (256, 4)])
def test_scored_options(opt, d, G):
    b, q = batch([1500, 64, 129], d=d, G=G, wide=6.0, seed=1)
    kw = options(opt, b)
    out = scored(b, q, **kw)
    check(b, out, q, **kw)
    if not opt:
        plain = kvq.paged_decode_attn(b.cache, q, b.i32(b.lens), max(b.lens), b.table, b.kc, b.kp,
                                      b.vc, b.vp)
        assert float((plain - out).abs().max()) <= 1e-5


def test_scored_sees_nothing_and_idle_slots():
    b, q = batch([100, 0, 50], seed=2)
    out = scored(b, q, first=b.i32([100, 0, 10]))   # the first query's document is empty
    assert bool((out[0] == 0).all()) and bool((out[1] == 0).all())
    check(b, out, q, first=b.i32([100, 0, 10]))
    assert int(b.err.item()) == 0


def test_scored_reads_no_page_before_the_window():
    b, q = batch([900, 431], seed=3)
    want = scored(b, q, window=50)
    b.table[0, :(900 - 50) // 16] = -1
    b.table[1, :(431 - 50) // 16] = b.cache.NP + 7
    got = scored(b, q, window=50)
    assert int(b.err.item()) == 0 and torch.equal(got, want)


def test_scored_flags():
    b, q = batch([300, 90], seed=4)
    b.table[0, 2] = -3
    out = scored(b, q, cap=20.0)
    assert int(b.err.item()) == kvq.ERRF_PAGE
    ref, A, S, _ = reference(b, 0, 300, q, cap=20.0, skip_pages=[2])
    assert bool(((out[0].double() - ref).norm(dim=-1) <= float_tolerance(A, S, 300, 20.0)).all())
    b.err.zero_()
    out = scored(b, q, lens=[-1, 90], max_len=90)
    assert int(b.err.item()) == kvq.ERRF_LEN and bool((out[0] == 0).all())


def test_scored_rope():
    b, q = batch([200, 77], rope=True, seed=5)
    check(b, scored(b, q, cap=15.0), q, cap=15.0)


# ---- a shared prefix ---------------------------------------------------------

def share(b, prefix):
    """Makes every sequence begin with sequence 0's first `prefix` tokens."""
    P, n = b.P, prefix // b.P
    for s in range(1, len(b.lens)):
        if b.lens[s] == 0:
            b.table[s, :n] = -9      # never read
            continue
        b.table[s, :n] = b.table[0, :n]
        if prefix % P:
            a, c = int(b.table[0, n]), int(b.table[s, n])
            for pool in (b.kc, b.kp, b.vc, b.vp):
                pool[c, :, :prefix % P] = pool[a, :, :prefix % P]


def shared(b, q, prefix, cap=0.0, window=0, slopes=None, first=None, lens=None, **kw):
    lens = b.lens if lens is None else lens
    out = torch.full(q.shape, 5.0, dtype=torch.float16, device="cuda")
    kvq.shared_prefix_decode_attn(
        b.cache, q, prefix, b.i32(lens), max(lens), b.table, b.kc, b.kp, b.vc, b.vp, out=out,
        score=kvq.Score(cap, window, slopes, first), err=b.err, **kw)
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("d,G,P,kind,block", SHAPES)
@pytest.mark.parametrize("prefix", [0, 1, 64, 517])
def test_shared_shapes(d, G, P, kind, block, prefix):
    b, q = batch([prefix + 40, max(prefix, 1), prefix + 1, 0, prefix + 300], d=d, G=G, P=P, kind=kind,
                 block=block, wide=10.0)
    share(b, prefix)
    kw = options(dict(cap=30.0), b)
    check(b, shared(b, q, prefix, **kw), q, half=True, **kw)
    check(b, shared(b, q, prefix), q, half=True)
    assert int(b.err.item()) == 0


@pytest.mark.parametrize("opt", OPTS, ids=lambda o: "-".join(o) or "plain")
@pytest.mark.parametrize("S", [2, 33, 70])
def test_shared_options(opt, S):
    lens = [700 + 37 * (i % 9) for i in range(S)]
    b, q = batch(lens, H=1, G=4, wide=6.0, seed=6)
    share(b, 690)
    kw = options(opt, b)
    check(b, shared(b, q, 690, **kw), q, half=True, **kw)


def test_shared_long_prefix_is_split():
    b, q = batch([9000, 8201, 8200 + 64], d=128, H=2, G=8, P=32, block=128, wide=12.0, seed=7)
    share(b, 8200)
    check(b, shared(b, q, 8200), q, half=True)


def test_shared_rope():
    b, q = batch([300, 280, 257], rope=True, seed=8)
    share(b, 256)
    check(b, shared(b, q, 256), q, half=True)


def test_shared_bad_lengths_and_pages():
    b, q = batch([200, 150, 300], seed=9)
    share(b, 144)
    out = shared(b, q, 144, lens=[200, 100, 300])   # shorter than the prefix
    assert int(b.err.item()) == kvq.ERRF_LEN
    assert bool((out[1] == 0).all())
    lens, b.lens = b.lens, [200, 0, 300]
    check(b, out, q, half=True)
    b.lens = lens
    b.err.zero_()
    b.table[0, 4] = b.cache.NP
    b.table[1, 4] = b.table[2, 4] = b.cache.NP
    out = shared(b, q, 144)
    assert int(b.err.item()) == kvq.ERRF_PAGE
    for s in range(3):
        ref, A, S, vmax = reference(b, s, b.lens[s], q, skip_pages=[4])
        off = (out[s].double() - ref).norm(dim=-1)
        assert bool((off <= half_tolerance(ref, A, S, b.lens[s], vmax)).all())


def test_chain_append_prefill_then_decode_steps_behind_a_shared_prefix():
    """A run as a server makes it: the prompts are appended and attended in
    chunks, then every sequence decodes behind the common prompt."""
    g = torch.Generator().manual_seed(11)
    d, H, G, P, S, pre, new = 128, 2, 4, 16, 3, 100, 5
    Hq = H * G
    cache = kvq.Cache(d, H, P, 64, kvq.ROT_HADAMARD, 64)
    kc, kp = cache.new_pools(fill=0x7E)
    vc, vp = cache.new_pools(fill=0x7E)
    table = torch.full((S, 10), -1, dtype=torch.int32)
    table[:, :6] = torch.arange(6, dtype=torch.int32)
    for s in range(S):
        table[s, 6:10] = torch.arange(10 + 4 * s, 14 + 4 * s, dtype=torch.int32)
    table = table.cuda()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    kv = [torch.randn((pre + new, H, d), generator=g).half().cuda() for _ in range(2)]
    q = torch.randn((S, pre + new, Hq, d), generator=g).half().cuda()
    b = Batch([pre], [1], d=d, H=H, G=G, P=P, block=64)  # carries R and the geometry
    b.cache, b.kc, b.kp, b.vc, b.vp, b.table = cache, kc, kp, vc, vp, table
    # the common prompt, in two chunks, attended as it is written
    for lo, hi in ((0, 64), (64, pre)):
        n = hi - lo
        for s in range(S) if hi == pre else range(1):  # every sequence has its own copy of the last page
            kvq.quantize_append(cache, kv[0][lo:hi], kv[1][lo:hi], i32([s] * n),
                                i32(list(range(lo, hi))), table, kc, kp, vc, vp)
        out = kvq.paged_prefill_attn(cache, q[0, lo:hi], i32([0, n]), n, i32([hi]), hi, table[:1],
                                     kc, kp, vc, vp)
        b.lens, b.qn, b.q_start, b.q = [hi], [n], [0, n], q[0, lo:hi]
        b.check(out)
    for step in range(new):
        L = pre + step + 1
        kvq.quantize_append(cache, kv[0][L - 1:L].expand(S, H, d).contiguous(),
                            kv[1][L - 1:L].expand(S, H, d).contiguous(), i32(list(range(S))),
                            i32([L - 1] * S), table, kc, kp, vc, vp)
        qs = q[:, L - 1].contiguous()
        b.lens = [L] * S
        check(b, shared(b, qs, pre), qs, half=True)
        check(b, scored(b, qs, window=40, cap=20.0), qs, window=40, cap=20.0)


def test_graphs_on_another_stream_match_eager():
    """Captured calls (split and merge kernels, the prefix's part beside the
    own part) replayed twice between other calls on the same workspace."""
    b, q = batch([900, 700, 811], seed=13)
    share(b, 640)
    want_s, want_p = scored(b, q, cap=20.0, window=300), shared(b, q, 640, cap=20.0)
    lens = b.i32(b.lens)
    sc, sp = kvq.Score(20.0, 300), kvq.Score(20.0)
    ws = torch.empty(kvq.decode_workspace_bytes(b.cache, 3, 8, 900) +
                     kvq.shared_prefix_workspace_bytes(b.cache, 3, 8, 640, 900), dtype=torch.uint8,
                     device="cuda")
    o1, o2 = torch.zeros_like(want_s), torch.zeros_like(want_p)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        kvq.paged_decode_attn_scored(b.cache, q, lens, 900, b.table, b.kc, b.kp, b.vc, b.vp,
                                     score=sc, out=o1, workspace=ws, stream=st)
        kvq.shared_prefix_decode_attn(b.cache, q, 640, lens, 900, b.table, b.kc, b.kp, b.vc, b.vp,
                                      score=sp, out=o2, workspace=ws, stream=st)
    for _ in range(2):
        o1.zero_(), o2.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o1, want_s) and torch.equal(o2, want_p)
    # back to back on one stream and workspace, nothing waited for between
    for _ in range(20):
        kvq.shared_prefix_decode_attn(b.cache, q, 640, lens, 900, b.table, b.kc, b.kp, b.vc, b.vp,
                                      score=sp, out=o2, workspace=ws)
        kvq.paged_decode_attn_scored(b.cache, q, lens, 900, b.table, b.kc, b.kp, b.vc, b.vp,
                                     score=sc, out=o1, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(o1, want_s) and torch.equal(o2, want_p)


def test_shared_prefix_seen_through_a_window_and_documents():
    """Rows of which some see part of the prefix, some none of it."""
    b, q = batch([700, 520, 900, 513], seed=14)
    share(b, 512)
    for kw in (dict(window=250), dict(window=1), dict(first=b.i32([100, 512, 600, 512])),
               dict(first=b.i32([700, 0, 511, 513]))):
        out = shared(b, q, 512, **kw)
        check(b, out, q, half=True, **kw)
    assert bool((out[0] == 0).all())       # its document begins behind it


def test_tensors_of_another_device_are_refused():
    b, q = batch([100], seed=15)
    with pytest.raises(ValueError):
        kvq.paged_decode_attn_scored(b.cache, q.cpu(), b.i32([100]), 100, b.table, b.kc, b.kp, b.vc,
                                     b.vp)
    with pytest.raises(ValueError):
        scored(b, q, slopes=torch.zeros(3, device="cuda"))


def test_decode_tensors_that_would_be_misread_are_refused():
    b, q = batch([100, 60], seed=16)
    ls = b.i32(b.lens)
    wide = torch.cat([b.table, b.table], 1)[:, :b.table.shape[1]]
    odd = torch.empty((2, 9, 128), dtype=torch.float16, device="cuda")[:, :8]
    for kw in (dict(q=q.float()), dict(q=odd), dict(q=q[..., :64]), dict(lens=ls.long()),
               dict(lens=ls[:1]), dict(lens=ls.cpu()), dict(table=wide), dict(table=b.table[:1]),
               dict(table=b.table.long()), dict(out=torch.empty_like(q).double())):
        a = dict(q=q, lens=ls, table=b.table, out=None)
        a.update(kw)
        with pytest.raises(ValueError):
            kvq.paged_decode_attn_scored(b.cache, a["q"], a["lens"], 100, a["table"], b.kc, b.kp,
                                         b.vc, b.vp, out=a["out"])
        with pytest.raises(ValueError):
            kvq.shared_prefix_decode_attn(b.cache, a["q"], 32, a["lens"], 100, a["table"], b.kc,
                                          b.kp, b.vc, b.vp, out=a["out"])


@pytest.mark.parametrize("d", [128, 256])
def test_scored_masked_token_that_is_not_finite(d):
    b, q = batch([700, 333], d=d, seed=17)
    kw = dict(window=64)
    keep = scored(b, q, **kw)
    for s, L in enumerate(b.lens):
        at = L - 66                  # just before the window, in a page it begins in or next to
        b.kp[int(b.table[s, at // 16]), :, at % 16] = 0x7E007E00
        b.vp[int(b.table[s, at // 16]), :, at % 16] = 0x7C007C00
    assert torch.equal(scored(b, q, **kw), keep)


def test_shared_masked_token_that_is_not_finite():
    b, q = batch([310, 420, 555], seed=18)
    share(b, 300)
    kw = dict(window=200)
    keep = shared(b, q, 300, **kw)
    at = 290                         # seen by the first two sequences alone
    b.kp[int(b.table[0, at // 16]), :, at % 16] = 0x7E007E00
    b.vp[int(b.table[0, at // 16]), :, at % 16] = 0x7C007C00
    out = shared(b, q, 300, **kw)
    assert torch.equal(out[2], keep[2]) and bool(out[:2].isnan().all())
