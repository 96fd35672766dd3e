"""The prompt, scored and shared-prefix attention entry points where their
kernels' loops, number ranges and roundings are at their ends, against plain
float64 attention over the same pages."""

import math

import pytest
import torch

from attn_plain import attention, float_tolerance, half_tolerance, rows, seen_mask
from bit_rotated_kv_block_b200 import kvq
from test_gpu_prefill import Batch
from test_gpu_scored import batch, scored, share, shared

pytestmark = pytest.mark.gpu


def refill(b, k, v):
    """Writes other keys and values [tokens of all sequences][H][d] into the batch's cache."""
    ts = torch.cat([torch.full((n,), s, dtype=torch.int32) for s, n in enumerate(b.lens)])
    tp = torch.cat([torch.arange(n, dtype=torch.int32) for n in b.lens])
    kvq.quantize_append(b.cache, k.half().cuda().contiguous(), v.half().cuda().contiguous(),
                        ts.cuda(), tp.cuda(), b.table, b.kc, b.kp, b.vc, b.vp)


def rows_of(b, s, q, pos, cap=0.0, window=0):
    """Float64 results of one sequence's queries, with what their tolerances
    take: (out, A, S, largest seen value of each row [n][1])."""
    L = b.lens[s]
    pages = b.table[s, :-(-L // b.P)].long()
    k, v = rows(b.kc, b.kp, pages, b.d)[:L], rows(b.vc, b.vp, pages, b.d)[:L]
    seen = seen_mask(L, pos, window)
    ref, A, S = attention(q, k, v, pos, b.G, 1.0 / math.sqrt(b.d), b.R, cap, None, seen, b.rope)
    top = torch.where(seen, v.abs().amax(-1).amax(-1), torch.zeros((), dtype=torch.float64,
                                                                   device="cuda")).amax(1)
    return ref, A, S, top[:, None]


def check_prompt(b, out, cap=0.0, window=0):
    """As Batch.check, with each row's tolerance from the values that it sees."""
    for s, (L, n) in enumerate(zip(b.lens, b.qn)):
        a = b.q_start[s]
        ref, A, S, top = rows_of(b, s, b.q[a:a + n], torch.arange(L - n, L, device="cuda"), cap,
                                 window)
        off = (out[a:a + n].double() - ref).norm(dim=-1)
        tol = half_tolerance(ref, A, S, L, top, cap)
        assert bool((off <= tol).all()), (s, float((off / tol).max()), int(off.isnan().sum()))


def check_shared(b, out, q, cap=0.0, window=0):
    for s, L in enumerate(b.lens):
        ref, A, S, top = rows_of(b, s, q[s:s + 1], torch.tensor([L - 1], device="cuda"), cap, window)
        off = (out[s].double() - ref[0]).norm(dim=-1)
        tol = half_tolerance(ref, A, S, L, top, cap)[0]
        assert bool((off <= tol).all()), (s, float((off / tol).max()), int(off.isnan().sum()))


@pytest.mark.parametrize("d,opt", [(128, dict()), (256, dict()), (128, dict(cap=40.0, window=3500)),
                                   (256, dict(slopes=True))], ids=str)
def test_long_unsplit_prompt_with_rising_scores(d, opt):
    # 32 (64 at d 256) key tiles per block of rows, no split; every key scores
    # higher than the ones before it, so the reference maxima move all along
    L = 4096
    b = Batch([L], [L], d=d, H=1, G=4, block=64, seed=31)
    assert kvq.prefill_workspace_bytes(b.cache, 1, 4, L, L, L) == 0
    g = torch.Generator().manual_seed(32)
    u = torch.randn((1, 1, d), generator=g)
    at = torch.linspace(0.0, 1.5, L)[:, None, None]
    refill(b, u * at + 0.3 * torch.randn((L, 1, d), generator=g), torch.randn((L, 1, d), generator=g))
    b.qbuf.copy_((u.expand(L, 4, d) + 0.5 * torch.randn((L, 4, d), generator=g)).reshape(L, 4 * d))
    kw = dict(opt)
    if "slopes" in kw:
        kw["slopes"] = torch.tensor([2.0 ** (-4 - i) for i in range(4)], device="cuda")
    out = b.run(**kw)
    b.check(out, **kw)
    assert int(b.err.item()) == 0


def constant_tokens(b, value, at):
    """Standard normal keys and values, with tokens whose values are one constant
    in every channel (the Hadamard rotation gathers it in a channel per block).
    A row's stored minimum is a binary16 number, so a negative constant goes no
    lower than -65504 / sqrt(block); beyond it the cached row itself is infinite."""
    g = torch.Generator().manual_seed(33)
    T = sum(b.lens)
    v = torch.randn((T, b.H, b.d), generator=g)
    for i, t in enumerate(at):
        v[t] = value if i % 2 == 0 else -min(value, 65000.0 / math.sqrt(b.d))
    refill(b, torch.randn((T, b.H, b.d), generator=g), v)


@pytest.mark.parametrize("value", [3000.0, 11700.0, 20000.0, 50000.0])
@pytest.mark.parametrize("d,lens,qn", [(128, [300], [300]), (256, [200], [200]), (128, [2500], [40]),
                                       (128, [700, 333], [8, 16]), (256, [1500], [3])], ids=str)
def test_large_constant_values_are_finite(d, lens, qn, value):
    # a constant row of c decodes to c sqrt(block) in one channel, far above the
    # binary16 range for the larger ones, and is c again after the rotation back
    b = Batch(lens, qn, d=d, H=2, G=4, block=d)
    L, n = lens[0], qn[0]
    constant_tokens(b, value, [L - n, L - n // 2, 5])
    kw = dict(cap=30.0, window=100)
    check_prompt(b, b.run())
    check_prompt(b, b.run(**kw), **kw)
    check_prompt(b, b.run(window=1), window=1)
    assert int(b.err.item()) == 0


@pytest.mark.parametrize("value", [11700.0, 20000.0, 50000.0])
@pytest.mark.parametrize("d", [128, 256])
def test_large_constant_values_in_a_shared_prefix(d, value):
    b, q = batch([310, 420, 555], d=d, block=d, seed=34)
    constant_tokens(b, value, [7, 200, 299])
    share(b, 300)
    for kw in (dict(), dict(cap=30.0, window=300)):
        check_shared(b, shared(b, q, 300, **kw), q, **kw)
    assert int(b.err.item()) == 0


@pytest.mark.parametrize("size", [1e-3, 3e-4, 1e-4, 3e-5])
@pytest.mark.parametrize("d,lens,qn", [(128, [300], [300]), (256, [200], [200]), (128, [700, 333], [8, 16])],
                         ids=str)
def test_small_values_keep_their_bits(d, lens, qn, size):
    # value scales of a few binary16 subnormal steps; one-key windows give the
    # dequantized rows themselves
    b = Batch(lens, qn, d=d, H=2, G=4, block=64)
    g = torch.Generator().manual_seed(35)
    T = sum(lens)
    refill(b, torch.randn((T, 2, d), generator=g), size * torch.randn((T, 2, d), generator=g))
    for kw in (dict(window=1), dict(), dict(cap=20.0, window=50)):
        check_prompt(b, b.run(**kw), **kw)


@pytest.mark.parametrize("size", [1e-3, 1e-4, 3e-5])
def test_small_values_in_a_shared_prefix(size):
    b, q = batch([301, 302, 303], seed=36)
    g = torch.Generator().manual_seed(37)
    T = sum(b.lens)
    v = size * torch.randn((T, b.H, b.d), generator=g)
    refill(b, torch.randn((T, b.H, b.d), generator=g), v)
    share(b, 300)
    check_shared(b, shared(b, q, 300), q)


def lagging_batch(d, G, P, values, seed):
    """Sequences of 200 tokens of which one warp attends all (more pairs than
    resident warps), and queries whose score rises by about six bits at two
    tokens: less than moves the running reference. ``values(g, T, H)``: the
    value rows of a sequence, of which rows 100 and 130 are those tokens'."""
    b, q = batch([200] * 3 + [1] * 117, d=d, H=16, G=G, P=P, block=d, seed=seed)
    g = torch.Generator().manual_seed(seed)
    u = torch.randn((1, 1, d), generator=g)
    T = sum(b.lens)
    k = 0.02 * torch.randn((T, 16, d), generator=g)
    v = torch.randn((T, 16, d), generator=g)
    for s in range(3):
        k[200 * s + 100] = k[200 * s + 130] = 4.0 / math.sqrt(d) * u[0]
        v[200 * s:200 * s + 200] = values(g, 200, 16)
    refill(b, k, v)
    return b, (u + 0.05 * torch.randn(q.shape, generator=g)).half().cuda()


def check_scored(b, out, q, count, cap=0.0, window=0):
    for s in range(count):
        L = b.lens[s]
        ref, A, S, _ = rows_of(b, s, q[s:s + 1], torch.tensor([L - 1], device="cuda"), cap, window)
        off = (out[s].double() - ref[0]).norm(dim=-1)
        tol = float_tolerance(A, S, L, cap)[0]
        assert bool((off <= tol).all()), (s, float((off / tol).max()), int(off.isnan().sum()))


@pytest.mark.parametrize("size", [3e-5, 1e-4, 1e-3, 1e-2, 0.1, 30.0, 2000.0, 20000.0, 50000.0])
@pytest.mark.parametrize("d,G,P", [(128, 4, 16), (128, 8, 32), (128, 3, 64), (256, 4, 16), (256, 2, 64)])
def test_scored_over_value_sizes(d, G, P, size):
    def values(g, T, H):
        if size <= 30.0:
            return size * torch.randn((T, H, d), generator=g)
        v = torch.randn((T, H, d), generator=g)
        v[100], v[130] = size, -min(size, 65000.0 / math.sqrt(d))  # (binary16 minimum)
        return v
    b, q = lagging_batch(d, G, P, values, 41)
    for kw in (dict(), dict(cap=30.0, window=150)):
        check_scored(b, scored(b, q, **kw), q, 3, **kw)
    assert int(b.err.item()) == 0


@pytest.mark.parametrize("size", [1e-4, 20000.0])
@pytest.mark.parametrize("d", [128, 256])
def test_own_part_behind_a_prefix_over_value_sizes(d, size):
    # (a prefix of one token: nearly every position is the own part's)
    def values(g, T, H):
        v = min(size, 1.0) * torch.randn((T, H, d), generator=g)
        if size > 1.0:
            v[100] = v[130] = size
        return v
    b, q = lagging_batch(d, 4, 16, values, 42)
    share(b, 1)
    check_shared_some(b, shared(b, q, 1), q, 3)


def check_shared_some(b, out, q, count):
    lens, b.lens = b.lens, b.lens[:count]
    check_shared(b, out, q)
    b.lens = lens


@pytest.mark.parametrize("cap", [1e25, 1e30, 2e38, 3.4028234e38])
@pytest.mark.parametrize("d", [128, 256])
def test_a_huge_cap_is_none(d, cap):
    b, q = batch([700, 333], d=d, seed=51)
    share(b, 300)
    for call, chk in ((scored, lambda o: check_scored(b, o, q, 2)),
                      (lambda *a, **k: shared(*a[:2], 300, **k), lambda o: check_shared(b, o, q))):
        chk(call(b, q, cap=cap))
    p = Batch([300, 90], [300, 20], d=d, seed=52)
    p.check(p.run(cap=cap))
    if cap >= 1e30:
        assert torch.equal(p.run(cap=cap), p.run())
        assert torch.equal(scored(b, q, cap=cap), scored(b, q))


def test_pools_that_do_not_fit_the_cache_are_refused_by_every_call():
    b, q = batch([100, 60], seed=53)
    ls, qs = b.i32(b.lens), b.i32(b.q_start)
    calls = (lambda *p: kvq.paged_prefill_attn(b.cache, b.q, qs, 1, ls, 100, b.table, *p),
             lambda *p: kvq.paged_decode_attn_scored(b.cache, q, ls, 100, b.table, *p),
             lambda *p: kvq.shared_prefix_decode_attn(b.cache, q, 0, ls, 100, b.table, *p))
    for call in calls:
        call(b.kc, b.kp, b.vc, b.vp)
        for p in ((b.kc[:-1], b.kp, b.vc, b.vp), (b.kc, b.kp[:, :1].contiguous(), b.vc, b.vp),
                  (b.kc, b.kp, b.vc.transpose(1, 2), b.vp), (b.kc, b.kp, b.vc, b.vp.float())):
            with pytest.raises(ValueError):
                call(*p)
    torch.cuda.synchronize()


@pytest.mark.parametrize("d", [128, 256])
def test_rows_of_the_valid_sequence_beside_a_bad_range_when_keys_are_split(d):
    b = Batch([4000, 2500], [5, 3], d=d, tail=9, seed=11)
    b.q_start = [2, 7, 60]           # the second sequence's is no range of the rows
    out = b.run()
    assert int(b.err.item()) == kvq.ERRF_SEQ
    b.qn = [5, 0]
    b.check(out)
    assert bool((out[:2] == 7.0).all()) and bool((out[7:] == 7.0).all())


@pytest.mark.parametrize("word", [0x00007BFF, 0x7BFF7BFF, 0x7BFF0000, 0xFBFF7BFF - 2 ** 32, 0x7BFFFBFF],
                         ids=hex)
@pytest.mark.parametrize("d,lens,qn", [(128, [300], [200]), (256, [300], [200]), (128, [700], [9]),
                                       (128, [2500], [40])], ids=str)
def test_the_largest_finite_scales_and_minima(d, lens, qn, word):
    # (scale, minimum) of +-65504 and 0, one channel with code 15: values up to
    # 1.05e6. Zero queries weigh the seen tokens alike, so the results stay finite.
    b = Batch(lens, qn, d=d, H=2, G=4, block=d, seed=54)
    b.qbuf.zero_()
    at = 70
    page, slot = int(b.table[0, at // 16]), at % 16
    b.vp[page, :, slot] = word
    b.vc[page, :, slot] = 0
    b.vc[page, :, slot, 5] = 0x0F
    for kw in (dict(), dict(cap=20.0, window=250)):
        out = b.run(**kw)
        assert bool(out.isfinite().all())
        check_prompt(b, out, **kw)
        q = b.q[-1:].contiguous()
        check_scored(b, scored(b, q, **kw), q, 1, **kw)
    assert int(b.err.item()) == 0


def test_calls_on_two_streams_at_once():
    b, q = batch([900, 700, 811], seed=55)
    share(b, 640)
    p = Batch([500, 210], [30, 210], seed=56)
    want = shared(b, q, 640, cap=20.0), scored(b, q, window=300), p.run(cap=20.0)
    lens, plens, qs = b.i32(b.lens), p.i32(p.lens), p.i32(p.q_start)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    torch.cuda.synchronize()
    for _ in range(10):
        for st in streams:       # each call's output and workspace are its own
            pb, pp = (b.kc, b.kp, b.vc, b.vp), (p.kc, p.kp, p.vc, p.vp)
            outs.append((kvq.shared_prefix_decode_attn(b.cache, q, 640, lens, 900, b.table, *pb,
                                                       score=kvq.Score(20.0), stream=st),
                         kvq.paged_decode_attn_scored(b.cache, q, lens, 900, b.table, *pb,
                                                      score=kvq.Score(window=300), stream=st),
                         kvq.paged_prefill_attn(p.cache, p.q, qs, 210, plens, 500, p.table, *pp,
                                                score=kvq.Score(20.0), stream=st)))
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(x, y) for x, y in zip(o, want))


def test_many_sequences_with_few_tokens():
    S = 1500
    b = Batch([65 + i % 40 for i in range(S)], [1 + i % 3 for i in range(S)], H=1, G=4, seed=57)
    out = b.run()
    pick = list(range(0, S, 97))
    for s in pick:
        n = b.qn[s]
        ref, A, Sz, top = rows_of(b, s, b.q[b.q_start[s]:b.q_start[s] + n],
                                  torch.arange(b.lens[s] - n, b.lens[s], device="cuda"))
        off = (out[b.q_start[s]:b.q_start[s] + n].double() - ref).norm(dim=-1)
        assert bool((off <= half_tolerance(ref, A, Sz, b.lens[s], top)).all())
    share(b, 64)
    q = torch.randn((S, 4, 128), generator=torch.Generator().manual_seed(58)).half().cuda()
    got = shared(b, q, 64)
    for s in pick:
        ref, A, Sz, top = rows_of(b, s, q[s:s + 1], torch.tensor([b.lens[s] - 1], device="cuda"))
        off = (got[s].double() - ref[0]).norm(dim=-1)
        assert bool((off <= half_tolerance(ref, A, Sz, b.lens[s], top)[0]).all())
    assert int(b.err.item()) == 0
