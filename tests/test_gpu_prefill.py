"""Prompt attention (kvq_paged_prefill_attn) against plain float64 attention
over the same pages."""

import math

import numpy as np
import pytest
import torch

from attn_plain import attention, half_tolerance, rotation_matrix, rows, seen_mask
from bit_rotated_kv_block_b200 import kvq, workloads

pytestmark = pytest.mark.gpu


class Batch:
    """A filled cache and a ragged batch of query tokens."""

    def __init__(self, lens, qn, d=128, H=2, G=4, P=16, kind=1, block=64, seed=0, rope=False,
                 wide=1.0, pad_q=0, tail=0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.qn, self.d, self.H, self.G, self.P = lens, qn, d, H, G, P
        S = len(lens)
        npg = [-(-n // P) for n in lens]
        NP = sum(npg) + 2
        table = torch.full((S, max(npg + [0]) + 1), -1, dtype=torch.int32)
        perm = torch.randperm(NP, generator=g, dtype=torch.int32)
        o = 0
        for s in range(S):
            table[s, :npg[s]] = perm[o:o + npg[s]]
            o += npg[s]
        tbl = None
        if kind in (2, 3, 5):
            tbl = workloads.random_quaternions(seed, d)
        elif kind == 4:
            tbl = workloads.random_signs(seed, d)
        self.rope = torch.from_numpy(workloads.rope_table(max(lens) + 1, d)).cuda() if rope else None
        self.cache = kvq.Cache(d, H, P, NP, kind, block, tbl, rope=self.rope)
        self.R = rotation_matrix(d, kind, block, tbl)
        self.kc, self.kp = self.cache.new_pools(fill=0x7E)  # NaN parameters where nothing is written
        self.vc, self.vp = self.cache.new_pools(fill=0x7E)
        self.table = table.cuda()
        T = sum(lens)
        if T:
            mult = torch.ones((H, d))
            mult[:, 3] = mult[:, 77 % d] = wide
            kv = [(torch.randn((T, H, d), generator=g) * mult).half().cuda() for _ in range(2)]
            ts = torch.cat([torch.full((n,), s, dtype=torch.int32) for s, n in enumerate(lens)])
            tp = torch.cat([torch.arange(n, dtype=torch.int32) for n in lens])
            kvq.quantize_append(self.cache, kv[0], kv[1], ts.cuda(), tp.cuda(), self.table, self.kc,
                                self.kp, self.vc, self.vp)
        self.q_start = [0]
        for n in qn:
            self.q_start.append(self.q_start[-1] + n)
        self.T = self.q_start[-1] + tail
        Hq = H * G
        self.qbuf = torch.randn((max(1, self.T), Hq * d + pad_q), generator=g).half().cuda()
        self.q = self.qbuf[:self.T, :Hq * d].view(self.T, Hq, d) if pad_q == 0 else \
            self.qbuf.as_strided((self.T, Hq, d), (Hq * d + pad_q, d, 1))
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def i32(self, v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    def run(self, cap=0.0, window=0, slopes=None, first=None, bidir=None, sm_scale=None, **kw):
        sc = kvq.Score(cap, window, slopes, first, bidir)
        out = torch.full((self.T, self.H * self.G, self.d), 7.0, dtype=torch.float16, device="cuda")
        kvq.paged_prefill_attn(self.cache, self.q, self.i32(self.q_start),
                               max(1, max(self.qn)), self.i32(self.lens), max(self.lens),
                               self.table, self.kc, self.kp, self.vc, self.vp, out=out, score=sc,
                               err=self.err, sm_scale=sm_scale, **kw)
        torch.cuda.synchronize()
        return out

    def check(self, out, cap=0.0, window=0, slopes=None, first=None, bidir=None, sm_scale=None,
              bad_pages=()):
        sm = 1.0 / math.sqrt(self.d) if sm_scale is None else sm_scale
        for s, (L, n) in enumerate(zip(self.lens, self.qn)):
            if n == 0:
                continue
            a, b = self.q_start[s], self.q_start[s + 1]
            npg = -(-L // self.P)
            pages = self.table[s, :npg].long()
            badp = torch.zeros(npg, dtype=torch.bool, device="cuda")
            for ss, pg in bad_pages:
                if ss == s:
                    badp[pg] = True
            pages = torch.where(badp, torch.zeros_like(pages), pages)
            bad = badp.repeat_interleave(self.P)[:L]
            k = rows(self.kc, self.kp, pages, self.d)[:L]
            v = rows(self.vc, self.vp, pages, self.d)[:L]
            pos = torch.arange(L - n, L, device="cuda")
            seen = seen_mask(L, pos, window, None if first is None else first[a:b],
                             0 if bidir is None else int(bidir[s]), bad)
            ref, A, S = attention(self.q[a:b], k, v, pos, self.G, sm, self.R, cap, slopes, seen,
                                  self.rope)
            bias = 0.0 if slopes is None else float(slopes.abs().max()) * L
            tol = half_tolerance(ref, A, S, L, float(v[~bad].abs().max()) if (~bad).any() else 0.0,
                                 cap, bias)
            off = (out[a:b].double() - ref).norm(dim=-1)
            assert bool((off <= tol).all()), (s, float((off / tol).max()))


@pytest.mark.parametrize("d,G,P,kind,block", [
    (128, 4, 16, 1, 64), (128, 8, 32, 1, 128), (128, 1, 64, 1, 16), (128, 5, 16, 1, 32),
    (128, 3, 16, 0, 0), (128, 2, 32, 2, 0), (128, 4, 16, 3, 0), (128, 4, 16, 5, 0),
    (128, 4, 16, 4, 64), (256, 4, 16, 1, 256), (256, 2, 32, 1, 64), (256, 3, 64, 2, 0),
    (256, 1, 16, 4, 256), (128, 12, 16, 1, 64)])
def test_causal_chunks(d, G, P, kind, block):
    b = Batch([300, 1, 17, 129, 515], [300, 1, 5, 64, 33], d=d, G=G, P=P, kind=kind, block=block,
              wide=12.0)
    b.check(b.run())
    assert int(b.err.item()) == 0


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 256, 257])
@pytest.mark.parametrize("d", [128, 256])
def test_prompt_lengths(n, d):
    b = Batch([n], [n], d=d, H=1, G=4, block=128, seed=n)
    b.check(b.run())


@pytest.mark.parametrize("lens,qn", [([4000, 2500], [5, 3]), ([9001], [1]), ([2049], [17])])
@pytest.mark.parametrize("d", [128, 256])
def test_few_tokens_over_long_caches_split(lens, qn, d):
    b = Batch(lens, qn, d=d, H=2, G=4, block=64, wide=15.0, seed=3)
    assert kvq.prefill_workspace_bytes(b.cache, len(lens), 8, sum(qn), max(qn), max(lens)) > 0
    b.check(b.run())
    b.check(b.run(cap=30.0, window=1000), cap=30.0, window=1000)


OPTIONS = [dict(cap=50.0), dict(cap=5.0), dict(window=1), dict(window=100), dict(window=128),
           dict(slopes=True), dict(first=True), dict(bidir=True),
           dict(cap=30.0, window=70, slopes=True, first=True, bidir=True)]


@pytest.mark.parametrize("opt", OPTIONS, ids=lambda o: "-".join(o))
@pytest.mark.parametrize("d", [128, 256])
def test_options(opt, d):
    b = Batch([400, 129, 64], [390, 40, 64], d=d, H=2, G=4, wide=8.0, seed=5)
    kw = dict(opt)
    if "slopes" in kw:
        kw["slopes"] = torch.tensor([2.0 ** (-1 - i) for i in range(8)], device="cuda")
    if "first" in kw:
        pos = torch.cat([torch.arange(L - n, L) for L, n in zip(b.lens, b.qn)])
        f = pos // 50 * 50
        f[10] = pos[10] + 1      # a document that starts behind its token: sees nothing
        kw["first"] = f.to(torch.int32).cuda()
    if "bidir" in kw:
        kw["bidir"] = b.i32([200, 0, 64])
    out = b.run(**kw)
    b.check(out, **kw)
    if "first" in kw and not opt.get("bidir"):
        assert bool((out[10] == 0).all())


def test_rope_turns_each_query_by_its_position():
    b = Batch([200, 77], [60, 77], rope=True, seed=9)
    b.check(b.run())


def test_strided_queries_and_rows_behind_the_batch():
    b = Batch([90, 40], [33, 40], pad_q=64, tail=5)
    out = b.run()
    b.check(out)
    assert bool((out[b.q_start[-1]:] == 7.0).all())


def test_idle_and_bad_sequences():
    b = Batch([50, 60, 70], [10, 0, 20])
    b.check(b.run())
    assert int(b.err.item()) == 0
    b.lens = [50, 60, 15]          # fewer cached tokens than query tokens
    out = b.run()
    assert int(b.err.item()) == kvq.ERRF_LEN
    assert bool((out[10:] == 0).all())
    b.lens, b.qn = [50, 60], [10, 0]
    b.err.zero_()
    b.q_start, b.table = [0, 10, 31], b.table[:2].contiguous()  # past the T rows: not written
    out = b.run()
    assert int(b.err.item()) == kvq.ERRF_SEQ
    b.check(out[:10])
    assert bool((out[10:] == 7.0).all())


def test_bad_page_is_not_seen():
    b = Batch([200, 90], [20, 90], seed=4)
    b.table[0, 3] = b.cache.NP
    b.table[1, 0] = -5
    out = b.run()
    assert int(b.err.item()) == kvq.ERRF_PAGE
    b.check(out, bad_pages=[(0, 3), (1, 0)])


def test_pages_before_the_window_may_be_gone():
    b = Batch([600, 333], [8, 70], seed=6)
    keep = b.run(window=64)
    b.table[0, :(600 - 8 - 64) // 16] = -1
    b.table[1, :(333 - 70 - 64) // 16] = -1
    out = b.run(window=64)
    assert int(b.err.item()) == 0 and torch.equal(out, keep)


def test_extreme_scores_and_zero_query():
    b = Batch([300], [40], wide=30.0, seed=8)
    b.q[3] = 0
    b.q[5] *= 200
    b.check(b.run())
    b.check(b.run(sm_scale=-0.3), sm_scale=-0.3)
    b.check(b.run(sm_scale=0.0), sm_scale=0.0)


def test_graph_replay_on_another_stream_matches():
    b = Batch([500, 210], [30, 210], seed=2)
    want = b.run(cap=20.0)
    st = torch.cuda.Stream()
    out = torch.zeros_like(want)
    qs, ls = b.i32(b.q_start), b.i32(b.lens)
    need = kvq.prefill_workspace_bytes(b.cache, 2, 8, b.T, 210, 500)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    sc = kvq.Score(softcap=20.0)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        kvq.paged_prefill_attn(b.cache, b.q, qs, 210, ls, 500, b.table, b.kc, b.kp, b.vc, b.vp,
                               out=out, workspace=ws, score=sc, stream=st)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("d", [128, 256])
def test_rows_of_no_sequence_stay_as_they_were_when_keys_are_split(d):
    b = Batch([4000, 2500], [5, 3], d=d, tail=9, seed=11)
    assert kvq.prefill_workspace_bytes(b.cache, 2, 8, b.T, 5, 4000) > 0
    out = b.run(workspace=torch.full((1 << 24,), 0x3C, dtype=torch.uint8, device="cuda"))
    b.check(out)
    assert int(b.err.item()) == 0 and bool((out[8:] == 7.0).all())
    b.q_start = [2, 7, 60]           # two rows before the first sequence; the second's is no range
    out = b.run(workspace=torch.full((1 << 24,), 0x3C, dtype=torch.uint8, device="cuda"))
    assert int(b.err.item()) == kvq.ERRF_SEQ
    assert bool((out[:2] == 7.0).all()) and bool((out[7:] == 7.0).all())
    assert bool((out[2:7] != 7.0).any())


@pytest.mark.parametrize("word", [0x7C007C00, 0x7E007E00, 0x3C00FC00, 0x7BFF0000, 0x00007BFF])
@pytest.mark.parametrize("key", [False, True], ids=["value", "key"])
@pytest.mark.parametrize("d,lens,qn", [(128, [300], [300]), (256, [150], [150]), (128, [2500], [40])])
def test_a_token_that_is_not_finite_reaches_only_the_queries_that_see_it(word, key, d, lens, qn):
    # (scale, minimum) of one token: infinities, NaN, a minimum of -infinity,
    # and finite pairs whose dequantized values leave the binary16 range
    b = Batch(lens, qn, d=d, H=1, G=4, seed=12)
    L, n = lens[0], qn[0]
    at = L - n + 21                  # inside the first tiles of the chunk
    keep = b.run(window=9)
    pool = b.kp if key else b.vp
    pool[int(b.table[0, at // 16]), 0, at % 16] = word
    if not key:
        b.vc[int(b.table[0, at // 16]), 0, at % 16] = 0xFF
    out = b.run(window=9)
    sees = torch.zeros(n, dtype=torch.bool, device="cuda")
    sees[21:30] = True
    assert torch.equal(out[~sees], keep[~sees])
    if word in (0x7C007C00, 0x7E007E00) or (word == 0x3C00FC00 and not key):
        assert bool(out[sees].isnan().all())
    assert int(b.err.item()) == 0


@pytest.mark.parametrize("lens,qn", [([300], [40]), ([4000], [5])])
def test_a_query_that_is_not_a_number_stays_one(lens, qn):
    b = Batch(lens, qn, seed=13)
    keep = b.run()
    b.q[2, 1, 5] = float("nan")
    out = b.run()
    assert bool(out[2, 1].isnan().all())
    out[2, 1] = keep[2, 1]
    assert torch.equal(out, keep)


def test_tensors_that_would_be_misread_are_refused():
    b = Batch([100, 60], [10, 20], seed=14)
    qs, ls = b.i32(b.q_start), b.i32(b.lens)

    def call(q=b.q, q_start=qs, lens=ls, table=b.table, out=None, vp=b.vp):
        return kvq.paged_prefill_attn(b.cache, q, q_start, 20, lens, 100, table, b.kc, b.kp, b.vc,
                                      vp, out=out)
    want = call()
    wide = torch.cat([b.table, b.table], 1)[:, :b.table.shape[1]]     # rows further apart
    for kw in (dict(q=b.q.float()), dict(q=b.q.bfloat16()), dict(q=b.q[:, :, :64]),
               dict(q=b.q.transpose(0, 1)), dict(q_start=qs.long()), dict(q_start=qs[:2]),
               dict(q_start=qs.cpu()), dict(lens=ls.long()), dict(lens=ls.cpu()),
               dict(table=b.table.long()), dict(table=b.table[:1]), dict(table=wide),
               dict(table=b.table.cpu()), dict(vp=b.vp.cpu()), dict(out=want.float()),
               dict(out=want[:5]), dict(out=want.transpose(0, 1).contiguous().transpose(0, 1))):
        with pytest.raises(ValueError):
            call(**kw)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    out = kvq.paged_prefill_attn(b.cache, b.q, qs, 20, ls, 100, b.table, b.kc, b.kp, b.vc, b.vp,
                                 stream=st)     # its workspace and output live on that stream
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("G,n", [(4, 15), (4, 16), (4, 17), (5, 12), (5, 13), (8, 8), (8, 9), (1, 64)])
@pytest.mark.parametrize("d", [128, 256])
def test_rows_around_half_a_tile(G, n, d):
    # up to 64 rows of a sequence the weights enter as two parts, on lanes of their own
    b = Batch([700, n, 333], [n, n, 1], d=d, H=2, G=G, wide=20.0, seed=21)
    b.check(b.run())
    b.check(b.run(cap=20.0, window=150), cap=20.0, window=150)
