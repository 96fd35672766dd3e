"""Host-side refusals of the attention entry points with options, through the
binding (no GPU)."""

import pytest
import torch

from bit_rotated_kv_block_b200 import kvq


def test_a_softcap_that_float32_cannot_hold_is_refused():
    for cap in (1e-50, -1e-60):
        with pytest.raises(ValueError):
            kvq.Score(softcap=cap)       # it would act as no cap
    assert kvq.Score(softcap=0.0).desc.softcap == 0.0
    assert kvq.Score(softcap=50.0).desc.softcap == 50.0


class Pools:
    """A small cache's geometry on the CPU, with pools that fit it."""

    def __init__(self):
        self.cache = kvq.Cache(128, 2, 16, 6, kvq.ROT_HADAMARD, 64, device="cpu")
        self.kc, self.kp = self.cache.new_pools(device="cpu", fill=0)
        self.vc, self.vp = self.cache.new_pools(device="cpu", fill=0)

    def check(self, workspace=None, err=None, **kw):
        p = dict(kc=self.kc, kp=self.kp, vc=self.vc, vp=self.vp)
        p.update(kw)
        kvq._memory(self.cache, p["kc"], p["kp"], p["vc"], p["vp"], workspace, err)


def test_pools_of_the_cache_are_taken():
    p = Pools()
    p.check()
    p.check(workspace=torch.empty(64, dtype=torch.uint8), err=torch.zeros(1, dtype=torch.int32))
    layers = torch.zeros((3, 6, 2, 16, 64), dtype=torch.uint8)
    p.check(kc=layers[1], vc=layers[2])                          # a layer of a larger tensor
    p.check(kc=torch.zeros((9, 2, 16, 64), dtype=torch.uint8))   # more pages than the cache names
    p.check(kp=p.kp.view(6, 32), vc=p.vc.view(-1))               # the same bytes, fewer dimensions


@pytest.mark.parametrize("name", ["kc", "kp", "vc", "vp"])
def test_pools_that_would_be_misread_or_read_past_their_end_are_refused(name):
    p = Pools()
    t = getattr(p, name)
    layers = torch.zeros((t.shape[0], 3, *t.shape[1:]), dtype=t.dtype)
    for bad in (t[:5], t[:, :1].contiguous(), layers[:, 1], t.transpose(1, 2),
                t.transpose(1, 2).contiguous(), t.float(), t.view(-1)[:-1],
                torch.zeros((6, 4, *t.shape[2:]), dtype=t.dtype),
                t.view(torch.int16) if name in ("kp", "vp") else t.view(torch.int32)):
        with pytest.raises(ValueError):
            p.check(**{name: bad})


def test_workspace_and_error_words_that_do_not_fit_are_refused():
    p = Pools()
    for ws in (torch.empty((64, 2), dtype=torch.uint8)[:, 0], torch.empty((4, 8)).t()):
        with pytest.raises(ValueError):
            p.check(workspace=ws)
    for err in (torch.zeros(1, dtype=torch.uint8), torch.zeros(1), torch.zeros(0, dtype=torch.int32),
                torch.zeros(1, dtype=torch.int64)):
        with pytest.raises(ValueError):
            p.check(err=err)


@pytest.mark.parametrize("value", [2 ** 31, 2 ** 32, 2 ** 32 + 64, -2 ** 31 - 1])
def test_sizes_beyond_32_bits_are_refused(monkeypatch, value):
    # (ctypes would cut them to their low 32 bits)
    p = Pools()
    monkeypatch.setattr(kvq, "_fit", lambda cache, q, seqs, *a: (q.shape, 0))
    monkeypatch.setattr(kvq, "_ints", lambda *a: None)
    monkeypatch.setattr(kvq, "_stream", lambda *a: None)

    class Library:
        def __getattr__(self, name):
            return lambda *a: 0
    monkeypatch.setattr(kvq, "lib", lambda: Library())
    q = torch.zeros((2, 4, 128), dtype=torch.float16)
    lens, table = torch.zeros(2, dtype=torch.int32), torch.zeros((2, 4), dtype=torch.int32)
    qs, pools = torch.zeros(3, dtype=torch.int32), (p.kc, p.kp, p.vc, p.vp)
    ws = torch.zeros(64, dtype=torch.uint8)
    good = lambda v=16: (
        lambda: kvq.paged_prefill_attn(p.cache, q, qs, v, lens, 64, table, *pools, workspace=ws),
        lambda: kvq.paged_prefill_attn(p.cache, q, qs, 4, lens, v, table, *pools, workspace=ws),
        lambda: kvq.paged_decode_attn_scored(p.cache, q, lens, v, table, *pools, workspace=ws),
        lambda: kvq.shared_prefix_decode_attn(p.cache, q, v, lens, 64, table, *pools, workspace=ws),
        lambda: kvq.shared_prefix_decode_attn(p.cache, q, 16, lens, v, table, *pools, workspace=ws),
        lambda: kvq.prefill_workspace_bytes(p.cache, 2, 4, 2, v, 64),
        lambda: kvq.prefill_workspace_bytes(p.cache, 2, 4, 2, 4, v),
        lambda: kvq.shared_prefix_workspace_bytes(p.cache, 2, 4, v, 64),
        lambda: kvq.shared_prefix_workspace_bytes(p.cache, 2, 4, 16, v))
    for call in good():
        call()
    for call in good(value):
        with pytest.raises(ValueError):
            call()
