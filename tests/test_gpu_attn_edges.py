"""The prompt, scored and shared-prefix attention entry points where their
kernels' loops, number ranges and roundings are at their ends, against plain
float64 attention over the same pages."""

import pytest
import torch

from bit_rotated_kv_block_b200 import kvq
from test_gpu_prefill import Batch

pytestmark = pytest.mark.gpu


def refill(b, k, v):
    """Writes other keys and values [tokens of all sequences][H][d] into the batch's cache."""
    ts = torch.cat([torch.full((n,), s, dtype=torch.int32) for s, n in enumerate(b.lens)])
    tp = torch.cat([torch.arange(n, dtype=torch.int32) for n in b.lens])
    kvq.quantize_append(b.cache, k.half().cuda().contiguous(), v.half().cuda().contiguous(),
                        ts.cuda(), tp.cuda(), b.table, b.kc, b.kp, b.vc, b.vp)


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
