"""Measured cases of the attention operators over the rotated INT4 paged cache:
prompt attention (several query tokens per sequence), decode attention with
scored options (tanh cap, distance bias, window, document mask) and decode
attention for a batch that shares a prefix.

With ``own`` false ``run`` evaluates the operators' definitions in elementary
float32 torch operations; with ``own`` true it makes the library's calls.
Every state is a paged cache as a serving program holds it: packed codes and
(scale, minimum) words behind a shuffled block table, keys and values with
outlier channels (and, for some, a large first token), quantized row by row.
"""

import math

import torch

own = False

# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

_BASE = dict(op="prefill", S=1, q=1, q_lo=1, ctx=16, ctx_lo=16, H=8, G=4, d=128, P=16, block=64,
             cap=0.0, window=0, alibi=False, docs=False, bidir=0, prefix=0, sink=1.0)


def _case(name=None, **kw):
    c = dict(_BASE)
    c.update(kw)
    if name is not None:
        c["name"] = name
    return c


def listed():
    return [
        # checking a few guessed tokens of each running sequence in one pass: few rows, long caches
        _case("prefill_verify", op="prefill", S=8, q=5, q_lo=5, ctx=4101, ctx_lo=1000),
        # one prompt, every token new
        _case("prefill_prompt", op="prefill", S=1, q=4096, q_lo=4096, ctx=4096, ctx_lo=4096,
              sink=10.0),
        # chunks of long prompts with capped scores and a sliding window, uneven lengths
        _case("prefill_capped_window", op="prefill", S=4, q=2048, q_lo=777, ctx=16384,
              ctx_lo=9001, G=8, P=32, block=128, cap=50.0, window=4096),
        # wide heads with a distance bias, packed documents and a prefix seen from both sides
        _case("prefill_wide_bias", op="prefill", S=3, q=1500, q_lo=611, ctx=2999, ctx_lo=1801, H=4,
              d=256, block=256, alibi=True, docs=True, bidir=333),
        # a batch of prompts, the largest prompt work
        _case("prefill_batch", op="prefill", S=8, q=4096, q_lo=4096, ctx=4096, ctx_lo=4096,
              sink=10.0),
        # the smallest decode call: one short sequence, latency counts
        _case("scored_short", op="scored", S=1, ctx=301, ctx_lo=301, alibi=True),
        # a full decode batch with capped scores
        _case("scored_capped", op="scored", S=32, ctx=4097, ctx_lo=4097, cap=50.0, sink=10.0),
        # long contexts of which a layer with a sliding window reads the end
        _case("scored_window", op="scored", S=8, ctx=32768, ctx_lo=20011, G=8, P=32, block=128,
              window=4096),
        # ragged lengths, wide heads, distance bias and documents
        _case("scored_ragged_wide", op="scored", S=128, ctx=16384, ctx_lo=512, H=4, d=256,
              block=256, alibi=True, docs=True),
        # four requests behind a short common instruction
        _case("shared_short", op="shared", S=4, ctx=577, ctx_lo=515, prefix=512),
        # a batch behind one system prompt
        _case("shared_batch", op="shared", S=64, ctx=4096 + 640, ctx_lo=4096 + 33, prefix=4096),
        # many questions on one long document
        _case("shared_document", op="shared", S=96, ctx=32768 + 1024, ctx_lo=32768 + 1,
              prefix=32768, G=8, P=32, block=128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "scored", "shared"])
    d = 128 if op == "shared" or rng.random() < 0.7 else 256
    H = rng.choice([1, 2, 4, 8]) if d == 128 else rng.choice([1, 2, 4])
    G = rng.choice([1, 2, 3, 4, 5, 7, 8]) if d == 128 else rng.choice([1, 2, 3, 4])
    P = rng.choice([16, 32, 64])
    block = rng.choice([b for b in (16, 32, 64, 128, 256) if b <= d])
    c = _case(op=op, H=H, G=G, d=d, P=P, block=block, cap=rng.choice([0.0, 0.0, 30.0, 50.0]),
              alibi=rng.random() < 0.3, docs=rng.random() < 0.3, sink=rng.choice([1.0, 10.0]))
    if op == "prefill":
        c["S"] = _log(rng, 1, 8)
        c["q"] = _log(rng, 1, 2048)
        c["q_lo"] = max(1, int(c["q"] * rng.uniform(0.1, 1.0)))
        c["ctx"] = c["q"] + (0 if rng.random() < 0.4 else _log(rng, 1, 6000))
        c["ctx_lo"] = max(c["q"], int(c["ctx"] * rng.uniform(0.3, 1.0)))
        c["bidir"] = 0 if rng.random() < 0.7 else _log(rng, 1, c["ctx"])
        c["window"] = 0 if rng.random() < 0.6 else _log(rng, 1, c["ctx"])
    elif op == "scored":
        c["S"] = _log(rng, 1, 64)
        c["ctx"] = _log(rng, 1, 16384)
        c["ctx_lo"] = max(1, int(c["ctx"] * rng.uniform(0.1, 1.0)))
        c["window"] = 0 if rng.random() < 0.5 else _log(rng, 1, c["ctx"])
    else:
        c["S"] = _log(rng, 2, 96)
        c["prefix"] = _log(rng, 16, 24000)
        c["ctx_lo"] = c["prefix"] + rng.randint(1, 40)
        c["ctx"] = c["ctx_lo"] + _log(rng, 1, 1000)
        c["docs"] = False
    return c


def _spread(n, lo, hi):
    """n lengths in [lo, hi], the same for every seed; the first is hi."""
    return [hi - int((hi - lo) * ((i * 0.6180339887498949) % 1.0)) for i in range(n)]


def _lens(case):
    """(context, query tokens) of each sequence."""
    ctx = _spread(case["S"], case["ctx_lo"], case["ctx"])
    if case["op"] != "prefill":
        return ctx, [1] * case["S"]
    q = _spread(case["S"], case["q_lo"], case["q"])
    return ctx, [min(a, b) for a, b in zip(q[::-1], ctx)]


def _first(case, pos):
    """Start of the document that position `pos` belongs to (documents of 700 tokens)."""
    return pos // 700 * 700 if case["docs"] else 0


def _interval(case, L, p):
    """Positions [lo, hi) that a query at position p of L cached tokens sees."""
    hi = p + 1
    if case["bidir"]:
        hi = max(hi, min(case["bidir"], L))
    lo = _first(case, p)
    if case["window"]:
        lo = max(lo, p - case["window"] + 1)
    return max(lo, 0), max(hi, lo, 0)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _sylvester(n, dtype):
    i = torch.arange(n, device="cuda")
    x = i[:, None] & i[None, :]
    for s in (8, 4, 2, 1):
        x = x ^ (x >> s)
    return (1 - 2 * (x & 1)).to(dtype)


def _quantize(x, had):
    """Rows [..., d] -> (packed codes, parameter words) in the rotated basis."""
    b = had.shape[0]
    y = (x.reshape(*x.shape[:-1], x.shape[-1] // b, b) @ had).reshape(x.shape) / math.sqrt(b)
    mn, mx = y.amin(-1, keepdim=True), y.amax(-1, keepdim=True)
    m = (mn - mn.abs() * 2.0 ** -10).half()
    s = ((mx - m.float()) * ((1 + 2.0 ** -9) / 15)).half()
    c = ((y - m.float()) / s.float().clamp_min(1e-30)).round().clamp(0, 15).to(torch.uint8)
    codes = c[..., 0::2] | (c[..., 1::2] << 4)
    params = torch.cat([s, m], -1).view(torch.int32).squeeze(-1)
    return codes, params


def prepare(case, seed):
    S, H, G, d, P = (case[k] for k in ("S", "H", "G", "d", "P"))
    ctx, qn = _lens(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    pg = [-(-n // P) for n in ctx]
    npre = case["prefix"] // P
    width = max(pg) + 1
    total = npre + sum(n - npre for n in pg)
    NP = total + 3
    perm = torch.randperm(NP, generator=g, device="cuda", dtype=torch.int32)
    table = torch.full((S, width), -1, dtype=torch.int32, device="cuda")
    kc = torch.zeros((NP, H, P, d // 2), dtype=torch.uint8, device="cuda")
    vc = torch.zeros_like(kc)
    kp = torch.zeros((NP, H, P), dtype=torch.int32, device="cuda")
    vp = torch.zeros_like(kp)
    had = _sylvester(case["block"], torch.float32)
    if d == 256:  # per-channel scales, log-uniform
        mult = torch.exp(torch.empty((H, d), device="cuda").uniform_(math.log(0.1), math.log(20.0),
                                                                      generator=g))
    else:         # a few outlier channels per head
        mult = torch.ones((H, d), device="cuda")
        pick = torch.rand((H, d), generator=g, device="cuda").topk(3, dim=1).indices
        mult.scatter_(1, pick, torch.empty((H, 3), device="cuda").uniform_(10.0, 30.0, generator=g))

    def fill(pages, first):
        n = pages.numel() * P
        for codes, params in ((kc, kp), (vc, vp)):
            x = torch.randn((n, H, d), generator=g, device="cuda") * mult
            if first:
                x[0] *= case["sink"]
            c, w = _quantize(x.half().float(), had)
            codes[pages] = c.reshape(-1, P, H, d // 2).transpose(1, 2)
            params[pages] = w.reshape(-1, P, H).transpose(1, 2)

    off = npre
    if npre:
        fill(perm[:npre].long(), True)
        table[:, :npre] = perm[:npre]
    for s in range(S):
        n = pg[s] - npre
        if n > 0:
            table[s, npre:pg[s]] = perm[off:off + n]
            fill(perm[off:off + n].long(), npre == 0)
            off += n
    if case["prefix"] % P:  # the page that holds the prefix's end is each sequence's own copy
        shared = table[:, npre].long()
        r = case["prefix"] % P
        for pool in (kc, kp, vc, vp):
            pool[shared, :, :r] = pool[shared[0], :, :r].clone()

    T = sum(qn)
    q_start = [0]
    for n in qn:
        q_start.append(q_start[-1] + n)
    pos = [L - n + i for L, n in zip(ctx, qn) for i in range(n)]
    st = dict(case=case, T=T, had=had, table=table, kc=kc, kp=kp, vc=vc, vp=vp, NP=NP,
              max_q=max(qn), max_ctx=max(ctx), sm_scale=1.0 / math.sqrt(d))
    as_i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    st["q"] = torch.randn((T, H * G, d), generator=g, device="cuda").half()
    st["q_start"], st["lens"] = as_i32(q_start), as_i32(ctx)
    st["tok_seq"] = as_i32([s for s, n in enumerate(qn) for _ in range(n)])
    st["tok_idx"] = as_i32([i for n in qn for i in range(n)])
    st["pos"] = as_i32(pos)
    st["first"] = as_i32([_first(case, p) for p in pos]) if case["docs"] else None
    # one slope per query head, a geometric sequence from 1/2 to 1/256
    st["slopes"] = torch.tensor([2.0 ** (-1 - 7 * i / max(1, H * G - 1)) for i in range(H * G)],
                                device="cuda") if case["alibi"] else None
    st["bidir"] = torch.full((S,), case["bidir"], dtype=torch.int32, device="cuda") \
        .minimum(st["lens"]) if case["bidir"] else None
    return st


# ---------------------------------------------------------------------------
# the operators
# ---------------------------------------------------------------------------

def _dense(codes, params, table, d):
    """Cached rows of every sequence, [S][tokens][H][d] float32, rotated basis."""
    pages = table.clamp_min(0).long()
    c = codes[pages]                                           # [S][pages][H][P][d/2]
    c = torch.stack([c & 15, c >> 4], -1).flatten(-2)          # [S][pages][H][P][d]
    w = params[pages].view(torch.float16).reshape(*c.shape[:-1], 2).float()
    x = c.float().mul_(w[..., :1]).add_(w[..., 1:])
    return x.transpose(2, 3).flatten(1, 2)


def _rotate(x, had):
    b = had.shape[0]
    return (x.reshape(*x.shape[:-1], x.shape[-1] // b, b) @ had).reshape(x.shape) / math.sqrt(b)


def _plain(st):
    c = st["case"]
    S, H, G, d = c["S"], c["H"], c["G"], c["d"]
    k = _dense(st["kc"], st["kp"], st["table"], d)
    v = _dense(st["vc"], st["vp"], st["table"], d)
    n = st["max_q"]
    at = (st["q_start"][:-1, None] + torch.arange(n, device="cuda")).clamp_max(st["T"] - 1).long()
    q = _rotate(st["q"].float(), st["had"])[at].reshape(S, n, H, G, d)      # [S][n][H][G][d]
    pos = st["pos"][at]                                                     # [S][n]
    z = torch.matmul(q.permute(0, 2, 3, 1, 4).reshape(S, H, G * n, d), k.permute(0, 2, 3, 1))
    z = z.reshape(S, H, G, n, -1).mul_(st["sm_scale"])
    if c["cap"]:
        z.div_(c["cap"]).tanh_().mul_(c["cap"])
    j = torch.arange(z.shape[-1], device="cuda", dtype=torch.int32)
    if st["slopes"] is not None:
        dist = (pos[:, :, None] - j).abs_().float()
        z.addcmul_(-st["slopes"].reshape(1, H, G, 1, 1), dist[:, None, None])
    hi = pos + 1
    if st["bidir"] is not None:
        hi = hi.maximum(st["bidir"][:, None])
    seen = j < hi[:, :, None]
    if c["window"]:
        seen = seen & (j > pos[:, :, None] - c["window"])
    if st["first"] is not None:
        seen = seen & (j >= st["first"][at][:, :, None])
    z.masked_fill_(~seen[:, None, None], -math.inf)
    top = z.amax(-1, keepdim=True).clamp_min(-1e30)
    p = z.sub_(top).exp_()
    den = p.sum(-1, keepdim=True).clamp_min(1e-30)
    o = torch.matmul(p.reshape(S, H, G * n, -1), v.transpose(1, 2)).reshape(S, H, G, n, d) / den
    o = _rotate(o, st["had"]).permute(0, 3, 1, 2, 4).reshape(S, n, H * G, d)
    o = o[st["tok_seq"].long(), st["tok_idx"].long()]
    return o if c["op"] == "scored" else o.half()


def _handle(st):
    """The cache's descriptor, the scoring options and the buffers that a serving program keeps."""
    if "cache" not in st:
        from bit_rotated_kv_block_b200 import kvq
        c = st["case"]
        st["kvq"] = kvq
        st["cache"] = kvq.Cache(c["d"], c["H"], c["P"], st["NP"], kvq.ROT_HADAMARD, c["block"])
        st["score"] = kvq.Score(softcap=c["cap"], window=c["window"], alibi=st["slopes"],
                                first_pos=st["first"], prefix_lens=st["bidir"])
        Hq = c["H"] * c["G"]
        if c["op"] == "prefill":
            need = kvq.prefill_workspace_bytes(st["cache"], c["S"], Hq, st["T"], st["max_q"],
                                               st["max_ctx"])
        elif c["op"] == "scored":
            need = kvq.decode_workspace_bytes(st["cache"], c["S"], Hq, st["max_ctx"])
        else:
            need = kvq.shared_prefix_workspace_bytes(st["cache"], c["S"], Hq, c["prefix"],
                                                     st["max_ctx"])
        st["ws"] = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
        st["out"] = torch.empty(st["q"].shape, device="cuda",
                                dtype=torch.float32 if c["op"] == "scored" else torch.float16)
    return st["kvq"], st["cache"]


def run(st):
    if not own:
        return _plain(st)
    kvq, cache = _handle(st)
    op = st["case"]["op"]
    pools = (st["kc"], st["kp"], st["vc"], st["vp"])
    if op == "prefill":
        return kvq.paged_prefill_attn(cache, st["q"], st["q_start"], st["max_q"], st["lens"],
                                      st["max_ctx"], st["table"], *pools, out=st["out"],
                                      workspace=st["ws"], sm_scale=st["sm_scale"],
                                      score=st["score"])
    if op == "scored":
        return kvq.paged_decode_attn_scored(cache, st["q"], st["lens"], st["max_ctx"],
                                            st["table"], *pools, score=st["score"], out=st["out"],
                                            workspace=st["ws"], sm_scale=st["sm_scale"])
    return kvq.shared_prefix_decode_attn(cache, st["q"], st["case"]["prefix"], st["lens"],
                                         st["max_ctx"], st["table"], *pools, score=st["score"],
                                         out=st["out"], workspace=st["ws"],
                                         sm_scale=st["sm_scale"])


# ---------------------------------------------------------------------------
# work and exact values
# ---------------------------------------------------------------------------

def work(case):
    """Bytes: every cached row that some query sees (codes and parameters of K
    and V) once, a shared prefix once for the batch, queries and outputs once;
    operations: two products per seen (query head, position) pair."""
    H, G, d = case["H"], case["G"], case["d"]
    ctx, qn = _lens(case)
    row = 2 * (d // 2 + 4) * H
    kv = pairs = T = 0
    for s, (L, n) in enumerate(zip(ctx, qn)):
        lo_all, hi_all = L, 0
        for p in range(L - n, L):
            lo, hi = _interval(case, L, p)
            pairs += hi - lo
            if hi > lo:
                lo_all, hi_all = min(lo_all, lo), max(hi_all, hi)
        if case["op"] == "shared":
            lo_all = max(lo_all, case["prefix"])
        kv += max(0, hi_all - lo_all)
        T += n
    if case["op"] == "shared":
        kv += case["prefix"]
    out = 4 if case["op"] == "scored" else 2
    return {"bytes": float(kv * row + T * H * G * d * (2 + out)),
            "flops": float(4 * pairs * H * G * d)}


def exact(case, seed):
    """The definition in float64, one sequence and KV head at a time, straight
    from the packed bytes."""
    st = prepare(case, seed)
    H, G, d, b, P = case["H"], case["G"], case["d"], case["block"], case["P"]
    R = _sylvester(b, torch.float64) / math.sqrt(b)
    full = torch.zeros((d, d), dtype=torch.float64, device="cuda")
    for i in range(0, d, b):
        full[i:i + b, i:i + b] = R
    ctx, qn = _lens(case)
    out = torch.zeros((st["T"], H * G, d), dtype=torch.float64, device="cuda")
    t0 = 0
    for s, (L, n) in enumerate(zip(ctx, qn)):
        pages = st["table"][s, :-(-L // P)].long()
        sees = [_interval(case, L, p) for p in range(L - n, L)]
        lo = torch.tensor([a for a, _ in sees], device="cuda")[:, None]
        hi = torch.tensor([a for _, a in sees], device="cuda")[:, None]
        j = torch.arange(L, device="cuda")[None]
        seen = (j >= lo) & (j < hi)
        dist = (torch.arange(L - n, L, device="cuda")[:, None] - j).abs().double()
        for h in range(H):
            kv = []
            for codes, params in ((st["kc"], st["kp"]), (st["vc"], st["vp"])):
                by = codes[pages, h].reshape(-1, d // 2)[:L]
                x = torch.empty((L, d), dtype=torch.float64, device="cuda")
                x[:, 0::2] = (by & 15).double()
                x[:, 1::2] = (by >> 4).double()
                w = params[pages, h].reshape(-1, 1)[:L].view(torch.float16).double()
                kv.append(x * w[:, :1] + w[:, 1:])
            for g in range(h * G, (h + 1) * G):
                q = st["q"][t0:t0 + n, g].double() @ full
                z = (q @ kv[0].T) * float(st["sm_scale"])
                if case["cap"]:
                    z = case["cap"] * torch.tanh(z / case["cap"])
                if case["alibi"]:
                    z = z - st["slopes"][g].double() * dist
                z = torch.where(seen, z, torch.full_like(z, -math.inf))
                top = z.amax(1, keepdim=True)
                e = torch.where(seen, torch.exp(z - top), torch.zeros_like(z))
                den = e.sum(1, keepdim=True)
                o = torch.where(den > 0, (e @ kv[1]) / den, torch.zeros((), dtype=torch.float64,
                                                                       device="cuda"))
                out[t0:t0 + n, g] = o @ full.T
        t0 += n
    return out
