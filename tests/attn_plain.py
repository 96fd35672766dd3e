"""Plain float64 attention over a paged INT4 cache, straight from its bytes,
for the tests of the attention entry points with scoring options. It shares no
code with the library: rotations are dense matrices, every score is formed and
masked one by one."""

import math

import numpy as np
import torch


def rotation_matrix(d, kind, block=0, table=None):
    """R [d][d] float64 with y = R x for a row x (kinds as in kvq.h)."""
    R = np.zeros((d, d))
    if kind == 0:
        return np.eye(d)
    if kind in (1, 4):
        for b0 in range(0, d, block):
            for i in range(block):
                for j in range(block):
                    R[b0 + i, b0 + j] = (-1.0) ** bin(i & j).count("1") / math.sqrt(block)
        return R * np.asarray(table, np.float64)[None, :] if kind == 4 else R
    t = np.asarray(table, np.float64).reshape(d // 4, 2, 4)

    def mul(a, b):
        w, x, y, z = a
        p, q, r, s = b
        return np.array([w * p - x * q - y * r - z * s, w * q + x * p + y * s - z * r,
                         w * r - x * s + y * p + z * q, w * s + x * r - y * q + z * p])

    for j in range(d // 4):
        for c in range(4):
            e = np.zeros(4)
            e[c] = 1.0
            v = mul(t[j, 0], e)
            if kind in (2, 5):
                v = mul(v, t[j, 1] * np.array([1, -1, -1, -1]))
            R[4 * j:4 * j + 4, 4 * j + c] = v
    return R


def rows(codes, params, pages, d):
    """Dequantized rows [tokens][H][d] float64 of the listed pages (rotated basis)."""
    by = codes[pages].permute(0, 2, 1, 3).reshape(-1, codes.shape[1], d // 2)
    w = params.view(torch.float16).reshape(*params.shape, 2)[pages]
    w = w.permute(0, 2, 1, 3).reshape(-1, codes.shape[1], 2).double()
    x = torch.stack([by & 15, by >> 4], -1).flatten(-2).double()
    return x * w[..., :1] + w[..., 1:]


def seen_mask(L, pos, window=0, first=None, bidir=0, bad=None):
    """bool [len(pos)][L]: which positions each query sees."""
    j = torch.arange(L, device=pos.device)[None]
    p = pos[:, None]
    m = (j <= p) | (j < bidir)
    if window:
        m &= j > p - window
    if first is not None:
        m &= j >= first[:, None]
    if bad is not None:
        m &= ~bad[None]
    return m


def attention(q, k, v, pos, G, sm_scale, R, cap=0.0, slopes=None, seen=None, rope=None):
    """q [n][Hq][d] (original basis), k, v [L][H][d] (rotated) -> (out
    [n][Hq][d] in the original basis, A [n][Hq]: the 2-norm of sum_j p_j |v_j|,
    S [n][Hq]: the largest sum_i |q_i k_i| sm_scale of a seen position)."""
    n, Hq, d = q.shape
    L = k.shape[0]
    R = torch.as_tensor(R, dtype=torch.float64, device=q.device)
    x = q.double()
    if rope is not None:
        cs = rope[pos].double()[:, None]                   # [n][1][d/2][2]
        a, b = x[..., 0::2], x[..., 1::2]
        x = torch.stack([a * cs[..., 0] - b * cs[..., 1], a * cs[..., 1] + b * cs[..., 0]],
                        -1).flatten(-2)
    x = x @ R.T
    out = torch.zeros_like(x)
    A = torch.zeros((n, Hq), dtype=torch.float64, device=q.device)
    Sz = torch.zeros_like(A)
    for g in range(Hq):
        h = g // G
        z = x[:, g] @ k[:, h].T * sm_scale
        big = (x[:, g].abs() @ k[:, h].abs().T * abs(sm_scale))
        if cap:
            z = cap * torch.tanh(z / cap)
        if slopes is not None:
            z = z - slopes[g].double() * (pos[:, None] - torch.arange(L, device=q.device)).abs()
        z = torch.where(seen, z, torch.full_like(z, -math.inf))
        top = z.amax(1, keepdim=True) if L else torch.full((n, 1), -math.inf, device=q.device,
                                                           dtype=torch.float64)
        e = torch.where(seen, torch.exp(z - top), torch.zeros_like(z))
        den = e.sum(1, keepdim=True)
        p = torch.where(den > 0, e / den, torch.zeros_like(e))
        out[:, g] = (p @ v[:, h]) @ R
        A[:, g] = (p @ v[:, h].abs()).norm(dim=1)
        if L:
            Sz[:, g] = torch.where(seen, big, torch.zeros_like(big)).amax(1)
    return out, A, Sz


def half_tolerance(out, A, S, L, vmax, cap=0.0, bias=0.0):
    """2-norm bound per output row of a binary16 result whose weights and
    values were rounded to binary16 once each.

    Weights and values: relative 2^-11 each, so sum_j p_j |v_j| 2^-10 = A 2^-10
    (second-order terms and the binary32 sums: 1/64 of that). Output: 2^-11 of
    |out| <= A, plus the subnormal step 2^-25 per channel. Scores: the
    binary32 product of 2 d terms, the query's split and the offset stay below
    2^-20 S, the cap adds 2^-21 cap (its two approximate functions), the bias
    2^-22 of its size; a score off by t scales the weights by 2 t at most
    after normalisation. Weights below 2^-14 - 7 of the reference are
    subnormal: L terms of 2^-25 2^-7 of the largest |v|."""
    dz = S * 2.0 ** -20 + cap * 2.0 ** -21 + bias * 2.0 ** -22 + 2.0 ** -20
    d = out.shape[-1]
    return A * (2.0 ** -10 * (1 + 1 / 64) + 2.0 ** -11 + 2 * dz) \
        + math.sqrt(d) * 2.0 ** -25 + L * 2.0 ** -32 * vmax * math.sqrt(d)


def float_tolerance(A, S, L, cap=0.0, bias=0.0):
    """2-norm bound per output row of the binary32 decode: weights as hi + lo
    pairs (2^-22), products of 64 tokens summed with at most 8 truncations
    (2^-23 each), then one binary32 addition per 64 tokens and per split
    (at most L / 64 of both together and 64 more, 2^-24 each, doubled), the
    exponential 2^-21; scores as in half_tolerance."""
    dz = S * 2.0 ** -20 + cap * 2.0 ** -21 + bias * 2.0 ** -22 + 2.0 ** -20
    return A * ((L / 64 + 64) * 2.0 ** -23 + 2.0 ** -19 + 2 * dz) + 1e-30
