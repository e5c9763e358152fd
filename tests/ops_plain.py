"""Plain 64-bit forms of the operators of include/mk_ops.h, on the CPU, one
sequence and one token at a time; none of the package's code."""
import math

import torch

F64 = torch.float64


def rotate(x, pos, base):
    """x [heads][d]: pairs (2i, 2i + 1) turned by pos * base^(-2i / d)."""
    d = x.shape[-1]
    a = torch.tensor([pos * base ** (-2.0 * i / d) for i in range(d // 2)], dtype=F64)
    x = x.to(F64)
    e, o = x[..., 0::2], x[..., 1::2]
    return torch.stack((e * a.cos() - o * a.sin(), e * a.sin() + o * a.cos()), -1).flatten(-2)


def bf16_bound(ref):
    """Half a bf16 step at a value of this size (2^-8 of it; 2^-134 among the subnormals)."""
    return ref.abs() * 2.0 ** -8 + 2.0 ** -134


def gather_slots(pool, table, n):
    """pool [pages][n_kv][P][d] -> [n][n_kv][d]: the first n slots of a table's sequence."""
    P = pool.shape[2]
    return torch.stack([pool[table[s // P], :, s % P] for s in range(n)]) if n else pool[:0, :, 0]


def sees(i, n, ctx, window, mask_row, positions):
    """Which of the slots 0 .. ctx + n - 1 the i-th new token sees."""
    pos = positions if positions is not None else [ctx + j for j in range(n)]
    see = [True] * ctx + [bool((mask_row >> j) & 1) if mask_row is not None else j <= i for j in range(n)]
    if window:
        at = list(range(ctx)) + list(pos)
        see = [s and pos[i] - a < window for s, a in zip(see, at)]
    return torch.tensor(see)


def attention(q, k, v, see, scale):
    """q [n_q][d], k and v [slots][n_kv][d], see [slots] -> out [n_q][d], lse [n_q], and what the
    error bound needs: sum p |v| / sum p, and the largest |scale| sum |q k|.  Only what is seen is touched."""
    n_q, d = q.shape
    n_kv = k.shape[1]
    k, v = k[see].to(F64), v[see].to(F64)
    G = n_q // n_kv
    if k.shape[0] == 0:
        z = torch.zeros(n_q, d, dtype=F64)
        return z, torch.full((n_q,), -math.inf, dtype=F64), z, torch.zeros(n_q, dtype=F64)
    q = q.to(F64).view(n_kv, G, d)
    s = torch.einsum("hgd,shd->hgs", q, k) * scale
    size = torch.einsum("hgd,shd->hgs", q.abs(), k.abs()).amax(-1) * scale
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - lse[..., None])
    out = torch.einsum("hgs,shd->hgd", p, v).reshape(n_q, d)
    spread = torch.einsum("hgs,shd->hgd", p, v.abs()).reshape(n_q, d)
    return out, lse.reshape(n_q), spread, size.reshape(n_q)


def select(logits, scores, n_out, finished=None, eos=-1):
    """logits [R][W][V] -> every candidate's score, sorted by (score descending, index): (scores, beams, tokens)."""
    R, W, V = logits.shape
    x = logits.to(F64)
    cand = scores.to(F64)[..., None] + (x - torch.logsumexp(x, -1, keepdim=True))
    if finished is not None:
        only = torch.full_like(cand, -math.inf)
        only[..., eos] = scores.to(F64)
        cand = torch.where(finished.bool()[..., None], only, cand)
    cand = torch.where(cand.isnan(), -math.inf, cand).view(R, W * V)
    best, at = torch.sort(cand, dim=-1, descending=True, stable=True)
    return best[:, :n_out + 1], at[:, :n_out] // V, at[:, :n_out] % V


def commit(pool, table, ctx, path):
    """pool [L][pages][n_kv][P][d], in place."""
    P = pool.shape[3]
    old = pool.clone()
    for k, s in enumerate(path):
        a, b = ctx + s, ctx + k
        pool[:, table[b // P], :, b % P] = old[:, table[a // P], :, a % P]


def reorder(pools, tables, lens, parents, P):
    """tables [R][W][pages] -> new tables; the pools' open pages copied in place."""
    new = tables.clone()
    olds = [p.clone() for p in pools]
    for r, (n, par) in enumerate(zip(lens, parents)):
        W, full, used = len(par), n // P, n % P
        spare = [int(tables[r, w, full]) for w in range(W) if w not in par] if used else []
        had = set()
        for i, p in enumerate(par):
            new[r, i, :full] = tables[r, p, :full]
            if not used:
                continue
            src = int(tables[r, p, full])
            new[r, i, full] = src
            if p in had:
                dst = spare.pop(0)
                new[r, i, full] = dst
                for pool, old in zip(pools, olds):
                    pool[:, dst, :, :used] = old[:, src, :, :used]
            had.add(p)
    return new
