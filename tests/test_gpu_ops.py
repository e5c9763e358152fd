"""The operators beside the decode step (include/mk_ops.h) against plain 64-bit
forms (ops_plain.py), over types, head layouts, page sizes, lengths, strides
and masks; and runs of them together."""
import math

import pytest
import torch

import moe_decode_megakernel_gb300 as mk
import ops_plain as plain

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF = torch.bfloat16
BASE = 500000.0


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def new_status():
    return torch.zeros(8, dtype=torch.int32, device=DEV)


class Paged:
    """Pools (random, so that every unused row holds something) and shuffled tables for `slots` slots per row."""

    def __init__(self, g, slots, n_kv, P, d, layers=1, spare=2, extra_cols=1, fill=None):
        need = [-(-s // P) for s in slots]
        total = sum(need) + spare
        shape = (layers, total, n_kv, P, d)
        self.k, self.v = (torch.randn(shape, generator=g, device=DEV, dtype=BF) if fill is None else
                          torch.full(shape, fill, device=DEV, dtype=BF) for _ in range(2))
        ids = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
        self.tables = torch.full((len(slots), max(need, default=0) + extra_cols), -1, dtype=torch.int32, device=DEV)
        at = 0
        for r, n in enumerate(need):
            self.tables[r, :n] = ids[at:at + n]
            at += n
        self.cache = mk.KvCache(self.k, self.v, BASE)


def starts(counts, first=0):
    cu = [first]
    for n in counts:
        cu.append(cu[-1] + n)
    return cu


# -------------------------------------------------------------------- append

APPEND = [
    # n_q, n_kv, d, P, contexts, new tokens, positions, fused
    (4, 2, 64, 16, [0], [1], None, False),
    (4, 2, 64, 16, [15, 16, 0, 33], [1, 17, 0, 5], None, True),
    (32, 4, 128, 64, [8191, 100], [8, 3], "tree", True),
    (16, 2, 64, 64, [63, 64, 65], [130, 1, 64], "far", False),
    (5, 5, 128, 256, [250], [9], "far", True),
    (24, 4, 128, 32, [7], [700], None, True),
    (0, 1, 64, 128, [127, 0], [3, 300], None, False),
]


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("n_q,n_kv,d,P,ctx,new,where,fused", APPEND)
def test_append(dtype, n_q, n_kv, d, P, ctx, new, where, fused):
    g = gen(1 + sum(new))
    pg = Paged(g, [a + b for a, b in zip(ctx, new)], n_kv, P, d, layers=2)
    T, behind = sum(new), 3  # rows behind the last sequence
    heads = n_q + 2 * n_kv
    if fused:  # one projection's rows, with a gap between them
        rows = torch.randn(T + behind, heads * d + 16, generator=g, device=DEV).to(dtype)[:, :heads * d]
        x = rows.unflatten(1, (heads, d))
        q, k, v = x[:, :n_q], x[:, n_q:n_q + n_kv], x[:, n_q + n_kv:]
    else:
        q, k, v = (torch.randn(T + behind, h, d, generator=g, device=DEV).to(dtype) for h in (n_q, n_kv, n_kv))
    slot = [a + i for a, n in zip(ctx, new) for i in range(n)]
    pos = slot
    if where == "tree":
        pos = [s - i % 3 for i, s in enumerate(slot)]
    elif where == "far":
        pos = [(1 << 20) * (1 + i % 7) + 12345 * i for i in range(T)]
    positions = ints(pos + [0] * behind) if where else None
    q_out = torch.full((T + behind, n_q, d), 7.0, dtype=BF, device=DEV) if n_q else None
    want = {0: (pg.k.cpu(), pg.v.cpu())}
    st = new_status()
    mk.kv_append(pg.cache, 1, k, v, ints(starts(new)), ints(ctx), pg.tables, q=q if n_q else None, q_out=q_out,
                 positions=positions, status=st)
    mk.check_status(st)
    got_k, got_v = pg.k.cpu(), pg.v.cpu()
    old_k, old_v = want[0]
    kc, vc, tables = k.cpu(), v.cpu(), pg.tables.cpu()
    # rounding to bf16; the angle's error (pi 2^-24 and the sine's 2 ulp) and three fp32 roundings of e, o below 2^-20
    t = 0
    for b, n in enumerate(new):
        for i in range(n):
            s = ctx[b] + i
            page, row = tables[b, s // P], s % P
            ref = plain.rotate(kc[t], pos[t], BASE)
            mag = kc[t].to(torch.float64).abs().view(n_kv, d // 2, 2).sum(-1, keepdim=True).expand(-1, -1, 2).reshape(n_kv, d)
            err = (got_k[1, page, :, row].double() - ref).abs()
            assert (err <= plain.bf16_bound(ref) + mag * 2.0 ** -20).all()
            assert torch.equal(got_v[1, page, :, row], vc[t].to(BF))
            old_k[1, page, :, row] = got_k[1, page, :, row]
            old_v[1, page, :, row] = got_v[1, page, :, row]
            if n_q:
                qt = q[t].cpu()
                ref = plain.rotate(qt, pos[t], BASE)
                mag = qt.double().abs().view(n_q, d // 2, 2).sum(-1, keepdim=True).expand(-1, -1, 2).reshape(n_q, d)
                assert ((q_out[t].cpu().double() - ref).abs() <= plain.bf16_bound(ref) + mag * 2.0 ** -20).all()
            t += 1
    # nothing else was written: other slots, the other layer, the rows behind the last sequence
    assert torch.equal(got_k, old_k) and torch.equal(got_v, old_v)
    if n_q:
        assert (q_out[T:] == 7).all()


def test_append_in_place_and_offset_sequences():
    """q rotated onto itself inside a fused projection; sequences that start behind row 0."""
    g = gen(5)
    n_q, n_kv, d, P = 4, 2, 64, 16
    pg = Paged(g, [40, 40], n_kv, P, d)
    rows = torch.randn(12, (n_q + 2 * n_kv) * d, generator=g, device=DEV).to(BF)
    x = rows.unflatten(1, (-1, d))
    before = x.clone()
    args = (x[:, n_q:n_q + n_kv], x[:, n_q + n_kv:], ints([2, 5, 9]), ints([30, 7]), pg.tables)
    apart = torch.full((12, n_q, d), 3.0, dtype=BF, device=DEV)
    mk.kv_append(pg.cache, 0, *args, q=x[:, :n_q], q_out=apart)
    mk.kv_append(pg.cache, 0, *args, q=x[:, :n_q], q_out=x[:, :n_q])
    assert torch.equal(x[2:9, :n_q], apart[2:9])
    for r in (slice(0, 2), slice(9, 12)):
        assert torch.equal(x[r], before[r]) and (apart[r] == 3).all()
    assert torch.equal(x[:, n_q:], before[:, n_q:])


def test_append_negative_positions_turn_back():
    g = gen(6)
    pg = Paged(g, [4], 1, 16, 64)
    k = torch.randn(4, 1, 64, generator=g, device=DEV)
    mk.kv_append(pg.cache, 0, k, k, ints([0, 4]), ints([0]), pg.tables, positions=ints([-1, -77777, 0, -(1 << 31)]))
    got = pg.k[0, pg.tables[0, 0].item(), 0, :4].cpu().double()
    for t, p in enumerate([-1, -77777, 0, -(1 << 31)]):
        ref = plain.rotate(k[t].cpu(), p, BASE)[0]
        # at 2^31 the frequency's rounding (2^-53 of up to 0.16 turns) times the position is 2^-24 of a turn
        assert ((got[t] - ref).abs() <= plain.bf16_bound(ref) + 2.0 ** -18 * k[t].abs().max().item() * 4).all()


def test_append_leaves_out_what_is_out_of_range():
    g = gen(7)
    n_kv, d, P = 2, 64, 16
    pg = Paged(g, [48, 48, 48], n_kv, P, d, extra_cols=0)
    k = torch.randn(9, n_kv, d, generator=g, device=DEV)
    q, q_out = torch.randn(9, 4, d, generator=g, device=DEV), torch.full((9, 4, d), 5.0, dtype=BF, device=DEV)
    bad = pg.tables.clone()
    bad[0, 1], bad[1, 0] = pg.k.shape[1], -3
    before = pg.k.clone()
    st = new_status()
    # row 0's second page is beyond the pool, row 1 begins in a negative page and ends in a good one, row 2 overflows its table
    mk.kv_append(pg.cache, 0, k, k, ints([0, 3, 6, 9]), ints([15, 14, 46]), bad, q=q, q_out=q_out, status=st)
    with pytest.raises(mk.MkError) as e:
        mk.check_status(st)
    assert e.value.code == mk.MK_ERR_DEVICE and "kv_append" in str(e.value)
    t = pg.tables.tolist()
    changed = (pg.k != before).any(-1).any(2)[0]  # [page][row]
    want = torch.zeros_like(changed)
    want[t[0][0], 15] = True  # the first token of row 0
    want[t[1][1], 0] = True  # the third of row 1
    assert torch.equal(changed, want)
    assert (q_out[:6] != 5).any(-1).all() and (q_out[6:] == 5).all()
    # rows that the arrays do not have, a descending start
    st.zero_()
    before = pg.k.clone()
    mk.kv_append(pg.cache, 0, k, k, ints([0, 10, 10, 4]), ints([0, 0, 0]), pg.tables, status=st)
    with pytest.raises(mk.MkError):
        mk.check_status(st)
    assert torch.equal(pg.k, before)


# ----------------------------------------------------------------- attention

def mask_words(rows, words):
    low = (1 << 64) - 1
    return torch.tensor([[(w := (m >> (64 * j)) & low) - ((1 << 64) if w >> 63 else 0) for j in range(words)] for m in rows],
                        dtype=torch.int64, device=DEV)


def tree_of(g, n, kind):
    """Bit rows and depths of n drafted tokens."""
    import random
    r = random.Random(int(torch.randint(1 << 30, (1,), generator=g, device=DEV)))
    if kind == "random":  # any bits, rows with none among them; depths as they come
        rows = [0 if r.random() < 0.2 else r.getrandbits(n) for _ in range(n)]
        return rows, [r.randrange(0, n) for _ in range(n)]
    rows, depth = [], []
    for i in range(n):
        p = r.randint(max(-1, i - 4), i - 1) if i else -1
        rows.append((rows[p] if p >= 0 else 0) | (1 << i))
        depth.append(depth[p] + 1 if p >= 0 else 0)
    return rows, depth


def check_attn(pg, q, out, lse, tables, ctx, new, rows, positions, window, scale, n_kv, first=0, layer=0):
    """Every token against the plain form.  Bounds: the rounding of the probabilities (2^-8 of sum p |v| / sum p) and of the
    output (2^-8 of it); a score's error, d products summed in fp32 (d 2^-23 of sum |q k|, generous for any order), shifts
    exp by as much, and so do the exponential and the subtraction of the maximum (2^-20); sums over the slots in fp32."""
    d = q.shape[-1]
    kc, vc, qc, oc = pg.k[layer].cpu(), pg.v[layer].cpu(), q.cpu(), out.cpu().double()
    lc = lse.cpu().double() if lse is not None else None
    tables = tables.cpu().tolist()
    t = first
    for b, n in enumerate(new):
        if n == 0:
            continue
        k, v = plain.gather_slots(kc, tables[b], ctx[b] + n), plain.gather_slots(vc, tables[b], ctx[b] + n)
        for i in range(n):
            see = plain.sees(i, n, ctx[b], window, rows[b][i] if rows else None, positions[b] if positions else None)
            ref, ref_lse, spread, size = plain.attention(qc[t], k, v, see, scale)
            ds = (size * d * 2.0 ** -23 + 2.0 ** -20).unsqueeze(-1)
            tol = plain.bf16_bound(ref) + spread * (2.0 ** -8 + 2 * ds + see.numel() * 2.0 ** -24) * 1.01
            err = (oc[t] - ref).abs()
            assert (err <= tol).all(), (b, i, float((err - tol).max()), float(err.max()))
            if lc is not None:
                empty = ref_lse == -math.inf
                assert (lc[t][empty] == -math.inf).all() and (oc[t][empty] == 0).all()
                le = (lc[t] - ref_lse)[~empty].abs()
                assert (le <= ds[~empty, 0] + see.numel() * 2.0 ** -24 + ref_lse[~empty].abs() * 2.0 ** -22).all(), (b, i, float(le.max()))
            t += 1


ATTN = [
    # n_q, n_kv, d, P, contexts, new tokens, mask, window
    (4, 2, 64, 16, [0], [1], None, 0),
    (4, 2, 64, 16, [0], [1], "tree", 0),
    (8, 1, 128, 64, [130], [1], None, 0),
    (32, 4, 128, 64, [1000], [8], "tree", 0),
    (16, 2, 64, 64, [64, 0, 127, 128, 129, 500], [5, 3, 0, 1, 7, 4], "tree", 0),
    (16, 2, 64, 32, [64, 0, 127, 128, 129, 500], [5, 3, 0, 1, 7, 4], None, 0),
    (24, 4, 128, 16, [77, 300], [13, 45], "tree", 0),
    (24, 4, 128, 128, [77, 300], [13, 45], None, 0),
    (32, 4, 128, 64, [200, 10], [64, 33], "tree", 0),
    (16, 2, 64, 64, [333], [130], "tree", 0),
    (16, 2, 64, 64, [190], [130], "random", 0),
    (4, 4, 128, 256, [300, 260], [200, 3], None, 0),
    (40, 1, 128, 64, [70], [9], "tree", 0),
    (3, 1, 64, 16, [0, 1, 2], [70, 1, 129], "random", 0),
    # windows: inside the cache, at a tile's border, narrower than the tree, one slot
    (16, 2, 64, 64, [700, 40, 512], [5, 5, 9], "tree", 512),
    (16, 2, 64, 64, [700, 40, 512], [5, 5, 9], None, 512),
    (32, 4, 128, 64, [900], [40], "tree", 128),
    (8, 2, 128, 16, [300, 20], [60, 60], "tree", 3),
    (8, 2, 128, 16, [300, 20], [60, 60], None, 17),
    (8, 2, 64, 32, [150], [70], "random", 20),
    (4, 2, 64, 16, [33], [5], None, 1),
    # a long run over a cache, many tiles of queries
    (16, 2, 64, 64, [130], [300], None, 0),
    (8, 1, 128, 64, [0], [520], None, 100),
]


@pytest.mark.parametrize("n_q,n_kv,d,P,ctx,new,kind,window", ATTN)
def test_attn(n_q, n_kv, d, P, ctx, new, kind, window):
    g = gen(11 + sum(new) + window)
    pg = Paged(g, [a + b for a, b in zip(ctx, new)], n_kv, P, d, layers=2)
    # whatever lies in unused rows of the pages stays out of the sums
    used = torch.zeros(pg.k.shape[1], P, dtype=torch.bool, device=DEV)
    for b, (a, n) in enumerate(zip(ctx, new)):
        s = torch.arange(a + n, device=DEV)
        used[pg.tables[b].long()[s // P], s % P] = True
    for pool in (pg.k, pg.v):
        pool.masked_fill_(~used[None, :, None, :, None], math.nan)
    first, behind = 2, 3
    T = sum(new)
    x = (2 * torch.randn(first + T + behind, n_q * d + 24, generator=g, device=DEV)).to(BF)
    q = x[:, 8:8 + n_q * d].unflatten(1, (n_q, d))  # rows with a gap between them
    out = torch.full((first + T + behind, n_q * d + 8), 5.0, dtype=BF, device=DEV)[:, :n_q * d].unflatten(1, (n_q, d))
    lse = torch.full((first + T + behind, n_q), 5.0, device=DEV)
    rows = pos = mask = positions = None
    if kind:
        trees = [tree_of(g, n, kind) for n in new]
        rows, pos = [t[0] for t in trees], [[c + e for e in t[1]] for c, t in zip(ctx, trees)]
        words = -(-max(new) // 64) + 1  # a word more than it takes, its bits set
        junk = (1 << 64) - 1 << 64 * (words - 1)
        mask = mask_words([0] * first + [m | junk for r in rows for m in r] + [0] * behind, words)
        positions = ints([0] * first + [p for r in pos for p in r] + [0] * behind)
    st = new_status()
    ws = torch.empty(mk.tree_attn_workspace_bytes(pg.cache), dtype=torch.uint8, device=DEV)
    mk.tree_attn(pg.cache, 1, q, out, ints(starts(new, first)), ints(ctx), pg.tables, ws, tree_mask=mask, positions=positions,
                 window=window, lse=lse, status=st)
    mk.check_status(st)
    check_attn(pg, q, out, lse, pg.tables, ctx, new, rows, pos, window, 1 / math.sqrt(d), n_kv, first, layer=1)
    for r in (slice(0, first), slice(first + T, None)):
        assert (out[r] == 5).all() and (lse[r] == 5).all()


def run_attn(pg, q, ctx, new, ws=None, **kw):
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=DEV)
    if ws is None:
        ws = torch.empty(mk.tree_attn_workspace_bytes(pg.cache), dtype=torch.uint8, device=DEV)
    mk.tree_attn(pg.cache, 0, q, out, ints(starts(new)), ints(ctx), pg.tables, ws, lse=lse, **kw)
    return out, lse


@pytest.mark.parametrize("d,n_q,n_kv", [(64, 16, 2), (128, 8, 2)])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
def test_attn_masked_values_stay_out(value, d, n_q, n_kv):
    """NaN and infinities in K and V of tokens that some rows see: the others' outputs do not change at all."""
    g = gen(21)
    ctx, new, P = [150, 90], [20, 70], 16
    pg = Paged(g, [a + b for a, b in zip(ctx, new)], n_kv, P, d)
    q = torch.randn(sum(new), n_q, d, generator=g, device=DEV).to(BF)
    trees = [tree_of(g, n, "tree") for n in new]
    # token 4 of the first and token 66 of the second sequence are seen by themselves and their descendants only
    mask = mask_words([m for t in trees for m in t[0]], 2)
    pos = ints([c + e for c, t in zip(ctx, trees) for e in t[1]])
    clean, clean_lse = run_attn(pg, q, ctx, new, tree_mask=mask, positions=pos)
    for b, j in ((0, 4), (1, 66)):
        s = ctx[b] + j
        page = pg.tables[b, s // P].item()
        pg.v[0, page, :, s % P, ::3] = value
        pg.k[0, page, 0, s % P, 5] = value
    out, lse = run_attn(pg, q, ctx, new, tree_mask=mask, positions=pos)
    t = 0
    for b, n in enumerate(new):
        for i in range(n):
            if (trees[b][0][i] >> (4 if b == 0 else 66)) & 1:
                assert not out[t, :, ::3].isfinite().any()  # p * inf or NaN in every head
                h = n_q // n_kv  # heads whose K was finite: the other elements too
                assert out[t, h:].reshape(-1, d)[:, 1::3].isfinite().all() and out[t, h:].reshape(-1, d)[:, 2::3].isfinite().all()
            else:
                assert torch.equal(out[t], clean[t]) and torch.equal(lse[t], clean_lse[t])
            t += 1
    assert lse.isfinite().any()


@pytest.mark.parametrize("kind", [None, "tree"])
def test_attn_values_outside_the_window_stay_out(kind):
    g = gen(22)
    ctx, new, P, W = [400], [40], 16, 100
    pg = Paged(g, [440], 2, P, 64)
    q = torch.randn(40, 8, 64, generator=g, device=DEV).to(BF)
    rows, depth = tree_of(g, 40, "tree")
    pos = [400 + e for e in depth] if kind else [400 + i for i in range(40)]
    kw = dict(window=W)
    if kind:
        kw.update(tree_mask=mask_words(rows, 1), positions=ints(pos))
    clean, clean_lse = run_attn(pg, q, ctx, new, **kw)
    s = 400 - W + 3  # seen from positions up to 402
    pg.v[0, pg.tables[0, s // P].item(), :, s % P] = math.nan
    pg.k[0, pg.tables[0, 0].item()] = math.nan  # far outside
    pg.v[0, pg.tables[0, 1].item()] = math.inf
    out, lse = run_attn(pg, q, ctx, new, **kw)
    for i in range(40):
        if pos[i] - s < W:
            assert out[i].isnan().all()
        else:
            assert torch.equal(out[i], clean[i]) and torch.equal(lse[i], clean_lse[i])


LONG = [
    # n_q, n_kv, d, P, contexts, new tokens, mask, window: many tiles and many items for every SM
    (32, 4, 128, 64, [2900 + 37 * b for b in range(12)], [8] * 12, "tree", 0),
    (32, 4, 128, 16, [1500 + 91 * b for b in range(16)], [32, 17, 16, 33] * 4, "tree", 0),
    (16, 2, 64, 64, [6000, 100, 20000, 1], [64, 1, 5, 130], "tree", 0),
    (8, 8, 64, 32, [40 * b for b in range(200)], [1 + b % 3 for b in range(200)], None, 0),
    (4, 4, 128, 128, [5] * 700, [2] * 700, "tree", 0),
    (32, 4, 128, 64, [2000], [1100], None, 0),
    (32, 4, 128, 64, [9000, 300], [700, 500], None, 4096),
    (24, 4, 128, 64, [12000, 4097] * 6, [20, 11] * 6, "tree", 4096),
    (16, 2, 64, 16, [0], [3000], None, 512),
]


@pytest.mark.parametrize("n_q,n_kv,d,P,ctx,new,kind,window", LONG)
def test_attn_many_units(n_q, n_kv, d, P, ctx, new, kind, window):
    g = gen(71 + len(ctx))
    pg = Paged(g, [a + b for a, b in zip(ctx, new)], n_kv, P, d)
    T, B = sum(new), len(new)
    q = (2 * torch.randn(T, n_q, d, generator=g, device=DEV)).to(BF)
    trees = [tree_of(g, n, "tree") for n in new] if kind else None
    kw = {}
    if kind:
        kw = dict(tree_mask=mask_words([m for t in trees for m in t[0]], -(-max(new) // 64)),
                  positions=ints([c + e for c, t in zip(ctx, trees) for e in t[1]]))
    st = new_status()
    out, lse = run_attn(pg, q, ctx, new, window=window, status=st, **kw)
    mk.check_status(st)
    again = run_attn(pg, q, ctx, new, window=window, **kw)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    scale, t = 1 / math.sqrt(d), 0
    for b in range(B):
        n, c = new[b], ctx[b]
        s = torch.arange(c + n, device=DEV)
        k, v = (x[0][pg.tables[b].long()[s // P], :, s % P].double() for x in (pg.k, pg.v))
        if kind:
            see = torch.tensor([[True] * c + [bool(m >> j & 1) for j in range(n)] for m in trees[b][0]], device=DEV)
            mine = torch.tensor([c + e for e in trees[b][1]], device=DEV)
        else:
            mine = torch.arange(c, c + n, device=DEV)
            see = s[None] <= mine[:, None]
        if window:
            see = see & (mine[:, None] - torch.cat((s[:c], mine))[None] < window)
        for h in range(n_kv):
            G = n_q // n_kv
            x = q[t:t + n, h * G:(h + 1) * G].double().transpose(0, 1)
            w = (x @ k[:, h].T * scale).masked_fill(~see[None], -math.inf)
            size = (x.abs() @ k[:, h].T.abs() * scale).amax(-1)
            want = torch.logsumexp(w, -1)
            p = torch.exp(w - want[..., None])
            ref, spread = p @ v[:, h], p @ v[:, h].abs()
            # the bounds of check_attn
            ds = size * d * 2.0 ** -23 + 2.0 ** -20
            far = (c + n) * 2.0 ** -24
            tol = plain.bf16_bound(ref) + spread * (2.0 ** -8 + 2 * ds[..., None] + far) * 1.01
            err = (out[t:t + n, h * G:(h + 1) * G].double().transpose(0, 1) - ref).abs()
            assert (err <= tol).all(), (b, h, float((err - tol).max()))
            le = (lse[t:t + n, h * G:(h + 1) * G].double().T - want).abs()
            assert (le <= ds + far + want.abs() * 2.0 ** -22).all()
        t += n


@pytest.mark.parametrize("window", [1 << 30, (1 << 31) - 1])
@pytest.mark.parametrize("kind", [None, "tree"])
def test_attn_windows_longer_than_any_cache(kind, window):
    n_q, n_kv, d, ctx, new = 8, 2, 64, [300, 0], [150, 70]
    g = gen(97)
    pg = Paged(g, [a + b for a, b in zip(ctx, new)], n_kv, 64, d)
    q = torch.randn(sum(new), n_q, d, generator=g, device=DEV).to(BF)
    kw = {}
    if kind:
        trees = [tree_of(g, n, kind) for n in new]
        kw = dict(tree_mask=mask_words([m for t in trees for m in t[0]], 3),
                  positions=ints([c + e for c, t in zip(ctx, trees) for e in t[1]]))
    st = new_status()
    got = run_attn(pg, q, ctx, new, window=window, status=st, **kw)
    want = run_attn(pg, q, ctx, new, **kw)
    mk.check_status(st)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_attn_extreme_scores():
    """Scores far apart (one slot takes all), equal ones, and the lowest: the running maximum must carry them."""
    g = gen(23)
    ctx, new, P, d, n_q, n_kv = [700], [6], 64, 128, 8, 1
    pg = Paged(g, [706], n_kv, P, d)
    q = torch.zeros(6, n_q, d, device=DEV)
    q[:, :, 0] = 1
    pg.k[0, :, :, :, 0] = 0
    slots = torch.arange(706, device=DEV)
    ramp = slots.float() * 0.5 - 200  # rising along the cache: each tile raises the maximum
    for s, x in ((0, ramp), (1, -ramp), (2, torch.full_like(ramp, -3e4)), (3, torch.full_like(ramp, 3e4))):
        pg.k[0, pg.tables[0].long()[slots // P], 0, slots % P, s] = x.to(BF)
    q.zero_()
    for i in range(4):
        q[i, :, i] = 8
    q[4, :, 0], q[5, :, 1] = 40, 40
    q = q.to(BF)
    out, lse = run_attn(pg, q, ctx, new)
    check_attn(pg, q, out, lse, pg.tables, ctx, new, None, None, 0, 1 / math.sqrt(d), n_kv)


def test_attn_same_bits_again_on_another_stream_and_in_a_graph():
    g = gen(24)
    ctx, new = [3000, 17, 900], [9, 30, 1]
    pg = Paged(g, [a + b for a, b in zip(ctx, new)], 4, 64, 128)
    q = torch.randn(40, 32, 128, generator=g, device=DEV).to(BF)
    rows = [tree_of(g, n, "tree")[0] for n in new]
    mask = mask_words([m for r in rows for m in r], 1)
    ws = torch.empty(mk.tree_attn_workspace_bytes(pg.cache), dtype=torch.uint8, device=DEV).fill_(255)
    want, want_lse = run_attn(pg, q, ctx, new, ws, tree_mask=mask)
    check_attn(pg, q, want, want_lse, pg.tables, ctx, new, rows, None, 0, 1 / math.sqrt(128), 4)
    for _ in range(3):
        out, lse = run_attn(pg, q, ctx, new, ws, tree_mask=mask)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
    side = torch.cuda.Stream()
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=DEV)
    args = (pg.cache, 0, q, out, ints(starts(new)), ints(ctx), pg.tables, ws)
    side.wait_stream(torch.cuda.current_stream())
    mk.tree_attn(*args, tree_mask=mask, lse=lse, stream=side)
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mk.tree_attn(*args, tree_mask=mask, lse=lse)
    # other contexts, written into the captured call's arrays
    for c in ([100, 3, 64], ctx):  # within the pages that each table has
        args[5].copy_(ints(c))
        out.fill_(0)
        graph.replay()
        torch.cuda.synchronize()
        check_attn(pg, q, out, lse, pg.tables, c, new, rows, None, 0, 1 / math.sqrt(128), 4)
    assert torch.equal(out, want)


def test_attn_two_calls_at_once():
    """Calls on two streams, a workspace each."""
    g = gen(25)
    ctx, new = [5000, 300], [4, 20]
    pg = Paged(g, [a + b for a, b in zip(ctx, new)], 4, 64, 128)
    q = [torch.randn(24, 32, 128, generator=g, device=DEV).to(BF) for _ in range(2)]
    want = [run_attn(pg, x, ctx, new) for x in q]
    cu, cl = ints(starts(new)), ints(ctx)
    out = [torch.empty_like(x) for x in q]
    ws = [torch.empty(mk.tree_attn_workspace_bytes(pg.cache), dtype=torch.uint8, device=DEV) for _ in q]
    streams = [torch.cuda.Stream() for _ in q]
    torch.cuda.synchronize()
    for _ in range(5):
        for i in range(2):
            mk.tree_attn(pg.cache, 0, q[i], out[i], cu, cl, pg.tables, ws[i], stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(out[i], want[i][0])


def test_attn_leaves_out_what_is_out_of_range():
    g = gen(26)
    ctx, new, P = [100, 100, 100, 100], [4, 4, 70, 4], 16
    pg = Paged(g, [a + b for a, b in zip(ctx, new)], 2, P, 64, extra_cols=0)
    q = torch.randn(82, 4, 64, generator=g, device=DEV).to(BF)
    ws = torch.empty(mk.tree_attn_workspace_bytes(pg.cache), dtype=torch.uint8, device=DEV)
    cu = starts(new)
    every = mask_words([-1 % (1 << 64)] * 82, 1)

    def call(cu=cu, ctx=ctx, tables=pg.tables, **kw):
        out, st = torch.full_like(q, 5.0), new_status()
        mk.tree_attn(pg.cache, 0, q, out, ints(cu), ints(ctx), tables, ws, status=st, **kw)
        with pytest.raises(mk.MkError) as e:
            mk.check_status(st)
        assert e.value.code == mk.MK_ERR_DEVICE and "tree_attn" in str(e.value)
        return [bool((out[cu[b]:cu[b + 1]] != 5).all(-1).all()) if 0 <= cu[b] < cu[b + 1] <= 82 else None for b in range(4)], out

    assert call(tree_mask=every)[0] == [True, True, False, True]  # 70 tokens, 64 bits
    assert call(ctx=[100, -1, 100, 100])[0] == [True, False, True, True]
    assert call(ctx=[100, 100, 100, 1 << 30])[0] == [True, True, True, False]
    assert call(cu=[0, 4, 8, 78, 83])[0] == [True, True, True, None]
    tables = pg.tables.clone()
    tables[3, 2] = pg.k.shape[1]
    done, out = call(tables=tables)
    assert done[:3] == [True] * 3
    pos = ints([c + i for c, n in zip(ctx, new) for i in range(n)])
    good = torch.full_like(q, 5.0)
    mk.tree_attn(pg.cache, 0, q, good, ints(cu), ints(ctx), pg.tables, ws, positions=pos, window=50)
    pos[1] = 99
    done, out = call(positions=pos, window=50)
    assert done == [True] * 4 and torch.equal(out[4:], good[4:])


def test_attn_and_append_behind_four_gigabytes():
    """Offsets that pass 32 bits: pools of over 2^32 elements, pages at their far end, two layers."""
    P, n_kv, d = 64, 4, 128
    pages = (1 << 31) // (n_kv * P * d) + 100  # a layer of over 2^31 elements
    k = torch.empty(2, pages, n_kv, P, d, dtype=BF, device=DEV)
    v = torch.empty_like(k)
    cache = mk.KvCache(k, v, BASE)
    g = gen(27)
    ctx, n = 200, 6
    ids = [pages - 1, 3, pages - 7, pages // 2, pages - 2]
    tables = ints([ids])
    for pool in (k, v):
        pool[1, ids] = torch.randn(5, n_kv, P, d, generator=g, device=DEV, dtype=BF)
    x = torch.randn(n, 32 + 8, d, generator=g, device=DEV)
    q_out = torch.empty(n, 32, d, dtype=BF, device=DEV)
    cu, cl = ints([0, n]), ints([ctx])
    mk.kv_append(cache, 1, x[:, 32:36], x[:, 36:], cu, cl, tables, q=x[:, :32], q_out=q_out)
    s = torch.arange(ctx, ctx + n, device=DEV)
    page = tables[0].long()[s // P]
    assert torch.equal(v[1, page, :, s % P], x[:, 36:].to(BF))
    out, lse = torch.empty_like(q_out), torch.empty(n, 32, device=DEV)
    ws = torch.empty(mk.tree_attn_workspace_bytes(cache), dtype=torch.uint8, device=DEV)
    mk.tree_attn(cache, 1, q_out, out, cu, cl, tables, ws, lse=lse)

    class Small:
        pass
    small = Small()
    small.k, small.v = k[1:, ids], v[1:, ids]
    check_attn(small, q_out, out, lse, ints([[0, 1, 2, 3, 4]]), [ctx], [n], None, None, 0, 1 / math.sqrt(d), n_kv)


# -------------------------------------------------------------------- commit

@pytest.mark.parametrize("n_kv,d,P,layers", [(2, 64, 16, 3), (4, 128, 64, 2), (1, 64, 256, 1), (3, 128, 32, 5)])
def test_commit(n_kv, d, P, layers):
    g = gen(31)
    ctx = [0, 13, 16, 100, 5, 60]
    paths = [[0, 1, 2], [3], [], [1, 2, 4, 7, 11, 12, 13, 14, 15, 18, 29], [0, 2, 3, 9],
             [i + (i > 40) + (i > 3) for i in range(75)]]
    n = [30, 5, 4, 33, 10, 90]
    pg = Paged(g, [a + b for a, b in zip(ctx, n)], n_kv, P, d, layers=layers)
    width = 80
    want = [pg.k.cpu(), pg.v.cpu()]
    for b, p in enumerate(paths):
        for w in want:
            plain.commit(w, pg.tables[b].tolist(), ctx[b], p)
    new_lens, st = torch.full((6,), -9, dtype=torch.int32, device=DEV), new_status()
    mk.kv_commit(pg.cache, ints(ctx), ints([p + [-5] * (width - len(p)) for p in paths]), ints([len(p) for p in paths]), pg.tables,
                 new_lens=new_lens, status=st)
    mk.check_status(st)
    assert torch.equal(pg.k.cpu(), want[0]) and torch.equal(pg.v.cpu(), want[1])
    assert new_lens.tolist() == [a + len(p) for a, p in zip(ctx, paths)]


def test_commit_leaves_out_bad_paths():
    g = gen(32)
    P = 16
    pg = Paged(g, [40] * 6, 2, P, 64, layers=2, extra_cols=0)
    tables = pg.tables.clone()
    tables[4, 1] = 10 ** 6
    k = pg.k.clone()
    ctx, lens = [10, 10, 10, -4, 10, 10], [3, 2, 9, 1, 2, 2]
    path = [[1, 3, 3], [0, 38, 0], [0, 1, 2], [1, 0, 0], [0, 9, 0], [2, 5, 0]]
    new_lens, st = torch.empty(6, dtype=torch.int32, device=DEV), new_status()
    mk.kv_commit(pg.cache, ints(ctx), ints(path), ints(lens), tables, new_lens=new_lens, status=st)
    with pytest.raises(mk.MkError) as e:
        mk.check_status(st)
    assert e.value.code == mk.MK_ERR_DEVICE and "kv_commit" in str(e.value)
    assert new_lens.tolist() == [10, 10, 10, -4, 10, 12]  # the last path is good
    want = k.cpu()
    plain.commit(want, pg.tables[5].tolist(), 10, [2, 5])
    assert torch.equal(pg.k.cpu(), want)


def test_commit_entries_in_front_of_their_place():
    """A path that does not ascend may have entries whose place lies behind the table: nothing there is read."""
    g = gen(33)
    P = 16
    pg = Paged(g, [16, 16], 1, P, 64, extra_cols=0)  # one column: slot 16 has none
    k = pg.k.clone()
    new_lens, st = torch.empty(2, dtype=torch.int32, device=DEV), new_status()
    mk.kv_commit(pg.cache, ints([14, 14]), ints([[0, 0, 1], [0, 1, 1]]), ints([3, 3]), pg.tables, new_lens=new_lens, status=st)
    with pytest.raises(mk.MkError):
        mk.check_status(st)
    assert new_lens.tolist() == [14, 14] and torch.equal(pg.k, k)


# -------------------------------------------------------------------- select

def run_select(logits, scores, n, finished=None, eos=-1):
    R, W = scores.shape
    V = logits.shape[-1]
    flat = logits if logits.dim() == 2 else logits.view(R * W, V)
    out = (torch.empty(R, n, device=DEV), *(torch.empty(R, n, dtype=torch.int32, device=DEV) for _ in range(2)))
    ws = torch.empty(mk.beam_select_workspace_bytes(R, W, V, n), dtype=torch.uint8, device=DEV).fill_(255)
    mk.beam_select(flat, scores, *out, ws, finished=finished, eos=eos)
    return out


def check_select(got, logits, scores, n, finished=None, eos=-1):
    """Equal parents and tokens wherever the plain scores are apart by more than both forms' errors (an fp32 exponential's
    2 ulp in the sum, 2^-22 of a unit; doubles below that); scores to fp32."""
    best, beam, token = plain.select(logits.cpu(), scores.cpu(), n, None if finished is None else finished.cpu(), eos)
    s, p, t = (x.cpu() for x in got)
    ref = best[:, :n]
    assert torch.equal(s.isfinite(), ref.float().isfinite())
    fin = ref.isfinite()
    assert ((s.double() - ref)[fin].abs() <= ref[fin].abs() * 2.0 ** -23 + 2.0 ** -21).all()
    same = (p == beam) & (t == token)
    if not same.all():  # only among scores that are as good as equal and not of one beam
        for r, i in torch.nonzero(~same).tolist():
            near = [j for j in range(best.shape[1]) if j != i and abs(float(best[r, j] - best[r, i])) < 2.0 ** -20]
            assert near and any(int(beam[r, j]) != int(beam[r, i]) for j in near if j < n), (r, i)
    for r in range(s.shape[0]):  # no candidate twice
        assert len(set(zip(p[r].tolist(), t[r].tolist()))) == n


@pytest.mark.parametrize("R,W,V,n", [
    (1, 1, 1, 1), (1, 1, 7, 7), (3, 4, 7, 28), (1, 4, 1000, 4), (2, 3, 4096, 6), (1, 2, 4097, 128), (5, 8, 16385, 16),
    (2, 64, 300, 128), (1, 5, 65537, 10), (64, 4, 2000, 8), (1, 1, 100000, 1), (3, 7, 33, 100), (1, 64, 5000, 128)])
def test_select(R, W, V, n):
    g = gen(41 + V)
    logits = torch.randn(R, W, V, generator=g, device=DEV) * 3
    scores = -10 * torch.rand(R, W, generator=g, device=DEV)
    check_select(run_select(logits, scores, n), logits, scores, n)
    finished = (torch.rand(R, W, generator=g, device=DEV) < 0.4).to(torch.uint8)
    eos = V // 2
    check_select(run_select(logits, scores, n, finished, eos), logits, scores, n, finished, eos)


@pytest.mark.parametrize("V", [50, 4096, 9000])
def test_select_ties_go_to_the_lower_index(V):
    g = gen(42)
    R, W, n = 4, 4, 12
    logits = torch.randint(-2, 3, (R, W, V), generator=g, device=DEV).float()
    logits[0] = 0.0  # every continuation the same
    logits[1, 2] = logits[1, 1]  # twice the same beam
    logits[2] = logits[2].abs() * torch.where(torch.rand(W, V, generator=g, device=DEV) < 0.5, -0.0, 0.0)  # zeros of both signs
    scores = torch.zeros(R, W, device=DEV)
    got = run_select(logits, scores, n)
    best, beam, token = plain.select(logits.cpu(), scores.cpu(), n)
    for r in (0, 2):
        assert torch.equal(got[1][r].cpu().long(), beam[r]) and torch.equal(got[2][r].cpu().long(), token[r])
    check_select(got, logits, scores, n)
    # within a beam ties keep the order of the tokens
    for r in range(R):
        rows = {}
        for s, p, t in zip(*(x[r].tolist() for x in got)):
            key = (p, float(logits[r, p, t]))
            assert rows.get(key, -1) < t
            rows[key] = t


@pytest.mark.parametrize("order", ["up", "down"])
def test_select_sorted_logits(order):
    """Every tile better than the one before it, or the other way round."""
    V, n = 20000, 64
    x = torch.linspace(-5, 5, V, device=DEV)
    logits = torch.stack([x, x * 0.5]).view(1, 2, V)
    logits = logits if order == "up" else logits.flip(-1).contiguous()
    scores = torch.tensor([[-1.0, -1.5]], device=DEV)
    check_select(run_select(logits, scores, n), logits, scores, n)


def test_select_dead_beams_and_bad_logits():
    g = gen(43)
    R, W, V, n = 6, 3, 5000, 8
    logits = torch.randn(R, W, V, generator=g, device=DEV)
    scores = -torch.rand(R, W, generator=g, device=DEV)
    scores[0, 1:] = -math.inf  # the first step: one beam lives
    logits[1, 0, 77] = math.nan  # the row's sum is not a number: the beam is dead
    logits[2, 1, 5] = math.inf
    logits[3, :, 10:] = -math.inf  # ten tokens allowed
    logits[4, 2] = -math.inf  # none
    scores[5] = -math.inf
    got = run_select(logits, scores, n)
    check_select(got, logits, scores, n)
    best, beam, token = plain.select(logits.cpu(), scores.cpu(), n)
    assert torch.equal(got[1].cpu().long(), beam) and torch.equal(got[2].cpu().long(), token)
    # fewer living continuations than wanted: the rest in the order of the indices
    few = torch.full((1, 2, 40), -math.inf, device=DEV)
    few[0, 1, 30] = 1.0
    sc = torch.zeros(1, 2, device=DEV)
    fin = torch.tensor([[1, 0]], dtype=torch.uint8, device=DEV)
    got = run_select(few, sc, 5, fin, 3)
    assert got[1].tolist() == [[0, 1, 0, 0, 0]] and got[2].tolist() == [[3, 30, 0, 1, 2]]
    assert got[0].tolist() == [[0.0, 0.0, -math.inf, -math.inf, -math.inf]]


@pytest.mark.parametrize("pad,offset", [(0, 1), (3, 0), (5, 2)])
def test_select_strided_rows(pad, offset):
    g = gen(44)
    R, W, V, n = 2, 3, 9001, 6
    store = torch.full((R * W, V + pad + offset), 100.0, device=DEV)
    rows = store[:, offset:offset + V]
    rows.copy_(torch.randn(R * W, V, generator=g, device=DEV))
    scores = -torch.rand(R, W, generator=g, device=DEV)
    check_select(run_select(rows, scores, n), rows.reshape(R, W, V), scores, n)


def test_select_in_a_graph():
    g = gen(45)
    R, W, V, n = 3, 4, 40000, 8
    logits = torch.randn(R, W, V, generator=g, device=DEV)
    scores = -torch.rand(R, W, generator=g, device=DEV)
    out = (torch.empty(R, n, device=DEV), *(torch.empty(R, n, dtype=torch.int32, device=DEV) for _ in range(2)))
    ws = torch.empty(mk.beam_select_workspace_bytes(R, W, V, n), dtype=torch.uint8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    mk.beam_select(logits.view(R * W, V), scores, *out, ws)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        mk.beam_select(logits.view(R * W, V), scores, *out, ws)
    for _ in range(3):
        logits.copy_(torch.randn(R, W, V, generator=g, device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        check_select(out, logits, scores, n)


# ------------------------------------------------------------------- reorder

@pytest.mark.parametrize("n_kv,d,P,layers,W", [(2, 64, 16, 2, 4), (4, 128, 64, 3, 8), (1, 64, 256, 1, 1), (2, 128, 32, 2, 64),
                                               (3, 64, 16, 7, 5)])
def test_reorder(n_kv, d, P, layers, W):
    import random
    r = random.Random(W)
    g = gen(51)
    lens = [0, 1, P - 1, P, P + 1, 3 * P + 7, 4 * P]
    R = len(lens)
    pg = Paged(g, [6 * P] * (R * W), n_kv, P, d, layers=layers)
    parents = [[r.randrange(W) for _ in range(W)] for _ in range(R)]
    parents[1] = list(range(W))  # nobody moves
    parents[2] = list(reversed(range(W)))  # all do, no copies
    parents[5] = [W - 1] * W  # one survivor
    tables = pg.tables.view(R, W, -1).cpu()
    want = [pg.k.cpu(), pg.v.cpu()]
    new = plain.reorder(want, tables, lens, parents, P)
    out, st = torch.full_like(pg.tables, -7), new_status()
    mk.beam_reorder(pg.cache, ints(lens), ints(parents), pg.tables, out, status=st)
    mk.check_status(st)
    assert torch.equal(out.cpu().view(R, W, -1), new)
    assert torch.equal(pg.k.cpu(), want[0]) and torch.equal(pg.v.cpu(), want[1])


@pytest.mark.parametrize("R,W,layers,n_kv", [(700, 2, 2, 1), (300, 3, 3, 4), (1, 4, 30, 8), (90, 5, 4, 2), (20, 4, 20, 8)])
def test_reorder_few_and_many_requests(R, W, layers, n_kv):
    """Copies dealt to 8 up to hundreds of blocks per request, several units or less than one to a block."""
    import random
    r, P = random.Random(R), 16
    lens = [r.randrange(3 * P) for _ in range(R)]
    lens[0] = P + 5
    pg = Paged(gen(53), [3 * P] * (R * W), n_kv, P, 64, layers=layers)
    parents = [[r.randrange(W) for _ in range(W)] for _ in range(R)]
    tables = pg.tables.view(R, W, -1).cpu()
    want = [pg.k.cpu(), pg.v.cpu()]
    new = plain.reorder(want, tables, lens, parents, P)
    out, st = torch.full_like(pg.tables, -7), new_status()
    mk.beam_reorder(pg.cache, ints(lens), ints(parents), pg.tables, out, status=st)
    mk.check_status(st)
    assert torch.equal(out.cpu().view(R, W, -1), new)
    assert torch.equal(pg.k.cpu(), want[0]) and torch.equal(pg.v.cpu(), want[1])


def test_reorder_leaves_out_what_is_out_of_range():
    g = gen(52)
    P, W = 16, 3
    pg = Paged(g, [60] * 12, 2, P, 64, extra_cols=0)
    tables = pg.tables.clone()
    tables[9, 1] = -2  # request 3: the surviving beam's open page
    before = pg.k.clone()
    out, st = torch.full_like(tables, -7), new_status()
    mk.beam_reorder(pg.cache, ints([20, -1, 65, 20]), ints([[0, 3, 0], [0, 0, 0], [0, 0, 0], [0, 0, 0]]), tables, out, status=st)
    with pytest.raises(mk.MkError) as e:
        mk.check_status(st)
    assert e.value.code == mk.MK_ERR_DEVICE and "beam_reorder" in str(e.value)
    assert torch.equal(out[:9], tables[:9]) and torch.equal(pg.k, before)


# ------------------------------------------------------------------ together

def test_beam_search_keeps_each_beams_history():
    """Select, reorder and append, step after step: every beam's cache holds the rows of its own tokens' history."""
    g = gen(61)
    R, W, V, P, n_kv, d, L = 2, 4, 200, 16, 2, 64, 2
    prompt, steps = 21, 30
    cols = (prompt + steps) // P + 1
    shared = prompt // P
    pages = R * (shared + W * (cols - shared))
    k = torch.zeros(L, pages, n_kv, P, d, dtype=BF, device=DEV)
    cache = mk.KvCache(k, k.clone(), BASE)
    ids = torch.randperm(pages, generator=g, device=DEV).to(torch.int32).tolist()
    rows = []
    for r in range(R):
        common = [ids.pop() for _ in range(shared)]
        rows += [common + [ids.pop() for _ in range(cols - shared)] for _ in range(W)]
    tables = [ints(rows), torch.empty(R * W, cols, dtype=torch.int32, device=DEV)]
    emb = torch.randn(V, L, n_kv, d, generator=g, device=DEV).to(BF)  # a token's V in each layer
    st = new_status()
    hist = [[[int(x) for x in torch.randint(V, (prompt,), generator=g, device=DEV)]] * W for _ in range(R)]

    def append(tokens, lens, tab):
        n = len(tokens[0])
        x = emb[torch.tensor([t for row in tokens for t in row], device=DEV)]
        for layer in range(L):
            mk.kv_append(cache, layer, x[:, layer].contiguous(), x[:, layer].contiguous(), ints([n * i for i in range(len(tokens) + 1)]),
                         ints(lens), tab, status=st)
    # the prompt lies in beam 0's pages (the full ones are common); the other beams are not alive yet
    for r in range(R):
        append([hist[r][0]], [0], tables[0][r * W:r * W + 1])
    scores = torch.full((R, W), -math.inf, device=DEV)
    scores[:, 0] = 0
    out = [torch.empty(R, W, device=DEV), ints([[0] * W] * R), ints([[0] * W] * R)]
    ws = torch.empty(mk.beam_select_workspace_bytes(R, W, V, W), dtype=torch.uint8, device=DEV)
    for step in range(steps):
        logits = torch.randn(R * W, V, generator=g, device=DEV)
        if step % 7 == 3:
            logits[::W] += 30 * torch.rand(R, 1, generator=g, device=DEV) * (torch.arange(V, device=DEV) < W)
        mk.beam_select(logits, scores, *out, ws)
        mk.beam_reorder(cache, ints([prompt + step] * R), out[1], tables[0], tables[1], status=st)
        tables.reverse()
        append([[t] for row in out[2].tolist() for t in row], [prompt + step] * (R * W), tables[0])
        hist = [[hist[r][p] + [t] for p, t in zip(out[1][r].tolist(), out[2][r].tolist())] for r in range(R)]
        scores.copy_(out[0])
    mk.check_status(st)
    for r in range(R):
        for w in range(W):
            s = torch.arange(prompt + steps, device=DEV)
            page = tables[0][r * W + w].long()[s // P]
            got = cache.v_pool[:, page, :, s % P]  # [slots][layers]...
            want = emb[torch.tensor(hist[r][w], device=DEV)]
            assert torch.equal(got, want), (r, w)


def test_verified_tree_equals_the_run_it_accepts():
    """Drafts appended, attended as a tree, the accepted path committed: the cache and the outputs are those of the accepted
    tokens appended and attended as a run."""
    g = gen(62)
    B, n_q, n_kv, d, P = 3, 8, 2, 64, 16
    ctx, new = [30, 0, 129], [12, 7, 20]
    pg = Paged(g, [a + b for a, b in zip(ctx, new)], n_kv, P, d)
    pg2 = Paged(g, [a + b for a, b in zip(ctx, new)], n_kv, P, d)
    for b in range(B):  # the same contexts
        s = torch.arange(ctx[b], device=DEV)
        for a, c in ((pg.k, pg2.k), (pg.v, pg2.v)):
            c[0][pg2.tables[b].long()[s // P], :, s % P] = a[0][pg.tables[b].long()[s // P], :, s % P]
    trees = [tree_of(g, n, "tree") for n in new]
    paths = [[j for j in range(n) if (t[0][n - 1] >> j) & 1] for t, n in zip(trees, new)]  # the last token's ancestors
    qkv = torch.randn(sum(new), n_q + 2 * n_kv, d, generator=g, device=DEV)
    pos = ints([c + e for c, t in zip(ctx, trees) for e in t[1]])
    q1, st = torch.empty(sum(new), n_q, d, dtype=BF, device=DEV), new_status()
    cu, cl = ints(starts(new)), ints(ctx)
    mk.kv_append(pg.cache, 0, qkv[:, n_q:n_q + n_kv], qkv[:, n_q + n_kv:], cu, cl, pg.tables, q=qkv[:, :n_q], q_out=q1,
                 positions=pos, status=st)
    o1, l1 = run_attn(pg, q1, ctx, new, tree_mask=mask_words([m for t in trees for m in t[0]], 1), positions=pos, status=st)
    new_lens = torch.empty_like(cl)
    width = max(len(p) for p in paths)
    mk.kv_commit(pg.cache, cl, ints([p + [0] * (width - len(p)) for p in paths]), ints([len(p) for p in paths]), pg.tables,
                 new_lens=new_lens, status=st)
    # the same tokens as a run
    pick = torch.tensor([c + j for c, p in zip(starts(new), paths) for j in p], device=DEV)
    run = [len(p) for p in paths]
    x, q2 = qkv[pick], torch.empty(len(pick), n_q, d, dtype=BF, device=DEV)
    mk.kv_append(pg2.cache, 0, x[:, n_q:n_q + n_kv], x[:, n_q + n_kv:], ints(starts(run)), cl, pg2.tables, q=x[:, :n_q], q_out=q2,
                 status=st)
    o2, l2 = run_attn(pg2, q2, ctx, run, status=st)
    mk.check_status(st)
    assert new_lens.tolist() == [c + n for c, n in zip(ctx, run)]
    assert torch.equal(q1[pick], q2)
    for b in range(B):
        s = torch.arange(ctx[b] + run[b], device=DEV)
        for a, c in ((pg.k, pg2.k), (pg.v, pg2.v)):
            assert torch.equal(a[0][pg.tables[b].long()[s // P], :, s % P], c[0][pg2.tables[b].long()[s // P], :, s % P])
    # two orders of the same sums: each within its own bound of the exact value
    check_attn(pg2, q2, o2, l2, pg2.tables, ctx, run, None, None, 0, 1 / math.sqrt(d), n_kv)
    check_attn(pg2, q2, o1[pick], l1[pick], pg2.tables, ctx, run, None, None, 0, 1 / math.sqrt(d), n_kv)


@pytest.mark.parametrize("workload", ["tiny", "small"])
def test_agrees_with_the_decode_step(workload):
    """The operators on the decode step's own pools: attention of its last token in the last layer, from its queries, gives
    its attention output; the pools it wrote are read through the same tables."""
    import synth
    import synth.device
    import parity
    inp = synth.make_inputs(workload)
    w = inp.workload
    sh = w.shape
    model = parity._device_model(sh, w.seed, inp.router_bias)
    sched = mk.Sched(model, w.batch, int(inp.seq_lens.max()))
    sess = mk.Session(model, sched)
    kp, vp = synth.device.device_pools(sh, w.seed, inp.num_pages)
    tok, sl, bt = (torch.as_tensor(x, device=DEV) for x in (inp.tokens, inp.seq_lens, inp.block_tables))
    sess.step(tok, sl, bt, kp, vp, torch.empty(w.batch, sh.vocab, device=DEV))
    sess.check()
    q = sess.region("q", torch.float32, w.batch * sh.n_q * sh.head_dim).view(w.batch, sh.n_q, sh.head_dim)
    attn = sess.region("attn_out", torch.float32, w.batch * sh.n_q * sh.head_dim).view(w.batch, sh.n_q, sh.head_dim)
    cache = mk.KvCache(kp, vp, sh.rope_base)
    qb = q.to(BF)
    out = torch.empty_like(qb)
    ws = torch.empty(mk.tree_attn_workspace_bytes(cache), dtype=torch.uint8, device=DEV)
    st = new_status()
    mk.tree_attn(cache, sh.n_layers - 1, qb, out, ints(list(range(w.batch + 1))), sl - 1, bt, ws, status=st)
    mk.check_status(st)
    # q rounded to bf16 moves a score by at most 2^-8 of sum |q k| scale; p by as much of itself, twice over the quotient;
    # then the operator's own two roundings
    kc, vc = (x.view(BF)[sh.n_layers - 1].cpu() for x in (kp, vp))
    for b in range(w.batch):
        n = int(sl[b])
        k, v = plain.gather_slots(kc, bt[b].tolist(), n), plain.gather_slots(vc, bt[b].tolist(), n)
        ref, _, spread, size = plain.attention(q[b].cpu(), k, v, torch.ones(n, dtype=torch.bool), 1 / math.sqrt(sh.head_dim))
        tol = plain.bf16_bound(ref) + spread * (2.0 ** -8 + 2 * size[:, None] * 2.0 ** -8)
        assert ((out[b].cpu().double() - ref).abs() <= tol).all()
        assert ((attn[b].cpu().double() - ref).abs() <= tol).all()


@pytest.mark.parametrize("low", [-math.inf, -1e30, -3.4028234663852886e38])
def test_select_masked_vocabulary(low):
    """Constrained decoding: a few tokens allowed, all others at one low value (more of them than any bound keeps out)."""
    g = gen(46)
    R, W, V, n = 3, 4, 30000, 16
    logits = torch.full((R, W, V), low, device=DEV)
    allowed = torch.randint(V, (R, W, 10), generator=g, device=DEV)
    logits.scatter_(2, allowed, torch.randn(R, W, 10, generator=g, device=DEV))
    logits[1] = low  # nothing allowed
    logits[2, :, 29000:] = torch.randn(W, 1000, generator=g, device=DEV)  # the last tiles alone
    scores = -torch.rand(R, W, generator=g, device=DEV)
    got = run_select(logits, scores, n)
    best, beam, token = plain.select(logits.cpu(), scores.cpu(), n)
    check_select(got, logits, scores, n)
    for r in (0, 2):
        assert torch.equal(got[1][r].cpu().long(), beam[r]) and torch.equal(got[2][r].cpu().long(), token[r])


def test_calls_with_nothing_to_do():
    g = gen(81)
    pg = Paged(g, [20], 2, 16, 64)
    before = pg.k.clone()
    ws = torch.empty(mk.tree_attn_workspace_bytes(pg.cache), dtype=torch.uint8, device=DEV)
    e = lambda h: torch.empty(0, h, 64, dtype=BF, device=DEV)  # noqa: E731
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    for cu, cl, bt in ((ints([0, 0]), ints([5]), pg.tables), (ints([0]), none, pg.tables[:0])):
        mk.kv_append(pg.cache, 0, e(2), e(2), cu, cl, bt, q=e(4), q_out=e(4))
        mk.tree_attn(pg.cache, 0, e(4), e(4), cu, cl, bt, ws)
    # tokens, but no sequence that has them
    x = torch.ones(3, 2, 64, dtype=BF, device=DEV)
    q = torch.ones(3, 4, 64, dtype=BF, device=DEV)
    out = torch.full_like(q, 5.0)
    mk.kv_append(pg.cache, 0, x, x, ints([0, 0]), ints([5]), pg.tables)
    mk.tree_attn(pg.cache, 0, q, out, ints([3, 3]), ints([5]), pg.tables, ws)
    mk.kv_commit(pg.cache, ints([5]), ints([[]]).view(1, 0), ints([0]), pg.tables, new_lens=(n := ints([0])))
    assert n.tolist() == [5] and (out == 5).all() and torch.equal(pg.k, before)


def test_first_call_of_a_handle_inside_a_capture():
    g = gen(82)
    pg = Paged(g, [300], 2, 64, 64)
    q = torch.randn(3, 8, 64, generator=g, device=DEV).to(BF)
    cu, cl = ints([0, 3]), ints([297])
    want, _ = run_attn(pg, q, [297], [3])
    cache = mk.KvCache(pg.k, pg.v, BASE)
    out = torch.zeros_like(q)
    ws = torch.empty(mk.tree_attn_workspace_bytes(cache), dtype=torch.uint8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        mk.tree_attn(cache, 0, q, out, cu, cl, pg.tables, ws)
    assert (out == 0).all()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_many_sequences():
    """More sequences than threads of a block or lanes of a warp, some without tokens, one cache."""
    g = gen(83)
    B, n_kv, d, P = 600, 2, 64, 16
    new = [(7 * b) % 4 for b in range(B)]
    ctx = [(13 * b) % 50 for b in range(B)]
    pg = Paged(g, [a + n for a, n in zip(ctx, new)], n_kv, P, d)
    T = sum(new)
    qkv = torch.randn(T, 8, d, generator=g, device=DEV)
    q_out = torch.empty(T, 4, d, dtype=BF, device=DEV)
    st, cu, cl = new_status(), ints(starts(new)), ints(ctx)
    mk.kv_append(pg.cache, 0, qkv[:, 4:6], qkv[:, 6:], cu, cl, pg.tables, q=qkv[:, :4], q_out=q_out, status=st)
    out, lse = run_attn(pg, q_out, ctx, new, status=st)
    mk.check_status(st)
    check_attn(pg, q_out, out, lse, pg.tables, ctx, new, None, None, 0, 1 / math.sqrt(d), n_kv)
    slot = torch.tensor([a + i for a, n in zip(ctx, new) for i in range(n)], device=DEV)
    seq = torch.tensor([b for b, n in enumerate(new) for _ in range(n)], device=DEV)
    assert torch.equal(pg.v[0][pg.tables.long()[seq, slot // P], :, slot % P], qkv[:, 6:].to(BF))
    paths = [[n - 1] if n > 1 else [] for n in new]
    new_lens = torch.empty(B, dtype=torch.int32, device=DEV)
    want = pg.v.cpu()
    for b, p in enumerate(paths):
        plain.commit(want, pg.tables[b].tolist(), ctx[b], p)
    mk.kv_commit(pg.cache, cl, ints([p + [0] * (1 - len(p)) for p in paths]), ints([len(p) for p in paths]), pg.tables,
                 new_lens=new_lens, status=st)
    mk.check_status(st)
    assert torch.equal(pg.v.cpu(), want) and new_lens.tolist() == [a + len(p) for a, p in zip(ctx, paths)]


RUN_POSITIONS = {
    "repeated": lambda n: [0 if j < 7 * n // 10 else j for j in range(n)],
    "permuted": lambda n: [7 * j % n for j in range(n)],
    "reversed": lambda n: [n - 1 - j for j in range(n)],
    "blocks": lambda n: [(j + 300) % n for j in range(n)],
}


@pytest.mark.parametrize("order", list(RUN_POSITIONS))
@pytest.mark.parametrize("n_q,n_kv,d,P,ctx,new,window", [
    (2, 2, 64, 16, [0], [1000], 900), (8, 1, 128, 64, [0, 77], [1000, 501], 500), (8, 2, 64, 64, [300], [640], 128),
    (1, 1, 128, 32, [2000], [600], 599), (1, 1, 64, 16, [130], [600], 600)])
def test_attn_run_with_positions_and_a_window(n_q, n_kv, d, P, ctx, new, window, order):
    """A run whose positions are not its slots: new tokens can be a window apart in either order, so whole tiles of them are
    seen by some rows of a group only (not where the window holds all of them: the last two shapes)."""
    assert all(math.gcd(7, n) == 1 for n in new)
    g = gen(91)
    pg = Paged(g, [a + b for a, b in zip(ctx, new)], n_kv, P, d)
    q = torch.randn(sum(new), n_q, d, generator=g, device=DEV).to(BF)
    pos = [[c + p for p in RUN_POSITIONS[order](n)] for c, n in zip(ctx, new)]
    st = new_status()
    out, lse = run_attn(pg, q, ctx, new, window=window, positions=ints([p for row in pos for p in row]), status=st)
    mk.check_status(st)
    check_attn(pg, q, out, lse, pg.tables, ctx, new, None, pos, window, 1 / math.sqrt(d), n_kv)


@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_attn_run_with_positions_leaves_values_outside_the_window_out(value):
    g = gen(92)
    n, W, P, d = 700, 450, 16, 64
    pg = Paged(g, [n], 1, P, d)
    q = torch.randn(n, 2, d, generator=g, device=DEV).to(BF)
    pos = RUN_POSITIONS["permuted"](n - 1) + [n - 1]
    kw = dict(window=W, positions=ints(pos))
    clean, clean_lse = run_attn(pg, q, [0], [n], **kw)
    j = 300
    page = pg.tables[0, j // P].item()
    pg.v[0, page, :, j % P] = value
    pg.k[0, page, :, j % P, 3] = value
    out, lse = run_attn(pg, q, [0], [n], **kw)
    see = torch.tensor([j <= i and pos[i] - pos[j] < W for i in range(n)], device=DEV)
    assert torch.equal(out[~see], clean[~see]) and torch.equal(lse[~see], clean_lse[~see])
    if math.isnan(value):
        assert out[see].isnan().all()


@pytest.mark.parametrize("first,later,n", [(5, 0, 16), (3, 8, 16), (0, 9, 16), (0, 200, 16), (12, 3000, 16), (90, 20, 128), (40, 500, 128)])
def test_select_masked_vocabulary_over_several_tiles(first, later, n):
    """Enough rows that a block takes all tiles of one: fewer than n allowed tokens in its first tile, so that no bound holds
    there, and few or many behind it."""
    g = gen(94)
    R, W, V = 83, 4, 20000
    logits = torch.full((R, W, V), -math.inf, device=DEV)
    for lo, hi, count in ((0, 4096, first), (4096, V, later)):
        if count:
            at = torch.randint(lo, hi, (R, W, count), generator=g, device=DEV)
            logits.scatter_(2, at, torch.randn(R, W, count, generator=g, device=DEV))
    scores = -torch.rand(R, W, generator=g, device=DEV)
    got = run_select(logits, scores, n)
    check_select(got, logits, scores, n)
    best, beam, token = plain.select(logits.cpu(), scores.cpu(), n)
    dead = best[:, :n] == -math.inf  # in the order of the indices
    assert torch.equal(got[1].cpu().long()[dead], beam[dead]) and torch.equal(got[2].cpu().long()[dead], token[dead])
    for _ in range(20):
        assert all(torch.equal(a, b) for a, b in zip(got, run_select(logits, scores, n)))


def test_attention_right_behind_an_append_in_place():
    """Q rotated onto itself (rows that share cache lines with their neighbours) and read by the next kernel, which is let in
    before the append has ended; with and without a wait between the calls."""
    g = gen(95)
    n_q, n_kv, d, P, n = 5, 1, 64, 16, 900
    pg = Paged(g, [n + 40], n_kv, P, d)
    src = torch.randn(n, (n_q + 2 * n_kv) * d + 24, generator=g, device=DEV).to(BF)
    cu, cl = ints([0, n]), ints([40])
    ws = torch.empty(mk.tree_attn_workspace_bytes(pg.cache), dtype=torch.uint8, device=DEV)

    def run(wait):
        rows = src.clone()
        x = rows[:, :(n_q + 2 * n_kv) * d].unflatten(1, (-1, d))
        out = torch.empty(n, n_q, d, dtype=BF, device=DEV)
        torch.cuda.synchronize()
        mk.kv_append(pg.cache, 0, x[:, n_q:n_q + 1], x[:, n_q + 1:], cu, cl, pg.tables, q=x[:, :n_q], q_out=x[:, :n_q])
        if wait:
            torch.cuda.synchronize()
        mk.tree_attn(pg.cache, 0, x[:, :n_q], out, cu, cl, pg.tables, ws)
        return x[:, :n_q].clone(), out
    q, want = run(True)
    for _ in range(30):
        again = run(False)
        assert torch.equal(again[0], q) and torch.equal(again[1], want)


@pytest.mark.parametrize("score", [-math.inf, math.nan])
@pytest.mark.parametrize("eos", [0, 2, 5, 39])
def test_select_finished_beams_without_a_score(score, eos):
    """A finished beam whose score is -inf (or no number) has no better continuation than any other: the lowest indices."""
    logits = torch.randn(1, 2, 40, generator=gen(51), device=DEV)
    fin = torch.ones(1, 2, dtype=torch.uint8, device=DEV)
    scores = torch.tensor([[score, -2.0]], device=DEV)
    got = run_select(logits, scores, 6, fin, eos)
    # the living score first, then 0, 1, 2, ... of beam 0
    assert got[0].tolist() == [[-2.0] + [-math.inf] * 5]
    assert got[1].tolist() == [[1] + [0] * 5] and got[2].tolist() == [[eos, 0, 1, 2, 3, 4]]
    got = run_select(logits[:, :1].contiguous(), scores[:, :1].contiguous(), 6, fin[:, :1].contiguous(), eos)
    assert got[0].tolist() == [[-math.inf] * 6] and got[2].tolist() == [[0, 1, 2, 3, 4, 5]]


@pytest.mark.parametrize("R,W,V,n", [(1, 4, 1000, 6), (2, 3, 4096, 128), (1, 2, 9000, 16), (1, 64, 40, 33)])
@pytest.mark.parametrize("low", [-1e30, -3.4028234663852886e38])
def test_select_scores_that_absorb_the_logits(R, W, V, n, low):
    """A beam's score so far from zero that all its continuations score the same in 64 bits: the lowest tokens, not the
    largest logits."""
    g = gen(47)
    logits = torch.randn(R, W, V, generator=g, device=DEV) * 3
    for lows in (range(W), range(1, W), [w for w in range(W) if w % 2]):
        scores = -torch.rand(R, W, generator=g, device=DEV)
        scores[:, list(lows)] = low
        x = logits.clone()
        if 0 not in lows:  # the other beams have few continuations, so that the absorbed ones are wanted
            for w in set(range(W)) - set(lows):
                x[:, w, 3:] = -math.inf
        got = run_select(x, scores, n)
        best, beam, token = plain.select(x.cpu(), scores.cpu(), n)
        assert torch.equal(got[1].cpu().long(), beam) and torch.equal(got[2].cpu().long(), token)
        check_select(got, x, scores, n)


def test_select_logits_below_the_last_bit_of_the_score():
    g = gen(48)
    # all logits far below the last bit of their log-sum-exp: every score of a beam is the same
    logits = torch.randn(1, 2, 9000, generator=g, device=DEV) * 1e-30
    scores = torch.tensor([[-1.0, -0.5]], device=DEV)
    for n in (1, 7, 128):
        got = run_select(logits, scores, n)
        assert got[1].tolist() == [[1] * n] and got[2].tolist() == [list(range(n))]


@pytest.mark.parametrize("n", [3, 8, 16, 40])
def test_select_ties_of_different_logits(n):
    """Two groups of logits that differ by less than the scores' last bit within a group: a tie at the border is broken by
    the index, across beams, and what lies above it is kept."""
    V, W, a = 6000, 3, 5
    r = torch.Generator().manual_seed(49)
    logits, groups = torch.rand(1, W, V, generator=r) * 1e-7, []
    for w in range(W):
        at = torch.randperm(V, generator=r)[:a].sort().values
        logits[0, w, at] = 1 + torch.arange(a).flip(0) * 2.0 ** -22
        groups.append(at.tolist())
    scores = torch.full((1, W), -1e12)
    # the groups hold together and apart, whatever the last bits of the log-sum-exp
    cand = scores.double()[..., None] + (logits.double() - torch.logsumexp(logits.double(), -1, keepdim=True))
    for shift in (-2.0 ** -20, 2.0 ** -20):
        moved = scores.double()[..., None] + (logits.double() - torch.logsumexp(logits.double(), -1, keepdim=True) + shift)
        assert torch.equal(cand, moved) and len(cand.unique()) == 2
    got = run_select(logits.to(DEV), scores.to(DEV), n)
    top = [(w, t) for w in range(W) for t in groups[w]]
    rest = [(0, t) for t in range(V) if t not in groups[0]]
    want = (top + rest)[:n]
    assert list(zip(got[1][0].tolist(), got[2][0].tolist())) == want


def test_select_infinite_score():
    """A beam of score +inf: all its finite continuations are worth the same."""
    logits = torch.randn(1, 2, 500, generator=gen(50), device=DEV)
    logits[0, 1, :4] = -math.inf
    got = run_select(logits, torch.tensor([[-1.0, math.inf]], device=DEV), 6)
    assert got[0].tolist() == [[math.inf] * 6] and got[1].tolist() == [[1] * 6] and got[2].tolist() == [[4, 5, 6, 7, 8, 9]]


def test_select_absorbed_scores_beside_finished_beams_and_in_long_rows():
    g = gen(52)
    # a finished beam of the same score as the absorbed ones around it
    logits = torch.randn(2, 4, 300, generator=g, device=DEV)
    scores = torch.full((2, 4), -1e30, device=DEV)
    scores[1, 0] = -2e30
    fin = torch.tensor([[1, 0, 1, 0], [0, 1, 0, 0]], dtype=torch.uint8, device=DEV)
    got = run_select(logits, scores, 5, fin, 7)
    assert got[1].tolist() == [[0, 1, 1, 1, 1], [1, 2, 2, 2, 2]] and got[2].tolist() == [[7, 0, 1, 2, 3]] * 2
    # several tiles to a part, ties behind many tiles without any
    R, W, V, n = 83, 4, 13000, 16
    logits = torch.full((R, W, V), -math.inf, device=DEV)
    logits[:, :, 12000:] = torch.randn(R, W, 1000, generator=g, device=DEV)
    scores = torch.full((R, W), -3e38, device=DEV)
    got = run_select(logits, scores, n)
    assert (got[1] == 0).all() and (got[2] == torch.arange(12000, 12000 + n, device=DEV, dtype=torch.int32)).all()


def test_records_name_the_page_that_is_out_of_range():
    """A good source and a bad destination, and the other way round: the message has the bad one."""
    P = 16
    pg = Paged(gen(93), [32, 32], 1, P, 64, extra_cols=0)
    for column, slot_from, bad in ((0, 3, 54321), (1, 3, 54321), (0, 3, -17)):
        tables, st = pg.tables.clone(), new_status()
        tables[0, column] = bad
        mk.kv_commit(pg.cache, ints([14, 14]), ints([[slot_from], [slot_from]]), ints([1, 1]), tables, status=st)  # 17 -> 14
        with pytest.raises(mk.MkError) as e:
            mk.check_status(st)
        assert f"page id {bad} out of range" in str(e.value)
    for row, bad in ((0, 54321), (1, 54321), (1, -17)):  # beam 0 survives, beam 1's open page takes the copy
        tables, st = pg.tables.clone(), new_status()
        tables[row, 1] = bad
        mk.beam_reorder(pg.cache, ints([20]), ints([[0, 0]]), tables, torch.empty_like(tables), status=st)
        with pytest.raises(mk.MkError) as e:
            mk.check_status(st)
        assert f"page id {bad} out of range" in str(e.value)


def test_select_as_many_rows_as_it_takes():
    g = gen(96)
    R, W, V, n = 16383, 4, 20, 4
    logits = torch.randn(R, W, V, generator=g, device=DEV) * 3
    scores = -10 * torch.rand(R, W, generator=g, device=DEV)
    check_select(run_select(logits, scores, n), logits, scores, n)


@pytest.mark.parametrize("cu", [[0, 3, 2, 2], [9, 12, 12, 12], [-7, -2, 0, 3], [0, 9, 9, 8], [3, 3, 3, -1]])
def test_append_records_sequences_without_a_token(cu):
    """Lengths below zero and rows that the arrays do not have, where no token belongs to the sequence."""
    pg = Paged(gen(97), [20] * 3, 2, 16, 64)
    k, st = torch.ones(9, 2, 64, dtype=BF, device=DEV), new_status()
    mk.kv_append(pg.cache, 0, k, k, ints(cu), ints([0, 0, 0]), pg.tables, status=st)
    with pytest.raises(mk.MkError) as e:
        mk.check_status(st)
    assert e.value.code == mk.MK_ERR_DEVICE and "kv_append" in str(e.value)


def test_attn_odd_values_in_a_long_run_end_in_time():
    """A NaN among 40000 new tokens, each of which may lie outside a row's window: what it adds to the rows that see it is
    found within the kernel's wait limits."""
    g = gen(98)
    n, W, P, d = 40001, 20000, 64, 64
    assert math.gcd(7, n) == 1
    pg = Paged(g, [n], 1, P, d)
    q = torch.randn(n, 2, d, generator=g, device=DEV).to(BF)
    pos = torch.arange(n, device=DEV) * 7 % n
    st = new_status()
    kw = dict(window=W, positions=pos.to(torch.int32), status=st)
    clean, clean_lse = run_attn(pg, q, [0], [n], **kw)
    j = 20011
    pg.v[0, pg.tables[0, j // P].item(), :, j % P] = math.nan
    out, lse = run_attn(pg, q, [0], [n], **kw)
    mk.check_status(st)
    see = (torch.arange(n, device=DEV) >= j) & (pos - pos[j] < W)
    assert out[see].isnan().all() and torch.equal(out[~see], clean[~see]) and torch.equal(lse, clean_lse)


# ------------------------------------------------------- beside the decode step

def decode_setup(shape, seed, batch, max_len):
    import parity
    model = parity._device_model(shape, seed, None)
    return mk.Session(model, mk.Sched(model, batch, max_len))


@pytest.mark.parametrize("R,W", [(1, 2), (2, 4)])
def test_beam_search_over_the_decode_step(R, W):
    """mk_decode_step, beam_select and beam_reorder, step after step: each surviving beam's cache and logits are those of its
    own history, decoded again without any reordering."""
    import synth
    import synth.device
    sh, seed = synth.MODELS["tiny"], 5
    P, V, B, prompt, steps = sh.page_size, sh.vocab, R * W, 37, 21
    cols, full = (prompt + steps + P - 1) // P, prompt // P
    pages = R * full + B * (cols - full)
    kp, vp = synth.device.device_pools(sh, seed, pages + B * cols)
    ids = torch.randperm(pages + B * cols, generator=torch.Generator().manual_seed(seed)).tolist()
    rows, again = [], [[ids.pop() for _ in range(cols)] for _ in range(B)]
    for r in range(R):
        common = [ids.pop() for _ in range(full)]
        rows += [common + [ids.pop() for _ in range(cols - full)] for _ in range(W)]
    for b in range(B):  # the prompt's rows (the generator's values), the same for the beams of a request
        for c in range(full + 1):
            for pool in (kp, vp):
                if c == full and b % W:
                    pool[:, rows[b][c]] = pool[:, rows[b - b % W][c]]
                pool[:, again[b][c]] = pool[:, rows[b][c]]
    cache = mk.KvCache(kp, vp, sh.rope_base)
    sess, st = decode_setup(sh, seed, B, prompt + steps), new_status()
    tables, again = [ints(rows), torch.empty(B, cols, dtype=torch.int32, device=DEV)], ints(again)
    logits, ws = torch.empty(B, V, device=DEV), torch.empty(mk.beam_select_workspace_bytes(R, W, V, W), dtype=torch.uint8, device=DEV)
    scores = torch.full((R, W), -math.inf, device=DEV)
    scores[:, 0] = 0
    out = [torch.empty(R, W, device=DEV), ints([[0] * W] * R), ints([[0] * W] * R)]
    hist = [[[7 + r]] * W for r in range(R)]
    tokens, moved = ints([h[-1] for row in hist for h in row]), 0
    for t in range(steps):
        n = prompt + t  # tokens in the caches before this step's
        sess.step(tokens, ints([n + 1] * B), tables[0], kp, vp, logits)
        sess.check()
        if t + 1 == steps:
            break
        spiced = logits + 0.7 * torch.randn(B, V, generator=gen(100 + t), device=DEV)  # so that beams die and multiply
        mk.beam_select(spiced, scores, *out, ws)
        mk.beam_reorder(cache, ints([n + 1] * R), out[1], tables[0], tables[1], status=st)
        tables.reverse()
        parents = out[1].tolist()
        moved += sum(len(set(p)) < W for p in parents)
        hist = [[hist[r][p] + [w] for p, w in zip(parents[r], out[2].tolist()[r])] for r in range(R)]
        tokens = out[2].flatten().clone()
        scores.copy_(out[0])
    mk.check_status(st)
    assert moved > 4
    want = torch.empty_like(logits)
    for t in range(steps):
        sess.step(ints([h[t] for row in hist for h in row]), ints([prompt + t + 1] * B), again, kp, vp, want)
        sess.check()
    # two runs of the step on the same history: fp32 sums in any order, K and V rounded to bf16 behind them
    assert ((logits - want).abs() <= 1e-3 * want.abs().amax(-1, keepdim=True)).all()
    s = torch.arange(prompt + steps, device=DEV)
    for b in range(B):
        for pool in (kp.view(BF), vp.view(BF)):
            a, c = (pool[:, tab[b].long()[s // P], :, s % P].double() for tab in (tables[0], again))
            assert torch.equal(a[:prompt], c[:prompt])
            assert ((a - c).abs() <= c.abs() * 2.0 ** -7 + 1e-3 * c.abs().amax(-1, keepdim=True)).all(), b


def test_append_rotates_as_the_decode_step():
    """The step's K of one token at several positions against kv_append of its K at position 0, where nothing turns."""
    import dataclasses

    import synth
    import synth.device
    for name in ("tiny", "small"):
        sh = dataclasses.replace(synth.MODELS[name], n_layers=1)
        P, at = sh.page_size, [0, 1, 2, 77, 500, 1023]
        cols = at[-1] // P + 1
        kp, vp = synth.device.device_pools(sh, 3, 2 * cols)
        tab = ints([list(range(cols)), list(range(cols, 2 * cols))])
        sess = decode_setup(sh, 3, 1, at[-1] + 1)
        cache, st = mk.KvCache(kp, vp, sh.rope_base), new_status()
        logits = torch.empty(1, sh.vocab, device=DEV)
        raw = None
        for p in at:
            sess.step(ints([11]), ints([p + 1]), tab[:1].contiguous(), kp, vp, logits)
            sess.check()
            k, v = (x.view(BF)[0, p // P, :, p % P].clone()[None] for x in (kp, vp))
            if raw is None:
                raw = k, v
            mk.kv_append(cache, 0, *raw, ints([0, 1]), ints([p]), tab[1:].contiguous(), status=st)
            got_k, got_v = (x.view(BF)[0, cols + p // P, :, p % P] for x in (kp, vp))
            assert torch.equal(got_v, raw[1][0]) and torch.equal(v, raw[1])
            # K at position 0 is rounded (2^-8 of either element of a pair), and each side's result; angles below 2^-20
            mag = raw[0][0].double().abs().unflatten(-1, (-1, 2)).sum(-1, keepdim=True).expand(-1, -1, 2).flatten(-2)
            assert ((got_k.double() - k[0].double()).abs() <= mag * (2.0 ** -8 + 2.0 ** -20) + 2 * plain.bf16_bound(k[0].double()) * 1.01).all(), p
        mk.check_status(st)


@pytest.mark.parametrize("lens", [[513, 1400], [512, 100], [1500]])
def test_agrees_with_the_decode_steps_sliding_layers(lens):
    """As test_agrees_with_the_decode_step, in a layer that sees a window of 512."""
    import dataclasses

    import synth
    import synth.device
    sh = dataclasses.replace(synth.MODELS["dense"], n_layers=1)
    assert sh.window == 512 and not sh.is_full_layer(0)
    B, P = len(lens), sh.page_size
    need = [-(-n // P) for n in lens]
    ids = torch.randperm(sum(need), generator=torch.Generator().manual_seed(4)).tolist()
    bt = ints([[ids.pop() for _ in range(n)] + [-1] * (max(need) - n) for n in need])
    kp, vp = synth.device.device_pools(sh, 4, sum(need))
    sess, sl = decode_setup(sh, 4, B, max(lens)), ints(lens)
    sess.step(ints([3 + 5 * b for b in range(B)]), sl, bt, kp, vp, torch.empty(B, sh.vocab, device=DEV))
    sess.check()
    q, attn = (sess.region(x, torch.float32, B * sh.n_q * sh.head_dim).view(B, sh.n_q, sh.head_dim) for x in ("q", "attn_out"))
    cache, st = mk.KvCache(kp, vp, sh.rope_base), new_status()
    qb = q.to(BF)
    out = torch.empty_like(qb)
    ws = torch.empty(mk.tree_attn_workspace_bytes(cache), dtype=torch.uint8, device=DEV)
    mk.tree_attn(cache, 0, qb, out, ints(list(range(B + 1))), sl - 1, bt, ws, window=sh.window, status=st)
    mk.check_status(st)
    kc, vc = (x.view(BF)[0].cpu() for x in (kp, vp))
    for b, n in enumerate(lens):
        k, v = plain.gather_slots(kc, bt[b].tolist(), n), plain.gather_slots(vc, bt[b].tolist(), n)
        ref, _, spread, size = plain.attention(q[b].cpu(), k, v, torch.arange(n) > n - 1 - sh.window, 1 / math.sqrt(sh.head_dim))
        tol = plain.bf16_bound(ref) + spread * (2.0 ** -8 + 2 * size[:, None] * 2.0 ** -8)
        assert ((out[b].cpu().double() - ref).abs() <= tol).all()
        assert ((attn[b].cpu().double() - ref).abs() <= tol).all()
