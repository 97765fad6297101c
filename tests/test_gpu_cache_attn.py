"""GPU parity of attention over a key/value cache (cp_cache_attn, cp_cache_attn_partial)
with the fp64 oracle.

Tolerances, from the arithmetic: a score is an fp32 sum of D exact products, which the
tensor core adds 16 at a time and may truncate by 2^-23 of the running sum, so it is off
by at most e = (D / 16) 2^-23 scale sum |q k| (largest over rows), plus 2^-22 |score| of
the scaling; exponentials carry 2^-21, and P is kept to 2^-17 in two bf16 terms. So
|lse - ref| <= e + 2^-22 |ref| + 2^-20, and an output is off by at most
2 (e + 2^-17 + 2^-20) max |v| and, where it is bf16, half a step: 2^-8 |ref|.
"""
import numpy as np
import pytest
import torch

import context_long_sequence_cp_b200 as cp
from oracle import cache_attention as CA

pytestmark = pytest.mark.gpu

JUNK = float("nan")


def case(B, T, Hq, Hkv, D, cap, lengths, seed=0, tree=True):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(B, T, Hq, D, generator=g).to(torch.bfloat16)
    k, v = (torch.randn(B, cap, Hkv, D, generator=g).to(torch.bfloat16) for _ in range(2))
    for b, n in enumerate(lengths):   # rows past the drafted ones were never written
        k[b, n + T:] = JUNK
        v[b, n + T:] = JUNK
    words = None
    if tree:
        words = torch.zeros(B, T, dtype=torch.int64)
        for b in range(B):
            for t in range(T):
                up = int(torch.randint(-1, t, (1,), generator=g)) if t > 0 else -1
                w = (int(words[b, up]) if up >= 0 else 0) & (2 ** 64 - 1) | 1 << t
                words[b, t] = w - 2 ** 64 if w >= 2 ** 63 else w
    return q, k, v, torch.tensor(lengths, dtype=torch.int32), words


def slack(q, k, v, lengths, T):
    """(score error e, max |v|) over the rows that are seen."""
    D, G, e, top = q.shape[-1], q.shape[2] // k.shape[2], 0.0, 0.0
    for b, n in enumerate(lengths):
        m = n + T
        kk = k[b, :m].abs().float().repeat_interleave(G, 1)
        if m:
            e = max(e, float(torch.einsum("thd,shd->ths", q[b].abs().float(), kk).max()))
            top = max(top, float(v[b, :m].abs().max()))
    return (D / 16) * 2.0 ** -23 * e / D ** 0.5, top


def assert_close(o, lse, ref, q, k, v, lengths, T, bf16=True):
    e, top = slack(q, k, v, [int(n) for n in lengths], T)
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    err = np.abs(o - ref[0])
    bound = 2 * (e + 2.0 ** -17 + 2.0 ** -20) * top + (2.0 ** -8 * np.abs(ref[0]) if bf16 else 0.0)
    assert np.all(err <= bound), float((err - bound).max())
    none = np.isneginf(ref[1])
    assert np.array_equal(none, np.isneginf(lse))
    d, r = np.abs(lse[~none] - ref[1][~none]), np.abs(ref[1][~none])
    assert np.all(d <= e + 2.0 ** -22 * r + 2.0 ** -20), float(d.max())


def words_of(tree):
    return None if tree is None else [[int(w) & (2 ** 64 - 1) for w in row] for row in tree.tolist()]


@pytest.mark.parametrize("B,T,Hq,Hkv,D,cap,lengths,tree", [
    (1, 1, 1, 1, 64, 1, (0,), False),                        # one token, an empty cache
    (2, 1, 4, 4, 128, 130, (127, 128), False),               # the new key at a tile's end and start
    (3, 3, 6, 2, 64, 300, (0, 126, 297), True),              # drafted keys across a tile's border; a full cache
    (1, 64, 2, 1, 128, 200, (100,), True),                   # the most drafted tokens, 128 rows
    (1, 64, 12, 4, 64, 1000, (700,), True),                  # 192 rows: two query tiles
    (2, 5, 35, 5, 128, 600, (513, 1), True),                 # 7 heads a group: 18 tokens would fit
    (1, 2, 128, 1, 64, 500, (333,), True),                   # 128 heads a group: a tile per token
    (4, 16, 8, 2, 128, 2100, (0, 2084, 5, 1000), True),      # uneven
    (1, 7, 4, 1, 128, 9000, (8990,), False),                 # one unit cut among many CTAs, a chain
    (5, 1, 2, 2, 64, 700, (1, 2, 3, 64, 699), False),
    (40, 2, 2, 1, 64, 40, tuple(range(0, 38)) + (0, 38), True),
])
def test_matches_oracle(B, T, Hq, Hkv, D, cap, lengths, tree):
    q, k, v, n, words = case(B, T, Hq, Hkv, D, cap, lengths, seed=cap + T, tree=tree)
    plan = cp.CachePlan(B, Hq, Hkv, D, cap, T)
    dev = [t.cuda() for t in (q, k, v, n)]
    w = None if words is None else words.cuda()
    o, lse = cp.cache_attn(plan, *dev, tree=w)
    assert cp.cache_check(plan) == 0
    ref = CA.attend(q.double().numpy(), k.double().numpy(), v.double().numpy(), lengths, words_of(words))
    assert_close(o, lse, ref, q, k, v, lengths, T)
    again = cp.cache_attn(plan, *dev, tree=w)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])
    # the partial form: the same rows in fp32
    op, lp = cp.cache_attn_partial(plan, *dev, own_drafts=True, tree=w)
    assert_close(op.view(B, T, Hq, D), lp.view(B, T, Hq).transpose(1, 2), ref, q, k, v, lengths, T, bf16=False)


def test_divided_cache_merges_to_the_whole():
    """Context-parallel ranks hold parts of the cache, the last one the drafted rows too."""
    B, T, Hq, Hkv, D = 2, 3, 8, 2, 128
    lengths, cuts = (700, 150), ((0, 300, 600), (0, 0, 100))
    q, k, v, n, words = case(B, T, Hq, Hkv, D, 800, lengths, seed=3)
    parts = []
    for r in range(3):
        last = r == 2
        ks, vs = (torch.full((B, 400, Hkv, D), JUNK, dtype=torch.bfloat16) for _ in range(2))
        ns = []
        for b in range(B):
            lo, hi = cuts[b][r], lengths[b] if last else cuts[b][r + 1]
            rows = hi - lo + (T if last else 0)
            ks[b, :rows], vs[b, :rows] = k[b, lo:lo + rows], v[b, lo:lo + rows]
            ns.append(hi - lo)
        plan = cp.CachePlan(B, Hq, Hkv, D, 400, T)
        parts.append(cp.cache_attn_partial(plan, q.cuda(), ks.cuda(), vs.cuda(), torch.tensor(ns, dtype=torch.int32).cuda(),
                                           own_drafts=last, tree=words.cuda() if last else None))
        assert cp.cache_check(plan) == 0
    o, lse = cp.merge_partials(torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts]))
    ref = CA.attend(q.double().numpy(), k.double().numpy(), v.double().numpy(), lengths, words_of(words))
    assert_close(o.view(B, T, Hq, D), lse.view(B, T, Hq).transpose(1, 2), ref, q, k, v, lengths, T)
    # a rank that holds nothing: all rows empty
    empty = parts[0][1].view(B, T, Hq)[1]
    assert torch.all(torch.isneginf(empty)) and torch.all(parts[0][0].view(B, T, Hq, D)[1] == 0)


def test_masked_rows_of_every_kind():
    """Words without bits, bits past T, stale infinities and NaNs past the last key, a cache's
    lowest values, and lengths outside the cache (NaN, the neighbours untouched)."""
    B, T, Hq, Hkv, D, cap = 5, 2, 2, 1, 64, 200
    lengths = [0, 60, -1, cap - 1, 130]
    q, k, v, _, _ = case(B, T, Hq, Hkv, D, cap, (0, 60, 0, 0, 130), seed=8, tree=False)
    k[1, 62:], v[1, 62:] = float("inf"), -float("inf")
    k[4, :130] = torch.finfo(torch.bfloat16).min            # scores of -inf and inf
    q[4] = q[4].abs()
    tree = torch.tensor([[0, 2], [1, 3], [1, 3], [1, 3], [1 | 1 << 40, 3 | 1 << 63 - 1]], dtype=torch.int64)
    plan = cp.CachePlan(B, Hq, Hkv, D, cap, T)
    o, lse = cp.cache_attn(plan, q.cuda(), k.cuda(), v.cuda(), torch.tensor(lengths, dtype=torch.int32).cuda(), tree.cuda())
    assert cp.cache_check(plan) == 0
    o, lse = o.cpu(), lse.cpu()
    assert torch.all(o[0, 0] == 0) and torch.all(torch.isneginf(lse[0, :, 0]))      # sees nothing at all
    assert torch.isfinite(o[0, 1].float()).all() and torch.isfinite(lse[0, :, 1]).all()
    ref = CA.attend(q[:2].double().numpy(), k[:2].double().numpy(), v[:2].double().numpy(), lengths[:2], words_of(tree[:2]))
    assert_close(o[:2], lse[:2], ref, q[:2], k[:2, :62], v[:2, :62], lengths[:2], T)
    for b in (2, 3):
        assert torch.all(torch.isnan(o[b].float())) and torch.all(torch.isnan(lse[b]))
    # the cached keys' scores are about -1e39 or lower: only the drafted rows count, bits past T do not
    ref = CA.attend(q[4:].double().numpy(), k[4:, 130:].double().numpy(), v[4:, 130:].double().numpy(), [0], [[1, 3]])
    assert_close(o[4:], lse[4:], ref, q[4:], k[4:, 130:132], v[4:, 130:132], [0], T)


@pytest.mark.parametrize("T,used,n", [(20, 13, 100), (64, 3, 120), (64, 40, 128), (2, 0, 0), (64, 63, 200)])
def test_padding_of_a_short_tree_may_hold_anything(T, used, n):
    """Drafted tokens that no token sees: their words are 0 and their rows were never written,
    in the tile that holds the last cached key and in the one after."""
    B, Hq, Hkv, D, cap = 2, 4, 2, 128, 400
    q, k, v, lens, words = case(B, T, Hq, Hkv, D, cap, (n, n + 5), seed=T + used)
    for b, m in enumerate((n, n + 5)):
        k[b, m + used:], v[b, m + used:], words[b, used:] = JUNK, JUNK, 0
    hole = 1 if used > 2 else None                                  # a token that only itself would see
    if hole is not None:
        words &= ~(1 << hole)
        k[0, n + hole], v[0, n + hole] = JUNK, JUNK
    plan = cp.CachePlan(B, Hq, Hkv, D, cap, T)
    o, lse = cp.cache_attn(plan, q.cuda(), k.cuda(), v.cuda(), lens.cuda(), words.cuda())
    assert cp.cache_check(plan) == 0
    clean = [torch.where(torch.isnan(x), torch.zeros_like(x), x) for x in (k, v)]
    ref = CA.attend(q.double().numpy(), *(x.double().numpy() for x in clean), lens.tolist(), words_of(words))
    assert_close(o, lse, ref, q, *clean, lens, T)


def test_lengths_grow_on_the_device_in_a_graph():
    """Decoding as a captured step: the lengths are device memory, the replays follow them."""
    B, T, Hq, Hkv, D, cap = 2, 1, 8, 2, 64, 600
    q, k, v, _, _ = case(B, T, Hq, Hkv, D, cap, (cap - 1, cap - 1), seed=4, tree=False)
    plan = cp.CachePlan(B, Hq, Hkv, D, cap, T)
    dev = [t.cuda() for t in (q, k, v)]
    n = torch.tensor([125, 300], dtype=torch.int32, device="cuda")
    cp.cache_attn(plan, *dev, n)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = cp.cache_attn(plan, *dev, n)
        n.add_(1)
    n.copy_(torch.tensor([125, 300], dtype=torch.int32))
    for step in range(6):
        graph.replay()
        torch.cuda.synchronize()
        lens = [125 + step, 300 + step]
        ref = CA.attend(q.double().numpy(), k.double().numpy(), v.double().numpy(), lens)
        assert_close(o, lse, ref, q, k, v, lens, T)
    assert cp.cache_check(plan) == 0


def test_streams_and_given_outputs():
    B, T, Hq, Hkv, D, cap = 3, 4, 8, 4, 128, 3000
    sets = [case(B, T, Hq, Hkv, D, cap, ls, seed=i) for i, ls in enumerate(((2990, 17, 1500), (5, 2000, 800)))]
    sets = [[t.cuda() for t in s] for s in sets]
    plan = cp.CachePlan(B, Hq, Hkv, D, cap, T)
    refs = [cp.cache_attn(plan, *s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [(i, cp.cache_attn(plan, *sets[i], stream=streams[i])) for _ in range(8) for i in range(2)]
    torch.cuda.synchronize()
    assert cp.cache_check(plan) == 0
    for i, (o, lse) in got:
        assert torch.equal(o, refs[i][0]) and torch.equal(lse, refs[i][1])
    o, lse = torch.empty_like(refs[0][0]), torch.empty_like(refs[0][1])
    ws = torch.empty(plan.workspace_bytes(), dtype=torch.uint8, device="cuda")
    a, b = cp.cache_attn(plan, *sets[0], o=o, lse=lse, workspace=ws)
    assert a is o and b is lse and torch.equal(o, refs[0][0]) and torch.equal(lse, refs[0][1])


def test_same_as_the_fused_forward_on_a_full_context():
    """A chain of the last 64 tokens over the tokens before them is the tail of causal attention."""
    B, H, S, D, T = 1, 4, 512, 128, 64
    g = torch.Generator().manual_seed(11)
    q, k, v = (torch.randn(B, S, H, D, generator=g).to(torch.bfloat16) for _ in range(3))
    plan = cp.Plan(B, H, S, D, 1, True, "contiguous")
    o_full, lse_full = cp.attn_fwd(plan, *(t[None].cuda() for t in (q, k, v)))
    c = cp.CachePlan(B, H, H, D, S, T)
    o, lse = cp.cache_attn(c, q[:, S - T:].contiguous().cuda(), k.cuda(), v.cuda(),
                           torch.tensor([S - T], dtype=torch.int32, device="cuda"))
    ref = CA.attend(q[:, S - T:].double().numpy(), k.double().numpy(), v.double().numpy(), [S - T])
    assert_close(o, lse, ref, q[:, S - T:], k, v, [S - T], T)
    # the fused forward keeps P in one bf16 term: its own tolerance
    assert torch.max(torch.abs(o_full[0, :, S - T:].float() - o.float())) <= 2e-2
    assert torch.max(torch.abs(lse_full[:, :, S - T:] - lse)) <= 1e-3


def test_overlapping_buffers_are_refused():
    """Outputs and the workspace over the cache, the lengths, the words, the queries or one another."""
    B, T, Hq, Hkv, D, cap = 2, 3, 4, 2, 64, 300
    q, k, v, n, words = (t.cuda() for t in case(B, T, Hq, Hkv, D, cap, (200, 297), seed=1))
    plan = cp.CachePlan(B, Hq, Hkv, D, cap, T)
    rows = B * T * Hq
    o, lse = torch.empty(2 * rows * D, device="cuda"), torch.empty(rows, device="cuda")
    ws = torch.empty(plan.workspace_bytes(), dtype=torch.uint8, device="cuda")
    p = {name: t.data_ptr() for name, t in dict(q=q, k=k, v=v, n=n, words=words, o=o, lse=lse, ws=ws).items()}

    def whole(**over):
        a = {**p, **over}
        return cp.lib().cp_cache_attn(plan.handle, a["q"], a["k"], a["v"], a["n"], a["words"], a["o"], a["lse"], a["ws"], None)

    def part(**over):
        a = {**p, **over}
        return cp.lib().cp_cache_attn_partial(plan.handle, a["q"], a["k"], a["v"], a["n"], 1, a["words"], a["o"], a["lse"],
                                              a["ws"], None)
    end_k, end_v = p["k"] + 2 * k.numel(), p["v"] + 2 * v.numel()
    for call in (whole, part):
        assert call() == 0
        for bad in (dict(o=p["k"]), dict(o=end_v - 16), dict(lse=end_k - 4), dict(ws=p["v"]), dict(ws=p["q"]),
                    dict(o=p["n"]), dict(lse=p["n"]), dict(ws=p["words"]), dict(lse=p["o"] + 64), dict(o=p["ws"] + 1024),
                    dict(lse=p["ws"]), dict(o=p["q"] + 16), dict(lse=p["q"])):
            assert call(**bad) == -1, bad
    assert part(o=p["q"]) == -1                                   # fp32 rows are twice as long
    torch.cuda.synchronize()
    assert cp.cache_check(plan) == 0


@pytest.mark.parametrize("lengths", [(200, 297, 0), (8000, 3, 4000), (60, 61, 62)])
def test_output_in_place_of_the_queries(lengths):
    """Units whole in a CTA and cut among several, two query tiles per head: the same bits."""
    B, T, Hq, Hkv, D = 3, 40, 8, 2, 128
    q, k, v, n, words = (t.cuda() for t in case(B, T, Hq, Hkv, D, max(lengths) + T, lengths, seed=2))
    plan = cp.CachePlan(B, Hq, Hkv, D, max(lengths) + T, T)
    o, lse = cp.cache_attn(plan, q, k, v, n, words)
    for _ in range(5):
        mine = q.clone()
        got, l2 = cp.cache_attn(plan, mine, k, v, n, words, o=mine)
        assert got is mine and torch.equal(mine, o) and torch.equal(l2, lse)
    assert cp.cache_check(plan) == 0
