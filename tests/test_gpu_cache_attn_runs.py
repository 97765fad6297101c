"""GPU parity of cp_cache_attn and cp_cache_attn_partial where a CTA gets many key tiles: the
second warpgroup's accumulator, maxima that grow within a run, the ring of tiles and the barriers
reused from unit to unit, units cut at both ends of a CTA's run, and the empty slots that stand
for a unit's start from two tiles per SM on.

Reference: the formula in 64 bits, one product per sequence and key/value head.

Tolerances, from the arithmetic, per row. A score is off by e and an output by the products of P
as in test_gpu_cache_attn.py: e = (D / 16) 2^-23 scale sum |q k| of the row's largest, 2^-22 of
the score (at most X) for the scaling, 2^-20 for the exponential, 2^-17 for P in two bf16 terms. What
long runs add, in a run of R tiles of 128 keys of a warpgroup: the exponent's argument, a fused
product of a score in log2 units and the maximum, is rounded to 2^-24 of it, and arguments below
-40 have no weight: 40 ln 2 2^-24 < 2^-19; a sum of 64 exponentials of a tile adds 64 roundings, and
each tile at most one more, and a rescaling by an approximate power of two (2^-22) and its
rounding: (64 + 6 R) 2^-24; the tensor core adds P V, which may truncate by 2^-23 of the sum of
|P V|, 16 times a tile, and the rescaling of the accumulator counts once more per tile:
(16 2 + 6) R 2^-24; and the pieces of a unit, joined by at most J of them: 6 J 2^-24. So with
    w = e + 2^-22 X + 2^-20 + 2^-19 + (64 + 6 R + 6 J) 2^-24
|lse - ref| <= w + 2^-22 |ref| and |o - ref| <= (2 w + 2^-17 + (38 R + 6 J) 2^-24) max |v|, and
half a step, 2^-8 |ref|, where it is bf16."""
import pytest
import torch

import context_long_sequence_cp_b200 as cp

pytestmark = pytest.mark.gpu

TILE = 128


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def tree_words(B, T, g):
    """Random trees: token t sees its ancestors and itself."""
    words = torch.zeros(B, T, dtype=torch.int64)
    for b in range(B):
        for t in range(T):
            up = int(torch.randint(-1, t, (1,), generator=g)) if t else -1
            w = ((int(words[b, up]) if up >= 0 else 0) | 1 << t) & (2 ** 64 - 1)
            words[b, t] = w - 2 ** 64 if w >= 2 ** 63 else w
    return words


def reference(q, k, v, lengths, words):
    """(o [B, T, Hq, D], lse [B, Hq, T], largest |score|, largest scale sum |q k|, largest |v|)."""
    B, T, Hq, D = q.shape
    Hkv = k.shape[2]
    G = Hq // Hkv
    o = torch.zeros(B, T, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq, T), -torch.inf, dtype=torch.float64, device="cuda")
    u = torch.arange(T, device="cuda")
    top, mag, vmax = 0.0, 0.0, 0.0
    for b, n in enumerate(lengths):
        drafted = (words[b].cuda()[:, None] >> u) & 1 == 1                           # [T, T]
        seen = torch.cat([torch.ones(T, n, dtype=torch.bool, device="cuda"), drafted], 1)
        for h in range(Hkv):
            kk, vv = k[b, :n + T, h].double(), v[b, :n + T, h].double()
            qq = q[b, :, h * G:(h + 1) * G].double().reshape(T * G, D)
            s = (qq @ kk.T / D ** 0.5).reshape(T, G, -1)
            mag = max(mag, float((qq.abs() @ kk.abs().T).max()) / D ** 0.5)
            top, vmax = max(top, float(s.abs().max())), max(vmax, float(vv.abs().max()))
            s = torch.where(seen[:, None], s, -torch.inf)
            lse[b, h * G:(h + 1) * G] = torch.logsumexp(s, -1).T
            o[b, :, h * G:(h + 1) * G] = torch.softmax(s, -1) @ vv
    return o, lse, top, mag, vmax


def check(q, k, v, lengths, words, run, pieces):
    """Both entry points against the reference; `run`: tiles of a warpgroup in one CTA at most."""
    B, T, Hq, D = q.shape
    plan = cp.CachePlan(B, Hq, k.shape[2], D, k.shape[1], T)
    dev = [t.cuda() for t in (q, k, v)] + [torch.tensor(lengths, dtype=torch.int32, device="cuda")]
    o, lse = cp.cache_attn(plan, *dev, tree=words.cuda())
    op, lp = cp.cache_attn_partial(plan, *dev, own_drafts=True, tree=words.cuda())
    again = cp.cache_attn(plan, *dev, tree=words.cuda())
    assert cp.cache_check(plan) == 0
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])
    ref, ref_lse, top, mag, vmax = reference(*dev[:3], lengths, words)
    w = (D / 16) * 2.0 ** -23 * mag + 2.0 ** -22 * top + 2.0 ** -20 + 2.0 ** -19 + (64 + 6 * run + 6 * pieces) * 2.0 ** -24
    bound = (2 * w + 2.0 ** -17 + (38 * run + 6 * pieces) * 2.0 ** -24) * vmax
    err = (op.view(B, T, Hq, D).double() - ref).abs()
    assert torch.all(err <= bound), ("partial", float(err.max()), bound)
    err = (o.double() - ref).abs() - 2.0 ** -8 * ref.abs()
    assert torch.all(err <= bound), ("o", float(err.max()), bound)
    for got in (lse, lp.view(B, T, Hq).transpose(1, 2)):
        assert torch.equal(torch.isneginf(got), torch.isneginf(ref_lse))
        d = torch.where(torch.isneginf(ref_lse), 0.0, got.double() - ref_lse).abs()
        assert torch.all(d <= w + 2.0 ** -22 * torch.where(torch.isneginf(ref_lse), 0.0, ref_lse).abs()), float(d.max())


def tiles(lengths, T):
    return sum(-(-(n + T) // TILE) for n in lengths)


@pytest.mark.parametrize("D,Hq,Hkv,T", [(128, 8, 2, 5), (64, 6, 2, 21), (128, 4, 1, 1), (64, 16, 1, 8)])
def test_maxima_that_grow_within_a_run(D, Hq, Hkv, T):
    """Runs of 12 tiles per CTA whose rows' largest scores move by 9 log2 units, upwards in half of
    the rows and downwards in the others, every few tiles: in steps of five tiles, so that both
    warpgroups see each of them, and 18 units in all, so that what came before still counts."""
    per = 12
    n = per * sms() // Hkv * TILE - 37
    assert tiles([n], T) * Hkv >= (per - 1) * sms()
    g = torch.Generator().manual_seed(D + T)
    q = torch.randn(1, T, Hq, D, generator=g) * 0.5
    k, v = (torch.randn(1, n + T, Hkv, D, generator=g) for _ in range(2))
    # the first feature carries the level: a key's score moves by +- its level, in log2 units
    level = torch.tensor([0.0, 0.0, 9.0, 9.0, 18.0])[(torch.arange(n + T) // TILE) % 5]
    q[..., 0] = torch.where(torch.randn(1, T, Hq, generator=g) > 0, 1.0, -1.0) * 8.0
    k[..., 0] = (level * (0.6931471805599453 * D ** 0.5 / 8.0))[None, :, None]
    q, k, v = (t.to(torch.bfloat16) for t in (q, k, v))
    grow = k[0, ::TILE, 0, 0].float() * 8.0 / D ** 0.5 / 0.6931471805599453
    assert float(grow.max()) > 17 and float(grow[2] - grow[1]) > 8.5    # past the 8 units of a rescaling
    check(q, k, v, [n], tree_words(1, T, g), per // 2 + 1, sms())


@pytest.mark.parametrize("D", [64, 128])
def test_several_units_of_several_tiles_per_run(D):
    """Uneven lengths: two or three units of one to six tiles in each CTA's run, cut at both ends,
    and more than two tiles per SM (empty slots before each unit)."""
    B, Hkv, G, T = 64, 8, 2, 3
    g = torch.Generator().manual_seed(D)
    lengths = torch.randint(0, 700, (B,), generator=g).tolist()
    lengths[3], lengths[5], lengths[9] = 0, 125, 126                       # one tile, one tile exactly full, two
    total = tiles(lengths, T) * Hkv
    assert total >= 8 * sms() and B * Hkv >= 2 * sms()
    q = torch.randn(B, T, Hkv * G, D, generator=g).to(torch.bfloat16)
    k, v = (torch.randn(B, 720, Hkv, D, generator=g).to(torch.bfloat16) for _ in range(2))
    check(q, k, v, lengths, tree_words(B, T, g), 3, 2)


@pytest.mark.parametrize("more", [-1, 0, 1])
def test_both_sides_of_two_tiles_per_sm(more):
    """One tile fewer than two per SM, as many, one more: without and with the empty slots. Units
    of one to nine tiles, some of them whole in a CTA and others cut among several."""
    D, G, T, B = 128, 3, 2, 60
    want = 2 * sms() + more
    sizes = [1 + i % 9 for i in range(B)]
    sizes[-1] += want - sum(sizes)
    assert min(sizes) >= 1 and sum(sizes) == want
    lengths = [s * TILE - T - (7 * i) % 100 for i, s in enumerate(sizes)]
    assert tiles(lengths, T) == want
    g = torch.Generator().manual_seed(3 + more)
    q = torch.randn(B, T, G, D, generator=g).to(torch.bfloat16)
    k, v = (torch.randn(B, max(lengths) + T, 1, D, generator=g).to(torch.bfloat16) for _ in range(2))
    check(q, k, v, lengths, tree_words(B, T, g), 2, 16)


def test_one_token_of_each_sequence_over_long_caches():
    """Decoding: grouped heads, 24 sequences of up to 8k keys, one token each, some caches short."""
    B, Hq, Hkv, D, cap = 24, 8, 2, 128, 8192
    g = torch.Generator().manual_seed(8)
    lengths = [cap - 1 - 331 * b for b in range(B - 2)] + [0, 1]
    assert tiles(lengths, 1) * Hkv >= 8 * sms()
    q = torch.randn(B, 1, Hq, D, generator=g).to(torch.bfloat16)
    k, v = (torch.randn(B, cap, Hkv, D, generator=g).to(torch.bfloat16) for _ in range(2))
    check(q, k, v, lengths, tree_words(B, 1, g), 10, 8)
