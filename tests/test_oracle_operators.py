"""Pins of the oracles of multi-axis rotary, decayed linear attention and cache attention:
special cases in closed form, other oracles, finite differences, planted mistakes."""
import numpy as np
import pytest

from oracle import attention as A
from oracle import cache_attention as CA
from oracle import linear_attention as LA
from oracle import rope as R
from oracle import rope_axes as RA


# ------------------------------------------------------------------------- rope_axes
def test_one_axis_is_the_rope_oracle():
    x = np.random.default_rng(0).standard_normal((7, 3, 64))
    pos = np.array([0, 1, 2, 5, 77, 1000, 12345])
    got = RA.rotate(x, RA.angles(pos[None], [32], 64))
    # two ways to round theta (a few 2^-53): angles up to 12345 differ by less than 6e-12, times |x| < 5
    assert np.allclose(got, R.rope(x, pos), rtol=0, atol=3e-11)
    # one axis: both frequency readings are the same table
    assert np.allclose(RA.angles(pos[None], [32], 64, freqs="per_axis"), RA.angles(pos[None], [32], 64), rtol=1e-12)


@pytest.mark.parametrize("pairing", ["adjacent", "half"])
@pytest.mark.parametrize("freqs", ["shared", "per_axis"])
def test_rotation_keeps_norms_and_inverts(pairing, freqs):
    g = np.random.default_rng(1)
    x, pos = g.standard_normal((5, 2, 64)), g.integers(-50, 50, (3, 5))
    ang = RA.angles(pos, [8, 12, 12], 64, freqs=freqs)
    y = RA.rotate(x, ang, pairing)
    assert np.allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1))
    assert np.allclose(RA.rotate(y, ang, pairing, inverse=True), x)
    # scores depend on position differences axis by axis
    q, k = g.standard_normal((2, 1, 1, 64))
    dots = [np.sum(RA.rotate(q, RA.angles(p[:, None], [8, 12, 12], 64, freqs=freqs), pairing) *
                   RA.rotate(k, RA.angles(p[:, None] + np.array([[3], [-4], [9]]), [8, 12, 12], 64, freqs=freqs), pairing))
            for p in (np.array([0, 0, 0]), np.array([11, 5, -7]))]
    assert np.isclose(dots[0], dots[1])


def test_pairings_are_a_permutation_of_features():
    g = np.random.default_rng(2)
    x, pos = g.standard_normal((4, 2, 64)), g.integers(0, 99, (2, 4))
    ang = RA.angles(pos, [20, 12], 64)
    perm = np.concatenate([np.arange(0, 64, 2), np.arange(1, 64, 2)])
    assert np.allclose(RA.rotate(x, ang)[..., perm], RA.rotate(x[..., perm], ang, "half"))
    assert not np.allclose(RA.rotate(x, ang), RA.rotate(x, ang, "half"))


def test_per_axis_frequencies_restart():
    ang = RA.angles(np.ones((2, 1)), [16, 16], 64, freqs="per_axis")[0]
    assert np.allclose(ang[:16], ang[16:]) and ang[0] == 1.0 and np.isclose(ang[1], 10000.0 ** (-1 / 16))
    assert np.isclose(RA.angles(np.ones((2, 1)), [16, 16], 64)[0][16], 0.01)   # 10000^(-32/64)


# ------------------------------------------------------------------ linear attention
def _qkv(B, S, H, D, seed):
    g = np.random.default_rng(seed)
    return [g.standard_normal((B, S, H, D)) for _ in range(4)]


def test_linear_attention_is_the_masked_product():
    q, k, v, _ = _qkv(2, 9, 3, 4, 3)
    ld = np.log(np.array([1.0, 0.9, 0.3]))
    o, s = LA.forward(q, k, v, ld, 0.5)
    i = np.arange(9)
    for h in range(3):
        w = np.where(i[:, None] >= i[None], np.exp(ld[h]) ** np.maximum(i[:, None] - i[None], 0), 0.0)
        for b in range(2):
            assert np.allclose(o[b, :, h], 0.5 * ((q[b, :, h] @ k[b, :, h].T) * w) @ v[b, :, h])
            assert np.allclose(s[b, h], (k[b, :, h] * (np.exp(ld[h]) ** (8 - i))[:, None]).T @ v[b, :, h])


def test_linear_attention_decay_of_zero_sees_only_itself():
    q, k, v, _ = _qkv(1, 5, 1, 4, 4)
    o, s = LA.forward(q, k, v, np.array([-np.inf]), 1.0)
    assert np.allclose(o[0, :, 0], np.sum(q * k, -1)[0, :, 0, None] * v[0, :, 0])
    assert np.allclose(s[0, 0], np.outer(k[0, -1, 0], v[0, -1, 0]))


def test_linear_attention_splits_at_any_token():
    q, k, v, do = _qkv(1, 10, 2, 4, 5)
    ld, g = np.log(np.array([0.95, 0.5])), np.random.default_rng(6)
    s0, ds = g.standard_normal((1, 2, 4, 4)), g.standard_normal((1, 2, 4, 4))
    o, s = LA.forward(q, k, v, ld, 0.7, s0)
    o1, s1 = LA.forward(q[:, :3], k[:, :3], v[:, :3], ld, 0.7, s0)
    o2, s2 = LA.forward(q[:, 3:], k[:, 3:], v[:, 3:], ld, 0.7, s1)
    assert np.allclose(np.concatenate([o1, o2], 1), o) and np.allclose(s2, s)
    whole = LA.backward(q, k, v, ld, 0.7, do, s0, ds)
    late = LA.backward(q[:, 3:], k[:, 3:], v[:, 3:], ld, 0.7, do[:, 3:], s1, ds)
    early = LA.backward(q[:, :3], k[:, :3], v[:, :3], ld, 0.7, do[:, :3], s0, late[3])
    for w, e, l in zip(whole[:3], early[:3], late[:3]):
        assert np.allclose(np.concatenate([e, l], 1), w)
    assert np.allclose(early[3], whole[3])


def test_linear_attention_gradients_against_differences():
    q, k, v, do = _qkv(1, 6, 2, 3, 7)
    ld, g = np.log(np.array([0.9, 0.4])), np.random.default_rng(8)
    s0, ds = g.standard_normal((1, 2, 3, 3)), g.standard_normal((1, 2, 3, 3))

    def loss(q, k, v, s0):
        o, s = LA.forward(q, k, v, ld, 0.6, s0)
        return np.sum(o * do) + np.sum(s * ds)

    args, grads, eps = [q, k, v, s0], LA.backward(q, k, v, ld, 0.6, do, s0, ds), 1e-5
    for a, (x, dx) in enumerate(zip(args, grads)):
        for _ in range(12):
            at = tuple(g.integers(0, n) for n in x.shape)
            up, down = [y.copy() for y in args], [y.copy() for y in args]
            up[a][at] += eps
            down[a][at] -= eps
            # the loss is at most quadratic in one entry: central differences are exact but for rounding
            assert np.isclose((loss(*up) - loss(*down)) / (2 * eps), dx[at], rtol=1e-6, atol=1e-7)


# -------------------------------------------------------------------- cache attention
def test_chain_over_a_cache_is_causal_attention():
    g = np.random.default_rng(9)
    q, k, v = (g.standard_normal((1, 12, 2, 8)) for _ in range(3))
    o_ref, lse_ref = A.attention(q, k, v, causal=True)
    o, lse = CA.attend(q[:, 7:], k, v, [7])
    assert np.allclose(o, o_ref[:, 7:]) and np.allclose(lse, lse_ref[:, :, 7:])


def test_tree_words_pick_rows_and_groups_share_keys():
    g = np.random.default_rng(10)
    q, k, v = g.standard_normal((1, 3, 4, 8)), g.standard_normal((1, 9, 2, 8)), g.standard_normal((1, 9, 2, 8))
    o, lse = CA.attend(q, k, v, [5], [[0b001, 0b011, 0b101]])
    # token 2 sees token 0 and itself, not token 1: rows 0-4, 5 and 7
    rows = [0, 1, 2, 3, 4, 5, 7]
    s = k[0, rows, 1] @ q[0, 2, 3] / np.sqrt(8)
    p = np.exp(s) / np.exp(s).sum()
    assert np.allclose(o[0, 2, 3], p @ v[0, rows, 1]) and np.isclose(lse[0, 3, 2], np.log(np.exp(s).sum()))


def test_empty_rows_and_unread_rows():
    g = np.random.default_rng(11)
    q, k, v = (g.standard_normal((2, 2, 1, 4)) for _ in range(3))
    k[0, :], v[1, 1] = np.nan, np.nan
    o, lse = CA.attend(q, k, v, [0, 1], own_drafts=False)
    assert np.all(o[0] == 0) and np.all(np.isneginf(lse[0])) and np.allclose(o[1], v[1, 0])
    o, lse = CA.attend(q[1:], k[1:], v[1:, :1].repeat(2, 1), [0], [[0, 1]])
    assert np.all(o[0, 0] == 0) and np.isneginf(lse[0, 0, 0]) and np.isfinite(lse[0, 0, 1])


def test_split_cache_merges_to_the_whole():
    g = np.random.default_rng(12)
    q, k, v = g.standard_normal((1, 3, 2, 4)), g.standard_normal((1, 11, 2, 4)), g.standard_normal((1, 11, 2, 4))
    o, lse = CA.attend(q, k, v, [8])
    a = CA.attend(q, k[:, :5], v[:, :5], [5], own_drafts=False)
    b = CA.attend(q, k[:, 5:], v[:, 5:], [3])
    m, l = A.merge([(x[0].reshape(-1, 4), x[1].transpose(0, 2, 1).reshape(-1)) for x in (a, b)])
    assert np.allclose(m, o.reshape(-1, 4)) and np.allclose(l, lse.transpose(0, 2, 1).reshape(-1))


def test_planted_mistakes_are_seen():
    q, k, v, _ = _qkv(1, 6, 1, 4, 13)
    ld = np.log(np.array([0.8]))
    o, s = LA.forward(q, k, v, ld, 1.0)
    late = LA.forward(q, np.roll(k, 1, 1), v, ld, 1.0)[0]                 # keys one token late
    assert not np.allclose(o, late)
    assert not np.allclose(o[:, 1:], LA.forward(q, k, v, ld / 2, 1.0)[0][:, 1:])
