"""The operators on tensors of more than 2^31 elements: offsets that pass 32 bits."""
import numpy as np
import pytest
import torch

import context_long_sequence_cp_b200 as cp

pytestmark = pytest.mark.gpu

B, S, H, D = 5, 131072, 32, 128   # 2.7e9 elements, 5.4 GB in bf16


@pytest.fixture(scope="module")
def plan():
    assert B * S * H * D > 2 ** 31
    return cp.Plan(B, H, S, D, 1, True, "contiguous")


def _randn(shape, seed):
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(seed))


def test_rope_axes(plan):
    """A token's rotation depends on its positions alone: the last tokens equal a short call's."""
    x = _randn((B, S, H, D), 1)
    pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (2, B, S), dtype=torch.int32, device="cuda")
    n = 96
    short = cp.Plan(1, H, n, D, 1, True, "contiguous")
    args = dict(sections=[40, 24], freqs="per_axis", pairing="half")
    y = cp.rope_axes(plan, x, pos, **args)
    want = cp.rope_axes(short, x[-1:, -n:].contiguous(), pos[:, -1:, -n:].contiguous(), **args)
    assert torch.equal(y.view(B, S, H, D)[-1, -n:], want.view(n, H, D))
    back = cp.rope_axes(plan, y, pos, inverse=True, **args)
    want = cp.rope_axes(short, want, pos[:, -1:, -n:].contiguous(), inverse=True, **args)
    assert torch.equal(back[-1, -n:], want.view(n, H, D))


def test_linear_attention_forward_and_backward(plan):
    """Decays of e^-0.05 a token: what is 1500 tokens away counts e^-75, less than any rounding."""
    q, k, v, do = (_randn((1, B, S, H, D), s) for s in (2, 3, 4, 5))
    ld = torch.full((H,), -0.05, device="cuda")
    o, _ = cp.linattn_fwd(plan, q, k, v, ld)
    dq, dk, dv, _ = cp.linattn_bwd(plan, q, k, v, ld, do)
    assert cp.check(plan) == 0
    W, b, h = 1600, B - 1, H - 1
    i = torch.arange(W, dtype=torch.float64)
    m = torch.tril(torch.exp(-0.05 * (i[:, None] - i))) / D ** 0.5
    last = {n: t[0, b, -W:, h].double().cpu() for n, t in dict(q=q, k=k, v=v, do=do).items()}
    s, p = (last["q"] @ last["k"].T) * m, (last["do"] @ last["v"].T) * m
    for name, got, left, right in (("o", o, s, "v"), ("dq", dq, p, "k"), ("dk", dk, p.T, "q"), ("dv", dv, s.T, "do")):
        ref, mag = (left @ last[right])[-64:], (left.abs() @ last[right].abs())[-64:]   # rows next to the end
        err = (got[0, b, -64:, h].double().cpu() - ref).abs()
        # bf16 roundings of the scores or state and of the output, fp32 arithmetic below 2^-15
        assert torch.all(err <= 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -15) * (1 + 2.0 ** -8) * mag), name


def test_cache_attention():
    """A key of the last head near the cache's end that outweighs a million others by e^26."""
    cap, Hkv, T, row = 1_100_000, 16, 2, 1_090_000
    assert row * Hkv * D > 2 ** 31
    k, v = (torch.zeros(1, cap, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = torch.full((1, T, Hkv, D), 1.0, dtype=torch.bfloat16, device="cuda")
    k[0, row, Hkv - 1] = 3.625                                    # score 3.625 sqrt(128) = 41.01
    want = _randn((D,), 6)
    v[0, row, Hkv - 1] = want
    plan = cp.CachePlan(1, Hkv, Hkv, D, cap, T)
    o, lse = cp.cache_attn(plan, q, k, v, torch.tensor([cap - T], dtype=torch.int32, device="cuda"))
    assert cp.cache_check(plan) == 0
    # the others' weight is 1.1e6 e^-41 = 1.7e-12 and P is kept to 2^-17: a bf16 value plus less than half a step
    assert torch.all((o[0, :, -1].float() - want.float()).abs() <= 2.0 ** -8 * want.float().abs())
    assert torch.all(o[0, :, :-1] == 0)
    lse = lse.double().cpu().numpy()[0]
    assert np.all(np.abs(lse[-1] - 3.625 * 128 ** 0.5) <= 2.0 ** -22 * 41.1 + 2.0 ** -20 + 8 * 2.0 ** -23 * 41.1)
    # 59 tiles a run and 128 keys a tile: fewer than 8192 additions to a row's sum, each off by 2^-24 of it
    seen = np.log(cap - T + 1 + np.arange(T))
    assert np.all(np.abs(lse[:-1] - seen) <= 2.0 ** -20 + 2.0 ** -22 * 14 + 8192 * 2.0 ** -24)
