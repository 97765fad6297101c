"""The rotary map, linear attention and cache attention as a model uses them: a hybrid of
one linear and one softmax layer on image-like positions, trained, and then served from a
prompt through a tree of drafted tokens."""
import numpy as np
import pytest
import torch

import context_long_sequence_cp_b200 as cp
from oracle import attention as A
from oracle import cache_attention as CA
from oracle import linear_attention as LA
from oracle import rope_axes as RA
from tests import gpu_util as G

pytestmark = pytest.mark.gpu

B, H, S, D, N, SECTIONS = 1, 4, 384, 64, 2, (8, 12, 12)


def grid_positions(n):
    """time, height, width of n tokens of 8 x 6 frames."""
    i = np.arange(n)
    return np.stack([i // 48, i // 6 % 8, i % 6]).astype(np.int32)[:, None]


def f64(t):
    return t.double().cpu().numpy()


def rel(x, ref):
    return np.linalg.norm(f64(x) - ref) / np.linalg.norm(ref)


def test_hybrid_layers_forward_and_backward():
    """rope -> linear attention -> rope -> softmax attention on zigzag ranks, and back. Each
    stage takes the GPU's own input, so its error is its own: bf16 operands and outputs, at most
    three roundings of relative rms 2^-8 / sqrt(3), below 2^-7 in all."""
    g = torch.Generator().manual_seed(1)
    x, k, v, dy = ((torch.randn(B, S, H, D, generator=g) * s).to(torch.bfloat16).cuda() for s in (0.5, 0.5, 1.0, 1.0))
    ld = torch.tensor([-0.03, -0.01, -0.003, -0.5], device="cuda")
    pos = torch.from_numpy(grid_positions(S)).cuda()
    ang = RA.angles(grid_positions(S), SECTIONS, D)
    plan = cp.Plan(B, H, S, D, N, True, "zigzag")
    nat = lambda t: G.from_layout(t, N, "zigzag")
    qr, kr = (cp.rope_axes(plan, t, pos, SECTIONS) for t in (x, k))
    vr = cp.layout_permute(plan, v, 0).view_as(qr)
    mid, state = cp.linattn_fwd(plan, qr, kr, vr, ld, want_state=True)
    back = cp.layout_permute(plan, mid, 1).view(B, S, H, D)
    q2 = cp.rope_axes(plan, back, pos, SECTIONS)
    o, lse = cp.attn_fwd(plan, q2, kr, vr)
    assert cp.check(plan) == 0
    assert rel(nat(qr), RA.rotate(f64(x), ang)) <= 2.0 ** -8
    ref_mid, ref_s = LA.forward(f64(nat(qr)), f64(nat(kr)), f64(v), f64(ld), plan.scale)
    assert rel(nat(mid), ref_mid) <= 2.0 ** -7 and rel(state, ref_s) <= 1e-6
    ref_o, _ = A.attention(f64(nat(q2)), f64(nat(kr)), f64(v), causal=True)
    assert rel(nat(o), ref_o) <= 2.0 ** -7
    # backward, stage by stage
    do = G.to_layout(dy.cpu(), N, "zigzag").cuda()
    dq2, _, _ = cp.attn_bwd(plan, q2, kr, vr, o, lse, do)
    dback = cp.rope_axes(plan, dq2, pos, SECTIONS, inverse=True)
    dmid = cp.layout_permute(plan, dback, 0).view_as(mid)
    dqr, dkr, dvr, _ = cp.linattn_bwd(plan, qr, kr, vr, ld, dmid)
    dx = cp.rope_axes(plan, dqr, pos, SECTIONS, inverse=True)
    assert cp.check(plan) == 0
    assert rel(dback, RA.rotate(f64(nat(dq2)), ang, inverse=True)) <= 2.0 ** -8
    refs = LA.backward(f64(nat(qr)), f64(nat(kr)), f64(v), f64(ld), plan.scale, f64(dback))
    for got, ref in zip((dqr, dkr, dvr), refs):
        assert rel(nat(got), ref) <= 2.0 ** -7
    assert rel(dx, RA.rotate(f64(nat(dqr)), ang, inverse=True)) <= 2.0 ** -8


def test_prompt_then_drafted_tree():
    """Prompt into cache and state; then three drafted tokens, two of them at one position: the
    softmax layer checks the tree, the linear layer steps along the accepted branch."""
    T, cap = 3, S + 16
    g = torch.Generator().manual_seed(2)
    q, k, v = ((torch.randn(B, S + T, H, D, generator=g) * 0.5).to(torch.bfloat16).cuda() for _ in range(3))
    ld = torch.tensor([-0.03, -0.01, -0.003, -0.1], device="cuda")
    pos = grid_positions(S + T)
    pos[:, :, S + 2] = pos[:, :, S + 1]                     # siblings share their depth's position
    depth = torch.from_numpy(pos).cuda()
    prompt, few = cp.Plan(B, H, S, D, 1, True, "contiguous"), cp.Plan(B, H, T, D, 1, True, "contiguous")
    k_cache, v_cache = (torch.full((B, cap, H, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kr = cp.rope_axes(prompt, k[:, :S].contiguous(), depth[:, :, :S].contiguous(), SECTIONS)
    k_cache[:, :S], v_cache[:, :S] = kr[0], v[:, :S]
    _, state = cp.linattn_fwd(prompt, q[None, :, :S].contiguous(), kr, v[None, :, :S].contiguous(), ld, want_state=True)
    qd, kd = (cp.rope_axes(few, t[:, S:].contiguous(), depth[:, :, S:].contiguous(), SECTIONS)[0] for t in (q, k))
    k_cache[:, S:S + T], v_cache[:, S:S + T] = kd, v[:, S:]
    tree = torch.tensor([[0b001, 0b011, 0b101]], device="cuda")
    c = cp.CachePlan(B, H, H, D, cap, T)
    o, lse = cp.cache_attn(c, qd.contiguous(), k_cache, v_cache, torch.tensor([S], dtype=torch.int32, device="cuda"), tree)
    assert cp.cache_check(c) == 0 and cp.check(prompt) == 0
    ref, _ = CA.attend(f64(qd), f64(k_cache), f64(v_cache), [S], [[0b001, 0b011, 0b101]])
    assert rel(o, ref) <= 2.0 ** -8
    # tokens 0 and 2 were accepted
    pick = [0, 2]
    step = cp.linattn_step(*(t[:, pick].contiguous() for t in (qd, kd, v[:, S:])), ld, state)
    args = [np.concatenate([f64(a), f64(b[:, pick])], 1) for a, b in
            ((q[:, :S], qd), (kr[0], kd), (v[:, :S], v[:, S:]))]
    ref_o, ref_s = LA.forward(*args, f64(ld), D ** -0.5)
    assert rel(step, ref_o[:, S:]) <= 2.0 ** -8 and rel(state, ref_s) <= 2e-6
