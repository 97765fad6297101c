"""GPU parity of linear attention with a decay per head (cp_linattn_fwd, _bwd, _step) with
the fp64 recurrence.

Tolerances, from the arithmetic, per element, with M the sum of the absolute values of
the terms of that element (oracle.linear_attention.magnitudes):
  * bf16 outputs: three roundings to bf16, of at most half a step (2^-8 of the value):
    a decayed score or a state entry once, both as operands of terms that add to at most
    M, and the output; plus the fp32 arithmetic, below 2^-15 M. So
    |gpu - oracle| <= 2^-8 |oracle| + (2^-8 + 2^-15) M (1 + 2^-8).
    The roundings are independent: over a tensor the 2-norm of the error stays below
    2^-8 of the result's (two roundings of relative rms at most 2^-8 / sqrt(3) each).
  * fp32 states: the weighted rows are exact to 2^-24 in three terms, their weights (an
    fp32 exponential of an fp64 product) to 2^-22; the tensor core adds in fp32 and may
    truncate, by 2^-23 of the running sum, once for each 16 rows and term: 24 times a
    chunk; and the chunk sums are added with one rounding, 2^-24, per chunk of 128 rows
    (n of them). |gpu - oracle| <= (2^-22 + 24 2^-23 + n 2^-24) M.
  * the recurrent form sums the state in fp32, one rounding of 2^-23 (decay and product)
    per token.
"""
import numpy as np
import pytest
import torch

import context_long_sequence_cp_b200 as cp
from oracle import linear_attention as LA
from tests import gpu_util as G

pytestmark = pytest.mark.gpu


def decays(H, kind):
    """natural log of the decays: slow (as used), none and mixed with fast ones."""
    if kind == "slow":
        return torch.log1p(-torch.exp2(-(5 + 7 * torch.arange(H, dtype=torch.float64) / H))).float()
    table = torch.tensor([0.0, -1e-6, -0.3749, -0.3751, -1.0, -3.0, -30.0, -float("inf")])
    return table[torch.arange(H) % len(table)].contiguous()


def inputs(B, S, H, D, seed):
    g = torch.Generator().manual_seed(seed)
    q, k, v, do = ((torch.randn(B, S, H, D, generator=g) * s).to(torch.bfloat16) for s in (0.5, 0.5, 1.0, 1.0))
    s0, ds = (torch.randn(B, H, D, D, generator=g) for _ in range(2))
    return q, k, v, do, s0, ds


def f64(t):
    return t.detach().double().cpu().numpy()


def assert_rows(gpu, ref, mag, what):
    gpu = f64(gpu)
    err, bound = np.abs(gpu - ref), 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -15) * (1 + 2.0 ** -8) * mag + 1e-30
    assert np.all(err <= bound), (what, float((err / bound).max()))
    if ref.size >= 4096:
        assert np.linalg.norm(gpu - ref) <= 2.0 ** -8 * np.linalg.norm(ref), (what, np.linalg.norm(gpu - ref) / np.linalg.norm(ref))


def assert_state(gpu, ref, mag, S, what):
    err = np.abs(f64(gpu) - ref)
    bound = (2.0 ** -22 + 24 * 2.0 ** -23 + (S // 128 + 16) * 2.0 ** -24) * mag + 1e-30
    assert np.all(err <= bound), (what, float((err / bound).max()))


SHAPES = [
    # B, H, S, D, N, layout: one token; a chunk and its neighbours; ragged pieces; many short pieces
    (1, 1, 1, 64, 1, "contiguous"), (2, 3, 1, 128, 1, "contiguous"), (1, 2, 127, 128, 1, "contiguous"),
    (1, 2, 128, 64, 1, "contiguous"), (1, 2, 129, 128, 1, "contiguous"), (3, 5, 1000, 64, 5, "contiguous"),
    (2, 3, 996, 128, 3, "zigzag"), (2, 8, 80, 64, 8, "zigzag"), (1, 2, 2000, 128, 1, "zigzag"),
    (1, 8, 1536, 128, 4, "zigzag"), (2, 8, 16, 128, 8, "zigzag"),
]


@pytest.mark.parametrize("kind", ["slow", "mixed"])
@pytest.mark.parametrize("B,H,S,D,N,layout", SHAPES)
def test_forward_and_backward_match_oracle(B, H, S, D, N, layout, kind):
    q, k, v, do, s0, ds = inputs(B, S, H, D, seed=S + D)
    ld = decays(H, kind)
    plan = cp.Plan(B, H, S, D, N, True, layout)
    lay = lambda t: G.to_layout(t, N, layout).cuda()
    nat = lambda t: G.from_layout(t, N, layout)
    dev = [lay(t) for t in (q, k, v)] + [ld.cuda()]
    for first in (None, s0):
        ref, ref_s = LA.forward(f64(q), f64(k), f64(v), ld.double().numpy(), plan.scale, None if first is None else f64(first))
        mag, mag_s = LA.magnitudes(f64(q), f64(k), f64(v), ld.double().numpy(), plan.scale, None if first is None else f64(first))
        z = None if first is None else first.cuda()
        o, s = cp.linattn_fwd(plan, *dev, state_in=z, want_state=True)
        o2, none = cp.linattn_fwd(plan, *dev, state_in=z)
        assert cp.check(plan) == 0 and none is None
        assert_rows(nat(o), ref, mag, "o")
        assert_rows(nat(o2), ref, mag, "o without state")
        assert_state(s, ref_s, mag_s, S, "state")
    for first, last in ((None, None), (s0, ds), (None, ds)):
        n = [None if t is None else f64(t) for t in (first, last)]
        args = (f64(q), f64(k), f64(v), ld.double().numpy(), plan.scale, f64(do), *n)
        refs, mags = LA.backward(*args), LA.magnitudes_backward(*args)
        got = cp.linattn_bwd(plan, *dev, lay(do), state_in=None if first is None else first.cuda(),
                             dstate_out=None if last is None else last.cuda(), want_dstate=first is not None)
        assert cp.check(plan) == 0 and (got[3] is None) == (first is None)
        for g, r, m, name in zip(got[:3], refs, mags, ("dq", "dk", "dv")):
            assert_rows(nat(g), r, m, name)
        if got[3] is not None:
            assert_state(got[3], refs[3], mags[3], S, "dstate")


def test_many_segments_and_many_units():
    """Sequences cut into many segments (one head), and more (batch, head) than SMs (one segment)."""
    for B, H, S in ((1, 1, 6000), (8, 40, 150)):
        q, k, v, do, s0, ds = inputs(B, S, H, 64, seed=B + S)
        ld = decays(H, "slow")
        plan = cp.Plan(B, H, S, 64, 1, True, "contiguous")
        dev = [t[None].cuda() for t in (q, k, v)] + [ld.cuda()]
        args = (f64(q), f64(k), f64(v), ld.double().numpy(), plan.scale)
        o, s = cp.linattn_fwd(plan, *dev, state_in=s0.cuda(), want_state=True)
        got = cp.linattn_bwd(plan, *dev, do[None].cuda(), state_in=s0.cuda(), dstate_out=ds.cuda(), want_dstate=True)
        assert cp.check(plan) == 0
        ref, mag = LA.forward(*args, f64(s0)), LA.magnitudes(*args, f64(s0))
        assert_rows(o[0], ref[0], mag[0], "o")
        assert_state(s, ref[1], mag[1], S, "state")
        ref, mag = (f(*args, f64(do), f64(s0), f64(ds)) for f in (LA.backward, LA.magnitudes_backward))
        for g, r, m, name in zip(got[:3], ref, mag, ("dq", "dk", "dv")):
            assert_rows(g[0], r, m, name)
        assert_state(got[3], ref[3], mag[3], S, "dstate")


def test_ranks_pass_the_state():
    """Each rank on its own tokens from its predecessor's state: the whole sequence's rows and
    gradients, to the tolerance of both."""
    B, H, S, D, N = 1, 3, 768, 128, 3
    q, k, v, do, s0, ds = inputs(B, S, H, D, seed=9)
    ld = decays(H, "slow").cuda()
    one = cp.Plan(B, H, S // N, D, 1, True, "contiguous")
    parts = lambda t: [x.cuda() for x in G.to_layout(t, N, "contiguous")[:, None]]
    qs, ks, vs, dos = (parts(t) for t in (q, k, v, do))
    states, outs = [s0.cuda()], []
    for r in range(N):
        o, s = cp.linattn_fwd(one, qs[r], ks[r], vs[r], ld, state_in=states[-1], want_state=True)
        outs.append(o)
        states.append(s)
    grads, g = [None] * N, ds.cuda()
    for r in reversed(range(N)):
        grads[r] = cp.linattn_bwd(one, qs[r], ks[r], vs[r], ld, dos[r], state_in=states[r], dstate_out=g, want_dstate=True)
        g = grads[r][3]
    assert cp.check(one) == 0
    args = (f64(q), f64(k), f64(v), f64(ld), one.scale)
    ref, mag = LA.forward(*args, f64(s0)), LA.magnitudes(*args, f64(s0))
    join = lambda ts: G.from_layout(torch.cat(ts), N, "contiguous")
    assert_rows(join(outs), ref[0], mag[0], "o")
    assert_state(states[-1], ref[1], mag[1], S, "state")
    ref, mag = (f(*args, f64(do), f64(s0), f64(ds)) for f in (LA.backward, LA.magnitudes_backward))
    for i, name in enumerate(("dq", "dk", "dv")):
        assert_rows(join([x[i] for x in grads]), ref[i], mag[i], name)
    assert_state(g, ref[3], mag[3], S, "dstate")


@pytest.mark.parametrize("B,T,H,D,kind", [(1, 1, 1, 64, "slow"), (2, 1, 3, 128, "mixed"), (3, 5, 5, 64, "mixed"),
                                          (1, 16, 8, 128, "mixed"), (5, 7, 70, 64, "slow"), (10, 2, 33, 128, "slow")])
def test_step_matches_oracle_and_updates_in_place(B, T, H, D, kind):
    q, k, v, _, s0, _ = inputs(B, T, H, D, seed=B + T)
    ld = decays(H, kind)
    st = s0.cuda()
    o = cp.linattn_step(q.cuda(), k.cuda(), v.cuda(), ld.cuda(), st)
    args = (f64(q), f64(k), f64(v), ld.double().numpy(), D ** -0.5, f64(s0))
    ref, mag = LA.forward(*args), LA.magnitudes(*args)
    # fp32 throughout: one bf16 rounding of the output, (T + D) fp32 roundings of sums of at most M
    err = np.abs(f64(o) - ref[0])
    assert np.all(err <= 2.0 ** -8 * np.abs(ref[0]) + (T + D) * 2.0 ** -23 * mag[0])
    # the decay's own relative error, 2^-22, counts once per token it is applied
    assert np.all(np.abs(f64(st) - ref[1]) <= T * (2.0 ** -23 + 2.0 ** -22) * mag[1] + 1e-30)
    # token by token: the same
    one = s0.cuda()
    rows = [cp.linattn_step(*(x[:, t:t + 1].contiguous().cuda() for x in (q, k, v)), ld.cuda(), one) for t in range(T)]
    assert torch.equal(torch.cat(rows, 1), o) and torch.equal(one, st)


def test_prompt_then_steps():
    """A prompt's last state decodes on: the recurrent rows are the chunked form's."""
    B, H, S, D, T = 2, 4, 300, 64, 5
    q, k, v, _, _, _ = inputs(B, S + T, H, D, seed=77)
    ld = decays(H, "slow")
    plan = cp.Plan(B, H, S, D, 1, True, "contiguous")
    head = [t[None, :, :S].contiguous().cuda() for t in (q, k, v)]
    _, st = cp.linattn_fwd(plan, *head, ld.cuda(), want_state=True)
    o = cp.linattn_step(*(t[:, S:].contiguous().cuda() for t in (q, k, v)), ld.cuda(), st)
    args = (f64(q), f64(k), f64(v), ld.double().numpy(), D ** -0.5)
    ref, mag = LA.forward(*args), LA.magnitudes(*args)
    assert_rows(o, ref[0][:, S:], mag[0][:, S:], "o")
    assert_state(st, ref[1], mag[1], S + 128 * T, "state")


def test_inputs_stay_and_rows_do_not_depend_on_neighbours():
    """No input is written; a batch row's results are bit-identical alone and in a batch of the
    same plan shape with other rows changed; two calls give the same bits."""
    B, H, S, D, N = 2, 3, 600, 128, 2
    q, k, v, do, s0, ds = (t.cuda() for t in inputs(B, S, H, D, seed=5))
    lay = lambda t: G.to_layout(t.cpu(), N, "zigzag").cuda()
    ld = decays(H, "slow").cuda()
    plan = cp.Plan(B, H, S, D, N, True, "zigzag")
    args = [lay(q), lay(k), lay(v), ld]
    keep = [t.clone() for t in args]
    o, s = cp.linattn_fwd(plan, *args, state_in=s0, want_state=True)
    again = cp.linattn_fwd(plan, *args, state_in=s0, want_state=True)
    assert torch.equal(o, again[0]) and torch.equal(s, again[1])
    g = cp.linattn_bwd(plan, *args, lay(do), state_in=s0, dstate_out=ds, want_dstate=True)
    for a, b in zip(args, keep):
        assert torch.equal(a, b)
    args[0][:, 1], args[1][:, 1], args[2][:, 1] = 7.0, -3.0, 2.0
    o2, s2 = cp.linattn_fwd(plan, *args, state_in=s0, want_state=True)
    assert torch.equal(o[:, 0], o2[:, 0]) and torch.equal(s[0], s2[0])
    g2 = cp.linattn_bwd(plan, *args, lay(do), state_in=s0, dstate_out=ds, want_dstate=True)
    assert all(torch.equal(x[:, 0], y[:, 0]) for x, y in zip(g[:3], g2[:3])) and torch.equal(g[3][0], g2[3][0])


def test_unaligned_to_32_outputs_and_slices_of_buffers():
    """Tensors that start at any 16-byte boundary inside a larger buffer, the rest of it left as it was."""
    B, H, S, D = 1, 2, 200, 64
    q, k, v, do, _, _ = inputs(B, S, H, D, seed=6)
    n = B * S * H * D

    def inside(t):
        buf = torch.full((n + 64,), 5.0, dtype=torch.bfloat16, device="cuda")
        view = buf[8:8 + n].view(1, B, S, H, D)
        view.copy_(t[None])
        return buf, view
    bufs = [inside(t) for t in (q, k, v, torch.zeros_like(q))]
    ld = decays(H, "slow").cuda()
    plan = cp.Plan(B, H, S, D, 1, True, "contiguous")
    o, _ = cp.linattn_fwd(plan, *(x[1] for x in bufs[:3]), ld, o=bufs[3][1])
    ref, _ = cp.linattn_fwd(plan, *(t[None].cuda() for t in (q, k, v)), ld)
    assert torch.equal(o, ref)
    for buf, _ in bufs:
        assert torch.all(buf[:8] == 5) and torch.all(buf[8 + n:] == 5)


def test_streams_graphs_and_two_calls_at_once():
    B, H, S, D, N = 1, 4, 1024, 64, 2
    sets = [[G.to_layout(t, N, "zigzag").cuda() for t in inputs(B, S, H, D, seed=s)[:4]] for s in (1, 2)]
    ld = decays(H, "slow").cuda()
    plan = cp.Plan(B, H, S, D, N, True, "zigzag")
    refs = [(cp.linattn_fwd(plan, *x[:3], ld, want_state=True), cp.linattn_bwd(plan, *x[:3], ld, x[3])) for x in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = []
    for _ in range(5):   # interleaved on two streams, one plan, a workspace each
        for x, s in zip(sets, streams):
            got.append((x is sets[1], cp.linattn_fwd(plan, *x[:3], ld, want_state=True, stream=s),
                        cp.linattn_bwd(plan, *x[:3], ld, x[3], stream=s)))
    torch.cuda.synchronize()
    assert cp.check(plan) == 0
    for which, f, b in got:
        rf, rb = refs[int(which)]
        assert torch.equal(f[0], rf[0]) and torch.equal(f[1], rf[1])
        assert all(torch.equal(x, y) for x, y in zip(b[:3], rb[:3]))
    graph, live = torch.cuda.CUDAGraph(), [t.clone() for t in sets[0]]
    with torch.cuda.graph(graph):
        f = cp.linattn_fwd(plan, *live[:3], ld, want_state=True)
        b = cp.linattn_bwd(plan, *live[:3], ld, live[3])
    for i in (1, 0):
        for a, t in zip(live, sets[i]):
            a.copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(f[0], refs[i][0][0]) and torch.equal(f[1], refs[i][0][1])
        assert all(torch.equal(x, y) for x, y in zip(b[:3], refs[i][1][:3]))


def test_refusals_with_a_device():
    plan = cp.Plan(1, 2, 4096, 64, 1, True, "contiguous")
    assert plan.linattn_workspace_bytes() > 0
    q = torch.zeros(1, 1, 4096, 2, 64, dtype=torch.bfloat16, device="cuda")
    ld, st = torch.zeros(2, device="cuda"), torch.zeros(1, 2, 64, 64, device="cuda")
    with pytest.raises(ValueError, match="workspace"):
        cp.linattn_fwd(plan, q, q, q, ld, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert cp.lib().cp_linattn_fwd(plan.handle, q.data_ptr(), q.data_ptr(), q.data_ptr(), ld.data_ptr(), None,
                                   q.data_ptr(), None, None, None) == -6
    with pytest.raises(cp.CpAttnError):
        cp.linattn_fwd(plan, q, q, q, ld, state_in=st, state_out=st)
    with pytest.raises(cp.CpAttnError):
        cp.linattn_fwd(cp.Plan(1, 2, 4096, 64, 1, False, "contiguous"), q, q, q, ld)
    with pytest.raises(ValueError, match="q"):
        cp.linattn_fwd(plan, q.transpose(2, 3), q, q, ld)
    with pytest.raises(cp.CpAttnError):
        cp.linattn_step(*([torch.zeros(1, 17, 2, 64, dtype=torch.bfloat16, device="cuda")] * 3), ld, st)


def test_outputs_over_inputs_are_refused():
    """Other CTAs read the rows and states that an output in place would overwrite."""
    plan = cp.Plan(1, 2, 300, 64, 1, True, "contiguous")
    q, k, v, do = (torch.zeros(1, 1, 300, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(4))
    ld, st = torch.zeros(2, device="cuda"), torch.zeros(1, 2, 64, 64, device="cuda")
    for x in (q, k, v):
        with pytest.raises(cp.CpAttnError):
            cp.linattn_fwd(plan, q, k, v, ld, o=x)
    new = [torch.empty_like(q) for _ in range(3)]
    ptr = lambda t: None if t is None else t.data_ptr()
    ws = torch.empty(plan.linattn_workspace_bytes() + 16, dtype=torch.uint8, device="cuda")
    for grads, dsi in ((new, st), ([do] + new[1:], None), ([new[0], q, new[2]], None), (new[:2] + [k], None)):
        assert cp.lib().cp_linattn_bwd(plan.handle, ptr(q), ptr(k), ptr(v), ptr(ld), ptr(do), ptr(st), None,
                                       *(ptr(g) for g in grads), ptr(dsi), ptr(ws), None) == -1
    a = [torch.zeros(1, 1, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    for x in a:
        with pytest.raises(cp.CpAttnError):
            cp.linattn_step(*a, ld, st, o=x)


def test_a_long_sequence_of_one_head_and_its_gradients():
    """Many segments, whose states dv's scan takes from dk's; and the state chained by hand."""
    B, H, S, D = 1, 1, 6200, 128
    q, k, v, do, s0, ds = inputs(B, S, H, D, seed=5)
    ld = torch.tensor([-0.002])
    plan = cp.Plan(B, H, S, D, 1, True, "contiguous")
    assert plan.linattn_workspace_bytes() > 0
    lay = lambda t: G.to_layout(t, 1, "contiguous").cuda()
    dev = [lay(t) for t in (q, k, v, do)]
    dq, dk, dv, dsi = cp.linattn_bwd(plan, *dev[:3], ld.cuda(), dev[3], state_in=s0.cuda(), dstate_out=ds.cuda(),
                                     want_dstate=True)
    assert cp.check(plan) == 0
    scale = 1 / D ** 0.5
    w = torch.exp(ld.double()[0] * (torch.arange(S, dtype=torch.float64)[:, None] - torch.arange(S, dtype=torch.float64)))
    m = torch.tril(w) * scale
    Q, K, V, DO = (t[0, :, 0].double() for t in (q, k, v, do))
    G1, S0 = ds[0, 0].double(), s0[0, 0].double()
    up = torch.exp(ld.double()[0] * (torch.arange(S, dtype=torch.float64) + 1))[:, None]
    down = torch.exp(ld.double()[0] * (S - 1 - torch.arange(S, dtype=torch.float64)))[:, None]
    a, b = (DO @ V.T) * m, (Q @ K.T) * m
    refs = (a @ K + scale * up * (DO @ S0.T), a.T @ Q + down * (V @ G1.T), b.T @ DO + down * (K @ G1),
            scale * (up * Q).T @ DO + torch.exp(ld.double()[0] * S) * G1)
    mags = (a.abs() @ K.abs() + scale * up * (DO.abs() @ S0.abs().T), a.abs().T @ Q.abs() + down * (V.abs() @ G1.abs().T),
            b.abs().T @ DO.abs() + down * (K.abs() @ G1.abs()),
            scale * (up * Q).abs().T @ DO.abs() + torch.exp(ld.double()[0] * S) * G1.abs())
    for got, ref, mag, name in zip((dq, dk, dv), refs, mags, ("dq", "dk", "dv")):
        assert_rows(G.from_layout(got.cpu(), 1, "contiguous")[0, :, 0], ref.numpy(), mag.numpy(), name)
    assert_state(dsi[0, 0], refs[3].numpy(), mags[3].numpy(), S, "dstate_in")


def test_step_keeps_slow_decays_over_thousands_of_tokens():
    """A state kept over 4096 tokens. A token's update is d S + k v^T rounded to fp32: with d as a
    pair of fp32 numbers (2^-48 of d) the inner sum k v^T + lo S is rounded once, by at most 2^-24
    of its value (k v^T itself is exact), and the outer one once, by at most half a step of the
    new state. Later decays do not enlarge these. They need not be of either sign by chance: where
    the state and the row lie on one grid, what d takes off a token may be rounded away each time
    (all of it, for d nearer to 1 than half a step), so they are added as they are, in the 2-norm:
        |error| <= sum_t (|half steps of S_t| + 2^-24 (|k_t v_t^T| + 2^-24 |S_t|)),
    with 1% for entries whose computed value lies across a power of two. A decay kept as one fp32
    exponential is off by up to 2^-23 of d, twice a half step, and exceeds this sum."""
    S, H, D = 4096, 4, 64
    q, k, v, _, s0, _ = (t.cuda() for t in inputs(1, S, H, D, seed=12))
    ld = torch.tensor([-1e-6, -2e-8, -1e-4, 0.0], device="cuda")
    one, many = s0.clone(), s0.clone()
    for t in range(S):
        cp.linattn_step(*(x[:, t:t + 1] for x in (q, k, v)), ld, one)
    for t in range(0, S, 16):
        cp.linattn_step(*(x[:, t:t + 16] for x in (q, k, v)), ld, many)
    assert torch.equal(one, many)
    ref, d = s0.double(), torch.exp(ld.double())[None, :, None, None]
    norm = lambda x: x.square().sum((0, 2, 3)).sqrt()
    bound = torch.zeros(H, dtype=torch.float64, device="cuda")
    for t in range(S):
        new = k[:, t].double()[..., :, None] * v[:, t].double()[..., None, :]
        ref = d * ref + new
        half_step = torch.exp2(torch.floor(torch.log2(ref.abs().clamp(min=2.0 ** -126))) - 24)
        bound += 1.01 * norm(half_step) + 2.0 ** -24 * (norm(new) + 2.0 ** -24 * norm(ref))
    err = norm(one.double() - ref)
    assert torch.all(err <= bound), (err / bound).tolist()


def test_outputs_over_one_another_are_refused():
    """The same buffer as two outputs, or as an output and the workspace, also in part: several CTAs
    would write its bytes in no order."""
    plan = cp.Plan(1, 2, 4096, 64, 1, True, "contiguous")
    n = 4096 * 2 * 64
    rows = torch.zeros(4, n, dtype=torch.bfloat16, device="cuda")
    q, k, v, do = (x.data_ptr() for x in rows)
    ld, zs = torch.zeros(2, device="cuda"), torch.zeros(4, 1, 2, 64, 64, device="cuda")
    z = [x.data_ptr() for x in zs]
    buf = torch.zeros(4 * n + plan.linattn_workspace_bytes(), dtype=torch.bfloat16, device="cuda")
    at = lambda i: buf.data_ptr() + 2 * i                    # element i
    ws = at(4 * n)

    def fwd(o=at(0), so=z[0], ws=ws):
        return cp.lib().cp_linattn_fwd(plan.handle, q, k, v, ld.data_ptr(), z[1], o, so, ws, None)

    def bwd(dq=at(0), dk=at(n), dv=at(2 * n), dsi=z[0], ws=ws):
        return cp.lib().cp_linattn_bwd(plan.handle, q, k, v, ld.data_ptr(), do, z[1], z[2], dq, dk, dv, dsi, ws, None)
    assert fwd() == 0 and bwd() == 0
    for bad in (dict(o=z[0]), dict(so=at(n - 8)), dict(ws=at(0)), dict(ws=z[0]), dict(ws=z[1]), dict(o=ws + 64),
                dict(ws=q), dict(so=ld.data_ptr())):
        assert fwd(**bad) == -1, bad
    for bad in (dict(dq=at(n)), dict(dk=at(2 * n)), dict(dv=at(0)), dict(dq=at(8)), dict(dv=at(n + 8)), dict(dsi=at(0)),
                dict(ws=at(3 * n - 8)), dict(ws=z[2]), dict(dv=do + 16), dict(dsi=z[1] + 16)):
        assert bwd(**bad) == -1, bad
    assert fwd(o=at(n), so=None, ws=at(3 * n)) == 0 and bwd(dsi=None) == 0          # next to one another
    s = [torch.zeros(1, 1, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(4)]

    def step(o=s[3].data_ptr(), st=z[0]):
        return cp.lib().cp_linattn_step(1, 1, 2, 64, *(x.data_ptr() for x in s[:3]), ld.data_ptr(), 0.1, st, o, None)
    assert step() == 0
    for bad in (dict(o=z[0]), dict(o=z[0] + 2 * 64 * 64 * 4 - 16), dict(st=s[0].data_ptr()), dict(o=ld.data_ptr())):
        assert step(**bad) == -1, bad
    torch.cuda.synchronize()
    assert cp.check(plan) == 0
