"""GPU parity of the multi-axis rotary map (cp_rope_axes_permute) and of its inverse with
the fp64 oracle.

Tolerance per element, from the arithmetic: the angle is reduced in fp64, its sine and
cosine are fp32 (error below 1e-6 with the fp32 products), the result is rounded to bf16
once, by at most half a step, 2^-8 of the value: |gpu - oracle| <= 2^-8 |oracle| + 1e-5 |pair|.
"""
import ctypes

import numpy as np
import pytest
import torch

import context_long_sequence_cp_b200 as cp
from oracle import rope_axes as RA
from tests import gpu_util as G
from workloads import make_small

pytestmark = pytest.mark.gpu


def pair_norm(ref, pairing):
    D = ref.shape[-1]
    a, b = (ref[..., 0::2], ref[..., 1::2]) if pairing == "adjacent" else (ref[..., :D // 2], ref[..., D // 2:])
    n = np.sqrt(a * a + b * b)
    return np.stack([n, n], -1).reshape(ref.shape) if pairing == "adjacent" else np.concatenate([n, n], -1)


def assert_close(gpu, ref, pairing):
    err = np.abs(gpu - ref)
    bound = 2.0 ** -8 * np.abs(ref) + 1e-5 * pair_norm(ref, pairing)
    assert np.all(err <= bound), float((err - bound).max())


def shards(x, N):
    B, S, H, D = x.shape
    return x.reshape(B, N, S // N, H, D).permute(1, 0, 2, 3, 4).contiguous()


def groups(x, N):
    B, S, H, D = x.shape
    return x.reshape(B, S, N, H // N, D).permute(2, 0, 1, 3, 4).contiguous()


def ungroup(y):
    N, B, S, h, D = y.shape
    return y.permute(1, 2, 0, 3, 4).reshape(B, S, N * h, D)


@pytest.mark.parametrize("B,H,S,D,N,layout,sections,freqs,pairing,top", [
    (1, 2, 256, 64, 4, "contiguous", (32,), "shared", "adjacent", 256),
    (2, 3, 1002, 128, 3, "zigzag", (16, 24, 24), "shared", "adjacent", 4000),
    (2, 3, 1002, 128, 3, "zigzag", (16, 24, 24), "per_axis", "half", 4000),
    (1, 1, 10, 64, 1, "zigzag", (1, 30, 1), "per_axis", "half", 100),          # the fewest lanes per unit
    (3, 1, 1, 128, 1, "contiguous", (60, 4), "shared", "half", 100),           # one token
    (1, 37, 64, 128, 2, "contiguous", (8,) * 8, "per_axis", "adjacent", 500),  # a ragged last vector round
    (2, 8, 512, 64, 4, "ulysses", (10, 11, 11), "shared", "adjacent", 4000),
    (1, 8, 24, 128, 8, "ulysses", (32, 32), "shared", "half", 4000),           # one head per run
    (1, 2, 64, 128, 1, "contiguous", (32, 32), "shared", "adjacent", 2 ** 31 - 1),
])
def test_both_directions_match_oracle(B, H, S, D, N, layout, sections, freqs, pairing, top):
    x, dy, _ = make_small(B, H, S, D, seed=51)
    g = torch.Generator().manual_seed(52)
    pos = torch.randint(-top // 2 if top < 2 ** 30 else 0, top, (len(sections), B, S), generator=g).to(torch.int32)
    ang = RA.angles(pos.numpy(), sections, D, freqs=freqs)
    plan = cp.Plan(B, H, S, D, N, False, layout)
    kw = dict(sections=sections, freqs=freqs, pairing=pairing)
    to_in = (lambda t: shards(t, N)) if layout == "ulysses" else (lambda t: t)
    out = cp.rope_axes(plan, to_in(x).cuda(), pos.cuda(), **kw).cpu()
    nat = ungroup(out) if layout == "ulysses" else G.from_layout(out, N, layout)
    assert_close(nat.double().numpy(), RA.rotate(x.double().numpy(), ang, pairing), pairing)
    dlay = groups(dy, N) if layout == "ulysses" else G.to_layout(dy, N, layout)
    dx = cp.rope_axes(plan, dlay.cuda(), pos.cuda(), inverse=True, **kw).cpu()
    ref = RA.rotate(dy.double().numpy(), ang, pairing, inverse=True)
    dnat = dx if layout != "ulysses" else dx.permute(1, 0, 2, 3, 4).reshape(B, S, H, D)
    assert_close(dnat.double().numpy(), ref, pairing)
    # the inverse is the gradient: <rot(x), dy> = <x, inverse(dy)> in 64 bits, and both are the oracle's above
    assert np.isclose(np.sum(RA.rotate(x.double().numpy(), ang, pairing) * dy.double().numpy()),
                      np.sum(x.double().numpy() * ref))


def test_one_axis_equals_rope_permute():
    """One axis, natural positions: the same bits as the single-position map."""
    B, H, S, D, N = 2, 5, 384, 128, 4
    x = make_small(B, H, S, D, seed=53)[0].cuda()
    plan = cp.Plan(B, H, S, D, N, True, "zigzag")
    pos = (torch.arange(S, dtype=torch.int32, device="cuda") + 777).repeat(1, B, 1)
    one = cp.rope_permute(plan, x, pos_offset=777)   # in the shape of x
    assert bool(torch.equal(cp.rope_axes(plan, x, pos, [D // 2]).view_as(one), one))


def test_given_output_other_stream_and_graph():
    B, H, S, D, N = 1, 4, 200, 64, 2
    x, y, _ = (t.cuda() for t in make_small(B, H, S, D, seed=54))
    plan = cp.Plan(B, H, S, D, N, True, "contiguous")
    pos = torch.randint(0, 99, (2, B, S), dtype=torch.int32, device="cuda")
    ref = cp.rope_axes(plan, x, pos, [16, 16])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    side = cp.rope_axes(plan, x, pos, [16, 16], stream=s)
    raw = cp.rope_axes(plan, x, pos, [16, 16], stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(side, ref) and torch.equal(raw, ref)
    out = torch.empty_like(ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        assert cp.rope_axes(plan, x, pos, [16, 16], out=out) is out
    x.copy_(y)
    pos.add_(3)
    graph.replay()
    assert torch.equal(out, cp.rope_axes(plan, y, pos, [16, 16]))


def test_in_place_is_refused():
    plan = cp.Plan(1, 2, 64, 64, 1, True, "contiguous")
    x = torch.zeros(1, 64, 2, 64, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(1, 1, 64, dtype=torch.int32, device="cuda")
    with pytest.raises(cp.CpAttnError):
        cp.rope_axes(plan, x, pos, [32], out=x.view(1, 1, 64, 2, 64))


def test_overlaps_are_refused():
    """Rows move in the map: an output that begins inside the input, or over the positions."""
    B, S, H, D = 2, 64, 2, 64
    plan = cp.Plan(B, H, S, D, 2, True, "zigzag")
    n = B * S * H * D
    buf = torch.zeros(4 * n, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(2 * B * S + 2 * n, dtype=torch.int32, device="cuda")
    sections = (ctypes.c_int * 2)(16, 16)

    def call(x, y, inverse):
        return cp.lib().cp_rope_axes_permute(plan.handle, inverse, x, y, pos.data_ptr(), 2, sections, 1e4, 0, 0, None)
    at = lambda i: buf.data_ptr() + 2 * i
    for inverse in (0, 1):
        for x, y in ((at(0), at(n - 8)), (at(n - 8), at(0)), (at(8), at(0)), (at(0), at(0)), (at(0), pos.data_ptr()),
                     (at(0), pos.data_ptr() + 4 * 2 * B * S - 16)):
            assert call(x, y, inverse) == -1
        assert call(at(0), at(n), inverse) == 0 and call(at(n), at(0), inverse) == 0
        assert call(at(0), pos.data_ptr() + 4 * 2 * B * S, inverse) == 0
    torch.cuda.synchronize()
    assert cp.check(plan) == 0
