"""Host-side checks of the rotary, linear-attention and cache-attention entry points: what
they refuse, with which status, before anything is enqueued. No GPU needed; the pointers
of refused calls are never read."""
import ctypes
import math

import pytest
import torch

import context_long_sequence_cp_b200 as cp
from context_long_sequence_cp_b200 import build as cpbuild

INVALID, UNSUPPORTED, ALIGNMENT, CUDA, WORKSPACE = -1, -2, -3, -4, -6
P = 1 << 20          # an aligned address that is never read
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="the call would reach the GPU")


@pytest.fixture(scope="module", autouse=True)
def built():
    cpbuild.build()


def _rope(plan, direction=0, x=P, y=2 * P, pos=P, sections=(16, 24, 24), base=1e4, freqs=0, pairing=0, axes=None):
    arr = (ctypes.c_int * max(len(sections), 1))(*sections)
    return cp.lib().cp_rope_axes_permute(plan, direction, x, y, pos, len(sections) if axes is None else axes, arr,
                                         base, freqs, pairing, None)


def test_rope_axes_refusals():
    keep = cp.Plan(2, 4, 256, 128, 2, True, "zigzag")
    plan = keep.handle
    for bad in (dict(direction=2), dict(direction=-1), dict(x=None), dict(y=None), dict(pos=None), dict(freqs=2),
                dict(pairing=-1), dict(base=1.0), dict(base=math.inf), dict(base=math.nan), dict(axes=0),
                dict(axes=-1), dict(sections=(16, 24, 23)), dict(sections=(16, 24, 25)), dict(sections=(64, 0)),
                dict(sections=(65, -1)), dict(sections=(2**31 - 1, 2**31 - 1))):
        assert _rope(plan, **bad) == INVALID, bad
    assert _rope(None) == INVALID
    for bad in (dict(x=P + 8), dict(y=P + 2), dict(pos=P + 2)):
        assert _rope(plan, **bad) == ALIGNMENT, bad


def _linattn(plan, q=P, k=P, v=P, ld=P, si=None, o=P, so=None, ws=P):
    return cp.lib().cp_linattn_fwd(plan, q, k, v, ld, si, o, so, ws, None)


def _linattn_bwd(plan, q=P, k=P, v=P, ld=P, do=P, si=None, ds=None, dq=P, dk=P, dv=P, dsi=None, ws=P):
    return cp.lib().cp_linattn_bwd(plan, q, k, v, ld, do, si, ds, dq, dk, dv, dsi, ws, None)


def test_linattn_refusals():
    keep = cp.Plan(2, 4, 256, 128, 2, True, "zigzag")
    plan = keep.handle
    for f, names in ((_linattn, ("q", "k", "v", "ld", "o")), (_linattn_bwd, ("q", "k", "v", "ld", "do", "dq", "dk", "dv"))):
        assert f(None) == INVALID
        for name in names:
            assert f(plan, **{name: None}) == INVALID, name
            assert f(plan, **{name: P + 2}) == ALIGNMENT, name
    assert _linattn(plan, si=P + 4) == ALIGNMENT and _linattn(plan, so=P + 8) == ALIGNMENT
    assert _linattn(plan, ws=P + 8) == ALIGNMENT and _linattn_bwd(plan, dsi=P + 8) == ALIGNMENT
    assert _linattn(plan, si=P, so=P) == INVALID            # every segment reads the first state
    assert _linattn_bwd(plan, ds=P, dsi=P) == INVALID
    for bad in (cp.Plan(1, 4, 256, 64, 2, False, "contiguous"), cp.Plan(1, 4, 256, 64, 2, False, "ulysses")):
        assert _linattn(bad.handle) == UNSUPPORTED and _linattn_bwd(bad.handle) == UNSUPPORTED
        assert cp.lib().cp_linattn_workspace_bytes(bad.handle) == 0
    assert cp.lib().cp_linattn_workspace_bytes(None) == 0


def test_linattn_step_refusals():
    def step(B=1, T=1, H=2, D=64, q=P, k=P, v=P, ld=P, scale=0.1, st=P, o=P):
        return cp.lib().cp_linattn_step(B, T, H, D, q, k, v, ld, scale, st, o, None)
    for bad in (dict(B=-1), dict(T=-1), dict(H=0), dict(scale=math.nan), dict(scale=math.inf), dict(q=None),
                dict(k=None), dict(v=None), dict(ld=None), dict(st=None), dict(o=None)):
        assert step(**bad) == INVALID, bad
    for bad in (dict(D=96), dict(D=32), dict(T=17), dict(B=2**30, H=2**10)):
        assert step(**bad) == UNSUPPORTED, bad
    for bad in (dict(q=P + 2), dict(k=P + 8), dict(v=P + 8), dict(ld=P + 2), dict(st=P + 4), dict(o=P + 8)):
        assert step(**bad) == ALIGNMENT, bad
    assert step(B=0) == 0 and step(T=0, q=None) == 0         # nothing to do


def test_cache_plan_refusals():
    def plan(B=2, Hq=8, Hkv=2, D=128, cap=1000, T=4, scale=0.0):
        h = ctypes.c_void_p()
        rc = cp.lib().cp_cache_plan(ctypes.byref(h), B, Hq, Hkv, D, cap, T, scale)
        if rc == 0:
            assert cp.lib().cp_cache_attn_workspace_bytes(h) > 0
            cp.lib().cp_cache_plan_destroy(h)
        else:
            assert h.value is None
        return rc
    assert plan() == 0 and plan(T=64) == 0 and plan(B=1024) == 0 and plan(Hq=256, Hkv=2) == 0 and plan(scale=0.3) == 0
    for bad in (dict(B=0), dict(Hq=0), dict(Hkv=0), dict(cap=0), dict(T=0), dict(scale=math.nan), dict(scale=math.inf)):
        assert plan(**bad) == INVALID, bad
    for bad in (dict(D=96), dict(T=65), dict(B=1025), dict(Hq=9), dict(Hq=258, Hkv=2), dict(cap=2**31 - 1),
                dict(B=1024, Hkv=2**17, Hq=2**17)):
        assert plan(**bad) == UNSUPPORTED, bad
    assert cp.lib().cp_cache_plan(None, 1, 1, 1, 64, 10, 1, 0.0) == INVALID
    assert cp.lib().cp_cache_plan_destroy(None) == 0
    assert cp.lib().cp_cache_attn_workspace_bytes(None) == 0


def test_cache_attn_refusals():
    plan = cp.CachePlan(2, 8, 2, 128, 1000, 4)

    def call(h=plan.handle, q=P, k=P, v=P, n=P, tree=P, o=P, lse=P, ws=P):
        return cp.lib().cp_cache_attn(h, q, k, v, n, tree, o, lse, ws, None)

    def partial(own=1, o=P, lse=P, ws=P):
        return cp.lib().cp_cache_attn_partial(plan.handle, P, P, P, P, own, P, o, lse, ws, None)
    for bad in (dict(h=None), dict(q=None), dict(k=None), dict(v=None), dict(n=None), dict(o=None)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(q=P + 8), dict(k=P + 8), dict(v=P + 8), dict(n=P + 2), dict(tree=P + 4), dict(o=P + 8),
                dict(lse=P + 2), dict(ws=P + 8)):
        assert call(**bad) == ALIGNMENT, bad
    assert call(ws=None) == WORKSPACE
    for bad in (dict(own=2), dict(own=-1), dict(o=None), dict(lse=None)):
        assert partial(**bad) == INVALID, bad
    assert partial(o=P + 8) == ALIGNMENT and partial(ws=None) == WORKSPACE


@no_gpu
def test_without_a_device_every_launch_says_so():
    keep = cp.Plan(1, 2, 256, 64, 2, True, "zigzag")
    plan = keep.handle
    assert _rope(plan, sections=(16, 16)) == CUDA
    assert _linattn(plan) == CUDA and _linattn_bwd(plan) == CUDA
    assert cp.lib().cp_linattn_step(1, 1, 2, 64, P, P, P, P, 0.1, P, P, None) == CUDA
    c = cp.CachePlan(1, 2, 1, 64, 100, 2)
    assert cp.lib().cp_cache_attn(c.handle, P, P, P, P, P, P, P, P, None) == CUDA
    assert cp.cache_check(c, stream=0) == CUDA


def test_python_refuses_what_does_not_fit():
    """Types, shapes, strides and devices are checked before the library is called."""
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    plan = cp.Plan(1, 2, 8, 64, 2, True, "zigzag")
    pos = torch.zeros(2, 1, 8, dtype=torch.int32)
    x, q = bf(1, 8, 2, 64), bf(2, 1, 4, 2, 64)
    ld, st = torch.zeros(2), torch.zeros(1, 2, 64, 64)
    with pytest.raises(ValueError, match="positions"):
        cp.rope_axes(plan, x, pos.long(), [16, 16])
    with pytest.raises(ValueError, match="positions"):
        cp.rope_axes(plan, x, pos[:1], [16, 16])
    with pytest.raises(ValueError, match="x:"):
        cp.rope_axes(plan, q, pos, [16, 16])                   # the layout of the other direction
    with pytest.raises(ValueError, match="freqs"):
        cp.rope_axes(plan, x, pos, [16, 16], freqs="each")
    with pytest.raises(ValueError, match="v:"):
        cp.linattn_fwd(plan, q, q, q.float(), ld)
    with pytest.raises(ValueError, match="k:"):
        cp.linattn_fwd(plan, q, bf(2, 1, 4, 2, 128)[..., ::2], q, ld)   # strided
    with pytest.raises(ValueError, match="log_decay"):
        cp.linattn_fwd(plan, q, q, q, ld.double())
    with pytest.raises(ValueError, match="state_in"):
        cp.linattn_fwd(plan, q, q, q, ld, state_in=st.half())
    with pytest.raises(ValueError, match="dout"):
        cp.linattn_bwd(plan, q, q, q, ld, x)
    with pytest.raises(ValueError, match="state"):
        cp.linattn_step(bf(1, 1, 2, 64), bf(1, 1, 2, 64), bf(1, 1, 2, 64), ld, st[:, :1])
    c = cp.CachePlan(1, 4, 2, 64, 32, 3)
    kv, n = bf(1, 32, 2, 64), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="k_cache"):
        cp.cache_attn(c, bf(1, 3, 4, 64), bf(1, 31, 2, 64), kv, n)
    with pytest.raises(ValueError, match="lengths"):
        cp.cache_attn(c, bf(1, 3, 4, 64), kv, kv, n.long())
    with pytest.raises(ValueError, match="tree"):
        cp.cache_attn(c, bf(1, 3, 4, 64), kv, kv, n, tree=torch.zeros(1, 3, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):              # all that fits, but on the CPU
        cp.cache_attn(c, bf(1, 3, 4, 64), kv, kv, n)
    with pytest.raises(ValueError, match="CUDA"):
        cp.linattn_step(bf(1, 1, 2, 64), bf(1, 1, 2, 64), bf(1, 1, 2, 64), ld, st)


def test_linattn_workspace_depends_on_the_plan_alone():
    """Sized with any device current, or none: a caller that lays out its buffers first gets the
    bytes that the call will use. 8 heads of 64 chunks: 16 segments forward, 15 of whose states
    are kept (the backward: 6, three scans of 5)."""
    plan = cp.Plan(1, 8, 64 * 128, 64, 1, True, "contiguous")
    sms = 148 if not torch.cuda.is_available() else torch.cuda.get_device_properties(0).multi_processor_count
    n = int(cp.lib().cp_linattn_workspace_bytes(plan.handle))
    assert n > 0 and n % (8 * 64 * 64 * 4) == 0
    assert sms != 148 or n == 15 * 8 * 64 * 64 * 4
    assert plan.linattn_workspace_bytes() == n


def test_python_refuses_a_stream_of_another_device():
    """Entering such a stream would make its device current, and the kernel would run there on the
    tensors' addresses."""
    class Stream:
        cuda_stream, device = 0, torch.device("cuda", 1)
    with pytest.raises(ValueError, match="stream"):
        cp._enqueue(torch.device("cuda", 0), Stream(), lambda s: pytest.fail("launched"))


@pytest.mark.parametrize("scale", [math.nan, math.inf, -math.inf])
def test_python_refuses_a_scale_that_is_no_number(scale):
    """As the library does; NaN is not one of the values that select the default."""
    x, ld, st = torch.zeros(1, 1, 2, 64, dtype=torch.bfloat16), torch.zeros(2), torch.zeros(1, 2, 64, 64)
    with pytest.raises(ValueError, match="scale"):
        cp.linattn_step(x, x, x, ld, st, scale=scale)


def test_linattn_segments_are_those_of_the_measured_comment():
    """The rule that cuts a sequence into segments, restated, and its choices for the sizes whose
    times stand beside it; the library's show in the bytes it asks for (the states of all segments
    but the last, of one scan forward and of three backward)."""
    def choose(ctas, state_ctas, chunks, sms=148):
        def cost(s):
            per = -(-chunks // s)
            c = -(-ctas * s // sms) * (per + 2.5 + 0.35 * (s - 1))
            return c + (-(-state_ctas * (s - 1) // sms) * (0.45 * per + 2.0) if s > 1 else 0.0)
        return min(range(1, min(chunks, 64) + 1), key=cost)
    assert choose(32, 32, 256) == 4 and choose(8, 8, 64) == 16 and choose(3 * 8, 2 * 8, 64) == 6
    assert choose(3 * 4, 2 * 4, 256) == 12
    if torch.cuda.is_available() and torch.cuda.get_device_properties(0).multi_processor_count != 148:
        pytest.skip("the comment's figures are of 148 SMs")
    for heads, chunks in ((32, 256), (8, 64), (4, 256), (16, 32), (1, 57), (300, 10)):
        f, b = choose(heads, heads, chunks), choose(3 * heads, 2 * heads, chunks)
        plan = cp.Plan(1, heads, chunks * 128, 64, 1, True, "contiguous")
        assert plan.linattn_workspace_bytes() == max(f - 1, 3 * (b - 1)) * heads * 64 * 64 * 4
