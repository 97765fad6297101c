"""Cases of the rotary, linear-attention and cache-attention operators, their plain
forms in elementary torch operations, and their values from the definitions in 64 bits.

  rope_axes      rotary embedding with one position per axis (time, height, width),
                 fused into the layout map of a context-parallel plan; its inverse
                 is the gradient.
  linattn_fwd / linattn_bwd / linattn_step
                 causal linear attention with a decay for each head: chunked over a
                 prompt or a training sequence in the plan's layout, and its
                 recurrent form for a few tokens on a kept state.
  cache_attn     attention of a tree of drafted tokens (or of single tokens) over a
                 key/value cache.

``run`` computes the plain form where ``own`` is false and makes the library's calls
where it is true; both take what ``prepare`` gives.
"""
import math

import torch

own = False

_LAYOUTS = ("contiguous", "zigzag", "ulysses")


# ---------------------------------------------------------------------- the cases
def listed():
    return [
        # Keys or queries of a 32k-token video clip on the way into zigzag attention.
        dict(name="rope_video_32k", op="rope", B=1, S=32768, H=32, D=128, N=8, layout="zigzag", sections="16,24,24",
             freqs="shared", pairing="adjacent", inverse=False),
        # Gradient of an image batch's rotation, half pairing, odd lengths and head count.
        dict(name="rope_grad_odd", op="rope", B=3, S=1998, H=5, D=64, N=3, layout="zigzag", sections="16,16",
             freqs="per_axis", pairing="half", inverse=True),
        # The rotation of one decoding step: latency.
        dict(name="rope_decode", op="rope", B=4, S=1, H=32, D=128, N=1, layout="contiguous", sections="16,24,24",
             freqs="shared", pairing="adjacent", inverse=False),
        # Prompt of 32k tokens, the state kept for decoding.
        dict(name="linear_prompt_32k", op="linear_fwd", B=1, S=32768, H=32, D=128, N=8, layout="zigzag",
             state_in=False, state_out=True),
        # A ragged batch of a small model, continued from a state (contiguous ranks of 200 tokens).
        dict(name="linear_prompt_odd", op="linear_fwd", B=3, S=1000, H=5, D=64, N=5, layout="contiguous",
             state_in=True, state_out=True),
        # Training: the backward of 4k tokens, and of a batch of 16k tokens.
        dict(name="linear_train_4k", op="linear_bwd", B=1, S=4096, H=16, D=128, N=4, layout="zigzag",
             state_in=False, state_out=False),
        dict(name="linear_train_16k", op="linear_bwd", B=2, S=16384, H=32, D=128, N=8, layout="contiguous",
             state_in=True, state_out=True),
        # Decoding: one token of each of 64 sequences, and a few tokens of three small ones.
        dict(name="linear_step_64", op="linear_step", B=64, T=1, H=32, D=128),
        dict(name="linear_step_few", op="linear_step", B=3, T=5, H=5, D=64),
        # A tree of 32 drafted tokens over a 128k-token cache, grouped heads.
        dict(name="cache_tree_128k", op="cache", B=1, T=32, Hq=32, Hkv=8, D=128, cap=131072, lengths="full"),
        # A served batch of uneven lengths, 16 drafted tokens each.
        dict(name="cache_batch_uneven", op="cache", B=16, T=16, Hq=32, Hkv=8, D=128, cap=8192, lengths="uneven"),
        # Single tokens over short caches, one key/value head per query head.
        dict(name="cache_token_short", op="cache", B=2, T=1, Hq=16, Hkv=16, D=64, cap=500, lengths="full"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_tokens(rng, budget, layout):
    """(B, S, H, D, N) with B*S*H*D within the budget."""
    while True:
        D = rng.choice([64, 128])
        N = rng.choice([1, 1, 2, 3, 4, 5, 8])
        unit = 2 * N if layout == "zigzag" else N
        S = unit * max(1, _log_int(rng, 1, 32768) // unit)
        H = _log_int(rng, 1, 48)
        if layout == "ulysses":
            H = N * max(1, H // N)
        B = _log_int(rng, 1, 16)
        if B * S * H * D <= budget:
            return B, S, H, D, N


def draw(rng):
    op = rng.choice(["rope", "linear_fwd", "linear_bwd", "linear_step", "cache"])
    if op == "rope":
        layout = rng.choice(_LAYOUTS)
        B, S, H, D, N = _draw_tokens(rng, 1 << 27, layout)
        axes = rng.choice([1, 2, 3, 3, 4])
        cuts = sorted(rng.sample(range(1, D // 2), axes - 1))
        sections = ",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [D // 2]))
        return dict(op=op, B=B, S=S, H=H, D=D, N=N, layout=layout, sections=sections,
                    freqs=rng.choice(["shared", "per_axis"]), pairing=rng.choice(["adjacent", "half"]),
                    inverse=rng.choice([False, True]))
    if op in ("linear_fwd", "linear_bwd"):
        layout = rng.choice(_LAYOUTS[:2])
        B, S, H, D, N = _draw_tokens(rng, 1 << 27, layout)
        return dict(op=op, B=B, S=S, H=H, D=D, N=N, layout=layout, state_in=rng.choice([False, True]),
                    state_out=rng.choice([False, True]))
    if op == "linear_step":
        D = rng.choice([64, 128])
        return dict(op=op, B=_log_int(rng, 1, 64), T=rng.choice([1, 1, 2, 3, 5, 8, 16]), H=_log_int(rng, 1, 32), D=D)
    while True:
        D = rng.choice([64, 128])
        Hkv = _log_int(rng, 1, 16)
        G = rng.choice([1, 2, 3, 4, 5, 8, 16])
        B = _log_int(rng, 1, 32)
        T = rng.choice([1, 1, 2, 5, 8, 16, 31, 64])
        cap = _log_int(rng, T + 1, 131072)
        if B * Hkv * D * cap <= 1 << 27 and B * Hkv * G * T * cap <= 1 << 28:
            return dict(op=op, B=B, T=T, Hq=Hkv * G, Hkv=Hkv, D=D, cap=cap,
                        lengths=rng.choice(["full", "uneven", "uneven"]))


# ---------------------------------------------------------------- helpers of both sides
def _positions(c):
    """Natural position of rank r's local token l, [N * S/N] in rank-major order."""
    N, S = c["N"], c["S"]
    p = torch.arange(S, device="cuda")
    if c["layout"] == "zigzag":   # rank r holds chunk r, then chunk 2N-1-r, of 2N
        chunks = p.reshape(2 * N, S // (2 * N))
        return torch.cat([chunks[:N], chunks[N:].flip(0)], 1).reshape(-1)
    return p


def _natural(x, pos):
    """Rank-major [N, B, S/N, H, D] -> natural [B, S, H, D]."""
    N, B, T, H, D = x.shape
    out = torch.empty(B, N * T, H, D, dtype=x.dtype, device=x.device)
    out[:, pos] = x.permute(1, 0, 2, 3, 4).reshape(B, N * T, H, D)
    return out


def _ranked(x, pos, N):
    """Natural [B, S, H, D] -> rank-major [N, B, S/N, H, D]."""
    B, S, H, D = x.shape
    return x[:, pos].reshape(B, N, S // N, H, D).permute(1, 0, 2, 3, 4).contiguous()


def _groups(x, N):
    """Natural [B, S, H, D] -> Ulysses head groups [N, B, S, H/N, D]."""
    B, S, H, D = x.shape
    return x.reshape(B, S, N, H // N, D).permute(2, 0, 1, 3, 4).contiguous()


def _lengths(c):
    """Cached tokens of each sequence, before the T drafted ones."""
    room = c["cap"] - c["T"]
    if c["lengths"] == "full" or c["B"] == 1:
        return [room] * c["B"]
    return [room * b // (c["B"] - 1) for b in range(c["B"])]   # an empty cache among them


def _log_decay(H):
    """Natural log of head h's decay 1 - 2^-(5 + 7 h / H): windows from 32 to about 4096 tokens."""
    h = torch.arange(H, dtype=torch.float64, device="cuda")
    return torch.log1p(-torch.exp2(-(5 + 7 * h / H))).float()


def _randn(gen, *shape, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)


# --------------------------------------------------------------------- prepare and run
def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator("cuda")
    gen.manual_seed(seed)
    st = {"case": c}
    if c["op"] == "rope":
        B, S, H, D, N = (c[x] for x in "BSHDN")
        st["sections"] = [int(x) for x in c["sections"].split(",")]
        A = len(st["sections"])
        st["positions"] = torch.randint(0, 40000, (A, B, S), generator=gen, device="cuda", dtype=torch.int32)
        shape = (B, S, H, D)
        if c["layout"] == "ulysses":
            shape = (N, B, S, H // N, D) if c["inverse"] else (N, B, S // N, H, D)
        elif c["inverse"]:
            shape = (N, B, S // N, H, D)
        st["x"] = _randn(gen, *shape)
        if own:
            import context_long_sequence_cp_b200 as cp
            st["plan"] = cp.Plan(B, H, S, D, N, False, c["layout"])
    elif c["op"] in ("linear_fwd", "linear_bwd"):
        B, S, H, D, N = (c[x] for x in "BSHDN")
        shape = (N, B, S // N, H, D)
        st["q"], st["k"], st["v"] = (_randn(gen, *shape, scale=s) for s in (0.5, 0.5, 1.0))
        st["log_decay"] = _log_decay(H)
        st["state_in"] = _randn(gen, B, H, D, D, dtype=torch.float32) if c["state_in"] else None
        if c["op"] == "linear_bwd":
            st["dout"] = _randn(gen, *shape)
            st["dstate"] = _randn(gen, B, H, D, D, dtype=torch.float32) if c["state_out"] else None
        if own:
            import context_long_sequence_cp_b200 as cp
            st["plan"] = cp.Plan(B, H, S, D, N, True, c["layout"])
    elif c["op"] == "linear_step":
        B, T, H, D = (c[x] for x in "BTHD")
        st["q"], st["k"], st["v"] = (_randn(gen, B, T, H, D, scale=s) for s in (0.5, 0.5, 1.0))
        st["log_decay"] = _log_decay(H)
        st["state"] = _randn(gen, B, H, D, D, scale=4.0, dtype=torch.float32)
    else:
        B, T, Hq, Hkv, D, cap = (c[x] for x in ("B", "T", "Hq", "Hkv", "D", "cap"))
        st["q"] = _randn(gen, B, T, Hq, D)
        st["k"], st["v"] = (_randn(gen, B, cap, Hkv, D) for _ in range(2))
        st["lengths"] = torch.tensor(_lengths(c), dtype=torch.int32, device="cuda")
        # a random tree: token t hangs from an earlier one (or from the cache, -1) and sees its ancestors and itself
        parents = (torch.rand(B, T, generator=gen, device="cuda") * (torch.arange(T, device="cuda") + 1)).long().cpu() - 1
        tree = torch.zeros(B, T, dtype=torch.int64)
        for t in range(T):
            up = parents[:, t]
            seen = torch.where(up >= 0, tree.gather(1, up.clamp(min=0)[:, None])[:, 0], torch.zeros(B, dtype=torch.int64))
            tree[:, t] = seen | (-(1 << 63) if t == 63 else 1 << t)
        st["tree"] = tree.cuda()
        if own:
            import context_long_sequence_cp_b200 as cp
            st["plan"] = cp.CachePlan(B, Hq, Hkv, D, cap, T)
    return st


def run(st):
    c = st["case"]
    if own:
        return _run_own(st, c)
    with torch.no_grad():
        if c["op"] == "rope":
            return _rope_plain(st, c)
        if c["op"] == "linear_fwd":
            return _linear_fwd_plain(st, c)
        if c["op"] == "linear_bwd":
            return _linear_bwd_plain(st, c)
        if c["op"] == "linear_step":
            return _linear_step_plain(st, c)
        return _cache_plain(st, c)


def _run_own(st, c):
    import context_long_sequence_cp_b200 as cp
    if c["op"] == "rope":
        return cp.rope_axes(st["plan"], st["x"], st["positions"], st["sections"], freqs=c["freqs"],
                            pairing=c["pairing"], inverse=c["inverse"])
    if c["op"] == "linear_fwd":
        o, s = cp.linattn_fwd(st["plan"], st["q"], st["k"], st["v"], st["log_decay"], state_in=st["state_in"],
                              want_state=c["state_out"])
        return [o] + ([s] if c["state_out"] else [])
    if c["op"] == "linear_bwd":
        dq, dk, dv, ds = cp.linattn_bwd(st["plan"], st["q"], st["k"], st["v"], st["log_decay"], st["dout"],
                                        state_in=st["state_in"], dstate_out=st["dstate"], want_dstate=c["state_in"])
        return [dq, dk, dv] + ([ds] if c["state_in"] else [])
    if c["op"] == "linear_step":
        o = cp.linattn_step(st["q"], st["k"], st["v"], st["log_decay"], st["state"])
        return [o, st["state"]]
    o, lse = cp.cache_attn(st["plan"], st["q"], st["k"], st["v"], st["lengths"], st["tree"])
    return [o, lse]


# ------------------------------------------------------------------------ plain forms
def _thetas(st, c):
    """(axis of each feature pair, its frequency in 64 bits)."""
    D, sections = c["D"], st["sections"]
    n = torch.tensor(sections, device="cuda")
    axis = torch.repeat_interleave(torch.arange(len(sections), device="cuda"), n)
    pair = torch.arange(D // 2, device="cuda", dtype=torch.float64)
    if c["freqs"] == "per_axis":
        pair = (pair - torch.repeat_interleave(torch.cumsum(n, 0) - n, n)) * (D // 2) / n[axis]
    return axis, torch.pow(torch.tensor(10000.0, dtype=torch.float64, device="cuda"), -2 * pair / D)


def _rope_plain(st, c):
    B, S, H, D, N = (c[x] for x in "BSHDN")
    pos = _positions(c)
    x = st["x"].float()
    if c["layout"] == "ulysses":
        x = x.permute(1, 2, 0, 3, 4) if c["inverse"] else x.permute(1, 0, 2, 3, 4)
        x = x.reshape(B, S, H, D)
    elif c["inverse"]:
        x = _natural(x, pos)
    axis, theta = _thetas(st, c)
    angle = st["positions"].double()[axis].permute(1, 2, 0) * theta   # [B, S, D/2]
    cos, sin = torch.cos(angle).float()[:, :, None], torch.sin(angle).float()[:, :, None]
    sin = -sin if c["inverse"] else sin
    if c["pairing"] == "half":
        a, b = x[..., :D // 2], x[..., D // 2:]
        y = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    else:
        a, b = x[..., 0::2], x[..., 1::2]
        y = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).reshape(B, S, H, D)
    y = y.to(torch.bfloat16)
    if c["layout"] == "ulysses":
        return y.reshape(B, N, S // N, H, D).permute(1, 0, 2, 3, 4).contiguous() if c["inverse"] else _groups(y, N)
    return y if c["inverse"] else _ranked(y, pos, N)


def _decays(log_decay, powers):
    """exp(log_decay[h] * powers), powers of 0 giving 1; fp32 of the value in 64 bits."""
    x = log_decay.double().reshape(-1, *[1] * powers.dim()) * powers.double()
    return torch.exp(x).float()


def _linear_scan(a, b, v, log_decay, first, e):
    """y_i = sum_{j<=i} d^(i-j) (a_i . b_j) v_j + d^(i+e) a_i^T first, all [B, S, H, D] fp32, by chunks of 128
    whose states are joined by one product with the lower triangle of chunk decays."""
    B, S, H, D = a.shape
    C = min(128, S)
    n = -(-S // C)
    pad = n * C - S
    a, b, v = (torch.nn.functional.pad(x, (0, 0, 0, 0, 0, pad)).reshape(B, n, C, H, D).permute(0, 3, 1, 2, 4)
               for x in (a, b, v))                                     # [B, H, n, C, D]
    p = torch.arange(C, device="cuda")
    within = _decays(log_decay, (p[:, None] - p[None]).clamp(min=0)) * (p[:, None] >= p[None])   # [H, C, C]
    y = (a @ b.transpose(-1, -2) * within[:, None]) @ v
    kv = (b * _decays(log_decay, C - 1 - p)[:, None, :, None]).transpose(-1, -2) @ v              # [B, H, n, D, D]
    m = torch.arange(n, device="cuda")
    gap = m[:, None] - 1 - m[None]
    join = _decays(log_decay, (C * gap).clamp(min=0)) * (gap >= 0)                                # [H, n, n]
    before = (join @ kv.reshape(B, H, n, D * D)).reshape(B, H, n, D, D)
    if first is not None:
        before = before + _decays(log_decay, C * m + e - 1)[:, :, None, None] * first[:, :, None]
    y = y + _decays(log_decay, p + 1)[:, None, :, None] * (a @ before)
    return y.permute(0, 2, 3, 1, 4).reshape(B, n * C, H, D)[:, :S]


def _linear_state(k, v, log_decay, powers, first):
    """sum_i d^powers_i k_i v_i^T + d^S first: [B, H, D, D] fp32."""
    w = _decays(log_decay, powers).transpose(0, 1)[None, :, :, None]
    s = (k * w).permute(0, 2, 3, 1) @ v.permute(0, 2, 1, 3)
    if first is not None:
        s = s + _decays(log_decay, torch.tensor([k.shape[1]], device="cuda"))[:, :, None] * first
    return s


def _linear_fwd_plain(st, c):
    pos, scale, ld = _positions(c), 1 / math.sqrt(c["D"]), st["log_decay"]
    q, k, v = (_natural(st[x], pos).float() for x in "qkv")
    o = scale * _linear_scan(q, k, v, ld, st["state_in"], 1)
    out = [_ranked(o.to(torch.bfloat16), pos, c["N"])]
    if c["state_out"]:
        out.append(_linear_state(k, v, ld, c["S"] - 1 - torch.arange(c["S"], device="cuda"), st["state_in"]))
    return out


def _linear_bwd_plain(st, c):
    pos, scale, ld = _positions(c), 1 / math.sqrt(c["D"]), st["log_decay"]
    q, k, v, do = (_natural(st[x], pos).float() for x in ("q", "k", "v", "dout"))
    s0, ds = st["state_in"], st["dstate"]
    dq = scale * _linear_scan(do, v, k, ld, None if s0 is None else s0.transpose(-1, -2), 1)
    back = [x.flip(1) for x in (q * scale, k, v, do)]
    dk = _linear_scan(back[2], back[3], back[0], ld, None if ds is None else ds.transpose(-1, -2), 0).flip(1)
    dv = _linear_scan(back[1], back[0], back[3], ld, ds, 0).flip(1)
    out = [_ranked(x.to(torch.bfloat16), pos, c["N"]) for x in (dq, dk, dv)]
    if c["state_in"]:
        out.append(_linear_state(q * scale, do, ld, 1 + torch.arange(c["S"], device="cuda"), ds))
    return out


def _linear_step_plain(st, c):
    ld, T = st["log_decay"], c["T"]
    q, k, v = (st[x].float() for x in "qkv")
    o = (1 / math.sqrt(c["D"])) * _linear_scan(q, k, v, ld, st["state"], 1)
    st["state"].copy_(_linear_state(k, v, ld, T - 1 - torch.arange(T, device="cuda"), st["state"]))
    return [o.to(torch.bfloat16), st["state"]]


def _seen(st, c):
    """Which cache row each drafted token sees: [B, T, cap]."""
    T = c["T"]
    row = torch.arange(c["cap"], device="cuda")[None]
    draft = row - st["lengths"][:, None]                                # [B, cap]
    bit = (st["tree"][:, :, None] >> draft.clamp(0, T - 1)[:, None]) & 1
    return (draft < 0)[:, None] | ((draft >= 0) & (draft < T))[:, None] & (bit == 1)


def _cache_plain(st, c):
    B, T, Hq, Hkv, D = (c[x] for x in ("B", "T", "Hq", "Hkv", "D"))
    seen = _seen(st, c)[:, None, None]                                  # [B, 1, 1, T, cap]
    q = st["q"].float().reshape(B, T, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4)
    k = st["k"].float().permute(0, 2, 3, 1)[:, :, None]                 # [B, Hkv, 1, D, cap]
    v = st["v"].float().permute(0, 2, 1, 3)[:, :, None]
    s = (q.reshape(B, Hkv, 1, -1, D) @ k).reshape(B, Hkv, Hq // Hkv, T, -1) / math.sqrt(D)
    s = torch.where(seen, s, -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(s - m)
    total = p.sum(-1, keepdim=True)
    o = (p.reshape(B, Hkv, 1, -1, c["cap"]) @ v).reshape(B, Hkv, Hq // Hkv, T, D) / torch.where(total > 0, total, 1.0)
    lse = (m + torch.log(total))[..., 0].reshape(B, Hq, T)
    return [o.permute(0, 3, 1, 2, 4).reshape(B, T, Hq, D).to(torch.bfloat16), lse]


# ---------------------------------------------------- the definitions, in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    c = st["case"]
    with torch.no_grad():
        if c["op"] == "rope":
            return _rope_exact(st, c)
        if c["op"] == "linear_fwd":
            return _linear_fwd_exact(st, c)
        if c["op"] == "linear_bwd":
            return _linear_bwd_exact(st, c)
        if c["op"] == "linear_step":
            return _linear_step_exact(st, c)
        return _cache_exact(st, c)


def _rope_exact(st, c):
    """One complex multiplication per feature pair, token by token in the order of the output."""
    B, S, H, D, N = (c[x] for x in "BSHDN")
    first = [sum(st["sections"][:a]) for a in range(len(st["sections"]))]
    angle = torch.empty(B, S, D // 2, dtype=torch.float64, device="cuda")
    for a, (f, n) in enumerate(zip(first, st["sections"])):
        for j in range(n):
            t = 10000.0 ** (-j / n) if c["freqs"] == "per_axis" else 10000.0 ** (-2 * (f + j) / D)
            angle[:, :, f + j] = st["positions"][a].double() * t
    turn = torch.polar(torch.ones_like(angle), -angle if c["inverse"] else angle)

    def rotate(x, t):   # x [..., heads, D], t [..., D/2]
        x = x.double()
        z = torch.complex(x[..., :D // 2], x[..., D // 2:]) if c["pairing"] == "half" else torch.view_as_complex(
            x.reshape(*x.shape[:-1], D // 2, 2).contiguous())
        z = z * t[..., None, :]
        return torch.cat([z.real, z.imag], -1) if c["pairing"] == "half" else torch.view_as_real(z).flatten(-2)

    x, T = st["x"], S // N
    if c["layout"] == "ulysses":
        if c["inverse"]:
            out = torch.empty(N, B, T, H, D, dtype=torch.float64, device="cuda")
            for g in range(N):
                for r in range(N):
                    at = slice(r * T, (r + 1) * T)
                    out[r, :, :, g * (H // N):(g + 1) * (H // N)] = rotate(x[g][:, at], turn[:, at])
            return out
        out = torch.empty(N, B, S, H // N, D, dtype=torch.float64, device="cuda")
        for g in range(N):
            for r in range(N):
                at = slice(r * T, (r + 1) * T)
                out[g][:, at] = rotate(x[r][:, :, g * (H // N):(g + 1) * (H // N)], turn[:, at])
        return out
    C = S // (2 * N)
    out = torch.empty((B, S, H, D) if c["inverse"] else (N, B, T, H, D), dtype=torch.float64, device="cuda")
    for r in range(N):
        pieces = [(0, r * C, C), (C, (2 * N - 1 - r) * C, C)] if c["layout"] == "zigzag" else [(0, r * T, T)]
        for local, glob, n in pieces:
            li, gi = slice(local, local + n), slice(glob, glob + n)
            if c["inverse"]:
                out[:, gi] = rotate(x[r][:, li], turn[:, gi])
            else:
                out[r][:, li] = rotate(x[:, gi], turn[:, gi])
    return out


def _by_heads(x, c, pos):
    """Rank-major [N, B, T, H, D] -> fp64 [B, H, S, D] in natural order."""
    return _natural(x, pos).double().permute(0, 2, 1, 3).contiguous()


def _from_heads(x, c, pos):
    return _ranked(x.permute(0, 2, 1, 3), pos, c["N"])


def _blocks(S):
    return [(i, min(S, i + 256)) for i in range(0, S, 256)]


def _linear_fwd_exact(st, c):
    pos, ld, S, scale = _positions(c), st["log_decay"].double(), c["S"], 1 / math.sqrt(c["D"])
    q, k, v = (_by_heads(st[x], c, pos) for x in "qkv")
    o = torch.empty_like(v)
    t = torch.arange(S, device="cuda", dtype=torch.float64)
    for i, j in _blocks(S):   # rows i..j against every earlier token
        w = torch.exp(ld[:, None, None] * (t[i:j, None] - t[None, :j]).clamp(min=0)) * (t[i:j, None] >= t[None, :j])
        o[:, :, i:j] = ((q[:, :, i:j] @ k[:, :, :j].transpose(-1, -2)) * w) @ v[:, :, :j]
        if st["state_in"] is not None:
            o[:, :, i:j] += torch.exp(ld[:, None] * (t[i:j] + 1))[:, :, None] * (q[:, :, i:j] @ st["state_in"].double())
    out = [_from_heads(o * scale, c, pos)]
    if c["state_out"]:
        w = torch.exp(ld[:, None] * (S - 1 - t))[:, :, None]
        s = (k * w).transpose(-1, -2) @ v
        if st["state_in"] is not None:
            s = s + torch.exp(ld * S)[:, None, None] * st["state_in"].double()
        out.append(s)
    return out


def _linear_bwd_exact(st, c):
    pos, ld, S, scale = _positions(c), st["log_decay"].double(), c["S"], 1 / math.sqrt(c["D"])
    q, k, v, do = (_by_heads(st[x], c, pos) for x in ("q", "k", "v", "dout"))
    dq, dk, dv = torch.empty_like(q), torch.zeros_like(k), torch.zeros_like(v)
    t = torch.arange(S, device="cuda", dtype=torch.float64)
    for i, j in _blocks(S):
        w = scale * torch.exp(ld[:, None, None] * (t[i:j, None] - t[None, :j]).clamp(min=0)) * (t[i:j, None] >= t[None, :j])
        p = (q[:, :, i:j] @ k[:, :, :j].transpose(-1, -2)) * w
        dp = (do[:, :, i:j] @ v[:, :, :j].transpose(-1, -2)) * w
        dq[:, :, i:j] = dp @ k[:, :, :j]
        dk[:, :, :j] += dp.transpose(-1, -2) @ q[:, :, i:j]
        dv[:, :, :j] += p.transpose(-1, -2) @ do[:, :, i:j]
    up = scale * torch.exp(ld[:, None] * (t + 1))[:, :, None]          # weight of the first state in each output
    if st["state_in"] is not None:
        dq += up * (do @ st["state_in"].double().transpose(-1, -2))
    if st["dstate"] is not None:
        g, w = st["dstate"].double(), torch.exp(ld[:, None] * (S - 1 - t))[:, :, None]
        dk += w * (v @ g.transpose(-1, -2))
        dv += w * (k @ g)
    out = [_from_heads(x, c, pos) for x in (dq, dk, dv)]
    if c["state_in"]:
        ds = (q * up).transpose(-1, -2) @ do
        if st["dstate"] is not None:
            ds = ds + torch.exp(ld * S)[:, None, None] * st["dstate"].double()
        out.append(ds)
    return out


def _linear_step_exact(st, c):
    d = torch.exp(st["log_decay"].double())[None, :, None, None]
    s = st["state"].double()
    o = []
    for t in range(c["T"]):
        q, k, v = (st[x][:, t].double() for x in "qkv")                # [B, H, D]
        s = d * s + k[..., :, None] * v[..., None, :]
        o.append((q[..., None, :] @ s)[..., 0, :] / math.sqrt(c["D"]))
    return [torch.stack(o, 1), s]


def _cache_exact(st, c):
    B, T, Hq, Hkv, D = (c[x] for x in ("B", "T", "Hq", "Hkv", "D"))
    o = torch.zeros(B, T, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq, T), -math.inf, dtype=torch.float64, device="cuda")
    tree = st["tree"].cpu()
    for b, n in enumerate(_lengths(c)):
        seen = torch.ones(T, n + T, dtype=torch.bool)
        for t in range(T):
            for u in range(T):
                seen[t, n + u] = bool((int(tree[b, t]) >> u) & 1)
        seen = seen.cuda()
        for h in range(Hkv):
            heads = range(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            k, v = st["k"][b, :n + T, h].double(), st["v"][b, :n + T, h].double()
            s = st["q"][b][:, heads].double() @ k.T / math.sqrt(D)     # [T, G, n + T]
            s = s.masked_fill(~seen[:, None], -math.inf)
            o[b][:, heads] = torch.softmax(s, -1) @ v
            lse[b, heads] = torch.logsumexp(s, -1).T
    return [o, lse]


# ----------------------------------------------------------------------------- work
def work(case):
    c = case
    if c["op"] == "rope":
        n = c["B"] * c["S"] * c["H"] * c["D"]
        axes = c["sections"].count(",") + 1
        return {"bytes": 4 * n + 4 * axes * c["B"] * c["S"], "flops": 3 * n}
    if c["op"] in ("linear_fwd", "linear_bwd"):
        n, state = c["B"] * c["S"] * c["H"] * c["D"], 4 * c["B"] * c["H"] * c["D"] ** 2
        tensors, products = (4, 2) if c["op"] == "linear_fwd" else (7, 5)
        # products with (or onto) a D x D state: 2 D^2 each per token and head
        states = c["state_in"] * (1 if c["op"] == "linear_fwd" else 2) + c["state_out"]
        return {"bytes": 2 * tensors * n + states * state, "flops": 2 * products * n * c["D"]}
    if c["op"] == "linear_step":
        n, state = c["B"] * c["T"] * c["H"] * c["D"], 4 * c["B"] * c["H"] * c["D"] ** 2
        return {"bytes": 8 * n + 2 * state, "flops": 4 * n * c["D"]}
    rows = sum(_lengths(c)) + c["B"] * c["T"]
    qo = c["B"] * c["T"] * c["Hq"]
    pairs = sum(n + (c["T"] + 1) / 2 for n in _lengths(c)) * c["T"] * c["Hq"]
    return {"bytes": 4 * rows * c["Hkv"] * c["D"] + 4 * qo * c["D"] + 4 * qo, "flops": 4 * pairs * c["D"]}
