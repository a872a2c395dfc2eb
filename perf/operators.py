"""The serving and long-context operators beside the dense attention: what is
measured of them, and their plain forms.

Four operators that are used together:
  rope          rotary positions with one or several axes, on queries and keys
                in one launch; ``inverse`` is its gradient.
  append        rotation of new queries and keys, and the append of new keys and
                values to a paged e4m3 cache with one power-of-two scale per
                page and head.
  paged         attention over that cache: one query token per sequence, a few
                drafted tokens, or a chunk of a prompt; grouped heads, window
                and sinks.
  window        sliding-window attention with sinks, forward and backward.

Where ``own`` is false, ``run`` computes them with elementary torch operations
in 32 bits and rounds once at the end; where it is true, it calls the
framework.
"""

import math

import torch

own = False

F8 = torch.float8_e4m3fn
E_MIN, E_MAX = -100, 120  # exponents of a cache block's scale


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # One decode step of eight sequences: latency alone.
        dict(name="rope_token", op="rope", layout="packed", B=1, H=32, Hkv=8, N=8, d=128, rot=128, axes=1,
             interleaved=False, inverse=False),
        # A prompt of images or video: time, height and width positions.
        dict(name="rope_axes3", op="rope", layout="dense", B=2, H=32, Hkv=8, N=8191, d=128, rot=128, axes=3,
             interleaved=False, inverse=False),
        # The gradient of a partial rotation in a training batch, odd length.
        dict(name="rope_grad_partial", op="rope", layout="packed", B=1, H=16, Hkv=16, N=16381, d=64, rot=32, axes=1,
             interleaved=True, inverse=True),
        # One new token for each of 128 sequences.
        dict(name="append_decode", op="append", B=128, H=32, Hkv=8, new=1, ctx=8192, page=64, d=128, rot=128, axes=1,
             interleaved=False),
        # Prompts of ragged lengths entering the cache behind a shared context.
        dict(name="append_prompt", op="append", B=6, H=32, Hkv=8, new=4001, ctx=6000, page=16, d=128, rot=128, axes=3,
             interleaved=False),
        # One sequence answering in a chat: a short cache, window and sinks.
        dict(name="decode_one", op="paged", B=1, H=8, Hkv=8, new=1, ctx=2047, page=16, d=64, window=512, sinks=4),
        # A full serving batch with ragged contexts.
        dict(name="decode_batch", op="paged", B=64, H=32, Hkv=8, new=1, ctx=32768, page=64, d=128, window=0, sinks=0),
        # Five drafted tokens per sequence checked in one call.
        dict(name="verify_drafts", op="paged", B=16, H=32, Hkv=8, new=5, ctx=16200, page=32, d=128, window=0, sinks=0),
        # Chunks of long prompts over what the cache holds already.
        dict(name="prompt_chunk", op="paged", B=2, H=16, Hkv=2, new=2048, ctx=16384, page=64, d=128, window=0, sinks=0),
        # A long prompt through a layer with a window.
        dict(name="window_prompt", op="window", B=2, H=32, Hkv=8, N=8192, M=8192, d=64, window=1024, sinks=4,
             train=False),
        # One training step of a windowed layer.
        dict(name="window_step", op="window", B=1, H=16, Hkv=4, N=8192, M=8192, d=128, window=1024, sinks=4,
             train=True),
        # A short training step with wide heads and odd sizes.
        dict(name="window_step_wide", op="window", B=2, H=8, Hkv=2, N=1001, M=1203, d=256, window=129, sinks=1,
             train=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "paged", "paged", "window", "window"])
    d = rng.choice([64, 128, 256])
    hkv = rng.choice([1, 2, 4, 8])
    h = hkv * rng.choice([1, 2, 4, 8] if d < 256 else [1, 2, 4])
    if op == "rope":
        b = rng.choice([1, 1, 2, 3])
        return dict(op=op, layout="dense" if b > 1 else rng.choice(["dense", "packed"]), B=b, H=h, Hkv=hkv,
                    N=_log(rng, 1, max(1, 16384 * 1024 // (b * h * d))), d=d,
                    rot=rng.choice([d, d, d // 2]), axes=rng.choice([1, 1, 2, 3]),
                    interleaved=rng.random() < 0.5, inverse=rng.random() < 0.5)
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        b = _log(rng, 1, 64)
        new = _log(rng, 1, max(1, 16384 // b))
        return dict(op=op, B=b, H=h, Hkv=hkv, new=new, ctx=new + _log(rng, 1, 8000), page=page, d=d,
                    rot=rng.choice([d, d, d // 2]), axes=rng.choice([1, 1, 2, 3]), interleaved=rng.random() < 0.5)
    window = rng.choice([0, 0, _log(rng, 1, 4096)])
    sinks = rng.choice([0, 1, 4, 64]) if window else 0
    if op == "paged":
        kind = rng.choice(["token", "drafts", "chunk"])
        b = _log(rng, 1, {"token": 48, "drafts": 12, "chunk": 3}[kind])
        new = {"token": 1, "drafts": rng.randint(2, 8), "chunk": _log(rng, 17, 1024)}[kind]
        return dict(op=op, B=b, H=h, Hkv=hkv, new=new, ctx=max(new, _log(rng, 16, 16000)), page=page, d=d,
                    window=window, sinks=sinks)
    n = _log(rng, 1, 4096)
    m = n if rng.random() < 0.6 else _log(rng, 1, 4096)
    b = rng.choice([1, 2])
    while b * h * n * m > 6 * 4096 * 4096 and h > hkv:
        h //= 2
    while b * h * n * m > 6 * 4096 * 4096 and hkv > 1:
        h, hkv = h // 2, hkv // 2
    return dict(op=op, B=b, H=h, Hkv=hkv, N=n, M=m, d=d, window=window, sinks=sinks, train=rng.random() < 0.6)


def _lengths(case):
    """New tokens and cache length (new ones among it) of each sequence: ragged, and of the case alone."""
    B, new, ctx = case["B"], case["new"], case["ctx"]
    n = [new if new < 16 else new - (b * 7919 % (new // 3 + 1)) for b in range(B)]
    k = [max(n[b], ctx - (b * 104729 % (ctx * 3 // 4 + 1))) for b in range(B)]
    return n, k


def _pairs(n, k, window, sinks):
    """Visible (query, key) pairs of n queries at the end of k keys."""
    total = 0
    if window <= 0:
        lo = max(0, k - n)  # position of the first query that sees a key, and of those before it none
        return sum(range(lo + 1, k + 1))
    for p in range(max(0, k - n), k):
        total += min(p + 1, window) + min(sinks, max(0, p + 1 - window))
    return total


def work(case):
    d, H, Hkv = case["d"], case["H"], case["Hkv"]
    if case["op"] == "rope":
        T = case["B"] * case["N"]
        heads = H + Hkv
        # each value read and written once, the table's rows of the positions, the positions
        return {"bytes": T * heads * d * 4 + T * case["rot"] * 4 + T * case["axes"] * 4,
                "flops": T * heads * case["rot"] * 3}
    if case["op"] == "append":
        n, k = _lengths(case)
        T = sum(n)
        # q read and written, k and v read, codes written, the table's rows
        return {"bytes": T * d * (4 * H + (4 + 2) * Hkv) + T * case["rot"] * 4,
                "flops": T * (H + Hkv) * case["rot"] * 3 + T * Hkv * d * 4}
    if case["op"] == "paged":
        n, k = _lengths(case)
        W, S = case["window"], case["sinks"]
        keys = sum(kb if W <= 0 else min(kb, W + nb - 1 + S) for nb, kb in zip(n, k))
        pairs = sum(_pairs(nb, kb, W, S) for nb, kb in zip(n, k))
        return {"bytes": keys * Hkv * d * 2 + sum(n) * H * (4 * d + 4), "flops": 4 * H * d * pairs}
    B, N, M = case["B"], case["N"], case["M"]
    pairs = B * H * _pairs(N, M, case["window"], case["sinks"])
    io = 2 * d * (B * H * N + 2 * B * Hkv * M)  # q, k, v
    fwd = {"bytes": io + B * H * N * (2 * d + 4), "flops": 4 * d * pairs}
    if not case["train"]:
        return fwd
    return {"bytes": fwd["bytes"] + io + B * H * N * (4 * d + 4) + io, "flops": fwd["flops"] + 10 * d * pairs}


# ----------------------------------------------------------------- the inputs
def _sections(case):
    half = case["rot"] // 2
    a = case["axes"]
    if a == 1:
        return [half]
    first = half // 4 if a == 3 else half // 2
    rest = (half - first) // (a - 1)
    return [first] + [rest] * (a - 2) + [half - first - rest * (a - 2)]


def _table(rot, rows, device):
    """cos | sin of row * 10000^(-2i / rot), formed in 64 bits."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot)
    ang = torch.arange(rows, dtype=torch.float64, device=device)[:, None] * inv
    return torch.cat([ang.cos(), ang.sin()], 1).float()


def _positions(case, base, total, g):
    """int32 [axes][total]: text positions on the first axis, grid coordinates on the others."""
    rows = [base]
    for a in range(1, case["axes"]):
        rows.append((torch.arange(total, device="cuda") // (1 if a == 1 else 24)) % 24 + a)
    return torch.stack(rows).to(torch.int32).contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(torch.bfloat16)

    d, H, Hkv = case["d"], case["H"], case["Hkv"]
    st = dict(case)
    if case["op"] == "rope":
        B, N = case["B"], case["N"]
        rows = 32768 if N <= 32768 - 64 else N + 64
        shift = int(torch.randint(0, rows - N - 32, (1,), generator=g, device="cuda"))
        base = (torch.arange(N, device="cuda") + shift).repeat(B)
        pos = _positions(case, base, B * N, g)
        st["table"] = _table(case["rot"], rows, "cuda")
        if case["layout"] == "dense":
            st.update(q=normal(B, H, N, d), k=normal(B, Hkv, N, d), positions=pos.view(case["axes"], B, N))
        else:
            # queries and keys as a projection leaves them: one row per token
            qk = normal(N, H + Hkv, d)
            st.update(q=qk[:, :H], k=qk[:, H:], positions=pos)
        st["sections"] = _sections(case)
        return st
    if case["op"] in ("append", "paged"):
        n, k = _lengths(case)
        B, page = case["B"], case["page"]
        total = sum(n)
        pages = [-(-x // page) for x in k]
        width = max(pages)
        num = sum(pages) + 7
        perm = torch.randperm(num, generator=g, device="cuda")
        table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b in range(B):
            table[b, : pages[b]] = perm[at : at + pages[b]].to(torch.int32)
            at += pages[b]
        cu = [0]
        for x in n:
            cu.append(cu[-1] + x)
        # Blocks of tokens of different sizes of values: scales of several powers of two.
        amp = torch.exp2(torch.randint(-2, 3, (num, Hkv, 1, 1), generator=g, device="cuda").float())
        cache = []
        for _ in range(2):
            vals = torch.randn((num, Hkv, page, d), generator=g, device="cuda")
            vals *= amp if case["op"] == "append" else amp.sqrt()
            e = _exponent(vals.abs().amax((2, 3)))
            cache.append((((vals * torch.exp2(-e.float())[:, :, None, None]).to(F8)), torch.exp2(e.float())))
        st.update(k_cache=cache[0][0], k_scale=cache[0][1], v_cache=cache[1][0], v_scale=cache[1][1], page_table=table,
                  cu=torch.tensor(cu, dtype=torch.int32, device="cuda"),
                  seqlens_k=torch.tensor(k, dtype=torch.int32, device="cuda"), max_q=max(n), max_k=max(k))
        if case["op"] == "paged":
            st["q"] = normal(total, H, d)
            return st
        qkv = normal(total, H + 2 * Hkv, d, scale=2.0)
        st.update(q=qkv[:, :H], k=qkv[:, H : H + Hkv], v=qkv[:, H + Hkv :])
        seq = torch.repeat_interleave(torch.arange(B, device="cuda"), torch.tensor(n, device="cuda"))
        st["slot"] = torch.arange(total, device="cuda") - st["cu"][seq].long() + (st["seqlens_k"][seq].long() - torch.tensor(n, device="cuda")[seq])
        st["seq"] = seq
        st["positions"] = _positions(case, st["slot"], total, g)
        st["table"] = _table(case["rot"], max(k) + 64, "cuda")
        st["sections"] = _sections(case)
        return st
    B, N, M = case["B"], case["N"], case["M"]
    st.update(q=normal(B, H, N, d), k=normal(B, Hkv, M, d), v=normal(B, Hkv, M, d))
    if case["train"]:
        st["dout"] = normal(B, H, N, d)
    return st


# ------------------------------------------------------------- the plain forms
def _exponent(amax):
    """The least e with amax <= 448 * 2^e, within the scale's range."""
    f, ex = torch.frexp(amax.float())
    e = ex - 9 + (f > 0.875).to(ex.dtype)
    e = torch.where(amax > 0, e, torch.full_like(e, E_MIN))
    return e.clamp(E_MIN, E_MAX)


def _cos_sin(st):
    """[..., rot / 2] cosines and sines of each token, each pair by its axis."""
    half = st["rot"] // 2
    axis = torch.repeat_interleave(torch.arange(st["axes"], device="cuda"), torch.tensor(st["sections"], device="cuda"))
    pos = st["positions"].long()[axis].movedim(0, -1)  # [..., half]
    col = torch.arange(half, device="cuda")
    return st["table"][pos, col], st["table"][pos, col + half]


def _rotate(x, cos, sin, rot, interleaved, inverse):
    x = x.float()
    if inverse:
        sin = -sin
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., : rot // 2], x[..., rot // 2 : rot]
        y[..., : rot // 2], y[..., rot // 2 : rot] = a * cos - b * sin, b * cos + a * sin
    return y


def _plain_rope(st):
    cos, sin = _cos_sin(st)
    dim = 1 if st["layout"] == "dense" else -2
    cos, sin = cos.unsqueeze(dim), sin.unsqueeze(dim)
    args = (cos, sin, st["rot"], st["interleaved"], st["inverse"])
    return _rotate(st["q"], *args).bfloat16(), _rotate(st["k"], *args).bfloat16()


def _plain_append_one(x, cache, scale, st):
    """New rows x [tokens][Hkv][d] (32 bits) into the cache, in place."""
    page, Hkv, d = st["page"], st["Hkv"], st["d"]
    block = st["slot"] // page
    touched = st["page_table"][st["seq"], block].long()  # page of each token
    inside = st["slot"] - block * page
    pages, inv = torch.unique(touched, return_inverse=True)
    first = torch.full((pages.numel(),), page, dtype=torch.long, device="cuda").scatter_reduce(0, inv, inside, "amin")
    amax = torch.zeros((pages.numel(), Hkv), device="cuda").index_reduce_(0, inv, x.abs().amax(-1), "amax")
    e_new = _exponent(amax)
    old = torch.where((first > 0)[:, None], scale[pages], torch.zeros_like(amax))
    s = torch.maximum(torch.exp2(e_new.float()), old)
    held = cache[pages].float()  # tokens before the first new one are kept, at the block's new scale
    again = (held * (old / s)[:, :, None, None]).to(F8)
    keep = torch.arange(page, device="cuda")[None, :] < first[:, None]
    codes = torch.where(keep[:, None, :, None], again.view(torch.uint8), cache[pages].view(torch.uint8))
    codes[inv, :, inside] = (x / s[inv][:, :, None]).to(F8).view(torch.uint8)
    cache.view(torch.uint8)[pages] = codes
    scale[pages] = s


def _plain_append(st):
    cos, sin = _cos_sin(st)
    cos, sin = cos.unsqueeze(-2), sin.unsqueeze(-2)
    args = (cos, sin, st["rot"], st["interleaved"], False)
    _plain_append_one(_rotate(st["k"], *args), st["k_cache"], st["k_scale"], st)
    _plain_append_one(st["v"].float(), st["v_cache"], st["v_scale"], st)
    return _rotate(st["q"], *args).bfloat16()


def _visible(pos, keys, window, sinks):
    """pos [..., n, 1] positions of queries, keys [k]: key j is seen iff j <= p and (j > p - window or j < sinks)."""
    m = keys <= pos
    if window > 0:
        m = m & ((keys > pos - window) | (keys < sinks))
    return m


def _softmax(s, m):
    """Row maxima, exponentials and sums of scores s with visible places m; rows with none give 0 and -inf."""
    s = s.masked_fill(~m, -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(s - top)
    l = p.sum(-1, keepdim=True)
    return p / l.clamp_min(1e-38), (top + torch.log(l)).squeeze(-1)


def _plain_paged(st):
    B, H, Hkv, d, n = st["B"], st["H"], st["Hkv"], st["d"], st["max_q"]
    total, width, page = st["q"].shape[0], st["page_table"].shape[1], st["page"]
    lq = (st["cu"][1:] - st["cu"][:-1]).long()
    seq = torch.repeat_interleave(torch.arange(B, device="cuda"), lq, output_size=total)
    i = torch.arange(total, device="cuda") - st["cu"][seq].long()
    q = torch.zeros((B, n, H, d), device="cuda")
    q[seq, i] = st["q"].float()
    q = q.view(B, n, Hkv, H // Hkv, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, d)
    ids = st["page_table"].clamp_min(0).long()

    def values(cache, scale):
        x = cache[ids].float() * scale[ids][..., None, None]  # [B, width, Hkv, page, d]
        return x.permute(0, 2, 1, 3, 4).reshape(B, Hkv, width * page, d)

    s = q @ values(st["k_cache"], st["k_scale"]).transpose(-1, -2) * (d ** -0.5)
    pos = (st["seqlens_k"].long() - lq)[:, None] + torch.arange(n, device="cuda")
    keys = torch.arange(width * page, device="cuda")
    m = _visible(pos[:, :, None], keys, st["window"], st["sinks"])  # [B, n, keys]
    s = s.view(B, Hkv, H // Hkv, n, -1)
    p, lse = _softmax(s, m[:, None, None])
    v = values(st["v_cache"], st["v_scale"])
    o = (p.reshape(B, Hkv, -1, p.shape[-1]) @ v).view(B, Hkv * (H // Hkv), n, d)
    return o[seq, :, i].bfloat16(), lse.reshape(B, H, n)[seq, :, i].t().contiguous()


def _plain_window(st):
    B, H, Hkv, N, M, d = (st[x] for x in ("B", "H", "Hkv", "N", "M", "d"))
    scale = d ** -0.5
    g = H // Hkv
    q = st["q"].float().view(B, Hkv, g, N, d)
    k, v = st["k"].float()[:, :, None], st["v"].float()[:, :, None]
    pos = torch.arange(N, device="cuda")[:, None] + (M - N)
    m = _visible(pos, torch.arange(M, device="cuda"), st["window"], st["sinks"])
    p, lse = _softmax(q @ k.transpose(-1, -2) * scale, m)
    o = p @ v
    outs = [o.reshape(B, H, N, d).bfloat16(), lse.reshape(B, H, N)]
    if st["train"]:
        do = st["dout"].float().view(B, Hkv, g, N, d)
        dv = (p.transpose(-1, -2) @ do).sum(2)
        ds = p * (do @ v.transpose(-1, -2) - (do * o).sum(-1, keepdim=True))
        dq = ds @ k * scale
        dk = (ds.transpose(-1, -2) @ q).sum(2) * scale
        outs += [dq.reshape(B, H, N, d).bfloat16(), dk.bfloat16(), dv.bfloat16()]
    return outs


# ------------------------------------------------------------------- one pass
def run(st):
    op = st["op"]
    if own:
        import exact_attention_80_gb300 as fa

        if op == "rope":
            return fa.rope(st["q"], st["k"], st["table"], st["positions"], sections=st["sections"],
                           interleaved=st["interleaved"], inverse=st["inverse"])
        if op == "append":
            q = fa.kv_append_fp8(st["q"], st["k"], st["v"], st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"],
                                 st["page_table"], st["cu"], st["seqlens_k"], st["max_q"], table=st["table"],
                                 positions=st["positions"], sections=st["sections"], interleaved=st["interleaved"])
            return q, st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"]
        if op == "paged":
            return fa.attention_paged_fp8(st["q"], st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"],
                                          st["page_table"], st["cu"], st["seqlens_k"], st["max_q"], st["max_k"],
                                          window=st["window"], sinks=st["sinks"])
        o, lse = fa.attention_window(st["q"], st["k"], st["v"], st["window"], st["sinks"])
        if not st["train"]:
            return o, lse
        return (o, lse, *fa.attention_window_backward(st["q"], st["k"], st["v"], o, lse, st["dout"], st["window"],
                                                      st["sinks"]))
    if op == "rope":
        return _plain_rope(st)
    if op == "append":
        q = _plain_append(st)
        return q, st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"]
    if op == "paged":
        return _plain_paged(st)
    return tuple(_plain_window(st))


# -------------------------------------------- the definitions again, in 64 bits
def _exact_turn(x, st, t, sign):
    """Rows x [heads][d] of one stretch of tokens t [tokens]: x [tokens][heads][d] turned pair by pair, as complex numbers."""
    rot, half = st["rot"], st["rot"] // 2
    x = x.double()
    pos = st["positions"].reshape(st["axes"], -1)[:, t].long()
    angle_cos = torch.empty((len(t), half), dtype=torch.float64, device=x.device)
    angle_sin = torch.empty_like(angle_cos)
    at = 0
    for axis, size in enumerate(st["sections"]):
        rows = st["table"][pos[axis]].double()
        angle_cos[:, at : at + size] = rows[:, at : at + size]
        angle_sin[:, at : at + size] = rows[:, half + at : half + at + size]
        at += size
    turn = torch.complex(angle_cos, sign * angle_sin)[:, None, :]
    out = x.clone()
    if st["interleaved"]:
        z = torch.view_as_complex(x[..., :rot].reshape(*x.shape[:-1], half, 2).contiguous()) * turn
        out[..., :rot] = torch.view_as_real(z).reshape(*x.shape[:-1], rot)
    else:
        z = torch.complex(x[..., :half].contiguous(), x[..., half:rot].contiguous()) * turn
        out[..., :half], out[..., half:rot] = z.real, z.imag
    return out


def _exact_rope(st):
    sign = -1.0 if st["inverse"] else 1.0
    outs = []
    for x in (st["q"], st["k"]):
        if st["layout"] == "packed":
            outs.append(_exact_turn(x, st, torch.arange(x.shape[0], device=x.device), sign))
        else:
            B, heads, N, d = x.shape
            rows = x.transpose(1, 2).reshape(B * N, heads, d)
            y = _exact_turn(rows, st, torch.arange(B * N, device=x.device), sign)
            outs.append(y.view(B, N, heads, d).transpose(1, 2).contiguous())
    return tuple(outs)


def _exact_append(st):
    """q, and the four parts of the cache, block by block: codes as the e4m3 values they are."""
    T = st["q"].shape[0]
    t = torch.arange(T, device="cuda")
    q = _exact_turn(st["q"], st, t, 1.0)
    outs = [q]
    new = {"k": _exact_turn(st["k"], st, t, 1.0), "v": st["v"].double()}
    seqs, lens = st["cu"].tolist(), st["seqlens_k"].tolist()
    page = st["page"]
    codes, scales = {}, {}
    for which in ("k", "v"):
        c, s = st[which + "_cache"].double(), st[which + "_scale"].double()
        for b in range(st["B"]):
            n = seqs[b + 1] - seqs[b]
            pos = lens[b] - n
            done = 0
            while done < n:
                blk, lo = divmod(pos + done, page)
                count = min(page - lo, n - done)
                x = new[which][seqs[b] + done : seqs[b] + done + count].transpose(0, 1)  # [Hkv][count][d]
                pg = st["page_table"][b, blk].long()
                amax = x.abs().amax((1, 2))
                f, ex = torch.frexp((amax / 448.0).clamp_min(2.0 ** E_MIN))  # f in [1/2, 1): a power of two has f = 1/2
                want = torch.exp2((ex - (f == 0.5).to(ex.dtype)).clamp(E_MIN, E_MAX).double())
                if lo > 0:
                    want = torch.maximum(want, s[pg])
                    c[pg, :, :lo] = (c[pg, :, :lo] * (s[pg] / want)[:, None, None]).to(F8).double()
                c[pg, :, lo : lo + count] = _round_e4m3(x / want[:, None, None])
                s[pg] = want
                done += count
        codes[which], scales[which] = c, s
    return tuple(outs + [codes["k"], codes["v"], scales["k"], scales["v"]])


def _round_e4m3(x):
    """64-bit values rounded to three mantissa bits (nearest, ties to even), least step 2^-9."""
    _, ex = torch.frexp(x)
    step = torch.exp2((ex - 4).clamp_min(-9).double())
    return torch.round(x / step) * step


def _exact_rows(q, k, v, first, scale, window, sinks, do=None):
    """One head: queries q [n][d] at positions first.., keys and values [m][d], 64 bits, a stretch of queries at a time.
    Returns o, lse and, with do, dq, dk, dv."""
    n, m = q.shape[0], k.shape[0]
    o, lse = torch.zeros_like(q), torch.full((n,), -math.inf, dtype=torch.float64, device=q.device)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    j = torch.arange(m, device=q.device)
    for a in range(0, n, 1024):
        z = min(n, a + 1024)
        p = torch.arange(first + a, first + z, device=q.device)[:, None]
        seen = j[None, :] <= p
        if window > 0:
            seen &= (p - j[None, :] < window) | (j[None, :] < sinks)
        s = (q[a:z] @ k.T) * scale
        s = torch.where(seen, s, torch.full_like(s, -math.inf))
        some = seen.any(1)
        lse[a:z] = torch.logsumexp(s, 1)
        w = torch.where(some[:, None], torch.exp(s - torch.where(some, lse[a:z], torch.zeros_like(lse[a:z]))[:, None]),
                        torch.zeros_like(s))
        o[a:z] = w @ v
        if do is not None:
            dv += w.T @ do[a:z]
            ds = w * (do[a:z] @ v.T - (do[a:z] * o[a:z]).sum(1, keepdim=True))
            dq[a:z] = ds @ k * scale
            dk += ds.T @ q[a:z] * scale
    return o, lse, dq, dk, dv


def _exact_paged(st):
    H, Hkv, d, page = st["H"], st["Hkv"], st["d"], st["page"]
    o = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros((H, st["q"].shape[0]), dtype=torch.float64, device="cuda")
    cu, lens = st["cu"].tolist(), st["seqlens_k"].tolist()
    for b in range(st["B"]):
        ids = st["page_table"][b, : -(-lens[b] // page)].long()
        for c in range(Hkv):
            k = (st["k_cache"][ids, c].double() * st["k_scale"][ids, c].double()[:, None, None]).reshape(-1, d)[: lens[b]]
            v = (st["v_cache"][ids, c].double() * st["v_scale"][ids, c].double()[:, None, None]).reshape(-1, d)[: lens[b]]
            for h in range(c * (H // Hkv), (c + 1) * (H // Hkv)):
                x = st["q"][cu[b] : cu[b + 1], h].double()
                o[cu[b] : cu[b + 1], h], lse[h, cu[b] : cu[b + 1]] = _exact_rows(
                    x, k, v, lens[b] - x.shape[0], d ** -0.5, st["window"], st["sinks"])[:2]
    return o, lse


def _exact_window(st):
    B, H, Hkv, d = st["B"], st["H"], st["Hkv"], st["d"]
    f64 = dict(dtype=torch.float64, device="cuda")
    o, lse = torch.empty(st["q"].shape, **f64), torch.empty(st["q"].shape[:3], **f64)
    dq, dk, dv = torch.empty(st["q"].shape, **f64), torch.zeros(st["k"].shape, **f64), torch.zeros(st["k"].shape, **f64)
    for b in range(B):
        for h in range(H):
            c = h // (H // Hkv)
            r = _exact_rows(st["q"][b, h].double(), st["k"][b, c].double(), st["v"][b, c].double(), st["M"] - st["N"],
                            d ** -0.5, st["window"], st["sinks"], st["dout"][b, h].double() if st["train"] else None)
            o[b, h], lse[b, h], dq[b, h] = r[:3]
            dk[b, c] += r[3]
            dv[b, c] += r[4]
    return (o, lse, dq, dk, dv) if st["train"] else (o, lse)


def exact(case, seed):
    st = prepare(case, seed)
    return {"rope": _exact_rope, "append": _exact_append, "paged": _exact_paged, "window": _exact_window}[case["op"]](st)
