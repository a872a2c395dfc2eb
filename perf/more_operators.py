"""Operators on ragged batches beside the paged cache and the windowed layers:
what is measured of them, and their plain forms.

Three kinds of calls that are used together:
  packed      causal attention over packed sequences of different lengths with
              grouped heads, a window and sinks, forward and backward.
  prefix      attention over the paged e4m3 cache for a batch whose sequences
              begin with the same pages, which are attended to once for all.
  read        keys and values of cached tokens back as packed bf16 tensors.

Where ``own`` is false, ``run`` computes them with elementary torch operations
in 32 bits and rounds once at the end; where it is true, it calls the
framework.
"""

import math

import torch

own = False

F8 = torch.float8_e4m3fn


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # A few short prompts that arrive together: latency alone.
        dict(name="prompts_short", op="packed", B=5, new=130, ctx=0, H=32, Hkv=8, d=128, window=0, sinks=0, train=False),
        # Whole prompts of very different lengths in one batch.
        dict(name="prompts_mixed", op="packed", B=8, new=8001, ctx=0, H=32, Hkv=8, d=128, window=0, sinks=0,
             train=False),
        # Chunks of prompts behind a context that was read back from the cache.
        dict(name="prompts_continued", op="packed", B=3, new=1500, ctx=16000, H=16, Hkv=2, d=64, window=0, sinks=0,
             train=False),
        # One training step of a layer on packed documents.
        dict(name="documents_step", op="packed", B=24, new=2047, ctx=0, H=16, Hkv=4, d=128, window=0, sinks=0,
             train=True),
        # The same with long documents and a window.
        dict(name="documents_step_window", op="packed", B=6, new=8191, ctx=0, H=16, Hkv=8, d=64, window=1024, sinks=4,
             train=True),
        # A short step with wide heads and odd sizes.
        dict(name="documents_step_wide", op="packed", B=7, new=777, ctx=0, H=8, Hkv=2, d=256, window=0, sinks=0,
             train=True),
        # Four chats behind the same instructions: latency.
        dict(name="prefix_chat", op="prefix", B=4, new=1, prefix=1024, suffix=100, H=8, Hkv=8, d=64, page=16),
        # A full serving batch behind one long document.
        dict(name="prefix_batch", op="prefix", B=64, new=1, prefix=16384, suffix=2000, H=32, Hkv=8, d=128, page=64),
        # Drafted tokens checked for every sequence of such a batch.
        dict(name="prefix_drafts", op="prefix", B=16, new=5, prefix=8160, suffix=4000, H=32, Hkv=8, d=128, page=32),
        # Wide heads, many query heads per kv head.
        dict(name="prefix_wide", op="prefix", B=31, new=1, prefix=4096, suffix=500, H=16, Hkv=2, d=256, page=128),
        # The context of one short chat read back.
        dict(name="read_one", op="read", B=1, new=500, Hkv=8, d=64, page=16),
        # The contexts of a batch read back behind a prefix that is held already.
        dict(name="read_batch", op="read", B=8, new=16200, Hkv=8, d=128, page=64),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["packed", "packed", "packed", "prefix", "prefix", "read"])
    d = rng.choice([64, 128, 256])
    hkv = rng.choice([1, 2, 4, 8])
    h = hkv * rng.choice([1, 2, 3, 4, 7, 8] if d < 256 else [1, 2, 3, 4])
    if op == "read":
        b = _log(rng, 1, 64)
        return dict(op=op, B=b, new=_log(rng, 1, max(1, 60000 * 1024 // (b * hkv * d))), Hkv=hkv, d=d, page=rng.choice([16, 32, 64, 128]))
    if op == "prefix":
        page = rng.choice([16, 32, 64, 128])
        kind = rng.choice(["token", "token", "drafts"])
        b = _log(rng, 1, 64 if kind == "token" else 16)
        new = 1 if kind == "token" else rng.randint(2, 8)
        return dict(op=op, B=b, new=new, prefix=page * max(1, _log(rng, 16, 16384) // page),
                    suffix=max(new, _log(rng, 1, 2000)), H=h, Hkv=hkv, d=d, page=page)
    window = rng.choice([0, 0, _log(rng, 1, 4096)])
    sinks = rng.choice([0, 1, 4, 64]) if window else 0
    train = rng.random() < 0.5
    b = _log(rng, 1, 48)
    new = _log(rng, 1, max(1, min(6000, 24000 // b)))
    ctx = 0 if train and rng.random() < 0.7 else rng.choice([0, _log(rng, 1, 4000)])
    while b * new * (new + 2 * ctx) * h * d > 4 * 4096 * 4096 * 16 * 128 and h > hkv:
        h = hkv * max(1, h // hkv // 2)
    while b * new * (new + 2 * ctx) * h * d > 4 * 4096 * 4096 * 16 * 128 and hkv > 1:
        h, hkv = h // 2, hkv // 2
    return dict(op=op, B=b, new=new, ctx=ctx, H=h, Hkv=hkv, d=d, window=window, sinks=sinks, train=train)


def _ragged(count, most, step):
    """Lengths of `count` sequences, the first the longest, others down to an eighth of it; every seventh a few tokens."""
    out = []
    for b in range(count):
        x = most - (b * step) % (7 * most // 8 + 1)
        out.append(max(1, x if b % 7 != 6 else min(x, 1 + b % 40)))
    return out


def _lengths(case):
    """Query tokens and keys of each sequence."""
    B = case["B"]
    if case["op"] == "packed":
        n = _ragged(B, case["new"], 7919)
        c = _ragged(B, case["ctx"], 104729) if case["ctx"] else [0] * B
        return n, [a + b for a, b in zip(n, c)]
    if case["op"] == "prefix":
        n = [case["new"]] * B
        s = [max(case["new"], x) for x in _ragged(B, case["suffix"], 7919)]
        return n, [case["prefix"] + x for x in s]
    n = _ragged(B, case["new"], 7919)
    first = [(b * 131) % 257 for b in range(B)]  # tokens of each sequence that are not read
    return n, [a + b for a, b in zip(n, first)]


def _pairs(n, k, window, sinks):
    """Visible (query, key) pairs of n queries at the end of k keys."""
    p0 = max(0, k - n)
    if window <= 0:
        return (k * (k + 1) - p0 * (p0 + 1)) // 2
    return sum(min(p + 1, window) + min(sinks, max(0, p + 1 - window)) for p in range(p0, k))


def work(case):
    d, Hkv = case["d"], case["Hkv"]
    n, k = _lengths(case)
    if case["op"] == "read":
        return {"bytes": sum(n) * Hkv * d * 6, "flops": sum(n) * Hkv * d * 2}
    H = case["H"]
    if case["op"] == "prefix":
        keys = case["prefix"] + sum(x - case["prefix"] for x in k)
        pairs = sum(_pairs(a, b, 0, 0) for a, b in zip(n, k))
        return {"bytes": keys * Hkv * d * 2 + sum(n) * H * (4 * d + 4), "flops": 4 * H * d * pairs}
    pairs = H * sum(_pairs(a, b, case["window"], case["sinks"]) for a, b in zip(n, k))
    rows = H * sum(n)
    io = 2 * d * (rows + 2 * Hkv * sum(k))  # q, k, v
    fwd = {"bytes": io + rows * (2 * d + 4), "flops": 4 * d * pairs}
    if not case["train"]:
        return fwd
    return {"bytes": fwd["bytes"] + io + rows * (4 * d + 4) + io, "flops": fwd["flops"] + 10 * d * pairs}


# ----------------------------------------------------------------- the inputs
def _starts(lengths):
    cu = [0]
    for x in lengths:
        cu.append(cu[-1] + x)
    return cu


def _int32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _codes(shape, g):
    """Codes of blocks of values of different sizes, and the power-of-two scale of each block."""
    num, Hkv = shape[:2]
    amp = torch.exp2(torch.randint(-2, 3, (num, Hkv, 1, 1), generator=g, device="cuda").float())
    vals = torch.randn(shape, generator=g, device="cuda") * amp.sqrt()
    e = torch.ceil(torch.log2(vals.abs().amax((2, 3)) / 448.0))
    return (vals * torch.exp2(-e)[:, :, None, None]).clamp(-448, 448).to(F8), torch.exp2(e)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)

    st = dict(case)
    d, Hkv, B = case["d"], case["Hkv"], case["B"]
    n, k = _lengths(case)
    st.update(n=n, k=k, cu_n=_starts(n), cu_k=_starts(k), max_n=max(n), max_k=max(k), total=sum(n))
    st["cu_q"], st["cu_keys"] = _int32(st["cu_n"]), _int32(st["cu_k"])
    if case["op"] == "packed":
        H = case["H"]
        if sum(n) == sum(k):  # a fused projection's rows
            qkv = normal(sum(n), H + 2 * Hkv, d)
            st.update(q=qkv[:, :H], key=qkv[:, H : H + Hkv], value=qkv[:, H + Hkv :])
        else:
            st.update(q=normal(sum(n), H, d), key=normal(sum(k), Hkv, d), value=normal(sum(k), Hkv, d))
        if case["train"]:
            st["dout"] = normal(sum(n), H, d)
        return st
    page = case["page"]
    shared = case.get("prefix", 0) // page
    own_pages = [-(-x // page) - shared for x in k]
    num = shared + sum(own_pages) + 5
    perm = torch.randperm(num, generator=g, device="cuda").to(torch.int32)
    table = torch.full((B, shared + max(own_pages)), -1, dtype=torch.int32, device="cuda")
    table[:, :shared] = perm[:shared]
    at = shared
    for b in range(B):
        table[b, shared : shared + own_pages[b]] = perm[at : at + own_pages[b]]
        at += own_pages[b]
    st["k_cache"], st["k_scale"] = _codes((num, Hkv, page, d), g)
    st["v_cache"], st["v_scale"] = _codes((num, Hkv, page, d), g)
    st["page_table"], st["seqlens_k"] = table, _int32(k)
    if case["op"] == "prefix":
        st["q"] = normal(sum(n), case["H"], d)
    else:
        st["starts"] = _int32([b - a for a, b in zip(n, k)])
    return st


# ------------------------------------------------------------- the plain forms
def _visible(pos, keys, window, sinks):
    """pos [n, 1] positions of queries, keys [k]: key j is seen iff j <= p and (j > p - window or j < sinks)."""
    m = keys <= pos
    if window > 0:
        m = m & ((keys > pos - window) | (keys < sinks))
    return m


def _softmax(s):
    """Weights and log of the sum of exponentials of scores; rows of -inf alone give 0 and -inf."""
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(s - top)
    l = p.sum(-1, keepdim=True)
    return p / l.clamp_min(1e-38), (top + torch.log(l)).squeeze(-1)


def _plain_packed(st):
    H, Hkv, d = st["H"], st["Hkv"], st["d"]
    G, scale = H // Hkv, st["d"] ** -0.5
    q, k, v = st["q"], st["key"], st["value"]
    o = torch.empty((st["total"], H, d), device="cuda")
    lse = torch.empty((H, st["total"]), device="cuda")
    dq, dk, dv = torch.empty_like(o), torch.empty(k.shape, device="cuda"), torch.empty(v.shape, device="cuda")
    for b in range(st["B"]):
        n, m = st["n"][b], st["k"][b]
        rows, cols = slice(st["cu_n"][b], st["cu_n"][b + 1]), slice(st["cu_k"][b], st["cu_k"][b + 1])
        pos = torch.arange(n, device="cuda")[:, None] + (m - n)
        hidden = ~_visible(pos, torch.arange(m, device="cuda"), st["window"], st["sinks"])
        for c in range(Hkv):
            heads = slice(c * G, (c + 1) * G)
            qc = q[rows, heads].float().transpose(0, 1)  # [G, n, d]
            kc, vc = k[cols, c].float(), v[cols, c].float()
            w, ll = _softmax((qc @ kc.T * scale).masked_fill_(hidden, -math.inf))
            oc = w @ vc
            o[rows, heads] = oc.transpose(0, 1)
            lse[heads, rows] = ll
            if st["train"]:
                do = st["dout"][rows, heads].float().transpose(0, 1)
                dv[cols, c] = (w.transpose(-1, -2) @ do).sum(0)
                ds = w * (do @ vc.T - (do * oc).sum(-1, keepdim=True))
                dq[rows, heads] = (ds @ kc * scale).transpose(0, 1)
                dk[cols, c] = (ds.transpose(-1, -2) @ qc).sum(0) * scale
    if not st["train"]:
        return o.bfloat16(), lse
    return o.bfloat16(), lse, dq.bfloat16(), dk.bfloat16(), dv.bfloat16()


def _values(cache, scale, ids):
    """Cached values of pages `ids` [..., pages] as [..., Hkv, tokens, d], 32 bits."""
    x = cache[ids].float() * scale[ids][..., None, None]  # [..., pages, Hkv, page, d]
    x = x.transpose(-4, -3)
    return x.reshape(*x.shape[:-3], -1, x.shape[-1])


def _plain_prefix(st):
    B, H, Hkv, d, n = st["B"], st["H"], st["Hkv"], st["d"], st["new"]
    G, L = H // Hkv, st["prefix"]
    shared = L // st["page"]
    q = st["q"].float().view(B, n, Hkv, G, d).permute(0, 2, 3, 1, 4)  # [B, Hkv, G, n, d]
    ids = st["page_table"].long()
    first, rest = ids[0, :shared], ids[:, shared:].clamp_min(0)
    kp, vp = _values(st["k_cache"], st["k_scale"], first), _values(st["v_cache"], st["v_scale"], first)
    ks, vs = _values(st["k_cache"], st["k_scale"], rest), _values(st["v_cache"], st["v_scale"], rest)
    sp = torch.einsum("bcgnd,ckd->bcgnk", q, kp)
    ss = torch.einsum("bcgnd,bckd->bcgnk", q, ks)
    pos = (st["seqlens_k"].long() - L - n)[:, None] + torch.arange(n, device="cuda")  # within the rest
    hidden = torch.arange(ks.shape[2], device="cuda") > pos[:, None, None, :, None]
    s = torch.cat([sp, ss.masked_fill(hidden, -math.inf)], -1) * d ** -0.5
    p, lse = _softmax(s)
    o = torch.einsum("bcgnk,ckd->bcgnd", p[..., :L], vp) + torch.einsum("bcgnk,bckd->bcgnd", p[..., L:], vs)
    o = o.permute(0, 3, 1, 2, 4).reshape(B * n, H, d)
    return o.bfloat16(), lse.permute(1, 2, 0, 3).reshape(H, B * n).contiguous()


def _plain_read(st):
    T = st["total"]
    lens = (st["cu_q"][1:] - st["cu_q"][:-1]).long()
    seq = torch.repeat_interleave(torch.arange(st["B"], device="cuda"), lens, output_size=T)
    at = torch.arange(T, device="cuda") - st["cu_q"][seq].long() + st["starts"][seq].long()
    page, slot = st["page_table"][seq, at // st["page"]].long(), at % st["page"]
    return tuple((st[c][page, :, slot].float() * st[s][page][..., None]).bfloat16()
                 for c, s in (("k_cache", "k_scale"), ("v_cache", "v_scale")))


# ------------------------------------------------------------------- one pass
def run(st):
    op = st["op"]
    if own:
        import exact_attention_80_gb300 as fa

        if op == "packed":
            batch = (st["cu_q"], st["cu_keys"], st["max_n"], st["max_k"], st["window"], st["sinks"])
            o, lse = fa.attention_packed(st["q"], st["key"], st["value"], *batch)
            if not st["train"]:
                return o, lse
            return (o, lse, *fa.attention_packed_backward(st["q"], st["key"], st["value"], o, lse, st["dout"], *batch))
        cache = (st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"], st["page_table"])
        if op == "prefix":
            return fa.attention_prefix_fp8(st["q"], *cache, st["cu_q"], st["seqlens_k"], st["max_n"], st["max_k"],
                                           st["prefix"])
        return fa.kv_read_fp8(*cache, st["cu_q"], st["starts"], st["total"])
    return {"packed": _plain_packed, "prefix": _plain_prefix, "read": _plain_read}[op](st)


# -------------------------------------------- the definitions again, in 64 bits
def _exact_head(q, k, v, window, sinks, do=None):
    """One head: queries q [n][d], the last of the keys k and values v [m][d], a stretch of rows at a time.
    Returns o, lse, dq, dk, dv (the last three of sum(o * do))."""
    n, m, scale = q.shape[0], k.shape[0], q.shape[1] ** -0.5
    o, dq, dk, dv = torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    lse = torch.full((n,), -math.inf, dtype=torch.float64, device=q.device)
    for a in range(0, n, 2048):
        z = min(n, a + 2048)
        lo = max(0, m - n + a - window + 1) if window > 0 else 0
        cols = torch.arange(m, device=q.device)
        if lo > sinks:
            cols = torch.cat([cols[:sinks], cols[lo:]])
        cols = cols[cols < m - n + z]  # no row of the stretch sees the others
        if cols.numel() == 0:
            continue
        age = torch.arange(m - n + a, m - n + z, device=q.device)[:, None] - cols[None, :]
        seen = age >= 0
        if window > 0:
            seen &= (age < window) | (cols[None, :] < sinks)
        kk, vv = k[cols], v[cols]
        s = torch.where(seen, q[a:z] @ kk.T * scale, -math.inf)
        lse[a:z] = torch.logsumexp(s, 1)
        w = torch.exp(s - torch.where(seen.any(1), lse[a:z], 0.0)[:, None])
        o[a:z] = w @ vv
        if do is not None:
            dv.index_add_(0, cols, w.T @ do[a:z])
            ds = w * (do[a:z] @ vv.T - (do[a:z] * o[a:z]).sum(1, keepdim=True))
            dq[a:z] = ds @ kk * scale
            dk.index_add_(0, cols, ds.T @ q[a:z] * scale)
    return o, lse, dq, dk, dv


def _exact_packed(st):
    f64 = dict(dtype=torch.float64, device="cuda")
    H, G = st["H"], st["H"] // st["Hkv"]
    o, dq = torch.zeros(st["q"].shape, **f64), torch.zeros(st["q"].shape, **f64)
    lse = torch.zeros((H, st["total"]), **f64)
    dk, dv = torch.zeros(st["key"].shape, **f64), torch.zeros(st["value"].shape, **f64)
    for b in range(st["B"]):
        i0, i1, j0, j1 = st["cu_n"][b], st["cu_n"][b + 1], st["cu_k"][b], st["cu_k"][b + 1]
        for h in range(H):
            c = h // G
            do = st["dout"][i0:i1, h].double() if st["train"] else None
            r = _exact_head(st["q"][i0:i1, h].double(), st["key"][j0:j1, c].double(), st["value"][j0:j1, c].double(),
                            st["window"], st["sinks"], do)
            o[i0:i1, h], lse[h, i0:i1], dq[i0:i1, h] = r[:3]
            dk[j0:j1, c] += r[3]
            dv[j0:j1, c] += r[4]
    return (o, lse, dq, dk, dv) if st["train"] else (o, lse)


def _exact_tokens(st, which, b, c, lo, hi):
    """Cached values of tokens lo .. hi - 1 of sequence b, kv head c."""
    page = st["page"]
    t = torch.arange(lo, hi, device="cuda")
    pg = st["page_table"][b].long()[torch.div(t, page, rounding_mode="floor")]
    return st[which + "_cache"][pg, c, t % page].double() * st[which + "_scale"][pg, c].double()[:, None]


def _exact_prefix(st):
    H, G, d = st["H"], st["H"] // st["Hkv"], st["d"]
    o = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros((H, st["total"]), dtype=torch.float64, device="cuda")
    for c in range(st["Hkv"]):
        head = [_exact_tokens(st, x, 0, c, 0, st["prefix"]) for x in "kv"]
        for b in range(st["B"]):
            tail = [_exact_tokens(st, x, b, c, st["prefix"], st["k"][b]) for x in "kv"]
            k, v = (torch.cat(x) for x in zip(head, tail))
            i0, i1 = st["cu_n"][b], st["cu_n"][b + 1]
            for h in range(c * G, (c + 1) * G):
                o[i0:i1, h], lse[h, i0:i1] = _exact_head(st["q"][i0:i1, h].double(), k, v, 0, 0)[:2]
    return o, lse


def _exact_read(st):
    outs = []
    for x in "kv":
        y = torch.zeros((st["total"], st["Hkv"], st["d"]), dtype=torch.float64, device="cuda")
        for b in range(st["B"]):
            for c in range(st["Hkv"]):
                y[st["cu_n"][b] : st["cu_n"][b + 1], c] = _exact_tokens(st, x, b, c, st["k"][b] - st["n"][b], st["k"][b])
        outs.append(y)
    return tuple(outs)


def exact(case, seed):
    st = prepare(case, seed)
    return {"packed": _exact_packed, "prefix": _exact_prefix, "read": _exact_read}[case["op"]](st)
