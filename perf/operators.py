"""Operators of the paged KV cache, as a serving engine calls them, with their plain forms.

Three families:

* ``write`` / ``read`` -- quantising K/V rows into an 8-bit paged cache (e4m3 values with one
  power-of-two scale per token and KV head) and reading rows back.
* ``attend`` -- one ragged attention step over that 8-bit cache: the step's new K/V rows are
  quantised into their slots, then every query row attends its request's positions.
* ``shared`` -- one decode step over a bf16 paged cache in which groups of requests share a
  long prompt prefix, whose pages stand once in the pool.

With ``own`` false, ``run`` is elementary torch arithmetic in 32 bits; with ``own`` true it is
the calls that a user of this library makes. ``exact`` is the definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ELT = {"bf16": 2, "f32": 4}
E4M3_MAX = 448.0


# ------------------------------------------------------------------ cases


def listed():
    return [
        # the K/V of one decode step of 64 requests, written to their slots
        dict(name="write_decode_rows", op="write", tokens=64, kv_heads=8, head_dim=128,
             block=16, dtype="bf16"),
        # the K/V of many long prompts at once, an odd count
        dict(name="write_prompts", op="write", tokens=50021, kv_heads=8, head_dim=128,
             block=16, dtype="bf16"),
        # one short request read back in full precision
        dict(name="read_one_request_f32", op="read", tokens=1337, kv_heads=4, head_dim=64,
             block=32, dtype="f32"),
        # a resumed batch read back from its pages
        dict(name="read_batch", op="read", tokens=131072, kv_heads=8, head_dim=128, block=16,
             dtype="bf16"),
        # a few short chats, where latency counts
        dict(name="attend_few_short", op="attend", requests=4, q_lo=1, q_hi=1, ctx_lo=15,
             ctx_hi=300, q_heads=32, kv_heads=8, head_dim=128, block=16, dtype="bf16", window=0,
             lens=3),
        # the ordinary decode batch
        dict(name="attend_decode_batch", op="attend", requests=64, q_lo=1, q_hi=1, ctx_lo=127,
             ctx_hi=2047, q_heads=32, kv_heads=8, head_dim=128, block=16, dtype="bf16", window=0,
             lens=1),
        # long contexts, the largest cache stream
        dict(name="attend_long", op="attend", requests=16, q_lo=1, q_hi=1, ctx_lo=32767,
             ctx_hi=32767, q_heads=64, kv_heads=8, head_dim=128, block=16, dtype="bf16",
             window=0, lens=2),
        # a few drafted tokens of each request checked at once, full precision, a window
        dict(name="attend_drafts_f32", op="attend", requests=11, q_lo=1, q_hi=6, ctx_lo=100,
             ctx_hi=5000, q_heads=16, kv_heads=4, head_dim=64, block=32, dtype="f32",
             window=2000, lens=5),
        # two chunks of long prompts
        dict(name="attend_chunks", op="attend", requests=2, q_lo=700, q_hi=960, ctx_lo=1000,
             ctx_hi=4096, q_heads=32, kv_heads=8, head_dim=128, block=16, dtype="bf16",
             window=0, lens=7),
        # a handful of requests behind a common system prompt
        dict(name="shared_few", op="shared", groups=1, per_group=6, prefix=1024, suf_lo=1,
             suf_hi=120, q_heads=32, kv_heads=8, head_dim=128, block=16, dtype="bf16", lens=4),
        # the decode batch behind a long common document
        dict(name="shared_batch", op="shared", groups=1, per_group=64, prefix=8192, suf_lo=16,
             suf_hi=1024, q_heads=32, kv_heads=8, head_dim=128, block=16, dtype="bf16", lens=6),
        # many samples from each of four very long prompts
        dict(name="shared_samples", op="shared", groups=4, per_group=37, prefix=32768, suf_lo=1,
             suf_hi=700, q_heads=64, kv_heads=8, head_dim=128, block=32, dtype="bf16", lens=8),
    ]


HEADS = [(32, 8), (64, 8), (16, 16), (16, 4), (8, 1), (10, 5), (16, 1)]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "read", "attend", "attend", "attend", "shared", "shared"])
    hq, hkv = rng.choice(HEADS)
    d = rng.choice([64, 128, 128])
    block = rng.choice([16, 16, 32, 64, 128])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("write", "read"):
        top = 131072 * 8 * 128 // (hkv * d) * 2 // ELT[dtype] // 2
        return dict(op=op, tokens=_log_int(rng, 1, min(top, 131072)), kv_heads=hkv, head_dim=d,
                    block=block, dtype=dtype)
    if op == "attend":
        kind = rng.choice(["decode", "decode", "drafts", "chunk"])
        if kind == "chunk":
            n, q_lo, q_hi = rng.randint(1, 4), rng.randint(17, 200), rng.randint(200, 800)
            ctx_hi = _log_int(rng, 64, 4096)
        else:
            n = _log_int(rng, 1, 128)
            q_lo, q_hi = 1, (1 if kind == "decode" else rng.randint(2, 8))
            ctx_hi = _log_int(rng, 32, min(32768, 300000 // n))
        window = rng.choice([0, 0, 0, _log_int(rng, 16, 4096)])
        return dict(op=op, requests=n, q_lo=q_lo, q_hi=q_hi, ctx_lo=rng.randint(0, ctx_hi // 2),
                    ctx_hi=ctx_hi, q_heads=hq, kv_heads=hkv, head_dim=d, block=block,
                    dtype=dtype, window=window, lens=rng.randint(10, 1 << 20))
    groups = rng.choice([1, 1, 2, 3, 5])
    per_group = _log_int(rng, 2, 192 // groups)
    pages = _log_int(rng, max(1, 256 // block), 32768 // groups // block)
    return dict(op="shared", groups=groups, per_group=per_group, prefix=pages * block,
                suf_lo=1, suf_hi=_log_int(rng, 2, 1500), q_heads=hq, kv_heads=hkv, head_dim=d,
                block=block, dtype="bf16", lens=rng.randint(10, 1 << 20))


# ------------------------------------------------------------------ lengths and pages


def _lengths(case):
    """(q_len, context) of each request: from the case alone."""
    r = np.random.RandomState(case["lens"])
    if case["op"] == "attend":
        q = r.randint(case["q_lo"], case["q_hi"] + 1, size=case["requests"])
        ctx = r.randint(case["ctx_lo"], case["ctx_hi"] + 1, size=case["requests"])
    else:
        n = case["groups"] * case["per_group"]
        q = np.ones(n, np.int64)
        # the suffix counts this step's token
        ctx = case["prefix"] + r.randint(case["suf_lo"], case["suf_hi"] + 1, size=n) - 1
    return q.astype(np.int32), ctx.astype(np.int32)


def _pages(case, q, ctx, rng):
    """Block table [R, stride] over a shuffled pool and the slot of each new token."""
    bs, n = case["block"], len(q)
    seq = q + ctx
    need = -(-seq // bs)
    first = case["prefix"] // bs if case["op"] == "shared" else 0
    groups = case["groups"] if case["op"] == "shared" else 0
    own_pages = need - first
    total = 2 + int(math.ceil(1.2 * (own_pages.sum() + groups * first)))
    free = rng.permutation(np.arange(2, total))
    stride = int(need.max())
    bt = np.zeros((n, stride), np.int32)
    if first:
        head = free[:groups * first].reshape(groups, 1, first)
        bt[:, :first] = np.broadcast_to(head, (groups, n // groups, first)).reshape(n, first)
    col = np.arange(stride)[None, :]
    mine = (col >= first) & (col < need[:, None])
    bt[mine] = free[groups * first:groups * first + int(own_pages.sum())]
    qsl = np.zeros(n + 1, np.int32)
    qsl[1:] = np.cumsum(q)
    r_of_t = np.repeat(np.arange(n), q)
    pos = ctx[r_of_t] + np.arange(qsl[-1]) - qsl[r_of_t]
    slots = bt[r_of_t, pos // bs].astype(np.int64) * bs + pos % bs
    return bt, qsl, seq.astype(np.int32), slots, total


# ------------------------------------------------------------------ quantising, plain


def _quantise(x):
    """Rows [..., D] -> (e4m3 [..., D], scale code [...]): the scale is 2^(code - 127) with the
    smallest exponent for which the largest finite magnitude is at most 448 scales."""
    x = x.float()
    a = torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x)).amax(-1)
    m, e = torch.frexp(a)
    e = e.to(torch.int32) - 9 + (m > 0.875).to(torch.int32)
    e = torch.where(a > 0, e.clamp(min=-126), torch.zeros_like(e))
    inv = ((127 - e) << 23).view(torch.float32)
    y = (x * inv.unsqueeze(-1)).clamp(-E4M3_MAX, E4M3_MAX)
    return y.to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _scale(code):
    return (code.to(torch.int32) << 23).view(torch.float32)


def _write_plain(x, cache, scale, slots):
    v, c = _quantise(x)
    nb, bs, h, d = cache.shape
    cache.view(torch.uint8).view(nb * bs, h, d)[slots] = v.view(torch.uint8)
    scale.view(torch.uint8).view(nb * bs, h)[slots] = c


def _rows_plain(cache, scale, slots):
    """Rows of the cache at `slots` (any shape), in 32 bits."""
    nb, bs, h, d = cache.shape
    v = cache.view(torch.uint8).view(nb * bs, h, d)[slots].view(torch.float8_e4m3fn).float()
    return v * _scale(scale.view(torch.uint8).view(nb * bs, h)[slots]).unsqueeze(-1)


# ------------------------------------------------------------------ state


def _rows(gen, shape, dtype):
    """K or V rows: normal values whose size differs from token to token and head to head."""
    x = torch.randn(shape, generator=gen, device="cuda")
    s = torch.exp(0.5 * torch.randn(shape[:-1], generator=gen, device="cuda"))
    return (x * s.unsqueeze(-1)).to(dtype)


def _fill(gen, shape, dtype):
    """A pool [NB, BS, H, D], filled some pages at a time."""
    out = torch.empty(shape, dtype=dtype, device="cuda")
    step = max(1, (1 << 26) // int(np.prod(shape[1:])))
    for b in range(0, shape[0], step):
        out[b:b + step] = _rows(gen, out[b:b + step].shape, dtype)
    return out


def _fill_q8(gen, shape):
    out = torch.empty(shape, dtype=torch.float8_e4m3fn, device="cuda")
    code = torch.empty(shape[:-1], dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 26) // int(np.prod(shape[1:])))
    for b in range(0, shape[0], step):
        out[b:b + step], code[b:b + step] = _quantise(_rows(gen, out[b:b + step].shape, torch.float32))
    return out, code.view(torch.float8_e8m0fnu)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rng = np.random.RandomState(seed % (1 << 32))
    dt = DTYPES[case["dtype"]]
    h, d, bs = case["kv_heads"], case["head_dim"], case["block"]
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    s = dict(case=case)
    if case["op"] in ("write", "read"):
        t = case["tokens"]
        nb = 2 + -(-int(1.2 * t) // bs)
        # whole pages in a shuffled order, as a scheduler hands them out
        page = rng.permutation(np.arange(2, nb))[:-(-t // bs)]
        if len(page) * bs < t:
            raise ValueError("pool too small")
        pos = np.arange(t)
        s["slots"] = dev(page[pos // bs].astype(np.int64) * bs + pos % bs)
        s["k_cache"], s["k_scale"] = _fill_q8(gen, (nb, bs, h, d))
        s["v_cache"], s["v_scale"] = _fill_q8(gen, (nb, bs, h, d))
        if case["op"] == "write":
            s["k"], s["v"] = _rows(gen, (t, h, d), dt), _rows(gen, (t, h, d), dt)
        else:
            s["k"] = torch.empty((t, h, d), dtype=dt, device="cuda")
            s["v"] = torch.empty((t, h, d), dtype=dt, device="cuda")
        return s
    q, ctx = _lengths(case)
    bt, qsl, seq, slots, nb = _pages(case, q, ctx, rng)
    t, hq = int(qsl[-1]), case["q_heads"]
    s.update(h_qsl=qsl, h_seq=seq, q_max=int(q.max()), s_max=int(seq.max()), bt=dev(bt),
             qsl=dev(qsl), seq=dev(seq), slots=dev(slots))
    s["q"] = torch.randn((t, hq, d), generator=gen, device="cuda").to(dt)
    s["k"], s["v"] = _rows(gen, (t, h, d), dt), _rows(gen, (t, h, d), dt)
    s["out"] = torch.empty((t, hq, d), dtype=dt, device="cuda")
    shape = (nb, bs, h, d)
    if case["op"] == "attend":
        s["k_cache"], s["k_scale"] = _fill_q8(gen, shape)
        s["v_cache"], s["v_scale"] = _fill_q8(gen, shape)
    else:
        s["k_cache"], s["v_cache"] = _fill(gen, shape, dt), _fill(gen, shape, dt)
        s["h_prefix"] = np.full(len(q), case["prefix"], np.int32)
        s["prefix"] = dev(s["h_prefix"])
        s["h_group"] = np.arange(0, len(q) + 1, case["per_group"], dtype=np.int32)
    if own:
        import paged_kv_attention_cb_gb300 as cb

        if case["op"] == "attend":
            chunk = int(seq[q > 1].sum())
            s["workspace"] = cb.alloc_workspace_q8(len(q), t, hq, h, d, bs, chunk)
        else:
            s["workspace"] = cb.alloc_workspace_shared(len(q), t, hq, h, d)
    return s


# ------------------------------------------------------------------ one pass


def _softmax_rows(scores):
    m = scores.amax(-1, keepdim=True)
    e = torch.exp(scores - m)
    return e / e.sum(-1, keepdim=True)


def _attend_plain(s):
    c = s["case"]
    _write_plain(s["k"], s["k_cache"], s["k_scale"], s["slots"])
    _write_plain(s["v"], s["v_cache"], s["v_scale"], s["slots"])
    bs, hkv, d = c["block"], c["kv_heads"], c["head_dim"]
    g = c["q_heads"] // hkv
    n, qm, sm = c["requests"], s["q_max"], s["s_max"]
    pos = torch.arange(sm, device="cuda")
    slots = s["bt"][:, pos // bs].long() * bs + pos % bs
    k = _rows_plain(s["k_cache"], s["k_scale"], slots)  # [n, sm, hkv, d]
    v = _rows_plain(s["v_cache"], s["v_scale"], slots)
    i = torch.arange(qm, device="cuda")
    row = s["qsl"][:-1, None].long() + i  # [n, qm]
    live = row < s["qsl"][1:, None]
    q = s["q"][row.clamp(max=s["q"].shape[0] - 1)].float().view(n, qm, hkv, g, d)
    sc = torch.matmul(q.permute(0, 2, 1, 3, 4).reshape(n, hkv, qm * g, d), k.permute(0, 2, 3, 1))
    sc = sc.view(n, hkv, qm, g, sm) * (1.0 / math.sqrt(d))
    last = (s["seq"] - (s["qsl"][1:] - s["qsl"][:-1]))[:, None] + i  # [n, qm]
    ok = pos <= last[..., None]
    if c["window"]:
        ok = ok & (pos > last[..., None] - c["window"])
    sc = sc.masked_fill(~ok[:, None, :, None, :], -math.inf)
    sc = torch.where(live[:, None, :, None, None], sc, torch.zeros_like(sc))
    # positions past a request hold pages of others: their weight is zero
    v = torch.where((pos < s["seq"][:, None])[..., None, None], v, torch.zeros_like(v))
    p = _softmax_rows(sc).view(n, hkv, qm * g, sm)
    o = torch.matmul(p, v.permute(0, 2, 1, 3)).view(n, hkv, qm, g, d).permute(0, 2, 1, 3, 4)
    o = o.reshape(n * qm, hkv * g, d).to(s["out"].dtype)
    t = torch.arange(s["q"].shape[0], device="cuda")
    r = torch.searchsorted(s["qsl"][1:].long(), t, right=True)
    s["out"].copy_(o[r * qm + (t - s["qsl"].long()[r])])


def _shared_plain(s):
    c = s["case"]
    bs, hkv, d, p = c["block"], c["kv_heads"], c["head_dim"], c["prefix"]
    g, ng, n = c["q_heads"] // hkv, c["groups"], c["per_group"]
    flat = lambda x: x.view(-1, hkv, d)
    flat(s["k_cache"])[s["slots"]] = s["k"]
    flat(s["v_cache"])[s["slots"]] = s["v"]
    # the prefix, once for each group: [ng, hkv, n * g, p]
    pos = torch.arange(p, device="cuda")
    slots = s["bt"][::n][:, pos // bs].long() * bs + pos % bs
    kp, vp = flat(s["k_cache"])[slots].float(), flat(s["v_cache"])[slots].float()
    q = s["q"].float().view(ng, n, hkv, g, d)
    sp = torch.matmul(q.permute(0, 2, 1, 3, 4).reshape(ng, hkv, n * g, d), kp.permute(0, 2, 3, 1))
    # the suffix of each request: [ng * n, hkv, g, s_max - p]
    pos = torch.arange(p, s["s_max"], device="cuda")
    slots = s["bt"][:, pos // bs].long() * bs + pos % bs
    ok = pos < s["seq"][:, None]
    ks, vs = flat(s["k_cache"])[slots].float(), flat(s["v_cache"])[slots].float()
    vs = torch.where(ok[..., None, None], vs, torch.zeros_like(vs))
    ss = torch.matmul(q.reshape(ng * n, hkv, g, d), ks.permute(0, 2, 3, 1))
    ss = ss.masked_fill(~ok[:, None, None, :], -math.inf)
    ss = ss.view(ng, n, hkv, g, -1).permute(0, 2, 1, 3, 4).reshape(ng, hkv, n * g, -1)
    w = _softmax_rows(torch.cat([sp, ss], -1) * (1.0 / math.sqrt(d)))
    op = torch.matmul(w[..., :p], vp.permute(0, 2, 1, 3)).view(ng, hkv, n, g, d)
    ws = w[..., p:].view(ng, hkv, n, g, -1).permute(0, 2, 1, 3, 4).reshape(ng * n, hkv, g, -1)
    os = torch.matmul(ws, vs.permute(0, 2, 1, 3)).view(ng, n, hkv, g, d)
    s["out"].copy_((op.permute(0, 2, 1, 3, 4) + os).reshape(ng * n, hkv * g, d))


def run(s):
    op = s["case"]["op"]
    if own:
        import paged_kv_attention_cb_gb300 as cb

        if op == "write":
            cb.write_kv_q8(s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_scale"],
                           s["v_scale"], s["slots"])
        elif op == "read":
            cb.read_kv_q8(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["slots"],
                          s["k"], s["v"])
        elif op == "attend":
            cb.paged_attention_q8(s["out"], s["q"], s["k_cache"], s["v_cache"], s["k_scale"],
                                  s["v_scale"], s["qsl"], s["seq"], s["bt"], s["h_qsl"],
                                  s["h_seq"], s["workspace"], sliding_window=s["case"]["window"],
                                  k_new=s["k"], v_new=s["v"], slot_mapping=s["slots"])
        else:
            cb.paged_attention_shared(s["out"], s["q"], s["k_cache"], s["v_cache"], s["qsl"],
                                      s["seq"], s["bt"], s["prefix"], s["h_qsl"], s["h_seq"],
                                      s["h_prefix"], s["h_group"], s["workspace"], k_new=s["k"],
                                      v_new=s["v"], slot_mapping=s["slots"])
    elif op == "write":
        _write_plain(s["k"], s["k_cache"], s["k_scale"], s["slots"])
        _write_plain(s["v"], s["v_cache"], s["v_scale"], s["slots"])
    elif op == "read":
        s["k"].copy_(_rows_plain(s["k_cache"], s["k_scale"], s["slots"]))
        s["v"].copy_(_rows_plain(s["v_cache"], s["v_scale"], s["slots"]))
    elif op == "attend":
        _attend_plain(s)
    else:
        _shared_plain(s)
    if op == "read":
        return dict(k=s["k"], v=s["v"])
    outs = dict(k_cache=s["k_cache"], v_cache=s["v_cache"])
    if op != "shared":
        outs.update(k_scale=s["k_scale"], v_scale=s["v_scale"])
    if op != "write":
        outs.update(out=s["out"])
    return outs


# ------------------------------------------------------------------ work


def work(case):
    h, d, e = case["kv_heads"], case["head_dim"], ELT[case["dtype"]]
    if case["op"] in ("write", "read"):
        # rows in one form read, in the other written, and the slots
        t = case["tokens"]
        return dict(bytes=2 * t * h * (d * e + d + 1) + 8 * t, flops=2 * t * h * d)
    q, ctx = (a.astype(np.int64) for a in _lengths(case))
    t, hq = int(q.sum()), case["q_heads"]
    if case["op"] == "attend":
        w = case["window"] or 1 << 40
        first = np.maximum(0, ctx - w + 1)  # first position the request attends
        kept = int((ctx - first).sum())     # positions read from the cache
        pairs = 0
        for a, b in zip(q.tolist(), ctx.tolist()):
            pairs += int(np.minimum(np.arange(b + 1, b + a + 1), w).sum())
        rows, row = kept, 2 * h * (d + 1)
    else:
        p = case["prefix"]
        rows, row = case["groups"] * p + int((ctx - p).sum()), 2 * h * d * e
        pairs = int((ctx + 1).sum())
    # the cache's rows; q and out; the new rows, read and written
    return dict(bytes=rows * row + 2 * t * hq * d * e + 2 * t * h * d * e + t * row + 8 * t,
                flops=4 * hq * d * pairs)


# ------------------------------------------------------------------ the definition in 64 bits


def _quantise64(x):
    """(value / scale, scale) of rows in float64, from the definition."""
    x = x.double()
    top = x.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(top / E4M3_MAX))
    e = torch.where(top > E4M3_MAX * torch.exp2(e), e + 1, e)  # log2 may round either way
    e = torch.where(top <= E4M3_MAX * torch.exp2(e - 1), e - 1, e)
    scale = torch.exp2(torch.where(top > 0, e.clamp(min=-126.0), torch.zeros_like(e)))
    y = x / scale
    # e4m3: 3 fraction bits, smallest exponent -6; halves go to the even neighbour
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -20))).clamp(min=-6.0) - 3)
    return torch.round(y / step) * step, scale.squeeze(-1)


def _values(cache, scale):
    """An 8-bit cache's stored values and scales in float64, flat over the slots."""
    nb, bs, h, d = cache.shape
    return cache.double().view(nb * bs, h, d), scale.double().view(nb * bs, h)


def exact(case, seed):
    s = prepare(case, seed)
    h, d = case["kv_heads"], case["head_dim"]
    if case["op"] != "shared":
        kv, ks = _values(s["k_cache"], s["k_scale"])
        vv, vs = _values(s["v_cache"], s["v_scale"])
        if case["op"] == "read":
            pick = lambda v, c: v[s["slots"]] * c[s["slots"]].unsqueeze(-1)
            return dict(k=pick(kv, ks), v=pick(vv, vs))
        kv[s["slots"]], ks[s["slots"]] = _quantise64(s["k"])
        vv[s["slots"]], vs[s["slots"]] = _quantise64(s["v"])
        outs = dict(k_cache=kv, v_cache=vv, k_scale=ks, v_scale=vs)
        if case["op"] == "write":
            return outs
        at = lambda v, c, i: v[i] * c[i].unsqueeze(-1)
        key, val = lambda i: at(kv, ks, i), lambda i: at(vv, vs, i)
    else:
        kv, vv = s["k_cache"].double().view(-1, h, d), s["v_cache"].double().view(-1, h, d)
        kv[s["slots"]], vv[s["slots"]] = s["k"].double(), s["v"].double()
        outs = dict(k_cache=kv, v_cache=vv)
        key, val = lambda i: kv[i], lambda i: vv[i]
    # request by request: each query row over the positions it attends
    g = case["q_heads"] // h
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    window = case.get("window", 0) or 1 << 40
    for r in range(len(s["h_seq"])):
        a, b, n = int(s["h_qsl"][r]), int(s["h_qsl"][r + 1]), int(s["h_seq"][r])
        p = torch.arange(n, device="cuda")
        slot = s["bt"][r].long()[p // case["block"]] * case["block"] + p % case["block"]
        k, v = key(slot), val(slot)
        q = s["q"][a:b].double().view(b - a, h, g, d)
        sc = torch.einsum("qhgd,shd->hgqs", q, k) / math.sqrt(d)
        row = torch.arange(n - (b - a), n, device="cuda")[:, None]
        sc = torch.where((p <= row) & (p > row - window), sc, -math.inf)
        out[a:b] = torch.einsum("hgqs,shd->qhgd", torch.softmax(sc, -1), v).reshape(b - a, h * g, d)
    outs["out"] = out
    return outs
