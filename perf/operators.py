"""Cases that time and check the decoder-layer operators next to the int4g linears: RMS norm with the residual, rotary
positions, the write into the 8-bit key/value cache and the attention that reads it.

`own` False: the operators in plain torch, 32-bit arithmetic (64 for angles).  `own` True: the library's calls.
"""
import math
import random

import torch

own = False

E4M3_MAX, INT8_MAX = 448.0, 127.0


# ------------------------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # the latency of one request's next token: a short context
        dict(name="attention 1x1 of 517", op="attention", fmt="e4m3", batch=1, q=1, q_min=1, kv=517, kv_min=517, heads=32,
             kv_heads=8, dim=128, block=64, window=0),
        # a serving batch's next tokens, contexts of every length
        dict(name="attention 48x1 ragged", op="attention", fmt="e4m3", batch=48, q=1, q_min=1, kv=8100, kv_min=130,
             heads=32, kv_heads=8, dim=128, block=64, window=0),
        # a few requests with very long contexts
        dict(name="attention 3x1 long int8", op="attention", fmt="int8", batch=3, q=1, q_min=1, kv=131000, kv_min=60000,
             heads=32, kv_heads=4, dim=128, block=128, window=0),
        # drafted tokens checked in one pass, heads of 64, small blocks
        dict(name="attention 16x5 drafted", op="attention", fmt="int8", batch=16, q=5, q_min=2, kv=4001, kv_min=37,
             heads=24, kv_heads=8, dim=64, block=16, window=0),
        # a whole prompt, one key head for each query head
        dict(name="attention prompt 4095", op="attention", fmt="e4m3", batch=1, q=4095, q_min=4095, kv=4095, kv_min=4095,
             heads=32, kv_heads=32, dim=128, block=64, window=0),
        # chunks of two prompts after long contexts
        dict(name="attention chunks long", op="attention", fmt="int8", batch=2, q=2048, q_min=1500, kv=33000,
             kv_min=20000, heads=32, kv_heads=4, dim=128, block=32, window=0),
        # the write of one token for each request of a serving batch
        dict(name="append 48x1", op="append", fmt="int8", batch=48, q=1, q_min=1, kv=4100, kv_min=130, kv_heads=8, dim=128,
             block=64),
        # the write of prompts
        dict(name="append prompts", op="append", fmt="e4m3", batch=5, q=4095, q_min=900, kv=5000, kv_min=4096, kv_heads=8,
             dim=128, block=64),
        # one token through a norm
        dict(name="norm 1x4096", op="norm", rows=1, heads=1, width=4096, residual=True, out8=False, group=0),
        # a prompt's tokens, the normed values in 16 and in 8 bits
        dict(name="norm 8191x4096 8 bits", op="norm", rows=8191, heads=1, width=4096, residual=True, out8=True, group=128),
        # one token for each request, one axis
        dict(name="rope 48 tokens", op="rope", tokens=48, heads=32, kv_heads=8, dim=128, rot=128, axes=1, far=131072,
             halves=True),
        # a long prompt of video and text: time, height and width
        dict(name="rope 16381 video", op="rope", tokens=16381, heads=32, kv_heads=4, dim=128, rot=128, axes=3, far=32768,
             halves=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tokens", "tokens", "prompt", "prompt", "append", "norm", "rope"])
    dim = rng.choice([64, 128, 128])
    kv_heads = rng.choice([1, 2, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 7, 8])
    fmt, block = rng.choice(["e4m3", "int8"]), rng.choice([16, 32, 64, 128])
    if op == "tokens":
        batch = _log(rng, 1, 128)
        kv = _log(rng, 64, min(131072, 524288 // batch))
        q = rng.choice([1, 1, 1, 2, 3, 4])
        return dict(op="attention", fmt=fmt, batch=batch, q=q, q_min=1, kv=kv, kv_min=max(q, kv // 8), heads=heads,
                    kv_heads=kv_heads, dim=dim, block=block, window=rng.choice([0, 0, 0, 1000]))
    if op == "prompt":
        batch = rng.choice([1, 1, 2, 3])
        q = _log(rng, 20, 4096 // batch)
        kv = _log(rng, q, 24000)
        return dict(op="attention", fmt=fmt, batch=batch, q=q, q_min=max(1, q // 3), kv=kv, kv_min=max(q, kv // 2),
                    heads=heads, kv_heads=kv_heads, dim=dim, block=block, window=rng.choice([0, 0, 0, 1000]))
    if op == "append":
        batch = _log(rng, 1, 64)
        q = _log(rng, 1, 16384 // batch)
        kv = _log(rng, q, 20000)
        return dict(op="append", fmt=fmt, batch=batch, q=q, q_min=max(1, q // 4), kv=kv, kv_min=q, kv_heads=kv_heads,
                    dim=dim, block=block)
    if op == "norm":
        if rng.random() < 0.3:     # each head's query or key normed by itself
            return dict(op="norm", rows=_log(rng, 1, 16384), heads=heads, width=dim, residual=False, out8=False, group=0)
        group = rng.choice([0, 64, 128, 256])
        width = rng.randrange(1, 65) * 256 if rng.random() < 0.8 else 8 * rng.randrange(20, 1000)
        return dict(op="norm", rows=_log(rng, 1, 8191), heads=1, width=min(width, 8192), residual=rng.random() < 0.7,
                    out8=width % 256 == 0 and rng.random() < 0.6, group=group)
    rot = dim if rng.random() < 0.7 else dim // 2
    return dict(op="rope", tokens=_log(rng, 1, 16381), heads=heads, kv_heads=kv_heads, dim=dim, rot=rot,
                axes=rng.choice([1, 2, 3]), far=_log(rng, 1000, 1000000), halves=rng.random() < 0.7)


def _lengths(case):
    """The query and cache lengths of a case's sequences: part of the case, not of its values."""
    r = random.Random("%(batch)d %(q)d %(q_min)d %(kv)d %(kv_min)d %(block)d" % case)
    q = [r.randint(case["q_min"], case["q"]) for _ in range(case["batch"])]
    q[0] = case["q"]
    kv = [max(n, r.randint(case["kv_min"], case["kv"])) for n in q]
    kv[-1] = max(q[-1], case["kv"])
    return q, kv


def _visible(case):
    """Sum over query tokens of the keys that each sees, and the keys of all sequences that any token sees."""
    pairs = keys = 0
    for q, kv in zip(*_lengths(case)):
        w = case["window"] or kv
        first = kv - q + 1                       # keys that the first token sees without a window
        full = min(q, max(0, w - first + 1))     # tokens that see fewer keys than the window, or just as many
        pairs += full * first + full * (full - 1) // 2 + (q - full) * w
        keys += min(kv, w + q - 1)
    return pairs, keys


def work(case):
    op = case["op"]
    if op == "attention":
        pairs, keys = _visible(case)
        tokens = sum(_lengths(case)[0])
        return {"bytes": 2 * keys * case["kv_heads"] * case["dim"] + 8 * keys * case["kv_heads"] / case["block"]
                + 4 * tokens * case["heads"] * case["dim"] + 4 * tokens * case["heads"],
                "flops": 4 * pairs * case["heads"] * case["dim"]}
    if op == "append":
        tokens = sum(_lengths(case)[0])
        return {"bytes": 2 * tokens * case["kv_heads"] * (3 * case["dim"] + 4 / case["block"]),
                "flops": 4 * tokens * case["kv_heads"] * case["dim"]}
    if op == "norm":
        n = case["rows"] * case["heads"] * case["width"]
        b = n * (2 + 2 + (4 if case["residual"] else 0) + (1 if case["out8"] else 0)) + 2 * case["width"]
        if case["out8"]:
            b += 4 * case["rows"] * case["heads"] * (case["width"] // case["group"] if case["group"] else 1)
        return {"bytes": b, "flops": 8 * n}
    n = case["tokens"] * (case["heads"] + case["kv_heads"])
    return {"bytes": 4 * n * case["dim"] + 4 * case["axes"] * case["tokens"] + 4 * case["rot"], "flops": 3 * n * case["rot"]}


# ------------------------------------------------------------------------------------------------------------ inputs

def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _heads(g, n, heads, dim):
    """Keys or values as a projection gives them: some channels larger than others."""
    gain = torch.exp(0.5 * _normal(g, 1, heads, dim))
    return (_normal(g, n, heads, dim) * gain).to(torch.bfloat16)


def _least_scale(amax, fmt):
    """The least power of two that brings amax within the type's range; 2^-126 where amax is 0."""
    top, bits = (E4M3_MAX, 9) if fmt == "e4m3" else (INT8_MAX, 7)
    m, e = torch.frexp(amax.float())                                # amax = m 2^e, and top = (top / 2^bits) 2^bits
    e = e - bits + (m > top / 2.0 ** bits).to(e.dtype)
    e = torch.where(amax > 0, e, -126).clamp(min=-126)
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _codes(x, fmt):
    """x in units of its scale, rounded to the 8-bit type and held as bytes."""
    if fmt == "e4m3":
        return x.to(torch.float8_e4m3fn).view(torch.uint8)
    return torch.round(x).to(torch.int8).view(torch.uint8)


def _values(codes, fmt):
    return codes.view(torch.float8_e4m3fn if fmt == "e4m3" else torch.int8).float()


def _cache(g, case, blocks):
    """A cache of codes [blocks, kv_heads, block, dim] with a scale for each block and head."""
    shape = (blocks, case["kv_heads"], case["block"], case["dim"])
    gain = torch.exp(0.5 * _normal(g, 1, shape[1], 1, shape[3]))
    x = _normal(g, *shape).mul_(gain).to(torch.bfloat16).float()
    scale = _least_scale(x.abs().amax(dim=(2, 3)), case["fmt"])
    return _codes(x / scale[:, :, None, None], case["fmt"]), scale


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 17)
    op = case["op"]
    s = {"case": dict(case)}
    if op in ("attention", "append"):
        q, kv = _lengths(case)
        block = case["block"]
        most = -(-max(kv) // block)
        blocks = sum(-(-n // block) for n in kv) + 3
        order = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32).cpu()
        table = torch.zeros((len(kv), most), dtype=torch.int32)
        at = 0
        for b, n in enumerate(kv):
            m = -(-n // block)
            table[b, :m] = order[at:at + m]
            at += m
        s["table"] = table.cuda()
        s["cu_q"] = torch.tensor([0] + q, dtype=torch.int32).cumsum(0).to(torch.int32).cuda()
        s["kv_lens"] = torch.tensor(kv, dtype=torch.int32).cuda()
        s["max_q"] = max(q)
        s["k_cache"], s["k_scale"] = _cache(g, case, blocks)
        s["v_cache"], s["v_scale"] = _cache(g, case, blocks)
        if op == "attention":
            # queries out of one fused projection: rows that are wider than the queries alone
            wide = case["heads"] + 2 * case["kv_heads"]
            s["qkv"] = _normal(g, sum(q), wide, case["dim"]).mul_(1.3).to(torch.bfloat16)
            s["scale"] = 1.0 / math.sqrt(case["dim"])
        else:
            s["k"] = _heads(g, sum(q), case["kv_heads"], case["dim"])
            s["v"] = _heads(g, sum(q), case["kv_heads"], case["dim"])
    elif op == "norm":
        n, h, w = case["rows"], case["heads"], case["width"]
        s["x"] = _normal(g, n, h, w).to(torch.bfloat16)
        s["w"] = (1 + 0.2 * _normal(g, w)).to(torch.bfloat16)
        s["r"] = _normal(g, n, h, w).mul_(3).to(torch.bfloat16) if case["residual"] else None
    else:
        n = case["tokens"]
        s["q"] = _normal(g, n, case["heads"], case["dim"]).to(torch.bfloat16)
        s["k"] = _normal(g, n, case["kv_heads"], case["dim"]).to(torch.bfloat16)
        pairs = case["rot"] // 2
        s["inv_freq"] = 10000.0 ** (-torch.arange(pairs, dtype=torch.float64) / pairs).cuda()
        s["positions"] = torch.randint(0, case["far"], (case["axes"], n), generator=g, device="cuda", dtype=torch.int32)
        # each axis has a run of the pairs, the first axis the shortest
        a = case["axes"]
        s["sections"] = [pairs - (a - 1) * (pairs // a + (1 if a > 1 else 0))] + [pairs // a + 1] * (a - 1)
        s["pair_axis"] = torch.repeat_interleave(torch.arange(a), torch.tensor(s["sections"])).cuda()
    return s


# ---------------------------------------------------------------------------------------------------------- own calls

def _run_own(s):
    import int4_group_quantized_int4g_gb300 as fl
    case = s["case"]
    op = case["op"]
    if op == "attention":
        fmt = fl.FL_KV8_E4M3 if case["fmt"] == "e4m3" else fl.FL_KV8_INT8
        out, lse = fl.fl_kv8_attention(s["qkv"][:, :case["heads"]], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                                       s["table"], s["kv_lens"], cu_q=s["cu_q"], max_q=s["max_q"], fmt=fmt,
                                       scale=s["scale"], window=case["window"], return_lse=True)
        return {"out": out, "lse": lse}
    if op == "append":
        fmt = fl.FL_KV8_E4M3 if case["fmt"] == "e4m3" else fl.FL_KV8_INT8
        fl.fl_kv8_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"],
                         s["kv_lens"], cu_q=s["cu_q"], max_q=s["max_q"], fmt=fmt)
        return _cache_out(s)
    if op == "norm":
        r = fl.fl_rmsnorm(s["x"], s["w"], 1e-6, residual=s["r"], out8=case["out8"], group=case["group"])
        return {k: v.view(torch.float8_e4m3fn) if k == "codes" else v for k, v in r.items()}
    q, k = fl.fl_rope(s["q"], s["k"], s["positions"], s["inv_freq"], sections=s["sections"], halves=case["halves"])
    return {"q": q, "k": k}


def _cache_out(s):
    """The whole cache: e4m3 codes as the values they are, int8 codes as whole numbers, each in units of its scale."""
    t = torch.float8_e4m3fn if s["case"]["fmt"] == "e4m3" else torch.int8
    return {"k": s["k_cache"].view(t), "v": s["v_cache"].view(t), "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


# -------------------------------------------------------------------------------------------------------- plain forms

def _attention(s):
    case = s["case"]
    hq, hk, d, block, fmt = case["heads"], case["kv_heads"], case["dim"], case["block"], case["fmt"]
    table, cu = s["table"].long(), s["cu_q"].long()
    batch, n = table.shape[0], table.shape[1] * block
    q_len, kv_len = cu[1:] - cu[:-1], s["kv_lens"].long()
    k = (_values(s["k_cache"][table], fmt) * s["k_scale"][table][..., None, None]).transpose(1, 2).reshape(batch, hk, n, d)
    v = (_values(s["v_cache"][table], fmt) * s["v_scale"][table][..., None, None]).transpose(1, 2).reshape(batch, hk, n, d)
    at = torch.arange(s["max_q"], device="cuda")
    real = at[None] < q_len[:, None]                                         # [batch, max_q]
    row = torch.where(real, cu[:-1, None] + at[None], 0)
    q = s["qkv"][:, :hq].float()[row]                                        # [batch, max_q, hq, d]
    q = q.view(batch, s["max_q"], hk, hq // hk, d).permute(0, 2, 3, 1, 4).reshape(batch, hk, -1, d)
    x = torch.matmul(q, k.transpose(2, 3)).mul_(s["scale"]).view(batch, hk, hq // hk, s["max_q"], n)
    last = (kv_len - q_len)[:, None] + at[None]                              # the last key that a token sees
    j = torch.arange(n, device="cuda")
    hide = j[None, None] > last[..., None]
    if case["window"]:
        hide |= j[None, None] <= last[..., None] - case["window"]
    x.masked_fill_(hide[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True).clamp_(min=-1e30)
    p = x.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(batch, hk, -1, n), v).view(batch, hk, hq // hk, s["max_q"], d) / total.clamp(min=1e-30)
    lse = (top + total.log()).squeeze(-1)
    out = o.permute(0, 3, 1, 2, 4).reshape(batch, s["max_q"], hq, d)[real]
    return {"out": out.to(torch.bfloat16), "lse": lse.permute(0, 3, 1, 2).reshape(batch, s["max_q"], hq)[real]}


def _append_one(s, x, cache, scale):
    """Writes x [tokens, kv_heads, dim] into the cache, every block that gets a token at once."""
    case = s["case"]
    fmt, block, blocks = case["fmt"], case["block"], cache.shape[0]
    cu, kv_len = s["cu_q"].long(), s["kv_lens"].long()
    token = torch.arange(x.shape[0], device="cuda")
    b = torch.searchsorted(cu[1:].contiguous(), token, right=True)
    pos = kv_len[b] - (cu[b + 1] - token)
    where, slot = s["table"].long()[b, pos // block], pos % block
    touched = torch.zeros(blocks, dtype=torch.bool, device="cuda")
    touched[where] = True
    first = torch.full((blocks,), block, dtype=torch.int64, device="cuda")
    first.scatter_reduce_(0, where, slot, "amin")                            # the block's tokens before are kept
    x = x.float()
    amax = torch.zeros((blocks, x.shape[1]), device="cuda")
    amax.scatter_reduce_(0, where[:, None].expand(-1, x.shape[1]), x.abs().amax(-1), "amax")
    new = _least_scale(amax, fmt)
    new = torch.where(touched[:, None], torch.where((first > 0)[:, None], torch.maximum(new, scale), new), scale)
    rows = touched.nonzero()[:, 0]
    old = _values(cache[rows], fmt) * (scale[rows] / new[rows])[..., None, None]
    keep = torch.arange(block, device="cuda")[None] < first[rows][:, None]
    raised = (new[rows] > scale[rows])[:, :, None] & keep[:, None, :]
    cache[rows] = torch.where(raised[..., None], _codes(old, fmt), cache[rows])
    cache[where, :, slot] = _codes(x / new[where][..., None], fmt)
    scale.copy_(new)


def _norm(s):
    case = s["case"]
    x = s["x"].float()
    out = {}
    if s["r"] is not None:
        x = x + s["r"].float()
        out["residual"] = x.to(torch.bfloat16)
    n = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * s["w"].float()
    out["y"] = n.to(torch.bfloat16)
    if case["out8"]:
        group = case["group"] or case["width"]
        n = n.view(*n.shape[:2], -1, group)
        scale = n.abs().amax(-1) / E4M3_MAX
        code = n / scale.clamp(min=1e-38)[..., None]
        out["codes"] = code.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).reshape(x.shape)
        out["scales"] = scale
    return out


def _rotate(x, cos, sin, rot, halves):
    u, v = (x[..., :rot // 2], x[..., rot // 2:rot]) if halves else (x[..., 0:rot:2], x[..., 1:rot:2])
    a, b = u * cos - v * sin, v * cos + u * sin
    turned = torch.cat((a, b), -1) if halves else torch.stack((a, b), -1).flatten(-2)
    return torch.cat((turned, x[..., rot:]), -1)


def _rope(s):
    case = s["case"]
    angle = s["positions"].double()[s["pair_axis"]].t() * s["inv_freq"][None]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    return {n: _rotate(s[n].float(), cos, sin, case["rot"], case["halves"]).to(torch.bfloat16) for n in ("q", "k")}


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "attention":
        return _attention(state)
    if op == "append":
        _append_one(state, state["k"], state["k_cache"], state["k_scale"])
        _append_one(state, state["v"], state["v_cache"], state["v_scale"])
        return _cache_out(state)
    return _norm(state) if op == "norm" else _rope(state)


# ------------------------------------------------------------------------------------------------------------ 64 bits

def _exact_attention(s):
    case = s["case"]
    hq, hk, d, block = case["heads"], case["kv_heads"], case["dim"], case["block"]
    t = torch.float8_e4m3fn if case["fmt"] == "e4m3" else torch.int8
    out = torch.zeros((s["qkv"].shape[0], hq, d), dtype=torch.float64, device="cuda")
    lse = torch.zeros((s["qkv"].shape[0], hq), dtype=torch.float64, device="cuda")
    at = 0
    for b, (q, kv) in enumerate(zip(*_lengths(case))):
        ids = s["table"][b, :-(-kv // block)].long()
        see = torch.arange(kv, device="cuda")[None] <= torch.arange(kv - q, kv, device="cuda")[:, None]
        if case["window"]:
            see &= torch.arange(kv, device="cuda")[None] > torch.arange(kv - q, kv, device="cuda")[:, None] - case["window"]
        for g in range(hk):
            kk, vv = ((s[c][ids, g].view(t).double() * s[sc][ids, g].double()[:, None, None]).reshape(-1, d)[:kv]
                      for c, sc in (("k_cache", "k_scale"), ("v_cache", "v_scale")))
            for h in range(g * (hq // hk), (g + 1) * (hq // hk)):
                x = (s["qkv"][at:at + q, h].double() @ kk.t()) * s["scale"]
                x = torch.where(see, x, -math.inf)
                lse[at:at + q, h] = torch.logsumexp(x, -1)
                out[at:at + q, h] = torch.softmax(x, -1) @ vv
        at += q
    return {"out": out, "lse": lse}


def _exact_append(s):
    case = s["case"]
    block, top = case["block"], 448.0 if case["fmt"] == "e4m3" else 127.0
    t = torch.float8_e4m3fn if case["fmt"] == "e4m3" else torch.int8
    got = {}
    for n in ("k", "v"):
        code, scale = s[n + "_cache"].view(t).double(), s[n + "_scale"].double().clone()
        at = 0
        for b, (q, kv) in enumerate(zip(*_lengths(case))):
            for j in range((kv - q) // block, -(-kv // block)):
                lo, hi = max(kv - q, j * block), min(kv, (j + 1) * block)
                c = int(s["table"][b, j])
                x = s[n][at + lo - (kv - q):at + hi - (kv - q)].double().transpose(0, 1)         # [heads, tokens, dim]
                need = x.abs().amax((1, 2)) / top
                new = torch.tensor([2.0 ** max(-126, math.frexp(a)[1] - (math.frexp(a)[0] == 0.5)) if a else 2.0 ** -126
                                    for a in need.tolist()], dtype=torch.float64, device="cuda")
                if lo % block:
                    new = torch.maximum(new, scale[c])
                    code[c, :, :lo % block] *= (scale[c] / new)[:, None, None]
                code[c, :, lo - j * block:hi - j * block] = x / new[:, None, None]
                scale[c] = new
            at += q
        got[n], got[n + "_scale"] = code, scale
    return got


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "attention":
        return None if work(case)["flops"] > 6e12 else _exact_attention(s)
    if op == "append":
        return _exact_append(s) if sum(_lengths(case)[0]) // case["block"] + 2 * case["batch"] < 4000 else None
    if op == "norm":
        x = s["x"].double() + (s["r"].double() if s["r"] is not None else 0)
        n = x / torch.sqrt(torch.mean(x * x, -1, keepdim=True) + 1e-6) * s["w"].double()
        out = {"y": n}
        if s["r"] is not None:
            out["residual"] = x
        if case["out8"]:
            parts = n.reshape(*n.shape[:2], -1, case["group"] or case["width"])
            out["scales"] = parts.abs().amax(-1) / 448
            out["codes"] = (parts / out["scales"][..., None]).reshape(n.shape)
        return out
    pairs = case["rot"] // 2
    out = {}
    axis = s["pair_axis"]
    turn = torch.polar(torch.ones((case["tokens"], pairs), dtype=torch.float64, device="cuda"),
                       torch.stack([s["positions"][int(a)].double() * s["inv_freq"][i] for i, a in enumerate(axis)], 1))
    for n in ("q", "k"):
        x = s[n].double().clone()
        even, odd = (slice(0, pairs), slice(pairs, 2 * pairs)) if case["halves"] else (slice(0, 2 * pairs, 2), slice(1, 2 * pairs, 2))
        z = torch.complex(x[..., even], x[..., odd]) * turn[:, None]
        x[..., even], x[..., odd] = z.real, z.imag
        out[n] = x
    return out
