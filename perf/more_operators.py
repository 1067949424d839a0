"""Cases that time and check what stands around the decoder layers of a program that generates text: the linear layer in
8-bit integers, the logits' penalties, biases and masks with the choice of a token, and the pages of the 8-bit cache.

`own` False: the operators in plain torch, 32-bit arithmetic.  `own` True: the library's calls.
"""
import math
import random

import torch

own = False


# ------------------------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one token through a square projection
        dict(name="linear 1x4096x4096", op="linear", rows=1, k=4096, n=4096, codes=False, out="bf16", weights=1),
        # a serving batch's last tokens through the head: fp32 logits of a ragged vocabulary
        dict(name="linear head 24 rows", op="linear", rows=24, k=4096, n=128003, codes=False, out="fp32", weights=1),
        # a chunk's tokens, rounded to 8 bits once for two products (gate and up)
        dict(name="linear chunk 301 two products", op="linear", rows=301, k=4096, n=11008, codes=True, out="bf16", weights=2),
        # a long prompt through the widest layer
        dict(name="linear prompt 8190", op="linear", rows=8190, k=4096, n=11008, codes=False, out="bf16", weights=1),
        # one request's next token: logits of one row, a short history, no grammar
        dict(name="logits 1x128003", op="logits", rows=1, vocab=128003, dtype="fp32", history=517, grammar=False, biases=0),
        # a serving batch whose answers follow grammars, with some biases
        dict(name="logits 48x151655 grammar", op="logits", rows=48, vocab=151655, dtype="bf16", history=4100, grammar=True,
             biases=300),
        # a large batch of many continuations
        dict(name="logits 512x128003", op="logits", rows=512, vocab=128003, dtype="fp32", history=2000, grammar=False,
             biases=20),
        # long documents in every history
        dict(name="logits 12x32000 long histories", op="logits", rows=12, vocab=32000, dtype="fp32", history=131000,
             grammar=False, biases=0),
        # four continuations of one prompt
        dict(name="pages fork 1x4", op="fork", prompts=1, ways=4, tokens=517, new=1, layers=8, kv_heads=8, dim=128, block=64),
        # a serving batch of prompts with five continuations each, a few drafted tokens
        dict(name="pages fork 48x5", op="fork", prompts=48, ways=5, tokens=4001, new=3, layers=2, kv_heads=8, dim=128,
             block=32),
        # a small pool after a few requests have left
        dict(name="pages compact 300", op="compact", blocks=300, live=0.4, slots=20, layers=1, kv_heads=4, dim=128, block=16),
        # a large pool, two layers of it
        dict(name="pages compact 9001", op="compact", blocks=9001, live=0.6, slots=256, layers=2, kv_heads=8, dim=128,
             block=64),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear", "logits", "logits", "fork", "compact"])
    if op == "linear":
        rows = rng.choice([1, _log(rng, 1, 32), _log(rng, 2, 512), _log(rng, 32, 8190)])
        k = 16 * _log(rng, 16, 896)
        n = _log(rng, 100, 130000 if rows <= 64 else 16000)
        weights = rng.choice([1, 1, 2])
        while weights * rows * k * n > 8190 * 4096 * 11008 or weights * k * n > 4096 * 128003:
            n = n // 2 + 1
        return dict(op="linear", rows=rows, k=k, n=n, codes=rng.random() < 0.4, out=rng.choice(["bf16", "bf16", "fp32"]),
                    weights=weights)
    if op == "logits":
        vocab = _log(rng, 1000, 262144)
        rows = _log(rng, 1, max(1, 60000000 // vocab)) if rng.random() < 0.8 else 1
        return dict(op="logits", rows=min(rows, 512), vocab=vocab, dtype=rng.choice(["bf16", "fp32"]),
                    history=min(_log(rng, 1, 131072), 4000000 // min(rows, 512)), grammar=rng.random() < 0.5,
                    biases=rng.choice([0, 0, 5, 300]))
    shape = dict(layers=rng.choice([1, 2, 4]), kv_heads=rng.choice([1, 2, 4, 8]), dim=rng.choice([64, 128, 128]),
                 block=rng.choice([16, 32, 64, 128]))
    if op == "fork":
        prompts = _log(rng, 1, 48)
        tokens = min(_log(rng, 1, 4001), 1200000000 // (prompts * _page_bytes(shape)) * shape["block"] + 1)
        return dict(op="fork", prompts=prompts, ways=rng.choice([2, 3, 4, 5]), tokens=tokens,
                    new=rng.choice([1, 1, 2, 3, 5]), **shape)
    blocks = min(_log(rng, 20, 9001), 2400000000 // _page_bytes(shape))
    return dict(op="compact", blocks=blocks, live=rng.choice([0.05, 0.3, 0.5, 0.8, 0.95]), slots=_log(rng, 1, 256), **shape)


def _lengths(case):
    """Token counts of a case's histories or prompts: part of the case, not of its values."""
    r = random.Random(str(sorted((k, v) for k, v in case.items() if k != "name")))
    if case["op"] == "logits":
        got = [r.randint(case["history"] // 2, case["history"]) for _ in range(case["rows"])]
        got[0] = case["history"]
        return got, [r.randint(0, n) for n in got]
    got = [r.randint(max(1, case["tokens"] // 8), case["tokens"]) for _ in range(case["prompts"])]
    got[0] = case["tokens"]
    return got


def _live(case):
    """Which pages of a pool to be compacted are in use, and how many move."""
    r = random.Random(str(sorted((k, v) for k, v in case.items() if k != "name")))
    live = [r.random() < case["live"] for _ in range(case["blocks"])]
    live[r.randrange(case["blocks"])] = True
    n = sum(live)
    return live, sum(live[n:])


def _page_bytes(case):
    return case["layers"] * 2 * case["kv_heads"] * (case["block"] * case["dim"] + 4)


def work(case):
    op = case["op"]
    if op == "linear":
        m, k, n, w = case["rows"], case["k"], case["n"], case["weights"]
        out = w * m * n * (2 if case["out"] == "bf16" else 4)
        return {"bytes": w * n * (k + 4) + 2 * m * k + out + (m * (k + 4) if case["codes"] else 0), "flops": 2 * m * k * n * w}
    if op == "logits":
        b, v = case["rows"], case["vocab"]
        return {"bytes": b * v * ((2 if case["dtype"] == "bf16" else 4) + 4 + (1 / 8 if case["grammar"] else 0))
                + 4 * sum(_lengths(case)[0]) + 8 * b * case["biases"] + 40 * b, "flops": 4 * b * v}
    if op == "fork":
        block, ways, new = case["block"], case["ways"], case["new"]
        lens = _lengths(case)
        copies = sum(ways - 1 for n in lens if n % block)
        entries = sum(ways * (-(-(n + new) // block)) for n in lens)
        return {"bytes": 2 * copies * _page_bytes(case) + 4 * 4 * entries, "flops": entries}
    moves = _live(case)[1]
    return {"bytes": 2 * moves * _page_bytes(case) + 4 * 3 * case["blocks"], "flops": case["blocks"]}


# ------------------------------------------------------------------------------------------------------------ inputs

def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _whole(g, lo, hi, *shape, dtype=torch.int32):
    return torch.randint(lo, hi, shape, generator=g, device="cuda", dtype=dtype)


def _caches(g, case, blocks):
    shape = (blocks, case["kv_heads"], case["block"], case["dim"])
    return ([_whole(g, 0, 256, *shape, dtype=torch.uint8) for _ in range(2 * case["layers"])],
            [torch.exp2(torch.floor(_normal(g, *shape[:2]))) for _ in range(2 * case["layers"])])


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 29)
    r = random.Random(seed * 7919 + 31)
    op = case["op"]
    s = {"case": dict(case)}
    if op == "linear":
        # activations with some channels larger than the rest; weights as they come out of a loader, already in 8 bits
        gain = torch.exp(0.5 * _normal(g, 1, case["k"]))
        s["x"] = (_normal(g, case["rows"], case["k"]) * gain).to(torch.bfloat16)
        s["w"] = [_normal(g, case["n"], case["k"]).mul_(32).round_().clamp_(-127, 127).to(torch.int8)
                  for _ in range(case["weights"])]
        s["w_scale"] = [torch.exp(0.3 * _normal(g, case["n"])) * 1e-3 for _ in range(case["weights"])]
    elif op == "logits":
        b, v = case["rows"], case["vocab"]
        lens, prompt = _lengths(case)
        dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        s["logits"] = _normal(g, b, v).mul_(3).to(dtype)
        # repeated tokens come often: half of every history is of a few hundred tokens
        few = _whole(g, 0, v, b, 300)
        n = case["history"]
        pick = few.gather(1, _whole(g, 0, 300, b, n, dtype=torch.int64))
        s["history"] = torch.where(_normal(g, b, n) > 0, pick, _whole(g, 0, v, b, n))
        s["history_lens"], s["prompt_lens"] = _i32(lens), _i32(prompt)
        s["repetition"] = 1 + 0.3 * _normal(g, b).abs()
        s["frequency"] = 0.2 * _normal(g, b)
        s["presence"] = 0.4 * _normal(g, b)
        s["temperature"] = 0.4 + _normal(g, b).abs()
        s["bias_offsets"] = s["bias_ids"] = s["bias"] = s["allowed"] = None
        if case["biases"]:
            k = min(case["biases"], v // 2)
            s["bias_offsets"] = _i32([k * i for i in range(b + 1)])
            # different tokens in each row: an odd step through the vocabulary from anywhere
            start, step = _whole(g, 0, v, b, 1, dtype=torch.int64), v // k
            s["bias_ids"] = ((start + step * torch.arange(k, device="cuda")) % v).to(torch.int32).reshape(-1)
            s["bias"] = 5 * _normal(g, b * k)
        if case["grammar"]:
            # one in eight tokens is allowed in most rows, every one in some
            bits = _whole(g, -2 ** 31, 2 ** 31, 3, b, -(-v // 32), dtype=torch.int64)
            bits = bits[0] & bits[1] & bits[2]
            s["allowed"] = torch.where(_whole(g, 0, 4, b, 1) == 0, -1, bits).to(torch.int32)
    elif op == "fork":
        lens, block, ways = _lengths(case), case["block"], case["ways"]
        pages = [-(-n // block) for n in lens]
        most = max(-(-(n + case["new"]) // block) for n in lens) + 1
        blocks = sum(pages) + len(lens) * ways * (2 + case["new"] // block) + 5
        order = list(range(blocks))
        r.shuffle(order)
        slots = len(lens) * ways + 1
        table, refs, at = torch.full((slots, most), -1, dtype=torch.int32), torch.zeros(blocks, dtype=torch.int32), 0
        kv = [0] * slots
        for i, n in enumerate(pages):           # prompt i is slot i, its continuations come after all prompts
            table[i, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
            refs[order[at:at + n]] = 1
            kv[i] = lens[i]
            at += n
        s["table"], s["refs"], s["kv_lens"] = table.cuda(), refs.cuda(), _i32(kv)
        parents = [i for i in range(len(lens)) for _ in range(ways - 1)]
        children = list(range(len(lens), len(lens) * ways))
        s["parents"], s["children"] = _i32(parents), _i32(children)
        # continuations first, so that each prompt's own sequence keeps the page that all share
        s["seqs"] = _i32(children + list(range(len(lens))))
        s["keep"] = _i32([0] * len(children) + lens)
        s["new"] = _i32([case["new"]] * (len(children) + len(lens)))
        s["codes"], s["scales"] = _caches(g, case, blocks)
    else:
        live, _ = _live(case)
        block = case["block"]
        pages = [i for i, a in enumerate(live) if a]
        r.shuffle(pages)
        # sequences of these pages, and now and then one more that shares the first pages of the one before
        runs, at = [[] for _ in range(case["slots"])], 0
        per = -(-len(pages) // case["slots"])
        for i in range(case["slots"]):
            mine = pages[at:at + per]
            at += len(mine)
            runs[i] = (runs[i - 1][:r.randint(0, len(runs[i - 1]))] if i % 3 == 2 else []) + mine
        most = 2 * per + 2
        table, refs = torch.full((len(runs), most), -1, dtype=torch.int32), torch.zeros(case["blocks"], dtype=torch.int32)
        for i, p in enumerate(runs):
            if p:
                table[i, :len(p)] = torch.tensor(p, dtype=torch.int32)
                refs[p] += 1
        s["table"], s["refs"] = table.cuda(), refs.cuda()
        s["kv_lens"] = _i32([max(0, len(p) * block - r.randrange(block)) for p in runs])
        s["codes"], s["scales"] = _caches(g, case, case["blocks"])
    return s


# ---------------------------------------------------------------------------------------------------------- own calls

def _run_own(s):
    import int4_group_quantized_int4g_gb300 as fl
    case = s["case"]
    op = case["op"]
    if op == "linear":
        dtype = torch.bfloat16 if case["out"] == "bf16" else torch.float32
        if not case["codes"]:
            return {"y": [fl.fl_int8_linear(s["x"], w, t, out_dtype=dtype) for w, t in zip(s["w"], s["w_scale"])]}
        codes, scale = fl.fl_int8_quantize(s["x"])
        return {"codes": codes, "scale": scale,
                "y": [fl.fl_int8_linear(codes, w, t, x_scale=scale, out_dtype=dtype) for w, t in zip(s["w"], s["w_scale"])]}
    if op == "logits":
        return fl.fl_logits_process(s["logits"], history=s["history"], history_lens=s["history_lens"],
                                    prompt_lens=s["prompt_lens"], repetition=s["repetition"], frequency=s["frequency"],
                                    presence=s["presence"], bias_offsets=s["bias_offsets"], bias_ids=s["bias_ids"],
                                    bias=s["bias"], allowed=s["allowed"], temperature=s["temperature"])
    pool, block = (s["refs"], s["table"], s["kv_lens"]), case["block"]
    if op == "fork":
        fl.fl_kv8_pages_free(*pool, s["seqs"], block, keep=s["keep"])
        fl.fl_kv8_pages_fork(*pool, s["parents"], s["children"], block)
        granted, pairs, count = fl.fl_kv8_pages_alloc(*pool, s["seqs"], s["new"], block)
        got = {"granted": granted, "refs": s["refs"], "table": s["table"], "kv_lens": s["kv_lens"]}
    else:
        table, refs, pairs, count, moved = fl.fl_kv8_pages_compact(*pool, block, in_place=False)
        got = {"refs": refs, "table": table, "moved": moved}
    fl.fl_kv8_pages_copy(s["codes"][0::2], s["codes"][1::2], s["scales"][0::2], s["scales"][1::2], pairs, count)
    return {**got, "pairs": pairs, "count": count, "codes": s["codes"], "scales": s["scales"]}


# -------------------------------------------------------------------------------------------------------- plain forms

def _quantize(x):
    x = x.float()
    top = x.abs().amax(-1)
    scale = top / torch.full_like(top, 127.0)
    # the nearest whole number to the quotient itself: 32 bits would round some of them onto a border first
    code = torch.round(x.double() / scale.double()[:, None]).float()
    return torch.where(scale[:, None] > 0, code, torch.zeros_like(x)), scale


def _linear(s):
    case = s["case"]
    dtype = torch.bfloat16 if case["out"] == "bf16" else torch.float32
    q, scale = _quantize(s["x"])
    y = [(torch.matmul(q, w.float().t()) * (scale[:, None] * t[None])).to(dtype) for w, t in zip(s["w"], s["w_scale"])]
    return {"codes": q.to(torch.int8), "scale": scale, "y": y} if case["codes"] else {"y": y}


def _counts(s):
    """How often each token stands in a row's output, and whether in its prompt."""
    case = s["case"]
    at = torch.arange(s["history"].shape[1], device="cuda")[None]
    real = at < s["history_lens"][:, None]
    answer = real & (at >= s["prompt_lens"][:, None])
    ids = s["history"].long()
    count = torch.zeros((case["rows"], case["vocab"]), device="cuda")
    count.scatter_add_(1, ids, answer.float())
    seen = torch.zeros((case["rows"], case["vocab"]), device="cuda")
    seen.scatter_add_(1, ids, real.float())
    return count, seen > 0


def _logits(s):
    case = s["case"]
    x = s["logits"].float()
    count, seen = _counts(s)
    r = s["repetition"][:, None]
    x = torch.where(seen, torch.where(x > 0, x / r, x * r), x)
    x = x - s["frequency"][:, None] * count
    x = torch.where(count > 0, x - s["presence"][:, None], x)
    if s["bias"] is not None:
        k = s["bias"].numel() // case["rows"]
        x = x.scatter_add(1, s["bias_ids"].view(-1, k).long(), s["bias"].view(-1, k))
    x = x * (1.0 / s["temperature"])[:, None]
    if s["allowed"] is not None:
        bit = (s["allowed"][:, :, None] >> torch.arange(32, device="cuda", dtype=torch.int32)) & 1
        x = torch.where(bit.view(case["rows"], -1)[:, :case["vocab"]] == 1, x, -math.inf)
    top = x.amax(-1, keepdim=True)
    some = top > -math.inf                          # a row without a token that may come: -1, and no probability
    token = torch.where(x == top, torch.arange(case["vocab"], device="cuda", dtype=torch.int32)[None], case["vocab"]).amin(-1)
    log_sum = (x - torch.where(some, top, 0.0)).exp().sum(-1, keepdim=True).log()
    return {"logits": x, "token": torch.where(some[:, 0], token, -1).to(torch.int32), "lse": (top + log_sum)[:, 0],
            "logprob": torch.where(some, -log_sum, -math.inf)[:, 0]}


def _pages(n, block):
    return (n + block - 1) // block


def _free_plain(s, block):
    table, lens, keep, seqs = s["table"], s["kv_lens"], s["keep"].long(), s["seqs"].long()
    old = lens[seqs].long()
    at = torch.arange(table.shape[1], device="cuda")[None]
    gone = (at >= _pages(keep, block)[:, None]) & (at < _pages(old, block)[:, None])
    rows = table[seqs]
    s["refs"].index_add_(0, rows.clamp(min=0).long().view(-1), -gone.to(torch.int32).view(-1))
    table[seqs] = torch.where(gone, -1, rows)
    lens[seqs] = torch.minimum(old, keep).to(torch.int32)


def _fork_plain(s, block):
    table, lens, parents, children = s["table"], s["kv_lens"], s["parents"].long(), s["children"].long()
    n = lens[parents]
    has = torch.arange(table.shape[1], device="cuda")[None] < _pages(n, block)[:, None]
    rows = table[parents]
    s["refs"].index_add_(0, rows.clamp(min=0).long().view(-1), has.to(torch.int32).view(-1))
    table[children] = torch.where(has, rows, table[children])
    lens[children] = n


def _alloc_plain(s, block):
    table, lens, refs = s["table"], s["kv_lens"], s["refs"]
    seqs, new = s["seqs"].long(), s["new"].long()
    order = torch.arange(seqs.numel(), device="cuda")
    old = lens[seqs].long()
    end = old + new
    page = table[seqs, torch.clamp(old // block, max=table.shape[1] - 1)].long().clamp(min=0)
    shared = (old % block > 0) & (new > 0) & (refs[page] > 1)
    # of the sequences that share a page, the last keeps it when nobody else has it
    sharers = torch.zeros_like(refs).index_add_(0, page, shared.to(torch.int32))
    last = torch.full(refs.shape, -1, dtype=torch.int64, device="cuda")
    last.scatter_reduce_(0, page, torch.where(shared, order, -1), "amax")
    copy = shared & ~((sharers[page] == refs[page]) & (last[page] == order))
    need = _pages(end, block) - _pages(old, block) + copy.long()
    upto = need.cumsum(0)
    ok = upto <= (refs == 0).sum()
    copy &= ok
    at = torch.arange(table.shape[1], device="cuda")[None]
    first = torch.where(copy, old // block, _pages(old, block))
    fresh = ok[:, None] & (at >= first[:, None]) & (at < _pages(end, block)[:, None])
    # free pages in ascending order, taken in the order of the list
    free = torch.sort((refs > 0).to(torch.int8), stable=True).indices
    rank = ((upto - need)[:, None] + at - first[:, None]).clamp(0, refs.numel() - 1)
    rows = torch.where(fresh, free[rank].to(torch.int32), table[seqs])
    table[seqs] = rows
    lens[seqs] = torch.where(ok, end, old).to(torch.int32)
    refs.index_add_(0, page, -copy.to(torch.int32))
    refs.index_add_(0, rows.clamp(min=0).long().view(-1), fresh.to(torch.int32).view(-1))
    pairs = torch.full((seqs.numel() + 1, 2), -1, dtype=torch.int32, device="cuda")
    to = torch.where(copy, copy.long().cumsum(0) - 1, seqs.numel())
    fill = rows.gather(1, torch.clamp(old // block, max=table.shape[1] - 1)[:, None])[:, 0]
    pairs[to] = torch.stack((page.to(torch.int32), fill), 1)
    return ok.to(torch.int32), pairs[:-1], copy.sum(dtype=torch.int32).view(1)


def _compact_plain(s, block):
    refs, table = s["refs"], s["table"]
    live = refs > 0
    n = live.sum()
    at = torch.arange(refs.numel(), device="cuda")
    high, hole = live & (at >= n), ~live & (at < n)
    holes = torch.sort((~hole).to(torch.int8), stable=True).indices     # the holes first, ascending
    moved = torch.where(high, holes[(high.long().cumsum(0) - 1).clamp(min=0)], at)
    moved = torch.where(live, moved, -1).to(torch.int32)
    to = torch.where(live, moved.long(), refs.numel())
    new_refs = torch.zeros(refs.numel() + 1, dtype=torch.int32, device="cuda")
    new_refs[to] = refs
    has = torch.arange(table.shape[1], device="cuda")[None] < _pages(s["kv_lens"], block)[:, None]
    new_table = torch.where(has, moved[table.clamp(min=0).long()], table)
    half = refs.numel() // 2
    pairs = torch.full((half + 1, 2), -1, dtype=torch.int32, device="cuda")
    pairs[torch.where(high, high.long().cumsum(0) - 1, half)] = torch.stack((at.to(torch.int32), moved), 1)
    return new_table, new_refs[:-1], pairs[:-1], high.sum(dtype=torch.int32).view(1), moved


def _pages_plain(s):
    case = s["case"]
    block = case["block"]
    if case["op"] == "fork":
        _free_plain(s, block)
        _fork_plain(s, block)
        granted, pairs, count = _alloc_plain(s, block)
        got = {"granted": granted, "refs": s["refs"], "table": s["table"], "kv_lens": s["kv_lens"]}
    else:
        table, refs, pairs, count, moved = _compact_plain(s, block)
        got = {"refs": refs, "table": table, "moved": moved}
    real = pairs[pairs[:, 0] >= 0].long()
    for t in s["codes"] + s["scales"]:
        t[real[:, 1]] = t[real[:, 0]]
    pairs = torch.where(pairs[:, :1] >= 0, pairs, -1)
    return {**got, "pairs": pairs, "count": count, "codes": s["codes"], "scales": s["scales"]}


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "linear":
        return _linear(state)
    return _logits(state) if op == "logits" else _pages_plain(state)


# ------------------------------------------------------------------------------------------------------------ 64 bits

def _exact_linear(s):
    case = s["case"]
    x = s["x"].double()
    scale = x.abs().max(-1).values / 127
    scale = scale.float().double()                      # the scale is held in 32 bits, and codes are of what is held
    q = torch.round(x / scale.clamp(min=1e-300)[:, None])
    y = []
    for w, t in zip(s["w"], s["w_scale"]):
        part = torch.empty((x.shape[0], w.shape[0]), dtype=torch.float64, device="cuda")
        for i in range(0, w.shape[0], 4096):
            part[:, i:i + 4096] = q @ w[i:i + 4096].double().t()
        y.append(part * scale[:, None] * t.double()[None])
    return {"codes": q, "scale": scale, "y": y} if case["codes"] else {"y": y}


def _exact_logits(s):
    case = s["case"]
    v = case["vocab"]
    lens, prompts = _lengths(case)
    out = s["logits"].double()
    token, lse = [], []
    for b in range(case["rows"]):
        h = s["history"][b, :lens[b]].long()
        x = out[b]
        for t in torch.unique(h).split(100000):
            x[t] = torch.where(x[t] > 0, x[t] / s["repetition"][b].double(), x[t] * s["repetition"][b].double())
        t, c = torch.unique(h[prompts[b]:], return_counts=True)
        x[t] -= c.double() * s["frequency"][b].double() + s["presence"][b].double()
        if s["bias"] is not None:
            lo, hi = s["bias_offsets"][b:b + 2].tolist()
            x[s["bias_ids"][lo:hi].long()] += s["bias"][lo:hi].double()
        x /= s["temperature"][b].double()
        if s["allowed"] is not None:
            i = torch.arange(v, device="cuda")
            x[(s["allowed"][b].long()[i // 32] >> (i % 32)) & 1 == 0] = -math.inf
        lse.append(torch.logsumexp(x, -1))
    lse = torch.stack(lse)
    return {"logits": out, "token": None, "lse": lse, "logprob": out.max(-1).values - lse}


def exact(case, seed):
    if case["op"] == "linear":
        flops = work(case)["flops"]
        return _exact_linear(prepare(case, seed)) if flops < 2e12 else None
    return _exact_logits(prepare(case, seed)) if case["op"] == "logits" else None
