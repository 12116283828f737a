"""Measured cases of a hybrid stack's serving step: packed prompts, tables built on the GPU, linear attention.

Operators (op of a case):
  packed    causal grouped-query attention over whole prompts of different lengths, packed one
            after another, q, k and v as they leave a fused projection (no cache is read)
  grow      the step's tokens enter the sequences: blocks from a free list on the GPU, block
            tables, lengths, row offsets, cache slots and positions of every token
  free      blocks of finished or evicted sequences go back to the free list
  linear    linear attention with a decay for each head, a chunk of tokens a sequence
            (S_t = a S_{t-1} + k_t v_t^T, o_t = scale q_t^T S_t; S carried in 32 bits)
  linear1   the same for one token a sequence
"""
import math
import random

import torch

own = False

BS = 16  # tokens a block


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one short prompt that nobody else waits beside: the latency of a call
        {"name": "packed 1x37", "op": "packed", "batch": 1, "heads": 32, "kv_heads": 8, "dim": 128, "lo": 37, "hi": 37},
        # a server's prefill step of cold prompts of all lengths, one of them empty
        {"name": "packed 48 ragged", "op": "packed", "batch": 48, "heads": 32, "kv_heads": 8, "dim": 128, "lo": 0, "hi": 1300},
        # head dim 64 and a group of 3, 7 prompts around 1500 tokens
        {"name": "packed 7 d64 g3", "op": "packed", "batch": 7, "heads": 24, "kv_heads": 8, "dim": 64, "lo": 801, "hi": 2203},
        # one long document, group 8: the largest
        {"name": "packed 1x16384", "op": "packed", "batch": 1, "heads": 16, "kv_heads": 2, "dim": 128, "lo": 16384, "hi": 16384},
        # a decode step: one token for each of 64 sequences of about 1088
        {"name": "grow 64x1", "op": "grow", "batch": 64, "lo": 1024, "hi": 1152, "new_lo": 1, "new_hi": 1, "spare": 64},
        # a step of 256 requests, prompts and decodes mixed, whose last ones find no blocks left
        {"name": "grow 256 mixed", "op": "grow", "batch": 256, "lo": 0, "hi": 8000, "new_lo": 0, "new_hi": 700, "spare": -500},
        # the blocks of a few finished sequences out of 64
        {"name": "free 64x72", "op": "free", "batch": 64, "lo": 0, "hi": 72, "width": 72},
        # what an eviction of 32 long sequences gave up
        {"name": "free 32x2048", "op": "free", "batch": 32, "lo": 300, "hi": 2000, "width": 2048},
        # one user's token in a layer of 32 heads: the latency of a call
        {"name": "linear1 1", "op": "linear1", "batch": 1, "heads": 32, "kv_heads": 32, "dim": 128},
        # a batched decode step
        {"name": "linear1 64", "op": "linear1", "batch": 64, "heads": 32, "kv_heads": 32, "dim": 128},
        # chunks of a mixed step: 24 sequences, some fresh, some with a state, the shortest of one token
        {"name": "linear 24 ragged", "op": "linear", "batch": 24, "heads": 16, "kv_heads": 16, "dim": 128, "lo": 1, "hi": 1100},
        # one long prompt
        {"name": "linear 1x20000", "op": "linear", "batch": 1, "heads": 32, "kv_heads": 32, "dim": 128, "lo": 20000, "hi": 20000},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def _draw(rng):
    op = rng.choice(["packed", "packed", "packed", "grow", "free", "linear1", "linear", "linear"])
    kvh = rng.choice([1, 2, 3, 4, 8, 8, 16])
    dim = rng.choice([64, 128, 128])
    if op == "packed":
        hi = _log(rng, 1, 16384)
        return {"op": op, "batch": _log(rng, 1, 64), "heads": kvh * rng.choice([1, 1, 2, 3, 4, 5, 8, 8]), "kv_heads": kvh, "dim": dim,
                "lo": rng.choice([0, hi // 2, hi]), "hi": hi}
    if op == "grow":
        hi, new = _log(rng, 1, 30000), _log(rng, 1, 2000)
        return {"op": op, "batch": _log(rng, 1, 512), "lo": rng.choice([0, hi // 2]), "hi": hi, "new_lo": rng.choice([0, 1, new]), "new_hi": new,
                "spare": rng.choice([1000, 0, -_log(rng, 1, 1000)])}
    if op == "free":
        width = _log(rng, 1, 3000)
        hi = rng.randint(0, width)
        return {"op": op, "batch": _log(rng, 1, 256), "lo": rng.choice([0, hi // 2]), "hi": hi, "width": width}
    if op == "linear1":
        return {"op": op, "batch": _log(rng, 1, 128), "heads": kvh * rng.choice([1, 1, 2, 4]), "kv_heads": kvh, "dim": dim}
    hi = _log(rng, 1, 20000)
    return {"op": op, "batch": _log(rng, 1, 64), "heads": kvh * rng.choice([1, 1, 1, 2, 3, 4]), "kv_heads": kvh, "dim": dim,
            "lo": rng.choice([0, hi // 2, hi]), "hi": hi}


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 100)


def _room(case):
    """Values of the largest tensors that the plain form makes."""
    n, per = case.get("hi", 1), case["batch"] * case.get("heads", 1)
    if case["op"] == "packed":
        return per * n * n
    if case["op"] == "linear":
        return 8 * per * (n + 64) * case["dim"]
    return 0


def draw(rng):
    most = {op: max(_cost(c) for c in listed() if c["op"] == op) for op in ("packed", "grow", "free", "linear", "linear1")}
    while True:
        c = _draw(rng)
        if _cost(c) <= most[c["op"]] and _room(c) <= 4.5e9:
            return c


# ------------------------------------------------------------------------------------ the inputs
def _lens(case, lo="lo", hi="hi"):
    """Lengths of the sequences, of the case alone; both ends of the range are among them."""
    r = random.Random("%d %d %d" % (case["batch"], case[lo], case[hi]))
    v = [r.randint(case[lo], case[hi]) for _ in range(case["batch"])]
    v[0] = case[hi]
    if len(v) > 1:
        v[-1] = case[lo]
    return v


def _cu(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def _blocks(n):
    return (n + BS - 1) // BS


def _grown(case):
    """grow: each sequence's length, its new tokens, the blocks those take, and how many blocks the free list holds."""
    lens, new = _lens(case), _lens(case, "new_lo", "new_hi")
    need = [_blocks(a + b) - _blocks(a) for a, b in zip(lens, new)]
    return lens, new, need, max(0, sum(need) + case["spare"])


def _counts(case):
    """free: how many blocks each row gives back; in a narrow table only every eighth sequence has finished."""
    v = _lens(case)
    return v if case["width"] > 1000 else [n if i % 8 == 0 else 0 for i, n in enumerate(v)]


def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)
    op, s, batch = case["op"], {"case": case}, case["batch"]
    if op == "free":
        counts, width = _counts(case), case["width"]
        total, room = batch * width, 1000
        perm = torch.randperm(total + room, device="cuda", generator=gen).to(torch.int32)
        there = torch.arange(width, device="cuda") < _ints(counts)[:, None]
        s["ids"] = torch.where(there, perm[:total].view(batch, width), torch.full((), -1, dtype=torch.int32, device="cuda"))
        s["counts"] = _ints(counts)
        s["free"] = torch.cat([perm[total:], torch.full((total,), -1, dtype=torch.int32, device="cuda")])
        s["num_free"] = _ints([room])
        return s
    if op == "grow":
        lens, new, _, have = _grown(case)
        width = _blocks(case["hi"] + case["new_hi"])
        used = sum(_blocks(n) for n in lens)
        perm = torch.randperm(used + have + 1, device="cuda", generator=gen).to(torch.int32)
        count = _ints([_blocks(n) for n in lens], torch.int64)
        j = torch.arange(width, device="cuda")
        at = ((count.cumsum(0) - count)[:, None] + j).clamp(max=len(perm) - 1)
        s["tables"] = torch.where(j < count[:, None], perm[at], torch.full((), -1, dtype=torch.int32, device="cuda"))
        s["lens"], s["new"] = _ints(lens), _ints(new)
        s["free"], s["num_free"] = perm[used:].contiguous(), _ints([have])
        s["max_tokens"] = _max_tokens(case)
        return s
    heads, kvh, d = case["heads"], case["kv_heads"], case["dim"]
    rows = batch if op == "linear1" else sum(_lens(case))
    # q, k and v of a token lie side by side, as a fused projection leaves them
    qkv = torch.randn(rows, heads + 2 * kvh, d, device="cuda", generator=gen).to(torch.bfloat16)
    s["q"], s["k"], s["v"] = qkv[:, :heads], qkv[:, heads:heads + kvh], qkv[:, heads + kvh:]
    s["scale"] = 1.0 / math.sqrt(d)
    if op != "linear1":
        s["cu"], s["most"] = _ints(_cu(_lens(case))), case["hi"]
    if op != "packed":
        slots = batch + 3
        s["state"] = torch.randn(slots, kvh, d, d, device="cuda", generator=gen)
        s["slots"] = torch.randperm(slots, device="cuda", generator=gen)[:batch].to(torch.int32)
        # heads remember between a few and a few hundred tokens
        span = torch.rand(kvh, device="cuda", generator=gen, dtype=torch.float64) * math.log(350) + math.log(1.4)
        s["log_decay"] = (-torch.exp(-span)).float()
        # every third sequence begins with this call
        before = torch.randint(1, 5000, (batch,), device="cuda", generator=gen, dtype=torch.int32)
        before[::3] = 0
        s["lens"] = before + (1 if op == "linear1" else s["cu"][1:] - s["cu"][:-1])
    return s


def _max_tokens(case):
    """Rows of a step's buffers: its tokens, rounded up to a multiple of 64 as a captured step pads them."""
    return (sum(_lens(case, "new_lo", "new_hi")) + 63) // 64 * 64


# ------------------------------------------------------------------------------------ one pass
def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import paged_kv_gqa_slot_gb300 as pa
    op = s["case"]["op"]
    if op == "packed":
        return pa.pa_prefill_packed(s["q"], s["k"], s["v"], s["cu"], s["scale"], s["most"])
    if op == "grow":
        return pa.pa_kv_grow(s["tables"], s["lens"], s["new"], s["free"], s["num_free"], s["max_tokens"])
    if op == "free":
        return s["free"], pa.pa_kv_free(s["ids"], s["counts"], s["free"], s["num_free"])
    if op == "linear1":
        out = pa.pa_linear_decode(s["state"], s["slots"], s["q"], s["k"], s["v"], s["log_decay"], s["lens"], s["scale"])
    else:
        out = pa.pa_linear_prefill(s["state"], s["slots"], s["q"], s["k"], s["v"], s["log_decay"], s["cu"], s["lens"], s["scale"], s["most"])
    return out, s["state"]


def _run_plain(s):
    return {"packed": _plain_packed, "grow": _plain_grow, "free": _plain_free, "linear": _plain_linear, "linear1": _plain_linear1}[s["case"]["op"]](s)


def _rows_of(s):
    """Sequence and place of every packed row; the row of every place of a padded batch, and whether there is one."""
    cu = s["cu"].long()
    t = torch.arange(s["q"].shape[0], device=cu.device)
    seq = torch.bucketize(t, cu[1:], right=True)
    i = torch.arange(max(s["most"], 1), device=cu.device)
    there = i < (cu[1:] - cu[:-1])[:, None]
    return seq, t - cu[seq], (cu[:-1, None] + i).clamp(max=max(len(t) - 1, 0)), there


def _plain_packed(s):
    if s["q"].shape[0] == 0:
        return torch.zeros(s["q"].shape, dtype=torch.bfloat16, device=s["q"].device)
    seq, place, row, there = _rows_of(s)
    kvh, heads, d = s["k"].shape[1], s["q"].shape[1], s["q"].shape[2]
    b, n = row.shape
    q = s["q"][row].float().view(b, n, kvh, heads // kvh, d).permute(0, 2, 3, 1, 4)  # [b, kvh, g, n, d]
    k, v = (x[row].float().masked_fill(~there[:, :, None, None], 0.0).transpose(1, 2).unsqueeze(2) for x in (s["k"], s["v"]))  # [b, kvh, 1, n, d]
    x = (q @ k.transpose(3, 4)).mul_(s["scale"])
    i = torch.arange(n, device=row.device)
    x.masked_fill_(i > i[:, None], -math.inf)  # a row past a sequence's end sees its first keys, and is not read
    p = x.sub_(x.amax(-1, keepdim=True)).exp_()
    o = (p @ v) / p.sum(-1, keepdim=True)
    return o.permute(0, 3, 1, 2, 4).reshape(b, n, heads, d)[seq, place].to(torch.bfloat16)


def _plain_grow(s):
    tables, lens, new, rows = s["tables"], s["lens"].long(), s["new"].long(), s["max_tokens"]
    need = (lens + new + BS - 1) // BS - (lens + BS - 1) // BS
    got = ((need == 0) | (need.cumsum(0) <= s["num_free"])) & (new.cumsum(0) <= rows)  # in order, while blocks and rows last
    new, need = torch.where(got, new, torch.zeros_like(new)), torch.where(got, need, torch.zeros_like(need))
    cu = torch.nn.functional.pad(new.cumsum(0), (1, 0))
    first = need.cumsum(0) - need
    j = torch.arange(tables.shape[1], device=tables.device) - ((lens + BS - 1) // BS)[:, None]
    at = (s["num_free"].long() - 1 - first[:, None] - j).clamp(0, len(s["free"]) - 1)  # the list is used up from its end
    tables.copy_(torch.where((j >= 0) & (j < need[:, None]), s["free"][at], tables))
    t = torch.arange(rows, device=tables.device)
    seq = torch.bucketize(t, cu[1:], right=True)
    there = seq < len(lens)
    seq = seq.clamp(max=len(lens) - 1)
    pos = torch.where(there, lens[seq] + t - cu[seq], torch.zeros_like(t))
    slots = torch.where(there, tables[seq, pos // BS].long() * BS + pos % BS, torch.full_like(t, -1))
    return (tables, (lens + new).int(), (s["num_free"] - need.sum()).int(), cu.int(), slots, pos.int(),
            torch.where(there, seq, torch.full_like(seq, -1)).int())


def _plain_free(s):
    ids, free = s["ids"], s["free"]
    mine = (torch.arange(ids.shape[1], device=ids.device) < s["counts"][:, None]) & (ids >= 0)
    flat = mine.reshape(-1)
    at = s["num_free"].long() + flat.long().cumsum(0) - 1
    room = torch.cat([free, free.new_zeros(1)])  # what does not leave goes to a place of its own
    room[torch.where(flat, at, torch.full_like(at, len(free)))] = ids.reshape(-1)
    free.copy_(room[:-1])
    return free, (s["num_free"] + flat.sum()).int()


def _plain_linear1(s):
    state, at = s["state"], s["slots"].long()
    kvh, heads = s["k"].shape[1], s["q"].shape[1]
    a = torch.exp(s["log_decay"].double()).float()
    old = torch.where((s["lens"] > 1)[:, None, None, None], state[at], torch.zeros_like(state[:1]))
    now = old * a[:, None, None] + s["k"].float().unsqueeze(3) * s["v"].float().unsqueeze(2)
    state[at] = now
    q = s["q"].float().reshape(len(at), kvh, heads // kvh, -1)
    return ((q @ now) * s["scale"]).reshape(s["q"].shape).to(torch.bfloat16), state


def _plain_linear(s):
    """In chunks of 64: within a chunk the masked products, between chunks one product with the decays."""
    state, at, c = s["state"], s["slots"].long(), 64
    kvh, heads, d = s["k"].shape[1], s["q"].shape[1], s["q"].shape[2]
    if s["q"].shape[0] == 0:
        return torch.zeros(s["q"].shape, dtype=torch.bfloat16, device=state.device), state
    seq, place, row, there = _rows_of(s)
    b, pad = row.shape[0], -row.shape[1] % c
    row, there = torch.nn.functional.pad(row, (0, pad)), torch.nn.functional.pad(there, (0, pad))
    m, g = row.shape[1] // c, heads // kvh
    hide = ~there[:, :, None, None]
    q, k, v = (x[row].float().masked_fill(hide, 0.0).view(b, m, c, x.shape[1], d).permute(0, 3, 1, 2, 4) for x in (s["q"], s["k"], s["v"]))  # [b, h, m, c, d]
    la = s["log_decay"].double()
    i = torch.arange(c, device=row.device)
    far = torch.exp(la[:, None, None] * (i[:, None] - i).clamp(min=0)).tril().float()  # [h, c, c]
    q = q.reshape(b, kvh, g, m, c, d)
    inner = ((q @ k.transpose(3, 4).unsqueeze(2)) * far[:, None, None]) @ v.unsqueeze(2)
    left = (s["cu"][1:] - s["cu"][:-1]).long()[:, None] - torch.arange(1, m + 1, device=row.device) * c  # tokens behind each chunk
    mine = (left + c).clamp(0, c)  # tokens in each chunk
    rest = torch.exp(la[:, None, None] * (mine[:, None, :, None] - 1 - i).clamp(min=0)).float()  # [b, h, m, c]
    add = (k * rest[..., None]).transpose(3, 4) @ v  # [b, h, m, d, d]
    begin = torch.nn.functional.pad(mine.cumsum(1), (1, 0)).double()  # tokens before each chunk, and all of them
    gap = begin[:, :, None] - begin[:, None, 1:]  # from the end of chunk n to the begin of chunk m
    w = torch.exp(la[:, None, None] * gap[:, None].clamp(min=0)) * (torch.arange(m + 1, device=row.device)[:, None] > torch.arange(m, device=row.device))
    old = torch.where((s["lens"].long() > left[:, 0] + c)[:, None, None, None], state[at], torch.zeros_like(state[:1]))
    carried = torch.exp(la[:, None] * begin[:, None]).float()[..., None, None] * old.unsqueeze(2)
    carried = carried + (w.float() @ add.reshape(b, kvh, m, d * d)).view(b, kvh, m + 1, d, d)
    state[at] = torch.where((left[:, 0] + c > 0)[:, None, None, None], carried[:, :, m], state[at])
    outer = (q @ carried[:, :, :m].unsqueeze(2)) * torch.exp(la[:, None] * (i + 1)).float()[:, None, None, :, None]
    o = ((inner + outer) * s["scale"]).permute(0, 3, 4, 1, 2, 5).reshape(b, m * c, heads, d)
    return o[seq, place].to(torch.bfloat16), state


# ------------------------------------------------------------------------------------ what it takes
def work(case):
    op, batch = case["op"], case["batch"]
    if op == "free":
        n = sum(_counts(case))
        return {"bytes": 8 * n + 4 * batch + 8, "flops": n}
    if op == "grow":
        lens, _, need, have = _grown(case)
        rows = _max_tokens(case)
        return {"bytes": batch * 16 + 4 + 8 * min(sum(need), have) + 4 * sum(1 for a in lens if a % BS) + 16 * rows + 8, "flops": 2 * rows}
    heads, kvh, d = case["heads"], case["kv_heads"], case["dim"]
    lens = [1] * batch if op == "linear1" else _lens(case)
    rows = sum(lens) * (2 * heads + 2 * kvh) * d * 2 + 4 * batch
    if op == "packed":
        return {"bytes": rows, "flops": 4 * sum(n * (n + 1) // 2 for n in lens) * heads * d}
    seen = sum(1 + (i % 3 != 0) for i, n in enumerate(lens) if n)  # states written, and read unless they begin
    return {"bytes": rows + seen * kvh * d * d * 4 + 8 * batch + 4 * kvh, "flops": sum(lens) * (3 * kvh + 2 * heads) * d * d}


# ------------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    op = case["op"]
    if op in ("grow", "free"):
        s = prepare(case, seed)
        if op == "free":
            free, n = s["free"].tolist(), int(s["num_free"].item())
            for ids, count in zip(s["ids"].tolist(), s["counts"].tolist()):
                for block in ids[:count]:
                    if block >= 0:
                        free[n] = block
                        n += 1
            return torch.tensor(free, dtype=torch.int32), torch.tensor([n], dtype=torch.int32)
        tables, lens, free = s["tables"].tolist(), s["lens"].tolist(), s["free"].tolist()[:s["num_free"].item()]
        cu, slots, pos, seq = [0], [], [], []
        asked_blocks = asked_rows = 0
        have = len(free)
        for b, new in enumerate(s["new"].tolist()):
            need = _blocks(lens[b] + new) - _blocks(lens[b])
            asked_blocks, asked_rows = asked_blocks + need, asked_rows + new
            if (need and asked_blocks > have) or asked_rows > s["max_tokens"]:
                new = need = 0
            for j in range(need):
                tables[b][_blocks(lens[b]) + j] = free.pop()
            for p in range(lens[b], lens[b] + new):
                slots.append(tables[b][p // BS] * BS + p % BS)
                pos.append(p)
                seq.append(b)
            lens[b] += new
            cu.append(cu[-1] + new)
        more = s["max_tokens"] - len(slots)
        whole = [torch.tensor(v, dtype=torch.int32) for v in (tables, lens, [len(free)], cu, pos + [0] * more, seq + [-1] * more)]
        return whole[0], whole[1], whole[2], whole[3], torch.tensor(slots + [-1] * more, dtype=torch.int64), whole[4], whole[5]
    heads, kvh, d = case["heads"], case["kv_heads"], case["dim"]
    lens = [1] * case["batch"] if op == "linear1" else _lens(case)
    if sum(n * n for n in lens) * heads * d * 4 > 8e12:
        return None
    s = prepare(case, seed)
    group, cu = heads // kvh, _cu(lens)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    if op == "packed":
        for b, n in enumerate(lens):
            for h in range(heads):
                q, k, v = (x[cu[b]:cu[b + 1], i].double() for x, i in ((s["q"], h), (s["k"], h // group), (s["v"], h // group)))
                x = torch.mm(q, k.T) * s["scale"]
                x.masked_fill_(torch.ones(n, n, dtype=torch.bool, device="cuda").triu_(1), -math.inf)
                out[cu[b]:cu[b + 1], h] = torch.softmax(x, 1) @ v
        return out
    state = s["state"].double()
    slots, total = s["slots"].tolist(), s["lens"].tolist()
    for b, n in enumerate(lens):
        if n == 0:
            continue
        i = torch.arange(n, device="cuda", dtype=torch.float64)
        for h in range(kvh):
            a = s["log_decay"][h].double()
            k, v = (x[cu[b]:cu[b + 1], h].double() for x in (s["k"], s["v"]))
            old = state[slots[b], h] * (0.0 if total[b] == n else 1.0)
            apart = i[:, None] - i
            far = torch.where(apart >= 0, torch.exp(a * apart.clamp(min=0)), torch.zeros_like(apart))
            for hq in range(h * group, (h + 1) * group):
                q = s["q"][cu[b]:cu[b + 1], hq].double()
                out[cu[b]:cu[b + 1], hq] = (((q @ k.T) * far) @ v + torch.exp(a * (i + 1))[:, None] * (q @ old)) * s["scale"]
            state[slots[b], h] = torch.exp(a * n) * old + (k * torch.exp(a * (n - 1 - i))[:, None]).T @ v
    return out, state
