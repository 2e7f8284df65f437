"""What the operators of the block-scaled INT8 cache are measured on.

Four operators of a serving program whose paged cache needs no calibration: every block of tokens has, for each KV
head, a scale of its own for its keys and one for its values, and the query stays bfloat16.

  append_gqa_block_paged        new keys and values into the cache; a block that is partly full is rescaled in place
  attn_gqa_block_paged          attention of packed new rows (single tokens, drafts, chunks, prompts), with the rows'
                                log-sum-exp
  attn_weights_gqa_block_paged  adds up, for each cached token and KV head, the attention weight that it gets
  evict_gqa_block_paged         keeps the first and the last tokens and those with the most weight, in other pages

New tokens are packed: rows q_start[b] .. q_start[b + 1] - 1 of q, k, v and out are the last tokens of the
kv_lens[b]-token context of sequence b.
"""
import itertools
import math
import random

import torch

own = False

DEV = "cuda"
D = 128                       # head size of the attention calls
MOST_SCORES = 1 << 31         # B * Hq * S * T of the largest case
NEG = float("-inf")


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # a decode step's input: 16 sequences, one new token each, inside a block that has others already
        dict(name="append_decode", op="append", B=16, S=1, T=4096, ragged=False, Hkv=8, D=128, page=64, block=64, mix=1),
        # prompts and single tokens in one batch of a server that prefills in chunks
        dict(name="append_prompt", op="append", B=16, S=4096, T=4096, ragged=True, Hkv=8, D=128, page=64, block=32, mix=2),
        # another head size and count, small blocks in pages that are no power of two, ragged lengths
        dict(name="append_odd", op="append", B=5, S=777, T=1500, ragged=True, Hkv=5, D=80, page=48, block=16, mix=3),
        # a decode step: 16 sequences, one row each, 4096 tokens of context
        dict(name="attn_decode", op="attn", B=16, S=1, T=4096, ragged=False, Hq=64, Hkv=8, page=64, block=64, mix=1),
        # a chunked-prefill step: one sequence with 512 new rows beside seven with one or some
        dict(name="attn_mixed", op="attn", B=8, S=512, T=4096, ragged=True, Hq=64, Hkv=8, page=64, block=32, mix=2),
        # a long chunk with as long a cached prefix
        dict(name="attn_long", op="attn", B=1, S=4096, T=8192, ragged=False, Hq=64, Hkv=8, page=128, block=128, mix=1),
        # a few drafted tokens to verify over a long context, odd group size, small blocks
        dict(name="attn_draft", op="attn", B=3, S=5, T=20001, ragged=True, Hq=35, Hkv=7, page=48, block=16, mix=4),
        # the weights of a decode step
        dict(name="weights_decode", op="weights", B=16, S=1, T=4096, ragged=False, Hq=64, Hkv=8, page=64, block=64, mix=1),
        # the weights of a prompt's chunk, before its cache is cut down
        dict(name="weights_prompt", op="weights", B=1, S=4096, T=8192, ragged=False, Hq=64, Hkv=8, page=64, block=64, mix=1),
        # drafts and short chunks, odd sizes
        dict(name="weights_odd", op="weights", B=5, S=37, T=5000, ragged=True, Hq=20, Hkv=5, page=80, block=16, mix=5),
        # sixteen contexts cut down to a quarter
        dict(name="evict_quarter", op="evict", B=16, T=4096, ragged=False, Hkv=8, D=128, page=64, block=64, budget=1024,
             sinks=4, recent=256, mix=1),
        # a long and some short contexts, odd sizes; what fits the budget is kept whole
        dict(name="evict_odd", op="evict", B=3, T=20001, ragged=True, Hkv=5, D=128, page=48, block=16, budget=2047,
             sinks=1, recent=129, mix=6),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["append", "attn", "attn", "weights", "evict"])
    hkv, g = rng.choice([1, 2, 3, 4, 5, 8]), rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 12, 16])
    block = rng.choice([16, 16, 32, 48, 64, 128])
    page = block * rng.choice([1, 1, 2, 3, 4])
    b, t = _log(rng, 1, 32), _log(rng, 1, 20001 if op in ("attn", "evict") else 8192)
    case = dict(op=op, B=b, ragged=rng.random() < 0.6, Hkv=hkv, page=page, block=block, mix=rng.randrange(1, 1 << 20))
    if op == "evict":
        while b * t * hkv > 16 * 4096 * 8:
            b, t = max(1, b // 2), t if b > 1 else t // 2
        budget = _log(rng, 1, max(1, min(t + t // 4, 4096)))
        sinks = min(rng.choice([0, 0, 1, 4, 16]), budget)
        return dict(case, B=b, T=t, D=rng.choice([64, 80, 128, 256]), budget=budget, sinks=sinks,
                    recent=rng.randint(0, budget - sinks))
    s = _log(rng, 1, min(t, 4096))
    if op == "append":
        d = rng.choice([64, 80, 128, 192, 256])
        while b * s * hkv * d > 16 * 2048 * 8 * 128:
            s, b = max(1, s // 2), b if s > 1 else max(1, b // 2)
        return dict(case, B=b, S=s, T=t, D=d)
    while b * s * t * g * hkv > MOST_SCORES // 4:
        if b > 1:
            b //= 2
        elif s > 64:
            s //= 2
        else:
            t //= 2
    return dict(case, B=b, S=min(s, t), T=t, Hq=g * hkv)


def _lens(case):
    """New rows and context length of each sequence (a function of the case alone). Ragged: the first sequence has
    the most rows and the longest context; the others one row or some."""
    b, s, t = case["B"], case.get("S", 0), case["T"]
    if not case["ragged"]:
        return [s] * b, [t] * b
    r = random.Random(case["mix"])
    ql = [s] + [(1 if r.random() < 0.5 else r.randint(0, max(1, s // 8))) if s else 0 for _ in range(b - 1)]
    return ql, [t] + [r.randint(max(q, 1), t) for q in ql[1:]]


# --------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _sigma(g, *shape):
    return torch.exp(torch.rand(shape, generator=g, device=DEV) * math.log(4.0) + math.log(0.5))


def _codes(g, shape):
    return (torch.randn(shape, generator=g, device=DEV) * (127 / 4.5)).round().clamp(-127, 127).to(torch.int8)


def _start(ql):
    return [0] + list(itertools.accumulate(ql))


def _scales(g, num, case, heads):
    """Scales of all blocks of a pool: a size of the head's own times one of the block's."""
    per = case["page"] // case["block"]
    return (_sigma(g, num, per, heads) * _sigma(g, heads) * (2.0 / 127)).contiguous()


def prepare(case, seed):
    g = _gen(seed)
    hkv, ps, bs, b = case["Hkv"], case["page"], case["block"], case["B"]
    d = case.get("D", D)
    ql, kl = _lens(case)
    start = _start(ql)
    n = start[-1] + 2                                              # two rows behind the last sequence
    most, kept = -(-case["T"] // ps), -(-case.get("budget", 0) // ps)
    num = b * (most + kept) + 3                                    # a few spare pages, all in a shuffled order
    perm = torch.randperm(num, generator=g, device=DEV).to(torch.int32)
    st = {"op": case["op"], "case": case, "n": n, "S": max(max(ql), 1), "T": max(max(kl), 1), "sm": 1.0 / math.sqrt(d)}
    st["table"] = perm[:b * most].reshape(b, most).contiguous()
    st["q_start"] = torch.tensor(start, dtype=torch.int32, device=DEV)
    st["kv_lens"] = torch.tensor(kl, dtype=torch.int32, device=DEV)
    # the program's own list of rows: which sequence, which of its new rows; and of cached tokens
    st["row_b"] = torch.tensor([i for i, q in enumerate(ql) for _ in range(q)], dtype=torch.int64, device=DEV)
    st["row_i"] = torch.tensor([i for q in ql for i in range(q)], dtype=torch.int64, device=DEV)
    st["tok_b"] = torch.repeat_interleave(torch.arange(b, device=DEV), st["kv_lens"].long())
    st["tok_t"] = torch.cat([torch.arange(k, device=DEV) for k in kl])
    st["k"] = _codes(g, (num, ps, hkv, d))
    st["k_scale"] = _scales(g, num, case, hkv)
    if case["op"] != "weights":
        st["v"] = _codes(g, (num, ps, hkv, d))
        st["v_scale"] = _scales(g, num, case, hkv)
    _spoil(st, kl, num)
    if case["op"] == "append":
        size = torch.cat([_sigma(g, hkv), _sigma(g, hkv)]) / 4
        kv = torch.randn(n, 2 * hkv, d, generator=g, device=DEV) * size[:, None]
        st["kv"] = kv.bfloat16()                                   # keys and values of one projection, side by side
        return st
    if case["op"] in ("evict", "weights"):
        w = torch.exp(2 * torch.randn(num, hkv, ps, generator=g, device=DEV))
        w = torch.where(w < 0.3, torch.zeros_like(w), w)               # many tokens that nothing looked at
        st["weights"] = w / 32
    if case["op"] == "evict":
        st["new_table"] = perm[b * most:b * (most + kept)].reshape(b, kept).contiguous()
        st["kept"] = torch.full((b, hkv, case["budget"]), -1, dtype=torch.int32, device=DEV)
        st["new_lens"] = torch.zeros(b, dtype=torch.int32, device=DEV)
        return st
    q = torch.randn(n, case["Hq"], d, generator=g, device=DEV) * _sigma(g, case["Hq"])[:, None]
    q[start[-1]:] = float("nan")                                   # nobody's rows
    st["q"] = q.bfloat16()
    st["lse"] = torch.full((n, case["Hq"]), 0.5, device=DEV)
    if case["op"] == "weights":
        _, st["lse"][:start[-1]] = _softmax(st)                    # of the attention call before
    else:
        st["out"] = torch.full((n, case["Hq"], d), 0.01, dtype=torch.bfloat16, device=DEV)
    return st


def _spoil(st, kl, num):
    """Scales of blocks that hold no token yet are whatever memory held: NaN here."""
    c = st["case"]
    live = torch.zeros(num * (c["page"] // c["block"]), dtype=torch.bool, device=DEV)
    live[_block_of(st, st["tok_b"], st["tok_t"])] = True
    for s in ("k_scale", "v_scale"):
        if s in st:
            st[s][~live.view(num, -1)] = float("nan")


# --------------------------------------------------------------------------- one pass
def run(st):
    if own:
        from int8_head_kv_gb300 import fa3
        c = st["case"]
        if st["op"] == "append":
            hkv = c["Hkv"]
            fa3.append_gqa_block_paged(st["kv"][:, :hkv], st["kv"][:, hkv:], st["k"], st["v"], st["k_scale"],
                                       st["v_scale"], st["table"], st["q_start"], st["kv_lens"])
        elif st["op"] == "attn":
            fa3.attn_gqa_block_paged(st["q"], st["k"], st["v"], st["k_scale"], st["v_scale"], st["q_start"],
                                     st["kv_lens"], st["table"], st["sm"], out=st["out"], lse=st["lse"])
        elif st["op"] == "weights":
            fa3.attn_weights_gqa_block_paged(st["q"], st["k"], st["k_scale"], st["lse"], st["weights"], st["q_start"],
                                             st["kv_lens"], st["table"], st["sm"])
        else:
            fa3.evict_gqa_block_paged(st["k"], st["v"], st["k_scale"], st["v_scale"], st["weights"], st["table"],
                                      st["kv_lens"], st["new_table"], c["budget"], sinks=c["sinks"],
                                      recent=c["recent"], kept=st["kept"], new_lens=st["new_lens"])
    else:
        {"append": _plain_append, "attn": _plain_attn, "weights": _plain_weights, "evict": _plain_evict}[st["op"]](st)
    return _outputs(st)


def _outputs(st):
    # The int8 codes are whole numbers and are compared as such: what they are is defined to the last bit.
    names = {"append": ("k", "v", "k_scale", "v_scale"), "attn": ("out", "lse"), "weights": ("weights",),
             "evict": ("kept", "new_lens", "k", "v", "k_scale", "v_scale", "weights")}
    return {x: st[x] for x in names[st["op"]]}


def _page_of(st, b, t):
    ps = st["case"]["page"]
    return st["table"][b, t // ps].long(), t % ps


def _block_of(st, b, t):
    """Number, in the pool, of the block that token t of sequence b lies in."""
    c = st["case"]
    page, at = _page_of(st, b, t)
    return page * (c["page"] // c["block"]) + at // c["block"]


def _plain_append(st):
    c = st["case"]
    hkv, bs, used = c["Hkv"], c["block"], st["row_b"].numel()
    first = (st["kv_lens"] - (st["q_start"][1:] - st["q_start"][:-1])).long()        # position of the first new token
    pos = first[st["row_b"]] + st["row_i"]
    page, at = _page_of(st, st["row_b"], pos)
    blk = _block_of(st, st["row_b"], pos)
    # the partly full block in front of each sequence's new tokens (a sequence without new ones: none)
    has = (st["q_start"][1:] > st["q_start"][:-1]) & (first % bs != 0)
    seq = torch.arange(c["B"], device=DEV)
    lead = _block_of(st, seq, first.clamp(max=st["table"].shape[1] * c["page"] - 1))
    old_at = torch.arange(bs, device=DEV)
    old_pos = (first - first % bs)[:, None] + old_at
    old = has[:, None] & (old_at < (first % bs)[:, None])
    op, oa = _page_of(st, seq[:, None], old_pos.clamp(max=st["table"].shape[1] * c["page"] - 1))
    for x, pool, scale in ((st["kv"][:used, :hkv], st["k"], st["k_scale"]), (st["kv"][:used, hkv:], st["v"], st["v_scale"])):
        flat = scale.view(-1, hkv)
        top = torch.zeros_like(flat).index_reduce_(0, blk, x.float().abs().amax(-1), "amax", include_self=True)
        top = top / torch.full_like(top, 127.0)                      # a scale: IEEE division
        before = torch.where(has[:, None], flat[lead], torch.zeros_like(flat[lead]))
        top[lead] = torch.where(has[:, None], torch.maximum(top[lead], before), top[lead])
        now = top[lead]
        ratio = torch.where(now > 0, before / now, torch.zeros_like(now))
        moved = (pool[op, oa].double() * ratio.double()[:, None, :, None]).round().to(torch.int8)
        pool[op[old], oa[old]] = moved[old]
        touched = torch.zeros(flat.shape[0], dtype=torch.bool, device=DEV)
        touched[blk] = True
        flat.copy_(torch.where(touched[:, None], top, flat))
        s = flat[blk][:, :, None]
        code = torch.where(s > 0, x.float() / s, torch.zeros_like(s)).round().clamp(-127, 127)
        pool[page, at] = code.to(torch.int8)


def _values(st, codes, scales):
    """float32 [B, T, Hkv, D] of all sequences' cached keys or values, zero behind each context."""
    c = st["case"]
    t = torch.arange(st["T"], device=DEV)
    seq = torch.arange(c["B"], device=DEV)[:, None]
    page, at = _page_of(st, seq, t[None, :].expand(c["B"], -1))
    x = codes[page, at].float() * scales.view(-1, c["Hkv"])[_block_of(st, seq, t[None, :])][..., None]
    return x.masked_fill_((t >= st["kv_lens"][:, None])[:, :, None, None], 0.0)


def _scores(st):
    """float32 [B, Hkv, G, S, T]; -inf where a row does not see a token, and for rows that are nobody's."""
    c = st["case"]
    b, s, t, hkv, g = c["B"], st["S"], st["T"], c["Hkv"], c["Hq"] // c["Hkv"]
    k = _values(st, st["k"], st["k_scale"]).permute(0, 2, 3, 1)                       # [B, Hkv, D, T]
    ql, kl = st["q_start"][1:] - st["q_start"][:-1], st["kv_lens"]
    i = torch.arange(s, device=DEV)
    rows = (st["q_start"][:-1, None] + i).clamp(max=st["n"] - 1).long()
    q = st["q"][rows].float().reshape(b, s, hkv, g, D).permute(0, 2, 3, 1, 4)
    x = torch.matmul(q.reshape(b, hkv, g * s, D), k).reshape(b, hkv, g, s, t).mul_(st["sm"])
    last = torch.where(i < ql[:, None], (kl - ql)[:, None] + i, torch.full_like(rows, -1))
    return x.masked_fill_(torch.arange(t, device=DEV) > last[:, None, None, :, None], NEG)


def _softmax(st):
    """Weights before the division, their sums and each row's log-sum-exp, in the rows' order."""
    x = _scores(st)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top.isinf(), torch.zeros_like(top), top)
    p = x.sub_(top).exp_()
    z = p.sum(-1, keepdim=True)
    b, hkv, g, s, _ = x.shape
    lse = (z.log() + top).permute(0, 3, 1, 2, 4).reshape(b, s, hkv * g)
    return (p, z), lse[st["row_b"], st["row_i"]]


def _plain_attn(st):
    (p, z), lse = _softmax(st)
    b, hkv, g, s, t = p.shape
    v = _values(st, st["v"], st["v_scale"]).transpose(1, 2)                           # [B, Hkv, T, D]
    o = torch.matmul(p.reshape(b, hkv, g * s, t), v).reshape(b, hkv, g, s, D)
    o = torch.where(z > 0, o / z, torch.zeros_like(o)).permute(0, 3, 1, 2, 4).reshape(b, s, hkv * g, D)
    used = st["row_b"].numel()
    st["out"][:used] = o[st["row_b"], st["row_i"]].bfloat16()
    st["lse"][:used] = lse


def _plain_weights(st):
    x = _scores(st)
    b, hkv, g, s, _ = x.shape
    rows = (st["q_start"][:-1, None] + torch.arange(s, device=DEV)).clamp(max=st["n"] - 1).long()
    lse = st["lse"][rows].reshape(b, s, hkv, g).permute(0, 2, 3, 1)[..., None]
    w = x.sub_(lse).exp_().sum((2, 3))                                                # [B, Hkv, T]
    tb, tt = st["tok_b"], st["tok_t"]
    page, at = _page_of(st, tb, tt)
    new = tt >= (st["kv_lens"] - (st["q_start"][1:] - st["q_start"][:-1])).long()[tb]
    got = w[tb, :, tt]
    st["weights"][page, :, at] = torch.where(new[:, None], got, st["weights"][page, :, at] + got)


def _plain_evict(st):
    c = st["case"]
    b, hkv, t, bs, m = c["B"], c["Hkv"], st["T"], c["block"], c["budget"]
    at = torch.arange(t, device=DEV)
    seq, head = torch.arange(b, device=DEV)[:, None, None], torch.arange(hkv, device=DEV)[None, :, None]
    lens = st["kv_lens"].long()[:, None, None]
    page, off = _page_of(st, seq, at)                                                 # [B, 1, T]
    w = st["weights"][page, head, off]
    rank = torch.where((at < c["sinks"]) | (at >= lens - c["recent"]), torch.full_like(w, float("inf")), w)
    rank = torch.where(at < lens, rank, torch.full_like(w, NEG))
    best = rank.sort(dim=-1, descending=True, stable=True).indices[..., :m]
    best = torch.nn.functional.pad(best, (0, m - best.shape[-1]), value=t)
    slot = torch.arange(m, device=DEV)
    live = slot < lens.clamp(max=m)                                                   # [B, 1, m]
    best = torch.where(live, best, torch.full_like(best, t)).sort(-1).values
    live = live.expand_as(best)
    src = best.clamp(max=t - 1)
    page, off = _page_of(st, seq, src)
    to = st["new_table"][seq, slot // c["page"]].long()
    to, put = to.expand_as(best), (slot % c["page"]).expand_as(best)
    hd = head.expand_as(best)
    pad = -m % bs
    for pool, scale in ((st["k"], st["k_scale"]), (st["v"], st["v_scale"])):
        s = torch.where(live, scale[page, off // bs, hd], torch.zeros((), device=DEV))
        new = torch.nn.functional.pad(s, (0, pad)).view(b, hkv, -1, bs).amax(-1).repeat_interleave(bs, -1)[..., :m]
        ratio = torch.where(new > 0, s / new, torch.zeros_like(new))
        code = (pool[page, off, hd].double() * ratio.double()[..., None]).round().to(torch.int8)
        pool[to[live], put[live], hd[live]] = code[live]
        scale[to[live], put[live] // bs, hd[live]] = new[live]
    st["weights"][to[live], hd[live], put[live]] = st["weights"][page, hd, off][live]
    st["kept"].copy_(torch.where(live, best, torch.full_like(best, -1)))
    st["new_lens"].copy_(st["kv_lens"].clamp(max=m))


# --------------------------------------------------------------------------- the floor
def work(case):
    hkv, bs = case["Hkv"], case["block"]
    ql, kl = _lens(case)
    n = sum(ql)
    blocks = lambda k: -(-k // bs)                                                    # noqa: E731
    if case["op"] == "append":
        values = n * 2 * hkv * case["D"]
        scales = sum(blocks(k) - (k - q) // bs for q, k in zip(ql, kl) if q) * 2 * hkv
        return {"bytes": values * 3 + scales * 4 + 12 * case["B"], "flops": values * 3}
    if case["op"] == "evict":
        kept = [min(k, case["budget"]) for k in kl]
        rows = sum(kept) * hkv
        size = sum(k for k, m in zip(kl, kept) if k > m) * hkv * 4                    # weights to choose by
        size += rows * (2 * 2 * case["D"] + 4 + 4 + 4) + sum(blocks(m) for m in kept) * hkv * 2 * 4
        return {"bytes": size, "flops": rows * 2 * case["D"]}
    hq = case["Hq"]
    live = [k if q else 0 for q, k in zip(ql, kl)]
    pairs = sum(q * (k - q) + q * (q + 1) // 2 for q, k in zip(ql, kl)) * hq
    size = sum(live) * hkv * D + sum(map(blocks, live)) * hkv * 4 + n * hq * D * 2 + n * hq * 4
    size += 4 * sum(-(-k // case["page"]) for k in live)
    if case["op"] == "weights":
        return {"bytes": size + (2 * sum(live) - n) * hkv * 4, "flops": 2 * D * pairs}
    return {"bytes": size + sum(live) * hkv * D + sum(map(blocks, live)) * hkv * 4 + n * hq * D * 2,
            "flops": 4 * D * pairs}


# --------------------------------------------------------------------------- the definition in 64 bits
def _rows_of(st, b, t):
    """Rows, in the flattened pool, of tokens t of sequence b."""
    ps = st["case"]["page"]
    return st["table"][b].long()[torch.div(t, ps, rounding_mode="floor")] * ps + t % ps


def exact(case, seed):
    st = prepare(case, seed)
    return _outputs(st) if _EXACT[case["op"]](st, case, *_lens(case)) is None else None


def _exact_append(st, case, ql, kl):
    hkv, bs = case["Hkv"], case["block"]
    start = _start(ql)
    for b, (n, end) in enumerate(zip(ql, kl)):
        for lo in range((end - n) // bs * bs, end if n else 0, bs):                  # the blocks that get new tokens
            old = torch.arange(lo, max(lo, end - n), device=DEV)
            new = torch.arange(max(lo, end - n), min(lo + bs, end), device=DEV)
            row = start[b] + new - (end - n)
            blk = _rows_of(st, b, torch.tensor([lo], device=DEV))[0] // bs
            for pool, scale, x in ((st["k"], st["k_scale"], st["kv"][row, :hkv]), (st["v"], st["v_scale"], st["kv"][row, hkv:])):
                flat, sc = pool.view(-1, hkv, pool.shape[-1]), scale.view(-1, hkv)
                s = (x.double().abs().amax(-1).amax(0) / 127).float()
                if old.numel():
                    at = _rows_of(st, b, old)
                    s = torch.maximum(s, sc[blk])
                    flat[at] = torch.round(flat[at].double() * (sc[blk].double() / s.double()).float().double()[:, None]).to(torch.int8)
                sc[blk] = s
                quotient = (x.double() / s.double()[:, None]).float()                # the float32 quotient decides
                flat[_rows_of(st, b, new)] = torch.clamp(torch.round(quotient), -127, 127).to(torch.int8)


def _cached(st, case, b, end, codes, scales):
    rows = _rows_of(st, b, torch.arange(end, device=DEV))
    hkv = case["Hkv"]
    return codes.view(-1, hkv, D)[rows].double() * scales.view(-1, hkv)[rows // case["block"]].double()[..., None]


def _exact_rows(st, case, ql, kl, use):
    """Calls use(rows, head, scores in 64 bits, sequence) for every sequence and query head."""
    start, g = _start(ql), case["Hq"] // case["Hkv"]
    for b, (n, end) in enumerate(zip(ql, kl)):
        if not n:
            continue
        k = _cached(st, case, b, end, st["k"], st["k_scale"])
        for h in range(case["Hq"]):
            x = st["q"][start[b]:start[b + 1], h].double() @ k[:, h // g].T * st["sm"]
            x += torch.full_like(x, NEG).triu(end - n + 1)
            use(slice(start[b], start[b + 1]), h, x, b)


def _exact_attn(st, case, ql, kl):
    g, out, lse = case["Hq"] // case["Hkv"], st["out"].double(), st["lse"].double()
    last = {}

    def use(rows, h, x, b):
        if b not in last:
            last.clear()
            last[b] = _cached(st, case, b, kl[b], st["v"], st["v_scale"])
        lse[rows, h] = torch.logsumexp(x, -1)
        out[rows, h] = torch.softmax(x, -1) @ last[b][:, h // g]

    _exact_rows(st, case, ql, kl, use)
    st["out"], st["lse"] = out, lse


def _exact_weights(st, case, ql, kl):
    g, ps, pool = case["Hq"] // case["Hkv"], case["page"], st["weights"].double()

    def use(rows, h, x, b):
        t = torch.arange(kl[b], device=DEV)
        page, at = st["table"][b].long()[torch.div(t, ps, rounding_mode="floor")], t % ps
        got = torch.exp(x - st["lse"][rows, h].double()[:, None]).sum(0)
        if h % g == 0:
            pool[page, h // g, at] *= t < kl[b] - ql[b]                              # new tokens begin with nothing
        pool[page, h // g, at] += got

    _exact_rows(st, case, ql, kl, use)
    st["weights"] = pool


def _exact_evict(st, case, ql, kl):
    hkv, bs, m, ps = case["Hkv"], case["block"], case["budget"], case["page"]
    d = case["D"]
    k_scale, v_scale = st["k_scale"].view(-1, hkv), st["v_scale"].view(-1, hkv)
    for b, end in enumerate(kl):
        t = torch.arange(end, device=DEV)
        rows = _rows_of(st, b, t)
        count = min(end, m)
        slots = torch.arange(count, device=DEV)
        to = st["new_table"][b].long()[torch.div(slots, ps, rounding_mode="floor")] * ps + slots % ps
        for h in range(hkv):
            w = st["weights"][rows // ps, h, rows % ps].double()
            if end > m:
                must = (t < case["sinks"]) | (t >= end - case["recent"])
                others = t[~must]
                # the most weight first, of equal ones the earliest: a stable sort of the reversed order's mirror
                order = torch.argsort(-w[~must], stable=True)[:m - int(must.sum())]
                keep = torch.cat([t[must], others[order]]).sort().values
            else:
                keep = t
            src = rows[keep]
            for pool, scale in ((st["k"], k_scale), (st["v"], v_scale)):
                s = scale[src // bs, h]
                new = torch.stack([x.max() for x in s.split(bs)]).repeat_interleave(bs)[:count]
                r = (s.double() / new.double()).float().double()
                flat = pool.view(-1, hkv, d)
                flat[to, h] = torch.round(flat[src, h].double() * r[:, None]).to(torch.int8)
                scale[to // bs, h] = new
            st["weights"][to // ps, h, to % ps] = w[keep].float()
            st["kept"][b, h, :count] = keep.to(torch.int32)
        st["new_lens"][b] = count


_EXACT = {"append": _exact_append, "attn": _exact_attn, "weights": _exact_weights, "evict": _exact_evict}
