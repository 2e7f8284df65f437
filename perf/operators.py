"""What the attention-input and chunk-attention operators are measured on.

Four operators of a serving program that keeps its keys and values in an INT8 cache:

  norm_rope               per-head RMS norm and position rotation of q and k in one pass
  rope_append_gqa_paged   the same on the way into the paged INT8 cache; q becomes codes, v is quantized
  prefill_attn_gqa_paged  attention of a chunk of new tokens (one to thousands) over the paged cache
  cross_attn_gqa          attention to an encoder's INT8 states of another length

New tokens are packed: rows q_start[b] .. q_start[b + 1] - 1 of q, k, v and out belong to sequence b.
"""
import itertools
import math
import random

import torch

own = False

DEV = "cuda"
D = 128                       # head size of every INT8 attention call
EPS = 1e-6
MOST_SCORES = 1 << 31         # B * Hq * S * T of the largest case


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # calibration looks at q and k as attention sees them: a batch laid out (B, H, S, D)
        dict(name="norm_rope_calib", op="norm_rope", B=4, S=2048, Hq=64, Hkv=8, D=128, rot=128, norm=True,
             interleaved=False, transposed=True, f32=False),
        # the same for one new token of 16 sequences: latency
        dict(name="norm_rope_decode", op="norm_rope", B=16, S=1, Hq=64, Hkv=8, D=128, rot=128, norm=True,
             interleaved=False, transposed=False, f32=False),
        # neighbouring pairs, a part of the head rotated, no norm, float32 out, odd row count and head size
        dict(name="norm_rope_odd", op="norm_rope", B=3, S=333, Hq=20, Hkv=5, D=80, rot=32, norm=False,
             interleaved=True, transposed=False, f32=True),
        # a decode step's input: 16 sequences, one new token each, pages of 64
        dict(name="append_decode", op="append", B=16, S=1, T=4096, ragged=False, Hq=64, Hkv=8, rot=128, norm=True,
             interleaved=False, page=64, mix=1),
        # a mixed step of a server that prefills in chunks: one sequence with 2048 new tokens, 15 with one
        dict(name="append_mixed", op="append", B=16, S=2048, T=4096, ragged=True, Hq=64, Hkv=8, rot=128, norm=True,
             interleaved=False, page=64, mix=2),
        # a large prompt batch without norms, odd pages and head counts, ragged lengths
        dict(name="append_odd", op="append", B=7, S=1111, T=1600, ragged=True, Hq=20, Hkv=5, rot=64, norm=False,
             interleaved=True, page=24, mix=3),
        # single tokens among the chunk calls: 16 sequences, one row each, 4096 tokens of context
        dict(name="chunk_decode", op="chunk", B=16, S=1, T=4096, ragged=False, Hq=64, Hkv=8, page=64, mix=1),
        # a chunked-prefill step: one sequence with 512 new rows beside seven with one
        dict(name="chunk_mixed", op="chunk", B=8, S=512, T=4096, ragged=True, Hq=64, Hkv=8, page=64, mix=2),
        # a long chunk with as long a cached prefix
        dict(name="chunk_long", op="chunk", B=1, S=4096, T=8192, ragged=False, Hq=64, Hkv=8, page=128, mix=1),
        # a few drafted tokens to verify over a long context, odd group size, pages that end inside a key tile
        dict(name="chunk_draft", op="chunk", B=3, S=5, T=20001, ragged=True, Hq=35, Hkv=7, page=48, mix=4),
        # one decoder token of 16 sequences over an encoder's states
        dict(name="cross_decode", op="cross", B=16, S=1, T=1500, ragged=True, Hq=16, Hkv=16, mix=5),
        # a decoder's prompt over an encoder's states, ragged on both sides
        dict(name="cross_prompt", op="cross", B=8, S=448, T=2048, ragged=True, Hq=32, Hkv=8, mix=6),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "append", "chunk", "chunk", "cross"])
    hkv, g = rng.choice([1, 2, 3, 4, 5, 8]), rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 12, 16])
    if op == "norm_rope":
        d = rng.choice([64, 80, 96, 128, 192, 256])
        n = _log(rng, 1, max(1, min(8192, (8192 * 72 * 128) // ((g + 1) * hkv * d))))
        b = rng.choice([x for x in (1, 2, 3, 4, 5, 16) if x <= n])
        return dict(op=op, B=b, S=max(1, n // b), Hq=g * hkv, Hkv=hkv, D=d, rot=rng.choice([d, d // 2, 32]),
                    norm=rng.random() < 0.6, interleaved=rng.random() < 0.4, transposed=rng.random() < 0.5,
                    f32=rng.random() < 0.3)
    b, t = _log(rng, 1, 32), _log(rng, 1, 20001 if op == "chunk" else 4096)
    s = _log(rng, 1, min(t, 4096)) if op != "cross" else _log(rng, 1, 2048)
    if op == "append":
        while b * s * (g + 2) * hkv > 2048 * 80:
            s = max(1, s // 2)
            b = max(1, b // 2) if s == 1 else b
        return dict(op=op, B=b, S=s, T=t, ragged=rng.random() < 0.6, Hq=g * hkv, Hkv=hkv,
                    rot=rng.choice([128, 64, 32]), norm=rng.random() < 0.5, interleaved=rng.random() < 0.4,
                    page=rng.choice([1, 7, 16, 24, 64, 100, 128]), mix=rng.randrange(1, 1 << 20))
    while b * s * t * g * hkv > MOST_SCORES // 4:
        if b > 1:
            b //= 2
        elif s > 64:
            s //= 2
        else:
            t //= 2
    case = dict(op=op, B=b, S=min(s, t) if op == "chunk" else s, T=t, ragged=rng.random() < 0.6, Hq=g * hkv, Hkv=hkv,
                mix=rng.randrange(1, 1 << 20))
    if op == "chunk":
        case["page"] = rng.choice([1, 16, 24, 48, 64, 100, 128, 256])
    return case


def _lens(case):
    """New rows and context length of each sequence (a function of the case alone). Ragged: the first sequence
    has the most rows; the others one row or some, and a cross-attended state may be empty."""
    b, s, t = case["B"], case["S"], case["T"]
    if not case["ragged"]:
        return [s] * b, [t] * b
    r = random.Random(case["mix"])
    cross = case["op"] == "cross"
    ql = [s] + [1 if r.random() < 0.5 else r.randint(0, max(1, s // 8)) for _ in range(b - 1)]
    kl = [t] + [r.randint(0 if cross else max(q, 1), t) for q in ql[1:]]
    if cross and b > 2:
        kl[-1] = 0
    return ql, kl


# --------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _table(n, rot):
    """cos and sin of position p times 10000^(-2i / rot), in 64 bits, rounded to float32: [n][rot], cos first."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
    a = torch.arange(n, dtype=torch.float64, device=DEV)[:, None] * inv[None, :]
    return torch.cat([a.cos(), a.sin()], 1).float().contiguous()


def _sigma(g, n):
    return torch.exp(torch.rand(n, generator=g, device=DEV) * math.log(4.0) + math.log(0.5))


def _codes(g, shape):
    return (torch.randn(shape, generator=g, device=DEV) * (127 / 4.5)).round().clamp(-127, 127).to(torch.int8)


def _paging(case, kl, g):
    """A pool with a few spare pages and the pages of each sequence in a shuffled order."""
    ps = case["page"]
    b, most = case["B"], max(1, -(-case["T"] // ps))
    num = b * most + 3
    perm = torch.randperm(num, generator=g, device=DEV).to(torch.int32)
    return num, perm[:b * most].reshape(b, most).contiguous()


def _start(ql):
    return [0] + list(itertools.accumulate(ql))


def prepare(case, seed):
    g = _gen(seed)
    hq, hkv = case["Hq"], case["Hkv"]
    st = {"op": case["op"], "case": case}
    if case["op"] == "norm_rope":
        b, s, d = case["B"], case["S"], case["D"]
        qkv = torch.randn(b, s, hq + 2 * hkv, d, generator=g, device=DEV)
        qkv *= torch.cat([_sigma(g, hq), _sigma(g, 2 * hkv)])[None, None, :, None]
        st["qkv"] = qkv.bfloat16()                                 # q, k and v of one projection, side by side
        st["cos_sin"] = _table(8192 + s, case["rot"])
        st["pos"] = (torch.randint(0, 8192, (b, 1), generator=g, device=DEV)
                     + torch.arange(s, device=DEV)).to(torch.int32)
        st["wq"] = (1 + 0.2 * torch.randn(d, generator=g, device=DEV)).bfloat16() if case["norm"] else None
        st["wk"] = (1 + 0.2 * torch.randn(d, generator=g, device=DEV)).bfloat16() if case["norm"] else None
        t = torch.float32 if case["f32"] else torch.bfloat16
        if case["transposed"]:
            st["q_out"] = torch.empty(b, hq, s, d, dtype=t, device=DEV).transpose(1, 2)
            st["k_out"] = torch.empty(b, hkv, s, d, dtype=t, device=DEV).transpose(1, 2)
        else:
            st["q_out"] = torch.empty(b, s, hq, d, dtype=t, device=DEV)
            st["k_out"] = torch.empty(b, s, hkv, d, dtype=t, device=DEV)
        return st
    ql, kl = _lens(case)
    start = _start(ql)
    n = max(1, start[-1]) + 2                                      # two rows behind the last sequence
    st["q_start"] = torch.tensor(start, dtype=torch.int32, device=DEV)
    st["kv_lens"] = torch.tensor(kl, dtype=torch.int32, device=DEV)
    st["n"] = n
    # the program's own list of rows: which sequence, which of its new rows
    st["row_b"] = torch.tensor([b for b, q in enumerate(ql) for _ in range(q)], dtype=torch.int64, device=DEV)
    st["row_i"] = torch.tensor([i for q in ql for i in range(q)], dtype=torch.int64, device=DEV)
    sq, sk, sv = _sigma(g, hq), _sigma(g, hkv), _sigma(g, hkv)
    st["q_scale"], st["k_scale"], st["v_scale"] = sq * (4.5 / 127), sk * (4.5 / 127), sv * (4.5 / 127)
    if case["op"] != "cross":
        num, st["table"] = _paging(case, kl, g)
        st["k"] = _codes(g, (num, case["page"], hkv, D))
        st["v"] = _codes(g, (num, case["page"], hkv, D))
    if case["op"] == "append":
        if case["norm"]:                                            # the norm leaves every head near 1
            st["q_scale"], st["k_scale"] = (torch.full_like(x, 4.5 / 127) for x in (sq, sk))
        qkv = torch.randn(n, hq + 2 * hkv, D, generator=g, device=DEV)
        st["qkv"] = (qkv * torch.cat([sq, sk, sv])[None, :, None]).bfloat16()
        st["cos_sin"] = _table(case["T"], case["rot"])
        st["wq"] = (1 + 0.2 * torch.randn(D, generator=g, device=DEV)).bfloat16() if case["norm"] else None
        st["wk"] = (1 + 0.2 * torch.randn(D, generator=g, device=DEV)).bfloat16() if case["norm"] else None
        st["q8"] = torch.zeros(n, hq, D, dtype=torch.int8, device=DEV)
        return st
    st["q"] = _codes(g, (n, hq, D))
    st["out"] = torch.full((n, hq, D), 0.5, dtype=torch.bfloat16, device=DEV)
    st["sm"] = 1.0 / math.sqrt(D)
    st["S"], st["T"] = max(max(ql), 1), max(max(kl), 1)
    if case["op"] == "cross":
        st["k"] = _codes(g, (case["B"], case["T"], hkv, D))
        st["v"] = _codes(g, (case["B"], case["T"], hkv, D))
    return st


# --------------------------------------------------------------------------- one pass
def run(st):
    if own:
        from int8_head_kv_gb300 import fa3
        c = st["case"]
        if st["op"] == "norm_rope":
            hq, hkv = c["Hq"], c["Hkv"]
            q, k = fa3.norm_rope(st["qkv"][:, :, :hq], st["qkv"][:, :, hq:hq + hkv], st["cos_sin"], st["pos"],
                                 q_weight=st["wq"], k_weight=st["wk"], eps=EPS, interleaved=c["interleaved"],
                                 q_out=st["q_out"], k_out=st["k_out"])
            return {"q": q, "k": k}
        if st["op"] == "append":
            hq, hkv = c["Hq"], c["Hkv"]
            x = st["qkv"]
            fa3.rope_append_gqa_paged(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], st["cos_sin"], st["q_scale"],
                                      st["k_scale"], st["v_scale"], st["k"], st["v"], st["table"], st["q_start"],
                                      st["kv_lens"], q_weight=st["wq"], k_weight=st["wk"], eps=EPS,
                                      interleaved=c["interleaved"], q_out=st["q8"])
            return {"q": st["q8"], "k": st["k"], "v": st["v"]}
        if st["op"] == "chunk":
            return fa3.prefill_attn_gqa_paged(st["q"], st["k"], st["v"], st["q_scale"], st["k_scale"], st["v_scale"],
                                              st["q_start"], st["kv_lens"], st["table"], st["sm"], out=st["out"])
        return fa3.cross_attn_gqa(st["q"], st["k"], st["v"], st["q_scale"], st["k_scale"], st["v_scale"],
                                  st["q_start"], st["kv_lens"], st["sm"], out=st["out"])
    if st["op"] == "norm_rope":
        return _plain_norm_rope(st)
    return _plain_append(st) if st["op"] == "append" else _plain_attention(st)


def _norm(x, w):
    if w is None:
        return x
    return x * (1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)) * w.to(x.dtype)


def _rotate(x, cs, interleaved):
    """x [..., H, D], cs [..., rot] of the row's position."""
    rot = cs.shape[-1]
    c, s = cs[..., None, :rot // 2].to(x.dtype), cs[..., None, rot // 2:].to(x.dtype)
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * c - b * s, b * c + a * s
    return y


def _plain_norm_rope(st):
    c, x = st["case"], st["qkv"]
    hq, hkv = c["Hq"], c["Hkv"]
    cs = st["cos_sin"][st["pos"].long()]
    st["q_out"].copy_(_rotate(_norm(x[:, :, :hq].float(), st["wq"]), cs, c["interleaved"]))
    st["k_out"].copy_(_rotate(_norm(x[:, :, hq:hq + hkv].float(), st["wk"]), cs, c["interleaved"]))
    return {"q": st["q_out"], "k": st["k_out"]}


def _plain_append(st):
    # The codes are whole numbers and decide at half steps: the rotated values are taken in 64 bits, so that no
    # code depends on how 32 bits round. v's quotient is the float32 one of the quantizer.
    c = st["case"]
    hq, hkv, used = c["Hq"], c["Hkv"], st["row_b"].numel()
    x, b = st["qkv"][:used], st["row_b"]
    pos = (st["kv_lens"] - (st["q_start"][1:] - st["q_start"][:-1])).long()[b] + st["row_i"]
    cs = st["cos_sin"][pos]
    q = _rotate(_norm(x[:, :hq].double(), st["wq"]), cs, c["interleaved"]) / st["q_scale"].double()[:, None]
    k = _rotate(_norm(x[:, hq:hq + hkv].double(), st["wk"]), cs, c["interleaved"]) / st["k_scale"].double()[:, None]
    v = x[:, hq + hkv:].float() / st["v_scale"][:, None]
    page, at = st["table"][b, pos // c["page"]].long(), pos % c["page"]
    st["q8"][:used] = q.round().clamp(-127, 127).to(torch.int8)
    st["k"][page, at] = k.round().clamp(-127, 127).to(torch.int8)
    st["v"][page, at] = v.round().clamp(-127, 127).to(torch.int8)
    return {"q": st["q8"], "k": st["k"], "v": st["v"]}


def _plain_attention(st):
    c = st["case"]
    b, s, t, hkv, g = c["B"], st["S"], st["T"], c["Hkv"], c["Hq"] // c["Hkv"]
    at = torch.arange(t, device=DEV)
    if st["op"] == "chunk":
        page = st["table"][:, at // c["page"]].long()
        k, v = st["k"][page, at % c["page"]], st["v"][page, at % c["page"]]
    else:
        k, v = st["k"][:, :t], st["v"][:, :t]
    k = (k.float() * st["k_scale"][:, None]).permute(0, 2, 3, 1)                        # [B, Hkv, D, T]
    v = (v.float() * st["v_scale"][:, None]).transpose(1, 2)                            # [B, Hkv, T, D]
    ql, kl = st["q_start"][1:] - st["q_start"][:-1], st["kv_lens"]
    i = torch.arange(s, device=DEV)
    rows = (st["q_start"][:-1, None] + i).clamp(max=st["n"] - 1).long()
    q = (st["q"][rows].float() * st["q_scale"][:, None]).reshape(b, s, hkv, g, D).permute(0, 2, 3, 1, 4)
    x = torch.matmul(q.reshape(b, hkv, g * s, D), k).reshape(b, hkv, g, s, t) * st["sm"]
    last = (kl - ql)[:, None] + i if st["op"] == "chunk" else kl[:, None] - 1 + 0 * i   # last key of each row
    x.masked_fill_(at > last[:, None, None, :, None], float("-inf"))
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x.sub_(torch.where(top.isinf(), torch.zeros_like(top), top)))
    z = p.sum(-1, keepdim=True)
    o = torch.matmul(p.reshape(b, hkv, g * s, t), v).reshape(b, hkv, g, s, D)
    o = torch.where(z > 0, o / z, torch.zeros_like(o)).permute(0, 3, 1, 2, 4).reshape(b, s, hkv * g, D)
    st["out"][:st["row_b"].numel()] = o[st["row_b"], st["row_i"]].bfloat16()
    return st["out"]


# --------------------------------------------------------------------------- the floor
def work(case):
    hq, hkv = case["Hq"], case["Hkv"]
    if case["op"] == "norm_rope":
        n, d = case["B"] * case["S"], case["D"]
        values = n * (hq + hkv) * d
        return {"bytes": values * (2 + (4 if case["f32"] else 2)) + n * (4 + 4 * case["rot"]), "flops": values * 8}
    ql, kl = _lens(case)
    n = sum(ql)
    if case["op"] == "append":
        values = n * (hq + 2 * hkv) * D
        return {"bytes": values * 3 + n * (8 + 4 * case["rot"]), "flops": values * 10}
    live = [k if q else 0 for q, k in zip(ql, kl)]
    size = n * hq * D * 3 + sum(live) * hkv * D * 2
    if case["op"] == "chunk":
        size += 4 * sum(-(-k // case["page"]) for k in live)
        pairs = sum(q * (k - q) + q * (q + 1) // 2 for q, k in zip(ql, kl))
    else:
        pairs = sum(q * k for q, k in zip(ql, kl))
    return {"bytes": size, "flops": 4 * D * hq * pairs}


# --------------------------------------------------------------------------- the definition in 64 bits
def _turn(x, weight, cs, interleaved):
    """Rows x [H][D] of one token in float64, as complex numbers turned by the table's angle."""
    x = x.double()
    if weight is not None:
        x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS) * weight.double()
    rot = cs.shape[-1]
    turn = torch.complex(cs[..., :rot // 2].double(), cs[..., rot // 2:].double()).unsqueeze(-2)
    head, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        z = torch.complex(head[..., ::2].contiguous(), head[..., 1::2].contiguous()) * turn
        head = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(head[..., :rot // 2].contiguous(), head[..., rot // 2:].contiguous()) * turn
        head = torch.cat([z.real, z.imag], -1)
    return torch.cat([head, rest], -1)


def exact(case, seed):
    st = prepare(case, seed)
    hq, hkv = case["Hq"], case["Hkv"]
    g = hq // hkv
    if case["op"] == "norm_rope":
        cs = st["cos_sin"][st["pos"].long()]
        return {"q": _turn(st["qkv"][:, :, :hq], st["wq"], cs, case["interleaved"]),
                "k": _turn(st["qkv"][:, :, hq:hq + hkv], st["wk"], cs, case["interleaved"])}
    ql, kl = _lens(case)
    start = _start(ql)
    if case["op"] == "append":
        # the codes are whole numbers: what they are in 64 bits
        for b, (n, end) in enumerate(zip(ql, kl)):
            if not n:
                continue
            x, pos = st["qkv"][start[b]:start[b + 1]], torch.arange(end - n, end, device=DEV)
            cs = st["cos_sin"][pos]
            rows = st["table"][b].long()[torch.div(pos, case["page"], rounding_mode="floor")] * case["page"] + pos % case["page"]
            code = lambda y, sc: torch.clamp(torch.round(y / sc.double()[None, :, None]), -127, 127).to(torch.int8)  # noqa: E731
            st["q8"][start[b]:start[b + 1]] = code(_turn(x[:, :hq], st["wq"], cs, case["interleaved"]), st["q_scale"])
            st["k"].view(-1, hkv, D)[rows] = code(_turn(x[:, hq:hq + hkv], st["wk"], cs, case["interleaved"]), st["k_scale"])
            st["v"].view(-1, hkv, D)[rows] = torch.clamp(torch.round(x[:, hq + hkv:].float() / st["v_scale"][:, None]),
                                                         -127, 127).to(torch.int8)
        return {"q": st["q8"], "k": st["k"], "v": st["v"]}
    out = st["out"].double()
    for b, (n, end) in enumerate(zip(ql, kl)):
        if not n:
            continue
        if not end:
            out[start[b]:start[b + 1]] = 0
            continue
        if case["op"] == "chunk":
            t = torch.arange(end, device=DEV)
            rows = st["table"][b].long()[torch.div(t, case["page"], rounding_mode="floor")] * case["page"] + t % case["page"]
            kb, vb = st["k"].view(-1, hkv, D)[rows], st["v"].view(-1, hkv, D)[rows]
        else:
            kb, vb = st["k"][b, :end], st["v"][b, :end]
        for h in range(hq):
            qh = st["q"][start[b]:start[b + 1], h].double()
            logit = qh @ kb[:, h // g].double().T
            logit *= st["q_scale"][h].double() * st["k_scale"][h // g].double() * st["sm"]
            if case["op"] == "chunk":
                logit += torch.full_like(logit, float("-inf")).triu(end - n + 1)
            p = torch.softmax(logit, -1)
            out[start[b]:start[b + 1], h] = p @ vb[:, h // g].double() * st["v_scale"][h // g].double()
    return out
