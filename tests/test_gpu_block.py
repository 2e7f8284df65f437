"""GPU parity of the block-scaled paged cache (append, attention, attention weights, eviction) against the float64
oracle.

Tolerances.  Codes, scales and positions are equal bit for bit.  A score is a sum of 128 exact products in float32: it is off
by 128 2^-24 of sum |q k| at most, and by a few roundings of itself; with that error d (absolute, of a natural
exponent), attention is off by 2 d of the weighted mean of |v|, by 2^-11 of it for the weights' fp16 rounding, by
T 2^-32 of the largest |v| for weights in fp16's subnormals, and by half a bf16 step of the result, 2^-8 of it.  The
log-sum-exp is off by d, by the roundings of T / 16 additions, and by its own.  A token's weight is off by d, 2^-22
for the exponential and |s| + |lse| in 2^-22 in each term, and by 68 2^-24 of the sum for 64 additions a step and a
compensated sum of steps.
"""
import numpy as np
import pytest
import torch

import workloads as W
from helpers import fa3
from oracle import fa3_oracle as O

pytestmark = pytest.mark.gpu
SM = 128 ** -0.5
U = 2.0 ** -24


def _t(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _bf(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(torch.bfloat16)


def _f(t):
    return t.detach().float().cpu().numpy()


def _same(got, ref):
    """Equal values (NaN is NaN's equal), array by array."""
    assert len(got) == len(ref)
    ok = True
    for i, (g, r) in enumerate(zip(got, ref)):
        g = g.cpu().numpy() if isinstance(g, torch.Tensor) else g
        if not np.array_equal(g, r, equal_nan=r.dtype.kind == "f"):
            at = np.argwhere((g != r) & ~((g != g) & (r != r)))
            print(f"array {i}: {len(at)} of {g.size} differ, first at {at[:3].tolist()}: {g[tuple(at[0])]} not {r[tuple(at[0])]}")
            ok = False
    return ok


def _cache(rng, kv_lens, page, block, Hkv, D=128, spare=3, extra=0, wide=2.0):
    """Pools whose dead scales are NaN and whose dead table entries lie outside the pool."""
    B, mp = len(kv_lens), -(-max(max(kv_lens), 1) // page) + 1
    num = B * (mp + extra) + spare
    perm = rng.permutation(num)
    table = perm[:B * mp].reshape(B, mp).astype(np.int32)
    c = dict(page=page, block=block, Hkv=Hkv, D=D, num=num, rest=perm[B * mp:].astype(np.int32),
             kv_lens=np.asarray(kv_lens, np.int32))
    code = lambda: np.clip(np.rint(rng.standard_t(5, (num, page, Hkv, D)) * 30), -127, 127).astype(np.int8)  # noqa: E731
    scale = lambda: (W.log_uniform(rng, 1 / wide, wide, (num, page // block, Hkv)) / 40).astype(np.float32)  # noqa: E731
    c["k"], c["v"], c["ks"], c["vs"] = code(), code(), scale(), scale()
    live = np.zeros((num, page // block), bool)
    for b, kv in enumerate(kv_lens):
        for t in range(0, kv, block):
            live[table[b, t // page], t % page // block] = True
        table[b, -(-kv // page):] = num + 5
    c["ks"][~live], c["vs"][~live] = np.nan, np.nan
    c["table"] = table
    return c


def _rows(rng, c, q_lens, Hq, lead=0, behind=2, size=1.0):
    c["q_start"] = (lead + np.concatenate([[0], np.cumsum(q_lens)])).astype(np.int32)
    n = int(c["q_start"][-1]) + behind
    q = rng.standard_normal((n, Hq, c["D"])) * W.log_uniform(rng, 0.5, 2, (Hq,))[None, :, None] * size
    used = np.zeros(n, bool)
    used[c["q_start"][0]:c["q_start"][-1]] = True
    q[~used] = np.nan                                              # nobody's rows
    c["q"], c["used"] = _f(_bf(q)), used
    return c


def _attend(F, c, err=None, sm=SM, lse=True, strided=False, **kw):
    q = _bf(c["q"]).cuda()
    if strided:
        big = torch.full((q.shape[0], q.shape[1] + 3, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
        big[:, 1:-2] = q
        q = big[:, 1:-2]
    out = torch.full(c["q"].shape, 3.0, dtype=torch.bfloat16, device="cuda")
    l = torch.full(c["q"].shape[:2], 3.0, device="cuda") if lse else None  # noqa: E741
    a = [_t(c[x]) for x in ("k", "v", "ks", "vs", "q_start", "kv_lens", "table")]
    torch.cuda.synchronize()
    F.attn_gqa_block_paged(q, *a, sm, out=out, lse=l, dev_err=err, **kw)
    torch.cuda.synchronize()
    return _f(out), None if l is None else _f(l)


def _score_error(c, sm=SM):
    """Of each row and head [n][Hq]: the bound d of the module's comment."""
    d = np.zeros(c["q"].shape[:2])
    a = dict(c, q=np.abs(np.nan_to_num(c["q"])), k=np.abs(c["k"]))
    for b, rows, h, s in O.block_scores(a["q"], a["k"], c["ks"], c["table"], c["q_start"], c["kv_lens"], sm):
        d[rows, h] = np.where(np.isfinite(s), s, 0).max(1) * 136 * U
    return d


def _check_attention(c, out, lse, sm=SM, keep=3.0, rows=None):
    ref, rl = O.attention_block(np.nan_to_num(c["q"]), c["k"], c["v"], c["ks"], c["vs"], c["table"], c["q_start"], c["kv_lens"],
                                sm, np.full(c["q"].shape, keep), np.full(c["q"].shape[:2], keep))
    mean, _ = O.attention_block(np.nan_to_num(c["q"]), c["k"], np.abs(c["v"]), c["ks"], c["vs"], c["table"], c["q_start"],
                                c["kv_lens"], sm, np.full(c["q"].shape, keep), np.full(c["q"].shape[:2], keep))
    d, used = _score_error(c, sm), c["used"] if rows is None else rows
    T = int(c["kv_lens"].max())
    most = 127 * float(np.nanmax(c["vs"]))
    tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -11 + 2 * d[..., None] + 2 * (np.abs(rl) * 2 * U)[..., None]) * mean + T * 2.0 ** -32 * most
    bad = np.abs(out - ref) > tol
    assert np.all(np.isfinite(out[used])) and not bad[used].any(), (np.argwhere(bad & used[:, None, None])[:4],
                                                                    np.abs(out - ref)[bad][:4], tol[bad][:4])
    assert np.all(out[~used] == keep) or rows is not None
    if lse is not None:
        tl = d + (T / 16 + 64) * U + np.abs(rl) * 8 * U
        assert not (np.abs(lse - rl) > tl)[used].any(), (np.abs(lse - rl) / tl)[used].max()
        assert np.all(lse[~used] == keep) or rows is not None
    return ref, rl


# ---------------------------------------------------------------------- append
APPEND = [                        # q_lens, kv_lens, page, block, Hkv, D
    ([1], [1], 16, 16, 1, 128),
    ([1, 1, 1], [17, 64, 130], 64, 64, 8, 128),
    ([3, 0, 40], [19, 7, 41], 48, 16, 3, 80),
    ([100, 5, 1], [300, 5, 77], 96, 32, 2, 64),
    ([257], [260], 128, 128, 2, 256),
    ([1] * 40, list(range(1, 41)), 32, 16, 2, 8),
    ([200, 300], [513, 300], 256, 256, 1, 192),
]


def _kv(rng, n, Hkv, D, size=1.0):
    x = _f(_bf(rng.standard_t(4, (n, 2 * Hkv, D)) * size * W.log_uniform(rng, 0.1, 3, (2 * Hkv,))[None, :, None]))
    return x[:, :Hkv], x[:, Hkv:], x


@pytest.mark.parametrize("q_lens,kv_lens,page,block,Hkv,D", APPEND)
@pytest.mark.parametrize("wide", [True, False])
def test_append_codes_and_scales_are_exact(q_lens, kv_lens, page, block, Hkv, D, wide):
    F, rng = fa3(), np.random.default_rng(len(q_lens) + D)
    c = _cache(rng, kv_lens, page, block, Hkv, D)
    q_start = np.concatenate([[1], 1 + np.cumsum(q_lens)]).astype(np.int32)
    n = int(q_start[-1]) + 2
    k, v, x = _kv(rng, n, Hkv, D, 0.5)
    ref = O.append_block_paged(k, v, c["k"], c["v"], c["ks"], c["vs"], c["table"], q_start, kv_lens)
    if wide:
        t = _bf(x).cuda()
    else:                                                          # rows that are 8-byte aligned only
        flat = torch.zeros(n * (2 * Hkv * D + 4) + 4, dtype=torch.bfloat16, device="cuda")
        t = flat[4:].as_strided((n, 2 * Hkv, D), (2 * Hkv * D + 4, D, 1))
        t.copy_(_bf(x))
    got = [_t(c[y]) for y in ("k", "v", "ks", "vs")]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    F.append_gqa_block_paged(t[:, :Hkv], t[:, Hkv:], *got, _t(c["table"]), _t(q_start), _t(c["kv_lens"]), dev_err=err)
    assert _same(got, ref)
    assert err.item() == 0


def test_append_token_by_token_and_values_at_half_steps():
    F, rng = fa3(), np.random.default_rng(5)
    c = _cache(rng, [0, 0], 32, 16, 2, 64, extra=2)
    table = np.arange(6, dtype=np.int32).reshape(2, 3)
    state = [c["k"], c["v"], c["ks"], c["vs"]]
    got, tab, start = [_t(x) for x in state], _t(table), np.array([0, 1, 2], np.int32)
    for t in range(40):
        k, v, _ = _kv(rng, 2, 2, 64, 2.0 ** rng.integers(-3, 4))
        k[0, 0, :40] = np.arange(-20, 20) + 0.5                    # half steps of scales that are whole
        k[0, 0, 40] = 127 * 2.0 ** (t // 10)
        lens = np.array([t + 1, t + 1], np.int32)
        state = O.append_block_paged(k, v, *state, table, start, lens)
        F.append_gqa_block_paged(_bf(k).cuda(), _bf(v).cuda(), *got, tab, _t(start), _t(lens))
    assert _same(got, state)


def test_append_codes_of_every_pair_of_mantissas():
    """Eight-bit mantissas against a block's eight-bit greatest: 127 x / a is a half step for many, and what the rounding
    of the scale makes of it decides."""
    F = fa3()
    c = _cache(np.random.default_rng(8), [5], 16, 16, 128, 256)
    m = np.arange(128, 256) / 128.0
    val = np.concatenate([m * 2.0 ** -e for e in range(10)])          # 1280 values a head, 5 tokens of 256
    x = np.broadcast_to(val, (128, 1280)).copy()
    x[np.broadcast_to(x[:, :128] > m[:, None], (128, 128)).nonzero()] /= 2   # none above the head's greatest
    x[:, ::3] *= -1
    x[np.arange(128), np.arange(128)] = m
    k = x.reshape(128, 5, 256).transpose(1, 0, 2).astype(np.float32)
    assert np.array_equal(_f(_bf(k)), k)
    for up in (1.0, 2.0 ** 20, 2.0 ** -40):
        ref = O.append_block_paged(k * np.float32(up), k[::-1] * np.float32(up), c["k"], c["v"], c["ks"], c["vs"], c["table"], [0, 5], [5])
        got = [_t(c[y]) for y in ("k", "v", "ks", "vs")]
        F.append_gqa_block_paged(_bf(k * up).cuda(), _bf(k[::-1] * up).cuda(), *got, _t(c["table"]), _t(np.array([0, 5], np.int32)),
                                 _t(c["kv_lens"]))
        assert _same(got, ref)


@pytest.mark.parametrize("old", [False, True])
def test_append_zero_tiny_and_not_finite_values(old):
    F, rng = fa3(), np.random.default_rng(6)
    c = _cache(rng, [20], 32, 32, 6, 16)
    if not old:
        c["kv_lens"][:] = 2
    k, v, _ = _kv(rng, 2, 6, 16)
    k[:, 0] = 0
    k[:, 1] = 2.0 ** -133
    k[0, 2, 3], k[1, 2, 5], k[1, 2, 6] = np.inf, -np.inf, np.nan
    k[:, 3] = np.inf
    k[:, 4] = 3e38
    k[0, 5], k[1, 5] = 1e-30, 1e30
    v[:, 2] = np.nan
    k, v = _f(_bf(k)), _f(_bf(v))
    c["ks"][c["table"][0, 0], 0, 0] = 0                             # a block of zeros so far
    ref = O.append_block_paged(k, v, c["k"], c["v"], c["ks"], c["vs"], c["table"], [0, 2], c["kv_lens"])
    got = [_t(c[y]) for y in ("k", "v", "ks", "vs")]
    F.append_gqa_block_paged(_bf(k).cuda(), _bf(v).cuda(), *got, _t(c["table"]), _t(np.array([0, 2], np.int32)), _t(c["kv_lens"]))
    assert _same(got, ref)


def test_append_bad_lengths_pages_and_starts():
    F, rng = fa3(), np.random.default_rng(7)
    c = _cache(rng, [40, 40, 40], 32, 16, 2, 64)
    k, v, _ = _kv(rng, 6, 2, 64)

    def run(table, start, lens):
        got = [_t(c[y]) for y in ("k", "v", "ks", "vs")]
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        F.append_gqa_block_paged(_bf(k).cuda(), _bf(v).cuda(), *got, _t(table), _t(np.asarray(start, np.int32)),
                                 _t(np.asarray(lens, np.int32)), dev_err=err)
        return [g.cpu().numpy() for g in got], err.item()
    before = [c[y] for y in ("k", "v", "ks", "vs")]
    table = c["table"].copy()
    table[1, 1] = -1
    got, e = run(table, [0, 2, 4, 6], [40, 40, 40])
    good = [table[[0, 2]], [0, 2, 4], [40, 40]]
    ref = O.append_block_paged(k[[0, 1, 4, 5]], v[[0, 1, 4, 5]], *before, *good)
    assert e == F.FA3_DEVERR_PAGE and _same(got, ref)
    for lens in ([40, 1, 40], [40, -3, 40], [40, 97, 40]):
        got, e = run(c["table"], [0, 2, 4, 6], lens)
        assert e == F.FA3_DEVERR_LENS and _same(got, O.append_block_paged(k[[0, 1, 4, 5]], v[[0, 1, 4, 5]], *before,
                                                                          c["table"][[0, 2]], [0, 2, 4], [40, 40]))
    got, e = run(c["table"], [0, 4, 2, 6], [40, 40, 40])
    assert e == F.FA3_DEVERR_LENS and _same(got, before)
    for start, rows, seqs in (([-1, 2, 4, 6], [2, 3, 4, 5], [1, 2]), ([0, 2, 4, 7], [0, 1, 2, 3], [0, 1])):
        got, e = run(c["table"], start, [40, 40, 40])
        assert e == F.FA3_DEVERR_LENS and _same(got, O.append_block_paged(k[rows], v[rows], *before, c["table"][seqs],
                                                                          [0, 2, 4], [40, 40]))


# ------------------------------------------------------------------- attention
ATTN = [                          # Hq, Hkv, page, block, q_lens, kv_lens
    (8, 1, 64, 64, [1], [1]),
    (8, 1, 16, 16, [1], [130]),
    (64, 8, 64, 64, [1, 1, 1], [300, 1, 129]),
    (5, 5, 48, 16, [1, 1], [500, 77]),
    (35, 7, 48, 48, [5, 1, 2], [700, 33, 2]),
    (16, 1, 32, 32, [1, 3, 0, 17], [400, 3, 9, 60]),
    (12, 4, 80, 16, [40, 1], [40, 900]),
    (8, 2, 64, 32, [200, 1, 33], [513, 257, 33]),
    (128, 1, 128, 128, [3], [200]),
    (6, 2, 256, 256, [300], [300]),
    (8, 8, 144, 48, [7, 130], [1000, 131]),
    (24, 2, 64, 16, [1] * 9, [1, 15, 16, 17, 127, 128, 129, 255, 640]),
]


@pytest.mark.parametrize("Hq,Hkv,page,block,q_lens,kv_lens", ATTN)
def test_attention(Hq, Hkv, page, block, q_lens, kv_lens):
    F, rng = fa3(), np.random.default_rng(Hq * 100 + sum(q_lens))
    c = _rows(rng, _cache(rng, kv_lens, page, block, Hkv), q_lens, Hq, lead=1)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = _attend(F, c, err)
    _check_attention(c, out, lse)
    assert err.item() == 0
    out2, none = _attend(F, c, lse=False, strided=True)
    assert none is None and np.array_equal(out, out2)


@pytest.mark.parametrize("page,block,wide", [(128, 128, 2.0), (384, 128, 2.0 ** 20), (256, 256, 2.0 ** 20), (4096, 4096, 2.0)])
def test_attention_of_blocks_that_hold_whole_key_tiles(page, block, wide):
    F, rng = fa3(), np.random.default_rng(12)
    for Hq, Hkv, q_lens, kv_lens in ((8, 2, [200, 1, 130], [700, 129, 130]), (4, 4, [300], [1100])):
        c = _rows(rng, _cache(rng, kv_lens, page, block, Hkv), q_lens, Hq, lead=1)
        c["vs"] *= np.exp2(rng.uniform(-np.log2(wide), 0, c["vs"].shape)).astype(np.float32)
        out, lse = _attend(F, c)
        _check_attention(c, out, lse)
        out2, _ = _attend(F, c, lse=False, strided=True)
        assert np.array_equal(out, out2)


def test_attention_of_one_query_expanded_over_rows():
    F, rng = fa3(), np.random.default_rng(10)
    for q_lens in ([1, 1, 1], [60, 30, 40]):
        c = _rows(rng, _cache(rng, [100, 130, 64], 32, 16, 2), q_lens, 4, behind=0)
        c["q"][:] = c["q"][:1]
        out, lse = _attend(F, c)
        a = [_t(c[x]) for x in ("k", "v", "ks", "vs", "q_start", "kv_lens", "table")]
        q = _bf(c["q"][:1]).cuda().expand(len(c["q"]), -1, -1)
        l2 = torch.zeros(c["q"].shape[:2], device="cuda")
        o2 = F.attn_gqa_block_paged(q, *a, SM, lse=l2)
        assert np.array_equal(out, _f(o2)) and np.array_equal(lse, _f(l2))
        if len(c["q"]) > 3:                                         # whole rows of heads may not overlap there
            w = F.attn_weight_pool(a[0])
            with pytest.raises(F.FA3Error):
                F.attn_weights_gqa_block_paged(q, a[0], a[2], l2, w, *a[4:], SM)


@pytest.mark.parametrize("Hq,Hkv,q_lens,kv_lens", [
    (8, 1, [4, 4], [900, 33]), (8, 1, [3, 4, 3], [3, 16, 17]), (16, 1, [2, 2, 2], [2, 700, 15]), (40, 8, [6, 5, 7], [6, 20, 400]),
    (11, 1, [2, 2], [129, 64]), (13, 1, [2, 2, 1, 0, 4], [500, 2, 1, 0, 77]), (2, 2, [32, 30, 20], [1500, 30, 21]),
    (8, 1, [20, 1, 1, 1, 1, 1], [3000, 1, 20, 300, 64, 5])])
def test_attention_units_of_32_columns(Hq, Hkv, q_lens, kv_lens):
    F, rng = fa3(), np.random.default_rng(9)
    c = _rows(rng, _cache(rng, kv_lens, 48, 16, Hkv), q_lens, Hq, lead=1)
    out, lse = _attend(F, c)
    _check_attention(c, out, lse)
    out2, _ = _attend(F, c, lse=False, strided=True)
    assert np.array_equal(out, out2)


def test_attention_long_contexts_split_over_the_gpu():
    F, rng = fa3(), np.random.default_rng(11)
    for q_lens, kv_lens, Hq, Hkv in (([1], [20000], 8, 1), ([70, 1], [9000, 3000], 6, 2)):
        c = _rows(rng, _cache(rng, kv_lens, 64, 32, Hkv), q_lens, Hq)
        out, lse = _attend(F, c)
        _check_attention(c, out, lse)


@pytest.mark.parametrize("q_lens,kv_lens", [([1, 1], [300, 200]), ([150, 90], [300, 200])])
def test_attention_blocks_of_very_different_sizes(q_lens, kv_lens):
    """Blocks of zeros, of tiny and of large values, with the weight on any of them; scores large enough that the
    softmax's reference moves."""
    F, rng = fa3(), np.random.default_rng(12)
    c = _rows(rng, _cache(rng, kv_lens, 64, 16, 2), q_lens, 8, size=2.0)
    live = np.isfinite(c["vs"])
    c["vs"] = np.where(live, 10.0 ** rng.uniform(-8, 4, c["vs"].shape), np.nan).astype(np.float32)
    zero = live & (rng.random(c["vs"].shape) < 0.2)
    c["vs"][zero] = 0
    c["ks"] = (c["ks"] * W.log_uniform(rng, 0.05, 4, c["ks"].shape)).astype(np.float32)
    c["ks"][live & (rng.random(c["ks"].shape) < 0.1)] = 0
    out, lse = _attend(F, c)
    # the largest |v| that has weight counts, not the largest of all: with weights relative to the values' sizes
    # a weight's rounding is relative to its contribution
    _check_attention(c, out, lse)
    ref, _ = O.attention_block(np.nan_to_num(c["q"]), c["k"], c["v"], c["ks"], c["vs"], c["table"], c["q_start"], c["kv_lens"],
                               SM, np.full(c["q"].shape, 3.0), np.full(c["q"].shape[:2], 3.0))
    mean, _ = O.attention_block(np.nan_to_num(c["q"]), c["k"], np.abs(c["v"]), c["ks"], c["vs"], c["table"], c["q_start"],
                                c["kv_lens"], SM, np.full(c["q"].shape, 3.0), np.full(c["q"].shape[:2], 3.0))
    d = _score_error(c)[..., None] + 64 * 2 * U
    top = mean.max(-1, keepdims=True)                               # a row's largest contribution is of this order
    tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -11 + 2 * d) * mean + 320 * 2.0 ** -32 * 128 * top
    assert not (np.abs(out - ref) > tol)[c["used"]].any()


def test_attention_values_all_zero():
    F, rng = fa3(), np.random.default_rng(13)
    c = _rows(rng, _cache(rng, [100, 300], 64, 32, 1), [1, 20], 4)
    c["vs"] = np.where(np.isfinite(c["vs"]), 0, np.nan).astype(np.float32)
    c["v"][:] = 0
    out, lse = _attend(F, c)
    assert np.all(out[c["used"]] == 0)
    _check_attention(c, out, lse)


def test_attention_bad_lengths_pages_and_starts():
    F, rng = fa3(), np.random.default_rng(14)
    c = _rows(rng, _cache(rng, [100, 130, 64], 32, 16, 2), [1, 2, 20], 4, behind=0)
    _check_attention(c, *_attend(F, c))
    for lens, start in (([100, 1, 64], None), ([100, 1000, 64], None), (None, [0, 4, 3, 23]), (None, [0, 1, 3, 24]),
                        (None, [-1, 1, 3, 23])):
        d = dict(c)
        if lens is not None:
            d["kv_lens"] = np.asarray(lens, np.int32)
        if start is not None:
            d["q_start"] = np.asarray(start, np.int32)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = _attend(F, d, err)
        assert err.item() == F.FA3_DEVERR_LENS
        rows = np.zeros(23, bool)
        if lens is not None:
            rows[[0, *range(3, 23)]] = True
        elif start[0] < 0:
            rows[1:] = True
        elif start[-1] > 23:
            rows[:3] = True
        # within the bounds, not the same bits: the work may be cut at other keys
        _check_attention(c, out, lse, rows=rows)
        assert np.all(out[~rows] == 3.0) and np.all(lse[~rows] == 3.0)
    for bad in (-1, 10 ** 6):
        d = dict(c, table=c["table"].copy())
        d["table"][1, 2] = bad
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = _attend(F, d, err)
        assert err.item() == F.FA3_DEVERR_PAGE
        rows = np.ones(23, bool)
        rows[1:3] = False
        _check_attention(c, out, lse, rows=rows)


# --------------------------------------------------------------------- weights
def _weigh(F, c, lse, w, err=None, **kw):
    wt = _t(w)
    a = [_bf(c["q"]).cuda(), _t(c["k"]), _t(c["ks"]), _t(lse.astype(np.float32)), wt, _t(c["q_start"]), _t(c["kv_lens"]),
         _t(c["table"])]
    torch.cuda.synchronize()
    F.attn_weights_gqa_block_paged(*a, SM, dev_err=err, **kw)
    torch.cuda.synchronize()
    return _f(wt)


def _check_weights(c, lse, before, got):
    q = np.nan_to_num(c["q"])
    lse = lse.astype(np.float32)
    ref = O.attention_weights_block(q, c["k"], c["ks"], lse, before, c["table"], c["q_start"], c["kv_lens"], SM)
    added = O.attention_weights_block(q, c["k"], c["ks"], lse, np.zeros_like(before), c["table"], c["q_start"], c["kv_lens"], SM)
    big = max((np.abs(s[np.isfinite(s)]).max() for *_, s in O.block_scores(q, c["k"], c["ks"], c["table"], c["q_start"],
                                                                           c["kv_lens"], SM)), default=0)
    each = _score_error(c).max() + (big + np.abs(lse[c["used"]]).max(initial=0) + 1) * 4 * U
    tol = added * (each + 68 * U) + np.abs(ref) * 2 * U
    bad = np.abs(got - ref) > tol
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], ref[bad][:4], tol[bad][:4])


@pytest.mark.parametrize("Hq,Hkv,page,block,q_lens,kv_lens", ATTN)
def test_weights(Hq, Hkv, page, block, q_lens, kv_lens):
    F, rng = fa3(), np.random.default_rng(Hq * 100 + sum(q_lens) + 1)
    c = _rows(rng, _cache(rng, kv_lens, page, block, Hkv), q_lens, Hq, lead=1)
    _, lse = O.attention_block(np.nan_to_num(c["q"]), c["k"], c["v"], c["ks"], c["vs"], c["table"], c["q_start"], c["kv_lens"],
                               SM, np.zeros(c["q"].shape), np.full(c["q"].shape[:2], np.nan))
    before = (rng.random((c["num"], Hkv, page)) * 0.01).astype(np.float32)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = _weigh(F, c, lse, before, err)
    _check_weights(c, lse, before, got)
    assert err.item() == 0
    assert np.array_equal(got, _weigh(F, c, lse, before))           # the same on every run


@pytest.mark.parametrize("q_lens,kv_lens,Hq,Hkv", [([400, 1, 30], [700, 5000, 31], 8, 1), ([300], [300], 4, 4),
                                                   ([1] * 70, list(range(1, 1400, 20)), 16, 2)])
def test_weights_of_cut_units(q_lens, kv_lens, Hq, Hkv):
    F, rng = fa3(), np.random.default_rng(21)
    c = _rows(rng, _cache(rng, kv_lens, 64, 64, Hkv), q_lens, Hq)
    _, lse = O.attention_block(np.nan_to_num(c["q"]), c["k"], c["v"], c["ks"], c["vs"], c["table"], c["q_start"], c["kv_lens"],
                               SM, np.zeros(c["q"].shape), np.full(c["q"].shape[:2], np.nan))
    before = (rng.random((c["num"], Hkv, 64)) * 0.01).astype(np.float32)
    _check_weights(c, lse, before, _weigh(F, c, lse, before))


def test_weights_bad_lengths_pages_and_starts():
    F, rng = fa3(), np.random.default_rng(22)
    c = _rows(rng, _cache(rng, [100, 130, 64], 32, 16, 2), [1, 2, 20], 4, behind=0)
    lse = np.full((23, 4), 2.0, np.float32)
    before = rng.random((c["num"], 2, 32)).astype(np.float32)
    whole = _weigh(F, c, lse, before)
    of = lambda b: np.unique(c["table"][b][c["table"][b] < c["num"]])  # noqa: E731
    for start, left in (([0, 4, 3, 23], [0, 1, 2]), ([0, 1, 3, 24], [2]), ([-1, 1, 3, 23], [0])):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = _weigh(F, dict(c, q_start=np.asarray(start, np.int32)), lse, before, err)
        ref = whole.copy()
        for b in left:
            ref[of(b)] = before[of(b)]
        assert err.item() == F.FA3_DEVERR_LENS and np.array_equal(got, ref)
    mine = np.unique(c["table"][1][c["table"][1] < c["num"]])
    for lens in ([100, 1, 64], [100, 1000, 64]):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = _weigh(F, dict(c, kv_lens=np.asarray(lens, np.int32)), lse, before, err)
        assert err.item() == F.FA3_DEVERR_LENS
        ref = whole.copy()
        ref[mine] = before[mine]
        assert np.array_equal(got, ref)
    d = dict(c, table=c["table"].copy())
    lost = d["table"][1, 2]
    d["table"][1, 2] = -7
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = _weigh(F, d, lse, before, err)
    whole[lost] = before[lost]
    assert err.item() == F.FA3_DEVERR_PAGE and np.array_equal(got, whole)


def _both(F, c, seed):
    """Attention and, with its log-sum-exps, attention weights."""
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = _attend(F, c, err)
    _check_attention(c, out, lse)
    before = np.random.default_rng(seed).random((c["num"], c["Hkv"], c["page"])).astype(np.float32)
    _check_weights(c, lse, before, _weigh(F, c, lse, before, err))
    assert err.item() == 0


@pytest.mark.parametrize("most,long", [(1, 0), (3, 0), (3, 2), (40, 4)])
def test_many_sequences_some_without_rows(most, long):
    """More sequences than a warp or a block looks at in one go, also without rows and without a context."""
    F, rng = fa3(), np.random.default_rng(61 + most + long)
    B = 141
    q_lens = rng.integers(0, most + 1, B)
    q_lens[[0, 31, 32, 33, 70, 139, 140]] = 0
    q_lens[rng.integers(34, 70, long)] = 90
    kv_lens = q_lens + rng.integers(0, 150, B)
    kv_lens[[0, 32, 140]] = 0
    _both(F, _rows(rng, _cache(rng, kv_lens.tolist(), 32, 16, 2), q_lens.tolist(), 8, lead=2), 62)


@pytest.mark.parametrize("q_lens,kv_lens,Hq,Hkv", [([1, 1, 2, 1], [90, 300, 2, 45], 8, 2), ([70, 40], [200, 41], 8, 2),
                                                  ([2, 1], [130, 40], 40, 1), ([30], [64], 100, 1)])
def test_queries_of_very_different_sizes(q_lens, kv_lens, Hq, Hkv):
    F, rng = fa3(), np.random.default_rng(63)
    c = _rows(rng, _cache(rng, kv_lens, 64, 32, Hkv), q_lens, Hq)
    n = c["q"].shape[0]
    c["q"] *= np.exp2(np.resize([0, -40, 9, -7, 5, -70, -3], n * Hq)).reshape(n, Hq, 1).astype(np.float32)
    c["q"][c["q_start"][0], 0] = 0
    _both(F, c, 64)


@pytest.mark.parametrize("q_lens", [[1, 2], [60, 30]])
def test_weights_of_rows_whose_sum_is_infinite(q_lens):
    F, rng = fa3(), np.random.default_rng(65)
    c = _rows(rng, _cache(rng, [200, 150], 32, 16, 2), q_lens, 8)
    before = rng.random((c["num"], 2, 32)).astype(np.float32)
    got = _weigh(F, c, np.full(c["q"].shape[:2], np.inf, np.float32), before)
    ref = before.copy()
    for b, (new, kv) in enumerate(zip(q_lens, (200, 150))):
        t = np.arange(kv - new, kv)
        ref[c["table"][b, t // 32], :, t % 32] = 0
    assert np.array_equal(got, ref)


# -------------------------------------------------------------------- eviction
EVICT = [                         # kv_lens, page, block, Hkv, D, budget, sinks, recent
    ([1], 16, 16, 1, 8, 1, 0, 0),
    ([100, 0, 17], 32, 16, 2, 64, 17, 1, 3),
    ([300, 65, 64, 63], 64, 64, 3, 128, 64, 4, 60),
    ([513], 48, 48, 2, 80, 100, 0, 0),
    ([2500], 96, 32, 1, 128, 1111, 5, 200),
    ([40, 41], 32, 32, 2, 16, 40, 20, 20),
    ([700], 128, 128, 2, 256, 5, 0, 1),
]


def _evict(F, c, w, new, budget, sinks, recent, err=None, **kw):
    got = [_t(c[x]) for x in ("k", "v", "ks", "vs")] + [_t(w)]
    kept, lens = F.evict_gqa_block_paged(*got, _t(c["table"]), _t(c["kv_lens"]), _t(new), budget, sinks=sinks, recent=recent,
                                         dev_err=err, **kw)
    return [x.cpu().numpy() for x in (kept, lens, *got)]


@pytest.mark.parametrize("kv_lens,page,block,Hkv,D,budget,sinks,recent", EVICT)
@pytest.mark.parametrize("ties", [False, True])
def test_eviction(kv_lens, page, block, Hkv, D, budget, sinks, recent, ties):
    F, rng = fa3(), np.random.default_rng(budget + ties)
    pages = -(-budget // page)
    c = _cache(rng, kv_lens, page, block, Hkv, D, extra=pages)
    new = c["rest"][:len(kv_lens) * pages].reshape(-1, pages).copy()
    w = np.exp(3 * rng.standard_normal((c["num"], Hkv, page))).astype(np.float32)
    if ties:
        w = np.where(w < 2, np.where(rng.random(w.shape) < 0.5, -0.0, 0.0), np.rint(w)).astype(np.float32)
        w[rng.random(w.shape) < 0.01] = np.nan
        w[rng.random(w.shape) < 0.01] = np.inf
        w[rng.random(w.shape) < 0.02] = -1.5
    ref = O.evict_block_paged(c["k"], c["v"], c["ks"], c["vs"], w, c["table"], c["kv_lens"], new, budget, sinks, recent)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = _evict(F, c, w, new, budget, sinks, recent, err)
    assert _same(got, ref)
    assert err.item() == 0


def test_eviction_longer_than_shared_memory():
    """Weights that do not fit in shared memory are read again; many equal ones, so that the choice falls inside a tie."""
    F, rng = fa3(), np.random.default_rng(31)
    T, budget = 60001, 20000
    c = _cache(rng, [T], 64, 32, 1, 8, extra=313)
    new = c["rest"][:313].reshape(1, 313).copy()
    for w in (rng.random((c["num"], 1, 64)), rng.integers(0, 3, (c["num"], 1, 64))):
        w = w.astype(np.float32)
        got = _evict(F, c, w, new, budget, 3, 77)
        t = np.arange(T)
        ref = O.kept_tokens(w[c["table"][0, t // 64], 0, t % 64], budget, 3, 77)
        assert got[0][0, 0].tolist() == ref


@pytest.mark.parametrize("T,page,values", [(30000, 48, 1), (30001, 64, 2), (9000, 16, 3)])
def test_eviction_among_many_equal_weights(T, page, values):
    """More equal weights than are put aside, which shared memory holds."""
    F, rng = fa3(), np.random.default_rng(33)
    B, Hkv, budget = 3, 4, 5000
    pages = -(-budget // page)
    c = _cache(rng, [T] * B, page, 16, Hkv, 8, extra=pages)
    new = c["rest"][:B * pages].reshape(B, pages).copy()
    w = (1 + rng.integers(0, values, (c["num"], Hkv, page)) / 64).astype(np.float32)
    kept = _evict(F, c, w, new, budget, 5, 100)[0]
    t = np.arange(T)
    for b in range(B):
        for g in range(Hkv):
            assert kept[b, g].tolist() == O.kept_tokens(w[c["table"][b, t // page], g, t % page], budget, 5, 100)


def test_eviction_bad_lengths_and_pages():
    F, rng = fa3(), np.random.default_rng(32)
    c = _cache(rng, [100, 90, 80], 32, 16, 2, 64, extra=1)
    new = c["rest"][:3].reshape(3, 1).copy()
    w = rng.random((c["num"], 2, 32)).astype(np.float32)
    ref = O.evict_block_paged(c["k"], c["v"], c["ks"], c["vs"], w, c["table"], c["kv_lens"], new, 30, 1, 3)
    for length in (-1, 1000):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = _evict(F, dict(c, kv_lens=np.array([100, length, 80], np.int32)), w, new, 30, 1, 3, err)
        assert err.item() == F.FA3_DEVERR_LENS
        assert np.all(got[0][1] == -1) and got[1][1] == 0 and np.array_equal(got[0][[0, 2]], ref[0][[0, 2]])
        keep = new[1, 0]
        for g, r, b in zip(got[2:], ref[2:], (c["k"], c["v"], c["ks"], c["vs"], w)):
            r = r.copy()
            r[keep] = b[keep]
            assert np.array_equal(g, r, equal_nan=True)
    for which in ("new", "old"):
        d, to, err = dict(c, table=c["table"].copy()), new.copy(), torch.zeros(1, dtype=torch.int32, device="cuda")
        if which == "new":
            to[1, 0] = -5
        else:
            d["table"][1, 1] = 10 ** 7
        got = _evict(F, d, w, to, 30, 1, 3, err)
        assert err.item() == F.FA3_DEVERR_PAGE
        for b in (0, 2):
            assert np.array_equal(got[0][b], ref[0][b]) and np.array_equal(got[2][new[b, 0]], ref[2][new[b, 0]])


# -------------------------------------------------------- together, streams, graphs
def test_a_cache_that_is_filled_read_cut_and_read_again():
    """Prompts, then decode steps with an eviction in between, all four calls on one cache as a server runs them."""
    F, rng = fa3(), np.random.default_rng(41)
    Hq, Hkv, page, block, budget = 8, 2, 32, 16, 48
    num = 40
    pool = np.zeros((num, page, Hkv, 128), np.int8)
    scale = np.full((num, page // block, Hkv), np.nan, np.float32)
    w0 = np.full((num, Hkv, page), 7.0, np.float32)
    perm = rng.permutation(num).astype(np.int32)
    table = perm[:12].reshape(2, 6).copy()
    state = [pool, pool, scale, scale]
    dev = [_t(x) for x in state] + [_t(w0)]
    weights = w0
    lens = np.zeros(2, np.int32)

    def step(q_lens):
        nonlocal state, weights, lens
        start = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
        lens = lens + np.asarray(q_lens, np.int32)
        n = int(start[-1])
        k, v, _ = _kv(rng, n, Hkv, 128, 0.5)
        q = _f(_bf(rng.standard_normal((n, Hq, 128))))
        state = list(O.append_block_paged(k, v, *state, table, start, lens))
        tt, ts, tl, tq = _t(table), _t(start), _t(lens), _bf(q).cuda()
        F.append_gqa_block_paged(_bf(k).cuda(), _bf(v).cuda(), *dev[:4], tt, ts, tl)
        lse = torch.full((n, Hq), 3.0, device="cuda")
        out = F.attn_gqa_block_paged(tq, *dev[:4], ts, tl, tt, SM, lse=lse)
        F.attn_weights_gqa_block_paged(tq, dev[0], dev[2], lse, dev[4], ts, tl, tt, SM)
        assert _same(dev[:4], state)
        c = dict(page=page, block=block, Hkv=Hkv, D=128, num=num, kv_lens=lens, table=table, q_start=start, q=q,
                 used=np.ones(n, bool), k=state[0], v=state[1], ks=state[2], vs=state[3])
        _check_attention(c, _f(out), _f(lse))
        _check_weights(c, _f(lse), weights, _f(dev[4]))
        weights = _f(dev[4])

    step([90, 33])
    step([1, 1])
    new = perm[12:16].reshape(2, 2).copy()
    ref = O.evict_block_paged(*state, weights, table, lens, new, budget, 2, 10)
    kept, nl = F.evict_gqa_block_paged(*dev, _t(table), _t(lens), _t(new), budget, sinks=2, recent=10)
    assert _same((kept, nl, *dev), ref)
    state, weights, lens = list(ref[2:6]), ref[6], ref[1]
    table = np.concatenate([new, perm[16:20].reshape(2, 2)], 1)
    step([1, 1])
    step([3, 20])


def _many(c, n_steps=2):
    """Device copies of everything that the four calls take."""
    t = dict(q=_bf(np.nan_to_num(c["q"])).cuda(), out=torch.zeros(c["q"].shape, dtype=torch.bfloat16, device="cuda"),
             lse=torch.zeros(c["q"].shape[:2], device="cuda"))
    for x in ("k", "v", "ks", "vs", "q_start", "kv_lens", "table"):
        t[x] = _t(c[x])
    t["w"] = torch.full((c["num"], c["Hkv"], c["page"]), 0.25, device="cuda")
    n = c["q"].shape[0]
    g = torch.Generator().manual_seed(n)
    t["kv"] = torch.randn(n, 2 * c["Hkv"], 128, generator=g).bfloat16().cuda()
    pages = -(-40 // c["page"])
    t["new"] = _t(c["rest"][:len(c["kv_lens"]) * pages].reshape(-1, pages))
    t["kept"] = torch.full((len(c["kv_lens"]), c["Hkv"], 40), -1, dtype=torch.int32, device="cuda")
    t["nl"] = torch.zeros(len(c["kv_lens"]), dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    return t


def _all_calls(F, t, stream=None):
    h = t["kv"].shape[1] // 2
    pools = (t["k"], t["v"], t["ks"], t["vs"])
    F.append_gqa_block_paged(t["kv"][:, :h], t["kv"][:, h:], *pools, t["table"], t["q_start"], t["kv_lens"], stream=stream)
    F.attn_gqa_block_paged(t["q"], *pools, t["q_start"], t["kv_lens"], t["table"], SM, out=t["out"], lse=t["lse"], stream=stream)
    F.attn_weights_gqa_block_paged(t["q"], t["k"], t["ks"], t["lse"], t["w"], t["q_start"], t["kv_lens"], t["table"], SM,
                                   stream=stream)
    F.evict_gqa_block_paged(*pools, t["w"], t["table"], t["kv_lens"], t["new"], 40, sinks=1, recent=5, kept=t["kept"],
                            new_lens=t["nl"], stream=stream)


RESULTS = ("k", "v", "ks", "vs", "out", "lse", "w", "kept", "nl")


@pytest.mark.parametrize("q_lens,kv_lens", [([1, 1, 1], [300, 90, 1000]), ([60, 1, 100], [300, 90, 1000])])
def test_other_streams_and_graphs(q_lens, kv_lens):
    F, rng = fa3(), np.random.default_rng(51)
    make = lambda: _rows(np.random.default_rng(52), _cache(np.random.default_rng(53), kv_lens, 64, 32, 2, extra=1),  # noqa: E731
                         q_lens, 8, behind=0)
    ref = _many(make())
    _all_calls(F, ref)
    torch.cuda.synchronize()
    same = lambda a: all(torch.equal(a[x].view(torch.uint8), ref[x].view(torch.uint8)) for x in RESULTS)  # noqa: E731
    a, b = _many(make()), _many(make())
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    _all_calls(F, a, stream=s1)                                    # two streams at once, neither the current one
    with torch.cuda.stream(s2):
        _all_calls(F, b)
    torch.cuda.synchronize()
    assert same(a) and same(b)
    # two graphs that replay at the same time share no workspace
    a, b = _many(make()), _many(make())
    graphs = []
    for t in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            _all_calls(F, t)
        graphs.append(g)
    fresh = _many(make())
    for t in (a, b):
        for x in RESULTS:
            t[x].copy_(fresh[x])
    torch.cuda.synchronize()
    for g, s in zip(graphs, (s1, s2)):
        with torch.cuda.stream(s):
            g.replay()
    torch.cuda.synchronize()
    assert same(a) and same(b)


@pytest.mark.parametrize("q_lens", [[1, 2], [150, 40]])
def test_pages_beyond_32_bit_offsets(q_lens):
    """The same calls on the first and on the last pages of pools of 4.6 GB give the same."""
    F, rng = fa3(), np.random.default_rng(71)
    num, page, block, Hkv, Hq, budget = 70000, 64, 32, 8, 16, 70
    lens = np.array([400, 130], np.int32)
    n, fill = sum(q_lens), int(lens.sum())
    k, v, _ = _kv(rng, fill, Hkv, 128)
    k, v, q = _bf(k).cuda(), _bf(v).cuda(), _bf(rng.standard_normal((n, Hq, 128))).cuda()
    pools = [torch.empty(num, page, Hkv, 128, dtype=torch.int8, device="cuda") for _ in range(2)]
    scales = [F.block_scale_pool(pools[0], block) for _ in range(2)]
    w = F.attn_weight_pool(pools[0])
    start = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    results = []
    for first in (0, num - 20):
        table = first + np.arange(14, dtype=np.int32).reshape(2, 7)
        new = first + np.arange(14, 18, dtype=np.int32).reshape(2, 2)
        tt, tl, ts = _t(table), _t(lens), _t(start)
        F.append_gqa_block_paged(k, v, *pools, *scales, tt, _t(np.array([0, 400, 530], np.int32)), tl)
        lse = torch.zeros(n, Hq, device="cuda")
        out = F.attn_gqa_block_paged(q, *pools, *scales, ts, tl, tt, SM, lse=lse)
        F.attn_weights_gqa_block_paged(q, pools[0], scales[0], lse, w, ts, tl, tt, SM)
        kept, nl = F.evict_gqa_block_paged(*pools, *scales, w, tt, tl, _t(new), budget, sinks=1, recent=5)
        at = [(first + 14 + 2 * b + t // page, t % page) for b in range(2) for t in range(budget)]
        pg, row = (torch.tensor(x, device="cuda") for x in zip(*at))
        results.append([out, lse, kept, nl, pools[0][pg, row], pools[1][pg, row], scales[0][pg, row // block],
                        scales[1][pg, row // block], w[pg, :, row]])
    assert all(torch.equal(x, y) for x, y in zip(*results))
    assert results[0][8].sum() > 0 and results[0][3].tolist() == [budget, budget]


def test_refusals_on_the_gpu():
    F = fa3()
    pool = torch.zeros(4, 32, 2, 128, dtype=torch.int8, device="cuda")
    s, w = F.block_scale_pool(pool, 16), F.attn_weight_pool(pool)
    table, start, lens = (torch.zeros(1, 2, dtype=torch.int32, device="cuda"), torch.tensor([0, 1], dtype=torch.int32).cuda(),
                          torch.ones(1, dtype=torch.int32, device="cuda"))
    x = torch.zeros(1, 2, 128, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(1, 2, device="cuda")
    for bad in (s[:3], s[..., :1], F.block_scale_pool(pool, 32), s.double(), s[:, :1].expand(4, 3, 2).contiguous()):
        with pytest.raises((ValueError, TypeError)):
            F.append_gqa_block_paged(x, x, pool, pool, s, bad, table, start, lens)
        with pytest.raises((ValueError, TypeError)):
            F.attn_gqa_block_paged(x, pool, pool, s, bad, start, lens, table, SM)
    for q in (x.float(), x[..., :64], x[:, :1].expand(1, 2, 128), x[0]):
        with pytest.raises((ValueError, TypeError)):
            F.attn_gqa_block_paged(q, pool, pool, s, s, start, lens, table, SM)
        with pytest.raises((ValueError, TypeError)):
            F.attn_weights_gqa_block_paged(q, pool, s, lse, w, start, lens, table, SM)
    with pytest.raises(ValueError):
        F.attn_gqa_block_paged(x, pool, pool, s, s, start, lens, table, SM, lse=lse[:, :1])
    with pytest.raises(ValueError):
        F.attn_gqa_block_paged(x, pool, pool, s, s, start, lens, table, SM, out=x[:, :1])
    with pytest.raises(F.FA3Error):
        F.attn_gqa_block_paged(x, pool, pool, s, s, start, lens, table, 0.0)
    with pytest.raises(F.FA3Error):
        F.attn_gqa_block_paged(x, pool, pool, s, s, start, lens, table, SM, workspace=torch.zeros(16, device="cuda"))
    with pytest.raises(F.FA3Error):
        F.attn_weights_gqa_block_paged(x, pool, s, lse, w, start, lens, table, SM, workspace=torch.zeros(16, device="cuda"))
    with pytest.raises(ValueError):
        F.attn_weights_gqa_block_paged(x, pool, s, lse, w[:, :1], start, lens, table, SM)
    for kw in (dict(budget=0), dict(budget=65), dict(budget=4, sinks=3, recent=2), dict(budget=4, sinks=-1),
               dict(budget=4, kept=torch.zeros(1, 2, 5, dtype=torch.int32, device="cuda")),
               dict(budget=4, new_lens=torch.zeros(2, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            F.evict_gqa_block_paged(pool, pool, s, s, w, table, lens, table, **kw)
    # no rows: nothing to do
    F.append_gqa_block_paged(x[:0], x[:0], pool, pool, s, s, table, start, lens)
    assert F.attn_gqa_block_paged(x[:0], pool, pool, s, s, start, lens, table, SM).shape == (0, 2, 128)
    F.attn_weights_gqa_block_paged(x[:0], pool, s, lse[:0], w, start, lens, table, SM)
