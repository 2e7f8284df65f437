"""Block-scaled cache at the edges of its numbers: query rows and log-sum-exps that are not finite, scores of very different
sizes side by side, scales far from one, and tables far wider than their contexts.

Tolerances beside test_gpu_block.py's.  A token's weight is added up term by term: the row's term exp(s - lse) is off by its own
d (a score's error) and by what its exponent's parts lose.  Those are f = fl(k_scale fl(sm log2 e)), two roundings of |s|;
fl(lse log2 e) and, in the kernel that takes it through the product, fl(1 / f), two of |lse|; and there the tensor pipe's last
sum of nine terms, each cut off below 2^-24 of the greatest, |lse|: 16 U (|s| + |lse| + 1) holds them, U = 2^-24, and 4 U for
the exponential.  Where that is no small number e, the term lies within exp(+-e).  64 additions a step and the compensated
sum of steps: 68 U of the sum.  A term below 2^-126, float32's smallest normal number, may be lost: 2^-126 for each.
"""
import numpy as np
import pytest
import torch

from helpers import fa3
from oracle import fa3_oracle as O
from test_gpu_block import ATTN, SM, U, _attend, _bf, _cache, _check_attention, _f, _rows, _score_error, _t, _weigh

pytestmark = pytest.mark.gpu


def _weight_bounds(c, lse, before, sm=SM):
    """The weights pool in float64 and each weight's tolerance."""
    lse = lse.astype(np.float32).astype(np.float64)
    q, ps, g = np.nan_to_num(c["q"]), c["page"], c["q"].shape[1] // c["Hkv"]
    d = _score_error(c, sm)
    ref, tol = before.astype(np.float64), np.zeros(before.shape)
    for b, rows, h, s in O.block_scores(q, c["k"], c["ks"], c["table"], c["q_start"], c["kv_lens"], sm):
        le = lse[rows, h][:, None]
        with np.errstate(invalid="ignore"):
            term = np.where(s == -np.inf, 0.0, np.exp(s - le))
            e = d[rows, h][:, None] + (np.abs(np.where(s == -np.inf, 0.0, s)) + np.abs(le) + 1) * 16 * U + 4 * U
            off = np.where(term == 0, 0.0, term * np.expm1(e))
        t = np.arange(int(c["kv_lens"][b]))
        at = (c["table"][b, t // ps], h // g, t % ps)
        if h % g == 0:
            ref[at] = np.where(t >= len(t) - (rows.stop - rows.start), 0.0, ref[at])
        ref[at] += term.sum(0)
        tol[at] += off.sum(0) + 68 * U * term.sum(0) + len(term) * 2.0 ** -126
    return ref, tol + np.abs(ref) * 2 * U


def _lse(c, sm=SM):
    return O.attention_block(np.nan_to_num(c["q"]), c["k"], c["v"], c["ks"], c["vs"], c["table"], c["q_start"], c["kv_lens"], sm,
                             np.zeros(c["q"].shape), np.zeros(c["q"].shape[:2]))[1]


def _within(got, ref, tol):
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), got[bad][:4], ref[bad][:4], tol[bad][:4])


# ------------------------------------------------- query rows that are not finite
# Hq, Hkv, q_lens, kv_lens: units of 8, 16 and 32 columns, one long context, two row tiles, one row tile, cut units of both
SHAPES = [(8, 2, [1, 1, 1], [300, 2, 129]), (16, 1, [1, 1], [500, 77]), (8, 1, [4, 4, 4, 4], [900, 33, 64, 5]),
          (8, 1, [1], [20000]), (8, 2, [200, 40, 130], [700, 129, 130]), (8, 2, [30, 25], [400, 25]), (8, 1, [70], [9000]),
          (8, 2, [20], [6000])]


def _spoil(c, value, rng):
    """Some rows' queries of one head get `value`; which (row, head) did."""
    hit = np.zeros(c["q"].shape[:2], bool)
    q = c["q"].copy()
    starts = c["q_start"]
    for b in range(len(starts) - 1):
        row = int(rng.integers(starts[b], starts[b + 1]))
        hit[row, rng.integers(0, q.shape[1])] = True
    hit[starts[0], 0] = True
    q[hit, 5] = value
    return dict(c, q=q), hit


@pytest.mark.parametrize("Hq,Hkv,q_lens,kv_lens", SHAPES)
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("block", [16, 32, 128])
def test_a_query_that_is_not_finite_shows_in_its_row_alone(Hq, Hkv, q_lens, kv_lens, value, block):
    F, rng = fa3(), np.random.default_rng(81)
    c = _rows(rng, _cache(rng, kv_lens, 128, block, Hkv), q_lens, Hq)
    out, _ = _attend(F, c)
    _check_attention(c, out, None)
    for code in (None, -77):                                       # any codes; all scores infinite and of one sign
        d = c
        if code is not None:
            d = dict(c, k=c["k"].copy())
            d["k"][..., 5] = code
            out, _ = _attend(F, d)
        spoiled, hit = _spoil(d, value, rng)
        got, _ = _attend(F, spoiled)
        assert np.all(np.isnan(got[hit]))
        assert np.array_equal(got[~hit], out[~hit])


@pytest.mark.parametrize("Hq,Hkv,q_lens,kv_lens", SHAPES)
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_the_log_sum_exp_of_a_query_that_is_not_finite_is_not_a_number(Hq, Hkv, q_lens, kv_lens, value):
    F, rng = fa3(), np.random.default_rng(82)
    c = _rows(rng, _cache(rng, kv_lens, 64, 32, Hkv), q_lens, Hq)
    for code in (None, -77):
        if code is not None:
            c["k"][..., 5] = code
        _, lse = _attend(F, c)
        spoiled, hit = _spoil(c, value, rng)
        _, got = _attend(F, spoiled)
        assert np.all(np.isnan(got[hit]))
        assert np.array_equal(got[~hit], lse[~hit])


# ------------------------------------------------------------ log-sum-exps and weights
# Hq, Hkv, q_lens, kv_lens: fa3_few.cu's kernel with one and with several chunks of columns, fa3_weights.cu's with units
# whole and cut
WEIGHT_SHAPES = [(8, 2, [1, 3], [300, 129]), (16, 1, [5, 1], [500, 77]), (8, 2, [70, 40], [200, 41]), (100, 1, [30], [64]),
                 (8, 1, [400, 30], [5000, 31])]


@pytest.mark.parametrize("Hq,Hkv,q_lens,kv_lens", WEIGHT_SHAPES)
@pytest.mark.parametrize("first", [True, False])
@pytest.mark.parametrize("query", [True, False])
def test_a_log_sum_exp_or_query_that_is_not_a_number_shows_in_the_weights(Hq, Hkv, q_lens, kv_lens, first, query):
    F, rng = fa3(), np.random.default_rng(83)
    c = _rows(rng, _cache(rng, kv_lens, 64, 32, Hkv), q_lens, Hq)
    before = rng.random((c["num"], Hkv, 64)).astype(np.float32)
    lse = _lse(c)
    row, h = int(c["q_start"][0]) + (0 if first else q_lens[0] - 1), 0 if first else Hq - 1
    sees = kv_lens[0] - q_lens[0] + (row - int(c["q_start"][0])) + 1
    without = lse.copy()
    without[row, h] = 1e4                                          # a row that gives nothing
    ref, tol = _weight_bounds(c, without, before)
    if query:
        c["q"][row, h, 77] = np.nan
    else:
        lse[row, h] = np.nan
    got = _weigh(F, c, lse, before)
    shown = np.zeros(got.shape, bool)
    t = np.arange(sees)
    shown[c["table"][0, t // 64], h // (Hq // Hkv), t % 64] = True
    assert np.all(np.isnan(got[shown]))
    _within(got[~shown], ref[~shown], tol[~shown])


@pytest.mark.parametrize("Hq,Hkv,q_lens,kv_lens", WEIGHT_SHAPES)
@pytest.mark.parametrize("size", [2.0 ** 14, 2.0 ** 17])
def test_weights_of_scores_of_a_million(Hq, Hkv, q_lens, kv_lens, size):
    """Queries of one power of two, so that a score's sum is exact; one key far above the others, which the weights are of."""
    F, rng = fa3(), np.random.default_rng(84)
    c = _rows(rng, _cache(rng, kv_lens, 64, 32, Hkv), q_lens, Hq)
    sign = np.where(rng.random(c["q"].shape) < 0.5, -1.0, 1.0)
    c["q"] = np.where(c["used"][:, None, None], sign * size, np.nan).astype(np.float32)
    c["ks"] = np.where(np.isfinite(c["ks"]), np.float32(0.5), np.float32(np.nan))
    lse = _lse(c).astype(np.float32)
    assert np.abs(lse[c["used"]]).max() > 4e5
    before = np.zeros((c["num"], Hkv, 64), np.float32)
    ps, g, ref = 64, Hq // Hkv, np.zeros(before.shape)
    low, high = np.zeros(before.shape), np.zeros(before.shape)
    for b, rows, h, s in O.block_scores(np.nan_to_num(c["q"]), c["k"], c["ks"], c["table"], c["q_start"], c["kv_lens"], SM):
        le = lse[rows, h].astype(np.float64)[:, None]
        seen = s > -np.inf
        x = np.where(seen, s, 0) - le
        e = (np.abs(np.where(seen, s, 0)) + np.abs(le) + 1) * 16 * U + 4 * U
        t = np.arange(int(c["kv_lens"][b]))
        at = (c["table"][b, t // ps], h // g, t % ps)
        low[at] += np.where(seen, np.exp(np.minimum(x - e, 80)), 0).sum(0)
        high[at] += np.where(seen, np.exp(np.minimum(x + e, 80)), 0).sum(0)
    got = _weigh(F, c, lse, before)
    assert np.all(np.isfinite(got))
    bad = (got < low * (1 - 2.0 ** -16) - 1e-30) | (got > high * (1 + 2.0 ** -16) + 1e-30)
    assert not bad.any(), (int(bad.sum()), got[bad][:4], low[bad][:4], high[bad][:4])


@pytest.mark.parametrize("Hq,Hkv,q_lens,kv_lens", WEIGHT_SHAPES)
@pytest.mark.parametrize("large", [0.0, 2.0 ** 6, 2.0 ** 10])
def test_weights_of_small_rows_beside_large_ones(Hq, Hkv, q_lens, kv_lens, large):
    """Every token's bound is that of its own rows: the first row of a sequence has the largest scores, in its group's
    first head, and another in the middle; they give their weight to few tokens."""
    F, rng = fa3(), np.random.default_rng(85)
    c = _rows(rng, _cache(rng, kv_lens, 64, 32, Hkv), q_lens, Hq)
    g = Hq // Hkv
    size = np.exp2(np.resize([0, -3, -40, -1, -7], c["q"].shape[0] * Hq)).reshape(-1, Hq)
    for b, n in enumerate(q_lens):
        for i in (0, n // 2):
            size[c["q_start"][b] + i, ::g] = large
    c["q"] *= size[..., None].astype(np.float32)
    lse = _lse(c)
    before = (rng.random((c["num"], Hkv, 64)) * 0.01).astype(np.float32)
    _within(_weigh(F, c, lse, before), *_weight_bounds(c, lse, before))


# ------------------------------------------------------------ scales far from one
@pytest.mark.parametrize("Hq,Hkv,q_lens,kv_lens", [(8, 2, [1, 1, 1], [300, 2, 129]), (8, 1, [4, 4], [900, 33]),
                                                   (8, 2, [200, 40, 130], [700, 129, 130]), (8, 2, [30, 25], [400, 25])])
@pytest.mark.parametrize("block", [16, 32, 128])
@pytest.mark.parametrize("exponent", [-95, -84, -60, 45, 75, 90])
def test_attention_of_key_scales_and_queries_that_make_up_for_one_another(Hq, Hkv, q_lens, kv_lens, block, exponent):
    """Queries 2^exponent as large and key scales 2^-exponent: the scores are ordinary, with half of the rows and the
    blocks' scales (the last block's aside) as far the other way, whose scores are next to nothing."""
    F, rng = fa3(), np.random.default_rng(86)
    c = _rows(rng, _cache(rng, kv_lens, 128, block, Hkv), q_lens, Hq)
    c["q"] = np.ldexp(c["q"], exponent).astype(np.float32)
    c["ks"] = np.ldexp(c["ks"], -exponent).astype(np.float32)
    out, lse = _attend(F, c)
    _check_attention(c, out, lse)
    some = rng.random(c["ks"].shape) < 0.3
    c["ks"][some & np.isfinite(c["ks"])] *= np.float32(2.0 ** -20)
    c["q"][::2] *= np.float32(2.0 ** -10)
    c["q"] = _f(_bf(c["q"]))
    out, lse = _attend(F, c)
    _check_attention(c, out, lse)


@pytest.mark.parametrize("Hq,Hkv,q_lens,kv_lens", WEIGHT_SHAPES)
@pytest.mark.parametrize("exponent", [-84, 45, 60])
def test_weights_of_key_scales_and_queries_that_make_up_for_one_another(Hq, Hkv, q_lens, kv_lens, exponent):
    F, rng = fa3(), np.random.default_rng(87)
    c = _rows(rng, _cache(rng, kv_lens, 64, 32, Hkv), q_lens, Hq)
    c["q"] = np.ldexp(c["q"], exponent).astype(np.float32)
    c["ks"] = np.ldexp(c["ks"], -exponent).astype(np.float32)
    c["ks"][(rng.random(c["ks"].shape) < 0.2) & np.isfinite(c["ks"])] = 0
    lse = _lse(c)
    before = (rng.random((c["num"], Hkv, 64)) * 0.01).astype(np.float32)
    _within(_weigh(F, c, lse, before), *_weight_bounds(c, lse, before))


# ------------------------------------------------------------ shapes that no other test has
@pytest.mark.parametrize("Hq,Hkv,q_lens,kv_lens", [(28, 4, [700, 1], [1900, 300]), (24, 2, [500], [2100]), (24, 8, [600], [600]),
                                                   (40, 8, [300, 200], [900, 1300])])
def test_weights_of_prompts_in_groups_that_do_not_divide_128(Hq, Hkv, q_lens, kv_lens):
    F, rng = fa3(), np.random.default_rng(88)
    c = _rows(rng, _cache(rng, kv_lens, 64, 64, Hkv), q_lens, Hq)
    lse = _lse(c)
    before = (rng.random((c["num"], Hkv, 64)) * 0.01).astype(np.float32)
    got = _weigh(F, c, lse, before)
    _within(got, *_weight_bounds(c, lse, before))
    assert np.array_equal(got, _weigh(F, c, lse, before))


@pytest.mark.parametrize("q_lens", [[1, 1], [60, 30], [300, 5]])
def test_tables_far_wider_than_the_contexts(q_lens):
    """A table for 2^30 tokens a sequence: plans in 64 bits, whichever kernel."""
    F, rng = fa3(), np.random.default_rng(89)
    page, wide = 16384, 65536
    lens = [600, 320]
    c = _rows(rng, _cache(rng, lens, page, 32, 1, spare=2, extra=1), q_lens, 8)
    table = np.full((2, wide), -1, np.int32)
    table[:, 0] = c["table"][:, 0]
    c["table"] = table
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = _attend(F, c, err)
    _check_attention(c, out, lse)
    before = (rng.random((c["num"], 1, page)) * 0.01).astype(np.float32)
    got = _weigh(F, c, lse, before, err)
    _within(got, *_weight_bounds(c, lse, before))
    assert err.item() == 0


@pytest.mark.parametrize("Hq,Hkv,page,block,q_lens,kv_lens", ATTN)
@pytest.mark.parametrize("mixed", [False, True])
def test_weights_within_the_bounds_of_their_own_rows(Hq, Hkv, page, block, q_lens, kv_lens, mixed):
    F, rng = fa3(), np.random.default_rng(90)
    c = _rows(rng, _cache(rng, kv_lens, page, block, Hkv), q_lens, Hq, lead=1)
    if mixed:
        n = c["q"].shape[0]
        c["q"] *= np.exp2(np.resize([0, -40, 9, -7, 5, -70, -3], n * Hq)).reshape(n, Hq, 1).astype(np.float32)
    _, lse = _attend(F, c)
    before = (rng.random((c["num"], Hkv, page)) * 0.01).astype(np.float32)
    _within(_weigh(F, c, lse, before), *_weight_bounds(c, lse, before))
