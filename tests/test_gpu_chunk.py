"""GPU parity of attention over packed new rows (chunks over a paged cache, cross attention) against the
float64 oracle."""
import sys
import threading

import numpy as np
import pytest
import torch

import workloads as W
from helpers import assert_attn_close, attn_errors, bf16_dev, fa3
from oracle import fa3_oracle as O

pytestmark = pytest.mark.gpu
SM = 128 ** -0.5
KEEP = 3.0                                       # what rows of no sequence hold before and after


def _t(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _case(rng, Hq, Hkv, q_lens, kv_lens, page=None, lead=0, behind=1):
    B = len(q_lens)
    q_start = (lead + np.concatenate([[0], np.cumsum(q_lens)])).astype(np.int32)
    n = int(q_start[-1]) + behind
    code = lambda *s: np.clip(np.rint(rng.standard_t(5, s) * 30), -127, 127).astype(np.int8)  # noqa: E731
    c = dict(q=code(n, Hq, 128), q_start=q_start, lens=np.asarray(kv_lens, np.int32), page=page,
             qs=(W.log_uniform(rng, 0.5, 2, Hq) / 30).astype(np.float32),
             ks=(W.log_uniform(rng, 0.5, 2, Hkv) / 30).astype(np.float32),
             vs=(W.log_uniform(rng, 0.5, 2, Hkv) / 30).astype(np.float32))
    T = max(max(kv_lens), 1)
    if page is None:
        c["k"], c["v"] = code(B, T, Hkv, 128), code(B, T, Hkv, 128)
    else:
        mp = -(-T // page) + 1
        num = B * mp + 2
        c["table"] = rng.permutation(num)[:B * mp].reshape(B, mp).astype(np.int32)
        for b, kv in enumerate(kv_lens):
            c["table"][b, -(-kv // page):] = num + 5                          # past the context: never read
        c["k"], c["v"] = code(num, page, Hkv, 128), code(num, page, Hkv, 128)
    return c


def _run(F, c, err=None, out=None, **kw):
    if out is None:
        out = torch.full(c["q"].shape, KEEP, dtype=torch.bfloat16, device="cuda")
    a = [_t(c[k]) for k in ("q", "k", "v", "qs", "ks", "vs", "q_start", "lens")]
    table = None if c["page"] is None else _t(c["table"])
    torch.cuda.synchronize()                                 # the call may be on another stream than the copies
    if c["page"] is None:
        o = F.cross_attn_gqa(*a, SM, out=out, dev_err=err, **kw)
    else:
        o = F.prefill_attn_gqa_paged(*a, table, SM, out=out, dev_err=err, **kw)
    torch.cuda.synchronize()
    return o.float().cpu().numpy()


def _ref(c):
    lens = np.where(np.diff(c["q_start"]) > 0, c["lens"], 0)
    if c["page"] is None:
        kv = [[x[b, :n] for b, n in enumerate(lens)] for x in (c["k"], c["v"])]
    else:
        kv = [[x[c["table"][b, np.arange(n) // c["page"]], np.arange(n) % c["page"]] for b, n in enumerate(lens)]
              for x in (c["k"], c["v"])]
    return O.packed_attention(c["q"], *kv, c["qs"], c["ks"], c["vs"], c["q_start"], lens, SM, c["page"] is not None,
                              np.full(c["q"].shape, KEEP))


def _gate(got, ref, c, what):
    """|got - ref| within what the arithmetic can be off.  The output rounds by half a step, 2^-8 of the value
    (with one key the output is bf16(v), so this alone can be the whole error, and a relative-RMS gate below 2^-8
    cannot hold for few distinct values).  Before that the output is a mean of v with weights off by: fp16 rounding
    2^-11 of a weight, twice (sum and product); at most 2^-25 for each of the T weights below fp16's normal range,
    twice, where the largest weight is at least 1; and the float32 score, |s| log2 units rounded about four times,
    2^-22 |s| (a relative error of the weight)."""
    T = max(1, int(c["lens"].max()))
    s = 128.0 * np.abs(c["q"].astype(np.int32)).max() * np.abs(c["k"].astype(np.int32)).max() * float(c["qs"].max()) \
        * float(c["ks"].max()) * SM * 1.4427
    v = 127.0 * float(c["vs"].max())
    tol = 2.0 ** -8 * np.abs(ref) * (1 + 2.0 ** -8) + (2.0 ** -10 + T * 2.0 ** -24 + 2.0 ** -22 * s) * v + 1e-30
    d = np.abs(np.asarray(got, np.float64) - ref)
    assert np.all(np.isfinite(got)), f"{what}: non-finite output"
    print(f"{what}: {float((d / tol).max()):.3f} of the tolerance")
    assert np.all(d <= tol), f"{what}: {float((d / tol).max()):.3f} of the tolerance"


def _check(F, c, what):
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got, ref = _run(F, c, err), _ref(c)
    assert int(err.item()) == 0
    s, e = c["q_start"][0], c["q_start"][-1]
    assert np.all(got[:s] == KEEP) and np.all(got[e:] == KEEP), f"{what}: rows of no sequence written"
    _gate(got[s:e], ref[s:e], c, what)
    return got


@pytest.mark.parametrize("Hq,Hkv,page", [(8, 1, 64), (4, 4, 16), (6, 2, 24), (10, 2, 7), (14, 2, 100), (16, 1, 128),
                                         (2, 1, 1), (128, 1, 48), (36, 3, 256)])
def test_ragged_chunks(Hq, Hkv, page):
    # group sizes 8, 1, 3, 5, 7, 16, 2, 128, 12; a sequence without new rows; single tokens; pages inside tiles
    F = fa3()
    rng = np.random.default_rng([Hq, Hkv, page])
    c = _case(rng, Hq, Hkv, [1, 40, 0, 3, 70], [300, 40, 7, 129, 200], page, lead=2)
    _check(F, c, f"chunk G={Hq // Hkv} page={page}")


@pytest.mark.parametrize("kv", [1, 2, 127, 128, 129, 255, 256, 257, 1023])
def test_single_tokens_at_key_tile_edges(kv):
    F = fa3()
    c = _case(np.random.default_rng(kv), 8, 2, [1, 1, 1], [kv, 1, max(1, kv - 1)], 32)
    _check(F, c, f"one token, {kv} keys")


@pytest.mark.parametrize("n", [15, 16, 17, 31, 32, 33, 64, 65, 129])
def test_row_block_edges(n):
    # 16 positions fill a tile of 128 rows at 8 heads, 32 a row block
    F = fa3()
    c = _case(np.random.default_rng(n), 8, 1, [n, n], [n, n + 130], 64)
    _check(F, c, f"{n} rows")


def test_many_sequences():
    F = fa3()
    rng = np.random.default_rng(3)
    ql = rng.integers(0, 4, 150)
    c = _case(rng, 4, 2, list(ql), list(ql + rng.integers(0, 60, 150)), 16)
    _check(F, c, "150 sequences")


def test_long_context_of_one_sequence():
    # one row block of each KV head: its keys are shared out over the whole GPU
    F = fa3()
    for q in (1, 5, 20):
        c = _case(np.random.default_rng(q), 16, 2, [q], [9001], 48)
        _check(F, c, f"{q} rows over 9001 keys")


def test_mixed_long_and_single():
    F = fa3()
    c = _case(np.random.default_rng(4), 16, 2, [1, 260, 1, 1], [3000, 1300, 2, 700], 64)
    _check(F, c, "mixed batch")


def test_growing_scores_force_rescales():
    F = fa3()
    c = _case(np.random.default_rng(5), 8, 1, [40, 1], [600, 1500], 64)
    sign = np.where(np.arange(128) % 3 == 0, -1, 1)
    T = 1500
    ramp = np.clip(np.arange(T) / T * 127, 1, 127)
    for b, n in enumerate(c["lens"]):
        for t in range(n):
            c["k"][c["table"][b, t // 64], t % 64] = np.rint(sign * ramp[t]).astype(np.int8)
    c["q"][:] = (sign * 100).astype(np.int8)
    c["qs"][:] = c["ks"][:] = 0.02
    _check(F, c, "growing scores")


def test_extreme_codes_and_zero_scales():
    F = fa3()
    c = _case(np.random.default_rng(6), 4, 2, [18, 1], [140, 400], 16)
    c["q"][:] = np.where(c["q"] > 0, 127, -127)
    c["k"][:] = np.where(c["k"] > 0, 127, -127)
    c["qs"][:] = c["ks"][:] = 1.0                                             # one key takes all the weight
    c["qs"][1] = 0.0                                                          # equal weights
    c["vs"][1] = 0.0
    _check(F, c, "extreme codes")


def test_bad_lengths_leave_their_rows():
    F = fa3()
    for page, bads in ((16, [3, -1, 4000]), (None, [-1, 4000])):
        for bad in bads:
            c = _case(np.random.default_rng(7), 8, 2, [4, 5, 30], [50, 60, 70], page)
            ref = _ref(c)
            c["lens"][1] = bad
            err = torch.zeros(1, dtype=torch.int32, device="cuda")
            got = _run(F, c, err)
            assert int(err.item()) == F.FA3_DEVERR_LENS
            assert np.all(got[4:9] == KEEP)
            for r in (slice(0, 4), slice(9, 39)):
                _gate(got[r], ref[r], c, f"beside lens {bad}")


@pytest.mark.parametrize("start", [[0, 9, 4, 39], [-3, 4, 9, 39], [0, 4, 9, 4000]])
def test_bad_q_start_is_reported(start):
    F = fa3()
    c = _case(np.random.default_rng(8), 8, 2, [4, 5, 30], [50, 60, 70], 16)
    c["q_start"] = np.asarray(start, np.int32)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = _run(F, c, err)
    assert int(err.item()) == F.FA3_DEVERR_LENS
    assert np.all(np.isfinite(got))


def test_bad_page_is_reported():
    F = fa3()
    c = _case(np.random.default_rng(9), 8, 2, [4, 5, 30], [50, 60, 70], 16)
    ref = _ref(c)
    for bad in (-1, c["k"].shape[0]):
        keep, c["table"][1, 2] = c["table"][1, 2], bad
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = _run(F, c, err)
        c["table"][1, 2] = keep
        assert int(err.item()) == F.FA3_DEVERR_PAGE
        for r in (slice(0, 4), slice(9, 39)):
            _gate(got[r], ref[r], c, "beside a bad page")


@pytest.mark.parametrize("Hq,Hkv", [(8, 1), (4, 4), (12, 4), (5, 1)])
def test_cross_ragged(Hq, Hkv):
    # states: none, one, inside a tile, several tiles; rows: none, one, many
    F = fa3()
    rng = np.random.default_rng([Hq, Hkv])
    c = _case(rng, Hq, Hkv, [3, 1, 0, 70, 1, 33], [0, 1, 9, 200, 515, 128], None, lead=1)
    got = _check(F, c, f"cross G={Hq // Hkv}")
    assert not got[1:4].any()                                                 # no states: zero rows


def test_cross_all_empty():
    F = fa3()
    c = _case(np.random.default_rng(10), 4, 2, [2, 40], [0, 0], None)
    got = _check(F, c, "no states")
    assert not got[:42].any()


def test_cross_many_empty_between_full():
    # a CTA's run of several units without keys beside units with keys, one and two row tiles
    F = fa3()
    rng = np.random.default_rng(18)
    lens = [0] * 90 + [300, 0, 0, 140] + [0] * 60
    rows = [1] * 90 + [1, 2, 1, 40] + list(rng.integers(0, 40, 60))
    c = _case(rng, 8, 2, rows, lens, None)
    _check(F, c, "many empty states")


def test_cross_long_runs_of_empty_states():
    # dozens of units without keys in one CTA's share, behind units with several key tiles
    F = fa3()
    rng = np.random.default_rng(19)
    lens = np.zeros(2000, int)
    lens[rng.choice(2000, 60, replace=False)] = rng.integers(1, 700, 60)
    c = _case(rng, 8, 2, [1] * 2000, list(lens), None)
    _check(F, c, "runs of empty states")


def test_more_sequences_than_a_warp_has_lanes():
    F = fa3()
    rng = np.random.default_rng(20)
    rows = list(rng.choice([0, 1, 1, 1, 3, 50], 1300))
    c = _case(rng, 8, 2, rows, [r + int(x) for r, x in zip(rows, rng.integers(0, 200, 1300))], 16)
    _check(F, c, "1300 sequences")


@pytest.mark.parametrize("seed", range(8))
def test_short_units_beside_longer_ones(seed):
    # parts of the line shorter than a unit's fixed cost and a key tile: cuts right behind a unit's begin
    F = fa3()
    rng = np.random.default_rng([25, seed])
    rows = list(rng.choice([1, 1, 1, 1, 1, 1, 20, 40], 6 * (seed + 1)))
    c = _case(rng, 8, 1 + seed % 2 * 3, rows, [r + int(x) for r, x in zip(rows, rng.choice([3, 60, 90, 500, 900], len(rows)))], 32)
    _check(F, c, "short units")


def test_table_of_a_very_long_context():
    # a table wide enough that the plan is made in 64 bits: the same cuts, the same bits
    F = fa3()
    rng = np.random.default_rng(21)
    c = _case(rng, 16, 2, [1, 70], [3000, 1900], 256)
    want = _run(F, c)
    _gate(want, _ref(c), c, "narrow table")
    wide = torch.full((2, 1 << 20), -1, dtype=torch.int32, device="cuda")
    wide[:, :c["table"].shape[1]] = _t(c["table"])
    out = torch.full(c["q"].shape, KEEP, dtype=torch.bfloat16, device="cuda")
    a = [_t(c[k]) for k in ("q", "k", "v", "qs", "ks", "vs", "q_start", "lens")]
    F.prefill_attn_gqa_paged(*a, wide, SM, out=out)
    assert np.array_equal(out.float().cpu().numpy(), want)


def test_agrees_with_the_decode_and_prefill_calls():
    # the same cache through the calls that were there: all within the gate of one oracle
    F = fa3()
    rng = np.random.default_rng(11)
    c = _case(rng, 16, 2, [1, 1, 1], [400, 33, 1], 16, behind=0)
    a = [_t(c[k]) for k in ("q", "k", "v", "qs", "ks", "vs", "lens")]
    ref = _ref(c)
    _gate(_run(F, c), ref, c, "chunk")
    _gate(F.decode_attn_gqa_paged(*a, _t(c["table"]), SM).float().cpu().numpy(), ref, c, "decode")
    c = _case(rng, 16, 2, [90], [90], 16, behind=0)
    ref = _ref(c)
    _gate(_run(F, c), ref, c, "chunk")
    k, v = (x[c["table"][0, np.arange(90) // 16], np.arange(90) % 16][None] for x in (c["k"], c["v"]))
    one = _t(np.array([90], np.int32))
    pre = F.prefill_attn_gqa(_t(c["q"][None]), _t(k), _t(v), _t(c["qs"]), _t(c["ks"]), _t(c["vs"]), one, one, SM)
    _gate(pre[0].float().cpu().numpy(), ref, c, "prefill")


def test_results_repeat_bit_for_bit():
    F = fa3()
    c = _case(np.random.default_rng(12), 16, 2, [1, 100, 7], [2500, 1300, 900], 64)
    first = _run(F, c)
    for _ in range(3):
        assert np.array_equal(first, _run(F, c))


def test_streams_and_graphs():
    # a side stream of its own; a captured call replayed on changed contents; two graphs replayed in turn
    F = fa3()
    rng = np.random.default_rng(13)
    c = _case(rng, 16, 2, [1, 37, 1], [2000, 700, 90], 64)
    d = _case(rng, 16, 2, [1, 37, 1], [1500, 64, 1999], 64)
    d["table"], d["k"], d["v"] = c["table"].copy(), c["k"], c["v"]
    full = np.random.default_rng(14).permutation(c["k"].shape[0])[:c["table"].size].reshape(c["table"].shape)
    c["table"] = full.astype(np.int32)
    d["table"] = full.astype(np.int32)
    want_c, want_d = _run(F, c), _run(F, d)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = _run(F, c, stream=s)
    assert np.array_equal(got, want_c)
    g, bufs = [], []
    for k in range(2):
        a = [_t(c[x]) for x in ("q", "k", "v", "qs", "ks", "vs", "q_start", "lens")] + [_t(c["table"])]
        out = torch.full(c["q"].shape, KEEP, dtype=torch.bfloat16, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            F.prefill_attn_gqa_paged(*a, SM, out=out)
        g.append(graph)
        bufs.append((a, out))
    for k, x in ((0, c), (1, d), (0, d), (1, c)):
        a, out = bufs[k]
        for t, name in zip(a, ("q", "k", "v", "qs", "ks", "vs", "q_start", "lens")):
            t.copy_(_t(x[name]))
        out.fill_(KEEP)
        g[k].replay()
        torch.cuda.synchronize()
        assert np.array_equal(out.float().cpu().numpy(), want_c if x is c else want_d)
    # both graphs at once on two streams
    s2 = torch.cuda.Stream()
    for a, out in bufs:
        out.fill_(KEEP)
    torch.cuda.synchronize()
    for st, graph in ((s, g[0]), (s2, g[1])):
        with torch.cuda.stream(st):
            graph.replay()
    torch.cuda.synchronize()
    assert np.array_equal(bufs[0][1].float().cpu().numpy(), want_d)
    assert np.array_equal(bufs[1][1].float().cpu().numpy(), want_c)


def test_two_streams_at_once():
    F = fa3()
    rng = np.random.default_rng(15)
    cs = [_case(rng, 16, 2, [1, 20], [3000, 900], 64) for _ in range(2)]
    want = [_run(F, c) for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    args = [[_t(c[k]) for k in ("q", "k", "v", "qs", "ks", "vs", "q_start", "lens")] + [_t(c["table"])] for c in cs]
    outs = [torch.full(c["q"].shape, KEEP, dtype=torch.bfloat16, device="cuda") for c in cs]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, a, o in zip(streams, args, outs):
            F.prefill_attn_gqa_paged(*a, SM, out=o, stream=s)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert np.array_equal(o.float().cpu().numpy(), w)


def test_pool_past_32_bit_offsets():
    F = fa3()
    c = _case(np.random.default_rng(16), 8, 8, [2], [100], 64, behind=0)
    num = (1 << 32) // (8 * 128 * 64) + 40
    big = [torch.zeros(num, 64, 8, 128, dtype=torch.int8, device="cuda") for _ in range(2)]
    table = np.array([[num - 1, num - 7, 0]], np.int32)
    for p, x in zip(big, (c["k"], c["v"])):
        p[num - 1], p[num - 7] = _t(x[c["table"][0, 0]]), _t(x[c["table"][0, 1]])
    out = F.prefill_attn_gqa_paged(_t(c["q"]), *big, _t(c["qs"]), _t(c["ks"]), _t(c["vs"]), _t(c["q_start"]),
                                   _t(c["lens"]), _t(table), SM)
    _gate(out.float().cpu().numpy(), _ref(c), c, "large pool")


def test_a_layer_as_it_is_served():
    """Calibrate on norm_rope's activations, append a prompt and then single tokens to the paged cache, attend
    to it, and cross-attend: every step against the oracle on the codes the step before left."""
    F = fa3()
    rng = np.random.default_rng(17)
    Hq, Hkv, D, page, eps = 8, 2, 128, 16, 1e-6
    prompts, steps = [40, 9], 3
    cs = F.rope_table(64, D)
    inv = 10000.0 ** (-np.arange(0, D, 2) / D)
    ang = np.arange(64)[:, None] * inv
    np.testing.assert_allclose(cs.cpu().numpy(), np.concatenate([np.cos(ang), np.sin(ang)], 1), atol=2.0 ** -24)
    w = [W.bf16_round(1 + 0.2 * rng.standard_normal(D).astype(np.float32)) for _ in range(2)]
    act = lambda n: W.bf16_round(W.student_t(rng, (n, Hq + 2 * Hkv, D), 4, 1.0))  # noqa: E731
    # calibration
    x = act(64)
    q, k = F.norm_rope(bf16_dev(x[:, :Hq]), bf16_dev(x[:, Hq:Hq + Hkv]), cs, torch.arange(64, dtype=torch.int32).cuda(),
                       bf16_dev(w[0]), bf16_dev(w[1]), eps)
    scales = []
    for y, H in ((q, Hq), (k, Hkv), (bf16_dev(x[:, Hq + Hkv:]), Hkv)):
        mn, mx = (torch.full((H,), s * float("inf"), device="cuda") for s in (1, -1))
        F.calibrate_perhead(y.transpose(0, 1).contiguous().reshape(H, -1), 0.9999, mn, mx)
        scales.append(F.qparams(mn, mx))
    num = 12
    pools = [torch.zeros(num, page, Hkv, D, dtype=torch.int8, device="cuda") for _ in range(2)]
    table = torch.from_numpy(rng.permutation(num)[:8].reshape(2, 4).astype(np.int32)).cuda()
    have = [0, 0]
    for ql in [prompts] + [[1, 1]] * steps:
        q_start = np.concatenate([[0], np.cumsum(ql)]).astype(np.int32)
        have = [h + n for h, n in zip(have, ql)]
        lens = np.array(have, np.int32)
        x = act(int(q_start[-1]))
        xd, before = bf16_dev(x), [p.cpu().numpy() for p in pools]
        q8 = F.rope_append_gqa_paged(xd[:, :Hq], xd[:, Hq:Hq + Hkv], xd[:, Hq + Hkv:], cs, *scales, *pools, table,
                                     _t(q_start), _t(lens), bf16_dev(w[0]), bf16_dev(w[1]), eps)
        out = F.prefill_attn_gqa_paged(q8, *pools, *scales, _t(q_start), _t(lens), table, SM)
        sc = [s.cpu().numpy() for s in scales]
        rq, rk, rv = O.rope_append_paged(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], *w, eps, cs.cpu().numpy(), False,
                                         *sc, np.zeros((len(x), Hq, D), np.int8), *before, table.cpu().numpy(),
                                         q_start, lens)
        assert np.array_equal(q8.cpu().numpy(), rq)
        assert all(np.array_equal(p.cpu().numpy(), r) for p, r in zip(pools, (rk, rv)))
        kv = [[O.gather_paged(r, table.cpu().numpy(), page, lens)[b, :n] for b, n in enumerate(lens)] for r in (rk, rv)]
        ref = O.packed_attention(rq, *kv, *sc, q_start, lens, SM, True, np.zeros(rq.shape))
        case = dict(q=rq, k=rk, qs=sc[0], ks=sc[1], vs=sc[2], lens=lens)
        _gate(out.float().cpu().numpy(), ref, case, f"layer step {ql}")
    # cross attention of the last rows to states written by quantize_append
    states = W.bf16_round(W.student_t(rng, (2, 25, Hkv, D), 4, 1.0))
    ck, cv = (torch.zeros(2, 25, Hkv, D, dtype=torch.int8, device="cuda") for _ in range(2))
    for cache, s in ((ck, scales[1]), (cv, scales[2])):
        F.quantize_append(bf16_dev(states), s, cache, torch.zeros(2, dtype=torch.int32, device="cuda"))
    enc = np.array([25, 11], np.int32)
    out = F.cross_attn_gqa(q8, ck, cv, *scales, _t(q_start), _t(enc), SM)
    kv = [[x.cpu().numpy()[b, :n] for b, n in enumerate(enc)] for x in (ck, cv)]
    ref = O.packed_attention(rq, *kv, *sc, q_start, enc, SM, False, np.zeros(rq.shape))
    case = dict(q=rq, k=ck.cpu().numpy(), qs=sc[0], ks=sc[1], vs=sc[2], lens=enc)
    _gate(out.float().cpu().numpy(), ref, case, "cross step")


def test_rows_shared_by_a_falling_q_start():
    # every second sequence would have all rows: more rows than there are, so no plan and no row written
    F = fa3()
    for B in (4, 80):
        c = _case(np.random.default_rng(22), 8, 2, [30] + [0] * (B - 1), [50] * B, 16)
        c["q_start"] = np.asarray(([0, 30] * B)[:B + 1], np.int32)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = _run(F, c, err)
        assert int(err.item()) == F.FA3_DEVERR_LENS
        assert np.all(got == KEEP)


def test_two_calls_in_one_graph():
    # their workspaces come from one pool, one after the other
    F = fa3()
    rng = np.random.default_rng(23)
    c, d = _case(rng, 16, 2, [1, 20], [1800, 400], 64), _case(rng, 8, 4, [5, 1], [900, 2500], None)
    want = [_run(F, c), _run(F, d)]
    a, b = ([_t(x[k]) for k in ("q", "k", "v", "qs", "ks", "vs", "q_start", "lens")] for x in (c, d))
    table = _t(c["table"])
    outs = [torch.full(x["q"].shape, KEEP, dtype=torch.bfloat16, device="cuda") for x in (c, d)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        F.prefill_attn_gqa_paged(*a, table, SM, out=outs[0])
        F.cross_attn_gqa(*b, SM, out=outs[1])
    for _ in range(3):
        for o in outs:
            o.fill_(KEEP)
        graph.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert np.array_equal(o.float().cpu().numpy(), w)


def test_calls_that_are_refused():
    F = fa3()
    c = _case(np.random.default_rng(24), 8, 2, [3, 2], [20, 30], 16, behind=0)
    q, k, v, qs, ks, vs, start, lens = (_t(c[x]) for x in ("q", "k", "v", "qs", "ks", "vs", "q_start", "lens"))
    good = dict(q=q, k=k, v=v, q_scale=qs, k_scale=ks, v_scale=vs, q_start=start, kv_lens=lens, block_table=_t(c["table"]),
                softmax_scale=SM)
    F.prefill_attn_gqa_paged(**good)
    need = F.chunk_workspace_size(5, 2, 8, 2, 128)
    bads = [(dict(q=q.float()), TypeError), (dict(q=q[:, :, :64]), ValueError), (dict(q=q[:, :7].contiguous(), q_scale=qs[:7]), F.FA3Error),
            (dict(q=q[:, ::2]), ValueError), (dict(v=v[:1]), ValueError), (dict(k=k.cpu()), TypeError), (dict(q_scale=qs[:2]), ValueError),
            (dict(k_scale=ks.double()), TypeError), (dict(q_start=start[:2]), ValueError), (dict(kv_lens=lens[:0]), ValueError),
            (dict(block_table=_t(c["table"])[:1]), ValueError), (dict(softmax_scale=0.0), F.FA3Error),
            (dict(softmax_scale=float("nan")), F.FA3Error), (dict(out=torch.zeros(5, 8, 128, device="cuda")), TypeError),
            (dict(out=torch.zeros(4, 8, 128, dtype=torch.bfloat16, device="cuda")), ValueError),
            (dict(workspace=torch.zeros(need - 1, dtype=torch.uint8, device="cuda")), F.FA3Error),
            (dict(workspace=torch.zeros(need + 1, dtype=torch.uint8, device="cuda")[1:]), F.FA3Error),
            (dict(workspace=torch.zeros(need, dtype=torch.uint8)), ValueError)]
    for bad, error in bads:
        with pytest.raises(error):
            F.prefill_attn_gqa_paged(**{**good, **bad})
    half = dict(k=k[..., :64].contiguous(), v=v[..., :64].contiguous(), q=q[..., :64].contiguous())
    with pytest.raises(F.FA3Error):                                           # head size 128 alone
        F.prefill_attn_gqa_paged(**{**good, **half})
    e = torch.zeros(2, 7, 2, 128, dtype=torch.int8, device="cuda")
    F.cross_attn_gqa(q, e, e, qs, ks, vs, start, lens * 0, SM)
    for k2, v2 in ((e[:1], e[:1]), (e, e[:, :6]), (e[:, :0], e[:, :0])):
        with pytest.raises((ValueError, F.FA3Error)):
            F.cross_attn_gqa(q, k2, v2, qs, ks, vs, start, lens * 0, SM)


def test_host_threads_on_one_stream():
    # All threads have the same current stream, so their calls share a workspace: the kernels of one call, which hand their
    # partial results on through it, stay together.  Batches of different sizes, and the decode call's own split.
    F = fa3()
    rng = np.random.default_rng(28)
    cs = [_case(rng, 16, 2, [1, 20], [3000, 900], 64), _case(rng, 8, 4, [5, 1, 70], [900, 2500, 300], 16), _case(rng, 8, 2, [3, 1], [2000, 64], None),
          _case(rng, 16, 2, [1, 1], [3000, 900], 64, behind=0), _case(rng, 8, 8, [1, 1, 1], [1200, 2, 2900], 32, behind=0)]
    args = [[_t(c[k]) for k in ("q", "k", "v", "qs", "ks", "vs", "q_start", "lens")] for c in cs]
    tables = [None if c["page"] is None else _t(c["table"]) for c in cs]

    def call(i):
        if cs[i]["page"] is None:
            return F.cross_attn_gqa(*args[i], SM)
        if i < 3:
            return F.prefill_attn_gqa_paged(*args[i], tables[i], SM)
        return F.decode_attn_gqa_paged(*args[i][:6], args[i][7], tables[i], SM)
    want = [call(i) for i in range(len(cs))]
    torch.cuda.synchronize()
    got, failed = [[] for _ in cs], []

    def run(i):
        try:
            for _ in range(150):
                got[i].append(call(i))
        except Exception as e:  # noqa: BLE001
            failed.append(e)
    interval = sys.getswitchinterval()
    sys.setswitchinterval(1e-6)
    try:
        threads = [threading.Thread(target=run, args=(i,)) for i in range(len(cs))]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    finally:
        sys.setswitchinterval(interval)
    torch.cuda.synchronize()
    assert not failed, failed
    for i, w in enumerate(want):
        assert all(torch.equal(o, w) for o in got[i]), f"batch {i}: {sum(not torch.equal(o, w) for o in got[i])} of 150 differ"


def _exact(c, values=None):
    """The packed attention of the case in float64, a sequence and KV head at a time; values in place of c's v."""
    out = np.full(c["q"].shape, KEEP)
    Hkv = c["k"].shape[2]
    G = c["q"].shape[1] // Hkv
    v_all = c["v"] if values is None else values
    for b, kv in enumerate(c["lens"]):
        s, e = int(c["q_start"][b]), int(c["q_start"][b + 1])
        t = np.arange(kv)
        at = (b, t) if c["page"] is None else (c["table"][b, t // c["page"]], t % c["page"])
        for g in range(Hkv if e > s else 0):
            q = c["q"][s:e, g * G:(g + 1) * G].reshape(-1, 128).astype(np.float64)
            x = q @ c["k"][at][:, g].T.astype(np.float64)
            x *= (np.tile(c["qs"][g * G:(g + 1) * G], e - s).astype(np.float64) * float(c["ks"][g]) * SM)[:, None]
            if c["page"] is not None:
                x[t[None] > (kv - (e - s) + np.repeat(np.arange(e - s), G))[:, None]] = -np.inf
            x = np.exp(x - x.max(1, keepdims=True))
            y = (x @ v_all[at][:, g].astype(np.float64)) / x.sum(1, keepdims=True) * float(c["vs"][g])
            out[s:e, g * G:(g + 1) * G] = y.reshape(e - s, G, 128)
    return out


def _tail_case(T, rows, weight, page, Hq, B):
    """B sequences over the same pages: one key that takes the weight 1 and T - 1 of weight 2^-weight each; values 0 and
    +-100 or so.  (With a unit to each SM no key is shared out, so one running maximum sees them all.)"""
    rng = np.random.default_rng([26, T, rows])
    mp = -(-T // page)
    c = dict(q=np.full((B * rows, Hq, 128), 64, np.int8), q_start=np.arange(0, B * rows + 1, rows, dtype=np.int32),
             lens=np.full(B, T, np.int32), page=page, k=np.zeros((mp, page, 1, 128), np.int8),
             table=np.broadcast_to(rng.permutation(mp).astype(np.int32), (B, mp)), qs=np.full(Hq, 0.01, np.float32),
             ks=np.full(1, weight / (128 * 64 * 100 * 0.01 * SM * 1.4426950408889634), np.float32),
             vs=np.full(1, 0.02, np.float32))
    value = rng.integers(90, 110, 128).astype(np.int8) * rng.choice([-1, 1], 128).astype(np.int8)
    c["v"] = np.broadcast_to(value, c["k"].shape).copy()
    sink = (c["table"][0, 70 // page], 70 % page)
    c["k"][sink], c["v"][sink] = 100, 0
    return c


@pytest.mark.parametrize("T,rows,weight,page,Hq,units", [
    (131072, 1, 25.2, 64, 8, 1), (131072, 1, 24.6, 64, 8, 1), (131072, 1, 26.9, 7, 2, 1), (100001, 20, 24.6, 64, 8, 1),
    (131072, 3, 28.0, 128, 128, 2), (20001, 1, 22.0, 48, 5, 1), (1 << 20, 1, 27.5, 64, 2, 1)])
def test_long_tails_of_small_weights(T, rows, weight, page, Hq, units):
    """A weight is off by 2^-11 of itself (fp16), or by 2^-32 of the largest (fp16's subnormals, half of 2^-24 against a
    largest of 2^7 or more), by the float32 score, |s| log2 units, 2^-22 |s|, and by the exponential, 2^-22; the sum of
    the weights counts them before the rounding.  So the output is off by those shares of the weighted mean of |v|, by
    T 2^-32 of max|v|, and by half a bf16 step."""
    F = fa3()
    B = torch.cuda.get_device_properties(0).multi_processor_count // units
    c = _tail_case(T, rows, weight, page, Hq, B)
    one = dict(c, q=c["q"][:rows], q_start=c["q_start"][:2], lens=c["lens"][:1])
    got, ref, mean = _run(F, c), _exact(one), np.abs(_exact(one, np.abs(c["v"])))
    tol = 2.0 ** -8 * np.abs(ref) * (1 + 2.0 ** -8) + (2.0 ** -11 + 2.0 ** -22 * (weight + 2) + 2.0 ** -22) * mean \
        + T * 2.0 ** -32 * 127 * float(c["vs"].max())
    d = np.abs(got.reshape((B,) + ref.shape) - ref)
    print(f"{T} keys of 2^-{weight}: {float((d / tol).max()):.3f} of the tolerance, largest output {float(np.abs(ref).max()):.2e}, "
          f"error {float(d.max()):.2e}")
    assert np.all(d <= tol)


@pytest.mark.parametrize("scale", [1.0, 30.0, 100.0])
@pytest.mark.parametrize("page", [64, 7, None])
def test_very_large_scores(scale, page):
    """Scores of up to 2^17 code products times 0.013 to 127 log2 units, 2^24 in all: the largest weights stay within fp16's
    range.  The reference of the weights is rounded up twice, by 2 units at most, so the largest is 2^3 or more and the others
    are off by 2^-28 of it, beside 2^-11 and, for five roundings of the factor, 2^-21 of their distance x from the largest,
    x 2^-x < 1 of it."""
    F = fa3()
    c = _case(np.random.default_rng(29), 8, 2, [1, 40, 3], [500, 300, 700], page, behind=0)
    c["qs"][:], c["ks"][:] = np.float32(0.1 * scale), np.float32(scale)
    got, ref, mean = _run(F, c), _exact(c), np.abs(_exact(c, np.abs(c["v"])))
    tol = 2.0 ** -8 * np.abs(ref) * (1 + 2.0 ** -8) + (2.0 ** -11 + 2.0 ** -21) * mean + 700 * 2.0 ** -28 * 127 * float(c["vs"].max())
    assert np.all(np.isfinite(got)) and np.all(np.abs(got - ref) <= tol), float((np.abs(got - ref) / tol).max())


@pytest.mark.parametrize("start", [[0, 9, 4, 39], [0, 4000, 9, 39], [5, 0, 9, 39], [0, 20, 39, 30]])
@pytest.mark.parametrize("empty", [0, 31, 40])
@pytest.mark.parametrize("page", [16, None])
def test_falling_q_start_with_room_behind(start, empty, page):
    # sequences that share rows though all their rows together are fewer than n: no row is written, also where the fall is beyond
    # the sequences that a warp looks at first, or at their edge
    F = fa3()
    c = _case(np.random.default_rng(38), 8, 2, [4, 5, 30] + [0] * empty, [50, 60, 70] + [1] * empty, page, behind=25)
    c["q_start"] = np.concatenate([np.full(empty, start[0], np.int32), np.asarray(start, np.int32)])
    c["lens"] = np.concatenate([np.ones(empty, np.int32), np.array([50, 60, 70], np.int32)])
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = _run(F, c, err)
    assert c["q"].shape[0] == 64 and int(err.item()) == F.FA3_DEVERR_LENS
    assert np.all(got == KEEP)


@pytest.mark.parametrize("Hq,Hkv,q_lens,kv_lens,page", [
    (16, 2, [1], [9001], 48), (16, 2, [5], [9001], 48), (16, 2, [20], [9001], 7), (8, 8, [1, 1, 1], [4096, 777, 64], 64),
    (16, 2, [1, 260, 1, 1], [3000, 1300, 100, 700], 64), (35, 7, [5, 1, 3], [6001, 900, 64], 48), (32, 8, [448, 60], [2048, 300], None),
    (16, 16, [1, 1, 1], [1500, 64, 900], None)])
def test_relative_rms_of_long_contexts(Hq, Hkv, q_lens, kv_lens, page):
    # outputs that are means over many keys are small beside max|v|: the project's bar on the relative RMS
    F = fa3()
    rng = np.random.default_rng([27, Hq, q_lens[0], kv_lens[0]])
    c = _case(rng, Hq, Hkv, q_lens, kv_lens, page, behind=0)
    got, ref = _run(F, c), _exact(c)
    for b in range(len(q_lens)):
        s, e = c["q_start"][b], c["q_start"][b + 1]
        assert_attn_close(got[s:e], ref[s:e], True, f"{kv_lens[b]} keys, {e - s} rows")
        # A head alone: the rounding of the output is up to 2^-8 of each value (and 2^-8 / sqrt 3 on average where
        # all lie just above powers of two, which is beyond the bar), the weights' 2^-11 in product and sum.
        for h in range(Hq):
            _, rms = attn_errors(got[s:e, h], ref[s:e, h])
            assert rms <= 2.0 ** -8 + 2.0 ** -10, f"{kv_lens[b]} keys, {e - s} rows, head {h}: relative RMS {rms:.3e}"
