"""GPU parity of the attention-input calls: norm_rope (bf16 / float32 results) and rope_append_gqa_paged
(INT8 codes into the paged cache), against the float64 oracle."""
import sys

import numpy as np
import pytest
import torch

import workloads as W
from helpers import bf16_dev, fa3
from oracle import fa3_oracle as O

pytestmark = pytest.mark.gpu
EPS = 1e-6


def _t(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _table(n, rot):
    inv = 10000.0 ** (-np.arange(0, rot, 2) / rot)
    a = np.arange(n)[:, None] * inv
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def _values(rng, shape):
    # heavy-tailed values of mixed head magnitudes, bf16-exact
    x = W.student_t(rng, shape, 4, W.log_uniform(rng, 0.05, 5.0, shape[:-2] + (shape[-2], 1)))
    return W.bf16_round(x)


def _check(got, y, m, f32):
    # float32 arithmetic: the sum of squares is at most 13 roundings deep (halved by the root), then mean, eps,
    # root, reciprocal, two products, one rotation product and one fma: below 16 * 2^-24 of the terms; a bf16
    # result adds half a step, 2^-8 of the value.
    tol = 2.0 ** -20 * m + (0 if f32 else 2.0 ** -8 * np.abs(y)) + 1e-38
    d = np.abs(got.double().cpu().numpy() - y)
    assert np.all(np.isfinite(d))
    assert np.all(d <= tol), float((d / tol).max())


@pytest.mark.parametrize("D,rot,interleaved", [(128, 128, False), (128, 64, True), (64, 64, True), (80, 32, False),
                                               (96, 96, True), (192, 64, False), (256, 256, False), (8, 8, True),
                                               (128, 8, False), (72, 56, False)])
@pytest.mark.parametrize("norm,f32", [(True, False), (False, True)])
def test_norm_rope(D, rot, interleaved, norm, f32):
    F = fa3()
    rng = np.random.default_rng([D, rot])
    n, Hq, Hkv, L = 37, 5, 3, 501
    x = _values(rng, (n, Hq + 2 * Hkv, D))
    wq, wk = (W.bf16_round(1 + 0.3 * rng.standard_normal(D).astype(np.float32)) for _ in range(2))
    pos = rng.integers(0, L, n).astype(np.int32)
    pos[:3] = [0, L - 1, 0]
    cs = _table(L, rot)
    xd = bf16_dev(x)
    q, k = F.norm_rope(xd[:, :Hq], xd[:, Hq:Hq + Hkv], _t(cs), _t(pos), bf16_dev(wq) if norm else None,
                       bf16_dev(wk) if norm else None, EPS, interleaved,
                       out_dtype=torch.float32 if f32 else torch.bfloat16)
    for got, sl, w in ((q, slice(0, Hq), wq), (k, slice(Hq, Hq + Hkv), wk)):
        _check(got, *O.norm_rope(x[:, sl], w if norm else None, EPS, cs, pos, interleaved), f32)


@pytest.mark.parametrize("what", ["norm_only", "rope_only", "q_only", "copy"])
def test_parts_of_the_pass(what):
    F = fa3()
    rng = np.random.default_rng(5)
    x = _values(rng, (9, 4, 128))
    w = W.bf16_round(1 + 0.3 * rng.standard_normal(128).astype(np.float32))
    pos = rng.integers(0, 64, 9).astype(np.int32)
    cs = _table(64, 128)
    use_w, use_t = what in ("norm_only", "q_only"), what in ("rope_only", "q_only")
    xd, wd = bf16_dev(x), bf16_dev(w)
    k = None if what == "q_only" else xd[:, 3:]
    q, ko = F.norm_rope(xd[:, :3], k, _t(cs) if use_t else None, _t(pos) if use_t else None, wd if use_w else None,
                        wd if use_w and k is not None else None, EPS)
    assert (ko is None) == (k is None)
    for got, sl in ((q, slice(0, 3)), (ko, slice(3, 4))):
        if got is not None:
            _check(got, *O.norm_rope(x[:, sl], w if use_w else None, EPS, cs if use_t else None, pos, False), False)
            if what == "copy":
                assert torch.equal(got, xd[:, sl])


def test_strided_transposed_and_in_place():
    F = fa3()
    rng = np.random.default_rng(6)
    B, S, H, D = 3, 21, 4, 128
    x = _values(rng, (B, S, H, D))
    pos = np.stack([np.arange(S) + 7 * b for b in range(B)]).astype(np.int32)
    cs = _table(64, 128)
    y, m = O.norm_rope(x.reshape(B * S, H, D), None, EPS, cs, pos.ravel(), False)
    xd = bf16_dev(x)
    out = torch.zeros(B, H, S, D, dtype=torch.bfloat16, device="cuda")
    F.norm_rope(xd, None, _t(cs), _t(pos), q_out=out.transpose(1, 2))
    _check(out.transpose(1, 2).reshape(B * S, H, D), y, m, False)
    heads_first = xd.transpose(1, 2).contiguous().transpose(1, 2)          # strided input
    q, _ = F.norm_rope(heads_first, None, _t(cs), _t(pos))
    assert torch.equal(q, out.transpose(1, 2))
    F.norm_rope(xd, None, _t(cs), _t(pos), q_out=xd)                        # in place
    assert torch.equal(xd, out.transpose(1, 2))
    # rotating the rope part alone of wider rows (an absorbed MLA query), the rest untouched
    wide = bf16_dev(np.concatenate([x, x], -1))
    keep = wide.clone()
    F.norm_rope(wide[..., D:], None, _t(cs), _t(pos), q_out=wide[..., D:])
    assert torch.equal(wide[..., :D], keep[..., :D]) and torch.equal(wide[..., D:], out.transpose(1, 2))


def test_bad_positions_skip_the_token():
    F = fa3()
    rng = np.random.default_rng(7)
    x = _values(rng, (4, 2, 64))
    cs = _table(10, 64)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((4, 2, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    pos = np.array([3, 10, -1, 9], np.int32)
    F.norm_rope(bf16_dev(x), None, _t(cs), _t(pos), q_out=out, dev_err=err)
    assert int(err.item()) == F.FA3_DEVERR_POS
    assert bool((out[1:3] == 9.0).all())
    y, m = O.norm_rope(x[[0, 3]], None, EPS, cs, pos[[0, 3]], False)
    _check(out[[0, 3]], y, m, False)


def test_calibrate_takes_what_norm_rope_lays_out():
    # norm_rope -> (B, H, S, D) -> calibrate -> qparams: the range of the very values it wrote
    F = fa3()
    rng = np.random.default_rng(8)
    B, S, H, D = 2, 40, 3, 128
    x = _values(rng, (B, S, H, D))
    w = W.bf16_round(1 + 0.3 * rng.standard_normal(D).astype(np.float32))
    pos = np.tile(np.arange(S, dtype=np.int32), (B, 1))
    out = torch.empty(B, H, S, D, dtype=torch.bfloat16, device="cuda")
    F.norm_rope(bf16_dev(x), None, _t(_table(S, D)), _t(pos), bf16_dev(w), q_out=out.transpose(1, 2))
    mn, mx = (torch.full((H,), s * float("inf"), device="cuda") for s in (1, -1))
    F.calibrate_perhead(out, 0.9999, mn, mx)
    scale = F.qparams(mn, mx).cpu().numpy()
    ref = O.qparams(*O.calibrate([out.float().cpu().numpy()], 0.9999))
    assert np.array_equal(scale, ref)


# --------------------------------------------------------------------- append
def _append_case(rng, Hq, Hkv, D, rot, page, q_lens, kv_lens, norm, lead=0, behind=2):
    B = len(q_lens)
    q_start = (lead + np.concatenate([[0], np.cumsum(q_lens)])).astype(np.int32)
    n = int(q_start[-1]) + behind
    mp = -(-max(kv_lens) // page) + 1
    num = B * mp + 3
    table = rng.permutation(num)[:B * mp].reshape(B, mp).astype(np.int32)
    for b, kv in enumerate(kv_lens):
        table[b, -(-kv // page):] = -1                                      # past the context: never read
    x = _values(rng, (n, Hq + 2 * Hkv, D))
    sc = (np.abs(x).max(axis=(0, 2)) / 127 * rng.uniform(0.3, 1.0, Hq + 2 * Hkv)).astype(np.float32)
    if norm:
        sc[:Hq + Hkv] = np.float32(4.0 / 127)
    if Hq:
        sc[0] = 0.0                                                         # an all-zero head's scale
    pools = [rng.integers(-127, 128, (num, page, Hkv, D)).astype(np.int8) for _ in range(2)]
    w = [W.bf16_round(1 + 0.3 * rng.standard_normal(D).astype(np.float32)) if norm else None for _ in range(2)]
    return dict(x=x, Hq=Hq, Hkv=Hkv, D=D, cs=_table(max(kv_lens) + 1, rot) if rot else None, q_start=q_start,
                kv_lens=np.asarray(kv_lens, np.int32), table=table, sc=sc, pools=pools, w=w, n=n)


def _run_append(F, c, interleaved, err=None, q=True):
    Hq, Hkv = c["Hq"], c["Hkv"]
    xd = bf16_dev(c["x"])
    kp, vp = (_t(p) for p in c["pools"])
    q_out = torch.full((c["n"], Hq, c["D"]), 77, dtype=torch.int8, device="cuda") if q else None
    w = [None if a is None else bf16_dev(a) for a in c["w"]]
    sc = _t(c["sc"])
    F.rope_append_gqa_paged(xd[:, :Hq] if q else None, xd[:, Hq:Hq + Hkv], xd[:, Hq + Hkv:],
                            None if c["cs"] is None else _t(c["cs"]), sc[:Hq].clone() if q else None,
                            sc[Hq:Hq + Hkv].clone(), sc[Hq + Hkv:].clone(), kp, vp, _t(c["table"]), _t(c["q_start"]),
                            _t(c["kv_lens"]), w[0] if q else None, w[1], EPS, interleaved, q_out=q_out, dev_err=err)
    torch.cuda.synchronize()
    return [None if a is None else a.cpu().numpy() for a in (q_out, kp, vp)]


def _ref_append(c, interleaved, q=True):
    Hq, Hkv, x, sc = c["Hq"], c["Hkv"], c["x"], c["sc"]
    q_out = np.full((c["n"], Hq, c["D"]), 77, np.int8)
    return O.rope_append_paged(x[:, :Hq] if q else None, x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], c["w"][0], c["w"][1], EPS,
                               c["cs"], interleaved, sc[:Hq], sc[Hq:Hq + Hkv], sc[Hq + Hkv:], q_out, *c["pools"],
                               c["table"], c["q_start"], c["kv_lens"])


def _same(got, ref):
    for g, r, name in zip(got, ref, ("q", "k", "v")):
        if r is not None:
            assert np.array_equal(g, r), f"{name}: {(g != r).sum()} of {g.size} codes differ"


@pytest.mark.parametrize("Hq,Hkv,D,rot,page,interleaved,norm", [
    (8, 2, 128, 128, 64, False, True), (8, 2, 128, 128, 64, False, False), (5, 1, 128, 64, 7, True, True),
    (3, 3, 80, 32, 1, True, False), (6, 2, 256, 256, 16, False, True), (1, 1, 64, 64, 24, True, False),
    (7, 5, 96, 96, 100, False, True), (4, 4, 128, 0, 16, False, False), (4, 4, 192, 0, 16, False, True)])
def test_append_bit_exact(Hq, Hkv, D, rot, page, interleaved, norm):
    F = fa3()
    rng = np.random.default_rng([Hq, D, page])
    c = _append_case(rng, Hq, Hkv, D, rot, page, [1, 0, 37, 5, 1], [130, 9, 37, 64, 1], norm, lead=1)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    _same(_run_append(F, c, interleaved, err), _ref_append(c, interleaved))
    assert int(err.item()) == 0


def test_append_without_q():
    F = fa3()
    c = _append_case(np.random.default_rng(11), 2, 3, 128, 128, 16, [3, 20], [50, 20], True)
    c["w"][0] = None
    _same(_run_append(F, c, False, q=False), _ref_append(c, False, q=False))


def test_append_ties_and_clamps():
    # power-of-two scales put many quotients exactly on half steps (position 0 turns nothing), far values clamp
    F = fa3()
    rng = np.random.default_rng(12)
    c = _append_case(rng, 4, 2, 128, 128, 16, [1, 1, 30], [1, 1, 30], False)
    c["x"] = W.bf16_round((rng.integers(-400, 401, c["x"].shape) / 64).astype(np.float32))
    c["x"][2, 0, :] = np.float32(2.0 ** 100)
    c["sc"][:] = np.float32(1 / 32)
    c["sc"][1] = np.float32(2.0 ** -120)                                    # beyond the exact-product range
    c["sc"][2] = np.float32(1e-41)                                          # a subnormal scale
    _same(_run_append(F, c, False), _ref_append(c, False))


def test_append_near_ties_are_decided_exactly():
    # 2.6 million rotated and normed codes: a few of them lie within float32 rounding of a half step
    F = fa3()
    rng = np.random.default_rng(13)
    for norm in (False, True):
        c = _append_case(rng, 16, 4, 128, 128, 64, [500, 41], [500, 600], norm)
        _same(_run_append(F, c, norm), _ref_append(c, norm))


def test_append_many_sequences():
    # more sequences than one 32-way step, then than two, finds
    F = fa3()
    for B in (33, 1100):
        rng = np.random.default_rng(B)
        ql = rng.integers(0, 3, B)
        ql[-1] = 1
        c = _append_case(rng, 1, 1, 64, 64, 4, list(ql), list(ql + rng.integers(1, 9, B)), False)
        _same(_run_append(F, c, False), _ref_append(c, False))


def test_append_errors_skip_what_is_wrong():
    F = fa3()
    rng = np.random.default_rng(14)
    c = _append_case(rng, 4, 2, 128, 128, 16, [3, 4, 2, 5], [20, 30, 40, 16], True)
    ref = list(_ref_append(c, False))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def untouched(ref, b):
        s, e = c["q_start"][b], c["q_start"][b + 1]
        ref[0][s:e] = 77
        for j in (1, 2):
            for p in range(c["kv_lens"][b] - (e - s), c["kv_lens"][b]):
                at = (c["table"][b, p // 16], p % 16)
                ref[j][at] = c["pools"][j - 1][at]

    good = c["kv_lens"].copy()
    for bad in (2, 100000, -5):                                              # fewer than the new rows; past T_max
        c["kv_lens"][1] = bad
        got = _run_append(F, c, False, err)
        assert int(err.item()) == F.FA3_DEVERR_LENS
        err.zero_()
        r = [a.copy() for a in ref]
        c["kv_lens"] = good.copy()
        untouched(r, 1)
        _same(got, r)
    table = c["table"].copy()
    c["table"][2, 39 // 16] = c["pools"][0].shape[0]                         # both new tokens of sequence 2
    got = _run_append(F, c, False, err)
    assert int(err.item()) == F.FA3_DEVERR_PAGE
    c["table"] = table
    r = [a.copy() for a in ref]
    untouched(r, 2)
    r[0] = ref[0]
    _same(got, r)
    err.zero_()
    c["cs"] = c["cs"][:39]                                                   # sequence 2's last position has no angle
    got = _run_append(F, c, False, err)
    assert int(err.item()) == F.FA3_DEVERR_POS
    r = [a.copy() for a in ref]
    row, at = c["q_start"][3] - 1, (c["table"][2, 39 // 16], 39 % 16)
    r[0][row] = 77
    for j in (1, 2):
        r[j][at] = c["pools"][j - 1][at]
    _same(got, r)


def test_v_codes_are_those_of_quantize_append_paged():
    F = fa3()
    rng = np.random.default_rng(15)
    x = _values(rng, (2, 6, 3, 128))
    sc = _t((np.abs(x).max(axis=(0, 1, 3)) / 127).astype(np.float32))
    table = _t(np.array([[2, 0], [1, 3]], np.int32))
    a, b, k = (torch.zeros(4, 8, 3, 128, dtype=torch.int8, device="cuda") for _ in range(3))
    F.quantize_append_paged(bf16_dev(x), sc, a, table, _t(np.array([4, 10], np.int32)))
    xd = bf16_dev(x).reshape(12, 3, 128)
    F.rope_append_gqa_paged(None, xd, xd, None, None, sc, sc, k, b, table, _t(np.array([0, 6, 12], np.int32)),
                            _t(np.array([10, 16], np.int32)))
    assert torch.equal(a, b) and torch.equal(a, k)


def test_append_past_32_bit_offsets():
    # a pool of more than 2^32 bytes, written near its end
    F = fa3()
    Hkv, D, page = 8, 128, 64
    num = (1 << 32) // (Hkv * D * page) + 40
    kp, vp = (torch.zeros(num, page, Hkv, D, dtype=torch.int8, device="cuda") for _ in range(2))
    rng = np.random.default_rng(16)
    x = _values(rng, (2, Hkv, D))
    sc = (np.abs(x).max(axis=(0, 2)) / 127).astype(np.float32)
    xd = bf16_dev(x)
    F.rope_append_gqa_paged(None, xd, xd, None, None, _t(sc), _t(sc), kp, vp, _t(np.array([[num - 1]], np.int32)),
                            _t(np.array([0, 2], np.int32)), _t(np.array([page], np.int32)))
    ref = O.quantize(x, sc[None, :, None])
    for p in (kp, vp):
        assert np.array_equal(p[num - 1, page - 2:].cpu().numpy(), ref)
        assert not p[:num - 1].any() and not p[num - 1, :page - 2].any()


def test_streams_and_graphs():
    # a side stream, and captured calls replayed on changed contents: the codes of the plain calls
    F = fa3()
    rng = np.random.default_rng(30)
    cs = [_append_case(rng, 8, 2, 128, 128, 16, [1, 20, 3], kv, True) for kv in ([40, 33, 3], [25, 60, 60])]
    cs[1]["table"] = cs[0]["table"] = np.arange(3 * 6, dtype=np.int32).reshape(3, 6)
    cs[1]["cs"] = cs[0]["cs"] = _table(64, 128)
    cs[1]["pools"] = [np.zeros((24, 16, 2, 128), np.int8) for _ in range(2)]
    cs[0]["pools"] = cs[1]["pools"]
    want = [_ref_append(c, False) for c in cs]
    names = ("x", "q_start", "kv_lens", "sc")
    buf = {n: (bf16_dev if n == "x" else _t)(cs[0][n]) for n in names}
    table, tab = _t(cs[0]["table"]), _t(cs[0]["cs"])
    pools = [_t(p) for p in cs[0]["pools"]]
    w = [bf16_dev(a) for a in cs[0]["w"]]
    cs[1]["w"] = cs[0]["w"]
    want[1] = _ref_append(cs[1], False)
    q_out = torch.full((cs[0]["n"], 8, 128), 77, dtype=torch.int8, device="cuda")
    rows = torch.zeros(cs[0]["n"], 8, 128, dtype=torch.bfloat16, device="cuda")
    pos = torch.arange(cs[0]["n"], dtype=torch.int32, device="cuda")

    def calls(stream=None):
        x, sc = buf["x"], buf["sc"]
        F.rope_append_gqa_paged(x[:, :8], x[:, 8:10], x[:, 10:], tab, sc[:8], sc[8:10], sc[10:], *pools, table,
                                buf["q_start"], buf["kv_lens"], *w, EPS, q_out=q_out, stream=stream)
        F.norm_rope(x[:, :8], None, tab, pos, w[0], eps=EPS, q_out=rows, stream=stream)

    def check(i):
        torch.cuda.synchronize()
        _same([t.cpu().numpy() for t in (q_out, *pools)], want[i])
        y, m = O.norm_rope(cs[i]["x"][:, :8], cs[0]["w"][0], EPS, cs[0]["cs"], np.arange(cs[0]["n"]), False)
        _check(rows, y, m, False)
        for t in (rows, *pools):
            t.zero_()
        q_out.fill_(77)
        torch.cuda.synchronize()

    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    calls(side)
    check(0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for i in (1, 0, 1):
        for n in names:
            buf[n].copy_((bf16_dev if n == "x" else _t)(cs[i][n]))
        graph.replay()
        check(i)


def test_calls_that_are_refused():
    F = fa3()
    rng = np.random.default_rng(31)
    x = bf16_dev(_values(rng, (6, 4, 128)))
    tab, pos = _t(_table(8, 128)), torch.zeros(6, dtype=torch.int32, device="cuda")
    w = bf16_dev(np.ones(128, np.float32))
    for bad, error in ((dict(q=x.float()), TypeError), (dict(cos_sin=tab.double()), TypeError), (dict(pos=None), ValueError),
                       (dict(pos=pos[:5]), ValueError), (dict(pos=pos.long()), TypeError), (dict(q_weight=w[:64]), ValueError),
                       (dict(k_weight=w), ValueError), (dict(k=x[:5]), ValueError), (dict(k=x, k_weight=w), ValueError),
                       (dict(q_out=x[:, :2]), ValueError), (dict(q_out=torch.zeros_like(x, dtype=torch.float16)), TypeError),
                       (dict(q_out=x[:, :1].expand(6, 4, 128)), ValueError), (dict(q=x[..., ::2]), ValueError),
                       (dict(q=x[..., :4]), ValueError), (dict(q=x[..., :12], cos_sin=None, pos=None), F.FA3Error), (dict(eps=-1.0), F.FA3Error), (dict(cos_sin=tab.cpu()), TypeError),
                       (dict(q=x[..., 2:122], cos_sin=tab[:, :120].contiguous()), F.FA3Error)):   # rows off 8 bytes
        with pytest.raises(error):
            F.norm_rope(**{**dict(q=x, k=None, cos_sin=tab, pos=pos), **bad})
    pool = torch.zeros(4, 8, 2, 128, dtype=torch.int8, device="cuda")
    sc, i32 = torch.ones(2, device="cuda"), lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    good = dict(q=x[:, :2], k=x[:, 2:], v=x[:, 2:], cos_sin=tab, q_scale=sc, k_scale=sc, v_scale=sc, k_cache=pool,
                v_cache=pool.clone(), block_table=i32(0, 1)[None], q_start=i32(0, 6), kv_lens=i32(6))
    F.rope_append_gqa_paged(**good)
    for bad, error in ((dict(k=x[:, 1:]), ValueError), (dict(v=x[:5, 2:]), ValueError), (dict(q=x[:, ::2]), ValueError),
                       (dict(q_scale=None), F.FA3Error), (dict(k_scale=sc[:1]), ValueError), (dict(q_start=i32(0)), ValueError),
                       (dict(kv_lens=i32(6).long()), TypeError), (dict(block_table=i32(0, 1)), ValueError),
                       (dict(v_cache=pool[:2]), ValueError), (dict(v_cache=pool.transpose(0, 1)), ValueError),
                       (dict(q_out=torch.zeros(6, 2, 64, dtype=torch.int8, device="cuda")), ValueError),
                       (dict(q=None, q_weight=w), ValueError), (dict(dev_err=i32(0).cpu()), TypeError)):
        with pytest.raises(error):
            F.rope_append_gqa_paged(**{**good, **bad})


@pytest.mark.parametrize("start", [[0, 9, 12, 4, 39], [0, 9, 4, 39, 39], [-3, 4, 9, 39, 39], [0, 4, 9, 4000, 39], [30, 20, 10, 5, 0]])
@pytest.mark.parametrize("empty", [0, 40])
def test_append_q_start_that_falls(start, empty):
    # A row's sequence is searched for, and a start that falls may lead the search to one that begins behind the
    # row: such a row is skipped.  Rows that are written are right for a sequence that holds them, nothing else is written.
    F = fa3()
    rng = np.random.default_rng([36, empty])
    c = _append_case(rng, 2, 1, 64, 64, 8, [9, 3, 1, 26], [9, 3, 1, 40], False, behind=1)
    assert c["n"] == 40
    B = 4 + empty                                                           # sequences without rows in front: the search takes two steps
    c["q_start"] = np.concatenate([np.zeros(empty, np.int32), np.asarray(start, np.int32)])
    c["kv_lens"] = np.concatenate([np.zeros(empty, np.int32), np.array([9, 3, 1, 40], np.int32)])
    c["table"] = np.arange(B * 6, dtype=np.int32).reshape(B, 6)
    c["pools"] = [rng.integers(-127, 128, (B * 6, 8, 1, 64)).astype(np.int8) for _ in range(2)]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    q, k, v = _run_append(F, c, False, err)
    assert int(err.item()) in (0, F.FA3_DEVERR_LENS)
    may = [p.reshape(-1, 64).copy() for p in c["pools"]]
    codes = lambda x, sc: O.quantize64(x, sc)  # noqa: E731
    seen = np.zeros(c["n"], bool)
    for b in range(B):
        q0, q1, kv = int(c["q_start"][b]), int(c["q_start"][b + 1]), int(c["kv_lens"][b])
        if not 0 <= q0 < q1 <= c["n"] or not q1 - q0 <= kv <= 48:
            continue
        for row in range(q0, q1):
            at = np.array([kv - (q1 - row)])
            x = c["x"][row:row + 1]
            y = codes(O.norm_rope(x[:, :2], None, EPS, c["cs"], at, False)[0], c["sc"][:2])[0]
            seen[row] |= np.array_equal(q[row], y)
            k8 = codes(O.norm_rope(x[:, 2:3], None, EPS, c["cs"], at, False)[0], c["sc"][2:3])[0, 0]
            v8 = O.quantize(x[:, 3:], c["sc"][3:][None, :, None])[0, 0]
            place = b * 48 + int(at[0])
            for got, new, keep in ((k, k8, may[0]), (v, v8, may[1])):
                if np.array_equal(got.reshape(-1, 64)[place], new):
                    keep[place] = new
    assert np.all(seen | np.all(q == 77, axis=(1, 2)))
    assert np.array_equal(k.reshape(-1, 64), may[0]) and np.array_equal(v.reshape(-1, 64), may[1])


@pytest.mark.parametrize("start", [[0, 9, 12, 4, 39], [0, 9, 4, 39, 39], [0, 0, -1, 0, 39], [0, 41, 41, 41, 41]])
@pytest.mark.parametrize("empty", [0, 1, 40, 300])
def test_append_reports_every_bad_start(start, empty):
    # also where every row finds a sequence that holds it, or no row looks at the bad one
    F = fa3()
    c = _append_case(np.random.default_rng(37), 2, 1, 64, 64, 8, [9, 3, 1, 26], [9, 3, 1, 40], False, behind=1)
    B = 4 + empty
    c["q_start"] = np.concatenate([np.zeros(empty, np.int32), np.asarray(start, np.int32)])
    c["kv_lens"] = np.concatenate([np.zeros(empty, np.int32), np.full(4, 40, np.int32)])
    c["table"] = np.arange(B * 6, dtype=np.int32).reshape(B, 6)
    c["pools"] = [np.zeros((B * 6, 8, 1, 64), np.int8) for _ in range(2)]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    _run_append(F, c, False, err)
    assert int(err.item()) == F.FA3_DEVERR_LENS


@pytest.mark.parametrize("eps", [0.0, 1e-6])
@pytest.mark.parametrize("D", [64, 80, 128, 192, 256])
def test_append_ties_after_the_norm(D, eps, monkeypatch):
    # Rows of one magnitude, and rows of one value beside zeros: the norm leaves +-w, or +-sqrt(D) w, exactly or (with
    # eps) by a relative eps / (2 x^2) less, which float64 still tells from a half step.  Weights (k + 1/2), and
    # for the rows of one value (k + 1/2) / sqrt(D) where that is a bf16 number, put them on half steps.  The codes are those of
    # float64 arithmetic, with rotation by 0 (position 0) and by the table's angles, and without rotation.
    monkeypatch.setattr(sys.modules[__name__], "EPS", eps)
    F = fa3()
    rng = np.random.default_rng([33, D])
    n, Hq, Hkv = 300, 6, 2
    for rot in (0, 32):
        c = _append_case(rng, Hq, Hkv, D, rot, 16, [n, 1, 1], [n, 1, 3], True)
        H = Hq + 2 * Hkv
        mag = W.bf16_round(np.exp(rng.uniform(np.log(1e-3 if eps == 0 else 300.0), np.log(3e6), (c["n"], H, 1))).astype(np.float32))
        c["x"] = mag * rng.choice([-1.0, 1.0], (c["n"], H, D)).astype(np.float32)
        c["sc"][:] = np.float32(1.0)
        c["sc"][2] = np.float32(4.0)
        c["w"] = [W.bf16_round((rng.integers(0, 60, D) + 0.5).astype(np.float32)) for _ in range(2)]
        if D in (64, 256):
            lone = rng.random((c["n"], H)) < 0.3
            at = rng.integers(0, D, (c["n"], H))
            c["x"][lone] *= (np.arange(D) == at[lone][:, None])
            c["w"] = [W.bf16_round(w / np.where(rng.random(D) < 0.5, 1.0, D ** 0.5).astype(np.float32)) for w in c["w"]]
        _same(_run_append(F, c, rot == 32), _ref_append(c, rot == 32))


def test_k_without_heads_of_q_is_refused():
    # the C call refuses a q without heads; a k_out that nothing writes must not come back
    F = fa3()
    x = bf16_dev(_values(np.random.default_rng(32), (6, 4, 128)))
    for shape in (x, x.reshape(2, 3, 4, 128)):
        with pytest.raises(F.FA3Error):
            F.norm_rope(shape[..., :0, :], shape, None, None)
    q, k = F.norm_rope(x[:0], x[:0, :2], None, None)                        # no tokens: nothing to write
    assert q.shape == (0, 4, 128) and k.shape == (0, 2, 128)


@pytest.mark.parametrize("interleaved", [False, True])
def test_append_codes_of_nan(interleaved, monkeypatch):
    monkeypatch.setattr(sys.modules[__name__], "bf16_dev", lambda a: torch.from_numpy(a).to(torch.bfloat16).cuda())   # NaN too
    # NaN in a weight or an angle, among finite ones: the code of those values is the one that quantize_append gives NaN
    F = fa3()
    rng = np.random.default_rng(39)
    c = _append_case(rng, 4, 2, 128, 64, 16, [30, 1], [30, 9], True)
    c["sc"][0] = c["sc"][1]
    ref = [a.copy() for a in _ref_append(c, interleaved)]
    pool, one = (torch.zeros(1, 1, 1, 8, dtype=torch.int8, device="cuda"), torch.ones(1, device="cuda"))
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    F.quantize_append(torch.full((1, 1, 1, 8), float("nan"), dtype=torch.bfloat16, device="cuda"), one, pool, zero)
    nan = int(pool[0, 0, 0, 0])
    c["w"] = [w.copy() for w in c["w"]]
    c["w"][0][100], c["w"][1][101] = np.nan, np.nan                         # beyond the rotated values: these alone
    c["cs"][5, 3] = np.nan                                                  # position 5: both members of pair 3
    ref[0][:31, :, 100] = nan
    row, pair = (5, (6, 7) if interleaved else (3, 35))                     # sequence 0's token at position 5
    for d in pair:
        ref[0][row, :, d] = nan
        ref[1][c["table"][0, 0], 5, :, d] = nan
    for b, n, kv in ((0, 30, 30), (1, 1, 9)):
        for p in range(kv - n, kv):
            ref[1][c["table"][b, p // 16], p % 16, :, 101] = nan
    _same(_run_append(F, c, interleaved), ref)


def _passes_a_task(tokens, heads, D):
    # heads_per_task of the kernels: passes of 32 / lanes rows that a warp takes of one token
    rows = 4 if D <= 64 else 2 if D <= 128 else 1
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return max(1, min(8, tokens * -(-heads // rows) // (sms * 24)))


# tokens enough for tasks of several passes: 20 + 5 and 35 + 7 heads leave a part of a task and of a pass at the end
@pytest.mark.parametrize("tokens,Hq,Hkv,D,rot,interleaved,norm,passes", [
    (2400, 20, 5, 128, 128, False, True, 8), (2700, 35, 7, 64, 64, True, True, 8), (1300, 20, 5, 256, 128, False, False, 8),
    (1100, 20, 5, 128, 64, True, False, 3), (1700, 35, 7, 80, 32, False, True, 8), (700, 35, 7, 192, 192, True, True, 7)])
def test_norm_rope_tasks_of_several_passes(tokens, Hq, Hkv, D, rot, interleaved, norm, passes):
    F = fa3()
    assert _passes_a_task(tokens, Hq + Hkv, D) >= passes
    rng = np.random.default_rng([34, tokens, D])
    x = _values(rng, (tokens, Hq + Hkv, D))
    w = [W.bf16_round(1 + 0.3 * rng.standard_normal(D).astype(np.float32)) if norm else None for _ in range(2)]
    pos, cs = rng.integers(0, 300, tokens).astype(np.int32), _table(300, rot)
    xd, wd, tab, at = bf16_dev(x), [None if a is None else bf16_dev(a) for a in w], _t(cs), _t(pos)
    want = [O.norm_rope(x[:, sl], a, EPS, cs, pos, interleaved) for sl, a in ((slice(0, Hq), w[0]), (slice(Hq, None), w[1]))]
    for dt in (torch.bfloat16, torch.float32):
        for got, ref in zip(F.norm_rope(xd[:, :Hq], xd[:, Hq:], tab, at, *wd, EPS, interleaved, out_dtype=dt), want):
            _check(got, *ref, dt is torch.float32)
    plain = F.norm_rope(xd[:, :Hq], xd[:, Hq:], tab, at, *wd, EPS, interleaved)
    F.norm_rope(xd[:, :Hq], xd[:, Hq:], tab, at, *wd, EPS, interleaved, q_out=xd[:, :Hq], k_out=xd[:, Hq:])   # in place
    assert torch.equal(xd[:, :Hq], plain[0]) and torch.equal(xd[:, Hq:], plain[1])


@pytest.mark.parametrize("tokens,Hq,Hkv,D,rot,page,interleaved,norm,passes", [
    (2000, 20, 5, 128, 128, 64, False, True, 8), (2300, 35, 7, 64, 64, 16, True, True, 8), (1000, 20, 5, 256, 128, 7, False, False, 8),
    (900, 20, 5, 128, 64, 24, True, False, 3), (1400, 35, 7, 80, 32, 64, False, True, 8), (700, 35, 7, 192, 192, 16, True, True, 8)])
def test_append_tasks_of_several_passes(tokens, Hq, Hkv, D, rot, page, interleaved, norm, passes):
    F = fa3()
    assert _passes_a_task(tokens, Hq + 2 * Hkv, D) >= passes
    rng = np.random.default_rng([35, tokens, D])
    c = _append_case(rng, Hq, Hkv, D, rot, page, [tokens - 44, 1, 0, 43], [tokens, 77, 3, 43], norm)
    c["sc"][[0, 9, Hq - 1, Hq + 3]] = np.float32(0.0)                       # heads of later passes
    c["sc"][[11, Hq + 4]] = np.float32(2.0 ** -120)                         # decided in float64
    _same(_run_append(F, c, interleaved), _ref_append(c, interleaved))
