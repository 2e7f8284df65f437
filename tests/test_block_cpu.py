"""CPU checks of the block-scaled cache's calls: the oracle's own pins, the host-side refusals of the C ABI and those
of the binding."""
import ctypes

import numpy as np
import pytest
import torch

from helpers import fa3
from oracle import fa3_oracle as O

EINVAL, ERANGE, EWORKSPACE = 1, 2, 4
FAKE = ctypes.c_void_p(4096)          # never dereferenced: validation fails first
ODD4 = ctypes.c_void_p(4096 + 4)
ODD8 = ctypes.c_void_p(4096 + 8)


@pytest.fixture(scope="module")
def L():
    return fa3().lib()


# ------------------------------------------------------------------ oracle pins
def test_append_by_hand():
    pool = np.zeros((3, 16, 1, 8), np.int8)
    scale = np.full((3, 1, 1), np.nan, np.float32)
    table = np.array([[2, 0]], np.int32)
    one = np.zeros((1, 1, 8), np.float32)
    one[0, 0, :3] = [127, 0.5, -1.5]
    k, _, ks, _ = O.append_block_paged(one, one, pool, pool, scale, scale, table, [0, 1], [1])
    assert ks[2, 0, 0] == 1 and list(k[2, 0, 0, :3]) == [127, 0, -2]          # half to even
    two = one * 2
    k2, _, ks2, _ = O.append_block_paged(two, two, k, k, ks, ks, table, [0, 1], [2])
    assert ks2[2, 0, 0] == 2 and list(k2[2, 0, 0, :3]) == [64, 0, -1]         # 63.5 -> 64, -1
    assert list(k2[2, 1, 0, :3]) == [127, 0, -2]
    k3, _, ks3, _ = O.append_block_paged(one, one, k2, k2, ks2, ks2, table, [0, 1], [3])
    assert ks3[2, 0, 0] == 2 and np.array_equal(k3[2, :2], k2[2, :2])         # a smaller token changes nothing
    assert np.isnan(ks3[0, 0, 0])


def test_a_block_scale_does_not_depend_on_the_split():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((20, 2, 8)).astype(np.float32)
    pool, scale = np.zeros((4, 16, 2, 8), np.int8), np.zeros((4, 1, 2), np.float32)
    table = np.array([[1, 3]], np.int32)
    whole = O.append_block_paged(x, -x, pool, pool, scale, scale, table, [0, 20], [20])
    step = (pool, pool, scale, scale)
    for t in range(20):
        step = O.append_block_paged(x[t:t + 1], -x[t:t + 1], *step, table, [0, 1], [t + 1])
    assert np.array_equal(whole[2], step[2]) and np.array_equal(whole[3], step[3])
    ref = x.reshape(20, 2, 8)
    got = O.cached_block_values(step[0], step[2], table, 0, 20)
    # written within half a step, and moved by half a step at most for each time that the scale grew (15 at most)
    assert np.all(np.abs(got - ref) <= 8.5 * step[2].max())
    got = O.cached_block_values(whole[0], whole[2], table, 0, 20)
    assert np.all(np.abs(got - ref) <= 0.5001 * whole[2].max())


def test_attention_equals_torch_and_weights_sum_to_the_rows():
    rng = np.random.default_rng(2)
    code = lambda *s: rng.integers(-127, 128, s).astype(np.int8)  # noqa: E731
    k, v = code(4, 16, 2, 128), code(4, 16, 2, 128)
    ks, vs = (rng.uniform(0.001, 0.01, (4, 1, 2)).astype(np.float32) for _ in range(2))
    table = np.array([[2, 0, 3]], np.int32)
    q = rng.standard_normal((9, 4, 128))
    out, lse = O.attention_block(q, k, v, ks, vs, table, [0, 9], [41], 0.09, np.zeros((9, 4, 128)), np.zeros((9, 4)))
    keys = torch.from_numpy(O.cached_block_values(k, ks, table, 0, 41)).repeat_interleave(2, 1).transpose(0, 1)
    vals = torch.from_numpy(O.cached_block_values(v, vs, table, 0, 41)).repeat_interleave(2, 1).transpose(0, 1)
    mask = torch.arange(41)[None] <= torch.arange(32, 41)[:, None]
    tq = torch.from_numpy(q).transpose(0, 1)
    ref = torch.nn.functional.scaled_dot_product_attention(tq, keys, vals, attn_mask=mask, scale=0.09)
    np.testing.assert_allclose(out, ref.transpose(0, 1).numpy(), rtol=1e-9, atol=1e-12)
    full = torch.logsumexp((tq @ keys.transpose(1, 2) * 0.09).masked_fill(~mask, -np.inf), -1)
    np.testing.assert_allclose(lse, full.T.numpy(), rtol=1e-12)
    before = np.full((4, 2, 16), 5.0)
    w = O.attention_weights_block(q, k, ks, lse, before, table, [0, 9], [41], 0.09)
    old = np.zeros_like(before)
    old[2], old[0] = 5.0, 5.0                                                  # the first 32 tokens had 5 each
    used = np.zeros((4, 2, 16), bool)
    used[2], used[0], used[3, :, :9] = True, True, True
    assert np.all(w[~used] == 5.0)
    np.testing.assert_allclose((w - old)[used].sum(), 9 * 4, rtol=1e-12)


def test_kept_tokens():
    w = [9, 1, 5, 5, -0.0, 0.0, 7, 5, 2, 3]
    assert O.kept_tokens(w, 10, 0, 0) == list(range(10)) and O.kept_tokens(w, 11, 3, 3) == list(range(10))
    assert O.kept_tokens(w, 3, 0, 0) == [0, 2, 6]                             # the earliest of three fives
    assert O.kept_tokens(w, 4, 2, 1) == [0, 1, 6, 9]
    assert O.kept_tokens(w, 4, 2, 2) == [0, 1, 8, 9]
    assert O.kept_tokens([0.0, -0.0, 0.0], 2, 0, 0) == [0, 1]
    assert O.kept_tokens([1.0, float("nan"), float("inf")], 1, 0, 0) == [1]


def test_eviction_keeps_values_within_half_a_step():
    rng = np.random.default_rng(3)
    k, v = (rng.integers(-127, 128, (6, 16, 2, 8)).astype(np.int8) for _ in range(2))
    ks, vs = (rng.uniform(0.5, 2, (6, 1, 2)).astype(np.float32) for _ in range(2))
    w = rng.random((6, 2, 16)).astype(np.float32)
    table, new = np.array([[4, 1, 5]], np.int32), np.array([[0, 2]], np.int32)
    kept, lens, k2, v2, ks2, vs2, w2 = O.evict_block_paged(k, v, ks, vs, w, table, [45], new, 20, 1, 4)
    assert lens[0] == 20 and list(kept[0, 0, -4:]) == [41, 42, 43, 44] and kept[0, 0, 0] == 0
    for a, a2, s, s2 in ((k, k2, ks, ks2), (v, v2, vs, vs2)):
        old, got = O.cached_block_values(a, s, table, 0, 45), O.cached_block_values(a2, s2, new, 0, 20)
        for h in range(2):
            step = np.repeat([s2[0, 0, h], s2[2, 0, h]], 16)[:20, None]
            assert np.all(np.abs(got[:, h] - old[kept[0, h], h]) <= 0.50001 * step)
    assert np.array_equal(k2[[1, 3, 4, 5]], k[[1, 3, 4, 5]])


# ------------------------------------------------------------------- C refusals
def test_append_validation(L):
    def call(k=FAKE, v=FAKE, kc=FAKE, ks=FAKE, bt=FAKE, st=FAKE, kl=FAKE, n=4, B=2, Hkv=2, D=128, kst=256, vst=256, npg=8,
             ps=64, mp=4, block=32):
        return L.fa3_append_gqa_block_paged(k, v, kc, FAKE, ks, FAKE, bt, st, kl, n, B, Hkv, D, kst, vst, npg, ps, mp, block,
                                            None, None)
    for bad in (dict(k=None), dict(v=None), dict(kc=None), dict(ks=None), dict(bt=None), dict(st=None), dict(kl=None),
                dict(n=0), dict(B=0), dict(Hkv=0), dict(D=0), dict(npg=0), dict(ps=0), dict(mp=0), dict(block=0),
                dict(block=48), dict(block=128)):
        assert call(**bad) == EINVAL, bad
    for bad in (dict(block=8), dict(ps=8192, block=8192), dict(D=12), dict(D=264), dict(kst=254), dict(vst=-4), dict(k=ODD4),
                dict(kc=ODD4), dict(ks=ctypes.c_void_p(4098)), dict(ps=1 << 20, mp=1 << 12), dict(npg=1 << 25),
                dict(B=(1 << 30) + 1), dict(Hkv=65536)):
        assert call(**bad) == ERANGE, bad


def test_attention_validation(L):
    def call(q=FAKE, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, st=FAKE, kl=FAKE, bt=FAKE, out=FAKE, n=4, B=2, Hq=16, Hkv=2, D=128,
             qs=2048, npg=8, ps=64, mp=4, block=32, sc=0.09, ws=FAKE, wsb=1 << 40):
        return L.fa3_attn_gqa_block_paged(q, k, v, ks, vs, st, kl, bt, out, None, n, B, Hq, Hkv, D, qs, npg, ps, mp, block,
                                          sc, ws, wsb, None, None)
    for bad in (dict(q=None), dict(k=None), dict(v=None), dict(ks=None), dict(vs=None), dict(st=None), dict(kl=None),
                dict(bt=None), dict(out=None), dict(n=0), dict(B=0), dict(Hq=15), dict(Hkv=0), dict(sc=0.0),
                dict(sc=float("nan")), dict(ps=0), dict(npg=0), dict(block=48), dict(D=0)):
        assert call(**bad) == EINVAL, bad
    for bad in (dict(D=64), dict(Hq=258), dict(q=ODD8), dict(k=ODD8), dict(out=ODD8), dict(qs=2052), dict(qs=-8),
                dict(block=8), dict(ps=1 << 20, mp=1 << 12), dict(n=1 << 27), dict(B=(1 << 30) + 1)):
        assert call(**bad) == ERANGE, bad


def test_weights_validation(L):
    def call(q=FAKE, k=FAKE, ks=FAKE, lse=FAKE, w=FAKE, st=FAKE, kl=FAKE, bt=FAKE, n=4, B=2, Hq=16, Hkv=2, D=128, qs=2048,
             npg=8, ps=64, mp=4, block=32, sc=0.09):
        return L.fa3_attn_weights_gqa_block_paged(q, k, ks, lse, w, st, kl, bt, n, B, Hq, Hkv, D, qs, npg, ps, mp, block, sc,
                                                  FAKE, 1 << 30, None, None)
    for bad in (dict(q=None), dict(k=None), dict(ks=None), dict(lse=None), dict(w=None), dict(st=None), dict(kl=None),
                dict(bt=None), dict(n=0), dict(B=0), dict(Hq=15), dict(Hkv=0), dict(sc=-1.0), dict(sc=float("inf")),
                dict(block=48), dict(D=0)):
        assert call(**bad) == EINVAL, bad
    for bad in (dict(D=64), dict(Hq=258), dict(q=ODD8), dict(k=ODD8), dict(qs=2052), dict(qs=1024), dict(block=8),
                dict(n=1 << 27)):
        assert call(**bad) == ERANGE, bad
    assert L.fa3_attn_weights_workspace_size() > 0


def test_values_of_four_bytes_are_aligned(L):
    odd = ctypes.c_void_p(4098)
    for at in (3, 4, 9):
        a = [FAKE] * 10
        a[at] = odd
        assert L.fa3_attn_gqa_block_paged(*a, 4, 2, 16, 2, 128, 2048, 8, 64, 4, 32, 0.09, FAKE, 1 << 40, None, None) == ERANGE
    for at in (2, 3, 4):
        a = [FAKE] * 8
        a[at] = odd
        assert L.fa3_attn_weights_gqa_block_paged(*a, 4, 2, 16, 2, 128, 2048, 8, 64, 4, 32, 0.09, FAKE, 1 << 30, None, None) == ERANGE


def test_eviction_validation(L):
    def call(k=FAKE, v=FAKE, ks=FAKE, w=FAKE, bt=FAKE, kl=FAKE, nt=FAKE, kept=FAKE, nl=FAKE, B=2, Hkv=2, D=128, npg=8, ps=64,
             mp=4, block=32, new=2, budget=100, sinks=4, recent=10):
        return L.fa3_evict_gqa_block_paged(k, v, ks, FAKE, w, bt, kl, nt, kept, nl, B, Hkv, D, npg, ps, mp, block, new, budget,
                                           sinks, recent, None, None)
    for bad in (dict(k=None), dict(v=None), dict(ks=None), dict(w=None), dict(bt=None), dict(kl=None), dict(nt=None),
                dict(kept=None), dict(nl=None), dict(B=0), dict(Hkv=0), dict(D=0), dict(new=0), dict(budget=0),
                dict(sinks=-1), dict(recent=-1), dict(sinks=50, recent=51), dict(budget=129), dict(block=48)):
        assert call(**bad) == EINVAL, bad
    for bad in (dict(D=12), dict(D=264), dict(block=8), dict(k=ODD4), dict(B=65536), dict(w=ctypes.c_void_p(4098))):
        assert call(**bad) == ERANGE, bad


def test_eviction_refuses_lengths_in_place_and_budgets_beyond_32_bits(L):
    def call(kl, nl, budget=100, new=2):
        return L.fa3_evict_gqa_block_paged(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, kl, FAKE, FAKE, nl, 4, 2, 128, 8, 64, 4, 32, new,
                                           budget, 4, 10, None, None)
    at = FAKE.value
    for d in (0, 4, 12, -12):
        assert call(FAKE, ctypes.c_void_p(at + d)) == EINVAL, d
    assert call(FAKE, ctypes.c_void_p(at + 16), (1 << 31) - 65535, 1 << 25) == ERANGE


def test_call_block_knows_the_calls(L):
    F = fa3()
    for name, count in (("fa3_append_gqa_block_paged", 21), ("fa3_attn_gqa_block_paged", 25),
                        ("fa3_attn_weights_gqa_block_paged", 23), ("fa3_evict_gqa_block_paged", 23)):
        i, pack, n = F._CALLS[name]
        assert n == count
        args = pack(*([0] * n))
        assert L.fa3_call(i, args, n) == EINVAL and L.fa3_call(i, args, n - 1) == EINVAL


# ------------------------------------------------------------- binding refusals
def test_binding_refuses_host_tensors_and_shapes():
    F = fa3()
    pool = torch.zeros(3, 32, 2, 128, dtype=torch.int8)
    with pytest.raises(ValueError):
        F.block_scale_pool(pool, 24)
    with pytest.raises(ValueError):
        F.block_scale_pool(pool, 0)
    with pytest.raises(ValueError):
        F.attn_weight_pool(pool[0])
    s, w = F.block_scale_pool(pool, 16), F.attn_weight_pool(pool)
    assert s.shape == (3, 2, 2) and w.shape == (3, 2, 32)
    i = torch.zeros(1, dtype=torch.int32)
    x = torch.zeros(1, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        F.append_gqa_block_paged(x, x, pool, pool, s, s, i[None], i, i)
    with pytest.raises(TypeError):
        F.attn_gqa_block_paged(x, pool, pool, s, s, i, i, i[None], 0.1)
    with pytest.raises(TypeError):
        F.attn_weights_gqa_block_paged(x, pool, s, x, w, i, i, i[None], 0.1)
    with pytest.raises(TypeError):
        F.evict_gqa_block_paged(pool, pool, s, s, w, i[None], i, i[None], 4)
