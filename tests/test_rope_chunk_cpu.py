"""CPU checks of the attention-input and packed-attention calls: the oracle's own pins, the host-side
refusals of the C ABI and those of the binding."""
import ctypes
import threading
import types
from collections import OrderedDict

import numpy as np
import pytest
import torch

from helpers import fa3
from oracle import fa3_oracle as O

EINVAL, ERANGE, EWORKSPACE = 1, 2, 4
FAKE = ctypes.c_void_p(4096)          # never dereferenced: validation fails first
ODD4 = ctypes.c_void_p(4096 + 4)


@pytest.fixture(scope="module")
def L():
    return fa3().lib()


# ------------------------------------------------------------------ oracle pins
def _table(n, rot):
    a = np.arange(n)[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / rot)
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_complex_product(interleaved):
    rng = np.random.default_rng(1)
    x, cs, pos = rng.standard_normal((7, 3, 16)), _table(50, 8), rng.integers(0, 50, 7)
    y, m = O.norm_rope(x, None, 0.0, cs, pos, interleaved)
    z = x[..., 0:8:2] + 1j * x[..., 1:8:2] if interleaved else x[..., :4] + 1j * x[..., 4:8]
    z = z * (cs[pos, :4] + 1j * cs[pos, 4:].astype(np.float64))[:, None]
    got = y[..., 0:8:2] + 1j * y[..., 1:8:2] if interleaved else y[..., :4] + 1j * y[..., 4:8]
    np.testing.assert_allclose(got, z, rtol=1e-12, atol=1e-14)
    assert np.array_equal(y[..., 8:], x[..., 8:])
    assert np.all(m >= np.abs(y) - 1e-12)


def test_rotated_scores_depend_on_the_distance_only():
    rng = np.random.default_rng(2)
    q, k, cs = rng.standard_normal((1, 1, 64)), rng.standard_normal((1, 1, 64)), _table(200, 64)
    dot = lambda i, j: float((O.norm_rope(q, None, 0, cs, np.array([i]), False)[0]  # noqa: E731
                              * O.norm_rope(k, None, 0, cs, np.array([j]), False)[0]).sum())
    assert abs(dot(10, 3) - dot(150, 143)) < 1e-4
    assert abs(dot(10, 3) - dot(10, 4)) > 1e-3


def test_norm_against_hand_values():
    y, _ = O.norm_rope(np.array([[[3.0, 4.0, 0, 0, 0, 0, 0, 0]]]), np.array([2.0, 1, 1, 1, 1, 1, 1, 1]), 0.0, None,
                       np.array([0]), False)
    np.testing.assert_allclose(y[0, 0, :2], [6 / np.sqrt(25 / 8), 4 / np.sqrt(25 / 8)], rtol=1e-14)


def test_packed_attention_equals_prefill_and_cross():
    rng = np.random.default_rng(3)
    code = lambda *s: rng.integers(-127, 128, s).astype(np.int8)  # noqa: E731
    q, k, v = code(1, 9, 4, 128), code(1, 12, 2, 128), code(1, 12, 2, 128)
    qs, ks, vs = (rng.uniform(0.001, 0.01, n).astype(np.float32) for n in (4, 2, 2))
    ref = O.gqa_prefill(q, k, v, qs, ks, vs, np.array([9]), np.array([12]), 0.09)
    got = O.packed_attention(q[0], [k[0]], [v[0]], qs, ks, vs, [0, 9], [12], 0.09, True, np.zeros((9, 4, 128)))
    np.testing.assert_allclose(got, ref[0], rtol=1e-9, atol=1e-12)
    got = O.packed_attention(q[0], [k[0]], [v[0]], qs, ks, vs, [0, 9], [12], 0.09, False, np.zeros((9, 4, 128)))
    dq = torch.from_numpy(q[0] * qs[None, :, None].astype(np.float64)).transpose(0, 1)
    dk, dv = (torch.from_numpy(np.repeat(x[0] * s[None, :, None].astype(np.float64), 2, 1)).transpose(0, 1)
              for x, s in ((k, ks), (v, vs)))
    full = torch.nn.functional.scaled_dot_product_attention(dq, dk, dv, scale=0.09).transpose(0, 1).numpy()
    np.testing.assert_allclose(got, full, rtol=1e-9, atol=1e-12)


def test_append_oracle_places_rows():
    rng = np.random.default_rng(4)
    k = rng.standard_normal((3, 1, 8))
    pool = np.zeros((4, 2, 1, 8), np.int8)
    one = np.ones(1, np.float32) / 20
    _, kp, vp = O.rope_append_paged(None, k, k, None, None, 0.0, None, False, None, one, one, None, pool, pool,
                                    np.array([[3, 1]], np.int32), np.array([0, 3]), np.array([4]))
    assert kp[3, 1].any() and kp[1].any() and not kp[3, 0].any() and not kp[0].any() and not kp[2].any()
    assert np.array_equal(kp, vp)


# ------------------------------------------------------------------- C refusals
def test_norm_rope_validation(L):
    def call(q=FAKE, k=FAKE, qw=FAKE, kw=FAKE, eps=1e-6, cs=FAKE, tl=10, rot=64, pos=FAKE, qo=FAKE, ko=FAKE, S=4, Hkv=2,
             D=128, qss=1024, qsb=0):
        return L.fa3_norm_rope(q, k, qw, kw, eps, cs, tl, rot, 0, pos, qo, ko, 0, 1, S, 8, Hkv, D, qsb, qss, 128, 0,
                               256, 128, 0, 1024, 128, 0, 256, 128, None, None)
    assert call(q=None) == EINVAL
    assert call(qo=None) == EINVAL
    assert call(pos=None) == EINVAL
    assert call(ko=None) == EINVAL
    assert call(k=None, ko=None) == EINVAL            # Hkv without k
    assert call(kw=None) == EINVAL
    assert call(S=0) == EINVAL
    assert call(eps=-1.0) == EINVAL
    assert call(eps=float("nan")) == EINVAL
    assert call(tl=0) == EINVAL
    assert call(rot=136) == EINVAL
    assert call(rot=12) == ERANGE
    assert call(D=12, rot=8) == ERANGE
    assert call(D=264) == ERANGE
    assert call(qss=1022) == ERANGE
    assert call(qsb=-4) == ERANGE
    assert call(q=ODD4) == ERANGE
    assert call(S=1 << 30, Hkv=2) in (ERANGE, 5, 3)    # too many tasks, or no device here


def test_rope_append_validation(L):
    def call(q=FAKE, k=FAKE, qw=None, qs=FAKE, qo=FAKE, kc=FAKE, bt=FAKE, st=FAKE, n=4, B=2, Hq=8, D=128, stride=1024,
             npg=8, ps=16, mp=4, rot=64):
        return L.fa3_rope_append_gqa_paged(q, k, FAKE, qw, None, 1e-6, FAKE, 10, rot, 0, qs, FAKE, FAKE, qo, kc, FAKE,
                                           bt, st, FAKE, n, B, Hq, 2, D, stride, stride, stride, npg, ps, mp, None, None)
    assert call(k=None) == EINVAL
    assert call(bt=None) == EINVAL
    assert call(st=None) == EINVAL
    assert call(qo=None) == EINVAL
    assert call(qs=None) == EINVAL
    assert call(q=None, qo=None, qw=FAKE) == EINVAL
    assert call(n=0) == EINVAL
    assert call(B=0) == EINVAL
    assert call(Hq=0) == EINVAL
    assert call(ps=0) == EINVAL
    assert call(ps=1 << 20, mp=1 << 12) == ERANGE
    assert call(rot=4) == ERANGE
    assert call(D=20, rot=8) == ERANGE
    assert call(stride=1026) == ERANGE
    assert call(kc=ODD4) == ERANGE


def test_packed_attention_validation(L):
    UN = ctypes.c_void_p(4096 + 8)

    def chunk(q=FAKE, st=FAKE, bt=FAKE, out=FAKE, n=4, B=2, Hq=16, Hkv=2, D=128, npg=8, ps=16, mp=4, sc=0.09):
        return L.fa3_prefill_attn_gqa_paged(q, FAKE, FAKE, FAKE, FAKE, FAKE, st, FAKE, bt, out, n, B, Hq, Hkv, D, npg,
                                            ps, mp, sc, FAKE, 1 << 40, None, None)

    def cross(k=FAKE, n=4, B=2, T=64, Hq=16, Hkv=2, D=128, sc=0.09):
        return L.fa3_cross_attn_gqa(FAKE, k, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, n, B, T, Hq, Hkv, D, sc, FAKE,
                                    1 << 40, None, None)
    assert chunk(q=None) == EINVAL and chunk(st=None) == EINVAL and chunk(bt=None) == EINVAL
    assert chunk(out=None) == EINVAL and chunk(n=0) == EINVAL and chunk(B=0) == EINVAL
    assert chunk(Hq=15) == EINVAL and chunk(sc=0.0) == EINVAL and chunk(sc=float("inf")) == EINVAL
    assert chunk(ps=0) == EINVAL and chunk(npg=0) == EINVAL
    assert chunk(D=64) == ERANGE and chunk(Hq=258) == ERANGE and chunk(q=UN) == ERANGE and chunk(out=UN) == ERANGE
    assert chunk(ps=1 << 20, mp=1 << 12) == ERANGE
    assert cross(k=None) == EINVAL and cross(T=0) == EINVAL and cross(Hkv=0) == EINVAL
    assert cross(D=256) == ERANGE and cross(k=UN) == ERANGE and cross(sc=-1.0) == EINVAL


# ------------------------------------------------------------- binding refusals
def test_binding_refuses_cpu_tensors_and_wrong_types():
    from int8_head_kv_gb300 import fa3 as F
    x = torch.zeros(2, 4, 128, dtype=torch.bfloat16)
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(TypeError):
        F.norm_rope(x, None, None, None)
    with pytest.raises(TypeError):
        F.norm_rope(x.float(), None, None, None)
    c = torch.zeros(2, 16, 1, 128, dtype=torch.int8)
    with pytest.raises(TypeError):
        F.rope_append_gqa_paged(None, x[:, :1], x[:, :1], None, None, None, None, c, c, None, i, i[:2])
    with pytest.raises(TypeError):
        F.prefill_attn_gqa_paged(None, c, c, None, None, None, i, i[:2], None, 0.1)
    with pytest.raises(TypeError):
        F.cross_attn_gqa(None, c, c, None, None, None, i, i[:2], 0.1)


def test_rope_table_checks_and_far_positions():
    from int8_head_kv_gb300 import fa3 as F
    for bad in ((0, 8), (4, 7), (4, 0)):
        with pytest.raises(ValueError):
            F.rope_table(*bad, device="cpu")
    with pytest.raises(ValueError):
        F.rope_table(4, 8, device="cpu", inv_freq=torch.ones(3))
    t = F.rope_table(100001, 4, device="cpu").numpy()
    ang = 100000 * np.array([1.0, 0.01])
    np.testing.assert_allclose(t[100000], np.concatenate([np.cos(ang), np.sin(ang)]), atol=2.0 ** -24)


def test_calls_in_one_block(L):
    from int8_head_kv_gb300 import fa3 as F
    for name, (i, pack, count) in F._CALLS.items():
        kinds = F._SIGS[name][1]
        zero = [0.0 if k is F._F else 0 for k in kinds]
        assert len(kinds) == count and L.fa3_call(i, pack(*zero), count) == EINVAL          # the call's own check
        assert L.fa3_call(i, pack(*zero), count - 1) == EINVAL
        assert L.fa3_call(i, None, count) == EINVAL
        for at, k in enumerate(kinds):                                                      # beyond an int
            for v in (1 << 31, -(1 << 31) - 1) if k is F._I else (-1,) if k is F._SZ else ():
                assert L.fa3_call(i, pack(*zero[:at], v, *zero[at + 1:]), count) == ERANGE, (name, at)
    assert L.fa3_call(len(F._CALLS), b"", 0) == EINVAL
    # the same answer as the call itself where the arguments are looked at one by one: a head size of 12
    args = [1 << 20, 0, 0, 0, 1e-6, 0, 0, 0, 0, 0, 1 << 20, 0, 0, 1, 1, 1, 0, 12] + [0] * 14
    i, pack, count = F._CALLS["fa3_norm_rope"]
    assert L.fa3_call(i, pack(*args), count) == L.fa3_norm_rope(*args) == ERANGE
    args[4] = float("nan")
    assert L.fa3_call(i, pack(*args), count) == L.fa3_norm_rope(*args) == EINVAL


def test_workspace_cache_is_looked_up_as_one_step(monkeypatch):
    # another host thread drops the entry between the look-up and what follows it
    from int8_head_kv_gb300 import fa3 as F
    stream, device, threads = types.SimpleNamespace(cuda_stream=77), torch.device("cuda", 0), []

    class Cache(OrderedDict):
        def get(self, key, default=None):
            found = super().get(key, default)
            threads.append(threading.Thread(target=F._forget_workspace, args=("chunk", device, stream)))
            threads[-1].start()
            threads[-1].join(0.3)
            return found

    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    for look_up in (lambda: F._chunk_workspace(100, device, stream, 0, 77), lambda: F._workspace("chunk", 100, device, stream=stream)):
        have = torch.empty(100, dtype=torch.uint8)
        monkeypatch.setattr(F, "_ws_cache", Cache({("chunk", 0, 77): have}))
        assert look_up() is have
        for t in threads:
            t.join()
        assert not F._ws_cache


def test_more_sequences_than_the_kernels_count_are_refused(L):
    for B in ((1 << 30) + 1, (1 << 31) - 1):
        assert L.fa3_rope_append_gqa_paged(None, FAKE, FAKE, None, None, 1e-6, None, 0, 0, 0, None, FAKE, FAKE, None, FAKE, FAKE, FAKE, FAKE, FAKE, 4,
                                           B, 0, 2, 128, 0, 1024, 1024, 8, 16, 4, None, None) == ERANGE
        assert L.fa3_prefill_attn_gqa_paged(*[FAKE] * 10, 4, B, 16, 2, 128, 8, 16, 4, 0.09, FAKE, 1 << 40, None, None) == ERANGE
        assert L.fa3_cross_attn_gqa(*[FAKE] * 9, 4, B, 1, 16, 2, 128, 0.09, FAKE, 1 << 40, None, None) == ERANGE
