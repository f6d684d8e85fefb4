"""Refusals of the calls after the verify attention: no GPU needed, nothing is launched."""
import ctypes as C
import struct

import numpy as np
import pytest

import _step as S


@pytest.fixture(scope="module")
def pkv():
    import __graft_entry__
    __graft_entry__._build_module().build()
    import paged_kv_cache_int64_gb300 as m
    return m


ACCEPT = dict(tp=16, tsr=400, tst=100, dp=16, dsr=300, dst=100, dt=0, ids=16, ua=16, us=16, nd=None, R=1, T=4, V=100, out=16,
              num=16, err=None, stream=None)
WEIGHTS = dict(q=16, k=16, fmt=0, ks=None, nb=4, sb=16384, st=1024, sh=256, ssb=64, sst=4, bt=16, bts=1, mb=1, sl=16, qv=None,
               R=1, T=1, hq=16, hkv=4, d=256, bs=16, scale=0.0625, lse=None, split=0, splits=0, prev=None, pl=None, w=16, wr=64,
               wh=16, mc=16, ws=16, wsb=1 << 24, err=None, stream=None)
SELECT = dict(s=16, sr=64, sh=16, mc=16, sl=16, R=1, hkv=4, sinks=1, recent=2, budget=8, keep=16, nl=16, err=None, stream=None)
COMPACT = dict(k=16, v=16, fmt=0, nb=4, sb=16384, st=1024, sh=256, ks=None, vs=None, ssb=0, sst=0, ssh=0, t=16, ts=1, tb=1, u=16,
               us=1, ub=1, keep=16, nl=16, R=1, hkv=4, budget=8, bs=16, d=256, w=None, wr=0, wh=0, mc=0, ws=16, wsb=1 << 20,
               err=None, stream=None)
INT8 = dict(fmt=1, ks=16, vs=16, ssb=64, sst=4, ssh=1)
FP4 = dict(fmt=3, ks=16, vs=16, ssb=1024, sst=64, ssh=16, sb=8192, st=512, sh=128)


@pytest.mark.parametrize("call,base,change,status", [
    ("pkv_spec_verify_accept", ACCEPT, dict(R=0, tp=None), 0),
    ("pkv_spec_verify_accept", ACCEPT, dict(R=-1), 1),
    ("pkv_spec_verify_accept", ACCEPT, dict(T=0), 1),
    ("pkv_spec_verify_accept", ACCEPT, dict(V=0), 1),
    ("pkv_spec_verify_accept", ACCEPT, dict(V=(1 << 30) + 1), 2),
    ("pkv_spec_verify_accept", ACCEPT, dict(dt=3), 1),
    ("pkv_spec_verify_accept", ACCEPT, dict(tp=None), 1),
    ("pkv_spec_verify_accept", ACCEPT, dict(ids=None), 1),
    ("pkv_spec_verify_accept", ACCEPT, dict(ua=None), 1),
    ("pkv_spec_verify_accept", ACCEPT, dict(us=None), 1),
    ("pkv_spec_verify_accept", ACCEPT, dict(out=None), 1),
    ("pkv_spec_verify_accept", ACCEPT, dict(num=None), 1),
    ("pkv_spec_verify_accept", ACCEPT, dict(tp=18), 1),
    ("pkv_spec_verify_accept", ACCEPT, dict(dp=17, dt=1), 1),
    ("pkv_spec_verify_accept", ACCEPT, dict(tst=-1), 1),
    ("pkv_kv_attn_weights", WEIGHTS, dict(R=0, q=None), 0),
    ("pkv_kv_attn_weights", WEIGHTS, dict(d=128), 2),
    ("pkv_kv_attn_weights", WEIGHTS, dict(fmt=3), 1),
    ("pkv_kv_attn_weights", WEIGHTS, dict(q=None), 1),
    ("pkv_kv_attn_weights", WEIGHTS, dict(w=None), 1),
    ("pkv_kv_attn_weights", WEIGHTS, dict(ws=None), 1),
    ("pkv_kv_attn_weights", WEIGHTS, dict(fmt=1), 1),
    ("pkv_kv_attn_weights", WEIGHTS, dict(fmt=2), 1),
    ("pkv_kv_attn_weights", WEIGHTS, dict(T=0), 1),
    ("pkv_kv_attn_weights", WEIGHTS, dict(hq=15), 2),
    ("pkv_kv_attn_weights", WEIGHTS, dict(hq=129, hkv=1), 2),
    ("pkv_kv_attn_weights", WEIGHTS, dict(bs=12), 2),
    ("pkv_kv_attn_weights", WEIGHTS, dict(bts=0), 1),
    ("pkv_kv_attn_weights", WEIGHTS, dict(mc=0), 1),
    ("pkv_kv_attn_weights", WEIGHTS, dict(mb=1 << 28, bts=1 << 28), 2),
    ("pkv_kv_attn_weights", WEIGHTS, dict(mb=1 << 20, bts=1 << 20, bs=2040, R=1000), 2),
    ("pkv_kv_attn_weights", WEIGHTS, dict(q=24), 1),
    ("pkv_kv_attn_weights", WEIGHTS, dict(k=24), 1),
    ("pkv_kv_attn_weights", WEIGHTS, dict(sh=260), 1),
    ("pkv_kv_attn_weights", WEIGHTS, dict(w=18), 1),
    ("pkv_kv_attn_weights", WEIGHTS, dict(sb=0), 1),
    ("pkv_kv_attn_weights", WEIGHTS, dict(fmt=1, ks=16, sst=3), 1),
    ("pkv_kv_attn_weights", WEIGHTS, dict(fmt=1, ks=18), 1),
    ("pkv_kv_attn_weights", WEIGHTS, dict(scale=0.0), 1),
    ("pkv_kv_attn_weights", WEIGHTS, dict(scale=float("nan")), 1),
    ("pkv_kv_attn_weights", WEIGHTS, dict(lse=16), 1),
    ("pkv_kv_attn_weights", WEIGHTS, dict(lse=16, split=128), 1),
    ("pkv_kv_attn_weights", WEIGHTS, dict(wh=15), 1),
    ("pkv_kv_attn_weights", WEIGHTS, dict(R=2, wr=8), 1),
    ("pkv_kv_attn_weights", WEIGHTS, dict(wsb=8), 1),
    ("pkv_kv_attn_weights", WEIGHTS, dict(ws=20), 1),
    ("pkv_kv_evict_select", SELECT, dict(R=0, s=None), 0),
    ("pkv_kv_evict_select", SELECT, dict(budget=0, sinks=0, recent=0), 1),
    ("pkv_kv_evict_select", SELECT, dict(sinks=6, recent=3), 1),
    ("pkv_kv_evict_select", SELECT, dict(sinks=2 ** 31 - 1, recent=2 ** 31 - 1), 1),
    ("pkv_kv_evict_select", SELECT, dict(sinks=-1), 1),
    ("pkv_kv_evict_select", SELECT, dict(recent=-1), 1),
    ("pkv_kv_evict_select", SELECT, dict(mc=0), 1),
    ("pkv_kv_evict_select", SELECT, dict(mc=1 << 31), 2),
    ("pkv_kv_evict_select", SELECT, dict(s=None), 1),
    ("pkv_kv_evict_select", SELECT, dict(s=18), 1),
    ("pkv_kv_evict_select", SELECT, dict(keep=None), 1),
    ("pkv_kv_evict_select", SELECT, dict(nl=None), 1),
    ("pkv_kv_evict_select", SELECT, dict(sr=-1), 1),
    ("pkv_kv_cache_compact", COMPACT, dict(R=0, k=None), 0),
    ("pkv_kv_cache_compact", COMPACT, dict(d=128), 2),
    ("pkv_kv_cache_compact", COMPACT, dict(fmt=4), 1),
    ("pkv_kv_cache_compact", COMPACT, dict(k=None), 1),
    ("pkv_kv_cache_compact", COMPACT, dict(u=None), 1),
    ("pkv_kv_cache_compact", COMPACT, dict(keep=None), 1),
    ("pkv_kv_cache_compact", COMPACT, dict(ws=None), 1),
    ("pkv_kv_cache_compact", COMPACT, dict(wsb=3), 1),
    ("pkv_kv_cache_compact", COMPACT, dict(budget=0), 1),
    ("pkv_kv_cache_compact", COMPACT, dict(us=0), 1),
    ("pkv_kv_cache_compact", COMPACT, dict(k=24), 1),
    ("pkv_kv_cache_compact", COMPACT, dict(st=1020), 1),
    ("pkv_kv_cache_compact", COMPACT, dict(sh=0), 1),
    ("pkv_kv_cache_compact", COMPACT, dict(w=16), 1),
    ("pkv_kv_cache_compact", COMPACT, dict(w=18, mc=16), 1),
    ("pkv_kv_cache_compact", COMPACT, dict(w=16, mc=16, wr=64, wh=8), 1),
    ("pkv_kv_cache_compact", COMPACT, dict(fmt=1), 1),
    ("pkv_kv_cache_compact", COMPACT, {**INT8, "vs": 18}, 1),
    ("pkv_kv_cache_compact", COMPACT, {**INT8, "sst": 0}, 1),
    ("pkv_kv_cache_compact", COMPACT, {**FP4, "ks": None}, 1),
    ("pkv_kv_cache_compact", COMPACT, {**FP4, "ssh": 8}, 1),
    ("pkv_kv_cache_compact", COMPACT, {**FP4, "ks": 20}, 1),
])
def test_refusals(pkv, call, base, change, status):
    got = getattr(pkv.lib, call)(*{**base, **change}.values())
    assert got == status, pkv.lib.pkv_last_error()
    assert bool(pkv.lib.pkv_last_error()) == bool(status)


CALLS = ("pkv_spec_verify_accept", "pkv_kv_attn_weights", "pkv_kv_evict_select", "pkv_kv_cache_compact")


def packed(pkv, call, values, size=None):
    b = b"".join(struct.pack("=d" if isinstance(v, float) else "=q", v or 0) for v in values)
    return pkv.lib.pkv_call_packed(call, b, len(b) if size is None else size)


def test_packed_calls_refuse_alike(pkv):
    cases = test_refusals.pytestmark[0].args[1]
    assert {c[0] for c in cases} == set(CALLS)
    for call, base, change, status in cases:
        values = list({**base, **change}.values())
        assert getattr(pkv.lib, call)(*values) == status
        message = pkv.lib.pkv_last_error()
        assert packed(pkv, CALLS.index(call), values) == status
        assert pkv.lib.pkv_last_error() == message


def test_packed_calls_refuse_what_does_not_fit(pkv):
    for i, base in enumerate((ACCEPT, WEIGHTS, SELECT, COMPACT)):
        values = list({**base, "R": 0}.values())
        assert packed(pkv, i, values) == 0
        for bad in (values[:-1], values + [0]):
            assert packed(pkv, i, bad) == 1 and b"bytes" in pkv.lib.pkv_last_error()
        for r in (1 << 32, -(1 << 31) - 1):
            assert packed(pkv, i, list({**base, "R": r}.values())) == 1 and b"range" in pkv.lib.pkv_last_error()
        assert pkv.lib.pkv_call_packed(i, None, 8 * len(values)) == 1
    for i in (-1, 4):
        assert packed(pkv, i, [0]) == 1 and b"unknown" in pkv.lib.pkv_last_error()


def test_workspace_bytes(pkv):
    assert pkv.kv_attn_weights_workspace_bytes(0, 4, 1) == 0 and pkv.kv_cache_compact_workspace_bytes(1, 0, 1) == 0
    assert pkv.kv_attn_weights_workspace_bytes(8, 16, 152) >= 8 * 16 * 4
    assert pkv.kv_cache_compact_workspace_bytes(2, 4, 65) % 4 == 0
    # sizes past 32 bits
    assert pkv.kv_cache_compact_workspace_bytes(1 << 16, 1 << 8, 1 << 10) > 1 << 28


def test_binding_refuses(pkv):
    torch = pytest.importorskip("torch")
    P = torch.zeros(1, 2, 8)
    i, f = torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, 1)
    with pytest.raises(AssertionError):  # not on the GPU
        pkv.spec_verify_accept(P, None, i, f, f[0], torch.zeros(1, 2, dtype=torch.int32), i[0])
    with pytest.raises(AssertionError):  # a type that probabilities do not have
        pkv.spec_verify_accept(P.double(), None, i, f, f[0], torch.zeros(1, 2, dtype=torch.int32), i[0])
    with pytest.raises(AssertionError):
        pkv.kv_evict_select(torch.zeros(1, 1, 8), i[0], 0, 1, 4, torch.zeros(1, 1, 4, dtype=torch.int32), i[0])


def test_plain_accept_by_hand():
    P = np.array([[[0.5, 0.25, 0.25], [0.0, 0.5, 0.5]]], dtype=np.float32)
    Q = np.array([[[0.25, 0.5, 0.25]]], dtype=np.float32)
    run = lambda x, ua, us: S.accept(P, Q, np.array([[x]]), np.array([[ua]]), np.array([us]), [1])  # noqa: E731
    assert [v.tolist() for v in run(0, 0.99, 0.0)] == [[[0, 1]], [2]]   # 0.99 * 0.25 < 0.5; then the first with p > 0
    assert [v.tolist() for v in run(0, 0.99, 0.5)] == [[[0, 2]], [2]]   # 0.5 is not above 0.5
    assert [v.tolist() for v in run(1, 0.5, 0.9)] == [[[0, -1]], [1]]   # 0.5 * 0.5 = p: goes; max(p - q, 0) = (0.25, 0, 0)
    assert [v.tolist() for v in run(1, 0.25, 0.9)] == [[[1, 2]], [2]]


def test_plain_select_by_hand():
    s = np.array([9, 1, 5, 5, np.nan, 5, 2, 0], dtype=np.float32)
    assert S.select(s, 8, 1, 1, 4).tolist() == [0, 2, 3, 7]
    assert S.select(s, 8, 0, 0, 7).tolist() == [0, 1, 2, 3, 5, 6, 7]
    assert S.select(s, 3, 1, 1, 4).tolist() == [0, 1, 2]
    assert S.select(s, 8, 2, 2, 4).tolist() == [0, 1, 6, 7]


def test_plain_weights_by_hand():
    """One query head, two tokens: a causal softmax written out."""
    q, k = np.zeros((2, 1, 256)), np.zeros((3, 1, 256))
    q[:, 0, 0] = [1.0, 2.0]
    k[:, 0, 0] = [0.0, np.log(2.0), np.log(3.0)]
    w, bound = S.weights(q, k, 3, 2, 1.0, 2)
    assert np.allclose(w[0], [1 / 3 + 1 / 14, 2 / 3 + 4 / 14, 9 / 14], rtol=1e-14)
    assert (bound > 0).all() and bound.max() < 1e-4
    assert np.allclose(S.weights(q, k, 3, 2, 1.0, 1)[0][0], [1 / 3, 2 / 3, 0], rtol=1e-14)
