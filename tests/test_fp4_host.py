"""The 4-bit cache on the host: the numpy statement of its formats is held to hand-made values, and the
three calls' argument checks refuse bad calls before any CUDA call is reached."""
import numpy as np
import pytest

import _fp4 as F


@pytest.fixture(scope="module")
def pkv():
    import __graft_entry__
    __graft_entry__._build_module().build()
    import paged_kv_cache_int64_gb300 as m
    return m


def test_formats_by_hand():
    # ties of e2m1 go to the even code, magnitudes past 6 saturate
    x = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.001, 7.0, 1e9, 0.2501, 0.7499])
    assert F._nearest_even(x, F.E2M1).tolist() == [0, 2, 2, 4, 4, 6, 6, 7, 7, 7, 1, 1]
    assert F.E4M3[0x7E] == 448 and F.E4M3[0x01] == 2.0 ** -9 and F.E4M3[0x08] == 2.0 ** -6 and np.isnan(F.E4M3[0x7F])
    # e4m3: 17 lies between 16 (even) and 18; 19 between 18 and 20 (even); past 448 saturates
    assert [F.E4M3[i] for i in F._nearest_even([17.0, 19.0, 1e4], F._POS)] == [16.0, 20.0, 448.0]


def test_quantizer_by_hand():
    # scale 1: a group whose largest magnitude is 6 has s = 1 and stores small halves exactly
    x = np.zeros(256, dtype=np.float32)
    x[:16] = [6, -6, 3, -3, 1.5, 0.5, 0, -0.0, 4, 2, 1, -1, 2.5, 3.5, 0.25, -0.25]
    x[16:32] = 12.0                     # s = 2, codes 6
    x[32] = np.inf                      # saturates: s = 448, code 7
    x[48] = np.nan                      # NaN scale, zero codes
    u = F.f32_to_bf16(np.where(np.isnan(x), 0, x))
    u[48] = 0x7FC0
    c, s = F.quantize(u, 1.0)
    assert [F.E4M3[b] for b in s[:3]] == [1.0, 2.0, 448.0] and s[3] == 0x7F
    lo = F.values(c, s)
    assert lo[:14].tolist() == [6, -6, 3, -3, 1.5, 0.5, 0, 0, 4, 2, 1, -1, 2, 4]
    assert (lo[14:16] == 0).all() and (lo[16:32] == 12).all() and lo[32] == 6 * 448 and (c[24:32] == 0).all()
    assert c[3] >> 4 == 8  # the sign of a negative zero is kept


# pointers are small fake addresses (multiples of 32): no check reads them

def _write(pkv, **kw):
    a = dict(kn=64, vn=64, nst=1024, bt=64, bts=1, mb=1, sl=64, qsl=64, R=1, max_q=1, kc=64, vc=64, kb=64, vb=64, ks=64,
             vs=64, nb=4, sb=8192, st=512, sh=128, ssb=1024, sst=64, ssh=16, bs=16, hkv=4, d=256, err=None, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return pkv.lib.pkv_kv_cache_write_fp4(*[a[k] for k in (
        "kn", "vn", "nst", "bt", "bts", "mb", "sl", "qsl", "R", "max_q", "kc", "vc", "kb", "vb", "ks", "vs", "nb", "sb",
        "st", "sh", "ssb", "sst", "ssh", "bs", "hkv", "d", "err", "stream")])


def _read(pkv, **kw):
    a = dict(kc=64, vc=64, kb=64, vb=64, ks=64, vs=64, nb=4, sb=8192, st=512, sh=128, ssb=1024, sst=64, ssh=16, bt=64,
             bts=1, mb=1, pb=64, pe=64, R=1, max_t=1, bs=16, hkv=4, d=256, kd=64, vd=64, ctx=16, err=None, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return pkv.lib.pkv_kv_fp4_dequant_dense(*[a[k] for k in (
        "kc", "vc", "kb", "vb", "ks", "vs", "nb", "sb", "st", "sh", "ssb", "sst", "ssh", "bt", "bts", "mb", "pb", "pe",
        "R", "max_t", "bs", "hkv", "d", "kd", "vd", "ctx", "err", "stream")])


def _attend(pkv, **kw):
    a = dict(q=64, kc=64, vc=64, kb=64, vb=64, ks=64, vs=64, nb=4, sb=8192, st=512, sh=128, ssb=1024, sst=64, ssh=16,
             bt=64, bts=1, mb=1, sl=64, R=1, T=1, hq=16, hkv=4, d=256, bs=16, scale=0.0625, out=64, ws=64, wsb=1 << 30,
             err=None, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return pkv.lib.pkv_spec_verify_attn_fp4(*[a[k] for k in (
        "q", "kc", "vc", "kb", "vb", "ks", "vs", "nb", "sb", "st", "sh", "ssb", "sst", "ssh", "bt", "bts", "mb", "sl", "R",
        "T", "hq", "hkv", "d", "bs", "scale", "out", "ws", "wsb", "err", "stream")])


CACHE_BAD = [
    (dict(d=128), 2),      # head_dim
    (dict(kc=None), 1),    # null pointers
    (dict(vb=None), 1),
    (dict(ks=None), 1),
    (dict(bt=None), 1),
    (dict(nb=0), 1),       # sizes
    (dict(bs=0), 1),
    (dict(mb=2), 1),       # table stride below its columns
    (dict(hkv=0), 1),
    (dict(st=-512), 1),    # strides
    (dict(ssh=0), 1),
    (dict(sh=136), 1),     # alignment
    (dict(ssh=8), 1),
    (dict(kc=72), 1),
    (dict(vb=72), 1),
]


@pytest.mark.parametrize("kw,status", CACHE_BAD + [
    (dict(kn=None), 1), (dict(qsl=None), 1), (dict(max_q=-1), 1), (dict(R=-1), 1),
    (dict(nst=512), 1),    # token stride below a token's rows
    (dict(nst=1032), 1),   # not a multiple of 16 elements
    (dict(kn=80), 1),      # rows 16- but not 32-byte aligned
])
def test_write_refuses(pkv, kw, status):
    assert _write(pkv, **kw) == status and pkv.lib.pkv_last_error()


@pytest.mark.parametrize("kw,status", CACHE_BAD + [
    (dict(pb=None), 1), (dict(pe=None), 1), (dict(kd=None), 1), (dict(kd=80), 1), (dict(ctx=0), 1), (dict(max_t=-1), 1),
])
def test_read_refuses(pkv, kw, status):
    assert _read(pkv, **kw) == status and pkv.lib.pkv_last_error()


@pytest.mark.parametrize("kw,status", CACHE_BAD + [
    (dict(q=None), 1), (dict(sl=None), 1), (dict(out=None), 1), (dict(ws=None), 1), (dict(R=-1), 1), (dict(T=0), 1),
    (dict(hq=15), 2), (dict(hq=132), 2),     # heads: not a multiple, more than 32 a KV head
    (dict(bs=20), 2),                        # block_size not a multiple of 8
    (dict(q=72), 1), (dict(out=72), 1), (dict(ws=72), 1), (dict(wsb=1024), 1),
    (dict(scale=0.0), 1), (dict(scale=float("nan")), 1), (dict(R=1 << 30, T=1 << 20), 1),
    (dict(mb=1 << 27, bts=1 << 27), 2),      # table columns past 2^31 - 128 positions
])
def test_attend_refuses(pkv, kw, status):
    assert _attend(pkv, **kw) == status and pkv.lib.pkv_last_error()


def test_nothing_to_do_launches_nothing(pkv):
    assert _write(pkv, R=0) == 0 and _write(pkv, max_q=0, kn=None) == 0
    assert _read(pkv, R=0) == 0 and _read(pkv, max_t=0, kc=None) == 0
    assert _attend(pkv, R=0) == 0


def test_workspace_bytes(pkv):
    one = pkv.spec_verify_fp4_workspace_bytes(1)
    assert one > 0 and one % 16 == 0 and pkv.spec_verify_fp4_workspace_bytes(152) == 152 * one
    assert pkv.spec_verify_fp4_workspace_bytes(0) == 0 and pkv.spec_verify_fp4_workspace_bytes(-3) == 0
