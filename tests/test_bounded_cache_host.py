"""The calls after the verify attention, refused for how their buffers lie: no GPU needed, nothing is launched."""
import numpy as np
import pytest

from test_step_host import ACCEPT, COMPACT, SELECT, WEIGHTS, pkv  # noqa: F401


def refused(pkv, call, values, word):  # noqa: F811
    status = getattr(pkv.lib, call)(*values.values())
    assert status == pkv.PKV_ERR_INVALID_ARG and word in pkv.lib.pkv_last_error(), (status, pkv.lib.pkv_last_error())


@pytest.mark.parametrize("change", [
    dict(nl=0x1000),                          # the lengths updated in place
    dict(nl=0x1004), dict(nl=0x0ffc),         # a part of them
    dict(keep=0x1000), dict(keep=0x1004), dict(keep=0x1000 - 4 * 2 * 4 * 8 + 4),
    dict(nl=0x2000 + 4 * 2 * 4 * 8 - 4), dict(nl=0x2000 - 4),
])
def test_select_refuses_outputs_over_its_lengths(pkv, change):  # noqa: F811
    """Every CTA of a request reads its length while one of them writes the new one."""
    base = {**SELECT, "s": 0x100000, "R": 2, "sl": 0x1000, "keep": 0x2000, "nl": 0x3000}
    refused(pkv, "pkv_kv_evict_select", {**base, **change}, b"overlap")


@pytest.mark.parametrize("call,base", [("pkv_kv_attn_weights", dict(WEIGHTS)), ("pkv_kv_cache_compact", {**COMPACT, "w": 16})])
def test_rows_of_weights_that_overlap_are_refused(pkv, call, base):  # noqa: F811
    """Each stride holds a row, but request 0's next head, or its third, is another request's."""
    base = {**base, "hkv": 2, "mc": 16, "R": 2}
    for change in (dict(wr=16, wh=16), dict(wr=31, wh=16), dict(wr=16, wh=31), dict(wr=2 ** 62, wh=15), dict(wr=15, wh=2 ** 62),
                   dict(hkv=4, wr=48, wh=16), dict(hkv=4, wr=63, wh=16), dict(R=5, wr=16, wh=79),
                   dict(R=2 ** 20, wr=2 ** 44, wh=2 ** 63 - 1)):
        refused(pkv, call, {**base, **change}, b"rows of weights")


@pytest.mark.parametrize("call,base", [("pkv_kv_attn_weights", dict(WEIGHTS)), ("pkv_kv_cache_compact", {**COMPACT, "w": 16})])
def test_rows_of_weights_in_any_order_are_taken(pkv, call, base):  # noqa: F811
    """Requests inside heads or heads inside requests, one of either with any stride: the check after this one refuses."""
    last = dict(ws=20, d=256) if call == "pkv_kv_attn_weights" else dict(ws=18)
    base = {**base, "hkv": 2, "mc": 16, "R": 3, **last}
    for change in (dict(wr=32, wh=16), dict(wr=16, wh=48), dict(wr=2 ** 62, wh=16), dict(R=1, wr=0, wh=16), dict(hkv=1, wr=16, wh=0),
                   dict(R=1, hkv=1, wr=0, wh=0)):
        refused(pkv, call, {**base, **change}, b"workspace")


W0 = 0x100000


@pytest.mark.parametrize("R,hkv,wr,wh,mc,shift", [
    (1, 1, 16, 16, 16, 1), (1, 1, 16, 16, 16, -15),                 # a key's place against another's
    (2, 3, 48, 16, 16, 16), (2, 3, 48, 16, 16, 48), (2, 3, 48, 16, 16, -95), (2, 3, 48, 16, 16, 95),  # a head's, a request's
    (2, 3, 96, 32, 16, 1), (2, 3, 96, 32, 16, 32 + 15), (2, 3, 96, 32, 16, 17),  # rows with room in between
    (3, 2, 32, 96, 16, -64 + 15),
])
def test_earlier_weights_beside_their_own_place_are_refused(pkv, R, hkv, wr, wh, mc, shift):  # noqa: F811
    base = {**WEIGHTS, "R": R, "hkv": hkv, "hq": hkv, "wr": wr, "wh": wh, "mc": mc, "w": W0}
    refused(pkv, "pkv_kv_attn_weights", {**base, "prev": W0 + 4 * shift}, b"prev must be")


@pytest.mark.parametrize("R,hkv,wr,wh,mc,shift", [
    (1, 1, 16, 16, 16, 0), (2, 3, 48, 16, 16, 0), (1, 1, 16, 16, 16, 16), (2, 3, 48, 16, 16, -96), (2, 3, 48, 16, 16, 96),
    (2, 3, 96, 32, 16, 16), (2, 3, 96, 32, 16, -16),                # interleaved rows
    (2, 3, 192, 32, 16, 96), (3, 2, 32, 96, 16, 16), (20000, 4, 64, 16, 16, 20000 * 64),
])
def test_earlier_weights_apart_or_in_place_are_taken(pkv, R, hkv, wr, wh, mc, shift):  # noqa: F811
    """The check after this one refuses."""
    base = {**WEIGHTS, "R": R, "hkv": hkv, "hq": hkv, "wr": wr, "wh": wh, "mc": mc, "w": W0, "ws": 20}
    refused(pkv, "pkv_kv_attn_weights", {**base, "prev": W0 + 4 * shift}, b"workspace")


@pytest.mark.parametrize("change", [
    dict(out=0x1000), dict(out=0x1000 + 4 * 2 * 3 - 4), dict(out=0x1000 - 4 * 2 * 4 + 4),  # tokens over the drafts
    dict(num=0x1000), dict(num=0x1000 - 4), dict(num=0x2000), dict(num=0x2000 + 4 * 2 * 4 - 4),
    dict(nd=0x2004), dict(nd=0x3004), dict(nd=0x2ffc),
])
def test_accept_refuses_outputs_over_its_drafts(pkv, change):  # noqa: F811
    """A request's drafts are read while another's tokens are written."""
    base = {**ACCEPT, "tp": 0x100000, "dp": 0x200000, "R": 2, "ids": 0x1000, "out": 0x2000, "num": 0x3000, "nd": 0x4000}
    refused(pkv, "pkv_spec_verify_accept", {**base, **change}, b"overlap")
