"""The bound of tests/_fp4_bound.py sees what it is to see: coarser query rows, a lost tile or piece, a mask off
by one; and a query row's digits are as exact as the header says."""
import os
import re

import numpy as np
import pytest

import _fp4 as F
import _fp4_bound as B


def outlier_rows(rng, rows, big):
    """Query rows with one element of each 16 `big` times the others."""
    q = rng.standard_normal((rows, 256))
    q[:, rng.integers(0, 16, 16) + 16 * np.arange(16)] *= big
    return F.bf16_to_f32(F.f32_to_bf16(q.astype(np.float32))).astype(np.float64)


@pytest.mark.parametrize("big", [1, 30, 100, 1000, 3e5])
def test_query_digits(big):
    """Elements down to 2^-9 of their 16's largest and 2^-11 of the row's are exact; the others within half a
    step: 2^-17 of the 16's largest or 2^-19 of the row's."""
    rng = np.random.default_rng(int(big))
    q = outlier_rows(rng, 64, big)
    got = B.q_terms(q)
    assert (np.abs(got - q) <= B.q_lost(q)).all()
    a = np.abs(q)
    block = np.repeat(a.reshape(64, 16, 16).max(-1), 16, axis=-1)
    fine = (a >= 2.0 ** -9 * block) & (a >= 2.0 ** -11 * a.max(-1, keepdims=True))
    assert fine.any() and np.array_equal(got[fine], q[fine])
    assert (np.abs(got - q) <= np.maximum(2.0 ** -17 * block, 2.0 ** -19 * a.max(-1, keepdims=True))).all()


def test_query_digits_of_the_whole_range():
    """Every bf16 magnitude, 256 of one exponent range a row: subnormal numbers, the largest, mixed signs."""
    rng = np.random.default_rng(1)
    bits = np.arange(0x7F80, dtype=np.uint16)
    bits = np.concatenate([bits, rng.permutation(0x7F80).astype(np.uint16)])
    bits = bits[:len(bits) // 256 * 256].reshape(-1, 256) | (rng.integers(0, 2, (len(bits) // 256, 256)) << 15).astype(np.uint16)
    q = F.bf16_to_f32(bits).astype(np.float64)
    assert (np.abs(B.q_terms(q) - q) <= B.q_lost(q)).all()


def _cache(rng, n, channel=None):
    x = rng.standard_normal((n, 256)).astype(np.float32) * (1 if channel is None else channel)
    return F.values(*F.quantize(F.f32_to_bf16(x), 0.013)) * float(np.float32(0.013))


def _exceeds(got, want, tol):
    return (np.abs(got - want) > tol).any()


@pytest.mark.parametrize("big", [30, 100])
def test_bound_sees_coarser_query_rows(big):
    """Outlier channels that meet small ones of K (none of their codes is left): six digits stay inside, four do not."""
    rng = np.random.default_rng(big)
    at = rng.integers(0, 16, 16) + 16 * np.arange(16)
    q = rng.standard_normal((4, 256))
    q[:, at] *= big
    q = F.bf16_to_f32(F.f32_to_bf16(q.astype(np.float32))).astype(np.float64)
    channel = np.ones(256, dtype=np.float32)
    channel[at] = 1 / big
    k, v = _cache(rng, 2000, channel), _cache(rng, 2000)
    want, tol = B._rows(q, k, v, 0.25)
    for terms in (6, 4):
        _, p = B.probabilities(B.q_terms(q, terms), k, 0.25)
        assert _exceeds(p @ v, want, tol) == (terms == 4)


@pytest.mark.parametrize("n", [64, 300, 1000, 9000, 40000])
def test_bound_sees_lost_keys(n):
    """Rows of equal norms under a small scale, so that every key carries weight: leaving out the newest key, one
    tile or a piece of five tiles, or taking a key twice, passes the bound; an exact row rounded to bf16 does not."""
    rng = np.random.default_rng(n)
    q = F.bf16_to_f32(F.f32_to_bf16(rng.standard_normal((4, 256)).astype(np.float32))).astype(np.float64)
    k, v = _cache(rng, n), _cache(rng, n)
    want, tol = B._rows(q, k, v, 1 / 64)
    _, p = B.probabilities(q, k, 1 / 64)
    rounded = F.bf16_to_f32(F.f32_to_bf16(want.astype(np.float32)))
    assert not _exceeds(rounded, want, tol)

    def with_weights(w):
        return (p * w) @ v / (p * w).sum(-1, keepdims=True)

    for lo, hi in [(n - 1, n), (0, 1)] + [(a, min(a + size, n)) for size in (128, 640) for a in range(0, n, size)][:80]:
        if hi - lo == n:
            continue
        for weight in (0.0, 2.0):
            w = np.ones(n)
            w[lo:hi] = weight
            assert _exceeds(with_weights(w), want, tol), (lo, hi, weight)


CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_cache_int64_gb300", "csrc")


def code(name):
    """A source file without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


def test_merge_reads_the_workspace_by_plain_loads():
    """The read-only path promises data that no grid writes while the reading one is resident; the merge is
    launched beside the grid that writes its workspace."""
    text = code("spec_verify_fp4.cu")
    merge = text[text.index("spec_verify_fp4_merge_kernel("):]
    merge = merge[:merge.index("\n}")]
    assert "ws.lm" in merge and "ws.notes" in merge and "ws.o" in merge
    assert re.findall(r"__ld\w+\(([^)]*)\)", merge) == ["v_scale"]


@pytest.mark.parametrize("name", ["kv_fp4_write.cu", "kv_fp4_dequant.cu", "spec_verify_fp4.cu"])
def test_rules_take_the_device_s_sm_count(name):
    """What depends on how many warps or CTAs the device holds asks the device."""
    text = code(name)
    assert "num_sms()" in text and not re.search(r"\b1(32|4[48]|5[26]|60)\b", text)
