"""spec_verify_accept against exact integers."""
import numpy as np
import pytest
import torch

import _step as S
from _devsetup import DEV, dev_err

pytestmark = pytest.mark.gpu

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module")
def pkv():
    import paged_kv_cache_int64_gb300 as m
    return m


def make(R, T, V, dtype, drafted, seed, sharp=2.0):
    g = torch.Generator().manual_seed(seed)
    base = sharp * torch.randn(R, T, V, generator=g)
    near = base[:, :T - 1] + 0.7 * torch.randn(R, T - 1, V, generator=g)
    P = torch.softmax(base, -1).to(TYPES[dtype])
    Q = torch.softmax(near, -1).to(TYPES[dtype]) if drafted else None
    ids = torch.multinomial(torch.softmax(near, -1).reshape(-1, V), 1, generator=g).reshape(R, T - 1).int() if T > 1 else \
        torch.zeros(R, 0, dtype=torch.int32)
    return P, Q, ids, torch.rand(R, T - 1, generator=g), torch.rand(R, generator=g), \
        torch.randint(0, T, (R,), generator=g, dtype=torch.int32)


def run(pkv, P, Q, ids, ua, us, nd, stream=None):
    R, T, _ = P.shape
    out = torch.full((R, T), 77, dtype=torch.int32, device=DEV)
    num, err = torch.full((R,), 77, dtype=torch.int32, device=DEV), dev_err()
    dev = lambda x: None if x is None else x if x.is_cuda else x.to(DEV)  # noqa: E731
    pkv.spec_verify_accept(dev(P), dev(Q), dev(ids), dev(ua), dev(us), out, num, num_drafts=dev(nd), dev_err=err, stream=stream)
    torch.cuda.synchronize()
    return out.cpu().numpy(), num.cpu().numpy(), err.item()


def check(pkv, P, Q, ids, ua, us, nd, status=0):
    got = run(pkv, P, Q, ids, ua, us, nd)
    R, T, _ = P.shape
    f = lambda x: None if x is None else x.cpu().float().numpy()  # noqa: E731
    want = S.accept(f(P), f(Q), ids.cpu().numpy(), ua.cpu().numpy(), us.cpu().numpy(), [T - 1] * R if nd is None else nd.cpu().numpy())
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1]), (got[:2], want)
    assert got[2] == status


@pytest.mark.parametrize("R,T,V", [(1, 1, 1), (1, 1, 7), (2, 2, 33), (3, 4, 1000), (5, 9, 4097), (16, 3, 32000), (2, 40, 515),
                                   (4, 5, 50021), (2, 3, 131072), (1, 2, 262144)])
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("drafted", [True, False])
def test_accept(pkv, R, T, V, dtype, drafted):
    P, Q, ids, ua, us, nd = make(R, T, V, dtype, drafted, seed=R * 100 + T)
    check(pkv, P, Q, ids, ua, us, nd)
    check(pkv, P, Q, ids, ua, us, None)


def test_accept_all_and_none(pkv):
    P, Q, ids, ua, us, _ = make(4, 6, 2000, "fp32", True, seed=3)
    check(pkv, P, Q, ids, torch.zeros_like(ua), us, None)  # 0 < p: every draft stays
    got = run(pkv, P, Q, ids, torch.zeros_like(ua), us, None)
    assert (got[1] == 6).all()
    P2 = P.clone()
    P2.scatter_(2, torch.nn.functional.pad(ids, (0, 1))[..., None].long(), 0.0)
    check(pkv, P2, Q, ids, ua, us, None)  # p = 0: the first draft goes
    assert (run(pkv, P2, Q, ids, ua, us, None)[1] == 1).all()


@pytest.mark.parametrize("u", [0.0, 1e-30, 2.0 ** -24, 0.25, 0.5, 0.75, 1.0 - 2.0 ** -24, 1.0, -1.0, float("nan")])
def test_borders_of_the_running_sum(pkv, u):
    """Dyadic probabilities: u times the total falls on the borders themselves."""
    V = 4096
    P = torch.zeros(3, 1, V)
    P[0, 0, [5, 1000, 2049, 4095]] = 0.25
    P[1, 0, :] = 1.0 / V
    P[2, 0, 4095] = 1.0
    e = torch.zeros(3, 0)
    check(pkv, P, None, e.int(), e, torch.full((3,), u), None)


def test_residual_that_is_empty_draws_from_the_target(pkv):
    P, _, ids, ua, us, _ = make(3, 3, 700, "fp32", True, seed=5)
    Q = P[:, :2].clone()
    ids = torch.zeros(3, 2, dtype=torch.int32)
    P[:, 0, 0] = 0.0  # not accepted, and max(p - q, 0) = 0 everywhere
    check(pkv, P, Q, ids, ua, us, None)
    P1 = torch.zeros(1, 2, 300)
    P1[0, :, 17] = 1.0
    check(pkv, P1, None, torch.tensor([[17]], dtype=torch.int32), torch.tensor([[0.5]]), torch.tensor([0.9]), None)  # one-hot: greedy
    check(pkv, P1, None, torch.tensor([[16]], dtype=torch.int32), torch.tensor([[0.5]]), torch.tensor([0.9]), None)


@pytest.mark.parametrize("V", [4096, 50021])
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_low_parts_of_one_sign(pkv, V, dtype):
    """p halfway between two multiples of 2^-23 and q one less, everywhere: every difference is 2^-23, all of it from the
    parts below 2^-23 (p rounds down to the even multiple, q up to it)."""
    R = 16
    P = torch.full((R, 2, V), 64.5 * 2.0 ** -23).to(TYPES[dtype])
    Q = torch.full((R, 1, V), 63.5 * 2.0 ** -23).to(TYPES[dtype])
    assert (P.double() == 64.5 * 2.0 ** -23).all() and (Q.double() == 63.5 * 2.0 ** -23).all()
    ids = torch.arange(R, dtype=torch.int32)[:, None]
    P[torch.arange(R), 0, ids[:, 0].long()] = 0.0  # the draft goes
    us = (torch.arange(R) + 0.25) / R
    check(pkv, P, Q, ids, torch.full((R, 1), 0.5), us, None)


def test_values_out_of_range(pkv):
    P, Q, ids, ua, us, _ = make(4, 4, 600, "fp32", True, seed=6)
    P[0, 0, :300] = float("nan")
    P[1, 0, 3] = float("inf")
    P[2, 1, 9] = -1.0
    Q[3, 0, 5] = float("nan")
    check(pkv, P, Q, ids, ua, us, None)
    check(pkv, torch.zeros(2, 1, 50), None, ids[:2, :0], ua[:2, :0], us[:2], None, status=pkv.PKV_ERR_DEVICE_BOUNDS)  # token 0
    bad = ids.clone()
    bad[0, 1], bad[1, 0], bad[2, 2] = 600, -1, 2 ** 31 - 1
    for q in (Q, None):
        check(pkv, P, q, bad, torch.zeros_like(ua), us, None, status=pkv.PKV_ERR_DEVICE_BOUNDS)
    check(pkv, P, Q, ids, ua, us, torch.tensor([-1, 4, 3, 0], dtype=torch.int32), status=pkv.PKV_ERR_DEVICE_BOUNDS)


@pytest.mark.parametrize("offset", [0, 1])
def test_strided_and_unaligned_rows(pkv, offset):
    """Rows inside a wider tensor, at odd offsets; requests and tokens interleaved."""
    R, T, V = 3, 4, 1021
    P, Q, ids, ua, us, nd = make(R, T, V, "bf16", True, seed=8)
    wide = torch.full((T, R, V + 11), float("nan"), dtype=torch.bfloat16, device=DEV)
    view = wide.permute(1, 0, 2)[:, :, offset:offset + V]
    view.copy_(P)
    wq = torch.full((R, T - 1, V + 16), float("nan"), dtype=torch.bfloat16, device=DEV)
    vq = wq[..., 8:8 + V]
    vq.copy_(Q)
    got = run(pkv, view, vq, ids, ua, us, nd)
    want = run(pkv, P, Q, ids, ua, us, nd)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])


def test_distribution(pkv):
    """Emitted first tokens have the target's distribution: chi-square over 20,000 requests, 11 degrees of freedom, the
    value that 1 in a million draws passes (48.2)."""
    R, V = 20000, 12
    g = torch.Generator().manual_seed(11)
    p, q = torch.softmax(torch.randn(V, generator=g), 0), torch.softmax(torch.randn(V, generator=g), 0)
    ids = torch.multinomial(q.expand(R, V), 1, generator=g).int()
    out, _, _ = run(pkv, p.expand(R, 2, V), q.expand(R, 1, V), ids, torch.rand(R, 1, generator=g), torch.rand(R, generator=g), None)
    seen = np.bincount(out[:, 0], minlength=V)
    want = R * p.double().numpy() / p.double().sum().item()
    assert ((seen - want) ** 2 / want).sum() < 48.2


def test_graph_and_other_stream(pkv):
    P, Q, ids, ua, us, nd = (x.to(DEV) for x in make(7, 5, 9001, "fp32", True, seed=12))
    out, num = torch.zeros(7, 5, dtype=torch.int32, device=DEV), torch.zeros(7, dtype=torch.int32, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    pkv.spec_verify_accept(P, Q, ids, ua, us, out, num, num_drafts=nd, stream=side)
    side.synchronize()
    want = run(pkv, P, Q, ids, ua, us, nd)
    assert np.array_equal(out.cpu().numpy(), want[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.spec_verify_accept(P, Q, ids, ua, us, out, num, num_drafts=nd)
    for seed in (1, 2):
        us.copy_(torch.rand(7, generator=torch.Generator().manual_seed(seed)))
        out.fill_(5)
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(out.cpu().numpy(), run(pkv, P, Q, ids, ua, us, nd)[0])
