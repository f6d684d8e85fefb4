"""Workloads of a speculative-decoding step over a bounded cache: verification of drafted tokens against the
target's probabilities, the attention weight that each cached key collects, the choice of the keys that stay, and
the move of their rows to the front.

`own` or plain, the layouts are the library's: caches [num_blocks][block_size][kv_heads][256] behind an int32 block
table, weights and scores fp32 [requests][kv_heads][positions].
"""
import functools
import math
import random

import numpy as np
import torch

own = False  # False: plain torch forms; True: the library's calls

D = 256
DEV = "cuda"
SPLIT = 4096  # keys of one split of the verify attention that ran before
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------------

def _accept(name, reqs, T, vocab, dtype, drafted, ragged):
    c = dict(op="accept", reqs=reqs, T=T, vocab=vocab, dtype=dtype, drafted=drafted, ragged=ragged)
    return dict(c, name=name) if name else c


def _weights(name, reqs, ctx, ragged, holes, T, hkv, group, block, kv, lse, prev):
    c = dict(op="weights", reqs=reqs, ctx=ctx, ragged=ragged, holes=holes, T=T, hkv=hkv, group=group, block=block, kv=kv,
             lse=lse, prev=prev)
    return dict(c, name=name) if name else c


def _select(name, reqs, ctx, ragged, hkv, budget, sinks, recent):
    c = dict(op="select", reqs=reqs, ctx=ctx, ragged=ragged, holes=False, hkv=hkv, budget=budget, sinks=sinks, recent=recent)
    return dict(c, name=name) if name else c


def _compact(name, reqs, ctx, ragged, hkv, block, budget, sinks, recent, inplace):
    c = dict(op="compact", reqs=reqs, ctx=ctx, ragged=ragged, holes=False, hkv=hkv, block=block, budget=budget, sinks=sinks,
             recent=recent, inplace=inplace)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one user, three drafts of a small draft model: latency
        _accept("accept_b1_32k", 1, 4, 32000, "fp32", True, False),
        # a batch of verify steps, seven drafts each
        _accept("accept_b64_128k", 64, 8, 131072, "fp32", True, False),
        # drafts looked up in the prompt (no draft probabilities), some requests with few or none; odd vocabulary
        _accept("accept_b256_odd", 256, 5, 50021, "bf16", False, True),
        # one user, one token, after the int8 verify attention: the weight of each key goes on top of the earlier steps'
        _weights("weights_b1_1k", 1, 1024, False, False, 1, 4, 4, 16, "int8", True, True),
        # a batch of verify steps of eight tokens, some rejected, int8 cache in large pages
        _weights("weights_b32_40k", 32, 40960, True, False, 8, 4, 4, 880, "int8", True, True),
        # the last 32 queries of two prompts look back at the whole prompt (bf16 cache, no earlier weights)
        _weights("weights_window_24k", 2, 24576, False, False, 32, 4, 4, 880, "bf16", False, False),
        # a padded batch: an empty request, a one-token one, odd heads and lengths, e4m3 cache in small pages
        _weights("weights_padded_odd", 7, 5003, True, True, 3, 2, 7, 48, "fp8", False, True),
        # half of a short context stays
        _select("select_b1_1k", 1, 1024, False, 4, 512, 4, 64),
        # a batch is cut back to a budget, lengths ragged (some within it)
        _select("select_b32_40k", 32, 40960, True, 4, 8192, 4, 256),
        # one very long context
        _select("select_b1_256k", 1, 262144, False, 4, 16384, 4, 1024),
        # in place, one user
        _compact("compact_b1_1k", 1, 1024, False, 4, 16, 512, 4, 64, True),
        # a batch's kept rows moved to the front of their own blocks
        _compact("compact_b16_32k", 16, 32768, True, 4, 880, 8192, 4, 256, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("accept", "weights", "weights", "select", "compact"))
    if op == "accept":
        vocab = _log(rng, 1000, 200000)
        return _accept(None, _log(rng, 1, min(256, 8388608 // vocab)), rng.randint(1, 9), vocab, rng.choice(("fp32", "fp32", "bf16", "fp16")),
                       rng.random() < 0.6, rng.random() < 0.5)
    reqs, hkv = _log(rng, 1, 32), rng.choice((1, 2, 3, 4, 5, 8))
    ragged = rng.random() < 0.7
    if op == "weights":
        kv = rng.choice(("bf16", "int8", "fp8"))
        ctx = _log(rng, 33, min(262144, 1_300_000 // (reqs * hkv)))
        group = rng.choice((1, 2, 3, 4, 5, 6, 7, 8, 12, 16))
        T = min(ctx, rng.choice((1, 1, rng.randint(2, 8), rng.randint(9, 40))))
        return _weights(None, reqs, ctx, ragged, rng.random() < 0.3, T, hkv, group, rng.choice((8, 16, 24, 32, 48, 64, 128, 176, 256, 880)),
                        kv, rng.random() < 0.5, rng.random() < 0.5)
    ctx = _log(rng, 100, min(262144, 2_000_000 // (reqs * hkv)))
    budget = max(2, int(ctx * rng.uniform(0.1, 0.9)))
    sinks = rng.randint(0, min(8, budget // 4))
    recent = rng.randint(1, max(1, budget // 4))
    if op == "select":
        return _select(None, reqs, ctx, ragged, hkv, budget, sinks, recent)
    ctx = min(ctx, 500_000 // (reqs * hkv))
    budget = max(2, min(budget, ctx - 1))
    return _compact(None, reqs, ctx, ragged, hkv, rng.choice((8, 16, 24, 48, 64, 176, 880)), budget, min(sinks, budget // 4),
                    max(1, min(recent, budget // 4)), rng.random() < 0.5)


def _lens(c):
    """The batch's lengths: the first is ctx; ragged ones spread over a factor of eight; `holes`: a batch padded with an
    empty request and a one-token request."""
    rng = random.Random(c["reqs"] * 1000003 + c["ctx"] * 101 + c["hkv"])
    lens = [c["ctx"]] + [_log(rng, max(1, c["ctx"] / 8), c["ctx"]) if c["ragged"] else c["ctx"] for _ in range(c["reqs"] - 1)]
    if c["holes"] and c["reqs"] >= 2:
        lens[-1] = 0
    if c["holes"] and c["reqs"] >= 3:
        lens[-2] = 1
    return lens


def _drafts(c):
    rng = random.Random(c["reqs"] * 101 + c["vocab"])
    return [rng.randint(0, c["T"] - 1) if c["ragged"] else c["T"] - 1 for _ in range(c["reqs"])]


def work(c):
    if c["op"] == "accept":
        size = 4 if c["dtype"] == "fp32" else 2
        # the row of probabilities that the last token is drawn from, and the draft's beside it
        rows = sum(2 if c["drafted"] and n else 1 for n in _drafts(c))
        return {"bytes": rows * c["vocab"] * size + c["reqs"] * c["T"] * 16, "flops": 2 * rows * c["vocab"]}
    lens = _lens(c)
    keys = sum(lens) * c["hkv"]
    if c["op"] == "weights":
        hq = c["hkv"] * c["group"]
        row = {"bf16": 512, "int8": 260, "fp8": 256}[c["kv"]]
        b = keys * (row + 4 + (4 if c["prev"] else 0)) + len(lens) * c["T"] * hq * 2 * D
        seen = sum(max(0, n - c["T"] + t + 1) for n in lens for t in range(c["T"]))
        return {"bytes": b, "flops": 2 * seen * hq * D}
    kept = sum(min(n, c["budget"]) for n in lens) * c["hkv"]
    if c["op"] == "select":
        return {"bytes": 4 * (keys + kept), "flops": keys}
    # rows that change their place: in place, requests within the budget and the first rows stay where they are
    moved = sum(c["budget"] - c["sinks"] for n in lens if n > c["budget"]) * c["hkv"] if c["inplace"] else kept
    return {"bytes": moved * (2 * 2 * 2 * D + 4 + 8), "flops": 0}


# ------------------------------------------------------------------------------------------------
# the plain forms
# ------------------------------------------------------------------------------------------------

def _plain_accept(s):
    P, Q, ids = s["target"], s["draft"], s["ids"].long()
    R, T, V = P.shape
    n = torch.zeros(R, dtype=torch.long, device=DEV)
    if T > 1:
        p = P[:, :-1].gather(2, ids[..., None])[..., 0].double()
        q = Q.gather(2, ids[..., None])[..., 0].double() if Q is not None else torch.ones_like(p)
        ok = (s["u_accept"].double() * q < p) & (torch.arange(T - 1, device=DEV) < s["num_drafts"].long()[:, None])
        n = ok.long().cumprod(1).sum(1)
    row = torch.arange(R, device=DEV)
    p = P[row, n].double()
    w = p
    if T > 1:
        at = n.clamp(max=T - 2)
        q = Q[row, at].double() if Q is not None else torch.zeros_like(p).scatter_(1, ids[row, at][:, None], 1.0)
        w = torch.where((n < s["num_drafts"])[:, None], (p - q).clamp(min=0.0), p)
    w = torch.where(w.sum(1, keepdim=True) > 0, w, p)
    c = w.cumsum(1)
    token = (c <= s["u_sample"].double()[:, None] * c[:, -1:]).sum(1)
    t = torch.arange(T, device=DEV)
    out = torch.where(t < n[:, None], torch.nn.functional.pad(ids, (0, 1)), torch.full_like(t, -1))
    return out.scatter(1, n[:, None], token[:, None]).int(), (n + 1).int()


def _slots(s, table, pos, req):
    """Flat slot (block * block_size + slot) of position pos of request req."""
    blk = table[req, (pos // s["block"]).long()].clamp(min=0).long()
    return blk * s["block"] + (pos % s["block"]).long()


def _keys(s):
    """K rows in fp32 [reqs][positions][hkv][256] and which of them are live."""
    pos, req = torch.arange(s["ctx"], device=DEV), torch.arange(s["reqs"], device=DEV)
    live = pos[None, :] < s["seq_lens"].long()[:, None]
    slot = _slots(s, s["bt"], pos[None, :].expand(s["reqs"], -1), req[:, None])
    k = s["k"].view(-1, s["hkv"], D)[slot]
    if s["kv"] == "int8":
        k = k.float() * s["k_scale"].view(-1, s["hkv"])[slot][..., None]
    elif s["kv"] == "fp8":
        k = k.view(torch.float8_e4m3fn).float() * s["k_scale"]
    return torch.where(live[..., None, None], k.float(), torch.zeros((), device=DEV)), live


def _plain_weights(s):
    R, T, hkv, g = s["reqs"], s["T"], s["hkv"], s["group"]
    k, live = _keys(s)
    q = s["q"].float().view(R, T, hkv, g, D).permute(0, 2, 1, 3, 4).reshape(R, hkv, T * g, D)
    w = torch.matmul(q, k.permute(0, 2, 3, 1)) * s["softmax_scale"]
    del k
    pos, t = torch.arange(s["ctx"], device=DEV), torch.arange(T, device=DEV)
    at = s["seq_lens"].long()[:, None] - T + t[None, :]  # the queries' own positions
    seen = (pos[None, None, :] <= at[:, :, None]) & live[:, None, :]
    seen = seen[:, None, :, None, :].expand(-1, 1, -1, g, -1).reshape(R, 1, T * g, -1)
    w = w.masked_fill(~seen, -math.inf)
    if s["part_lse"] is not None:
        x = torch.arange(s["part_lse"].shape[0], device=DEV)[:, None, None] * SPLIT < s["seq_lens"].long()[None, :, None]
        x = torch.where(x[..., None], s["part_lse"].view(-1, R, T, hkv * g), torch.full((), -math.inf, device=DEV))
        lse = torch.logsumexp(x, 0).view(R, T, hkv, g).permute(0, 2, 1, 3).reshape(R, hkv, T * g, 1)
    else:
        m = w.amax(-1, keepdim=True)
        m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
        lse = m + torch.log(torch.exp(w - m).sum(-1, keepdim=True))
    counted = (t[None, :] < s["q_valid"].long()[:, None]).repeat_interleave(g, 1)[:, None, :, None]
    w = torch.where(counted & ~torch.isinf(lse), torch.exp(w - lse), torch.zeros((), device=DEV)).sum(2)
    if s["prev"] is not None:
        w = w + torch.where((pos[None, :] < s["prev_lens"].long()[:, None])[:, None, :], s["prev"], torch.zeros((), device=DEV))
    s["weights"].copy_(torch.where(live[:, None, :], w, s["weights"]))
    return s["weights"]


def _plain_select(s):
    sc = s["scores"]
    n = s["seq_lens"].long()[:, None, None]
    pos = torch.arange(sc.shape[2], device=DEV)[None, None, :]
    sc = torch.where((pos < s["sinks"]) | (pos >= n - s["recent"]), torch.full((), math.inf, device=DEV), sc)
    sc = torch.where(pos < n, sc, torch.full((), -math.inf, device=DEV))
    first = torch.sort(sc, dim=-1, descending=True, stable=True)[1][..., :s["budget"]]
    new = n.clamp(max=s["budget"])
    j = torch.arange(s["budget"], device=DEV)
    kept = torch.sort(torch.where(j < new, first, torch.full_like(first, 1 << 40)), dim=-1)[0]
    s["keep"].copy_(torch.where(j < new, kept, s["keep"].long()).int())
    s["new_lens"].copy_(new.flatten().int())
    return s["keep"], s["new_lens"]


def _plain_compact(s):
    R, hkv, budget = s["keep"].shape
    j = torch.arange(budget, device=DEV).view(1, 1, -1).expand(R, hkv, -1)
    live = j < s["new_lens"].long()[:, None, None]
    r, h, j = (x[live] for x in (torch.arange(R, device=DEV).view(-1, 1, 1).expand(R, hkv, budget),
                                 torch.arange(hkv, device=DEV).view(1, -1, 1).expand(R, hkv, budget), j))
    at = s["keep"].long()[live]
    src, dst = _slots(s, s["bt"], at, r), _slots(s, s["dst"], j, r)
    k, v = s["k"].view(-1, hkv, D), s["v"].view(-1, hkv, D)
    k[dst, h] = k[src, h]
    v[dst, h] = v[src, h]
    s["weights"][r, h, j] = s["weights"][r, h, at]
    return s["k"], s["v"], s["weights"]


# ------------------------------------------------------------------------------------------------
# the library's calls
# ------------------------------------------------------------------------------------------------

def _own_accept(s):
    import paged_kv_cache_int64_gb300 as pkv
    pkv.spec_verify_accept(s["target"], s["draft"], s["ids"], s["u_accept"], s["u_sample"], s["tokens"], s["num_out"],
                           num_drafts=s["num_drafts"], dev_err=s["err"])
    return s["tokens"], s["num_out"]


@functools.lru_cache(None)
def _workspace(name, *sizes):
    """A call's workspace, which a program keeps for all its calls of these sizes on one stream."""
    import paged_kv_cache_int64_gb300 as pkv
    return torch.empty(getattr(pkv, name)(*sizes), dtype=torch.uint8, device=DEV)


def _own_weights(s):
    import paged_kv_cache_int64_gb300 as pkv
    kv = {"bf16": pkv.PKV_KV_BF16, "int8": pkv.PKV_KV_INT8, "fp8": pkv.PKV_KV_FP8}[s["kv"]]
    pkv.kv_attn_weights(s["q"], s["k"], s["bt"], s["seq_lens"], s["T"], s["softmax_scale"], s["weights"],
                        _workspace("kv_attn_weights_workspace_bytes", s["q"].shape[0], s["q"].shape[1]), kv_dtype=kv,
                        k_scale=s["k_scale"], prev=s["prev"], prev_lens=s["prev_lens"], q_valid=s["q_valid"],
                        part_lse=s["part_lse"], split_tokens=SPLIT, dev_err=s["err"])
    return s["weights"]


def _own_select(s):
    import paged_kv_cache_int64_gb300 as pkv
    pkv.kv_evict_select(s["scores"], s["seq_lens"], s["sinks"], s["recent"], s["budget"], s["keep"], s["new_lens"],
                        dev_err=s["err"])
    return s["keep"], s["new_lens"]


def _own_compact(s):
    import paged_kv_cache_int64_gb300 as pkv
    pkv.kv_cache_compact(s["k"], s["v"], s["bt"], s["dst"], s["keep"], s["new_lens"],
                         _workspace("kv_cache_compact_workspace_bytes", *s["keep"].shape), weights=s["weights"], dev_err=s["err"])
    return s["k"], s["v"], s["weights"]


# ------------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------------

def _probabilities(logits, dtype):
    """Softmax of rows whose logits are peaked as a language model's are: a few likely tokens, a long tail."""
    return torch.softmax(logits, -1).to(dtype)


def _prepare_accept(c, gen):
    R, T, V, dt = c["reqs"], c["T"], c["vocab"], TYPES[c["dtype"]]
    nd = _drafts(c)
    base = 2.5 * torch.randn(R, T, V, generator=gen, device=DEV)
    target = _probabilities(base, dt)
    s = dict(target=target, draft=None, num_drafts=torch.tensor(nd, dtype=torch.int32, device=DEV))
    # the draft model's rows: the target's logits, less sure
    guess = base[:, :T - 1] + 0.7 * torch.randn(R, T - 1, V, generator=gen, device=DEV)
    race = torch.empty(R, T - 1, V, device=DEV).exponential_(generator=gen)
    s["ids"] = (torch.softmax(guess, -1) / race).argmax(-1).int() if T > 1 else torch.zeros(R, 0, dtype=torch.int32, device=DEV)
    if c["drafted"]:
        s["draft"] = _probabilities(guess, dt)
    s["u_accept"] = torch.rand(R, T - 1, generator=gen, device=DEV)
    s["u_sample"] = torch.rand(R, generator=gen, device=DEV)
    s["tokens"] = torch.full((R, T), -1, dtype=torch.int32, device=DEV)
    s["num_out"] = torch.zeros(R, dtype=torch.int32, device=DEV)
    return s


def _table(lens, block, order, nb):
    """Block table of the requests over the first blocks of a permutation of nb."""
    pages = [-(-n // block) for n in lens]
    perm, at = order.permutation(nb), 0
    bt = np.full((len(lens), max(1, max(pages))), -1, dtype=np.int32)
    for r, n in enumerate(pages):
        bt[r, :n] = perm[at:at + n]
        at += n
    return bt


def _split_lse(s, q, k):
    """Split log-sum-exps of the scores, as the verify attention leaves them: natural, fp32, [splits][R*T][Hq]."""
    R, T, hkv, g, ctx = s["reqs"], s["T"], s["hkv"], s["group"], s["ctx"]
    S = -(-ctx // SPLIT)
    part = torch.full((S, R * T, hkv * g), math.nan, device=DEV)
    lens = s["seq_lens"].tolist()
    for r, n in enumerate(lens):
        qr = q[r * T:(r + 1) * T].double().view(T, hkv, g, D).permute(1, 0, 2, 3).reshape(hkv, T * g, D)
        for i in range(-(-n // SPLIT)):
            lo, hi = i * SPLIT, min(n, (i + 1) * SPLIT)
            z = torch.matmul(qr.float(), k[r, lo:hi].permute(1, 2, 0)).double() * s["softmax_scale"]
            own_pos = (n - T + torch.arange(T, device=DEV)).repeat_interleave(g)[None, :, None]
            z = z.masked_fill(torch.arange(lo, hi, device=DEV)[None, None, :] > own_pos, -math.inf)
            part[i, r * T:(r + 1) * T] = torch.logsumexp(z, -1).view(hkv, T, g).permute(1, 0, 2).reshape(T, hkv * g).float()
    return part


def _prepare_weights(c, gen, order, lens, s):
    R, T, hkv, g, block = c["reqs"], c["T"], c["hkv"], c["group"], c["block"]
    nb = sum(-(-n // block) for n in lens) + 3
    s.update(T=T, group=g, kv=c["kv"], bt=torch.from_numpy(_table(lens, block, order, nb)).to(DEV), softmax_scale=1.0 / math.sqrt(D),
             prev=None, prev_lens=None, part_lse=None, k_scale=None)
    # K rows with channels of different sizes
    x = torch.randn(nb, block, hkv, D, generator=gen, device=DEV) * torch.exp(0.6 * torch.randn(hkv, D, generator=gen, device=DEV))
    if c["kv"] == "int8":
        a = x.abs().amax(-1)
        s["k_scale"], s["k"] = a / 127.0, torch.round(x * (127.0 / a)[..., None]).to(torch.int8)
    elif c["kv"] == "fp8":
        s["k_scale"] = (x.abs().amax() / 448.0).reshape(1)
        s["k"] = (x / s["k_scale"]).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        s["k"] = x.to(torch.bfloat16)
    del x
    s["q"] = torch.randn(R * T, hkv * g, D, generator=gen, device=DEV).to(torch.bfloat16)
    s["weights"] = torch.zeros(R, hkv, s["ctx"], device=DEV)
    # a verify step of several tokens: some of each request's drafts were rejected; a window counts whole
    s["q_valid"] = torch.randint(1, T + 1, (R,), generator=gen, device=DEV, dtype=torch.int32) if c["prev"] else \
        torch.full((R,), T, dtype=torch.int32, device=DEV)
    if c["prev"]:
        s["prev"] = torch.rand(R, hkv, s["ctx"], generator=gen, device=DEV) ** 4
        s["prev_lens"] = (s["seq_lens"] - T).clamp(min=0)
    if c["lse"]:
        s["part_lse"] = _split_lse(s, s["q"], _keys(s)[0])


def _prepare_compact(c, gen, order, lens, s):
    R, hkv, block, budget = c["reqs"], c["hkv"], c["block"], c["budget"]
    new = [min(n, budget) for n in lens]
    pages = sum(-(-n // block) for n in lens) + 3
    extra = 0 if c["inplace"] else sum(-(-n // block) for n in new)
    bt = _table(lens, block, order, pages)
    s["bt"] = torch.from_numpy(bt).to(DEV)
    # the same table, or blocks that are not the requests' own
    s["dst"] = s["bt"] if c["inplace"] else torch.from_numpy(np.where((t := _table(new, block, order, extra)) >= 0, t + pages, -1).astype(np.int32)).to(DEV)
    for name in ("k", "v"):
        s[name] = torch.randn(pages + extra, block, hkv, D, generator=gen, device=DEV).to(torch.bfloat16)
    s["weights"] = torch.rand(R, hkv, s["ctx"], generator=gen, device=DEV)
    # kept positions: the first, the last, and a random choice in between
    n = s["seq_lens"].long()[:, None, None]
    pos = torch.arange(s["ctx"], device=DEV)[None, None, :]
    sc = torch.rand(R, hkv, s["ctx"], generator=gen, device=DEV)
    sc = torch.where((pos < c["sinks"]) | (pos >= n - c["recent"]), sc + 2.0, sc).masked_fill(pos >= n, -1.0)
    first = torch.sort(sc, dim=-1, descending=True, stable=True)[1][..., :budget]
    live = torch.arange(budget, device=DEV) < n
    s["keep"] = torch.where(live, torch.sort(torch.where(live, first, torch.full_like(first, 1 << 40)), dim=-1)[0], torch.full_like(first, -1)).int()
    s["new_lens"] = torch.tensor(new, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEV).manual_seed(seed)
    order = np.random.RandomState(seed % (1 << 31))
    if c["op"] == "accept":
        s = _prepare_accept(c, gen)
    else:
        lens = _lens(c)
        s = dict(reqs=c["reqs"], ctx=max(lens), hkv=c["hkv"], seq_lens=torch.tensor(lens, dtype=torch.int32, device=DEV),
                 block=c.get("block"))
        if c["op"] == "weights":
            _prepare_weights(c, gen, order, lens, s)
        elif c["op"] == "compact":
            _prepare_compact(c, gen, order, lens, s)
        else:
            # accumulated attention: a few large sums, a long tail of small ones, some keys that nothing looked at
            x = torch.exp(2.0 * torch.randn(c["reqs"], c["hkv"], s["ctx"], generator=gen, device=DEV) - 6.0)
            s["scores"] = torch.where(torch.rand(x.shape, generator=gen, device=DEV) < 0.02, torch.zeros_like(x), x)
            s.update(sinks=c["sinks"], recent=c["recent"], budget=c["budget"],
                     keep=torch.full((c["reqs"], c["hkv"], c["budget"]), -1, dtype=torch.int32, device=DEV),
                     new_lens=torch.zeros(c["reqs"], dtype=torch.int32, device=DEV))
    s.update(op=c["op"], err=torch.zeros(1, dtype=torch.int32, device=DEV))
    return s


def run(state):
    s = state
    if s["op"] == "accept":
        tokens, count = _own_accept(s) if own else _plain_accept(s)
        return {"tokens": tokens, "num_out": count}
    if s["op"] == "weights":
        return {"weights": _own_weights(s) if own else _plain_weights(s)}
    if s["op"] == "select":
        keep, new = _own_select(s) if own else _plain_select(s)
        return {"keep": keep, "new_lens": new}
    k, v, w = _own_compact(s) if own else _plain_compact(s)
    return {"k": k, "v": v, "weights": w}


# ------------------------------------------------------------------------------------------------
# from the definition, in 64 bits
# ------------------------------------------------------------------------------------------------

def _exact_accept(c, s):
    P = s["target"].double().cpu().numpy()
    Q = None if s["draft"] is None else s["draft"].double().cpu().numpy()
    ids, ua, us, nd = (s[k].cpu().numpy() for k in ("ids", "u_accept", "u_sample", "num_drafts"))
    tokens = np.full((c["reqs"], c["T"]), -1, dtype=np.int32)
    count = np.zeros(c["reqs"], dtype=np.int32)
    for r in range(c["reqs"]):
        t = 0
        while t < nd[r] and float(ua[r, t]) * (1.0 if Q is None else Q[r, t, ids[r, t]]) < P[r, t, ids[r, t]]:
            tokens[r, t] = ids[r, t]
            t += 1
        w = P[r, t].copy()
        if t < nd[r]:
            if Q is None:
                w[ids[r, t]] = 0.0
            else:
                w = np.maximum(w - Q[r, t], 0.0)
        cdf = np.cumsum(w)
        tokens[r, t] = np.searchsorted(cdf, float(us[r]) * cdf[-1], side="right")
        count[r] = t + 1
    return {"tokens": torch.from_numpy(tokens), "num_out": torch.from_numpy(count)}


def _exact_weights(c, s, lens):
    T, hkv, g = c["T"], c["hkv"], c["group"]
    out = torch.zeros(c["reqs"], hkv, s["ctx"], dtype=torch.float64, device=DEV)
    valid = s["q_valid"].tolist()
    for r, n in enumerate(lens):
        if n == 0:
            continue
        pos = torch.arange(n, device=DEV)
        rows = s["bt"][r].long()[pos // c["block"]] * c["block"] + pos % c["block"]
        k = s["k"].view(-1, hkv, D)[rows]
        if c["kv"] == "fp8":
            b = k.double()
            e, m = torch.floor(b / 8) % 16, b % 8
            k = torch.where(e > 0, (1 + m / 8) * 2.0 ** (e - 7), m * 2.0 ** -9) * torch.where(b >= 128, -1.0, 1.0) * s["k_scale"].double()
        elif c["kv"] == "int8":
            k = k.double() * s["k_scale"].view(-1, hkv)[rows].double()[..., None]
        else:
            k = k.double()
        for t in range(valid[r]):
            m = n - T + t + 1
            if m <= 0:
                continue
            z = torch.einsum("hgd,nhd->hgn", s["q"][r * T + t].double().view(hkv, g, D), k[:m]) * s["softmax_scale"]
            if s["part_lse"] is not None:
                lse = torch.logsumexp(s["part_lse"][:-(-n // SPLIT), r * T + t].double(), 0).view(hkv, g, 1)
                out[r, :, :m] += torch.exp(z - lse).sum(1)
            else:
                out[r, :, :m] += torch.softmax(z, -1).sum(1)
        if c["prev"]:
            m = max(0, n - T)
            out[r, :, :m] += s["prev"][r, :, :m].double()
    return {"weights": out}


def exact(case, seed):
    c = case
    if c["op"] == "compact":
        return None  # rows and numbers are moved, none is computed
    s = prepare(c, seed)
    if c["op"] == "accept":
        return _exact_accept(c, s)
    lens = _lens(c)
    if c["op"] == "weights":
        return _exact_weights(c, s, lens)
    scores = s["scores"].double().cpu().numpy()
    keep = np.full((c["reqs"], c["hkv"], c["budget"]), -1, dtype=np.int32)
    for r, n in enumerate(lens):
        for h in range(c["hkv"]):
            if n <= c["budget"]:
                keep[r, h, :n] = np.arange(n)
                continue
            x = scores[r, h, :n].copy()
            x[:c["sinks"]] = x[n - c["recent"]:] = math.inf
            keep[r, h] = np.sort(np.lexsort((np.arange(n), -x))[:c["budget"]])
    return {"keep": torch.from_numpy(keep), "new_lens": torch.tensor([min(n, c["budget"]) for n in lens], dtype=torch.int32)}
