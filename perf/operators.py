"""Workloads of the 4-bit KV cache: quantizing K/V rows into it as they are written, reading it back
dense, and decode / speculative-verify attention over it.

The cache format (both sides, `own` or plain): a row of 256 elements is 128 bytes of e2m1 codes, the
even element in the low half of a byte, and 16 e4m3 scales, one per 16 elements; one fp32 scale per
tensor multiplies all of it. An element stands for e2m1 * e4m3 * scale.
"""
import functools
import math
import random

import numpy as np
import torch

own = False  # False: plain torch forms; True: the library's calls

D = 256
GROUP = 16
DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------------

def _case(name, op, reqs, ctx, ragged, holes, new, hkv, group, block):
    c = dict(op=op, reqs=reqs, ctx=ctx, ragged=ragged, holes=holes, new=new, hkv=hkv, group=group, block=block)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one user, one token: the append and the attention of a decode step, where launch latency counts
        _case("step_b1_1k", "append_attend", 1, 1024, False, False, 1, 4, 4, 16),
        # a batch of decode steps at mixed lengths, small pages
        _case("decode_b32_16k", "attend", 32, 16384, True, False, 1, 4, 4, 16),
        # speculative verify: eight draft tokens a request are appended and verified, large pages
        _case("verify_b32_40k", "append_attend", 32, 40960, True, False, 8, 4, 4, 880),
        # the same with 24 query heads on 4 KV heads (48 query rows a KV head)
        _case("verify_g6_20k", "attend", 8, 20008, False, False, 8, 4, 6, 880),
        # one very long context, one token
        _case("decode_b1_256k", "attend", 1, 262144, False, False, 1, 4, 4, 880),
        # a padded batch: an empty request, a one-token request, odd heads and lengths
        _case("padded_odd", "attend", 7, 5003, True, True, 3, 2, 7, 48),
        # decode rows of 64 users appended, then read back
        _case("append_b64", "write_read", 64, 1, False, False, 1, 4, 1, 16),
        # a 2,048-token prefill chunk written and read back for the chunk's attention
        _case("chunk_2048", "write_read", 1, 2048, False, False, 2048, 4, 1, 880),
        # prompts of many requests written at once (ragged), 8 KV heads
        _case("prompts_ragged", "write_read", 16, 8192, True, False, 8192, 8, 1, 64),
        # read back: a short prompt in odd pages, and one and many long contexts
        _case("read_777", "read", 1, 777, False, False, 0, 3, 1, 24),
        _case("read_47104", "read", 1, 47104, False, False, 0, 4, 1, 880),
        _case("read_b32_40k", "read", 32, 40960, True, False, 0, 4, 1, 16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("attend", "append_attend", "attend", "write_read", "read"))
    reqs = _log(rng, 1, 48)
    hkv = rng.choice((1, 2, 3, 4, 5, 8))
    block = rng.choice((8, 16, 24, 32, 48, 64, 128, 176, 256, 880))
    holes = rng.random() < 0.3
    ragged = rng.random() < 0.75
    if op in ("attend", "append_attend"):
        ctx = _log(rng, 17, min(262144, 2_560_000 // (reqs * hkv)))
        group = rng.choice((1, 2, 3, 4, 5, 6, 7, 8, 12, 16))
        return _case(None, op, reqs, ctx, ragged, holes, min(ctx, rng.randint(1, 12)), hkv, group, block)
    ctx = _log(rng, 3, min(65536, 560_000 // (reqs * hkv)))
    return _case(None, op, reqs, ctx, ragged, holes, ctx if op == "write_read" else 0, hkv, 1, block)


def _lens(c):
    """The batch's lengths: the first is ctx; ragged ones spread over a factor of eight; `holes`: a
    batch padded with an empty request and a one-token request."""
    rng = random.Random(c["reqs"] * 1000003 + c["ctx"] * 101 + c["hkv"])
    lens = [c["ctx"]] + [_log(rng, max(1, c["ctx"] / 8), c["ctx"]) if c["ragged"] else c["ctx"] for _ in range(c["reqs"] - 1)]
    if c["holes"] and c["reqs"] >= 2:
        lens[-1] = 0
    if c["holes"] and c["reqs"] >= 3:
        lens[-2] = 1
    return lens


def _new_lens(c):
    return [min(c["new"], n) for n in _lens(c)]


def work(c):
    lens = _lens(c)
    code_row, wide_row = D // 2 + D // GROUP, 2 * D  # bytes of one row of one tensor
    keys = sum(lens) * c["hkv"]
    new = sum(_new_lens(c)) * c["hkv"]
    meta = 4 * (2 * len(lens) + sum(-(-n // c["block"]) for n in lens))
    b, f = meta, 0
    if c["op"] in ("append_attend", "write_read"):
        b += 2 * new * (wide_row + code_row)
    if c["op"] in ("read", "write_read"):
        b += 2 * keys * (wide_row + code_row)
    if c["op"] in ("attend", "append_attend"):
        hq = c["hkv"] * c["group"]
        b += 2 * keys * code_row + 2 * len(lens) * c["new"] * hq * 2 * D
        seen = sum(max(0, n - c["new"] + t + 1) for n in lens for t in range(c["new"]))
        f += 4 * seen * hq * D
    return {"bytes": b, "flops": f}


# ------------------------------------------------------------------------------------------------
# the plain forms
# ------------------------------------------------------------------------------------------------

def _quantize(x, scale):
    """bf16 rows [..., 256] -> codes uint8 [..., 128], e4m3 scales as bytes [..., 16]."""
    x = x.float().unflatten(-1, (D // GROUP, GROUP))
    amax = x.abs().amax(-1)
    bs = (amax / (6.0 * scale)).clamp(max=448.0).to(torch.float8_e4m3fn)
    d = bs.float() * scale
    a = torch.where(((d >= 2.0 ** -126) & (d < math.inf))[..., None], (x / d[..., None]).abs(), torch.zeros_like(x))
    # nearest e2m1 magnitude, ties to the even code
    code = ((a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte() + (a > 2.5).byte() +
            (a >= 3.5).byte() + (a > 5.0).byte())
    code = code | (torch.signbit(x).byte() << 3)
    code = torch.where(torch.isnan(amax)[..., None], torch.zeros_like(code), code).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), bs.view(torch.uint8)


def _dequantize(codes, bscale, scale):
    """fp32 values [..., 256]."""
    two = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float32, device=codes.device)
    v = lut[two.int()].unflatten(-1, (D // GROUP, GROUP))
    return ((v * bscale.view(torch.float8_e4m3fn).float()[..., None]) * scale).flatten(-2)


def _slots(s, pos, req):
    """Flat slot (block * block_size + slot) of position pos of request req."""
    blk = s["bt"][req, (pos // s["block"]).long()].clamp(min=0).long()
    return blk * s["block"] + (pos % s["block"]).long()


def _plain_write(s):
    rows = torch.arange(s["k_new"].shape[0], device=DEV)
    req = torch.searchsorted(s["qsl"].long(), rows, right=True) - 1
    q0, q1 = s["qsl"].long()[req], s["qsl"].long()[req + 1]
    slot = _slots(s, s["seq_lens"].long()[req] - (q1 - q0) + (rows - q0), req)
    for t in ("k", "v"):
        codes, bs = _quantize(s[t + "_new"], s[t + "_scale"])
        s[t + "_fp4"].view(-1, s["hkv"], D // 2)[slot] = codes
        s[t + "_bscale"].view(-1, s["hkv"], D // GROUP)[slot] = bs


def _gather(s, t, slot):
    codes = s[t + "_fp4"].view(-1, s["hkv"], D // 2)[slot]
    bs = s[t + "_bscale"].view(-1, s["hkv"], D // GROUP)[slot]
    return _dequantize(codes, bs, s[t + "_scale"])


def _padded(s):
    pos = torch.arange(s["ctx"], device=DEV)
    req = torch.arange(s["reqs"], device=DEV)
    live = pos[None, :] < s["seq_lens"].long()[:, None]
    return _slots(s, pos[None, :].expand(s["reqs"], -1), req[:, None]), live


def _plain_read(s):
    slot, live = _padded(s)
    for t in ("k", "v"):
        v = _gather(s, t, slot).to(torch.bfloat16)
        s[t + "_dense"].copy_(torch.where(live[..., None, None], v, s[t + "_dense"]))


def _plain_attend(s):
    T, hkv, g = s["T"], s["hkv"], s["group"]
    slot, live = _padded(s)
    zero = torch.zeros((), device=DEV)
    q = s["q"].float().view(s["reqs"], T, hkv, g, D).permute(0, 2, 1, 3, 4).reshape(s["reqs"], hkv, T * g, D)
    k = torch.where(live[..., None, None], _gather(s, "k", slot), zero).permute(0, 2, 3, 1)
    w = torch.matmul(q, k) * s["softmax_scale"]
    del k
    pos = torch.arange(s["ctx"], device=DEV)
    last = s["seq_lens"].long()[:, None] - T + torch.arange(T, device=DEV)[None, :]  # the token's own position
    seen = (pos[None, None, :] <= last[:, :, None]) & live[:, None, :]
    seen = seen[:, None, :, None, :].expand(-1, 1, -1, g, -1).reshape(s["reqs"], 1, T * g, -1)
    w = w.masked_fill(~seen, -math.inf)
    m = w.amax(-1, keepdim=True)
    w = torch.exp(w - torch.where(torch.isinf(m), zero, m))
    total = w.sum(-1, keepdim=True)
    v = torch.where(live[..., None, None], _gather(s, "v", slot), zero).permute(0, 2, 1, 3)
    o = torch.matmul(w, v) / torch.where(total > 0, total, torch.ones_like(total))
    return o.view(s["reqs"], hkv, T, g, D).permute(0, 2, 1, 3, 4).reshape(s["reqs"] * T, hkv * g, D).to(torch.bfloat16)


# ------------------------------------------------------------------------------------------------
# the library's calls
# ------------------------------------------------------------------------------------------------

@functools.lru_cache(None)
def _workspace():
    """The attention's workspace, which a program keeps for all its calls on one stream."""
    import paged_kv_cache_int64_gb300 as pkv
    return torch.empty(pkv.spec_verify_fp4_workspace_bytes(), dtype=torch.uint8, device=DEV)


def _own_write(s):
    import paged_kv_cache_int64_gb300 as pkv
    pkv.kv_cache_write_fp4(s["k_new"], s["v_new"], s["bt"], s["seq_lens"], s["qsl"], s["max_new"], s["k_fp4"], s["v_fp4"],
                           s["k_bscale"], s["v_bscale"], s["k_scale"], s["v_scale"], dev_err=s["err"])


def _own_read(s):
    import paged_kv_cache_int64_gb300 as pkv
    pkv.kv_fp4_dequant_dense(s["k_fp4"], s["v_fp4"], s["k_bscale"], s["v_bscale"], s["bt"], s["zeros"], s["seq_lens"],
                             s["ctx"], s["k_scale"], s["v_scale"], s["k_dense"], s["v_dense"], dev_err=s["err"])


def _own_attend(s):
    import paged_kv_cache_int64_gb300 as pkv
    pkv.spec_verify_attn_fp4(s["q"], s["k_fp4"], s["v_fp4"], s["k_bscale"], s["v_bscale"], s["k_scale"], s["v_scale"],
                             s["bt"], s["seq_lens"], s["T"], s["softmax_scale"], s["out"], _workspace(), dev_err=s["err"])
    return s["out"]


# ------------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------------

def prepare(case, seed):
    c = case
    lens, new = _lens(c), _new_lens(c)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    order = np.random.RandomState(seed % (1 << 31))
    pages = [-(-n // c["block"]) for n in lens]
    nb = sum(pages) + 3
    perm, at = order.permutation(nb), 0
    bt = np.full((c["reqs"], max(1, max(pages))), -1, dtype=np.int32)
    for r, n in enumerate(pages):
        bt[r, :n] = perm[at:at + n]
        at += n
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)  # noqa: E731
    s = dict(op=c["op"], reqs=c["reqs"], ctx=max(lens), hkv=c["hkv"], group=c["group"], block=c["block"], T=c["new"],
             bt=torch.from_numpy(bt).to(DEV), seq_lens=i32(lens), zeros=i32([0] * len(lens)),
             qsl=i32([0] + np.cumsum(new).tolist()), max_new=max(new), softmax_scale=1.0 / math.sqrt(D),
             err=i32([0]))
    # K rows with channels of different sizes, V rows alike
    channel = {"k": torch.exp(0.6 * torch.randn(c["hkv"], D, generator=gen, device=DEV)), "v": torch.ones(c["hkv"], D, device=DEV)}
    for t in ("k", "v"):
        x = (torch.randn(nb * c["block"], c["hkv"], D, generator=gen, device=DEV) * channel[t]).to(torch.bfloat16)
        # a calibrated scale, with some room for rows that come later
        s[t + "_scale"] = (x.abs().amax().float() / (6.0 * 448.0) * 2.0 ** 0.1).reshape(1)
        codes, bs = _quantize(x, s[t + "_scale"])
        s[t + "_fp4"] = codes.view(nb, c["block"], c["hkv"], D // 2)
        s[t + "_bscale"] = bs.reshape(nb, c["block"], c["hkv"], D // GROUP)
        del x, codes, bs
        if c["op"] in ("append_attend", "write_read"):
            s[t + "_new"] = (torch.randn(sum(new), c["hkv"], D, generator=gen, device=DEV) * channel[t]).to(torch.bfloat16)
        if c["op"] in ("read", "write_read"):
            s[t + "_dense"] = torch.zeros(c["reqs"], max(lens), c["hkv"], D, dtype=torch.bfloat16, device=DEV)
    if c["op"] in ("attend", "append_attend"):
        s["q"] = torch.randn(c["reqs"] * c["new"], c["hkv"] * c["group"], D, generator=gen, device=DEV).to(torch.bfloat16)
        s["out"] = torch.empty_like(s["q"])
    return s


def run(state):
    s = state
    if s["op"] in ("append_attend", "write_read"):
        _own_write(s) if own else _plain_write(s)
    if s["op"] in ("read", "write_read"):
        _own_read(s) if own else _plain_read(s)
        return {"k": s["k_dense"], "v": s["v_dense"]}
    return {"out": _own_attend(s) if own else _plain_attend(s)}


# ------------------------------------------------------------------------------------------------
# from the definition, in 64 bits
# ------------------------------------------------------------------------------------------------

def _e4m3_values(byte):
    b = byte.double()
    e, m = torch.floor(b / 8) % 16, b % 8
    v = torch.where(e > 0, (1 + m / 8) * 2.0 ** (e - 7), m * 2.0 ** -9)
    return torch.where(b >= 128, -v, v)


def _stored(s, t, slot):
    """The values, in 64 bits, of the cache rows at `slot`."""
    codes = s[t + "_fp4"].view(-1, s["hkv"], D // 2)[slot].double()
    v = torch.empty(*codes.shape, 2, dtype=torch.float64, device=DEV)
    for half, n in enumerate((codes % 16, torch.floor(codes / 16))):
        m = n % 8
        a = torch.where(m < 2, m / 2, (2 + m % 2) * 2.0 ** (torch.floor(m / 2) - 2))
        v[..., half] = torch.where(n >= 8, -a, a)
    bs = _e4m3_values(s[t + "_bscale"].view(-1, s["hkv"], D // GROUP)[slot])
    return (v.view(*codes.shape[:-1], D // GROUP, GROUP) * bs[..., None]).flatten(-2) * s[t + "_scale"].double()


def _rounded(x, scale):
    """The values, in 64 bits, that the rows x stand for once they are quantized."""
    x = x.double().unflatten(-1, (D // GROUP, GROUP))
    g = scale.double()
    r = x.abs().amax(-1) / (6 * g)
    step = 2.0 ** (torch.floor(torch.log2(r.clamp(min=2.0 ** -6))) - 3)
    bs = (torch.round(r / step) * step).clamp(max=448.0)
    d = (bs * g)[..., None]
    a = torch.where(d > 0, x / d, torch.zeros_like(x)).abs()
    step = 2.0 ** (torch.floor(torch.log2(a.clamp(min=1.0))) - 1)
    a = (torch.round(a / step) * step).clamp(max=6.0)
    return (torch.sign(x) * a * d).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    lens, new = _lens(case), _new_lens(case)
    hkv, g, T = s["hkv"], s["group"], s["T"]
    out = {"k": [], "v": []} if case["op"] in ("read", "write_read") else []
    at = 0
    for r, n in enumerate(lens):
        pos = torch.arange(n, device=DEV)
        slot = _slots(s, pos, r) if n else pos
        val = {t: _stored(s, t, slot) for t in ("k", "v")}
        if case["op"] in ("append_attend", "write_read") and new[r]:
            for t in ("k", "v"):
                val[t][n - new[r]:] = _rounded(s[t + "_new"][at:at + new[r]], s[t + "_scale"])
            at += new[r]
        if case["op"] in ("read", "write_read"):
            for t in ("k", "v"):
                out[t].append(torch.cat((val[t], val[t].new_zeros(max(lens) - n, hkv, D))))
            continue
        q = s["q"][r * T:(r + 1) * T].double()
        for t in range(T):
            m = n - T + t + 1
            if m <= 0:
                out.append(torch.zeros(hkv * g, D, dtype=torch.float64, device=DEV))
                continue
            z = torch.einsum("hgd,nhd->hgn", q[t].view(hkv, g, D), val["k"][:m]) * s["softmax_scale"]
            out.append(torch.einsum("hgn,nhd->hgd", torch.softmax(z, -1), val["v"][:m]).reshape(hkv * g, D))
    if case["op"] in ("read", "write_read"):
        return {t: torch.stack(out[t]) for t in ("k", "v")}
    return {"out": torch.stack(out)}
