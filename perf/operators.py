"""What the attention-side operators next to the INT4 KV cache are measured on.

Three operators, in the order a layer runs them:

* ``norm_rope``: the norm of every query and key head and the rotation of its position, in one pass;
* ``prompt``: causal attention over whole prompts, packed one after another, with grouped heads;
* ``cache``: attention over the INT4 KV cache in pages (single tokens, a few tokens at once, a chunk of a prompt).

A case is a dict of plain values.  ``run`` computes it in plain torch (``own`` false) or through the library's
entry points (``own`` true).
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
_EPS = 1e-6


def _wq():
    import w4a16_bit_matmul_amd as wq
    return wq


# ---- the cases -----------------------------------------------------------------

def listed():
    return [
        # the decode step of 64 sequences of a 70B-style layer (64 query heads, 8 KV heads of 128)
        dict(name="norm_rope_decode", op="norm_rope", T=64, Hq=64, Hkv=8, D=128, rot=128, inter=False, dtype="bf16", far=131072),
        # a long prompt of the same layer
        dict(name="norm_rope_prompt", op="norm_rope", T=32768, Hq=64, Hkv=8, D=128, rot=128, inter=False, dtype="bf16", far=32768),
        # an odd number of tokens, narrow heads in groups of four, half of the channels rotated as neighbouring pairs
        dict(name="norm_rope_partial", op="norm_rope", T=4099, Hq=12, Hkv=3, D=64, rot=32, inter=True, dtype="f16", far=8192),
        # the first tokens of one conversation: the shortest call, latency alone
        dict(name="cache_one_short", op="cache", B=1, len_lo=201, len_hi=201, nq=1, Hq=64, Hkv=8, D=128, page=16, dtype="bf16"),
        # decode of 64 sequences with contexts up to 8K tokens
        dict(name="cache_decode_64", op="cache", B=64, len_lo=4097, len_hi=8192, nq=1, Hq=64, Hkv=8, D=128, page=64, dtype="bf16"),
        # one sequence that fills a 131072-row cache
        dict(name="cache_decode_long", op="cache", B=1, len_lo=131072, len_hi=131072, nq=1, Hq=64, Hkv=8, D=128, page=256, dtype="f16"),
        # draft tokens checked together: up to four queries a sequence, heads of 64, small pages
        dict(name="cache_few_tokens", op="cache", B=16, len_lo=999, len_hi=9001, nq=4, Hq=32, Hkv=8, D=64, page=16, dtype="f16"),
        # the next 512 tokens of two long prompts over what is already cached
        dict(name="cache_chunk", op="cache", B=2, len_lo=12000, len_hi=16384, nq=512, Hq=64, Hkv=8, D=128, page=64, dtype="bf16"),
        # a batch of short prompts, single tokens among them
        dict(name="prompt_short", op="prompt", B=48, len_lo=1, len_hi=300, Hq=64, Hkv=8, D=128, dtype="f16"),
        # ragged prompts, heads of 64 in groups of seven
        dict(name="prompt_ragged", op="prompt", B=16, len_lo=63, len_hi=1500, Hq=14, Hkv=2, D=64, dtype="f16"),
        # one 8K prompt
        dict(name="prompt_8k", op="prompt", B=1, len_lo=8192, len_hi=8192, Hq=64, Hkv=8, D=128, dtype="bf16"),
        # the largest: two prompts of around 12K tokens
        dict(name="prompt_long", op="prompt", B=2, len_lo=11001, len_hi=14000, Hq=64, Hkv=8, D=128, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "cache", "cache", "prompt"])
    D = rng.choice([64, 128, 128, 128, 256])
    Hkv = rng.choice([2, 3, 4, 8]) if D == 64 else rng.choice([1, 2, 3, 4, 8])
    if D == 64 and Hkv == 3:
        Hkv = 4  # a cache row is whole blocks of 128 values
    G = rng.choice([1, 2, 3, 4, 5, 7, 8])
    c = dict(op=op, Hq=Hkv * G, Hkv=Hkv, D=D, dtype=rng.choice(["bf16", "f16"]))
    if op == "norm_rope":
        heads = c["Hq"] + Hkv
        c["T"] = _log_int(rng, 1, min(32768, 32768 * 72 * 128 // (heads * D)))
        c["rot"] = rng.choice([D, D, D // 2, D // 4])
        c["inter"] = rng.random() < 0.5
        c["far"] = max(c["T"], _log_int(rng, 64, 131072))
        return c
    if op == "cache":
        c["nq"] = rng.choice([1, 1, 1, 2, 5, 8, _log_int(rng, 16, 512)])
        c["B"] = _log_int(rng, 1, 64) if c["nq"] <= 8 else rng.choice([1, 2])
        c["len_hi"] = _log_int(rng, 1, min(131072, 524288 // c["B"]) if c["nq"] <= 8 else 16384)
        c["len_lo"] = max(1, c["len_hi"] // rng.choice([1, 2, 10]))
        c["page"] = rng.choice([1, 4, 16, 32, 64, 256])
        return c
    c["B"] = _log_int(rng, 1, 64)
    # the squares of the lengths stay below those of one 13K prompt with 64 heads
    top = int(math.sqrt(1.7e8 * 64 * 128 / (c["B"] * c["Hq"] * D)))
    c["len_hi"] = _log_int(rng, 1, max(1, min(14000, top, 65536 // c["B"])))
    c["len_lo"] = max(1, c["len_hi"] // rng.choice([1, 2, 30]))
    return c


def _lengths(case):
    """The sequences' lengths: the case's own, not the seed's, so that every state of a case is the same work."""
    r = np.random.default_rng(case["B"] * 1000003 + case["len_hi"])
    n = r.integers(case["len_lo"], case["len_hi"] + 1, case["B"])
    n[int(r.integers(0, case["B"]))] = case["len_hi"]
    return [int(v) for v in n]


def _queries(case):
    """Queries of each sequence of a cache case (between one and nq, and nq in a chunk)."""
    lens = _lengths(case)
    if case["nq"] == 1:
        return [1] * len(lens)
    r = np.random.default_rng(case["B"] + 17 * case["nq"])
    if case["nq"] > 16:
        return [min(case["nq"], n) for n in lens]
    return [min(int(v), n) for v, n in zip(r.integers(1, case["nq"] + 1, len(lens)), lens)]


def work(case):
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    if case["op"] == "norm_rope":
        T, rows = case["T"], case["T"] * (Hq + Hkv)
        # q and k in and out, the cos and sin rows of every token, positions and weights
        return {"bytes": 2 * 2 * rows * D + 4 * T * case["rot"] + 4 * T + 2 * 2 * D,
                "flops": rows * (4 * D + 3 * case["rot"])}
    lens = _lengths(case)
    if case["op"] == "prompt":
        T = sum(lens)
        return {"bytes": 2 * T * D * (2 * Hq + 2 * Hkv) + 4 * (len(lens) + 1),
                "flops": 4 * D * Hq * sum(n * (n + 1) // 2 for n in lens)}
    hd = Hkv * D
    per_token = hd // 2 + 2 * (hd // 128) + (hd // 128 + 1) // 2
    nq = _queries(case)
    seen = sum(m * n - m * (m - 1) // 2 for m, n in zip(nq, lens))
    pages = sum(-(-n // case["page"]) for n in lens)
    return {"bytes": 2 * per_token * sum(lens) + 4 * pages + 4 * len(lens) + 2 * 2 * sum(nq) * Hq * D,
            "flops": 4 * D * Hq * seen}


# ---- inputs --------------------------------------------------------------------

def _normal(g, shape, dtype, scale=1.0, wide=0.0):
    """Normal values; a share `wide` of the channels is eight times larger in every row."""
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    if scale != 1.0:
        x *= scale
    if wide:
        ch = torch.rand(shape[1:], generator=g, device="cuda") < wide
        x *= torch.where(ch, 8.0, 1.0)
    return x.to(dtype)


# value e of eight neighbouring ones sits in this nibble of their 32-bit word
_NIBBLE = [4 * (e % 2) + e // 2 for e in range(8)]


def _int4_cache(g, S, hd, scale, wide):
    """An INT4 cache of S rows of hd values, quantized in blocks of 128: codes [S][hd/2] bytes, fp16 scales [S][hd/128],
    zero-points, two blocks a byte."""
    nb = hd // 128
    codes = torch.empty((S, hd // 2), dtype=torch.uint8, device="cuda")
    s_all = torch.empty((S, nb), dtype=torch.float16, device="cuda")
    zp = torch.zeros((S, (nb + 1) // 2), dtype=torch.uint8, device="cuda")
    ch = torch.where(torch.rand((hd,), generator=g, device="cuda") < wide, 8.0 * scale, scale)
    for r0 in range(0, S, 65536):
        r1 = min(S, r0 + 65536)
        x = (torch.randn((r1 - r0, hd), generator=g, device="cuda") * ch).view(r1 - r0, nb, 128)
        lo, hi = x.amin(-1, keepdim=True).clamp(max=0), x.amax(-1, keepdim=True).clamp(min=0)
        s = ((hi - lo) / 15).to(torch.float16)
        sf = s.float()
        inv = torch.where(sf > 0, 1.0 / sf, torch.zeros_like(sf))
        z = torch.round(-lo * inv).clamp(0, 15)
        q = torch.round(x * inv + z).clamp(0, 15).to(torch.int64).view(r1 - r0, hd // 8, 8)
        word = torch.zeros((r1 - r0, hd // 8), dtype=torch.int64, device="cuda")
        for e in range(8):
            word |= q[:, :, e] << (4 * _NIBBLE[e])
        for i in range(4):
            codes[r0:r1].view(-1, hd // 8, 4)[:, :, i] = ((word >> (8 * i)) & 255).to(torch.uint8)
        s_all[r0:r1] = s[:, :, 0]
        zi = z[:, :, 0].to(torch.uint8)
        zp[r0:r1] = zi[:, 0::2]
        zp[r0:r1, : nb // 2] |= zi[:, 1::2] << 4
    return codes, s_all, zp


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    dt = _DTYPES[case["dtype"]]
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    st = {"case": case}
    if case["op"] == "norm_rope":
        T, rot, far = case["T"], case["rot"], case["far"]
        # projections before their norm, of any size; weights around one
        st["q"] = _normal(g, (T, Hq, D), dt, 3.0, 0.01)
        st["k"] = _normal(g, (T, Hkv, D), dt, 2.0, 0.01)
        st["q_weight"] = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(dt)
        st["k_weight"] = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(dt)
        # the angles of far positions need 64 bits; the tables hold their cosines and sines in 32
        f = 10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64, device="cuda") * 2 / rot)
        ang = torch.arange(far, dtype=torch.float64, device="cuda")[:, None] * f
        st["cos"], st["sin"] = ang.cos().float(), ang.sin().float()
        # a prompt's tokens follow one another; the tokens of a decode step are anywhere
        pos = np.arange(T) + int(rng.integers(0, far - T + 1)) if T > 256 else rng.integers(0, far, T)
        st["positions"] = torch.from_numpy(pos.astype(np.int32)).cuda()
        return st
    lens = _lengths(case)
    if case["op"] == "prompt":
        T = sum(lens)
        st["q"] = _normal(g, (T, Hq, D), dt, 1.0, 0.01)
        st["k"] = _normal(g, (T, Hkv, D), dt, 1.0, 0.01)
        st["v"] = _normal(g, (T, Hkv, D), dt, 0.5)
        st["lens"] = lens
        st["seq_starts"] = torch.from_numpy(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)).cuda()
        return st
    page, hd, nq = case["page"], Hkv * D, _queries(case)
    pages = [-(-n // page) for n in lens]
    S = (sum(pages) + 3) * page
    order = rng.permutation(S // page)
    table = np.full((len(lens), max(pages)), -1, np.int32)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = order[at:at + n]
        at += n
    st["k_arrays"] = _int4_cache(g, S, hd, 1.0, 0.01)
    st["v_arrays"] = _int4_cache(g, S, hd, 0.5, 0.0)
    st["q"] = _normal(g, (sum(nq), Hq, D), dt)
    st["lens"], st["nq"], st["hd"], st["S"] = lens, nq, hd, S
    st["block_table"] = torch.from_numpy(table).cuda()
    st["context_lens"] = torch.from_numpy(np.array(lens, np.int32)).cuda()
    st["q_starts"] = torch.from_numpy(np.concatenate([[0], np.cumsum(nq)]).astype(np.int32)).cuda()
    if own:
        wq = _wq()
        st["k_cache"] = wq.KVCache(*st["k_arrays"], S, hd)
        st["v_cache"] = wq.KVCache(*st["v_arrays"], S, hd)
    return st


# ---- one pass ------------------------------------------------------------------

def run(st):
    return {"norm_rope": _run_norm_rope, "prompt": _run_prompt, "cache": _run_cache}[st["case"]["op"]](st)


def _run_norm_rope(st):
    c = st["case"]
    if own:
        return _wq().wq_qk_norm_rope(st["q"], st["k"], st["cos"], st["sin"], st["positions"], q_weight=st["q_weight"],
                                     k_weight=st["k_weight"], eps=_EPS, interleaved=c["inter"])
    at = st["positions"].long()
    cos, sin = st["cos"][at][:, None, :], st["sin"][at][:, None, :]
    rot, out = c["rot"], []
    for x, w in ((st["q"], st["q_weight"]), (st["k"], st["k_weight"])):
        n = x.float()
        n = n * torch.rsqrt((n * n).mean(-1, keepdim=True) + _EPS) * w.float()
        a, b = (n[..., 0:rot:2], n[..., 1:rot:2]) if c["inter"] else (n[..., : rot // 2], n[..., rot // 2: rot])
        a, b = a * cos - b * sin, b * cos + a * sin
        turned = torch.stack((a, b), -1).flatten(-2) if c["inter"] else torch.cat((a, b), -1)
        out.append(torch.cat((turned, n[..., rot:]), -1).to(x.dtype))
    return tuple(out)


def _attend(q, k, v, first, scale):
    """q [m][Hq][D], k and v [n][Hkv][D], all fp32: query i sees keys 0..first + i."""
    m, Hq, D = q.shape
    n, Hkv = k.shape[0], k.shape[1]
    kt, vh = k.permute(1, 2, 0).contiguous(), v.permute(1, 0, 2).contiguous()
    out = torch.empty_like(q)
    step = max(1, min(m, (1 << 28) // (Hq * n)))
    for i0 in range(0, m, step):
        i1 = min(m, i0 + step)
        e = min(n, first + i1)  # keys that some query of these sees
        qg = q[i0:i1].view(i1 - i0, Hkv, Hq // Hkv, D).permute(1, 0, 2, 3).reshape(Hkv, -1, D)
        p = torch.matmul(qg, kt[:, :, :e].contiguous()).view(Hkv, i1 - i0, Hq // Hkv, e) * scale
        hidden = torch.arange(e, device=q.device)[None, :] > first + torch.arange(i0, i1, device=q.device)[:, None]
        p = p.masked_fill(hidden[None, :, None, :], float("-inf"))
        p = torch.exp(p - p.amax(-1, keepdim=True))
        p = p / p.sum(-1, keepdim=True)
        o = torch.matmul(p.view(Hkv, -1, e), vh[:, :e].contiguous())
        out[i0:i1] = o.view(Hkv, i1 - i0, Hq // Hkv, D).permute(1, 0, 2, 3).reshape(i1 - i0, Hq, D)
    return out


def _run_prompt(st):
    if own:
        return _wq().wq_prompt_attention(st["q"], st["k"], st["v"], st["seq_starts"])
    D, at = st["case"]["D"], 0
    out = torch.empty_like(st["q"])
    for n in st["lens"]:
        s = slice(at, at + n)
        out[s] = _attend(st["q"][s].float(), st["k"][s].float(), st["v"][s].float(), 0, D ** -0.5).to(out.dtype)
        at += n
    return out


def _decode(arrays, rows, hd):
    """The named rows of a cache in fp32, [n][hd]."""
    codes, s, zp = (a[rows] for a in arrays)
    n, nb = rows.numel(), hd // 128
    b = codes.view(n, hd // 8, 4).int()
    word = b[:, :, 0] | (b[:, :, 1] << 8) | (b[:, :, 2] << 16) | (b[:, :, 3] << 24)
    q = torch.stack([(word >> (4 * k)) & 15 for k in _NIBBLE], -1).view(n, nb, 128)
    z = torch.stack((zp & 15, zp >> 4), -1).view(n, -1)[:, :nb].int()
    return ((q - z[:, :, None]).float() * s.float()[:, :, None]).view(n, hd)


def _rows(st, b):
    n, page = st["lens"][b], st["case"]["page"]
    t = torch.arange(n, device="cuda")
    return st["block_table"][b].long()[t // page] * page + t % page


def _run_cache(st):
    c = st["case"]
    if own:
        few = c["nq"] > 1
        return _wq().wq_kv_attention(st["q"], st["k_cache"], st["v_cache"], st["block_table"], st["context_lens"],
                                     page_size=c["page"], max_context=c["len_hi"],
                                     q_starts=st["q_starts"] if few else None, max_queries=c["nq"])
    out, at = torch.empty_like(st["q"]), 0
    for b, (n, m) in enumerate(zip(st["lens"], st["nq"])):
        rows = _rows(st, b)
        k, v = (_decode(st[a], rows, st["hd"]).view(n, c["Hkv"], c["D"]) for a in ("k_arrays", "v_arrays"))
        out[at:at + m] = _attend(st["q"][at:at + m].float(), k, v, n - m, c["D"] ** -0.5).to(out.dtype)
        at += m
    return out


# ---- the definition, in 64 bits --------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    D, Hq, Hkv = case["D"], case["Hq"], case["Hkv"]
    G = Hq // Hkv
    if case["op"] == "norm_rope":
        out = []
        c, s = (st[n].double()[st["positions"].long()] for n in ("cos", "sin"))
        r = case["rot"]
        first = torch.arange(0, r, 2) if case["inter"] else torch.arange(r // 2)
        second = first + (1 if case["inter"] else r // 2)
        for name in ("q", "k"):
            x = st[name].double()
            x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / D + _EPS) * st[name + "_weight"].double()
            y = x.clone()
            y[:, :, first.cuda()] = x[:, :, first.cuda()] * c[:, None] - x[:, :, second.cuda()] * s[:, None]
            y[:, :, second.cuda()] = x[:, :, second.cuda()] * c[:, None] + x[:, :, first.cuda()] * s[:, None]
            out.append(y)
        return tuple(out)
    lens = st["lens"]
    nq = st["nq"] if case["op"] == "cache" else lens
    out, at = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda"), 0
    for b, (n, m) in enumerate(zip(lens, nq)):
        if case["op"] == "cache":
            kv = []
            t = np.arange(n)
            rows = torch.from_numpy(st["block_table"][b].cpu().numpy()[t // case["page"]].astype(np.int64) * case["page"]
                                    + t % case["page"]).cuda()
            for name in ("k_arrays", "v_arrays"):
                codes, s, zp = (a.index_select(0, rows) for a in st[name])
                full = torch.empty((n, st["hd"]), dtype=torch.float64, device="cuda")
                for d in range(8):  # value d of every eight: byte and half of its word
                    byte = codes[:, _NIBBLE[d] // 2::4]
                    full[:, d::8] = (byte >> 4 if _NIBBLE[d] % 2 else byte & 15).double()
                for blk in range(st["hd"] // 128):
                    z = zp[:, blk // 2] >> 4 if blk % 2 else zp[:, blk // 2] & 15
                    cols = full[:, 128 * blk:128 * blk + 128]
                    cols.sub_(z.double()[:, None]).mul_(s[:, blk].double()[:, None])
                kv.append(full.view(n, Hkv, D))
            k, v = kv
        else:
            k, v = st["k"][at:at + n].double(), st["v"][at:at + n].double()
        for h in range(Hkv):
            kh, vh = k[:, h].t().contiguous(), v[:, h].contiguous()
            step = max(1, (1 << 26) // (n * G))
            for i0 in range(0, m, step):
                i1 = min(m, i0 + step)
                qh = st["q"][at + i0:at + i1, h * G:(h + 1) * G].double().reshape(-1, D)
                sc = (qh @ kh) / math.sqrt(D)
                last = n - m + torch.arange(i0, i1, device="cuda").repeat_interleave(G)
                sc[torch.arange(n, device="cuda")[None, :] > last[:, None]] = -math.inf
                out[at + i0:at + i1, h * G:(h + 1) * G] = (torch.softmax(sc, -1) @ vh).view(i1 - i0, G, D)
        at += m
    return out
