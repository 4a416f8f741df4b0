"""Attention on the HIP path where softmax weights and the sizes of the values
they meet differ by many powers of two: V scales of the INT4 cache from token to
token, a key that takes nearly all of the weight and has little value.  Against
plain 64-bit implementations, with a bound made of each row's own weights."""
import math

import numpy as np
import pytest
import torch

import attn_ref as ref
import oracle
import w4a16_bit_matmul_amd as wq
from parity import say
from test_gpu_attention import BF, HF, Cache, _run_cache, _run_prompt, _tables

pytestmark = pytest.mark.gpu

# A weight is rounded to fp16 relative to a reference point at most 2^-7 of the
# row's largest product of weight and V scale (scales enter as the power of two
# above them): half a step of fp16's subnormals there.
STEP = 2.0 ** -25 * 2.0 ** -7 * 2


def attend(q, k, v, s, seen, scale, dtype):
    """As attn_ref.attend, for one block of 128 values of v (or a head of 64): s
    [n] is its V scale of each token, v = s times integers up to 15.  The absolute
    part of a weight's rounding follows the largest weight times scale of the
    row, not the largest scale."""
    m, D = q.shape
    live = seen.any(-1)
    out, bound = torch.zeros((m, v.shape[1]), dtype=torch.float64), torch.zeros((m, v.shape[1]), dtype=torch.float64)
    if not bool(live.any()):
        return out, bound
    se = seen[live]
    sc = (q[live] @ k.T * scale).masked_fill(~se, -math.inf)
    big = q[live].abs() @ k.abs().T * scale
    mx = sc.amax(-1, keepdim=True)
    p = torch.exp(sc - mx)
    l = p.sum(-1, keepdim=True)
    o, mean_abs = p @ v / l, p @ v.abs() / l
    arg = (torch.where(se, mx - sc, torch.zeros_like(sc)) + mx.abs() + 90) * 1.4427  # (90: the powers of the scales)
    delta = (D + 8) * 2.0 ** -24 * big + 2.0 ** -23 * (2 + 2 * arg)
    n = k.shape[0]
    rel = (p * delta).sum(-1, keepdim=True) / l + n * 2.0 ** -24
    # (a scale of 0 counts as 2^-64)
    small = 15 * n * STEP * (p * s.clamp(min=2.0 ** -64)).amax(-1, keepdim=True) / l
    b = (ref.HALF[dtype] * o.abs() + ref.TINY[dtype] + (2.0 ** -11 + n * 2.0 ** -24) * mean_abs
         + (p * delta) @ v.abs() / l + rel * o.abs() + small)
    out[live], bound[live] = o, 1.01 * b
    return out, bound


# value e of eight neighbouring ones sits in this nibble of their 32-bit word
NIBBLE = [4 * (e % 2) + e // 2 for e in range(8)]


def _pack(q):
    """Codes [S][hd] (0..15) as the cache's bytes."""
    w = np.zeros((q.shape[0], q.shape[1] // 8), np.uint32)
    for e in range(8):
        w |= q[:, e::8].astype(np.uint32) << np.uint32(4 * NIBBLE[e])
    return w.view(np.uint8).reshape(q.shape[0], -1)


def _zeros(z):
    """Zero-points [S][blocks] as the cache's bytes."""
    out = np.zeros((z.shape[0], (z.shape[1] + 1) // 2), np.uint8)
    out |= z[:, 0::2]
    out[:, :z.shape[1] // 2] |= z[:, 1::2] << 4
    return out


def make_cache(seed, S, Hkv, D, pull, v_scale):
    """A cache whose scores and V scales are chosen: pull [S] in units of a score
    of about 1 (scores with the queries of `queries`, 0: random small ones),
    v_scale [S][blocks].  V's zero-points are low, so that values do not cancel."""
    rng = np.random.default_rng(seed)
    hd, nb = Hkv * D, Hkv * D // 128
    sign = rng.integers(0, 2, hd) * 2 - 1
    kq = rng.integers(0, 16, (S, hd))
    strong = pull != 0
    kq[strong] = np.where(sign * np.sign(pull[strong])[:, None] > 0, 15, 0)
    kz = np.where(strong[:, None], 7, rng.integers(6, 10, (S, nb)))
    # a row of codes 15 and 0 around 7 scores about 7.5 D times its scale, over sqrt(D)
    ks = np.where(strong[:, None], np.abs(pull)[:, None] / (7.5 * D ** 0.5), 0.01) * np.ones((1, nb))
    c = Cache.__new__(Cache)
    c.S, c.Hkv, c.D, c.hd = S, Hkv, D, hd
    v = (_pack(rng.integers(0, 16, (S, hd))), v_scale.astype(np.float16).view(np.uint16), _zeros(rng.integers(0, 4, (S, nb)).astype(np.uint8)))
    c.host = [(_pack(kq), ks.astype(np.float16).view(np.uint16), _zeros(kz.astype(np.uint8))), v]
    c.val = [torch.from_numpy(oracle.kv_dequant(x, S, hd)).view(S, Hkv, D).double() for x in c.host]
    c.sign = sign
    return c


def queries(seed, cache, T, Hq, dtype):
    rng = np.random.default_rng(seed)
    G = Hq // cache.Hkv
    sign = np.repeat(cache.sign.reshape(cache.Hkv, cache.D), G, axis=0)
    return torch.from_numpy((sign[None] * rng.uniform(0.9, 1.1, (T, Hq, cache.D))).astype(np.float32)).to(dtype)


def want(cache, q, table, page, lens, starts):
    """(out, bound) of every query row, block by block of 128 V values."""
    T, Hq, D = q.shape
    G = Hq // cache.Hkv
    out, bound = torch.zeros((T, Hq, D), dtype=torch.float64), torch.zeros((T, Hq, D), dtype=torch.float64)
    sv = torch.from_numpy(cache.host[1][1].view(np.float16).astype(np.float64))
    w = min(D, 128)
    for b, n in enumerate(lens):
        m = starts[b + 1] - starts[b]
        t = np.arange(n)
        rows = table[b][t // page].astype(np.int64) * page + t % page
        seen = torch.arange(n)[None, :] <= n - m + torch.arange(m)[:, None]
        s = slice(starts[b], starts[b + 1])
        for h in range(Hq):
            k, v = (x[rows, h // G] for x in cache.val)
            for d in range(0, D, w):
                out[s, h, d:d + w], bound[s, h, d:d + w] = attend(q[s, h].double(), k, v[:, d:d + w],
                                                                  sv[rows, (h // G * D + d) // 128], seen, D ** -0.5, q.dtype)
    return out, bound


def _check(cache, q, table, page, lens, starts, what, **kw):
    one = len(lens) == q.shape[0]
    o, b = want(cache, q, table, page, lens, starts)
    got, lse = _run_cache(cache.to_dev(), q.cuda(), table, page, lens, None if one else starts, **kw)
    ref.check(got, o, b, what)
    assert bool(torch.isfinite(lse).all())


# every kernel: sequences, queries of each, heads, and room for contexts (which picks it)
KERNELS = [
    (2, 1, 8, 1, 128, 256, "HP=1, RT=1, PK=1"), (2, 1, 64, 8, 64, 2 ** 20, "HP=4, RT=1, PK=2"), (2, 1, 16, 8, 64, 2 ** 20, "HP=4, RT=1, PK=4"),
    (2, 2, 40, 8, 64, 2 ** 20, "HP=2, RT=1, PK=1"), (2, 3, 48, 8, 64, 2 ** 20, "HP=2, RT=2, PK=1"), (2, 1, 64, 8, 128, 2 ** 20, "HP=2, RT=1, PK=2"),
    (2, 1, 18, 2, 128, 2 ** 20, "HP=2, RT=1, PK=1"), (2, 7, 24, 8, 128, 2 ** 20, "HP=1, RT=2, PK=1"), (2, 3, 8, 2, 256, 2 ** 20, "HP=1, RT=1, PK=1"),
    (3, 1, 6, 3, 256, 256, "HP=1, RT=1, PK=1"), (64, 16, 64, 8, 128, 256, "kv_chunk_kernel<D=128"), (64, 32, 32, 8, 64, 256, "kv_chunk_kernel<D=64")]


def _case(B, nq, Hq, Hkv, D, room, plan, page=16):
    p = wq.wq_kv_attention_plan(B * nq, Hq, Hkv, D, B, page, room, nq)
    assert plan in p, p
    say(f"{p} B={B} nq={nq} Hq={Hq} Hkv={Hkv}")
    lens = [200, 131, 170][:B] if B < 64 else [40 + b % 61 for b in range(B)]
    S = sum(-(-n // page) for n in lens) * page
    table = _tables(B, lens, page, S, width=room // page)
    return lens, S, table, [nq * b for b in range(B + 1)], page


@pytest.mark.parametrize("case", KERNELS)
@pytest.mark.parametrize("power", [14, 18, 27])
def test_one_token_with_a_large_v_scale_and_no_weight(case, power):
    """V scales of about 2^-12 and one token of 2^power times as much whose weight is
    e^-40: the others' weights keep their bits."""
    B, nq, Hq, Hkv, D, room, plan = case
    lens, S, table, starts, page = _case(*case)
    rng = np.random.default_rng(power)
    pull, vs = np.zeros(S), 2.0 ** -12 * rng.uniform(0.5, 1, (S, Hkv * D // 128))
    for b, n in enumerate(lens):
        t = n // 3
        row = table[b][t // page] * page + t % page
        pull[row], vs[row] = -40.0, 2.0 ** (power - 12)
    cache = make_cache(power + D, S, Hkv, D, pull, vs)
    _check(cache, queries(power, cache, B * nq, Hq, HF if power == 18 else BF), table, page, lens, starts, "out", max_context=room, max_queries=nq)


@pytest.mark.parametrize("case", [c for c in KERNELS if c[1] > 1])
def test_a_later_token_with_a_large_v_scale(case):
    """The last token's V scale is 2^27 times the others': queries before it do not
    see it and keep their bits."""
    B, nq, Hq, Hkv, D, room, plan = case
    lens, S, table, starts, page = _case(*case)
    rng = np.random.default_rng(D)
    vs = 2.0 ** -12 * rng.uniform(0.5, 1, (S, Hkv * D // 128))
    for b, n in enumerate(lens):
        vs[table[b][(n - 1) // page] * page + (n - 1) % page] = 2.0 ** 15
    cache = make_cache(D, S, Hkv, D, np.zeros(S), vs)
    _check(cache, queries(1, cache, B * nq, Hq, HF), table, page, lens, starts, "out", max_context=room, max_queries=nq)


@pytest.mark.parametrize("case", KERNELS)
@pytest.mark.parametrize("sink", [2.0 ** -24, 0.0])
def test_a_token_with_nearly_all_weight_and_no_value(case, sink):
    """The first token's score is 18 above the others' and its V scale fp16's smallest,
    or 0: what the others add is all of the output, with weights of e^-18."""
    B, nq, Hq, Hkv, D, room, plan = case
    lens, S, table, starts, page = _case(*case)
    rng = np.random.default_rng(D)
    pull, vs = np.zeros(S), 0.05 * rng.uniform(0.5, 1, (S, Hkv * D // 128))
    for b in range(B):
        pull[table[b][0] * page], vs[table[b][0] * page] = 18.0, sink
    cache = make_cache(D + 1, S, Hkv, D, pull, vs)
    _check(cache, queries(2, cache, B * nq, Hq, BF), table, page, lens, starts, "out", max_context=room, max_queries=nq)


@pytest.mark.parametrize("case", KERNELS)
@pytest.mark.parametrize("page", [16, 64])
def test_v_scales_over_all_of_fp16(case, page):
    """V scales spread over fp16's range from token to token and block to block (zeros
    among them; with fp16 outputs as far as those hold), scores from -30 to 30."""
    B, nq, Hq, Hkv, D, room, plan = case
    lens, S, table, starts, page = _case(*case, page=page)
    rng = np.random.default_rng(D + Hq)
    nb = Hkv * D // 128
    dtype = BF if nq > 1 else HF
    vs = np.where(rng.random((S, nb)) < 0.1, 0.0, np.exp2(rng.uniform(-24, 15.9 if dtype == BF else 11, (S, nb))))
    cache = make_cache(D + 2, S, Hkv, D, rng.uniform(-30, 30, S), vs)
    _check(cache, queries(3, cache, B * nq, Hq, dtype), table, page, lens, starts, "out", max_context=room, max_queries=nq)


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("first", [0, 1])
def test_two_blocks_of_a_head_or_two_heads_with_scales_far_apart(D, first):
    """One block's V scales are 2^33 times the other's: neither costs the other bits."""
    Hq, Hkv, page, n = 8, 256 // D, 16, 700
    S = -(-n // page) * page
    rng = np.random.default_rng(D)
    vs = rng.uniform(0.5, 1, (S, 2))
    vs[:, first] *= 2.0 ** 11
    vs[:, 1 - first] *= 2.0 ** -22
    cache = make_cache(D + 3, S, Hkv, D, np.zeros(S), vs)
    table = _tables(1, [n], page, S, width=2 ** 20 // page)
    for dtype in (BF, HF):
        _check(cache, queries(4, cache, 1, Hq, dtype), table, page, [n], [0, 1], f"out {dtype}", max_context=2 ** 20)


def test_a_sink_before_a_long_context():
    """131072 tokens behind a key that takes the weight (as often seen: the first
    token), shared out to many workgroups."""
    Hq, Hkv, D, page, n = 8, 1, 128, 64, 131072
    rng = np.random.default_rng(0)
    vs = 0.05 * rng.uniform(0.5, 1, (n, 1))
    vs[0] = 2.0 ** -20
    pull = np.zeros(n)
    pull[0] = 17.0
    cache = make_cache(9, n, Hkv, D, pull, vs)
    table = np.arange(n // page, dtype=np.int32)[None]
    _check(cache, queries(5, cache, 1, Hq, HF), table, page, [n], [0, 1], "out")


@pytest.mark.parametrize("n,Hq,Hkv,D", [(3000, 1, 1, 64), (3000, 2, 1, 128), (2100, 9, 9, 64), (2100, 9, 9, 128), (1500, 4, 4, 256), (900, 20, 20, 128)])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_a_prompt_behind_a_sink(n, Hq, Hkv, D, dtype):
    """The first key's score is 17 above the others' and its values are near 0: the
    output is the others', with weights of e^-17 (fp16: 2^-24.5)."""
    say(f"prompt behind a sink n={n} Hq={Hq} Hkv={Hkv} D={D} {dtype}")
    rng = np.random.default_rng(n + D)
    sign = rng.integers(0, 2, D) * 2 - 1
    q = torch.from_numpy((sign * rng.uniform(0.9, 1.1, (n, Hq, D))).astype(np.float32)).to(dtype)
    k = torch.from_numpy((0.05 * rng.standard_normal((n, Hkv, D))).astype(np.float32)).to(dtype)
    v = torch.from_numpy(rng.uniform(0.5, 1.5, (n, Hkv, D)).astype(np.float32)).to(dtype)
    k[0] = torch.from_numpy((sign * 17.0 / D ** 0.5).astype(np.float32)).to(dtype)
    v[0] = 2.0 ** -20
    got, _ = _run_prompt(q.cuda(), k.cuda(), v.cuda(), [0, n])
    got = got.double().cpu()
    seen = torch.tril(torch.ones((n, n), dtype=torch.bool))
    for h in range(0, Hq, 4):
        # the absolute part of a weight's rounding: half a step of fp16's subnormals at 2^-7 of
        # the largest weight (bf16 has none)
        kv = [x[:, h // (Hq // Hkv)].double() for x in (k, v)]
        o, b, _, _ = ref.attend(q[:, h].double(), *kv, seen, D ** -0.5, 2.0 ** -8 * float(v.abs().max()), dtype, ref.HALF[dtype])
        ref.check(got[:, h], o, b, f"head {h}")
