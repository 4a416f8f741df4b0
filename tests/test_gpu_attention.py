"""The operators next to the INT4 KV cache on the HIP path against plain 64-bit
implementations: head norm with rotation, causal attention over packed prompts,
attention over the cache in pages, and the three run together."""
import math

import numpy as np
import pytest
import torch

import attn_ref as ref
import oracle
import w4a16_bit_matmul_amd as wq
from parity import say

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16
NAN = float("nan")


# ---- norm and rotation -----------------------------------------------------------

def _rope_inputs(seed, T, Hq, Hkv, D, rot, dtype, P):
    q, k = ref.values(seed, (T, Hq, D), dtype, 3.0), ref.values(seed + 1, (T, Hkv, D), dtype, 0.5)
    rng = np.random.default_rng(seed + 2)
    w = [torch.from_numpy((1 + 0.3 * rng.standard_normal(D)).astype(np.float32)).to(dtype) for _ in range(2)]
    f = 10000.0 ** (-np.arange(rot // 2) * 2.0 / rot)
    ang = np.arange(P)[:, None] * f
    cos, sin = (torch.from_numpy(fn(ang).astype(np.float32)) for fn in (np.cos, np.sin))
    pos = torch.from_numpy(rng.integers(0, P, T).astype(np.int32))
    return q, k, w, cos, sin, pos


def _check_rope(got, x, w, cos, sin, pos, eps, inter, what, old=None):
    want, mag = ref.norm_rope(x, w, cos, sin, pos, eps, inter)
    bound = ref.norm_rope_bound(want, mag, x.dtype)
    pad = torch.isnan(want[:, 0, 0]) & ~torch.isnan(x.double()).any(-1).any(-1)
    got = got.cpu()
    if bool(pad.any()):
        assert torch.equal(got[pad].view(torch.int16), old[pad].view(torch.int16)), f"{what}: a padding row was written"
    ref.check(got[~pad], want[~pad], bound[~pad], what)


@pytest.mark.parametrize("T,Hq,Hkv,D,rot,inter", [
    (1, 1, 1, 128, 128, False), (64, 64, 8, 128, 128, False), (5, 3, 3, 64, 64, True), (33, 12, 3, 64, 32, False),
    (7, 14, 2, 64, 16, True), (19, 4, 1, 256, 256, False), (3, 5, 5, 256, 64, True), (2, 7, 1, 256, 128, False),
    (2501, 33, 1, 128, 96, False), (1025, 64, 8, 128, 128, True)])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_norm_rope(T, Hq, Hkv, D, rot, inter, dtype):
    say(f"norm rope T={T} Hq={Hq} Hkv={Hkv} D={D} rot={rot} inter={inter} {dtype}")
    q, k, w, cos, sin, pos = _rope_inputs(T + Hq, T, Hq, Hkv, D, rot, dtype, 777)
    dev = [t.cuda() for t in (q, k, cos, sin, pos, w[0], w[1])]
    qo, ko = wq.wq_qk_norm_rope(*dev[:5], q_weight=dev[5], k_weight=dev[6], eps=1e-5, interleaved=inter)
    torch.cuda.synchronize()
    _check_rope(qo, q, w[0], cos, sin, pos, 1e-5, inter, "q")
    _check_rope(ko, k, w[1], cos, sin, pos, 1e-5, inter, "k")


@pytest.mark.parametrize("inter", [False, True])
def test_norm_rope_slices_in_place_and_padding(inter):
    """q and k as slices of one fused projection, turned where they lie; tokens
    whose position is outside the table and the values between the slices keep
    their bytes; no weights."""
    T, Hq, Hkv, D = 37, 8, 2, 128
    q, k, _, cos, sin, pos = _rope_inputs(5, T, Hq, Hkv, D, 128, BF, 100)
    pos[3], pos[9], pos[36] = -1, 100, 2 ** 31 - 1
    fused = torch.full((T, (Hq + 2 * Hkv) * D + 8), 7.0, dtype=BF)
    fused[:, :Hq * D], fused[:, Hq * D:(Hq + Hkv) * D] = q.view(T, -1), k.view(T, -1)
    f = fused.cuda()
    qs, ks = f[:, :Hq * D].view(T, Hq, D), f[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D)
    wq.wq_qk_norm_rope(qs, ks, cos.cuda(), sin.cuda(), pos.cuda(), interleaved=inter, q_out=qs, k_out=ks)
    torch.cuda.synchronize()
    _check_rope(qs, q, None, cos, sin, pos, 1e-6, inter, "q", old=q)
    _check_rope(ks, k, None, cos, sin, pos, 1e-6, inter, "k", old=k)
    assert bool((f[:, (Hq + Hkv) * D:] == 7.0).all())


def test_norm_rope_far_positions_and_special_rows():
    """Positions whose rows lie past 2^31 bytes of the tables; rows of zeros, of
    the type's smallest and largest values; a NaN stays in its row."""
    T, D, P = 6, 128, 9_000_000
    q = ref.values(1, (T, 2, D), BF)
    q[0, 0], q[1, 0], q[2, 0], q[3, 1, 5] = 0.0, 1e-38, 1e18, NAN
    k = ref.values(2, (T, 1, D), BF)
    pos = torch.tensor([0, 1, P - 1, P - 2, 8_999_999 - 7, 5], dtype=torch.int32)
    cos, sin = torch.zeros((P, 64), device="cuda"), torch.zeros((P, 64), device="cuda")
    rows = torch.randn(T, 64)
    cos[pos.long().cuda()], sin[pos.long().cuda()] = rows.cos().cuda(), rows.sin().cuda()
    qo, ko = wq.wq_qk_norm_rope(q.cuda(), k.cuda(), cos, sin, pos.cuda())
    torch.cuda.synchronize()
    at = torch.arange(T, dtype=torch.int32)
    for got, x, what in ((qo, q, "q"), (ko, k, "k")):
        want, mag = ref.norm_rope(x, None, rows.cos(), rows.sin(), at, 1e-6, False)
        bound = ref.norm_rope_bound(want, mag, BF)
        nan = torch.isnan(want)
        assert torch.equal(torch.isnan(got.cpu()), nan), what
        ref.check(got.cpu().double().masked_fill(nan, 0), want.masked_fill(nan, 0), bound.masked_fill(nan, 0), what)


# ---- attention over packed prompts -------------------------------------------------

def _prompt_want(q, k, v, starts, scale):
    T, Hq, D = q.shape
    G = Hq // k.shape[1]
    half = ref.HALF[q.dtype]
    out, bound = torch.full((T, Hq, D), NAN, dtype=torch.float64), torch.zeros((T, Hq, D), dtype=torch.float64)
    lse, lb = torch.full((T, Hq), NAN, dtype=torch.float64), torch.zeros((T, Hq), dtype=torch.float64)
    none = torch.ones((T, Hq), dtype=torch.bool)
    for b in range(len(starts) - 1):
        s = slice(starts[b], starts[b + 1])
        none[s] = False
        n = starts[b + 1] - starts[b]
        seen = torch.tril(torch.ones((n, n), dtype=torch.bool))
        for h in range(Hq):
            vs = v[s, h // G].double()
            top = float(vs.abs().max()) if n else 0.0
            out[s, h], bound[s, h], lse[s, h], lb[s, h] = ref.attend(q[s, h].double(), k[s, h // G].double(), vs, seen, scale,
                                                                     top, q.dtype, half)
    return out, bound, lse, lb, none


def _check_rows(got, lse_got, want, old=7.0):
    """Rows of no sequence keep `old`; a row whose definition is NaN (an infinity
    in its query) is NaN."""
    out, bound, lse, lb, none = want
    got = got.cpu()
    assert bool((got[none] == old).all()), "a row of no sequence was written"
    nan = torch.isnan(lse) & ~none
    assert bool(torch.isnan(got[nan]).all())
    ref.check(got[~none & ~nan], out[~none & ~nan], bound[~none & ~nan], "out")
    if lse_got is not None:
        lse_got = lse_got.cpu().double()
        assert bool((lse_got[none] == old).all()), "an lse of no sequence was written"
        empty = torch.isinf(lse)
        assert bool(torch.isnan(lse_got[nan]).all())
        none = none | nan
        assert bool((lse_got[empty] == -math.inf).all()) and not bool(torch.isinf(lse_got[~empty & ~none]).any())
        ref.check(lse_got[~none & ~empty], lse[~none & ~empty], lb[~none & ~empty], "lse")


def _run_prompt(q, k, v, starts, scale=None, **kw):
    T, Hq, D = q.shape
    out = torch.full((T, Hq, D), 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full((T, Hq), 7.0, device="cuda")
    wq.wq_prompt_attention(q, k, v, torch.tensor(starts, dtype=torch.int32, device="cuda"), scale=scale, out=out, lse=lse, **kw)
    torch.cuda.synchronize()
    return out, lse


@pytest.mark.parametrize("lens,Hq,Hkv,D", [
    ([1], 1, 1, 128), ([1, 0, 2, 31, 0], 8, 1, 128), ([63, 64, 65], 2, 2, 128), ([127, 1, 128, 129], 4, 2, 64),
    ([300], 14, 2, 64), ([33, 200, 1], 3, 1, 256), ([257], 5, 5, 256), ([513, 90], 6, 2, 128), ([700], 64, 8, 128)])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_prompt_attention(lens, Hq, Hkv, D, dtype):
    say(f"prompt lens={lens} Hq={Hq} Hkv={Hkv} D={D} {dtype}")
    T = sum(lens)
    starts = [0] + list(np.cumsum(lens))
    starts = [int(x) for x in starts]
    q, k, v = (ref.values(T + i, (T, h, D), dtype, sc) for i, (h, sc) in enumerate(((Hq, 1.0), (Hkv, 1.0), (Hkv, 0.7))))
    got, lse = _run_prompt(q.cuda(), k.cuda(), v.cuda(), starts)
    _check_rows(got, lse, _prompt_want(q, k, v, starts, D ** -0.5))


def test_prompt_attention_many_sequences():
    """More sequences than a wave has lanes, some empty, with tokens before the
    first and behind the last."""
    rng = np.random.default_rng(3)
    lens = rng.integers(0, 12, 150)
    starts = [int(x) for x in 5 + np.concatenate([[0], np.cumsum(lens)])]
    T, Hq, Hkv, D = starts[-1] + 9, 2, 1, 64
    q, k, v = (ref.values(40 + i, (T, h, D), HF) for i, h in enumerate((Hq, Hkv, Hkv)))
    for t in (q, k, v):  # what lies outside every sequence must not matter
        t[:5], t[starts[-1]:] = NAN, NAN
    got, lse = _run_prompt(q.cuda(), k.cuda(), v.cuda(), starts, scale=0.3)
    _check_rows(got, lse, _prompt_want(q, k, v, starts, 0.3))


def test_prompt_attention_slices_and_large_scores():
    """q, k and v as slices of one fused tensor; scores far apart (weights that
    vanish) and large values."""
    lens, Hq, Hkv, D = [70, 133], 4, 2, 128
    T, starts = sum(lens), [0, 70, 203]
    fused = ref.values(9, (T, (Hq + 2 * Hkv) * D), HF, 4.0)
    f = fused.cuda()
    parts = [(0, Hq), (Hq, Hkv), (Hq + Hkv, Hkv)]
    dev = [f[:, a * D:(a + h) * D].view(T, h, D) for a, h in parts]
    cpu = [fused[:, a * D:(a + h) * D].reshape(T, h, D) for a, h in parts]
    got, lse = _run_prompt(*dev, starts, scale=1.0)
    _check_rows(got, lse, _prompt_want(*cpu, starts, 1.0))


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("bad", [NAN, math.inf, -math.inf])
def test_prompt_attention_later_tokens_do_not_reach_back(dtype, bad):
    """A NaN or an infinity in a key or value reaches its own query and later
    ones only; other sequences see nothing of it."""
    lens, Hq, Hkv, D = [90, 50], 4, 2, 128
    T, starts = 140, [0, 90, 140]
    q, k, v = (ref.values(70 + i, (T, h, D), dtype) for i, h in enumerate((Hq, Hkv, Hkv)))
    want = _prompt_want(q, k, v, starts, D ** -0.5)
    k[77, 0, 3], v[80, 1, 100], v[139, 0, 0] = bad, bad, bad
    got, _ = _run_prompt(q.cuda(), k.cuda(), v.cuda(), starts)
    got = got.cpu()
    out, bound = want[:2]
    ref.check(got[:77], out[:77], bound[:77], "before")
    ref.check(got[90:139], out[90:139], bound[90:139], "the next sequence")
    ref.check(got[80:90, 2:, :100], out[80:90, 2:, :100], bound[80:90, 2:, :100], "other channels")
    if math.isnan(bad):
        assert bool(torch.isnan(got[77:90, :2]).all())
    for t, h, c in ((80, slice(2, 4), 100), (89, slice(2, 4), 100), (139, slice(0, 2), 0)):
        x = got[t, h, c].double()
        assert bool((torch.isnan(x) if math.isnan(bad) else (x == bad) | torch.isnan(x)).all()), (t, x)


@pytest.mark.parametrize("lens,Hq,Hkv,D", [([40] * 60 + [0, 1, 129], 16, 8, 64), ([37] * 55 + [200], 6, 6, 128), ([530], 72, 72, 128),
                                           ([1200], 40, 20, 64), ([512, 700], 66, 33, 128)])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_prompt_attention_many_workgroups(lens, Hq, Hkv, D, dtype):
    """Prompts that fill the GPU, short and long: good values, then one value that
    is no number in a token that later ones see."""
    say(f"prompt, many workgroups: {len(lens)} of up to {max(lens)} Hq={Hq} Hkv={Hkv} D={D} {dtype}")
    starts = [int(x) for x in np.concatenate([[0], np.cumsum(lens)])]
    T = starts[-1]
    assert (T * (Hq // Hkv) // 128 + len(lens)) * Hkv >= 256
    q, k, v = (ref.values(T + i, (T, h, D), dtype, sc) for i, (h, sc) in enumerate(((Hq, 1.0), (Hkv, 1.0), (Hkv, 0.7))))
    want = _prompt_want(q, k, v, starts, D ** -0.5)
    got, lse = _run_prompt(q.cuda(), k.cuda(), v.cuda(), starts)
    _check_rows(got, lse, want)
    at, end, G = T - lens[-1] // 2, T, Hq // Hkv
    v[at, 1, 7] = math.inf
    got = _run_prompt(q.cuda(), k.cuda(), v.cuda(), starts)[0].cpu()
    hit = torch.zeros((T, Hq, D), dtype=torch.bool)
    hit[at:end, G:2 * G, 7] = True
    assert bool((torch.isnan(got[hit]) | torch.isinf(got[hit])).all())
    ref.check(got[~hit], want[0][~hit], want[1][~hit], "the others")


@pytest.mark.parametrize("D,n", [(64, 333), (128, 530), (256, 170)])
@pytest.mark.parametrize("bad", [NAN, math.inf])
def test_prompt_attention_values_that_are_no_numbers_in_longer_prompts(D, n, bad):
    """The same where a row walks many tiles (a prompt of 512 tokens or more with
    heads of 128 takes larger ones): bad values in a tile that all rows see, in one
    that some see, in the last token."""
    Hq, Hkv = 4, 2
    q, k, v = (ref.values(90 + i, (n, h, D), BF) for i, h in enumerate((Hq, Hkv, Hkv)))
    out, bound = _prompt_want(q, k, v, [0, n], D ** -0.5)[:2]
    at = n // 2
    v[at, 1, 5], v[n - 1, 0, D - 1] = bad, bad
    got = _run_prompt(q.cuda(), k.cuda(), v.cuda(), [0, n])[0].cpu()
    ref.check(got[:at], out[:at], bound[:at], "before")
    ref.check(got[at:n - 1, :2], out[at:n - 1, :2], bound[at:n - 1, :2], "other heads")
    keep = torch.ones(D, dtype=torch.bool)
    keep[5] = False
    ref.check(got[at:, 2:, keep], out[at:, 2:, keep], bound[at:, 2:, keep], "other channels")
    for x in (got[at:, 2:, 5], got[n - 1, :2, D - 1]):
        assert bool((torch.isnan(x) | (x == bad)).all())


# ---- attention over the cache ------------------------------------------------------

class Cache:
    """Host K and V caches of S rows (quantized by the oracle) and their device copies."""

    def __init__(self, seed, S, Hkv, D):
        self.S, self.Hkv, self.D, self.hd = S, Hkv, D, Hkv * D
        self.host, self.val = [], []
        for i, sc in enumerate((1.0, 0.5)):
            X = ref.values(seed + i, (S, self.hd), torch.float32, sc).numpy()
            c = oracle.kv_alloc(S, self.hd)
            oracle.kv_quantize(X, c)
            self.host.append(c)
            self.val.append(torch.from_numpy(oracle.kv_dequant(c, S, self.hd)).view(S, Hkv, D).double())

    def to_dev(self, keep=None):
        """keep: rows that are attended; the others get codes, NaN and infinite
        scales and zero-points that must not matter."""
        out = []
        for c in self.host:
            codes, s, z = (a.copy() for a in c)
            if keep is not None:
                junk = np.ones(self.S, bool)
                junk[keep] = False
                codes[junk], z[junk] = 0xA7, 0xFF
                s[junk] = np.where(np.arange(self.S)[:, None] % 2, 0x7C00, 0x7E00)[junk]
            d = wq.kv_cache_alloc(self.S, self.hd)
            d.codes.copy_(torch.from_numpy(codes))
            d.s.copy_(torch.from_numpy(s.view(np.int16)).view(torch.float16))
            d.zpacked.copy_(torch.from_numpy(z))
            out.append(d)
        return out

    def v_scale(self, rows):
        s = self.host[1][1].view(np.float16).astype(np.float64)
        return float(s[rows].max()) if len(rows) else 0.0


def _cache_want(cache, q, table, page, lens, starts, scale, max_context=None):
    T, Hq, D = q.shape
    G = Hq // cache.Hkv
    pages = cache.S // page
    out, bound = torch.full((T, Hq, D), NAN, dtype=torch.float64), torch.zeros((T, Hq, D), dtype=torch.float64)
    lse, lb = torch.full((T, Hq), NAN, dtype=torch.float64), torch.zeros((T, Hq), dtype=torch.float64)
    used = []
    none = torch.ones((T, Hq), dtype=torch.bool)
    for b, n in enumerate(lens):
        if max_context is not None:
            n = min(n, max_context)
        q0, q1 = starts[b], starts[b + 1]
        m = q1 - q0
        none[q0:q1] = False
        t = np.arange(max(n, 0))
        pg = table[b][t // page]
        ok = (pg >= 0) & (pg < pages)
        rows = np.where(ok, pg.astype(np.int64) * page + t % page, 0)
        used.append(rows[ok])
        seen = torch.from_numpy(ok)[None, :] & (torch.from_numpy(t)[None, :] <= n - m + torch.arange(m)[:, None])
        for h in range(Hq):
            kv = [x[rows, h // G] for x in cache.val]
            out[q0:q1, h], bound[q0:q1, h], lse[q0:q1, h], lb[q0:q1, h] = ref.attend(
                q[q0:q1, h].double(), kv[0], kv[1], seen, scale, 15 * cache.v_scale(rows[ok]), q.dtype, 2.0 ** -11)
    return (out, bound, lse, lb, none), np.unique(np.concatenate(used)) if used else np.zeros(0, np.int64)


def _run_cache(dev, q, table, page, lens, starts, **kw):
    T, Hq, D = q.shape
    out = torch.full((T, Hq, D), 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full((T, Hq), 7.0, device="cuda")
    one = starts is None
    wq.wq_kv_attention(q, *dev, torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"),
                       page_size=page, q_starts=None if one else torch.tensor(starts, dtype=torch.int32, device="cuda"),
                       out=out, lse=lse, **kw)
    torch.cuda.synchronize()
    return out, lse


def _tables(seed, lens, page, S, width=None):
    rng = np.random.default_rng(seed)
    need = [max(0, -(-n // page)) for n in lens]
    order = rng.permutation(S // page)
    assert sum(need) <= len(order)
    t = np.full((len(lens), width or max(1, max(need))), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        t[b, :n] = order[at:at + n]
        at += n
    return t


@pytest.mark.parametrize("lens,Hq,Hkv,D,page", [
    ([1], 1, 1, 128, 1), ([31, 32, 33, 0, 1], 8, 1, 128, 16), ([64, 100], 16, 2, 64, 32), ([7, 300], 32, 1, 128, 64),
    ([50, 0, 129], 6, 3, 256, 8), ([200, 77], 4, 4, 64, 4), ([513], 64, 8, 128, 128), ([90, 260], 40, 8, 256, 32),
    ([260, 1025], 17, 1, 128, 2)])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_cache_attention_single_tokens(lens, Hq, Hkv, D, page, dtype):
    say(f"cache lens={lens} Hq={Hq} Hkv={Hkv} D={D} page={page} {dtype}")
    B = len(lens)
    S = sum(-(-n // page) for n in lens) * page + 3 * page + (page - 1)  # a tail that is no whole page
    cache = Cache(sum(lens) + D, S, Hkv, D)
    table = _tables(B, lens, page, S)
    q = ref.values(B + Hq, (B, Hq, D), dtype)
    want, used = _cache_want(cache, q, table, page, lens, list(range(B + 1)), D ** -0.5)
    got, lse = _run_cache(cache.to_dev(used), q.cuda(), table, page, lens, None)
    _check_rows(got, lse, want)


@pytest.mark.parametrize("lens,nq,Hq,Hkv,D,page", [
    ([40, 3, 0, 100], [2, 3, 0, 4], 8, 1, 128, 16), ([5, 64], [9, 2], 4, 1, 128, 32), ([333], [33], 6, 2, 64, 64),
    ([150, 1], [17, 1], 3, 1, 256, 8), ([600], [200], 8, 1, 128, 64), ([96, 20], [5, 5], 64, 8, 128, 4)])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_cache_attention_several_tokens(lens, nq, Hq, Hkv, D, page, dtype):
    """Several queries of a sequence (more than it has tokens among them: those
    see nothing), rows of queries before the first and behind the last sequence."""
    say(f"cache lens={lens} nq={nq} Hq={Hq} Hkv={Hkv} D={D} page={page} {dtype}")
    starts = [int(x) for x in 2 + np.concatenate([[0], np.cumsum(nq)])]
    S = sum(-(-n // page) for n in lens) * page + 2 * page
    cache = Cache(sum(lens) + D, S, Hkv, D)
    table = _tables(len(lens), lens, page, S)
    q = ref.values(Hq, (starts[-1] + 3, Hq, D), dtype)
    want, used = _cache_want(cache, q, table, page, lens, starts, D ** -0.5)
    got, lse = _run_cache(cache.to_dev(used), q.cuda(), table, page, lens, starts)
    _check_rows(got, lse, want)


@pytest.mark.parametrize("B,most,Hq,Hkv,D,page", [(66, 125, 8, 8, 128, 16), (37, 12, 160, 16, 128, 64), (64, 250, 4, 4, 64, 1), (86, 33, 18, 6, 64, 32),
                                                  (171, 101, 3, 3, 128, 4)])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_cache_attention_many_rows(B, most, Hq, Hkv, D, page, dtype):
    """Many sequences with up to `most` queries each (the kernel for many rows):
    none or one among them, more queries than tokens, pages that are gone, page
    numbers behind the cache, lengths past max_context."""
    say(f"cache many rows B={B} most={most} Hq={Hq} Hkv={Hkv} D={D} page={page} {dtype}")
    rng = np.random.default_rng(B + D)
    nq = [0, 1, most, most] + [int(x) for x in rng.integers(0, most + 1, B - 4)]
    lens = [5, 1, most // 2, 300] + [int(x) for x in rng.integers(0, 170, B - 4)]
    starts = [int(x) for x in 1 + np.concatenate([[0], np.cumsum(nq)])]
    S = (sum(-(-n // page) for n in lens) + 3) * page
    cache = Cache(B + D, S, Hkv, D)
    table = _tables(B, lens, page, S)
    for b in range(5, B, 3):  # a page in the middle, or all of them
        gone = [lens[b] // 2 // page] if b % 2 else list(range(table.shape[1]))
        table[b, gone] = [-1, S // page, 2 ** 31 - 1, -2 ** 31][b % 4]
    q = ref.values(Hq, (starts[-1] + 2, Hq, D), dtype)
    cut = min(250, table.shape[1] * page)
    assert "kv_chunk_kernel" in wq.wq_kv_attention_plan(q.shape[0], Hq, Hkv, D, B, page, cut, most)
    want, used = _cache_want(cache, q, table, page, lens, starts, D ** -0.5, max_context=cut)
    got, lse = _run_cache(cache.to_dev(used), q.cuda(), table, page, lens, starts, max_context=cut, max_queries=most)
    _check_rows(got, lse, want)


@pytest.mark.parametrize("page", [16, 64])
def test_cache_attention_missing_pages_and_bounds(page):
    """Pages outside the cache (evicted ones) are not attended, a sequence whose
    pages are all gone gives zeros; lengths past max_context are cut there; the
    same page may serve two sequences, or one twice."""
    lens, Hq, Hkv, D = [150, 300, 64, 1000], 8, 2, 128
    S = 24 * page + 5
    cache = Cache(page, S, Hkv, D)
    rng = np.random.default_rng(page)
    table = rng.integers(0, S // page, (4, -(-320 // page))).astype(np.int32)
    table[0, 1], table[1, 2], table[1, 0] = -1, S // page, 2 ** 31 - 1
    table[2, :] = -5
    table[3, 1] = table[3, 0]
    q = ref.values(3, (4, Hq, D), BF)
    want, used = _cache_want(cache, q, table, page, lens, list(range(5)), 0.2, max_context=310)
    got, lse = _run_cache(cache.to_dev(used), q.cuda(), table, page, lens, None, scale=0.2, max_context=310)
    _check_rows(got, lse, want)
    assert bool((got[2] == 0).all())


@pytest.mark.parametrize("B,n,Hq,Hkv,D,page,nq", [(1, 9000, 8, 1, 128, 64, 1), (3, 4500, 4, 4, 64, 16, 1), (2, 5000, 4, 1, 256, 32, 1),
                                                 (1, 7000, 16, 8, 128, 32, 1), (2, 4000, 8, 2, 128, 16, 3)])
def test_cache_attention_long_contexts_are_split_and_joined(B, n, Hq, Hkv, D, page, nq):
    lens = [n - 1111 * b for b in range(B)]
    plan = wq.wq_kv_attention_plan(B * nq, Hq, Hkv, D, B, page, n, nq)
    say(plan)
    S = sum(-(-x // page) for x in lens) * page
    cache = Cache(n, S, Hkv, D)
    table = _tables(B, lens, page, S)
    q = ref.values(n, (B * nq, Hq, D), HF)
    starts = [nq * b for b in range(B + 1)]
    want, _ = _cache_want(cache, q, table, page, lens, starts, D ** -0.5)
    need = wq.wq_kv_attention_workspace_bytes(B * nq, Hq, Hkv, D, B, page, n, nq)
    assert (need > 0) == ("splits=1" not in plan.split()[-1:])
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")  # NaNs: no content is needed
    kw = dict(max_context=n, workspace=ws) if nq == 1 else dict(max_context=n, workspace=ws, max_queries=nq)
    got, lse = _run_cache(cache.to_dev(), q.cuda(), table, page, lens, None if nq == 1 else starts, **kw)
    _check_rows(got, lse, want)
    again, lse2 = _run_cache(cache.to_dev(), q.cuda(), table, page, lens, None if nq == 1 else starts, **kw)
    assert torch.equal(got, again) and torch.equal(lse, lse2)  # the same bits


@pytest.mark.parametrize("B,nq,most,room", [(3, 6, 4, 256), (2, 9, 2, 2 ** 20), (66, 140, 126, 256)])
def test_cache_attention_computes_the_first_max_queries(B, nq, most, room):
    """Sequences with more queries than are computed: the first ones are, and see
    what they would see among all; the rows of the others stay as they were."""
    Hq, Hkv, D, page = 8, 8, 128, 16
    lens, starts = [nq + 3 * b % 50 for b in range(B)], [nq * b for b in range(B + 1)]
    S = B * 16 * page
    cache = Cache(nq, S, Hkv, D)
    table = _tables(1, lens, page, S, width=room // page)
    q = ref.values(Hq, (starts[-1], Hq, D), HF)
    out, bound, lse, lb, none = _cache_want(cache, q, table, page, lens, starts, D ** -0.5)[0]
    none[torch.arange(starts[-1]) % nq >= most] = True
    got, got_lse = _run_cache(cache.to_dev(), q.cuda(), table, page, lens, starts, max_queries=most)
    _check_rows(got, got_lse, (out, bound, lse, lb, none))


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("Hq,Hkv,D,nq,plan", [
    (64, 8, 64, 1, "HP=4, RT=1, PK=2"), (12, 4, 64, 2, "HP=4, RT=1, PK=2"),
    (16, 8, 64, 1, "HP=4, RT=1, PK=4"), (8, 8, 64, 4, "HP=4, RT=1, PK=4"), (14, 2, 64, 1, "HP=2, RT=1, PK=2"), (40, 8, 64, 2, "HP=2, RT=1, PK=1"),
    (48, 8, 64, 3, "HP=2, RT=2, PK=1"), (64, 8, 128, 1, "HP=2, RT=1, PK=2"), (12, 4, 128, 2, "HP=2, RT=1, PK=2"), (18, 2, 128, 1, "HP=2, RT=1, PK=1"),
    (15, 5, 128, 5, "HP=1, RT=1, PK=1"), (24, 8, 128, 7, "HP=1, RT=2, PK=1"), (40, 4, 256, 3, "HP=1, RT=1, PK=1")])
def test_cache_attention_kernels_of_long_contexts(Hq, Hkv, D, nq, plan, page):
    """Room for a million tokens (which picks the kernel) with short and long
    contexts in it: heads that share a wave or a tile of rows differ in their
    scales by orders of magnitude."""
    say(f"cache room for long contexts Hq={Hq} Hkv={Hkv} D={D} nq={nq} page={page}")
    lens, width = [700, 0, 3, 1300, 129], 2 ** 20 // page
    starts = [0, nq, nq, 2 * nq, 3 * nq, 4 * nq] if nq > 1 else list(range(6))
    S = 2304
    cache = Cache(D + nq, S, Hkv, D)
    for i in range(2):
        X = ref.values(D + i, (S, Hkv, D), torch.float32).numpy() * (10.0 ** (np.arange(Hkv) % 4 - 2.0))[None, :, None].astype(np.float32)
        oracle.kv_quantize(np.ascontiguousarray(X.reshape(S, -1), np.float32), cache.host[i])
        cache.val[i] = torch.from_numpy(oracle.kv_dequant(cache.host[i], S, Hkv * D)).view(S, Hkv, D).double()
    table = _tables(D, lens, page, S, width=width)
    table[3, 700 // page] = -1
    q = ref.values(Hq, (starts[-1], Hq, D), HF)
    assert plan in wq.wq_kv_attention_plan(q.shape[0], Hq, Hkv, D, 5, page, 2 ** 20, nq)
    want, used = _cache_want(cache, q, table, page, lens, starts, D ** -0.5)
    got, lse = _run_cache(cache.to_dev(used), q.cuda(), table, page, lens, None if nq == 1 else starts, max_queries=nq)
    _check_rows(got, lse, want)


@pytest.mark.parametrize("Hq,Hkv,D,room", [(8, 2, 128, 128), (8, 2, 128, 2 ** 18), (4, 4, 64, 2 ** 18), (3, 1, 256, 256)])
def test_cache_attention_more_sequences_than_are_shared_out(Hq, Hkv, D, room):
    """300 sequences: a workgroup for each and its heads, however long they may be."""
    rng = np.random.default_rng(D)
    lens = [int(x) for x in rng.integers(0, 100, 300)]
    page, S = 32, 300 * 128
    cache = Cache(D, S, Hkv, D)
    table = _tables(D, lens, page, S, width=room // page)
    q = ref.values(Hq, (300, Hq, D), BF)
    assert wq.wq_kv_attention_plan(300, Hq, Hkv, D, 300, page, room, 1).endswith("whole units")
    want, used = _cache_want(cache, q, table, page, lens, list(range(301)), D ** -0.5)
    got, lse = _run_cache(cache.to_dev(used), q.cuda(), table, page, lens, None)
    _check_rows(got, lse, want)


@pytest.mark.parametrize("dtype,qs,ks,vs", [(BF, 1e30, 1e-3, 1e-4), (HF, 3e4, 1e-4, 1e-4), (BF, 1e-30, 1e3, 1e3), (HF, 1e-4, 1.0, 2e4),
                                            (BF, 1.0, 1.0, 1e-6), (HF, 1e4, 1e-3, 1e3)])
def test_cache_attention_value_ranges(dtype, qs, ks, vs):
    """Queries and cache values far from one: q in all of its type's range (infinite
    ones too, whose rows are NaN), K and V scales down to fp16's subnormals and up
    to its largest."""
    lens, Hq, Hkv, D, page = [70], 4, 1, 128, 16
    S = 80
    cache = Cache(2, S, Hkv, D)
    for i, sc in enumerate((ks, vs)):
        X = ref.values(60 + i, (S, D), torch.float32, sc, wide=0).numpy()
        X[::2] *= 0.05  # scales that differ from token to token
        oracle.kv_quantize(X, cache.host[i])
        cache.val[i] = torch.from_numpy(oracle.kv_dequant(cache.host[i], S, D)).view(S, Hkv, D).double()
    table = np.arange(5, dtype=np.int32)[None]
    q = ref.values(1, (1, Hq, D), torch.float32, qs, wide=0).to(dtype)
    scale = 2.0 / (D ** 0.5 * qs * ks)
    want, _ = _cache_want(cache, q, table, page, lens, [0, 1], float(np.float32(scale)))
    got, lse = _run_cache(cache.to_dev(), q.cuda(), table, page, lens, None, scale=scale)
    _check_rows(got, lse, want)


def test_cache_attention_nan_query_stays_in_its_row():
    cache = Cache(4, 64, 1, 128)
    q = ref.values(1, (2, 8, 128), BF)
    table = np.array([[0, 1], [2, 3]], np.int32)
    want, _ = _cache_want(cache, q, table, 16, [30, 20], [0, 1, 2], 0.1)
    q[0, 3, 17], q[1, 0, 0] = NAN, math.inf
    got, _ = _run_cache(cache.to_dev(), q.cuda(), table, 16, [30, 20], None, scale=0.1)
    got = got.cpu()
    assert bool(torch.isnan(got[0, 3]).all()) and bool(torch.isnan(got[1, 0]).any())
    keep = torch.ones((2, 8), dtype=torch.bool)
    keep[0, 3] = keep[1, 0] = False
    ref.check(got[keep], want[0][keep], want[1][keep], "other rows")


@pytest.mark.parametrize("nq,scale", [(3, 1e-20), (150, 1e-38), (3, 0.1)])
def test_cache_attention_zero_queries_with_small_scales(nq, scale):
    """Queries of zeros, whatever the scale: the mean of what they see."""
    lens, Hq, Hkv, D, page = [170, 200], 4, 1, 128, 16
    cache = Cache(5, 32 * page, Hkv, D)
    table = _tables(5, lens, page, 32 * page)
    table[0, 2] = -1
    q = ref.values(3, (2 * nq, Hq, D), HF)
    q[::2] = 0
    want, used = _cache_want(cache, q, table, page, lens, [0, nq, 2 * nq], float(np.float32(scale)))
    got, lse = _run_cache(cache.to_dev(used), q.cuda(), table, page, lens, [0, nq, 2 * nq], scale=scale)
    _check_rows(got, lse, want)


def test_cache_attention_rows_past_2_31_bytes():
    """A cache whose code bytes pass 2^32: pages at its start and its end."""
    Hkv, D, page = 8, 256, 64
    S = (2 ** 32 + 2 ** 26) // (Hkv * D // 2) // page * page
    small = Cache(6, 4 * page, Hkv, D)
    dev = []
    for c in small.host:
        d = wq.KVCache(torch.zeros((S, Hkv * D // 2), dtype=torch.uint8, device="cuda"),
                       torch.zeros((S, Hkv * D // 128), dtype=torch.float16, device="cuda"),
                       torch.zeros((S, Hkv * D // 256), dtype=torch.uint8, device="cuda"), S, Hkv * D)
        at = torch.cat([torch.arange(2 * page), torch.arange(S - 2 * page, S)]).cuda()
        d.codes[at], d.zpacked[at] = torch.from_numpy(c[0]).cuda(), torch.from_numpy(c[2]).cuda()
        d.s[at] = torch.from_numpy(c[1].view(np.int16)).view(torch.float16).cuda()
        dev.append(d)
    lens = [4 * page - 5]
    q = ref.values(2, (1, 16, D), BF)
    want, _ = _cache_want(small, q, np.array([[3, 0, 2, 1]], np.int32), page, lens, [0, 1], D ** -0.5)
    last = S // page - 1
    for pg in (page, 16):  # the paths of whole-tile and of small pages
        k = page // pg
        big = np.array([[x * k + i for x in (last, 0, last - 1, 1) for i in range(k)]], np.int32)
        got, lse = _run_cache(dev, q.cuda(), big, pg, lens, None)
        _check_rows(got, lse, want)


# ---- together, on streams and in graphs ----------------------------------------------

class Layer:
    """One attention layer's path: fused projection -> norm and rotation -> prompt
    attention, quantization into pages -> decode over the cache."""

    def __init__(self, lens, Hq=8, Hkv=2, D=128, page=16, dtype=BF, room=8):
        self.lens, self.Hq, self.Hkv, self.D, self.page, self.dtype = lens, Hq, Hkv, D, page, dtype
        B = len(lens)
        need = [-(-(n + room) // page) for n in lens]
        S = sum(need) * page
        self.caches = [wq.kv_cache_alloc(S, Hkv * D) for _ in range(2)]
        order = np.random.default_rng(B).permutation(sum(need)).astype(np.int32)
        self.table = np.full((B, max(need)), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        ang = np.arange(512)[:, None] * 10000.0 ** (-np.arange(D // 2) * 2.0 / D)
        self.cos, self.sin = (torch.from_numpy(f(ang).astype(np.float32)).cuda() for f in (np.cos, np.sin))
        self.w = [ref.values(i, (D,), dtype, 0.2, wide=0).add_(1).cuda() for i in range(2)]

    def slots(self, b, t):
        return self.table[b][t // self.page] * self.page + t % self.page

    def split(self, fused):
        T, D = fused.shape[0], self.D
        a, b = self.Hq * D, (self.Hq + self.Hkv) * D
        return fused[:, :a].view(T, -1, D), fused[:, a:b].view(T, -1, D), fused[:, b:].view(T, -1, D)

    def rope(self, fused, pos):
        q, k, v = self.split(fused)
        q, k = wq.wq_qk_norm_rope(q, k, self.cos, self.sin, pos, q_weight=self.w[0], k_weight=self.w[1])
        return q, k, v

    def append(self, k, v, slot):
        for x, c in ((k, self.caches[0]), (v, self.caches[1])):
            wq.wq_kv_quantize(x.reshape(x.shape[0], -1).contiguous(), c, slot=slot)


def test_a_layer_from_prompt_to_decode():
    """Prompts through all of the operators, then three decode steps; every
    attention against the plain form on what went in."""
    lens = [37, 1, 130]
    ly = Layer(lens)
    T, B = sum(lens), len(lens)
    starts = [0, 37, 38, 168]
    fused = ref.values(1, (T, (ly.Hq + 2 * ly.Hkv) * ly.D), ly.dtype).cuda()
    pos = torch.from_numpy(np.concatenate([np.arange(n) for n in lens]).astype(np.int32)).cuda()
    q, k, v = ly.rope(fused, pos)
    st = torch.tensor(starts, dtype=torch.int32, device="cuda")
    out = wq.wq_prompt_attention(q, k, v, st)
    slot = np.concatenate([ly.slots(b, np.arange(n)) for b, n in enumerate(lens)]).astype(np.int32)
    ly.append(k, v, torch.from_numpy(slot).cuda())
    torch.cuda.synchronize()
    want = _prompt_want(q.cpu(), k.cpu(), v.cpu(), starts, ly.D ** -0.5)
    _check_rows(out, None, want)
    table = torch.from_numpy(ly.table).cuda()
    view = Cache.__new__(Cache)
    view.S, view.Hkv, view.D, view.hd = ly.caches[0].S, ly.Hkv, ly.D, ly.Hkv * ly.D
    for step in range(3):
        fused = ref.values(10 + step, (B, (ly.Hq + 2 * ly.Hkv) * ly.D), ly.dtype).cuda()
        now = np.array(lens, np.int32) + step
        q, k, v = ly.rope(fused, torch.from_numpy(now).cuda())
        ly.append(k, v, torch.tensor([int(ly.slots(b, now[b])) for b in range(B)], dtype=torch.int32, device="cuda"))
        clens = torch.from_numpy(now + 1).cuda()
        out = wq.wq_kv_attention(q, *ly.caches, table, clens, page_size=ly.page)
        torch.cuda.synchronize()
        view.host = [(c.codes.cpu().numpy(), c.s.cpu().view(torch.int16).numpy().view(np.uint16), c.zpacked.cpu().numpy())
                     for c in ly.caches]
        view.val = [torch.from_numpy(oracle.kv_dequant(c, view.S, view.hd)).view(view.S, ly.Hkv, ly.D).double() for c in view.host]
        want, _ = _cache_want(view, q.cpu(), ly.table, ly.page, [int(x) + 1 for x in now], list(range(B + 1)), ly.D ** -0.5)
        _check_rows(out, None, want)


def test_decode_step_captured_and_replayed():
    """Norm and rotation, append and cache attention (split, with a workspace of
    its own) in one graph, replayed with new inputs and eager work in between."""
    lens = [3000, 2500]
    ly = Layer(lens, page=32)
    B = len(lens)
    ly.cos, ly.sin = (torch.randn(4096, 64, device="cuda") for _ in range(2))
    X = ref.values(3, (ly.caches[0].S, ly.Hkv * ly.D), torch.float32)
    for c in ly.caches:
        wq.wq_kv_quantize(X.cuda(), c)
    table = torch.from_numpy(ly.table).cuda()
    fused = torch.empty((B, (ly.Hq + 2 * ly.Hkv) * ly.D), dtype=ly.dtype, device="cuda")
    pos, slot = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(2))
    clens = torch.zeros(B, dtype=torch.int32, device="cuda")

    def step():
        q, k, v = ly.rope(fused, pos)
        ly.append(k, v, slot)
        return wq.wq_kv_attention(q, *ly.caches, table, clens, page_size=32, max_context=3008, lse=True)

    def fill(i):
        now = np.array(lens, np.int32) + i
        fused.copy_(ref.values(50 + i, tuple(fused.shape), ly.dtype))
        pos.copy_(torch.from_numpy(now))
        slot.copy_(torch.tensor([int(ly.slots(b, now[b])) for b in range(B)], dtype=torch.int32))
        clens.copy_(torch.from_numpy(now + 1 if i else np.zeros(B, np.int32)))

    fill(1)
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = step()
    for i in (1, 2, 0, 5, 3):
        fill(i)
        torch.cuda.synchronize()
        out.fill_(NAN)
        g.replay()
        torch.cuda.synchronize()
        got = out.clone(), lse.clone()
        want = step()
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), i


def test_calls_on_two_streams_at_once():
    """Split cache attention and prompt attention on two streams at the same
    time, each with its own workspace, give what they give alone."""
    cache = Cache(8, 8192, 2, 128)
    dev = cache.to_dev()
    table = np.arange(128, dtype=np.int32)[None]
    q = ref.values(1, (1, 8, 128), BF).cuda()
    tb, cl = torch.from_numpy(table).cuda(), torch.tensor([8192], dtype=torch.int32, device="cuda")
    p = [ref.values(2 + i, (600, h, 128), BF).cuda() for i, h in enumerate((4, 2, 2))]
    st = torch.tensor([0, 600], dtype=torch.int32, device="cuda")
    want = wq.wq_kv_attention(q, *dev, tb, cl, page_size=64), wq.wq_prompt_attention(*p, st)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for _ in range(10):
        for s in streams:
            outs.append((wq.wq_kv_attention(q, *dev, tb, cl, page_size=64, stream=s), wq.wq_prompt_attention(*p, st, stream=s)))
    torch.cuda.synchronize()
    for a, b in outs:
        assert torch.equal(a, want[0]) and torch.equal(b, want[1])
