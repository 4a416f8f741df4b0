"""The operators of a speculative decoding step on the HIP path: appending to the
INT4 cache against a definition that is fixed to the bit, attention of draft trees
against a plain 64-bit implementation, verification token by token in 64 bits, the
moving of accepted rows, and all of them run together."""
import math
import threading

import numpy as np
import pytest
import torch

import attn_ref as ref
import oracle
import spec_ref
import w4a16_bit_matmul_amd as wq
from parity import say
from test_gpu_attention import Cache, _check_rows, _tables

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
NAN = float("nan")
ODT = {BF: oracle.BF16, HF: oracle.F16}


def i32(x):
    return torch.as_tensor(np.asarray(x, np.int32)).cuda()


def bits(x):
    return x.cpu().contiguous().view(torch.int16).numpy().view(np.uint16)


def tables(rot, P):
    ang = np.arange(P)[:, None] * 10000.0 ** (-np.arange(rot // 2) * 2.0 / rot)
    return [torch.from_numpy(f(ang).astype(np.float32)) for f in (np.cos, np.sin)]


def host_of(c):
    return [c.codes.cpu().numpy(), c.s.cpu().view(torch.int16).numpy().view(np.uint16), c.zpacked.cpu().numpy()]


def same_cache(dev, host, what):
    for got, want, part in zip(host_of(dev), host, ("codes", "scales", "zero-points")):
        bad = np.argwhere(got != want)
        assert not len(bad), f"{what} {part}: {len(bad)} differ, first at {bad[0]}"


def filled_cache(seed, S, hd):
    rng = np.random.default_rng(seed)
    c = wq.kv_cache_alloc(S, hd)
    for t in (c.codes, c.zpacked):
        t.copy_(torch.from_numpy(rng.integers(0, 256, tuple(t.shape)).astype(np.uint8)))
    c.s.copy_(torch.from_numpy(rng.random(tuple(c.s.shape)).astype(np.float16)))
    return c


# ---- appending ---------------------------------------------------------------------

def check_append(lens, n, Hq, Hkv, D, rot, page, dtype, inter=False, norm=False, weights=True, k_out=False, first=0, extra=0,
                 positions=None, table=None, S=None, P=700, q=None, k=None, v=None, one=False, in_place=False, with_q=True):
    """Appends and compares every byte of the outputs and of both caches."""
    B = len(lens)
    starts = [int(x) for x in first + np.concatenate([[0], np.cumsum(n)])]
    T = starts[-1] + extra
    S = S or (sum(max(1, -(-x // page)) for x in lens) + 2) * page
    table = _tables(B + D, lens, page, S) if table is None else table
    say(f"append lens={lens[:6]} n={n[:6]} Hq={Hq} Hkv={Hkv} D={D} rot={rot} page={page} {dtype} inter={inter} norm={norm}")
    q = ref.values(1, (T, Hq, D), dtype, 2.0) if q is None else q
    k = ref.values(2, (T, Hkv, D), dtype) if k is None else k
    v = ref.values(3, (T, Hkv, D), dtype, 0.5) if v is None else v
    w = [ref.values(4 + i, (D,), dtype, 0.3, wide=0).add_(1) if weights and norm else None for i in range(2)]
    cos, sin = tables(rot, P)
    where = spec_ref.places(starts, T, lens)
    pos = [-1 if x is None else x[2] for x in where] if positions is None else positions
    pt = torch.tensor(pos, dtype=torch.int32)
    qw, kw = (spec_ref.turned(x, cos, sin, pt, inter, norm, wt, 1e-5) for x, wt in ((q, w[0]), (k, w[1])))
    kc, vc = filled_cache(1, S, Hkv * D), filled_cache(2, S, Hkv * D)
    hosts = [[a.copy() for a in host_of(c)] for c in (kc, vc)]
    live = [t for t in range(T) if where[t] is not None and 0 <= pos[t] < P]
    slot = np.full(T, -1, np.int32)
    for t in live:
        slot[t] = spec_ref.cache_row(table, page, S, where[t][0], where[t][2])
    for x, host in ((kw, hosts[0]), (v, hosts[1])):
        oracle.kv_quantize(bits(x).reshape(T, -1), host, slot=slot, dtype=ODT[dtype])
    # inputs as slices of one projection
    fused = torch.full((T, (Hq + 2 * Hkv) * D + 8), 7.0, dtype=dtype)
    a, b, c = Hq * D, (Hq + Hkv) * D, (Hq + 2 * Hkv) * D
    fused[:, :a], fused[:, a:b], fused[:, b:c] = q.view(T, -1), k.view(T, -1), v.view(T, -1)
    f = fused.cuda()
    qd, kd, vd = f[:, :a].view(T, Hq, D), f[:, a:b].view(T, Hkv, D), f[:, b:c].view(T, Hkv, D)
    qo = qd if in_place else torch.full((T, Hq, D), 7.0, dtype=dtype, device="cuda")
    ko = False if not k_out else kd if in_place else torch.full((T, Hkv, D), 7.0, dtype=dtype, device="cuda")
    got = wq.wq_kv_append(kd, vd, kc, vc, torch.from_numpy(table).cuda(), i32(lens), cos.cuda(), sin.cuda(), page_size=page,
                          q=qd if with_q else None, q_starts=None if one else i32(starts), positions=None if positions is None else pt.cuda(),
                          norm=norm, q_weight=None if w[0] is None else w[0].cuda(), k_weight=None if w[1] is None else w[1].cuda(),
                          eps=1e-5, interleaved=inter, q_out=qo if with_q else None, k_out=ko)
    torch.cuda.synchronize()
    assert (got[0] is None) == (not with_q) and (got[1] is None) == (not k_out)
    at = torch.zeros(T, dtype=torch.bool)
    at[live] = True
    for x, want, old, what in ((got[0], qw, q, "q"), (got[1], kw, k, "k")):
        if x is None:
            continue
        old = old if in_place else torch.full_like(old, 7.0)
        bad = np.argwhere(bits(x) != bits(torch.where(at[:, None, None], want, old)))
        assert not len(bad), f"{what}: {len(bad)} values differ, first at {bad[0]}"
    same_cache(kc, hosts[0], "K")
    same_cache(vc, hosts[1], "V")
    if in_place:
        assert bool((f[:, c:] == 7.0).all()) and np.array_equal(bits(f[:, b:c].reshape(T, Hkv, D)), bits(v))
    return qw, kw, q, k, w, cos, sin, pt, at


@pytest.mark.parametrize("lens,n,Hq,Hkv,D,rot,page", [
    ([1], [1], 1, 1, 128, 128, 1), ([5, 9, 600], [5, 2, 3], 8, 2, 128, 128, 16), ([70, 3], [70, 3], 14, 2, 64, 32, 4),
    ([33, 1, 64], [33, 1, 64], 3, 1, 256, 256, 32), ([130], [129], 6, 3, 128, 96, 64), ([20, 20], [1, 7], 4, 4, 64, 64, 2),
    ([9, 40], [9, 8], 10, 5, 256, 64, 8), ([300, 12, 7], [1, 1, 1], 64, 8, 128, 128, 256), ([50], [50], 24, 6, 64, 16, 128)])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("inter,norm", [(False, False), (True, True), (False, True), (True, False)])
def test_append(lens, n, Hq, Hkv, D, rot, page, dtype, inter, norm):
    """To the bit; and the rotated values against the formulas in 64 bits."""
    want, _, q, _, w, cos, sin, pos, _ = check_append(lens, n, Hq, Hkv, D, rot, page, dtype, inter, norm, k_out=n[0] % 2 == 1)
    if norm:
        exact, mag = ref.norm_rope(q, w[0], cos, sin, pos, 1e-5, inter)
        ref.check(want, exact, ref.norm_rope_bound(exact, mag, dtype), "the definition")


@pytest.mark.parametrize("B", [63, 64, 65, 300])
def test_append_many_sequences_some_empty(B):
    """Sequences found among many (the search takes 64 starts at a time), empty ones among them, tokens before the
    first and behind the last sequence, which nothing is written for."""
    rng = np.random.default_rng(B)
    n = [int(x) for x in rng.integers(0, 4, B)]
    lens = [x + int(y) for x, y in zip(n, rng.integers(0, 30, B))]
    check_append(lens, n, 4, 1, 128, 128, 16, BF, first=3, extra=5, k_out=True)
    check_append(lens, [1] * B, 4, 1, 128, 64, 16, HF, one=True)


def test_append_padding_missing_pages_and_positions():
    """Tokens whose position lies outside the tables are not written; those without a page (gone, behind the
    cache, past the table, before the sequence's start) are rotated and not cached."""
    lens, n, page = [40, 3, 500], [6, 5, 4], 8
    S = 30 * page + 3
    table = np.arange(15, dtype=np.int32).reshape(3, 5)
    table[0, 4] = -1  # tokens 32..39 of the first
    positions = [0, 699, 700, -1, 2 ** 31 - 1, 5, 6, 7, 8, 9, 10, 11, 12, 13, 14]
    check_append(lens, n, 8, 2, 128, 128, page, BF, table=table, S=S, positions=positions, k_out=True)
    table[0, 4], table[1, 0] = 20, S // page
    check_append(lens, n, 8, 2, 64, 64, page, HF, table=table, S=S, positions=positions, norm=True)
    check_append([2 ** 31 - 1, -5], [2, 1], 2, 1, 128, 128, page, HF, table=table[:2], S=S, positions=[1, 2, 3])


@pytest.mark.parametrize("norm", [False, True])
def test_append_in_place_without_queries_without_weights(norm):
    check_append([19, 7], [19, 7], 6, 3, 128, 128, 4, BF, norm=norm, in_place=True, k_out=True, weights=False)
    check_append([19, 7], [3, 7], 6, 3, 256, 128, 4, HF, norm=norm, in_place=True, k_out=True, inter=True)
    check_append([19, 7], [3, 7], 6, 3, 128, 64, 4, HF, norm=norm, with_q=False, k_out=True)
    check_append([19, 7], [3, 7], 2, 2, 64, 64, 4, BF, norm=norm, with_q=False)


def test_append_special_values():
    """Rows of zeros (scale 0), of the types' smallest and large values, blocks of one sign, values on the codes' halves."""
    T, Hkv, D = 8, 2, 128
    for dtype in (BF, HF):
        k, v = ref.values(5, (T, Hkv, D), dtype), ref.values(6, (T, Hkv, D), dtype)
        k[0], v[0] = 0.0, 0.0
        k[1], v[1] = 1e-38 if dtype == BF else 2.0 ** -24, 2.0 ** -24
        k[2], v[2] = 4e4, -6e4  # (turned by 45 degrees: 5.7e4, within fp16)
        v[3], k[4] = v[3].abs(), -k[4].abs()
        v[5] = (torch.arange(D) / 2.0 - 3).to(dtype)[None]
        v[6] = torch.tensor([0.0, 7.5, 0.5, 1.5] * (D // 4)).to(dtype)[None]
        for norm in (False, True):
            check_append([8], [8], 2, Hkv, D, 128, 4, dtype, norm=norm, k=k, v=v)


def test_append_far_rows_and_positions():
    """Rows of a cache past 2^32 bytes, tables past 2^31 bytes, a wide table."""
    Hkv, D, page, T = 8, 256, 64, 3
    S = (2 ** 32 + 2 ** 26) // (Hkv * D // 2) // page * page
    kc, vc = (wq.KVCache(torch.zeros((S, Hkv * D // 2), dtype=torch.uint8, device="cuda"),
                         torch.zeros((S, Hkv * D // 128), dtype=torch.float16, device="cuda"),
                         torch.zeros((S, Hkv * D // 256), dtype=torch.uint8, device="cuda"), S, Hkv * D) for _ in range(2))
    k, v = ref.values(1, (T, Hkv, D), BF), ref.values(2, (T, Hkv, D), BF)
    P = 5_000_000
    cos, sin = torch.zeros((P, 128), device="cuda"), torch.zeros((P, 128), device="cuda")
    rows = torch.randn(T, 128, generator=torch.Generator().manual_seed(1))
    pos = torch.tensor([P - 1, 3, P - 2], dtype=torch.int32)
    cos[pos.long().cuda()], sin[pos.long().cuda()] = rows.cos().cuda(), rows.sin().cuda()
    width = 2 ** 24 // page
    table = torch.full((2, width), -1, dtype=torch.int32, device="cuda")
    table[1, width - 1] = S // page - 1
    lens = i32([0, width * page])
    wq.wq_kv_append(k.cuda(), v.cuda(), kc, vc, table, lens, cos, sin, page_size=page, q_starts=i32([0, 0, T]), positions=pos.cuda())
    torch.cuda.synchronize()
    want = spec_ref.turned(k, rows.cos(), rows.sin(), torch.arange(T), False, False, None, 0.0)
    for c, x in ((kc, want), (vc, v)):
        host = oracle.kv_alloc(T, Hkv * D)
        oracle.kv_quantize(bits(x).reshape(T, -1), host, dtype=oracle.BF16)
        for got, w in zip((c.codes[-T:], c.s[-T:].view(torch.int16), c.zpacked[-T:]), host):
            assert np.array_equal(got.cpu().numpy().view(w.dtype), w)
        assert not bool(c.codes[:-T].any())


# ---- attention of draft trees -----------------------------------------------------

def tree_want(cache, q, table, page, lens, starts, masks, scale, max_context=None, most=None):
    """masks[b][i]: nodes that node i of sequence b sees."""
    T, Hq, D = q.shape
    G, pages = Hq // cache.Hkv, cache.S // page
    out, bound = torch.full((T, Hq, D), NAN, dtype=torch.float64), torch.zeros((T, Hq, D), dtype=torch.float64)
    lse, lb = torch.full((T, Hq), NAN, dtype=torch.float64), torch.zeros((T, Hq), dtype=torch.float64)
    none, used = torch.ones((T, Hq), dtype=torch.bool), []
    for b, n in enumerate(lens):
        n = max(0, n if max_context is None else min(n, max_context))
        q0, q1 = starts[b], starts[b + 1]
        m = q1 - q0
        t = np.arange(n)
        ok = (lambda pg: (pg >= 0) & (pg < pages))(table[b][t // page])
        rows = np.where(ok, table[b][t // page].astype(np.int64) * page + t % page, 0)
        used.append(rows[ok])
        q1 = q1 if most is None else min(q1, q0 + most)
        none[q0:q1] = False
        seen = np.zeros((q1 - q0, n), bool)
        for i in range(q1 - q0):
            seen[i, :max(0, n - m)] = True
            for j in masks[b][i]:
                if j < m and n - m + j >= 0:
                    seen[i, n - m + j] = True
        seen = torch.from_numpy(seen & ok[None, :])
        for h in range(Hq):
            kv = [x[rows, h // G] for x in cache.val]
            out[q0:q1, h], bound[q0:q1, h], lse[q0:q1, h], lb[q0:q1, h] = ref.attend(
                q[q0:q1, h].double(), kv[0], kv[1], seen, scale, 15 * cache.v_scale(rows[ok]), q.dtype, 2.0 ** -11)
    return (out, bound, lse, lb, none), np.unique(np.concatenate(used)) if used else np.zeros(0, np.int64)


def run_tree(dev, q, table, page, lens, starts, mask, **kw):
    T, Hq, D = q.shape
    out, lse = torch.full((T, Hq, D), 7.0, dtype=q.dtype, device="cuda"), torch.full((T, Hq), 7.0, device="cuda")
    wq.wq_kv_tree_attention(q, *dev, torch.from_numpy(table).cuda(), i32(lens), mask.cuda(), page_size=page,
                            q_starts=None if starts is None else i32(starts), out=out, lse=lse, **kw)
    torch.cuda.synchronize()
    return out, lse


def some_masks(seed, nq, T, first, words, kind="tree"):
    """Sets of seen nodes of every node, and the words of all T tokens of the call (of no sequence: all ones)."""
    rng = np.random.default_rng(seed)
    masks = []
    for n in nq:
        if kind == "tree":
            masks.append(spec_ref.random_tree(rng, n)[1] if n else [])
        else:  # anything: later nodes, not itself, nothing at all
            masks.append([set() if rng.random() < 0.2 else {int(j) for j in np.nonzero(rng.random(n) < 0.4)[0]} for _ in range(n)])
    mask = torch.full((T, words), -1, dtype=torch.int64)
    at = first
    for n, m in zip(nq, masks):
        if n:
            mask[at:at + n] = spec_ref.mask_words([{j for j in s if j < 64 * words} for s in m], words)
        at += n
    return [[{j for j in s if j < 64 * words} for s in m] for m in masks], mask


@pytest.mark.parametrize("lens,nq,Hq,Hkv,D,page,words", [
    ([1], [1], 1, 1, 128, 1, 1), ([40, 3, 0, 100, 12], [2, 3, 0, 4, 12], 8, 1, 128, 16, 1), ([64, 90], [33, 64], 4, 1, 128, 32, 1),
    ([333], [65], 6, 2, 64, 64, 2), ([150, 1], [17, 1], 3, 1, 256, 8, 1), ([600], [200], 8, 1, 128, 64, 4),
    ([96, 20], [5, 25], 64, 8, 128, 4, 1), ([70, 131, 260], [64, 127, 130], 14, 2, 64, 2, 3), ([127, 128, 129, 130], [2, 2, 2, 2], 5, 1, 256, 32, 1)])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("kind", ["tree", "any"])
def test_tree_attention(lens, nq, Hq, Hkv, D, page, words, dtype, kind):
    """Trees and masks of any kind (rows that see nothing among them), more nodes than tokens, rows of no
    sequence before the first and behind the last."""
    say(f"tree lens={lens} nq={nq} Hq={Hq} Hkv={Hkv} D={D} page={page} {dtype} {kind}")
    starts = [int(x) for x in 2 + np.concatenate([[0], np.cumsum(nq)])]
    S = sum(-(-n // page) for n in lens) * page + 2 * page
    cache = Cache(sum(lens) + D, S, Hkv, D)
    table = _tables(len(lens), lens, page, S)
    q = ref.values(Hq, (starts[-1] + 3, Hq, D), dtype)
    masks, mask = some_masks(D + page, nq, q.shape[0], 2, words, kind)
    want, used = tree_want(cache, q, table, page, lens, starts, masks, D ** -0.5, most=64 * words)
    got, lse = run_tree(cache.to_dev(used), q.cuda(), table, page, lens, starts, mask)
    _check_rows(got, lse, want)


@pytest.mark.parametrize("Hq,Hkv,D,nq,plan", [
    (64, 8, 64, 1, "HP=4, RT=1, PK=2"), (8, 8, 64, 4, "HP=4, RT=1, PK=4"), (14, 2, 64, 1, "HP=2, RT=1, PK=2"), (40, 8, 64, 2, "HP=2, RT=1, PK=1"),
    (48, 8, 64, 3, "HP=2, RT=2, PK=1"), (64, 8, 128, 1, "HP=2, RT=1, PK=2"), (18, 2, 128, 1, "HP=2, RT=1, PK=1"),
    (15, 5, 128, 5, "HP=1, RT=1, PK=1"), (24, 8, 128, 7, "HP=1, RT=2, PK=1"), (40, 4, 256, 3, "HP=1, RT=1, PK=1"),
    (64, 8, 128, 5, "kv_tree_kernel<D=128, RG=2"), (24, 2, 128, 9, "kv_tree_kernel<D=128, RG=4"), (32, 8, 64, 9, "kv_tree_kernel<D=64, RG=2"),
    (16, 2, 64, 30, "kv_tree_kernel<D=64, RG=4"), (7, 1, 128, 43, "kv_tree_kernel<D=128, RG=4")])
@pytest.mark.parametrize("page", [16, 64])
def test_tree_attention_kernels_of_long_contexts(Hq, Hkv, D, nq, plan, page):
    """Every variant, its steps shared out: short and long contexts under room for a million tokens, a page gone."""
    lens, width = [700, 0, 3, 1300, 129], 2 ** 20 // page
    nodes = [nq, 0, nq, nq, nq]
    starts = [0, nq, nq, 2 * nq, 3 * nq, 4 * nq] if nq > 1 else list(range(6))
    nodes = nodes if nq > 1 else [1] * 5
    S = 2304
    cache = Cache(D + nq, S, Hkv, D)
    table = _tables(D, lens, page, S, width=width)
    table[3, 700 // page] = -1
    q = ref.values(Hq, (starts[-1], Hq, D), HF)
    assert plan in wq.wq_kv_tree_attention_plan(q.shape[0], Hq, Hkv, D, 5, page, 2 ** 20, nq)
    masks, mask = some_masks(nq, nodes, q.shape[0], 0, 1, "any" if page == 16 else "tree")
    want, used = tree_want(cache, q, table, page, lens, starts, masks, D ** -0.5)
    got, lse = run_tree(cache.to_dev(used), q.cuda(), table, page, lens, None if nq == 1 else starts, mask, max_queries=nq)
    _check_rows(got, lse, want)


@pytest.mark.parametrize("B,most,Hq,Hkv,D,page", [(66, 125, 8, 8, 128, 16), (37, 12, 160, 16, 128, 64), (64, 250, 4, 4, 64, 1), (86, 33, 18, 6, 64, 32),
                                                  (300, 50, 1, 1, 128, 8), (40, 64, 8, 8, 64, 16)])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_tree_attention_many_rows(B, most, Hq, Hkv, D, page, dtype):
    """The kernel for many rows: sequences of none to `most` nodes, more nodes than tokens, pages that are gone,
    lengths past max_context."""
    rng = np.random.default_rng(B + D)
    nq = [0, 1, most, most] + [int(x) for x in rng.integers(0, most + 1, B - 4)]
    lens = [5, 1, most // 2, 300] + [int(x) for x in rng.integers(0, 170, B - 4)]
    starts = [int(x) for x in 1 + np.concatenate([[0], np.cumsum(nq)])]
    S = (sum(-(-n // page) for n in lens) + 3) * page
    cache = Cache(B + D, S, Hkv, D)
    table = _tables(B, lens, page, S)
    for b in range(5, B, 3):
        gone = [lens[b] // 2 // page] if b % 2 else list(range(table.shape[1]))
        table[b, gone] = [-1, S // page, 2 ** 31 - 1, -2 ** 31][b % 4]
    q = ref.values(Hq, (starts[-1] + 2, Hq, D), dtype)
    cut = min(250, table.shape[1] * page)
    assert "kv_tree_kernel" in wq.wq_kv_tree_attention_plan(q.shape[0], Hq, Hkv, D, B, page, cut, most)
    masks, mask = some_masks(B, nq, q.shape[0], 1, -(-most // 64), "any" if dtype == BF else "tree")
    want, used = tree_want(cache, q, table, page, lens, starts, masks, D ** -0.5, max_context=cut)
    got, lse = run_tree(cache.to_dev(used), q.cuda(), table, page, lens, starts, mask, max_context=cut, max_queries=most)
    _check_rows(got, lse, want)


@pytest.mark.parametrize("Hq,Hkv,D,nodes,room,plan", [
    (8, 8, 64, 4, 2 ** 20, "HP=4, RT=1, PK=4"), (8, 8, 64, 4, 1200, "HP=2, RT=1, PK=2"), (64, 8, 128, 2, 2 ** 20, "HP=2, RT=1, PK=1"),
    (64, 8, 128, 2, 1200, "HP=1, RT=1, PK=1"), (24, 8, 128, 7, 1200, "HP=1, RT=1"), (24, 8, 128, 7, 2 ** 20, "RT=2"), (48, 8, 64, 4, 1200, "HP=2, RT=1, PK=1"), (4, 1, 256, 30, 1200, "kv_attn_kernel<D=256"),
    (64, 8, 128, 8, 2 ** 20, "D=128, RG=2"), (64, 8, 128, 16, 2 ** 20, "D=128, RG=4"), (16, 8, 64, 20, 1200, "D=64, RG=2"),
    (28, 2, 64, 25, 1200, "D=64, RG=4")])
@pytest.mark.parametrize("bad", [NAN, math.inf, -math.inf])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_tree_attention_scales_of_other_branches(Hq, Hkv, D, nodes, room, plan, bad, dtype):
    """A node whose cache scales are infinite or NaN reaches the rows that see it and no other: two branches from the
    root by turns, the first of them bad in K, V or both, and a node that no row sees."""
    B, page = 6, 16
    lens = [nodes + x for x in (0, 3, 50, 200, 331, 1000)]
    starts = [nodes * b for b in range(B + 1)]
    S = (sum(-(-n // page) for n in lens) + 2) * page
    cache = Cache(D + nodes, S, Hkv, D)
    table = _tables(B, lens, page, S, width=room // page)
    q = ref.values(Hq, (starts[-1], Hq, D), dtype)
    # node i sees the root and the nodes of its parity, but for the last one, which only itself would
    tree = [{j for j in range(i + 1) if (j == 0 or j % 2 == i % 2) and j != nodes - 1} for i in range(nodes)]
    masks, mask = [tree] * B, torch.cat([spec_ref.mask_words(tree, 1)] * B)
    assert plan in wq.wq_kv_tree_attention_plan(q.shape[0], Hq, Hkv, D, B, page, room, nodes)
    want, used = tree_want(cache, q, table, page, lens, starts, masks, D ** -0.5)
    for which in ((0,), (1,), (0, 1)):
        dev = cache.to_dev(used)
        hit = torch.tensor([any(j % 2 for j in s) for s in tree] * B)
        for b in range(B):
            for j in [j for j in range(nodes) if j % 2 or j == nodes - 1]:
                at = lens[b] - nodes + j
                for c in which:
                    dev[c].s[table[b][at // page] * page + at % page] = bad
        got, lse = run_tree(dev, q.cuda(), table, page, lens, starts, mask)
        if 1 in which or math.isnan(bad):  # (a score of -inf has no weight)
            assert not bool(torch.isfinite(got.cpu()[hit]).all(-1).any())
        got[hit.cuda()], lse[hit.cuda()] = 7.0, 7.0
        none = want[4] | hit[:, None]
        _check_rows(got, lse, tuple(x.masked_fill(hit.view(-1, *[1] * (x.dim() - 1)), NAN) for x in want[:4]) + (none,))


@pytest.mark.parametrize("Hq,Hkv,D,page,n", [(8, 2, 128, 16, 5), (16, 8, 64, 32, 7), (4, 1, 256, 64, 30), (8, 8, 128, 16, 32)])
def test_a_chain_is_the_causal_attention_to_the_bit(Hq, Hkv, D, page, n):
    """Masks of a chain give what wq_kv_attention gives where the two take the same walk (up to 32 rows of a KV head,
    heads of 256)."""
    B = 3
    lens = [n + 7 * b % 90 + b for b in range(B)]
    S = (sum(-(-x // page) for x in lens) + 1) * page
    cache = Cache(n, S, Hkv, D)
    table = _tables(1, lens, page, S)
    starts = [n * b for b in range(B + 1)]
    q = ref.values(2, (n * B, Hq, D), BF)
    words = -(-n // 64)
    mask = spec_ref.mask_words([set(range(i + 1)) for i in range(n)], words).repeat(B, 1)
    dev = cache.to_dev()
    a, la = run_tree(dev, q.cuda(), table, page, lens, starts, mask, max_queries=n)
    b, lb = wq.wq_kv_attention(q.cuda(), *dev, torch.from_numpy(table).cuda(), i32(lens), page_size=page, q_starts=i32(starts),
                               max_queries=n, lse=True)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(la, lb)


def test_tree_attention_long_contexts_are_split_and_joined():
    for B, n, Hq, Hkv, D, page, nq in [(1, 9000, 8, 1, 128, 64, 6), (1, 9000, 8, 1, 128, 64, 9), (2, 7000, 20, 4, 64, 16, 40), (3, 4500, 16, 4, 64, 16, 12), (40, 2100, 8, 8, 128, 32, 40), (3, 4500, 4, 4, 64, 16, 1), (2, 5000, 4, 1, 256, 32, 3), (1, 7000, 16, 8, 128, 32, 12)]:
        lens = [n - min(1111, n // B) * b for b in range(B)]
        say(wq.wq_kv_tree_attention_plan(B * nq, Hq, Hkv, D, B, page, n, nq))
        S = sum(-(-x // page) for x in lens) * page
        cache = Cache(n, S, Hkv, D)
        table = _tables(B, lens, page, S)
        q = ref.values(n, (B * nq, Hq, D), HF)
        starts = [nq * b for b in range(B + 1)]
        masks, mask = some_masks(n, [nq] * B, B * nq, 0, 1)
        want, _ = tree_want(cache, q, table, page, lens, starts, masks, D ** -0.5)
        need = wq.wq_kv_tree_attention_workspace_bytes(B * nq, Hq, Hkv, D, B, page, n, nq)
        assert need > 0
        ws = torch.full((max(need, 1),), 0xFF, dtype=torch.uint8, device="cuda")  # NaNs: no content is needed
        got, lse = run_tree(cache.to_dev(), q.cuda(), table, page, lens, starts, mask, max_context=n, workspace=ws, max_queries=nq)
        _check_rows(got, lse, want)
        again, lse2 = run_tree(cache.to_dev(), q.cuda(), table, page, lens, starts, mask, max_context=n, workspace=ws, max_queries=nq)
        assert torch.equal(got, again) and torch.equal(lse, lse2)


# ---- verification --------------------------------------------------------------------

def check_verify(logits, tokens, uniform, starts, width, parents=None, draft=None, temperature=None, stride=None, one=False):
    """Compares every integer; logits float64 of values that `dtype` of the tensors holds."""
    T, V = logits.shape

    def dev(x):
        if stride is None:
            return x.cuda()
        wide = torch.full((T, stride), NAN, dtype=x.dtype)
        wide[:, 3:3 + V] = x
        return wide.cuda()[:, 3:3 + V]

    B = len(starts) - 1
    outs = [torch.full(s, 77, dtype=torch.int32, device="cuda") for s in ((B, width), (B, width), (B,))]
    got = wq.wq_verify_drafts(dev(logits), i32(tokens), torch.as_tensor(uniform, dtype=torch.float32).cuda(),
                              q_starts=None if one else i32(starts), max_queries=width, parents=None if parents is None else i32(parents),
                              draft_logits=None if draft is None else dev(draft),
                              temperature=None if temperature is None else torch.as_tensor(temperature, dtype=torch.float32).cuda(),
                              out_tokens=outs[0], path=outs[1], counts=outs[2],
                              workspace=torch.full((wq.wq_verify_drafts_workspace_bytes(T, V, B, draft is not None) + 256,), 0xFF,
                                                   dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    want = spec_ref.verify(logits.double().numpy(), tokens, uniform, starts, width, parents, None if draft is None else draft.double().numpy(),
                           temperature)
    for g, w, what in zip(got, want, ("out_tokens", "path", "counts")):
        g, w = g.cpu().numpy(), np.array(w, np.int32).reshape(g.shape)
        bad = np.argwhere(g != w)
        assert not len(bad), f"{what}: {len(bad)} differ, first at {bad[0]}: got {g[tuple(bad[0])]}, want {w[tuple(bad[0])]}"
    return want


def some_logits(rng, T, V, dtype, sharp=2.0):
    x = rng.standard_normal((T, V)) * sharp
    for r in range(T):
        x[r, rng.integers(0, V, min(V, 4))] += 5.0 + math.log(V) / 2
    return torch.from_numpy(x.astype(np.float32)).to(dtype)


def tree_inputs(seed, nq, V, dtype, first=0, extra=0, hit=0.7):
    """Trees whose nodes' tokens are often what their parent's row gives."""
    rng = np.random.default_rng(seed)
    starts = [int(x) for x in first + np.concatenate([[0], np.cumsum(nq)])]
    T = starts[-1] + extra
    x = some_logits(rng, T, V, dtype)
    u = rng.random(T).astype(np.float32)
    temp = rng.choice([0.0, 0.3, 1.0, 1.7], len(nq)).astype(np.float32)
    parents, tokens = np.full(T, -1, np.int32), rng.integers(0, V, T).astype(np.int32)
    xs = x.double().numpy()
    for b, n in enumerate(nq):
        if not n:
            continue
        p, _ = spec_ref.random_tree(rng, n)
        parents[starts[b]:starts[b + 1]] = p
        for i in range(1, n):
            if rng.random() < hit:
                row = starts[b] + p[i]
                top, w = spec_ref.probabilities(xs[row], temp[b])
                tokens[starts[b] + i] = top if w is None else spec_ref.take(w, u[row])
    return x, tokens, u, starts, parents, temp


@pytest.mark.parametrize("V", [1, 2, 7, 64, 999, 4096, 8191, 8192, 8193, 50001])
@pytest.mark.parametrize("dtype", [HF, BF, F32])
def test_verify_trees(V, dtype):
    nq = [5, 0, 1, 12, 3, 9] if V < 9000 else [4, 7]
    x, tokens, u, starts, parents, temp = tree_inputs(V, nq, V, dtype, first=2, extra=1)
    say(f"verify trees V={V} {dtype}")
    want = check_verify(x, tokens, u, starts, 12, parents, temperature=temp)
    assert V == 1 or max(want[2]) > 1
    check_verify(x, tokens, u, starts, 4, parents, temperature=temp, stride=V + 5)  # rows at any alignment, nodes cut off
    check_verify(x, tokens, u, starts, 12, temperature=None)  # chains of given tokens
    check_verify(x, tokens, u, list(range(x.shape[0] + 1)), 3, one=True)  # plain sampling


@pytest.mark.parametrize("V", [1, 2, 9, 500, 8192, 8200, 30011])
@pytest.mark.parametrize("dtype", [HF, BF, F32])
def test_verify_chains_of_a_draft_model(V, dtype):
    rng = np.random.default_rng(V)
    nq = [5, 0, 1, 12, 3, 9, 2, 2] if V < 9000 else [4, 7, 3]
    starts = [int(x) for x in 1 + np.concatenate([[0], np.cumsum(nq)])]
    T = starts[-1] + 2
    x = some_logits(rng, T, V, dtype)
    draft = (x.double() * 0.9 + torch.from_numpy(rng.standard_normal((T, V)) * 0.6)).to(dtype)
    temp = rng.choice([0.0, 0.4, 1.0, 1.5], len(nq)).astype(np.float32)
    u = rng.random(T).astype(np.float32)
    tokens = rng.integers(0, V, T).astype(np.int32)
    d = draft.double().numpy()
    for b, n in enumerate(nq):
        for i in range(1, n):  # drawn from the draft
            top, w = spec_ref.probabilities(d[starts[b] + i - 1], temp[b])
            tokens[starts[b] + i] = top if w is None else spec_ref.take(w, np.float32(rng.random()))
    say(f"verify chains V={V} {dtype}")
    want = check_verify(x, tokens, u, starts, 12, draft=draft, temperature=temp)
    if V < 9000:  # (few sequences above)
        assert max(want[2]) > 1 and (V < 9 or min(c - n for c, n in zip(want[2], nq)) < 0)
    check_verify(x, tokens, u, starts, 4, draft=draft, temperature=temp, stride=V + 4)
    check_verify(x, tokens, u, starts, 12, draft=draft)
    check_verify(x, tokens, u, starts, 12, draft=x, temperature=temp)  # the same distributions: all are accepted
    lone = tokens.copy()
    lone[starts[0] + 1:starts[0] + 5] = [-1, V, 2 ** 31 - 1, -2 ** 31]  # tokens that are none
    check_verify(x, lone, u, starts, 12, draft=draft, temperature=temp)


def test_verify_borders_and_ties():
    """Weights that are whole numbers: u on a border takes the next token; equal logits give the lowest greedy token;
    u of 0 and of the last number below 1; masked tokens are never taken."""
    V = 8
    x = torch.zeros((V + 3, V))
    u = [k / V for k in range(V)] + [0.0, float(np.float32(1) - np.float32(2.0 ** -24)), 0.5]
    starts = list(range(V + 4))
    assert [o[0] for o in check_verify(x, [0] * len(u), u, starts, 1)[0]][:V] == list(range(V))
    assert all(o[0] == 0 for o in check_verify(x, [0] * len(u), u, starts, 1, temperature=[0.0] * len(u))[0])
    y = torch.full((3, 20000), -math.inf)
    y[0, [7, 9000]], y[1, 19999], y[2, [5, 6]] = 1.0, -3.0, torch.tensor([2.0, 3.0])
    for uu in (0.0, 0.49, 0.5, 0.99999994):
        for t in (0.0, 1e-30, 0.5, 1e30, math.inf):
            want = check_verify(y, [0] * 3, [uu] * 3, [0, 1, 2, 3], 1, temperature=[t] * 3)
            assert want[0][1] == [19999] and want[0][0][0] in (7, 9000)
    check_verify(y.half(), [0] * 3, [0.7] * 3, [0, 1, 2, 3], 1)


@pytest.mark.parametrize("dtype", [HF, F32])
def test_verify_rows_that_are_no_distribution(dtype):
    """All masked, NaN or +inf anywhere: token -1, and the way ends; temperatures that are no numbers are greedy."""
    V, T = 9000, 12
    x, tokens, u, starts, parents, temp = tree_inputs(3, [T], V, dtype, hit=1.0)
    for bad in (math.nan, math.inf):
        for row, col in ((0, 0), (0, V - 1), (3, 8192)):
            for t in (0.0, 0.8):
                y = x.clone()
                y[row, col] = bad
                check_verify(y, tokens, u, starts, T, parents, temperature=[t])
                check_verify(y, tokens, u, starts, T, draft=x, temperature=[t])
                check_verify(x, tokens, u, starts, T, draft=y, temperature=[t])
    y = x.clone()
    y[0] = -math.inf
    assert check_verify(y, tokens, u, starts, T, parents)[0][0] == [-1] * T
    check_verify(y, tokens, u, starts, T, draft=x)
    check_verify(x, tokens, u, starts, T, draft=y)
    assert check_verify(x, tokens, u, starts, T, parents, temperature=[math.nan]) == check_verify(x, tokens, u, starts, T, parents, temperature=[-1.0])


def test_verify_odd_trees():
    """Siblings with one token (the first counts), parents that come later, are the node itself or no node, tokens of
    rows that give -1."""
    V = 50
    x, tokens, u, starts, _, _ = tree_inputs(9, [9], V, HF)
    first = spec_ref.take(spec_ref.probabilities(x[0].double().numpy(), 1.0)[1], u[0])
    tokens[1:4] = first
    check_verify(x, tokens, u, starts, 9, [-1, 0, 0, 0, 1, 2, 3, 4, 5])
    check_verify(x, tokens, u, starts, 9, [5, 1, 8, 0, 3, 3, 2 ** 31 - 1, -2 ** 31, 3])
    x[0], tokens[1] = -math.inf, -1
    check_verify(x, tokens, u, starts, 9, [-1, 0, 0, 0, 1, 2, 3, 4, 5])


def test_verify_many_nodes_and_long_ways():
    """1024 nodes, every one of the last few accepted; and ways as long as the tree."""
    V, n = 33, 1024
    rng = np.random.default_rng(1)
    x = torch.from_numpy(rng.standard_normal((n, V)).astype(np.float32))
    x[torch.arange(n), torch.from_numpy(rng.integers(0, V, n))] += 30
    tokens = np.concatenate([[0], x.argmax(-1).numpy()[:-1]]).astype(np.int32)
    u = rng.random(n).astype(np.float32)
    assert check_verify(x, tokens, u, [0, n], n)[2] == [n]
    assert check_verify(x, tokens, u, [0, n], n, draft=x)[2] == [n]
    x, tokens, u, starts, parents, temp = tree_inputs(5, [n], V, HF, hit=0.9)
    check_verify(x, tokens, u, starts, n, parents, temperature=temp)


def test_verify_without_rows():
    x = torch.zeros((0, 10), device="cuda")
    z = torch.zeros(0, dtype=torch.int32, device="cuda")
    for kw in ({}, dict(draft_logits=x)):
        out, path, counts = wq.wq_verify_drafts(x, z, z.float(), q_starts=i32([0, 0, 0]), max_queries=3, **kw)
        torch.cuda.synchronize()
        assert bool((out == -1).all()) and bool((path == -1).all()) and counts.tolist() == [0, 0]


def test_verify_keeps_the_targets_law():
    """Chains of one draft drawn from q: the first new token has the target's probabilities, whatever q is (20000
    sequences: within five standard deviations)."""
    V, B = 6, 20000
    rng = np.random.default_rng(4)
    p, q = np.array([0.05, 0.4, 0.25, 0.1, 0.15, 0.05]), np.array([0.3, 0.1, 0.1, 0.4, 0.05, 0.05])
    x = torch.from_numpy(np.log(np.repeat(p[None], 2 * B, 0))).float().cuda()
    d = torch.from_numpy(np.log(np.repeat(q[None], 2 * B, 0))).float().cuda()
    tokens = np.zeros(2 * B, np.int32)
    tokens[1::2] = rng.choice(V, B, p=q)
    out, _, counts = wq.wq_verify_drafts(x, i32(tokens), torch.from_numpy(rng.random(2 * B).astype(np.float32)).cuda(),
                                         q_starts=i32(np.arange(0, 2 * B + 1, 2)), max_queries=2, draft_logits=d)
    torch.cuda.synchronize()
    for got, n in ((out[:, 0].cpu().numpy(), B), (out[:, 1].cpu().numpy()[counts.cpu().numpy() == 2], None)):
        n = len(got)
        freq = np.bincount(got, minlength=V) / n
        assert n > 1000 and (np.abs(freq - p) <= 5 * np.sqrt(p * (1 - p) / n)).all(), freq


# ---- keeping rows ---------------------------------------------------------------------

def check_keep(lens, nq, paths, counts, hd, page, S, table, first=0):
    B, width = len(lens), len(paths[0])
    starts = [int(x) for x in first + np.concatenate([[0], np.cumsum(nq)])]
    caches = [filled_cache(i, S, hd) for i in range(2)]
    want = [[a.copy() for a in host_of(c)] for c in caches]
    for host in want:
        old = [a.copy() for a in host]
        for b in range(B):
            for j in range(min(counts[b], width, nq[b])):
                node = paths[b][j]
                if not j <= node < nq[b]:
                    continue
                to, at = (spec_ref.cache_row(table, page, S, b, lens[b] - nq[b] + i) for i in (j, node))
                if to >= 0 and at >= 0:
                    for a, o in zip(host, old):
                        a[to] = o[at]
    wq.wq_kv_keep(*caches, torch.from_numpy(table).cuda(), i32(lens), i32(paths), i32(counts), page_size=page, q_starts=i32(starts))
    torch.cuda.synchronize()
    for c, host, what in zip(caches, want, "KV"):
        same_cache(c, host, what)


@pytest.mark.parametrize("hd,page,B,most", [(128, 1, 1, 1), (128, 4, 7, 9), (1024, 16, 64, 8), (384, 2, 5, 64), (1152, 64, 9, 150), (4096, 8, 3, 30), (65536, 4, 2, 12)])
def test_keep(hd, page, B, most):
    rng = np.random.default_rng(hd + B)
    nq = [most] + [int(x) for x in rng.integers(0, most + 1, B - 1)]
    lens = [n + int(x) for n, x in zip(nq, rng.integers(0, 50, B))]
    S = (sum(-(-x // page) for x in lens) + 2) * page
    table = _tables(1, lens, page, S)
    paths, counts = np.full((B, most), -1, np.int64), []
    for b, n in enumerate(nq):
        way = sorted({0} | {int(x) for x in rng.integers(0, max(n, 1), n // 2)})[:n]
        paths[b, :len(way)] = way
        counts.append(len(way))
    check_keep(lens, nq, paths.tolist(), counts, hd, page, S, table, first=2)


def test_keep_odd_paths():
    """Nodes out of order, twice, before their place, of no node; counts past the path or the sequence, below zero;
    rows without a page or before the context's first token."""
    page, S = 4, 80
    lens, nq = [20, 20, 3, 20, 20], [10, 10, 8, 10, 10]
    table = _tables(2, [20] * 5, page, S + 40 * 4)
    S = S + 40 * 4
    paths = [[0, 3, 2, 9, 9, 5], [5, 5, 5, 0, 1, 10], [0, 5, 6, 7, 7, 7], [9, 9, 9, 9, 9, 2 ** 31 - 1], [1, 2, 3, 4, 5, 6]]
    counts = [6, 6, 100, 6, -3]
    check_keep(lens, nq, paths, counts, 256, page, S, table)
    table[0, 3], table[1, 2], table[3, 4] = -1, S // page, 2 ** 31 - 1
    check_keep(lens, nq, paths, counts, 256, page, S, table)
    check_keep(lens, nq, paths, [6, 3, 6, 2, 6], 128, page, S, table[:, :4].copy())


# ---- together ---------------------------------------------------------------------------

class Loop:
    """Steps of speculative decoding of one layer: append, tree attention, verification, keeping."""

    def __init__(self, lens, n, Hq=8, Hkv=2, D=128, page=16, V=300, dtype=BF, room=60):
        self.n, self.page, self.V, self.dims, self.dtype = n, page, V, (Hq, Hkv, D), dtype
        self.B = B = len(lens)
        need = [-(-(x + room) // page) for x in lens]
        self.S = (sum(need) + 1) * page
        self.table = _tables(B, [x * page for x in need], page, self.S)
        self.caches = [filled_cache(i, self.S, Hkv * D) for i in range(2)]
        rng = np.random.default_rng(B)
        self.parents, self.sees = zip(*[spec_ref.random_tree(rng, n, 3) for _ in range(B)])
        self.depth = i32([spec_ref.depth_of(p) for p in self.parents])
        self.mask = torch.cat([spec_ref.mask_words(s, 1) for s in self.sees]).cuda()
        self.par = i32(np.concatenate(self.parents))
        self.starts = i32(np.arange(B + 1) * n)
        self.tb, self.cos, self.sin = torch.from_numpy(self.table).cuda(), *(t.cuda() for t in tables(D, 4096))
        self.old = i32(lens)  # cached tokens before the step
        self.x = torch.empty((B * n, (Hq + 2 * Hkv) * D), dtype=dtype, device="cuda")
        self.logits = torch.empty((B * n, V), dtype=torch.float16, device="cuda")
        self.tokens, self.u = torch.zeros(B * n, dtype=torch.int32, device="cuda"), torch.zeros(B * n, device="cuda")

    def fill(self, seed):
        self.x.copy_(ref.values(seed, tuple(self.x.shape), self.dtype))
        rng = np.random.default_rng(seed)
        self.logits.copy_(some_logits(rng, self.B * self.n, self.V, HF, sharp=1.0))
        top = self.logits.float().topk(2, -1).indices.cpu().numpy()
        par = np.concatenate([[max(p, 0) + b * self.n for p in ps] for b, ps in enumerate(self.parents)])
        self.tokens.copy_(torch.from_numpy(top[par, rng.integers(0, 2, len(par))].astype(np.int32)))
        self.u.copy_(torch.from_numpy(rng.random(self.B * self.n).astype(np.float32)))

    def step(self):
        Hq, Hkv, D = self.dims
        T = self.x.shape[0]
        a, b = Hq * D, (Hq + Hkv) * D
        q, k, v = self.x[:, :a].view(T, Hq, D), self.x[:, a:b].view(T, Hkv, D), self.x[:, b:].view(T, Hkv, D)
        lens = self.old + self.n
        pos = (self.old[:, None] + self.depth).view(-1)
        q, _ = wq.wq_kv_append(k, v, *self.caches, self.tb, lens, self.cos, self.sin, q=q, page_size=self.page, q_starts=self.starts, positions=pos)
        out = wq.wq_kv_tree_attention(q, *self.caches, self.tb, lens, self.mask, page_size=self.page, q_starts=self.starts, max_queries=self.n)
        tokens, path, counts = wq.wq_verify_drafts(self.logits, self.tokens, self.u, q_starts=self.starts, max_queries=self.n, parents=self.par)
        wq.wq_kv_keep(*self.caches, self.tb, lens, path, counts, page_size=self.page, q_starts=self.starts)
        self.old.add_(counts)
        return q, out, tokens, path, counts


def test_steps_of_speculative_decoding():
    """Four steps: each attention against the plain form over what lies in the cache, each verification against
    the plain one, and at the end every kept row is its accepted token's, quantized at its place."""
    lens, n = [37, 0, 130], 9
    lp = Loop(lens, n)
    Hq, Hkv, D = lp.dims
    accepted = [[] for _ in lens]
    for step in range(4):
        lp.fill(step)
        before = lp.old.tolist()
        q, out, tokens, path, counts = lp.step()
        torch.cuda.synchronize()
        x = lp.x.cpu()
        want = spec_ref.verify(lp.logits.double().cpu().numpy(), lp.tokens.tolist(), lp.u.tolist(), lp.starts.tolist(), n, lp.par.tolist())
        assert [tokens.tolist(), path.tolist(), counts.tolist()] == [list(w) for w in want]
        # the cache as the attention saw it: before the rows were moved
        view = Cache.__new__(Cache)
        view.S, view.Hkv, view.D, view.hd = lp.S, Hkv, D, Hkv * D
        view.host = [tuple(host_of(c)) for c in lp.caches]
        pos = torch.tensor([before[b] + d for b in range(len(lens)) for d in spec_ref.depth_of(lp.parents[b])], dtype=torch.int32)
        k = spec_ref.turned(x[:, Hq * D:(Hq + Hkv) * D].reshape(-1, Hkv, D), lp.cos.cpu(), lp.sin.cpu(), pos, False, False, None, 0.0)
        v = x[:, (Hq + Hkv) * D:].reshape(-1, Hkv, D)
        rows = np.array([spec_ref.cache_row(lp.table, lp.page, lp.S, b, before[b] + i) for b in range(len(lens)) for i in range(n)], np.int32)
        for c, t in zip(view.host, (k, v)):
            oracle.kv_quantize(bits(t).reshape(len(rows), -1), c, slot=rows, dtype=ODT[lp.dtype])
        view.val = [torch.from_numpy(oracle.kv_dequant(c, lp.S, view.hd)).view(lp.S, Hkv, D).double() for c in view.host]
        wt, _ = tree_want(view, q.cpu(), lp.table, lp.page, [x + n for x in before], lp.starts.tolist(), lp.sees, D ** -0.5)
        _check_rows(out, None, wt)
        for b in range(len(lens)):
            for j, node in enumerate(path.tolist()[b][:counts.tolist()[b]]):
                accepted[b].append((spec_ref.cache_row(lp.table, lp.page, lp.S, b, before[b] + j), k[b * n + node], v[b * n + node]))
    assert sum(len(a) for a in accepted) > 4 * len(lens)
    for b, rows in enumerate(accepted):
        at = np.array([r for r, _, _ in rows], np.int64)
        for c, i in zip(lp.caches, (1, 2)):
            host = oracle.kv_alloc(len(rows), Hkv * D)
            oracle.kv_quantize(np.stack([bits(r[i]).reshape(-1) for r in rows]), host, dtype=ODT[lp.dtype])
            for got, want in zip(host_of(c), host):
                assert np.array_equal(got[at], want), b


@pytest.mark.parametrize("lens,page", [([3000, 2500], 32), ([30, 9, 77], 4)])
def test_a_step_captured_and_replayed(lens, page):
    """The whole step in one graph (its attention split with a workspace, lengths growing on the device), replayed
    with new inputs, against the same steps taken eagerly on a copy."""
    a, b = Loop(lens, 6, page=page), Loop(lens, 6, page=page)
    for lp in (a, b):
        lp.fill(0)
        lp.step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = a.step()
    for i in (1, 2, 3, 4):
        for lp in (a, b):
            lp.fill(i)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        want = b.step()
        torch.cuda.synchronize()
        for x, y in zip(outs, want):
            assert torch.equal(x, y), i
        assert torch.equal(a.old, b.old)
        for c, d in zip(a.caches, b.caches):
            assert torch.equal(c.codes, d.codes) and torch.equal(c.s, d.s) and torch.equal(c.zpacked, d.zpacked), i


def test_steps_on_two_streams_at_once():
    """Two loops on two streams, in turn, give what they give alone."""
    want, loops = [], []
    for seed in (1, 2):
        lp = Loop([2500, 40], 5, page=32)
        lp.fill(seed)
        want.append([t.clone() for t in lp.step()])
    torch.cuda.synchronize()
    for seed in (1, 2):
        lp = Loop([2500, 40], 5, page=32)
        lp.fill(seed)
        loops.append((lp, torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = []
    for lp, s in loops:
        with torch.cuda.stream(s):
            got.append(lp.step())
    torch.cuda.synchronize()
    for x, y in zip(got, want):
        for u, v in zip(x, y):
            assert torch.equal(u, v)
    # and with the stream as an argument
    lp, s = loops[0]
    s.wait_stream(torch.cuda.current_stream())
    out = wq.wq_verify_drafts(lp.logits, lp.tokens, lp.u, q_starts=lp.starts, max_queries=5, parents=lp.par, stream=s)
    s.synchronize()
    for u, v in zip(out, want[0][2:]):
        assert torch.equal(u, v)


def test_steps_in_two_threads():
    """Two threads, each with a loop and stream of its own and workspaces made for them, give what the loops give
    alone; a call that is refused in one of them is an error there."""
    want, loops = [], []
    for seed in (1, 2):
        lp = Loop([2500, 40], 5, page=32)
        lp.fill(seed)
        want.append([t.clone() for t in lp.step()])
        lp.fill(seed)
        loops.append(lp)
    torch.cuda.synchronize()
    failed = []

    def work(i):
        try:
            s, lp = torch.cuda.Stream(), loops[i]
            with torch.cuda.stream(s):
                for _ in range(20):
                    lp.old.copy_(i32([2500, 40]))
                    got = lp.step()
                    with pytest.raises(ValueError, match="uniform"):
                        wq.wq_verify_drafts(lp.logits, lp.tokens, lp.u[:-1])
                    s.synchronize()
                    for u, v in zip(got, want[i]):
                        assert torch.equal(u, v)
        except BaseException as e:
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed[0]
