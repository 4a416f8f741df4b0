"""What the operators of one speculative decoding step over the INT4 KV cache are measured on.

Four operators, in the order a step runs them (a sequence's nodes are its last token and the tokens drafted after it):

* ``append``: the rotation of queries and keys (with their norm, where a model has one) and the quantization of keys and
  values into the pages of the INT4 cache, in one pass;
* ``tree``: attention over that cache for the nodes of a draft tree, each of which sees the context and its ancestors;
* ``verify``: the drafted tokens against the target's distributions, from given random numbers: which are accepted, and the
  token that follows them;
* ``keep``: the cache rows of the accepted nodes moved together.

A case is a dict of plain values.  ``run`` computes it in plain torch (``own`` false) or through the library's entry
points (``own`` true).
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_EPS = 1e-6


def _wq():
    import w4a16_bit_matmul_amd as wq
    return wq


# ---- the cases -----------------------------------------------------------------

def listed():
    return [
        # the decode step of 64 sequences of a 70B-style layer (64 query heads, 8 KV heads of 128): a token each
        dict(name="append_decode_64", op="append", B=64, n_lo=1, n_hi=1, old=8192, Hq=64, Hkv=8, D=128, rot=128, inter=False, norm=False, k_out=False, page=64, dtype="bf16", far=131072),
        # draft trees of a small model (14 query heads, 2 KV heads of 64, normed heads, half of the channels rotated as
        # neighbouring pairs), tiny pages
        dict(name="append_trees", op="append", B=13, n_lo=3, n_hi=25, old=1000, Hq=14, Hkv=2, D=64, rot=32, inter=True, norm=True, k_out=False, page=4, dtype="f16", far=4096),
        # three long prompts of the 70B-style layer, whose rotated keys the prompt's own attention needs too
        dict(name="append_prompts", op="append", B=3, n_lo=9001, n_hi=12000, old=0, Hq=64, Hkv=8, D=128, rot=128, inter=False, norm=False, k_out=True, page=64, dtype="bf16", far=32768),
        # eight nodes after the first tokens of one conversation: the shortest call, latency alone
        dict(name="tree_one_short", op="tree", B=1, len_lo=300, len_hi=300, n_lo=8, n_hi=8, Hq=64, Hkv=8, D=128, page=16, dtype="bf16"),
        # trees of up to 16 nodes in a batch of 48 sequences
        dict(name="tree_batch", op="tree", B=48, len_lo=3001, len_hi=6000, n_lo=5, n_hi=16, Hq=64, Hkv=8, D=128, page=64, dtype="bf16"),
        # large trees of few sequences (two mask words a node), heads of 64 in groups of four, small pages
        dict(name="tree_large", op="tree", B=4, len_lo=7000, len_hi=12001, n_lo=100, n_hi=120, Hq=32, Hkv=8, D=64, page=16, dtype="f16"),
        # one sequence's tree of twelve nodes
        dict(name="verify_one", op="verify", B=1, n_lo=12, n_hi=12, V=32768, kind="tree", dtype="f16", greedy=0.0, masked=0.0),
        # trees of 64 sequences: the largest
        dict(name="verify_trees", op="verify", B=64, n_lo=16, n_hi=16, V=131072, kind="tree", dtype="f16", greedy=0.1, masked=0.0),
        # chains drawn from a draft model's distributions, some sequences greedy, some rows with all but the likely
        # tokens masked, an odd vocabulary
        dict(name="verify_chains", op="verify", B=33, n_lo=1, n_hi=6, V=50001, kind="chain", dtype="bf16", greedy=0.2, masked=0.3),
        # plain sampling of a token for each of 128 sequences, nothing drafted
        dict(name="verify_sample", op="verify", B=128, n_lo=1, n_hi=1, V=100003, kind="tree", dtype="f32", greedy=0.1, masked=0.5),
        # what 64 sequences accepted of eight nodes each
        dict(name="keep_64", op="keep", B=64, n_lo=8, n_hi=8, len_hi=2000, hd=1024, page=64),
        # large trees of many sequences, tiny pages, an odd number of blocks in a row
        dict(name="keep_many", op="keep", B=200, n_lo=30, n_hi=64, len_hi=500, hd=1152, page=4),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "tree", "tree", "verify", "verify", "keep"])
    D = rng.choice([64, 128, 128, 128, 256])
    Hkv = rng.choice([2, 4, 6, 8]) if D == 64 else rng.choice([1, 2, 3, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 5, 7, 8])
    page = rng.choice([1, 4, 16, 32, 64, 256])
    if op == "append":
        c = dict(op=op, Hq=Hq, Hkv=Hkv, D=D, page=page, dtype=rng.choice(["bf16", "f16"]), rot=rng.choice([D, D, D // 2, D // 4]),
                 inter=rng.random() < 0.5, norm=rng.random() < 0.4, k_out=rng.random() < 0.4)
        tokens = _log_int(rng, 1, min(30000, 30000 * 64 * 128 // (Hq * D)))
        c["B"] = min(tokens, _log_int(rng, 1, 100))
        c["n_hi"] = max(1, tokens // c["B"])
        c["n_lo"] = max(1, c["n_hi"] // rng.choice([1, 2, 10]))
        c["old"] = _log_int(rng, 1, 4096) if c["n_hi"] <= 64 else 0
        c["far"] = max(c["n_hi"] + c["old"], _log_int(rng, 64, 131072))
        return c
    if op == "tree":
        c = dict(op=op, Hq=Hq, Hkv=Hkv, D=D, page=page, dtype=rng.choice(["bf16", "f16"]))
        c["B"] = _log_int(rng, 1, 64)
        c["n_hi"] = _log_int(rng, 1, 128 if c["B"] <= 8 else 32)
        c["n_lo"] = max(1, c["n_hi"] // rng.choice([1, 2, 10]))
        most = 200_000_000 * 128 // max(D, 128)
        top = min(most // (c["B"] * Hq * c["n_hi"]), most // (c["B"] * Hkv * 128), 131072)
        c["len_hi"] = c["n_hi"] + _log_int(rng, 1, max(2, top - c["n_hi"]))
        c["len_lo"] = c["n_hi"] + (c["len_hi"] - c["n_hi"]) // rng.choice([1, 2, 10])
        return c
    if op == "verify":
        c = dict(op=op, kind=rng.choice(["tree", "tree", "chain"]), dtype=rng.choice(["bf16", "f16", "f32"]))
        c["V"] = _log_int(rng, 100, 200000)
        c["n_hi"] = _log_int(rng, 1, 64)
        c["n_lo"] = max(1, c["n_hi"] // rng.choice([1, 2, 10]))
        c["B"] = _log_int(rng, 1, max(1, min(256, 60_000_000 // (c["V"] * c["n_hi"]))))
        c["greedy"], c["masked"] = rng.choice([0.0, 0.2, 1.0]), rng.choice([0.0, 0.0, 0.5])
        return c
    c = dict(op=op, page=page, hd=128 * rng.choice([1, 2, 3, 4, 8, 16]))
    c["B"], c["n_hi"] = _log_int(rng, 1, 256), _log_int(rng, 1, 64)
    c["n_lo"] = max(1, c["n_hi"] // rng.choice([1, 2]))
    c["len_hi"] = c["n_hi"] + _log_int(rng, 1, 400)
    return c


def _nodes(case):
    """Tokens of the call in each sequence: the case's own, not the seed's, so that every state of a case is the same work."""
    r = np.random.default_rng(case["B"] * 1000003 + case["n_hi"])
    n = r.integers(case["n_lo"], case["n_hi"] + 1, case["B"])
    n[int(r.integers(0, case["B"]))] = case["n_hi"]
    return n.astype(np.int64)


def _lengths(case):
    """Cached tokens of each sequence, the call's own among them."""
    n, r = _nodes(case), np.random.default_rng(case["B"] * 7919 + case["n_hi"])
    if case["op"] == "append":
        return n + (r.integers(0, case["old"] + 1, case["B"]) if case["old"] else 0)
    if case["op"] == "keep":
        return n + r.integers(0, case["len_hi"] - case["n_hi"] + 1, case["B"])
    lens = r.integers(case["len_lo"], case["len_hi"] + 1, case["B"])
    lens[int(r.integers(0, case["B"]))] = case["len_hi"]
    return np.maximum(lens, n)


def _tree(case):
    """Parents of the nodes, [B][n_hi] (-1: the root, or no node), and their depths."""
    n, r = _nodes(case), np.random.default_rng(case["B"] * 31 + case["n_hi"])
    parents = np.full((case["B"], case["n_hi"]), -1, np.int64)
    depth = np.zeros_like(parents)
    at = np.arange(case["B"])
    for i in range(1, case["n_hi"]):
        # a node hangs from one of the last few: deep branches with siblings
        p = np.maximum(0, i - 1 - r.integers(0, 5, case["B"])) if case.get("kind") != "chain" else np.full(case["B"], i - 1)
        parents[:, i] = np.where(i < n, p, -1)
        depth[:, i] = np.where(i < n, depth[at, p] + 1, 0)
    return parents, depth


def _path(case):
    """Accepted nodes of each sequence, [B][n_hi] (-1 behind the last), and how many: the root and a way down the tree."""
    parents, _ = _tree(case)
    n, r = _nodes(case), np.random.default_rng(case["B"] * 131 + case["n_hi"])
    path, count = np.full_like(parents, -1), np.zeros(case["B"], np.int64)
    for b in range(case["B"]):
        way, node = [], int(r.integers(0, n[b]))
        while node >= 0:
            way.append(node)
            node = int(parents[b, node])
        count[b] = len(way)
        path[b, :len(way)] = way[::-1]
    return path, count


def _row_bytes(hd):
    return hd // 2 + 2 * (hd // 128) + (hd // 128 + 1) // 2


def work(case):
    n = int(_nodes(case).sum())
    if case["op"] == "append":
        Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
        # q, k, v in; q (and k) out; both caches' rows; the cos and sin rows and the page of every token
        out = Hq + (Hkv if case["k_out"] else 0)
        return {"bytes": n * (2 * D * (Hq + 2 * Hkv + out) + 2 * _row_bytes(Hkv * D) + 4 * case["rot"] + 4),
                "flops": n * D * (3 * (Hq + Hkv) + 8 * 2 * Hkv + (4 * (Hq + Hkv) if case["norm"] else 0))}
    if case["op"] == "tree":
        Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
        lens, nodes = _lengths(case), _nodes(case)
        _, depth = _tree(case)
        live = np.arange(case["n_hi"])[None, :] < nodes[:, None]
        seen = int(((lens - nodes)[:, None] + depth + 1)[live].sum())
        pages = int((-(-lens // case["page"])).sum())
        return {"bytes": 2 * _row_bytes(Hkv * D) * int(lens.sum()) + 4 * pages + 8 * n * -(-case["n_hi"] // 64) + 2 * 2 * n * Hq * D + 4 * n * Hq,
                "flops": 4 * D * Hq * seen}
    if case["op"] == "verify":
        size = {"f32": 4, "bf16": 2, "f16": 2}[case["dtype"]]
        rows = n + (n - case["B"] if case["kind"] == "chain" else 0)
        return {"bytes": rows * case["V"] * size + 16 * n + 4 * case["B"] * (2 * case["n_hi"] + 2), "flops": 4 * rows * case["V"]}
    path, count = _path(case)
    moved = int((path != np.arange(case["n_hi"])[None, :])[path >= 0].sum())
    return {"bytes": 2 * 2 * moved * _row_bytes(case["hd"]) + 4 * int(count.sum()), "flops": 0}


# ---- inputs --------------------------------------------------------------------

# value e of eight neighbouring ones sits in this nibble of their 32-bit word
_NIBBLE = [4 * (e % 2) + e // 2 for e in range(8)]


def _dev(x, dtype=np.int32):
    return torch.from_numpy(np.ascontiguousarray(x).astype(dtype)).cuda()


def _starts(n):
    return _dev(np.concatenate([[0], np.cumsum(n)]))


def _pages(case, seed, lens):
    """A block table in which the sequences' pages lie anywhere, and the cache rows that takes."""
    need = -(-lens // case["page"])
    order = np.random.default_rng(seed).permutation(int(need.sum()) + 3)
    table = np.full((case["B"], int(need.max())), -1, np.int32)
    table[np.arange(table.shape[1])[None, :] < need[:, None]] = order[:int(need.sum())]
    return _dev(table), len(order) * case["page"]


def _cache(g, S, hd, std, wide):
    """An INT4 cache of S rows of hd values: codes of normal values, fp16 scales, zero-points, two blocks a byte."""
    nb = hd // 128
    codes = torch.empty((S, hd // 2), dtype=torch.uint8, device="cuda")
    for r0 in range(0, S, 65536):  # codes near 7.5 with a spread of 2.6, as quantized normal values have
        x = torch.randn((min(S, r0 + 65536) - r0, hd // 2, 2), generator=g, device="cuda")
        x = (x * 2.6 + 7.5).round_().clamp_(0, 15).to(torch.uint8)
        codes[r0:r0 + 65536] = x[:, :, 0] | x[:, :, 1] << 4
    s = torch.rand((S, nb), generator=g, device="cuda") * 0.3 + 0.85
    s *= torch.where(torch.rand((1, nb), generator=g, device="cuda") < wide, 3.0, 1.0) * (std / 2.6)
    z = torch.randint(6, 10, (S, 2 * ((nb + 1) // 2)), generator=g, device="cuda", dtype=torch.uint8)
    z[:, nb:] = 0
    return [codes, s.to(torch.float16), z[:, 0::2] | z[:, 1::2] << 4]


def _tables(rot, far):
    # the angles of far positions need 64 bits; the tables hold their cosines and sines in 32
    f = 10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64, device="cuda") * 2 / rot)
    ang = torch.arange(far, dtype=torch.float64, device="cuda")[:, None] * f
    return ang.cos().float(), ang.sin().float()


def _masks(case):
    """The mask words of all nodes, [T][ceil(n_hi / 64)]: bit j of a node's words is set if it sees node j."""
    parents, _ = _tree(case)
    n, B, N = _nodes(case), case["B"], case["n_hi"]
    sees = np.zeros((B, N, 64 * -(-N // 64)), bool)
    at = np.arange(B)
    for i in range(N):
        if i:
            sees[:, i] = sees[at, np.maximum(parents[:, i], 0)]
        sees[:, i, i] = True
    words = np.packbits(sees, axis=-1, bitorder="little").view(np.int64)
    return words[np.arange(N)[None, :] < n[:, None]]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    st = {"case": case}
    n = _nodes(case)
    st["q_starts"] = _starts(n)
    if case["op"] == "verify":
        return _prepare_verify(case, g, st, n)
    lens = _lengths(case)
    st["context_lens"] = _dev(lens)
    st["block_table"], S = _pages(case, seed, lens)
    T = int(n.sum())
    if case["op"] == "keep":
        path, count = _path(case)
        st["path"], st["counts"] = _dev(path), _dev(count)
        st["k_arrays"], st["v_arrays"] = _cache(g, S, case["hd"], 1.0, 0.1), _cache(g, S, case["hd"], 0.5, 0.0)
        return st
    Hq, Hkv, D, dt = case["Hq"], case["Hkv"], case["D"], _DTYPES[case["dtype"]]
    st["k_arrays"], st["v_arrays"] = _cache(g, S, Hkv * D, 1.0, 0.1), _cache(g, S, Hkv * D, 0.5, 0.0)
    if case["op"] == "tree":
        st["q"] = torch.randn((T, Hq, D), generator=g, device="cuda").to(dt)
        st["tree_mask"] = torch.from_numpy(_masks(case)).cuda()
        return st
    # one fused projection, a few channels eight times larger, as a layer's matmul leaves it
    x = torch.randn((T, (Hq + 2 * Hkv) * D), generator=g, device="cuda")
    x *= torch.where(torch.rand((1, x.shape[1]), generator=g, device="cuda") < 0.01, 8.0, 1.0)
    x = x.to(dt)
    st["q"] = x[:, :Hq * D].view(T, Hq, D)
    st["k"] = x[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D)
    st["v"] = x[:, (Hq + Hkv) * D:].view(T, Hkv, D)
    st["q_weight"], st["k_weight"] = ((1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(dt) for _ in range(2))
    st["cos"], st["sin"] = _tables(case["rot"], case["far"])
    # a node's position is its depth's, not its row's; a prompt's tokens follow one another
    _, depth = _tree(case) if case["n_hi"] <= 64 else (None, np.arange(case["n_hi"])[None, :].repeat(case["B"], 0))
    pos = (lens - n)[:, None] + depth
    st["positions"] = _dev(pos[np.arange(case["n_hi"])[None, :] < n[:, None]])
    return st


def _prepare_verify(case, g, st, n):
    T, V, B, dt = int(n.sum()), case["V"], case["B"], _DTYPES[case["dtype"]]
    rand = lambda *s: torch.rand(s, generator=g, device="cuda")  # noqa: E731
    # a background of many unlikely tokens, and six per row that share most of the probability
    x = torch.randn((T, V), generator=g, device="cuda") * 2.0
    likely = torch.randint(0, V, (T, 6), generator=g, device="cuda")
    x.scatter_(1, likely, math.log(V) + 2.0 + 4.0 * rand(T, 6))
    if case["masked"]:
        rows = rand(T, 1) < case["masked"]
        x.masked_fill_(rows & (x < 3.0), -math.inf)
    st["logits"] = x.to(dt)
    st["temperature"] = torch.where(rand(B) < case["greedy"], torch.zeros(B, device="cuda"), 0.5 + 0.7 * rand(B))
    st["uniform"] = rand(T)
    row = st["q_starts"].long()[:-1, None] + torch.from_numpy(np.maximum(_tree(case)[0], 0)).cuda()
    live = torch.arange(case["n_hi"], device="cuda")[None, :] < torch.from_numpy(n).cuda()[:, None]
    parent_row = row[live]  # (a root's: its own)
    if case["kind"] == "chain":
        # the draft model agrees with the target up to some noise; its tokens are drawn from its own distributions
        d = torch.where(x > -math.inf, 0.9 * x + 0.7 * torch.randn((T, V), generator=g, device="cuda"), x)
        st["draft_logits"] = d.to(dt)
        t = st["temperature"].repeat_interleave(torch.from_numpy(n).cuda())[:, None].clamp(min=0.05)
        d = st["draft_logits"].float() / t - torch.log(-torch.log(rand(T, V).clamp(1e-30, 1 - 1e-7)))
        st["tokens"] = d.argmax(-1)[parent_row].int()
        return st
    st["parents"] = torch.from_numpy(_tree(case)[0]).cuda()[live].int()
    # a node's token is one of its parent's likely ones: the first child has the likeliest, and so on
    i = torch.arange(T, device="cuda")
    elder = torch.zeros(T, dtype=torch.int64, device="cuda")
    for k in range(1, min(8, T)):
        elder[k:] += (parent_row[k:] == parent_row[:T - k]) & (i[k:] != parent_row[k:]) & (i[:T - k] != parent_row[:T - k])
    top = torch.topk(st["logits"].float(), 6, -1).indices
    st["tokens"] = top[parent_row, elder.clamp(max=5)].int()
    return st


# ---- one pass ------------------------------------------------------------------

def run(st):
    return {"append": _run_append, "tree": _run_tree, "verify": _run_verify, "keep": _run_keep}[st["case"]["op"]](st)


def _own_caches(wq, st, hd):
    return [wq.KVCache(*st[a], st[a][0].shape[0], hd) for a in ("k_arrays", "v_arrays")]


def _places(st):
    """Sequence, place in it and sequence's first place of every token of the call."""
    starts = st["q_starts"].long()
    t = torch.arange(st["q"].shape[0] if "q" in st else st["logits"].shape[0], device="cuda")
    b = torch.searchsorted(starts[1:], t, right=True)
    return b, t - starts[b], starts


def _normed(x, w):
    """The norm of every head, each step one operation in 32 bits but for the sum of squares, which is taken in 64 (the
    cache's codes must not hang on the order of a sum)."""
    x = x.float()
    ms = (x.double().square().sum(-1, keepdim=True) / x.shape[-1]).float()
    r = (ms + _EPS).double().sqrt().float().double().reciprocal().float()
    return x * r * w.float()


def _turned(x, cos, sin, inter):
    """The rotation, each product and sum rounded to 32 bits."""
    r = 2 * cos.shape[-1]
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if inter else (x[..., : r // 2], x[..., r // 2: r])
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((a, b), -1).flatten(-2) if inter else torch.cat((a, b), -1)
    return torch.cat((turned, x[..., r:]), -1)


def _quantized(x):
    """Rows of hd values as cache rows: codes, scales, zero-points; every step one operation rounded to 32 bits."""
    T, hd = x.shape
    x = x.float().view(T, hd // 128, 128)
    lo, hi = x.amin(-1, keepdim=True).clamp(max=0), x.amax(-1, keepdim=True).clamp(min=0)
    s16 = ((hi - lo).double() / 15).float().to(torch.float16)
    s = s16.float()
    some = s > 0
    d = torch.where(some, s, torch.ones_like(s)).double()
    z = torch.where(some, (-lo / d).float().round().clamp(0, 15), torch.zeros_like(s))
    q = ((x / d).float() + z).round().clamp(0, 15)
    q = torch.where(some, q, torch.zeros_like(q)).to(torch.int64).view(T, hd // 8, 8)
    word = (q << torch.tensor([4 * p for p in _NIBBLE], device=q.device)).sum(-1)
    codes = ((word[..., None] >> torch.tensor([0, 8, 16, 24], device=q.device)) & 255).to(torch.uint8).view(T, hd // 2)
    z = torch.nn.functional.pad(z[:, :, 0].to(torch.uint8), (0, hd // 128 % 2))
    return codes, s16[:, :, 0], z[:, 0::2] | z[:, 1::2] << 4


def _run_append(st):
    c = st["case"]
    if own:
        wq = _wq()
        kc, vc = _own_caches(wq, st, c["Hkv"] * c["D"])
        q, k = wq.wq_kv_append(st["k"], st["v"], kc, vc, st["block_table"], st["context_lens"], st["cos"], st["sin"], q=st["q"],
                               page_size=c["page"], q_starts=st["q_starts"], positions=st["positions"], norm=c["norm"],
                               q_weight=st["q_weight"] if c["norm"] else None, k_weight=st["k_weight"] if c["norm"] else None,
                               eps=_EPS, interleaved=c["inter"], k_out=c["k_out"])
        return [q] + ([k] if c["k_out"] else []) + st["k_arrays"] + st["v_arrays"]
    at = st["positions"].long()
    cos, sin = st["cos"][at][:, None, :], st["sin"][at][:, None, :]
    q, k = ((_normed(st[a], st[a + "_weight"]) if c["norm"] else st[a].float()) for a in ("q", "k"))
    q, k = (_turned(x, cos, sin, c["inter"]).to(st["q"].dtype) for x in (q, k))
    b, i, starts = _places(st)
    token = st["context_lens"].long()[b] - (starts[b + 1] - starts[b]) + i
    rows = st["block_table"].long()[b, token // c["page"]] * c["page"] + token % c["page"]
    for x, arrays in ((k, st["k_arrays"]), (st["v"], st["v_arrays"])):
        for to, made in zip(arrays, _quantized(x.reshape(x.shape[0], -1))):
            to[rows] = made
    return [q] + ([k] if c["k_out"] else []) + st["k_arrays"] + st["v_arrays"]


def _decoded(arrays, rows, hd):
    """The named rows of a cache in fp32, [...][hd]."""
    codes, s, zp = (a[rows] for a in arrays)
    shape, nb = rows.shape, hd // 128
    b = codes.view(*shape, hd // 8, 4).int()
    word = b[..., 0] | (b[..., 1] << 8) | (b[..., 2] << 16) | (b[..., 3] << 24)
    q = torch.stack([(word >> (4 * k)) & 15 for k in _NIBBLE], -1).view(*shape, nb, 128)
    z = torch.stack((zp & 15, zp >> 4), -1).view(*shape, -1)[..., :nb].int()
    return ((q - z[..., None]).float() * s.float()[..., None]).view(*shape, hd)


def _run_tree(st):
    c = st["case"]
    Hq, Hkv, D, B, N, L = c["Hq"], c["Hkv"], c["D"], c["B"], c["n_hi"], c["len_hi"]
    G = Hq // Hkv
    if own:
        wq = _wq()
        kc, vc = _own_caches(wq, st, Hkv * D)
        return wq.wq_kv_tree_attention(st["q"], kc, vc, st["block_table"], st["context_lens"], st["tree_mask"], page_size=c["page"],
                                       q_starts=st["q_starts"], max_context=L, max_queries=N, lse=True)
    starts, lens = st["q_starts"].long(), st["context_lens"].long()
    n = starts[1:] - starts[:-1]
    t = torch.arange(L, device="cuda")
    page = st["block_table"].long()[:, t // c["page"]].clamp(min=0)
    rows = torch.where(t < lens[:, None], page * c["page"] + t % c["page"], 0)
    # [B][Hkv][...]: the sequences padded to the longest, the heads of a group among the rows of their KV head
    kt = _decoded(st["k_arrays"], rows, Hkv * D).view(B, L, Hkv, D).permute(0, 2, 3, 1).contiguous()
    v = _decoded(st["v_arrays"], rows, Hkv * D).view(B, L, Hkv, D).permute(0, 2, 1, 3).contiguous()
    at = torch.minimum(starts[:-1, None] + torch.arange(N, device="cuda"), starts[-1] - 1)
    q = st["q"].float()[at].view(B, N, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, N * G, D)
    word = st["tree_mask"][at]
    bits = ((word[..., None] >> torch.arange(64, device="cuda")) & 1).bool().view(B, N, -1)
    node = t - (lens - n)[:, None]
    seen = (node < 0)[:, None, :] | torch.gather(bits, 2, node.clamp(0, bits.shape[2] - 1)[:, None, :].expand(B, N, L))
    seen &= (t < lens[:, None])[:, None, :]
    p = torch.matmul(q, kt).mul_(D ** -0.5)
    p.view(B, Hkv, N, G, L).masked_fill_(~seen[:, None, :, None, :], -math.inf)
    m = p.amax(-1, keepdim=True).clamp(min=-1e30)
    p = p.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / l.clamp(min=1e-30)
    lse = (m + torch.log(l))[..., 0]
    b, i, _ = _places(st)
    o = o.view(B, Hkv, N, G, D)[b, :, i].reshape(-1, Hq, D)
    return o.to(st["q"].dtype), lse.view(B, Hkv, N, G)[b, :, i].reshape(-1, Hq)


def _distributions(x, t):
    """Per row of logits: the likeliest token (the first of equals), and weights in proportion to the probabilities at
    temperature t (0: the likeliest alone), in 64 bits."""
    x = x.double()
    m = x.amax(-1, keepdim=True)
    ids = torch.arange(x.shape[1], device=x.device)
    top = torch.where(x == m, ids, x.shape[1]).amin(-1)
    w = torch.where(t[:, None] > 0, torch.exp((x - m) / t[:, None]), (ids == top[:, None]).double())
    return top, w


def _picked(w, u):
    """The first token whose cumulated weight is above u of the whole."""
    cdf = w.cumsum(-1)
    at = (cdf <= u.double()[:, None] * cdf[:, -1:]).sum(-1)
    last = torch.where(w > 0, torch.arange(w.shape[1], device=w.device), -1).amax(-1)
    return torch.minimum(at, last)


def _run_verify(st):
    c = st["case"]
    if own:
        return _wq().wq_verify_drafts(st["logits"], st["tokens"], st["uniform"], q_starts=st["q_starts"], max_queries=c["n_hi"],
                                      parents=st.get("parents"), draft_logits=st.get("draft_logits"), temperature=st["temperature"])
    N = c["n_hi"]
    b, i, starts = _places(st)
    n = starts[1:] - starts[:-1]
    at = torch.minimum(starts[:-1, None] + torch.arange(N, device="cuda"), starts[-1] - 1)  # [B][N] rows
    live = torch.arange(N, device="cuda") < n[:, None]
    tokens, u, t = st["tokens"].long(), st["uniform"], st["temperature"]
    top, w = _distributions(st["logits"], t[b])
    if c["kind"] == "chain":
        dtop, d = _distributions(st["draft_logits"], t[b])
        p, q = w / w.sum(-1, keepdim=True), d / d.sum(-1, keepdim=True)
        draft = tokens[(at + 1).clamp(max=tokens.numel() - 1)]  # the token drafted after a row
        coin = u.double()[(at + 1).clamp(max=tokens.numel() - 1)]
        yes = torch.where(t[:, None] > 0, coin * q[at, draft] < p[at, draft], top[at] == draft)
        yes = yes & (torch.arange(N, device="cuda") < n[:, None] - 1)
        took = yes.long().cumprod(-1).sum(-1)  # drafts accepted
        last = starts[:-1] + took
        left = torch.where(((took < n - 1) & (t > 0))[:, None], (p[last] - q[last]).clamp(min=0), p[last])
        left = torch.where(left.sum(-1, keepdim=True) > 0, left, p[last])
        new = _picked(left, u[starts[:-1]])
        kept = torch.arange(N, device="cuda") <= took[:, None]
        path = torch.where(kept, torch.arange(N, device="cuda"), -1)
        count = took + 1
    else:
        pick = _picked(w, u)
        mother = st["parents"].long()[at]  # of node j of sequence b; the root has none
        matched = (tokens[at] == pick[(starts[:-1, None] + mother).clamp(0, tokens.numel() - 1)]) & (mother >= 0) & live
        # of siblings with one token the first counts
        j = torch.arange(N, device="cuda")
        twin = (mother[:, :, None] == mother[:, None, :]) & (tokens[at][:, :, None] == tokens[at][:, None, :]) & (j[None, :] < j[:, None])
        matched &= ~(twin & live[:, None, :]).any(-1)
        # a node is accepted if it and all of its ancestors are: ways to the root by doubling steps
        good = matched | (j == 0) & live
        step = mother.clamp(min=0)
        for _ in range(max(1, (N - 1).bit_length())):
            good = good & torch.gather(good, 1, step)
            step = torch.gather(step, 1, step)
        path = torch.where(good, j, N).sort(-1).values
        path = torch.where(path < N, path, -1)
        count = good.sum(-1)
        new = pick[starts[:-1] + torch.gather(path, 1, (count - 1)[:, None])[:, 0]]
    j = torch.arange(N, device="cuda")
    after = tokens[torch.gather(at, 1, torch.roll(path, -1, 1).clamp(min=0))]
    out = torch.where(j < (count - 1)[:, None], after, torch.where(j == (count - 1)[:, None], new[:, None], -1))
    return out.int(), path.int(), count.int()


def _run_keep(st):
    c = st["case"]
    if own:
        wq = _wq()
        kc, vc = _own_caches(wq, st, c["hd"])
        wq.wq_kv_keep(kc, vc, st["block_table"], st["context_lens"], st["path"], st["counts"], page_size=c["page"],
                      q_starts=st["q_starts"])
        return st["k_arrays"] + st["v_arrays"]
    starts, path = st["q_starts"].long(), st["path"].long()
    first = st["context_lens"].long() - (starts[1:] - starts[:-1])
    j = torch.arange(path.shape[1], device="cuda").expand_as(path)
    kept = (j < st["counts"][:, None]) & (path >= j)
    b = torch.arange(c["B"], device="cuda")[:, None].expand_as(path)[kept]

    def rows(node):
        token = first[b] + node[kept]
        return st["block_table"].long()[b, token // c["page"]] * c["page"] + token % c["page"]

    source, target = rows(path), rows(j)
    for x in st["k_arrays"] + st["v_arrays"]:
        x[target] = x[source]
    return st["k_arrays"] + st["v_arrays"]


# ---- the definition, in 64 bits --------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    return {"append": _exact_append, "tree": _exact_tree, "verify": _exact_verify, "keep": _exact_keep}[case["op"]](case, st)


def _cache_row(case, table, token):
    return int(table[token // case["page"]]) * case["page"] + token % case["page"]


def _exact_append(case, st):
    n, lens, rot = _nodes(case), _lengths(case), case["rot"]
    pos = st["positions"].long()
    c, s = st["cos"].double()[pos][:, None], st["sin"].double()[pos][:, None]
    first = torch.arange(0, rot, 2) if case["inter"] else torch.arange(rot // 2)
    second = first + (1 if case["inter"] else rot // 2)
    first, second = first.cuda(), second.cuda()
    made = []
    for name in ("q", "k"):
        x = st[name].double()
        if case["norm"]:
            x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / case["D"] + _EPS) * st[name + "_weight"].double()
        y = x.clone()
        y[:, :, first] = x[:, :, first] * c - x[:, :, second] * s
        y[:, :, second] = x[:, :, second] * c + x[:, :, first] * s
        made.append(y)
    table = st["block_table"].cpu().numpy()
    rows = torch.tensor([_cache_row(case, table[b], int(lens[b] - n[b]) + i) for b in range(case["B"]) for i in range(int(n[b]))], device="cuda")
    caches = []
    for x, name in ((made[1].to(st["k"].dtype).double(), "k_arrays"), (st["v"].double(), "v_arrays")):
        hd = case["Hkv"] * case["D"]
        x = x.reshape(-1, hd // 128, 128)
        low, high = torch.clamp(x.min(-1).values, max=0), torch.clamp(x.max(-1).values, min=0)
        scales = st[name][1].double()
        scales[rows] = ((high - low) / 15).to(torch.float16).double()
        # codes and zero-points are whole numbers of one rounding each: their bits are the definition in 32 bits, not this one
        caches += [None, scales, None]
    return made[:2 if case["k_out"] else 1] + caches


def _exact_tree(case, st):
    n, lens = _nodes(case), _lengths(case)
    if float((n * lens).sum()) * case["Hq"] * case["D"] > 1.2e12:
        return None
    D, Hq, Hkv = case["D"], case["Hq"], case["Hkv"]
    G, hd, at = Hq // Hkv, Hkv * D, 0
    parents, _ = _tree(case)
    table = st["block_table"].cpu().numpy().astype(np.int64)
    out = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(st["q"].shape[:2], dtype=torch.float64, device="cuda")
    for b in range(case["B"]):
        m, ln = int(n[b]), int(lens[b])
        t = np.arange(ln)
        rows = torch.from_numpy(table[b][t // case["page"]] * case["page"] + t % case["page"]).cuda()
        sees = np.ones((m, ln), bool)
        sees[:, ln - m:] = False
        for i in range(m):
            node = i
            while node >= 0:
                sees[i, ln - m + node] = True
                node = int(parents[b, node])
        hidden = torch.from_numpy(~sees).cuda().repeat_interleave(G, 0)
        kv = []
        for name in ("k_arrays", "v_arrays"):
            codes, s, zp = (a.index_select(0, rows) for a in st[name])
            full = torch.empty((ln, hd), dtype=torch.float64, device="cuda")
            for d in range(8):  # value d of every eight: byte and half of its word
                byte = codes[:, _NIBBLE[d] // 2::4]
                full[:, d::8] = (byte >> 4 if _NIBBLE[d] % 2 else byte & 15).double()
            for blk in range(hd // 128):
                z = zp[:, blk // 2] >> 4 if blk % 2 else zp[:, blk // 2] & 15
                full[:, 128 * blk:128 * blk + 128].sub_(z.double()[:, None]).mul_(s[:, blk].double()[:, None])
            kv.append(full.view(ln, Hkv, D))
        for h in range(Hkv):
            qh = st["q"][at:at + m, h * G:(h + 1) * G].double().reshape(m * G, D)
            sc = (qh @ kv[0][:, h].t().contiguous()) / math.sqrt(D)
            sc[hidden] = -math.inf
            lse[at:at + m, h * G:(h + 1) * G] = torch.logsumexp(sc, -1).view(m, G)
            out[at:at + m, h * G:(h + 1) * G] = (torch.softmax(sc, -1) @ kv[1][:, h].contiguous()).view(m, G, D)
        at += m
    return out, lse


def _exact_verify(case, st):
    """Sequence by sequence, token by token."""
    n, N, B = _nodes(case), case["n_hi"], case["B"]
    if int(n.sum()) * case["V"] > 3e8:
        return None
    at = np.concatenate([[0], np.cumsum(n)])
    tokens, u, t = (st[k].cpu().numpy() for k in ("tokens", "uniform", "temperature"))
    parents, _ = _tree(case)
    out, path, count = np.full((B, N), -1, np.int32), np.full((B, N), -1, np.int32), np.zeros(B, np.int32)

    def probabilities(name, row, temp):
        x = st[name][row].double()
        if temp == 0:
            p = torch.zeros_like(x)
            p[int((x == x.max()).nonzero()[0])] = 1
            return p
        return torch.softmax(x / float(temp), -1)

    def sample(p, coin):
        cdf = torch.cumsum(p, 0)
        return min(int(torch.searchsorted(cdf, float(coin) * float(cdf[-1]), right=True)), int((p > 0).nonzero()[-1]))

    for b in range(B):
        node, way, temp = 0, [0], np.float64(t[b])
        while True:
            row = int(at[b]) + node
            p = probabilities("logits", row, temp)
            if case["kind"] == "chain":
                if node + 1 == n[b]:
                    new = sample(p, u[at[b]])
                    break
                x = int(tokens[row + 1])
                if temp == 0:
                    if p[x] == 1:
                        node += 1
                        way.append(node)
                        continue
                    new = int(p.argmax())
                    break
                d = probabilities("draft_logits", row, temp)
                if float(u[row + 1]) * float(d[x]) < float(p[x]):
                    node += 1
                    way.append(node)
                    continue
                new = sample((p - d).clamp(min=0), u[at[b]])
                break
            new = sample(p, u[row])
            nexts = [i for i in range(node + 1, int(n[b])) if parents[b, i] == node and tokens[at[b] + i] == new]
            if not nexts:
                break
            node = nexts[0]
            way.append(node)
        count[b] = len(way)
        path[b, :len(way)] = way
        out[b, :len(way)] = [tokens[at[b] + i] for i in way[1:]] + [new]
    return tuple(torch.from_numpy(x).cuda() for x in (out, path, count))


def _exact_keep(case, st):
    n, lens = _nodes(case), _lengths(case)
    table, path, count = (st[k].cpu().numpy() for k in ("block_table", "path", "counts"))
    source, target = [], []
    for b in range(case["B"]):
        for j in range(int(count[b])):
            source.append(_cache_row(case, table[b], int(lens[b] - n[b]) + int(path[b, j])))
            target.append(_cache_row(case, table[b], int(lens[b] - n[b]) + j))
    out = []
    for x in st["k_arrays"] + st["v_arrays"]:
        y = x.double() if x.is_floating_point() else x.clone()
        y[torch.tensor(target, device="cuda")] = x.to(y.dtype)[torch.tensor(source, device="cuda")]
        out.append(y)
    return out
