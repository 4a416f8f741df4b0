"""Argument checks of the operators of a speculative decoding step (host only:
every refusal happens before anything is enqueued), and their plain forms."""
import ctypes

import numpy as np
import pytest
import torch

import spec_ref
import w4a16_bit_matmul_amd as wq

P = ctypes.c_void_p
A, A2, B = P(0x10000), P(0x20000), P(0x10002)  # placeholder addresses, never dereferenced
ODD = P(0x10001)
OK, EINVAL, EUNSUP, EALIGN, EWS = wq.WQ_OK, wq.WQ_EINVAL, wq.WQ_EUNSUPPORTED, wq.WQ_EALIGN, wq.WQ_EWORKSPACE
BF, HF, F32 = wq.WQ_BF16, wq.WQ_F16, wq.WQ_F32


def append(**kw):
    a = dict(q=A, k=A, v=A, dtype=BF, T=2, Hq=8, Hkv=2, D=128, qs=1024, ks=256, vs=256, norm=0, qw=None, kw=None, eps=1e-6, pos=None,
             cos=A, sin=A, P=16, rot=128, inter=0, kc=A, ksc=A, kz=A, vc=A, vsc=A, vz=A, S=4096, nseq=2, table=A, width=64, page=16,
             lens=A, starts=None, qo=A2, ko=None, qos=1024, kos=256, stream=None)
    a.update(kw)
    return wq.lib().wq_kv_append(*a.values())


def tree(**kw):
    a = dict(q=A, dtype=BF, T=2, Hq=8, Hkv=2, D=128, qs=1024, kc=A, ks=A, kz=A, vc=A, vs=A, vz=A, S=4096, nseq=2, table=A, width=64,
             page=16, lens=A, max_context=1024, starts=None, max_queries=1, mask=A, words=1, scale=0.1, out=A2, lse=None, ws=A,
             wsb=1 << 20, stream=None)
    a.update(kw)
    return wq.lib().wq_kv_tree_attention(*a.values())


def verify(**kw):
    a = dict(logits=A, dtype=HF, T=4, V=1000, stride=1000, draft=None, ds=0, nseq=2, starts=A, most=4, tokens=A, parents=A, u=A, temp=A,
             out=A2, path=A2, counts=A2, ws=A, wsb=1 << 20, stream=None)
    a.update(kw)
    return wq.lib().wq_verify_drafts(*a.values())


def keep(**kw):
    a = dict(kc=A, ks=A, kz=A, vc=A, vs=A, vz=A, S=4096, hd=1024, T=8, nseq=2, table=A, width=64, page=16, lens=A, starts=A, path=A, pw=4,
             counts=A, stream=None)
    a.update(kw)
    return wq.lib().wq_kv_keep(*a.values())


def test_nothing_to_do_is_no_error():
    assert append(T=0, nseq=0) == append(T=3, nseq=0, starts=A) == append(T=0, nseq=0, k=None) == OK
    assert tree(T=0, nseq=0, max_queries=0, mask=None) == tree(T=3, starts=A, max_queries=0) == OK
    assert verify(T=0, nseq=0, starts=None) == verify(nseq=0, out=None) == OK
    assert keep(T=0) == keep(nseq=0) == keep(pw=0) == OK


@pytest.mark.parametrize("call", [append, tree])
def test_heads_and_types(call):
    assert call(dtype=F32) == call(dtype=7) == call(T=-1) == call(Hq=0) == call(Hkv=-2) == EINVAL
    assert call(D=96) == call(Hq=7) == call(Hkv=1, Hq=8, D=64, qs=512) == EUNSUP
    assert call(qs=1016) == call(qs=2 ** 23) == EINVAL and call(qs=1028) == EALIGN


@pytest.mark.parametrize("call", [append, tree, keep])
def test_pages(call):
    assert call(page=0) == call(page=24) == call(page=-16) == call(page=8192) == EUNSUP
    assert call(S=0) == call(S=2 ** 31) == call(width=-1) == call(nseq=-1) == call(nseq=2 ** 24 + 1) == EINVAL
    assert call(T=3, starts=None) == EINVAL  # one token a sequence unless starts says otherwise
    assert call(table=None) == call(lens=None) == EINVAL and call(table=B) == call(lens=B) == call(starts=B) == EALIGN
    for name in ("kc", "kz", "vc", "vz"):
        assert call(**{name: None}) == EINVAL, name
    assert call(kc=B) == call(vc=B) == EALIGN


def test_append_refusals():
    for name in ("k", "v", "cos", "sin", "ksc", "vsc"):
        assert append(**{name: None}) == EINVAL, name
    for name in ("q", "k", "v", "cos", "sin", "qo", "ko", "pos", "qw", "kw"):
        assert append(**{name: B}) == EALIGN, name
    assert append(qw=P(0x10008)) == append(ksc=ODD) == append(vsc=ODD) == EALIGN
    assert append(q=None) == append(qo=None) == EINVAL  # both, or neither
    assert append(norm=2) == append(inter=2) == append(P=0) == append(eps=-1.0) == append(eps=float("nan")) == EINVAL
    assert append(rot=0) == append(rot=24) == append(rot=144) == EUNSUP
    assert append(ks=248) == append(vs=255) == append(qos=1016) == append(ko=A2, kos=248) == EINVAL
    assert append(vs=260) == append(ko=A2, kos=260) == EALIGN
    assert append(T=2 ** 26, starts=A) == append(T=2 ** 25, Hq=64, qs=8192, qos=8192, starts=A) == EUNSUP  # workgroups


def test_tree_refusals():
    assert tree(mask=None) == tree(words=0) == tree(words=65537) == EINVAL and tree(mask=P(0x10004)) == EALIGN
    assert tree(T=80, starts=A, max_queries=65, nseq=1) == EINVAL  # more nodes than the mask has bits
    assert tree(max_context=64 * 16 + 1) == tree(max_queries=2) == tree(scale=0.0) == tree(out=None) == EINVAL
    need = wq.wq_kv_tree_attention_workspace_bytes(2, 8, 2, 128, 2, 16, 65536)
    long = dict(S=1 << 20, width=4096, max_context=65536)
    assert need > 0 and tree(**long, ws=None) == tree(**long, wsb=need - 1) == EWS and tree(**long, ws=B, wsb=need) == EALIGN
    assert wq.wq_kv_tree_attention_plan(2, 8, 2, 128, 2, 16, 65536) == wq.wq_kv_attention_plan(2, 8, 2, 128, 2, 16, 65536) + ", tree masks"
    assert wq.lib().wq_kv_tree_attention_plan(2, 8, 2, 96, 2, 16, 1024, 1, ctypes.create_string_buffer(64), 64) == EUNSUP


def test_verify_refusals():
    for name in ("logits", "tokens", "u", "out", "path", "counts"):
        assert verify(**{name: None}) == EINVAL, name
    for name in ("starts", "tokens", "parents", "u", "temp", "out", "path", "counts"):
        assert verify(**{name: B}) == EALIGN, name
    assert verify(logits=ODD) == verify(dtype=F32, logits=B) == verify(dtype=BF, draft=ODD, ds=1000, parents=None) == EALIGN
    assert verify(dtype=5) == verify(T=-1) == verify(V=0) == verify(stride=999) == verify(most=0) == verify(nseq=-1) == EINVAL
    assert verify(draft=A, ds=999, parents=None) == verify(starts=None) == EINVAL
    assert verify(draft=A, ds=1000) == verify(most=1025) == verify(V=2 ** 24 + 1, stride=2 ** 25) == EUNSUP
    assert verify(T=2 ** 26) == verify(T=2 ** 25, draft=A, ds=1000, parents=None) == verify(T=2 ** 20, V=2 ** 18, stride=2 ** 18) == EUNSUP
    need = wq.wq_verify_drafts_workspace_bytes(4, 1000, 2)
    both = wq.wq_verify_drafts_workspace_bytes(4, 1000, 2, drafts=True)
    assert 0 < need < both
    assert verify(ws=None) == verify(wsb=need - 1) == verify(draft=A, ds=1000, parents=None, wsb=both - 1) == EWS and verify(ws=B) == EALIGN
    assert wq.wq_verify_drafts_workspace_bytes(0, 1000, 2) == wq.wq_verify_drafts_workspace_bytes(4, 0, 2) == 0
    assert wq.wq_verify_drafts_workspace_bytes(2 ** 25, 1000, 2, drafts=True) == 0


def test_keep_refusals():
    assert keep(path=None) == keep(counts=None) == EINVAL and keep(path=B) == keep(counts=B) == EALIGN
    assert keep(hd=0) == keep(hd=2 ** 23 + 128) == keep(pw=-1) == EINVAL and keep(hd=1000) == EUNSUP
    assert keep(nseq=2 ** 23) == EUNSUP


def test_binding_rejects_before_any_call():
    x = torch.zeros((2, 4, 128), dtype=torch.float16)
    k = x[:, :2]
    i = torch.zeros(2, dtype=torch.int32)
    tb, cs = torch.zeros((2, 4), dtype=torch.int32), torch.zeros((5, 64))
    c = wq.KVCache(torch.zeros((16, 128), dtype=torch.uint8), torch.zeros((16, 2), dtype=torch.float16),
                   torch.zeros((16, 1), dtype=torch.uint8), 16, 256)
    bad = wq.KVCache(c.codes, c.s.float(), c.zpacked, 16, 256)
    for m, a, kw in [("on the GPU", (k, k, c, c, tb, i, cs, cs), dict(q=x)), ("caches", (x, x, c, c, tb, i, cs, cs), {}),
                     ("heads", (k, x, c, c, tb, i, cs, cs), {}), ("k_cache.s", (k, k, bad, c, tb, i, cs, cs), {}),
                     ("block_table", (k, k, c, c, tb[0], i, cs, cs), {}), ("context_lens", (k, k, c, c, tb, i[:1], cs, cs), {}),
                     ("sin", (k, k, c, c, tb, i, cs, cs[:4]), {}), ("norm=True", (k, k, c, c, tb, i, cs, cs), dict(k_weight=cs[0])),
                     ("k_weight", (k, k, c, c, tb, i, cs, cs), dict(norm=True, k_weight=cs[0])), ("tokens", (k, k[:1], c, c, tb, i, cs, cs), {}),
                     ("q_out", (k, k, c, c, tb, i, cs, cs), dict(q_out=x)), ("k_out", (k, k, c, c, tb, i, cs, cs), dict(k_out=x)),
                     ("positions", (k, k, c, c, tb, i, cs, cs), dict(positions=i.long())),
                     ("q_starts", (k, k, c, c, tb, i, cs, cs), dict(q_starts=i))]:
        with pytest.raises(ValueError, match=m):
            wq.wq_kv_append(*a, page_size=4, **kw)
    mask = torch.zeros((2, 1), dtype=torch.int64)
    with pytest.raises(ValueError, match="tree_mask"):
        wq.wq_kv_tree_attention(x, c, c, tb, i, mask[:1], page_size=4)
    with pytest.raises(ValueError, match="tree_mask"):
        wq.wq_kv_tree_attention(x, c, c, tb, i, mask.int(), page_size=4)
    with pytest.raises(ValueError, match="words"):
        wq.wq_kv_tree_attention(x, c, c, tb, i, mask[0], page_size=4)
    with pytest.raises(ValueError, match="on the GPU"):
        wq.wq_kv_tree_attention(x, c, c, tb, i, mask, page_size=4)
    l, u = torch.zeros((2, 9)), torch.zeros(2)
    for m, a, kw in [("on the GPU", (l, i, u), {}), ("float32", (l.double(), i, u), {}), ("contiguous rows", (l.t(), i, u), {}),
                     ("tokens", (l, i.long(), u), {}), ("uniform", (l, i, u[:1]), {}), ("parents", (l, i, u), dict(parents=u)),
                     ("draft_logits", (l, i, u), dict(draft_logits=l[:, :5])), ("draft_logits", (l, i, u), dict(draft_logits=l.half())),
                     ("temperature", (l, i, u), dict(temperature=u[:1])), ("q_starts", (l, i, u), dict(q_starts=i[:0])),
                     ("out_tokens", (l, i, u), dict(out_tokens=i)), ("counts", (l, i, u), dict(counts=i[:1])),
                     ("workspace", (l, i, u), dict(workspace=torch.empty(8, device="meta")))]:
        with pytest.raises(ValueError, match=m):
            wq.wq_verify_drafts(*a, **kw)
    with pytest.raises(ValueError, match="path"):
        wq.wq_kv_keep(c, c, tb, i, i, i, page_size=4, q_starts=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="q_starts"):
        wq.wq_kv_keep(c, c, tb, i, tb, i, page_size=4, q_starts=i)
    with pytest.raises(ValueError, match="on the GPU"):
        wq.wq_kv_keep(c, c, tb, i, tb, i, page_size=4, q_starts=torch.zeros(3, dtype=torch.int32))


def test_the_plain_chain_has_the_targets_law():
    """Over all drafts and tests together the first new token has the target's
    probabilities: for every token sum over drafts x of q(x) [accepted as it, or
    refused and taken from the rest] = p, by a grid of random numbers."""
    p, q = np.array([0.1, 0.6, 0.3]), np.array([0.5, 0.25, 0.25])
    N = 1000
    hits = np.zeros(3)
    grid = (np.arange(N) + 0.5) / N
    for x in range(3):
        yes = (grid * q[x] < p[x]).mean()
        hits[x] += q[x] * yes
        left = np.maximum(p - q, 0)
        got = np.array([spec_ref.take(left, u) for u in grid])
        for y in range(3):
            hits[y] += q[x] * (1 - yes) * (got == y).mean()
    assert np.abs(hits - p).max() <= 2 / N  # a step of the grid in each of two factors


def test_binding_takes_tensors_and_sizes_of_32_bits():
    x = torch.zeros((2, 2, 128), dtype=torch.float16)
    i = torch.zeros(2, dtype=torch.int32)
    tb, cs, mask = torch.zeros((2, 4), dtype=torch.int32), torch.zeros((5, 64)), torch.zeros((2, 1), dtype=torch.int64)
    c = wq.KVCache(torch.zeros((16, 128), dtype=torch.uint8), torch.zeros((16, 2), dtype=torch.float16),
                   torch.zeros((16, 1), dtype=torch.uint8), 16, 256)
    starts = torch.zeros(3, dtype=torch.int32)
    for page in (2 ** 31, -2 ** 31 - 1, 2 ** 32 + 4):
        for call in (lambda: wq.wq_kv_append(x, x, c, c, tb, i, cs, cs, page_size=page),
                     lambda: wq.wq_kv_tree_attention(x, c, c, tb, i, mask, page_size=page),
                     lambda: wq.wq_kv_keep(c, c, tb, i, tb, i, page_size=page, q_starts=starts)):
            with pytest.raises(ValueError, match="page_size"):
                call()
    for page in (4.0, None, "4"):
        with pytest.raises(TypeError):
            wq.wq_kv_append(x, x, c, c, tb, i, cs, cs, page_size=page)
    with pytest.raises(TypeError, match="context_lens must be a tensor"):
        wq.wq_kv_append(x, x, c, c, tb, [1, 2], cs, cs, page_size=4)
    with pytest.raises(TypeError, match="tree_mask must be a tensor"):
        wq.wq_kv_tree_attention(x, c, c, tb, i, None, page_size=4)
    with pytest.raises(TypeError, match="uniform must be a tensor"):
        wq.wq_verify_drafts(cs[:2], i, 0.5)
    with pytest.raises(TypeError):
        wq.wq_verify_drafts(cs[:2], i, cs[:2, 0].contiguous(), max_queries="1")
    with pytest.raises(TypeError, match="counts must be a tensor"):
        wq.wq_kv_keep(c, c, tb, i, tb, None, page_size=4, q_starts=starts)
    with pytest.raises(ValueError, match=r"positions must be a contiguous torch.int32 tensor of shape \(2,\) on cpu "
                                         r"\(got torch.int64, shape \(2,\), on cpu\)"):
        wq.wq_kv_append(x, x, c, c, tb, i, cs, cs, page_size=4, positions=i.long())
