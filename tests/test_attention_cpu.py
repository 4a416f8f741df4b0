"""Argument checks of the attention-side operators (host only: every refusal
happens before anything is enqueued) and the plans of the cache attention."""
import ctypes
import re

import pytest
import torch

import w4a16_bit_matmul_amd as wq

P = ctypes.c_void_p
A, A2, B = P(0x10000), P(0x20000), P(0x10002)  # placeholder addresses, never dereferenced
EINVAL, EUNSUP, EALIGN, EWS = wq.WQ_EINVAL, wq.WQ_EUNSUPPORTED, wq.WQ_EALIGN, wq.WQ_EWORKSPACE
BF, HF = wq.WQ_BF16, wq.WQ_F16


def rope(**kw):
    a = dict(q=A, k=A, dtype=BF, T=4, Hq=8, Hkv=2, D=128, qs=1024, ks=256, qw=A, kw=A, eps=1e-6, pos=A, cos=A, sin=A, P=16, rot=128,
             inter=0, qo=A2, ko=A2, qos=1024, kos=256, stream=None)
    a.update(kw)
    return wq.lib().wq_qk_norm_rope(*a.values())


def prompt(**kw):
    a = dict(q=A, k=A, v=A, dtype=BF, T=4, Hq=8, Hkv=2, D=128, qs=1024, ks=256, vs=256, nseq=1, starts=A, scale=0.1, out=A2, lse=None,
             stream=None)
    a.update(kw)
    return wq.lib().wq_prompt_attention(*a.values())


def cache(**kw):
    a = dict(q=A, dtype=BF, T=2, Hq=8, Hkv=2, D=128, qs=1024, kc=A, ks=A, kz=A, vc=A, vs=A, vz=A, S=4096, nseq=2, table=A, width=64,
             page=16, lens=A, max_context=1024, starts=None, max_queries=1, scale=0.1, out=A2, lse=None, ws=None, wsb=0, stream=None)
    a.update(kw)
    return wq.lib().wq_kv_attention(*a.values())


def test_nothing_to_do_is_no_error():
    assert rope(T=0) == rope(T=0, q=None) == wq.WQ_OK
    assert prompt(T=0) == prompt(nseq=0) == wq.WQ_OK
    assert cache(T=0, nseq=0, max_queries=0) == wq.WQ_OK
    assert cache(T=3, starts=A, max_queries=0) == cache(T=3, nseq=0, starts=A, max_queries=3) == wq.WQ_OK


@pytest.mark.parametrize("call", [rope, prompt, cache])
def test_heads_and_types(call):
    assert call(dtype=wq.WQ_F32) == call(dtype=7) == EINVAL
    assert call(T=-1) == call(Hq=0) == call(Hkv=0) == call(Hkv=-2) == EINVAL
    assert call(D=96) == call(D=512) == call(Hq=7) == EUNSUP
    assert call(qs=1016) == EINVAL and call(qs=1028) == EALIGN
    assert call(q=None) == EINVAL and call(q=B) == EALIGN


def test_norm_rope_refusals():
    for name in ("q", "k", "pos", "cos", "sin", "qo", "ko"):
        assert rope(**{name: None}) == EINVAL, name
        assert rope(**{name: B}) == (EALIGN), name
    assert rope(qw=P(0x10004)) == rope(kw=P(0x10004)) == EALIGN
    assert rope(eps=-1e-6) == rope(eps=float("nan")) == rope(eps=float("inf")) == EINVAL
    assert rope(P=0) == rope(inter=2) == EINVAL
    assert rope(rot=0) == rope(rot=8) == rope(rot=24) == rope(rot=144) == EUNSUP
    assert rope(ks=255) == rope(qos=8) == rope(kos=248) == EINVAL
    assert rope(ks=260) == rope(qos=1025) == EALIGN


def test_prompt_refusals():
    for name in ("q", "k", "v", "starts", "out"):
        assert prompt(**{name: None}) == EINVAL, name
        assert prompt(**{name: B}) == EALIGN, name
    assert prompt(lse=B) == EALIGN
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert prompt(scale=s) == cache(scale=s) == EINVAL
    assert prompt(nseq=-1) == prompt(ks=248) == EINVAL and prompt(vs=257) == EALIGN
    assert prompt(T=2 ** 31 - 1, Hq=4096, qs=4096 * 128, Hkv=1024, ks=1024 * 128, vs=1024 * 128) == EUNSUP


def test_cache_refusals():
    for name in ("q", "kc", "ks", "kz", "vc", "vs", "vz", "table", "lens", "out"):
        assert cache(**{name: None}) == EINVAL, name
    for name in ("q", "kc", "vc", "table", "lens", "out", "lse"):
        assert cache(**{name: B}) == EALIGN, name
    assert cache(ks=P(0x10001)) == cache(vs=P(0x10001)) == EALIGN
    assert cache(page=0) == cache(page=24) == cache(page=-16) == cache(page=8192) == EUNSUP
    assert cache(Hkv=1, Hq=8, D=64, qs=512) == EUNSUP  # a cache row is whole blocks of 128 values
    assert cache(S=0) == cache(max_context=64 * 16 + 1) == cache(width=-1) == cache(nseq=-1) == EINVAL
    # one query per sequence unless q_starts says otherwise
    assert cache(T=3) == cache(max_queries=0) == cache(max_queries=2) == cache(T=2, starts=A, max_queries=3) == EINVAL
    need = wq.wq_kv_attention_workspace_bytes(2, 8, 2, 128, 2, 16, 65536)
    long = dict(S=1 << 20, width=4096, max_context=65536)
    assert need > 0
    assert cache(**long) == cache(**long, ws=A, wsb=need - 1) == cache(**long, ws=None, wsb=need) == EWS
    assert cache(**long, ws=B, wsb=need) == EALIGN
    assert wq.wq_kv_attention_workspace_bytes(2, 8, 2, 100, 2, 16, 65536) == 0
    assert wq.wq_kv_attention_workspace_bytes(0, 8, 2, 128, 0, 16, 65536, 0) == 0
    buf = ctypes.create_string_buffer(64)
    f = wq.lib().wq_kv_attention_plan
    assert f(2, 8, 2, 128, 2, 16, 1024, 1, None, 64) == f(-1, 8, 2, 128, 2, 16, 1024, 1, buf, 64) == EINVAL
    assert f(2, 8, 2, 96, 2, 16, 1024, 1, buf, 64) == EUNSUP


def test_cache_plans_and_their_workspace():
    """Long contexts of few sequences and heads are shared out equally (with a
    workspace for the results of the units that several workgroups hold); many,
    or short ones, are a workgroup each."""
    for T, Hq, Hkv, D, nb, page, ctx, nq, shared in [
            (1, 64, 8, 128, 1, 16, 1, 1, False), (1, 64, 8, 128, 1, 16, 200, 1, False), (64, 64, 8, 128, 64, 64, 8192, 1, True),
            (1, 8, 1, 256, 1, 256, 131072, 1, True), (16, 8, 8, 64, 4, 8, 5000, 4, True), (512, 64, 8, 128, 1, 64, 16384, 512, False),
            (1, 6, 3, 256, 1, 1, 10 ** 6, 1, True), (600, 8, 8, 128, 600, 16, 8192, 1, False), (257, 1, 1, 128, 257, 16, 65536, 1, False)]:
        d = wq.wq_kv_attention_plan(T, Hq, Hkv, D, nb, page, ctx, nq)
        grid, heads, rt = (int(re.search(n + r"=(\d+)", d).group(1)) for n in ("grid", "HP", "RT"))
        rows = nq * Hq // Hkv
        assert Hkv % heads == 0 and heads * D in (128, 256), d
        units = nb * (Hkv // heads) * (-(-rows // (16 * rt)))
        need = wq.wq_kv_attention_workspace_bytes(T, Hq, Hkv, D, nb, page, ctx, nq)
        assert (d.split()[-1] == "shares") == shared == (need > 0), d
        assert grid <= 512 if shared else grid == units, d
        assert need == (2 * grid * heads * min(rows, 16 * rt) * (D + 2) * 4 if shared else 0), d


def test_shares_are_counted_in_32_bits():
    """Steps of 128 tokens of all units together: past 2^31 each unit is a
    workgroup again."""
    below = wq.wq_kv_attention_plan(1, 508, 254, 128, 1, 4096, 2 ** 30, 1)  # 127 units of 2^23 steps
    at = wq.wq_kv_attention_plan(1, 512, 512, 128, 1, 4096, 2 ** 30, 1)  # 256 units
    assert "HP=2" in below and "grid=512" in below and below.endswith("shares")
    assert "HP=2" in at and "grid=256" in at and at.endswith("whole units")
    assert wq.wq_kv_attention_workspace_bytes(1, 512, 512, 128, 1, 4096, 2 ** 30) == 0


def test_limits_of_the_cache_attention():
    plan = lambda *a: wq.lib().wq_kv_attention_plan(*a, ctypes.create_string_buffer(160), 160)
    assert plan(1, 8, 2, 128, 1, 16, 2 ** 30, 1) == wq.WQ_OK and plan(1, 8, 2, 128, 1, 16, 2 ** 30 + 1, 1) == EINVAL
    assert plan(2 ** 24 + 1, 8, 2, 128, 2 ** 24 + 1, 16, 64, 1) == EINVAL
    # a grid holds 2^24 workgroups less one
    assert plan(2 ** 23 - 1, 8, 2, 128, 2 ** 23 - 1, 16, 64, 1) == wq.WQ_OK and plan(2 ** 23, 8, 2, 128, 2 ** 23, 16, 64, 1) == EUNSUP
    assert cache(T=2 ** 23, nseq=2 ** 23) == EUNSUP
    assert plan(2 ** 31 - 1, 65536, 1, 128, 2 ** 24, 16, 64, 2 ** 31 - 1) == EUNSUP
    assert prompt(T=2 ** 28, Hq=8, Hkv=8, qs=1024, ks=1024, vs=1024) == prompt(nseq=2 ** 23) == EUNSUP
    assert rope(T=2 ** 28) == rope(T=2 ** 26, Hq=64, Hkv=8, qs=8192, ks=1024, qos=8192, kos=1024) == EUNSUP
    # strides (in values) from 2^23 on
    assert prompt(ks=2 ** 23) == prompt(qs=2 ** 23) == cache(qs=2 ** 23) == rope(kos=2 ** 23) == EINVAL


def test_binding_rejects_before_any_call():
    x = torch.zeros((2, 4, 128), dtype=torch.float16)
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="bfloat16 or float16"):
        wq.wq_prompt_attention(x.float(), x, x, i)
    with pytest.raises(ValueError, match="contiguous"):
        wq.wq_prompt_attention(x.transpose(0, 1), x, x, i)
    with pytest.raises(ValueError, match="tokens"):
        wq.wq_prompt_attention(x, x[:1], x, i)
    with pytest.raises(ValueError, match="expected"):
        wq.wq_prompt_attention(x, x.bfloat16(), x, i)
    with pytest.raises(ValueError, match="heads"):
        wq.wq_prompt_attention(x, x, x[:, :2], i)
    with pytest.raises(ValueError, match="seq_starts"):
        wq.wq_prompt_attention(x, x, x, i.long())
    with pytest.raises(ValueError, match="on the GPU"):
        wq.wq_prompt_attention(x, x, x, i)
    t = torch.zeros((5, 64))
    with pytest.raises(ValueError, match="positions"):
        wq.wq_qk_norm_rope(x, x, t, t, i)
    with pytest.raises(ValueError, match="sin"):
        wq.wq_qk_norm_rope(x, x, t, t[:4], i[:2])
    with pytest.raises(ValueError, match="q_weight"):
        wq.wq_qk_norm_rope(x, x, t, t, i[:2], q_weight=t[0])
    c = wq.KVCache(torch.zeros((16, 128), dtype=torch.uint8), torch.zeros((16, 2), dtype=torch.float16),
                   torch.zeros((16, 1), dtype=torch.uint8), 16, 256)
    bad = wq.KVCache(c.codes, c.s.float(), c.zpacked, 16, 256)
    tb = torch.zeros((2, 4), dtype=torch.int32)
    with pytest.raises(ValueError, match="v_cache.s"):
        wq.wq_kv_attention(x, c, bad, tb, i[:2], page_size=4)
    with pytest.raises(ValueError, match="block_table"):
        wq.wq_kv_attention(x, c, c, tb[0], i[:2], page_size=4)
    with pytest.raises(ValueError, match="context_lens"):
        wq.wq_kv_attention(x, c, c, tb, i, page_size=4)
    with pytest.raises(ValueError, match="caches"):
        wq.wq_kv_attention(torch.zeros((2, 4, 100), dtype=torch.float16), c, c, tb, i[:2], page_size=4)
    for ws in (torch.empty(1 << 20, dtype=torch.uint8, device="meta"), torch.empty((1 << 10, 2), dtype=torch.uint8)[:, 0]):
        with pytest.raises(ValueError, match="workspace"):
            wq.wq_kv_attention(x, c, c, tb, i[:2], page_size=4, workspace=ws)
    with pytest.raises(ValueError, match="q_starts"):
        wq.wq_kv_attention(x, c, c, tb, i[:2], page_size=4, q_starts=i[:2])
