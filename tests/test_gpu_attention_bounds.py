"""Cache attention on the HIP path at the edges of the bounds that its caller
gives: max_context, max_queries and workspaces sized from them."""
import numpy as np
import pytest
import torch

import attn_ref as ref
import w4a16_bit_matmul_amd as wq
from parity import say
from test_gpu_attention import BF, HF, Cache, _cache_want, _check_rows, _run_cache, _tables

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("most", [7, 6, 100])
def test_a_workspace_sized_for_more_queries_than_there_are(most):
    """The bytes that wq_kv_attention_workspace_bytes names for these bounds fit the
    call with the same bounds."""
    lens, nq, Hq, Hkv, D, page, room = [3000, 2100], [4, 2], 8, 2, 128, 32, 4096
    T, starts = 6, [0, 4, 6]
    need = wq.wq_kv_attention_workspace_bytes(T, Hq, Hkv, D, 2, page, room, most)
    assert need > 0
    S = 4096 + 2048
    cache = Cache(most, S, Hkv, D)
    table = _tables(1, lens, page, S, width=room // page)
    q = ref.values(2, (T, Hq, D), BF)
    want, used = _cache_want(cache, q, table, page, lens, starts, D ** -0.5)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    got, lse = _run_cache(cache.to_dev(used), q.cuda(), table, page, lens, starts, max_context=room, max_queries=most, workspace=ws)
    _check_rows(got, lse, want)


@pytest.mark.parametrize("Hq,Hkv,D,nq", [(8, 2, 128, 1), (4, 4, 64, 3), (3, 1, 256, 2), (64, 8, 128, 160)])
def test_no_room_for_any_token(Hq, Hkv, D, nq):
    """A block table without columns, or max_context 0, whatever the lengths: every
    query sees nothing."""
    B = 8
    starts = [nq * b for b in range(B + 1)]
    cache = Cache(D, 16, Hkv, D)
    q = ref.values(3, (B * nq, Hq, D), HF).cuda()
    if nq == 160:
        assert "kv_chunk_kernel" in wq.wq_kv_attention_plan(B * nq, Hq, Hkv, D, B, 16, 0, nq)
    for width, kw in ((0, {}), (3, dict(max_context=0))):
        out, lse = _run_cache(cache.to_dev(), q, np.full((B, width), -1, np.int32), 16, [0, 5] * (B // 2), None if nq == 1 else starts,
                              **kw, **({} if nq == 1 else dict(max_queries=nq)))
        assert bool((out == 0).all()) and bool((lse == -np.inf).all())


@pytest.mark.parametrize("lens,nq,Hq,Hkv,D,page,room,shared", [
    ([700, 300, 90, 1000], [4, 1, 3, 0], 8, 2, 128, 16, 256, False), ([5000, 4100, 3000], [3, 5, 2], 8, 8, 64, 64, 4096, True),
    ([1500, 1024, 1025], [9, 2, 9], 4, 1, 256, 32, 1024, True), ([700], [512], 16, 2, 128, 16, 400, False)])
def test_lengths_past_max_context_count_as_it(lens, nq, Hq, Hkv, D, page, room, shared):
    """A sequence of more tokens than max_context has that many, and its queries are the
    last of those."""
    say(f"lens={lens} past {room}, nq={nq} Hq={Hq} Hkv={Hkv} D={D}")
    starts = [int(x) for x in np.concatenate([[0], np.cumsum(nq)])]
    S = (sum(-(-min(n, room) // page) for n in lens) + 2) * page
    cache = Cache(room + D, S, Hkv, D)
    table = _tables(D, [min(n, room) for n in lens], page, S, width=-(-max(lens) // page))
    q = ref.values(4, (starts[-1], Hq, D), BF)
    plan = wq.wq_kv_attention_plan(starts[-1], Hq, Hkv, D, len(lens), page, room, max(nq))
    assert plan.endswith("shares") == shared, plan
    want, used = _cache_want(cache, q, table, page, lens, starts, D ** -0.5, max_context=room)
    got, lse = _run_cache(cache.to_dev(used), q.cuda(), table, page, lens, starts, max_context=room, max_queries=max(nq))
    _check_rows(got, lse, want)


@pytest.mark.parametrize("T,Hq,Hkv,D,B,page,room,nq", [(1, 8, 1, 128, 1, 64, 9000, 1), (3, 4, 4, 64, 3, 16, 4500, 1), (2, 4, 1, 256, 2, 32, 5000, 1),
                                                      (1, 16, 8, 128, 1, 32, 7000, 1), (6, 8, 2, 128, 2, 16, 4000, 3)])
def test_shared_out_calls_need_their_workspace(T, Hq, Hkv, D, B, page, room, nq):
    """The long contexts of test_gpu_attention.py are shared out, and the call refuses
    less than the bytes named for it."""
    assert wq.wq_kv_attention_plan(T, Hq, Hkv, D, B, page, room, nq).endswith("shares")
    need = wq.wq_kv_attention_workspace_bytes(T, Hq, Hkv, D, B, page, room, nq)
    assert need > 0
    S = -(-room // page) * page
    c = Cache(D, S, Hkv, D).to_dev()
    for x in c:
        x.s.zero_()
    q = torch.zeros((T, Hq, D), dtype=HF, device="cuda")
    table = torch.zeros((B, S // page), dtype=torch.int32, device="cuda")
    lens = torch.full((B,), nq, dtype=torch.int32, device="cuda")
    starts = None if nq == 1 else torch.arange(0, T + 1, nq, dtype=torch.int32, device="cuda")
    call = lambda n: wq.wq_kv_attention(q, *c, table, lens, page_size=page, max_context=room, q_starts=starts, max_queries=nq,
                                        workspace=torch.empty(n, dtype=torch.uint8, device="cuda"))
    with pytest.raises(wq.WQError):
        call(need - 1)
    assert bool((call(need) == 0).all())


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 128), (4, 4, 64), (3, 1, 256)])
def test_one_long_context_among_more_sequences_than_are_shared_out(Hq, Hkv, D):
    """300 sequences of up to 90 tokens and one of 5000: a workgroup walks each, whatever
    the others' lengths."""
    rng = np.random.default_rng(D + 1)
    lens = [int(x) for x in rng.integers(0, 91, 300)]
    lens[117] = 5000
    page, S = 32, 300 * 96 + 5024
    cache = Cache(D + 7, S, Hkv, D)
    table = _tables(D, lens, page, S)
    q = ref.values(Hq, (300, Hq, D), HF)
    assert wq.wq_kv_attention_plan(300, Hq, Hkv, D, 300, page, 5024, 1).endswith("whole units")
    want, used = _cache_want(cache, q, table, page, lens, list(range(301)), D ** -0.5)
    got, lse = _run_cache(cache.to_dev(used), q.cuda(), table, page, lens, None)
    _check_rows(got, lse, want)


@pytest.mark.parametrize("Hq,Hkv,D,B,nq,kernel", [(64, 8, 128, 64, 16, "kv_chunk_kernel<D=128"), (32, 8, 64, 64, 32, "kv_chunk_kernel<D=64"),
                                                 (16, 4, 128, 64, 4, "shares"), (8, 1, 256, 20, 3, "shares")])
def test_short_contexts_under_a_large_max_context(Hq, Hkv, D, B, nq, kernel):
    """Room for a million tokens a sequence and at most 120 in it."""
    rng = np.random.default_rng(B + D)
    lens = [0, 1, nq] + [int(x) for x in rng.integers(0, 121, B - 3)]
    page, room = 16, 2 ** 20
    S = (sum(-(-n // page) for n in lens) + 1) * page
    cache = Cache(D + nq, S, Hkv, D)
    table = _tables(D, lens, page, S, width=room // page)
    starts = [nq * b for b in range(B + 1)]
    q = ref.values(nq, (B * nq, Hq, D), BF)
    assert kernel in wq.wq_kv_attention_plan(B * nq, Hq, Hkv, D, B, page, room, nq)
    want, used = _cache_want(cache, q, table, page, lens, starts, D ** -0.5)
    got, lse = _run_cache(cache.to_dev(used), q.cuda(), table, page, lens, starts, max_queries=nq)
    _check_rows(got, lse, want)
