"""Cache scales that are infinite or NaN in the attention of draft trees, K's as V's:
every row that sees such a token is infinite or NaN in all of its values, and no other
row is touched."""
import math

import pytest
import torch

import attn_ref as ref
import spec_ref
import w4a16_bit_matmul_amd as wq
from test_gpu_attention import Cache, _check_rows, _tables
from test_gpu_spec import BF, HF, NAN, run_tree, tree_want

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq,Hkv,D,nodes,room,plan", [
    (8, 8, 64, 4, 2 ** 20, "HP=4, RT=1, PK=4"), (8, 8, 64, 4, 1200, "HP=2, RT=1, PK=2"), (64, 8, 128, 2, 2 ** 20, "HP=2, RT=1, PK=1"),
    (64, 8, 128, 2, 1200, "HP=1, RT=1, PK=1"), (24, 8, 128, 7, 2 ** 20, "RT=2"), (48, 8, 64, 4, 1200, "HP=2, RT=1, PK=1"),
    (4, 1, 256, 30, 1200, "kv_attn_kernel<D=256"), (64, 8, 128, 8, 2 ** 20, "D=128, RG=2"), (64, 8, 128, 16, 2 ** 20, "D=128, RG=4"),
    (16, 8, 64, 20, 1200, "D=64, RG=2"), (28, 2, 64, 25, 1200, "D=64, RG=4")])
@pytest.mark.parametrize("bad", [NAN, math.inf, -math.inf])
@pytest.mark.parametrize("page", [16, 64])
def test_rows_that_see_a_bad_scale_show_it(Hq, Hkv, D, nodes, room, plan, bad, page):
    """One node of a branch, and in one sequence a token before the nodes, with a bad scale of K alone, V alone or both
    in the last cache block of every head."""
    B, dtype = 6, HF if page == 16 else BF
    lens = [nodes + x for x in (0, 3, 50, 200, 331, 1000)]
    starts = [nodes * b for b in range(B + 1)]
    S = (sum(-(-n // page) for n in lens) + 2) * page
    cache = Cache(D + nodes, S, Hkv, D)
    table = _tables(B, lens, page, S, width=room // page)
    q = ref.values(Hq, (starts[-1], Hq, D), dtype)
    # node i sees the root and the nodes of its parity; node 1 is bad
    tree = [{j for j in range(i + 1) if j == 0 or j % 2 == i % 2} for i in range(nodes)]
    mask = torch.cat([spec_ref.mask_words(tree, 1)] * B)
    assert plan in wq.wq_kv_tree_attention_plan(q.shape[0], Hq, Hkv, D, B, page, room // page * page, nodes)
    want, used = tree_want(cache, q, table, page, lens, starts, [tree] * B, D ** -0.5)
    hit = torch.tensor([1 in s for s in tree] * B)
    hit[starts[5]:] = True  # by a token before the nodes
    for which in ((0,), (1,), (0, 1)):
        dev = cache.to_dev(used)
        for b in range(B):
            for at in [lens[b] - nodes + 1] + ([700] if b == 5 else []):
                for c in which:
                    rows = dev[c].s[int(table[b][at // page]) * page + at % page]
                    rows[(1 if D == 256 else 0)::(2 if D == 256 else 1)] = bad
        got, lse = run_tree(dev, q.cuda(), table, page, lens, starts, mask)
        seen = got.cpu()[hit]
        if D == 256 and 0 not in which:  # V's scale of a block reaches its own 128 values
            seen = seen[..., 128:]
        assert not bool(torch.isfinite(seen).any()), f"{int(torch.isfinite(seen).sum())} of {seen.numel()} values hide it"
        got[hit.cuda()], lse[hit.cuda()] = 7.0, 7.0
        none = want[4] | hit[:, None]
        _check_rows(got, lse, tuple(x.masked_fill(hit.view(-1, *[1] * (x.dim() - 1)), NAN) for x in want[:4]) + (none,))
