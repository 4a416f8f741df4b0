"""The largest calls of a speculative decoding step on the HIP path."""
import numpy as np
import pytest
import torch

import w4a16_bit_matmul_amd as wq
from test_gpu_spec import HF, i32, tree_inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("most", [16, 20])
def test_verify_of_millions_of_sequences(most):
    """Three trees among 2^22 sequences, all others empty: the answers of the three alone."""
    B, at = 2 ** 22 + 3, [0, 777_777, 2 ** 22 + 2]
    x, tokens, u, starts, parents, temp = tree_inputs(4, [9, 16, 12], 300, HF)
    args = [x.cuda(), i32(tokens), torch.from_numpy(u).cuda()]
    want = wq.wq_verify_drafts(*args, q_starts=i32(starts), max_queries=most, parents=i32(parents), temperature=torch.from_numpy(temp).cuda())
    n, t = np.zeros(B, np.int64), np.ones(B, np.float32)
    n[at], t[at] = np.diff(starts), temp
    many = i32(np.concatenate([[0], np.cumsum(n)]))
    got = wq.wq_verify_drafts(*args, q_starts=many, max_queries=most, parents=i32(parents), temperature=torch.from_numpy(t).cuda())
    torch.cuda.synchronize()
    assert min(want[2].tolist()) >= 1 and max(want[2].tolist()) > 1
    for g, w, nothing in zip(got, want, (-1, -1, 0)):
        assert torch.equal(g[at], w)
        rest = torch.ones(B, dtype=torch.bool, device="cuda")
        rest[at] = False
        assert bool((g[rest] == nothing).all())
