"""The largest calls of a speculative decoding step (host only): a grid holds less than
2^32 threads, which the checks count before anything is enqueued."""
import w4a16_bit_matmul_amd as wq
from test_spec_cpu import A, A2, EUNSUP, append, verify

MOST = 2 ** 26 - 4  # waves of 64 threads, four a workgroup


def test_append_counts_the_last_workgroup():
    keys = dict(q=None, qo=None, starts=A)  # two waves a token
    assert append(T=2 ** 25 - 1, **keys) == EUNSUP
    assert append(T=MOST // 2 + 1, **keys) == EUNSUP
    assert append(T=MOST // 4 + 1, starts=A) == EUNSUP  # and two for its eight heads of q


def test_verify_counts_the_last_workgroup():
    most = lambda T, V, drafts=False: wq.wq_verify_drafts_workspace_bytes(T, V, 1, drafts=drafts)  # noqa: E731
    for V, chunks in ((1, 1), (2048, 1), (2049, 2), (4096, 2), (5000, 3), (6144, 3), (131072, 64)):
        for drafts in (False, True):
            T = MOST // chunks // (1 + drafts)
            assert most(T, V, drafts) > 0 and most(T + 1, V, drafts) == 0, (V, drafts)
    for T in (2 ** 26 - 1, 2 ** 26 - 3):
        assert verify(T=T) == EUNSUP
    assert verify(T=2 ** 25 - 1, V=4096, stride=4096) == EUNSUP
    assert verify(T=2 ** 25 - 1, draft=A2, ds=1000, parents=None) == EUNSUP
