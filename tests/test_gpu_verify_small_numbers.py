"""Random numbers at and near 0 in the verification of drafts: a token is taken as by
a number of 2^-60 at least, whatever lies before it, and a row that is a distribution
always gives a token."""
import math

import numpy as np
import pytest
import torch

import spec_ref
from test_gpu_spec import BF, F32, HF, check_verify

pytestmark = pytest.mark.gpu

INF = math.inf
NUMBERS = [0.0, 1e-45, 2.0 ** -100, 2.0 ** -61, 2.0 ** -60, 2.0 ** -55, 2.0 ** -49, 2.0 ** -24, 0.5, 1 - 2.0 ** -24]


@pytest.fixture(autouse=True)
def numbers_of_a_power_at_least(monkeypatch):
    plain = spec_ref.take
    monkeypatch.setattr(spec_ref, "take", lambda w, u: plain(w, max(float(np.float32(u)), 2.0 ** -60)))


def every_form(row, t, dtype, numbers=NUMBERS):
    """The row with each number: as plain sampling, as trees of one node among those for up to 80, and as the end of
    a chain.  Returns the tokens."""
    n = len(numbers)
    x = torch.as_tensor(row).to(dtype).repeat(n, 1)
    starts, kw = list(range(n + 1)), dict(temperature=[t] * n)
    want = check_verify(x, [0] * n, numbers, starts, 1, **kw)[0]
    check_verify(x, [0] * n, numbers, starts, 80, **kw)
    check_verify(x, [0] * n, numbers, starts, 1, draft=x, **kw)
    return [w[0] for w in want]


def row_of(V, values):
    x = torch.full((V,), -INF)
    for at, v in values:
        x[at] = v
    return x


@pytest.mark.parametrize("dtype", [HF, BF, F32])
def test_weights_far_below_the_largest_of_their_chunk(dtype):
    """Weights of 2^-72 of the largest and less, which a sum need not hold, before the token that is taken."""
    x = np.random.default_rng(1).standard_normal(2048) * 2
    x[1500] = 20.0
    assert every_form(torch.from_numpy(x), 0.2, dtype)[0] == 1500
    assert every_form(row_of(2048, [(0, 0.0), (1500, 60.0)]), 1.0, dtype)[0] == 1500
    # 1536 weights of 2^-72.5, 2^-61.9 together, decide whether the one of 2^-60.2 behind them passes 2^-60
    row = row_of(2048, [(slice(0, 1536), -50.25), (1600, -41.75), (2000, 0.0)])
    assert every_form(row, 1.0, dtype)[:2] == [1600, 1600]
    # 2^-70 in the first chunk, 2^-50 in the second, the rest in the fourth
    row = row_of(9001, [(10, -48.5), (3000, -34.75), (7000, 0.0)])
    assert every_form(row, 1.0, dtype) == [3000] * 6 + [7000] * 4


@pytest.mark.parametrize("dtype", [HF, BF, F32])
def test_weights_at_the_end_of_64_bits(dtype):
    """A first chunk whose weights are 2^-1060 to 2^-1080 of the row's largest, at the end of what 64 bits hold."""
    rng = np.random.default_rng(2)
    for t, at in ((0.05, -36.75), (0.05, -37.0), (0.05, -37.25), (0.0625, -46.25), (0.0625, -46.5), (1.0, -740.0), (1.0, -744.0), (1.0, -748.0)):
        for _ in range(8):
            x = torch.full((2 * 2048 + 100,), -INF)
            x[:2048] = torch.from_numpy((at + rng.standard_normal(2048) * (0.4 if t == 1.0 else 0.02)).astype(np.float32))
            x[2048:] = -2.0
            x[3000] = 0.0
            tokens = every_form(x, t, dtype)
            assert min(tokens) >= 2048


@pytest.mark.parametrize("dtype", [HF, BF, F32])
@pytest.mark.parametrize("V", [3, 500, 2048, 2100, 20011])
def test_wide_rows(dtype, V):
    """Logits spread over hundreds of powers of two, some masked."""
    rng = np.random.default_rng(V)
    for spread, t in ((60.0, 1.0), (8.0, 0.1), (3.0, 0.04)):
        x = rng.standard_normal(V) * spread
        x[rng.random(V) < 0.3] = -INF
        x[rng.integers(0, V)] = spread
        every_form(torch.from_numpy(x), t, dtype)


@pytest.mark.parametrize("dtype", [HF, BF, F32])
@pytest.mark.parametrize("n", [4, 20])
def test_what_a_refused_draft_leaves(dtype, n):
    """max(p - q, 0) over wide rows, with small numbers for the token and large ones for the drafts."""
    rng = np.random.default_rng(n)
    B, V = 12, 6001
    starts = [n * b for b in range(B + 1)]
    x = torch.from_numpy(rng.standard_normal((n * B, V)) * 12).to(dtype)
    draft = torch.from_numpy(rng.standard_normal((n * B, V)) * 12).to(dtype)
    u = np.full(n * B, 1 - 2.0 ** -24, np.float32)
    u[starts[:-1]] = (NUMBERS + [0.0, 2.0 ** -30])[:B]
    tokens = rng.integers(0, V, n * B).astype(np.int32)
    likely = draft.double().argmax(-1).numpy()
    for b in range(B):  # refused, as a rule: what the draft likes best
        tokens[starts[b] + 1:starts[b + 1]] = likely[starts[b]:starts[b + 1] - 1]
    check_verify(x, tokens, u, starts, n, draft=draft)
    check_verify(x, tokens, u, starts, n, draft=draft, temperature=[0.3] * B)
