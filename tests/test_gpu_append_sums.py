"""The head norm's sum of squares in appending, where its order shows: 64-bit sums of
eight neighbouring values in order, then of neighbours, pair by pair."""
import numpy as np
import pytest
import torch

import oracle
import w4a16_bit_matmul_amd as wq
from test_gpu_spec import ODT, HF, bits, filled_cache, host_of, i32, same_cache

pytestmark = pytest.mark.gpu


def f32(x):
    return x.astype(np.float32).astype(np.float64)


def in_order(sq):
    s = np.zeros(sq.shape[:-1] + (sq.shape[-1] // 8,))
    for i in range(8):
        s = s + sq[..., i::8]
    while s.shape[-1] > 1:
        s = s[..., 0::2] + s[..., 1::2]
    return s[..., 0]


def one_by_one(sq):
    s = np.zeros(sq.shape[:-1])
    for i in range(sq.shape[-1]):
        s = s + sq[..., i]
    return s


def normed(x, w, eps, add):
    """x [T][H][D] times its norm and w, rounded to fp16, every step one fp32 operation."""
    mean = f32(add(x * x) / x.shape[-1])
    r = f32(1.0 / f32(np.sqrt(f32(mean + np.float64(np.float32(eps))))))
    return f32(f32(x * r[..., None]) * w).astype(np.float16)


def telling_pairs(D):
    """(x, w): the rounded r w tells r of a sum of x^2 + 1000^2 from r of the next fp32 number's."""
    x = 4.0 * (1024 + np.arange(390))  # the sum is a multiple of 16 in [2^24, 2^25), whose fp32 numbers are 2 apart
    w = (1 + np.arange(1024) / 1024)
    y = []
    for up in (0.0, 2.0):
        r = f32(1.0 / f32(np.sqrt(f32(f32((x * x + 1e6 + up) / D) + np.float64(np.float32(1e-5))))))
        y.append(f32(r[:, None] * w).astype(np.float16))
    at = np.argwhere(y[0] != y[1])
    return x[at[:, 0]], w[at[:, 1]]


@pytest.mark.parametrize("D", [64, 128, 256])
def test_the_norms_sum_is_in_its_order(D):
    """Heads of large values x and 1000, a 1 that puts the sum on an fp32 midpoint, and values of 2^-15 that lift it
    off only where they are added up before they meet x^2, beside which (64-bit numbers 2^-28 apart) each is lost."""
    rng = np.random.default_rng(D)
    T, Hq, Hkv, page, groups = 300, 6, 2, 16, D // 8
    xs, ws = telling_pairs(D)
    pair = rng.integers(0, len(xs), (2, groups))  # of each group of eight, with q's and with k's weights
    w = np.ones((2, D), np.float16)
    w[:, 2::8] = ws[pair]
    heads = np.zeros((T, Hq + Hkv, groups, 8))
    for t in range(T):
        for h in range(Hq + Hkv):
            g = int(rng.integers(0, groups))
            heads[t, h, g, :3] = xs[pair[int(h >= Hq), g]], 1000.0, 1.0
            if rng.random() < 0.5:  # behind x in its eight: lost
                heads[t, h, g, 3:] = 2.0 ** -15
            else:  # eight of others: kept
                heads[t, h, (g + 1 + int(rng.integers(0, groups - 1))) % groups] = 2.0 ** -15
    heads = heads.reshape(T, Hq + Hkv, D)
    q, k = (torch.from_numpy(x.astype(np.float16)) for x in (heads[:, :Hq], heads[:, Hq:]))
    v = torch.from_numpy(rng.standard_normal((T, Hkv, D)).astype(np.float16))
    want, other = [[normed(x.double().numpy(), wt.astype(np.float64), 1e-5, add) for x, wt in ((q, w[0]), (k, w[1]))]
                   for add in (in_order, one_by_one)]
    assert min((a != b).sum() for a, b in zip(want, other)) >= T // 5  # the order shows
    S = -(-T // page) * page
    kc, vc = filled_cache(1, S, Hkv * D), filled_cache(2, S, Hkv * D)
    hosts = [[a.copy() for a in host_of(c)] for c in (kc, vc)]
    table = np.random.default_rng(3).permutation(S // page).astype(np.int32)[None]
    slot = (table[0][np.arange(T) // page] * page + np.arange(T) % page).astype(np.int32)
    for x, host in ((torch.from_numpy(want[1]), hosts[0]), (v, hosts[1])):
        oracle.kv_quantize(bits(x).reshape(T, -1), host, slot=slot, dtype=ODT[HF])
    one, zero = torch.ones((1, D // 2), device="cuda"), torch.zeros((1, D // 2), device="cuda")  # position 0: no turn
    got = wq.wq_kv_append(k.cuda(), v.cuda(), kc, vc, torch.from_numpy(table).cuda(), i32([T]), one, zero, page_size=page, q=q.cuda(),
                          q_starts=i32([0, T]), positions=i32([0] * T), norm=True, q_weight=torch.from_numpy(w[0]).cuda(),
                          k_weight=torch.from_numpy(w[1]).cuda(), eps=1e-5, k_out=True)
    torch.cuda.synchronize()
    for g, x, what in zip(got, want, "qk"):
        bad = np.argwhere(bits(g) != x.view(np.uint16))
        assert not len(bad), f"{what}: {len(bad)} values differ, first at {bad[0]}"
    same_cache(kc, hosts[0], "K")
    same_cache(vc, hosts[1], "V")
