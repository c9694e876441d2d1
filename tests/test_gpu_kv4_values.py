"""Attention over the 4-bit cache where the values' sizes differ by far: keys whose
values are all zero, groups of a head that are all zero, groups of different
sizes, values that are not finite (needs a B200).  Every output channel is held
to a bound of its own group's scales."""
import numpy as np
import pytest
import torch

import kv4_ref as ref
import weight_only_quantization_wise_b200 as qz
from test_gpu_kv4 import Cache, dev, randn  # noqa: F401  (dev is a fixture)

pytestmark = pytest.mark.gpu


def expected(q, kq, vq, L, new, D, g, window=0, left_out=None):
    """float64 result and bound of one sequence; left_out: (key, channel) pairs
    that count with weight but without value (their channels are not compared).

    Per channel, with the scales S of its own group (0 for a group of zeros,
    which adds nothing): bf16's half step; 2^-11 of each weight P S, and 2^-25
    of the largest for weights below fp16's normal range (2^-24 taken), times
    |c - Z| <= 15; queries of 16 bits move a score by at most |scale| 2^-15 max|q|
    sum|k| (and 2^-21 for its conversion), a P by the exponential of twice that;
    ex2 and the fp32 sums 2^-20, a P below 2^-126 counts as 0; 16 keys per tensor
    core sum, each off by at most 2^-22 of the largest magnitude, sum P S 15.
    """
    T, Hq, _ = q.shape
    kf, vf = ref.values(*kq, g), ref.values(*vq, g)
    codes, s, z = vq
    S = ref.bf16_f64(s) * (codes.reshape(L, -1, D // g, g) != z[..., None]).any(-1)
    S = np.repeat(S, g, -1)                                     # per channel
    if left_out is not None:
        S, vf = S.copy(), vf.copy()
        S[left_out], vf[left_out] = 0.0, 0.0
    H = kf.shape[1]
    out, lim = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    scale = D ** -0.5
    for i in range(new):
        p = L - new + i
        keep = np.arange(L) <= p
        if window:
            keep &= np.arange(L) > p - window
        n = keep.sum()
        if n == 0:
            continue
        for h in range(Hq):
            kh, vh, Sh = (x[keep][:, h // (Hq // H)] for x in (kf, vf, S))
            qh = q[i, h].double().numpy()
            e = scale * (kh @ qh)
            e = np.exp(e - e.max())
            P = (e / e.sum())[:, None]
            out[i, h] = (P * vh).sum(0)
            pv = (P * np.abs(vh)).sum(0)
            delta = scale * np.abs(qh).max() * np.abs(kh).sum(-1).max() * (2.0 ** -15 + 2.0 ** -21)
            lim[i, h] = (2.0 ** -8 * np.abs(out[i, h]) +
                         ((2.0 ** -11 + 2.0 ** -20) * pv +
                          np.minimum(np.expm1(2 * delta) * pv, 2 * np.abs(vh).max(0))) * (1 + 2.0 ** -8) +
                         (n / 16 + 8) * 2.0 ** -22 * 15 * (P * Sh).sum(0) +
                         n * 15 * (2.0 ** -24 * (P * Sh).max(0) + 2.0 ** -126 * Sh.max(0)) + 2.0 ** -133)
    return out, lim


def check(dev, k, v, q, new, g, window=0):  # noqa: F811
    L, H, D = k.shape
    k, v, q = (x.to(torch.bfloat16) for x in (k, v, q))
    c = Cache(dev, [L], H, D, 16, g)
    c.append(k.to(dev), v.to(dev), [L], [L])
    got = c.attend(q.to(dev), [L], [new], window=window).cpu().double().numpy()
    want, lim = expected(q, ref.quantize(k, g), ref.quantize(v, g), L, new, D, g, window)
    worst = (np.abs(got - want) / lim).max()
    assert worst <= 1.0, worst                      # a NaN fails too
    return got


def led_keys(L, D, at, lead, seed):
    """Keys of small scores, but for one that leads by about `lead` powers of two
    under a query of ones."""
    k = randn((L, 1, D), seed, 0.3).float()
    k[at] = lead * 0.6931 / D ** 0.5
    return k


@pytest.mark.parametrize("D,g", ref.COMBOS)
@pytest.mark.parametrize("at", [0, 17, 200, 399])
@pytest.mark.parametrize("std,lead", [(0.02, 14), (1e-3, 8), (1e-3, 14), (1e-5, 4), (1e-6, 0),
                                      (1e-30, 6)])
def test_a_key_of_zeros_beside_small_values(dev, D, g, at, std, lead):  # noqa: F811
    """A key whose value is zero (its scale is stored as 1) holds most of the
    weight; the others' small values still count in full."""
    L = 400
    v = randn((L, 1, D), 61).float() * std
    v[at] = 0.0
    check(dev, led_keys(L, D, at, lead, 60), v, torch.ones(1, 2, D), 1, g)


@pytest.mark.parametrize("D,g", [c for c in ref.COMBOS if c[0] > c[1]])
@pytest.mark.parametrize("std", [1.0, 1e-3, 1e-6])
@pytest.mark.parametrize("alive_from", [10 ** 6, 250, 385, 398])
def test_a_group_of_zeros(dev, D, g, std, alive_from):  # noqa: F811
    """The last group of a padded head is zero in every key, or up to a late one:
    the live groups, and the late values, count in full."""
    L, new = 400, 4
    k, v = randn((L, 1, D), 62, 0.3), randn((L, 1, D), 63).float() * std
    v[:alive_from, :, -g:] = 0.0
    got = check(dev, k, v, randn((new, 2, D), 64), new, g)
    if alive_from > L:
        assert (got[..., -g:] == 0.0).all()


@pytest.mark.parametrize("D,g", [c for c in ref.COMBOS if c[0] > c[1]])
@pytest.mark.parametrize("power", [-60, -40, -20, -12, 12, 20, 40, 60])
def test_groups_of_different_sizes(dev, D, g, power):  # noqa: F811
    L, new = 300, 2
    k, v = randn((L, 1, D), 65, 0.3), randn((L, 1, D), 66).float()
    v[..., :g] *= 2.0 ** power
    check(dev, k, v, randn((new, 4, D), 67), new, g)


@pytest.mark.parametrize("D,g", ref.COMBOS)
@pytest.mark.parametrize("rise", [0.0, 0.02, 0.3, 3.0])
@pytest.mark.parametrize("alive", [None, 37, 180, 399])
def test_zeros_alone_while_scores_rise(dev, D, g, rise, alive):  # noqa: F811
    """Every value zero, or all but one key's: scores that rise by `rise` powers of
    two a key move the maximum far while no exponent has been set."""
    L = 400
    v = torch.zeros(L, 1, D)
    if alive is not None:
        v[alive] = randn((1, D), 75) * 1e-3
    k = (torch.arange(L).float() * rise * 0.6931 / D ** 0.5)[:, None, None].expand(L, 1, D)
    got = check(dev, k, v, torch.ones(1, 2, D), 1, g)
    if alive is None:
        assert (got == 0.0).all()


@pytest.mark.parametrize("D,g", ref.COMBOS)
@pytest.mark.parametrize("L,new,share,window", [(9000, 1, 8, 0), (700, 70, 8, 0), (700, 70, 8, 40),
                                                (48, 48, 2, 0)])
def test_zeros_among_many_rows_and_parts(dev, D, g, L, new, share, window):  # noqa: F811
    """Keys of zeros at the front and scattered, zero groups, small values, over
    parts of CTAs, 16-row tiles, windows and rows that see zeros alone."""
    H = 2
    k, v = randn((L, H, D), 68, 0.3).float(), randn((L, H, D), 69).float() * 1e-4
    gen = torch.Generator().manual_seed(70)
    v *= (torch.rand(L, H, D // g, 1, generator=gen) < 0.7).expand(L, H, D // g, g).reshape(L, H, D)
    v[:33] = 0.0
    k[:2] += 0.5
    check(dev, k, v, torch.ones(new, H * share, D) + randn((new, H * share, D), 71, 0.2), new, g, window)


@pytest.mark.parametrize("D,g", ref.COMBOS)
@pytest.mark.parametrize("L,at,new", [(400, 150, 1), (400, 398, 1), (400, 399, 3), (400, 0, 2)])
@pytest.mark.parametrize("value", [float("inf"), float("-inf")])
def test_an_infinite_value_stays_in_its_group(dev, D, g, L, at, new, value):  # noqa: F811
    """The channels of the group that holds it are not finite in the rows that see
    the key, whatever step of the sequence it stands in; all others are right."""
    k, v = randn((L, 1, D), 72, 0.3), randn((L, 1, D), 73)
    fine = v.clone()
    v[at, 0, 5] = value
    c = Cache(dev, [L], 1, D, 16, g)
    c.append(k.to(dev), v.to(dev), [L], [L])
    q = randn((new, 2, D), 74)
    got = c.attend(q.to(dev), [L], [new]).cpu().double().numpy()
    left_out = np.zeros((L, 1, D), bool)
    left_out[at, 0, :g] = True                       # the group's other values at that key too
    want, lim = expected(q, ref.quantize(k, g), ref.quantize(fine, g), L, new, D, g, 0, left_out)
    for i in range(new):
        sees = at <= L - new + i
        good = slice(g if sees else 0, None)
        if sees:
            assert not np.isfinite(got[i, :, :g]).any()
        assert (np.abs(got[i, :, good] - want[i, :, good]) <= lim[i, :, good]).all(), i
    assert qz.qz_device_status() == 0
