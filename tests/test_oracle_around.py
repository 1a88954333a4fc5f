"""Pins for the fp64 oracle of the operators around the decode (rotary
positions, cache append, attention weights, accumulation, eviction)."""
import itertools
import math

import numpy as np
import pytest

from oracle import around_ref as ar
from oracle import sparse_mla_ref as ref


@pytest.mark.parametrize("interleaved", [True, False])
def test_rope_is_complex_multiplication(interleaved):
    rng = np.random.default_rng(1)
    x, pos = rng.standard_normal((3, 2, 20)), np.array([0, 7, 100000])
    f = ar.rope_frequencies(12)
    y = ar.rope(x, pos, f, offset=5, interleaved=interleaved, mscale=1.5)
    part = x[..., 5:17]
    z = part[..., 0::2] + 1j * part[..., 1::2] if interleaved else part[..., :6] + 1j * part[..., 6:]
    want = 1.5 * z * np.exp(1j * pos[:, None, None] * f)
    got = y[..., 5:17]
    got = got[..., 0::2] + 1j * got[..., 1::2] if interleaved else got[..., :6] + 1j * got[..., 6:]
    assert np.abs(got - want).max() < 1e-12
    assert np.array_equal(np.delete(y, np.s_[5:17], -1), np.delete(x, np.s_[5:17], -1))


def test_rope_transpose_is_the_gradient_and_the_inverse():
    rng = np.random.default_rng(2)
    x, g, pos = rng.standard_normal((4, 1, 8)), rng.standard_normal((4, 1, 8)), np.arange(4) * 31
    f = ar.rope_frequencies(8)
    y = ar.rope(x, pos, f, offset=0, interleaved=False, mscale=1.3)
    back = ar.rope(g, pos, f, offset=0, interleaved=False, mscale=1.3, transpose=True)
    assert abs((y * g).sum() - (x * back).sum()) < 1e-12           # <R x, g> = <x, R' g>
    one = ar.rope(x, pos, f, offset=0, interleaved=False)
    assert np.abs(ar.rope(one, pos, f, offset=0, interleaved=False, transpose=True) - x).max() < 1e-12


def test_rope_scores_depend_on_the_distance_alone():
    rng = np.random.default_rng(3)
    q, k = rng.standard_normal((1, 1, 64)), rng.standard_normal((1, 1, 64))
    f = ar.rope_frequencies(64)
    dot = [float((ar.rope(q, [a], f, offset=0, interleaved=True) * ar.rope(k, [b], f, offset=0, interleaved=True)).sum())
           for a, b in ((5, 3), (1005, 1003), (2, 0))]
    assert max(dot) - min(dot) < 1e-9


def test_frequencies():
    assert np.allclose(ar.rope_frequencies(4, base=100.0), [1.0, 0.1], rtol=1e-15)
    assert np.allclose(ar.rope_frequencies(4, base=100.0, scaling="linear", factor=4), [0.25, 0.025], rtol=1e-15)
    plain = ar.rope_frequencies(64)
    yarn = ar.rope_frequencies(64, scaling="yarn", factor=40.0, original_ctx=4096)
    # pairs that turn more than 32 times over 4096 positions keep their frequency, those that turn less than once
    # are divided by the factor, the others lie between, falling steadily
    turns = plain * 4096 / (2 * math.pi)
    assert np.allclose(yarn[turns > 36], plain[turns > 36]) and np.allclose(yarn[turns < 0.9], plain[turns < 0.9] / 40)
    ratio = yarn / plain
    assert np.all(np.diff(ratio) <= 1e-15) and ratio[0] == 1.0 and abs(ratio[-1] - 1 / 40) < 1e-15


def test_append_rows_norm_then_rotation():
    rng = np.random.default_rng(4)
    x, w = rng.standard_normal((5, 576)), rng.standard_normal(512)
    y = ar.append_rows(x, norm_weight=w, eps=0.0)
    assert np.allclose(((y[:, :512] / w) ** 2).mean(1), 1.0) and np.array_equal(y[:, 512:], x[:, 512:])
    f = ar.rope_frequencies(64)
    z = ar.append_rows(x, norm_weight=w, eps=0.0, freq=f, positions=np.arange(5))
    assert np.array_equal(z[0, 512:], x[0, 512:]) and np.allclose(z[:, :512], y[:, :512])
    assert np.allclose(np.linalg.norm(z[:, 512:], axis=1), np.linalg.norm(x[:, 512:], axis=1))
    # 512-dim rows: the rotated dims are normed first
    u = ar.append_rows(x[:, :512], norm_weight=w, eps=0.0, freq=f, positions=np.arange(5))
    assert np.allclose(u[0], y[0, :512])


def test_group_exponent():
    for amax, want in ((448.0, 0), (448.0001, 1), (224.0, -1), (1.0, -8), (0.0, -126), (2.0 ** -140, -126),
                       (1.75, -8), (1.7500001, -7)):
        assert ar.group_exponent(amax) == want, amax
        assert amax <= 448 * 2.0 ** want


def test_slot_rows():
    pt = np.array([[3, 1], [0, 2]])
    assert ar.slot_rows([0, 65, -1, 127], [0, 0, 0, 1], pt).tolist() == [192, 65, -1, 191]
    assert ar.slot_rows([5, -1], None, None).tolist() == [5, -1]


def test_attention_weights_sum_to_the_heads_and_match_the_decode():
    rng = np.random.default_rng(5)
    q, rows = rng.standard_normal((6, 576)), rng.standard_normal((9, 576))
    out, lse = ref.attend_rows(q, rows, 0.04, 512)
    w = ar.attention_weights(q, rows, lse, 0.04)
    assert abs(w.sum() - 6) < 1e-12 and np.all(w > 0)
    # equal queries: the mean output is the weighted mean of the values
    q1 = np.repeat(q[:1], 6, 0)
    out, lse = ref.attend_rows(q1, rows, 0.04, 512)
    w = ar.attention_weights(q1, rows, lse, 0.04)
    assert np.allclose(w @ rows[:, :512] / 6, out[0])
    assert np.all(ar.attention_weights(q, rows, np.full(6, -np.inf), 0.04) == 0)


def test_accumulate_brute_force():
    acc = np.array([[1.0, 2.0, 3.0]])
    got = ar.accumulate(acc, np.array([[2, -1, 0, 2, 7]]), np.array([[1.0, 5.0, 0.25, 2.0, 9.0]]), 0.5)
    assert got.tolist() == [[0.75, 1.0, 4.5]]


def test_evict_select_brute_force():
    rng = np.random.default_rng(6)
    for n, budget, sinks, recent in itertools.product((0, 1, 5, 8), (1, 3, 5, 8), (0, 1), (0, 2)):
        if sinks + recent > budget:
            continue
        acc = rng.integers(0, 3, 8).astype(float)          # ties
        kept = ar.evict_select(acc, n, budget, sinks, recent)
        assert len(kept) == min(n, budget) and kept == sorted(set(kept))
        if n <= budget:
            assert kept == list(range(n))
            continue
        assert set(range(min(sinks, n))) | set(range(n - recent, n)) <= set(kept)
        for i in set(range(n)) - set(kept):                # no evicted position beats a kept, unprotected one
            for j in kept:
                if sinks <= j < n - recent:
                    assert (acc[j], -j) > (acc[i], -i)
    assert ar.evict_select(np.array([np.nan, 0.0, 1.0, np.nan]), 4, 2, 0, 0) == [1, 2]


@pytest.mark.parametrize("mistake", ["mean over the row", "no decay", "ties to the higher", "half as interleaved"])
def test_planted_mistakes_fail_a_pin(mistake):
    rng = np.random.default_rng(7)
    if mistake == "mean over the row":
        x = rng.standard_normal((2, 576))
        wrong = x[:, :512] / np.sqrt((x ** 2).mean(1, keepdims=True))
        assert not np.allclose((wrong ** 2).mean(1), 1.0)
    elif mistake == "no decay":
        assert ar.accumulate(np.ones((1, 2)), np.array([[0]]), np.array([[1.0]]), 0.5).tolist() != [[2.0, 1.0]]
    elif mistake == "ties to the higher":
        assert ar.evict_select(np.zeros(4), 4, 2, 0, 0) == [0, 1]
    else:
        x, f = rng.standard_normal((1, 1, 8)), ar.rope_frequencies(8)
        a, b = (ar.rope(x, [3], f, offset=0, interleaved=i) for i in (True, False))
        assert np.abs(a - b).max() > 1e-3
