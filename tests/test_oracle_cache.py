"""Pins of the oracle of the 8-bit cache and of the pages to facts outside it."""
from __future__ import annotations

from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle
from oracle import cache as C


def test_need_exponent_is_the_smallest_that_holds_the_maximum():
    rng = np.random.default_rng(0)
    for x in list(np.exp(rng.uniform(-60, 60, 200))) + [448.0, 449.0, 447.0, 224.0, 1e-20, 2.0 ** -90]:
        e = C.need_exponent(float(x))
        assert Fraction(448) * Fraction(2) ** e >= Fraction(float(x)) > Fraction(448) * Fraction(2) ** (e - 1)
    assert C.need_exponent(0.0) == -100 and C.need_exponent(1e38) == 100


def test_append_matches_torch_casts_and_keeps_the_other_rows():
    rng = np.random.default_rng(1)
    g, rows, T = 8, 40, 13
    codes = rng.integers(0, 120, size=(rows, 576)).astype(np.uint8)
    scale = 2.0 ** rng.integers(-3, 3, size=rows // g)
    kv = rng.standard_normal((T, 576)) * 100
    off = 16
    q_pos = np.arange(3, 3 + T)
    new_codes, new_scale = C.quantize_append(codes, scale, g, kv, np.zeros(T, int), q_pos, lambda s, p: off + p)
    for r in list(range(off)) + list(range(off + 16, rows)):
        assert np.array_equal(new_codes[r], codes[r])
    assert np.array_equal(new_scale[[0, 1, 4]], scale[[0, 1, 4]])
    for t in range(T):
        s = new_scale[(off + 3 + t) // g]
        ref = torch.tensor(kv[t] / s, dtype=torch.float64).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
        assert np.array_equal(new_codes[off + 3 + t], ref)
    for r in range(off, off + 3):                       # rows of the first block that were there before
        f = scale[2] / new_scale[2]
        assert f <= 1
        ref = torch.tensor(oracle.e4m3_decode(codes[r]) * f).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
        assert np.array_equal(new_codes[r], ref)


def test_re_encoding_is_exact_above_the_smallest_step():
    codes = np.arange(126, dtype=np.uint8)[None, :].repeat(5, 0)
    codes = np.pad(codes, ((0, 3), (0, 450)))
    kv = np.full((1, 576), 448.0 * 4)                   # needs a scale of 4: the old rows' exponents fall by 2
    new, s = C.quantize_append(codes, np.ones(1), 8, kv, [0], [5], lambda q, p: p)
    assert s[0] == 4.0
    before, after = oracle.e4m3_decode(codes[0]), oracle.e4m3_decode(new[0]) * 4
    big = np.abs(before) >= 2.0 ** -3                   # 8 times the smallest normal: three bits below it are kept
    assert np.array_equal(before[big], after[big])
    assert np.abs(before - after).max() <= 4 * 2.0 ** -10


def _held(pool):
    want = np.zeros_like(pool.refs)
    for s in range(pool.table.shape[0]):
        n = pool.pages(pool.lens[s])
        assert (pool.table[s, :n] >= 0).all()
        np.add.at(want, pool.table[s, :n], 1)
    return want


@pytest.mark.parametrize("seed", range(6))
def test_pool_invariants_under_random_calls(seed):
    """Random resizes, forks and compactions: counts stay those of the tables, and
    what a sequence reads is what was written to it (rows carry unique stamps)."""
    rng = np.random.default_rng(seed)
    S, N, P, pps = 9, 40, 4, 8
    pool = C.Pool(np.full((S, pps), -1), np.zeros(S, int), np.zeros(N, int), P)
    data = np.zeros((N, P), np.int64)
    wrote = {s: [] for s in range(S)}
    stamp = 1
    for _ in range(60):
        what = rng.integers(3)
        if what == 0:
            n = rng.integers(1, S + 1)
            seqs = rng.permutation(S)[:n]
            lens = rng.integers(0, 2 * P * 3, size=n)
            before = pool.lens.copy()
            pool.no_pages = False
            for a, b in pool.resize(seqs, lens):
                data[b] = data[a]
            for s in seqs:
                s = int(s)
                wrote[s] = wrote[s][:pool.lens[s]]
                for x in range(before[s], pool.lens[s]):     # append: written once per new row
                    data[pool.table[s, x // P], x % P] = stamp
                    wrote[s].append(stamp)
                    stamp += 1
        elif what == 1:
            src = rng.integers(0, S, size=2)
            dst = rng.integers(0, S, size=2)
            before = pool.lens.copy()
            pool.fork(src, dst)
            done = set()
            for a, b in zip(map(int, src), map(int, dst)):
                if before[b] == 0 and b not in done and a not in dst:
                    wrote[b] = list(wrote[a])
                done.add(b)
        else:
            _, copies = pool.compact()
            for a, b in copies:
                data[b] = data[a]
            live = np.flatnonzero(pool.refs)
            assert live.size == 0 or live.max() == live.size - 1
        assert np.array_equal(_held(pool), pool.refs)
        for s in range(S):
            got = [data[pool.table[s, x // P], x % P] for x in range(pool.lens[s])]
            assert got == wrote[s], s


def test_growth_is_all_or_nothing_and_lists_are_checked():
    pool = C.Pool(np.full((3, 4), -1), np.zeros(3, int), np.zeros(5, int), 4)
    pool.resize([0, 1], [8, 8])
    assert list(pool.table[0, :2]) == [0, 1] and list(pool.table[1, :2]) == [2, 3]
    pool.resize([0, 1, 2], [4, 12, 8])                  # frees one page, wants three
    assert pool.no_pages and list(pool.lens) == [4, 8, 0] and pool.refs.sum() == 3
    pool.bad = False
    pool.resize([2, 2, 9, 1], [4, 8, 4, 17])            # twice, out of range, too long
    assert pool.bad and list(pool.lens) == [4, 8, 4]
