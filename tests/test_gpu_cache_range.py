"""The 8-bit cache over the range of its inputs, on lists that are not cut into parts: one
CTA then goes through all tiles of a list, with the reference of its weights running
(shorter batches are cut into parts of a tile, which the combine joins).
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
from sparse_attention_weight_b200 import binding as B
from sparse_attention_weight_b200 import build, inputs
from tests.test_gpu_cache import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    B.lib()


class Whole(Case):
    """One sequence of n rows and as many equal queries at its end as keep the lists whole:
    at least one per SM."""

    def __init__(self, seed, n, H, dense, g=64, page=64):
        super().__init__(seed, [n], 1, H, 0, g, page)
        T = torch.cuda.get_device_properties(0).multi_processor_count + 1
        self.k = 0 if dense else n
        self.T = T
        self.q_seq, self.q_pos = np.zeros(T, np.int32), np.full(T, n - 1, np.int32)
        self.idx = None if dense else np.tile(np.arange(n, dtype=np.int32), (T, 1))
        self.q = np.repeat(self.q, T, 0)

    def run(self, dev, **kw):
        db = kw.get("batch") or self.batch(dev)
        assert B.q8_workspace(B.Q8_MLA, db, H=self.H, k=self.k, device=dev).numel() == 256   # no parts
        return super().run(dev, **kw)


# ------------------------------------------------------------------- a sink and thousands of small weights
@pytest.mark.parametrize("n,dense", [(2048, False), (2048, True), (8191, True), (32768, True)])
@pytest.mark.parametrize("where", ["first", "last", "middle"])
def test_small_weights_beside_a_sink(cuda_device, n, dense, where):
    """One row holds 0.5 to 0.95 of the weight, the others (unit-normal logits, values of
    mean 1 and variance 1) the rest, each too small to be held by itself.

    Tolerance: 3e-3 of the norm of a head's output, whatever the length.  The sink is held
    at 2^7 or more (it is at least the sum of the others, which the reference puts there),
    and small weights in steps of 2^-9, u = 2^-16 of the sink, rounded up or down in the
    proportion that keeps their mean, so that a weight w (the sink 1) has a variance of at
    most u w and the sum over all of them, (1 - p) / p, one of u (1 - p) / p.
    Divided by the sum of the weights, 1 / p, that is a deviation of sqrt(u p (1 - p)) <=
    2^-9 of the values' size sqrt(2), against an output of at least sqrt(1 + p^2) per dim:
    2.5e-3 at p = 0.5.  The bf16 output adds 2^-8 / sqrt(3) of a mantissa's mean square,
    1.7e-3, independently: 3.0e-3 together.
    """
    H = 16
    c = Whole(40 + n, n, H, dense)
    r = np.random.default_rng(n)
    sink = {"first": 0, "last": n - 1, "middle": n // 2}[where]
    rows = np.zeros((n, 576))
    rows[:, :512] = r.standard_normal((n, 512)) + 1
    rows[:, 512:575] = r.standard_normal((n, 63))
    rows[sink, 512:575] = 0
    rows[sink, 575] = 16
    c.codes[c.row(0, np.arange(n))] = inputs.to_e4m3_bytes(rows.astype(np.float32))
    c.scale[:] = 1.0
    sm = 1 / np.sqrt(63)
    v = oracle.e4m3_decode(c.codes[c.row(0, np.arange(n))])
    q = np.zeros((H, 576))
    q[:, 512:575] = oracle.bf16_decode(inputs.to_bf16_bits(r.standard_normal((H, 63)).astype(np.float32)))
    z = sm * (q @ v.T)
    z[:, sink] = -np.inf
    want = np.array([0.5, 0.8, 0.9, 0.95])[np.arange(H) % 4]
    q[:, 575] = (np.log(np.exp(z).sum(1)) + np.log(want / (1 - want))) / (sm * 16)
    c.q = np.repeat(inputs.to_bf16_bits(q.astype(np.float32))[None], c.T, 0)
    out, lse = c.run(cuda_device, sm=sm)
    assert (out == out[0]).all() and (lse == lse[0]).all()
    got, q = oracle.bf16_decode(out[0]), oracle.bf16_decode(c.q[0])
    ref, ref_lse = oracle.sparse_mla(q[None], v, np.arange(n)[None], sm)
    p = np.exp(sm * (q @ v[sink]) - ref_lse[0])
    assert (p > 0.4).all() and (p < 0.97).all()
    err = np.linalg.norm(got - ref[0], axis=1) / np.linalg.norm(ref[0], axis=1)
    print(f"sink {where} of {n}: " + " ".join(f"{x * 1e3:.2f}" for x in err))
    assert (err <= 3e-3).all()
    assert (np.abs(lse[0] - ref_lse[0]) <= 1e-3).all()


# ------------------------------------------------------------------- the running reference
@pytest.mark.parametrize("dense", [False, True])
@pytest.mark.parametrize("tops", [(-100, 40), (-100, 20, 60, 90), (40, -100), (40, -100, 40), (-100, 40, -100, 90),
                                  (-60, 70), (0, 0, 100, -100)], ids=str)
def test_scales_from_end_to_end_of_a_whole_list(cuda_device, tops, dense):
    """Runs of one to three tiles whose scales lie 2^100 and more apart, in rising, falling
    and mixed order: the reference moves by more than fp32's exponents, and every row keeps
    its share of the denominator."""
    n = 1024
    c = Whole(50 + len(tops), n, 16, dense, g=8)
    part = n // len(tops)
    for i, e in enumerate(tops):
        c.scale[np.unique(c.row(0, np.arange(i * part, n if i + 1 == len(tops) else (i + 1) * part)) // 8)] = 2.0 ** e
    sm = 2.0 ** (-max(tops) - 10)                        # logits of about 1
    c.check(*c.run(cuda_device, sm=sm), sm=sm, rows=[0, c.T - 1])


@pytest.mark.parametrize("dense", [False, True])
@pytest.mark.parametrize("order", ["rising", "falling", "both"])
def test_growing_logits_of_a_whole_list(cuda_device, order, dense):
    """Logits that rise, fall, or rise and fall by far more than a factor of 2^8 per tile."""
    n, H = 2000, 16
    c = Whole(60, n, H, dense)
    at = {"rising": np.arange(n), "falling": np.arange(n)[::-1],
          "both": np.where(np.arange(n) < n // 2, np.arange(n), n - np.arange(n)) * 2}[order]
    rows = np.zeros((n, 576))
    rows[:, :512] = np.random.default_rng(2).standard_normal((n, 512))
    rows[:, 575] = at / 40.0
    c.codes[c.row(0, np.arange(n))] = inputs.to_e4m3_bytes(rows.astype(np.float32))
    c.scale[:] = 1.0
    q = np.random.default_rng(3).standard_normal((H, 576)).astype(np.float32)
    q[:, 575] = np.linspace(1, 200, H)
    c.q = np.repeat(inputs.to_bf16_bits(q)[None], c.T, 0)
    c.check(*c.run(cuda_device), rows=[0, c.T - 1])


@pytest.mark.parametrize("first,then", [(0, 1), (127, 0), (128, 300), (300, 2), (999, 0)])
@pytest.mark.parametrize("dense", [False, True])
def test_tiles_without_usable_rows_in_a_whole_list(cuda_device, first, then, dense):
    """The first rows, and every other tile after them, cannot be used (empty slots, or
    scales that are none): the reference is set by the first tile that has one."""
    n = 1000
    c = Whole(65, n, 24, dense, g=1)
    off = np.arange(n) < first
    off |= (np.arange(n) // 128 % 2 == 1) & (np.arange(n) % 128 >= then % 128) & (np.arange(n) != n - 1)
    if dense:
        c.scale[c.row(0, np.flatnonzero(off))] = 0.0
        skip = c.scale == 0
        c.check(*c.run(cuda_device, flags=B.DEV_BAD_SCALE if off.any() else 0), rows=[0, c.T - 1], skip=skip)
    else:
        c.idx[:, off] = -1
        c.check(*c.run(cuda_device), rows=[0, c.T - 1])


# ------------------------------------------------------------------- logits beyond fp32
@pytest.mark.parametrize("n,whole", [(100, True), (1000, True), (1000, False)])
@pytest.mark.parametrize("dense", [False, True])
@pytest.mark.parametrize("sign", [1, -1])
def test_a_largest_logit_beyond_fp32_gives_nan(cuda_device, n, whole, dense, sign):
    """Heads whose largest logit passes fp32's range (either way) are NaN; a row far below
    the others counts nothing; the other heads are as without them."""
    H = 16
    if whole:
        c = Whole(70, n, H, dense)
    else:
        c = Case(70, [n], 1, H, 0 if dense else n, 64, 64)
        if not dense:
            c.idx[0] = np.arange(n)
    vals = oracle.e4m3_decode(c.codes)
    vals[:, 575] = 64.0                                  # of one sign in every row
    c.codes = inputs.to_e4m3_bytes(vals.astype(np.float32))
    c.scale[:] = 1.0
    sm = 1.0 / 24
    ref = c.run(cuda_device, sm=sm)
    c.check(*ref, sm=sm, rows=[0])
    c.q = c.q.copy()
    beyond = np.zeros((H, 576), np.float32)
    beyond[:, 575] = sign * 3e38
    c.q[:, [2, 5]] = inputs.to_bf16_bits(beyond)[None, [2, 5]]
    out, lse = c.run(cuda_device, sm=sm)
    nan = np.isnan(oracle.bf16_decode(out))
    assert nan[:, [2, 5]].all() and np.isnan(lse[:, [2, 5]]).all()
    rest = [h for h in range(H) if h not in (2, 5)]
    assert np.array_equal(out[:, rest], ref[0][:, rest]) and np.array_equal(lse[:, rest], ref[1][:, rest])


@pytest.mark.parametrize("whole", [True, False])
@pytest.mark.parametrize("dense", [False, True])
@pytest.mark.parametrize("at", [0, 500, 999])
def test_one_logit_beyond_fp32(cuda_device, at, dense, whole):
    """Above the others in one row of a list it makes its head NaN, below them it takes the
    row out: the head (all other logits 0) is then the mean of the other rows.
    Tolerance: half a step of bf16, and 2^-8 of the mean magnitude for weights of 8 bits."""
    n, H = 1000, 16
    if whole:
        c = Whole(71, n, H, dense)
    else:
        c = Case(71, [n], 1, H, 0 if dense else n, 64, 64)
        if not dense:
            c.idx[0] = np.arange(n)
    vals = oracle.e4m3_decode(c.codes)
    vals[:, 575] = 0
    vals[c.row(0, np.arange(n))[at], 575] = 64.0
    c.codes = inputs.to_e4m3_bytes(vals.astype(np.float32))
    c.scale[:] = 1.0
    q = np.zeros((H, 576), np.float32)
    q[:, 575] = np.where(np.arange(H) % 2, 3e38, -3e38)
    c.q = np.repeat(inputs.to_bf16_bits(q)[None], c.T, 0)
    out, lse = c.run(cuda_device, sm=1.0)
    got = oracle.bf16_decode(out)
    assert np.isnan(got[:, 1::2]).all() and np.isnan(lse[:, 1::2]).all()
    v = np.delete(oracle.e4m3_decode(c.codes[c.row(0, np.arange(n))])[:, :512], at, 0)
    ref = v.mean(0)
    assert (np.abs(got[:, 0::2] - ref) <= 2.0 ** -8 * (np.abs(ref) + np.abs(v).mean(0))).all()
    assert (np.abs(lse[:, 0::2] - np.log(n - 1)) <= 2.0 ** -16).all()


@pytest.mark.parametrize("queries", [1, 3, 700])
def test_any_bound_of_the_lengths(cuda_device, queries):
    """max_kv_len only has to be no less than any length: the largest number will do, for
    batches whose lists it cuts into parts and for ones whose lists it leaves whole."""
    c = Case(80, [700], queries, 16, 0, 64, 0)
    want = c.run(cuda_device)
    db = c.batch(cuda_device)
    db.struct.max_kv_len = 2 ** 31 - 1
    got = c.run(cuda_device, batch=db)
    rows = [0, queries // 2, queries - 1]
    c.check(*want, rows=rows)
    c.check(*got, rows=rows)
    if queries > 3:
        assert B.q8_workspace(B.Q8_MLA, db, H=c.H, k=0, device=cuda_device).numel() == 256
        assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])


# ------------------------------------------------------------------- appends to scales that are not powers of two
@pytest.mark.parametrize("g", [2, 16, 64])
@pytest.mark.parametrize("T", [3, 4000])
def test_append_into_blocks_of_any_scale(cuda_device, g, T):
    """A block's earlier scale may be any number in range (a cache quantised elsewhere): new
    codes are E4M3 of the exact quotient, and re-encoded ones of the exact product."""
    from oracle import cache as C
    from tests.test_gpu_cache import _append, _same_codes
    r = np.random.default_rng(g + T)
    per = -(-T // 60)
    n = -(-T // per)
    old = r.integers(1, 70, n)
    new = np.minimum(r.integers(1, per + 1, n), per)
    c = Case(90 + g, [int(x) for x in old + new], 1, 8, 0, g, 64)
    c.scale = (2.0 ** r.integers(-8, 6, c.scale.size) * r.uniform(1, 2, c.scale.size)).astype(np.float32)
    q_seq = np.repeat(np.arange(n), new)
    q_pos = np.concatenate([np.arange(o, o + m) for o, m in zip(old, new)])
    kv = oracle.bf16_decode(inputs.to_bf16_bits((r.standard_normal((q_seq.size, 576))
                                                 * np.exp2(r.integers(-3, 8, (q_seq.size, 1)))).astype(np.float32)))
    # quotients next to E4M3's ties: the scale of every other sequence's block is an entry over a tie
    for s in range(0, n, 2):
        b = int(c.row(s, int(old[s]))) // g
        tie = (2 * r.integers(8, 16) + 1) / 2.0 * 2.0 ** r.integers(-4, 4)
        x = max(abs(kv[int(np.flatnonzero(q_seq == s)[0]), 5]), 2.0 ** -6)
        c.scale[b] = np.float32(x / tie)
    bits = inputs.to_bf16_bits(kv.astype(np.float32))
    codes, scale = _append(cuda_device, c, bits, q_seq, q_pos)
    want = C.quantize_append(c.codes, c.scale, g, oracle.bf16_decode(bits), q_seq, q_pos, lambda s, p: int(c.row(s, p)))
    assert np.array_equal(scale, want[1].astype(np.float32)) and _same_codes(codes, want[0])


@pytest.mark.parametrize("exp", [-100, -60, 0, 60, 99])
def test_append_into_blocks_of_any_scale_at_the_ends(cuda_device, exp):
    """The same at the smallest and largest scales, with entries of every size, infinite
    ones and NaN among the new rows."""
    from oracle import cache as C
    from tests.test_gpu_cache import _append, _same_codes
    r = np.random.default_rng(exp + 200)
    g, n = 16, 40
    c = Case(95, [16] * n, 1, 8, 0, g, 64)
    c.scale = (2.0 ** float(exp) * r.uniform(1, 2, c.scale.size)).astype(np.float32)
    q_seq, q_pos = np.repeat(np.arange(n), 3), np.tile([5, 6, 7], n)
    size = np.clip(exp + r.integers(-14, 9 if exp < 99 else 5, (q_seq.size, 1)) + r.integers(-2, 3, (q_seq.size, 576)), -132, 126)
    kv = (r.standard_normal((q_seq.size, 576)) * np.exp2(size.astype(float))).astype(np.float32)
    kv[::7, 3], kv[1::7, 4], kv[2::7, 5] = np.inf, -np.inf, np.nan
    kv[3::7, 6:9] = [0.0, -0.0, 1e-40]
    bits = inputs.to_bf16_bits(kv)
    codes, scale = _append(cuda_device, c, bits, q_seq, q_pos)
    want = C.quantize_append(c.codes, c.scale, g, oracle.bf16_decode(bits), q_seq, q_pos, lambda s, p: int(c.row(s, p)))
    assert np.array_equal(scale, want[1].astype(np.float32)) and _same_codes(codes, want[0])
