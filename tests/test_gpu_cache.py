"""The 8-bit latent cache on the GPU against the float64 oracle.

Append: codes and scales must equal the oracle's (one rounding, nearest even).

Attention tolerance, per output value, from the number formats (all sums in
float64 on the oracle's side; p, v the exact weights and values, s the row scales):
  output     half a step of bf16: 2^-8 |ref| (at least the smallest step)
  weights    p_i s_i is held as hi + lo of E4M3 by way of fp16: half a step of fp16 (2^-12
             relative), then of lo, which is at most half a step of hi (2^-4 of 2^-4
             relative) or half of E4M3's smallest step (2^-10) where that is more, with
             a largest weight of at least 2^5:
             (2^-8 + 2^-12) sum p|v| + 2^-15 max_i(p_i s_i) sum_i |code_i|
  logits     an error dz of every logit moves each weight by 2 dz relative: 2 dz sum p|v|
             dz = |sm| (2^-17 max|q| max_i sum_d |c_id|        (query entries, two E4M3 numbers)
                        + 2^-15 max_i sum_d |q_d c_id|)        (fp32 sums of 36 partial products)
                  + 2^-19 (1 + max|z|)                         (scaling and exponentials in fp32)
  lse        dz + 2^-19 (1 + |lse|)
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
from oracle import cache as C
from sparse_attention_weight_b200 import binding as B
from sparse_attention_weight_b200 import build, inputs
from sparse_attention_weight_b200.configs import Workload

pytestmark = pytest.mark.gpu
SM = 1 / 24


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    B.lib()


class Case:
    """A cache with random codes and scales, queries and a selection, on the host."""

    def __init__(self, seed, lens, qs, H, k, g, page, scale_exp=(-7, -4), holes=0.0, dup=False, gap=0):
        r = np.random.default_rng(seed)
        self.H, self.k, self.g, self.page = H, k, g, page
        self.lens = np.array(lens, np.int32)
        self.n = len(lens)
        need = [-(-x // (page or g)) for x in lens]
        unit = page or g
        units = sum(need) + 2
        perm = r.permutation(units) if page else np.arange(units)
        self.pps = max(1, max(need))
        self.table = np.full((self.n, self.pps), -1, np.int32)
        self.off = np.zeros(self.n, np.int64)
        at = 0
        for b, m in enumerate(need):
            self.table[b, :m] = perm[at:at + m]
            self.off[b] = at * unit + gap
            at += m
        self.rows = units * unit + gap
        self.codes = r.integers(0, 256, size=(self.rows, 576)).astype(np.uint8)
        self.codes[(self.codes & 0x7F) == 0x7F] = 0x3A
        self.codes = np.where(np.abs(oracle.e4m3_decode(self.codes)) > 200, self.codes ^ 0x20, self.codes).astype(np.uint8)
        self.scale = (2.0 ** r.integers(*scale_exp, size=-(-self.rows // g), endpoint=True)).astype(np.float32)
        self.q_seq = np.repeat(np.arange(self.n, dtype=np.int32), qs)
        self.q_pos = np.concatenate([np.arange(x - qs, x) for x in lens]).astype(np.int32)
        T = self.T = self.q_seq.size
        self.q = inputs.to_bf16_bits(r.standard_normal((T, H, 576), dtype=np.float32))
        self.idx = None
        if k:
            self.idx = np.full((T, k), -1, np.int32)
            for t in range(T):
                n = int(self.q_pos[t]) + 1
                m = min(n, k) if not dup else k
                m -= int(m * holes)
                sel = r.choice(n, size=m, replace=dup)
                self.idx[t, np.sort(r.choice(k, size=m, replace=False))] = sel if dup else np.sort(sel)

    def row(self, b, pos):
        pos = np.asarray(pos)
        if self.page:
            return self.table[b, pos // self.page].astype(np.int64) * self.page + pos % self.page
        return self.off[b] + pos

    def batch(self, dev):
        class Host:
            kv_offset, kv_len, q_seq, q_pos = self.off, self.lens, self.q_seq, self.q_pos
        return B.DeviceBatch.from_host(Host, dev, kv_rows=self.rows, page_size=self.page,
                                       page_table=self.table if self.page else None)

    def run(self, dev, sm=SM, flags=0, batch=None, stream=None):
        db = batch or self.batch(dev)
        t = {n: B.bits_to_tensor(getattr(self, n), dev) for n in ("q", "codes", "scale")}
        idx = None if self.idx is None else torch.as_tensor(self.idx, device=dev)
        out = torch.full((self.T + 1, self.H, 512), 0x4242, dtype=torch.int16, device=dev)
        lse = torch.full((self.T + 1, self.H), 7.0, device=dev)
        ws = B.q8_workspace(B.Q8_MLA, db, H=self.H, k=self.k, device=dev)
        B.dsa_sparse_mla_q8(db, t["q"], t["codes"], t["scale"], self.g, idx, self.k, self.H, sm, out, lse, ws)
        assert B.read_device_status(ws) == flags
        out, lse = B.tensor_to_bits(out), lse.cpu().numpy()
        assert (out[self.T] == 0x4242).all() and (lse[self.T] == 7.0).all()     # rows behind the last are not written
        return out[:self.T], lse[:self.T]

    def check(self, out_bits, lse, sm=SM, rows=None, skip=None):
        got = oracle.bf16_decode(out_bits)
        q = oracle.bf16_decode(self.q)
        for t in range(self.T) if rows is None else rows:
            b = int(self.q_seq[t])
            pos = np.arange(self.q_pos[t] + 1) if self.idx is None else self.idx[t][self.idx[t] >= 0]
            rr = self.row(b, pos.astype(np.int64))
            s = self.scale[rr // self.g].astype(np.float64)
            if skip is not None:
                keep = ~skip[rr // self.g]
                rr, s = rr[keep], s[keep]
            if rr.size == 0:
                assert (out_bits[t] == 0).all() and (lse[t] == -np.inf).all()
                continue
            code = oracle.e4m3_decode(self.codes[rr])
            c = code * s[:, None]
            ref, ref_lse = oracle.sparse_mla(q[t:t + 1], c, np.arange(rr.size)[None], sm)
            ref, ref_lse = ref[0], ref_lse[0]
            z = sm * (q[t] @ c.T)
            p = np.exp(z - ref_lse[:, None])
            pv = p @ np.abs(c[:, :512])
            w = (p * s).max(1)[:, None] * np.abs(code[:, :512]).sum(0)[None]
            dz = abs(sm) * (2.0 ** -17 * np.abs(q[t]).max(1) * np.abs(c).sum(1).max()
                            + 2.0 ** -15 * (np.abs(q[t]) @ np.abs(c).T).max(1)) + 2.0 ** -19 * (1 + np.abs(z).max(1))
            bound = 2.0 ** -8 * np.abs(ref) + 2.0 ** -133 + (2.0 ** -8 + 2.0 ** -12 + 2 * dz[:, None]) * pv + 2.0 ** -15 * w
            err = np.abs(got[t] - ref)
            assert (err <= bound).all(), (t, float((err / bound).max()))
            assert (np.abs(lse[t] - ref_lse) <= dz + 2.0 ** -19 * (1 + np.abs(ref_lse))).all(), t


# ------------------------------------------------------------------- attention
@pytest.mark.parametrize("H", [8, 16, 24, 32, 40, 64, 72, 128])
def test_sparse_heads(cuda_device, H):
    c = Case(H, [300, 17, 129], 2, H, 100, 16, 64, holes=0.2)
    c.check(*c.run(cuda_device))


@pytest.mark.parametrize("k", [1, 2, 31, 32, 63, 64, 65, 127, 128, 129, 255, 256, 257, 1000, 2047, 2048])
def test_sparse_selection_widths(cuda_device, k):
    c = Case(k, [2500, 700], 1, 72, k, 64, 0, holes=0.1 if k > 10 else 0.0)
    c.check(*c.run(cuda_device))


@pytest.mark.parametrize("g", [1, 2, 4, 8, 16, 32, 64])
@pytest.mark.parametrize("page", [0, 64, 128, 192])
def test_blocks_and_pages(cuda_device, g, page):
    c = Case(g + page, [400, 65, 64, 1], 1, 16, 150, g, page)
    c.check(*c.run(cuda_device))


def test_contiguous_sequences_need_no_alignment(cuda_device):
    c = Case(3, [100, 333], 2, 32, 80, 16, 0, gap=5)
    c.check(*c.run(cuda_device))


@pytest.mark.parametrize("lens", [[1], [2, 1, 3], [63, 64, 65], [127, 128, 129], [255, 256, 257], [1000, 31],
                                  [5003]], ids=str)
@pytest.mark.parametrize("page", [0, 64])
def test_dense(cuda_device, lens, page):
    c = Case(sum(lens), lens, 1, 128 if sum(lens) < 600 else 40, 0, 32, page)
    c.check(*c.run(cuda_device))


def test_dense_several_queries_see_their_own_prefix(cuda_device):
    c = Case(5, [140, 71], 70, 16, 0, 64, 64)
    c.check(*c.run(cuda_device))


def test_dense_equals_the_full_selection(cuda_device):
    c = Case(6, [900, 411], 3, 64, 0, 8, 64)
    out, lse = c.run(cuda_device)
    c.k = 1024
    c.idx = np.full((c.T, 1024), -1, np.int32)
    for t in range(c.T):
        c.idx[t, :c.q_pos[t] + 1] = np.arange(c.q_pos[t] + 1)
    out2, lse2 = c.run(cuda_device)
    c.check(out2, lse2)
    c.idx, c.k = None, 0
    c.check(out, lse)


def test_prefill_rows(cuda_device):
    """Many queries of one sequence (more than there are SMs), ragged selections."""
    c = Case(8, [700], 650, 24, 96, 64, 64, holes=0.3)
    c.check(*c.run(cuda_device), rows=range(0, 650, 13))


def test_long_context_decode(cuda_device):
    c = Case(9, [40000, 9000], 2, 128, 2048, 64, 64)
    c.check(*c.run(cuda_device))


def test_repeated_rows_count_each_time(cuda_device):
    c = Case(10, [50, 9], 2, 16, 200, 4, 64, dup=True)
    c.check(*c.run(cuda_device))


def test_rows_that_a_mask_leaves_empty(cuda_device):
    c = Case(11, [300, 200, 100], 2, 24, 130, 64, 64, holes=0.5)
    c.idx[1] = -1                                        # nothing
    c.idx[3, :] = -1
    c.idx[3, 129] = 7                                    # one row, in the last slot
    c.idx[4, :128] = -1                                  # only slots of the second tile
    c.idx[4, 128:] = [3, 5]
    c.check(*c.run(cuda_device))


def test_scales_far_apart(cuda_device):
    c = Case(12, [200, 90], 1, 16, 120, 8, 64, scale_exp=(-14, 0))
    c.check(*c.run(cuda_device))
    c = Case(13, [200, 90], 1, 16, 120, 8, 64, scale_exp=(-95, -90))
    c.check(*c.run(cuda_device))
    c = Case(14, [200, 90], 1, 16, 120, 8, 64, scale_exp=(90, 95))
    c.check(*c.run(cuda_device, sm=2.0 ** -96), sm=2.0 ** -96)


def test_scales_that_are_not_powers_of_two(cuda_device):
    c = Case(15, [200, 90], 1, 16, 120, 8, 64)
    c.scale *= np.random.default_rng(1).uniform(0.5, 2, c.scale.shape).astype(np.float32)
    c.check(*c.run(cuda_device))


@pytest.mark.parametrize("sm", [0.0, -0.05, 1.0])
def test_softmax_scales(cuda_device, sm):
    c = Case(16, [260, 90], 1, 16, 150, 8, 64)
    c.check(*c.run(cuda_device, sm=sm), sm=sm)


def test_peaked_and_growing_logits(cuda_device):
    """Logits that rise over the rows by far more than a factor of 2^8 per tile (the
    running maximum changes in every tile), and one row that holds nearly all weight."""
    c = Case(17, [1200], 1, 16, 1024, 64, 0)
    c.idx[0] = np.arange(1024)
    base = np.arange(c.rows) / 40.0
    codes = np.zeros((c.rows, 576))
    codes[:, :512] = np.random.default_rng(2).standard_normal((c.rows, 512))
    codes[:, 575] = base
    c.codes = inputs.to_e4m3_bytes(codes.astype(np.float32))
    c.scale[:] = 1.0
    q = np.random.default_rng(3).standard_normal((1, 16, 576)).astype(np.float32)
    q[..., 575] = 200.0
    c.q = inputs.to_bf16_bits(q)
    c.check(*c.run(cuda_device))
    c.idx[0] = np.arange(1024)[::-1]                     # and falling
    c.check(*c.run(cuda_device))


def test_queries_of_any_size(cuda_device):
    c = Case(18, [200, 90], 1, 16, 120, 8, 64)
    for f in (1e-30, 1e-3, 3e4):
        r = np.random.default_rng(4).standard_normal((c.T, 16, 576)).astype(np.float32) * np.float32(f)
        c.q = inputs.to_bf16_bits(r)
        c.check(*c.run(cuda_device, sm=SM / f if f > 1 else SM), sm=SM / f if f > 1 else SM)
    c.q[:] = 0
    c.check(*c.run(cuda_device))


def test_nan_and_infinity_stay_where_they_are(cuda_device):
    c = Case(19, [200, 150], 2, 16, 60, 8, 64)
    ref = c.run(cuda_device)
    used = np.zeros(c.rows, bool)
    for t in range(c.T):
        used[c.row(c.q_seq[t], c.idx[t][c.idx[t] >= 0])] = True
    c.codes[~used] = 0x7F                                # rows that nobody selects
    got = c.run(cuda_device)
    assert np.array_equal(got[0], ref[0]) and np.array_equal(got[1], ref[1])
    c.check(*got)
    c.codes[c.row(c.q_seq[2], c.idx[2, 5])] = 0xFF       # a row of query 2
    hit = np.array([(c.row(c.q_seq[t], c.idx[t][c.idx[t] >= 0]) == c.row(c.q_seq[2], c.idx[2, 5])).any()
                    for t in range(c.T)])
    q = c.q.copy()
    q[0, 3, 7], q[0, 9, 575] = 0x7F80, 0xFF80            # +inf and -inf in two heads of query 0
    q[1, 2, 0] = 0x7FC0                                  # NaN
    c.q = q
    out, lse = c.run(cuda_device)
    nan = np.isnan(oracle.bf16_decode(out)).all(2)
    assert np.array_equal(nan, np.isnan(oracle.bf16_decode(out)).any(2)) and np.array_equal(nan, np.isnan(lse))
    want = np.zeros((c.T, 16), bool)
    want[hit] = True
    want[0, [3, 9]] = want[1, 2] = True
    assert np.array_equal(nan, want)
    assert np.array_equal(out[~want], ref[0][~want])


@pytest.mark.parametrize("T,H", [(1, 128), (10, 128), (20, 64)])
@pytest.mark.parametrize("dense", [False, True])
def test_nan_in_a_part_of_a_split_list(cuda_device, T, H, dense):
    """A NaN row makes its query NaN, whichever part of the list it lies in (the last query
    too, behind whose parts nothing is), and no other query; an empty part stays out of it."""
    lens = [2300 + 64 * t for t in range(T)]
    c = Case(30 + T, lens, 1, H, 0 if dense else 2048, 64, 64)
    if not dense and T > 1:
        c.idx[1] = -1
        c.idx[1, :300] = np.arange(300)                  # later parts empty
    want = c.run(cuda_device)
    for t in {0, T // 2, T - 1}:
        pos = 1234 if dense else int(c.idx[t][c.idx[t] >= 0][-1])
        c.codes[c.row(t, np.array([pos]))] = 0x7F
    out, lse = c.run(cuda_device)
    hit = np.zeros(T, bool)
    hit[[0, T // 2, T - 1]] = True
    nan = np.isnan(oracle.bf16_decode(out))
    assert nan[hit].all() and np.isnan(lse[hit]).all() and not nan[~hit].any()
    assert np.array_equal(out[~hit], want[0][~hit]) and np.array_equal(lse[~hit], want[1][~hit])


def test_flags(cuda_device):
    c = Case(20, [200, 150, 90], 1, 16, 60, 8, 64)
    good = c.idx.copy()
    c.idx[1, 3] = 150                                    # beyond its sequence
    out, lse = c.run(cuda_device, flags=B.DEV_BAD_INDEX)
    c.idx[1, 3] = -1
    c.check(out, lse)                                    # the entry was skipped
    c.idx = good
    skip = np.zeros(c.scale.size, bool)
    blocks = [int(c.row(0, c.idx[0, 4]) // 8), int(c.row(2, c.idx[2, 0]) // 8), int(c.row(2, c.idx[2, 9]) // 8)]
    for i, bad in zip(blocks, (np.float32("nan"), np.float32(0), np.float32(-1))):
        c.scale[i] = bad
        skip[i] = True
    c.check(*c.run(cuda_device, flags=B.DEV_BAD_SCALE), skip=skip)
    c = Case(21, [200, 150, 90], 1, 16, 60, 8, 64)
    c.table[1, 1] = 1 << 20
    out, lse = c.run(cuda_device, flags=B.DEV_BAD_INDEX)
    c.idx[1][c.idx[1] // 64 == 1] = -1
    c.check(out, lse)


def test_dense_flags(cuda_device):
    c = Case(22, [200, 150, 90], 1, 16, 0, 8, 64)
    c.q_pos[1] = 150
    out, lse = c.run(cuda_device, flags=B.DEV_BAD_QUERY)
    assert (out[1] == 0).all() and (lse[1] == -np.inf).all()
    c.check(out, lse, rows=[0, 2])
    c.q_pos[1], c.q_seq[2] = 149, 3
    out, lse = c.run(cuda_device, flags=B.DEV_BAD_QUERY)
    assert (out[2] == 0).all() and (lse[2] == -np.inf).all()
    c.check(out, lse, rows=[0, 1])


def test_no_queries(cuda_device):
    c = Case(23, [20], 1, 8, 4, 1, 0)
    db = c.batch(cuda_device)
    db.struct.num_q = 0
    ws = B.q8_workspace(B.Q8_MLA, db, H=8, k=4, device=cuda_device)
    e = torch.empty(16, dtype=torch.uint8, device=cuda_device)
    B.dsa_sparse_mla_q8(db, e, e, e, 1, e, 4, 8, SM, e, None, ws)
    B.dsa_quantize_append(db, e, e, e, 1, ws)
    assert B.read_device_status(ws) == 0


def test_no_queries_and_no_pointers(cuda_device):
    """Empty tensors have no address: an empty batch takes them in either form."""
    c = Case(23, [20], 1, 8, 4, 1, 0)
    c.q_seq, c.q_pos = c.q_seq[:0], c.q_pos[:0]
    db = c.batch(cuda_device)
    e = torch.empty(0, dtype=torch.uint8, device=cuda_device)
    for k, idx in ((4, e), (4, None), (0, None)):
        ws = B.q8_workspace(B.Q8_MLA, db, H=8, k=k, device=cuda_device)
        B.dsa_sparse_mla_q8(db, e, e, e, 1, idx, k, 8, SM, e, None, ws)
        assert B.read_device_status(ws) == 0


@pytest.mark.parametrize("top,rest,dense", [(40, -100, False), (40, -100, True), (90, -80, True), (8, -100, False)])
def test_scales_at_both_ends_in_one_query(cuda_device, top, rest, dense):
    """Rows of the smallest scale (what the append gives to a block of zeros) beside rows of
    a large one: they add nothing to the output but their full share to the denominator."""
    c = Case(28, [900, 2500], 1, 16, 0 if dense else 700, 8, 64)
    c.scale[:] = 2.0 ** rest
    for b in range(2):
        for pos in (1, 160, 500):                        # before, beside and after rows of the small scale
            c.scale[c.row(b, pos) // 8] = 2.0 ** top
            if not dense:
                c.idx[b, pos] = pos
    sm = SM * 2.0 ** (-top - 6)                          # logits of about 1
    c.check(*c.run(cuda_device, sm=sm), sm=sm)


def test_dense_beyond_the_stated_length(cuda_device):
    """A position far behind max_kv_len is refused, not answered from part of its rows."""
    c = Case(29, [900, 100], 1, 16, 0, 8, 64)
    db = c.batch(cuda_device)
    db.struct.max_kv_len = 128
    out, lse = c.run(cuda_device, flags=B.DEV_BAD_QUERY, batch=db)
    assert (out[0] == 0).all() and (lse[0] == -np.inf).all()
    c.check(out, lse, rows=[1])


@pytest.mark.parametrize("T", [74, 75, 147, 148, 149, 297])
@pytest.mark.parametrize("H,k", [(72, 300), (16, 0)])
def test_items_around_the_number_of_sms(cuda_device, T, H, k):
    r = np.random.default_rng(T)
    c = Case(T, [int(x) for x in r.integers(1, 400, T)], 1, H, k, 16, 64, holes=0.2 if k else 0.0)
    if k:
        c.idx[::5] = -1                                  # items without rows between the others
        c.check(*c.run(cuda_device), rows=range(0, T, 7))
    else:
        c.check(*c.run(cuda_device), rows=range(0, T, 7))


def test_results_repeat_bit_for_bit(cuda_device):
    c = Case(24, [3000, 800, 77], 1, 128, 512, 64, 64)
    a, b = c.run(cuda_device), c.run(cuda_device)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


def test_captured_calls_on_two_streams(cuda_device):
    """Two captured graphs, each with its own workspace, replayed together on two
    streams give what eager calls give."""
    cases = [Case(25, [2000, 500], 1, 128, 700, 64, 64), Case(26, [900], 3, 64, 0, 16, 0)]
    want = [c.run(cuda_device) for c in cases]
    graphs, outs, keep = [], [], []
    for c in cases:
        db = c.batch(cuda_device)
        t = [B.bits_to_tensor(x, cuda_device) for x in (c.q, c.codes, c.scale)]
        idx = None if c.idx is None else torch.as_tensor(c.idx, device=cuda_device)
        out = torch.zeros((c.T, c.H, 512), dtype=torch.int16, device=cuda_device)
        lse = torch.zeros((c.T, c.H), device=cuda_device)
        ws = B.q8_workspace(B.Q8_MLA, db, H=c.H, k=c.k, device=cuda_device)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            B.dsa_sparse_mla_q8(db, t[0], t[1], t[2], c.g, idx, c.k, c.H, SM, out, lse, ws)
        graphs.append(g)
        outs.append((out, lse, ws))
        keep.append((db, t, idx))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for (out, lse, ws), (w_out, w_lse) in zip(outs, want):
        assert B.read_device_status(ws) == 0
        assert np.array_equal(B.tensor_to_bits(out), w_out) and np.array_equal(lse.cpu().numpy(), w_lse)


def test_rows_beyond_32_bit_offsets(cuda_device):
    """A cache of more than 2^32 bytes: attention and append at its end."""
    free, _ = torch.cuda.mem_get_info()
    if free < 12 << 30:
        pytest.skip("needs 12 GB of free device memory")
    rows = (1 << 23) + 1024                              # 4.8 GB of codes
    c = Case(27, [500], 2, 16, 200, 64, 0)
    off = rows - 576
    kv8 = torch.zeros((rows, 576), dtype=torch.uint8, device=cuda_device)
    scale = torch.ones(rows // 64, device=cuda_device)
    kv8[off:off + 500] = torch.as_tensor(c.codes[:500], device=cuda_device)
    scale[off // 64:off // 64 + 8] = torch.as_tensor(c.scale[:8], device=cuda_device)
    small = c.run(cuda_device)

    class Host:
        kv_offset, kv_len, q_seq, q_pos = np.array([off]), c.lens, c.q_seq, c.q_pos
    db = B.DeviceBatch.from_host(Host, cuda_device, kv_rows=rows)
    out = torch.zeros((2, 16, 512), dtype=torch.int16, device=cuda_device)
    lse = torch.zeros((2, 16), device=cuda_device)
    ws = B.q8_workspace(B.Q8_MLA, db, H=16, k=200, device=cuda_device)
    B.dsa_sparse_mla_q8(db, B.bits_to_tensor(c.q, cuda_device), kv8, scale, 64,
                        torch.as_tensor(c.idx, device=cuda_device), 200, 16, SM, out, lse, ws)
    assert B.read_device_status(ws) == 0
    assert np.array_equal(B.tensor_to_bits(out), small[0]) and np.array_equal(lse.cpu().numpy(), small[1])
    kv = np.random.default_rng(5).standard_normal((2, 576)).astype(np.float32) * 50
    bits = inputs.to_bf16_bits(kv)
    want_codes, want_scale = C.quantize_append(c.codes[:512], c.scale[:8], 64, oracle.bf16_decode(bits), c.q_seq,
                                               c.q_pos, lambda s, p: p)
    B.dsa_quantize_append(db, B.bits_to_tensor(bits, cuda_device), kv8, scale, 64, ws)
    assert B.read_device_status(ws) == 0
    assert np.array_equal(kv8[off:off + 500].cpu().numpy(), want_codes[:500])
    assert np.array_equal(scale[off // 64:off // 64 + 8].cpu().numpy(), want_scale)
    assert not kv8[:off].any()


# ------------------------------------------------------------------- append
def _append(dev, c, bits, q_seq, q_pos, flags=0):
    class Host:
        kv_offset, kv_len = c.off, c.lens
    Host.q_seq, Host.q_pos = np.asarray(q_seq, np.int32), np.asarray(q_pos, np.int32)
    db = B.DeviceBatch.from_host(Host, dev, kv_rows=c.rows, page_size=c.page, page_table=c.table if c.page else None)
    kv8, scale = B.bits_to_tensor(c.codes, dev), B.bits_to_tensor(c.scale, dev)
    ws = B.q8_workspace(B.Q8_APPEND, db, device=dev)
    B.dsa_quantize_append(db, B.bits_to_tensor(bits, dev), kv8, scale, c.g, ws)
    assert B.read_device_status(ws) == flags
    return kv8.cpu().numpy(), scale.cpu().numpy()


def _same_codes(got, want):
    """Equal codes; the two zeros and the two NaN codes are one each."""
    canon = lambda x: np.where((x & 0x7F) == 0x7F, 0x7F, x)  # noqa: E731
    return np.array_equal(canon(got), canon(want))


@pytest.mark.parametrize("g", [1, 2, 4, 8, 16, 32, 64])
@pytest.mark.parametrize("page", [0, 64, 192])
@pytest.mark.parametrize("new", [[1, 1, 1, 1], [2, 3, 1, 5], [64, 65, 1, 200], [300, 0, 127, 128]], ids=str)
def test_append_matches_oracle(cuda_device, g, page, new):
    r = np.random.default_rng(g + page + sum(new))
    old = np.array([0, 5, 64, 131])
    lens = old + np.array(new)
    c = Case(1, [int(max(1, x)) for x in lens], 1, 8, 0, g, page)
    c.lens = lens.astype(np.int32)
    q_seq = np.repeat(np.arange(4), new)
    q_pos = np.concatenate([np.arange(o, o + n) for o, n in zip(old, new)])
    kv = r.standard_normal((q_seq.size, 576)).astype(np.float32) * np.exp2(r.integers(-6, 6, (q_seq.size, 1))).astype(np.float32)
    bits = inputs.to_bf16_bits(kv)
    codes, scale = _append(cuda_device, c, bits, q_seq, q_pos)
    want_codes, want_scale = C.quantize_append(c.codes, c.scale, g, oracle.bf16_decode(bits), q_seq, q_pos,
                                               lambda s, p: int(c.row(s, p)))
    assert np.array_equal(scale, want_scale.astype(np.float32)) and _same_codes(codes, want_codes)


def test_append_long_list(cuda_device):
    """More tokens than the short-list rule takes: windows of several tokens per CTA."""
    r = np.random.default_rng(3)
    new = np.array([3000, 1, 2, 900, 1, 1, 700])
    old = np.array([0, 77, 10, 3, 64, 63, 130])
    c = Case(2, [int(x) for x in old + new], 1, 8, 0, 16, 64)
    q_seq = np.repeat(np.arange(7), new)
    q_pos = np.concatenate([np.arange(o, o + n) for o, n in zip(old, new)])
    bits = inputs.to_bf16_bits(r.standard_normal((q_seq.size, 576)).astype(np.float32))
    codes, scale = _append(cuda_device, c, bits, q_seq, q_pos)
    want = C.quantize_append(c.codes, c.scale, 16, oracle.bf16_decode(bits), q_seq, q_pos, lambda s, p: int(c.row(s, p)))
    assert np.array_equal(scale, want[1].astype(np.float32)) and _same_codes(codes, want[0])


@pytest.mark.parametrize("T", [1023, 1024, 1025])
def test_append_around_the_short_list_rule_captured(cuda_device, T):
    """Lists at the rule's edge, appended by two captured graphs with a workspace each,
    replayed one after the other on another stream."""
    r = np.random.default_rng(T)
    c = Case(5, [T - 100, 100], 1, 8, 0, 8, 64)
    q_seq = np.repeat([0, 1], [T - 100, 100])
    q_pos = np.concatenate([np.arange(T - 100), np.arange(100)])
    class Host:
        kv_offset, kv_len = c.off, c.lens
    Host.q_seq, Host.q_pos = q_seq.astype(np.int32), q_pos.astype(np.int32)
    db = B.DeviceBatch.from_host(Host, cuda_device, kv_rows=c.rows, page_size=64, page_table=c.table)
    kv8, scale = B.bits_to_tensor(c.codes, cuda_device), B.bits_to_tensor(c.scale, cuda_device)
    bits = [inputs.to_bf16_bits(r.standard_normal((T, 576)).astype(np.float32) * f) for f in (4, 1)]
    kv = [B.bits_to_tensor(x, cuda_device) for x in bits]
    ws = [B.q8_workspace(B.Q8_APPEND, db, device=cuda_device) for _ in range(2)]
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g, x, w in zip(graphs, kv, ws):
        with torch.cuda.graph(g):
            B.dsa_quantize_append(db, x, kv8, scale, 8, w)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        for _ in range(3):
            for g in graphs:
                g.replay()
    torch.cuda.synchronize()
    assert [B.read_device_status(w) for w in ws] == [0, 0]
    want = c.codes, c.scale
    for x in bits:
        want = C.quantize_append(want[0], want[1], 8, oracle.bf16_decode(x), q_seq, q_pos, lambda s, p: int(c.row(s, p)))
    assert np.array_equal(scale.cpu().numpy(), want[1].astype(np.float32)) and _same_codes(kv8.cpu().numpy(), want[0])


@pytest.mark.parametrize("T", [2047, 2048, 2049, 9000])
def test_append_on_both_sides_of_the_search_for_runs(cuda_device, T):
    test_append_around_the_short_list_rule_captured(cuda_device, T)


@pytest.mark.parametrize("page", [0, 64])
@pytest.mark.parametrize("g", [1, 64])
def test_append_many_short_runs(cuda_device, g, page):
    """A long list of one to three tokens per sequence, more runs than CTAs, among them
    runs that are refused (no page, a sequence too short) and ones that raise a scale."""
    r = np.random.default_rng(g)
    n = 1500
    old, new = r.integers(0, 130, n), r.integers(1, 4, n)
    c = Case(6, [int(x) for x in old + new], 1, 8, 0, g, page)
    q_seq = np.repeat(np.arange(n), new)
    q_pos = np.concatenate([np.arange(o, o + k) for o, k in zip(old, new)])
    assert q_seq.size > 2048
    bits = inputs.to_bf16_bits(r.standard_normal((q_seq.size, 576)).astype(np.float32)
                               * np.exp2(r.integers(-6, 6, (q_seq.size, 1))).astype(np.float32))
    bad, flags = np.zeros(n, bool), 0
    c.lens = c.lens.copy()
    c.lens[[5, 700]] = old[[5, 700]]
    bad[[5, 700]], flags = True, B.DEV_BAD_QUERY
    if page:
        c.table[[9, 901], (old // 64)[[9, 901]]] = -1
        whole = old // 64 == (old + new - 1) // 64
        assert whole[[9, 901]].all()
        bad[[9, 901]], flags = True, flags | B.DEV_BAD_INDEX
    codes, scale = _append(cuda_device, c, bits, q_seq, q_pos, flags=flags)
    keep = ~bad[q_seq]
    want = C.quantize_append(c.codes, c.scale, g, oracle.bf16_decode(bits[keep]), q_seq[keep], q_pos[keep],
                             lambda s, p: int(c.row(s, p)))
    assert np.array_equal(scale, want[1].astype(np.float32)) and _same_codes(codes, want[0])


def test_append_extreme_values(cuda_device):
    c = Case(4, [64 * 9], 1, 8, 0, 64, 0)
    kv = np.zeros((64 * 9, 576), np.float32)
    kv[64:128] = 1e-38                                   # needs less than the smallest scale
    kv[128:192] = 3e38                                   # more than the largest: saturates
    kv[192:256] = np.random.default_rng(1).standard_normal((64, 576))
    kv[200, 5], kv[201, 6], kv[202, 7] = np.inf, -np.inf, np.nan
    kv[256:320] = 448.0
    kv[320:384] = 449.0 + 3                              # bf16 452: just above 448
    kv[384:448] = np.inf
    kv[448:512] = np.nan
    kv[512] = -0.0
    bits = inputs.to_bf16_bits(kv)
    codes, scale = _append(cuda_device, c, bits, np.zeros(64 * 9), np.arange(64 * 9))
    want = C.quantize_append(c.codes, c.scale, 64, oracle.bf16_decode(bits), np.zeros(64 * 9), np.arange(64 * 9),
                             lambda s, p: p)
    assert np.array_equal(scale, want[1].astype(np.float32)) and _same_codes(codes, want[0])
    assert scale[4] == 1.0 and scale[5] == 2.0


def test_append_step_by_step_equals_the_definition(cuda_device):
    """Tokens appended one call at a time: the block's scale grows, earlier rows follow."""
    r = np.random.default_rng(6)
    c = Case(5, [80, 70], 1, 8, 0, 32, 64)
    mags = np.exp2(r.integers(-3, 10, 40))
    codes, scale = c.codes, c.scale
    for i in range(40):
        kv = r.standard_normal((2, 576)).astype(np.float32) * np.float32(mags[i])
        bits = inputs.to_bf16_bits(kv)
        pos = [30 + i, 20 + i]
        c.codes, c.scale = codes, scale
        want = C.quantize_append(codes, scale, 32, oracle.bf16_decode(bits), [0, 1], pos, lambda s, p: int(c.row(s, p)))
        codes, scale = _append(cuda_device, c, bits, [0, 1], pos)
        assert np.array_equal(scale, want[1].astype(np.float32)) and _same_codes(codes, want[0])
        scale = scale.astype(np.float32)


def test_append_flags(cuda_device):
    c = Case(7, [100, 90], 1, 8, 0, 16, 64)
    bits = inputs.to_bf16_bits(np.random.default_rng(1).standard_normal((3, 576)).astype(np.float32))
    row = lambda s, p: int(c.row(s, p))  # noqa: E731
    kv = oracle.bf16_decode(bits)
    # beyond the sequence's end: the tokens before it are appended
    codes, scale = _append(cuda_device, c, bits, [0, 0, 0], [98, 99, 100], flags=B.DEV_BAD_QUERY)
    want = C.quantize_append(c.codes, c.scale, 16, kv[:2], [0, 0], [98, 99], row)
    assert np.array_equal(scale, want[1].astype(np.float32)) and _same_codes(codes, want[0])
    # an unknown sequence
    codes, scale = _append(cuda_device, c, bits, [0, 1, 2], [99, 89, 0], flags=B.DEV_BAD_QUERY)
    want = C.quantize_append(c.codes, c.scale, 16, kv[:2], [0, 1], [99, 89], row)
    assert np.array_equal(scale, want[1].astype(np.float32)) and _same_codes(codes, want[0])
    # sequences out of order: the first one is appended
    codes, scale = _append(cuda_device, c, bits[:2], [1, 0], [89, 99], flags=B.DEV_BAD_QUERY)
    want = C.quantize_append(c.codes, c.scale, 16, kv[:1], [1], [89], row)
    assert np.array_equal(scale, want[1].astype(np.float32)) and _same_codes(codes, want[0])
    # a page outside the pool
    c.table[0, 1] = 1 << 20
    codes, scale = _append(cuda_device, c, bits[:2], [0, 1], [99, 89], flags=B.DEV_BAD_INDEX)
    want = C.quantize_append(c.codes, c.scale, 16, kv[1:2], [1], [89], row)
    assert np.array_equal(scale, want[1].astype(np.float32)) and _same_codes(codes, want[0])
    # an earlier scale that is none
    c = Case(8, [100, 90], 1, 8, 0, 16, 64)
    c.scale[row(0, 99) // 16] = np.nan
    codes, scale = _append(cuda_device, c, bits[:1], [0], [99], flags=B.DEV_BAD_SCALE)
    want = C.quantize_append(c.codes, c.scale, 16, kv[:1], [0], [99], row)
    assert np.array_equal(scale, want[1].astype(np.float32)) and _same_codes(codes, want[0])
    # a contiguous sequence that shares a block with its neighbour
    c = Case(9, [100, 90], 1, 8, 0, 16, 0, gap=3)
    codes, scale = _append(cuda_device, c, bits[:1], [0], [99], flags=B.DEV_BAD_QUERY)
    assert np.array_equal(codes, c.codes) and np.array_equal(scale, c.scale)


# ------------------------------------------------------------------- the paths that call them
def test_project_append_q8_equals_project_then_append(cuda_device):
    dev, HI, H, d = cuda_device, 8, 16, 256
    c = Case(30, [150, 70], 3, H, 0, 16, 64)
    n_all = HI * 128 + 128 + HI + 576 + H * 576
    ins = inputs.projection_inputs(c.T, d, n_all)
    hid, w_all = (B.bits_to_tensor(ins[n], dev) for n in ("hidden", "w_all"))
    db = c.batch(dev)
    new = lambda: [torch.zeros((c.T, HI, 128), dtype=torch.uint8, device=dev),  # noqa: E731
                   torch.zeros((c.T, HI), device=dev), torch.zeros((c.T, H, 576), dtype=torch.int16, device=dev),
                   torch.zeros((c.rows, 128), dtype=torch.uint8, device=dev)]
    a, b = new(), new()
    kv = torch.zeros((c.rows, 576), dtype=torch.int16, device=dev)
    ws = B.workspace(B.OP_PROJECT, db, H_I=HI, H=H, device=dev)
    B.dsa_project_append(db, hid, w_all, d, HI, H, 1e4, *a, kv, ws)
    assert B.read_device_status(ws) == 0
    rows = torch.as_tensor(np.concatenate([c.row(s, [p]) for s, p in zip(c.q_seq, c.q_pos)]), device=dev)
    kv8 = [B.bits_to_tensor(c.codes, dev).clone() for _ in range(2)]
    scale = [B.bits_to_tensor(c.scale, dev).clone() for _ in range(2)]
    B.dsa_quantize_append(db, kv[rows].contiguous(), kv8[0], scale[0], 16, ws)
    ws = B.q8_workspace(B.Q8_PROJECT, db, H_I=HI, H=H, device=dev)
    B.dsa_project_append_q8(db, hid, w_all, d, HI, H, 1e4, *b, kv8[1], scale[1], 16, ws)
    assert B.read_device_status(ws) == 0
    for x, y in zip(a + [kv8[0], scale[0]], b + [kv8[1], scale[1]]):
        assert torch.equal(x, y)


@pytest.mark.parametrize("wl", [
    Workload("q8_decode", 61, "decode", k=512, h_index=16, heads=128, batch=3, ctx_min=700, ctx_max=3000, q_per_seq=2),
    Workload("q8_prefill", 62, "prefill", k=128, h_index=4, heads=16, seq_len=400)], ids=lambda w: w.name)
def test_forward_q8_is_indexer_topk_and_attention(cuda_device, wl):
    dev = cuda_device
    ins = inputs.make_inputs(wl)
    bh = ins["batch"]
    c = Case(31, [int(x) for x in bh.kv_len], 1, wl.heads, 0, 64, 0)
    c.q_seq, c.q_pos, c.q, c.T, c.k = bh.q_seq, bh.q_pos, ins["q"], bh.num_q, wl.k
    db = c.batch(dev)
    k_idx = np.zeros((c.rows, 128), np.uint8)
    for b in range(bh.num_seqs):
        k_idx[c.off[b]:c.off[b] + c.lens[b]] = ins["k_idx"][bh.kv_offset[b]:bh.kv_offset[b] + c.lens[b]]
    t = {n: B.bits_to_tensor(x, dev) for n, x in (("q_idx", ins["q_idx"]), ("k_idx", k_idx), ("w", ins["w"]),
                                                   ("q", c.q), ("kv8", c.codes), ("scale", c.scale))}
    ld = (int(c.lens.max()) + 3) // 4 * 4
    scores = torch.zeros((c.T, ld), device=dev)
    idx = torch.zeros((c.T, wl.k), dtype=torch.int32, device=dev)
    ws = B.workspace(B.OP_INDEXER, db, H_I=wl.h_index, H=wl.heads, k=wl.k, device=dev)
    B.dsa_indexer_scores(db, t["q_idx"], t["k_idx"], t["w"], wl.h_index, scores, ld, ws)
    B.dsa_topk(db, scores, ld, wl.k, idx, ws)
    c.idx = idx.cpu().numpy()
    ref = c.run(dev)
    out = torch.zeros((c.T, wl.heads, 512), dtype=torch.int16, device=dev)
    lse = torch.zeros((c.T, wl.heads), device=dev)
    ws = B.q8_workspace(B.Q8_FORWARD, db, H_I=wl.h_index, H=wl.heads, k=wl.k, device=dev)
    B.dsa_forward_q8(db, t["q_idx"], t["k_idx"], t["w"], wl.h_index, t["q"], t["kv8"], t["scale"], 64, wl.heads, wl.k,
                     SM, out, lse, ws)
    assert B.read_device_status(ws) == 0
    assert np.array_equal(B.tensor_to_bits(out), ref[0]) and np.array_equal(lse.cpu().numpy(), ref[1])
    c.check(*ref, rows=range(0, c.T, max(1, c.T // 20)))
