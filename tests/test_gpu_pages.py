"""The page calls on the GPU against the sequential oracle: all results are whole
numbers and copied bytes, so they must be equal."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
from oracle import cache as C
from sparse_attention_weight_b200 import binding as B
from sparse_attention_weight_b200 import build, inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    B.lib()


def _pool(r, S, N, P, pps, filled, live):
    table = np.full((S, pps), -1, np.int32)
    lens = np.zeros(S, np.int32)
    refs = np.zeros(N, np.int32)
    perm, at = r.permutation(N), 0
    for s in filled:
        w = int(min(r.integers(0, pps, endpoint=True), live - at, N - at))
        table[s, :w] = perm[at:at + w]
        lens[s] = 0 if w <= 0 else (w - 1) * P + int(r.integers(1, P, endpoint=True))
        refs[perm[at:at + w]] += 1
        at += max(0, w)
    return table, lens, refs


class Dev:
    """A pool on the device beside its oracle, with page data."""

    def __init__(self, dev, table, lens, refs, P, sizes=(576 * 64, 4, 132), in_place=False, seed=0):
        self.dev, self.P = dev, P
        self.ref = C.Pool(table, lens, refs, P)
        up = lambda x: torch.as_tensor(np.array(x, np.int32), device=dev)  # noqa: E731
        self.state = B.PageState(up(table), up(lens), up(refs), P)
        self.in_place = in_place
        r = np.random.default_rng(seed)
        self.data = [r.integers(0, 256, size=(len(refs), n)).astype(np.uint8) for n in sizes]
        self.bufs = [torch.as_tensor(x, device=dev) for x in self.data]
        self.buffers = B.PageBuffers(self.bufs, len(refs))

    def dst(self):
        return self.state if self.in_place else self.state.like()

    def copied(self, copies):
        for a, b in copies:
            for x in self.data:
                x[b] = x[a]

    def check(self, out, ws, flags=0):
        assert B.read_device_status(ws) == flags
        for got, want in ((out.page_table, self.ref.table), (out.seq_len, self.ref.lens), (out.ref_count, self.ref.refs)):
            assert np.array_equal(got.cpu().numpy(), want)
        for got, want in zip(self.bufs, self.data):
            assert np.array_equal(got.cpu().numpy(), want)
        self.state = out

    def resize(self, seqs, lens, flags=0):
        a, b = (torch.as_tensor(np.array(x, np.int32), device=self.dev) for x in (seqs, lens))
        ws, out = B.pages_workspace(self.state, len(seqs), device=self.dev), self.dst()
        B.dsa_pages_resize(self.state, out, a, b, self.buffers, ws)
        self.copied(self.ref.resize(seqs, lens))
        self.check(out, ws, flags)

    def fork(self, src, dst, flags=0):
        a, b = (torch.as_tensor(np.array(x, np.int32), device=self.dev) for x in (src, dst))
        ws, out = B.pages_workspace(self.state, len(src), device=self.dev), self.dst()
        B.dsa_pages_fork(self.state, out, a, b, ws)
        self.ref.fork(src, dst)
        self.check(out, ws, flags)

    def compact(self, with_map=True):
        ws, out = B.pages_workspace(self.state, 0, device=self.dev), self.dst()
        n = len(self.ref.refs)
        m = torch.full((n,), 5, dtype=torch.int32, device=self.dev) if with_map else None
        B.dsa_pages_compact(self.state, out, self.buffers, m, ws)
        want, copies = self.ref.compact()
        self.copied(copies)
        self.check(out, ws)
        if with_map:
            assert np.array_equal(m.cpu().numpy(), want)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("S,N,P,pps", [(1, 1, 64, 1), (3, 10, 64, 4), (7, 1025, 128, 33), (64, 4099, 64, 70),
                                       (1500, 9000, 192, 5)])
def test_random_calls(cuda_device, S, N, P, pps, in_place):
    r = np.random.default_rng(S + N)
    d = Dev(cuda_device, *_pool(r, S, N, P, pps, range(0, S, 2), N // 2), P, sizes=(576, 4, 132, 1024),
            in_place=in_place)
    for step in range(24):
        what = int(r.integers(4))
        if what <= 1:
            n = int(r.integers(1, S, endpoint=True))
            seqs = r.permutation(S)[:n]
            now = d.ref.lens[seqs].astype(np.int64)
            top = pps * P
            lens = np.where(r.random(n) < 0.4, r.integers(0, now + 1), np.minimum(now + r.integers(0, 2 * P, n), top))
            d.ref.no_pages = False
            probe = C.Pool(d.ref.table, d.ref.lens, d.ref.refs, P)
            probe.resize(seqs, lens)
            d.resize(seqs, lens, flags=B.DEV_NO_PAGES if probe.no_pages else 0)
        elif what == 2:
            empty = np.flatnonzero(d.ref.lens == 0)
            full = np.flatnonzero(d.ref.lens > 0)
            if empty.size and full.size:
                n = int(r.integers(1, empty.size, endpoint=True))
                d.fork(r.choice(full, n), r.permutation(empty)[:n])
        else:
            d.compact(with_map=bool(step % 2))


def test_copy_on_write_of_shared_last_pages(cuda_device):
    """Four holders of a partly filled page: three grow and one does not; then all do."""
    P, S, N, pps = 64, 6, 30, 4
    table = np.full((S, pps), -1, np.int32)
    table[0, :2] = [9, 4]
    lens = np.array([100, 0, 0, 0, 0, 0], np.int32)
    refs = np.zeros(N, np.int32)
    refs[[9, 4]] = 1
    d = Dev(cuda_device, table, lens, refs, P)
    d.fork([0, 0, 0], [3, 1, 2])
    d.resize([2, 0, 3], [101, 130, 128])                 # every one of them copies, sequence 1 keeps page 4
    assert int(d.ref.table[1, 1]) == 4 and d.ref.refs[4] == 1
    d.fork([1, 1], [4, 5])
    d.resize([4, 1, 5], [101, 128, 200])                 # the last one listed keeps it
    assert int(d.ref.table[5, 1]) == 4
    d.resize([5, 4], [70, 0])
    d.fork([5], [4])
    d.resize([5, 4], [20, 71])                           # one leaves the page in the same call: no copy
    assert int(d.ref.table[4, 1]) == 4
    d.resize([0, 5], [192, 64])                          # full pages need no copy


def test_lists_are_checked(cuda_device):
    P, S, N, pps = 64, 5, 12, 3
    d = Dev(cuda_device, *_pool(np.random.default_rng(0), S, N, P, pps, [0, 1], 6), P)
    d.resize([0, 4, 0, -1, 5, 2, 3], [10, 64, 100, 5, 5, 193, -1], flags=B.DEV_BAD_QUERY)
    d.fork([0, 0, 0, 1, 4, -1, 0], [3, 3, 4, 0, 2, 2, 9], flags=B.DEV_BAD_QUERY)
    d.resize([], [])
    d.fork([], [])


def test_too_few_pages_grow_nobody(cuda_device):
    P, S, N, pps = 64, 4, 5, 4
    d = Dev(cuda_device, *_pool(np.random.default_rng(0), S, N, P, pps, [], 0), P)
    d.resize([0, 1], [128, 128])
    d.resize([0, 1, 2], [64, 200, 128], flags=B.DEV_NO_PAGES)       # one page comes back, three are wanted
    d.resize([2], [128])
    d.resize([3], [1], flags=B.DEV_NO_PAGES)


def test_table_entries_outside_the_pool_are_left_alone(cuda_device):
    P, S, N, pps = 64, 3, 8, 4
    table = np.full((S, pps), -1, np.int32)
    table[0] = [1, 99, 2, -7]
    lens = np.array([230, 0, 0], np.int32)
    refs = np.zeros(N, np.int32)
    refs[[1, 2]] = 1
    up = lambda x: torch.as_tensor(np.array(x, np.int32), device=cuda_device)  # noqa: E731
    src = B.PageState(up(table), up(lens), up(refs), P)
    dst = src.like()
    ws = B.pages_workspace(src, 4, device=cuda_device)
    B.dsa_pages_resize(src, dst, up([0]), up([10]), None, ws)
    assert B.read_device_status(ws) == B.DEV_BAD_INDEX
    assert dst.page_table.cpu().tolist()[0] == [1, 99, -1, -7] and dst.seq_len.cpu().tolist() == [10, 0, 0]
    assert dst.ref_count.cpu().tolist() == [0, 1, 0, 0, 0, 0, 0, 0]
    B.dsa_pages_resize(src, dst, up([0]), up([240]), None, ws)      # the last page is outside: no copy
    assert B.read_device_status(ws) == B.DEV_BAD_INDEX
    assert dst.page_table.cpu().tolist()[0] == table[0].tolist() and dst.seq_len.cpu().tolist() == [240, 0, 0]
    B.dsa_pages_fork(src, dst, up([0]), up([2]), ws)
    assert B.read_device_status(ws) == B.DEV_BAD_INDEX
    assert dst.page_table.cpu().tolist()[2] == table[0].tolist() and dst.ref_count.cpu().tolist()[1:3] == [2, 2]
    B.dsa_pages_compact(src, dst, None, None, ws)
    assert B.read_device_status(ws) == B.DEV_BAD_INDEX
    assert dst.page_table.cpu().tolist()[0] == [1, 99, 0, -7]


def test_compact_of_empty_full_and_large_pools(cuda_device):
    for live in (0, 1, 5000, 10000):
        r = np.random.default_rng(live)
        d = Dev(cuda_device, *_pool(r, 100, 10000, 64, 200, range(100), live), 64, sizes=(64,))
        d.compact()


def test_many_entries(cuda_device):
    """More list entries than the planning CTA has threads, and more pages than one pass takes."""
    r = np.random.default_rng(1)
    d = Dev(cuda_device, *_pool(r, 3000, 40000, 64, 16, range(1500), 12000), 64, sizes=(16,))
    d.fork(r.integers(0, 1500, 1200), 1500 + r.permutation(1500)[:1200])
    seqs = r.permutation(3000)[:2500]
    lens = np.minimum(d.ref.lens[seqs] + r.integers(-300, 300, 2500), 16 * 64).clip(0)
    d.resize(seqs, lens)
    d.compact()


def test_pool_beyond_32_bit_offsets(cuda_device):
    free, _ = torch.cuda.mem_get_info()
    if free < 12 << 30:
        pytest.skip("needs 12 GB of free device memory")
    N, P, n = 131072, 64, 576 * 64                       # 4.8 GB
    buf = torch.zeros((N, n), dtype=torch.uint8, device=cuda_device)
    table = np.full((2, 4), -1, np.int32)
    table[0] = [N - 1, N - 2, 7, N - 5]
    lens = np.array([250, 0], np.int32)
    refs = np.zeros(N, np.int32)
    refs[table[0]] = 1
    for i, pg in enumerate(table[0]):
        buf[int(pg)] = i + 1
    up = lambda x: torch.as_tensor(np.array(x, np.int32), device=cuda_device)  # noqa: E731
    st = B.PageState(up(table), up(lens), up(refs), P)
    ws = B.pages_workspace(st, 4, device=cuda_device)
    B.dsa_pages_compact(st, st, B.PageBuffers([buf], N), None, ws)
    assert B.read_device_status(ws) == 0
    got = st.page_table.cpu().tolist()[0]
    assert sorted(got) == [0, 1, 2, 3]
    for i, pg in enumerate(got):
        assert (buf[pg] == i + 1).all()


def test_captured_step(cuda_device):
    """A captured decode step (grow by a token, in place): each replay grows again."""
    P, S, N, pps = 64, 4, 16, 4
    st = B.PageState.empty(S, N, P, pps, device=cuda_device)
    ws = B.pages_workspace(st, S, device=cuda_device)
    seqs = torch.arange(S, dtype=torch.int32, device=cuda_device)
    lens = torch.full((S,), 62, dtype=torch.int32, device=cuda_device)
    B.dsa_pages_resize(st, st, seqs, lens, None, ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lens.add_(1)
        B.dsa_pages_resize(st, st, seqs, lens, None, ws)
    for _ in range(4):
        g.replay()
    assert B.read_device_status(ws) == 0
    assert st.seq_len.cpu().tolist() == [66] * S and int(st.ref_count.sum()) == 8
    assert st.page_table.cpu()[:, :2].tolist() == [[0, 4], [1, 5], [2, 6], [3, 7]]


# ------------------------------------------------------------------- together
def test_serving_run(cuda_device):
    """Prompts, appends, a fork, steps that diverge, a freed sequence and a compaction:
    at every step the attention over the paged 8-bit cache is that of the rows that
    were appended (kept apart on the host)."""
    from .test_gpu_cache import Case, SM
    dev, P, S, N, pps, H, g = cuda_device, 64, 6, 40, 6, 16, 16
    r = np.random.default_rng(7)
    st = B.PageState.empty(S, N, P, pps, device=dev)
    kv8 = torch.zeros((N * P, 576), dtype=torch.uint8, device=dev)
    scale = torch.ones(N * P // g, device=dev)
    bufs = B.PageBuffers([kv8, scale], N)
    ws = B.pages_workspace(st, S, device=dev)
    up = lambda x: torch.as_tensor(np.array(x, np.int32), device=dev)  # noqa: E731
    host = {s: (np.zeros((pps * P, 576), np.uint8), np.ones(pps * P // g), 0) for s in range(S)}

    def append(new):                                     # {sequence: tokens}
        seqs = sorted(new)
        old = [host[s][2] for s in seqs]
        B.dsa_pages_resize(st, st, up(seqs), up([o + new[s] for o, s in zip(old, seqs)]), bufs, ws)
        assert B.read_device_status(ws) == 0
        q_seq = np.repeat(seqs, [new[s] for s in seqs])
        q_pos = np.concatenate([np.arange(o, o + new[s]) for o, s in zip(old, seqs)])
        kv = r.standard_normal((q_seq.size, 576)).astype(np.float32) * np.exp2(r.integers(-2, 3, (q_seq.size, 1))).astype(np.float32)
        bits = inputs.to_bf16_bits(kv)
        db = B.DeviceBatch.from_pages(st, up(q_seq), up(q_pos), pps * P)
        wa = B.q8_workspace(B.Q8_APPEND, db, device=dev)
        B.dsa_quantize_append(db, B.bits_to_tensor(bits, dev), kv8, scale, g, wa)
        assert B.read_device_status(wa) == 0
        for s, o in zip(seqs, old):
            mine = q_seq == s
            codes, sc = C.quantize_append(host[s][0], host[s][1], g, oracle.bf16_decode(bits[mine]), q_seq[mine],
                                          q_pos[mine], lambda _, p: p)
            host[s] = (codes, sc, o + new[s])

    def attend():
        live = [s for s in range(S) if host[s][2]]
        q = inputs.to_bf16_bits(r.standard_normal((len(live), H, 576)).astype(np.float32))
        db = B.DeviceBatch.from_pages(st, up(live), up([host[s][2] - 1 for s in live]), pps * P)
        out = torch.zeros((len(live), H, 512), dtype=torch.int16, device=dev)
        lse = torch.zeros((len(live), H), device=dev)
        wm = B.q8_workspace(B.Q8_MLA, db, H=H, k=0, device=dev)
        B.dsa_sparse_mla_q8(db, B.bits_to_tensor(q, dev), kv8, scale, g, None, 0, H, SM, out, lse, wm)
        assert B.read_device_status(wm) == 0
        for i, s in enumerate(live):
            c = Case(0, [host[s][2]], 1, H, 0, g, 0)
            c.codes = np.concatenate([host[s][0], c.codes])[:max(c.rows, pps * P)]
            c.scale = host[s][1].astype(np.float32)
            c.q = q[i:i + 1]
            c.check(B.tensor_to_bits(out)[i:i + 1], lse.cpu().numpy()[i:i + 1])

    append({0: 100, 1: 7, 2: 200})
    attend()
    B.dsa_pages_fork(st, st, up([0, 0]), up([3, 4]), ws)
    host[3], host[4] = host[0], host[0]
    attend()
    for step in range(4):
        append({0: 1, 1: 1, 3: 2, 4: 1})
    attend()
    B.dsa_pages_resize(st, st, up([2, 0]), up([0, 70]), bufs, ws)   # freed, and cut
    host[2] = (host[2][0], host[2][1], 0)
    host[0] = (host[0][0], host[0][1], 70)
    attend()
    B.dsa_pages_compact(st, st, bufs, None, ws)
    assert B.read_device_status(ws) == 0
    attend()
    append({0: 60, 1: 1, 5: 130})
    attend()
    used = int((st.ref_count > 0).sum())
    assert used == len({int(p) for s in range(S) for p in st.page_table[s, :-(-host[s][2] // P)].cpu()})


@pytest.mark.parametrize("n", [1023, 1024, 1025])
@pytest.mark.parametrize("in_place", [False, True])
def test_lists_around_one_pass(cuda_device, n, in_place):
    """As many entries as a pass of the planning threads takes, and one more or fewer, with
    a repeated sequence at the end."""
    r = np.random.default_rng(n)
    d = Dev(cuda_device, *_pool(r, 1100, 5000, 64, 4, range(0, 1100, 2), 2500), 64, sizes=(132,), in_place=in_place)
    seqs = r.permutation(1100)[:n]
    seqs[-1] = seqs[3]
    lens = r.integers(0, 2 * 64, n)
    d.resize(seqs, lens, flags=B.DEV_BAD_QUERY)
    d.compact()


@pytest.mark.parametrize("in_place", [False, True])
def test_compaction_of_more_pages_than_shared_memory_has_masks_for(cuda_device, in_place):
    r = np.random.default_rng(1)
    N = 131072 + 77
    d = Dev(cuda_device, *_pool(r, 40, N, 64, 2000, range(40), 60000), 64, sizes=(4, 16), in_place=in_place)
    d.compact()
    d.resize(np.arange(0, 40, 3), np.zeros(14, np.int64))
    d.compact(with_map=False)


def test_two_captured_steps_in_place_on_another_stream(cuda_device):
    """Fork, growth with copies, and compaction of one pool in place, captured as two graphs
    and replayed on a side stream."""
    P, S, N, pps = 64, 8, 64, 6
    r = np.random.default_rng(2)
    table, lens, refs = _pool(r, S, N, P, pps, range(4), 20)
    lens[0], table[0, :2] = 100, [60, 61]
    refs[:] = 0
    lens[1:4] = 0
    refs[[60, 61]] = 1
    d = Dev(cuda_device, table, lens, refs, P, in_place=True)
    up = lambda x: torch.as_tensor(np.array(x, np.int32), device=cuda_device)  # noqa: E731
    a, b, c, e = up([0, 0]), up([5, 6]), up([5, 6, 0]), up([130, 101, 128])
    ws = [B.pages_workspace(d.state, 3, device=cuda_device) for _ in range(3)]
    torch.cuda.synchronize()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        B.dsa_pages_fork(d.state, d.state, a, b, ws[0])
        B.dsa_pages_resize(d.state, d.state, c, e, d.buffers, ws[1])
    with torch.cuda.graph(g2):
        B.dsa_pages_compact(d.state, d.state, d.buffers, None, ws[2])
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        g1.replay()
        g2.replay()
    torch.cuda.synchronize()
    d.ref.fork([0, 0], [5, 6])
    d.copied(d.ref.resize([5, 6, 0], [130, 101, 128]))
    d.copied(d.ref.compact()[1])
    assert [B.read_device_status(w) for w in ws] == [0, 0, 0]
    d.check(d.state, ws[2])


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("N", [49152, 49153, 120001])
def test_resize_of_pools_around_what_shared_memory_holds(cuda_device, N, in_place):
    r = np.random.default_rng(N)
    S, P, pps = 300, 64, 700
    d = Dev(cuda_device, *_pool(r, S, N, P, pps, range(0, S, 2), N // 2), P, sizes=(4, 132), in_place=in_place)
    d.fork(np.arange(0, 20, 2), np.arange(1, 21, 2))
    for _ in range(4):
        n = int(r.integers(1, S))
        seqs = r.permutation(S)[:n]
        now = d.ref.lens[seqs].astype(np.int64)
        lens = np.where(r.random(n) < 0.4, r.integers(0, now + 1), np.minimum(now + r.integers(0, 3000, n), pps * P))
        probe = C.Pool(d.ref.table, d.ref.lens, d.ref.refs, P)
        probe.resize(seqs, lens)
        d.resize(seqs, lens, flags=B.DEV_NO_PAGES if probe.no_pages else 0)


def test_sequences_that_meet_in_the_hash_table(cuda_device):
    """Many entries of few sequences, sequences far apart, and every sequence twice."""
    r = np.random.default_rng(5)
    S = 200000
    d = Dev(cuda_device, np.full((S, 1), -1, np.int32), np.zeros(S, np.int32), np.zeros(3000, np.int32), 64, sizes=(4,))
    seqs = (np.arange(1024, dtype=np.int64) * 2048 * 97) % S
    seqs = np.concatenate([np.unique(seqs)[:500], np.unique(seqs)[:500], [7] * 24])
    d.resize(r.permutation(seqs), r.integers(0, 65, seqs.size), flags=B.DEV_BAD_QUERY)
    d.resize(np.arange(1024) * 190, r.integers(0, 65, 1024))
