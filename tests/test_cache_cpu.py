"""Host-side checks of the 8-bit cache's and the page calls' entry points: bad
arguments are refused before anything is launched (addresses are never followed)."""
from __future__ import annotations

import ctypes
import os
import re

import pytest

from sparse_attention_weight_b200 import binding as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P, WS, BIG = 0x60000, 0x50000, 1 << 40


@pytest.fixture(scope="module")
def lib():
    from sparse_attention_weight_b200 import build
    build.build()
    return B.lib()


def _batch(T=16, page_size=0, pps=0, table=0, kv_rows=6016):
    return B.DsaBatch(2, T, 3000, 0, kv_rows, 0x10000, 0x20000, 0x30000, 0x40000, page_size, pps, table)


def _state(seqs=4, pages=100, page_size=64, pps=8, table=0x10000, lens=0x20000, refs=0x30000):
    return B.DsaPageState(seqs, pages, page_size, pps, table, lens, refs)


def test_constants_match_the_header():
    src = open(os.path.join(ROOT, "include", "dsa.h")).read()
    defs = {n: int(v) for n, v in re.findall(r"^#define (DSA_\w+) (\d+)u?\b", src, flags=re.M)}
    assert defs["DSA_DEV_BAD_SCALE"] == B.DEV_BAD_SCALE and defs["DSA_DEV_NO_PAGES"] == B.DEV_NO_PAGES
    assert [defs["DSA_Q8_" + n] for n in ("APPEND", "MLA", "FORWARD", "PROJECT")] == [
        B.Q8_APPEND, B.Q8_MLA, B.Q8_FORWARD, B.Q8_PROJECT]
    assert defs["DSA_MAX_PAGE_BUFFERS"] == B.MAX_PAGE_BUFFERS
    assert ctypes.sizeof(B.DsaPageState) == 40 and ctypes.sizeof(B.DsaPageBuffers) == 8 + 16 * B.MAX_PAGE_BUFFERS


def test_q8_workspace_sizes(lib):
    b = _batch()
    sz = lambda op, hi=64, h=128, k=2048: lib.dsa_q8_workspace_size(op, ctypes.byref(b), hi, h, k)  # noqa: E731
    assert sz(B.Q8_APPEND, 0, 0, 0) >= 256 and sz(B.Q8_MLA, 0, 128, 0) >= 256
    assert sz(B.Q8_FORWARD) >= 16 * 3000 * 4 + 16 * 2048 * 4
    assert sz(B.Q8_PROJECT) >= 16 * 576 * 2 + lib.dsa_workspace_size(B.OP_PROJECT, ctypes.byref(b), 64, 128, 0, 0)
    for bad in (sz(4), sz(-1), sz(B.Q8_MLA, h=12), sz(B.Q8_MLA, k=2049), sz(B.Q8_MLA, k=-1), sz(B.Q8_FORWARD, k=0),
                sz(B.Q8_FORWARD, hi=10), sz(B.Q8_PROJECT, hi=6), lib.dsa_q8_workspace_size(1, None, 64, 128, 1)):
        assert bad == 0


def test_quantize_append_host_checks(lib):
    def call(b=None, kv=P, kv8=P, scale=P, g=64, ws=WS, n=BIG):
        b = b or _batch()
        return lib.dsa_quantize_append(ctypes.byref(b), kv, kv8, scale, g, ws, n, None)
    assert lib.dsa_quantize_append(None, P, P, P, 64, WS, BIG, None) == 1
    assert call(kv=0) == 1 and call(kv8=0) == 1 and call(scale=0) == 1 and call(ws=0) == 1
    for g in (0, -1, 3, 48, 128):
        assert call(g=g) == 2
    assert call(kv=P + 2) == 2 and call(kv8=P + 8) == 2 and call(ws=WS + 4) == 2
    assert call(b=_batch(page_size=32, pps=94, table=P)) == 2       # pages of a multiple of 64
    assert call(n=255) == 3


def test_sparse_mla_q8_host_checks(lib):
    def call(b=None, q=P, kv8=P, scale=P, g=64, idx=P, k=2048, H=128, sm=0.1, out=P, ws=WS, n=BIG):
        b = b or _batch()
        return lib.dsa_sparse_mla_q8(ctypes.byref(b), q, kv8, scale, g, idx, k, H, sm, out, None, ws, n, None)
    assert call(q=0) == 1 and call(kv8=0) == 1 and call(scale=0) == 1 and call(out=0) == 1 and call(ws=0) == 1
    assert call(sm=float("inf")) == 1 and call(sm=float("nan")) == 1
    assert call(H=12) == 2 and call(H=136) == 2 and call(k=0) == 2 and call(k=2049) == 2
    assert call(idx=0) == 2                                          # the dense form takes k = 0
    assert call(g=5) == 2 and call(q=P + 8) == 2 and call(out=P + 4) == 2 and call(kv8=P + 4) == 2
    assert call(b=_batch(page_size=128, pps=24, table=P, kv_rows=8000)) == 2
    assert call(n=128) == 3 and call(idx=0, k=0, n=128) == 3


def test_forward_and_project_q8_host_checks(lib):
    b = _batch()
    fwd = lambda **a: lib.dsa_forward_q8(  # noqa: E731
        ctypes.byref(b), a.get("qi", P), P, P, a.get("hi", 64), P, a.get("kv8", P), P, a.get("g", 64), 128,
        a.get("k", 2048), a.get("sm", 0.1), P, None, WS, a.get("n", BIG), None)
    assert fwd(qi=0) == 1 and fwd(kv8=0) == 1 and fwd(sm=float("nan")) == 1
    assert fwd(hi=10) == 2 and fwd(g=7) == 2 and fwd(k=0) == 2 and fwd(n=1024) == 3
    prj = lambda **a: lib.dsa_project_append_q8(  # noqa: E731
        ctypes.byref(b), a.get("h", P), P, a.get("d", 7168), 64, 128, a.get("base", 1e4), P, P, P, P,
        a.get("kv8", P), a.get("scale", P), a.get("g", 64), WS, a.get("n", BIG), None)
    assert prj(h=0) == 1 and prj(kv8=0) == 1 and prj(scale=0) == 1 and prj(base=0.0) == 1
    assert prj(d=7170) == 2 and prj(g=0) == 2 and prj(kv8=P + 8) == 2 and prj(n=1024) == 3


def test_pages_host_checks(lib):
    s, o = _state(), _state(table=0x40000, lens=0x70000, refs=0x80000)
    size = lib.dsa_pages_workspace_size(ctypes.byref(s), 10)
    assert size >= 256 + 100 * 4
    for bad in (_state(seqs=0), _state(pages=0), _state(page_size=32), _state(page_size=96), _state(pps=0),
                _state(page_size=1 << 20, pps=1 << 12)):
        assert lib.dsa_pages_workspace_size(ctypes.byref(bad), 1) == 0
    assert lib.dsa_pages_workspace_size(ctypes.byref(s), -1) == 0 and lib.dsa_pages_workspace_size(None, 1) == 0

    def resize(a=s, b=o, n=4, l1=P, l2=P, bufs=None, ws=WS, nb=BIG):
        return lib.dsa_pages_resize(ctypes.byref(a), ctypes.byref(b), n, l1, l2, bufs, ws, nb, None)
    assert resize(n=-1) == 1 and resize(l1=0) == 1 and resize(l2=0) == 1 and resize(ws=0) == 1
    assert resize(a=_state(table=0)) == 1 and resize(b=_state(refs=0)) == 1
    assert resize(b=_state(seqs=5)) == 1 and resize(b=_state(pages=99)) == 1 and resize(b=_state(page_size=128)) == 1
    assert resize(b=_state(lens=0x70000)) == 1                       # in place, or wholly apart
    assert resize(a=_state(page_size=32), b=_state(page_size=32)) == 2
    assert resize(ws=WS + 4) == 2
    assert resize(nb=size - 1 - 6 * 16) == 3

    def bufs(*parts):
        t = B.DsaPageBuffers()
        t.num = len(parts)
        for j, (base, n) in enumerate(parts):
            t.base[j], t.page_bytes[j] = base, n
        return t
    assert resize(bufs=bufs((0, 64))) == 1 and resize(bufs=bufs((P, 0))) == 1
    assert resize(bufs=bufs((P, 66))) == 2 and resize(bufs=bufs((P + 2, 64))) == 2
    many = bufs()
    many.num = 9
    assert resize(bufs=many) == 1
    assert lib.dsa_pages_fork(ctypes.byref(s), ctypes.byref(o), 2, 0, P, WS, BIG, None) == 1
    assert lib.dsa_pages_fork(ctypes.byref(s), ctypes.byref(o), 2, P, P, WS, 300, None) == 3
    assert lib.dsa_pages_compact(ctypes.byref(s), None, None, None, WS, BIG, None) == 1
    assert lib.dsa_pages_compact(ctypes.byref(s), ctypes.byref(o), bufs((P, 6)), None, WS, BIG, None) == 2


def test_page_sums_stay_in_32_bits(lib):
    big, fits = _state(seqs=1 << 16, pps=1 << 15), _state(seqs=(1 << 16) - 2, pps=1 << 15)
    assert lib.dsa_pages_workspace_size(ctypes.byref(fits), 1) > 0
    assert lib.dsa_pages_workspace_size(ctypes.byref(big), 1) == 0
    assert lib.dsa_pages_resize(ctypes.byref(big), ctypes.byref(big), 1, P, P, None, WS, BIG, None) == 2
    assert lib.dsa_pages_fork(ctypes.byref(big), ctypes.byref(big), 1, P, P, WS, BIG, None) == 2
    assert lib.dsa_pages_compact(ctypes.byref(big), ctypes.byref(big), None, None, WS, BIG, None) == 2


def test_binding_takes_the_current_device_only(monkeypatch):
    """Tensors of another device (here: the CPU's, with device 0 current), strided ones and
    page buffers of another pool size are refused before the library is called."""
    import numpy as np
    import torch
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(B, "_stream", lambda s: None)

    class NoCall:
        def __getattr__(self, name):
            return lambda *a: pytest.fail(name + " was called")
    monkeypatch.setattr(B, "lib", lambda: NoCall())

    class Host:
        kv_offset, kv_len, q_seq, q_pos = np.array([0]), np.array([8]), np.array([0]), np.array([7])
    b = B.DeviceBatch.from_host(Host, "cpu")
    x = torch.zeros(64, dtype=torch.int32)
    s = B.PageState.empty(2, 4, 64, 2, device="cpu")
    bufs = B.PageBuffers([torch.zeros(8, 4)], 4)
    calls = [lambda: B.dsa_quantize_append(b, x, x, x, 1, x),
             lambda: B.dsa_project_append_q8(b, x, x, 8, 4, 8, 1e4, x, x, x, x, x, x, 1, x),
             lambda: B.dsa_sparse_mla_q8(b, x, x, x, 1, None, 0, 8, 1.0, x, None, x),
             lambda: B.dsa_forward_q8(b, x, x, x, 4, x, x, x, 1, 8, 4, 1.0, x, None, x),
             lambda: B.dsa_pages_resize(s, s, x, x, None, x),
             lambda: B.dsa_pages_fork(s, s, x, x, x),
             lambda: B.dsa_pages_compact(s, s, None, None, x)]
    for call in calls:
        with pytest.raises(ValueError, match="current CUDA device"):
            call()
    with pytest.raises(ValueError, match="another number of pages"):
        B._buffers(bufs, B.PageState.empty(2, 8, 64, 2, device="cpu"), -1)
    with pytest.raises(ValueError, match="contiguous"):
        B._dev(torch.zeros(4, 4).t()[1:], -1)


def test_batches_and_states_of_mixed_devices_are_refused():
    import torch
    lists = [torch.zeros(2, dtype=torch.int32) for _ in range(2)]
    on_cpu = B.PageState.empty(2, 4, 64, 2, device="cpu")
    assert B.DeviceBatch.from_pages(on_cpu, *lists, 128).struct.kv_rows == 256
    on_cpu.device = 0                                    # as if its arrays lay on a GPU
    with pytest.raises(ValueError, match="page state's device"):
        B.DeviceBatch.from_pages(on_cpu, *lists, 128)
    meta = torch.zeros(2, dtype=torch.int32, device="meta")
    meta.get_device = lambda: 0
    with pytest.raises(ValueError, match="one device"):
        B.PageState(torch.zeros(2, 2, dtype=torch.int32), meta, torch.zeros(4, dtype=torch.int32), 64)
    on_cpu.device = -1
    with pytest.raises(ValueError, match="one length"):
        B.DeviceBatch.from_pages(on_cpu, lists[0], lists[1][:1], 128)
