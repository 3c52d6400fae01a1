"""The 8-bit latent cache and its pages, as cases that can be measured.

Each case names one operator ("op") and its sizes.  ``run`` computes it either
in plain torch operations in 32 bits (``own`` false) or through this
repository's library (``own`` true); ``exact`` computes it from its definition
in 64 bits.

The cache: row r holds 576 E4M3 codes (512 latent + 64 RoPE), its value is
``scale[r // g]`` times the codes, g = scale_block tokens.  The scales are
powers of two.  A paged cache maps key s of sequence b to row
``table[b, s // P] * P + s % P``.
"""
import math

import numpy as np
import torch

D_QK, D_V, D_INDEX = 576, 512, 128
E4M3_MAX = 448.0
MIN_EXP, MAX_EXP = -100, 100          # exponents that a block's scale can take
SM_SCALE = 1.0 / math.sqrt(D_QK)

own = False


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one new token of one sequence at 131072, rows picked by the top-k: the least work a step can have
        {"name": "mla decode 1 x 128K", "op": "mla", "seqs": 1, "q_per_seq": 1, "ctx_min": 131072, "ctx_max": 131072,
         "heads": 128, "k": 2048, "g": 64, "page": 64, "dense": False},
        # a serving batch of mixed contexts, one token each
        {"name": "mla decode 64 x 4K-32K", "op": "mla", "seqs": 64, "q_per_seq": 1, "ctx_min": 4096,
         "ctx_max": 32768, "heads": 128, "k": 2048, "g": 64, "page": 64, "dense": False},
        # a chunk of a long prompt: queries of one sequence at the end of a 64K context
        {"name": "mla prefill chunk 4096", "op": "mla", "seqs": 1, "q_per_seq": 4096, "ctx_min": 65536,
         "ctx_max": 65536, "heads": 128, "k": 2048, "g": 64, "page": 0, "dense": False},
        # no selection (a dense layer, or contexts that a selection does not pay for): ragged lengths, every key
        {"name": "mla dense 24 x 1-8191", "op": "mla", "seqs": 24, "q_per_seq": 1, "ctx_min": 1, "ctx_max": 8191,
         "heads": 128, "k": 0, "g": 16, "page": 64, "dense": True},
        # the cache append of a decode step, two tokens per sequence: blocks partly filled, a scale that may grow
        {"name": "append decode 64 x 2", "op": "append", "seqs": 64, "new_min": 2, "new_max": 2, "old_min": 4096,
         "old_max": 8191, "g": 64, "page": 64, "grow": 0.25},
        # prompts of odd lengths going into the cache
        {"name": "append prompts 16 x 1K-8K", "op": "append", "seqs": 16, "new_min": 1000, "new_max": 8192,
         "old_min": 0, "old_max": 77, "g": 64, "page": 64, "grow": 0.25},
        # a decode step: every sequence one token longer, few pages wanted of a large pool
        {"name": "resize decode 64", "op": "resize", "seqs": 64, "entries": 64, "pages": 16384, "per_seq": 512,
         "page": 64, "grow": 1, "free": 0.0, "share": 0.0},
        # a scheduling step: prompts admitted, finished and cut sequences freed, forked last pages copied on write
        {"name": "resize schedule 256", "op": "resize", "seqs": 256, "entries": 256, "pages": 24576, "per_seq": 512,
         "page": 64, "grow": 2048, "free": 0.3, "share": 0.5},
        # four samples of each of a few prompts
        {"name": "fork 24 of 8", "op": "fork", "seqs": 32, "entries": 24, "pages": 4096, "per_seq": 512, "page": 64},
        # beams of long contexts
        {"name": "fork 192 of 64", "op": "fork", "seqs": 256, "entries": 192, "pages": 65536, "per_seq": 2048,
         "page": 64},
        # a small pool after sequences have left it
        {"name": "compact 4096 pages", "op": "compact", "seqs": 64, "pages": 4096, "per_seq": 128, "page": 64,
         "live": 0.5},
        # the pool of sixteen 128K contexts after half of them have left
        {"name": "compact 32768 pages", "op": "compact", "seqs": 256, "pages": 32768, "per_seq": 2048, "page": 64,
         "live": 0.5},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["mla", "mla", "mla", "append", "append", "resize", "fork", "compact"])
    g = 1 << rng.randrange(7)
    page = rng.choice([0, 64, 64, 128, 192])
    if op == "mla":
        heads = 8 * rng.randint(1, 16)
        if rng.random() < 0.3:                        # every visible key
            seqs = _log(rng, 1, 32)
            hi = _log(rng, 1, 8191)
            return {"op": op, "seqs": seqs, "q_per_seq": rng.randint(1, 2), "ctx_min": max(2, hi // 8),
                    "ctx_max": max(2, hi), "heads": heads, "k": 0, "g": g, "page": page, "dense": True}
        k = _log(rng, 1, 2048)
        if rng.random() < 0.3:                        # a chunk of a prompt
            n = _log(rng, 16, 2000)
            ctx = n + _log(rng, 1, 30000)
            return {"op": op, "seqs": 1, "q_per_seq": n, "ctx_min": ctx, "ctx_max": ctx, "heads": heads, "k": k,
                    "g": g, "page": page, "dense": False}
        hi = _log(rng, 16, 32768)
        return {"op": op, "seqs": _log(rng, 1, 100), "q_per_seq": rng.randint(1, 4), "ctx_min": max(4, hi // 8),
                "ctx_max": hi, "heads": heads, "k": k, "g": g, "page": page, "dense": False}
    if op == "append":
        hi = _log(rng, 1, 8000)
        return {"op": op, "seqs": _log(rng, 1, 60000 // (hi + 500)), "new_min": max(1, hi // 8), "new_max": hi,
                "old_min": 0, "old_max": _log(rng, 1, 8000), "g": g, "page": page, "grow": rng.random()}
    page = page or 64
    if op == "resize":
        pages = _log(rng, 512, 24000)
        seqs = _log(rng, 1, 256)
        return {"op": op, "seqs": seqs, "entries": rng.randint(1, seqs), "pages": pages, "per_seq": _log(rng, 8, 512),
                "page": page, "grow": _log(rng, 1, 2048), "free": rng.random(), "share": rng.random()}
    if op == "fork":
        src = _log(rng, 1, 64)
        entries = _log(rng, 1, 190)
        return {"op": op, "seqs": src + entries, "entries": entries, "pages": _log(rng, 512, 65536),
                "per_seq": _log(rng, 8, 2048), "page": page}
    return {"op": op, "seqs": _log(rng, 2, 256), "pages": _log(rng, 256, 32768 * 64 // page), "per_seq": _log(rng, 8, 2048),
            "page": page, "live": rng.uniform(0.05, 0.95)}


# ------------------------------------------------------------------- inputs
def _host(case, seed):
    return np.random.default_rng([int(seed), sum(map(ord, case["op"]))])


def _lengths(case):
    """Lengths of the sequences, by the case alone: (cached before, new).  mla: every row is cached, the last ones ask."""
    r = np.random.default_rng([7, case["seqs"]])
    between = lambda a: r.integers(case[a + "_min"], case[a + "_max"], size=case["seqs"], endpoint=True)  # noqa: E731
    if case["op"] == "append":
        return between("old"), between("new")
    lens = between("ctx")
    m = min(case["q_per_seq"], int(lens.min()))
    return lens - m, np.full(case["seqs"], m)


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _layout(r, lens, page, g):
    """Rows of sequences of the given lengths: (kv_offset, table or None, rows)."""
    lens = lens.astype(np.int64)
    if page == 0:                                     # contiguous, every sequence on a block of its own
        room = -(-lens // g) * g
        off = np.concatenate([[0], np.cumsum(room)])
        return off[:-1], None, int(max(off[-1], g))
    need = -(-lens // page)
    pps = int(max(1, need.max()))
    total = int(need.sum()) + 3
    perm = r.permutation(total)
    start = np.concatenate([[0], np.cumsum(need)])[:-1]
    j = np.arange(pps)[None, :]
    table = np.where(j < need[:, None], perm[np.minimum(start[:, None] + j, total - 1)], -1).astype(np.int32)
    return np.zeros(len(lens), np.int64), table, total * page


def _random_cache(rows, g, gen):
    """Codes of unit-normal rows under scales of 2^-7 .. 2^-5 (a block's largest entry is near 448)."""
    kv8 = torch.empty((rows, D_QK), dtype=torch.uint8, device="cuda")
    blocks = -(-rows // g)
    scale = torch.exp2(torch.randint(-7, -4, (blocks,), generator=gen, device="cuda").float())
    step = 1 << 18
    per = torch.repeat_interleave(scale, g)[:rows]
    for a in range(0, rows, step):
        b = min(rows, a + step)
        x = torch.randn((b - a, D_QK), generator=gen, device="cuda") / per[a:b, None]
        kv8[a:b] = x.clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
    return kv8, scale


def _prepare_mla(case, seed):
    r, gen = _host(case, seed), _gen(seed)
    n, k = case["seqs"], case["k"]
    old, new = _lengths(case)
    lens, m = (old + new).astype(np.int32), int(new[0])
    off, table, rows = _layout(r, lens, case["page"], case["g"])
    q_seq = np.repeat(np.arange(n, dtype=np.int32), m)
    q_pos = (lens[q_seq] - m + np.tile(np.arange(m), n)).astype(np.int32)
    kv8, scale = _random_cache(rows, case["g"], gen)
    T = n * m
    q = torch.randn((T, case["heads"], D_QK), generator=gen, device="cuda").to(torch.bfloat16)
    s = {"op": "mla", "g": case["g"], "page": case["page"], "heads": case["heads"], "k": k, "kv8": kv8,
         "scale": scale, "q": q, "rows": rows, "kv_offset": torch.as_tensor(off, device="cuda"),
         "kv_len": torch.as_tensor(lens, device="cuda"), "q_seq": torch.as_tensor(q_seq, device="cuda"),
         "q_pos": torch.as_tensor(q_pos, device="cuda"), "max_len": int(lens.max()), "idx": None,
         "table": None if table is None else torch.as_tensor(table, device="cuda")}
    if not case["dense"]:
        # ascending distinct positions, one in each of k equal stretches of the context; all where it is no longer than k
        seen = (s["q_pos"].long() + 1)[:, None]
        j = torch.arange(k, device="cuda")[None, :]
        lo, hi = j * seen // k, (j + 1) * seen // k
        u = torch.rand((T, k), generator=gen, device="cuda", dtype=torch.float64)
        pick = lo + ((hi - lo).double() * u).long()
        s["idx"] = torch.where(seen > k, pick, torch.where(j < seen, j, -1)).int().contiguous()
    s["out"] = torch.zeros((T, case["heads"], D_V), dtype=torch.bfloat16, device="cuda")
    s["lse"] = torch.zeros((T, case["heads"]), device="cuda")
    if own:
        B = _binding()
        s["batch"] = _device_batch(s, off, lens, q_seq, q_pos, table)
        s["ws"] = B.q8_workspace(B.Q8_MLA, s["batch"], H=case["heads"], k=k, device="cuda")
    return s


def _prepare_append(case, seed):
    r, gen = _host(case, seed), _gen(seed)
    n, g = case["seqs"], case["g"]
    old, new = _lengths(case)
    lens = (old + new).astype(np.int32)
    off, table, rows = _layout(r, lens, case["page"], g)
    T = int(new.sum())
    q_seq = np.repeat(np.arange(n, dtype=np.int32), new)
    first = np.concatenate([[0], np.cumsum(new)])[:-1]
    q_pos = (np.arange(T) - first[q_seq] + old[q_seq]).astype(np.int32)
    kv8, scale = _random_cache(rows, g, gen)
    # unit-normal rows, some of them eight times as large: these raise their block's scale
    kv = torch.randn((T, D_QK), generator=gen, device="cuda")
    big = torch.rand((T, 1), generator=gen, device="cuda") < case["grow"]
    kv = torch.where(big, 8 * kv, kv).to(torch.bfloat16)
    s = {"op": "append", "g": g, "page": case["page"], "kv": kv, "kv8": kv8, "scale": scale, "rows": rows,
         "kv_offset": torch.as_tensor(off, device="cuda"), "kv_len": torch.as_tensor(lens, device="cuda"),
         "q_seq": torch.as_tensor(q_seq, device="cuda"), "q_pos": torch.as_tensor(q_pos, device="cuda"),
         "max_len": int(lens.max()), "table": None if table is None else torch.as_tensor(table, device="cuda")}
    if own:
        B = _binding()
        s["batch"] = _device_batch(s, off, lens, q_seq, q_pos, table)
        s["ws"] = B.q8_workspace(B.Q8_APPEND, s["batch"], device="cuda")
    return s


def _pool(r, case, filled):
    """Sequences `filled` with random lengths on random pages: (table, lens, refs), numpy."""
    P, pps, N = case["page"], case["per_seq"], case["pages"]
    table = np.full((case["seqs"], pps), -1, np.int32)
    lens = np.zeros(case["seqs"], np.int32)
    refs = np.zeros(N, np.int32)
    room = int(N * case.get("live", 0.5))
    perm = r.permutation(N)
    most = max(1, min(pps, 2 * room // max(1, len(filled))))
    want = r.integers(0, most, size=len(filled), endpoint=True)
    want = np.minimum(np.cumsum(want), room) - np.minimum(np.cumsum(want) - want, room)
    at = 0
    for s, w in zip(filled, want):
        table[s, :w] = perm[at:at + w]
        lens[s] = 0 if w == 0 else (w - 1) * P + int(r.integers(1, P, endpoint=True))
        at += w
    refs[perm[:at]] = 1
    return table, lens, refs


def _prepare_pages(case, seed):
    r, gen = _host(case, seed), _gen(seed)
    P, pps, S, N, op = case["page"], case["per_seq"], case["seqs"], case["pages"], case["op"]
    if op == "fork":
        srcs = S - case["entries"]
        table, lens, refs = _pool(r, case, np.arange(srcs))
        a = r.integers(0, srcs, size=case["entries"]).astype(np.int32)
        b = (srcs + r.permutation(case["entries"])).astype(np.int32)
    elif op == "resize":
        table, lens, refs = _pool(r, case, np.arange(S))
        # sequences that share all of another's pages, as after a fork
        free = np.flatnonzero(r.random(S) < case["share"] / 2)
        keep = np.setdiff1d(np.arange(S), free)
        for s in free if keep.size else []:
            used = table[s][table[s] >= 0]
            refs[used] = 0
            o = int(keep[r.integers(keep.size)])
            table[s], lens[s] = table[o], lens[o]
            refs[table[s][table[s] >= 0]] += 1
        a = r.permutation(S)[:case["entries"]].astype(np.int32)
        now = lens[a].astype(np.int64)
        cut = r.random(a.size) < case["free"]
        b = np.where(cut, np.where(r.random(a.size) < 0.7, 0, now // 2),
                     np.minimum(now + r.integers(1, case["grow"], size=a.size, endpoint=True), pps * P)).astype(np.int32)
    else:
        table, lens, refs = _pool(r, case, np.arange(S))
        a = b = np.zeros(0, np.int32)
    dev = lambda x: torch.as_tensor(x, device="cuda")  # noqa: E731
    s = {"op": op, "page": P, "table": dev(table), "lens": dev(lens), "refs": dev(refs), "a": dev(a), "b": dev(b),
         "table_out": torch.zeros((S, pps), dtype=torch.int32, device="cuda"),
         "lens_out": torch.zeros(S, dtype=torch.int32, device="cuda"),
         "refs_out": torch.zeros(N, dtype=torch.int32, device="cuda")}
    if op != "fork":                                  # the pool's buffers: latent codes, their scales, indexer keys
        s["kv8"] = torch.randint(0, 256, (N, P * D_QK), generator=gen, device="cuda", dtype=torch.uint8)
        s["scale"] = torch.exp2(torch.randint(-7, -4, (N, P // 64), generator=gen, device="cuda").float())
        s["k_idx"] = torch.randint(0, 256, (N, P * D_INDEX), generator=gen, device="cuda", dtype=torch.uint8)
    if op == "compact":
        s["map"] = torch.zeros(N, dtype=torch.int32, device="cuda")
    if own:
        B = _binding()
        s["src"] = B.PageState(s["table"], s["lens"], s["refs"], P)
        s["dst"] = B.PageState(s["table_out"], s["lens_out"], s["refs_out"], P)
        s["buffers"] = B.PageBuffers([s["kv8"], s["scale"], s["k_idx"]], N) if op != "fork" else None
        s["ws"] = B.pages_workspace(s["src"], len(a), device="cuda")
    return s


def prepare(case, seed):
    if case["op"] == "mla":
        return _prepare_mla(case, seed)
    if case["op"] == "append":
        return _prepare_append(case, seed)
    return _prepare_pages(case, seed)


# ------------------------------------------------------------------- the library's calls
def _binding():
    from sparse_attention_weight_b200 import binding
    return binding


def _device_batch(s, off, lens, q_seq, q_pos, table):
    class Host:
        pass
    h = Host()
    h.kv_offset, h.kv_len, h.q_seq, h.q_pos = off, lens, q_seq, q_pos
    return _binding().DeviceBatch.from_host(h, "cuda", kv_rows=s["rows"], page_size=s["page"], page_table=table)


def _run_own(s):
    B = _binding()
    if s["op"] == "mla":
        B.dsa_sparse_mla_q8(s["batch"], s["q"], s["kv8"], s["scale"], s["g"], s["idx"], s["k"], s["heads"], SM_SCALE,
                            s["out"], s["lse"], s["ws"])
        return {"out": s["out"], "lse": s["lse"]}
    if s["op"] == "append":
        B.dsa_quantize_append(s["batch"], s["kv"], s["kv8"], s["scale"], s["g"], s["ws"])
        return {"codes": s["kv8"].view(torch.float8_e4m3fn), "scale": s["scale"]}
    state = {"table": s["table_out"], "lens": s["lens_out"], "refs": s["refs_out"]}
    if s["op"] == "fork":
        B.dsa_pages_fork(s["src"], s["dst"], s["a"], s["b"], s["ws"])
        return state
    if s["op"] == "resize":
        B.dsa_pages_resize(s["src"], s["dst"], s["a"], s["b"], s["buffers"], s["ws"])
    else:
        B.dsa_pages_compact(s["src"], s["dst"], s["buffers"], s["map"], s["ws"])
        state["map"] = s["map"]
    return {**state, "kv8": s["kv8"], "scale": s["scale"], "k_idx": s["k_idx"]}


# ------------------------------------------------------------------- the plain forms
def _row_of(s, seq, pos):
    """Cache rows of positions `pos` of sequences `seq` (tensors of one shape)."""
    if s["table"] is None:
        return s["kv_offset"][seq] + pos
    P = s["page"]
    return s["table"][seq, pos // P].long() * P + pos % P


def _plain_mla(s, real=torch.float32):
    T, H = s["q"].shape[:2]
    if s["idx"] is None:
        pos = torch.arange(s["max_len"], device="cuda")[None, :].expand(T, -1)
        valid = pos <= s["q_pos"].long()[:, None]
    else:
        pos, valid = s["idx"].long(), s["idx"] >= 0
    seq = s["q_seq"].long()[:, None].expand_as(pos)
    row = _row_of(s, seq, torch.where(valid, pos, 0))
    keys = s["kv8"][row].view(torch.float8_e4m3fn).to(real)
    keys *= s["scale"].to(real)[row // s["g"]][..., None]
    z = torch.matmul(s["q"].to(real), keys.transpose(1, 2)) * SM_SCALE
    z.masked_fill_(~valid[:, None, :], -math.inf)
    top = z.amax(dim=2, keepdim=True)
    p = torch.exp(z - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(dim=2, keepdim=True)
    out = torch.matmul(p, keys[..., :D_V]) / torch.where(total == 0, 1.0, total)
    lse = (torch.log(total) + top)[..., 0]
    return out, lse


def _plain_append(s):
    g, T = s["g"], s["kv"].shape[0]
    x = s["kv"].float()
    row = _row_of(s, s["q_seq"].long(), s["q_pos"].long())
    block = row // g
    first = s["q_pos"].long() // g * g                # the block's first position
    # the block's old rows are those before the first new one
    new_at = torch.full((s["scale"].numel(),), 1 << 30, dtype=torch.int64, device="cuda")
    new_at = new_at.scatter_reduce(0, block, s["q_pos"].long(), "amin")[block]
    # the exponent that 448 times a power of two needs to hold the block's new rows
    amax = x.abs().amax(dim=1)
    mant, e = torch.frexp(amax)                       # amax = mant * 2^e, mant in [0.5, 1): amax <= 448 * 2^(e - 9 or e - 8)
    need = torch.where(amax == 0, MIN_EXP, torch.where(mant <= 0.875, e - 9, e - 8)).clamp(MIN_EXP, MAX_EXP).float()
    need = torch.full_like(s["scale"], MIN_EXP).scatter_reduce(0, block, need, "amax")[block]
    before = s["scale"][block]
    now = torch.where(new_at > first, torch.maximum(before, torch.exp2(need)), torch.exp2(need))
    # the old rows of a sequence's first new block, under its new scale
    t = torch.searchsorted(s["q_seq"], torch.arange(s["kv_len"].numel(), dtype=torch.int32, device="cuda"))
    at = ((block * g)[t][:, None] + torch.arange(g, device="cuda")).clamp(max=s["rows"] - 1)
    codes = s["kv8"][at]
    held = codes.view(torch.float8_e4m3fn).float() * (before / now)[t][:, None, None]
    old = (torch.arange(g, device="cuda") < (new_at - first)[t][:, None])[..., None]
    s["kv8"][at] = torch.where(old, held.to(torch.float8_e4m3fn).view(torch.uint8), codes)
    s["kv8"][row] = (x / now[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
    s["scale"][block] = now
    return {"codes": s["kv8"].view(torch.float8_e4m3fn), "scale": s["scale"]}


def _plain_fork(s):
    P, a, b = s["page"], s["a"].long(), s["b"].long()
    table, lens, refs = s["table"].clone(), s["lens"].clone(), s["refs"].clone()
    rows = table[a]
    used = torch.arange(table.shape[1], device="cuda")[None, :] < ((lens[a].long() + P - 1) // P)[:, None]
    refs.scatter_add_(0, torch.where(used, rows, 0).long().reshape(-1), used.int().reshape(-1))
    table[b] = torch.where(used, rows, -1)
    lens[b] = lens[a]
    return {"table": table, "lens": lens, "refs": refs}


def _plain_resize(s):
    P, a = s["page"], s["a"].long()
    table, lens, refs = s["table"].clone(), s["lens"].clone(), s["refs"].clone()
    N, pps = refs.numel(), table.shape[1]
    old, new = lens[a].long(), s["b"].long()
    have, want = (old + P - 1) // P, (new + P - 1) // P
    rows = table[a].long()
    j = torch.arange(pps, device="cuda")[None, :]
    # pages that are given back
    drop = (j >= want[:, None]) & (j < have[:, None])
    refs.scatter_add_(0, torch.where(drop, rows, 0).reshape(-1), -drop.int().reshape(-1))
    rows = torch.where(drop, -1, rows)
    # a growing sequence copies a shared, partly filled last page; of those that share it the last one keeps it
    last = rows.gather(1, (have - 1).clamp(min=0)[:, None])[:, 0]
    part = (new > old) & (old % P != 0)
    same = (last[:, None] == last[None, :]) & part[:, None] & part[None, :]
    rank = torch.tril(same.int(), -1).sum(1)
    copy = part & (refs[last.clamp(min=0)] - rank > 1)
    take = copy.long() + (want - have).clamp(min=0)
    start = torch.cumsum(take, 0) - take
    # the lowest free pages, in the entries' order (there are enough of them)
    is_free = refs == 0
    order = torch.cumsum(is_free.long(), 0) - 1
    free = torch.zeros(N + 1, dtype=torch.int64, device="cuda")
    free.scatter_(0, torch.where(is_free, order, N), torch.arange(N, device="cuda"))
    enough = take.sum() <= is_free.sum()
    copy, take = copy & enough, take * enough
    grow = (j >= have[:, None]) & (j < want[:, None]) & enough
    got = free[(start[:, None] + copy[:, None].long() + (j - have[:, None])).clamp(0, N)]
    rows = torch.where(grow, got, rows)
    refs.scatter_add_(0, torch.where(grow, rows, 0).reshape(-1), grow.int().reshape(-1))
    to = free[start.clamp(max=N)]
    rows = torch.where(copy[:, None] & (j == (have - 1)[:, None]), to[:, None], rows)
    refs.scatter_add_(0, torch.where(copy, last, 0), -copy.int())
    refs.scatter_add_(0, torch.where(copy, to, 0), copy.int())
    table[a] = rows.int()
    lens[a] = torch.where((new > old) & ~enough, old, new).int()
    frm, to = last[copy], to[copy]
    s["kv8"][to], s["scale"][to], s["k_idx"][to] = s["kv8"][frm], s["scale"][frm], s["k_idx"][frm]
    return {"table": table, "lens": lens, "refs": refs, "kv8": s["kv8"], "scale": s["scale"], "k_idx": s["k_idx"]}


def _plain_compact(s):
    table, lens, refs, P = s["table"], s["lens"].clone(), s["refs"], s["page"]
    N = refs.numel()
    live = refs > 0
    count = live.sum()
    page = torch.arange(N, device="cuda")
    frm, to = page[live & (page >= count)], page[~live & (page < count)]
    new = torch.where(live, page, -1)
    new[frm] = to
    used = torch.arange(table.shape[1], device="cuda")[None, :] < ((lens.long() + P - 1) // P)[:, None]
    out = torch.where(used, new[table.long().clamp(min=0)].int(), table)
    moved = refs.clone()
    moved[to], moved[frm] = refs[frm], 0
    s["kv8"][to], s["scale"][to], s["k_idx"][to] = s["kv8"][frm], s["scale"][frm], s["k_idx"][frm]
    return {"table": out, "lens": lens, "refs": moved, "map": new.int(), "kv8": s["kv8"], "scale": s["scale"],
            "k_idx": s["k_idx"]}


def run(state):
    if own:
        return _run_own(state)
    if state["op"] == "mla":
        out, lse = _plain_mla(state)
        return {"out": out.to(torch.bfloat16), "lse": lse}
    return {"append": _plain_append, "fork": _plain_fork, "resize": _plain_resize,
            "compact": _plain_compact}[state["op"]](state)


# ------------------------------------------------------------------- work
def work(case):
    s = _sizes(case)
    if case["op"] == "mla":
        H, T = case["heads"], s["T"]
        return {"bytes": T * H * (D_QK + D_V) * 2 + T * H * 4 + s["distinct"] * (D_QK + 4 / case["g"])
                + (0 if case["dense"] else 4 * T * case["k"]),
                "flops": 2 * H * (D_QK + D_V) * s["picked"]}
    if case["op"] == "append":
        return {"bytes": s["T"] * (3 * D_QK + 8) + 4 * s["T"] / case["g"], "flops": 2 * s["T"] * D_QK}
    meta = 4 * (case["seqs"] * (case["per_seq"] + 1) + case["pages"])
    return {"bytes": 2 * meta + 2 * s["moved"] * (case["page"] * (D_QK + D_INDEX) + 4 * (case["page"] // 64)),
            "flops": 0}


def _sizes(case):
    """Rows that are attended to, rows of the cache that they are, new rows; the pages that are moved as expected."""
    if case["op"] == "mla":
        old, new = _lengths(case)
        m = int(new[0])
        seen = old[:, None] + 1 + np.arange(m)[None, :]
        picked = seen if case["dense"] else np.minimum(seen, case["k"])
        return {"T": seen.size, "picked": int(picked.sum()),
                "distinct": int(np.minimum(picked.sum(1), old + new).sum())}
    if case["op"] == "append":
        return {"T": int(_lengths(case)[1].sum())}
    live = case.get("live", 0.5)
    if case["op"] == "compact":
        most = min(case["per_seq"], 2 * int(case["pages"] * live) / case["seqs"])
        live = min(live, case["seqs"] * most / 2 / case["pages"])
        return {"moved": case["pages"] * live * (1 - live)}
    if case["op"] == "resize":                        # last pages that two growing sequences share
        return {"moved": case["entries"] * case["share"] / 2 * (1 - case["free"]) ** 2}
    return {"moved": 0}


# ------------------------------------------------------------------- from the definitions, in 64 bits
def _round_e4m3(x):
    """float64 values rounded to E4M3 (nearest, ties to even, 448 at most)."""
    e = torch.floor(torch.log2(torch.clamp(x.abs(), min=2.0 ** -40)))
    e = torch.where(torch.exp2(e) > x.abs(), e - 1, e).clamp(min=-6)
    step = torch.exp2(e - 3)
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _decode_table():
    v = [(-1.0) ** (c >> 7) * ((c & 7) / 8 * 2.0 ** -6 if (c >> 3 & 15) == 0 else (1 + (c & 7) / 8) * 2.0 ** ((c >> 3 & 15) - 7))
         for c in range(256)]
    v[127] = v[255] = math.nan
    return torch.tensor(v, dtype=torch.float64, device="cuda")


def _exact_mla(case, seed):
    s = _prepare_mla(case, seed)
    code, outs, lses = _decode_table(), [], []
    for t in range(0, s["q"].shape[0], 64):
        seq, last = s["q_seq"][t:t + 64].long(), s["q_pos"][t:t + 64].long()
        if case["dense"]:
            pos = torch.arange(int(last.max()) + 1, device="cuda").repeat(seq.numel(), 1)
            live = pos <= last[:, None]
        else:
            pos = s["idx"][t:t + 64].long()
            live = pos >= 0
        pos = pos.clamp(min=0)
        if case["page"]:
            row = s["table"].long()[seq[:, None], pos // case["page"]] * case["page"] + pos % case["page"]
        else:
            row = s["kv_offset"][seq][:, None] + pos
        kv = code[s["kv8"][row].int()] * s["scale"].double()[row // case["g"]].unsqueeze(-1)
        logit = torch.einsum("thd,tkd->thk", s["q"][t:t + 64].double(), kv) * SM_SCALE
        logit = torch.where(live[:, None, :], logit, torch.full_like(logit, -math.inf))
        lses.append(torch.logsumexp(logit, dim=-1))
        outs.append(torch.einsum("thk,tkd->thd", torch.softmax(logit, dim=-1), kv[..., :D_V]))
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}


def _exact_append(case, seed):
    s = _prepare_append(case, seed)
    g, code = case["g"], _decode_table()
    kv, seqs, pos = s["kv"].double().cpu(), s["q_seq"].cpu().numpy(), s["q_pos"].cpu().numpy()
    scale, off = s["scale"].double(), s["kv_offset"].cpu().numpy()
    table = None if s["table"] is None else s["table"].cpu().numpy()
    values = code[s["kv8"].int()]
    # runs of new tokens of one sequence within one block
    cut = np.flatnonzero(np.concatenate([[True], (np.diff(seqs) != 0) | (pos[1:] // g != pos[:-1] // g)]))
    end = np.concatenate([cut[1:], [len(pos)]])
    big = np.maximum.reduceat(kv.abs().amax(1).numpy(), cut)
    kv = kv.cuda()
    rows_old, rows_new, f_old, f_new, blocks, f_block = [], [], [], [], [], []
    for a, b, m in zip(cut, end, big):
        p0, q = int(pos[a]), int(seqs[a])
        base = p0 // g * g
        row = int(off[q]) + base if table is None else int(table[q, base // case["page"]]) * case["page"] + base % case["page"]
        e = MIN_EXP
        if m > 0:
            e = int(math.ceil(math.log2(m / E4M3_MAX)))
            e += int(448.0 * 2.0 ** e < m) - int(448.0 * 2.0 ** (e - 1) >= m)
        now = 2.0 ** min(max(e, MIN_EXP), MAX_EXP)
        if p0 > base:
            was = float(s["scale"][row // g])
            now = max(was, now)
            rows_old += range(row, row + p0 - base)
            f_old += [was / now] * (p0 - base)
        rows_new += range(row + p0 - base, row + p0 - base + b - a)
        f_new += [now] * int(b - a)
        blocks.append(row // g)
        f_block.append(now)
    d = lambda v, t: torch.tensor(v, dtype=t, device="cuda")  # noqa: E731
    if rows_old:
        r = d(rows_old, torch.int64)
        values[r] = _round_e4m3(values[r] * d(f_old, torch.float64)[:, None])
    values[d(rows_new, torch.int64)] = _round_e4m3(kv / d(f_new, torch.float64)[:, None])
    scale[d(blocks, torch.int64)] = d(f_block, torch.float64)
    return {"codes": values, "scale": scale}


def exact(case, seed):
    if case["op"] == "mla":
        return _exact_mla(case, seed)
    if case["op"] == "append":
        return _exact_append(case, seed)
    return None                                       # whole numbers and moved bytes
