"""Cases, inputs and plain forms of the operators of a bounded cache.

Three operators, with the head shape of this library (256 values per head, 24
query heads over 4 KV heads), over paged pools of its formats:

  attend  causal attention of each sequence's newest tokens, one or a whole
          prompt, over a sliding window of its keys and the first few;
  move    rows of the cache moved to other positions, their keys turned from
          the old position's angle to the new one's, and read back;
  blocks  whole blocks moved within the pools, and the block tables rewritten.

``run`` computes them in elementary torch operations, or, where ``own`` is
true, by the framework's calls.  ``exact`` computes them in 64 bits, apart
from the plain form.
"""
import functools
import math

import numpy as np
import torch

own = False

HQ, HK, D = 24, 4, 256
GQA = HQ // HK
SCALE = 0.0625
THETA = 1e7
FMT = {"f16": 1, "q4_0": 2, "q8_0": 8}  # the pool formats' numbers
ROW = {"f16": 512, "q4_0": 144, "q8_0": 272}  # bytes of a stored row
IO = {"f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one user's step far into an endless conversation
        {"name": "attend 1 token, window 512", "op": "attend", "seqs": 1, "tok": 1, "mixed": False, "len": 33000, "window": 512, "sinks": 4,
         "page": 16, "kt": "q8_0", "vt": "q8_0", "io": "bf16"},
        # a decode step of eight sequences on a 4-bit cache
        {"name": "attend 8 tokens, window 4096", "op": "attend", "seqs": 8, "tok": 1, "mixed": False, "len": 32768, "window": 4096, "sinks": 4,
         "page": 16, "kt": "q4_0", "vt": "q4_0", "io": "bf16"},
        # a large batch, a window without first tokens, the formats of the per-call workload
        {"name": "attend 64 tokens, window 1024", "op": "attend", "seqs": 64, "tok": 1, "mixed": False, "len": 8192, "window": 1024, "sinks": 0,
         "page": 64, "kt": "q8_0", "vt": "q4_0", "io": "f16"},
        # verification of four drafted tokens on a 16-bit cache, pages of the verify workload
        {"name": "attend 8 x 4 tokens, window 2048", "op": "attend", "seqs": 8, "tok": 4, "mixed": False, "len": 20000, "window": 2048, "sinks": 16,
         "page": 256, "kt": "f16", "vt": "f16", "io": "f16"},
        # a step that mixes two chunks of prompt with single tokens and an idle sequence, pages that are no power of two
        {"name": "attend 700 + 600 + 3 tokens", "op": "attend", "seqs": 6, "tok": 700, "mixed": True, "len": 9000, "window": 2048, "sinks": 16,
         "page": 48, "kt": "q8_0", "vt": "q8_0", "io": "bf16"},
        # a large chunk of a long prompt
        {"name": "attend 2048 tokens, window 1024", "op": "attend", "seqs": 1, "tok": 2048, "mixed": False, "len": 16384, "window": 1024, "sinks": 4,
         "page": 16, "kt": "q8_0", "vt": "q4_0", "io": "bf16"},
        # a prompt from its first token on, every key visible, a 16-bit cache
        {"name": "attend 4096 tokens, no window", "op": "attend", "seqs": 1, "tok": 4096, "mixed": False, "len": 4096, "window": 0, "sinks": 0,
         "page": 64, "kt": "f16", "vt": "f16", "io": "bf16"},
        # three accepted of eight drafted tokens each, moved up to follow one another
        {"name": "move 8 x 3 accepted drafts", "op": "move", "how": "drafts", "rows": 24, "seqs": 8, "len": 9000, "page": 16, "kt": "q4_0",
         "vt": "q4_0", "rot": 64, "inter": False},
        # the middle of a full context dropped: the later rows move down over it, their keys to the new positions
        {"name": "move 12000 rows down by 777", "op": "move", "how": "shift", "rows": 12000, "seqs": 1, "len": 777, "page": 16, "kt": "q8_0",
         "vt": "q8_0", "rot": 64, "inter": False},
        # a context grown past what its frequencies were made for: every key turned to others where it lies
        {"name": "move 65536 rows, frequencies", "op": "move", "how": "rescale", "rows": 65536, "seqs": 4, "len": 0, "page": 256, "kt": "q8_0",
         "vt": "q4_0", "rot": 256, "inter": True},
        # a few holes of a small pool closed
        {"name": "blocks 40 of 16 rows", "op": "blocks", "move": 40, "live": 300, "seqs": 5, "page": 16, "kt": "q4_0", "vt": "q4_0"},
        # a pool brought to its front after most of its sequences have ended
        {"name": "blocks 5000 of 64 rows", "op": "blocks", "move": 5000, "live": 6000, "seqs": 40, "page": 64, "kt": "q8_0", "vt": "q4_0"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "move", "blocks"])
    kt, vt = rng.choice(list(FMT)), rng.choice(list(FMT))
    page = rng.choice([16, 32, 48, 64, 256])
    if op == "blocks":
        move = _log(rng, 1, 2000)
        return {"op": op, "move": move, "live": move + _log(rng, 1, 2000), "seqs": rng.randint(1, 40), "page": rng.choice([16, 32, 48, 64]), "kt": kt, "vt": vt}
    if op == "move":
        how = rng.choice(["drafts", "shift", "rescale", "fork"])
        rows = _log(rng, 1, 300 if how == "drafts" else 20000)
        if kt == "q4_0" and how in ("shift", "rescale"):  # one step of 4 bits is as large as a value: few rows
            rows = min(rows, 700)
        return {"op": op, "how": how, "rows": rows, "seqs": rng.randint(1, min(rows, 9)), "len": _log(rng, 1, 30000), "page": page, "kt": kt, "vt": vt,
                "rot": rng.choice([32, 64, 128, 256]), "inter": rng.random() < 0.3}
    kind = rng.choice(["step", "step", "chunk", "mixed"])
    if kind == "step":
        seqs, tok = _log(rng, 1, 64), rng.choice([1, 1, 1, 2, 3, 5, 8])
    else:
        seqs, tok = rng.randint(1, 4) if kind == "chunk" else rng.randint(2, 9), _log(rng, 9, 1500)
    window = rng.choice([0, _log(rng, 1, 8192), _log(rng, 64, 8192)])
    room = 3_500_000 // (seqs * tok)  # visible keys of a token, so that a draw stays below the work of the largest listed case
    length = tok + _log(rng, 1, max(2, min(40000, room if window == 0 else 40000, 120000 // seqs)))
    return {"op": op, "seqs": seqs, "tok": tok, "mixed": kind == "mixed", "len": length, "window": window if window == 0 else max(1, min(window, room)),
            "sinks": rng.choice([0, 1, 4, 16, 100]), "page": page, "kt": kt, "vt": vt, "io": rng.choice(["f16", "bf16"])}


def _tokens(case):
    """New tokens and lengths of a case's sequences, ragged, from the case alone."""
    new, lens = [], []
    for i in range(case["seqs"]):
        if not case["mixed"]:
            n = case["tok"]
        elif i < 2:
            n = case["tok"] - case["tok"] // 7 * i
        else:
            n = 0 if i % 4 == 3 else 1
        history = max(0, case["len"] - case["tok"])
        new.append(n)
        lens.append(n + history - (97 * i) % (history // 4 + 1))
    return new, lens


def _spans(case):
    """(new tokens, length, first key in a window, sinks before it) of each sequence."""
    got = []
    for n, length in zip(*_tokens(case)):
        lo = max(0, length - n - case["window"] + 1) if case["window"] and n else 0
        got.append((n, length, lo, min(case["sinks"], lo)))
    return got


def _visible(n, length, window, sinks):
    """Pairs of a token and a key that it sees."""
    p = np.arange(length - n, length, dtype=np.int64)
    lo = np.maximum(0, p - window + 1) if window else np.zeros_like(p)
    return int((p - lo + 1 + np.minimum(sinks, lo)).sum())


def work(case):
    op, per = case["op"], HK * (ROW[case["kt"]] + ROW[case["vt"]])
    if op == "attend":
        tokens = sum(s[0] for s in _spans(case))
        keys = sum(length - lo + first for n, length, lo, first in _spans(case) if n)
        pairs = sum(_visible(n, length, case["window"], case["sinks"]) for n, length, _, _ in _spans(case) if n)
        return {"bytes": keys * per + tokens * HQ * D * 4, "flops": 4 * D * HQ * pairs}
    if op == "blocks":
        return {"bytes": 2 * case["move"] * case["page"] * per + 8 * case["live"], "flops": 0}
    # rows in and out, read back; where keys are turned in place the values stay
    r, k = case["rows"], HK * ROW[case["kt"]]
    moved = k if case["how"] == "rescale" else per
    return {"bytes": r * (2 * moved + per + 2 * HK * D * 2 + 24), "flops": r * HK * D * 8}


# ------------------------------------------------------------------ pool bytes (groups of 16 rows)

@functools.lru_cache(None)
def _bytes_of(fmt, is_v):
    """Where in its group byte c of row r is: [16, bytes of a row], a row's eight scales (if it has them) before its quants."""
    at = np.zeros((16, ROW[fmt]), np.int64)
    scales = 0 if fmt == "f16" else 16
    body = ROW[fmt] - scales
    for r in range(16):
        for b in range(scales // 2):
            first = 64 * (b // 2) + 16 * (r % 8 // 2) + 8 * (b % 2) + 4 * (r // 8) + 2 * (r % 2) if is_v else 16 * r + 2 * b
            at[r, 2 * b: 2 * b + 2] = first, first + 1
        c = np.arange(body)
        at[r, scales:] = 16 * scales + body * r + ((c // 16) ^ (r % 8)) * 16 + c % 16
    return torch.from_numpy(at).cuda()


def _dequantised(rows, fmt):
    """Rows of bytes [..., bytes of a row] as values in 32 bits."""
    if fmt == "f16":
        return rows.contiguous().view(torch.float16).float()
    d = rows[..., :16].contiguous().view(torch.float16).float()[..., None]
    q = rows[..., 16:]
    if fmt == "q8_0":
        q = q.contiguous().view(torch.int8).float().reshape(*q.shape[:-1], 8, 32)
    else:
        q = q.reshape(*q.shape[:-1], 8, 16)
        q = torch.cat([q & 15, q >> 4], -1).float() - 8.0
    return (q * d).flatten(-2)


def _quantised(x, fmt):
    """Rows [..., 256] in 32 bits as bytes, every operation rounded on its own."""
    if fmt == "f16":
        return x.half().view(torch.uint8)
    x = x.reshape(*x.shape[:-1], 8, 32)
    if fmt == "q8_0":
        d = x.abs().amax(-1, keepdim=True) / 127.0
        y = x * torch.where(d != 0, 1.0 / d, torch.zeros_like(d))
        q = torch.trunc(y)
        q = (q + torch.where((y - q).abs() >= 0.5, torch.sign(y), torch.zeros_like(y))).to(torch.int8).view(torch.uint8)
    else:
        size = x.abs()
        first = torch.where(size == size.amax(-1, keepdim=True), torch.arange(32, device=x.device), 32).amin(-1, keepdim=True)
        d = x.gather(-1, first) / -8.0
        q = torch.trunc(x * torch.where(d != 0, 1.0 / d, torch.zeros_like(d)) + 8.5).clamp_max(15.0).to(torch.uint8)
        q = q[..., :16] | (q[..., 16:] << 4)
    return torch.cat([d.squeeze(-1).half().view(torch.uint8), q.flatten(-2)], -1)


def _pool(groups, fmt, is_v, g):
    """A pool of random rows."""
    got = torch.empty(groups, 16 * ROW[fmt], dtype=torch.uint8, device="cuda")
    back = torch.argsort(_bytes_of(fmt, is_v).reshape(-1))
    step = max(1, (1 << 28) // (16 * D * 4))
    for i in range(0, groups, step):
        n = min(step, groups - i)
        got[i: i + n] = _quantised(torch.randn(n, 16, D, device="cuda", generator=g), fmt).reshape(n, -1)[:, back]
    return got.reshape(-1)


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _shares(n, k):
    """n cut into k nearly equal parts."""
    return [n // k + (1 if i < n % k else 0) for i in range(k)]


def _freq(rot, wide=1.0):
    """Radians per position; wide: for contexts that are so many times longer (a larger base)."""
    base = THETA * wide ** (rot / (rot - 2))
    return [base ** (-2.0 * i / rot) for i in range(rot // 2)]


def _table(used, pages, g):
    """A block table [sequences][pages] over a shuffled pool: used[i], the pages that sequence i has; the others' entries are -1."""
    n = sum(len(u) for u in used)
    order = torch.randperm(n, device="cuda", generator=g).to(torch.int32).cpu().numpy()
    table, at = np.full((len(used), pages), -1, np.int32), 0
    for i, u in enumerate(used):
        table[i, u] = order[at: at + len(u)]
        at += len(u)
    return torch.from_numpy(table).cuda(), n


def _prepare_attend(case, g, page):
    spans = _spans(case)
    used = []
    for n, length, lo, first in spans:  # pages outside the windows have been given back
        used.append(sorted(set(range(-(-first // page))) | set(range(lo // page, -(-length // page)))) if n else [])
    table, n_blocks = _table(used, max(1, max(-(-s[1] // page) for s in spans)), g)
    rows = sum(s[0] for s in spans)
    qkv = torch.randn(rows, HQ + 2 * HK, D, device="cuda", generator=g).to(IO[case["io"]])
    lens = np.array([s[1] for s in spans], np.int32)
    return {"q": qkv[:, :HQ], "table": table, "new": np.array([s[0] for s in spans], np.int32), "lens_host": lens, "lens": torch.from_numpy(lens).cuda(),
            "out": torch.empty(rows, HQ, D, dtype=qkv.dtype, device="cuda")}, n_blocks


def _prepare_move(case, g, page, seed):
    """Rows to move: (sequence, position) from and to."""
    rng = np.random.default_rng(seed)
    seq, src, dst, to = [], [], [], []
    for i, n in enumerate(_shares(case["rows"], case["seqs"])):
        at = case["len"] + 7 * i
        if case["how"] == "drafts":  # n of the tokens drafted from position `at` on, in order
            a, b = at + np.sort(rng.choice(3 * n, n, replace=False)), at + np.arange(n)
        elif case["how"] == "shift":  # four rows stay, `len` rows behind them go
            a, b = 4 + at + np.arange(n), 4 + np.arange(n)
        elif case["how"] == "fork":  # the sequence's copy has pages of its own
            a = b = at + np.arange(n)
        else:
            a = b = np.arange(n)
        src.append(a)
        dst.append(b)
        seq.append(np.full(n, i))
        to.append(np.full(n, i + case["seqs"] if case["how"] == "fork" else i))
    dev = lambda x: torch.from_numpy(np.concatenate(x).astype(np.int32)).cuda()  # noqa: E731
    used = [sorted(set(a // page) | set(b // page)) if case["how"] != "fork" else sorted(set(a // page)) for a, b in zip(src, dst)]
    if case["how"] == "fork":
        used += used
    table, n_blocks = _table(used, 1 + max(max(u) for u in used), g)
    return {"src_seq": dev(seq), "src": dev(src), "dst_seq": dev(to), "dst": dev(dst), "table": table,
            "k_out": torch.empty(case["rows"], HK, D, dtype=torch.float16, device="cuda"),
            "v_out": torch.empty(case["rows"], HK, D, dtype=torch.float16, device="cuda")}, n_blocks


def _prepare_blocks(case, seed):
    """Live blocks of a pool, `move` of them behind the first `live` places, which have as many holes."""
    rng = np.random.default_rng(seed)
    move, live = case["move"], case["live"]
    n_blocks = 2 * live
    holes = np.sort(rng.choice(live, move, replace=False))
    behind = np.sort(live + rng.choice(n_blocks - live, move, replace=False))
    blocks = rng.permutation(np.concatenate([np.setdiff1d(np.arange(live), holes), behind]))
    table = np.full((case["seqs"], -(-live // case["seqs"]) + 3), -1, np.int32)
    for i, part in enumerate(np.array_split(blocks, case["seqs"])):
        table[i, : len(part)] = part
    dev = lambda x: torch.from_numpy(x.astype(np.int32)).cuda()  # noqa: E731
    return {"src": dev(behind), "dst": dev(holes), "table": dev(table), "table_out": torch.empty(table.shape, dtype=torch.int32, device="cuda")}, n_blocks


def prepare(case, seed):
    g, op, page = _gen(seed), case["op"], case["page"]
    if op == "attend":
        s, n_blocks = _prepare_attend(case, g, page)
    elif op == "move":
        s, n_blocks = _prepare_move(case, g, page, seed)
    else:
        s, n_blocks = _prepare_blocks(case, seed)
    n_blocks = max(1, n_blocks)
    groups = n_blocks * HK * (page // 16)
    s.update(case=case, k_pool=_pool(groups, case["kt"], False, g), v_pool=_pool(groups, case["vt"], True, g))
    if own:
        from paged_kv_gqa_11_gb300.cache import PagedKVCache
        s["cache"] = PagedKVCache(n_blocks, page, FMT[case["kt"]], FMT[case["vt"]], k_pool=s["k_pool"], v_pool=s["v_pool"])
        if op == "move":
            from paged_kv_gqa_11_gb300.rope import Rope
            s["rope"] = s["rope_from"] = None
            if case["how"] in ("shift", "rescale"):
                s["rope_from"] = Rope(_freq(case["rot"]), interleaved=case["inter"])
                s["rope"] = Rope(_freq(case["rot"], 4.0), interleaved=case["inter"]) if case["how"] == "rescale" else s["rope_from"]
    return s


# ------------------------------------------------------------------ the plain forms

def _groups(s, seq, pos):
    """Pool group of each (row, head), and the row in it."""
    page = s["case"]["page"]
    block = s["table"][seq.long(), (pos // page).long()].long().clamp_min(0)
    head = torch.arange(HK, device="cuda")
    return (block[..., None] * HK + head) * (page // 16) + ((pos % page) // 16).long()[..., None], (pos % 16).long()


def _rows(s, name, seq, pos):
    """Rows of bytes of a pool [..., 4, bytes of a row]."""
    fmt = s["case"]["kt" if name == "k_pool" else "vt"]
    grp, row = _groups(s, seq, pos)
    return s[name][grp[..., None] * (16 * ROW[fmt]) + _bytes_of(fmt, name == "v_pool")[row][..., None, :]]


def _write(s, name, seq, pos, rows):
    fmt = s["case"]["kt" if name == "k_pool" else "vt"]
    grp, row = _groups(s, seq, pos)
    s[name][grp[..., None] * (16 * ROW[fmt]) + _bytes_of(fmt, name == "v_pool")[row][..., None, :]] = rows


def _turned(x, angle, inter):
    """Heads [n, h, 256], their first values turned by angles [n, pairs] (in 64 bits)."""
    rot = 2 * angle.shape[-1]
    c, s = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    y = x.clone()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if inter else (x[..., : rot // 2], x[..., rot // 2: rot])
    if inter:
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * s, b * c + a * s
    else:
        y[..., : rot // 2], y[..., rot // 2: rot] = a * c - b * s, b * c + a * s
    return y


def _move(s):
    case = s["case"]
    k, v = _rows(s, "k_pool", s["src_seq"], s["src"]), _rows(s, "v_pool", s["src_seq"], s["src"])
    if case["how"] in ("shift", "rescale"):
        freq = lambda wide: torch.tensor(_freq(case["rot"], wide), dtype=torch.float64, device="cuda")  # noqa: E731
        angle = s["dst"].double()[:, None] * freq(4.0 if case["how"] == "rescale" else 1.0) - s["src"].double()[:, None] * freq(1.0)
        turned = _quantised(_turned(_dequantised(k, case["kt"]), angle, case["inter"]), case["kt"])
        blocks = -(-case["rot"] // 32)  # the blocks of 32 values that are turned; the others keep their bytes
        if case["kt"] == "f16":
            turned[..., 64 * blocks:] = k[..., 64 * blocks:]
        else:
            body = (ROW[case["kt"]] - 16) // 8
            turned[..., 2 * blocks: 16] = k[..., 2 * blocks: 16]
            turned[..., 16 + body * blocks:] = k[..., 16 + body * blocks:]
        same = torch.tensor([case["how"] != "rescale"], device="cuda") & (s["src"] == s["dst"])  # nothing to turn
        k = torch.where(same[:, None, None], k, turned)
    _write(s, "k_pool", s["dst_seq"], s["dst"], k)
    _write(s, "v_pool", s["dst_seq"], s["dst"], v)
    return {"k": _dequantised(_rows(s, "k_pool", s["dst_seq"], s["dst"]), case["kt"]).half(),
            "v": _dequantised(_rows(s, "v_pool", s["dst_seq"], s["dst"]), case["vt"]).half()}


def _attend(s):
    case, spans = s["case"], _spans(s["case"])
    n, t = len(spans), max(x[0] for x in spans)
    col = lambda v: torch.tensor(v, device="cuda")[:, None]  # noqa: E731
    new, length, lo, first = (col([x[i] for x in spans]) for i in range(4))
    # each sequence's keys: its sinks, then those from its first window on, in whole groups of 16 rows
    first, lo = (first + 15) // 16 * 16, lo // 16 * 16
    first = torch.minimum(first, lo)
    keys = max((x[1] - x[2] // 16 * 16) + min((x[3] + 15) // 16 * 16, x[2] // 16 * 16) for x in spans if x[0])
    at = torch.arange(0, -(-keys // 16) * 16, device="cuda")[None, :]
    pos = torch.where(at < first, at, lo + at - first)
    live = pos < length
    lead = torch.where(live, pos, 0)[:, ::16]
    grp, _ = _groups(s, torch.arange(n, device="cuda")[:, None].expand_as(lead), lead)
    kv = []
    for name, fmt in (("k_pool", case["kt"]), ("v_pool", case["vt"])):
        b = s[name].reshape(-1, 16 * ROW[fmt])[grp]  # [n, groups, 4, bytes]
        b = b[..., _bytes_of(fmt, name == "v_pool").reshape(-1)].reshape(*b.shape[:-1], 16, ROW[fmt])
        kv.append(_dequantised(b, fmt).permute(0, 2, 1, 3, 4).reshape(n, HK, -1, D))
    k, v = kv
    # queries, padded to the longest sequence's new tokens
    start = torch.cumsum(new, 0) - new
    tok = torch.arange(t, device="cuda")[None, :]
    row = torch.where(tok < new, start + tok, 0)
    q = s["q"][row].float().reshape(n, t, HK, GQA, D).permute(0, 2, 1, 3, 4).reshape(n, HK, t * GQA, D)
    mine = (length - new + tok)[:, :, None]  # positions of the tokens
    seen = (pos[:, None, :] <= mine) & live[:, None, :]
    if case["window"]:
        seen &= (pos[:, None, :] > mine - case["window"]) | (pos[:, None, :] < case["sinks"])
    logit = torch.matmul(q, k.transpose(-1, -2)).mul_(SCALE).reshape(n, HK, t, GQA, -1)
    logit.masked_fill_(~seen[:, None, :, None, :], float("-inf"))
    p = torch.exp(logit - logit.amax(-1, keepdim=True))
    o = torch.matmul(p.reshape(n, HK, t * GQA, -1), v).reshape(n, HK, t, GQA, D) / p.sum(-1, keepdim=True)
    o = o.permute(0, 2, 1, 3, 4).reshape(n, t, HQ, D)
    return {"out": o[(tok < new).expand(n, t)].to(IO[case["io"]])}


def _blocks(s):
    table = s["table"]
    for name, fmt in (("k_pool", s["case"]["kt"]), ("v_pool", s["case"]["vt"])):
        pool = s[name].reshape(-1, HK * s["case"]["page"] * ROW[fmt])
        pool[s["dst"].long()] = pool[s["src"].long()]
    to = torch.arange(2 * s["case"]["live"], dtype=torch.int32, device="cuda")
    to[s["src"].long()] = s["dst"]
    s["table_out"].copy_(torch.where(table >= 0, to[table.long().clamp_min(0)], table))
    return {"table": s["table_out"], "k_pool": s["k_pool"], "v_pool": s["v_pool"]}


def run(state):
    s, case = state, state["case"]
    if not own:
        return {"attend": _attend, "move": _move, "blocks": _blocks}[case["op"]](s)
    c = s["cache"]
    if case["op"] == "attend":
        return {"out": c.attend_window(s["q"], s["table"], s["lens"], s["lens_host"], s["new"], case["window"], case["sinks"], SCALE,
                                       out=s["out"], want_lse=False)[0]}
    if case["op"] == "move":
        c.move_rows(s["src_seq"], s["src"], s["dst_seq"], s["dst"], s["table"], rope=s["rope"], rope_from=s["rope_from"],
                    disjoint=case["how"] in ("fork", "rescale"))
        k, v = c.read_rows(s["dst_seq"], s["dst"], s["table"], k_out=s["k_out"], v_out=s["v_out"])
        return {"k": k, "v": v}
    return {"table": c.move_blocks(s["src"], s["dst"], s["table"], table_out=s["table_out"]), "k_pool": s["k_pool"], "v_pool": s["v_pool"]}


# ------------------------------------------------------------------ in 64 bits, apart from the above

def _half_at(flat, at):
    """The binary16 numbers whose bytes start at `at`, in 64 bits."""
    bits = flat[at].long() | (flat[at + 1].long() << 8)
    sign = 1.0 - 2.0 * (bits >> 15).double()
    e, m = (bits >> 10) & 31, (bits & 1023).double()
    return sign * torch.where(e == 0, m * 2.0 ** -24, (1024.0 + m) * torch.pow(2.0, (e - 25).double()))


def _values(s, name, seq, pos, head):
    """Rows of one head in 64 bits, each value found by its own byte."""
    fmt, page, pool = s["case"]["kt" if name == "k_pool" else "vt"], s["case"]["page"], s[name]
    block = s["table"].long()[seq, pos // page]
    base = (((block * HK + head) * page + pos % page // 16 * 16) * ROW[fmt])[:, None]
    r, i = (pos % 16)[:, None], torch.arange(D, device="cuda")[None, :]
    chunk = lambda at, row: base + row * r + ((at // 16) ^ (r % 8)) * 16 + at % 16  # noqa: E731
    if fmt == "f16":
        return _half_at(pool, chunk(2 * i, 512))
    b = i // 32
    scale = 64 * (b // 2) + 16 * (r % 8 // 2) + 8 * (b % 2) + 4 * (r // 8) + 2 * (r % 2) if name == "v_pool" else 16 * r + 2 * b
    d = _half_at(pool, base + scale)
    if fmt == "q8_0":
        x = pool[256 + chunk(i, 256)].long()
        return torch.where(x > 127, x - 256, x).double() * d
    x = pool[256 + chunk(16 * b + i % 16, 128)].long()
    return (torch.where(i % 32 >= 16, x >> 4, x & 15) - 8).double() * d


def _stored(x, fmt):
    """What rows in 64 bits come back as from a cache of this format. The formats' rule is one of 32-bit operations, each rounded:
    every one is done in 64 bits here and rounded to 32."""
    if fmt == "f16":
        return x.half().double()
    r32 = lambda y: y.float().double()  # noqa: E731
    b = r32(x).reshape(*x.shape[:-1], 8, 32)
    if fmt == "q8_0":
        d = r32(b.abs().max(-1, keepdim=True).values / 127)
        y = r32(b * r32(1 / d))
        q = torch.sign(y) * torch.floor(y.abs() + 0.5)
    else:
        size = b.abs()
        lead = (size == size.max(-1, keepdim=True).values).int().argmax(-1, keepdim=True)
        d = b.gather(-1, lead) / -8
        q = torch.trunc(r32(r32(b * r32(1 / d)) + 8.5)).clamp(max=15) - 8
    return torch.where(d == 0, torch.zeros_like(q), q * d.half().double()).reshape(x.shape)


def _exact_move(s, case):
    k, v = (torch.stack([_values(s, n, s["src_seq"].long(), s["src"].long(), h) for h in range(HK)], 1) for n in ("k_pool", "v_pool"))
    if case["how"] in ("shift", "rescale"):
        old, now = (torch.tensor(_freq(case["rot"], w), dtype=torch.float64, device="cuda") for w in (1.0, 4.0 if case["how"] == "rescale" else 1.0))
        turn = torch.polar(torch.ones(1, 1, dtype=torch.float64, device="cuda"), torch.outer(s["dst"].double(), now) - torch.outer(s["src"].double(), old))
        head, pairs = k[..., : case["rot"]], case["rot"] // 2
        head = head.unflatten(-1, (pairs, 2)) if case["inter"] else head.unflatten(-1, (2, pairs)).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(head.contiguous()) * turn[:, None])
        z = (z if case["inter"] else z.transpose(-1, -2)).flatten(-2)
        z = _stored(torch.cat([z, k[..., case["rot"]:]], -1), case["kt"])
        whole = -(-case["rot"] // 32) * 32
        z[..., whole:] = k[..., whole:]
        still = (s["src"] == s["dst"]) & (case["how"] == "shift")
        k = torch.where(still[:, None, None], k, z)
    return {"k": k, "v": v}


def exact(case, seed):
    global own
    if case["op"] == "blocks":  # whole numbers
        return None
    was, own = own, False
    s = prepare(case, seed)
    own = was
    if case["op"] == "move":
        return _exact_move(s, case)
    out, at = torch.zeros(s["q"].shape[0], HQ, D, dtype=torch.float64, device="cuda"), 0
    for i, (n, length, _, _) in enumerate(_spans(case)):
        for t0 in range(0, n, 512):  # so many tokens at once
            t1 = min(n, t0 + 512)
            mine = torch.arange(length - n + t0, length - n + t1, device="cuda")
            pos = torch.arange(length - n + t1, device="cuda")
            if case["window"]:
                pos = pos[(pos >= int(mine[0]) - case["window"] + 1) | (pos < case["sinks"])]
            sees = pos[None] <= mine[:, None]
            if case["window"]:
                sees &= (mine[:, None] - pos[None] < case["window"]) | (pos[None] < case["sinks"])
            seq = torch.full_like(pos, i)
            for h in range(HK):
                k, v = (_values(s, name, seq, pos, h) for name in ("k_pool", "v_pool"))
                q = s["q"][at + t0: at + t1, GQA * h: GQA * (h + 1)].double()
                z = torch.where(sees[:, None], q @ k.T / 16, float("-inf"))
                out[at + t0: at + t1, GQA * h: GQA * (h + 1)] = torch.softmax(z, -1) @ v
        at += n
    return {"out": out}
