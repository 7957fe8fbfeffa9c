"""Cases, inputs and plain forms of the cache operators around the decode.

Four operators, with the head shape of this library (256 values per head, 24
query heads over 4 KV heads):

  norm_rope  RMS norm of every query and key head and the position rotation;
  append     the same norm and rotation of new keys on their way into a paged
             cache (quantised to its format, with the values), the queries
             rotated beside them, and the new rows read back from the cache;
  read       rows of a paged cache as floating values;
  prefix     decode attention of sequences that share a long prefix.

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
EPS = 1e-6
THETA = 1e7
FMT = {"f16": 1, "q4_0": 2, "q8_0": 8}  # the pool formats' numbers
ROW = {"f16": 512, "q4_0": 144, "q8_0": 272}  # bytes of a stored row
IO = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
IO_BYTES = {"f16": 2, "bf16": 2, "f32": 4}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token of one sequence: what a single user's step pays before its attention
        {"name": "norm-rope 1 token", "op": "norm_rope", "rows": 1, "io": "bf16", "out": "bf16", "rot": 64, "inter": False},
        # a prefill chunk
        {"name": "norm-rope 4096 tokens", "op": "norm_rope", "rows": 4096, "io": "bf16", "out": "bf16", "rot": 256, "inter": False},
        # a decode step of eight sequences on a 4-bit cache
        {"name": "append 8 tokens q4_0", "op": "append", "rows": 8, "seqs": 8, "page": 16, "kt": "q4_0", "vt": "q4_0",
         "io": "bf16", "rot": 64, "inter": False, "far": 33000},
        # a chunk of prompt, ragged over three sequences, pages of another size
        {"name": "append 777 tokens q8_0", "op": "append", "rows": 777, "seqs": 3, "page": 48, "kt": "q8_0", "vt": "q8_0",
         "io": "f16", "rot": 128, "inter": True, "far": 0},
        # a large prefill chunk, the formats of the per-call workload, far positions
        {"name": "append 8192 tokens q8_0/q4_0", "op": "append", "rows": 8192, "seqs": 2, "page": 256, "kt": "q8_0", "vt": "q4_0",
         "io": "bf16", "rot": 256, "inter": False, "far": 250000},
        # a short prompt read back from a 16-bit cache
        {"name": "read 300 rows f16", "op": "read", "rows": 300, "seqs": 1, "page": 16, "kt": "f16", "vt": "f16", "out": "f32"},
        # a whole cached prefix as 16-bit rows
        {"name": "read 32768 rows q4_0", "op": "read", "rows": 32768, "seqs": 1, "page": 16, "kt": "q4_0", "vt": "q4_0", "out": "f16"},
        # two continuations of one short prompt
        {"name": "prefix 2 x (300 + 40)", "op": "prefix", "seqs": 2, "groups": 1, "prefix": 300, "suffix": 40, "page": 16,
         "kt": "q8_0", "vt": "q8_0", "tok": 1, "io": "f16"},
        # the shared-prefix workload of the benchmark
        {"name": "prefix 8 x (32768 + 1024)", "op": "prefix", "seqs": 8, "groups": 1, "prefix": 32768, "suffix": 1024, "page": 16,
         "kt": "q4_0", "vt": "q4_0", "tok": 1, "io": "bf16"},
        # four system prompts under a batch of 64
        {"name": "prefix 64 x (8192 + 300)", "op": "prefix", "seqs": 64, "groups": 4, "prefix": 8192, "suffix": 300, "page": 64,
         "kt": "q8_0", "vt": "q4_0", "tok": 1, "io": "f16"},
        # verification of four drafted tokens, pages of the verify workload
        {"name": "prefix 8 x (16384 + 2048), 4 tokens", "op": "prefix", "seqs": 8, "groups": 1, "prefix": 16384, "suffix": 2048,
         "page": 256, "kt": "q8_0", "vt": "q8_0", "tok": 4, "io": "bf16"},
        # a 16-bit cache, odd lengths, pages that are no power of two
        {"name": "prefix 17 x (4111 + 500) f16", "op": "prefix", "seqs": 17, "groups": 3, "prefix": 4111, "suffix": 500, "page": 48,
         "kt": "f16", "vt": "f16", "tok": 1, "io": "f16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "append", "read", "prefix", "prefix"])
    kt, vt = rng.choice(list(FMT)), rng.choice(list(FMT))
    page = rng.choice([16, 32, 48, 64, 256])
    rot, inter = rng.choice([32, 64, 128, 256]), rng.random() < 0.3
    if op == "norm_rope":
        return {"op": op, "rows": _log(rng, 1, 4096), "io": rng.choice(["f16", "bf16"]), "out": rng.choice(["f16", "bf16", "f32"]),
                "rot": rot, "inter": inter}
    if op == "append":
        rows = _log(rng, 1, 4096)
        return {"op": op, "rows": rows, "seqs": rng.randint(1, min(rows, 9)), "page": page, "kt": kt, "vt": vt,
                "io": rng.choice(["f16", "bf16"]), "rot": rot, "inter": inter, "far": rng.choice([0, 1000, 60000, 250000])}
    if op == "read":
        rows = _log(rng, 1, 32768)
        return {"op": op, "rows": rows, "seqs": rng.randint(1, min(rows, 9)), "page": page, "kt": kt, "vt": vt,
                "out": rng.choice(["f16", "bf16"])}
    seqs, tok = _log(rng, 2, 40), rng.choice([1, 1, 2, 3, 5, 8])
    rows = seqs * tok  # a draw stays below the work of the largest listed case
    return {"op": op, "seqs": seqs, "groups": rng.randint(1, max(1, seqs // 2)), "prefix": _log(rng, 200, min(32768, 400000 // rows)),
            "suffix": _log(rng, 16, min(1024, 100000 // rows)),
            "page": page, "kt": kt, "vt": vt, "tok": tok, "io": rng.choice(["f16", "bf16"])}


def _shares(n, k):
    """n cut into k nearly equal parts."""
    return [n // k + (1 if i < n % k else 0) for i in range(k)]


def _prefix_shape(case):
    """Sizes of the groups, their prefix lengths, and the sequences' lengths: ragged, from the case alone."""
    sizes = _shares(case["seqs"], case["groups"])
    pre = [case["prefix"] - (97 * g) % (case["prefix"] // 8 + 1) for g in range(len(sizes))]
    lens, i = [], 0
    for g, b in enumerate(sizes):
        for _ in range(b):
            lens.append(pre[g] + max(case["tok"], case["suffix"] - (61 * i) % (case["suffix"] // 2 + 1)))
            i += 1
    return sizes, pre, lens


def work(case):
    op = case["op"]
    if op == "norm_rope":
        n = case["rows"] * (HQ + HK) * D
        return {"bytes": n * (IO_BYTES[case["io"]] + IO_BYTES[case["out"]]) + 4 * case["rows"], "flops": 8 * n}
    if op == "append":
        r, b = case["rows"], IO_BYTES[case["io"]]
        stored = r * HK * (ROW[case["kt"]] + ROW[case["vt"]])
        # queries in and out, keys and values in, stored rows out and in again, values out
        return {"bytes": r * (2 * HQ + 2 * HK) * D * b + 2 * stored + r * 2 * HK * D * 2 + 8 * r, "flops": r * (HQ + 3 * HK) * D * 8}
    if op == "read":
        r = case["rows"]
        return {"bytes": r * HK * (ROW[case["kt"]] + ROW[case["vt"]] + 2 * D * IO_BYTES[case["out"]]) + 8 * r, "flops": r * 2 * HK * D}
    sizes, pre, lens = _prefix_shape(case)
    live = sum(pre) + sum(n - p for n, p in zip(lens, [p for b, p in zip(sizes, pre) for _ in range(b)]))  # each shared row once
    rows = len(lens) * case["tok"] * HQ
    return {"bytes": live * HK * (ROW[case["kt"]] + ROW[case["vt"]]) + rows * (2 * D * IO_BYTES[case["io"]] + 4),
            "flops": 4 * D * HQ * sum(case["tok"] * (n - case["tok"]) + case["tok"] * (case["tok"] + 1) // 2 for n in lens)}


# ------------------------------------------------------------------ pool bytes (groups of 16 rows)

def _swizzle(chunks, device):
    """Where chunk position p of row r comes from: chunk p xor (r mod 8)."""
    r, p = torch.arange(16, device=device)[:, None], torch.arange(chunks, device=device)[None, :]
    return p ^ (r & 7)


def _quants(x, fmt):
    """Rows [..., 256] in 32 bits to (scale of each 32 values, whole numbers), every operation rounded on its own."""
    x = x.reshape(*x.shape[:-1], 8, 32)
    if fmt == "q8_0":
        d = x.abs().amax(-1, keepdim=True) / 127.0
        inv = torch.where(d != 0, 1.0 / d, torch.zeros_like(d))
        y = x * inv
        q = torch.trunc(y)
        q = q + torch.where((y - q).abs() >= 0.5, torch.sign(y), torch.zeros_like(y))
    else:
        size = x.abs()
        first = torch.where(size == size.amax(-1, keepdim=True), torch.arange(32, device=x.device), 32).amin(-1, keepdim=True)
        d = x.gather(-1, first) / -8.0
        inv = torch.where(d != 0, 1.0 / d, torch.zeros_like(d))
        q = torch.trunc(x * inv + 8.5).clamp_max(15.0)
    return d.squeeze(-1).half(), q


def _pack(x, fmt, is_v):
    """Groups [G, 16, 256] as the pool's bytes [G, 16 * row bytes]."""
    g, dev = x.shape[0], x.device
    if fmt == "f16":
        scales, body = None, x.half().view(torch.uint8).reshape(g, 16, 32, 16)
    else:
        d, q = _quants(x, fmt)
        if fmt == "q8_0":
            body = q.to(torch.int8).view(torch.uint8).reshape(g, 16, 16, 16)
        else:
            q = q.to(torch.uint8)
            body = (q[..., :16] | (q[..., 16:] << 4)).reshape(g, 16, 8, 16)
        if is_v:  # [block / 2][(row % 8) / 2][block % 2][row / 8][row % 2]
            d = d.reshape(g, 2, 4, 2, 4, 2).permute(0, 4, 2, 5, 1, 3)
        scales = d.contiguous().reshape(g, 128).view(torch.uint8)
    at = _swizzle(body.shape[2], dev)[None, :, :, None].expand_as(body)
    body = body.gather(2, at).reshape(g, -1)
    return body if scales is None else torch.cat([scales, body], 1)


def _unpack(b, fmt, is_v, wide=torch.float32):
    """The values [G, 16, 256] of the pool's bytes."""
    g, dev = b.shape[0], b.device
    scales, body = (None, b) if fmt == "f16" else (b[:, :256], b[:, 256:])
    body = body.reshape(g, 16, -1, 16)
    at = _swizzle(body.shape[2], dev)[None, :, :, None].expand_as(body)
    body = body.gather(2, at).contiguous()
    if fmt == "f16":
        return body.reshape(g, 16, 512).view(torch.float16).to(wide)
    d = scales.contiguous().view(torch.float16)
    d = d.reshape(g, 4, 4, 2, 2, 2).permute(0, 4, 2, 5, 1, 3).reshape(g, 16, 8) if is_v else d.reshape(g, 16, 8)
    if fmt == "q8_0":
        q = body.view(torch.int8).reshape(g, 16, 8, 32).to(wide)
    else:
        q = torch.cat([body & 15, body >> 4], -1).to(wide) - 8.0
    return (q * d.to(wide)[..., None]).reshape(g, 16, 256)


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _inv_freq(rot):
    return [THETA ** (-2.0 * i / rot) for i in range(rot // 2)]


def _new_rows(case, g):
    """A projection's output [rows][24 + 4 + 4 heads][256] and the norms' weights."""
    qkv = torch.randn(case["rows"], HQ + 2 * HK, D, device="cuda", generator=g) * 1.7
    w = 1.0 + 0.2 * torch.randn(2, D, device="cuda", generator=g)
    t = IO[case["io"]]
    return qkv.to(t), w[0].to(t).contiguous(), w[1].to(t).contiguous()


def _pages(n_pages, stride, seqs, g):
    """A block table over a shuffled pool: seqs rows of `stride` entries, of which each sequence uses all."""
    order = torch.randperm(n_pages, device="cuda", generator=g).to(torch.int32)
    return order[: seqs * stride].reshape(seqs, stride).contiguous()


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    if op == "norm_rope":
        qkv, wq, wk = _new_rows(case, g)
        pos = torch.randint(0, 262144, (case["rows"],), device="cuda", generator=g, dtype=torch.int32)
        out = IO[case["out"]]
        s = {"case": case, "q": qkv[:, :HQ], "k": qkv[:, HQ:HQ + HK], "wq": wq, "wk": wk, "pos": pos,
             "q_out": torch.empty(case["rows"], HQ, D, dtype=out, device="cuda"),
             "k_out": torch.empty(case["rows"], HK, D, dtype=out, device="cuda")}
        if own:
            from paged_kv_gqa_11_gb300.rope import Rope
            s["rope"] = Rope(_inv_freq(case["rot"]), interleaved=case["inter"], eps=EPS)
        return s
    page, kt, vt = case["page"], case["kt"], case["vt"]
    if op in ("append", "read"):
        counts = _shares(case["rows"], case["seqs"])
        far = case.get("far", 0)
        seq = torch.repeat_interleave(torch.arange(len(counts)), torch.tensor(counts)).to(torch.int32)
        pos = torch.cat([far + 7 * i + torch.arange(c) for i, c in enumerate(counts)]).to(torch.int32)
        first = far // page  # pages before it hold nothing that is used here
        used = int(pos.max()) // page + 1 - first
        table = torch.zeros(len(counts), first + used, dtype=torch.int32, device="cuda")
        table[:, first:] = _pages(len(counts) * used, used, len(counts), g)
        s = {"case": case, "seq": seq.cuda(), "pos": pos.cuda(), "table": table}
        n_blocks, groups = len(counts) * used, len(counts) * used * HK * (page // 16)
        if op == "append":
            qkv, wq, wk = _new_rows(case, g)
            s.update(q=qkv[:, :HQ], k=qkv[:, HQ:HQ + HK], v=qkv[:, HQ + HK:], wq=wq, wk=wk,
                     k_pool=torch.zeros(groups * 16 * ROW[kt], dtype=torch.uint8, device="cuda"),
                     v_pool=torch.zeros(groups * 16 * ROW[vt], dtype=torch.uint8, device="cuda"),
                     q_out=torch.empty(case["rows"], HQ, D, dtype=IO[case["io"]], device="cuda"))
            out = torch.float16
        else:
            s.update(k_pool=_pack(torch.randn(groups, 16, D, device="cuda", generator=g), kt, False).reshape(-1),
                     v_pool=_pack(torch.randn(groups, 16, D, device="cuda", generator=g), vt, True).reshape(-1))
            out = IO[case["out"]]
        s.update(k_out=torch.empty(case["rows"], HK, D, dtype=out, device="cuda"),
                 v_out=torch.empty(case["rows"], HK, D, dtype=out, device="cuda"))
    else:
        sizes, pre, lens = _prefix_shape(case)
        stride = -(-max(lens) // page)
        shared = [p // page for p in pre]  # whole pages of a prefix are shared; the page it ends in is each sequence's own copy
        n_blocks = sum(shared) + sum(-(-n // page) - sh for n, sh in zip(lens, [h for b, h in zip(sizes, shared) for _ in range(b)]))
        order = torch.randperm(n_blocks, device="cuda", generator=g).to(torch.int32).cpu().numpy()
        table, at, i = np.zeros((len(lens), stride), np.int32), 0, 0
        copies = []  # (block of the group's first sequence, block of another), rows of the prefix in both
        for b, sh, p in zip(sizes, shared, pre):
            head = order[at: at + sh]
            at += sh
            for j in range(b):
                mine = -(-lens[i] // page) - sh
                table[i, :sh], table[i, sh: sh + mine] = head, order[at: at + mine]
                at += mine
                if p % page and j:
                    copies.append((table[i - j, sh], table[i, sh], p % page))
                i += 1
        groups = n_blocks * HK * (page // 16)
        kv = []
        for fmt, is_v in ((kt, False), (vt, True)):
            x = torch.randn(n_blocks, HK, page, D, device="cuda", generator=g)
            for a, b, n in copies:
                x[int(b), :, :n] = x[int(a), :, :n]
            kv.append(_pack(x.reshape(groups, 16, D), fmt, is_v).reshape(-1))
            del x
        q = torch.randn(len(lens), case["tok"], HQ, D, device="cuda", generator=g).to(IO[case["io"]])
        s = {"case": case, "q": q, "k_pool": kv[0], "v_pool": kv[1], "table": torch.from_numpy(table).cuda(),
             "lens_host": np.array(lens, np.int32), "lens": torch.tensor(lens, dtype=torch.int32, device="cuda"),
             "sizes": np.array(sizes, np.uint32), "pre": np.array(pre, np.int32),
             "out": torch.empty_like(q), "lse": torch.empty(len(lens), case["tok"], HQ, dtype=torch.float32, device="cuda")}
    if own:
        from paged_kv_gqa_11_gb300.cache import PagedKVCache
        s["cache"] = PagedKVCache(n_blocks, page, FMT[kt], FMT[vt], k_pool=s["k_pool"], v_pool=s["v_pool"])
        if op == "append":
            from paged_kv_gqa_11_gb300.rope import Rope
            s["rope"] = Rope(_inv_freq(case["rot"]), interleaved=case["inter"], eps=EPS)
    return s


# ------------------------------------------------------------------ the plain forms

def _normed(x, w):
    x = x.float()
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()


def _rotated(x, pos, rot, inter):
    """Heads [n, h, 256] turned by their rows' positions; angles in 64 bits, a far position times a frequency loses its fraction in 32."""
    ang = pos.double()[:, None, None] * torch.tensor(_inv_freq(rot), dtype=torch.float64, device=x.device)
    c, s = torch.cos(ang).float(), torch.sin(ang).float()
    y = x.clone()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if inter else (x[..., : rot // 2], x[..., rot // 2: rot])
    if inter:
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * s, b * c + a * s
    else:
        y[..., : rot // 2], y[..., rot // 2: rot] = a * c - b * s, b * c + a * s
    return y


def _group_of(s, seq, pos):
    """Pool group of each (row, head), and the row in it."""
    page = s["case"]["page"]
    block = s["table"][seq.long(), (pos // page).long()].long()
    head = torch.arange(HK, device="cuda")
    grp = (block[..., None] * HK + head) * (page // 16) + ((pos % page) // 16).long()[..., None]
    return grp, (pos % 16).long()


def _read(s, out):
    case = s["case"]
    grp, row = _group_of(s, s["seq"], s["pos"])
    got = []
    for pool, fmt, is_v in ((s["k_pool"], case["kt"], False), (s["v_pool"], case["vt"], True)):
        x = _unpack(pool.reshape(-1, 16 * ROW[fmt]), fmt, is_v)
        got.append(x[grp, row[:, None]].to(out))
    return got


def _append(s):
    case = s["case"]
    k = _rotated(_normed(s["k"], s["wk"]), s["pos"], case["rot"], case["inter"])
    q = _rotated(_normed(s["q"], s["wq"]), s["pos"], case["rot"], case["inter"]).to(IO[case["io"]])
    grp, row = _group_of(s, s["seq"], s["pos"])
    for name, x, fmt, is_v in (("k_pool", k, case["kt"], False), ("v_pool", s["v"].float(), case["vt"], True)):
        # a row's bytes as a group of its own would hold them, then those of its place in its group
        one = torch.zeros(x.shape[0] * HK, 16, D, device="cuda")
        flat = row[:, None].expand(-1, HK).reshape(-1)
        one[torch.arange(one.shape[0], device="cuda"), flat] = x.reshape(-1, D)
        one = _pack(one, fmt, is_v)
        at, byte = _mask(fmt, is_v)[flat].nonzero(as_tuple=True)
        s[name].reshape(-1, 16 * ROW[fmt])[grp.reshape(-1)[at], byte] = one[at, byte]
    return q


def _mask(fmt, is_v):
    """Which bytes of a group belong to each of its 16 rows."""
    r, row_q = torch.arange(16, device="cuda"), {"f16": 512, "q8_0": 256, "q4_0": 128}[fmt]
    body = (torch.arange(16 * row_q, device="cuda") // row_q)[None, :] == r[:, None]
    if fmt == "f16":
        return body
    i = torch.arange(128, device="cuda")
    owner = (((i >> 3) & 3) << 1) | (i & 1) | (((i >> 1) & 1) << 3) if is_v else i >> 3
    return torch.cat([(owner[None, :] == r[:, None]).repeat_interleave(2, 1), body], 1)


def _attend(s):
    case, t = s["case"], s["case"]["tok"]
    n, longest = s["lens"].numel(), int(s["lens_host"].max())
    pos = torch.arange(longest, device="cuda", dtype=torch.int32)[None, :].expand(n, -1)
    seq = torch.arange(n, device="cuda")[:, None].expand_as(pos)
    grp, row = _group_of(s, seq, pos)
    k, v = (_unpack(s[p].reshape(-1, 16 * ROW[case[f]]), case[f], p == "v_pool") for p, f in (("k_pool", "kt"), ("v_pool", "vt")))
    k, v = (x[grp, row[..., None]].permute(0, 2, 1, 3) for x in (k, v))  # [n, 4, longest, 256]
    q = s["q"].float().reshape(n, t, HK, GQA, D).permute(0, 2, 1, 3, 4).reshape(n, HK, t * GQA, D)
    logit = torch.matmul(q, k.transpose(-1, -2)) / 16.0
    last = s["lens"][:, None] - t + torch.arange(t, device="cuda")  # the last key that a token sees
    seen = pos[:, None, :] <= last[:, :, None]
    logit = logit.reshape(n, HK, t, GQA, longest).masked_fill(~seen[:, None, :, None, :], float("-inf"))
    top = logit.amax(-1, keepdim=True)
    p = torch.exp(logit - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.reshape(n, HK, t * GQA, longest), v).reshape(n, HK, t, GQA, D) / total
    lse = (top + torch.log(total))[..., 0]
    return {"out": o.permute(0, 2, 1, 3, 4).reshape(n, t, HQ, D).to(IO[case["io"]]), "lse": lse.permute(0, 2, 1, 3).reshape(n, t, HQ)}


def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if op == "norm_rope":
        if own:
            q, k = s["rope"].apply(s["q"], s["k"], s["pos"], s["wq"], s["wk"], q_out=s["q_out"], k_out=s["k_out"])
        else:
            q, k = (_rotated(_normed(s[n], s[w]), s["pos"], case["rot"], case["inter"]).to(IO[case["out"]]) for n, w in (("q", "wq"), ("k", "wk")))
        return {"q": q, "k": k}
    if op == "append":
        if own:
            c = s["cache"]
            q = c.append_rope(s["rope"], s["k"], s["v"], s["seq"], s["pos"], s["table"], k_weight=s["wk"], q=s["q"], q_weight=s["wq"],
                              q_out=s["q_out"])
            k, v = c.read_rows(s["seq"], s["pos"], s["table"], k_out=s["k_out"], v_out=s["v_out"])
        else:
            q = _append(s)
            k, v = _read(s, torch.float16)
        return {"q": q, "k": k, "v": v}
    if op == "read":
        if own:
            k, v = s["cache"].read_rows(s["seq"], s["pos"], s["table"], k_out=s["k_out"], v_out=s["v_out"])
        else:
            k, v = _read(s, IO[case["out"]])
        return {"k": k, "v": v}
    if own:
        out, lse = s["cache"].decode_prefix(s["q"], s["table"], s["lens"], s["lens_host"], s["sizes"], s["pre"], case["tok"], 0.0625,
                                            out=s["out"], lse=s["lse"])
        return {"out": out, "lse": lse}
    return _attend(s)


# ------------------------------------------------------------------ in 64 bits, apart from the above

@functools.lru_cache(None)
def _places(fmt, is_v):
    """For each row of a group: where its scales sit, and where its value i has its byte (and, for 4 bits, which half)."""
    scale = np.zeros((16, 8), np.int64)
    for r in range(16):
        for b in range(8):
            scale[r, b] = 64 * (b // 2) + 16 * ((r % 8) // 2) + 8 * (b % 2) + 4 * (r // 8) + 2 * (r % 2) if is_v else 16 * r + 2 * b
    byte, high = np.zeros((16, D), np.int64), np.zeros(D, bool)
    for i in range(D):
        at = 2 * i if fmt == "f16" else i if fmt == "q8_0" else 16 * (i // 32) + i % 16
        high[i] = fmt == "q4_0" and i % 32 >= 16
        for r in range(16):
            per = {"f16": 512, "q8_0": 256, "q4_0": 128}[fmt]
            byte[r, i] = (0 if fmt == "f16" else 256) + r * per + ((at // 16) ^ (r % 8)) * 16 + at % 16
    return torch.from_numpy(scale).cuda(), torch.from_numpy(byte).cuda(), torch.from_numpy(high).cuda()


def _half_at(flat, at):
    """The binary16 numbers whose bytes start at `at`, in 64 bits."""
    bits = flat[at].long() | (flat[at + 1].long() << 8)
    sign = 1.0 - 2.0 * (bits >> 15).double()
    e, m = (bits >> 10) & 31, (bits & 1023).double()
    return sign * torch.where(e == 0, m * 2.0 ** -24, (1024.0 + m) * torch.pow(2.0, (e - 25).double()))


def _value_rows(pool, fmt, is_v, base, row):
    """Rows in 64 bits: base, the first byte of their groups, row, their place in them."""
    scale, byte, high = _places(fmt, is_v)
    b = base[..., None] + byte[row]
    if fmt == "f16":
        return _half_at(pool, b)
    d = _half_at(pool, base[..., None] + scale[row]).repeat_interleave(32, -1)
    x = pool[b].long()
    x = torch.where(x > 127, x - 256, x) if fmt == "q8_0" else torch.where(high, x >> 4, x & 15) - 8
    return x.double() * d


def _base(s, seq, pos, head, fmt):
    page = s["case"]["page"]
    block = s["table"].long()[seq.long(), pos.long() // page]
    return ((block * HK + head) * page + (pos.long() % page) // 16 * 16) * ROW[fmt]


def _turned(x, w, pos, rot, inter):
    """The norm and the rotation in 64 bits, by complex numbers."""
    x, w = x.double(), w.double()
    x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / D + EPS) * w
    ang = pos.double()[:, None, None] * torch.tensor([THETA ** (-2.0 * i / rot) for i in range(rot // 2)], dtype=torch.float64, device=x.device)
    turn = torch.polar(torch.ones_like(ang), ang)
    head = x[..., :rot]
    z = torch.complex(head[..., 0::2].contiguous(), head[..., 1::2].contiguous()) if inter else torch.complex(head[..., : rot // 2].contiguous(), head[..., rot // 2:].contiguous())
    z = torch.view_as_real(z * turn)
    head = z.flatten(-2) if inter else torch.cat([z[..., 0], z[..., 1]], -1)
    return torch.cat([head, x[..., rot:]], -1)


def _stored(x, fmt):
    """What rows in 64 bits come back as from a cache of this format. The formats' rule is one of 32-bit operations, each rounded:
    every one is done in 64 bits here and rounded to 32 (a product, quotient or sum of two 32-bit numbers rounds the same either way)."""
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


def exact(case, seed):
    global own
    was, own = own, False
    s = prepare(case, seed)
    own = was
    op = case["op"]
    if op == "norm_rope":
        return {n: _turned(s[n], s["w" + n], s["pos"], case["rot"], case["inter"]) for n in ("q", "k")}
    if op == "append":
        k = _turned(s["k"], s["wk"], s["pos"], case["rot"], case["inter"])
        return {"q": _turned(s["q"], s["wq"], s["pos"], case["rot"], case["inter"]), "k": _stored(k, case["kt"]), "v": _stored(s["v"].double(), case["vt"])}
    if op == "read":
        got = {}
        for n, fmt in (("k", case["kt"]), ("v", case["vt"])):
            parts = []
            for h in range(HK):
                base, row = _base(s, s["seq"], s["pos"], h, fmt), (s["pos"] % 16).long()
                parts.append(_value_rows(s[n + "_pool"], fmt, n == "v", base, row))
            got[n] = torch.stack(parts, 1)
        return got
    t, n = case["tok"], len(s["lens_host"])
    out, lse = torch.zeros(n, t, HQ, D, dtype=torch.float64, device="cuda"), torch.zeros(n, t, HQ, dtype=torch.float64, device="cuda")
    for i in range(n):
        length = int(s["lens_host"][i])
        pos = torch.arange(length, device="cuda")
        seq, row = torch.full_like(pos, i), pos % 16
        for h in range(HK):
            k = _value_rows(s["k_pool"], case["kt"], False, _base(s, seq, pos, h, case["kt"]), row)
            v = _value_rows(s["v_pool"], case["vt"], True, _base(s, seq, pos, h, case["vt"]), row)
            for j in range(t):
                m = length - t + 1 + j
                z = s["q"][i, j, GQA * h: GQA * (h + 1)].double() @ k[:m].T / 16
                lse[i, j, GQA * h: GQA * (h + 1)] = torch.logsumexp(z, -1)
                out[i, j, GQA * h: GQA * (h + 1)] = torch.softmax(z, -1) @ v[:m]
    return {"out": out, "lse": lse}
