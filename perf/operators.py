"""The cases that the paged-serving operators of kvq are measured on.

Three operators, the parts of one serving step over paged packed caches:

* ``pages``: the block table, the free list and the slot map of the step, from the
  requests' lengths (``kvq.pages_assign``);
* ``append``: the step's new tokens, a packed ragged batch of [tokens][n_kv][128]
  rows, quantized and bit-packed into the slots of that map
  (``kvq.paged_append_ragged``);
* ``prefix``: decode attention for a batch whose sequences share long prefixes: each
  shared prefix is read once for all its sequences, then merged with every
  sequence's own tokens (``kvq.paged_prefix_decode_attn``).

With ``own`` false, ``run`` computes them in elementary torch operations, in 32 bits;
with ``own`` true it makes the framework's calls. ``exact`` gives the attention in 64
bits, from the packed bits, read bit by bit. Sizes are those of the repository's
workloads (16 query heads on 2 KV heads at K3V3, 28 on 4 at K3V2, 32 on 8 at K2V2, the
4-on-1 tiny reference) and of ordinary serving batches around them.
"""
import math
import random

import numpy as np
import torch

own = False

D, HALF, TILE = 128, 64, 32
DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of a full serving batch: every request gets one token, some a page
        dict(name="pages_decode_256", op="pages", batch=256, new=1, old=4000, page_tiles=2, done=8),
        # a few prompts arrive in a small deployment
        dict(name="pages_prompts_9", op="pages", batch=9, new=700, old=0, page_tiles=1, done=0),
        # chunked prefill of a large batch, with finished requests handing back their pages
        dict(name="pages_prefill_1000", op="pages", batch=1000, new=512, old=3000, page_tiles=4, done=50),
        # one token for each of 16 sequences (28 query heads on 4 KV heads, K3V2)
        dict(name="append_step_16", op="append", batch=16, new=1, old=1000, n_kv=4, bits_k=3, bits_v=2,
             dtype="bf16", page_tiles=4),
        # prompts of odd lengths joining sequences that end inside a tile, K3V3
        dict(name="append_ragged_33", op="append", batch=33, new=77, old=45, n_kv=2, bits_k=3, bits_v=3,
             dtype="fp16", page_tiles=1),
        # fp32 rows, wide codes: a handful of sequences extended by a chunk
        dict(name="append_wide_5", op="append", batch=5, new=301, old=10, n_kv=3, bits_k=5, bits_v=6,
             dtype="fp32", page_tiles=2),
        # a prefill batch of whole prompts (8 KV heads, K2V2)
        dict(name="append_prefill_24", op="append", batch=24, new=2500, old=0, n_kv=8, bits_k=2, bits_v=2,
             dtype="bf16", page_tiles=8),
        # the tiny reference: two sequences, one short shared prompt
        dict(name="prefix_tiny", op="prefix", batch=2, groups=1, prefix=257, suffix=20, n_q=4, n_kv=1,
             bits_k=2, bits_v=2, dtype="fp32", page_tiles=1),
        # a serving step behind one system prompt (28 query heads on 4 KV heads, K3V2)
        dict(name="prefix_serve_16", op="prefix", batch=16, groups=1, prefix=8192, suffix=512, n_q=28,
             n_kv=4, bits_k=3, bits_v=2, dtype="bf16", page_tiles=4),
        # three shared documents, sequences of uneven lengths (32 query heads on 8 KV heads, K2V2)
        dict(name="prefix_docs_48", op="prefix", batch=48, groups=3, prefix=4001, suffix=300, n_q=32,
             n_kv=8, bits_k=2, bits_v=2, dtype="bf16", page_tiles=2),
        # wide codes, half precision, odd sizes
        dict(name="prefix_wide_9", op="prefix", batch=9, groups=2, prefix=2900, suffix=700, n_q=8, n_kv=1,
             bits_k=5, bits_v=4, dtype="fp16", page_tiles=1),
        # many samples of one 128K context (16 query heads on 2 KV heads, K3V3)
        dict(name="prefix_long_64", op="prefix", batch=64, groups=1, prefix=131072, suffix=1500, n_q=16,
             n_kv=2, bits_k=3, bits_v=3, dtype="bf16", page_tiles=8),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["pages", "append", "prefix", "prefix"])
    page_tiles = rng.choice([1, 2, 4, 8])
    if op == "pages":
        batch = _log(rng, 1, 1000)
        return dict(op=op, batch=batch, new=_log(rng, 1, 600), old=_log(rng, 1, 4000),
                    page_tiles=page_tiles, done=rng.randrange(1 + batch // 4))
    if op == "append":
        n_kv, batch = rng.choice([1, 2, 3, 4, 8]), _log(rng, 1, 64)
        return dict(op=op, batch=batch, new=_log(rng, 1, max(2, 400000 // (n_kv * batch) // 2)),
                    old=rng.randrange(3000), n_kv=n_kv, bits_k=rng.randint(1, 6), bits_v=rng.randint(1, 6),
                    dtype=rng.choice(["bf16", "fp16", "fp32"]), page_tiles=page_tiles)
    n_kv, batch = rng.choice([1, 2, 3, 4, 8]), _log(rng, 1, 64)
    return dict(op=op, batch=batch, groups=rng.randint(1, 4), prefix=_log(rng, 1, 32000 // n_kv),
                suffix=_log(rng, 1, 1500), n_q=n_kv * rng.choice([1, 2, 4, 5, 7, 8, 16]), n_kv=n_kv,
                bits_k=rng.randint(1, 6), bits_v=rng.randint(1, 6),
                dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]), page_tiles=page_tiles)


def _lens(case, what, n, mean, least=0):
    """Ragged lengths around `mean`: the first is the longest, one is the least."""
    r = random.Random("%s %d %d %d" % (what, n, mean, case["batch"]))
    if mean <= 1:
        return [mean] * n
    got = [max(least, int(mean * r.uniform(0.2, 1.8))) for _ in range(n)]
    got[0] = max(least, int(1.8 * mean))
    if n > 2:
        got[n // 2] = least
    return got


def _sizes(case):
    if case["op"] == "prefix":
        pre = _lens(case, "prefix", case["groups"], case["prefix"])
        pre[0] = case["prefix"]
        return pre, _lens(case, "suffix", case["batch"], case["suffix"])
    old, new = _lens(case, "old", case["batch"], case["old"]), _lens(case, "new", case["batch"], case["new"])
    if case["op"] == "pages":  # finished requests: no tokens left, their pages go back
        for i in random.Random(case["batch"]).sample(range(case["batch"]), case["done"]):
            old[i] = new[i] = 0
    return old, new


def _rec_words(case):
    return D * (case["bits_k"] + case["bits_v"]) + TILE


def work(case):
    a, b = _sizes(case)
    if case["op"] == "pages":
        span = TILE * case["page_tiles"]
        pages = sum(-(-(x + y) // span) - -(-x // span) for x, y in zip(a, b))
        return {"bytes": 16 * len(a) + 4 * (len(a) + 1) + 8 * pages + 12 * sum(b), "flops": 0}
    rec = 4 * _rec_words(case)
    if case["op"] == "append":
        size = 4 if case["dtype"] == "fp32" else 2
        rows = sum(b) * case["n_kv"]
        return {"bytes": rows * (2 * D * size + rec / TILE) + 8 * sum(b), "flops": rows * 2 * D * 7}
    size = 4 if case["dtype"] == "fp32" else 2
    tokens = sum(a) + sum(b)
    groups = _group_start(case)
    pairs = sum(b) + sum(n * (e - s) for n, s, e in zip(a, groups[:-1], groups[1:]))
    return {"bytes": tokens * case["n_kv"] * rec / TILE + 2 * case["batch"] * case["n_q"] * D * size,
            "flops": 4 * D * pairs * case["n_q"]}


def _group_start(case):
    n, k = case["batch"], case["groups"]
    r = random.Random("groups %d %d" % (n, k))
    return [0] + sorted(r.randint(0, n) for _ in range(k - 1)) + [n]


# ------------------------------------------------- codebooks, plans, tables
_books = {}


def _codebook(bits):
    """Gaussian Lloyd-Max levels of 2^bits, rounded to fp16: (levels, midpoints) in fp32."""
    if bits not in _books:
        n = 1 << (bits - 1)  # the positive half; the other is its mirror image
        # companded start, then Newton's method on c_m = E[x | cell m] (tridiagonal)
        inv = lambda p: math.sqrt(2.0) * float(torch.erfinv(torch.tensor(2 * p - 1, dtype=torch.float64)))  # noqa: E731
        c = np.array([math.sqrt(3.0) * inv(0.5 + (m + 0.5) / (2 * n)) for m in range(n)])
        pdf = lambda x: np.exp(-0.5 * x * x) / math.sqrt(2 * math.pi)  # noqa: E731
        tail = np.vectorize(lambda x: 0.5 * math.erfc(x / math.sqrt(2)))
        for _ in range(200):
            t = np.concatenate([[0.0], 0.5 * (c[1:] + c[:-1]), [40.0]])
            mass, mom = tail(t[:-1]) - tail(t[1:]), pdf(t[:-1]) - pdf(t[1:])
            mean = mom / mass
            # d mean_m / d t_lower, d t_upper
            lo, hi = pdf(t[:-1]) * (mean - t[:-1]) / mass, pdf(t[1:]) * (t[1:] - mean) / mass
            lo[0] = 0.0  # the border at zero does not move
            hi[-1] = 0.0
            J = np.eye(n) - 0.5 * (np.diag(lo + hi) + np.diag(hi[:-1], 1) + np.diag(lo[1:], -1))
            step = np.linalg.solve(J, mean - c)
            c = c + step
            if np.max(np.abs(step)) < 1e-13:
                break
        lv = np.concatenate([-c[::-1], c]).astype(np.float16).astype(np.float64)
        _books[bits] = (lv.astype(np.float32), (0.5 * (lv[1:] + lv[:-1])).astype(np.float32))
    return _books[bits]


def _distortion(bits):
    if bits == 0:
        return 1.0
    lv, th = (x.astype(np.float64) for x in _codebook(bits))
    t = np.concatenate([[-40.0], th, [40.0]])
    cdf = np.array([0.5 * math.erfc(-x / math.sqrt(2)) for x in t])
    pdf = np.exp(-0.5 * t * t) / math.sqrt(2 * math.pi)
    m0, m1 = np.diff(cdf), -np.diff(pdf)
    m2 = m0 - np.diff(t * pdf)
    return float(np.sum(m2 - 2 * lv * m1 + lv * lv * m0))


_gain = []


def _plan(energy, bits_k, bits_v, rng):
    """One KV head's plan: integer widths by greedy gain, scales, order, segments, signs."""
    if not _gain:
        d = [_distortion(b) for b in range(9)]
        _gain.extend([d[b] - d[b + 1] for b in range(8)] + [0.0])
    width = np.zeros(HALF, np.int64)
    gain = np.array(_gain)
    for _ in range(HALF * bits_k):
        g = np.where(width < 8, energy * gain[width], -1.0)
        width[int(np.argmax(g))] += 1
    a = np.sqrt(energy / (2 * energy.sum()))
    order = [j for w in range(8, 0, -1) for j in range(HALF) if width[j] == w]
    seg = np.concatenate([[0], np.cumsum([2 * width[j] for j in order])])
    return dict(width=width, a_hat=a.astype(np.float32), g=(1.0 / a).astype(np.float32), order=order,
                seg=seg, sign=rng.integers(0, 2, D), bits_k=bits_k, bits_v=bits_v, energy=energy)


def _plan_record(p, head):
    """The plan as the 1024-byte record of the C interface."""
    r = np.zeros(1024, np.uint8)
    put = lambda off, v, t: r.__setitem__(slice(off, off + np.asarray(v, t).nbytes), np.atleast_1d(np.asarray(v, t)).view(np.uint8))  # noqa: E731
    order, n = p["order"], len(p["order"])
    put(0, [0x5051564B], "<u4")
    put(4, [p["bits_k"], p["bits_v"], n, 0, head, D * p["bits_k"], D * p["bits_v"]], "<i4")
    put(32, p["g"], "<f4")
    put(288, p["a_hat"], "<f4")
    put(544, p["width"], "u1")
    put(608, order, "u1")
    put(672, p["seg"], "<u2")
    steps = []  # (width, first rank, count): runs of one width in groups of four
    i = 0
    while i < n:
        w = p["width"][order[i]]
        k = 1
        while k < 4 and i + k < n and p["width"][order[i + k]] == w:
            k += 1
        steps.append((w, i, k))
        i += k
    put(802, [len(steps)], "u1")
    for off, col in ((804, 0), (836, 1), (868, 2)):
        put(off, [s[col] for s in steps], "u1")
    put(900, np.packbits(p["sign"].astype(np.uint8), bitorder="little").view("<u4"), "<u4")
    put(920, [p["energy"].sum()], "<f8")
    first = [i for i, s in enumerate(steps) if i == 0 or steps[i - 1][0] != s[0]]
    last = [b - 1 for b in first[1:] + [len(steps)]]
    put(928, [len(first)], "u1")
    put(936, [steps[i][0] for i in first], "u1")
    put(944, first, "u1")
    put(952, [b - a + 1 for a, b in zip(first, last)], "u1")
    put(960, [steps[b][2] for b in last], "u1")
    put(968, [p["seg"][steps[i][1]] for i in first], "<u2")
    return r


def _tables(plans):
    """Where each code of a tile record sits: first bit, width, level table; per head."""
    n_kv = len(plans)
    bit = np.zeros((2, n_kv, TILE, D), np.int64)
    wid = np.zeros((2, n_kv, D), np.int64)
    t = np.arange(TILE)
    sk, sv = 4 * (t % 8) + t // 8, 8 * ((t % 8) // 2) + 2 * (t // 8) + t % 2
    for h, p in enumerate(plans):
        wid[0, h] = np.tile(p["width"], 2)
        wid[1, h] = p["bits_v"]
        for r, j in enumerate(p["order"]):
            w = int(p["width"][j])
            bit[0, h, :, j] = 32 * p["seg"][r] + sk * 2 * w
            bit[0, h, :, j + HALF] = bit[0, h, :, j] + w
        bit[1, h] = 32 * D * p["bits_k"] + 32 * p["bits_v"] * np.arange(D)[None] + (sv * p["bits_v"])[:, None]
    level, thr = np.zeros((9, 256), np.float32), np.full((9, 255), np.inf, np.float32)
    for b in range(1, 9):
        level[b, :1 << b], thr[b, :(1 << b) - 1] = _codebook(b)
    up = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(DEV)  # noqa: E731
    return dict(bit=up(bit), wid=up(wid), level=up(level), thr=up(thr[wid.reshape(-1)]),
                g=up(np.stack([np.tile(p["g"], 2) for p in plans])),
                a_hat=up(np.stack([np.tile(p["a_hat"], 2) for p in plans])),
                flip=up(np.stack([1.0 - 2.0 * p["sign"] for p in plans]).astype(np.float32)))


# ------------------------------------------------------------- plain forms
def _hadamard(y):
    """Walsh-Hadamard transform of the last axis, stages of distance 1, 2, ..., 64."""
    for e in range(7):
        v = y.view(*y.shape[:-1], HALF >> e, 2, 1 << e)
        y = torch.stack([v[..., 0, :] + v[..., 1, :], v[..., 0, :] - v[..., 1, :]], -2).flatten(-3)
    return y


def _norm(x):
    """fp16 norms of rows of 128 in the format's order of sums, and their reciprocals."""
    s = x * x
    s = ((s[..., :32] + s[..., 32:64]) + s[..., 64:96]) + s[..., 96:]
    s = s[..., :16] + s[..., 16:]
    s = s[..., :8] + s[..., 8:]
    s = s[..., :4] + s[..., 4:]
    s = s[..., :2] + s[..., 2:]
    n = (s[..., 0] + s[..., 1]).sqrt().clamp(max=65504.0).half()
    return n, torch.where(n > 0, 1.0 / n.float(), 0.0)


def _codes(T, which, z):
    """Codes of z [tokens, n_kv, 128]: the number of its width's thresholds below it."""
    n, rows = z.shape[0], z.shape[1] * D
    thr = T["thr"].view(2, rows, 255)[which]
    return torch.searchsorted(thr, z.reshape(n, rows).t().contiguous()).t().reshape(z.shape)


def _append_plain(T, pool, k, v, slots, seq, old_len, first):
    """Tokens k, v [n, n_kv, 128] into the tile records pool [records, n_kv, words] (int32) at
    their slots; `seq`: the token's sequence, old_len: lengths before, first: each sequence's
    first token. Slots below zero are left out."""
    live = (slots >= 0).nonzero()[:, 0]
    k, v, slots, seq = k[live].float(), v[live].float(), slots[live], seq[live]
    n, n_kv, words = len(live), pool.shape[1], pool.shape[2]
    nk, rk = _norm(k)
    nv, rv = _norm(v)
    zk = (k * rk[..., None]) * T["g"]
    zv = _hadamard(v * T["flip"]) * rv[..., None]
    codes = torch.stack([torch.where(nk[..., None] > 0, _codes(T, 0, zk), 0),
                         torch.where(nv[..., None] > 0, _codes(T, 1, zv), 0)])
    rec, at = torch.unique(slots // TILE, return_inverse=True)
    pos = slots % TILE
    bit, wid = T["bit"][:, :, pos].transpose(1, 2), T["wid"][:, None].expand(2, n, n_kv, D)
    word, shift = bit >> 5, bit & 31
    row = (at[:, None] * n_kv + torch.arange(n_kv, device=DEV)) * (words + 1)
    to = (row[None, ..., None] + word).reshape(-1)
    new = torch.zeros(len(rec) * n_kv * (words + 1), dtype=torch.int64, device=DEV)
    mask = torch.zeros_like(new)
    for buf, x in ((new, codes), (mask, (1 << wid) - 1)):  # a code may reach into the next word
        x = (x << shift).reshape(-1)
        buf.index_add_(0, to, x & 0xFFFFFFFF)
        buf.index_add_(0, to + 1, x >> 32)
    # norms: 16-bit fields behind the code words
    base = words - TILE
    for i, x in enumerate((nk, nv)):
        to = (row + base + 16 * i + (pos // 2)[:, None]).reshape(-1)
        sh = (16 * (pos % 2))[:, None]
        new.index_add_(0, to, ((x.view(torch.int16).long() & 0xFFFF) << sh).reshape(-1))
        mask.index_add_(0, to, (torch.full_like(x, 0, dtype=torch.int64) + (0xFFFF << sh)).reshape(-1))
    new, mask = (b.view(len(rec), n_kv, words + 1)[..., :words] for b in (new, mask))
    # a tile that held no token before starts from zero code words
    held = old_len[seq] > old_len[seq] + (torch.arange(len(slots), device=DEV) - first[seq]) - pos
    kept = torch.zeros(len(rec), dtype=torch.bool, device=DEV).index_put_((at,), held)
    old = pool[rec].long() & 0xFFFFFFFF
    old[..., :base] = torch.where(kept[:, None, None], old[..., :base], 0)
    got = (old & ~mask) | new
    pool[rec] = torch.where(got >= 1 << 31, got - (1 << 32), got).int()


def _assign_plain(table, held, ids, ring, lens, n_new, n_slots, span):
    """Block table, pages held, free ring and slot map for lens + n_new tokens."""
    n_pages, P = len(ids), table.shape[1]
    cu = torch.nn.functional.pad(n_new.long().cumsum(0), (1, 0))
    need = (lens.long() + n_new + span - 1) // span
    ok = (need <= P) & (cu[1:] <= n_slots)
    j = torch.arange(P, device=DEV)
    head, count = ring[0], ring[1]
    back = ok[:, None] & (j >= need[:, None]) & (j < held[:, None])
    freed = table[back]
    ids[(head + count + torch.arange(len(freed), device=DEV)) % n_pages] = freed
    avail = count + len(freed)
    take = torch.where(ok, (need - held).clamp(min=0), 0)
    ok = ok & ((take.cumsum(0) <= avail) | (take == 0))
    take = torch.where(ok, take, 0)
    first = take.cumsum(0) - take
    got = ids[(head + first[:, None] + j - held[:, None]) % n_pages]
    fill = ok[:, None] & (j >= held[:, None]) & (j < need[:, None])
    table.copy_(torch.where(fill, got, torch.where(back, -1, table)))
    held.copy_(torch.where(ok, need, held))
    ring.copy_(torch.stack([(head + take.sum()) % n_pages, avail - take.sum()]))
    seq = torch.repeat_interleave(torch.arange(len(lens), device=DEV), n_new.long(), output_size=n_slots)
    pos = lens[seq].long() + torch.arange(n_slots, device=DEV) - cu[seq]
    page = table[seq, (pos // span).clamp(max=P - 1)].long()
    slots = torch.where(ok[seq], page * span + pos % span, -1)
    return cu.int(), slots, pos.int(), seq


def _unpack(T, recs, which):
    """Levels [n, n_kv, 32, 128] of the tile records recs [n, n_kv, words] (int32)."""
    bit, wid = T["bit"][which], T["wid"][which]
    w = torch.nn.functional.pad(recs, (0, 1)).long() & 0xFFFFFFFF
    at = (bit >> 5).reshape(1, bit.shape[0], -1).expand(len(recs), -1, -1)
    x = w.gather(2, at) | (w.gather(2, at + 1) << 32)
    x = (x.view(len(recs), *bit.shape) >> (bit & 31)) & ((1 << wid) - 1)[:, None]
    return T["level"][wid[:, None].expand_as(bit), x]


def _cache(T, pool, table, n_tokens, page_tiles):
    """k^ and rotated v^ [rows, n_kv, tokens, 128] of the rows of a block table, in fp32."""
    n_tiles = -(-n_tokens // TILE)
    tile = torch.arange(n_tiles, device=DEV)
    rec = table[:, tile // page_tiles].long().clamp(min=0) * page_tiles + tile % page_tiles
    recs = pool[rec.reshape(-1)]
    norms = recs[..., -TILE:].contiguous().view(torch.float16).float().view(*recs.shape[:2], 2, TILE, 1)
    k = _unpack(T, recs, 0) * T["a_hat"][:, None] * norms[:, :, 0]
    v = _unpack(T, recs, 1) * norms[:, :, 1]
    shape = (len(table), n_tiles, recs.shape[1], TILE, D)
    return [x.view(shape).transpose(1, 2).reshape(shape[0], shape[2], -1, D) for x in (k, v)]


def _prefix_plain(s):
    T, q = s["T"], s["q"].float()
    B, n_q, n_kv = q.shape[0], q.shape[1], s["n_kv"]
    G, n_groups = n_q // n_kv, len(s["prefix_lens"])
    q = q.view(B, n_kv, G, D) / math.sqrt(D)
    start = s["group_start"].long()
    b = torch.arange(B, device=DEV)
    g = (b[:, None] >= start[1:]).sum(1)
    i = b - start[g]
    kp, vp = _cache(T, s["pool"], s["prefix_table"], s["max_prefix"], s["page_tiles"])
    ks, vs = _cache(T, s["pool"], s["table"], s["max_len"], s["page_tiles"])
    # the sequences of a group, side by side: [groups, n_kv, sequences * G, 128]
    qg = torch.zeros(n_groups, n_kv, s["most"], G, D, device=DEV)
    qg[g, :, i] = q
    sp = qg.flatten(2, 3) @ kp.transpose(2, 3)
    ss = q @ ks.transpose(2, 3)
    t = torch.arange(sp.shape[3], device=DEV)
    sp = sp.masked_fill_((t >= s["prefix_lens"][:, None])[:, None, None], -math.inf)
    ss = ss.masked_fill_((torch.arange(ss.shape[3], device=DEV) >= s["lens"][:, None])[:, None, None], -math.inf)
    mp = sp.amax(3).view(n_groups, n_kv, -1, G)
    m = torch.maximum(mp[g, :, i], ss.amax(3))
    m = torch.where(m == -math.inf, 0.0, m)
    mg = torch.zeros_like(mp)
    mg[g, :, i] = m
    sp = sp.sub_(mg.flatten(2, 3)[..., None]).exp_()
    ss = ss.sub_(m[..., None]).exp_()
    lsum = sp.sum(3).view_as(mp)[g, :, i] + ss.sum(3)
    o = (sp @ vp).view(n_groups, n_kv, -1, G, D)[g, :, i] + ss @ vs
    o = _hadamard(o) * T["flip"][:, None] / (D * torch.where(lsum > 0, lsum, 1.0)[..., None])
    return o.reshape(B, n_q, D).to(s["q"].dtype)


# ----------------------------------------------------------------- inputs
def _rows(n, plans, dtype, gen):
    """Post-RoPE keys of the plans' block energies, one coordinate in 100 an outlier, and values."""
    sig = torch.tensor(np.stack([np.tile(np.sqrt(p["energy"] / 2), 2) for p in plans]), device=DEV).float()
    k = torch.randn(n, len(plans), D, generator=gen, device=DEV) * sig
    out = torch.rand(n, len(plans), D, generator=gen, device=DEV) < 0.01
    v = torch.randn(n, len(plans), D, generator=gen, device=DEV)
    return torch.where(out, 8 * k, k).to(dtype), v.to(dtype)


def _page_state(rows, need, spare, extra, rng):
    """Rows holding their first `need` pages of a shuffled pool; the rest is the free ring."""
    total, wide = int(sum(need)), int(max(need)) + extra
    n_pages = total + spare
    ids = torch.from_numpy(rng.permutation(n_pages).astype(np.int32)).to(DEV)
    # one buffer: table, held, free ids and ring are views of it
    sizes = [rows * wide, rows, n_pages]
    ints = sum(sizes) + (sum(sizes) & 1)
    flat = torch.zeros(4 * ints + 16, dtype=torch.uint8, device=DEV)
    state = dict(flat=flat, n_pages=n_pages, wide=wide, rows=rows)
    table, held, free, ring = _page_views(state, flat)
    need = torch.tensor(need, device=DEV)
    table.fill_(-1)
    j = torch.arange(wide, device=DEV)
    table[j < need[:, None]] = ids[:total]
    held.copy_(need)
    free[:spare] = ids[total:]
    ring[1] = spare
    return state


def _page_views(state, flat):
    rows, wide, n = state["rows"], state["wide"], state["n_pages"]
    ints = flat[:-16].view(torch.int32)
    return (ints[:rows * wide].view(rows, wide), ints[rows * wide:rows * (wide + 1)],
            ints[rows * (wide + 1):rows * (wide + 1) + n], flat[-16:].view(torch.int64))


def prepare(case, seed):
    rng, gen = np.random.default_rng(seed), torch.Generator(device=DEV).manual_seed(seed)
    a, b = _sizes(case)
    span = TILE * case["page_tiles"]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    if case["op"] == "pages":
        need = [-(-x // span) for x in a]
        gone = random.Random(case["batch"]).sample(range(case["batch"]), case["done"])
        held = [1 + case["old"] // span if i in gone else n for i, n in enumerate(need)]
        grow = sum(-(-(x + y) // span) for x, y in zip(a, b)) - sum(need)
        state = _page_state(len(a), held, grow + 5, 2 + max(b) // span, rng)
        return dict(op="pages", pages=state, now=state["flat"].clone(), lens=i32(a), n_new=i32(b),
                    n_slots=sum(b), page_tiles=case["page_tiles"])
    energy = np.exp(-np.arange(HALF) / 6.0 + rng.standard_normal((case["n_kv"], HALF)))
    plans = [_plan(e, case["bits_k"], case["bits_v"], rng) for e in energy]
    T = _tables(plans)
    state = dict(op=case["op"], T=T, n_kv=case["n_kv"], bits_k=case["bits_k"], bits_v=case["bits_v"],
                 page_tiles=case["page_tiles"],
                 plans=torch.from_numpy(np.stack([_plan_record(p, h) for h, p in enumerate(plans)])).to(DEV))
    dtype = DTYPES[case["dtype"]]

    def fill(pool, pages, rows, lens, n_new):
        table, held, free, ring = _page_views(pages, pages["flat"])
        cu, slots, pos, seq = _assign_plain(table, held, free, ring, lens, n_new, rows, span)
        return table, cu, slots, seq

    words = _rec_words(case)
    if case["op"] == "append":
        need = [-(-x // span) for x in a]
        total = sum(-(-(x + y) // span) for x, y in zip(a, b))
        pages = _page_state(len(a), need, total - sum(need) + 3, 2 + max(b) // span, rng)
        pool = torch.zeros(pages["n_pages"] * case["page_tiles"], case["n_kv"], words, dtype=torch.int32,
                           device=DEV)
        lens, n_new = i32(a), i32(b)
        # the tokens already in the last, part-filled tile of each sequence
        part = lens % TILE
        table, cu, slots, seq = fill(pool, pages, int(part.sum()), lens - part, part)
        k, v = _rows(len(slots), plans, dtype, gen)
        if len(slots):
            _append_plain(T, pool, k, v, slots, seq, lens - part, cu[:-1])
        table, cu, slots, seq = fill(pool, pages, sum(b), lens, n_new)
        k, v = _rows(sum(b), plans, dtype, gen)
        return dict(state, pool=pool, k=k, v=v, slots=slots, seq=seq, cu=cu, lens0=lens, lens=lens.clone(),
                    n_pages=pages["n_pages"], batch=len(a))
    lens, n_groups = i32([0] * (len(a) + len(b))), len(a)
    need = [-(-x // span) for x in a + b]
    pages = _page_state(len(a + b), [0] * len(a + b), sum(need) + 2, max(need) + 1, rng)
    pool = torch.zeros(pages["n_pages"] * case["page_tiles"], case["n_kv"], words, dtype=torch.int32, device=DEV)
    table, cu, slots, seq = fill(pool, pages, sum(a + b), lens, i32(a + b))
    for at in range(0, len(slots), 32768):  # the caches are filled in parts: whole tiles but for the last
        k, v = _rows(len(slots[at:at + 32768]), plans, torch.bfloat16, gen)
        cut = slice(at, at + 32768)
        done = (at - cu[:-1]).clamp(min=0)
        _append_plain(T, pool, k, v, slots[cut], seq[cut], done, (cu[:-1] - at).clamp(min=0))
    start = _group_start(case)
    q = torch.randn(case["batch"], case["n_q"], D, generator=gen, device=DEV).to(dtype)
    return dict(state, pool=pool, prefix_table=table[:n_groups].contiguous(), table=table[n_groups:].contiguous(),
                prefix_lens=i32(a), lens=i32(b), group_start=i32(start), max_prefix=max(max(a), 1),
                max_len=max(max(b), 1), most=max(y - x for x, y in zip(start, start[1:])), q=q,
                n_pages=pages["n_pages"])


# -------------------------------------------------------------------- run
def _handle(s):
    """What a user's program keeps between calls: the configuration, page descriptions, buffers."""
    if "handle" not in s:
        from bit_kv_cache_19_b200 import kvq

        h = s["handle"] = dict(kvq=kvq, status=torch.zeros(1, dtype=torch.int32, device=DEV))
        if s["op"] == "pages":
            table, held, free, ring = _page_views(s["pages"], s["now"])
            h["state"] = kvq.make_page_state(table, held, free, ring, s["page_tiles"])
            h["cu"] = torch.empty(len(s["lens"]) + 1, dtype=torch.int32, device=DEV)
            h["slots"] = torch.empty(s["n_slots"], dtype=torch.int64, device=DEV)
            h["pos"] = torch.empty(s["n_slots"], dtype=torch.int32, device=DEV)
            h["ws"] = torch.zeros(kvq.pages_assign_workspace_bytes(len(s["lens"])), dtype=torch.uint8, device=DEV)
            return h
        h["cfg"] = cfg = kvq.make_cfg(s["n_kv"], s["bits_k"], s["bits_v"])
        batch = s["batch"] if s["op"] == "append" else len(s["lens"])
        h["plans"] = torch.full((batch,), s["plans"].data_ptr(), dtype=torch.int64, device=DEV)
        if s["op"] == "prefix":
            h["prefix"] = kvq.make_pages(s["pool"], s["prefix_table"], s["n_pages"], s["page_tiles"])
            h["pages"] = kvq.make_pages(s["pool"], s["table"], s["n_pages"], s["page_tiles"])
            n = kvq.prefix_decode_workspace_bytes(cfg, batch, s["q"].shape[1], len(s["prefix_lens"]))
            h["ws"] = torch.zeros(n, dtype=torch.uint8, device=DEV)
            h["out"] = torch.empty_like(s["q"])
    return s["handle"]


def run(s):
    if s["op"] == "pages":
        s["now"].copy_(s["pages"]["flat"])  # every pass starts from the same pages
        table, held, free, ring = _page_views(s["pages"], s["now"])
        if own:
            h = _handle(s)
            h["kvq"].pages_assign(h["state"], s["lens"], s["n_new"], h["cu"], h["slots"], h["pos"], h["ws"],
                                  h["status"])
            return dict(table=table, held=held, free=free, ring=ring, cu=h["cu"], slots=h["slots"], pos=h["pos"])
        cu, slots, pos, _ = _assign_plain(table, held, free, ring, s["lens"], s["n_new"], s["n_slots"],
                                          TILE * s["page_tiles"])
        return dict(table=table, held=held, free=free, ring=ring, cu=cu, slots=slots, pos=pos)
    if s["op"] == "append":
        s["lens"].copy_(s["lens0"])
        if own:
            h = _handle(s)
            h["kvq"].paged_append_ragged(h["cfg"], h["plans"], s["k"], s["v"], s["cu"], s["slots"], s["pool"],
                                         s["n_pages"], s["page_tiles"], s["lens"], h["status"])
        else:
            _append_plain(s["T"], s["pool"], s["k"], s["v"], s["slots"], s["seq"], s["lens"], s["cu"][:-1].long())
            s["lens"] += s["cu"][1:] - s["cu"][:-1]
        return dict(pool=s["pool"], lens=s["lens"])
    if own:
        h = _handle(s)
        h["kvq"].paged_prefix_decode_attn(h["cfg"], h["plans"], h["prefix"], s["prefix_lens"], s["group_start"],
                                          s["max_prefix"], h["pages"], s["lens"], s["max_len"], s["q"], h["out"],
                                          h["ws"], h["status"])
        return h["out"]
    return _prefix_plain(s)


# ------------------------------------------------------------------ exact
def exact(case, seed):
    """The attention's outputs in 64 bits: codes read bit by bit from the packed records, one
    sequence and head at a time. Tables, slots, packed words and lengths are whole numbers."""
    if case["op"] == "pages":
        return None
    s = prepare(case, seed)
    if case["op"] == "append":
        return None
    n_kv, G, bk, bv = s["n_kv"], case["n_q"] // case["n_kv"], s["bits_k"], s["bits_v"]
    rec = s["plans"].cpu().numpy()
    pool = s["pool"].cpu().numpy()
    tables = [s["prefix_table"].cpu().numpy(), s["table"].cpu().numpy()]
    H = np.array([[1.0]])
    while len(H) < D:
        H = np.block([[H, H], [H, -H]])

    def tokens(which, row, h, n):
        """k^, v^ [n, 128] of one row and head, float64 on the GPU."""
        n_tiles = -(-n // TILE)
        tile = np.arange(n_tiles)
        at = tables[which][row, tile // s["page_tiles"]].astype(np.int64) * s["page_tiles"] + tile % s["page_tiles"]
        raw = np.ascontiguousarray(pool[at, h])
        bits = np.unpackbits(raw.view(np.uint8), axis=1, bitorder="little")
        norms = raw[:, -TILE:].copy().view(np.float16).astype(np.float64)
        p = rec[h]
        width, a_hat = p[544:608], p[288:544].view("<f4").astype(np.float64)
        seg, sign = p[672:802].view("<u2"), 1.0 - 2.0 * np.unpackbits(p[900:916], bitorder="little")
        k, v = np.zeros((n_tiles, TILE, D)), np.zeros((n_tiles, TILE, D))
        slot_k = [4 * (t % 8) + t // 8 for t in range(TILE)]
        slot_v = [8 * ((t % 8) // 2) + 2 * (t // 8) + t % 2 for t in range(TILE)]

        def field(x, n_bits):  # [n_tiles, 32, n_bits] bits -> numbers
            return (x.astype(np.int64) << np.arange(n_bits)).sum(-1)
        for r in range(int(p[12:16].view("<i4")[0])):
            j = int(p[608 + r])
            w = int(width[j])
            f = bits[:, 32 * int(seg[r]):32 * int(seg[r]) + 64 * w].reshape(n_tiles, TILE, 2, w)[:, slot_k]
            lv = _codebook(w)[0].astype(np.float64)
            k[:, :, j] = lv[field(f[:, :, 0], w)] * a_hat[j]
            k[:, :, j + HALF] = lv[field(f[:, :, 1], w)] * a_hat[j]
        lv = _codebook(bv)[0].astype(np.float64)
        for i in range(D):
            at = 32 * (D * bk + i * bv)
            v[:, :, i] = lv[field(bits[:, at:at + 32 * bv].reshape(n_tiles, TILE, bv)[:, slot_v], bv)]
        k *= norms[:, :TILE, None]
        v *= norms[:, TILE:, None]
        k, v = (torch.from_numpy(x.reshape(-1, D)[:n]).to(DEV) for x in (k, v))
        return k, v @ torch.from_numpy(H * sign / D).to(DEV)

    if sum(map(sum, _sizes(case))) * n_kv > 500_000:
        return None  # the bits are read one by one on the host: over about 20 seconds
    q = s["q"].double()
    out = torch.zeros_like(q)
    start = s["group_start"].tolist()
    for h in range(n_kv):
        for g, (lo, hi) in enumerate(zip(start, start[1:])):
            if hi == lo:
                continue
            kp, vp = tokens(0, g, h, int(s["prefix_lens"][g]))
            for b in range(lo, hi):
                ks, vs = tokens(1, b, h, int(s["lens"][b]))
                k, v = torch.cat([kp, ks]), torch.cat([vp, vs])
                if len(k):
                    x = q[b, h * G:(h + 1) * G] @ k.T / math.sqrt(D)
                    out[b, h * G:(h + 1) * G] = torch.softmax(x, -1) @ v
    return out
