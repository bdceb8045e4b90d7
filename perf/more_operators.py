"""The measured cases of the 4-bit cache's operators and of its pages'.

Three operators of serving the hybrid's attention layers from a paged cache in
4 bits: ``store`` (rows of k and v into the cache and back out of it),
``attn`` (attention of a batch through page tables over that cache) and
``pages`` (growing and trimming sequences, forking them, compacting the pool).
``run`` computes them in plain torch operations, or, with ``own`` set, through
gated_deltanet_linear_06_gb300's public calls; ``exact`` gives the same
outputs from the definitions, in 64 bits where they are computed numbers.

The cache.  uint8 [pages][h_kv][page / 16][18 d]: 16 tokens of a head are 18 d
bytes, 8 d of K codes, 8 d of V codes, and bf16 scales [token][K groups | V
groups] of 32 channels each.  A group's scale is s = -m / 8, m its element of
largest magnitude; a code is clamp(rint(x / s), -8, 7) + 8.  Codes stand eight
to a 32-bit word, the words in 16-byte vectors [vector][32 lanes][4]: word
w = (token / 8) * (d / 32) + channel / 32 is in vector w / 4, place w % 4, and
  K: lane (token % 8) * 4 + (channel % 32) / 8, nibble (channel % 8) / 2 +
     4 * (channel % 2), the word then turned left by 3 bits;
  V: lane (channel % 32) / 4 * 4 + (token % 8) / 2, nibble channel % 4 + 4 * (token % 2).
"""
from __future__ import annotations

import math

import torch

own = False

BF, F32, F64, I32, U8 = torch.bfloat16, torch.float32, torch.float64, torch.int32, torch.uint8
TINY = 2.0 ** -90      # a group whose largest magnitude is below this is held as zeros


# ---------------------------------------------------------------- the cases

def _store(name, tokens, h_kv, d, page, f32_out=False, runs=True):
    """runs: the rows follow each other through the pages, as a prompt's do; else
    each token is another sequence's next one."""
    return {"name": name, "op": "store", "tokens": tokens, "h_kv": h_kv, "d": d, "page": page,
            "f32_out": f32_out, "runs": runs}


def _attn(name, batch, steps, h_q, h_kv, d, lo, hi, page=64, gated=True):
    return {"name": name, "op": "attn", "batch": batch, "steps": steps, "h_q": h_q, "h_kv": h_kv,
            "d": d, "lo": lo, "hi": hi, "page": page, "gated": gated}


def _pages(name, op, seqs, lo, hi, page, pages, layers=0, h_kv=2, d=256, kv4=True, steps=0, children=0):
    """pages: of the pool; layers: caches that share its tables; kv4: 4-bit caches,
    else bf16 ones; children: sequences forked off the first `seqs`, in turn."""
    return {"name": name, "op": op, "seqs": seqs, "lo": lo, "hi": hi, "page": page, "pages": pages,
            "layers": layers, "h_kv": h_kv, "d": d, "kv4": kv4, "steps": steps, "children": children}


def listed():
    return [
        # one decode step of a full server batch: a row each, all over the pool; launch latency
        _store("store_decode_256", 256, 2, 256, 64, runs=False),
        # a prompt chunk of odd length in small pages, read back in fp32
        _store("store_chunk_2049", 2049, 8, 128, 16, f32_out=True),
        # a whole long prompt
        _store("store_prompt_32768", 32768, 2, 256, 64),
        # one user's turn after a short prompt: latency
        _attn("attn_b1_833", 1, 1, 16, 2, 256, 833, 833),
        # verifying 4 drafted tokens of 17 sequences, small pages, odd lengths
        _attn("attn_b17_s4_6001", 17, 4, 32, 8, 128, 4, 6001, page=16, gated=False),
        # one very long document: the work of one sequence over the whole GPU
        _attn("attn_b1_131072", 1, 1, 32, 8, 128, 131072, 131072, gated=False),
        # narrow heads, ragged and short sequences, large pages
        _attn("attn_b96_d64", 96, 1, 64, 8, 64, 1, 2900, page=128, gated=False),
        # the largest: a full server batch with contexts of all lengths
        _attn("attn_b256_8000", 256, 1, 16, 2, 256, 100, 8000),
        # a speculative step's tables: 4 tokens more for 256 sequences, all of them taken back
        _pages("pages_step_256", "step", 256, 100, 8000, 64, 65536, steps=4),
        # 48 answers sampled from one prompt whose last page is half full, 12 layers
        _pages("pages_fork_48", "fork", 1, 5003, 5003, 64, 4096, layers=12, children=48),
        # a beam of 5 over bf16 caches in small pages
        _pages("pages_fork_5_bf16", "fork", 2, 170, 333, 16, 1021, layers=8, h_kv=8, d=128, kv4=False, children=5),
        # a pool with holes all over it drawn together, 12 layers
        _pages("pages_compact_12", "compact", 64, 100, 8000, 64, 6144 + 512, layers=12),
    ]


def _logint(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["store", "store", "attn", "attn", "attn", "step", "fork", "compact"])
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "store":
        d, h = rng.choice([64, 128, 256]), rng.choice([1, 2, 4, 8])
        tokens = min(_logint(rng, 1, 32768), 32768 * 512 // (h * d))
        # rows all over a pool take a page each
        return _store(None, tokens, h, d, page, f32_out=tokens <= 8192 and rng.random() < 0.4,
                      runs=rng.random() < 0.5 or tokens * page * h * d > 1 << 29)
    if op == "attn":
        d = rng.choice([64, 128, 256])
        h_kv, g = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 5, 8])
        steps = rng.choice([1, 1, 1, 2, 4])
        batch, hi = _logint(rng, 1, 256), _logint(rng, steps, 131072)
        while batch * h_kv * d * hi > 256 * 512 * 8000 or batch * g * h_kv * steps * hi > 256 * 16 * 8000 * 2:
            batch, hi = max(1, batch * 3 // 4), max(steps, hi * 2 // 3)
        return _attn(None, batch, steps, g * h_kv, h_kv, d, min(hi, rng.choice([0, 1, steps, 50])), hi,
                     page=page, gated=rng.random() < 0.6)
    if op == "step":
        seqs, hi = _logint(rng, 1, 256), _logint(rng, 16, 8000)
        used = seqs * (hi // page + 2)
        return _pages(None, op, seqs, min(hi, 10), hi, page, used + _logint(rng, 64, 40000), steps=rng.randint(1, 8))
    d, h, kv4 = rng.choice([64, 128, 256]), rng.choice([1, 2, 4, 8]), rng.random() < 0.7
    if op == "fork":
        seqs, kids, hi = rng.randint(1, 4), _logint(rng, 2, 48), _logint(rng, 16, 5000)
        layers = rng.randint(1, 12)
    else:
        seqs, kids, hi = _logint(rng, 2, 64), 0, _logint(rng, 100, 6000)
        layers = rng.randint(1, 8)
    while True:
        pages = (seqs * (hi // page + 2) + kids) * 8 // 5 + rng.randint(1, 64)
        if layers * pages * _page_bytes({"page": page, "h_kv": h, "d": d, "kv4": kv4}) <= 2_000_000_000:
            return _pages(None, op, seqs, max(1, min(hi, 60)), hi, page, pages, layers=layers, h_kv=h, d=d,
                          kv4=kv4, children=kids)
        layers, hi = max(1, layers // 2), max(1, hi * 2 // 3)


# --------------------------------------------------------------- the inputs

def _lens(n, lo, hi):
    """n lengths spread over [lo, hi], both ends among them, in an order that is
    not sorted (fixed by the case, as its work is)."""
    if n == 1:
        return [hi]
    step = next(s for s in (67, 71, 73, 79, 83) if math.gcd(s, n) == 1)
    return [lo + (hi - lo) * ((i * step) % n) // (n - 1) for i in range(n)]


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 23)
    return g


def _randn(g, *shape, std=1.0, dtype=BF):
    return (torch.randn(*shape, generator=g, device="cuda", dtype=F32) * std).to(dtype)


def _page_bytes(c):
    return c["page"] * c["h_kv"] * c["d"] * 18 // 16 if c["kv4"] else c["page"] * c["h_kv"] * c["d"] * 2


def prepare(case, seed):
    g = _gen(seed)
    return {"store": _prepare_store, "attn": _prepare_attn}.get(case["op"], _prepare_pages)(case, g)


def _rows_of(g, tokens, h, d):
    """k or v rows: a few channels are far larger than the others, as keys' are."""
    wide = 1.0 + 6.0 * (torch.rand(h, d, generator=g, device="cuda") < 0.03)
    return _randn(g, tokens, h, d, dtype=F32) * wide


def _prepare_store(case, g):
    T, h, d, page = (case[k] for k in ("tokens", "h_kv", "d", "page"))
    kv = torch.stack([_rows_of(g, T, h, d), _rows_of(g, T, h, d)], 1).to(BF)       # [T][2][h][d], a projection's
    t = torch.arange(T, device="cuda")
    if case["runs"]:
        pages = (T + page - 1) // page + 3
        perm = torch.randperm(pages, generator=g, device="cuda")
        slot = perm[t // page] * page + t % page
    else:
        pages = T + 3
        perm = torch.randperm(pages, generator=g, device="cuda")
        slot = perm[t] * page + torch.randint(0, page, (T,), generator=g, device="cuda")
    out = F32 if case["f32_out"] else BF
    return {"case": case, "k": kv[:, 0], "v": kv[:, 1], "slot": slot.to(I32),
            "cache": torch.zeros(pages, h, page // 16, 18 * d, dtype=U8, device="cuda"),
            "k_out": torch.empty(T, h, d, dtype=out, device="cuda"),
            "v_out": torch.empty(T, h, d, dtype=out, device="cuda")}


def _prepare_attn(case, g):
    B, S, hq, hk, d, page = (case[k] for k in ("batch", "steps", "h_q", "h_kv", "d", "page"))
    lens = _lens(B, case["lo"], case["hi"])
    per = [(n + page - 1) // page for n in lens]
    width, pages = max(1, max(per)), sum(per) + 1
    host = torch.randperm(pages, generator=g, device="cuda").to(I32).cpu()
    table, at = torch.zeros(B, width, dtype=I32), 0
    for b in range(B):
        table[b, :per[b]] = host[at:at + per[b]]
        at += per[b]
    cache = torch.empty(pages, hk, page // 16, 18 * d, dtype=U8, device="cuda")
    step = max(1, (1 << 25) // (page * hk * d))
    for p in range(0, pages, step):
        n = min(step, pages - p)
        k, v = (_quantised(_randn(g, n * page, hk, d)) for _ in range(2))
        cache[p:p + n] = _packed(k, v, n, page)
    qg = _randn(g, B, S, hq, 2 * d)
    return {"case": case, "cache": cache, "table": table.cuda(),
            "len": torch.tensor(lens, dtype=I32, device="cuda"),
            # scores q.k / sqrt(d) of standard deviation 2: maps as peaked as a trained layer's
            "q": (qg[..., :d].float() * 2.0).to(BF).contiguous(),
            "gate": qg[..., d:] if case["gated"] else None,
            "out": torch.empty(B, S, hq, d, dtype=BF, device="cuda")}


def _prepare_pages(case, g):
    c = case
    n, kids, page, P = c["seqs"], c["children"], c["page"], c["pages"]
    lens = _lens(n, c["lo"], c["hi"])
    width = max(lens) // page + 2 + c["steps"]
    host = torch.randperm(P, generator=g, device="cuda").to(I32).cpu()
    table, refs, at = torch.full((n + kids, width), -1, dtype=I32), torch.zeros(P, dtype=I32), 0
    for b in range(n):
        k = (lens[b] + page - 1) // page
        # every third sequence shares the first pages of the one before it
        same = min(lens[b] // page, lens[b - 1] // page) // 2 if b % 3 == 2 else 0
        table[b, :same] = table[b - 1, :same]
        table[b, same:k] = host[at:at + k - same]
        at += k - same
        refs[table[b, :k].long()] += 1
    pad = -P % 4, -(n + kids) % 4
    # one buffer holds a pool's integers, so that one copy takes it back
    ints = torch.cat([refs, torch.zeros(pad[0], dtype=I32), torch.tensor(lens + [0] * kids, dtype=I32),
                      torch.zeros(pad[1], dtype=I32), table.flatten()]).cuda()
    cache = torch.randint(0, 256, (c["layers"], P, _page_bytes(c)), generator=g, device="cuda", dtype=U8)
    a, b = P + pad[0], n + kids + pad[1]
    child = torch.arange(n, n + kids, dtype=I32, device="cuda")
    return {"case": c, "ints": ints, "ints0": ints.clone(), "refs": ints[:P], "len": ints[a:a + n + kids],
            "table": ints[a + b:].view(n + kids, width), "cache": cache, "seen": torch.empty_like(ints),
            "len0": torch.tensor(lens, dtype=I32, device="cuda"),
            "slot": torch.zeros(n, max(1, c["steps"]), dtype=I32, device="cuda"),
            "child": child, "parent": (child - n) % n, "live": torch.zeros(1, dtype=I32, device="cuda")}


# ------------------------------------------- the cache's format in plain torch

def _quantised(x):
    """bf16 [T, h, d] -> (codes 0..15 [T, h, d], bf16 scales [T, h, d / 32])."""
    T, h, d = x.shape
    x = x.float().reshape(T, h, d // 32, 32)
    hi, lo = x.amax(-1), x.amin(-1)
    m = torch.where(hi >= -lo, hi, lo)
    s = torch.where(m.abs() < TINY, torch.zeros_like(m), m / -8.0)
    s = torch.where(torch.isfinite(x).all(-1), s, torch.full_like(s, float("nan")))
    safe = torch.where(s.abs() > 0, s, torch.ones_like(s))[..., None]
    n = torch.where((s.abs() > 0)[..., None], torch.round(x / safe).clamp(-8, 7), torch.zeros_like(x))
    return (n + 8.0).to(U8).view(T, h, d), s.to(BF)


def _word(n, place):
    """Nibbles along the last axis into 32-bit words held in 64."""
    return (n.to(torch.int64) << (4 * place)).sum(-1)


def _packed(k, v, pages, page):
    """(codes, scales) of k and v, tokens in order -> [pages, h, page / 16, 18 d] bytes."""
    (kn, ks), (vn, vs) = k, v
    T, h, d = kn.shape
    U, R = page // 16, d // 32
    at = torch.arange(8, device=kn.device)
    # K: [pages, U, 2 halves, 8 tokens, h, R, 4 lanes, 8 channels]
    kn = kn.view(pages, U, 2, 8, h, R, 4, 8)
    w = _word(kn, at // 2 + 4 * (at % 2))
    w = ((w << 3) | (w >> 29)) & 0xFFFFFFFF
    kw = w.permute(0, 4, 1, 2, 5, 3, 6).reshape(pages, h, U, d // 64, 4, 32).transpose(-1, -2)
    # V: [pages, U, 2 halves, 4 lanes, 2 tokens, h, R, 8 lanes, 4 channels]
    vn = vn.view(pages, U, 2, 4, 2, h, R, 8, 4).permute(0, 5, 1, 2, 6, 7, 3, 4, 8)
    w = _word(vn.reshape(pages, h, U, 2, R, 8, 4, 8), at)
    vw = w.reshape(pages, h, U, d // 64, 4, 32).transpose(-1, -2)

    def raw(w):
        return torch.where(w >= 1 << 31, w - (1 << 32), w).to(I32).contiguous().view(U8).view(pages, h, U, 8 * d)

    sc = torch.cat([ks, vs], -1).view(pages, U, 16, h, 2 * R).permute(0, 3, 1, 2, 4)
    sc = sc.reshape(pages, h, U, 32 * R).contiguous().view(U8)
    return torch.cat([raw(kw), raw(vw), sc], -1)


def _unpacked(rows):
    """Whole pages [n, h, U, 18 d] -> k and v values, fp32 [n, U * 16, h, d]."""
    n, h, U, d = rows.shape[0], rows.shape[1], rows.shape[2], rows.shape[3] // 18
    R = d // 32
    e = torch.arange(8, device=rows.device, dtype=I32)

    def words(part):
        return part.contiguous().view(I32).view(n, h, U, d // 64, 32, 4).transpose(-1, -2).reshape(n, h, U, 2, R, 32)

    w = words(rows[..., :8 * d])
    w = ((w >> 3) & 0x1FFFFFFF) | (w << 29)
    k = ((w[..., None] >> (4 * (e // 2 + 4 * (e % 2)))) & 15).reshape(n, h, U, 2, R, 8, 32)
    k = k.permute(0, 2, 3, 5, 1, 4, 6).reshape(n, U * 16, h, R, 32)
    w = words(rows[..., 8 * d:16 * d])
    v = ((w[..., None] >> (4 * e)) & 15).reshape(n, h, U, 2, R, 8, 4, 2, 4)
    v = v.permute(0, 2, 3, 6, 7, 1, 4, 5, 8).reshape(n, U * 16, h, R, 32)
    sc = rows[..., 16 * d:].contiguous().view(BF).view(n, h, U, 16, 2, R).permute(4, 0, 2, 3, 1, 5).float()
    sc = sc.reshape(2, n, U * 16, h, R, 1)
    return ((k - 8).float() * sc[0]).reshape(n, U * 16, h, d), ((v - 8).float() * sc[1]).reshape(n, U * 16, h, d)


# ---------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return {"store": _own_store, "attn": _own_attn, "step": _own_step, "fork": _own_fork,
                "compact": _own_compact}[op](state)
    return {"store": _plain_store, "attn": _plain_attn, "step": _plain_step, "fork": _plain_fork,
            "compact": _plain_compact}[op](state)


def _own_store(s):
    import gated_deltanet_linear_06_gb300 as gdn
    if "dims" not in s:
        c = s["case"]
        s["dims"] = gdn.make_attn_dims(h_q=c["h_kv"], h_kv=c["h_kv"], d=c["d"], rot=0)
    gdn.gdn_kv4_store(s["dims"], s["k"], s["v"], s["cache"], slot=s["slot"])
    gdn.gdn_kv4_load(s["dims"], s["cache"], s["k_out"], s["v_out"], slot=s["slot"])
    return s["k_out"], s["v_out"]


def _own_attn(s):
    import gated_deltanet_linear_06_gb300 as gdn
    if "dims" not in s:
        c = s["case"]
        s["dims"] = gdn.make_attn_dims(h_q=c["h_q"], h_kv=c["h_kv"], d=c["d"], rot=0)
        n = gdn.gdn_attn_decode_kv4_workspace_bytes(s["dims"], c["batch"], c["steps"])
        s["ws"] = torch.empty(n, dtype=U8, device="cuda")
    gdn.gdn_attn_decode_kv4(s["dims"], s["q"], s["cache"], s["table"], s["len"], s["out"], s["ws"],
                            gate=s["gate"])
    return s["out"]


def _own_pool(gdn, s):
    if "pool" not in s:
        s["pool"] = gdn.make_page_pool(s["refs"], s["table"], s["len"], s["case"]["page"])
        s["caches"] = gdn.make_page_caches([s["cache"][i] for i in range(s["case"]["layers"])])
        s["ws"] = torch.empty(gdn.gdn_pages_workspace_bytes(s["pool"]), dtype=U8, device="cuda")
    return s["pool"], s["caches"], s["ws"]


def _own_step(s):
    import gated_deltanet_linear_06_gb300 as gdn
    pool, caches, ws = _own_pool(gdn, s)
    gdn.gdn_pages_extend(pool, s["slot"], ws)
    s["seen"].copy_(s["ints"])                     # the tables as the step's attention reads them
    gdn.gdn_pages_trim(pool, caches, s["len0"], ws)
    return s["slot"], s["seen"], s["ints"]


def _own_fork(s):
    import gated_deltanet_linear_06_gb300 as gdn
    pool, caches, ws = _own_pool(gdn, s)
    gdn.gdn_pages_fork(pool, caches, s["parent"], s["child"], ws)
    s["seen"].copy_(s["ints"])
    gdn.gdn_pages_free(pool, s["child"], ws)
    return s["seen"], s["ints"], s["cache"]


def _own_compact(s):
    import gated_deltanet_linear_06_gb300 as gdn
    pool, caches, ws = _own_pool(gdn, s)
    s["ints"].copy_(s["ints0"])                    # the pool as it was: its moved pages still hold their bytes
    gdn.gdn_pages_compact(pool, caches, ws, n_live=s["live"])
    return s["ints"], s["live"], s["cache"]


# --------------------------------------------------------- the plain forms

def _plain_store(s):
    c = s["case"]
    h, d, page = c["h_kv"], c["d"], c["page"]
    slot = s["slot"].long()
    T, R = slot.numel(), d // 32
    # a token's codes alone, in a page of which the other tokens' are zero bits, then merged by masks
    unit, j = slot // 16, slot % 16
    (kn, ks), (vn, vs) = _quantised(s["k"]), _quantised(s["v"])
    at = torch.arange(8, device="cuda")
    kw = _word(kn.view(T, h, R, 4, 8), at // 2 + 4 * (at % 2))
    kw = (((kw << 3) | (kw >> 29)) & 0xFFFFFFFF)                                # [T, h, R, 4]
    vw = _word(vn.view(T, h, R, 8, 4), at[:4])                                         # [T, h, R, 8], 16 bits
    page_at, in_page = unit // (page // 16), unit % (page // 16)
    r = torch.arange(R, device="cuda")
    head = torch.arange(h, device="cuda")[None, :, None, None]
    w = ((j // 8)[:, None] * R + r)[:, None, :, None]                                  # [T, 1, R, 1]
    lane_k = ((j % 8) * 4)[:, None, None, None] + at[:4]
    lane_v = at * 4 + ((j % 8) // 2)[:, None, None, None]
    words = s["cache"].view(I32).view(-1, h, page // 16, 18 * d // 4)
    p4, u4 = page_at[:, None, None, None], in_page[:, None, None, None]
    signed = torch.where(kw >= 1 << 31, kw - (1 << 32), kw).to(I32)
    words[p4, head, u4, (w // 4) * 128 + lane_k * 4 + w % 4] = signed
    halves = s["cache"].view(torch.int16).view(-1, h, page // 16, 9 * d)
    v16 = torch.where(vw >= 1 << 15, vw - (1 << 16), vw).to(torch.int16)
    place = 4 * d + ((w // 4) * 128 + lane_v * 4 + w % 4) * 2 + (j % 2)[:, None, None, None]
    halves[p4, head, u4, place] = v16
    sc = s["cache"].view(BF).view(-1, h, page // 16, 9 * d)
    place = 8 * d + j[:, None, None] * 2 * R + torch.arange(2 * R, device="cuda")
    sc[page_at[:, None, None], torch.arange(h, device="cuda")[:, None], in_page[:, None, None], place] = \
        torch.cat([ks, vs], -1)
    # and back: the rows' words, halves and scales gathered again
    kb = words[p4, head, u4, (w // 4) * 128 + lane_k * 4 + w % 4]
    kb = ((kb >> 3) & 0x1FFFFFFF) | (kb << 29)
    kb = ((kb[..., None] >> (4 * (at // 2 + 4 * (at % 2))).to(I32)) & 15).reshape(T, h, R, 32)
    vb = halves[p4, head, u4, 4 * d + ((w // 4) * 128 + lane_v * 4 + w % 4) * 2 + (j % 2)[:, None, None, None]]
    vb = ((vb.to(I32)[..., None] >> (4 * at[:4]).to(I32)) & 15).reshape(T, h, R, 32)
    sb = sc[page_at[:, None, None], torch.arange(h, device="cuda")[:, None], in_page[:, None, None], place].float()
    s["k_out"].copy_(((kb - 8).float() * sb[..., :R, None]).view(T, h, d))
    s["v_out"].copy_(((vb - 8).float() * sb[..., R:, None]).view(T, h, d))
    return s["k_out"], s["v_out"]


def _plain_attn(s):
    c = s["case"]
    B, S, hq, hk, d = (c[k] for k in ("batch", "steps", "h_q", "h_kv", "d"))
    G = hq // hk
    N = s["table"].shape[1] * c["page"]
    k, v = _unpacked(s["cache"][s["table"].flatten().long()])
    k, v = k.reshape(B, N, hk, d).permute(0, 2, 1, 3), v.reshape(B, N, hk, d).permute(0, 2, 1, 3)
    q = s["q"].float().reshape(B, S, hk, G, d).permute(0, 2, 1, 3, 4).reshape(B, hk, S * G, d) * d ** -0.5
    t = torch.matmul(q, k.transpose(-1, -2)).reshape(B, hk, S, G, N)
    key = torch.arange(N, device="cuda")
    last = s["len"][:, None] - S + torch.arange(S, device="cuda")                # [B, S]
    keep = (key <= last[..., None])[:, None, :, None]                             # [B, 1, S, 1, N]
    t = t.masked_fill(~keep, float("-inf"))
    top = t.amax(-1, keepdim=True)
    t = torch.exp(t - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    den = t.sum(-1, keepdim=True)
    v = v.masked_fill((key >= s["len"][:, None])[:, None, :, None], 0.0)
    o = torch.matmul(t.reshape(B, hk, S * G, N), v).reshape(B, hk, S, G, d)
    o = (o / torch.where(den > 0, den, torch.ones_like(den))).permute(0, 2, 1, 3, 4).reshape(B, S, hq, d)
    if s["gate"] is not None:
        o = o * torch.sigmoid(s["gate"].float())
    s["out"].copy_(o)
    return s["out"]


def _free_first(refs):
    """Page indices, the free ones first, both kinds ascending."""
    return torch.sort((refs > 0).int(), stable=True).indices


def _drop(s, rows):
    """One reference less for every page in rows (entries below zero: none)."""
    s["refs"].index_add_(0, rows.clamp(min=0).flatten().long(), -(rows >= 0).int().flatten())


def _plain_step(s):
    c = s["case"]
    page, steps, n = c["page"], c["steps"], c["seqs"]
    table, ln = s["table"][:n], s["len"][:n]
    col = torch.arange(table.shape[1], device="cuda")
    had, want = (ln + page - 1) // page, (ln + steps + page - 1) // page
    first = (torch.cumsum(want - had, 0) - (want - had))[:, None] + col - had[:, None]
    new = (col >= had[:, None]) & (col < want[:, None])
    fresh = _free_first(s["refs"])[first.clamp(0, s["refs"].numel() - 1)].to(I32)
    table.copy_(torch.where(new, fresh, table))
    s["refs"].index_add_(0, fresh.flatten().long(), new.int().flatten())
    at = ln[:, None] + torch.arange(steps, device="cuda")
    s["slot"].copy_(table.gather(1, (at // page).long()) * page + at % page)
    ln.add_(steps)
    s["seen"].copy_(s["ints"])
    keep = (s["len0"] + page - 1) // page
    gone = col >= keep[:, None]
    _drop(s, torch.where(gone, table, torch.full_like(table, -1)))
    table.masked_fill_(gone, -1)
    ln.copy_(s["len0"])
    return s["slot"], s["seen"], s["ints"]


def _plain_fork(s):
    c = s["case"]
    page, n = c["page"], c["children"]
    src, dst = s["parent"].long(), s["child"].long()
    ln = s["len"][src]
    full, part = (ln // page).long(), ln % page > 0
    col = torch.arange(s["table"].shape[1], device="cuda")
    last = s["table"][src, full]
    fresh = _free_first(s["refs"])[torch.cumsum(part, 0) - part.long()].to(I32)
    rows = torch.where(col < full[:, None], s["table"][src], torch.full_like(s["table"][src], -1))
    rows.scatter_(1, full[:, None], torch.where(part, fresh, torch.full_like(fresh, -1))[:, None])
    s["refs"].index_add_(0, rows.clamp(min=0).flatten().long(), (rows >= 0).int().flatten())
    s["table"][dst] = rows
    s["len"][dst] = ln
    # where no page is half full one is copied onto itself
    s["cache"][:, torch.where(part, fresh, last).long()] = s["cache"][:, last.long()]
    s["seen"].copy_(s["ints"])
    _drop(s, s["table"][dst])
    s["table"][dst] = -1
    s["len"][dst] = 0
    return s["seen"], s["ints"], s["cache"]


def _plain_compact(s):
    s["ints"].copy_(s["ints0"])
    refs, table = s["refs"], s["table"]
    at = torch.arange(refs.numel(), device="cuda")
    used = refs > 0
    live = used.sum()
    hole, late = (~used & (at < live)).nonzero()[:, 0], (used & (at >= live)).nonzero()[:, 0]
    to = at.clone()
    to[late] = hole
    s["cache"][:, hole] = s["cache"][:, late]
    refs[hole] = refs[late]
    refs[late] = 0
    table.copy_(torch.where(table >= 0, to[table.clamp(min=0).long()].to(I32), table))
    s["live"].copy_(live)
    return s["ints"], s["live"], s["cache"]


# ------------------------------------------------------- the work of a pass

def work(case):
    c = case
    if c["op"] == "store":
        n = c["tokens"] * c["h_kv"] * c["d"]
        # rows in, codes and scales out, codes and scales in again, values out
        return {"bytes": 4 * n + 2 * (n * 9 // 8) + n * (8 if c["f32_out"] else 4) + 8 * c["tokens"],
                "flops": 10 * n}
    if c["op"] == "attn":
        B, S, hq, hk, d = (c[k] for k in ("batch", "steps", "h_q", "h_kv", "d"))
        lens = _lens(B, c["lo"], c["hi"])
        rows = B * S * hq * d
        return {"bytes": sum(lens) * hk * d * 9 // 8 + rows * (4 + (2 if c["gated"] else 0))
                + sum(4 * -(-n // c["page"]) for n in lens),
                "flops": 4 * S * hq * d * sum(lens)}
    lens, page = _lens(c["seqs"], c["lo"], c["hi"]), c["page"]
    held = sum(-(-n // page) for n in lens)
    if c["op"] == "step":
        new = sum(-(-(n + c["steps"]) // page) - -(-n // page) for n in lens)
        # the lengths read and written twice, rows out, each new page's entry and count twice, and the
        # counts read until enough free pages are found
        return {"bytes": 4 * (c["seqs"] * (4 + c["steps"]) + 6 * new + 2 * new * c["pages"] // (c["pages"] - held))
                + 8 * (c["pages"] + 2 * c["seqs"]), "flops": 0}
    if c["op"] == "fork":
        mine = [lens[i % c["seqs"]] for i in range(c["children"])]
        moved = sum(1 for n in mine if n % page)
        return {"bytes": 2 * moved * c["layers"] * _page_bytes(c) + 28 * sum(-(-n // page) for n in mine), "flops": 0}
    # about as many pages are above the line as a random pool leaves there
    return {"bytes": int(2 * held * (1 - held / c["pages"]) * c["layers"] * _page_bytes(c))
            + 8 * c["pages"] + 8 * held, "flops": 0}


# --------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"store": _exact_store, "attn": _exact_attn, "step": _exact_step, "fork": _exact_fork,
            "compact": _exact_compact}[case["op"]](case, s)


def _exact_store(c, s):
    def held(x):
        x = x.double().unflatten(-1, (-1, 32))
        big = x.abs().amax(-1, keepdim=True)
        sign = torch.where((x == big).any(-1, keepdim=True), 1.0, -1.0).double()
        unit = big / 8                                        # values lie on unit * (-sign) * {-8 .. 7}
        n = torch.round(-sign * x / torch.where(big > 0, unit, torch.ones_like(unit))).clamp(-8, 7)
        v = torch.where(big < TINY, torch.zeros_like(x), -sign * unit * n)
        return torch.where(torch.isfinite(x).all(-1, keepdim=True), v, torch.full_like(v, math.nan)).flatten(-2)
    return held(s["k"]), held(s["v"])


def _exact_attn(c, s):
    B, S, hq, hk, d, page = (c[k] for k in ("batch", "steps", "h_q", "h_kv", "d", "page"))
    lens, G = _lens(B, c["lo"], c["hi"]), hq // hk
    if sum(lens) * hk * d > 1 << 31 or B * hk * S > 8192:
        return None
    # where each nibble of a token's row lies, byte by byte
    j, ch = torch.arange(16, device="cuda")[:, None], torch.arange(d, device="cuda")[None]
    w = (j // 8) * (d // 32) + ch // 32
    bit = (4 * ((ch % 8) // 2 + 4 * (ch % 2)) + 3 + torch.arange(4, device="cuda")[:, None, None]) % 32
    byte_k = (w // 4) * 512 + ((j % 8) * 4 + ch % 32 // 8) * 16 + w % 4 * 4 + bit // 8      # [4 bits, 16, d]
    nib = ch % 4 + 4 * (j % 2)
    byte_v = 8 * d + (w // 4) * 512 + (ch % 32 // 4 * 4 + j % 8 // 2) * 16 + w % 4 * 4 + nib // 2
    out = torch.zeros(B, S, hq, d, dtype=F64, device="cuda")
    for b in range(B):
        if lens[b] == 0:
            continue
        rows = s["cache"][s["table"][b, :-(-lens[b] // page)].long()]                     # [n, h, U, 18 d]
        for h in range(hk):
            u = rows[:, h].reshape(-1, 18 * d)
            k = sum(((u[:, byte_k[i]] >> (bit[i] % 8).to(U8)) & 1).double() * 2 ** i for i in range(4))
            v = ((u[:, byte_v] >> (nib % 2 * 4).to(U8)) & 15).double()
            sc = u[:, 16 * d:].contiguous().view(BF).view(-1, 16, 2, d // 32).double()
            k = ((k - 8).unflatten(-1, (-1, 32)) * sc[:, :, 0, :, None]).reshape(-1, d)
            v = ((v - 8).unflatten(-1, (-1, 32)) * sc[:, :, 1, :, None]).reshape(-1, d)
            for i in range(S):
                seen = lens[b] - (S - 1 - i)
                if seen > 0:
                    a = s["q"][b, i, h * G:(h + 1) * G].double() @ k[:seen].t() / math.sqrt(d)
                    out[b, i, h * G:(h + 1) * G] = torch.softmax(a, -1) @ v[:seen]
    if s["gate"] is not None:
        out /= 1.0 + torch.exp(-s["gate"].double())
    return out


def _host_pool(s):
    return s["refs"].tolist(), s["table"].tolist(), s["len"].tolist()


def _ints_of(s, refs, table, ln):
    n = s["ints"].clone()
    P, N = len(refs), len(ln)
    n[:P] = torch.tensor(refs, dtype=I32)
    a = P + -P % 4
    n[a:a + N] = torch.tensor(ln, dtype=I32)
    n[a + N + -N % 4:] = torch.tensor([e for row in table for e in row], dtype=I32)
    return n


def _exact_step(c, s):
    refs, table, ln = _host_pool(s)
    page, slots, free = c["page"], [], 0
    for b in range(c["seqs"]):
        slots.append([])
        for _ in range(c["steps"]):
            if ln[b] % page == 0:
                while refs[free]:
                    free += 1
                refs[free], table[b][ln[b] // page] = 1, free
            slots[-1].append(table[b][ln[b] // page] * page + ln[b] % page)
            ln[b] += 1
    seen = _ints_of(s, refs, table, ln)
    return torch.tensor(slots, dtype=I32), seen, s["ints0"]


def _exact_fork(c, s):
    refs, table, ln = _host_pool(s)
    page, free = c["page"], 0
    cache = s["cache"].clone()
    for src, dst in zip(s["parent"].tolist(), s["child"].tolist()):
        ln[dst] = ln[src]
        for i in range(ln[src] // page):
            table[dst][i] = table[src][i]
            refs[table[src][i]] += 1
        if ln[src] % page:
            while refs[free]:
                free += 1
            i = ln[src] // page
            refs[free], table[dst][i] = 1, free
            cache[:, free] = cache[:, table[src][i]]
    return _ints_of(s, refs, table, ln), s["ints0"], cache


def _exact_compact(c, s):
    refs, table, ln = _host_pool(s)
    pages = [p for p, r in enumerate(refs) if r > 0]
    keep = set(pages)
    holes = [p for p in range(len(pages)) if p not in keep]
    late = [p for p in pages if p >= len(pages)]
    to = dict(zip(late, holes))
    cache = s["cache"].clone()
    for a, b in to.items():
        cache[:, b] = cache[:, a]
        refs[b], refs[a] = refs[a], 0
    table = [[to.get(e, e) for e in row] for row in table]
    return _ints_of(s, refs, table, ln), torch.tensor([len(pages)], dtype=I32), cache
