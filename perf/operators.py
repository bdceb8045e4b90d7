"""The measured cases of the attention-layer and expert-layer operators.

Three operators of a hybrid model's decode path, next to the Gated DeltaNet
layer: ``prep`` (per-head norms of q and k, rotary positions with one or
several axes, and the write into the paged cache, in one pass), ``shared``
(attention of a batch of sequences that share one long prefix, each with a
paged tail of its own) and ``moe`` (a whole mixture-of-experts layer for a few
tokens).  ``run`` computes them in plain torch operations, or, with ``own``
set, through gated_deltanet_linear_06_gb300's public calls; ``exact`` gives
the same outputs from the definitions in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
NORM_EPS = 1e-6
THETA = 1.0e7          # rotary base of long-context models


# ---------------------------------------------------------------- the cases

def _prep(name, tokens, h_q, h_kv, d, rot, axes=1, interleave=False, pairs=False, gated=False,
          far=0, page=64):
    """gated: q is a strided view of a [tokens][h_q][2 d] projection whose other
    half is the output gate; far: the first token's position."""
    return {"name": name, "op": "prep", "tokens": tokens, "h_q": h_q, "h_kv": h_kv, "d": d,
            "rot": rot, "axes": axes, "interleave": interleave, "pairs": pairs, "gated": gated,
            "far": far, "page": page}


def _shared(name, batch, steps, h_q, h_kv, d, prefix, tail_lo, tail_hi, page=64, gated=True):
    return {"name": name, "op": "shared", "batch": batch, "steps": steps, "h_q": h_q, "h_kv": h_kv,
            "d": d, "prefix": prefix, "tail_lo": tail_lo, "tail_hi": tail_hi, "page": page,
            "gated": gated}


def _moe(name, tokens, hidden, inter, experts, top_k, shared_inter=0, renorm=True, f32_out=False):
    return {"name": name, "op": "moe", "tokens": tokens, "hidden": hidden, "inter": inter,
            "experts": experts, "top_k": top_k, "shared_inter": shared_inter, "renorm": renorm,
            "f32_out": f32_out}


def listed():
    return [
        # one decode step of 8 sequences far into their contexts: all launch latency
        _prep("prep_decode_8", 8, 16, 2, 256, 64, gated=True, far=131000),
        # a prompt chunk with pictures in it: three axes, frequencies dealt out in turn, odd length
        _prep("prep_image_2049", 2049, 32, 8, 128, 128, axes=3, interleave=True),
        # a whole long prompt, q read out of the projection that also holds the output gate
        _prep("prep_prompt_32768", 32768, 16, 2, 256, 64, gated=True),
        # one user's turn after a short system prompt
        _shared("shared_b1_p700", 1, 1, 16, 2, 256, 700, 133, 133),
        # verifying 4 drafted tokens of 17 sequences, small pages, odd lengths
        _shared("shared_b17_s4_p5000", 17, 4, 32, 8, 128, 5000, 4, 900, page=16, gated=False),
        # agents of one long document: the prefix dominates, and its products bound it
        _shared("shared_b64_p32768", 64, 1, 16, 2, 256, 32768, 0, 700),
        # a full server batch under a common prompt: own tails dominate
        _shared("shared_b256_p4096", 256, 1, 16, 2, 256, 4096, 100, 3000),
        # the largest: a full batch over a long document
        _shared("shared_b256_p32768", 256, 1, 16, 2, 256, 32768, 1, 1100),
        # one token of one user through 256 experts and the shared one
        _moe("moe_t1", 1, 2048, 512, 256, 8, shared_inter=512),
        # a few tokens (one speculative window of one user), 64 wider experts, odd sizes
        _moe("moe_t5_wide", 5, 2048, 1408, 64, 6, renorm=False, f32_out=True),
        # a small batch
        _moe("moe_t16", 16, 2048, 512, 256, 8, shared_inter=512),
        # the most tokens one call takes, 512 experts: nearly every weight is read
        _moe("moe_t64", 64, 2048, 512, 512, 10, shared_inter=512),
    ]


def _logint(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prep", "shared", "shared", "moe", "moe"])
    if op == "prep":
        d = rng.choice([64, 128, 256])
        h_kv = rng.choice([1, 2, 4, 8])
        h_q = h_kv * rng.choice([1, 2, 4, 5, 8])
        tokens = _logint(rng, 1, 32768)
        # no more than the largest listed case moves
        tokens = max(1, min(tokens, 32768 * 18 * 256 // ((h_q + h_kv) * d)))
        axes = rng.choice([1, 1, 2, 3])
        return _prep(None, tokens, h_q, h_kv, d, rng.choice([d, d // 2, d // 4]), axes=axes,
                     interleave=rng.random() < 0.5, pairs=rng.random() < 0.3,
                     gated=rng.random() < 0.5, far=rng.choice([0, 0, rng.randrange(1 << 20)]),
                     page=rng.choice([16, 32, 64, 128]))
    if op == "shared":
        d = rng.choice([64, 128, 256])
        h_kv = rng.choice([1, 2, 4, 8])
        g = rng.choice([1, 2, 4, 6, 8])
        steps = rng.choice([1, 1, 1, 2, 4, 8])
        batch = _logint(rng, 1, 256)
        prefix = _logint(rng, 16, 32768)
        while batch * steps * g * h_kv * d * prefix > 256 * 16 * 256 * 32768:
            batch = max(1, batch // 2)
        hi = _logint(rng, steps, 3000)
        while batch * h_kv * d * hi > 256 * 2 * 256 * 1500 and hi > steps:
            hi = max(steps, hi // 2)
        return _shared(None, batch, steps, g * h_kv, h_kv, d, prefix, min(hi, rng.choice([0, 1, steps])),
                       hi, page=rng.choice([16, 32, 64, 128]), gated=rng.random() < 0.7)
    hidden = rng.choice([512, 1024, 1536, 2048, 2056, 2880])
    inter = rng.choice([128, 256, 512, 520, 768, 1408])
    experts = rng.choice([8, 16, 64, 128, 256, 512])
    while experts * inter * hidden > 512 * 512 * 2048:
        experts //= 2
    return _moe(None, _logint(rng, 1, 64), hidden, inter, experts, rng.randint(1, min(10, experts)),
                shared_inter=rng.choice([0, 0, 256, 512]), renorm=rng.random() < 0.6,
                f32_out=rng.random() < 0.3)


# --------------------------------------------------------------- the inputs

def _tails(case):
    """Tail lengths of a shared case: spread over [tail_lo, tail_hi], both ends
    among them, in an order that is not sorted (fixed by the case, as its work is)."""
    b, lo, hi = case["batch"], case["tail_lo"], case["tail_hi"]
    if b == 1:
        return [hi]
    step = next(s for s in (67, 71, 73, 79, 83) if math.gcd(s, b) == 1)
    return [lo + (hi - lo) * ((i * step) % b) // (b - 1) for i in range(b)]


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _randn(g, *shape, std=1.0, dtype=BF):
    return (torch.randn(*shape, generator=g, device="cuda", dtype=F32) * std).to(dtype)


def _randn_big(g, rows, *shape, std=1.0):
    """bf16 [rows, *shape] drawn in blocks of rows (no fp32 copy of the whole)."""
    out = torch.empty(rows, *shape, device="cuda", dtype=BF)
    step = max(1, (1 << 26) // max(1, math.prod(shape)))
    for r in range(0, rows, step):
        out[r:r + step] = torch.randn(min(step, rows - r), *shape, generator=g, device="cuda",
                                      dtype=F32) * std
    return out


def prepare(case, seed):
    g = _gen(seed)
    return {"prep": _prepare_prep, "shared": _prepare_shared, "moe": _prepare_moe}[case["op"]](case, g)


def _prepare_prep(case, g):
    T, hq, hk, d, rot, ax = (case[k] for k in ("tokens", "h_q", "h_kv", "d", "rot", "axes"))
    qg = _randn(g, T, hq, (2 if case["gated"] else 1) * d)
    kv = _randn(g, T, 2, hk, d)
    nf = rot // 2
    inv_freq = torch.tensor([THETA ** (-2.0 * i / rot) for i in range(nf)], dtype=F64, device="cuda")
    if ax > 1 and case["interleave"]:
        axis = [i % ax for i in range(nf)]
    else:
        axis = [min(i * ax // nf, ax - 1) for i in range(nf)]
    # text positions, with runs of picture patches whose axes part (time, row, column)
    t = torch.arange(T, device="cuda")
    pos = [case["far"] + t]
    if ax > 1:
        inside = (t // 256) % 2 == 1
        patch = t % 256
        base = case["far"] + t - patch
        pos = [torch.where(inside, base, pos[0])]
        pos += [torch.where(inside, base + (patch // 16 if a == 1 else patch % 16), case["far"] + t)
                for a in range(1, ax)]
    pages = (T + case["page"] - 1) // case["page"] + 3
    perm = torch.randperm(pages, generator=g, device="cuda")
    slot = (perm[t // case["page"]] * case["page"] + t % case["page"]).to(torch.int32)
    w = 1.0 + 0.25 * torch.randn(2, d, generator=g, device="cuda", dtype=F32)
    return {"case": case, "q": qg[:, :, :d], "k": kv[:, 0], "v": kv[:, 1], "q_w": w[0].contiguous(),
            "k_w": w[1].contiguous(), "inv_freq": inv_freq,
            "axis": torch.tensor(axis, dtype=torch.int32, device="cuda"),
            "pos": torch.stack(pos).to(torch.int32).contiguous(), "slot": slot,
            "q_out": torch.empty(T, hq, d, dtype=BF, device="cuda"),
            "k_cache": torch.zeros(pages, case["page"], hk, d, dtype=BF, device="cuda"),
            "v_cache": torch.zeros(pages, case["page"], hk, d, dtype=BF, device="cuda")}


def _prepare_shared(case, g):
    B, S, hq, hk, d, page = (case[k] for k in ("batch", "steps", "h_q", "h_kv", "d", "page"))
    lens = _tails(case)
    n_pre = (case["prefix"] + page - 1) // page
    per = [(n + page - 1) // page for n in lens]
    width = max(1, max(per))
    pages = n_pre + sum(per) + 1
    perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    tail = torch.zeros(B, width, dtype=torch.int32)
    at, host = n_pre, perm.cpu()
    for b in range(B):
        tail[b, :per[b]] = host[at:at + per[b]]
        at += per[b]
    # scores q.k / sqrt(d) of standard deviation 2: maps as peaked as a trained layer's
    qg = _randn(g, B, S, hq, 2 * d)
    st = {"case": case, "q": (qg[..., :d].float() * 2.0).to(BF).contiguous(),
          "gate": qg[..., d:] if case["gated"] else None,
          "k_cache": _randn_big(g, pages, page, hk, d), "v_cache": _randn_big(g, pages, page, hk, d),
          "prefix_pages": perm[:n_pre].contiguous(), "tail_pages": tail.cuda(),
          "tail_len": torch.tensor(lens, dtype=torch.int32, device="cuda"),
          "out": torch.empty(B, S, hq, d, dtype=BF, device="cuda")}
    return st


def _prepare_moe(case, g):
    T, H, I, E, Is = (case[k] for k in ("tokens", "hidden", "inter", "experts", "shared_inter"))
    st = {"case": case, "x": _randn(g, T, H), "w_router": _randn(g, E, H, std=H ** -0.5),
          "w_gate_up": _randn_big(g, E, 2 * I, H, std=H ** -0.5),
          "w_down": _randn_big(g, E, H, I, std=I ** -0.5),
          "y": torch.empty(T, H, dtype=F32 if case["f32_out"] else BF, device="cuda"),
          "ids": torch.empty(T, case["top_k"], dtype=torch.int32, device="cuda"),
          "wts": torch.empty(T, case["top_k"], dtype=F32, device="cuda"),
          "s_gate_up": None, "s_down": None, "s_gate": None}
    if Is:
        st["s_gate_up"] = _randn(g, 2 * Is, H, std=H ** -0.5)
        st["s_down"] = _randn(g, H, Is, std=Is ** -0.5)
        st["s_gate"] = _randn(g, H, std=H ** -0.5)
    return st


# ---------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return {"prep": _own_prep, "shared": _own_shared, "moe": _own_moe}[op](state)
    return {"prep": _plain_prep, "shared": _plain_shared, "moe": _plain_moe}[op](state)


def _attn_dims(gdn, c):
    return gdn.make_attn_dims(h_q=c["h_q"], h_kv=c["h_kv"], d=c["d"], rot=c.get("rot", 0),
                              n_axes=c.get("axes", 1), rope_pairs=int(c.get("pairs", False)),
                              norm_eps=NORM_EPS)


def _own_prep(s):
    import gated_deltanet_linear_06_gb300 as gdn
    if "dims" not in s:
        s["dims"] = _attn_dims(gdn, s["case"])
    gdn.gdn_attn_prep(s["dims"], s["q"], s["k"], s["v"], s["q_w"], s["k_w"], s["inv_freq"], s["axis"],
                      s["pos"], s["q_out"], s["k_cache"], s["v_cache"], slot=s["slot"])
    return s["q_out"], s["k_cache"], s["v_cache"]


def _own_shared(s):
    import gated_deltanet_linear_06_gb300 as gdn
    if "dims" not in s:
        c = s["case"]
        s["dims"] = _attn_dims(gdn, c)
        n = gdn.gdn_attn_decode_shared_workspace_bytes(s["dims"], c["batch"], c["steps"])
        s["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    gdn.gdn_attn_decode_shared(s["dims"], s["q"], s["k_cache"], s["v_cache"], s["prefix_pages"],
                               s["case"]["prefix"], s["tail_pages"], s["tail_len"], s["out"], s["ws"],
                               gate=s["gate"])
    return s["out"]


def _own_moe(s):
    import gated_deltanet_linear_06_gb300 as gdn
    if "dims" not in s:
        c = s["case"]
        s["dims"] = gdn.make_moe_dims(hidden=c["hidden"], inter=c["inter"], experts=c["experts"],
                                      top_k=c["top_k"], shared_inter=c["shared_inter"],
                                      renorm=int(c["renorm"]))
        n = gdn.gdn_moe_step_workspace_bytes(s["dims"], c["tokens"])
        s["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    gdn.gdn_moe_step(s["dims"], s["x"], s["w_router"], s["w_gate_up"], s["w_down"], s["y"], s["ws"],
                     w_shared_gate_up=s["s_gate_up"], w_shared_down=s["s_down"],
                     w_shared_gate=s["s_gate"], topk_id=s["ids"], topk_w=s["wts"])
    return s["y"], s["ids"], s["wts"]


# --------------------------------------------------------- the plain forms

def _plain_prep(s):
    c = s["case"]
    rot, nf, d = c["rot"], c["rot"] // 2, c["d"]
    # the angle of a far position needs 64 bits; its sine and cosine then hold in 32
    ang = s["pos"].double()[s["axis"].long()].t() * s["inv_freq"]          # [T, nf]
    cos, sin = ang.cos().float()[:, None], ang.sin().float()[:, None]

    def normed(x, w):
        x = x.float()
        return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + NORM_EPS) * w

    def rotated(x):
        y = x.clone()
        if c["pairs"]:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
        else:
            a, b = x[..., :nf], x[..., nf:rot]
            y[..., :nf], y[..., nf:rot] = a * cos - b * sin, b * cos + a * sin
        return y

    s["q_out"].copy_(rotated(normed(s["q"], s["q_w"])))
    rows = s["slot"].long()
    s["k_cache"].view(-1, c["h_kv"], d)[rows] = rotated(normed(s["k"], s["k_w"])).to(BF)
    s["v_cache"].view(-1, c["h_kv"], d)[rows] = s["v"]
    return s["q_out"], s["k_cache"], s["v_cache"]


def _plain_shared(s):
    c = s["case"]
    B, S, hq, hk, d, L = (c[k] for k in ("batch", "steps", "h_q", "h_kv", "d", "prefix"))
    G = hq // hk
    q = s["q"].float().view(B, S, hk, G, d) * d ** -0.5
    kp = s["k_cache"][s["prefix_pages"].long()].view(-1, hk, d)[:L].float()
    vp = s["v_cache"][s["prefix_pages"].long()].view(-1, hk, d)[:L].float()
    # the prefix, once for all rows of a key head
    qh = q.permute(2, 0, 1, 3, 4).reshape(hk, B * S * G, d)
    sp = torch.matmul(qh, kp.permute(1, 2, 0)).view(hk, B, S, G, L)
    # the tails
    N = s["tail_pages"].shape[1] * c["page"]
    kt = s["k_cache"][s["tail_pages"].long()].view(B, N, hk, d).permute(2, 0, 1, 3).float()
    vt = s["v_cache"][s["tail_pages"].long()].view(B, N, hk, d).permute(2, 0, 1, 3).float()
    qt = qh.view(hk, B, S * G, d)
    tt = torch.matmul(qt, kt.transpose(-1, -2)).view(hk, B, S, G, N)
    key = torch.arange(N, device="cuda")
    last = s["tail_len"][:, None] - S + torch.arange(S, device="cuda")      # [B, S]
    keep = key <= last[..., None]                                           # [B, S, N]
    tt = tt.masked_fill(~keep[None, :, :, None], float("-inf"))
    top = torch.maximum(sp.amax(-1), tt.amax(-1)) if L else tt.amax(-1)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)[..., None]
    sp, tt = torch.exp(sp - top), torch.exp(tt - top)
    den = sp.sum(-1) + tt.sum(-1)
    o = torch.matmul(sp.view(hk, B * S * G, L), vp.permute(1, 0, 2)).view(hk, B, S * G, d)
    # a masked key has no weight, whatever stands in its value row
    vt = vt.masked_fill((key >= s["tail_len"][:, None])[None, ..., None], 0.0)
    o = o + torch.matmul(tt.view(hk, B, S * G, N), vt)
    o = o.view(hk, B, S, G, d) / torch.where(den > 0, den, torch.ones_like(den))[..., None]
    o = o.permute(1, 2, 0, 3, 4).reshape(B, S, hq, d)
    if s["gate"] is not None:
        o = o * torch.sigmoid(s["gate"].float())
    s["out"].copy_(o)
    return s["out"]


def _plain_moe(s):
    c = s["case"]
    T, I = c["tokens"], c["inter"]
    # 64 bits: logits next to each other decide which experts run
    logits = s["x"].double() @ s["w_router"].double().t()
    p = torch.softmax(logits, -1)
    ids = torch.sort(-logits, dim=-1, stable=True).indices[:, :c["top_k"]]
    w = p.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    x = s["x"].float()
    y = torch.zeros(T, c["hidden"], dtype=F32, device="cuda")
    for t in range(T):
        gu = torch.einsum("kih,h->ki", s["w_gate_up"][ids[t]].float(), x[t])
        a = gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:]
        y[t] = torch.einsum("khi,ki->h", s["w_down"][ids[t]].float(), a * w[t, :, None].float())
    if c["shared_inter"]:
        gu = x @ s["s_gate_up"].float().t()
        g, u = gu.chunk(2, -1)
        share = torch.sigmoid(x @ s["s_gate"].float())[:, None]
        y += share * ((g * torch.sigmoid(g) * u) @ s["s_down"].float().t())
    s["y"].copy_(y)
    s["ids"].copy_(ids)
    s["wts"].copy_(w)
    return s["y"], s["ids"], s["wts"]


# ------------------------------------------------------- the work of a pass

def work(case):
    c = case
    if c["op"] == "prep":
        T, hq, hk, d = c["tokens"], c["h_q"], c["h_kv"], c["d"]
        rows = T * (hq + hk)
        return {"bytes": T * d * (4 * hq + 8 * hk) + 4 * T * (c["axes"] + 1) + 8 * d + 6 * c["rot"],
                "flops": rows * (4 * d + 3 * c["rot"])}
    if c["op"] == "shared":
        B, S, hq, hk, d, L = (c[k] for k in ("batch", "steps", "h_q", "h_kv", "d", "prefix"))
        tail = sum(_tails(c))
        rows = B * S * hq * d
        kv = (L + tail) * hk * d * 4
        return {"bytes": kv + rows * (4 + (2 if c["gated"] else 0)),
                "flops": 4 * S * hq * d * (B * L + tail)}
    T, H, I, E, k, Is = (c[n] for n in ("tokens", "hidden", "inter", "experts", "top_k", "shared_inter"))
    # experts that T tokens of k choices each reach when every choice is alike
    hit = E * (1.0 - (1.0 - k / E) ** T)
    return {"bytes": int(6 * H * (hit * I + Is) + 2 * E * H + (2 * H if Is else 0)
                         + T * H * (2 + (4 if c["f32_out"] else 2)) + 8 * T * k),
            "flops": 2 * T * H * E + 6 * T * H * (k * I + Is)}


# --------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"prep": _exact_prep, "shared": _exact_shared, "moe": _exact_moe}[case["op"]](case, s)


def _exact_prep(c, s):
    d, rot, nf = c["d"], c["rot"], c["rot"] // 2

    def turn(x, w):
        # norm, then each pair as a complex number times e^{i angle}
        x = x.double()
        x = x / ((x ** 2).sum(-1, keepdim=True) / d + NORM_EPS).sqrt() * w.double()
        first = list(range(0, rot, 2)) if c["pairs"] else list(range(nf))
        second = [i + 1 for i in first] if c["pairs"] else [i + nf for i in first]
        ang = torch.stack([s["pos"][int(s["axis"][i])].double() * s["inv_freq"][i] for i in range(nf)], -1)
        z = torch.complex(x[..., first], x[..., second]) * torch.polar(torch.ones_like(ang), ang)[:, None]
        y = x.clone()
        y[..., first], y[..., second] = z.real, z.imag
        return y

    kc, vc = s["k_cache"].double().flatten(0, 1), s["v_cache"].double().flatten(0, 1)
    kc[s["slot"].long()] = turn(s["k"], s["k_w"])
    vc[s["slot"].long()] = s["v"].double()
    return turn(s["q"], s["q_w"]), kc.view_as(s["k_cache"]), vc.view_as(s["v_cache"])


def _exact_shared(c, s):
    B, S, hq, hk, d, L, page = (c[k] for k in ("batch", "steps", "h_q", "h_kv", "d", "prefix", "page"))
    G = hq // hk
    if 4.0 * S * hq * d * (B * L + sum(_tails(c))) > 4e11:
        return None
    rows = torch.arange(L, device="cuda")
    rows = s["prefix_pages"].long()[rows // page] * page + rows % page
    kall, vall = s["k_cache"].flatten(0, 1), s["v_cache"].flatten(0, 1)
    out = torch.zeros(B, S, hq, d, dtype=F64, device="cuda")
    lens = _tails(c)
    for h in range(hk):
        kp, vp = kall[rows, h].double(), vall[rows, h].double()
        for b in range(B):
            n = torch.arange(lens[b], device="cuda")
            own_rows = s["tail_pages"][b].long()[n // page] * page + n % page
            k = torch.cat([kp, kall[own_rows, h].double()])
            v = torch.cat([vp, vall[own_rows, h].double()])
            for i in range(S):
                seen = L + max(0, lens[b] - (S - 1 - i))
                if seen == 0:
                    continue
                sc = s["q"][b, i, h * G:(h + 1) * G].double() @ k[:seen].t() / math.sqrt(d)
                out[b, i, h * G:(h + 1) * G] = torch.softmax(sc, -1) @ v[:seen]
    if s["gate"] is not None:
        out /= 1.0 + torch.exp(-s["gate"].double())
    return out


def _exact_moe(c, s):
    T, I, k, Is = c["tokens"], c["inter"], c["top_k"], c["shared_inter"]
    x = s["x"].double()
    logits = (s["w_router"].double() @ x.t()).t()
    order = torch.argsort(logits, dim=-1, descending=True, stable=True)[:, :k]
    e = torch.exp(logits - logits.amax(-1, keepdim=True))
    w = torch.gather(e, 1, order) / (1.0 if c["renorm"] else e.sum(-1, keepdim=True))
    if c["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    y = torch.zeros(T, c["hidden"], dtype=F64, device="cuda")
    for ex in order.unique().tolist():                       # expert by expert
        t, slot = (order == ex).nonzero(as_tuple=True)
        gu = s["w_gate_up"][ex].double() @ x[t].t()
        act = gu[:I] / (1.0 + torch.exp(-gu[:I])) * gu[I:]
        y.index_add_(0, t, (s["w_down"][ex].double() @ act).t() * w[t, slot, None])
    if Is:
        gu = s["s_gate_up"].double() @ x.t()
        act = gu[:Is] / (1.0 + torch.exp(-gu[:Is])) * gu[Is:]
        y += (s["s_down"].double() @ act).t() / (1.0 + torch.exp(-(x @ s["s_gate"].double())))[:, None]
    return y, order.to(torch.int32), w
