"""The serving operators next to the prefill path, measured: rotary positions with several axes, appending
to a paged key/value cache, and attention over that cache for a batch that shares a prefix.

`run` takes each in its plain form (elementary torch operations in 32 bits, angles in 64) or, with `own`
set, through the calls of the library's binding.  `exact` is the definition in 64 bits.
"""
import math

import torch

own = False

D = 128  # head dimension the library is compiled for
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# --- cases -----------------------------------------------------------------------------------------


def _rotary(name, B, N, Hq, Hkv, dtype="bf16", rot=D, axes=1, pairs="half", inverse=False, far=0):
    return {"name": name, "op": "rotary", "B": B, "N": N, "Hq": Hq, "Hkv": Hkv, "dtype": dtype, "rot": rot,
            "axes": axes, "pairs": pairs, "inverse": inverse, "far": far}


def _append(name, nseq, new_lo, new_hi, old_hi, page, Hq, Hkv, dtype="bf16", rot=D, axes=1, pairs="half", prefix=0):
    return {"name": name, "op": "append", "nseq": nseq, "new_lo": new_lo, "new_hi": new_hi, "old_hi": old_hi,
            "page": page, "Hq": Hq, "Hkv": Hkv, "dtype": dtype, "rot": rot, "axes": axes, "pairs": pairs,
            "prefix": prefix}


def _attend(name, nseq, new_lo, new_hi, old_lo, old_hi, prefix, page, Hq, Hkv, dtype="bf16"):
    return {"name": name, "op": "attend", "nseq": nseq, "new_lo": new_lo, "new_hi": new_hi, "old_lo": old_lo,
            "old_hi": old_hi, "prefix": prefix, "page": page, "Hq": Hq, "Hkv": Hkv, "dtype": dtype}


def listed():
    return [
        # a short prompt of one small head before its plan: the call's latency
        _rotary("rotary_1k", 1, 1024, 1, 1),
        # the rotation before the 128K prefill, 32 query heads over 8 KV heads
        _rotary("rotary_128k", 1, 131072, 32, 8),
        # the gradient's way through the rotation of an image/video prompt (time, height, width), odd length
        _rotary("rotary_axes_inverse", 2, 9973, 32, 8, dtype="fp16", axes=3, inverse=True),
        # one decode step of 64 sequences behind a 32K shared prefix
        _append("append_step", 64, 1, 1, 200, 16, 32, 8, prefix=32768),
        # chunks of seven prompts with image tokens in them, ragged, landing in pages of 64
        _append("append_chunks", 7, 1, 4096, 500, 64, 32, 8, axes=3),
        # one sequence, a 1K prompt and its first answers: the latency of a step
        _attend("attend_one", 1, 1, 1, 0, 100, 1024, 16, 32, 8),
        # a step of 64 chats behind a 32K document
        _attend("attend_batch", 64, 1, 1, 0, 1023, 32768, 64, 32, 8),
        # a step of 256 short answers to one 128K document: the largest
        _attend("attend_wide", 256, 1, 1, 0, 511, 131072, 64, 32, 8),
        # 16 unrelated long sequences of very different lengths: no prefix, bound by the cache reads
        _attend("attend_own", 16, 1, 1, 0, 32767, 0, 16, 32, 8, dtype="fp16"),
        # five drafted tokens of 33 sequences checked at once, prefix ending inside a page, groups of 8
        _attend("attend_drafts", 33, 5, 5, 0, 700, 5001, 32, 16, 2),
        # prompt chunks of five sequences behind an 8K instruction, ending inside a page
        _attend("attend_chunks", 5, 1, 1023, 0, 3000, 8191, 128, 32, 8, dtype="fp16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rotary", "append", "attend", "attend"))
    Hq, Hkv = rng.choice(((32, 8), (32, 8), (16, 2), (8, 8), (12, 4), (3, 1), (1, 1)))
    dtype = rng.choice(("bf16", "bf16", "fp16"))
    if op != "attend":
        rot = rng.choice((128, 128, 64, 96, 32))
        axes = rng.choice((1, 1, 2, 3))
        pairs = rng.choice(("half", "half", "adjacent"))
    if op == "rotary":
        B = rng.choice((1, 1, 2, 3))
        c = _rotary("", B, _log(rng, 1, 131072 // B), Hq, Hkv, dtype, rot, axes, pairs, rng.random() < 0.4,
                    rng.choice((0, 0, 1 << 20)))
    elif op == "append":
        nseq = _log(rng, 1, 256)
        hi = _log(rng, 1, max(1, 16384 // nseq))
        c = _append("", nseq, min(hi, rng.choice((0, 1, 1))), hi, _log(rng, 1, max(2, 65536 // nseq)),
                    rng.choice((16, 32, 64, 128)), Hq, Hkv, dtype, rot, axes, pairs, rng.choice((0, 0, 4999, 32768)))
    else:
        page = rng.choice((16, 32, 64, 128))
        kind = rng.choice(("step", "step", "drafts", "chunks"))
        if kind == "chunks":
            nseq = rng.randint(1, 6)
            hi = _log(rng, 9, 1024)
            prefix, old = rng.choice((0, _log(rng, 1, 8192))), _log(rng, 1, 4096)
        else:
            nseq = _log(rng, 1, 256)
            hi = 1 if kind == "step" else rng.randint(2, 8)
            prefix = rng.choice((0, _log(rng, 1, 131072 // hi)))
            old = _log(rng, 2, 131072 // nseq)
        lo = 1 if kind == "chunks" else hi
        c = _attend("", nseq, lo, hi, 0, old, prefix, page, Hq, Hkv, dtype)
    del c["name"]
    return c


# --- inputs ----------------------------------------------------------------------------------------


def _spread(lo, hi, n, seed):
    """n whole numbers of [lo, hi], the same for every seed of a case's work: both ends, and evenly between,
    in an order that goes by the seed."""
    v = [lo + (hi - lo) * i // max(1, n - 1) for i in range(n)] if n > 1 else [hi]
    g = torch.Generator().manual_seed(seed)
    return [v[i] for i in torch.randperm(n, generator=g).tolist()]


def _lengths(case, seed):
    new = _spread(case["new_lo"], case["new_hi"], case["nseq"], seed)
    old = _spread(case.get("old_lo", 0), case["old_hi"], case["nseq"], seed + 1)
    return new, old


def _sections(rot, axes):
    """Frequencies of each axis: 1/4, 3/8, 3/8 of them for three (time, height, width), halves for two."""
    F = rot // 2
    return {1: (F,), 2: (F // 2, F - F // 2), 3: (F // 4, (F - F // 4) // 2, F - F // 4 - (F - F // 4) // 2)}[axes]


def _inv_freq(rot, theta=500000.0):
    return [theta ** (-2.0 * i / rot) for i in range(rot // 2)]


def _positions(axes, shape, start):
    """Positions of text with a picture in it: time runs on, height and width walk a grid 61 wide."""
    t = torch.arange(shape[-1], device="cuda").expand(shape) + start
    p = [t, start + (t // 61) % 97, start + t % 61][:axes]
    return torch.stack([x.to(torch.int32) for x in p]).contiguous()


def _rotary_config(case):
    import score_keys_pooled_b200 as s2o
    return s2o.make_rotary(case["rot"], theta=500000.0, sections=_sections(case["rot"], case["axes"]),
                           interleaved=case["pairs"] == "adjacent")


def _cache_config(case, Tq, max_pages, num_pages):
    import score_keys_pooled_b200 as s2o
    return s2o.make_cache(case["Hq"], case["Hkv"], case["page"], num_pages, case["nseq"], max_pages, Tq,
                          max_q=case["new_hi"], prefix_len=case["prefix"],
                          dtype=s2o.BF16 if case["dtype"] == "bf16" else s2o.FP16)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = TYPES[case["dtype"]]
    Hq, Hkv = case["Hq"], case["Hkv"]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(t)

    s = {"case": case, "t": t}
    if case["op"] == "rotary":
        B, N = case["B"], case["N"]
        if case["inverse"]:  # gradients as the prefill's layout has them: [B, H, N, d]
            s["q"] = normal(B, Hq, N, D).transpose(1, 2)
            s["k"] = normal(B, Hkv, N, D).transpose(1, 2)
        else:  # one packed projection: [B, N, (Hq + 2 Hkv) d]
            qkv = normal(B, N, Hq + 2 * Hkv, D)
            s["q"], s["k"] = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv]
        s["pos"] = _positions(case["axes"], (B, N), case["far"])
        if own:
            s["rotary"] = _rotary_config(case)
        return s

    nseq, page, P = case["nseq"], case["page"], case["prefix"]
    new, old = _lengths(case, seed)
    Tq, length = sum(new), [a + b for a, b in zip(new, old)]
    max_pages = max(1, -(-(case["new_hi"] + case["old_hi"]) // page))
    pre = -(-P // page) if case["op"] == "attend" else 0
    used = [max(0, -(-n // page)) for n in length]
    num_pages = pre + nseq * max_pages + 3
    ids = torch.randperm(num_pages, generator=g, device="cuda").to(torch.int32)
    s["prefix_pages"] = ids[:pre].contiguous()
    # each sequence's pages in its row of the table; what lies behind them is never read
    at = torch.tensor([0] + used, device="cuda").cumsum(0)[:-1] + pre
    col = torch.arange(max_pages, device="cuda")
    mine = col[None] < torch.tensor(used, device="cuda")[:, None]
    s["table"] = torch.where(mine, ids[torch.where(mine, at[:, None] + col, 0)], -1).to(torch.int32)
    s["q_start"] = torch.tensor([0] + new, device="cuda").cumsum(0).to(torch.int32)
    s["kv_len"] = torch.tensor(length, device="cuda", dtype=torch.int32)
    s["max_len"], s["Tq"] = max(length), Tq
    # stale values of earlier requests fill the cache behind the lengths
    s["k_cache"], s["v_cache"] = normal(num_pages, Hkv, page, D), normal(num_pages, Hkv, page, D)
    if case["op"] == "append":
        qkv = normal(Tq, Hq + 2 * Hkv, D)
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        s["pos"] = _positions(case["axes"], (Tq,), P) if case["axes"] > 1 else None
        s["q_out"] = torch.empty(Tq, Hq, D, device="cuda", dtype=t)
    else:
        # queries drift along the direction that the first keys of the prefix (or of each sequence) stand out in
        u = torch.nn.functional.normalize(torch.randn(Hkv, D, generator=g, device="cuda"), dim=-1)
        s["q"] = (torch.randn(Tq, Hkv, Hq // Hkv, D, generator=g, device="cuda") + u[:, None]).reshape(Tq, Hq, D).to(t)
        first = s["prefix_pages"][:1].long() if P else s["table"][:, 0].clamp(min=0).long()
        s["k_cache"][first, :, :4] = (s["k_cache"][first, :, :4].float() + 4.0 * u[:, None]).to(t)
        s["O"] = torch.empty(Tq, Hq, D, device="cuda", dtype=t)
        s["lse"] = torch.empty(Tq, Hq, device="cuda", dtype=torch.float32)
    if own:
        import score_keys_pooled_b200 as s2o
        s["cfg"] = _cache_config(case, Tq, max_pages, num_pages)
        if case["op"] == "append":
            s["rotary"] = _rotary_config(case)
        else:
            s["workspace"] = s2o.alloc_attention_paged(s["cfg"])
    return s


# --- one pass --------------------------------------------------------------------------------------


def run(s):
    if own:
        return _own(s)
    return {"rotary": _plain_rotary, "append": _plain_append, "attend": _plain_attend}[s["case"]["op"]](s)


def _own(s):
    import score_keys_pooled_b200 as s2o
    op = s["case"]["op"]
    if op == "rotary":
        return s2o.rotary(s["rotary"], s["q"], s["k"], s["pos"], inverse=s["case"]["inverse"])
    if op == "append":
        s2o.cache_append(s["cfg"], s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["q_start"],
                         s["kv_len"], rotary=s["rotary"], positions=s["pos"], q_out=s["q_out"])
        return s["q_out"], s["k_cache"], s["v_cache"]
    return s2o.attention_paged(s["cfg"], s["q"], s["k_cache"], s["v_cache"], s["table"], s["q_start"], s["kv_len"],
                               prefix_pages=s["prefix_pages"], O=s["O"], lse=s["lse"], workspace=s["workspace"])


def _cos_sin(case, pos, inverse):
    """cos and sin of every frequency's angle, [..., rot / 2] in 32 bits; the angles are formed in 64."""
    rot = case["rot"]
    n = torch.tensor(_sections(rot, case["axes"]), device="cuda")
    axis = torch.repeat_interleave(torch.arange(case["axes"], device="cuda"), n, output_size=rot // 2)
    f = torch.tensor(_inv_freq(rot), device="cuda", dtype=torch.float64)
    phi = pos.movedim(0, -1)[..., axis].double() * f
    return phi.cos().float(), (-phi if inverse else phi).sin().float()


def _turn(x, c, s, pairs):
    """x [..., H, d] turned by the angles [..., rot / 2]."""
    F = c.shape[-1]
    c, s, x = c[..., None, :], s[..., None, :], x.float()
    if pairs == "half":
        a, b = x[..., :F], x[..., F:2 * F]
        return torch.cat((a * c - b * s, a * s + b * c, x[..., 2 * F:]), -1)
    a, b = x[..., 0:2 * F:2], x[..., 1:2 * F:2]
    return torch.cat((torch.stack((a * c - b * s, a * s + b * c), -1).flatten(-2), x[..., 2 * F:]), -1)


def _plain_rotary(s):
    case = s["case"]
    c, sn = _cos_sin(case, s["pos"], case["inverse"])
    return tuple(_turn(s[n], c, sn, case["pairs"]).to(s["t"]) for n in ("q", "k"))


def _tokens(s):
    """Of every token: its sequence, its place among the sequence's new tokens, and in its own keys."""
    t = torch.arange(s["Tq"], device="cuda")
    start = s["q_start"].long()
    seq = torch.searchsorted(start, t, right=True) - 1
    j = t - start[seq]
    return seq, j, s["kv_len"].long()[seq] - (start[seq + 1] - start[seq]) + j


def _plain_append(s):
    case = s["case"]
    seq, _, at = _tokens(s)
    pos = s["pos"] if s["pos"] is not None else (at + case["prefix"])[None]
    c, sn = _cos_sin(case, pos, False)
    page = s["table"][seq, at // case["page"]].long()
    s["q_out"].copy_(_turn(s["q"], c, sn, case["pairs"]))
    s["k_cache"][page, :, at % case["page"]] = _turn(s["k"], c, sn, case["pairs"]).to(s["t"])
    s["v_cache"][page, :, at % case["page"]] = s["v"]
    return s["q_out"], s["k_cache"], s["v_cache"]


def _plain_attend(s):
    case = s["case"]
    nseq, P, Hq, Hkv, Tq = case["nseq"], case["prefix"], case["Hq"], case["Hkv"], s["Tq"]
    G, Q, scale = Hq // Hkv, case["new_hi"], 1.0 / math.sqrt(D)
    seq, j, at = _tokens(s)
    q = s["q"].float() * scale
    # the shared prefix: every row of a KV head against the same keys
    rows = q.view(Tq, Hkv, G, D).permute(1, 0, 2, 3).reshape(Hkv, Tq * G, D)
    pk, pv = (s[n][s["prefix_pages"].long()].permute(1, 0, 2, 3).reshape(Hkv, -1, D)[:, :P].float()
              for n in ("k_cache", "v_cache"))
    sp = (rows @ pk.transpose(1, 2)).view(Hkv, Tq, G, P)
    # the sequences' own keys, padded to the longest
    L = s["max_len"]
    pages = s["table"][:, :-(-L // case["page"])].clamp(min=0).long()
    ok, ov = (s[n][pages].permute(0, 2, 1, 3, 4).reshape(nseq, Hkv, -1, D)[:, :, :L].float()
              for n in ("k_cache", "v_cache"))
    key = torch.arange(L, device="cuda")
    ov = torch.where((key[None] < s["kv_len"][:, None])[:, None, :, None], ov, 0.0)
    padded = torch.zeros(nseq, Q, Hq, D, device="cuda")
    padded[seq, j] = q
    limit = torch.full((nseq, Q), -1, device="cuda")
    limit[seq, j] = at
    so = padded.view(nseq, Q, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(nseq, Hkv, Q * G, D) @ ok.transpose(2, 3)
    so = so.view(nseq, Hkv, Q, G, L)
    so = torch.where(key <= limit[:, None, :, None, None], so, -math.inf)
    # one softmax over both
    none = torch.full((Tq, Hkv, G), -math.inf, device="cuda")
    mo = so.amax(-1).permute(0, 2, 1, 3)[seq, j] if L else none
    mp = sp.amax(-1).transpose(0, 1) if P else none
    m = torch.maximum(mo, mp)
    m = torch.where(m == -math.inf, 0.0, m)
    ep = torch.exp(sp - m.transpose(0, 1)[..., None])
    mpad = torch.zeros(nseq, Q, Hkv, G, device="cuda")
    mpad[seq, j] = m
    eo = torch.exp(so - mpad.permute(0, 2, 1, 3)[..., None])
    total = ep.sum(-1).transpose(0, 1) + eo.sum(-1).permute(0, 2, 1, 3)[seq, j]
    acc = (ep.view(Hkv, Tq * G, P) @ pv).view(Hkv, Tq, G, D).transpose(0, 1)
    acc = acc + (eo.view(nseq, Hkv, Q * G, L) @ ov).view(nseq, Hkv, Q, G, D).permute(0, 2, 1, 3, 4)[seq, j]
    O = torch.where(total[..., None] > 0, acc / total[..., None], 0.0)
    return O.reshape(Tq, Hq, D).to(s["t"]), (m + torch.log(total)).reshape(Tq, Hq)


# --- what a pass cannot do without -----------------------------------------------------------------


def work(case):
    Hq, Hkv, row = case["Hq"], case["Hkv"], 2 * D
    if case["op"] == "rotary":
        n = case["B"] * case["N"]
        return {"bytes": n * (2 * (Hq + Hkv) * row + 4 * case["axes"]), "flops": 3 * n * (Hq + Hkv) * case["rot"]}
    new, old = _lengths(case, 0)  # the totals are those of any seed, to within which old meets which new
    Tq = sum(new)
    if case["op"] == "append":
        return {"bytes": Tq * (2 * (Hq + 2 * Hkv) * row + (4 * case["axes"] if case["axes"] > 1 else 0)),
                "flops": 3 * Tq * (Hq + Hkv) * case["rot"]}
    keys = sum(n * case["prefix"] + n * o + n * (n + 1) // 2 for n, o in zip(new, old))
    return {"bytes": 2 * Hkv * row * (case["prefix"] + sum(new) + sum(old)) + Tq * Hq * (2 * row + 4),
            "flops": 4 * D * Hq * keys}


# --- the definition in 64 bits ---------------------------------------------------------------------


def _rotated(case, x, pos):
    """Pairs of x [n, H, d] as complex numbers times exp(i phi), phi = position of the pair's axis * frequency."""
    rot = case["rot"]
    F = rot // 2
    phi, f = torch.empty(x.shape[0], F, dtype=torch.float64, device=x.device), 0
    for axis, n in enumerate(_sections(rot, case["axes"])):
        for _ in range(n):
            phi[:, f] = pos[axis].double() * math.exp(-2.0 * f / rot * math.log(500000.0))
            f += 1
    e = torch.polar(torch.ones_like(phi), -phi if case.get("inverse") else phi)
    out = x.double()
    for h in range(x.shape[1]):
        y = x[:, h, :rot].double()
        z = torch.complex(y[:, :F], y[:, F:]) if case["pairs"] == "half" else torch.complex(y[:, ::2], y[:, 1::2])
        z = z * e
        out[:, h, :rot] = torch.cat((z.real, z.imag), 1) if case["pairs"] == "half" else torch.view_as_real(z).flatten(1)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotary":
        return tuple(torch.stack([_rotated(case, s[n][b], s["pos"][:, b]) for b in range(case["B"])]) for n in "qk")
    page, P, Hkv, G = case["page"], case["prefix"], case["Hkv"], case["Hq"] // case["Hkv"]
    new, old = _lengths(case, seed)
    start = [sum(new[:i]) for i in range(len(new))]
    if case["op"] == "append":
        at = torch.cat([torch.arange(o, o + n, device="cuda") for n, o in zip(new, old)])
        pos = s["pos"] if s["pos"] is not None else (at + P)[None]
        q, k = _rotated(case, s["q"], pos), _rotated(case, s["k"], pos)
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        for b, (n, o) in enumerate(zip(new, old)):
            where = torch.arange(o, o + n, device="cuda")
            ids = s["table"][b].long()[where // page]
            kc[ids, :, where % page] = k[start[b]:start[b] + n]
            vc[ids, :, where % page] = s["v"][start[b]:start[b] + n].double()
        return q, kc, vc

    def keys(pages, n, name):
        c = s[name].index_select(0, pages[:-(-n // page)].long())
        return torch.cat(tuple(c), 1)[:, :n].double() if n else torch.zeros(Hkv, 0, D, dtype=torch.float64, device="cuda")

    pk, pv = keys(s["prefix_pages"], P, "k_cache"), keys(s["prefix_pages"], P, "v_cache")
    O = torch.zeros(s["Tq"], case["Hq"], D, dtype=torch.float64, device="cuda")
    lse = torch.full((s["Tq"], case["Hq"]), -math.inf, dtype=torch.float64, device="cuda")
    for b, (n, o) in enumerate(zip(new, old)):
        if n == 0:
            continue
        k, v = keys(s["table"][b], o + n, "k_cache"), keys(s["table"][b], o + n, "v_cache")
        q = s["q"][start[b]:start[b] + n].double().view(n, Hkv, G, D).permute(1, 2, 0, 3).reshape(Hkv, G * n, D)
        hidden = torch.arange(o + n, device="cuda")[None] > o + torch.arange(n, device="cuda")[:, None]
        x = (q @ k.mT).view(Hkv, G, n, o + n).masked_fill(hidden, -math.inf).view(Hkv, G * n, o + n)
        x = torch.cat((q @ pk.mT, x), 2) / math.sqrt(D)
        p = torch.softmax(x, 2)
        y = p[:, :, :P] @ pv + p[:, :, P:] @ v
        O[start[b]:start[b] + n] = y.view(Hkv, G, n, D).permute(2, 0, 1, 3).reshape(n, case["Hq"], D)
        lse[start[b]:start[b] + n] = torch.logsumexp(x, 2).view(Hkv, G, n).permute(2, 0, 1).reshape(n, case["Hq"])
    return O, lse
