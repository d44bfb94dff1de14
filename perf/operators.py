"""What the rotary, paged-cache and shared-prefix attention operators are measured on.

Three operators that follow one another in a serving step, the first also in a training step:

  rope    rotary positions of q and k (half or interleaved pairs, part of the head, frequencies
          scaled for long contexts), forward and backward
  append  new keys and values into a paged cache, q and k rotated on the way
  attend  attention of the new tokens over a prefix that the whole batch shares and over each
          sequence's own pages

``own`` False computes the plain forms with elementary torch operations, True calls the library.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
BF = torch.bfloat16


# ---- cases ------------------------------------------------------------------------------------

def _rope(name, B, S, Hq, Hkv, D, rot, inter=False, scaling="none", back=False, fused=False,
          start=0, given=False):
    return {"name": name, "op": "rope", "B": B, "S": S, "Hq": Hq, "Hkv": Hkv, "D": D, "rot": rot,
            "inter": inter, "scaling": scaling, "back": back, "fused": fused, "start": start,
            "given": given}


def _append(name, B, T, Hq, Hkv, D, rot, page, own_len, ragged=False, inter=False,
            scaling="none", start=0):
    return {"name": name, "op": "append", "B": B, "T": T, "Hq": Hq, "Hkv": Hkv, "D": D,
            "rot": rot, "page": page, "own_len": own_len, "ragged": ragged, "inter": inter,
            "scaling": scaling, "start": start}


def _attend(name, B, T, Hq, Hkv, D, page, prefix, own_len, ragged=False, lse=False, peaky=False,
            head_major=False):
    return {"name": name, "op": "attend", "B": B, "T": T, "Hq": Hq, "Hkv": Hkv, "D": D,
            "page": page, "prefix": prefix, "own_len": own_len, "ragged": ragged, "lse": lse,
            "peaky": peaky, "head_major": head_major}


def listed():
    return [
        # one new token of one sequence: nothing but latency
        _rope("rope_one_token", 1, 1, 32, 8, 128, 128, start=40000),
        # a training step's q and k at the 8K shape
        _rope("rope_8k", 1, 8192, 32, 8, 128, 128),
        # its gradient for a packed batch with given positions: interleaved pairs, half the head,
        # odd length
        _rope("rope_8k_back_part", 2, 4097, 64, 8, 128, 64, inter=True, scaling="ntk", back=True,
              given=True),
        # a 128K prompt far inside a long context, read out of the rows of a fused projection
        _rope("rope_128k_fused", 1, 131072, 32, 8, 128, 128, scaling="parts", fused=True,
              start=900001),
        # one decode step of one sequence
        _append("append_one_token", 1, 1, 32, 8, 128, 128, 64, 5000),
        # one step of a batch with drafted tokens, padded rows behind the last sequence
        _append("append_batch_ragged", 96, 5, 64, 8, 128, 128, 16, 3000, ragged=True,
                scaling="parts", start=70000),
        # a long prompt's keys and values into the pages that a batch will share
        _append("append_prefix_32k", 1, 32768, 32, 8, 128, 128, 64, 32768),
        # a few sequences on a short instruction: the smallest serving step
        _attend("attend_small", 4, 1, 32, 8, 128, 16, 500, 60),
        # one sequence alone on a long cache, nothing shared
        _attend("attend_one_long", 1, 1, 32, 8, 128, 64, 0, 131072, lse=True),
        # a decode step of a batch on a shared document
        _attend("attend_batch_32k", 64, 1, 32, 8, 128, 16, 32768, 1500),
        # drafted tokens (none to five a sequence) on a very long shared document, many heads, a
        # few keys that stand out
        _attend("attend_draft_128k", 96, 5, 64, 8, 128, 64, 131000, 700, ragged=True, lse=True,
                peaky=True),
        # no shared heads, small heads, head-major pages
        _attend("attend_d64", 40, 2, 16, 16, 64, 32, 7777, 900, head_major=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def _unnamed(c):
    return {k: v for k, v in c.items() if k != "name"}


def draw(rng):
    heads = [(32, 8), (64, 8), (16, 16), (4, 4), (28, 4), (40, 8), (8, 1), (24, 8), (10, 2)]
    kind = rng.choice(["rope", "append", "attend", "attend"])
    Hq, Hkv = rng.choice(heads)
    if kind == "rope":
        D = rng.choice([64, 80, 128, 128, 192, 256])
        rot = rng.choice([D, D, D // 2 // 16 * 16])
        room = 130000 * 40 * 128 // ((Hq + Hkv) * D + 2)
        n = _log(rng, 1, room)
        B = min(n, rng.choice([1, 1, 2, 3, 7]))
        return _unnamed(_rope("", B, max(1, n // B), Hq, Hkv, D, rot, rng.random() < 0.5,
                     rng.choice(["none", "linear", "ntk", "parts"]), rng.random() < 0.5,
                     rng.random() < 0.4, rng.choice([0, rng.randrange(1 << 20)]),
                     rng.random() < 0.4))
    page = rng.choice([16, 32, 48, 64, 128, 256])
    if kind == "append":
        D = rng.choice([64, 128, 128])
        B = _log(rng, 1, 128)
        T = rng.choice([1, 1, rng.randrange(1, 9), _log(rng, 1, max(1, 16384 // B))])
        return _unnamed(_append("", B, T, Hq, Hkv, D, rng.choice([D, D // 2]), page,
                       T + _log(rng, 1, 3000), rng.random() < 0.5, rng.random() < 0.5,
                       rng.choice(["none", "linear", "ntk", "parts"]),
                       rng.choice([0, rng.randrange(1 << 18)])))
    D = rng.choice([64, 128, 128])
    B = _log(rng, 1, 128)
    T = rng.choice([1, 1, 1, rng.randrange(2, 9)])
    prefix = rng.choice([0, _log(rng, 1, 131072), _log(rng, 1, 131072), _log(rng, 1, 131072)])
    own_len = T + _log(rng, 1, 4096 if B > 1 else 131072)
    c = _attend("", B, T, Hq, Hkv, D, page, prefix, own_len, rng.random() < 0.4,
                rng.random() < 0.4, rng.random() < 0.3, rng.random() < 0.3)
    most = work(next(x for x in listed() if x["name"] == "attend_draft_128k"))
    while work(c)["flops"] > most["flops"] or work(c)["bytes"] > most["bytes"]:
        c["prefix"] //= 2
        c["own_len"] = c["T"] + (c["own_len"] - c["T"] + 1) // 2
    return _unnamed(c)


# ---- what a case fixes: counts and lengths (the seed only orders them) ------------------------

def _counts(c):
    """New tokens and own length (new tokens among them) of each sequence."""
    B, T = c["B"], c["T"]
    n = [b % (T + 1) for b in range(B)] if c["ragged"] else [T] * B
    if c["ragged"] and B == 1:
        n = [T]
    before = c["own_len"] - T
    return n, [n[b] + (before * (b + 1)) // B for b in range(B)]


def _rows(c):
    """Rows of a packed call: the sequences' tokens and, in a ragged batch, a few rows behind."""
    n, _ = _counts(c)
    return sum(n) + 3 if c["ragged"] else sum(n)


def work(c):
    D = c["D"]
    if c["op"] == "rope":
        n = c["B"] * c["S"]
        elems = n * (c["Hq"] + c["Hkv"])
        return {"bytes": elems * D * 4 + (8 * n if c["given"] else 0),
                "flops": elems * c["rot"] * 3}
    n, lens = _counts(c)
    if c["op"] == "append":
        tok = sum(n)
        return {"bytes": tok * (c["Hq"] + 2 * c["Hkv"]) * D * 4,
                "flops": tok * (c["Hq"] + c["Hkv"]) * c["rot"] * 3}
    keys = c["prefix"] + sum(lens)
    seen = sum(x * c["prefix"] + x * (m - x) + x * (x + 1) // 2 for x, m in zip(n, lens))
    return {"bytes": keys * c["Hkv"] * D * 4 + sum(n) * c["Hq"] * (4 * D + (4 if c["lse"] else 0)),
            "flops": 4 * seen * c["Hq"] * D}


# ---- inputs -----------------------------------------------------------------------------------

THETA, FACTOR, TRAINED, FAST, SLOW = 500000.0, 8.0, 8192, 32.0, 1.0


def _frequencies(rot, scaling):
    """Radians a position, in 64 bits, and the factor of cos and sin."""
    theta, m = THETA, 1.0
    if scaling == "ntk":
        theta *= FACTOR ** (rot / (rot - 2))
    f = theta ** (-np.arange(0, rot, 2, dtype=np.float64) / rot)
    if scaling == "linear":
        f = f / FACTOR
    if scaling == "parts":
        turns = TRAINED * f / (2 * math.pi)
        g = np.clip((turns - SLOW) / (FAST - SLOW), 0.0, 1.0)
        f = f * (g + (1 - g) / FACTOR)
        m = 0.1 * math.log(FACTOR) + 1.0
    return f, m


def _phases(f):
    """The frequencies as the library keeps them: 2^-64 of a turn a position, as 64-bit words."""
    w = [int(x / (2 * math.pi) * 2.0 ** 64) & (2 ** 64 - 1) for x in f]
    return torch.tensor([x - 2 ** 64 if x >= 2 ** 63 else x for x in w], dtype=torch.int64)


def _angles(c):
    f, m = _frequencies(c["rot"], c["scaling"])
    return {"freq": torch.from_numpy(f).to(DEV), "mscale": m, "phases": _phases(f).to(DEV)}


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(shape, g):
    return torch.randn(shape, generator=g, device=DEV, dtype=BF)


def prepare(c, seed):
    g = _gen(seed)
    rng = np.random.default_rng(seed)
    D, Hq, Hkv = c["D"], c["Hq"], c["Hkv"]
    s = {"case": c}
    if c["op"] == "rope":
        B, S = c["B"], c["S"]
        if c["fused"]:  # q, k and v of one projection side by side in a row
            x = _normal((B, S, (Hq + 2 * Hkv) * D), g)
            s["q"] = x[..., :Hq * D].unflatten(-1, (Hq, D))
            s["k"] = x[..., Hq * D:(Hq + Hkv) * D].unflatten(-1, (Hkv, D))
        else:
            s["q"], s["k"] = _normal((B, S, Hq, D), g), _normal((B, S, Hkv, D), g)
        if c["given"]:  # packed documents: positions start again at odd places
            p = torch.arange(S, device=DEV).repeat(B, 1) + c["start"]
            cut = torch.randint(0, S, (B, 1), generator=g, device=DEV)
            s["pos"] = torch.where(p - c["start"] >= cut, p - c["start"] - cut, p)
        s.update(_angles(c))
        return s
    n, lens = _counts(c)
    B, T = c["B"], c["T"]
    order = rng.permutation(B)
    n, lens = [n[i] for i in order], [lens[i] for i in order]
    rows = _rows(c)
    shape = (rows,) if c["ragged"] else (B, T)
    ps = c["page"]
    need = [-(-m // ps) for m in lens]
    prefix = c.get("prefix", 0)
    shared = -(-prefix // ps)
    pages = shared + sum(need) + 2
    perm = rng.permutation(pages)
    table = np.full((B, -(-c["own_len"] // ps)), -1, dtype=np.int32)
    at = shared
    for b in range(B):
        table[b, :need[b]] = perm[at:at + need[b]]
        at += need[b]
    s["table"] = torch.from_numpy(table).to(DEV)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    s["cu"] = (torch.tensor([0] + list(np.cumsum(n)), dtype=torch.int32, device=DEV)
               if c["ragged"] else None)
    s["q"] = _normal(shape + (Hq, D), g)
    s["o"] = torch.zeros_like(s["q"])
    if c["op"] == "append":
        s["k"], s["v"] = _normal(shape + (Hkv, D), g), _normal(shape + (Hkv, D), g)
        s["kp"], s["vp"] = _normal((pages, ps, Hkv, D), g), _normal((pages, ps, Hkv, D), g)
        s.update(_angles(c))
        return s
    if c["head_major"]:
        s["kp"] = _normal((pages, Hkv, ps, D), g).transpose(1, 2)
        s["vp"] = _normal((pages, Hkv, ps, D), g).transpose(1, 2)
    else:
        s["kp"], s["vp"] = _normal((pages, ps, Hkv, D), g), _normal((pages, ps, Hkv, D), g)
    if c["peaky"]:
        s["kp"][:, 3] *= 4
    s["ptable"] = torch.from_numpy(perm[:shared].astype(np.int32)).to(DEV)
    # slots that no token has been written to hold anything
    for b in range(B):
        if lens[b] % ps:
            s["kp"][int(table[b, need[b] - 1]), lens[b] % ps:] = float("nan")
            s["vp"][int(table[b, need[b] - 1]), lens[b] % ps:] = float("nan")
    if prefix % ps:
        s["kp"][int(perm[shared - 1]), prefix % ps:] = float("nan")
        s["vp"][int(perm[shared - 1]), prefix % ps:] = float("inf")
    if c["lse"]:
        s["lse"] = torch.zeros((Hq, rows) if c["ragged"] else (B, Hq, T), device=DEV)
    return s


# ---- one pass ---------------------------------------------------------------------------------

def run(s):
    c = s["case"]
    if c["op"] == "rope":
        return _run_rope(s, c)
    return _run_append(s, c) if c["op"] == "append" else _run_attend(s, c)


def _run_rope(s, c):
    if own:
        import context_parallelism_gb300 as up
        call = up.rope_backward if c["back"] else up.rope_forward
        q, k = call(s["q"], s["k"], s["phases"], mscale=s["mscale"], interleaved=c["inter"],
                    positions=s.get("pos"), start=c["start"])
        return {"q": q, "k": k}
    B, S = c["B"], c["S"]
    pos = s["pos"] if c["given"] else (torch.arange(S, device=DEV) + c["start"]).expand(B, S)
    cos, sin = _cos_sin(s, pos)
    if c["back"]:
        sin = -sin
    return {"q": _rotate(s["q"], cos, sin, c), "k": _rotate(s["k"], cos, sin, c)}


def _cos_sin(s, pos):
    a = pos.to(torch.float64).unsqueeze(-1) * s["freq"]  # far positions: angles in 64 bits
    return ((torch.cos(a) * s["mscale"]).float().unsqueeze(-2),
            (torch.sin(a) * s["mscale"]).float().unsqueeze(-2))


def _rotate(x, cos, sin, c):
    rot = c["rot"]
    f = x[..., :rot].float()
    if c["inter"]:
        a, b = f[..., 0::2], f[..., 1::2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = f[..., :rot // 2], f[..., rot // 2:]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((y.to(x.dtype), x[..., rot:]), -1)


def _tokens(s, c):
    """Sequence and place among the new tokens of each row that belongs to a sequence."""
    B, T = c["B"], c["T"]
    if c["ragged"]:
        r = torch.arange(_rows(c) - 3, device=DEV)
        seq = torch.searchsorted(s["cu"][1:].long(), r, right=True)
        return r, seq, r - s["cu"].long()[seq], (s["cu"][1:] - s["cu"][:-1]).long()
    r = torch.arange(B * T, device=DEV)
    return r, r // T, r % T, torch.full((B,), T, device=DEV)


def _run_append(s, c):
    if own:
        import context_parallelism_gb300 as up
        up.kv_append(s["k"], s["v"], s["kp"], s["vp"], s["table"], s["lens"], q=s["q"],
                     q_out=s["o"], phases=s["phases"], mscale=s["mscale"],
                     interleaved=c["inter"], start=c["start"], cu_seqlens=s["cu"])
        return {"q": s["o"], "kp": s["kp"], "vp": s["vp"]}
    r, seq, i, n = _tokens(s, c)
    at = s["lens"].long()[seq] - n[seq] + i
    cos, sin = _cos_sin(s, at + c["start"])
    q, k, v = (s[x].reshape(-1, s[x].shape[-2], c["D"])[r] for x in ("q", "k", "v"))
    page, slot = s["table"].long()[seq, at // c["page"]], at % c["page"]
    s["kp"][page, slot] = _rotate(k, cos, sin, c)
    s["vp"][page, slot] = v
    s["o"].view(-1, c["Hq"], c["D"])[r] = _rotate(q, cos, sin, c)
    return {"q": s["o"], "kp": s["kp"], "vp": s["vp"]}


def _run_attend(s, c):
    if own:
        import context_parallelism_gb300 as up
        up.paged_attention(s["q"], s["kp"], s["vp"], s["table"], s["lens"],
                           prefix_table=s["ptable"], prefix_len=c["prefix"],
                           cu_seqlens=s["cu"], max_q=c["T"], max_len=c["own_len"], out=s["o"],
                           lse=s.get("lse"))
    else:
        _plain_attend(s, c)
    return {"o": s["o"], "lse": s["lse"]} if c["lse"] else {"o": s["o"]}


def _plain_attend(s, c):
    B, T, Hq, Hkv, D, ps = c["B"], c["T"], c["Hq"], c["Hkv"], c["D"], c["page"]
    G, P, L = Hq // Hkv, c["prefix"], c["own_len"]
    r, seq, i, n = _tokens(s, c)
    q = s["q"].reshape(-1, Hkv, G, D)[r].float() / math.sqrt(D)
    # scores against the shared prefix
    ids = torch.arange(P, device=DEV)
    pk = s["kp"][s["ptable"].long()[ids // ps], ids % ps].float()
    pv = s["vp"][s["ptable"].long()[ids // ps], ids % ps].float()
    sp = torch.einsum("nhgd,khd->nhgk", q, pk)
    # scores against each sequence's own tokens, the batch padded to T new tokens
    j = torch.arange(L, device=DEV)
    page = s["table"].long()[:, j // ps]
    live = (j < s["lens"].long()[:, None])[..., None, None]
    ok = torch.where(live, s["kp"][page.clamp(min=0), j % ps].float(), 0.0)
    ov = torch.where(live, s["vp"][page.clamp(min=0), j % ps].float(), 0.0)
    qp = torch.zeros((B, T, Hkv, G, D), device=DEV)
    qp[seq, i] = q
    so = torch.einsum("bthgd,blhd->bthgl", qp, ok)
    last = (s["lens"].long() - n)[:, None] + torch.arange(T, device=DEV)
    so = so.masked_fill((j > last[..., None])[:, :, None, None, :], -math.inf)[seq, i]
    m = torch.cat((sp, so), -1).amax(-1, keepdim=True)
    base = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    sp, so = torch.exp(sp - base), torch.exp(so - base)
    total = sp.sum(-1, keepdim=True) + so.sum(-1, keepdim=True)
    wide = torch.zeros((B, T, Hkv, G, L), device=DEV)
    wide[seq, i] = so
    o = torch.einsum("nhgk,khd->nhgd", sp, pv) + \
        torch.einsum("bthgl,blhd->bthgd", wide, ov)[seq, i]
    o = torch.where(total > 0, o / total, 0.0)
    s["o"].view(-1, Hq, D)[r] = o.reshape(-1, Hq, D).to(BF)
    if c["lse"]:
        lse = (base + torch.log(total)).reshape(-1, Hq)
        if c["ragged"]:
            s["lse"][:, r] = lse.t()
        else:
            s["lse"].copy_(lse.view(B, T, Hq).transpose(1, 2))


# ---- the definitions in 64 bits ---------------------------------------------------------------

def _turned(x, pos, s, c, back=False):
    """x [..., heads, D] with each pair as a complex number times m e^{i pos f}."""
    rot = c["rot"]
    z = torch.polar(torch.full_like(s["freq"], s["mscale"]).expand(*pos.shape, -1).contiguous(),
                    pos.to(torch.float64)[..., None] * s["freq"] * (-1 if back else 1))
    f = x[..., :rot].double()
    pairs = f.unflatten(-1, (rot // 2, 2) if c["inter"] else (2, rot // 2))
    if not c["inter"]:
        pairs = pairs.transpose(-1, -2)
    y = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * z.unsqueeze(-2))
    if not c["inter"]:
        y = y.transpose(-1, -2)
    return torch.cat((y.flatten(-2), x[..., rot:].double()), -1)


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "rope":
        S = c["S"]
        pos = s["pos"] if c["given"] else c["start"] + torch.arange(S, device=DEV).repeat(c["B"], 1)
        return {x: _turned(s[x], pos, s, c, c["back"]) for x in ("q", "k")}
    B, T, D, ps = c["B"], c["T"], c["D"], c["page"]
    lens = s["lens"].tolist()
    first = s["cu"].tolist() if c["ragged"] else [T * b for b in range(B + 1)]
    o = s["o"].double()
    flat = o.view(-1, c["Hq"], D)
    rows = {x: s[x].reshape(-1, *s[x].shape[-2:]) for x in ("q", "k", "v") if x in s}
    if c["op"] == "append":
        kp, vp = s["kp"].double(), s["vp"].double()
        for b in range(B):
            lo, hi = first[b], first[b + 1]
            if lo == hi:
                continue
            at = torch.arange(lens[b] - (hi - lo), lens[b], device=DEV)
            flat[lo:hi] = _turned(rows["q"][lo:hi], at + c["start"], s, c)
            page = s["table"][b, at // ps].long()
            kp[page, at % ps] = _turned(rows["k"][lo:hi], at + c["start"], s, c)
            vp[page, at % ps] = rows["v"][lo:hi].double()
        return {"q": o, "kp": kp, "vp": vp}
    P, Hkv = c["prefix"], c["Hkv"]
    G = c["Hq"] // Hkv
    used = first[-1]
    lse = torch.zeros((rows["q"].shape[0], c["Hq"]), dtype=torch.float64, device=DEV)
    for h in range(Hkv):
        q = rows["q"][:used, h * G:(h + 1) * G].double() / D ** 0.5
        pk = s["kp"][s["ptable"].long(), :, h].reshape(-1, D)[:P].double()
        pv = s["vp"][s["ptable"].long(), :, h].reshape(-1, D)[:P].double()
        for b in range(B):
            lo, hi = first[b], first[b + 1]
            if lo == hi:
                continue
            ids = s["table"][b, :-(-lens[b] // ps)].long()
            k = torch.cat((pk, s["kp"][ids, :, h].reshape(-1, D)[:lens[b]].double()))
            v = torch.cat((pv, s["vp"][ids, :, h].reshape(-1, D)[:lens[b]].double()))
            t = q[lo:hi] @ k.t()
            n = hi - lo
            late = torch.ones((n, n), dtype=torch.bool, device=DEV).triu(1)[:, None]
            t[..., -n:] = t[..., -n:].masked_fill(late, -math.inf)
            flat[lo:hi, h * G:(h + 1) * G] = torch.softmax(t, -1) @ v
            lse[lo:hi, h * G:(h + 1) * G] = torch.logsumexp(t, -1)
    if not c["lse"]:
        return {"o": o}
    return {"o": o, "lse": lse.t().contiguous() if c["ragged"]
            else lse.view(B, T, -1).transpose(1, 2).contiguous()}
