"""What the operators around the attention and the readout are measured on: tokens in, norms and
positions of q and k, tokens out.

  norm    norm of each head of q and k, and the rotation of its positions, in one pass: forward,
          backward (with the gradients of the norms' weights) and on the way into a paged cache
  embed   token embedding with a factor, and its gradient: a sum over the places of each token
  logp    log probabilities of given tokens out of the readout h w^T, with the entropy and the most
          likely alternatives

``own`` False computes the plain forms with elementary torch operations, True calls the library.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
BF = torch.bfloat16
EPS = 1e-6


# ---- cases ------------------------------------------------------------------------------------

def _norm(name, B, S, Hq, Hkv, D, rot, inter=False, scaling="none", back=False, fused=False,
          start=0, given=False, wide=False, offset=0.0):
    return {"name": name, "op": "norm", "B": B, "S": S, "Hq": Hq, "Hkv": Hkv, "D": D, "rot": rot,
            "inter": inter, "scaling": scaling, "back": back, "fused": fused, "start": start,
            "given": given, "wide": wide, "offset": offset}


def _append(name, B, T, Hq, Hkv, D, rot, page, own_len, ragged=False, inter=False,
            scaling="none", start=0, wide=False, offset=0.0):
    return {"name": name, "op": "append", "B": B, "T": T, "Hq": Hq, "Hkv": Hkv, "D": D,
            "rot": rot, "page": page, "own_len": own_len, "ragged": ragged, "inter": inter,
            "scaling": scaling, "start": start, "wide": wide, "offset": offset}


def _embed(name, S, Dm, V, back=False, scaled=False):
    return {"name": name, "op": "embed", "S": S, "Dm": Dm, "V": V, "back": back,
            "scaled": scaled}


def _logp(name, S, Dm, V, top):
    return {"name": name, "op": "logp", "S": S, "Dm": Dm, "V": V, "top": top}


def listed():
    return [
        # a training step's q and k at the 8K shape
        _norm("norm_rope_8k", 1, 8192, 32, 8, 128, 128),
        # a 128K prompt far inside a long context, read out of the rows of a fused projection
        _norm("norm_rope_128k_fused", 1, 131072, 32, 8, 128, 128, scaling="parts", fused=True,
              start=900001),
        # the gradient for a packed batch with given positions: interleaved pairs, half the head,
        # odd length, weights in 32 bits that are kept as their distance from one
        _norm("norm_rope_8k_back_part", 2, 4097, 64, 8, 128, 64, inter=True, scaling="ntk",
              back=True, given=True, wide=True, offset=1.0),
        # the gradient of a long training sequence
        _norm("norm_rope_32k_back", 1, 32768, 32, 8, 128, 128, back=True),
        # one decode step of a batch with drafted tokens, padded rows behind the last sequence
        _append("norm_append_batch", 96, 5, 64, 8, 128, 128, 16, 3000, ragged=True,
                scaling="parts", start=70000),
        # the tokens of one decode step of a batch
        _embed("embed_step", 64, 4096, 128256),
        # a long training sequence or prompt, scaled by the root of the width
        _embed("embed_128k", 131072, 4096, 128256, scaled=True),
        # its gradient: the whole table is written, the commonest tokens have thousands of places
        _embed("embed_back_128k", 131072, 4096, 128256, back=True, scaled=True),
        # the gradient of a short sequence for a small table of odd sizes
        _embed("embed_back_odd", 4097, 1000, 32003, back=True),
        # one new token of one sequence: the weights' bytes
        _logp("logp_step", 1, 4096, 128256, 5),
        # a decode step of a batch with many alternatives asked for
        _logp("logp_batch", 48, 4096, 128256, 20),
        # scoring a prompt
        _logp("logp_prompt_4k", 4096, 4096, 128256, 5),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def _unnamed(c):
    return {k: v for k, v in c.items() if k != "name"}


def draw(rng):
    heads = [(32, 8), (64, 8), (16, 16), (4, 4), (28, 4), (40, 8), (8, 1), (24, 8), (10, 2)]
    kind = rng.choice(["norm", "norm", "append", "embed", "embed", "logp", "logp"])
    Hq, Hkv = rng.choice(heads)
    scaling = rng.choice(["none", "linear", "ntk", "parts"])
    inter, wide = rng.random() < 0.5, rng.random() < 0.5
    offset = rng.choice([0.0, 0.0, 1.0])
    if kind == "norm":
        back = rng.random() < 0.5
        D = rng.choice([64, 80, 128, 128, 192, 256])
        rot = rng.choice([D, D, D // 2 // 16 * 16])
        room = (32768 if back else 130000) * 40 * 128 // ((Hq + Hkv) * D + 2)
        n = _log(rng, 1, room)
        B = min(n, rng.choice([1, 1, 2, 3, 7]))
        return _unnamed(_norm("", B, max(1, n // B), Hq, Hkv, D, rot, inter, scaling, back,
                              rng.random() < 0.4, rng.choice([0, rng.randrange(1 << 20)]),
                              rng.random() < 0.4, wide, offset))
    if kind == "append":
        D = rng.choice([64, 128, 128])
        B = _log(rng, 1, 128)
        T = rng.choice([1, 1, rng.randrange(1, 9), _log(rng, 1, max(1, 16384 // B))])
        return _unnamed(_append("", B, T, Hq, Hkv, D, rng.choice([D, D // 2]),
                                rng.choice([16, 32, 48, 64, 128, 256]), T + _log(rng, 1, 3000),
                                rng.random() < 0.5, inter, scaling,
                                rng.choice([0, rng.randrange(1 << 18)]), wide, offset))
    Dm = rng.choice([256, 1000, 1024, 2048, 2568, 4096, 5120])
    V = _log(rng, 1000, 128256)
    if kind == "embed":
        return _unnamed(_embed("", _log(rng, 1, 131072 * 4096 // max(Dm, 4096)), Dm,
                               min(V, 128256 * 4096 // max(Dm, 4096)), rng.random() < 0.5,
                               rng.random() < 0.5))
    S = _log(rng, 1, min(16384, 4096 * 4096 * 128256 // (Dm * V)))
    return _unnamed(_logp("", S, Dm, min(V, 128256 * 4096 // max(Dm, 4096)),
                          rng.choice([0, 1, 5, 8, 20])))


# ---- what a case fixes ------------------------------------------------------------------------

def _counts(c):
    """New tokens and own length (new tokens among them) of each sequence of an append."""
    B, T = c["B"], c["T"]
    n = [b % (T + 1) for b in range(B)] if c["ragged"] and B > 1 else [T] * B
    before = c["own_len"] - T
    return n, [n[b] + (before * (b + 1)) // B for b in range(B)]


def _rows(c):
    """Rows of an append: the sequences' tokens and, in a ragged batch, a few rows behind."""
    n, _ = _counts(c)
    return sum(n) + 3 if c["ragged"] else sum(n)


def _frequency(V):
    """How often the tokens of a text come, the commonest first."""
    p = 1.0 / (np.arange(V, dtype=np.float64) + 2.7)
    return p / p.sum()


def work(c):
    if c["op"] in ("norm", "append"):
        n = c["B"] * c["S"] if c["op"] == "norm" else sum(_counts(c)[0])
        turned = n * (c["Hq"] + c["Hkv"])
        if c["op"] == "append":
            return {"bytes": (turned + n * c["Hkv"]) * c["D"] * 4,
                    "flops": turned * (4 * c["D"] + 3 * c["rot"])}
        back = c["back"]
        return {"bytes": turned * c["D"] * (6 if back else 4) + (8 * n if c["given"] else 0),
                "flops": turned * ((11 if back else 4) * c["D"] + 3 * c["rot"])}
    S, Dm, V = c["S"], c["Dm"], c["V"]
    if c["op"] == "embed":
        if c["back"]:
            return {"bytes": 2 * S * Dm + 4 * V * Dm + 8 * S, "flops": S * Dm}
        rows = float((1 - (1 - _frequency(V)) ** S).sum())
        return {"bytes": int(2 * rows * Dm) + 2 * S * Dm + 8 * S, "flops": S * Dm}
    return {"bytes": 2 * (S + V) * Dm + S * (20 + 12 * c["top"]), "flops": 2 * S * V * Dm}


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


def _normal(shape, g):
    return torch.randn(shape, generator=g, device=DEV, dtype=BF)


def prepare(c, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = {"case": c}
    if c["op"] == "embed":
        return _prepare_embed(c, g, s)
    if c["op"] == "logp":
        return _prepare_logp(c, g, s)
    f, m = _frequencies(c["rot"], c["scaling"])
    s.update(freq=torch.from_numpy(f).to(DEV), mscale=m, phases=_phases(f).to(DEV))
    for x in ("qw", "kw"):  # learned weights: around one, or kept as their distance from it
        y = 1 + 0.3 * torch.randn(c["D"], generator=g, device=DEV) - c["offset"]
        s[x] = y if c["wide"] else y.to(BF)
    return _prepare_norm(c, g, s) if c["op"] == "norm" else _prepare_append(c, g, s, seed)


def _prepare_norm(c, g, s):
    B, S, D, Hq, Hkv = c["B"], c["S"], c["D"], c["Hq"], c["Hkv"]
    if c["fused"]:  # q, k and v of one projection side by side in a row
        x = _normal((B, S, (Hq + 2 * Hkv) * D), g)
        s["q"] = x[..., :Hq * D].unflatten(-1, (Hq, D))
        s["k"] = x[..., Hq * D:(Hq + Hkv) * D].unflatten(-1, (Hkv, D))
    else:
        s["q"], s["k"] = _normal((B, S, Hq, D), g), _normal((B, S, Hkv, D), g)
    s["k"][:, ::7] *= 8  # some keys are large before the norm
    if c["back"]:
        s["dq"], s["dk"] = _normal((B, S, Hq, D), g), _normal((B, S, Hkv, D), g)
    if c["given"]:  # packed documents: positions start again at odd places
        p = torch.arange(S, device=DEV).repeat(B, 1) + c["start"]
        cut = torch.randint(0, S, (B, 1), generator=g, device=DEV)
        s["pos"] = torch.where(p - c["start"] >= cut, p - c["start"] - cut, p)
    return s


def _prepare_append(c, g, s, seed):
    rng = np.random.default_rng(seed)
    n, lens = _counts(c)
    B, T, D, Hq, Hkv, ps = c["B"], c["T"], c["D"], c["Hq"], c["Hkv"], c["page"]
    order = rng.permutation(B)
    n, lens = [n[i] for i in order], [lens[i] for i in order]
    shape = (_rows(c),) if c["ragged"] else (B, T)
    need = [-(-m // ps) for m in lens]
    pages = sum(need) + 2
    perm = rng.permutation(pages)
    table = np.full((B, -(-c["own_len"] // ps)), -1, dtype=np.int32)
    at = 0
    for b in range(B):
        table[b, :need[b]] = perm[at:at + need[b]]
        at += need[b]
    s["table"] = torch.from_numpy(table).to(DEV)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    s["cu"] = (torch.tensor([0] + list(np.cumsum(n)), dtype=torch.int32, device=DEV)
               if c["ragged"] else None)
    s["q"] = _normal(shape + (Hq, D), g)
    s["o"] = torch.zeros_like(s["q"])
    s["k"], s["v"] = _normal(shape + (Hkv, D), g), _normal(shape + (Hkv, D), g)
    s["kp"], s["vp"] = _normal((pages, ps, Hkv, D), g), _normal((pages, ps, Hkv, D), g)
    return s


def _prepare_embed(c, g, s):
    S, Dm, V = c["S"], c["Dm"], c["V"]
    names = torch.randperm(V, generator=g, device=DEV)
    often = torch.from_numpy(_frequency(V)).to(DEV)
    s["tokens"] = names[torch.multinomial(often, S, replacement=True, generator=g)]
    if S > 8:  # the end of the last sequence is padding
        s["tokens"][-3:] = -1
    s["scale"] = math.sqrt(Dm) if c["scaled"] else 1.0
    if c["back"]:
        s["dh"] = _normal((S, Dm), g)
    else:
        s["w"] = _normal((V, Dm), g) * 0.03
    return s


def _prepare_logp(c, g, s):
    S, Dm, V = c["S"], c["Dm"], c["V"]
    s["w"] = _normal((V, Dm), g) * (2 / math.sqrt(Dm))
    s["target"] = torch.randint(0, V, (S,), generator=g, device=DEV)
    # from tokens that the model does not expect to ones that it is nearly certain of
    sure = 5 * torch.rand((S, 1), generator=g, device=DEV)
    s["h"] = (torch.randn((S, Dm), generator=g, device=DEV) +
              sure * s["w"][s["target"]].float()).to(BF)
    s["target"][S // 16 * 15 + 1:] = -1  # the end of the last sequence is padding
    return s


# ---- one pass ---------------------------------------------------------------------------------

def run(s):
    c = s["case"]
    return {"norm": _run_norm, "append": _run_append, "embed": _run_embed,
            "logp": _run_logp}[c["op"]](s, c)


def _run_norm(s, c):
    if own:
        import context_parallelism_gb300 as up
        how = dict(phases=s["phases"], mscale=s["mscale"], eps=EPS, offset=c["offset"],
                   interleaved=c["inter"], positions=s.get("pos"), start=c["start"])
        if c["back"]:
            dq, dk, dqw, dkw = up.norm_rope_backward(s["dq"], s["dk"], s["q"], s["k"], s["qw"],
                                                     s["kw"], **how)
            return {"dq": dq, "dk": dk, "dqw": dqw, "dkw": dkw}
        q, k = up.norm_rope_forward(s["q"], s["k"], s["qw"], s["kw"], **how)
        return {"q": q, "k": k}
    B, S = c["B"], c["S"]
    pos = s["pos"] if c["given"] else (torch.arange(S, device=DEV) + c["start"]).expand(B, S)
    cos, sin = _cos_sin(s, pos)
    if c["back"]:
        dq, dqw = _plain_back(s["dq"], s["q"], s["qw"], cos, sin, c)
        dk, dkw = _plain_back(s["dk"], s["k"], s["kw"], cos, sin, c)
        return {"dq": dq, "dk": dk, "dqw": dqw, "dkw": dkw}
    return {"q": _plain(s["q"], s["qw"], cos, sin, c), "k": _plain(s["k"], s["kw"], cos, sin, c)}


def _cos_sin(s, pos):
    a = pos.to(torch.float64).unsqueeze(-1) * s["freq"]  # far positions: angles in 64 bits
    return ((torch.cos(a) * s["mscale"]).float().unsqueeze(-2),
            (torch.sin(a) * s["mscale"]).float().unsqueeze(-2))


def _rotate(f, cos, sin, c):
    rot = c["rot"]
    if c["inter"]:
        a, b = f[..., 0:rot:2], f[..., 1:rot:2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = f[..., :rot // 2], f[..., rot // 2:rot]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((y, f[..., rot:]), -1)


def _plain(x, w, cos, sin, c):
    f = x.float()
    f = f * torch.rsqrt(f.square().mean(-1, keepdim=True) + EPS) * (c["offset"] + w.float())
    return _rotate(f, cos, sin, c).to(BF)


def _plain_back(dy, x, w, cos, sin, c):
    """The gradients of the input and of the weights."""
    f = x.float()
    r = torch.rsqrt(f.square().mean(-1, keepdim=True) + EPS)
    g = _rotate(dy.float(), cos, -sin, c)
    f = f * r
    dw = (g * f).flatten(0, -2).sum(0, dtype=torch.float64).float()  # a long sum
    g = g * (c["offset"] + w.float())
    return (r * (g - f * (g * f).mean(-1, keepdim=True))).to(BF), dw


def _run_append(s, c):
    if own:
        import context_parallelism_gb300 as up
        up.kv_append(s["k"], s["v"], s["kp"], s["vp"], s["table"], s["lens"], q=s["q"],
                     q_out=s["o"], phases=s["phases"], mscale=s["mscale"],
                     interleaved=c["inter"], start=c["start"], cu_seqlens=s["cu"],
                     q_weight=s["qw"], k_weight=s["kw"], eps=EPS, offset=c["offset"])
        return {"q": s["o"], "kp": s["kp"], "vp": s["vp"]}
    B, T, D = c["B"], c["T"], c["D"]
    if c["ragged"]:
        r = torch.arange(_rows(c) - 3, device=DEV)
        seq = torch.searchsorted(s["cu"][1:].long(), r, right=True)
        i, n = r - s["cu"].long()[seq], (s["cu"][1:] - s["cu"][:-1]).long()
    else:
        r = torch.arange(B * T, device=DEV)
        seq, i, n = r // T, r % T, torch.full((B,), T, device=DEV)
    at = s["lens"].long()[seq] - n[seq] + i
    cos, sin = _cos_sin(s, at + c["start"])
    q, k, v = (s[x].reshape(-1, s[x].shape[-2], D)[r] for x in ("q", "k", "v"))
    page, slot = s["table"].long()[seq, at // c["page"]], at % c["page"]
    s["kp"][page, slot] = _plain(k, s["kw"], cos, sin, c)
    s["vp"][page, slot] = v
    s["o"].view(-1, c["Hq"], D)[r] = _plain(q, s["qw"], cos, sin, c)
    return {"q": s["o"], "kp": s["kp"], "vp": s["vp"]}


def _run_embed(s, c):
    if own:
        import context_parallelism_gb300 as up
        if c["back"]:
            return {"dw": up.embed_backward(s["tokens"], s["dh"], c["V"], scale=s["scale"])}
        return {"h": up.embed_forward(s["tokens"], s["w"], scale=s["scale"])}
    t = s["tokens"]
    live = (t >= 0)[:, None]
    if c["back"]:
        dw = torch.zeros((c["V"], c["Dm"]), device=DEV)
        dw.index_add_(0, t.clamp(min=0), torch.where(live, s["dh"].float(), 0.0))
        return {"dw": dw * s["scale"]}
    return {"h": torch.where(live, s["w"][t.clamp(min=0)].float() * s["scale"], 0.0).to(BF)}


def _run_logp(s, c):
    if own:
        import context_parallelism_gb300 as up
        logp, entropy, lse, top_logp, top_index = up.token_logprobs(s["h"], s["w"], s["target"],
                                                                    top=c["top"])
        r = {"logp": logp, "entropy": entropy, "lse": lse}
        if c["top"]:
            r.update(top_logp=top_logp, top_index=top_index)
        return r
    t, top = s["target"], c["top"]
    live = t >= 0
    t = t.clamp(min=0)
    x = s["h"].float() @ s["w"].float().t()
    # the largest logits and the target's in 64 bits: which of two near ones is the larger, and how
    # far a probability near one is from it, are lost in 32
    near = x.topk(min(c["V"], top + 8), dim=-1).indices.sort(-1).values
    y = (s["w"][near].double() @ s["h"][..., None].double())[..., 0]
    yt = (s["w"][t].double() * s["h"].double()).sum(-1, keepdim=True)
    m = y.amax(-1, keepdim=True)
    d = (x - m.float()).scatter(1, near, (y - m).float())
    d = d.scatter(1, t[:, None], (yt - m).float())
    e = torch.exp(d)
    z = e.sum(-1, keepdim=True, dtype=torch.float64)
    log_z = torch.log(z)
    r = {"logp": torch.where(live, (yt - m - log_z)[:, 0], 0.0).float(),
         "entropy": (log_z - (e * d).sum(-1, keepdim=True, dtype=torch.float64) / z)[:, 0].float(),
         "lse": (m + log_z)[:, 0].float()}
    if top:
        by = torch.sort(y, dim=-1, descending=True, stable=True).indices[:, :top]
        r["top_index"] = near.gather(1, by)
        r["top_logp"] = (y.gather(1, by) - m - log_z).float()
    return r


# ---- the definitions in 64 bits ---------------------------------------------------------------

def _definition(x, w, pos, s, c):
    """x [..., heads, D], normed by its root mean square, each pair as a complex number times
    m e^{i pos f}."""
    rot = c["rot"]
    y = x / (x.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * (w + c["offset"])
    turn = torch.polar(torch.full_like(s["freq"], s["mscale"]).expand(*pos.shape, -1).contiguous(),
                       pos.double()[..., None] * s["freq"])
    z = y[..., :rot].unflatten(-1, (rot // 2, 2) if c["inter"] else (2, rot // 2))
    if not c["inter"]:
        z = z.transpose(-1, -2)
    z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * turn.unsqueeze(-2))
    if not c["inter"]:
        z = z.transpose(-1, -2)
    return torch.cat((z.flatten(-2), y[..., rot:]), -1)


def exact(c, seed):
    s = prepare(c, seed)
    return {"norm": _exact_norm, "append": _exact_append, "embed": _exact_embed,
            "logp": _exact_logp}[c["op"]](s, c)


def _exact_norm(s, c):
    pos = s["pos"] if c["given"] else \
        c["start"] + torch.arange(c["S"], device=DEV).repeat(c["B"], 1)
    r = {}
    for x in ("q", "k"):
        if not c["back"]:
            # long sequences in pieces: 64-bit copies of everything at once are large
            r[x] = torch.cat([_definition(a.double(), s[x + "w"].double(), p, s, c)
                              for a, p in zip(s[x].split(16384, 1), pos.split(16384, 1))], 1)
            continue
        parts, dw = [], 0
        for a, d, p in zip(s[x].split(8192, 1), s["d" + x].split(8192, 1), pos.split(8192, 1)):
            a = a.double().requires_grad_()
            w = s[x + "w"].double().requires_grad_()
            da, b = torch.autograd.grad(_definition(a, w, p, s, c), (a, w), d.double())
            parts.append(da)
            dw = dw + b
        r["d" + x], r["d" + x + "w"] = torch.cat(parts, 1), dw
    return r


def _exact_append(s, c):
    B, T, ps = c["B"], c["T"], c["page"]
    lens = s["lens"].tolist()
    first = s["cu"].tolist() if c["ragged"] else [T * b for b in range(B + 1)]
    o, kp, vp = s["o"].double(), s["kp"].double(), s["vp"].double()
    flat = o.view(-1, c["Hq"], c["D"])
    rows = {x: s[x].reshape(-1, *s[x].shape[-2:]).double() for x in ("q", "k", "v")}
    for b in range(B):
        lo, hi = first[b], first[b + 1]
        if lo == hi:
            continue
        at = torch.arange(lens[b] - (hi - lo), lens[b], device=DEV)
        flat[lo:hi] = _definition(rows["q"][lo:hi], s["qw"].double(), at + c["start"], s, c)
        page = s["table"][b, at // ps].long()
        kp[page, at % ps] = _definition(rows["k"][lo:hi], s["kw"].double(), at + c["start"], s, c)
        vp[page, at % ps] = rows["v"][lo:hi]
    return {"q": o, "kp": kp, "vp": vp}


def _exact_embed(s, c):
    live = s["tokens"] >= 0
    if c["back"]:
        # one-hot rows of the tokens that occur, times the gradients: a sum per token
        dw = torch.zeros((c["V"], c["Dm"]), dtype=torch.float64, device=DEV)
        order = torch.argsort(s["tokens"][live], stable=True)
        t, n = torch.unique_consecutive(s["tokens"][live][order], return_counts=True)
        d = s["dh"][live][order].double()
        if len(t):
            dw[t] = torch.segment_reduce(d, "sum", lengths=n, axis=0) * s["scale"]
        return {"dw": dw}
    h = torch.zeros((c["S"], c["Dm"]), dtype=torch.float64, device=DEV)
    h[live] = s["w"].double()[s["tokens"][live]] * s["scale"]
    return {"h": h}


def _exact_logp(s, c):
    S, V, top = c["S"], c["V"], c["top"]
    if 2 * S * V * c["Dm"] > 1e13:
        return None
    r = {x: [] for x in ("logp", "entropy", "lse") + (("top_logp", "top_index") if top else ())}
    w = s["w"].double()
    for h, t in zip(s["h"].split(512), s["target"].split(512)):
        p = torch.log_softmax(h.double() @ w.t(), -1)
        r["logp"].append(torch.where(t >= 0, p.gather(1, t.clamp(min=0)[:, None])[:, 0], 0.0))
        r["entropy"].append(-(p.exp() * p).sum(-1))
        r["lse"].append((h.double() * w[0]).sum(-1) - p[:, 0])
        if top:
            v, i = torch.sort(p, dim=-1, descending=True, stable=True)
            r["top_logp"].append(v[:, :top])
            r["top_index"].append(i[:, :top])
    return {x: torch.cat(y) for x, y in r.items()}
