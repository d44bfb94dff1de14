"""One layer from tokens to log probabilities, as the operators are used together: a training step with a
tied table, and a prefill with decoding steps over the paged cache (needs an sm_103a GPU).

Tolerances. Every intermediate is rounded to bf16 (2^-9 of its norm, as the roundings are independent):
embedding, projections, normed q and k, attention's weights and output, the second projection, and in
the backward the same again: fewer than 16 roundings on any way, 4 x 2^-9 together, and the attention's
own gradients are good to 2e-2. Log probabilities move by the change of a logit: a row of 128 features
off by 4 x 2^-9 of its norm, against rows of w of norm 2.
"""
import math

import pytest
import torch

import context_parallelism_gb300 as up

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16

V, Dm, Hq, Hkv, D = 640, 128, 4, 2, 64


def _model(seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def r(*s, scale=1.0):
        return (torch.randn(s, generator=g, device=DEV) * scale).to(BF)

    return {"w": r(V, Dm, scale=2 / math.sqrt(Dm)), "qkv": r((Hq + 2 * Hkv) * D, Dm, scale=Dm ** -0.5),
            "out": r(Dm, Hq * D, scale=(Hq * D) ** -0.5),
            "qn": (1 + 0.2 * r(D).float()).to(BF), "kn": (1 + 0.2 * r(D).float()).to(BF)}


SCALE = math.sqrt(Dm)


def _reference(m, t, start=0):
    """Hidden rows of tokens t [B, S] in 64 bits (autograd through m's tensors)."""
    B, S = t.shape
    x = m["w"][t] * SCALE
    qkv = (x @ m["qkv"].t()).unflatten(-1, (Hq + 2 * Hkv, D))
    q, k, v = qkv[..., :Hq, :], qkv[..., Hq:Hq + Hkv, :], qkv[..., Hq + Hkv:, :]
    f = 10000.0 ** (-torch.arange(0, D, 2, device=DEV, dtype=torch.float64) / D)
    a = (torch.arange(S, device=DEV)[:, None] + start) * f
    c, s = a.cos()[:, None], a.sin()[:, None]

    def turn(x, w):
        x = x * (x.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * w
        return torch.cat((x[..., :D // 2] * c - x[..., D // 2:] * s,
                          x[..., D // 2:] * c + x[..., :D // 2] * s), -1)

    q, k = turn(q, m["qn"]), turn(k, m["kn"])
    k, v = k.repeat_interleave(Hq // Hkv, 2), v.repeat_interleave(Hq // Hkv, 2)
    p = torch.einsum("bihd,bjhd->bhij", q, k) / math.sqrt(D)
    late = torch.ones(S, S, dtype=torch.bool, device=DEV).triu(1)
    o = torch.einsum("bhij,bjhd->bihd", p.masked_fill(late, -math.inf).softmax(-1), v)
    return x + o.flatten(2) @ m["out"].t()


def _split(qkv):
    qkv = qkv.unflatten(-1, (Hq + 2 * Hkv, D))
    return qkv[..., :Hq, :], qkv[..., Hq:Hq + Hkv, :], qkv[..., Hq + Hkv:, :].contiguous()


def _rel(x, ref):
    return ((x.double() - ref).norm() / ref.norm()).item()


def test_training_step_with_a_tied_table():
    m = _model()
    B, S = 1, 384
    t = torch.randint(0, V, (B, S), device=DEV)
    t[:, 50:60] = t[:, 49:50]
    target = t.roll(-1, 1)
    target[:, -1] = -1
    ph, ms = up.rope_phases(D)
    x = up.embed_forward(t, m["w"], scale=SCALE)
    q0, k0, v = _split(x @ m["qkv"].t())
    q, k = up.norm_rope_forward(q0, k0, m["qn"], m["kn"], ph, ms)
    q, k = q.contiguous(), k.contiguous()
    o, lse = up.attention_forward(q, k, v)
    h = (x.float() + (o.flatten(2) @ m["out"].t()).float()).to(BF)
    g = torch.full((S,), 1 / (S - 1), device=DEV)
    flat = h.view(S, Dm)
    loss, row_lse, dh, dw = up.ce_loss_fused(flat, m["w"], target.view(-1), g, seq_tile=128)
    logp, entropy, lse2, top, index = up.token_logprobs(flat, m["w"], target.view(-1), top=3)
    assert (logp + loss).abs().max() <= 1e-4 and (lse2 - row_lse).abs().max() <= 1e-4
    dh = dh.view(B, S, Dm)
    do = (dh @ m["out"]).unflatten(-1, (Hq, D)).contiguous()
    dq, dk, dv = up.attention_backward(q, k, v, o, lse, do)
    dq, dk, dqn, dkn = up.norm_rope_backward(dq, dk, q0, k0, m["qn"], m["kn"], ph, ms)
    dqkv = torch.cat((dq, dk, dv), 2).flatten(2)
    dx = (dh.float() + (dqkv @ m["qkv"]).float()).to(BF)
    readout = dw.clone()
    up.embed_backward(t, dx, V, scale=SCALE, dw=dw)
    up.upipe_sync_status()

    r = {n: p.double().requires_grad_() for n, p in m.items()}
    rh = _reference(r, t).view(S, Dm)
    p = torch.log_softmax(rh @ r["w"].t(), -1)
    live = target.view(-1) >= 0
    want = p.gather(1, target.view(-1).clamp(min=0)[:, None])[:, 0] * live
    grads = torch.autograd.grad(-(want * g).sum(), [r[n] for n in ("w", "qn", "kn", "qkv")])
    assert _rel(flat, rh.detach()) <= 4 * 2.0 ** -9
    assert _rel(logp, want.detach()) <= 1e-2
    for got, ref in ((dw, grads[0]), (dqn, grads[1]), (dkn, grads[2]),
                     (dqkv.view(S, -1).t().float() @ x.view(S, Dm).float(), grads[3])):
        assert _rel(got, ref) <= 4e-2
    # rows of the tokens alone; the last place has no target and no later query, so its gradient is zero
    changed = (dw != readout).any(1).nonzero().flatten().tolist()
    assert changed == sorted(set(t[0, :-1].tolist()))


@pytest.mark.parametrize("packed", [False, True])
def test_prefill_and_decode(packed):
    """A prompt through attention_forward and into pages, then steps that take the most likely token:
    each step's log probabilities are those of the whole text at once."""
    m = _model(1)
    B, P, steps, ps = 3, 200, 5, 16
    prompt = torch.randint(0, V, (1, P), device=DEV)
    ph, ms = up.rope_phases(D)
    pages = -(-P // ps)
    kp = torch.zeros((pages + B, ps, Hkv, D), dtype=BF, device=DEV)
    vp = torch.zeros_like(kp)
    shared = torch.arange(pages, dtype=torch.int32, device=DEV)
    table = pages + torch.arange(B, dtype=torch.int32, device=DEV)[:, None]
    norms = dict(q_weight=m["qn"], k_weight=m["kn"], eps=1e-6, phases=ph, mscale=ms)

    x = up.embed_forward(prompt, m["w"], scale=SCALE)
    q, k, v = _split(x @ m["qkv"].t())
    qr, kr = up.norm_rope_forward(q, k, m["qn"], m["kn"], ph, ms)
    up.kv_append(k, v, kp, vp, shared[None], torch.tensor([P], dtype=torch.int32, device=DEV), **norms)
    o, _ = up.attention_forward(qr.contiguous(), kr.contiguous(), v, with_lse=False)
    assert torch.equal(kp[:pages].flatten(0, 1)[:P], kr[0])  # the cache holds the normed, turned keys
    h = (x.float() + (o.flatten(2) @ m["out"].t()).float()).to(BF)
    _, _, _, top, index = up.token_logprobs(h[0, -1:], m["w"], top=B)
    tokens, logps = index[0].clone(), []           # each sequence goes on with another token
    text = [tokens]
    lens = torch.zeros(B, dtype=torch.int32, device=DEV)
    cu = torch.arange(B + 1, dtype=torch.int32, device=DEV) if packed else None
    for _ in range(steps):
        lens += 1
        x = up.embed_forward(tokens if packed else tokens[:, None], m["w"], scale=SCALE)
        q, k, v = _split(x @ m["qkv"].t())
        qr = up.kv_append(k, v, kp, vp, table, lens, q=q, start=P, cu_seqlens=cu, **norms)
        o, _ = up.paged_attention(qr, kp, vp, table, lens, prefix_table=shared, prefix_len=P,
                                  cu_seqlens=cu, max_q=1, max_len=steps)
        h = (x.float() + (o.flatten(-2) @ m["out"].t()).float()).to(BF)
        logp, entropy, _, top, index = up.token_logprobs(h.view(B, Dm), m["w"], tokens, top=4)
        tokens = index[:, 0].clone()
        logps.append((logp, entropy, top, index))
        text.append(tokens)
    up.upipe_sync_status()

    text = torch.stack(text[:-1], 1)
    r = {n: p.double() for n, p in m.items()}
    full = torch.cat((prompt.expand(B, P), text), 1)
    p = torch.log_softmax(_reference(r, full) @ r["w"].t(), -1)[:, P:]
    off = 4 * 2.0 ** -9 * 2 * _reference(r, full).norm(dim=-1).max().item()  # of a logit, twice below
    for i, (logp, entropy, top, index) in enumerate(logps):
        assert (logp.double() - p[:, i].gather(1, text[:, i:i + 1])[:, 0]).abs().max() <= 2 * off
        assert (top.double() - p[:, i].gather(1, index)).abs().max() <= 2 * off
        assert (top[:, :-1] >= top[:, 1:] - 1e-5).all()


def test_two_threads():
    """Calls from two threads at once, each on a stream of its own."""
    import threading

    m = _model(2)
    ph, _ = up.rope_phases(D)
    want, got, errors = [], [None, None], []

    def work(seed):
        g = torch.Generator(device=DEV).manual_seed(seed)
        t = torch.randint(-1, V, (3000,), generator=g, device=DEV)
        x = up.embed_forward(t, m["w"], scale=2.0)
        q = x.view(1, 3000, Dm // D, D)
        y, _ = up.norm_rope_forward(q, None, m["qn"], None, ph, start=seed)
        dx, _, dw, _ = up.norm_rope_backward(y, None, q, None, m["qn"], None, ph, start=seed)
        table = up.embed_backward(t, dx.view(3000, Dm), V, scale=2.0)
        out = up.token_logprobs(y.view(3000, Dm), m["w"], t, top=5)
        few = up.token_logprobs(y.view(3000, Dm)[:3].clone(), m["w"], t[:3].clone(), top=5)
        return [x, y, dx, dw, table, *out, *few]

    for seed in (0, 1):
        want.append(work(seed))
    torch.cuda.synchronize()

    def run(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(20):
                    got[i] = work(i)
            s.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in (0, 1)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not errors, errors
    up.upipe_sync_status()
    for a, b in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
