"""Linear attention with a decay per head and attention over a paged cache: the work that is measured.

Five calls of the library are covered: the chunked prefill (``la_forward``), its gradients
(``la_backward``), the single-token step on a recurrent state (``la_decode_step``) and the
single-token step on a paged key-value cache (``paged_decode_step``).  ``run`` computes each in
plain torch operations, or, where ``own`` is true, through the library.

The linear attention of one head with decay a = exp(g), g <= 0:

    S_t = a S_{t-1} + k_t v_t^T,    o_t = scale * S_t^T q_t.
"""
from __future__ import annotations

import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # a short user turn appended to a conversation whose state is carried: latency
        dict(name="la_prefill_turn", op="la_forward", B=1, T=61, H=32, dk=128, dv=128, dtype="bf16",
             state=True, decay="slopes"),
        # the library's 4096-token prompt of 16 heads
        dict(name="la_prefill_4k", op="la_forward", B=1, T=4096, H=16, dk=128, dv=128, dtype="bf16",
             state=False, decay="retention"),
        # the library's long-context prompt: few heads, 65536 tokens
        dict(name="la_prefill_64k", op="la_forward", B=1, T=65536, H=32, dk=128, dv=128, dtype="bf16",
             state=False, decay="slopes"),
        # a batch of long prompts that continue from carried states
        dict(name="la_prefill_batch", op="la_forward", B=4, T=16384, H=32, dk=128, dv=128, dtype="bf16",
             state=True, decay="retention"),
        # fp32 layers of small heads, a length that no tile divides
        dict(name="la_prefill_f32", op="la_forward", B=2, T=1023, H=8, dk=64, dv=64, dtype="f32",
             state=True, decay="retention"),
        # gradients of one training sequence
        dict(name="la_train_4k", op="la_backward", B=1, T=4096, H=16, dk=128, dv=128, dtype="bf16",
             state=False, decay="retention"),
        # gradients of a training batch of an odd length whose states are carried between segments
        dict(name="la_train_batch", op="la_backward", B=4, T=2047, H=32, dk=128, dv=128, dtype="bf16",
             state=True, decay="slopes"),
        # one conversation's next token
        dict(name="la_decode_1", op="la_decode", B=1, T=1, H=32, dk=128, dv=128, dtype="bf16",
             state=True, decay="slopes"),
        # the library's decode batch: 256 sequences of 32 heads
        dict(name="la_decode_256", op="la_decode", B=256, T=1, H=32, dk=128, dv=128, dtype="bf16",
             state=True, decay="retention"),
        # one long conversation: the split over the length has to fill the machine
        dict(name="paged_long", op="paged", B=1, H=32, Hkv=8, D=128, page=64, longest=131070, shortest=131070,
             dtype="bf16"),
        # a serving batch of ragged lengths, small pages, idle rows among them
        dict(name="paged_ragged", op="paged", B=64, H=32, Hkv=8, D=128, page=16, longest=8190, shortest=-1,
             dtype="bf16"),
        # fp32, one key-value head per query head, small heads and short caches: latency
        dict(name="paged_f32", op="paged", B=24, H=16, Hkv=16, D=64, page=16, longest=500, shortest=0,
             dtype="f32"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("la_forward", "la_forward", "la_backward", "la_decode", "paged", "paged"))
    dtype = "f32" if rng.random() < 0.25 else "bf16"
    if op == "paged":
        D, group = rng.choice((64, 128)), rng.choice((1, 2, 4, 7, 8))
        Hkv = rng.choice((1, 2, 4, 8))
        B = _log_int(rng, 1, 128)
        # the cache of a drawn batch holds no more than the largest listed one
        most = max(2, min(131070, 2 ** 30 // (B * Hkv * D * (8 if dtype == "f32" else 4))))
        longest = _log_int(rng, 1, most)
        shortest = rng.choice((-1, 0, longest // 2, longest))
        return dict(op=op, B=B, H=Hkv * group, Hkv=Hkv, D=D, page=rng.choice((8, 16, 32, 64, 100)),
                    longest=longest, shortest=shortest, dtype=dtype)
    dk, dv = (128, 128) if rng.random() < 0.6 else (rng.choice((64, 128)), rng.choice((64, 128)))
    case = dict(op=op, B=_log_int(rng, 1, 8), T=1, H=_log_int(rng, 1, 48), dk=dk, dv=dv, dtype=dtype,
                state=rng.random() < 0.6, decay=rng.choice(("slopes", "retention", "none")))
    if op == "la_decode":
        case.update(B=_log_int(rng, 1, 256), H=_log_int(rng, 1, 32), state=True)
        return case
    # tokens x heads of the largest listed case bound a drawn one (a fraction of it in fp32, and for gradients)
    most = 65536 * 32 // (case["B"] * case["H"] * (8 if dtype == "f32" else 2) * (4 if op == "la_backward" else 1))
    case["T"] = _log_int(rng, 1, max(2, min(65536, most)))
    return case


# ------------------------------------------------------------------------------- inputs
def _log_decay(kind, H, dev):
    """log of the decay of each head: geometric slopes, or 1 - 2^-(5..12)."""
    h = torch.arange(H, device=dev, dtype=torch.float64)
    if kind == "none":
        return None
    if kind == "slopes":
        return (-torch.pow(2.0, -8.0 * (h + 1) / H)).float()
    return torch.log1p(-torch.pow(2.0, -5.0 - 7.0 * h / max(H - 1, 1))).float()


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt = _TYPES[case["dtype"]]

    def normal(*shape, sd=1.0):
        return torch.randn(shape, generator=gen, device=dev).mul_(sd)

    if case["op"] == "paged":
        B, H, Hkv, D, page = case["B"], case["H"], case["Hkv"], case["D"], case["page"]
        lo, hi = case["shortest"], case["longest"]
        lengths = torch.randint(lo, hi + 1, (B,), generator=gen, device=dev, dtype=torch.int32)
        lengths[0] = hi
        per_seq = hi // page + 1                       # room for the new token
        pages = torch.randperm(B * per_seq + 3, generator=gen, device=dev)[: B * per_seq]
        shape = (B * per_seq + 3, page, Hkv, D)
        return dict(case=case, q=normal(B, H, D).to(dt), k=normal(B, Hkv, D).to(dt), v=normal(B, Hkv, D).to(dt),
                    k_cache=normal(*shape).to(dt), v_cache=normal(*shape).to(dt),
                    block_table=pages.to(torch.int32).reshape(B, per_seq).contiguous(), lengths=lengths)

    B, T, H, dk, dv = (case[n] for n in ("B", "T", "H", "dk", "dv"))
    lead = (B, H) if case["op"] == "la_decode" else (B, T, H)

    def unit(d):
        x = normal(*lead, d)
        return x.div_(x.norm(dim=-1, keepdim=True)).to(dt)

    s = dict(case=case, q=unit(dk), k=unit(dk), v=normal(*lead, dv).to(dt),
             log_decay=_log_decay(case["decay"], H, dev),
             state=normal(B, H, dk, dv, sd=0.1) if case["state"] else None)
    if case["op"] == "la_backward":
        s["grad_out"] = normal(*lead, dv).to(dt)
        s["grad_state"] = normal(B, H, dk, dv, sd=0.1) if case["state"] else None
    return s


# ------------------------------------------------------------------------------- plain forms
def _powers(g, n):
    """exp(g n) in 64 bits: g [H] or None (no decay), n any integer tensor -> [H, *n.shape]."""
    g = torch.zeros(1, device=n.device) if g is None else g
    return torch.exp(g.double().reshape((-1,) + (1,) * n.dim()) * n.double())


def _linear_attention(q, k, v, g, s0, late):
    """Unscaled outputs and last state of q, k, v [B, H, T, d] in fp32, by chunks and without a loop.

    The state enters token i of the sequence as a^(i + late) S0; after n tokens it is
    a^n S0 + sum_j a^(n - late - j) k_j v_j^T: late = 1 decays before the write (the forward
    recurrence), late = 0 after it (the adjoint's, in reversed time).
    """
    B, H, T, dk = q.shape
    dv, dev = v.shape[-1], q.device
    C = min(256, T)
    N = -(-T // C)
    pad = (0, 0, 0, N * C - T)
    q, k, v = (torch.nn.functional.pad(x, pad).reshape(B, H, N, C, -1) for x in (q, k, v))
    i = torch.arange(C, device=dev)
    n = torch.arange(N, device=dev)
    apart = i[:, None] - i[None, :]
    mask = torch.where(apart >= 0, _powers(g, apart.clamp(min=0)), 0.0).float()              # [H, C, C]
    out = ((q @ k.transpose(-1, -2)) * mask[:, None]) @ v
    count = torch.clamp(T - n * C, max=C)                                                    # tokens of each chunk
    left = count[:, None] - late - i[None, :]
    w = torch.where(left + late > 0, _powers(g, left.clamp(min=0)), 0.0).float()             # [H, N, C]
    local = (k * w[..., None]).transpose(-1, -2) @ v                                         # [B, H, N, dk, dv]
    since = n[:, None] - 1 - n[None, :]
    carry = torch.where(since >= 0, _powers(g, C * since.clamp(min=0)), 0.0).float()         # [H, N, N]
    start = (carry @ local.reshape(B, H, N, dk * dv)).reshape(B, H, N, dk, dv)
    if s0 is not None:
        start = start + _powers(g, n * C).float()[:, :, None, None] * s0[:, :, None]
    out = out + _powers(g, i + late).float()[:, None, :, None] * (q @ start)
    last = _powers(g, count[-1]).float()[:, None, None] * start[:, :, -1] + local[:, :, -1]
    return out.reshape(B, H, N * C, dv)[:, :, :T], last


def _heads(x):
    return x.float().transpose(1, 2)


def _tokens(x, dt):
    return x.transpose(1, 2).contiguous().to(dt)


def _plain_forward(s):
    q, k, v = (_heads(s[n]) for n in ("q", "k", "v"))
    out, last = _linear_attention(q, k, v, s["log_decay"], s["state"], 1)
    return _tokens(out * s["case"]["dk"] ** -0.5, s["q"].dtype), last


def _plain_backward(s):
    g, dt, scale = s["log_decay"], s["q"].dtype, s["case"]["dk"] ** -0.5
    q, k, v, do = (_heads(s[n]) for n in ("q", "k", "v", "grad_out"))
    s0, gs = s["state"], s["grad_state"]
    dq, _ = _linear_attention(do, v, k, g, None if s0 is None else s0.transpose(-1, -2), 1)
    # reversed time: the adjoint state is a linear attention's state over (q, do)
    rq, rk, rv, rdo = (x.flip(2) for x in (q * scale, k, v, do))
    dv, ds0 = _linear_attention(rk, rq, rdo, g, gs, 0)
    dk, _ = _linear_attention(rv, rdo, rq, g, None if gs is None else gs.transpose(-1, -2), 0)
    return dict(dq=_tokens(dq * scale, dt), dk=_tokens(dk.flip(2), dt), dv=_tokens(dv.flip(2), dt),
                dinitial_state=ds0)


def _plain_decode(s):
    q, k, v, state = s["q"].float(), s["k"].float(), s["v"].float(), s["state"]
    if s["log_decay"] is not None:
        state.mul_(torch.exp(s["log_decay"].double()).float()[:, None, None])
    state.add_(k[..., :, None] * v[..., None, :])
    out = (q[..., None, :] @ state).squeeze(-2) * s["case"]["dk"] ** -0.5
    return out.to(s["q"].dtype), state


def _plain_paged(s):
    case = s["case"]
    B, H, Hkv, D, page = case["B"], case["H"], case["Hkv"], case["D"], case["page"]
    table, lengths = s["block_table"].long(), s["lengths"].long()
    kc, vc = s["k_cache"], s["v_cache"]
    # the new token's key and value go to position `length` of every row that is not idle
    at = lengths.clamp(min=0)
    where = (table.gather(1, (at // page)[:, None])[:, 0], at % page)
    busy = (lengths >= 0)[:, None, None]
    kc[where] = torch.where(busy, s["k"], kc[where])
    vc[where] = torch.where(busy, s["v"], vc[where])
    k = kc[table].reshape(B, -1, Hkv, D).permute(0, 2, 1, 3).float()
    v = vc[table].reshape(B, -1, Hkv, D).permute(0, 2, 1, 3).float()
    seen = (torch.arange(k.shape[2], device=k.device) <= lengths[:, None])[:, None, None]    # [B, 1, 1, n]
    q = s["q"].float().reshape(B, Hkv, H // Hkv, D)
    x = (q @ k.transpose(-1, -2)) * D ** -0.5
    top = x.masked_fill(~seen, -math.inf).amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.where(seen, torch.exp(x - top), 0.0)
    out = (p @ v) / p.sum(-1, keepdim=True).clamp(min=1e-30)
    return out.reshape(B, H, D).to(s["q"].dtype), kc, vc


_PLAIN = {"la_forward": _plain_forward, "la_backward": _plain_backward, "la_decode": _plain_decode,
          "paged": _plain_paged}


# ------------------------------------------------------------------------------- the library's calls
def _own(s):
    import gated_delta_rule_109_b200 as kda

    op = s["case"]["op"]
    if op == "la_forward":
        return kda.la_forward(s["q"], s["k"], s["v"], s["log_decay"], s["state"])
    if op == "la_backward":
        return kda.la_backward(s["q"], s["k"], s["v"], s["log_decay"], s["grad_out"], s["state"], s["grad_state"])
    if op == "la_decode":
        return kda.la_decode_step(s["q"], s["k"], s["v"], s["log_decay"], s["state"]), s["state"]
    if "out" not in s:
        s["out"] = torch.zeros_like(s["q"])             # an idle row of the batch keeps what its output holds
    out = kda.paged_decode_step(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["block_table"], s["lengths"],
                                out=s["out"])
    return out, s["k_cache"], s["v_cache"]


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------------------- the work of one pass
def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "paged":
        B, H, Hkv, D = case["B"], case["H"], case["Hkv"], case["D"]
        # lengths are drawn evenly between the shortest and the longest; the first row has the longest
        mean = (max(case["shortest"], 0) + case["longest"]) / 2 + 1
        tokens = (B - 1) * mean + case["longest"] + 1
        return {"bytes": tokens * Hkv * D * 2 * e + 2 * B * H * D * e + 2 * B * Hkv * D * e,
                "flops": tokens * H * D * 4}
    B, T, H, dk, dv = (case[n] for n in ("B", "T", "H", "dk", "dv"))
    n, state = B * T * H, B * H * dk * dv * 4
    if case["op"] == "la_backward":
        carried = 2 if case["state"] else 0              # the state before, its gradient behind; one gradient written
        return {"bytes": n * (4 * dk + 3 * dv) * e + state * (carried + 1), "flops": n * dk * dv * 10}
    return {"bytes": n * (2 * dk + 2 * dv) * e + state * (2 if case["state"] else 1), "flops": n * dk * dv * 4}


# ------------------------------------------------------------------------------- the definitions in 64 bits
def _step(state, a, k, v):
    return state.mul_(a).addcmul_(k.unsqueeze(-1), v.unsqueeze(-2))


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "paged":
        page, group = case["page"], case["H"] // case["Hkv"]
        kc, vc, out = s["k_cache"], s["v_cache"], torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
        rows = s["lengths"].tolist()
        for b, n in enumerate(rows):
            if n >= 0:
                at = s["block_table"][b, n // page]
                kc[at, n % page], vc[at, n % page] = s["k"][b], s["v"][b]
        for b, n in enumerate(rows):
            if n < 0:
                continue
            pages = s["block_table"][b, : n // page + 1].long()
            for h in range(case["Hkv"]):
                k, v = (c[pages, :, h].reshape(-1, case["D"])[: n + 1].double() for c in (kc, vc))
                x = s["q"][b, h * group:(h + 1) * group].double() @ k.T / math.sqrt(case["D"])
                out[b, h * group:(h + 1) * group] = torch.softmax(x, -1) @ v
        return out, kc, vc
    B, T, H, dk, dv = (case[n] for n in ("B", "T", "H", "dk", "dv"))
    q, k, v = (s[n] for n in ("q", "k", "v"))
    scale, dev = 1.0 / math.sqrt(dk), q.device
    a = 1.0 if s["log_decay"] is None else torch.exp(s["log_decay"].double())[:, None, None]
    S = torch.zeros((B, H, dk, dv), dtype=torch.float64, device=dev) if s["state"] is None else s["state"].double()
    if case["op"] == "la_decode":
        S = _step(S, a, k.double(), v.double())
        return (q.double().unsqueeze(-2) @ S).squeeze(-2) * scale, S
    if case["op"] == "la_forward":
        out = torch.empty(v.shape, dtype=torch.float64, device=dev)
        for t in range(T):
            _step(S, a, k[:, t].double(), v[:, t].double())
            out[:, t] = (q[:, t].double().unsqueeze(-2) @ S).squeeze(-2) * scale
        return out, S
    do = s["grad_out"]
    dq, dkk, dvv = (torch.empty(x.shape, dtype=torch.float64, device=dev) for x in (q, k, v))
    for t in range(T):
        _step(S, a, k[:, t].double(), v[:, t].double())
        dq[:, t] = (S @ do[:, t].double().unsqueeze(-1)).squeeze(-1) * scale
    D = torch.zeros((B, H, dk, dv), dtype=torch.float64, device=dev)
    if s["grad_state"] is not None:
        D += s["grad_state"].double()
    for t in range(T - 1, -1, -1):
        D.addcmul_(q[:, t].double().unsqueeze(-1) * scale, do[:, t].double().unsqueeze(-2))
        dkk[:, t] = (D @ v[:, t].double().unsqueeze(-1)).squeeze(-1)
        dvv[:, t] = (k[:, t].double().unsqueeze(-2) @ D).squeeze(-2)
        D.mul_(a)
    return dict(dq=dq, dk=dkk, dv=dvv, dinitial_state=D)
