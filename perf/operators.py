"""Cases of the operators around the exact attention: rotary positions with several axes (applied
to whole sequences, undone for gradients, or written into a paged KV cache as tokens arrive) and
cross attention to an encoder's states (prefill, single token, training step).

Layouts are the library's: q [B, Hq, Nq, d], k and v [B, Hkv, Nk, d] with Hq a multiple of Hkv
(query head h reads key head h // (Hq // Hkv)), bf16, contiguous.
"""

import math

import torch

own = False

# Pairs of each axis at d = 128 and d = 64 (time, height, width, or height, width): the shares
# 1/4, 3/8, 3/8 of three axes and halves of two.
_SECTIONS = {(128, 3): (16, 24, 24), (64, 3): (8, 12, 12), (128, 2): (32, 32), (64, 2): (16, 16),
             (128, 1): (64,), (64, 1): (32,)}


def _rope(name, B, Hq, Hkv, N, d, axes, **more):
    c = {"name": name, "op": "rope", "B": B, "Hq": Hq, "Hkv": Hkv, "N": N, "d": d, "axes": axes, "base": 10000.0,
         "interleaved": False, "per_axis": False, "cyclic": False, "inverse": False}
    return {**c, **more}


def _paged(name, B, Hq, Hkv, T, d, axes, page, cache, **more):
    c = {"name": name, "op": "rope_paged", "B": B, "Hq": Hq, "Hkv": Hkv, "T": T, "d": d, "axes": axes, "page": page,
         "cache": cache, "base": 10000.0, "interleaved": False, "per_axis": False, "cyclic": False, "ragged": False}
    return {**c, **more}


def _cross(name, op, B, Hq, Hkv, Nq, Nk, d, lens="full"):
    return {"name": name, "op": op, "B": B, "Hq": Hq, "Hkv": Hkv, "Nq": Nq, "Nk": Nk, "d": d, "lens": lens}


def listed():
    return [
        # a video prompt of two sequences at the library's causal prefill size: q and k of one layer
        _rope("rope_video", 2, 16, 16, 8192, 128, 3),
        # the long ragged prompt with shared key heads; axes dealt out pair by pair, a larger base
        _rope("rope_ragged_shared", 1, 32, 8, 16381, 128, 3, cyclic=True, base=1000000.0),
        # an image encoder's training step: the gradients of q and k turned back; pairs side by side,
        # frequencies that start anew for each axis
        _rope("rope_image_grad", 4, 16, 16, 2048, 64, 2, interleaved=True, per_axis=True, inverse=True),
        # one new token of each of eight sequences into the paged cache (latency counts)
        _paged("paged_token", 8, 32, 32, 1, 128, 3, 64, 1000),
        # a chunk of a prompt into the paged cache, sequences of different new lengths
        _paged("paged_chunk", 4, 16, 16, 517, 64, 2, 128, 1500, ragged=True),
        # one token attends an image's states, shared key heads (latency counts)
        _cross("cross_token", "cross", 8, 32, 8, 1, 577, 128),
        # one token attends long encoder states of different lengths
        _cross("cross_token_long", "cross", 8, 32, 8, 1, 32768, 128, "ragged"),
        # decoder prompts against padded audio states at the library's prefill size
        _cross("cross_prefill", "cross", 4, 16, 16, 2048, 1500, 64, "ragged"),
        # long decoder prompts against long states
        _cross("cross_long", "cross", 2, 16, 16, 8192, 4096, 128),
        # small odd sizes, shared key heads, one sequence without an encoder's state
        _cross("cross_odd", "cross", 3, 12, 4, 333, 641, 64, "empty"),
        # training steps: forward and backward, whole and padded with shared key heads
        _cross("train_long", "cross_train", 2, 16, 16, 4096, 2048, 128),
        _cross("train_shared", "cross_train", 4, 16, 4, 2048, 1500, 64, "ragged"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    top = max(_cost(work(c)) for c in listed())
    while True:
        d, hkv, group = rng.choice((64, 128)), rng.choice((1, 2, 3, 4, 8, 16)), rng.choice((1, 1, 2, 4, 8))
        batch = rng.choice((1, 2, 3, 4, 8))
        op = rng.choice(("rope", "rope_paged", "cross", "cross", "cross_train"))
        flags = {"interleaved": rng.random() < 0.4, "per_axis": rng.random() < 0.4, "cyclic": rng.random() < 0.4,
                 "base": rng.choice((10000.0, 500000.0, 1000000.0))}
        if op == "rope":
            c = _rope("", batch, hkv * group, hkv, _log(rng, 1, 16384), d, rng.choice((1, 2, 3)),
                      inverse=rng.random() < 0.5, **flags)
        elif op == "rope_paged":
            c = _paged("", batch, hkv * group, hkv, rng.choice((1, _log(rng, 2, 2048))), d, rng.choice((1, 2, 3)),
                       rng.choice((64, 128, 192)), _log(rng, 64, 4096), ragged=rng.random() < 0.5, **flags)
        else:
            one = op == "cross" and rng.random() < 0.4
            # (a training step on one key alone has no gradient of q or k to speak of)
            c = _cross("", op, batch, hkv * group, hkv, 1 if one else _log(rng, 2, 8192),
                       _log(rng, 2 if op == "cross_train" else 1, 32768 if one else 4096), d,
                       rng.choice(("full", "ragged", "empty" if batch > 1 else "full")))
        del c["name"]
        if _cost(work(c)) <= top:
            return c


def _cost(w):
    return max(w["bytes"], w["flops"] / 50)


def _lens(case):
    """Keys of each sequence: all of them, spread over the upper half, or so with the last one empty."""
    B, Nk = case["B"], case["Nk"]
    if case["lens"] == "full":
        return [Nk] * B
    lens = [max(1, Nk - (b * Nk) // (2 * B)) for b in range(B)]
    if case["lens"] == "empty":
        lens[-1] = 0
    return lens


def _new(case):
    """New tokens of each sequence of a paged case."""
    B, T = case["B"], case["T"]
    return [max(1, T - (b * T) // (2 * B)) for b in range(B)] if case["ragged"] else [T] * B


def work(case):
    d, B, Hq, Hkv = case["d"], case["B"], case["Hq"], case["Hkv"]
    if case["op"] == "rope":
        rows = B * (Hq + Hkv) * case["N"]
        return {"bytes": rows * d * 4 + case["axes"] * B * case["N"] * 4, "flops": rows * d * 3}
    if case["op"] == "rope_paged":
        rows = sum(_new(case))
        return {"bytes": rows * ((Hq + 2 * Hkv) * d * 4 + case["axes"] * 4), "flops": rows * (Hq + Hkv) * d * 3}
    Nq, keys = case["Nq"], sum(_lens(case))
    q, kv, lse = B * Hq * Nq * d * 2, 2 * Hkv * keys * d * 2, B * Hq * Nq * 4
    pairs = Hq * Nq * keys
    if case["op"] == "cross":
        return {"bytes": 2 * q + kv + lse, "flops": 4 * pairs * d}
    # training: q, k, v, dout read; o, lse, dq, dk, dv written (dk and dv of padded keys too)
    return {"bytes": 4 * q + kv + lse + 2 * B * Hkv * case["Nk"] * d * 2, "flops": 14 * pairs * d}


def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(torch.bfloat16)


def _positions(gen, axes, B, N, start=0):
    """int32 [axes, B, N]: text positions, or frames of rows and columns behind a prompt of another length each."""
    n = torch.arange(N, device="cuda", dtype=torch.int64)
    first = torch.randint(0, 4096, (B, 1), generator=gen, device="cuda") + start
    wide = torch.randint(24, 49, (B, 1), generator=gen, device="cuda")
    t, h, w = n // (wide * wide), (n // wide) % wide, n % wide
    return torch.stack([first + x for x in ((n + 0 * wide,), (h, w), (t, h, w))[axes - 1]]).to(torch.int32).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    B, Hq, Hkv, d = case["B"], case["Hq"], case["Hkv"], case["d"]
    s = {"case": case}
    if case["op"] == "rope":
        N = case["N"]
        s["q"], s["k"] = _normal(gen, B, Hq, N, d), _normal(gen, B, Hkv, N, d)
        s["pos"] = _positions(gen, case["axes"], B, N)
        s["q_out"], s["k_out"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
    elif case["op"] == "rope_paged":
        T, page = case["T"], case["page"]
        pages = -(-(case["cache"] + T) // page)
        s["q"], s["k"], s["v"] = _normal(gen, B, Hq, T, d), _normal(gen, B, Hkv, T, d), _normal(gen, B, Hkv, T, d)
        s["pos"] = _positions(gen, case["axes"], B, T, case["cache"])
        s["q_out"] = torch.zeros_like(s["q"])
        s["k_pages"], s["v_pages"] = _normal(gen, B * pages, Hkv, page, d), _normal(gen, B * pages, Hkv, page, d)
        s["table"] = torch.randperm(B * pages, generator=gen, device="cuda").to(torch.int32).view(B, pages)
        s["seq_lens"] = torch.randint(0, case["cache"] + 1, (B,), generator=gen, device="cuda").to(torch.int32)
        s["new_lens"] = torch.tensor(_new(case), dtype=torch.int32, device="cuda") if case["ragged"] else None
    else:
        Nq, Nk = case["Nq"], case["Nk"]
        s["q"], s["k"], s["v"] = _normal(gen, B, Hq, Nq, d), _normal(gen, B, Hkv, Nk, d), _normal(gen, B, Hkv, Nk, d)
        s["lens"] = None if case["lens"] == "full" else torch.tensor(_lens(case), dtype=torch.int32, device="cuda")
        s["o"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(B, Hq, Nq, dtype=torch.float32, device="cuda")
        if case["op"] == "cross_train":
            s["dout"] = _normal(gen, B, Hq, Nq, d)
            s["dq"], s["dk"], s["dv"] = torch.empty_like(s["q"]), torch.empty_like(s["k"]), torch.empty_like(s["v"])
    if own and "pos" in s:  # the plan of a model's rotation, made once
        from exact_attention_06_gb300 import fattn
        s["plan"] = fattn.fa_rope_axes_plan(d, _SECTIONS[d, case["axes"]], case["base"],
                                            interleaved=case["interleaved"], per_axis=case["per_axis"],
                                            cyclic=case["cyclic"])
    return s


def run(s):
    case = s["case"]
    if own:
        return _run_own(s, case)
    if case["op"] == "rope":
        cos, sin = _angles(s["pos"], case)
        if case["inverse"]:
            sin = -sin
        return [_turn(s["q"], cos, sin, case["interleaved"]), _turn(s["k"], cos, sin, case["interleaved"])]
    if case["op"] == "rope_paged":
        return _plain_paged(s, case)
    if case["op"] == "cross":
        return list(_attend(s, case)[:2])
    return _plain_train(s, case)


def _run_own(s, case):
    from exact_attention_06_gb300 import fattn
    if case["op"] == "rope":
        fattn.fa_rope_axes(s["q"], s["k"], s["pos"], s["plan"], s["q_out"], s["k_out"], inverse=case["inverse"])
        return [s["q_out"], s["k_out"]]
    if case["op"] == "rope_paged":
        fattn.fa_rope_axes_paged(s["q"], s["k"], s["v"], s["pos"], s["plan"], s["q_out"], s["k_pages"], s["v_pages"],
                                 s["table"], s["seq_lens"], s["new_lens"])
        return [s["q_out"], s["k_pages"], s["v_pages"]]
    scale = case["d"] ** -0.5
    fattn.fa_cross_fwd(s["q"], s["k"], s["v"], s["o"], s["lse"], scale, kv_lens=s["lens"])
    if case["op"] == "cross":
        return [s["o"], s["lse"]]
    fattn.fa_cross_bwd(s["q"], s["k"], s["v"], s["o"], s["dout"], s["lse"], s["dq"], s["dk"], s["dv"], scale,
                       kv_lens=s["lens"])
    return [s["o"], s["lse"], s["dq"], s["dk"], s["dv"]]


# ---------------------------------------------------------------- plain forms

def _axis_and_rate(case):
    """The axis and the angle per position of each pair of dimensions."""
    sections = _SECTIONS[case["d"], case["axes"]]
    n = case["d"] // 2
    axis = [a for a, s in enumerate(sections) for _ in range(s)]
    if case["cyclic"]:  # in turn, over the axes that have pairs left
        axis = [a for _, a in sorted((i, a) for a, s in enumerate(sections) for i in range(s))]
    within = [axis[:i].count(a) for i, a in enumerate(axis)]
    rate = [case["base"] ** -(within[i] / sections[a] if case["per_axis"] else i / n) for i, a in enumerate(axis)]
    return axis, rate


def _angles(pos, case):
    axis, rate = _axis_and_rate(case)
    axis = torch.tensor(axis, device=pos.device)
    rate = torch.tensor(rate, dtype=torch.float64, device=pos.device)
    angle = pos[axis].to(torch.float64).permute(1, 2, 0) * rate  # [B, N, d/2]; far positions need 64 bits
    return angle.cos().float().unsqueeze(1), angle.sin().float().unsqueeze(1)


def _turn(x, cos, sin, interleaved):
    d = x.shape[-1]
    f = x.float()
    if interleaved:
        a, b = f[..., 0::2], f[..., 1::2]
        return torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2).to(torch.bfloat16)
    a, b = f[..., : d // 2], f[..., d // 2:]
    return torch.cat((a * cos - b * sin, a * sin + b * cos), -1).to(torch.bfloat16)


def _plain_paged(s, case):
    B, T, page = case["B"], case["T"], case["page"]
    cos, sin = _angles(s["pos"], case)
    q, k = _turn(s["q"], cos, sin, case["interleaved"]), _turn(s["k"], cos, sin, case["interleaved"])
    t = torch.arange(T, device=q.device)
    key = s["seq_lens"].long()[:, None] + t
    at, row = s["table"].long().gather(1, key // page), key % page
    if s["new_lens"] is None:
        s["q_out"].copy_(q)
        k, v = k.transpose(1, 2), s["v"].transpose(1, 2)
    else:
        real = (t < s["new_lens"][:, None])
        s["q_out"].copy_(torch.where(real[:, None, :, None], q, s["q_out"]))
        keep = real[:, :, None, None]
        k = torch.where(keep, k.transpose(1, 2), s["k_pages"][at, :, row])
        v = torch.where(keep, s["v"].transpose(1, 2), s["v_pages"][at, :, row])
    s["k_pages"][at, :, row] = k
    s["v_pages"][at, :, row] = v
    return [s["q_out"], s["k_pages"], s["v_pages"]]


def _attend(s, case):
    """o, lse, and what a backward pass needs: the probabilities and the 32-bit operands."""
    B, Hq, Hkv, Nq, Nk, d = (case[x] for x in ("B", "Hq", "Hkv", "Nq", "Nk", "d"))
    q = s["q"].float().view(B, Hkv, -1, d)  # the query heads of a key head, one under another
    k, v = s["k"].float(), s["v"].float()
    score = torch.matmul(q, k.transpose(-1, -2)) * d ** -0.5
    if s["lens"] is not None:
        real = torch.arange(Nk, device=q.device) < s["lens"][:, None]
        score = torch.where(real[:, None, None], score, -math.inf)
        k, v = (torch.where(real[:, None, :, None], x, 0.0) for x in (k, v))
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    lse = (top + total.log()).view(B, Hq, Nq)
    p = p / torch.where(total == 0, 1.0, total)
    o = torch.matmul(p, v)
    return o.to(torch.bfloat16).view(B, Hq, Nq, d), lse, o, p, q, k, v


def _plain_train(s, case):
    o16, lse, o, p, q, k, v = _attend(s, case)
    scale = case["d"] ** -0.5
    g = s["dout"].float().view_as(o)
    dv = torch.matmul(p.transpose(-1, -2), g)
    ds = p * (torch.matmul(g, v.transpose(-1, -2)) - (o * g).sum(-1, keepdim=True)) * scale
    dq, dk = torch.matmul(ds, k).view(s["q"].shape), torch.matmul(ds.transpose(-1, -2), q)
    return [o16, lse, dq.to(torch.bfloat16), dk.to(torch.bfloat16), dv.to(torch.bfloat16)]


# ---------------------------------------------------------------- 64 bits, from the definitions

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return [_exact_turn(s[x], s["pos"], case, case["inverse"]) for x in ("q", "k")]
    if case["op"] == "rope_paged":
        q, k = _exact_turn(s["q"], s["pos"], case, False), _exact_turn(s["k"], s["pos"], case, False)
        out = [s["q_out"].double(), s["k_pages"].double(), s["v_pages"].double()]
        for b, (first, n) in enumerate(zip(s["seq_lens"].tolist(), _new(case))):
            key = torch.arange(first, first + n, device="cuda")
            at, row = s["table"][b].long()[key // case["page"]], key % case["page"]
            out[0][b, :, :n] = q[b, :, :n]
            out[1][at, :, row] = k[b, :, :n].transpose(0, 1)
            out[2][at, :, row] = s["v"][b, :, :n].double().transpose(0, 1)
        return out
    return _exact_cross(s, case)


def _exact_turn(x, pos, case, back):
    """Pairs as complex numbers, turned by exp(i angle)."""
    n = case["d"] // 2
    axis, rate = _axis_and_rate(case)
    angle = torch.stack([pos[a].double() * r for a, r in zip(axis, rate)], -1)
    turn = torch.polar(torch.ones_like(angle), -angle if back else angle).unsqueeze(1)
    x = x.double()
    z = torch.view_as_complex(x.unflatten(-1, (n, 2)) if case["interleaved"] else
                              x.unflatten(-1, (2, n)).transpose(-1, -2).contiguous())
    y = torch.view_as_real(z * turn)
    return (y if case["interleaved"] else y.transpose(-1, -2)).flatten(-2).contiguous()


def _exact_cross(s, case):
    """Softmax and its derivatives by autograd in 64 bits, a sequence and a key head at a time."""
    B, Hq, Hkv, Nq, d = (case[x] for x in ("B", "Hq", "Hkv", "Nq", "d"))
    train, G = case["op"] == "cross_train", Hq // Hkv
    out = {"o": torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda"),
           "lse": torch.full((B, Hq, Nq), -math.inf, dtype=torch.float64, device="cuda")}
    if train:
        out.update({g: torch.zeros(s[x].shape, dtype=torch.float64, device="cuda")
                    for g, x in (("dq", "q"), ("dk", "k"), ("dv", "v"))})
    for b, n in enumerate(_lens(case)):
        for j in range(Hkv if n else 0):
            heads = slice(j * G, (j + 1) * G)
            q, k, v = (x.detach().double().requires_grad_(train)
                       for x in (s["q"][b, heads], s["k"][b, j, :n], s["v"][b, j, :n]))
            score = torch.einsum("gqc,kc->gqk", q, k) / math.sqrt(d)
            o = torch.einsum("gqk,kc->gqc", torch.softmax(score, -1), v)
            out["o"][b, heads], out["lse"][b, heads] = o.detach(), torch.logsumexp(score, -1).detach()
            if train:
                grads = torch.autograd.grad(o, (q, k, v), s["dout"][b, heads].double())
                out["dq"][b, heads], out["dk"][b, j, :n], out["dv"][b, j, :n] = grads
    return list(out.values())
