"""Cases of the operators of a model whose layers attend to a sliding window: the attention itself (prompts,
training steps, single tokens over the paged cache), the norms of queries and keys for each head with the rotary
position in the same pass (prompts, training steps, new tokens written into the paged cache), and the pages of
that cache (block tables and slot maps from the requests' lengths).

Layouts are the library's: q [B, Hq, N, d], k and v [B, Hkv, Nk, d] with Hq a multiple of Hkv (query head h reads
key head h // (Hq // Hkv)), pools [pages, Hkv, page_size, d], bf16, contiguous.  Query i stands at position
Nk - N + i and sees the `window` keys up to its own and the first `sinks` keys.
"""

import math

import torch

own = False

# Pairs of each axis at d = 128 and d = 64 (text; height and width; time, height and width).
_SECTIONS = {(128, 1): (64,), (64, 1): (32,), (128, 2): (32, 32), (64, 2): (16, 16),
             (128, 3): (16, 24, 24), (64, 3): (8, 12, 12)}
_EPS = 1e-6


def _window(name, op, B, Hq, Hkv, N, Nk, d, window, sinks):
    return {"name": name, "op": op, "B": B, "Hq": Hq, "Hkv": Hkv, "N": N, "Nk": Nk, "d": d, "window": window,
            "sinks": sinks}


def _decode(name, B, Hq, Hkv, d, page, cache, window, sinks, **more):
    c = {"name": name, "op": "window_decode", "B": B, "Hq": Hq, "Hkv": Hkv, "d": d, "page": page, "cache": cache,
         "window": window, "sinks": sinks, "empty": False}
    return {**c, **more}


def _norm(name, op, B, Hq, Hkv, N, d, axes, **more):
    c = {"name": name, "op": op, "B": B, "Hq": Hq, "Hkv": Hkv, "N": N, "d": d, "axes": axes, "interleaved": False,
         "wide_weights": False}
    return {**c, **more}


def _norm_paged(name, B, Hq, Hkv, N, d, axes, page, cache, **more):
    return _norm(name, "norm_rope_paged", B, Hq, Hkv, N, d, axes, page=page, cache=cache, **{"ragged": False, **more})


def _pages(name, B, N, page, cache, **more):
    return {"name": name, "op": "pages", "B": B, "N": N, "page": page, "cache": cache, "ragged": True, **more}


def listed():
    return [
        # the library's long ragged prompt with shared key heads, a wide window and a few sinks
        _window("window_long", "window", 1, 32, 8, 16381, 16381, 128, 4096, 4),
        # a chunk of a prompt behind 1500 earlier keys, a narrow window of odd width
        _window("window_chunk", "window", 4, 16, 4, 517, 2017, 64, 333, 0),
        # a training step at the library's causal size, shared key heads
        _window("window_train", "window_train", 2, 16, 4, 8192, 8192, 128, 1024, 4),
        # a training step of short sequences and a narrow window
        _window("window_train_narrow", "window_train", 4, 16, 16, 2048, 2048, 64, 256, 16),
        # one token of each of eight sequences (latency counts)
        _decode("decode_token", 8, 32, 8, 128, 64, 1000, 512, 4),
        # one token of many long sequences
        _decode("decode_long", 32, 32, 8, 128, 128, 32768, 8192, 16),
        # the long ragged prompt's queries and keys, normed and turned
        _norm("norm_rope_prompt", "norm_rope", 1, 32, 8, 16381, 128, 1),
        # a training step over video positions: forward and gradients, of the weights too
        _norm("norm_rope_train", "norm_rope_train", 2, 16, 4, 8192, 128, 3, wide_weights=True),
        # one new token of each of eight sequences into the paged cache (latency counts)
        _norm_paged("norm_paged_token", 8, 32, 8, 1, 128, 1, 64, 1000),
        # a chunk of a prompt into the paged cache, sequences of different new lengths
        _norm_paged("norm_paged_chunk", 4, 16, 16, 517, 64, 2, 128, 1500, ragged=True, interleaved=True),
        # rejected draft tokens of a serving step taken back, new ones placed (latency counts)
        _pages("pages_drafts", 64, 5, 64, 8000),
        # the pages of finished requests taken back, those of new prompts placed
        _pages("pages_prompts", 32, 16381, 128, 0, ragged=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    tops = [work(c) for c in listed()]
    most = {x: max(w[x] for w in tops) for x in ("bytes", "flops")}
    while True:
        d, hkv, group = rng.choice((64, 128)), rng.choice((1, 2, 3, 4, 8, 16)), rng.choice((1, 1, 2, 4, 5, 8))
        batch = rng.choice((1, 2, 3, 4, 8))
        op = rng.choice(("window", "window", "window_train", "window_decode", "window_decode", "norm_rope",
                         "norm_rope_train", "norm_rope_paged", "pages"))
        sinks, window = rng.choice((0, 0, 1, 4, 16, 100, 128)), _log(rng, 1, 8192)
        more = {"interleaved": rng.random() < 0.4, "wide_weights": rng.random() < 0.5}
        if op in ("window", "window_train"):
            n = _log(rng, 2, 16384)
            if op == "window_train":  # (a softmax of one key alone has no gradient of q or k to speak of)
                window = max(window, 2)
            c = _window("", op, batch, hkv * group, hkv, n, n + rng.choice((0, 0, _log(rng, 1, 8192))), d, window, sinks)
        elif op == "window_decode":
            batch = rng.choice((1, 3, 8, 32))
            c = _decode("", batch, hkv * group, hkv, d, rng.choice((64, 128, 192)), _log(rng, 1, 32768), window, sinks,
                        empty=batch > 1 and rng.random() < 0.3)
        elif op == "norm_rope_paged":
            c = _norm_paged("", batch, hkv * group, hkv, rng.choice((1, _log(rng, 2, 2048))), d, rng.choice((1, 2, 3)),
                            rng.choice((64, 128, 192)), _log(rng, 64, 4096), ragged=rng.random() < 0.5, **more)
        elif op == "pages":
            batch = _log(rng, 1, 512)
            c = _pages("", batch, rng.choice((1, _log(rng, 2, min(16384, 2**20 // batch)))), rng.choice((64, 128, 192)),
                       _log(rng, 1, 32768), ragged=rng.random() < 0.5)
        else:
            c = _norm("", op, batch, hkv * group, hkv, _log(rng, 1, 16384), d, rng.choice((1, 2, 3)), **more)
        del c["name"]
        w = work(c)
        if w["bytes"] <= most["bytes"] and w["flops"] <= most["flops"]:
            return c


def _seen(case):
    """Keys that the queries of a head see, added up, and keys that any of them sees."""
    N, Nk, W, S = case["N"], case["Nk"], case["window"], case["sinks"]
    pairs = sum(min(n, W) + min(S, max(n - W, 0)) for n in range(Nk - N + 1, Nk + 1))  # n keys up to its own
    first = max(0, Nk - N + 1 - W)
    return pairs, Nk - first + min(S, first)


def _cache_lens(case):
    """Lengths of a paged case's sequences: from half of the cache to all of it, perhaps one of none."""
    B, L = case["B"], case["cache"]
    lens = [max(min(1, L), L - (b * L) // (2 * B)) for b in range(B)]
    if case.get("empty"):
        lens[-1] = 0
    return lens


def _new(case):
    """New tokens of each sequence of a paged case."""
    B, N = case["B"], case["N"]
    return [max(1, N - (b * N) // (2 * B)) for b in range(B)] if case["ragged"] else [N] * B


def work(case):
    B = case["B"]
    if case["op"] == "pages":
        tokens, page = sum(_new(case)), case["page"]
        moved = sum(-(-(n + m) // page) - -(-n // page) for n, m in zip(_cache_lens(case), _new(case)))
        # lengths read and written by both calls, pages read and written by both, slots written
        return {"bytes": B * 4 * 8 + moved * 4 * 5 + B * case["N"] * 8, "flops": 2 * moved + tokens}
    d, Hq, Hkv = case["d"], case["Hq"], case["Hkv"]
    if case["op"] == "window_decode":
        keys = sum(min(n, case["window"]) + min(case["sinks"], max(n - case["window"], 0)) for n in _cache_lens(case))
        return {"bytes": B * Hq * (4 * d + 4) + 4 * Hkv * keys * d, "flops": 4 * Hq * keys * d}
    if case["op"] in ("window", "window_train"):
        pairs, keys = _seen(case)
        q, kv, lse = B * Hq * case["N"] * d * 2, 2 * B * Hkv * keys * d * 2, B * Hq * case["N"] * 4
        if case["op"] == "window":
            return {"bytes": 2 * q + kv + lse, "flops": 4 * B * Hq * pairs * d}
        # q, k, v, dout read; o, lse, dq, dk, dv written (dk and dv of keys that no query sees too)
        return {"bytes": 4 * q + kv + lse + 2 * B * Hkv * case["Nk"] * d * 2, "flops": 14 * B * Hq * pairs * d}
    if case["op"] == "norm_rope_paged":
        rows = sum(_new(case))
        return {"bytes": rows * ((Hq + 2 * Hkv) * d * 4 + case["axes"] * 4 + 8), "flops": rows * (Hq + Hkv) * d * 7}
    rows = B * (Hq + Hkv) * case["N"]
    if case["op"] == "norm_rope":
        return {"bytes": rows * d * 4 + case["axes"] * B * case["N"] * 4, "flops": rows * d * 7}
    # training: q, k and the gradients coming in read; both outputs and both gradients written
    return {"bytes": rows * d * 8 + case["axes"] * B * case["N"] * 4, "flops": rows * d * 20}


# ---------------------------------------------------------------- inputs

def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(torch.bfloat16)


def _positions(gen, axes, B, N, start=0):
    """int32 [axes, B, N]: text positions, or frames of rows and columns behind a prompt of another length each."""
    n = torch.arange(N, device="cuda", dtype=torch.int64)
    first = torch.randint(0, 4096, (B, 1), generator=gen, device="cuda") + start
    wide = torch.randint(24, 49, (B, 1), generator=gen, device="cuda")
    t, h, w = n // (wide * wide), (n // wide) % wide, n % wide
    return torch.stack([first + x for x in ((n + 0 * wide,), (h, w), (t, h, w))[axes - 1]]).to(torch.int32).contiguous()


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": case}
    if case["op"] == "pages":
        _prepare_pages(s, case, gen)
        return s
    B, Hq, Hkv, d = case["B"], case["Hq"], case["Hkv"], case["d"]
    if case["op"] == "window_decode":
        page, lens = case["page"], _cache_lens(case)
        pages = -(-case["cache"] // page)
        s["q"] = _normal(gen, B, Hq, d)
        s["k_pages"], s["v_pages"] = _normal(gen, B * pages, Hkv, page, d), _normal(gen, B * pages, Hkv, page, d)
        s["table"] = torch.randperm(B * pages, generator=gen, device="cuda").to(torch.int32).view(B, pages)
        order = torch.randperm(B, generator=gen, device="cuda")
        s["lens"] = _ints(lens)[order]
        s["o"], s["lse"] = torch.empty_like(s["q"]), torch.empty(B, Hq, dtype=torch.float32, device="cuda")
        return s
    if case["op"] in ("window", "window_train"):
        N, Nk = case["N"], case["Nk"]
        s["q"], s["k"], s["v"] = _normal(gen, B, Hq, N, d), _normal(gen, B, Hkv, Nk, d), _normal(gen, B, Hkv, Nk, d)
        s["o"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(B, Hq, N, dtype=torch.float32, device="cuda")
        if case["op"] == "window_train":
            s["dout"] = _normal(gen, B, Hq, N, d)
            s["dq"], s["dk"], s["dv"] = torch.empty_like(s["q"]), torch.empty_like(s["k"]), torch.empty_like(s["v"])
        return s
    N = case["N"]
    # queries and keys as a projection leaves them (heads of different sizes), weights around 1
    size = torch.exp(torch.randn(Hq + Hkv, 1, 1, generator=gen, device="cuda"))
    s["q"] = (size[:Hq] * torch.randn(B, Hq, N, d, generator=gen, device="cuda")).to(torch.bfloat16)
    s["k"] = (size[Hq:] * torch.randn(B, Hkv, N, d, generator=gen, device="cuda")).to(torch.bfloat16)
    for x in ("q_weight", "k_weight"):
        w = 1 + 0.2 * torch.randn(d, generator=gen, device="cuda")
        s[x] = w if case["wide_weights"] else w.to(torch.bfloat16)
    s["pos"] = _positions(gen, case["axes"], B, N, case.get("cache", 0))
    s["q_out"] = torch.zeros_like(s["q"])
    if case["op"] == "norm_rope_paged":
        page, lens = case["page"], _cache_lens(case)
        pages = -(-(case["cache"] + N) // page)
        s["v"] = _normal(gen, B, Hkv, N, d)
        s["k_pages"], s["v_pages"] = _normal(gen, B * pages, Hkv, page, d), _normal(gen, B * pages, Hkv, page, d)
        table = torch.randperm(B * pages, generator=gen, device="cuda").view(B, pages)
        key = _ints(lens).long()[:, None] + torch.arange(N, device="cuda")
        s["new_lens"] = _ints(_new(case)) if case["ragged"] else None
        s["slots"] = table.gather(1, key // page) * page + key % page
        if case["ragged"]:
            s["slots"] = torch.where(torch.arange(N, device="cuda") < s["new_lens"][:, None], s["slots"], -1)
    else:
        s["k_out"] = torch.empty_like(s["k"])
        if case["op"] == "norm_rope_train":
            s["dq_out"], s["dk_out"] = _normal(gen, B, Hq, N, d), _normal(gen, B, Hkv, N, d)
            s["dq"], s["dk"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
            s["dq_weight"], s["dk_weight"] = (torch.empty(d, device="cuda") for _ in range(2))
    if own:  # the plan of a model's rotation, made once
        from exact_attention_06_gb300 import fattn
        s["plan"] = fattn.fa_rope_axes_plan(d, _SECTIONS[d, case["axes"]], interleaved=case["interleaved"])
    return s


def _prepare_pages(s, case, gen):
    """Sequences with their new tokens in place; the pages that no table names are on the stack of free ones."""
    B, N, page, new = case["B"], case["N"], case["page"], _new(case)
    lens = [n + m for n, m in zip(_cache_lens(case), new)]
    max_pages = -(-(case["cache"] + N) // page)
    used = -(-_ints(lens).long() // page)
    num_pages = B * max_pages + 16
    ids = torch.randperm(num_pages, generator=gen, device="cuda").to(torch.int32)
    row = torch.arange(max_pages, device="cuda")
    taken, first = used[:, None] > row, torch.cumsum(used, 0) - used
    s["table"] = torch.where(taken, ids[(first[:, None] + row) % num_pages], -1).to(torch.int32)
    total = int(sum(-(-n // page) for n in lens))
    s["free_pages"] = torch.full((num_pages,), -1, dtype=torch.int32, device="cuda")
    s["free_pages"][:num_pages - total] = ids[total:]
    s["n_free"] = _ints([num_pages - total])
    s["lens"] = _ints(lens)
    order = torch.randperm(B, generator=gen, device="cuda")
    s["table"], s["lens"] = s["table"][order].contiguous(), s["lens"][order]
    s["more"] = _ints(new)[order]
    s["less"] = -s["more"]
    s["granted"] = torch.empty_like(s["lens"])
    s["slots"] = torch.empty(B, N, dtype=torch.int64, device="cuda")


def run(s):
    case = s["case"]
    if own:
        return _run_own(s, case)
    if case["op"] == "pages":
        _plain_extend(s, case, s["less"])
        s["slots"] = _plain_extend(s, case, s["more"])
        return [s[x] for x in ("table", "lens", "free_pages", "n_free", "granted", "slots")]
    if case["op"] == "window_decode":
        return _plain_decode(s, case)
    if case["op"] in ("window", "window_train"):
        return _plain_window(s, case)
    return _plain_norm(s, case)


def _run_own(s, case):
    from exact_attention_06_gb300 import fattn
    if case["op"] == "pages":
        fattn.fa_pages_extend(s["table"], s["lens"], s["less"], s["free_pages"], s["n_free"], s["granted"], None,
                              case["page"])
        fattn.fa_pages_extend(s["table"], s["lens"], s["more"], s["free_pages"], s["n_free"], s["granted"], s["slots"],
                              case["page"])
        return [s[x] for x in ("table", "lens", "free_pages", "n_free", "granted", "slots")]
    if case["op"] == "window_decode":
        fattn.fa_window_decode_paged(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"], s["o"], s["lse"],
                                     case["d"] ** -0.5, case["cache"], case["window"], case["sinks"])
        return [s["o"], s["lse"]]
    if case["op"] in ("window", "window_train"):
        args = case["d"] ** -0.5, case["window"], case["sinks"]
        fattn.fa_window_fwd(s["q"], s["k"], s["v"], s["o"], s["lse"], *args)
        if case["op"] == "window":
            return [s["o"], s["lse"]]
        fattn.fa_window_bwd(s["q"], s["k"], s["v"], s["o"], s["dout"], s["lse"], s["dq"], s["dk"], s["dv"], *args)
        return [s["o"], s["lse"], s["dq"], s["dk"], s["dv"]]
    weights = s["q_weight"], s["k_weight"], s["pos"], s["plan"]
    if case["op"] == "norm_rope_paged":
        fattn.fa_norm_rope_axes_paged(s["q"], s["k"], s["v"], *weights, s["q_out"], s["k_pages"], s["v_pages"], s["slots"],
                                      s["new_lens"], eps=_EPS)
        return [s["q_out"], s["k_pages"], s["v_pages"]]
    fattn.fa_norm_rope_axes(s["q"], s["k"], *weights, s["q_out"], s["k_out"], eps=_EPS)
    if case["op"] == "norm_rope":
        return [s["q_out"], s["k_out"]]
    fattn.fa_norm_rope_axes_bwd(s["q"], s["k"], *weights, s["dq_out"], s["dk_out"], s["dq"], s["dk"], s["dq_weight"],
                                s["dk_weight"], eps=_EPS)
    return [s[x] for x in ("q_out", "k_out", "dq", "dk", "dq_weight", "dk_weight")]


# ---------------------------------------------------------------- plain forms

def _plain_window(s, case):
    """A thousand queries at a time, against the keys that any of them sees."""
    B, Hq, Hkv, N, Nk, d, W, S = (case[x] for x in ("B", "Hq", "Hkv", "N", "Nk", "d", "window", "sinks"))
    train, scale, dev = case["op"] == "window_train", d ** -0.5, s["q"].device
    o, lse = torch.empty(s["q"].shape, device=dev), torch.empty(B, Hq, N, device=dev)
    if train:
        dq = torch.empty(s["q"].shape, device=dev)
        dk, dv = (torch.zeros(s["k"].shape, device=dev) for _ in range(2))
    for i in range(0, N, 1024):
        rows = slice(i, min(N, i + 1024))
        pos = torch.arange(Nk - N + i, Nk - N + rows.stop, device=dev)
        lo, hi = max(0, Nk - N + i - W + 1), Nk - N + rows.stop
        first = min(S, lo)
        key = torch.cat([torch.arange(first, device=dev), torch.arange(lo, hi, device=dev)])
        k, v = (torch.cat([s[x][:, :, :first], s[x][:, :, lo:hi]], 2).float() for x in ("k", "v"))
        seen = (key <= pos[:, None]) & ((key > pos[:, None] - W) | (key < S))
        seen = seen.repeat(Hq // Hkv, 1)
        part = (B, Hq, rows.stop - i)
        q = s["q"][:, :, rows].reshape(B, Hkv, -1, d).float()  # the query heads of a key head, one under another
        score = torch.where(seen, torch.matmul(q, k.transpose(-1, -2)) * scale, -math.inf)
        top = score.amax(-1, keepdim=True)
        p = torch.exp(score - top)
        total = p.sum(-1, keepdim=True)
        p = p / total
        out = torch.matmul(p, v)
        o[:, :, rows], lse[:, :, rows] = out.view(*part, d), (top + total.log()).view(part)
        if train:
            g = s["dout"][:, :, rows].reshape(B, Hkv, -1, d).float()
            ds = p * (torch.matmul(g, v.transpose(-1, -2)) - (out * g).sum(-1, keepdim=True)) * scale
            dq[:, :, rows] = torch.matmul(ds, k).view(*part, d)
            for grad, x in ((dk, torch.matmul(ds.transpose(-1, -2), q)), (dv, torch.matmul(p.transpose(-1, -2), g))):
                grad[:, :, :first] += x[:, :, :first]
                grad[:, :, lo:hi] += x[:, :, first:]
    out = [o.to(torch.bfloat16), lse]
    return out + [x.to(torch.bfloat16) for x in (dq, dk, dv)] if train else out


def _plain_decode(s, case):
    """The keys of each sequence's window and sinks gathered out of the pages."""
    B, Hq, Hkv, d, W, S, page = (case[x] for x in ("B", "Hq", "Hkv", "d", "window", "sinks", "page"))
    n = s["lens"].long()[:, None]
    first = torch.clamp(n - W, min=0)
    i = torch.arange(min(S, case["cache"]), device=n.device)
    j = first + torch.arange(min(W, case["cache"]), device=n.device)
    key = torch.cat([i.expand(B, -1), j], 1)
    seen = torch.cat([i < torch.minimum(first, n), j < n], 1)
    key = torch.where(seen, key, 0)
    at, row = s["table"].long().gather(1, key // page), key % page
    k, v = (s[x][at, :, row].transpose(1, 2).float() for x in ("k_pages", "v_pages"))  # [B, Hkv, keys, d]
    v = torch.where(seen[:, None, :, None], v, 0.0)
    score = torch.matmul(s["q"].float().view(B, Hkv, -1, d), k.transpose(-1, -2)) * d ** -0.5
    score = torch.where(seen[:, None, None], score, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p / torch.where(total == 0, 1.0, total), v)
    return [o.to(torch.bfloat16).view(B, Hq, d), (top + total.log()).view(B, Hq)]


def _axis_and_rate(case):
    """The axis and the angle per position of each pair of dimensions (base 10000)."""
    n = case["d"] // 2
    axis = [a for a, pairs in enumerate(_SECTIONS[case["d"], case["axes"]]) for _ in range(pairs)]
    return axis, [10000.0 ** -(i / n) for i in range(n)]


def _pairs(x, interleaved):
    n = x.shape[-1] // 2
    return (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :n], x[..., n:])


def _unpairs(a, b, interleaved):
    return torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)


def _plain_norm(s, case):
    axis, rate = _axis_and_rate(case)
    pos = s["pos"]
    angle = pos[torch.tensor(axis, device=pos.device)].double().permute(1, 2, 0)  # far positions need 64 bits
    angle = angle * torch.tensor(rate, dtype=torch.float64, device=pos.device)
    cos, sin = angle.cos().float().unsqueeze(1), angle.sin().float().unsqueeze(1)
    inter, out = case["interleaved"], {}
    for x in ("q", "k"):
        f, w = s[x].float(), s[x + "_weight"].float()
        r = torch.rsqrt((f * f).mean(-1, keepdim=True) + _EPS)
        a, b = _pairs(f * r * w, inter)
        out[x] = _unpairs(a * cos - b * sin, a * sin + b * cos, inter).to(torch.bfloat16)
        if case["op"] == "norm_rope_train":
            a, b = _pairs(s["d" + x + "_out"].float(), inter)
            g = _unpairs(a * cos + b * sin, b * cos - a * sin, inter)
            n, h = f * r, g * w
            out["d" + x] = (r * (h - n * (h * n).mean(-1, keepdim=True))).to(torch.bfloat16)
            out["d" + x + "_weight"] = (g * n).sum((0, 1, 2), dtype=torch.float64).float()
    if case["op"] == "norm_rope":
        return [out["q"], out["k"]]
    if case["op"] == "norm_rope_train":
        return [out[x] for x in ("q", "k", "dq", "dk", "dq_weight", "dk_weight")]
    b, t = torch.nonzero(s["slots"] >= 0, as_tuple=True) if case["ragged"] else (
        x.flatten() for x in torch.meshgrid(*(torch.arange(n, device=pos.device) for n in s["slots"].shape), indexing="ij"))
    slot = s["slots"][b, t]
    if case["ragged"]:
        real = torch.arange(case["N"], device=pos.device) < s["new_lens"][:, None]
        s["q_out"].copy_(torch.where(real[:, None, :, None], out["q"], s["q_out"]))
    else:
        s["q_out"].copy_(out["q"])
    s["k_pages"][slot // case["page"], :, slot % case["page"]] = out["k"][b, :, t]
    s["v_pages"][slot // case["page"], :, slot % case["page"]] = s["v"][b, :, t]
    return [s["q_out"], s["k_pages"], s["v_pages"]]


def _plain_extend(s, case, new):
    """Pages for new[b] more tokens of each sequence (fewer where negative), in place; the new tokens' slots."""
    page, stack, table = case["page"], s["free_pages"], s["table"].long()
    num, max_pages = stack.shape[0], table.shape[1]
    new, n, free = new.long(), s["lens"].long(), s["n_free"].long()
    had = (n + page - 1) // page
    want = (torch.clamp(n + new, min=0) + page - 1) // page
    take = torch.where(n + new <= max_pages * page, torch.clamp(want - had, min=0), 0)
    last = torch.cumsum(take, 0)
    ok = (n + new <= max_pages * page) & ((take == 0) | (last <= free))
    granted = torch.where((new > 0) & ~ok, 0, torch.maximum(new, -n))
    after = n + granted
    has = (after + page - 1) // page
    col = torch.arange(max_pages, device=n.device)
    more, less = (col >= had[:, None]) & (col < has[:, None]), (col >= has[:, None]) & (col < had[:, None])
    from_top = free - 1 - ((last - take)[:, None] + col - had[:, None])
    filled = torch.where(more, stack.long()[torch.clamp(from_top, 0, num - 1)], table)
    free = free - more.sum()
    back = torch.cumsum(had - torch.minimum(has, had), 0)
    to = free + back[-1] - 1 - ((back - (had - torch.minimum(has, had)))[:, None] + col - has[:, None])
    spare = torch.cat([stack, stack[:1]])  # one place more for what is not given back
    spare[torch.where(less, to, num).flatten()] = table.flatten().to(torch.int32)
    stack.copy_(spare[:num])
    s["table"].copy_(torch.where(less, -1, filled))
    s["lens"].copy_(after)
    s["n_free"].copy_(free + back[-1:])
    s["granted"].copy_(granted)
    t = torch.arange(case["N"], device=n.device)
    key = n[:, None] + t
    at = s["table"].long().gather(1, torch.clamp(key // page, max=max_pages - 1))
    return torch.where((t < granted[:, None]) & (at >= 0) & (at < num), at * page + key % page, -1)


# ---------------------------------------------------------------- 64 bits, from the definitions

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "pages":
        return _exact_pages(s, case)
    if case["op"] == "window_decode":
        return _exact_decode(s, case)
    if case["op"] in ("window", "window_train"):
        return _exact_window(s, case)
    return _exact_norm(s, case)


def _exact_window(s, case):
    """Softmax and its derivatives by autograd in 64 bits, a key head and some queries at a time."""
    B, Hq, Hkv, N, Nk, d, W, S = (case[x] for x in ("B", "Hq", "Hkv", "N", "Nk", "d", "window", "sinks"))
    train, G = case["op"] == "window_train", Hq // Hkv
    like = lambda x: torch.zeros(s[x].shape, dtype=torch.float64, device="cuda")  # noqa: E731
    out = {"o": like("q"), "lse": torch.zeros(B, Hq, N, dtype=torch.float64, device="cuda")}
    if train:
        out.update(dq=like("q"), dk=like("k"), dv=like("v"))
    for b in range(B):
        for j in range(Hkv):
            heads = slice(j * G, (j + 1) * G)
            for i in range(0, N, 2048):
                e = min(N, i + 2048)
                at = torch.arange(Nk - N + i, Nk - N + e, device="cuda")[:, None]
                key = torch.arange(Nk - N + e, device="cuda")
                hidden = (key > at) | ((at - key >= W) & (key >= S))
                some = torch.nonzero(~hidden.all(0))[:, 0]
                q, k, v = (x.detach().double().requires_grad_(train)
                           for x in (s["q"][b, heads, i:e], s["k"][b, j, some], s["v"][b, j, some]))
                score = torch.einsum("gqc,kc->gqk", q, k) / math.sqrt(d)
                score = score.masked_fill(hidden[:, some], -math.inf)
                o = torch.einsum("gqk,kc->gqc", torch.softmax(score, -1), v)
                out["o"][b, heads, i:e] = o.detach()
                out["lse"][b, heads, i:e] = torch.logsumexp(score, -1).detach()
                if train:
                    dq, dk, dv = torch.autograd.grad(o, (q, k, v), s["dout"][b, heads, i:e].double())
                    out["dq"][b, heads, i:e] = dq
                    out["dk"][b, j, some] += dk
                    out["dv"][b, j, some] += dv
    return list(out.values())


def _exact_decode(s, case):
    B, Hq, Hkv, d, page = (case[x] for x in ("B", "Hq", "Hkv", "d", "page"))
    o = torch.zeros(B, Hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["lens"].tolist()):
        if n == 0:
            continue
        key = torch.tensor([i for i in range(n) if i < case["sinks"] or n - i <= case["window"]], device="cuda")
        at = s["table"][b].long()[torch.div(key, page, rounding_mode="floor")]
        k, v = (s[x][at, :, key % page].double().permute(1, 0, 2) for x in ("k_pages", "v_pages"))
        q = s["q"][b].double().view(Hkv, -1, d)
        score = torch.einsum("hgc,hkc->hgk", q, k) / math.sqrt(d)
        o[b] = torch.einsum("hgk,hkc->hgc", torch.softmax(score, -1), v).reshape(Hq, d)
        lse[b] = torch.logsumexp(score, -1).flatten()
    return [o, lse]


def _exact_norm(s, case):
    """Pairs as complex numbers, turned by exp(i angle); gradients by autograd."""
    n, inter = case["d"] // 2, case["interleaved"]
    axis, rate = _axis_and_rate(case)
    angle = torch.stack([s["pos"][a].double() * r for a, r in zip(axis, rate)], -1)
    turn = torch.polar(torch.ones_like(angle), angle)
    out = {}
    for x in ("q", "k"):
        f = torch.zeros(s[x].shape, dtype=torch.float64, device="cuda")
        for b in range(case["B"]):  # (a sequence at a time)
            z = s[x][b].double().requires_grad_(True)
            w = s[x + "_weight"].double().requires_grad_(True)
            y = z / torch.sqrt(z.square().mean(-1, keepdim=True) + _EPS) * w
            c = torch.view_as_complex(y.unflatten(-1, (n, 2)).contiguous() if inter else
                                      y.unflatten(-1, (2, n)).transpose(-1, -2).contiguous())
            y = torch.view_as_real(c * turn[b])
            y = (y if inter else y.transpose(-1, -2)).flatten(-2)
            f[b] = y.detach()
            if case["op"] == "norm_rope_train":
                dz, dw = torch.autograd.grad(y, (z, w), s["d" + x + "_out"][b].double())
                out.setdefault("d" + x, []).append(dz)
                out["d" + x + "_weight"] = out.get("d" + x + "_weight", 0) + dw
        out[x] = f
    if case["op"] == "norm_rope":
        return [out["q"], out["k"]]
    if case["op"] == "norm_rope_train":
        out["dq"], out["dk"] = torch.stack(out["dq"]), torch.stack(out["dk"])
        return [out[x] for x in ("q", "k", "dq", "dk", "dq_weight", "dk_weight")]
    q, kp, vp = s["q_out"].double(), s["k_pages"].double(), s["v_pages"].double()
    for b, m in enumerate(_new(case)):
        slot = s["slots"][b, :m]
        at, row = torch.div(slot, case["page"], rounding_mode="floor"), slot % case["page"]
        q[b, :, :m] = out["q"][b, :, :m]
        kp[at, :, row] = out["k"][b, :, :m].transpose(0, 1)
        vp[at, :, row] = s["v"][b, :, :m].double().transpose(0, 1)
    return [q, kp, vp]


def _exact_pages(s, case):
    """The two calls on Python lists."""
    page, N = case["page"], case["N"]
    table, lens, stack, free = (s[x].tolist() for x in ("table", "lens", "free_pages", "n_free"))
    free = free[0]
    for new in (s["less"].tolist(), s["more"].tolist()):
        granted, slots, back = [], [[-1] * N for _ in lens], []
        for b, m in enumerate(new):
            had, want = -(-lens[b] // page), -(-(lens[b] + m) // page)
            for i in range(had, want):
                free -= 1
                table[b][i] = stack[free]
            for i in range(want, had):
                back.append(table[b][i])
                table[b][i] = -1
            for t in range(max(m, 0)):
                key = lens[b] + t
                slots[b][t] = table[b][key // page] * page + key % page
            granted.append(m)
            lens[b] += m
        for p in reversed(back):
            stack[free] = p
            free += 1
    ints = lambda x, t=torch.int32: torch.tensor(x, dtype=t, device="cuda")  # noqa: E731
    return [ints(table), ints(lens), ints(stack), ints([free]), ints(granted), ints(slots, torch.int64)]
