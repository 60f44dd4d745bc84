"""The serving operators over packed batches (sequences of different lengths, one after another): what is measured.

Three operators, each in a plain form of elementary torch operations in 32 bits (``own`` false) and as
the calls a user makes of the framework (``own`` true):

* ``packed``: attention over whole prompts, packed as [tokens, heads, D] with cumulative lengths;
* ``chunk``: the same for the newest tokens of each sequence over the paged cache that already holds them;
* ``append``: the rotation by position of the new tokens' q and k and the store of their k and v into the
  paged cache, for packed prompts and for one token of every sequence.

A case's lengths come from its own ``lens`` number, so that ``work`` knows them; the values, the
page order and the cache's contents come from the seed.
"""
import math

import numpy as np
import torch

own = False

_HEADS = ((12, 12), (32, 8), (16, 4), (8, 1), (8, 2), (12, 4), (6, 1), (16, 1))


def listed():
    return [
        # three short prompts of the GPT-2-small head shape: the smallest prefill call, where latency counts
        dict(name="packed_short_d64", op="packed", B=3, lo=5, hi=90, lens=1, Hq=12, Hkv=12, D=64, window=0, lse=False, pad=0),
        # a batch of GPT-2-small prompts of very different lengths (multi-head, D = 64)
        dict(name="packed_mha_d64", op="packed", B=8, lo=64, hi=1024, lens=2, Hq=12, Hkv=12, D=64, window=0, lse=False, pad=0),
        # a serving batch: many prompts of 1 to 1024 tokens, grouped heads, in a buffer padded for a captured graph
        dict(name="packed_gqa_batch", op="packed", B=32, lo=1, hi=1024, lens=3, Hq=32, Hkv=8, D=128, window=0, lse=False, pad=301),
        # a few long prompts, with the log-sum-exp that a later merge needs
        dict(name="packed_gqa_long", op="packed", B=4, lo=1024, hi=4096, lens=4, Hq=32, Hkv=8, D=128, window=0, lse=True, pad=0),
        # the largest: prompts of up to 8192 tokens with a sliding window
        dict(name="packed_gqa_window", op="packed", B=2, lo=5000, hi=8192, lens=5, Hq=32, Hkv=8, D=128, window=4096, lse=False, pad=0),
        # the smallest chunk call: two sequences, a few new tokens each
        dict(name="chunk_small_d64", op="chunk", B=2, lo=1, hi=9, lens=6, ctx=300, page=32, Hq=8, Hkv=2, D=64, window=0, lse=False, pad=0),
        # a continuous batch: chunks of 1 to 512 tokens over caches of up to 4096, page 16
        dict(name="chunk_gqa_mixed", op="chunk", B=8, lo=1, hi=512, lens=7, ctx=4096, page=16, Hq=32, Hkv=8, D=128, window=0, lse=False, pad=77),
        # long chunks over long caches
        dict(name="chunk_gqa_long", op="chunk", B=2, lo=1024, hi=2048, lens=8, ctx=8192, page=64, Hq=32, Hkv=8, D=128, window=0, lse=True, pad=0),
        # one decode step of 64 sequences
        dict(name="append_decode", op="append", B=64, lo=1, hi=1, lens=9, ctx=8192, page=16, Hq=32, Hkv=8, D=128, rot=128, interleaved=False, fp8=False, kout=False, pad=0),
        # the smallest: one token of three sequences, neighbouring pairs, an 8-bit cache
        dict(name="append_decode_small", op="append", B=3, lo=1, hi=1, lens=10, ctx=1000, page=16, Hq=12, Hkv=12, D=64, rot=64, interleaved=True, fp8=True, kout=False, pad=0),
        # packed prompts, a rotation of half of each head, an 8-bit cache, the rotated keys also kept for the prefill
        dict(name="append_prompts_fp8", op="append", B=16, lo=100, hi=512, lens=11, ctx=2048, page=64, Hq=32, Hkv=8, D=128, rot=64, interleaved=True, fp8=True, kout=True, pad=0),
        # a large packed batch of prompts into a 16-bit cache
        dict(name="append_prompts", op="append", B=24, lo=64, hi=2048, lens=12, ctx=4096, page=16, Hq=32, Hkv=8, D=128, rot=128, interleaved=False, fp8=False, kout=False, pad=55),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("packed", "packed", "chunk", "append"))
    Hq, Hkv = rng.choice(_HEADS)
    c = dict(op=op, lens=rng.randrange(1 << 30), Hq=Hq, Hkv=Hkv, D=rng.choice((64, 128)), pad=rng.choice((0, rng.randrange(1, 400))))
    if op == "append":
        c["D"] = rng.choice((64, 128, 128, 96, 256))
        decode = rng.random() < 0.4
        c["B"] = _log_int(rng, 1, 256 if decode else 24)
        # at most about the bytes of the largest listed append
        c["hi"] = 1 if decode else _log_int(rng, 2, max(2, min(2048, int(750e6 / (c["B"] * c["D"] * (4 * Hq + 9 * Hkv))))))
        c["lo"] = 1 if decode else rng.randrange(0, c["hi"] + 1)
        c["ctx"] = _log_int(rng, max(16, c["hi"]), 8192 if decode else 4096)
        c["page"] = rng.choice((16, 16, 32, 64, 128, 256))
        c["rot"] = rng.choice((c["D"], c["D"], c["D"] // 32 * 16))
        c["interleaved"], c["fp8"], c["kout"] = rng.random() < 0.5, rng.random() < 0.4, rng.random() < 0.3
        if decode:
            c["pad"] = 0
        return c
    c["B"] = _log_int(rng, 1, 48)
    # at most the padded scores of the largest listed case, B * Hq * longest^2
    scores = 2 * 32 * 8192 * 8192 / (c["B"] * Hq)
    most = int(math.sqrt(scores))
    if op == "packed":
        c["hi"] = _log_int(rng, 2, min(8192, most))
        c["lo"] = rng.randrange(0, c["hi"] + 1)
    else:
        c["page"] = rng.choice((16, 16, 32, 64, 128, 256))
        c["ctx"] = _log_int(rng, 16, 8192)
        c["hi"] = _log_int(rng, 1, min(c["ctx"], 2048, int(scores / c["ctx"])))
        c["lo"] = rng.randrange(0, c["hi"] + 1)
    c["window"] = rng.choice((0, 0, 0, _log_int(rng, 1, 4096)))
    c["lse"] = rng.random() < 0.4
    return c


def _lengths(case):
    """(new tokens, cached tokens with the new ones) of every sequence; the longest of the range is always among the new."""
    r = np.random.RandomState(case["lens"] % (1 << 31))
    n = r.randint(case["lo"], case["hi"] + 1, case["B"])
    n[r.randint(case["B"])] = case["hi"]
    if case["op"] == "packed":
        return n, n.copy()
    total = np.array([r.randint(x, case["ctx"] + 1) for x in n])
    return n, total


def _table(max_pos, rot, device):
    """cos and sin of every position's angles, formed in 64 bits: [max_pos, rot] = [cos | sin], each rot/2 wide."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot)
    a = torch.arange(max_pos, dtype=torch.float64, device=device)[:, None] * inv
    return torch.cat((a.cos(), a.sin()), 1).float().contiguous()


def _inputs(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    n, total = _lengths(case)
    B, Hq, Hkv, D = case["B"], case["Hq"], case["Hkv"], case["D"]
    T = int(n.sum()) + case["pad"]
    bf = lambda *s: torch.randn(s, generator=g, device=dev).to(torch.bfloat16)  # noqa: E731
    s = {"case": case, "n_max": int(n.max()), "k_max": int(total.max()), "scale": 1.0 / math.sqrt(D)}
    s["cu"] = torch.tensor(np.concatenate(([0], np.cumsum(n))), dtype=torch.int32, device=dev)
    s["q"] = bf(T, Hq, D)
    if case["op"] != "chunk":
        s["k"], s["v"] = bf(T, Hkv, D), bf(T, Hkv, D)
    if case["op"] != "append":
        s["out"] = torch.zeros((T, Hq, D), dtype=torch.bfloat16, device=dev)
        s["lse"] = torch.zeros((T, Hq), device=dev) if case["lse"] else None
    if case["op"] != "packed":
        page = case["page"]
        held = (total + page - 1) // page
        max_pages = -(-case["ctx"] // page)
        num = int(held.sum()) + 3
        order = torch.randperm(num, generator=g, device=dev).to(torch.int32).cpu()
        table = torch.full((B, max_pages), -1, dtype=torch.int32)
        at = 0
        for b in range(B):
            table[b, : held[b]] = order[at : at + held[b]]
            at += int(held[b])
        s["page_table"] = table.to(dev)
        s["seq_lens"] = torch.tensor(total, dtype=torch.int32, device=dev)
        s["k_pool"], s["v_pool"] = bf(num, Hkv, page, D), bf(num, Hkv, page, D)
        if case["op"] == "append":
            s["table"] = _table(case["ctx"], case["rot"], dev)
            s["q_out"] = torch.zeros_like(s["q"])
            s["k_out"] = torch.zeros_like(s["k"]) if case["kout"] else None
            if case["fp8"]:
                s["k_scale"], s["v_scale"] = 0.011, 0.009
                for p in ("k_pool", "v_pool"):
                    s[p] = (s[p].float() * 50).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return s


def prepare(case, seed):
    return _inputs(case, seed)


# ---------------------------------------------------------------- the plain forms


def _places(cu, T):
    """(sequence, index in it, whether any sequence holds it) of every row of a packed buffer."""
    t = torch.arange(T, device=cu.device)
    seq = (t[:, None] >= cu[None, 1:]).sum(1)
    real = seq < cu.numel() - 1
    seq = seq.clamp_max(cu.numel() - 2)
    return seq, torch.where(real, t - cu.long()[seq], torch.zeros_like(t)), real


def _plain_attention(q, k, v, lq, lk, window, scale):
    """Padded q [B,Sq,Hq,D] over k, v [B,Sk,Hkv,D] with true lengths lq, lk: causal at the end, in 32 bits."""
    B, Sq, Hq, D = q.shape
    Sk, Hkv = k.shape[1], k.shape[2]
    G = Hq // Hkv
    qf = (q.float() * scale).view(B, Sq, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * Sq, D)
    kf = k.float().permute(0, 2, 1, 3)
    vf = v.float().permute(0, 2, 1, 3)
    i = torch.arange(Sq, device=q.device)[None, :, None] + (lk - lq)[:, None, None]
    j = torch.arange(Sk, device=q.device)[None, None, :]
    hidden = (j > i) | (j >= lk[:, None, None])
    if window:
        hidden |= j <= i - window
    s = (qf @ kf.transpose(2, 3)).view(B, Hkv, G, Sq, Sk)
    s.masked_fill_(hidden[:, None, None], float("-inf"))
    m = s.amax(-1, keepdim=True)
    m0 = torch.where(m == float("-inf"), torch.zeros_like(m), m)
    p = s.sub_(m0).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.view(B, Hkv, G * Sq, Sk) @ vf).view(B, Hkv, G, Sq, D) / torch.where(total > 0, total, torch.ones_like(total))
    lse = torch.where(total > 0, m0 + total.log(), torch.full_like(total, float("-inf")))
    return o.permute(0, 3, 1, 2, 4).reshape(B, Sq, Hq, D), lse.permute(0, 3, 1, 2, 4).reshape(B, Sq, Hq)


def _to_rows(s, o, lse):
    seq, at, real = _places(s["cu"], s["q"].shape[0])
    s["out"].copy_(torch.where(real[:, None, None], o[seq, at].to(torch.bfloat16), s["out"]))
    if s["lse"] is not None:
        s["lse"].copy_(torch.where(real[:, None], lse[seq, at], s["lse"]))
    return [s["out"]] if s["lse"] is None else [s["out"], s["lse"]]


def _padded(x, cu, longest):
    at = (cu[:-1, None].long() + torch.arange(longest, device=cu.device)).clamp_max(max(x.shape[0] - 1, 0))
    return x[at]


def _plain_packed(s):
    cu, n = s["cu"], s["n_max"]
    lens = (cu[1:] - cu[:-1]).long()
    o, lse = _plain_attention(_padded(s["q"], cu, n), _padded(s["k"], cu, n), _padded(s["v"], cu, n), lens, lens, s["case"]["window"], s["scale"])
    return _to_rows(s, o, lse)


def _plain_chunk(s):
    cu, page = s["cu"], s["case"]["page"]
    j = torch.arange(s["k_max"], device=cu.device)
    lk = s["seq_lens"].long()
    phys = s["page_table"].long()[:, j // page].clamp_min(0)
    there = (j < lk[:, None])[:, :, None, None]
    k = s["k_pool"][phys, :, (j % page)[None, :]]
    v = torch.where(there, s["v_pool"][phys, :, (j % page)[None, :]], torch.zeros((), dtype=torch.bfloat16, device=cu.device))
    o, lse = _plain_attention(_padded(s["q"], cu, s["n_max"]), k, v, (cu[1:] - cu[:-1]).long(), lk, s["case"]["window"], s["scale"])
    return _to_rows(s, o, lse)


def _plain_rotate(x, cos, sin, rot, interleaved):
    """x [T,H,D] rotated by its row's angles (cos, sin [T, rot/2]), in 32 bits."""
    x = x.float()
    r, rest = x[..., :rot], x[..., rot:]
    cos, sin = cos[:, None], sin[:, None]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = r[..., : rot // 2], r[..., rot // 2 :]
        r = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((r, rest), -1)


def _append_places(s):
    case, cu = s["case"], s["cu"]
    seq, at, real = _places(cu, s["q"].shape[0])
    pos = (s["seq_lens"].long() - (cu[1:] - cu[:-1]).long())[seq] + at
    pos = torch.where(real, pos, torch.zeros_like(pos))
    return real, pos, s["page_table"].long()[seq, pos // case["page"]], pos % case["page"]


def _append_outputs(s):
    f8 = (lambda x: x.view(torch.float8_e4m3fn)) if s["case"]["fp8"] else (lambda x: x)
    got = [s["q_out"], f8(s["k_pool"]), f8(s["v_pool"])]
    return got if s["k_out"] is None else got + [s["k_out"]]


def _plain_append(s):
    case, rot = s["case"], s["case"]["rot"]
    real, pos, phys, slot = _append_places(s)
    cos, sin = s["table"][pos, : rot // 2], s["table"][pos, rot // 2 :]
    q = _plain_rotate(s["q"], cos, sin, rot, case["interleaved"])
    k = _plain_rotate(s["k"], cos, sin, rot, case["interleaved"])
    here = real[:, None, None]
    s["q_out"].copy_(torch.where(here, q.to(torch.bfloat16), s["q_out"]))
    if s["k_out"] is not None:
        s["k_out"].copy_(torch.where(here, k.to(torch.bfloat16), s["k_out"]))
    n = real.numel() - case["pad"]                 # the rows behind the last sequence go nowhere
    v = s["v"].float()
    if case["fp8"]:
        k = (k * (1.0 / s["k_scale"])).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        v = (v * (1.0 / s["v_scale"])).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        k, v = k.to(torch.bfloat16), v.to(torch.bfloat16)
    s["k_pool"][phys[:n], :, slot[:n]] = k[:n]
    s["v_pool"][phys[:n], :, slot[:n]] = v[:n]
    return _append_outputs(s)


def run(state):
    s, case = state, state["case"]
    if own:
        from scaled_dot_product_prefill_b200 import api

        if case["op"] == "packed":
            api.attn_prefill_packed(s["q"], s["k"], s["v"], s["cu"], window=case["window"], out=s["out"], lse=s["lse"])
            return [s["out"]] if s["lse"] is None else [s["out"], s["lse"]]
        if case["op"] == "chunk":
            api.attn_prefill_packed_paged(s["q"], s["k_pool"], s["v_pool"], s["cu"], s["page_table"], s["seq_lens"],
                                          max_seq_len=s["k_max"], window=case["window"], out=s["out"], lse=s["lse"])
            return [s["out"]] if s["lse"] is None else [s["out"], s["lse"]]
        cu = None if case["hi"] == 1 and case["lo"] == 1 else s["cu"]     # one token of every sequence
        if case["fp8"]:
            api.attn_kv_append_rope_fp8(s["q"], s["k"], s["v"], s["k_pool"], s["v_pool"], s["table"], s["page_table"], s["seq_lens"],
                                        k_scale=s["k_scale"], v_scale=s["v_scale"], cu_seqlens=cu, interleaved=case["interleaved"],
                                        q_out=s["q_out"], k_out=s["k_out"])
        else:
            api.attn_kv_append_rope(s["q"], s["k"], s["v"], s["k_pool"], s["v_pool"], s["table"], s["page_table"], s["seq_lens"],
                                    cu_seqlens=cu, interleaved=case["interleaved"], q_out=s["q_out"], k_out=s["k_out"])
        return _append_outputs(s)
    return {"packed": _plain_packed, "chunk": _plain_chunk, "append": _plain_append}[case["op"]](s)


# ---------------------------------------------------------------- what a pass cannot do without


def _visible(n, total, window):
    """Visible (query, key) pairs of one sequence: query i of n sits at position total - n + i."""
    last = np.arange(total - n, total, dtype=np.int64)
    seen = last + 1
    return int((np.minimum(seen, window) if window else seen).sum())


def work(case):
    n, total = _lengths(case)
    T, Hq, Hkv, D = int(n.sum()), case["Hq"], case["Hkv"], case["D"]
    if case["op"] == "append":
        elem = 1 if case["fp8"] else 2
        b = T * D * (Hq * 4 + Hkv * 4 + 2 * Hkv * elem + (Hkv * 2 if case["kout"] else 0)) + T * case["rot"] * 4
        return {"bytes": b, "flops": T * (Hq + Hkv) * case["rot"] // 2 * 6}
    pairs = sum(_visible(int(x), int(y), case["window"]) for x, y in zip(n, total))
    # keys that some query of the chunk sees
    keys = sum(min(int(y), int(x) + case["window"] - 1) if case["window"] and x else (int(y) if x else 0) for x, y in zip(n, total))
    return {"bytes": 2 * (2 * T * Hq * D + 2 * keys * Hkv * D) + (4 * T * Hq if case["lse"] else 0), "flops": 4 * D * Hq * pairs}


# ---------------------------------------------------------------- the definitions, in 64 bits


def _exact_attention(case, s, keys_of):
    n, total = _lengths(case)
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    G = Hq // Hkv
    out = s["out"].double()
    lse = None if s["lse"] is None else s["lse"].double()
    row = 0
    for b in range(case["B"]):
        x, y = int(n[b]), int(total[b])
        if x == 0:
            continue
        K, V = keys_of(b, y)
        behind = torch.arange(y - x, y, device=out.device)[:, None] - torch.arange(y, device=out.device)[None, :]
        seen = behind >= 0
        if case["window"]:
            seen &= behind < case["window"]
        for h in range(Hq):
            z = s["q"][row : row + x, h].double() @ K[:, h // G].double().t() / math.sqrt(D)
            z = torch.where(seen, z, torch.full_like(z, -math.inf))
            out[row : row + x, h] = torch.softmax(z, 1) @ V[:, h // G].double()
            if lse is not None:
                lse[row : row + x, h] = torch.logsumexp(z, 1)
        row += x
    return [out] if lse is None else [out, lse]


def exact(case, seed):
    s = _inputs(case, seed)
    n, total = _lengths(case)
    if case["op"] == "packed":
        first = np.concatenate(([0], np.cumsum(n)))
        return _exact_attention(case, s, lambda b, y: (s["k"][first[b] : first[b] + y], s["v"][first[b] : first[b] + y]))
    page = case["page"]

    def cached(b, y):
        own_pages = s["page_table"][b, : -(-y // page)].long()
        return tuple(p[own_pages].transpose(1, 2).reshape(-1, case["Hkv"], case["D"])[:y] for p in (s["k_pool"], s["v_pool"]))

    if case["op"] == "chunk":
        return _exact_attention(case, s, cached)
    # the append: the values themselves, not rounded to the cache's type (within its range)
    rot, half = case["rot"], case["rot"] // 2
    value = (lambda x: x.view(torch.float8_e4m3fn).double()) if case["fp8"] else (lambda x: x.double())
    q_out, k_pool, v_pool = s["q_out"].double(), value(s["k_pool"]), value(s["v_pool"])
    k_out = None if s["k_out"] is None else s["k_out"].double()
    first, second = (slice(0, rot, 2), slice(1, rot, 2)) if case["interleaved"] else (slice(0, half), slice(half, rot))

    def turned(x, angle):
        c, d, y = angle[:, None, :half].double(), angle[:, None, half:].double(), x.double()
        y[..., first] = x[..., first].double() * c - x[..., second].double() * d
        y[..., second] = x[..., second].double() * c + x[..., first].double() * d
        return y

    def stored(x, scale):
        return x if not case["fp8"] else (x / scale).clamp(-448.0, 448.0)

    row = 0
    for b in range(case["B"]):
        x, y = int(n[b]), int(total[b])
        at = slice(row, row + x)
        pos = torch.arange(y - x, y, device=q_out.device)
        phys = s["page_table"][b].long()[pos // page]
        q_out[at] = turned(s["q"][at], s["table"][pos])
        k = turned(s["k"][at], s["table"][pos])
        if k_out is not None:
            k_out[at] = k
        k_pool[phys, :, pos % page] = stored(k, s.get("k_scale"))
        v_pool[phys, :, pos % page] = stored(s["v"][at].double(), s.get("v_scale"))
        row += x
    return [q_out, k_pool, v_pool] if k_out is None else [q_out, k_pool, v_pool, k_out]
