"""The attention half of a quantized decoder layer as measured cases.

Four operators stand between the query / key / value projections (W4A4 GEMMs)
and the output projection:

* ``rope``    norms of queries and keys for each head and the position
              rotation, in one pass;
* ``write``   keys and values quantized to 8 bits as they enter a paged cache,
              one scale for each page and head, and the touched pages read
              back;
* ``read``    whole contexts of that cache read back to bf16;
* ``attend``  attention of a ragged batch of queries over that cache.

``own`` False: the plain form in elementary torch operations, in 32 bits (the
rotation angles in 64), rounded once at the end. ``own`` True: the calls a
user makes of the library.

The cache. ``kc``, ``vc``: int8 [pages, Hkv, P, d]; ``ks``, ``vs``: fp32
[pages, Hkv]; a code c stands for c * scale of its page and head. Token t of
sequence b is slot t % P of page ``table[b, t // P]``. A call's new tokens are
the last ones of each sequence: ``kv_len`` counts them already.

The quantizer, in binary32 (every operation rounded to nearest even):
a = max |x| over the finite new values of a page and head, s = max(s_old,
a / 127), s_old the page's scale if it holds earlier tokens of the sequence,
else 0; s < 2^-126 becomes 0. Earlier codes become rint(c * (s_old / s)), new
ones clamp(rint(x * (1 / s)), -127, 127), all zero where s is 0.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
TINY = 2.0 ** -126


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token of a decode step, 32 query and 8 key heads with head norms: pure latency
        {"name": "rope_one_token", "kind": "rope", "N": 1, "Hq": 32, "Hkv": 8, "d": 128, "rot": 128,
         "norm": True, "inter": False, "far": 4096},
        # a prefill of 4096 tokens at D = 4096 with grouped key heads, rotation only
        {"name": "rope_4096", "kind": "rope", "N": 4096, "Hq": 32, "Hkv": 8, "d": 128, "rot": 128,
         "norm": False, "inter": False, "far": 4096},
        # odd token count, half of each short head rotated in neighbouring pairs, positions up to a million
        {"name": "rope_odd_far", "kind": "rope", "N": 1237, "Hq": 20, "Hkv": 4, "d": 64, "rot": 32,
         "norm": True, "inter": True, "far": 1 << 20},
        # a decode step of 64 sequences: one token each into half-filled pages
        {"name": "write_decode_64", "kind": "write", "B": 64, "q": 1, "kv": 4096, "ragged": True, "Hkv": 8, "d": 128, "P": 64},
        # ragged prefill chunks, as many key heads as query heads, small pages
        {"name": "write_prefill_ragged", "kind": "write", "B": 7, "q": 2048, "kv": 2048, "ragged": True, "Hkv": 32, "d": 128, "P": 16},
        # whole contexts of four sequences read back in bf16
        {"name": "read_contexts", "kind": "read", "B": 4, "kv": 8192, "ragged": True, "Hkv": 8, "d": 128, "P": 128},
        # three short contexts of short heads, pages that end inside
        {"name": "read_short", "kind": "read", "B": 3, "kv": 77, "ragged": True, "Hkv": 5, "d": 64, "P": 16},
        # one sequence, one token, a short context: pure latency
        {"name": "attend_one", "kind": "attend", "B": 1, "q": 1, "kv": 200, "ragged": False, "Hq": 32, "Hkv": 32, "d": 128, "P": 16, "causal": True, "window": 0},
        # a decode step of 64 sequences at D = 4096 with grouped key heads
        {"name": "attend_decode_64", "kind": "attend", "B": 64, "q": 1, "kv": 4096, "ragged": True, "Hq": 32, "Hkv": 8, "d": 128, "P": 64, "causal": True, "window": 0},
        # two very long contexts at D = 8192
        {"name": "attend_decode_long", "kind": "attend", "B": 2, "q": 1, "kv": 131071, "ragged": False, "Hq": 64, "Hkv": 8, "d": 128, "P": 128, "causal": True, "window": 0},
        # prefill of two 4096-token prompts at D = 4096
        {"name": "attend_prefill", "kind": "attend", "B": 2, "q": 4096, "kv": 4096, "ragged": False, "Hq": 32, "Hkv": 8, "d": 128, "P": 64, "causal": True, "window": 0},
        # chunks of ragged prompts behind longer contexts, short heads, small pages, a sliding window
        {"name": "attend_chunk_window", "kind": "attend", "B": 6, "q": 511, "kv": 8000, "ragged": True, "Hq": 24, "Hkv": 8, "d": 64, "P": 16, "causal": True, "window": 1000},
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of lo .. hi."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.499)))))))


def draw(rng):
    case = _draw(rng)
    top = [work(c) for c in listed()]
    top = {k: max(w[k] for w in top) for k in top[0]}
    while any(work(case)[k] > top[k] for k in top):   # no dearer than the largest listed case
        k = "B" if case.get("B", 1) > 1 else "kv" if case.get("kv", 0) > 2 * case.get("q", 1) else "q"
        case[k] = max(1, case[k] // 2)
        if k == "q":
            case["kv"] = max(case["q"], case["kv"] // 2)
    return case


def _draw(rng):
    kind = rng.choice(["rope", "write", "read", "attend", "attend", "attend"])
    d, P = rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
    Hkv = rng.choice([1, 2, 4, 5, 8, 8, 16, 32])
    G = rng.choice([1, 1, 2, 3, 4, 4, 7, 8])
    while Hkv * G > 64:
        G = max(1, G // 2)
    if kind == "rope":
        rot = rng.choice([d, d, d // 2])
        return {"kind": kind, "N": _log(rng, 1, 8192), "Hq": Hkv * G, "Hkv": Hkv, "d": d, "rot": rot,
                "norm": rng.random() < 0.5, "inter": rng.random() < 0.4, "far": _log(rng, 4096, 1 << 20)}
    ragged = rng.random() < 0.6
    B = _log(rng, 1, 96)
    if kind == "write":
        q = rng.choice([1, _log(rng, 1, 4096)])
        B = max(1, min(B, 16384 // q))
        return {"kind": kind, "B": B, "q": q, "kv": q + _log(rng, 1, 8192) - 1, "ragged": ragged, "Hkv": Hkv, "d": d, "P": P}
    if kind == "read":
        return {"kind": kind, "B": B, "kv": max(1, _log(rng, 1, 32768) // B), "ragged": ragged, "Hkv": Hkv, "d": d, "P": P}
    causal = rng.random() < 0.85
    if rng.random() < 0.5:   # decode, or a few tokens of a draft to be checked
        q = rng.choice([1, 1, 1, rng.randint(2, 8)])
        kv = max(q, _log(rng, 16, 131072) // (1 if B <= 2 else B // 2))
    else:                    # prefill and chunks
        B = max(1, B // 8)
        q = _log(rng, 9, 4096)
        kv = q + rng.choice([0, _log(rng, 1, 8192) - 1])
        while B * Hkv * G * q * kv > 2 * 32 * 4096 * 4096:
            B, q, kv = (B // 2, q, kv) if B > 1 else (1, max(1, q // 2), max(q // 2, 1, kv // 2))
    return {"kind": kind, "B": B, "q": q, "kv": kv, "ragged": ragged, "Hq": Hkv * G, "Hkv": Hkv, "d": d, "P": P,
            "causal": causal, "window": rng.choice([0, 0, _log(rng, 1, 4096)]) if causal else 0}


def _lens(case):
    """([new or read tokens of each sequence], [its length with them])."""
    B, kv, q = case["B"], case["kv"], case.get("q", case["kv"])
    if not case["ragged"]:
        return [q] * B, [kv] * B
    r = random.Random(B * 7919 + q * 104729 + kv)
    least = 0 if case["kind"] == "attend" and q > 1 else 1   # some attended chunks are empty
    qs = [q] + [min(q, max(least, int(q * (1.1 * r.random() - 0.05)))) for _ in range(B - 1)]
    ks = [kv] + [max(a, 1, int(kv * (0.15 + 0.85 * r.random()))) for a in qs[1:]]
    return (qs if "q" in case else list(ks)), ks


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 2654435761 % (1 << 62) + 12345)
    return g


def _channels(g, H, d, n_out):
    """Channel gains of H heads: log-normal, and a few outlier channels."""
    c = torch.exp(0.4 * torch.randn(H, d, generator=g, device=DEV))
    c[:, torch.randperm(d, generator=g, device=DEV)[:n_out]] *= 6.0
    return c


def _cache(g, num, H, P, d, gain):
    """Codes and scales of `num` pages as earlier steps left them, made page
    by page from activations with the given channel gains."""
    x = torch.randn(num, H, P, d, generator=g, device=DEV) * gain[None, :, None, :]
    scale = x.abs().amax((2, 3)) / 127.0
    return (x / scale[:, :, None, None]).round_().clamp_(-127, 127).to(torch.int8), scale


def prepare(case, seed):
    g = _gen(seed)
    d, Hkv = case["d"], case["Hkv"]
    if case["kind"] == "rope":
        N, Hq, rot = case["N"], case["Hq"], case["rot"]
        w = (Hq + 2 * Hkv) * d
        qkv = (torch.randn(N, w, generator=g, device=DEV) * torch.exp(0.4 * torch.randn(w, generator=g, device=DEV))).bfloat16()
        s = {"case": case, "qkv": qkv,
             "pos": torch.randint(0, case["far"], (N,), generator=g, device=DEV, dtype=torch.int32),
             "inv_freq": (500000.0 ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)).float(),
             "qw": None, "kw": None,
             "q_out": torch.empty(N, Hq, d, dtype=torch.bfloat16, device=DEV),
             "k_out": torch.empty(N, Hkv, d, dtype=torch.bfloat16, device=DEV)}
        if case["norm"]:
            s["qw"] = (1.0 + 0.2 * torch.randn(d, generator=g, device=DEV)).bfloat16()
            s["kw"] = (1.0 + 0.2 * torch.randn(d, generator=g, device=DEV)).bfloat16()
        # views of the projections' output, as a user has them
        s["q"] = qkv[:, :Hq * d].view(N, Hq, d)
        s["k"] = qkv[:, Hq * d:(Hq + Hkv) * d].view(N, Hkv, d)
        return s
    B, P = case["B"], case["P"]
    qs, ks = _lens(case)
    N = sum(qs)
    pages = [-(-k // P) for k in ks]
    num = sum(pages) + 3
    order = (torch.randperm(num, generator=g, device=DEV)).to(torch.int32)
    width = max(pages) + 1
    # page ids of each sequence; behind its pages the table holds -1
    first = torch.tensor(np.cumsum([0] + pages[:-1]), device=DEV)
    col = torch.arange(width, device=DEV)
    have = torch.tensor(pages, device=DEV)
    at = (first[:, None] + col[None]).clamp(max=num - 1)
    table = torch.where(col[None] < have[:, None], order[at], torch.full_like(order[at], -1)).contiguous()
    kg, vg = _channels(g, Hkv, d, 2), _channels(g, Hkv, d, 1) * 0.5
    kc, ksc = _cache(g, num, Hkv, P, d, kg)
    vc, vsc = _cache(g, num, Hkv, P, d, vg)
    cu = torch.tensor(np.cumsum([0] + qs), dtype=torch.int32, device=DEV)
    s = {"case": case, "kc": kc, "vc": vc, "ks": ksc, "vs": vsc, "table": table, "cu": cu,
         "kv_len": torch.tensor(ks, dtype=torch.int32, device=DEV), "N": N,
         "ragged": bool(case["ragged"] and len(set(qs)) > 1)}
    if case["kind"] == "attend":
        Hq = case["Hq"]
        gain = kg.repeat_interleave(Hq // Hkv, 0)
        # logits of a standard deviation near 2: a few tokens carry most of the weight
        x = torch.randn(N, Hq, d, generator=g, device=DEV) * (2.0 / gain.square().mean(-1, keepdim=True))
        s["q"] = x.bfloat16()
        s["out"] = torch.empty(N, Hq, d, dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.empty(N, Hq, dtype=torch.float32, device=DEV)
        s["max_q"] = max(qs)
        return s
    if case["kind"] == "write":
        # new keys and values are slices of the projections' output; one token in 16 is larger,
        # so that some pages have to take a larger scale
        loud = 1.0 + 1.5 * (torch.rand(N, 1, 1, generator=g, device=DEV) < 1 / 16).float()
        kv = torch.empty(N, 2, Hkv, d, dtype=torch.bfloat16, device=DEV)
        kv[:, 0] = (torch.randn(N, Hkv, d, generator=g, device=DEV) * kg * loud).bfloat16()
        kv[:, 1] = (torch.randn(N, Hkv, d, generator=g, device=DEV) * vg * loud).bfloat16()
        s["k"], s["v"] = kv[:, 0], kv[:, 1]
        rs = [q + (k - q) % P for q, k in zip(qs, ks)]   # read back from the start of the first touched page
    else:
        rs = ks
    s["cu_read"] = torch.tensor(np.cumsum([0] + rs), dtype=torch.int32, device=DEV)
    s["R"] = sum(rs)
    s["k_out"] = torch.empty(s["R"], Hkv, d, dtype=torch.bfloat16, device=DEV)
    s["v_out"] = torch.empty(s["R"], Hkv, d, dtype=torch.bfloat16, device=DEV)
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    if own:
        return _run_own(s)
    kind = s["case"]["kind"]
    if kind == "rope":
        return _plain_rope(s)
    if kind == "attend":
        return _plain_attend(s)
    if kind == "write":
        _plain_write(s)
        k, v = _plain_read(s)
        return {"k": k, "v": v, "ks": s["ks"], "vs": s["vs"]}
    k, v = _plain_read(s)
    return {"k": k, "v": v}


def _run_own(s):
    import rotation_post_quantization_b200 as rq
    c = s["case"]
    if c["kind"] == "rope":
        rq.respin_qk_norm_rope(s["q"], s["k"], s["pos"], s["inv_freq"], s["q_out"], s["k_out"],
                               q_weight=s["qw"], k_weight=s["kw"], eps=1e-6, interleaved=c["inter"])
        return {"q": s["q_out"], "k": s["k_out"]}
    cache = rq.KvCache(s["kc"], s["vc"], s["ks"], s["vs"])
    if c["kind"] == "attend":
        if "ws" not in s:   # a program keeps its workspace
            n = rq.respin_kv_attention_workspace(cache, c["Hq"], s["N"], max_q=s["max_q"])
            s["ws"] = torch.empty(n, dtype=torch.uint8, device=DEV)
        rq.respin_kv_attention(cache, s["q"], s["kv_len"], s["table"], s["out"], s["ws"],
                               cu=s["cu"] if s["ragged"] else None, max_q=s["max_q"],
                               causal=c["causal"], window=c["window"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    if c["kind"] == "write":
        rq.respin_kv_append(cache, s["k"], s["v"], s["kv_len"], s["table"], cu=s["cu"] if s["ragged"] else None)
        rq.respin_kv_read(cache, s["k_out"], s["v_out"], s["kv_len"], s["table"], cu=s["cu_read"])
        return {"k": s["k_out"], "v": s["v_out"], "ks": s["ks"], "vs": s["vs"]}
    rq.respin_kv_read(cache, s["k_out"], s["v_out"], s["kv_len"], s["table"], cu=s["cu_read"])
    return {"k": s["k_out"], "v": s["v_out"]}


def _plain_rope(s):
    c = s["case"]
    rot = c["rot"]
    ang = s["pos"].double()[:, None] * s["inv_freq"].double()[None]
    cos, sin = ang.cos().float()[:, None], ang.sin().float()[:, None]

    def one(x, w):
        x = x.float()
        if w is not None:
            x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.float()
        y, rest = x[..., :rot], x[..., rot:]
        if c["inter"]:
            a, b = y[..., 0::2], y[..., 1::2]
            y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
        else:
            a, b = y[..., :rot // 2], y[..., rot // 2:]
            y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
        return torch.cat((y, rest), -1).bfloat16()

    return {"q": one(s["q"], s["qw"]), "k": one(s["k"], s["kw"])}


def _places(s, cu, N):
    """(sequence, position) of each row of a ragged batch of the last tokens."""
    row = torch.arange(N, device=DEV)
    seq = torch.searchsorted(cu[1:].long(), row, right=True)
    return seq, s["kv_len"].long()[seq] - (cu[seq + 1] - cu[seq]).long() + row - cu[seq].long()


def _plain_write(s):
    P = s["case"]["P"]
    seq, pos = _places(s, s["cu"], s["N"])
    page, slot = s["table"].long()[seq, pos // P], pos % P
    start = s["kv_len"].long()[seq] - (s["cu"][seq + 1] - s["cu"][seq]).long()
    older = (pos // P == start // P) & (start % P > 0)   # the page holds earlier tokens of the sequence
    first = s["cu"][:-1].long()                          # every sequence writes one token at least
    for x, codes, scale in ((s["k"], s["kc"], s["ks"]), (s["v"], s["vc"], s["vs"])):
        x = x.float()
        fin = torch.where(torch.isfinite(x), x, torch.zeros_like(x))
        top = fin.abs().amax(-1) / 127.0                                   # [N, H]
        was = torch.where(older[:, None], scale[page], torch.zeros_like(top))
        new = torch.zeros_like(scale).scatter_reduce(0, page[:, None].expand_as(top), torch.maximum(top, was), "amax")
        sc = new[page]
        sc = torch.where(sc < TINY, torch.zeros_like(sc), sc)
        div = torch.where(sc > 0, sc, torch.ones_like(sc))
        ratio, inv = torch.where(sc > 0, was / div, torch.zeros_like(sc)), torch.where(sc > 0, torch.ones_like(sc) / div, torch.zeros_like(sc))
        at, rt = page[first], ratio[first][:, :, None, None]               # each sequence's first touched page
        kept = codes[at]
        codes[at] = torch.where(older[first][:, None, None, None], (kept.float() * rt).round().to(torch.int8), kept)
        q = (x * inv[:, :, None]).clamp(-127.0, 127.0).round()
        codes[page, :, slot] = torch.where(torch.isnan(q) | (sc == 0)[:, :, None], torch.zeros_like(q), q).to(torch.int8)
        scale[page] = sc


def _plain_read(s):
    P = s["case"]["P"]
    seq, pos = _places(s, s["cu_read"], s["R"])
    page, slot = s["table"].long()[seq, pos // P], pos % P
    return tuple((codes[page, :, slot].float() * scale[page][:, :, None]).bfloat16()
                 for codes, scale in ((s["kc"], s["ks"]), (s["vc"], s["vs"])))


def _plain_attend(s):
    c = s["case"]
    B, Hq, Hkv, d, P = c["B"], c["Hq"], c["Hkv"], c["d"], c["P"]
    G, M = Hq // Hkv, s["max_q"]
    pages = s["table"][:, :-1].clamp(min=0).long()
    L = pages.shape[1] * P
    K, V = ((x[pages].float() * z[pages][..., None, None]).transpose(1, 2).reshape(B, Hkv, L, d)
            for x, z in ((s["kc"], s["ks"]), (s["vc"], s["vs"])))
    seq, pos = _places(s, s["cu"], s["N"])
    idx = torch.arange(s["N"], device=DEV) - s["cu"].long()[seq]
    Q = torch.zeros(B, M, Hkv, G, d, device=DEV)
    Q[seq, idx] = s["q"].float().view(-1, Hkv, G, d)
    where = torch.full((B, M), -1, device=DEV)
    where[seq, idx] = pos
    S = Q.permute(0, 2, 1, 3, 4).reshape(B, Hkv, M * G, d) @ K.transpose(2, 3)
    S *= d ** -0.5
    S = S.view(B, Hkv, M, G, L)
    j = torch.arange(L, device=DEV)
    ok = j[None, None] < s["kv_len"].long()[:, None, None]
    if c["causal"]:
        ok = ok & (j[None, None] <= where[:, :, None])
        if c["window"]:
            ok = ok & (j[None, None] > where[:, :, None] - c["window"])
    S.masked_fill_(~ok[:, None, :, None], -math.inf)
    m = S.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    S.sub_(m).exp_()
    l = S.sum(-1, keepdim=True)
    O = (S.view(B, Hkv, M * G, L) @ V).view(B, Hkv, M, G, d) / torch.where(l > 0, l, torch.ones_like(l))
    lse = (m + l.log())[..., 0]
    out = O.permute(0, 2, 1, 3, 4)[seq, idx].reshape(-1, Hq, d).bfloat16()
    return {"out": out, "lse": lse.permute(0, 2, 1, 3)[seq, idx].reshape(-1, Hq)}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    def _exact_rope(s, x, w):
        rot, inter = s["case"]["rot"], s["case"]["inter"]
        y = x.double().clone()
        if w is not None:
            y = y * w.double() * (y.pow(2).sum(-1, keepdim=True) / y.shape[-1] + 1e-6).rsqrt()
        out = y.clone()
        for i in range(rot // 2):
            t = s["pos"].double() * s["inv_freq"][i].double()
            a, b = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
            z = torch.complex(y[..., a], y[..., b]) * torch.polar(torch.ones_like(t), t)[:, None]
            out[..., a], out[..., b] = z.real, z.imag
        return out

    def _exact_write(s, qs, ks):
        """The quantizer in 64 bits with its binary32 roundings written out (a
        64-bit quotient or product of two binary32 numbers, rounded once more,
        is the correctly rounded one)."""
        P = s["case"]["P"]
        r32 = lambda x: x.float().double()  # noqa: E731
        row = 0
        for b, (q, n) in enumerate(zip(qs, ks)):
            for p in range((n - q) // P, -(-n // P) if q else 0):
                lo, hi = max(n - q, p * P), min(n, (p + 1) * P)
                page = int(s["table"][b, p])
                for x, codes, scale in ((s["k"], s["kc"], s["ks"]), (s["v"], s["vc"], s["vs"])):
                    new = x[row + lo - (n - q):row + hi - (n - q)].double().transpose(0, 1)   # [H, tokens, d]
                    old = scale[page].double() if lo > p * P else torch.zeros_like(scale[page]).double()
                    sc = torch.maximum(old, r32(torch.where(new.isfinite(), new, 0.0).abs().flatten(1).amax(1) / 127.0))
                    sc[sc < TINY] = 0.0
                    some = sc > 0
                    div = torch.where(some, sc, 1.0)
                    if lo > p * P:
                        c = codes[page, :, :lo - p * P].double()
                        codes[page, :, :lo - p * P] = (r32(c * r32(old / div)[:, None, None]).round() * some[:, None, None]).to(torch.int8)
                    c = r32(new * r32(1.0 / div)[:, None, None]).nan_to_num(0.0, 127.0, -127.0).clamp(-127, 127).round()
                    codes[page, :, lo - p * P:hi - p * P] = (c * some[:, None, None]).to(torch.int8)
                    scale[page] = sc.float()
            row += q

    def _exact_attend(s, qs, ks):
        c = s["case"]
        Hq, Hkv, d, P = c["Hq"], c["Hkv"], c["d"], c["P"]
        G = Hq // Hkv
        out = torch.zeros(s["N"], Hq, d, dtype=torch.float64, device=DEV)
        lse = torch.zeros(s["N"], Hq, dtype=torch.float64, device=DEV)
        row = 0
        for b, (q, n) in enumerate(zip(qs, ks)):
            ids = s["table"][b, :-(-n // P)].long()
            j = torch.arange(n, device=DEV)
            for h in range(Hkv if q else 0):
                K = (s["kc"][ids, h].double() * s["ks"][ids, h].double()[:, None, None]).flatten(0, 1)[:n]
                V = (s["vc"][ids, h].double() * s["vs"][ids, h].double()[:, None, None]).flatten(0, 1)[:n]
                step = max(1, (1 << 26) // (n * G))
                for i in range(0, q, step):
                    m = min(step, q - i)
                    at = (n - q + i + torch.arange(m, device=DEV))[:, None]
                    ok = (j[None] <= at) if c["causal"] else (j[None] >= 0).expand(m, n)
                    if c["window"]:
                        ok = ok & (at - j[None] < c["window"])
                    x = s["q"][row + i:row + i + m, h * G:(h + 1) * G].double()
                    t = torch.einsum("mgd,nd->mgn", x, K) / math.sqrt(d)
                    t = t.masked_fill(~ok[:, None], -math.inf)
                    z = torch.logsumexp(t, -1)
                    out[row + i:row + i + m, h * G:(h + 1) * G] = torch.einsum("mgn,nd->mgd", (t - z[..., None]).exp(), V)
                    lse[row + i:row + i + m, h * G:(h + 1) * G] = z
            row += q
        return {"out": out, "lse": lse}

    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "rope":
        return {"q": _exact_rope(s, s["q"], s["qw"]), "k": _exact_rope(s, s["k"], s["kw"])}
    qs, ks = _lens(case)
    if kind == "attend":
        return _exact_attend(s, qs, ks)
    if kind == "write":
        _exact_write(s, qs, ks)
    P = case["P"]
    outs = []
    for codes, scale in ((s["kc"], s["ks"]), (s["vc"], s["vs"])):
        rows = []
        for b, (q, n) in enumerate(zip(qs, ks)):
            begin = (n - q) // P * P if kind == "write" else 0
            ids = s["table"][b, :-(-n // P)].long()
            x = codes[ids].double() * scale[ids].double()[:, :, None, None]
            rows.append(x.permute(0, 2, 1, 3).reshape(-1, case["Hkv"], case["d"])[begin:n])
        outs.append(torch.cat(rows))
    got = {"k": outs[0], "v": outs[1]}
    if kind == "write":
        got |= {"ks": s["ks"].double(), "vs": s["vs"].double()}
    return got


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    d, Hkv = case["d"], case["Hkv"]
    if case["kind"] == "rope":
        n = case["N"] * (case["Hq"] + Hkv) * d
        return {"bytes": 4 * n + 4 * case["N"] + 2 * case["rot"], "flops": n * (3 + (4 if case["norm"] else 0))}
    qs, ks = _lens(case)
    P = case["P"]
    if case["kind"] == "read":
        n = sum(ks) * Hkv * d * 2
        return {"bytes": 3 * n + 8 * Hkv * sum(-(-k // P) for k in ks), "flops": n}
    if case["kind"] == "write":
        new = sum(qs) * Hkv * d * 2
        back = sum(q + (k - q) % P for q, k in zip(qs, ks)) * Hkv * d * 2
        touched = sum(-(-k // P) - (k - q) // P for q, k in zip(qs, ks) if q)
        # new values in, new codes out, touched pages' codes in and values out, their scales in and out
        return {"bytes": 2 * new + new + 3 * back + 16 * Hkv * touched, "flops": 3 * new + back}
    Hq = case["Hq"]
    pairs = seen = rows = 0
    for q, k in zip(qs, ks):
        if not q:
            continue
        rows += q
        w = case["window"] or k
        if case["causal"]:
            first = k - q + 1   # keys the first query sees without a window
            short = max(0, min(q, w - first + 1))
            pairs += short * first + short * (short - 1) // 2 + (q - short) * w
            seen += min(k, q + w - 1)
        else:
            pairs += q * k
            seen += k
    return {"bytes": seen * Hkv * d * 2 + rows * Hq * (4 * d + 4) + 8 * Hkv * (seen // P), "flops": 4 * pairs * Hq * d}
