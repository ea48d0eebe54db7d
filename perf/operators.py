"""The attention operators' measured cases: filling a paged 4-bit key/value cache, reading it
back, single-token attention over it and attention over whole prompts.

Every case gives head counts, the head size and the cache's page size; `lengths` derives the
sequence lengths from the case alone.  With `own` false, `run` computes the operators from
elementary torch operations in 32 bits; with `own` true it calls the library."""
import math
import random

import torch

own = False

DEV = "cuda"
TILE = 16  # tokens of one cache tile
THETA = 10000.0


# ---------------------------------------------------------------- cases
def listed():
    def c(name, op, heads, kv, dim, page, seqs, lo, hi, **more):
        return {"name": name, "op": op, "heads": heads, "kv_heads": kv, "dim": dim, "page": page, "rotary": dim,
                "seqs": seqs, "lo": lo, "hi": hi, "mix": 1, "past": 0, **more}

    return [
        # one stream of decode: the newest token of one sequence
        c("append_one", "append", 32, 8, 128, 64, 1, 1, 1, past=1000),
        # a decode step of a batch: one token of each of 64 sequences, partial rotation
        c("append_batch", "append", 32, 8, 128, 64, 64, 1, 1, past=1000, rotary=64),
        # prompts entering the cache
        c("append_prompt", "append", 32, 4, 128, 64, 5, 700, 3500),
        # a short cached prefix read back, small heads and pages
        c("gather_short", "gather", 8, 2, 64, 16, 1, 1501, 1501),
        # the prefixes of a batch of continued prompts
        c("gather_batch", "gather", 32, 8, 128, 64, 9, 1000, 12000),
        # one user decoding with a short context
        c("decode_short", "decode", 32, 8, 128, 64, 1, 777, 777),
        # a small model's batch: heads of 64, five query heads to a key head
        c("decode_small", "decode", 40, 8, 64, 16, 48, 50, 3000),
        # a serving batch, context lengths spread widely
        c("decode_batch", "decode", 32, 8, 128, 64, 64, 200, 16384),
        # one very long context, sixteen query heads to a key head
        c("decode_long", "decode", 32, 2, 128, 128, 1, 131072, 131072),
        # one short prompt
        c("prompt_short", "prompt", 32, 8, 128, 64, 1, 333, 333),
        # many short prompts packed, some with a cached prefix before them, heads of 64
        c("prompt_packed", "prompt", 24, 8, 64, 64, 24, 20, 700, past=150),
        # one long prompt
        c("prompt_long", "prompt", 32, 8, 128, 64, 1, 8192, 8192),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "gather", "decode", "decode", "prompt", "prompt"])
    heads, kv = rng.choice([(32, 8), (32, 4), (32, 2), (8, 8), (40, 8), (24, 8), (16, 1), (14, 2), (6, 6)])
    dim = rng.choice([64, 128])
    page = rng.choice([16, 32, 64, 128])
    rotary = rng.choice([dim, dim // 2, 32])
    past = 0
    if op == "append":
        seqs, hi = _spread(rng, 1, 48), _spread(rng, 1, 8192)
        hi = max(1, min(hi, 12000 // seqs))
        past = rng.randrange(0, 3000)
    elif op == "gather":
        seqs, hi = _spread(rng, 1, 32), _spread(rng, 20, 16384)
        hi = max(1, min(hi, 60000 // seqs))
    elif op == "decode":
        seqs, hi = _spread(rng, 1, 100), _spread(rng, 1, 100000)
        hi = max(1, min(hi, 400000 // seqs))
    else:
        seqs, hi = _spread(rng, 1, 32), _spread(rng, 1, 6000)
        hi = max(1, min(hi, 7000 // seqs))
        past = rng.choice([0, 0, rng.randrange(1, 1000)])
        past = min(past, 7000 // seqs)
    lo = hi if rng.random() < 0.3 else max(1, hi // rng.randrange(2, 30))
    return {"op": op, "heads": heads, "kv_heads": kv, "dim": dim, "page": page, "rotary": rotary, "seqs": seqs,
            "lo": lo, "hi": hi, "mix": rng.randrange(1 << 20), "past": past}


def lengths(case):
    """New tokens (queries, or cached tokens for gather and decode) and tokens before them, per sequence."""
    r = random.Random(case["mix"])
    lo, hi = case["lo"], case["hi"]
    new = [hi if lo == hi else _spread(r, lo, hi) for _ in range(case["seqs"])]
    past = [case["past"] and r.randrange(0, case["past"] + 1) for _ in new]
    return new, past


def work(case):
    H, KV, D = case["heads"], case["kv_heads"], case["dim"]
    new, past = lengths(case)
    n = sum(new)
    row = KV * 2 * (D // 2 + D // 64 * 4)  # cached bytes of a token
    if case["op"] == "append":  # q, k, v, cos and sin, slot and position in; rotated q and k and the cache out; read back
        moved = 2 * D * (H + 2 * KV) + 4 * case["rotary"] + 12 + 2 * D * (H + KV) + row + row + 4 * D * KV
        return {"bytes": n * moved, "flops": n * D * (3 * H + 13 * KV)}
    if case["op"] == "gather":
        return {"bytes": n * (row + 4 * D * KV), "flops": n * 4 * D * KV}
    if case["op"] == "decode":
        pages = sum(-(-x // case["page"]) for x in new)
        return {"bytes": n * row + 4 * D * H * len(new) + 4 * pages, "flops": n * 4 * D * H}
    pairs = sum(a * (a + 1) // 2 + a * b for a, b in zip(new, past))
    return {"bytes": 4 * D * H * n + 4 * D * KV * (n + sum(past)), "flops": pairs * 4 * D * H}


# ---------------------------------------------------------------- inputs
def _pages(case, counts, gen):
    """A page table over shuffled pages: int32 [seqs][most pages], and the number of pages."""
    need = [-(-c // case["page"]) for c in counts]
    order = torch.randperm(sum(need), generator=gen, device=DEV).to(torch.int32)
    table = torch.full((len(need), max(need)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for i, m in enumerate(need):
        table[i, :m] = order[at:at + m]
        at += m
    return table, at


def _spans(counts):
    cu = [0]
    for c in counts:
        cu.append(cu[-1] + c)
    return torch.tensor(cu, dtype=torch.int32, device=DEV)


def _tile_bytes(D):
    return TILE * (D + D // 64 * 8)


def _cached(case, pages, gen):
    """A filled cache, uint8 [pages][kv_heads][tiles][tile bytes]: a tile is 16 key code rows, 16 value
    code rows, then 16 rows of (scale, bias) words of the keys and of the values.  Word j*(D/64) + n of
    a code row holds channels 64n + 8j .. 64n + 8j + 7, the first in its lowest bits."""
    KV, D, P = case["kv_heads"], case["dim"], case["page"]
    n = D // 64
    cache = torch.empty(pages, KV, P // TILE, _tile_bytes(D), dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 26) // (KV * P * D))
    for a in range(0, pages, step):
        b = min(pages, a + step)
        shape = (b - a, KV, P // TILE, TILE, n, 64)
        out = []
        for _ in range(2):
            c, s, bias = _quantise(torch.randn(shape, generator=gen, device=DEV).to(torch.bfloat16).float())
            c = c.to(torch.uint8).view(*shape[:4], n, 8, 4, 2)
            c = (c[..., 0] | (c[..., 1] << 4)).transpose(-2, -3).reshape(*shape[:3], -1)
            sb = torch.stack([s, bias], -1).to(torch.bfloat16).reshape(*shape[:3], -1).view(torch.uint8)
            out.append((c, sb))
        cache[a:b] = torch.cat([out[0][0], out[1][0], out[0][1], out[1][1]], -1)
    return cache


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    H, KV, D, P = case["heads"], case["kv_heads"], case["dim"], case["page"]
    new, past = lengths(case)
    n, op = sum(new), case["op"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=DEV).to(torch.bfloat16)

    def empty(*shape):
        return torch.empty(shape, dtype=torch.bfloat16, device=DEV)

    s = {"case": case, "scale": D ** -0.5}
    if op == "append":
        R = case["rotary"]
        table, pages = _pages(case, [a + b for a, b in zip(new, past)], gen)
        at = torch.cat([torch.arange(b, a + b, device=DEV) for a, b in zip(new, past)])
        seq = torch.repeat_interleave(torch.arange(len(new), device=DEV), torch.tensor(new, device=DEV))
        far = torch.arange(max(a + b for a, b in zip(new, past)), device=DEV, dtype=torch.float64)
        angle = far[:, None] * THETA ** (-torch.arange(0, R, 2, device=DEV, dtype=torch.float64) / R)
        qkv = normal(n, H + 2 * KV, D)  # one fused projection's output: strided views
        s |= {"q": qkv[:, :H], "k": qkv[:, H:H + KV], "v": qkv[:, H + KV:],
              "rope": torch.stack([angle.cos(), angle.sin()], 1).float().contiguous(),  # [position][cos, sin][R/2]
              "positions": at.to(torch.int32),
              "slots": table[seq, at // P].long() * P + at % P, "table": table,
              "first": torch.tensor(past, dtype=torch.int32, device=DEV), "cu": _spans(new),
              "cache": torch.zeros(pages, KV, P // TILE, _tile_bytes(D), dtype=torch.uint8, device=DEV),
              "q_out": empty(n, H, D), "k_out": empty(n, KV, D), "kc": empty(n, KV, D), "vc": empty(n, KV, D)}
    elif op in ("gather", "decode"):
        table, pages = _pages(case, new, gen)
        s |= {"table": table, "cache": _cached(case, pages, gen)}
        if op == "gather":
            s |= {"cu": _spans(new), "kc": empty(n, KV, D), "vc": empty(n, KV, D)}
        else:
            s |= {"q": normal(len(new), H, D) * 2, "lens": torch.tensor(new, dtype=torch.int32, device=DEV),
                  "out": empty(len(new), H, D), "workspace": torch.zeros(32 << 20, dtype=torch.uint8, device=DEV)}
    else:
        keys = sum(past) + n
        s |= {"q": normal(n, H, D) * 2, "k": normal(keys, KV, D), "v": normal(keys, KV, D), "cu_q": _spans(new),
              "cu_k": _spans([a + b for a, b in zip(new, past)]), "out": empty(n, H, D)}
    return s


# ---------------------------------------------------------------- the plain forms
def _quantise(x):
    """Codes, scales and biases of groups of 64 (the last axis), fp32 holding bf16 values."""
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    s = ((hi * 0.5 - lo * 0.5) / 7.5).to(torch.bfloat16).float()
    c = torch.where(s > 0, torch.round((x * 0.5 - lo * 0.5) / (s * 0.5)), 0.0).clamp(0, 15)
    return c, s.squeeze(-1), lo.squeeze(-1)


def _as_cached(x):
    """The values that a cache stands for after x (bf16 [tokens][kv_heads][D]) went into it."""
    g = x.float().view(*x.shape[:-1], -1, 64)
    c, s, b = _quantise(g)
    return (s[..., None] * c + b[..., None]).view(x.shape).to(torch.bfloat16)


def _rotated(x, cos, sin):
    R = 2 * cos.shape[-1]
    x = x.float()
    a, b, rest = x[..., :R // 2], x[..., R // 2:R], x[..., R:]
    c, s = cos[:, None], sin[:, None]
    return torch.cat([a * c - b * s, b * c + a * s, rest], -1).to(torch.bfloat16)


def _values(state):
    """Keys and values of every slot of the table's pages, fp32 [seqs][kv_heads][tokens][D]."""
    case = state["case"]
    KV, D, n = case["kv_heads"], case["dim"], case["dim"] // 64
    t = state["cache"][state["table"].clamp(min=0).long()]  # [seqs][pages][kv][tiles][bytes]
    t = t.permute(0, 2, 1, 3, 4).reshape(t.shape[0], KV, -1, t.shape[-1])
    half, words = TILE * D // 2, TILE * n * 4
    out = []
    for codes, sb in ((t[..., :half], t[..., 2 * half:2 * half + words]), (t[..., half:2 * half], t[..., 2 * half + words:])):
        c = torch.stack([codes & 15, codes >> 4], -1).view(*t.shape[:3], TILE, 8, n, 8).transpose(-2, -3).float()
        sb = sb.contiguous().view(torch.bfloat16).view(*t.shape[:3], TILE, n, 1, 1, 2).float()
        out.append((c * sb[..., 0] + sb[..., 1]).reshape(t.shape[0], KV, -1, D))
    return out


def _softmax(scores, seen):
    """Softmax over the last axis where `seen`; rows that see nothing are zeros."""
    scores = torch.where(seen, scores, -math.inf)
    m = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(m == -math.inf, 0.0, m))
    return p / p.sum(-1, keepdim=True).clamp(min=1e-30)


def _of_spans(cu, n):
    """Each packed row's sequence and place in it."""
    at = torch.arange(n, device=cu.device)
    seq = torch.searchsorted(cu[1:].long(), at, right=True)
    return seq, at - cu[seq]


def run(state):
    if own:
        return _run_own(state)
    case = state["case"]
    KV, D = case["kv_heads"], case["dim"]
    G = case["heads"] // KV
    if case["op"] == "append":
        cs = state["rope"][state["positions"].long()]
        q, k = (_rotated(state[x], cs[:, 0], cs[:, 1]) for x in "qk")
        return {"q": q, "k": k, "kc": _as_cached(k), "vc": _as_cached(state["v"])}
    if case["op"] == "gather":
        k, v = _values(state)
        seq, at = _of_spans(state["cu"], state["kc"].shape[0])
        return {"kc": k[seq, :, at].to(torch.bfloat16), "vc": v[seq, :, at].to(torch.bfloat16)}
    if case["op"] == "decode":
        k, v = _values(state)
        q = state["q"].float().view(-1, KV, G, D) * state["scale"]
        seen = torch.arange(k.shape[2], device=DEV) < state["lens"][:, None, None, None]
        return (_softmax(q @ k.transpose(-1, -2), seen) @ v).to(torch.bfloat16).view(-1, KV * G, D)
    q, k, v = (state[x].float() for x in "qkv")
    n, keys = q.shape[0], k.shape[0]
    (sq, iq), (sk, ik) = _of_spans(state["cu_q"], n), _of_spans(state["cu_k"], keys)
    more = (state["cu_k"].diff() - state["cu_q"].diff())[sq]
    seen = (sq[:, None] == sk) & (ik <= (iq + more)[:, None])
    q = q.view(n, KV, G, D).permute(1, 2, 0, 3).reshape(KV, G * n, D) * state["scale"]
    p = _softmax((q @ k.permute(1, 2, 0)).view(KV, G, n, keys), seen).view(KV, G * n, keys)
    return (p @ v.transpose(0, 1)).view(KV, G, n, D).permute(2, 0, 1, 3).reshape(n, KV * G, D).to(torch.bfloat16)


# ---------------------------------------------------------------- the library's calls
_attn = None


def _run_own(s):
    global _attn
    if _attn is None:
        from bit_dequant_expert_softmax_b200 import attn as _attn
    case = s["case"]
    cfg = s.get("cfg")
    if cfg is None:
        cfg = s["cfg"] = _attn.fmoe_attn_config(case["heads"], case["kv_heads"], case["dim"], case["page"])
    if case["op"] == "append":
        _attn.fmoe_kv_append(cfg, s["q"], s["k"], s["v"], s["rope"], s["positions"], s["slots"], s["cache"], s["q_out"],
                             s["k_out"])
        _attn.fmoe_kv_gather(cfg, s["cache"], s["table"], s["cu"], s["kc"], s["vc"], first=s["first"])
        return {"q": s["q_out"], "k": s["k_out"], "kc": s["kc"], "vc": s["vc"]}
    if case["op"] == "gather":
        _attn.fmoe_kv_gather(cfg, s["cache"], s["table"], s["cu"], s["kc"], s["vc"])
        return {"kc": s["kc"], "vc": s["vc"]}
    if case["op"] == "decode":
        _attn.fmoe_attn_decode(cfg, s["q"], s["cache"], s["table"], s["lens"], s["out"], s["scale"], s["workspace"])
        return s["out"]
    _attn.fmoe_attn_prompt(cfg, s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], s["out"], s["scale"])
    return s["out"]


# ---------------------------------------------------------------- the definition in 64 bits
def _unpack64(s, page, head):
    """One page's keys and values of one head, fp64 [page tokens][D], word by word."""
    D = s["case"]["dim"]
    n = D // 64
    tiles = s["cache"][page, head].contiguous()
    words = tiles.view(torch.int32).long() & 0xFFFFFFFF
    per = TILE * D // 8
    found = []
    for i in range(2):
        w = words[..., i * per:(i + 1) * per].reshape(*words.shape[:-1], TILE, 8, n)
        sb = words[..., 2 * per + i * TILE * n:2 * per + (i + 1) * TILE * n].reshape(*words.shape[:-1], TILE, n)
        low, high = ((x & 0xFFFF).to(torch.int32) << 16 for x in (sb, sb >> 16))
        scale, bias = (x.view(torch.float32).double() for x in (low, high))
        ch = [((w >> 4 * b) & 15).double() for b in range(8)]
        x = torch.stack(ch, -1).movedim(-2, -3)  # [..., token, n, word, code]
        found.append((x * scale[..., None, None] + bias[..., None, None]).reshape(-1, D))
    return found


def _attend64(q, k, v, scale, seen=None):
    a = (q @ k.T) * scale
    if seen is not None:
        a = a.masked_fill(~seen, -math.inf)
    return torch.nan_to_num(torch.softmax(a, -1), nan=0.0) @ v


def exact(case, seed):
    s = prepare(case, seed)
    H, KV, D = case["heads"], case["kv_heads"], case["dim"]
    G = H // KV
    new, past = lengths(case)
    if case["op"] == "append":
        cs = s["rope"].double()[s["positions"].long()]
        turn = torch.complex(cs[:, 0], cs[:, 1])[:, None]
        R = case["rotary"]
        out = {"kc": None, "vc": None}
        for x in "qk":
            y = s[x].double().clone()
            z = torch.complex(y[..., :R // 2], y[..., R // 2:R]) * turn
            y[..., :R // 2], y[..., R // 2:R] = z.real, z.imag
            out[x] = y
        return out
    if case["op"] in ("gather", "decode"):
        outs = {"kc": [], "vc": [], "o": []}
        for i, L in enumerate(new):
            pages = s["table"][i, :-(-L // case["page"])].long()
            both = [_unpack64(s, pages, h) for h in range(KV)]
            k, v = (torch.stack([b[j][:L] for b in both]) for j in range(2))
            if case["op"] == "gather":
                outs["kc"].append(k.transpose(0, 1))
                outs["vc"].append(v.transpose(0, 1))
            else:
                q = s["q"][i].double().view(KV, G, D)
                outs["o"].append(torch.cat([_attend64(q[h], k[h], v[h], s["scale"]) for h in range(KV)]))
        if case["op"] == "gather":
            return {"kc": torch.cat(outs["kc"]), "vc": torch.cat(outs["vc"])}
        return torch.stack(outs["o"])
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
    a = b = 0
    for nq, before in zip(new, past):
        nk = nq + before
        seen = torch.ones(nq, nk, dtype=torch.bool, device=DEV).tril(nk - nq)
        for h in range(H):
            out[a:a + nq, h] = _attend64(s["q"][a:a + nq, h].double(), s["k"][b:b + nk, h // G].double(),
                                         s["v"][b:b + nk, h // G].double(), s["scale"], seen)
        a, b = a + nq, b + nk
    return out
