"""The operators of the 4-bit key/value cache, as they are measured: the cases, their inputs, one pass, its work.

A cache row of D dims is D e2m1 codes (two a byte, the even dim in the low nibble) and one e4m3 scale for each 16
dims; a value is code * scale * tensor scale (a power of two, one for the keys and one for the values).

The operators (field "op" of a case):
  attend      attention of the last nq tokens of each sequence over its cache; with "mass", each slot's attention weight
              over the call's rows is added to an accumulator
  store_load  rows of keys and values stored in the cache and read back in bf16
  mass        the attention weight of each key of a prompt, summed over query rows, from the forward's log-sum-exp
  evict       the slots with the highest accumulated weight and the most recent ones moved to a smaller cache, and the
              rows that it then holds read back in bf16
"""
import math

import torch

own = False

BLOCK = 16
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one user's next token over a short context: all latency (7b heads in groups of 4, as the grouped 128K workload)
        {"name": "attend_1k", "op": "attend", "B": 1, "H": 32, "Hkv": 8, "D": 128, "nq": 1, "cap": 1024, "ragged": False, "mass": False},
        # a serving batch with the skewed document lengths of the packed workload
        {"name": "attend_batch", "op": "attend", "B": 48, "H": 32, "Hkv": 8, "D": 128, "nq": 1, "cap": 33120, "ragged": True, "mass": False},
        # five tokens at once (drafted tokens checked together), 64 dims, an odd number of slots in use
        {"name": "attend_verify", "op": "attend", "B": 8, "H": 32, "Hkv": 4, "D": 64, "nq": 5, "cap": 4112, "ragged": True, "mass": False},
        # one user at 128K tokens, weights accumulated for a later eviction
        {"name": "attend_128k_mass", "op": "attend", "B": 1, "H": 32, "Hkv": 8, "D": 128, "nq": 1, "cap": 131072, "ragged": False, "mass": True},
        # one user at 1M tokens, the 13b workload's 40 heads in groups of 5
        {"name": "attend_1m", "op": "attend", "B": 1, "H": 40, "Hkv": 8, "D": 128, "nq": 1, "cap": 1048576, "ragged": False, "mass": False},
        # a decode step's new rows, one for each of 64 sequences
        {"name": "append_64", "op": "store_load", "B": 64, "Hkv": 8, "D": 128, "T": 1, "cap": 2048, "packed": False},
        # a prompt chunk of 16K tokens with 32 heads, read back for the next chunk
        {"name": "chunk_16k", "op": "store_load", "B": 1, "Hkv": 32, "D": 128, "T": 16384, "cap": 32768, "packed": False},
        # packed prompts of different lengths, 80 dims
        {"name": "packed_80", "op": "store_load", "B": 16, "Hkv": 8, "D": 80, "T": 40007, "cap": 8192, "packed": True},
        # the weight of every key of an 8K prompt with the 7b heads
        {"name": "mass_8k", "op": "mass", "H": 32, "Hkv": 32, "D": 128, "T": 8192, "window": 8192, "docs": 1},
        # a 128K prompt judged by its last 64 queries, grouped heads
        {"name": "mass_128k_window", "op": "mass", "H": 32, "Hkv": 8, "D": 128, "T": 131072, "window": 64, "docs": 1},
        # a 128K prompt cut to 4096 slots
        {"name": "evict_128k", "op": "evict", "B": 1, "Hkv": 8, "D": 128, "cap": 131072, "keep": 4096, "recent": 64, "ragged": False},
        # a serving batch cut back to 2048 slots after 128 tokens more
        {"name": "evict_batch", "op": "evict", "B": 48, "Hkv": 8, "D": 128, "cap": 2176, "keep": 2048, "recent": 256, "ragged": True},
    ]


def draw(rng):
    def spread(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(("attend", "attend", "store_load", "mass", "evict"))
    D = rng.choice((40, 64, 80, 96, 128, 128, 128, 256))
    Hkv = rng.choice((1, 2, 3, 4, 8))
    G = rng.choice((1, 2, 4, 5, 8))
    if op == "mass":
        T = spread(100, 12000)
        window = T if rng.random() < 0.5 else min(T, spread(1, 500))
        Hkv = min(Hkv, 4)
        return {"op": op, "H": Hkv * G, "Hkv": Hkv, "D": D, "T": T, "window": window,
                "docs": rng.choice((1, 1, 2, 5)) if window == T else 1}
    B = spread(1, 64)
    nq = rng.choice((1, 1, 1, 2, 3, 7, 16))
    top = max(64, min(262144, (1 << 30) // (B * Hkv * D), (1 << 27) // (B * Hkv * G * nq)))
    cap = (spread(48, top) + 15) // 16 * 16
    if op == "attend":
        return {"op": op, "B": B, "H": Hkv * G, "Hkv": Hkv, "D": D, "nq": nq,
                "cap": cap, "ragged": rng.random() < 0.6, "mass": rng.random() < 0.4}
    if op == "store_load":
        packed = rng.random() < 0.4
        cap = min(cap, 32768)
        T = spread(B, min(B * cap // 2, 60000)) if packed else spread(1, max(1, min(cap - 1, 60000 // B)))
        return {"op": op, "B": B, "Hkv": Hkv, "D": D, "T": T, "cap": cap, "packed": packed}
    keep = max(2, int(cap * rng.uniform(0.02, 0.95)))
    return {"op": op, "B": B, "Hkv": Hkv, "D": D, "cap": cap, "keep": keep, "recent": rng.randint(0, keep // 2),
            "ragged": rng.random() < 0.6}


# ------------------------------------------------------------------ inputs

def _gen(seed, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return g


def _rows(shape, g):
    """Keys or values in bf16: normal draws, with dims of different size, as trained heads have them."""
    size = torch.exp(0.5 * torch.randn(shape[-1], device="cuda", generator=g))
    return (torch.randn(shape, device="cuda", generator=g, dtype=torch.bfloat16) * size.bfloat16())


def _lengths(B, cap, lo, ragged, seed):
    """Used slots of each sequence: lognormal about a third of the capacity, clipped to [lo, cap]; or all in use but one."""
    if not ragged:
        return [max(lo, cap - 1)] * B
    x = torch.randn(B, generator=_gen(seed, "cpu"))
    return [max(lo, min(cap, int(cap / 3 * math.exp(1.0 * float(v))))) for v in x]


def _quantise(x, ts):
    """Codes 0..15 (sign in bit 3) and e4m3 scales of the last dim in blocks of 16, by the format's rounding to nearest even."""
    D = x.shape[-1]
    pad = (-D) % BLOCK
    f = torch.nn.functional.pad(x.float(), (0, pad)).unflatten(-1, (-1, BLOCK))
    six = torch.tensor(6.0 * ts, device=x.device)
    s8 = (f.abs().amax(-1) / six).clamp(max=448.0).to(torch.float8_e4m3fn)
    d = s8.float().unsqueeze(-1) * ts
    y = (f.abs() / d).where(d > 0, torch.zeros((), device=x.device))
    c = ((y > 0.25).to(torch.uint8) + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5) + (y > 5.0))
    c = (c | (torch.signbit(f).to(torch.uint8) << 3)).flatten(-2)[..., :D]
    return c, s8


def _packed_cache(B, Hkv, cap, D, ts, g):
    c, s = _quantise(_rows((B, Hkv, cap, D), g), ts)
    return c[..., 0::2] | (c[..., 1::2] << 4), s.view(torch.uint8)


def prepare(case, seed):
    g = _gen(seed)
    op, D = case["op"], case["D"]
    st = {"case": case, "levels": torch.tensor(LEVELS + tuple(-v for v in LEVELS), device="cuda"), "k_ts": 0.5, "v_ts": 1.0}
    if op == "mass":
        H, Hkv, T, w = case["H"], case["Hkv"], case["T"], case["window"]
        cuts = sorted({0, T} | set(torch.randint(1, max(2, T), (case["docs"] - 1,), generator=_gen(seed, "cpu")).tolist()))
        st["chunks"] = [(max(a, T - w), b, a, 0) for a, b in zip(cuts, cuts[1:])]
        st["ctx"] = torch.cat([torch.full((b - a,), a) for a, b in zip(cuts, cuts[1:])]).cuda()
        st["q"] = 2.0 * torch.randn((1, H, T, D), device="cuda", generator=g, dtype=torch.bfloat16)
        st["k"] = _rows((1, Hkv, T, D), g)
        st["lse"] = torch.zeros((1, H, T), device="cuda")
        st["r0"] = T - w
        t = torch.arange(T, device="cuda")
        seen = (t[None, :] <= t[T - w:, None]) & (t[None, :] >= st["ctx"][T - w:, None])
        for h in range(H):
            s = st["q"][0, h, T - w:].float() @ st["k"][0, h * Hkv // H].float().T / math.sqrt(D)
            st["lse"][0, h, T - w:] = torch.logsumexp(s.masked_fill_(~seen, -math.inf), -1)
        return st
    B, Hkv, cap = case["B"], case["Hkv"], case["cap"]
    if op == "store_load":
        if case["packed"]:
            share = torch.exp(torch.randn(B, generator=_gen(seed, "cpu")))
            n = torch.clamp((share / share.sum() * case["T"]).long(), max=cap - 1)
            short = case["T"] - int(n.sum())
            for b in range(B):                       # the rest goes where there is room
                more = min(short, cap - 1 - int(n[b]))
                n[b] += more
                short -= more
            st["lens"] = n.tolist()
            cu = [0] + torch.cumsum(n, 0).tolist()
            st["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
            st["k"], st["v"] = (_rows((cu[-1], Hkv, D), g) for _ in range(2))
            room = cap - n
        else:
            st["k"], st["v"] = (_rows((B, Hkv, case["T"], D), g) for _ in range(2))
            room = torch.full((B,), cap - case["T"])
        pos = (torch.rand(B, generator=_gen(seed + 1, "cpu")) * room).long()
        st["pos"] = pos.to(torch.int32).cuda()
        st["cache"] = [torch.zeros((B, Hkv, cap, n), dtype=torch.uint8, device="cuda") for n in (D // 2, -(-D // BLOCK)) * 2]
        return st
    lens = _lengths(B, cap, case.get("nq", 1), case["ragged"], seed)
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    st["cache"] = list(_packed_cache(B, Hkv, cap, D, st["k_ts"], g)) + list(_packed_cache(B, Hkv, cap, D, st["v_ts"], g))
    # accumulated weights: a few slots hold most of it
    if op == "evict" or case["mass"]:
        st["mass"] = torch.exp(2.0 * torch.randn((B, Hkv, cap), device="cuda", generator=g))
    if op == "attend":
        st["q"] = 2.0 * torch.randn((B, case["H"], case["nq"], D), device="cuda", generator=g, dtype=torch.bfloat16)
        if case["mass"]:
            st["mass_out"] = torch.zeros_like(st["mass"])
    else:
        keep = case["keep"]
        small = (keep + 15) // 16 * 16
        st["out"] = [torch.zeros((B, Hkv, small, n), dtype=torch.uint8, device="cuda") for n in (D // 2, -(-D // BLOCK)) * 2]
        st["mass_out"] = torch.zeros((B, Hkv, small), device="cuda")
        st["begin"] = torch.zeros(B, dtype=torch.int32, device="cuda")
    return st


# ------------------------------------------------------------------ plain forms

def _values(st, codes, scales, ts):
    """The values that packed codes and scales stand for, in 32 bits."""
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).int()
    s = scales.view(torch.float8_e4m3fn).float() * ts
    return st["levels"][c] * s.repeat_interleave(BLOCK, -1)[..., :c.shape[-1]]


def _plain_attend(st):
    c = st["case"]
    B, H, Hkv, nq, cap, D = (c[n] for n in ("B", "H", "Hkv", "nq", "cap", "D"))
    k = _values(st, st["cache"][0], st["cache"][1], st["k_ts"])
    v = _values(st, st["cache"][2], st["cache"][3], st["v_ts"])
    q = st["q"].float().view(B, Hkv, H // Hkv * nq, D)
    s = (q @ k.transpose(-1, -2)).view(B, Hkv, H // Hkv, nq, cap) / math.sqrt(D)
    last = st["lens"].long()[:, None] - nq + torch.arange(nq, device="cuda")             # [B, nq]
    seen = torch.arange(cap, device="cuda") <= last[:, None, None, :, None]
    s = s.masked_fill(~seen, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - top)
    total = p.sum(-1, keepdim=True)
    p = p / total
    o = (p.view(B, Hkv, -1, cap) @ v).view(B, H, nq, D).to(torch.bfloat16)
    lse = (top + torch.log(total)).view(B, H, nq)
    if not c["mass"]:
        return o, lse
    used = (torch.arange(cap, device="cuda") < st["lens"][:, None])[:, None]
    return o, lse, torch.where(used, st["mass"] + p.sum((2, 3)), st["mass_out"])


def _plain_store_load(st):
    out = []
    for x, ts in ((st["k"], st["k_ts"]), (st["v"], st["v_ts"])):
        code, s8 = _quantise(x, ts)
        d = (s8.float() * ts).repeat_interleave(BLOCK, -1)[..., :code.shape[-1]]
        out.append((st["levels"][code.int()] * d).to(torch.bfloat16))
    return out


def _plain_mass(st):
    c = st["case"]
    H, Hkv, T, D, r0 = c["H"], c["Hkv"], c["T"], c["D"], st["r0"]
    q = st["q"][0, :, r0:].float().view(Hkv, -1, D)
    s = (q @ st["k"][0].float().transpose(-1, -2)).view(Hkv, H // Hkv, T - r0, T)
    t = torch.arange(T, device="cuda")
    seen = (t <= t[r0:, None]) & (t >= st["ctx"][r0:, None])
    w = torch.exp(s / math.sqrt(D) - st["lse"][0, :, r0:].view(Hkv, H // Hkv, T - r0, 1))
    return (w * seen).sum((1, 2))[None]


def _plain_evict(st):
    c = st["case"]
    B, Hkv, cap, keep, D = c["B"], c["Hkv"], c["cap"], c["keep"], c["D"]
    lens = st["lens"].long()
    n = torch.clamp(lens, max=keep)
    slot = torch.arange(cap, device="cuda")
    recent = torch.minimum(n, torch.full_like(n, c["recent"]))
    rank = torch.where(slot >= (lens - recent)[:, None], math.inf, 0.0)[:, None] + st["mass"]
    rank = torch.where((slot < lens[:, None])[:, None], rank, -math.inf)
    order = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :keep]
    row = torch.arange(keep, device="cuda")
    there = (row < n[:, None])[:, None].expand(B, Hkv, keep)
    order = torch.sort(torch.where(there, order, cap), dim=-1).values
    at = torch.where(there, order, 0)[..., None]
    kv = [_values(st, st["cache"][i].gather(2, at.expand(-1, -1, -1, st["cache"][i].shape[-1])),
                  st["cache"][i + 1].gather(2, at.expand(-1, -1, -1, st["cache"][i + 1].shape[-1])), ts)
          for i, ts in ((0, st["k_ts"]), (2, st["v_ts"]))]
    kv = [torch.where(there[..., None], x, 0.0).to(torch.bfloat16) for x in kv]
    mass = st["mass_out"].clone()
    mass[..., :keep] = torch.where(there, st["mass"].gather(2, at[..., 0]), mass[..., :keep])
    return n.to(torch.int32), torch.where(there, order, -1).to(torch.int32), mass, kv[0], kv[1]


# ------------------------------------------------------------------ one pass

def _handles(st):
    """What a user's program sets up once: the cache handles and the workspace."""
    import chunked_causal_attention_gb300 as cca
    D = st["case"]["D"]
    st["handle"] = cca.KV4Cache(*st["cache"], D=D, k_scale=st["k_ts"], v_scale=st["v_ts"])
    if "out" in st:
        st["small"] = cca.KV4Cache(*st["out"], D=D, k_scale=st["k_ts"], v_scale=st["v_ts"])
    st["ws"] = cca.kv4_workspace(st["handle"], q=st.get("q"), mass="mass" in st)


def run(state):
    c = state["case"]
    op = c["op"]
    if not own:
        return {"attend": _plain_attend, "store_load": _plain_store_load, "mass": _plain_mass, "evict": _plain_evict}[op](state)
    import chunked_causal_attention_gb300 as cca
    if op == "mass":
        if "ws" not in state:
            state["ws"] = cca.key_mass_workspace(state["q"], state["k"], state["chunks"])
        return cca.key_mass(state["q"], state["k"], state["lse"], state["chunks"], ws=state["ws"])
    if "handle" not in state:
        _handles(state)
    cache, ws = state["handle"], state["ws"]
    if op == "attend":
        if not c["mass"]:
            return cca.kv4_attention(state["q"], cache, state["lens"], ws=ws)
        o, lse = cca.kv4_attention(state["q"], cache, state["lens"], mass_in=state["mass"], mass_out=state["mass_out"], ws=ws)
        return o, lse, state["mass_out"]
    if op == "store_load":
        cu = state.get("cu")
        cca.kv4_store(cache, state["k"], state["v"], state["pos"], cu_seqlens=cu, ws=ws)
        return list(cca.kv4_load(cache, state["pos"], state["k"].shape[0 if c["packed"] else 2], cu_seqlens=cu, ws=ws))
    lens, slots = cca.kv4_evict(cache, state["lens"], state["mass"], c["keep"], c["recent"], state["small"], state["mass_out"], ws=ws)
    k, v = cca.kv4_load(state["small"], state["begin"], c["keep"], ws=ws)
    return lens, slots, state["mass_out"], k, v


def work(case):
    D, op = case["D"], case["op"]
    row = 2 * (D // 2 + -(-D // BLOCK))                      # bytes of a cached key and value
    if op == "mass":
        H, Hkv, T, w = case["H"], case["Hkv"], case["T"], case["window"]
        pairs = w * (2 * T - w + 1) // 2 // (case["docs"] if w == T else 1)
        return {"bytes": H * w * (2 * D + 4) + Hkv * T * (2 * D + 4), "flops": 2 * D * H * pairs}
    B, Hkv, cap = case["B"], case["Hkv"], case["cap"]
    if op == "store_load":
        rows = Hkv * (case["T"] if case["packed"] else B * case["T"])
        return {"bytes": rows * (8 * D + row), "flops": 6 * D * rows}
    n = B * cap * (0.45 if case["ragged"] else 1.0)          # slots in use, about
    if op == "attend":
        H, nq = case["H"], case["nq"]
        return {"bytes": int(n * Hkv * (row + (8 if case["mass"] else 0)) + B * H * nq * (4 * D + 4)), "flops": int(4 * D * H * nq * n)}
    kept = Hkv * min(B * case["keep"], n)
    return {"bytes": int(4 * Hkv * n + kept * (2 * row + 12 + 4 * D)), "flops": int(Hkv * n)}


# ------------------------------------------------------------------ 64 bits

def _power64(e):
    """2^e for whole e in -64..63, exactly (pow is not exact to the last bit on every device)."""
    return torch.tensor([2.0 ** i for i in range(-64, 64)], dtype=torch.float64, device=e.device)[e.long() + 64]


def _decode64(codes, scales, ts, D):
    """Values of packed rows in 64 bits, from the bit fields: e2m1 codes (bias 1) and e4m3 scales (bias 7)."""
    out = torch.empty(codes.shape[:-1] + (D,), dtype=torch.float64, device=codes.device)
    for half in (0, 1):
        c = (codes >> (4 * half)).to(torch.float64) % 16
        neg = c >= 8
        c = c - 8 * neg
        e, m = torch.floor(c / 2), c % 2
        mag = torch.where(e > 0, (1 + m / 2) * _power64(e - 1), m / 2)
        out[..., half::2] = torch.where(neg, -mag, mag)
    b = scales.to(torch.float64)
    e, m = torch.floor(b / 8) % 16, b % 8
    s = torch.where(e > 0, (1 + m / 8) * _power64(e - 7), m * 2.0 ** -9) * ts
    for i in range(s.shape[-1]):
        out[..., i * BLOCK:(i + 1) * BLOCK] *= s[..., i:i + 1]
    return out


def _grid64(x, mantissa, lowest, largest):
    """x >= 0 rounded to nearest even on a floating grid: `mantissa` fraction bits, exponents from `lowest`, at most `largest`."""
    e = torch.clamp(torch.frexp(x).exponent - 1, min=lowest)
    step = _power64(e - mantissa)
    return torch.clamp(torch.round(x / step) * step, max=largest)


def _stored64(x, ts):
    """What a stored row stands for, from the definition: blocks of 16, scale and codes rounded to nearest even."""
    x = x.double()
    out = torch.empty_like(x)
    for a in range(0, x.shape[-1], BLOCK):
        part = x[..., a:a + BLOCK]
        s = _grid64(part.abs().amax(-1, keepdim=True) / 6 / ts, 3, -6, 448.0) * ts
        y = torch.where(s > 0, part.abs() / s, torch.zeros_like(part))
        out[..., a:a + BLOCK] = torch.sign(part) * _grid64(y, 1, 0, 6.0) * s
    return out


def exact(case, seed):
    st = prepare(case, seed)
    op, D = case["op"], case["D"]
    if op == "store_load":
        return [_stored64(st["k"], st["k_ts"]), _stored64(st["v"], st["v_ts"])]
    if op == "mass":
        H, G, T, r0 = case["H"], case["H"] // case["Hkv"], case["T"], st["r0"]
        mass = torch.zeros((1, case["Hkv"], T), dtype=torch.float64, device="cuda")
        for a, b, ctx, _ in st["chunks"]:
            causal = torch.ones((b - a, b - ctx), dtype=torch.bool, device="cuda").tril(a - ctx)
            for h in range(H):
                s = st["q"][0, h, a:b].double() @ st["k"][0, h // G, ctx:b].double().T * D ** -0.5
                mass[0, h // G, ctx:b] += torch.exp(s - st["lse"][0, h, a:b, None].double())[...].mul_(causal).sum(0)
        return mass
    B, Hkv, lens = case["B"], case["Hkv"], st["lens"].tolist()
    kc, ks, vc, vs = st["cache"]
    if op == "attend":
        H, nq = case["H"], case["nq"]
        G = H // Hkv
        o = torch.zeros((B, H, nq, D), dtype=torch.float64, device="cuda")
        lse = torch.full((B, H, nq), -math.inf, dtype=torch.float64, device="cuda")
        mass = st["mass_out"].double() if case["mass"] else None
        for b, n in enumerate(lens):
            for h in range(Hkv):
                k, v = (_decode64(c[b, h, :n], s[b, h, :n], ts, D) for c, s, ts in ((kc, ks, st["k_ts"]), (vc, vs, st["v_ts"])))
                s = st["q"][b, h * G:(h + 1) * G].double() @ k.T * D ** -0.5
                for i in range(nq):
                    s[:, i, n - nq + i + 1:] = -math.inf
                part = torch.logsumexp(s, -1)
                p = torch.exp(s - part[..., None])
                o[b, h * G:(h + 1) * G], lse[b, h * G:(h + 1) * G] = p @ v, part
                if case["mass"]:
                    mass[b, h, :n] = st["mass"][b, h, :n].double() + p.sum((0, 1))
        return (o, lse) if mass is None else (o, lse, mass)
    keep = case["keep"]
    slots = torch.full((B, Hkv, keep), -1, dtype=torch.int32, device="cuda")
    mass = st["mass_out"].double()
    k, v = (torch.zeros((B, Hkv, keep, D), dtype=torch.float64, device="cuda") for _ in range(2))
    for b, n in enumerate(lens):
        m = min(n, keep)
        r = min(case["recent"], m)
        for h in range(Hkv):
            w = st["mass"][b, h, :n - r].double()
            best = torch.sort(-w, stable=True).indices[:m - r]
            kept = torch.cat((torch.sort(best).values, torch.arange(n - r, n, device="cuda")))
            slots[b, h, :m] = kept.int()
            mass[b, h, :m] = st["mass"][b, h, kept].double()
            k[b, h, :m] = _decode64(kc[b, h, kept], ks[b, h, kept], st["k_ts"], D)
            v[b, h, :m] = _decode64(vc[b, h, kept], vs[b, h, kept], st["v_ts"], D)
    return torch.tensor([min(n, keep) for n in lens], dtype=torch.int32, device="cuda"), slots, mass, k, v
