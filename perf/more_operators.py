"""The operators of the paged key/value cache, as they are measured: the cases, their inputs, one pass, its work.

Keys and values lie in a pool of pages of `page` slots each, shared by all sequences; slot j of sequence b is slot
j % page of the page table[b][j // page], and a slot's number in the pool is page number * page + place in the page.

The operators (field "op" of a case):
  attend   attention of the newest tokens of each sequence, one or a chunk of many, over its pages
  store    rows of keys and values written to the slots that a slot map names
  reserve  slots for the next tokens of each sequence: pages taken from a stack of free ones, pages of ended sequences
           put back, block tables, lengths, offsets of the packed tokens and the slot map
"""
import math

import torch

own = False


def listed():
    return [
        # one user's next token over a short context: all latency (7b heads in groups of 4, as the grouped 128K workload)
        {"name": "next_1k", "op": "attend", "kind": "next", "B": 1, "H": 32, "Hkv": 8, "D": 128, "nq": 1, "cap": 1001, "page": 64, "ragged": False, "slots_first": False},
        # a serving batch's next tokens with the skewed document lengths of the packed workload, small pages
        {"name": "next_batch", "op": "attend", "kind": "next", "B": 48, "H": 32, "Hkv": 8, "D": 128, "nq": 1, "cap": 33120, "page": 16, "ragged": True, "slots_first": True},
        # one user at 1M tokens, the 13b workload's 40 heads in groups of 5
        {"name": "next_1m", "op": "attend", "kind": "next", "B": 1, "H": 40, "Hkv": 8, "D": 128, "nq": 1, "cap": 1048576, "page": 128, "ragged": False, "slots_first": False},
        # five tokens at once (drafted tokens checked together), 64 dims
        {"name": "verify", "op": "attend", "kind": "few", "B": 8, "H": 32, "Hkv": 4, "D": 64, "nq": 5, "cap": 4112, "page": 32, "ragged": True, "slots_first": False},
        # the last 2048 tokens of a 32K prompt, grouped heads
        {"name": "chunk_32k", "op": "attend", "kind": "chunk", "B": 1, "H": 32, "Hkv": 8, "D": 128, "nq": 2048, "cap": 32768, "page": 64, "ragged": False, "slots_first": False},
        # chunks of four prompts of different lengths, 32 heads of keys and values, 96 dims
        {"name": "chunks_mha", "op": "attend", "kind": "chunk", "B": 4, "H": 32, "Hkv": 32, "D": 96, "nq": 1500, "cap": 9000, "page": 128, "ragged": True, "slots_first": True},
        # one prompt's chunk among 23 users' next tokens
        {"name": "mixed", "op": "attend", "kind": "mixed", "B": 24, "H": 32, "Hkv": 8, "D": 128, "nq": 700, "cap": 8200, "page": 16, "ragged": True, "slots_first": False},
        # a decode step's new rows, one for each of 61 sequences in a batch padded to 64
        {"name": "rows_64", "op": "store", "Hkv": 8, "D": 128, "T": 64, "pad": 3, "page": 16, "pages": 2048, "slots_first": False},
        # a prompt chunk of 16K tokens with 32 heads
        {"name": "rows_16k", "op": "store", "Hkv": 32, "D": 128, "T": 16384, "pad": 0, "page": 64, "pages": 400, "slots_first": False},
        # one more token for each of 64 sequences
        {"name": "reserve_64", "op": "reserve", "B": 64, "page": 16, "max_pages": 2070, "T": 64, "ended": 0.0, "begun": 0.0, "tight": False},
        # 512 sequences, some ended, some that begin with their prompts
        {"name": "reserve_512", "op": "reserve", "B": 512, "page": 16, "max_pages": 2600, "T": 40007, "ended": 0.05, "begun": 0.05, "tight": False},
        # prompts of 128K tokens in all
        {"name": "reserve_128k", "op": "reserve", "B": 8, "page": 64, "max_pages": 2112, "T": 131072, "ended": 0.0, "begun": 1.0, "tight": False},
    ]


def draw(rng):
    def spread(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(("attend", "attend", "attend", "store", "reserve"))
    D = rng.choice((40, 64, 80, 96, 128, 128, 128, 256))
    Hkv = rng.choice((1, 2, 3, 4, 8))
    page = rng.choice((16, 16, 32, 64, 128, 256))
    first = rng.random() < 0.4
    if op == "attend":
        kind = rng.choice(("next", "next", "few", "chunk", "chunk", "mixed"))
        G = rng.choice((1, 2, 4, 5, 8))
        B = spread(1, 64) if kind == "next" else spread(1, 24) if kind in ("few", "mixed") else spread(1, 6)
        nq = 1 if kind == "next" else rng.randint(2, 16) if kind == "few" else spread(40, 2500)
        # what the plain form holds at once: scores of every head, keys of every head
        top = min(262144, (1 << 29) // (B * Hkv * D), (1 << 37) // (B * Hkv * G * nq * D))
        cap = spread(max(nq, 48), max(nq, 64, top))
        return {"op": op, "kind": kind, "B": B, "H": Hkv * G, "Hkv": Hkv, "D": D, "nq": nq, "cap": cap, "page": page,
                "ragged": rng.random() < 0.6, "slots_first": first}
    if op == "store":
        Hkv = rng.choice((1, 2, 3, 4, 8, 32))
        T = spread(1, min(60000, 60000 * 1024 // (Hkv * D)))
        return {"op": op, "Hkv": Hkv, "D": D, "T": T, "pad": rng.choice((0, 0, min(T - 1, 5), T // 7)), "page": page,
                "pages": -(-T // page) + spread(2, 300), "slots_first": first}
    B = spread(1, 700)
    T = B if rng.random() < 0.4 else max(B, spread(1, 131072))
    # no sequence's slots, at most T new ones among them, leave its table
    return {"op": op, "B": B, "page": page, "max_pages": -(-T // page) + spread(4, 600), "T": T,
            "ended": rng.choice((0.0, 0.05, 0.3)), "begun": rng.choice((0.0, 0.1, 1.0)), "tight": rng.random() < 0.25}


# ------------------------------------------------------------------ inputs

def _gen(seed, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return g


def _rows(shape, g):
    """Keys or values in bf16: normal draws, with dims of different size, as trained heads have them."""
    size = torch.exp(0.5 * torch.randn(shape[-1], device="cuda", generator=g))
    return torch.randn(shape, device="cuda", generator=g, dtype=torch.bfloat16) * size.bfloat16()


def _pool(case, pages, g):
    """A pool seen as [pages, Hkv, page, D], in memory that way or with a slot's heads next to each other. Every slot
    holds something: pages in use before still have their old rows."""
    Hkv, page, D = case["Hkv"], case["page"], case["D"]
    if case["slots_first"]:
        return [_rows((pages, page, Hkv, D), g).transpose(1, 2) for _ in range(2)]
    return [_rows((pages, Hkv, page, D), g) for _ in range(2)]


def _i32(x):
    return torch.as_tensor(x, dtype=torch.int32).cuda()


def _spread(B, lo, hi, ragged, cpu):
    """Lengths: lognormal about a third of hi, clipped to [lo, hi]; or all near hi."""
    if not ragged:
        return [hi] * B
    return [max(lo, min(hi, int(hi / 3 * math.exp(float(v))))) for v in torch.randn(B, generator=cpu)]


def _prepare_attend(case, seed):
    g, cpu = _gen(seed), _gen(seed + 1, "cpu")
    B, page = case["B"], case["page"]
    # a case's numbers of new tokens are the same for every seed, in another order
    if case["kind"] == "mixed":
        nq = [1] * (B - 1)
    else:
        nq = _spread(B - 1, 1, case["nq"], case["kind"] == "chunk" and case["ragged"], _gen(B, "cpu"))
    nq.append(case["nq"])
    nq = [nq[i] for i in torch.randperm(B, generator=cpu).tolist()]
    lens = [max(a, b) for a, b in zip(_spread(B, 1, case["cap"], case["ragged"], cpu), nq)]
    held = [-(-n // page) for n in lens]
    pages = sum(held) + 3
    order = torch.randperm(pages, generator=cpu).to(torch.int32)
    table = torch.full((B, max(held) + 1), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(held):
        table[b, :n] = order[at:at + n]
        at += n
    k, v = _pool(case, pages, g)
    cu = [0]
    for n in nq:
        cu.append(cu[-1] + n)
    q = 2.0 * torch.randn((cu[-1], case["H"], case["D"]), device="cuda", generator=g, dtype=torch.bfloat16)
    return {"case": case, "q": q, "k": k, "v": v, "table": table.cuda(), "lens": _i32(lens), "cu": _i32(cu), "most": (max(nq), max(lens))}


def _prepare_store(case, seed):
    g, cpu = _gen(seed), _gen(seed + 1, "cpu")
    page, T, pages = case["page"], case["T"], case["pages"]
    k, v = _pool(case, pages, g)
    rows = [_rows((T, case["Hkv"], case["D"]), g) for _ in range(2)]
    # slots of the pool but its last page, each once; a prompt's run of slots page by page. Padding has slot -1
    order = torch.randperm(pages - 1, generator=cpu)
    slots = (order[:, None] * page + torch.arange(page)).flatten()[:T].to(torch.int32)
    if case["pad"]:
        slots[T - case["pad"]:] = -1
    return {"case": case, "k": k, "v": v, "k_new": rows[0], "v_new": rows[1], "slots": slots.cuda()}


def _prepare_reserve(case, seed):
    B, page, most, T = case["B"], case["page"], case["max_pages"], case["T"]
    cpu = _gen(B, "cpu")                                         # a case's sequences are the same for every seed,
    u = torch.rand(B, generator=cpu)
    ended, begun = u < case["ended"], u > 1 - case["begun"]
    room = most * page - T
    lens = torch.clamp((room / 3 * torch.exp(torch.randn(B, generator=cpu))).long(), 1, room)
    lens[begun] = 0
    add = torch.where(ended, -1, 1)
    left = T - int((add > 0).sum())
    many = begun if bool(begun.any()) else ~ended                # who brings the other tokens
    if left > 0 and bool(many.any()):
        share = torch.exp(torch.randn(B, generator=cpu)) * many
        add = add + torch.where(many, (share / share.sum() * left).long(), 0)
    cpu = _gen(seed, "cpu")
    other = torch.randperm(B, generator=cpu)                     # in another order, with other pages
    lens, add, ended = lens[other], add[other], ended[other]
    held = -(-lens // page)
    need = torch.where(ended, 0, -(-(lens + add.clamp(min=0)) // page) - held)
    spare = int(need.sum()) // 2 if case["tight"] else int(need.sum()) + 7
    pages = int(held.sum()) + spare
    order = torch.randperm(pages, generator=cpu).to(torch.int32)
    table = torch.full((B, most), -1, dtype=torch.int32)
    there = torch.arange(most) < held[:, None]
    table[there] = order[:int(held.sum())]
    free = torch.full((pages,), -1, dtype=torch.int32)
    free[:spare] = order[int(held.sum()):]
    st = {"case": case, "add": _i32(add), "lens": _i32(lens), "table": table.cuda(), "free": free.cuda(), "n_free": _i32([spare])}
    # what the call writes, apart from what it reads, so that a pass can be made again
    st["lens_out"], st["n_free_out"] = torch.zeros_like(st["lens"]), torch.zeros_like(st["n_free"])
    return st


def prepare(case, seed):
    return {"attend": _prepare_attend, "store": _prepare_store, "reserve": _prepare_reserve}[case["op"]](case, seed)


# ------------------------------------------------------------------ plain forms

def _plain_attend(st):
    c = st["case"]
    B, H, Hkv, D, page = (c[n] for n in ("B", "H", "Hkv", "D", "page"))
    nq, n = st["most"]
    lens, cu = st["lens"].long(), st["cu"].long()
    new = cu[1:] - cu[:-1]
    at = st["table"][:, :-(-n // page)].long().clamp(min=0)
    k, v = (x[at].permute(0, 2, 1, 3, 4).flatten(2, 3).float() for x in (st["k"], st["v"]))       # [B, Hkv, slots, D]
    i = torch.arange(nq, device="cuda")
    tok = (cu[:-1, None] + torch.minimum(i, new[:, None] - 1).clamp(min=0)).clamp(max=st["q"].shape[0] - 1)
    q = st["q"][tok].float().view(B, nq, Hkv, H // Hkv, D).permute(0, 2, 3, 1, 4).flatten(2, 3)
    s = (q @ k.transpose(-1, -2)).view(B, Hkv, H // Hkv, nq, -1).mul_(1 / math.sqrt(D))
    last = lens[:, None] - new[:, None] + i                                                       # [B, nq]
    seen = torch.arange(k.shape[2], device="cuda") <= last[:, :, None]
    s.masked_fill_(~seen[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    s.sub_(top).exp_()
    total = s.sum(-1, keepdim=True)
    o = (s.flatten(2, 3) @ v).view(B, Hkv, H // Hkv, nq, D) / total
    lse = (top + torch.log(total))[..., 0]
    # back to the packed order
    t = torch.arange(st["q"].shape[0], device="cuda")
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, nq, H, D)[b, t - cu[b]].to(torch.bfloat16)
    return o, lse.permute(0, 3, 1, 2).reshape(B, nq, H)[b, t - cu[b]].T.contiguous()[None]


def _plain_store(st):
    page, slots = st["case"]["page"], st["slots"].long()
    there = (slots >= 0)[:, None, None]
    at = torch.where(slots >= 0, slots, st["case"]["pages"] * page - 1)              # the last slot, which no token has
    for pool, rows in ((st["k"], st["k_new"]), (st["v"], st["v_new"])):
        pool = pool.transpose(1, 2)
        pool[at // page, at % page] = torch.where(there, rows, pool[at // page, at % page])
    return st["k"], st["v"]


def _plain_reserve(st):
    c = st["case"]
    page, most, T = c["page"], c["max_pages"], c["T"]
    lens, add, n0 = st["lens"].long(), st["add"].long(), st["n_free"].long()
    j = torch.arange(most, device="cuda")
    held = (lens + page - 1) // page
    # pages of ended sequences go back first
    back = torch.where(add < 0, held, 0)
    to = n0 + torch.cumsum(back, 0)[:, None] - back[:, None] + j
    free = torch.cat((st["free"], st["free"][:1]))
    free[torch.where(j < back[:, None], to, len(free) - 1)] = st["table"]
    free = free[:-1]
    n1 = n0 + back.sum()
    # then in order, as long as there are enough
    new = add.clamp(min=0)
    need = torch.where(lens + new <= most * page, (lens + new + page - 1) // page - held, 0)
    before = torch.cumsum(need, 0) - need
    served = (add >= 0) & (lens + new <= most * page) & ((need == 0) | (before + need <= n1))
    need = torch.where(served, need, 0)
    mine = (j >= held[:, None]) & (j < (held + need)[:, None])
    table = torch.where(mine, free[(n1 - 1 - before[:, None] - j + held[:, None]).clamp(0, len(free) - 1)], st["table"])
    cu = torch.cat((torch.zeros_like(n0), torch.cumsum(new, 0)))
    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True).clamp(max=c["B"] - 1)
    s = lens[b] + t - cu[b]
    slots = table[b, (s // page).clamp(0, most - 1)].long() * page + s % page
    slots = torch.where((t < cu[-1]) & served[b], slots, -1)
    st["lens_out"].copy_(torch.where(add < 0, 0, torch.where(served, lens + new, lens)))
    st["n_free_out"].copy_(n1 - need.sum())
    st["table"].copy_(table)
    st["free"].copy_(free)
    return st["lens_out"], st["n_free_out"], cu.to(torch.int32), slots.to(torch.int32), st["table"], st["free"]


# ------------------------------------------------------------------ one pass

def _handles(st):
    """What a user's program sets up once: the handles and the workspace."""
    import chunked_causal_attention_gb300 as cca
    c = st["case"]
    if c["op"] == "reserve":
        st["handle"] = cca.PagedTables(st["table"], st["lens"], st["free"], st["n_free"], c["page"])
        st["ws"] = cca.paged_workspace(tables=st["handle"])
    else:
        st["handle"] = cca.PagedCache(st["k"], st["v"])
        st["ws"] = cca.paged_workspace(st["handle"], q=st.get("q"), B=c.get("B", 1))


def run(state):
    op = state["case"]["op"]
    if not own:
        return {"attend": _plain_attend, "store": _plain_store, "reserve": _plain_reserve}[op](state)
    import chunked_causal_attention_gb300 as cca
    if "handle" not in state:
        _handles(state)
    if op == "attend":
        return cca.paged_attention(state["q"], state["handle"], state["table"], state["lens"], state["cu"], ws=state["ws"])
    if op == "store":
        cca.paged_store(state["handle"], state["k_new"], state["v_new"], state["slots"], ws=state["ws"])
        return state["k"], state["v"]
    cu, slots = cca.paged_reserve(state["handle"], state["add"], state["case"]["T"], lens_out=state["lens_out"],
                                  n_free_out=state["n_free_out"], ws=state["ws"])
    return state["lens_out"], state["n_free_out"], cu, slots, state["table"], state["free"]


def work(case):
    op = case["op"]
    if op == "store":
        rows = (case["T"] - case["pad"]) * case["Hkv"]
        return {"bytes": 8 * case["D"] * rows + 4 * case["T"], "flops": 0}
    if op == "reserve":
        return {"bytes": 4 * case["T"] + 16 * case["B"] + 8 * (case["T"] // case["page"]), "flops": 0}
    B, H, Hkv, D = (case[n] for n in ("B", "H", "Hkv", "D"))
    few = 0.45 if case["ragged"] else 1.0                        # slots in use, about
    nq = [1] * (B - 1) + [case["nq"]] if case["kind"] == "mixed" else [case["nq"] * (few if case["kind"] == "chunk" else 1.0)] * B
    n = [max(case["cap"] * few, x) for x in nq]
    pairs = sum(x * (y - (x - 1) / 2) for x, y in zip(nq, n))
    return {"bytes": int(sum(n) * Hkv * D * 4 + sum(nq) * H * (4 * D + 4)), "flops": int(4 * D * H * pairs)}


# ------------------------------------------------------------------ 64 bits

def _exact_attend(case, seed):
    st = prepare(case, seed)
    page, D, G = case["page"], case["D"], case["H"] // case["Hkv"]
    cu, lens = st["cu"].tolist(), st["lens"].tolist()
    o = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros((1, case["H"], cu[-1]), dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        a, z = cu[b], cu[b + 1]
        pages = st["table"][b, :(n + page - 1) // page].long()
        unseen = torch.ones((z - a, n), dtype=torch.bool, device="cuda").triu(n - (z - a) + 1)
        for h in range(case["Hkv"]):
            k, v = (x[pages, h].reshape(-1, D)[:n].double() for x in (st["k"], st["v"]))
            for m in range(h * G, (h + 1) * G):
                s = (st["q"][a:z, m].double() @ k.T * D ** -0.5).masked_fill_(unseen, -math.inf)
                lse[0, m, a:z] = torch.logsumexp(s, -1)
                o[a:z, m] = s.sub_(lse[0, m, a:z, None]).exp_() @ v
    return o, lse


def _exact_store(case, seed):
    st = prepare(case, seed)
    slots = st["slots"].long()
    kept = torch.nonzero(slots >= 0)[:, 0]
    out = []
    for pool, rows in ((st["k"], st["k_new"]), (st["v"], st["v_new"])):
        pool = pool.double().transpose(1, 2).contiguous()
        pool.view(-1, case["Hkv"], case["D"]).index_copy_(0, slots[kept], rows[kept].double())
        out.append(pool.transpose(1, 2))
    return out


def exact(case, seed):
    if case["op"] == "reserve":
        return None                                              # whole numbers all
    return (_exact_attend if case["op"] == "attend" else _exact_store)(case, seed)
