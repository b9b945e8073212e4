"""The operators of the 4-bit KV cache, as they are measured: cases, inputs, plain forms and exact values.

A cache row (one slot of one kv head) is 128 values of 4 bits (e2m1: 0, 1/2, 1, 3/2, 2, 3, 4, 6 and a sign; the
value of dimension 2i in the low half of byte i) with one 8-bit scale (e4m3) for each 16 of them:

    value = 2^exp * scale * code        exp: one whole number for the keys of a cache, one for the values

Operators (`op` of a case):

    append     rows of keys and values are rounded into the slots behind a sequence's cache
    attention  rows of queries over the cache and, under an ancestor mask, the tree's own slots
    weights    attention weight that given rows (an accepted path) lay on every slot, added to a running score
    compact    the accepted nodes of a tree move to the slots behind the cache, in every layer
    evict      the slots with the least score leave the cache, in every layer

Where `own` is false `run` computes them from elementary torch operations in 32 bits, else it calls the library.
Codes and scales that an operator only moves are returned as the bytes that they are (they have to be equal); what
`append` rounds is returned as the values that the cache then stands for.
"""
import math

import torch

own = False

HD = 128            # head dimension
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
BORDERS = ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False))  # (value, up at a tie)
K_EXP, V_EXP = 0, -3
DEV = "cuda"


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # the chain of a 16-token draft block enters the cache of three sequences, one of them cut short
        dict(name="append_chain_b3", op="append", b=3, n=16, hq=32, hkv=8, at=1000, step=77, ragged=True),
        # a prompt of 4096 tokens of four sequences enters an empty cache
        dict(name="append_prompt_b4", op="append", b=4, n=4096, hq=32, hkv=8, at=0, step=0, ragged=False),
        # plain decoding of one sequence over a short context: latency
        dict(name="attention_token_b1", op="attention", b=1, t=1, hq=32, hkv=8, at=1000, step=0, tree=False),
        # plain decoding of sixteen sequences of uneven, long contexts: the bytes of the cache
        dict(name="attention_token_b16", op="attention", b=16, t=1, hq=32, hkv=8, at=32767, step=1531, tree=False),
        # the drafted chain of four sequences verified as it stands
        dict(name="attention_chain_b4", op="attention", b=4, t=16, hq=32, hkv=8, at=8191, step=801, tree=False),
        # a draft tree of 256 nodes and its root verified for two sequences
        dict(name="attention_tree_b2", op="attention", b=2, t=257, hq=32, hkv=8, at=8192, step=1000, tree=True),
        # the accepted path of one step votes on the slots it saw
        dict(name="weights_path_b1", op="weights", b=1, t=257, rows=9, hq=32, hkv=8, at=4096, step=0),
        # sixteen rows of each of eight sequences vote on long caches
        dict(name="weights_path_b8", op="weights", b=8, t=16, rows=16, hq=32, hkv=8, at=16384, step=1111),
        # one layer's accepted path moves
        dict(name="compact_b1", op="compact", layers=1, b=1, t=257, hkv=8, at=1000, step=0, most=7),
        # the paths of sixteen sequences move in all 36 layers
        dict(name="compact_36_b16", op="compact", layers=36, b=16, t=257, hkv=8, at=2048, step=99, most=15),
        # one layer of two sequences, one of them shorter than the budget
        dict(name="evict_b2", op="evict", layers=1, b=2, hkv=8, at=1263, step=700, budget=1000, sink=4, recent=256),
        # all 36 layers of one sequence go back from 8449 slots to 4096
        dict(name="evict_36_b1", op="evict", layers=36, b=1, hkv=8, at=8449, step=0, budget=4096, sink=4, recent=512),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("append", "attention", "attention", "attention", "weights", "compact", "evict"))
    hq, hkv = rng.choice(((32, 8), (32, 4), (16, 8), (40, 8), (8, 2), (4, 4)))
    most = [max(costs) for costs in zip(*(_cost(c) for c in listed() if c["op"] == op))]
    while True:
        b = _log(rng, 1, 16)
        at = _log(rng, 1, 32768) if rng.random() < 0.9 else 0
        step = rng.randint(0, max(0, at // max(1, b)))
        if op == "append":
            case = dict(op=op, b=b, n=_log(rng, 1, 4096), hq=hq, hkv=hkv, at=at, step=step, ragged=rng.random() < 0.5)
        elif op == "attention":
            case = dict(op=op, b=b, t=_log(rng, 1, 1025), hq=hq, hkv=hkv, at=at, step=step, tree=rng.random() < 0.5)
        elif op == "weights":
            rows = _log(rng, 1, 64)
            case = dict(op=op, b=b, t=rows + rng.choice((0, 1, 240)), rows=rows, hq=hq, hkv=hkv, at=at, step=step)
        elif op == "compact":
            case = dict(op=op, layers=_log(rng, 1, 36), b=b, t=rng.randint(64, 512), hkv=hkv, at=at, step=step, most=rng.randint(1, 15))
        else:
            at = max(at, 64)
            budget = rng.randint(at // 4 + 1, at)
            sink = rng.randint(0, min(8, budget // 2))
            case = dict(op=op, layers=_log(rng, 1, 36), b=b, hkv=hkv, at=at, step=step, budget=budget, sink=sink,
                        recent=rng.randint(0, (budget - sink) // 2))
        if all(c <= m for c, m in zip(_cost(case), most)):
            return case


def _cost(case):
    w = work(case)
    rows = case["b"] * case.get("layers", 1) * case["hkv"] * (case["at"] + case.get("t", case.get("n", 0)))
    return w["bytes"] + 64 * rows, w["flops"]


def _lens(case):
    """Slots of each sequence before the call."""
    return [max(0, case["at"] - s * case["step"]) for s in range(case["b"])]


def _new(case):
    """Rows of each sequence that enter (append) or vote (weights), nodes that move (compact)."""
    n = case["n"] if case["op"] == "append" else case["rows"] if case["op"] == "weights" else case["most"]
    if case["op"] == "append" and not case["ragged"]:
        return [n] * case["b"]
    return [n - (s * 5) % max(1, n // 2) for s in range(case["b"])]


def _cap(case):
    return (case["at"] + case.get("t", case.get("n", 0)) + 8) // 8 * 8


def _parents(t, seed):
    """A random tree of t nodes: node i hangs from an earlier one, more often from a late one."""
    g = torch.Generator().manual_seed(seed)
    i = torch.arange(1, t, dtype=torch.float64)
    p = (i * torch.rand(max(0, t - 1), generator=g, dtype=torch.float64).sqrt()).long()
    return [-1] + p.tolist()


def _ancestors(parents):
    t = len(parents)
    m = torch.zeros(t, t, dtype=torch.bool)
    for i, p in enumerate(parents):
        if p >= 0:
            m[i] = m[p]
        m[i, i] = True
    return m


def _bits(mask):
    """[..., t, t] truth values -> [..., t, ceil(t / 32)] words, bit j of word w for column 32 w + j."""
    t = mask.shape[-1]
    w = (t + 31) // 32
    full = torch.zeros(*mask.shape[:-1], 32 * w, dtype=torch.int64, device=mask.device)
    full[..., :t] = mask
    words = (full.view(*mask.shape[:-1], w, 32) << torch.arange(32, device=mask.device)).sum(-1)
    return torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32)


# ------------------------------------------------------------------------------------------------ inputs
def _codes(shape, g):
    """Random cache rows: codes as a block of 16 normal values leaves them, scales from 1/8 to 1/2."""
    x = torch.randn(65536, 2, generator=g, device=DEV) * 3.4   # a block's largest of 16 normal values stands near 6
    x[::16] = x[::16].sign() * 6
    c = _nearest(x.double(), torch.ones_like(x, dtype=torch.float64))
    table = (c[:, 0] + 16 * c[:, 1]).to(torch.uint8)
    pick = torch.randint(-32768, 32768, (*shape, HD // 2), generator=g, device=DEV, dtype=torch.int16)
    codes = table.view(-1)[pick.int().add_(32768).view(-1)].view(pick.shape) if pick.numel() < 1 << 26 else torch.cat(
        [table[p.int().add_(32768).view(-1)].view(p.shape) for p in pick.split(max(1, pick.shape[0] // 8))])
    scales = torch.randint(0x20, 0x31, (*shape, HD // 16), generator=g, device=DEV, dtype=torch.uint8)
    return codes, scales


def _cache(case, g, prefix=""):
    shape = (case.get("layers", 1), case["b"], case["hkv"], _cap(case))
    kc, ks = _codes(shape, g)
    vc, vs = _codes(shape, g)
    return {"k_codes": kc, "k_scales": ks, "v_codes": vc, "v_scales": vs}


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    op, b, hkv, lens = case["op"], case["b"], case["hkv"], _lens(case)
    st = {"case": dict(case), "scale": HD ** -0.5}
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    if op == "append":
        cap = _cap(case)
        z = lambda last: torch.zeros(1, b, hkv, cap, last, dtype=torch.uint8, device=DEV)  # noqa: E731
        st["cache"] = {"k_codes": z(HD // 2), "k_scales": z(HD // 16), "v_codes": z(HD // 2), "v_scales": z(HD // 16)}
        shape = (b, case["n"], hkv, HD)
        k = torch.randn(shape, generator=g, device=DEV)
        k[..., 5::32] *= 6                                          # keys have a few large dimensions
        st["k"], st["v"] = k.bfloat16(), (torch.randn(shape, generator=g, device=DEV) * 0.1).bfloat16()
        st["lens"], st["n_new"] = i32(lens), i32(_new(case))
        st["k_held"], st["v_held"] = torch.zeros_like(st["k"]), torch.zeros_like(st["v"])
    else:
        st["cache"] = _cache(case, g)
    if op in ("attention", "weights"):
        t, hq = case["t"], case["hq"]
        st["q"] = (torch.randn(b, t, hq, HD, generator=g, device=DEV) * 1.5).bfloat16()
        if op == "attention":
            st["lens"] = i32(lens)
            st["mask"] = torch.stack([_ancestors(_parents(t, seed * 131 + s)) for s in range(b)]).to(DEV) if case["tree"] else None
            st["anc"] = _bits(st["mask"]) if case["tree"] else None
            st["out"] = torch.zeros(b, t, hq, HD, dtype=torch.bfloat16, device=DEV)
            st["lse"] = torch.zeros(b, t, hq, dtype=torch.float32, device=DEV)
        else:
            rows = _new(case)
            st["n_rows"], st["lens"] = i32(rows), i32([n + r for n, r in zip(lens, rows)])
            pick = torch.zeros(b, case["rows"], dtype=torch.int32)          # the path's rows: the root, then its nodes
            for s in range(b):
                p = torch.randperm(t - 1, generator=torch.Generator().manual_seed(seed * 17 + s))[:rows[s] - 1].sort().values + 1
                pick[s, 1:rows[s]] = p.int()
            pick = pick.to(DEV)
            src = pick[:, 1:] + st["lens"][:, None] - st["n_rows"][:, None]
            st["rows"], st["src"] = pick, torch.nn.functional.pad(src, (0, 1), value=-1).contiguous()
            st["score"] = torch.rand(1, b, hkv, _cap(case), generator=g, device=DEV)
            st["score_out"] = st["score"].clone()
            st["lse"] = torch.zeros(b, t, hq, device=DEV)
            votes, see = _see(st)
            x = _scores(st, _picked(st, st["q"].float()))
            st["lse"][votes.nonzero()[:, 0], pick[votes].long()] = x.masked_fill(~see, -math.inf).logsumexp(-1)[votes]
    if op == "compact":
        a = _new(case)
        st["n_acc"], st["lens"] = i32(a), i32([n + 1 + k for n, k in zip(lens, a)])
        src = torch.full((b, 16), -1, dtype=torch.int32)
        for s in range(b):     # nodes behind the slots that the path goes to: a second pass finds the same rows
            p = torch.randperm(case["t"] - 17, generator=torch.Generator().manual_seed(seed * 19 + s))[:a[s]].sort().values
            src[s, :a[s]] = (lens[s] + 17 + p).int()
        st["src"] = src.to(DEV)
    if op == "evict":
        full = (case["layers"], b, hkv, _cap(case))
        st["score"] = torch.rand(full, generator=g, device=DEV).pow_(8) * 50       # most weight lies on few slots
        st["score"][torch.rand(full, generator=g, device=DEV) < 0.1] = 0.0         # some were never looked at: ties
        st["lens"], st["new_len"] = i32(lens), i32([0] * b)
        new = (case["layers"], b, hkv, (case["budget"] + 7) // 8 * 8 + 64)
        z = lambda last: torch.zeros(*new, last, dtype=torch.uint8, device=DEV)  # noqa: E731
        st["to"] = {"k_codes": z(HD // 2), "k_scales": z(HD // 16), "v_codes": z(HD // 2), "v_scales": z(HD // 16)}
        st["to_score"] = torch.zeros(new, device=DEV)
        st["kept"] = torch.zeros(*new[:3], case["budget"], dtype=torch.int32, device=DEV)
    if own:   # the handles that a program keeps: the cache, and a workspace
        from block_diffusion_draft_dflash_gb300 import _lib
        st["kv"] = _lib.Kv4Cache(k_exp=K_EXP, v_exp=V_EXP, **st["cache"])
        if op == "evict":
            st["kv_to"] = _lib.Kv4Cache(k_exp=K_EXP, v_exp=V_EXP, **st["to"])
        need = {"append": lambda: _lib.kv4_append_workspace_size(),
                "attention": lambda: _lib.kv4_attention_workspace_size(st["kv"], case["t"], case["hq"]),
                "weights": lambda: _lib.kv4_attention_weights_workspace_size(st["kv"], case["t"], case["hq"]),
                "compact": lambda: _lib.kv4_compact_workspace_size(),
                "evict": lambda: _lib.kv4_evict_workspace_size(st["kv"], case["budget"])}[op]
        st["ws"] = _lib.Workspace(need())
    return st


# ------------------------------------------------------------------------------------------------ plain forms
def _nearest(x, scale):
    """Codes of x / scale (64 bits: the borders between codes are met exactly); ties to the even code."""
    a = x.abs()
    c = torch.zeros(x.shape, dtype=torch.uint8, device=x.device)
    for t, up in BORDERS:
        c += (a >= t * scale) if up else (a > t * scale)
    return torch.where(scale > 0, c + 8 * torch.signbit(x).to(torch.uint8), torch.zeros_like(c))


def _round(x, exp):
    """x [..., 128] -> codes [..., 64], scales [..., 8] (bytes) and the values that they stand for."""
    blocks = x.double().view(*x.shape[:-1], HD // 16, 16) * 2.0 ** -exp
    scale = (blocks.abs().amax(-1) / 6).clamp(max=448.0).float().to(torch.float8_e4m3fn)
    s = scale.double()[..., None]
    c = _nearest(blocks, s)
    table = torch.tensor(GRID + tuple(-v for v in GRID), dtype=torch.float64, device=x.device)
    held = (table[c.long()] * s * 2.0 ** exp).view(x.shape).to(x.dtype)
    c = c.view(x.shape)
    return c[..., 0::2] | c[..., 1::2] << 4, scale.view(torch.uint8), held


def _values(codes, scales, exp):
    """The values of cache rows in 32 bits."""
    table = torch.tensor(GRID + tuple(-v for v in GRID), dtype=torch.float32, device=codes.device)
    c = torch.stack((codes & 15, codes >> 4), -1).view(*codes.shape[:-1], HD // 16, 16)
    s = scales.view(torch.float8_e4m3fn).float() * 2.0 ** exp
    return (table[c.int()] * s[..., None]).view(*codes.shape[:-1], HD)


def _scores(st, q):
    """Scaled scores of rows q [b][r][hq][128] against every slot: [b][r][hq][cap]."""
    c = st["cache"]
    k = _values(c["k_codes"][0], c["k_scales"][0], K_EXP)
    b, r, hq, _ = q.shape
    hkv = k.shape[1]
    grouped = q.view(b, r, hkv, hq // hkv, HD).transpose(1, 2).reshape(b, hkv, -1, HD)
    x = torch.matmul(grouped, k.transpose(-1, -2)) * st["scale"]
    return x.view(b, hkv, r, hq // hkv, -1).transpose(1, 2).reshape(b, r, hq, -1)


def _picked(st, x):
    return x.gather(1, st["rows"].long().view(*st["rows"].shape, *[1] * (x.dim() - 2)).expand(-1, -1, *x.shape[2:]))


def _see(st):
    """Rows that vote, and the slots that each of them sees ([b][rows][1][cap])."""
    j = torch.arange(st["rows"].shape[1], device=DEV)
    slot = torch.arange(st["score"].shape[-1], device=DEV)
    base = st["lens"] - st["n_rows"]
    votes = j < st["n_rows"][:, None]
    see = (slot <= (base[:, None] + j)[..., None]) & votes[..., None]
    return votes, see[:, :, None]


def _plain(st):
    case, c = st["case"], st["cache"]
    op, b = case["op"], case["b"]
    lens = st["lens"].long()
    if op == "append":
        n = case["n"]
        j = torch.arange(n, device=DEV)
        on = j < st["n_new"][:, None]
        s = torch.arange(b, device=DEV)[:, None].expand(b, n)[on]
        slot = (lens[:, None] + j)[on]
        for name, exp in (("k", K_EXP), ("v", V_EXP)):
            codes, scales, held = _round(st[name][on], exp)
            c[name + "_codes"][0, s, :, slot] = codes
            c[name + "_scales"][0, s, :, slot] = scales
            st[name + "_held"][on] = held
        return {"k_held": st["k_held"], "v_held": st["v_held"]}
    if op == "attention":
        t, hq, hkv, cap = case["t"], case["hq"], case["hkv"], _cap(case)
        x = _scores(st, st["q"].float())
        slot = torch.arange(cap, device=DEV)
        tail = slot - lens[:, None]
        if st["mask"] is None:
            see = tail[:, None] <= torch.arange(t, device=DEV)[:, None]
        else:
            own_slots = st["mask"].gather(2, tail.clamp(0, t - 1)[:, None].expand(b, t, cap))
            see = (tail < 0)[:, None] | (own_slots & (tail < t)[:, None])
        x = x.masked_fill(~see[:, :, None], -math.inf)
        m = x.amax(-1, keepdim=True)
        p = (x - m).exp()
        total = p.sum(-1, keepdim=True)
        v = _values(c["v_codes"][0], c["v_scales"][0], V_EXP)
        g = hq // hkv
        w = p.view(b, t, hkv, g, cap).transpose(1, 2).reshape(b, hkv, t * g, cap)
        o = torch.matmul(w, v).view(b, hkv, t, g, HD).transpose(1, 2).reshape(b, t, hq, HD) / total
        return {"out": o.bfloat16(), "lse": (m + total.log())[..., 0]}
    if op == "weights":
        _, see = _see(st)
        x = _scores(st, _picked(st, st["q"].float()))
        p = torch.where(see, (x - _picked(st, st["lse"])[..., None]).exp(), torch.zeros((), device=DEV))
        hkv = case["hkv"]
        mass = p.view(b, p.shape[1], hkv, -1, p.shape[-1]).sum((1, 3))
        slot = torch.arange(p.shape[-1], device=DEV)
        old = torch.where((slot < (lens - st["n_rows"])[:, None])[:, None], st["score"][0], torch.zeros((), device=DEV))
        live = (slot < lens[:, None])[:, None]
        return {"score": torch.where(live, old + mass, st["score"][0])[None]}
    if op == "compact":
        j = torch.arange(st["src"].shape[1], device=DEV)
        on = j < st["n_acc"][:, None]
        s = torch.arange(b, device=DEV)[:, None].expand(on.shape)[on]
        src = st["src"].long()[on]
        dst = (lens[:, None] - st["n_acc"][:, None] + j)[on]
        for rows in c.values():
            rows[:, s, :, dst] = rows[:, s, :, src]
        return dict(c)
    budget = case["budget"]
    slot = torch.arange(st["score"].shape[-1], device=DEV)
    kind = torch.where((slot < case["sink"]) | (slot >= (lens - case["recent"])[:, None]), 0, 1)
    kind = torch.where(slot < lens[:, None], kind, 2)[None, :, None].expand(st["score"].shape)
    order = st["score"].sort(dim=-1, descending=True, stable=True).indices
    order = order.gather(-1, kind.gather(-1, order).sort(dim=-1, stable=True).indices)
    new_len = lens.clamp(max=budget)
    left = torch.arange(budget, device=DEV) < new_len[None, :, None, None]
    if order.shape[-1] < budget:
        order = torch.nn.functional.pad(order, (0, budget - order.shape[-1]))
    kept = torch.where(left, order[..., :budget], slot.numel()).sort(-1).values
    at = torch.where(left, kept, 0)
    for name, rows in c.items():
        moved = rows.gather(3, at[..., None].expand(*at.shape, rows.shape[-1]))
        st["to"][name][..., :budget, :] = torch.where(left[..., None], moved, st["to"][name][..., :budget, :])
    st["to_score"][..., :budget] = torch.where(left, st["score"].gather(3, at), st["to_score"][..., :budget])
    return {**st["to"], "score": st["to_score"], "kept": torch.where(left, kept, -1).int(), "new_len": new_len.int()}


def run(st):
    if not own:
        return _plain(st)
    from block_diffusion_draft_dflash_gb300 import _lib
    case, kv, ws = st["case"], st["kv"], st["ws"]
    op = case["op"]
    if op == "append":
        _lib.kv4_append(kv, 0, st["k"], st["v"], st["lens"], ws, n_new=st["n_new"], k_held=st["k_held"], v_held=st["v_held"])
        return {"k_held": st["k_held"], "v_held": st["v_held"]}
    if op == "attention":
        _lib.kv4_attention(kv, 0, st["q"], st["lens"], st["anc"], st["scale"], st["out"], ws, lse=st["lse"])
        return {"out": st["out"], "lse": st["lse"]}
    if op == "weights":
        _lib.kv4_attention_weights(kv, 0, st["q"], st["lse"], st["lens"], st["scale"], st["score"], ws, n_rows=st["n_rows"],
                                   src_slot=st["src"], score_out=st["score_out"])
        return {"score": st["score_out"]}
    if op == "compact":
        _lib.kv4_compact(kv, st["src"], st["n_acc"], st["lens"], ws)
        return dict(st["cache"])
    _lib.kv4_evict(kv, st["score"], st["lens"], case["budget"], case["sink"], case["recent"], st["kv_to"], st["to_score"],
                   st["new_len"], st["kept"], ws)
    return {**st["to"], "score": st["to_score"], "kept": st["kept"], "new_len": st["new_len"]}


# ------------------------------------------------------------------------------------------------ what a pass needs
ROW = HD // 2 + HD // 16      # bytes of a cache row


def work(case):
    op, hkv, lens = case["op"], case["hkv"], _lens(case)
    if op == "append":
        rows = sum(_new(case)) * hkv
        return {"bytes": rows * 2 * (2 * HD * 2 + ROW), "flops": rows * 2 * HD * 4}
    if op == "attention":
        t, hq = case["t"], case["hq"]
        keys = sum(lens) + case["b"] * t
        tail = t * (t + 1) // 2 if not case["tree"] else int(t * (math.log2(t) + 1))   # a random tree's ancestors, about
        pairs = sum(t * n + tail for n in lens)
        mask = case["b"] * t * ((t + 31) // 32) * 4 if case["tree"] else 0
        return {"bytes": keys * hkv * 2 * ROW + case["b"] * t * hq * (2 * HD * 2 + 4) + mask, "flops": 4 * HD * hq * pairs}
    if op == "weights":
        hq, rows = case["hq"], _new(case)
        keys = sum(n + r for n, r in zip(lens, rows))
        return {"bytes": keys * hkv * (ROW + 8) + sum(rows) * hq * (HD * 2 + 4),
                "flops": 2 * HD * hq * sum(r * n + r * (r + 1) // 2 for n, r in zip(lens, rows))}
    if op == "compact":
        return {"bytes": case["layers"] * hkv * sum(_new(case)) * 2 * 2 * ROW, "flops": 0}
    kept = sum(min(n, case["budget"]) for n in lens)
    return {"bytes": case["layers"] * hkv * (4 * sum(lens) + kept * (2 * 2 * ROW + 4 + 4)), "flops": 0}


# ------------------------------------------------------------------------------------------------ exact values
def _rows64(codes, scales, exp):
    """Cache rows in 64 bits, from the fields of the codes: sign, two bits of exponent, one of mantissa."""
    both = torch.empty(*codes.shape[:-1], HD, dtype=torch.int64, device=codes.device)
    both[..., 0::2], both[..., 1::2] = codes % 16, codes // 16
    e, m = both // 2 % 4, both % 2
    size = torch.where(e == 0, 0.5 * m.double(), (1 + 0.5 * m) * 2.0 ** (e.double() - 1))
    se, sm = (scales.long() // 8 % 16).double(), (scales.long() % 8).double()
    s = torch.where(se == 0, sm / 8 * 2.0 ** -6, (1 + sm / 8) * 2.0 ** (se - 7)) * 2.0 ** exp
    return torch.where(both >= 8, -size, size) * s.repeat_interleave(16, -1)


def exact(case, seed):
    st = prepare(case, seed)
    op, b, lens, c = case["op"], case["b"], _lens(case), st["cache"]
    if op == "append":
        got = {}
        grid = torch.tensor(GRID, dtype=torch.float64, device=DEV)
        tenth = torch.arange(8, device=DEV)
        for name, exp in (("k", K_EXP), ("v", V_EXP)):
            out = torch.zeros(st[name].shape, dtype=torch.float64, device=DEV)
            for s, n in enumerate(_new(case)):
                x = st[name][s, :n].double().reshape(-1, 16) / 2.0 ** exp
                want = x.abs().max(1).values / 6
                e = torch.frexp(want).exponent.clamp(min=-5) - 4      # e4m3: three bits behind the first, down to 2^-9
                scale = torch.minimum((want / 2.0 ** e).round() * 2.0 ** e, torch.tensor(448.0, dtype=torch.float64, device=DEV))[:, None]
                far = (x.abs()[..., None] - scale[..., None] * grid).abs()
                tie = far == far.min(-1, keepdim=True).values         # two at a border: the even one
                code = torch.where(tie, tenth + 100 * (tenth % 2), 1000).min(-1).values % 100
                out[s, :n] = (grid[code] * scale * x.sign() * 2.0 ** exp).reshape(n, -1, HD)
            got[name + "_held"] = out
        return got
    if op == "attention":
        t, hq, g = case["t"], case["hq"], case["hq"] // case["hkv"]
        out = torch.zeros(b, t, hq, HD, dtype=torch.float64, device=DEV)
        lse = torch.zeros(b, t, hq, dtype=torch.float64, device=DEV)
        for s, n in enumerate(lens):
            mine = st["mask"][s] if case["tree"] else torch.ones(t, t, dtype=torch.bool, device=DEV).tril()
            see = torch.cat((torch.ones(t, n, dtype=torch.bool, device=DEV), mine), 1)
            for h in range(case["hkv"]):
                k = _rows64(c["k_codes"][0, s, h, :n + t], c["k_scales"][0, s, h, :n + t], K_EXP)
                v = _rows64(c["v_codes"][0, s, h, :n + t], c["v_scales"][0, s, h, :n + t], V_EXP)
                x = torch.einsum("tgd,nd->gtn", st["q"][s, :, h * g:(h + 1) * g].double(), k) / math.sqrt(HD)
                x[:, ~see] = -math.inf
                lse[s, :, h * g:(h + 1) * g] = x.logsumexp(-1).T
                out[s, :, h * g:(h + 1) * g] = torch.einsum("gtn,nd->tgd", x.softmax(-1), v)
        return {"out": out, "lse": lse}
    if op == "weights":
        g = case["hq"] // case["hkv"]
        score = st["score"].double()
        for s, (n, r) in enumerate(zip(lens, _new(case))):
            for h in range(case["hkv"]):
                k = _rows64(c["k_codes"][0, s, h, :n + r], c["k_scales"][0, s, h, :n + r], K_EXP)
                score[0, s, h, n:n + r] = 0
                x = torch.einsum("rgd,nd->rgn", st["q"][s, st["rows"][s, :r].long(), h * g:(h + 1) * g].double(), k) / math.sqrt(HD)
                p = (x - st["lse"][s, st["rows"][s, :r].long(), h * g:(h + 1) * g].double()[..., None]).exp()
                p = p * torch.ones(r, n + r, dtype=torch.float64, device=DEV).tril(n)[:, None]
                score[0, s, h, :n + r] += p.sum((0, 1))
        return {"score": score}
    if op == "compact":
        got = {k: v.clone() for k, v in c.items()}
        for s, (n, a) in enumerate(zip(lens, _new(case))):
            for k, v in c.items():
                got[k][:, s, :, n + 1:n + 1 + a] = v[:, s][:, :, st["src"][s, :a].long()]
        return got
    return None          # every output is a choice or a copy, which the plain form makes exactly
