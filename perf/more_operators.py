"""The operators on rows of logits, as they are measured: cases, inputs, plain forms and exact values.

A row holds one logit for each of V tokens.  Its tokens stand in order of their logits, the larger first, the lower
token id first among equal ones.  Operators (`op` of a case):

    sample    a token is drawn for every row with a given random number, from softmax(logits / T) cut by top-k, top-p
              and min-p (each keeps the first tokens of the order, the strictest counts):
                  top-k  the first k;  top-p  those before which less than p of the top-k's mass lies;
                  min-p  those with at least min_p times the first one's probability
              the token is the first one in the order at which the kept mass exceeds u times all of it
    top       the K first tokens of every row with their logits, and the row's log-sum at a temperature
    distill   loss of student rows against a teacher's top logits: the divergence of the distribution over the listed
              tokens and "any other" (weighted), or with `grad` its gradient by the student's logits as well
    backward  that gradient alone, from the statistics that the loss left and the gradients of the losses

Where `own` is false `run` computes them from elementary torch operations, else it calls the library.  Masses and what
is compared with them are 64-bit numbers in the plain form: which token a border falls on is a whole number.
"""
import math

import torch

own = False

DEV = "cuda"
VOCAB = 151936
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}

# (temperature, top_k, top_p, min_p) of the sequences of a batch, in turn
PARAMS = {
    "usual": [(0.6, 20, 0.95, 0.0)],
    "nucleus": [(1.0, 0, 0.9, 0.0)],
    "open": [(1.0, 0, 1.0, 0.0)],
    "minp": [(1.2, 0, 1.0, 0.05)],
    "mixed": [(0.6, 20, 0.95, 0.0), (0.0, 0, 1.0, 0.0), (1.0, 0, 0.9, 0.0), (0.8, 200, 0.98, 0.02), (1.3, 0, 1.0, 0.1),
              (1.0, 50, 1.0, 0.0), (0.7, 0, 0.8, 0.0), (1.0, 0, 1.0, 0.0)],
}


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # plain decoding of one sequence: latency
        dict(name="sample_token_b1", op="sample", rows=1, group=1, V=VOCAB, type="fp32", pad=0, params="usual", masked=False),
        # the target draws after every node of one tree of 256 nodes and its root
        dict(name="sample_tree_b1", op="sample", rows=257, group=257, V=VOCAB, type="fp32", pad=0, params="usual", masked=False),
        # chains of 16 rows of sixteen sequences, cut by mass alone
        dict(name="sample_nucleus_b16", op="sample", rows=256, group=16, V=VOCAB, type="bf16", pad=0, params="nucleus", masked=False),
        # trees of sixteen sequences, each with settings of its own
        dict(name="sample_mixed_b16", op="sample", rows=2064, group=129, V=VOCAB, type="bf16", pad=0, params="mixed", masked=False),
        # the teacher's list for one accepted path
        dict(name="top_path_b1", op="top", rows=16, V=VOCAB, type="fp32", pad=0, K=20, T=1.0),
        # lists for a prompt's every token
        dict(name="top_prompt_b2", op="top", rows=2048, V=VOCAB, type="bf16", pad=0, K=256, T=1.0),
        # validation on a small vocabulary of odd size: rows that start anywhere
        dict(name="distill_odd_b3", op="distill", rows=45, V=4001, type="bf16", pad=0, K=33, T=2.0, grad=False),
        # validation of sixteen drafted blocks
        dict(name="distill_eval_b16", op="distill", rows=240, V=VOCAB, type="fp32", pad=0, K=64, T=1.0, grad=False),
        # one drafted block teaches: loss and gradient in one call
        dict(name="distill_block_b1", op="distill", rows=15, V=VOCAB, type="fp32", pad=0, K=64, T=1.0, grad=True),
        # a training batch of 64 blocks
        dict(name="distill_block_b64", op="distill", rows=960, V=VOCAB, type="bf16", pad=0, K=128, T=1.0, grad=True),
        # gradient of a few rows of a vocabulary of odd size
        dict(name="backward_odd_b2", op="backward", rows=30, V=32003, type="bf16", pad=0, K=20, T=2.0),
        # gradient of a training batch, from kept statistics
        dict(name="backward_block_b64", op="backward", rows=960, V=VOCAB, type="fp32", pad=0, K=128, T=1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("sample", "sample", "top", "distill", "distill", "backward"))
    most = max(work(c)["bytes"] for c in listed() if c["op"] == op)
    while True:
        case = dict(op=op, rows=_log(rng, 1, 4096), V=_log(rng, 64, 262144), type=rng.choice(("fp32", "bf16")),
                    pad=rng.choice((0, 0, 1, 8, 37)))
        if op == "sample":
            group = _log(rng, 1, 257)
            case.update(group=group, rows=max(1, case["rows"] // group) * group, params=rng.choice(sorted(PARAMS)),
                        masked=rng.random() < 0.25)
        else:
            case.update(K=min(_log(rng, 1, 512), case["V"] // 2), T=rng.choice((1.0, 1.0, 0.75, 2.0)))
        if op == "distill":
            case["grad"] = rng.random() < 0.5
        if work(case)["bytes"] <= most:
            return case


def work(case):
    """Every logit is read once, every gradient written once; an exponential or two and a comparison for each."""
    es = 4 if case["type"] == "fp32" else 2
    n = case["rows"] * case["V"]
    if case["op"] == "sample":
        return {"bytes": n * es + case["rows"] * 16, "flops": 4 * n}
    lists = case["rows"] * case["K"] * 8
    if case["op"] == "top":
        return {"bytes": n * es + lists, "flops": 4 * n}
    if case["op"] == "distill":
        return {"bytes": n * es * (2 if case["grad"] else 1) + lists, "flops": (8 if case["grad"] else 4) * n}
    return {"bytes": n * es * 2 + lists, "flops": 4 * n}


# ------------------------------------------------------------------------------------------------ inputs
def _logits(rows, V, g, heads=24):
    """Rows as a language model gives them: a wide bell of unlikely tokens and a few likely ones, unevenly sure."""
    x = torch.randn(rows, V, generator=g, device=DEV).mul_(2.0).sub_(4.0)
    n = min(heads, V)
    at = torch.randint(0, V, (rows, n), generator=g, device=DEV)
    e = torch.empty(rows, n, device=DEV).exponential_(generator=g)
    sure = torch.rand(rows, 1, generator=g, device=DEV) * 4
    return x.scatter_reduce_(1, at, e * (1 + sure) + 4, "amax")


def _held(x, case):
    """The rows in the case's type, with `pad` unused values behind each."""
    whole = torch.zeros(case["rows"], case["V"] + case["pad"], dtype=TYPES[case["type"]], device=DEV)
    whole[:, :case["V"]] = x
    return whole[:, :case["V"]]


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    op, rows, V = case["op"], case["rows"], case["V"]
    st = {"case": dict(case)}
    f32 = lambda v: torch.tensor(v, dtype=torch.float32, device=DEV)  # noqa: E731
    zero = lambda *s, t=torch.float32: torch.zeros(s, dtype=t, device=DEV)  # noqa: E731
    x = _logits(rows, V, g)
    if op == "sample":
        if case["masked"]:                                       # a grammar allows few tokens
            no = torch.rand(rows, V, generator=g, device=DEV) < 0.9
            no[:, 0] = False                                     # the end of the text is one of them
            x.masked_fill_(no, -math.inf)
        each = PARAMS[case["params"]]
        each = [each[(s + seed) % len(each)] for s in range(rows // case["group"])]
        st["temperature"], st["top_p"], st["min_p"] = (f32([p[i] for p in each]) for i in (0, 2, 3))
        st["top_k"] = torch.tensor([p[1] for p in each], dtype=torch.int32, device=DEV)
        st["logits"], st["u"] = _held(x, case), torch.rand(rows, generator=g, device=DEV)
        st["token"], st["n_kept"], st["logprob"] = zero(rows, t=torch.int32), zero(rows, t=torch.int32), zero(rows)
    elif op == "top":
        st["logits"] = _held(x, case)
        st["id"], st["val"], st["lse"] = zero(rows, case["K"], t=torch.int32), zero(rows, case["K"]), zero(rows)
    else:
        T, K = case["T"], case["K"]
        st["val"], idx = x.topk(K, -1)                           # the teacher's lists, one for a node of a tree
        st["id"], st["lse"] = idx.int(), (x.double() / T).logsumexp(-1).float()
        st["teacher_row"] = torch.randperm(rows, generator=g, device=DEV).int()
        drop = torch.rand(rows, generator=g, device=DEV) < 0.1   # positions behind the accepted path teach nothing
        drop[0] = False
        x = x[st["teacher_row"].long()]                          # the student follows its teacher, more or less
        x.mul_(0.8).add_(torch.randn(x.shape, generator=g, device=DEV))
        st["teacher_row"].masked_fill_(drop, -1)
        st["weight"] = torch.exp(-(torch.arange(rows, device=DEV) % 15) / 7.0)   # early positions of a block count more
        st["student"] = _held(x, case)
        st["loss"], st["stats"] = zero(rows), zero(rows, 4)
        st["grad"] = torch.zeros_like(st["student"]) if case.get("grad", True) else None
        if op == "backward":
            st["grad_loss"] = torch.rand(rows, generator=g, device=DEV) + 0.5
            st["stats"] = _stats(st)
    if own:
        from block_diffusion_draft_dflash_gb300 import _lib
        size = {"sample": _lib.sample_workspace_size, "top": _lib.top_logits_workspace_size,
                "distill": _lib.distill_workspace_size, "backward": _lib.distill_workspace_size}[op]
        st["ws"] = _lib.Workspace(size(rows, V))
    return st


# ------------------------------------------------------------------------------------------------ plain forms
def _lists(st):
    """The teacher's list of every student row (ids, probabilities, what is left for the others) and which rows learn."""
    row = st["teacher_row"].long()
    at = row.clamp(min=0)
    t = (st["val"][at].double() / st["case"]["T"] - st["lse"][at, None].double()).exp()
    return st["id"][at].long(), t, (1 - t.sum(-1)).clamp(min=0), row >= 0


def _stats(st):
    """Largest logit of a row, log-sum of exp((z - largest) / T) over all tokens and over those not listed, 0."""
    ids, _, _, on = _lists(st)
    z = st["student"].float()
    m = z.amax(-1, keepdim=True)
    e = ((z - m) / st["case"]["T"]).exp()
    rest = e.scatter(1, ids, 0.0).sum(-1)
    s = torch.stack((m[:, 0], e.sum(-1).log(), rest.log(), torch.zeros_like(rest)), 1)
    return torch.where(on[:, None], s, 0.0)


def _gradient(st, stats, scale):
    ids, t, rho, on = _lists(st)
    T = st["case"]["T"]
    z = st["student"].float()
    scale = torch.where(on, scale / T, 0.0)[:, None]
    q = ((z - stats[:, :1]) / T - stats[:, 1:2]).exp()
    others = 1 - rho / (stats[:, 2] - stats[:, 1]).double().exp()
    grad = q * (scale * others[:, None].float())
    return grad.scatter(1, ids, (q.gather(1, ids) - t.float()) * scale).to(st["student"].dtype)


def _plain(st):
    case = st["case"]
    op = case["op"]
    if op == "sample":
        rows, V = st["logits"].shape
        per = lambda p: p.repeat_interleave(case["group"])[:, None]  # noqa: E731
        T, k, p, low = (per(st[n]) for n in ("temperature", "top_k", "top_p", "min_p"))
        first = T == 0
        x, order = st["logits"].float().sort(dim=-1, descending=True, stable=True)
        w = ((x.double() - x[:, :1]) / torch.where(first, 1.0, T).double()).exp()
        rank = torch.arange(V, device=DEV)
        keep = (x > -math.inf) & ((rank < k) | (k <= 0)) & ((rank == 0) | ~first)
        w = torch.where(keep, w, 0.0)
        before = torch.nn.functional.pad(w.cumsum(-1)[:, :-1], (1, 0))
        total = w.sum(-1, keepdim=True)
        keep &= ((before < p.double() * total) | (p >= 1)) & (w >= low.double())
        w = torch.where(keep, w, 0.0)
        total = w.sum(-1, keepdim=True)
        at = ((w.cumsum(-1) <= st["u"][:, None].double() * total) & keep).sum(-1, keepdim=True)
        n = keep.sum(-1, keepdim=True)
        at = torch.minimum(at, n - 1)
        return {"token": order.gather(1, at)[:, 0].int(), "n_kept": n[:, 0].int(),
                "logprob": (w.gather(1, at) / total).log()[:, 0].float()}
    if op == "top":
        x = st["logits"].float()
        val, order = x.sort(dim=-1, descending=True, stable=True)
        m = val[:, :1]
        total = ((x - m) / case["T"]).exp().sum(-1)
        return {"id": order[:, :case["K"]].int(), "val": val[:, :case["K"]].clone(), "lse": m[:, 0] / case["T"] + total.log()}
    if op == "backward":
        return {"grad": _gradient(st, st["stats"], st["weight"] * st["grad_loss"])}
    stats = _stats(st)
    ids, t, rho, on = _lists(st)
    log_q = (st["student"].gather(1, ids).double() - stats[:, :1]) / case["T"] - stats[:, 1:2].double()
    log_rest = (stats[:, 2] - stats[:, 1]).double()
    other = torch.where(rho > 0, rho * (rho.clamp(min=1e-300).log() - log_rest), 0.0)
    loss = torch.where(on, ((t * (t.log() - log_q)).sum(-1) + other) * st["weight"], 0.0).float()
    got = {"loss": loss, "stats": stats}
    if case["grad"]:
        got["grad"] = _gradient(st, stats, st["weight"])
    return got


def run(st):
    if not own:
        return _plain(st)
    from block_diffusion_draft_dflash_gb300 import _lib
    case = st["case"]
    op = case["op"]
    if op == "sample":
        _lib.sample(st["logits"], st["u"], st["token"], st["ws"], temperature=st["temperature"], top_k=st["top_k"],
                    top_p=st["top_p"], min_p=st["min_p"], group=case["group"], logprob=st["logprob"], n_kept=st["n_kept"])
        return {"token": st["token"], "n_kept": st["n_kept"], "logprob": st["logprob"]}
    if op == "top":
        _lib.top_logits(st["logits"], case["T"], st["id"], st["val"], st["lse"], st["ws"])
        return {"id": st["id"], "val": st["val"], "lse": st["lse"]}
    teacher = (st["id"], st["val"], st["lse"])
    if op == "backward":
        _lib.distill_backward(st["student"], *teacher, case["T"], st["stats"], st["grad"], st["ws"], grad_loss=st["grad_loss"],
                              teacher_row=st["teacher_row"], weight=st["weight"])
        return {"grad": st["grad"]}
    _lib.distill(st["student"], *teacher, case["T"], st["loss"], st["stats"], st["ws"], teacher_row=st["teacher_row"],
                 weight=st["weight"], grad=st["grad"])
    got = {"loss": st["loss"], "stats": st["stats"]}
    return {**got, "grad": st["grad"]} if case["grad"] else got


# ------------------------------------------------------------------------------------------------ exact values
def _exact_row(l, u, T, k, p, low):
    """One row's draw: token, kept tokens, log-probability (64 bits, token after token of the sorted row)."""
    live = (l > -math.inf).nonzero()[:, 0]
    if T == 0:
        return int(l.argmax()), 1, 0.0
    x, place = (l[live] / T).sort(descending=True, stable=True)
    if k > 0:
        x = x[:k]
    n = x.numel()
    log_mass = x.logcumsumexp(0)
    if p < 1:
        n = min(n, 1 + int((log_mass[:-1] < math.log(p) + log_mass[-1]).sum()))
    if low > 0:
        n = min(n, int((x - x[0] >= math.log(low)).sum()))
    at = int((log_mass[:n] <= (math.log(u) if u > 0 else -math.inf) + log_mass[n - 1]).sum()) if n > 1 else 0
    at = min(at, n - 1)
    return int(live[place[at]]), n, float(x[at] - log_mass[n - 1])


def exact(case, seed):
    st = prepare(case, seed)
    op, T = case["op"], case.get("T")
    if op == "sample":
        each = [st[n].tolist() for n in ("temperature", "top_k", "top_p", "min_p")]
        u = st["u"].tolist()
        rows = [_exact_row(st["logits"][r].double(), u[r], *(v[r // case["group"]] for v in each)) for r in range(case["rows"])]
        token, n, lp = zip(*rows)
        whole = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
        return {"token": whole(token), "n_kept": whole(n), "logprob": torch.tensor(lp, dtype=torch.float64)}
    if op == "top":
        x = st["logits"].double()
        return {"id": None, "val": None, "lse": (x / T).logsumexp(-1)}
    y = (st["student"].double() / T).log_softmax(-1)
    row = st["teacher_row"].tolist()
    loss, stats = torch.zeros(case["rows"], dtype=torch.float64), torch.zeros(case["rows"], 4, dtype=torch.float64)
    grad = torch.zeros_like(y)
    for r, a in enumerate(row):
        if a < 0:
            continue
        ids = st["id"][a].long()
        t = torch.exp(st["val"][a].double() / T - st["lse"][a].double())
        rho = max(0.0, 1.0 - float(t.sum()))
        other = torch.ones(case["V"], dtype=torch.bool, device=DEV)
        other[ids] = False
        log_rest = float(y[r][other].logsumexp(0))
        kl = float((t * (t.log() - y[r, ids])).sum()) + (rho * (math.log(rho) - log_rest) if rho > 0 else 0.0)
        w = float(st["weight"][r])
        loss[r] = w * kl
        m = float(st["student"][r].max())
        lse = float((st["student"][r].double() / T).logsumexp(0)) - m / T
        stats[r, :3] = torch.tensor([m, lse, lse + log_rest], dtype=torch.float64)
        if st["grad"] is not None:
            scale = w / T * (float(st["grad_loss"][r]) if op == "backward" else 1.0)
            d = y[r].exp() * (scale * (1 - rho / math.exp(log_rest)))
            d[ids] = (y[r, ids].exp() - t) * scale
            grad[r] = d
    if op == "backward":
        return {"grad": grad}
    return {"loss": loss, "stats": stats, "grad": grad} if case["grad"] else {"loss": loss, "stats": stats}
