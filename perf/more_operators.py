"""Cases for the operators that make and use token distributions around a training step:
sampling from logits (temperature, top-k, top-p, min-p, from given random numbers), a
teacher's top logits with the log sum of the rest, and the distillation loss on them with
its gradient.

`run` computes them in their plain form (elementary torch operations, in 32 bits, in 64
where a border decides about whole tokens) while `own` is false, and through the framework's
entry points while it is true; `exact` gives the same outputs in 64 bits."""
import math
import random

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}
MOST_TOP = 1024                                                     # entries of a teacher's row
LARGEST = {"sample": 1024 * 128256 * 2, "top": 4096 * 128256 * 2, "distill": 4096 * 128256 * 2}   # bytes of logits


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # one answer, one token at a time, with the usual filters: the smallest call, latency counts
        sample("sample_one", 1, 32000, "bf16", temperature=0.8, top_k=50, top_p=0.95),
        # a serving batch where every request has settings of its own (one in eight greedy)
        sample("sample_mixed_batch", 64, 128256, "bf16", mixed=True),
        # a step of rollouts for the policy loss: the whole distribution at temperature 1
        sample("sample_rollout", 1024, 128256, "bf16"),
        # fp32 logits of an odd vocabulary, nucleus sampling
        sample("sample_nucleus_f32", 500, 50257, "f32", temperature=0.7, top_p=0.9),
        # early in training: thousands of tokens in the nucleus; rows inside a padded vocabulary
        sample("sample_flat_nucleus", 2000, 32003, "bf16", top_p=0.95, min_p=0.002, scale=0.4, pad=61),
        # the teacher's side of a distillation step: few tokens, a micro-batch, odd fp32 rows
        top("top_few_tokens", 8, 32000, "bf16", k=20),
        top("top_batch", 4096, 128256, "bf16", k=64),
        top("top_odd_vocab_f32", 1023, 50257, "f32", k=100, temperature=2.0),
        # the student's side: few tokens
        distill("distill_few_tokens", 8, 32000, "bf16", k=20, gradient=True, rest=True),
        # a micro-batch of long answers with a large vocabulary, prompts masked
        distill("distill_batch", 4096, 128256, "bf16", k=64, gradient=True, rest=True, masked=0.25),
        # fp32 logits of an odd vocabulary, a teacher that kept its top entries alone, some rows fewer
        distill("distill_odd_vocab_f32", 1023, 50257, "f32", k=100, gradient=True, rest=False, masked=0.1,
                temperature=2.0, ragged=0.2),
        # evaluation: forward alone, many entries, rows inside a padded vocabulary
        distill("distill_score", 2000, 32003, "bf16", k=256, gradient=False, rest=True, masked=0.5, pad=61),
    ]


def sample(name, rows, vocab, dtype, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, mixed=False, scale=1.0, pad=0):
    return {"name": name, "op": "sample", "rows": rows, "vocab": vocab, "dtype": dtype, "temperature": temperature,
            "top_k": top_k, "top_p": top_p, "min_p": min_p, "mixed": mixed, "scale": scale, "pad": pad}


def top(name, rows, vocab, dtype, k, temperature=1.0, scale=1.0, pad=0):
    return {"name": name, "op": "top", "rows": rows, "vocab": vocab, "dtype": dtype, "k": k, "temperature": temperature,
            "scale": scale, "pad": pad}


def distill(name, rows, vocab, dtype, k, gradient, rest, masked=0.0, temperature=1.0, ragged=0.0, scale=1.0, pad=0):
    return {"name": name, "op": "distill", "rows": rows, "vocab": vocab, "dtype": dtype, "k": k, "gradient": gradient,
            "rest": rest, "masked": masked, "temperature": temperature, "ragged": ragged, "scale": scale, "pad": pad}


def spread(rng, least, most):
    """A whole number between least and most, spread over the logarithm."""
    return max(least, min(most, int(round(math.exp(rng.uniform(math.log(least), math.log(most)))))))


def draw(rng):
    op = rng.choice(("sample", "sample", "top", "distill"))
    dtype = rng.choice(("bf16", "f32"))
    vocab = spread(rng, 1000, 131072)
    rows = spread(rng, 1, max(1, min(8192, LARGEST[op] // (4 * vocab * SIZE[dtype]))))
    temperature = rng.choice((1.0, rng.uniform(0.5, 2.0)))
    more = {"scale": rng.choice((1.0, rng.uniform(0.1, 1.2))), "pad": rng.choice((0, rng.randrange(1, 128)))}
    if op == "sample":
        c = sample("", rows, vocab, dtype, rng.choice((temperature, temperature, 0.0)),
                   rng.choice((0, spread(rng, 1, 2000))), rng.choice((1.0, rng.uniform(0.05, 0.999))),
                   rng.choice((0.0, rng.uniform(0.001, 0.3))), rng.random() < 0.3, **more)
    elif op == "top":
        c = top("", rows, vocab, dtype, spread(rng, 1, min(MOST_TOP, vocab - 1)), temperature, **more)
    else:
        c = distill("", rows, vocab, dtype, spread(rng, 1, min(MOST_TOP, vocab - 1)), rng.random() < 0.75,
                    rng.random() < 0.6, rng.choice((0.0, rng.uniform(0.0, 0.6))), temperature,
                    rng.choice((0.0, rng.uniform(0.0, 0.5))), **more)
    del c["name"]
    return c


def work(case):
    rows, logits = case["rows"], case["rows"] * case["vocab"]
    size = SIZE[case["dtype"]]
    if case["op"] == "sample":
        settings = 4 * 4 * rows if case["mixed"] else 0
        return {"bytes": logits * size + rows * (4 + 8 + 4 + 4) + settings, "flops": 4 * logits}
    if case["op"] == "top":
        return {"bytes": logits * size + rows * (case["k"] * (size + 8) + 4), "flops": 4 * logits}
    live = rows - int(rows * case["masked"])
    entries = live * case["k"] * (size + 8) + rows * (4 + 4) + (live * 4 if case["rest"] else 0)
    wrote = logits * size if case["gradient"] else 0
    return {"bytes": live * case["vocab"] * size + wrote + entries + 4,
            "flops": live * case["vocab"] * (6 if case["gradient"] else 4)}


# ------------------------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return {"sample": prepare_sample, "top": prepare_top, "distill": prepare_distill}[case["op"]](case, g)


def normal_logits(case, n, g):
    """n rows of logits in fp32: a few tokens far above the rest, as a trained model has."""
    z = torch.randn(n, case["vocab"] + case["pad"], device="cuda", generator=g)
    return (z * 2.5 + 0.35 * z ** 3) * case["scale"]


def row_chunks(rows, vocab, least=1 << 27):
    step = max(1, least // vocab)
    return [(i, min(rows, i + step)) for i in range(0, rows, step)]


def prepare_logits(case, g):
    whole = torch.empty(case["rows"], case["vocab"] + case["pad"], device="cuda", dtype=TYPES[case["dtype"]])
    for a, b in row_chunks(case["rows"], case["vocab"]):
        whole[a:b] = normal_logits(case, b - a, g)
    return whole[:, :case["vocab"]]


def prepare_sample(case, g):
    rows = case["rows"]
    s = {"op": "sample", "logits": prepare_logits(case, g), "uniform": torch.rand(rows, device="cuda", generator=g)}
    if not case["mixed"]:
        return s | {k: case[k] for k in ("temperature", "top_k", "top_p", "min_p")}

    def some(share, on, off):   # the setting `on` in a share of the rows, `off` in the others
        return torch.where(torch.rand(rows, device="cuda", generator=g) < share, on, off)

    u = torch.rand(3, rows, device="cuda", generator=g)
    off = torch.zeros(rows, device="cuda")
    return s | {"temperature": some(0.875, 0.5 + u[0], off),
                "top_k": some(0.5, torch.exp2(10 * u[1]).round(), off).int(),
                "top_p": some(0.6, 0.8 + 0.19 * u[2], off + 1.0),
                "min_p": some(0.3, 0.02 + 0.1 * u[0], off)}


def prepare_top(case, g):
    return {"op": "top", "logits": prepare_logits(case, g), "k": case["k"], "temperature": case["temperature"]}


def prepare_distill(case, g):
    N, V, k, dt = case["rows"], case["vocab"], case["k"], TYPES[case["dtype"]]
    dev = "cuda"
    whole = torch.empty(N, V + case["pad"], device=dev, dtype=dt)
    value = torch.empty(N, k, device=dev, dtype=dt)
    index = torch.empty(N, k, device=dev, dtype=torch.int64)
    rest = torch.empty(N, device=dev) if case["rest"] else None
    for a, b in row_chunks(N, V):
        teacher = normal_logits(case, b - a, g)
        # a student on its way: the same tokens are likely, its logits are off by a little
        whole[a:b] = 0.85 * teacher + 0.7 * torch.randn(teacher.shape, device=dev, generator=g)
        teacher = teacher[:, :V].to(dt).float()
        v, index[a:b] = teacher.topk(k, dim=1)
        value[a:b] = v
        if rest is not None:
            teacher.scatter_(1, index[a:b], float("-inf"))
            rest[a:b] = torch.logsumexp(teacher.div_(case["temperature"]), 1)
    weight = torch.ones(N, device=dev)
    off = int(N * case["masked"])
    weight[torch.randperm(N, device=dev, generator=g)[:off]] = 0.0
    weight /= max(1, N - off)
    if case["ragged"] > 0:   # some rows keep fewer entries; the places behind them hold -1
        cut = torch.randint(1, k + 1, (N,), device=dev, generator=g)
        cut = torch.where(torch.rand(N, device=dev, generator=g) < case["ragged"], cut, k)
        index.masked_fill_(torch.arange(k, device=dev) >= cut[:, None], -1)
    return {"op": "distill", "logits": whole[:, :V], "value": value, "index": index, "weight": weight, "rest": rest,
            "temperature": case["temperature"],
            "dlogits": torch.empty(N, V, device=dev, dtype=dt) if case["gradient"] else None}


# ------------------------------------------------------------------------------- one pass
def run(state):
    op = state["op"]
    if own:
        return {"sample": own_sample, "top": own_top, "distill": own_distill}[op](state)
    return {"sample": plain_sample, "top": plain_top, "distill": plain_distill}[op](state)


def own_sample(s):
    from tiled_newton_schulz_tile_amd.sampling import sample as sample_tokens
    got = sample_tokens(s["logits"], s["uniform"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                        min_p=s["min_p"])
    return {"token": got.token, "logp": got.logp, "kept": got.kept}


def column(x, rows, dtype, device):
    """A setting as a column: one number for all rows, or one a row."""
    return x[rows, None].to(dtype) if torch.is_tensor(x) else torch.full((1, 1), x, dtype=dtype, device=device)


def plain_sample(s):
    N, V = s["logits"].shape
    parts = [plain_sample_rows(s, slice(a, b)) for a, b in row_chunks(N, V)]
    return {k: torch.cat([p[k] for p in parts]) for k in ("token", "logp", "kept")}


def plain_sample_rows(s, rows):
    dev = s["logits"].device
    z = s["logits"][rows].double() + 0.0   # (-0 is 0)
    V = z.shape[1]
    T, k, p, least = (column(s[n], rows, torch.float64, dev) for n in ("temperature", "top_k", "top_p", "min_p"))
    greedy = T == 0
    y = (z - z.amax(1, keepdim=True)) / torch.where(greedy, 1.0, T)
    e = y.exp()
    order = z.sort(dim=1, descending=True, stable=True).indices
    first = e.gather(1, order)
    sums = first.cumsum(1)
    before = torch.cat((torch.zeros_like(sums[:, :1]), sums[:, :-1]), 1)
    place = torch.arange(V, device=dev)
    k = torch.where((k > 0) & (k < V), k, V).long().expand(len(z), 1)
    keep = (place < k) & ((p >= 1) | (before < p * sums.gather(1, k - 1))) & (first >= least.clamp(max=1))
    keep = torch.where(greedy, False, keep) | (place == 0)
    keep = torch.zeros_like(keep).scatter_(1, order, keep)
    total = e.sum(1)
    sums = torch.where(keep, e, 0).cumsum(1)
    mass = sums[:, -1]
    token = (sums <= (s["uniform"][rows].double() * mass)[:, None]).sum(1).clamp(max=V - 1)
    logp = y.gather(1, token[:, None])[:, 0] - total.log()
    greedy = greedy[:, 0].expand(len(z))
    return {"token": token, "logp": torch.where(greedy, 0.0, logp).float(),
            "kept": torch.where(greedy, 1.0, mass / total).float()}


def own_top(s):
    from tiled_newton_schulz_tile_amd.distill import top_logits
    got = top_logits(s["logits"], s["k"], temperature=s["temperature"])
    return {"value": got.value, "index": got.index, "rest": got.rest}


def plain_top(s):
    k, out = s["k"], []
    for a, b in row_chunks(*s["logits"].shape):
        value, index = (s["logits"][a:b].float() + 0.0).sort(dim=1, descending=True, stable=True)
        y = value[:, k:] / s["temperature"]
        rest = (y - y[:, :1]).exp().sum(1).log() + y[:, 0]
        out.append((value[:, :k].to(s["logits"].dtype), index[:, :k], rest))
    return {n: torch.cat([x[i] for x in out]) for i, n in enumerate(("value", "index", "rest"))}


def own_distill(s):
    from tiled_newton_schulz_tile_amd.distill import distill_loss
    got = distill_loss(s["logits"], s["value"], s["index"], s["weight"], rest=s["rest"], temperature=s["temperature"],
                       dlogits=s["dlogits"])
    return {"loss": got.loss, "kl": got.kl} | ({} if s["dlogits"] is None else {"dlogits": got.dlogits})


def plain_distill(s):
    N, V = s["logits"].shape
    tau = 1.0 / s["temperature"]
    entry = (s["index"] >= 0) & (s["index"] < V)
    live = (s["weight"] != 0)[:, None]
    index = torch.where(entry, s["index"], 0)
    t = torch.where(entry, s["value"].float() * tau, -torch.inf)
    if s["rest"] is not None:
        t = torch.cat((t, s["rest"][:, None]), 1)
    t = t - t.amax(1, keepdim=True)
    logq = t - t.exp().sum(1, keepdim=True).log()
    q = logq.exp()
    logq = torch.where(q > 0, logq, 0.0)
    z = torch.where(live, s["logits"], 0.0).float() * tau
    z = z - z.amax(1, keepdim=True)
    e = z.exp()
    total = e.sum(1, keepdim=True)
    named = q[:, :entry.shape[1]]
    logp = z.gather(1, index) - total.log()
    kl = (named * (logq[:, :entry.shape[1]] - logp)).sum(1)
    share = 1 / total
    if s["rest"] is not None:
        mine = torch.where(entry, index, V)
        others = torch.cat((e, torch.zeros_like(total)), 1).scatter_(1, mine, 0.0).sum(1, keepdim=True)
        kl = kl + q[:, -1] * (logq[:, -1] - (others / total).log()[:, 0])
        share = share - q[:, -1:] / others
    kl = torch.where(live[:, 0], kl, 0.0)
    out = {"loss": (s["weight"] * kl).sum(), "kl": kl}
    if s["dlogits"] is None:
        return out
    grad = e * share
    at = torch.where(entry, e.gather(1, index) / total - named, grad.gather(1, index))
    grad = torch.cat((grad, torch.zeros_like(total)), 1).scatter_(1, torch.where(entry, index, V), at)[:, :V]
    s["dlogits"].copy_(torch.where(live, grad * (s["weight"] * tau)[:, None], 0.0))
    return out | {"dlogits": s["dlogits"]}


# ------------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"sample": exact_sample, "top": exact_top, "distill": exact_distill}[case["op"]](s)


def ranked(logits):
    """Per token one whole number, unlike any other of its row, that grows from the largest logit to the smallest and
    among equal ones with the index."""
    bits = (logits.float() + 0.0).view(torch.int32).long()
    up = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits)        # orders as the numbers do
    return (0x7FFFFFFF - up) * (1 << 31) + torch.arange(logits.shape[1], device=logits.device)


def exact_sample(s):
    N, V = s["logits"].shape
    dev, out = s["logits"].device, []
    for a, b in row_chunks(N, V, 1 << 26):
        rows = slice(a, b)
        T, k, p, least = (column(s[n], rows, torch.float64, dev).expand(b - a, 1)
                          for n in ("temperature", "top_k", "top_p", "min_p"))
        z = s["logits"][rows].double()
        rank = ranked(s["logits"][rows])
        line = rank.sort(dim=1).values
        lse = torch.logsumexp(z / torch.where(T > 0, T, 1.0), 1, keepdim=True)
        prob = torch.exp(z / torch.where(T > 0, T, 1.0) - lse)
        sums = prob.gather(1, line % (1 << 31)).cumsum(1)
        count = torch.where(k > 0, k.clamp(max=V), V).long()
        target = p * sums.gather(1, count - 1)
        count = torch.where(p < 1, torch.minimum(count, torch.searchsorted(sums, target) + 1), count)
        edge = z.amax(1, keepdim=True) + T * torch.log(least.clamp(max=1.0))   # log 0: no edge
        count = torch.minimum(count, (z >= edge).sum(1, keepdim=True).clamp(min=1))
        count = torch.where(T > 0, count, 1)
        keep = rank <= line.gather(1, count - 1)
        sums = torch.where(keep, prob, 0.0).cumsum(1)
        mass = sums[:, -1:]
        token = torch.searchsorted(sums, s["uniform"][rows, None].double() * mass, right=True)
        logp = torch.log(prob.gather(1, token))
        out.append([torch.where(T > 0, x, y)[:, 0] for x, y in
                    ((token, rank.argmin(1, keepdim=True)), (logp, 0.0), (mass, 1.0))])
    return {n: torch.cat([x[i] for x in out]) for i, n in enumerate(("token", "logp", "kept"))}


def exact_top(s):
    N, V = s["logits"].shape
    k, out = s["k"], []
    for a, b in row_chunks(N, V, 1 << 26):
        z = s["logits"][a:b]
        index = ranked(z).sort(dim=1).values % (1 << 31)
        y = z.double() / s["temperature"]
        out.append((z.double().gather(1, index[:, :k]), index[:, :k], torch.logsumexp(y.gather(1, index[:, k:]), 1)))
    return {n: torch.cat([x[i] for x in out]) for i, n in enumerate(("value", "index", "rest"))}


def exact_distill(s):
    """The loss by its definition, and its gradient by torch's derivative of that."""
    N, V = s["logits"].shape
    dev, T = s["logits"].device, s["temperature"]
    kl = torch.zeros(N, dtype=torch.float64, device=dev)
    loss = torch.zeros((), dtype=torch.float64, device=dev)
    grad = torch.zeros(N, V, dtype=torch.float64, device=dev) if s["dlogits"] is not None else None
    for a, b in row_chunks(N, V, 1 << 26):
        rows = torch.nonzero(s["weight"][a:b])[:, 0] + a
        if not rows.numel():
            continue
        w = s["weight"][rows].double()
        entry = (s["index"][rows] >= 0) & (s["index"][rows] < V)
        at = torch.where(entry, s["index"][rows], 0)
        teacher = torch.where(entry, s["value"][rows].double() / T, -torch.inf)
        if s["rest"] is not None:
            teacher = torch.cat((teacher, s["rest"][rows, None].double()), 1)
        logq = torch.log_softmax(teacher, 1)
        q = logq.exp()
        with torch.enable_grad():
            z = s["logits"][rows].double().requires_grad_(grad is not None)
            lp = torch.log_softmax(z / T, 1)
            student = lp.gather(1, at)
            if s["rest"] is not None:
                named = torch.zeros(lp.shape, dtype=torch.int32, device=dev).scatter_add_(1, at, entry.int()) > 0
                student = torch.cat((student, torch.logsumexp(lp.masked_fill(named, -torch.inf), 1, keepdim=True)), 1)
            term = torch.where(q > 0, q * (torch.where(q > 0, logq, 0.0) - student), 0.0).sum(1)
            part = (w * term).sum()
        kl[rows] = term.detach()
        loss += part.detach()
        if grad is not None:
            grad[rows] = torch.autograd.grad(part, z)[0]
    return {"loss": loss, "kl": kl} | ({} if grad is None else {"dlogits": grad})
