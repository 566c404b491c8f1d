"""Cases for the operators of a training step around the HiMuon update: the clipped policy
loss with its gradient, the gradient norm over many tensors, and the AdamW step over many
tensors with states in 32 or in 8 bits.

`run` computes them in their plain form (elementary torch operations in 32 bits) while
`own` is false, and through the framework's entry points while it is true; `exact` gives
the same outputs in 64 bits.

The parameters of a case are views of one flat buffer per kind, as a training program that
buckets its tensors keeps them; the gaps between tensors hold zeros, which every update
here leaves at zero, so a plain form works on the flat buffer."""
import math
import random

import torch

own = False

BLOCK = 256          # elements that share a scale of the 8-bit states
E4M3_MAX = 448.0     # largest value of the 8-bit type
TINY = 2.0 ** -100   # blocks whose largest magnitude is below are held as zeros
DITHER_M, DITHER_R = 0x9E3779B1, 0x85EBCA6B   # odd multipliers of the dither sequences
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # the loss of a few sampled tokens: the smallest call, latency counts
        policy("policy_few_tokens", 8, 32000, "bf16", gradient=True, masked=0.0, kl=0.0, temperature=1.0),
        # a micro-batch of long answers with a large vocabulary, prompts masked
        policy("policy_batch", 4096, 128256, "bf16", gradient=True, masked=0.25, kl=0.05, temperature=1.0),
        # an odd vocabulary (rows at every alignment), fp32 logits, sampled at a temperature
        policy("policy_odd_vocab_f32", 1023, 50257, "f32", gradient=True, masked=0.1, kl=0.02, temperature=0.7),
        # scoring sampled tokens under a frozen policy: forward alone, rows inside a padded vocabulary
        policy("policy_score", 2000, 32003, "bf16", gradient=False, masked=0.5, kl=0.1, temperature=1.0, pad=61),
        # the clip factor of a stack's norm gains: latency
        norm("norm_gains", "f32", count=65, least=4096, most=4096),
        # the whole gradient of a 16-layer decoder stack (2048 wide, 8192 hidden)
        norm("norm_stack", "bf16", count=112, least=2048 * 2048, most=2048 * 8192, two_sizes=True),
        # what HiMuon leaves to AdamW in a 32-layer stack: the gains, and nothing else
        adamw("adamw_gains", 32, "f32", "f32", count=65, least=4096, most=4096),
        # an embedding and a head of 32000 x 4096, fp32 master weights, bf16 gradients
        adamw("adamw_embeddings", 32, "f32", "bf16", count=2, least=32000 * 4096, most=32000 * 4096),
        # odd sizes packed without gaps (a flattened bucket), bf16 weights
        adamw("adamw_bucket", 32, "bf16", "bf16", count=301, least=1, most=400000, packed=True),
        # the same three with 8-bit states
        adamw("adamw8_gains", 8, "f32", "f32", count=65, least=4096, most=4096),
        adamw("adamw8_embeddings", 8, "f32", "bf16", count=2, least=32000 * 4096, most=32000 * 4096),
        adamw("adamw8_ragged", 8, "bf16", "bf16", count=301, least=1, most=400000),
    ]


def policy(name, tokens, vocab, dtype, gradient, masked, kl, temperature, pad=0):
    return {"name": name, "op": "policy", "tokens": tokens, "vocab": vocab, "dtype": dtype, "gradient": gradient,
            "masked": masked, "kl": kl, "temperature": temperature, "pad": pad}


def norm(name, grad, count, least, most, packed=False, two_sizes=False):
    return {"name": name, "op": "norm", "grad": grad, "count": count, "least": least, "most": most,
            "packed": packed, "two_sizes": two_sizes}


def adamw(name, bits, weight, grad, count, least, most, packed=False):
    return {"name": name, "op": "adamw", "bits": bits, "weight": weight, "grad": grad, "count": count,
            "least": least, "most": most, "packed": packed, "two_sizes": False}


def spread(rng, least, most):
    """A whole number between least and most, spread over the logarithm."""
    return max(least, min(most, int(round(math.exp(rng.uniform(math.log(least), math.log(most)))))))


def draw(rng):
    kind = rng.choice(("policy", "norm", "adamw32", "adamw8"))
    if kind == "policy":
        vocab = spread(rng, 1000, 131072)
        tokens = spread(rng, 1, min(8192, 4096 * 128256 // (2 * vocab)))
        c = policy("", tokens, vocab, rng.choice(("bf16", "f32")), rng.random() < 0.75,
                   rng.choice((0.0, rng.uniform(0.0, 0.6))), rng.choice((0.0, rng.uniform(0.01, 0.2))),
                   rng.choice((1.0, rng.uniform(0.5, 1.5))), rng.choice((0, rng.randrange(1, 128))))
    else:
        count = spread(rng, 1, 400)
        total = spread(rng, 3000, 200_000_000)   # the most that the tensors may hold together
        most = max(1, total // count)
        least = rng.choice((most, max(1, most // 100), 1))
        c = (norm("", rng.choice(("bf16", "f32")), count, least, most, packed=rng.random() < 0.5) if kind == "norm" else
             adamw("", 32 if kind == "adamw32" else 8, rng.choice(("f32", "bf16")), rng.choice(("f32", "bf16")), count,
                   least, most, packed=kind == "adamw32" and rng.random() < 0.5))
    del c["name"]
    return c


def sizes(case):
    """Element counts of a case's tensors (the same for every seed)."""
    n, least, most = case["count"], case["least"], case["most"]
    if case["two_sizes"]:   # per layer four square projections and three wide ones
        return [most if i % 7 >= 4 else least for i in range(n)]
    rng = random.Random(n * 1000003 + most * 17 + least)
    return [spread(rng, least, most) if most > least else most for _ in range(n)]


def layout(case):
    """(starts, sizes, length) of the tensors in a flat buffer: packed without gaps, or each
    at a multiple of 256 elements."""
    starts, at = [], 0
    size = sizes(case)
    for n in size:
        starts.append(at)
        at += n if case["packed"] else -(-n // BLOCK) * BLOCK
    return starts, size, at


def work(case):
    if case["op"] == "policy":
        rows = case["tokens"] - int(case["tokens"] * case["masked"])
        read = rows * case["vocab"] * SIZE[case["dtype"]]
        wrote = case["tokens"] * case["vocab"] * SIZE[case["dtype"]] if case["gradient"] else 0
        words = case["tokens"] * (8 + 4 * 4 + 4)   # label, weight, advantage, old, ref; the log probability out
        return {"bytes": read + wrote + words + 16, "flops": rows * case["vocab"] * (6 if case["gradient"] else 4)}
    n = sum(sizes(case))
    if case["op"] == "norm":
        return {"bytes": n * SIZE[case["grad"]] + 8, "flops": 2 * n}
    state = 16 if case["bits"] == 32 else 4 + 16 / BLOCK
    return {"bytes": n * (2 * SIZE[case["weight"]] + SIZE[case["grad"]] + state), "flops": 14 * n}


# ------------------------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return prepare_policy(case, g) if case["op"] == "policy" else prepare_tensors(case, g, seed)


def prepare_policy(case, g):
    N, V, dt = case["tokens"], case["vocab"], TYPES[case["dtype"]]
    dev = "cuda"

    def normal(std):
        return torch.randn(N, device=dev, generator=g) * std

    whole = torch.empty(N, V + case["pad"], device=dev, dtype=dt)
    label = torch.empty(N, device=dev, dtype=torch.int64)
    logp = torch.empty(N, device=dev)
    rows = max(1, (1 << 28) // V)
    for i in range(0, N, rows):
        z = torch.randn(min(rows, N - i), V + case["pad"], device=dev, generator=g)
        z = (z * 2.5 + 0.35 * z ** 3).to(dt)        # a few tokens far above the rest, as a trained model has
        whole[i:i + rows] = z
        z = z[:, :V].float() / case["temperature"]
        noise = torch.empty_like(z).exponential_(generator=g)
        label[i:i + rows] = (z - noise.log_()).argmax(1)   # sampled from the policy
        z = z - z.amax(1, keepdim=True)
        logp[i:i + rows] = (z.gather(1, label[i:i + rows, None]) - z.exp().sum(1, keepdim=True).log())[:, 0]
        del z, noise
    # the policy has moved a little since the tokens were sampled.  A token whose ratio lies on an edge of the
    # clip range has no gradient that rounding could not turn over: those are moved off it
    moved = normal(0.15)
    for edge in (math.log(0.8), math.log(1.28)):
        moved = torch.where((moved - edge).abs() < 1e-3, moved + 2e-3, moved)
    weight = torch.ones(N, device=dev)
    off = int(N * case["masked"])
    weight[torch.randperm(N, device=dev, generator=g)[:off]] = 0.0
    weight /= max(1, N - off)
    return {"op": "policy", "logits": whole[:, :V], "label": label, "weight": weight, "advantage": normal(1.0),
            "old": logp - moved, "ref": logp + normal(0.2) if case["kl"] > 0 else None, "kl": case["kl"],
            "temperature": case["temperature"], "clip": (0.2, 0.28),
            "dlogits": torch.empty(N, V, device=dev, dtype=dt) if case["gradient"] else None}


def prepare_tensors(case, g, seed):
    starts, size, length = layout(case)
    dev = "cuda"

    used = torch.zeros(length + 1, device=dev, dtype=torch.int32)
    used.index_add_(0, torch.tensor(starts + [s + n for s, n in zip(starts, size)], device=dev),
                    torch.tensor([1] * len(size) + [-1] * len(size), device=dev, dtype=torch.int32))
    used = used.cumsum(0, dtype=torch.int32)[:length] > 0

    def normal(std, dt):
        x = torch.randn(length, device=dev, generator=g)
        return x.mul_(std).mul_(used).to(dt)

    s = {"op": case["op"], "starts": starts, "sizes": size}
    # gradients: most entries small, a few large
    grad = normal(1.0, torch.float32)
    grad = grad.mul_(0.01).mul_(1 + grad.abs() * 50)
    s["grad"] = grad.to(TYPES[case["grad"]])
    if case["op"] == "norm":
        return s
    s["weight"] = normal(0.02, TYPES[case["weight"]])
    # states of a run in progress: moments of gradients like these
    m, r = normal(0.004, torch.float32), normal(0.01, torch.float32).abs_()
    r = r.add_(0.002).mul_(used)
    s |= {"bits": case["bits"], "lr": 1e-3, "beta1": 0.9, "beta2": 0.999, "eps": 1e-8, "decay": 0.1, "t": 50,
          "scale": torch.full((1,), 0.8, device=dev)}
    if case["bits"] == 32:
        s["m"], s["v"] = m, r.square_()
        return s
    rng = random.Random(seed)
    s["dither"] = (rng.getrandbits(32), rng.getrandbits(32))
    for name, x in (("m", m), ("r", r)):
        x = x.view(-1, BLOCK)
        unit = x.abs().amax(1) / E4M3_MAX
        x /= torch.where(unit > 0, unit, 1.0)[:, None]
        s[name] = x.clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(-1)
        s[name + "_scale"] = unit
    return s


# ------------------------------------------------------------------------------- one pass
def run(state):
    op = state["op"]
    if own:
        return {"policy": own_policy, "norm": own_norm, "adamw": own_adamw}[op](state)
    return {"policy": plain_policy, "norm": plain_norm, "adamw": plain_adamw}[op](state)


def own_policy(s):
    from tiled_newton_schulz_tile_amd.policy import policy_loss
    got = policy_loss(s["logits"], s["label"], s["weight"], s["advantage"], old_logp=s["old"], ref_logp=s["ref"],
                      clip=s["clip"], kl_coef=s["kl"], temperature=s["temperature"], dlogits=s["dlogits"])
    return {"stats": got.stats, "logp": got.logp} | ({} if s["dlogits"] is None else {"dlogits": got.dlogits})


def plain_policy(s):
    V, tau = s["logits"].shape[1], 1.0 / s["temperature"]
    live = (s["weight"] != 0) & (s["label"] >= 0) & (s["label"] < V)
    label = torch.where(live, s["label"], 0)[:, None]
    z = torch.where(live[:, None], s["logits"], 0.0).float() * tau
    z = z - z.amax(1, keepdim=True)
    e = z.exp()
    total = e.sum(1, keepdim=True)
    logp = (z.gather(1, label) - total.log())[:, 0]
    ratio = (logp - s["old"]).exp()
    u = ratio * s["advantage"]
    c = ratio.clamp(1 - s["clip"][0], 1 + s["clip"][1]) * s["advantage"]
    d = s["ref"] - logp if s["ref"] is not None else torch.zeros_like(logp)
    w = torch.where(live, s["weight"], 0.0)
    part, kl = -torch.minimum(u, c), d.exp() - d - 1
    stats = [(w * (part + s["kl"] * kl)).sum(), (w * part).sum(), (w * kl).sum(), (w * (u > c)).sum()]
    out = {"stats": torch.stack(stats), "logp": torch.where(live, logp, 0.0)}
    if s["dlogits"] is None:
        return out
    coef = torch.where(u > c, 0.0, -u) + s["kl"] * (1 - d.exp())
    coef = torch.where(live, w * coef * tau, 0.0)[:, None]
    grad = e * (-coef / total)
    grad.scatter_add_(1, label, coef)
    s["dlogits"].copy_(grad)
    return out | {"dlogits": s["dlogits"]}


def views(s, *names):
    """The tensors of a case: per tensor, its view of each named buffer."""
    return [tuple(s[k][a:a + n] for k in names) for a, n in zip(s["starts"], s["sizes"])]


def own_norm(s):
    from tiled_newton_schulz_tile_amd.adamw import GradNorm
    if "plan" not in s:
        s["plan"] = GradNorm([v[0] for v in views(s, "grad")])
    return {"norm_and_factor": s["plan"].compute(max_norm=1.0)}


def plain_norm(s):
    norm = s["grad"].float().square().sum().sqrt()
    return {"norm_and_factor": torch.stack((norm, (1.0 / (norm + 1e-6)).clamp(max=1.0)))}


def own_adamw(s):
    from tiled_newton_schulz_tile_amd.adamw import AdamW
    if "plan" not in s:
        if s["bits"] == 32:
            tensors = views(s, "weight", "grad", "m", "v")
        else:   # the scales of a tensor: those of its blocks of 256
            tensors = [v + (s["m_scale"][a // BLOCK:-(-(a + n) // BLOCK)], s["r_scale"][a // BLOCK:-(-(a + n) // BLOCK)])
                       for v, a, n in zip(views(s, "weight", "grad", "m", "r"), s["starts"], s["sizes"])]
        s["plan"] = AdamW(tensors, betas=(s["beta1"], s["beta2"]), eps=s["eps"], weight_decay=s["decay"])
    s["plan"].step(s["lr"], s["t"], scale=s["scale"], dither=s.get("dither"))
    return kept(s)


def kept(s):
    names = ("weight", "m", "v") if s["bits"] == 32 else ("weight", "m", "m_scale", "r", "r_scale")
    return {k: s[k] for k in names}


def plain_adamw(s):
    b1, b2 = s["beta1"], s["beta2"]
    g = s["grad"].float() * s["scale"]
    if s["bits"] == 32:
        m, v = s["m"], s["v"]
    else:
        m = (s["m"].float().view(-1, BLOCK) * s["m_scale"][:, None]).view(-1)
        v = (s["r"].float().view(-1, BLOCK) * s["r_scale"][:, None]).view(-1).square()
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    root = v.sqrt()
    step = m / (root * (1 / math.sqrt(1 - b2 ** s["t"])) + s["eps"])
    w = s["weight"].float() * (1 - s["lr"] * s["decay"]) - (s["lr"] / (1 - b1 ** s["t"])) * step
    s["weight"].copy_(w)
    if s["bits"] == 32:
        s["m"].copy_(m)
        s["v"].copy_(v)
    else:
        at = place(s, m.device)
        hold(m, at * DITHER_M + s["dither"][0], s["m"], s["m_scale"])
        hold(root, at * DITHER_R + s["dither"][1], s["r"], s["r_scale"], least=2.0 ** -9)
    return kept(s)


def place(s, device):
    """Each element's index inside its tensor, by blocks of 256."""
    first = torch.tensor(s["starts"], device=device) // BLOCK
    block = torch.arange(s["m_scale"].numel(), device=device)
    block = block - first[torch.searchsorted(first, block, right=True) - 1]
    return block[:, None] * BLOCK + torch.arange(BLOCK, device=device)


def hold(x, sequence, code, scale, least=0.0):
    """x in 8 bits (e4m3 values times one scale per block): the magnitude over the scale is rounded to a
    neighbour, down or up as the dither says, whose 16 bits are the upper half of `sequence` mod 2^32; a nonzero
    value becomes `least` at least."""
    x = x.view(-1, BLOCK)
    most = x.abs().amax(1)
    most = torch.where(most < TINY, 0.0, most)
    y = x.abs() * torch.where(most > 0, E4M3_MAX / most, 0.0)[:, None]
    dither = (((sequence >> 16) & 0xFFFF) << 4 | 8).to(torch.int32)
    low = torch.where(y < 2.0 ** -6, 2.0 ** -6, 0.0)   # below 2^-6 the values are 2^-9 apart, as just above it
    bits = (y + low).view(torch.int32)
    y = ((bits + dither) & ~0xFFFFF).view(torch.float32) - low
    y = torch.where(x != 0, y.clamp(least, E4M3_MAX), 0.0)
    y = torch.where(most[:, None] > 0, y, 0.0)
    code.copy_(torch.copysign(y, x).view(-1))
    scale.copy_(most / E4M3_MAX)


# ------------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"policy": exact_policy, "norm": exact_norm, "adamw": exact_adamw}[case["op"]](s)


def exact_policy(s):
    N, V = s["logits"].shape
    dev, tau = s["logits"].device, 1.0 / s["temperature"]
    low, high = 1 - s["clip"][0], 1 + s["clip"][1]
    logp = torch.zeros(N, dtype=torch.float64, device=dev)
    stats = torch.zeros(4, dtype=torch.float64, device=dev)
    grad = torch.zeros(N, V, dtype=torch.float64, device=dev) if s["dlogits"] is not None else None
    rows = max(1, (1 << 27) // V)
    for i in range(0, N, rows):
        at = torch.nonzero(s["weight"][i:i + rows])[:, 0] + i
        if not at.numel():
            continue
        z = s["logits"][at].double() * tau
        y = s["label"][at]
        lse = torch.logsumexp(z, 1)
        lp = z[torch.arange(len(at), device=dev), y] - lse
        w, A = s["weight"][at].double(), s["advantage"][at].double()
        rho = torch.exp(lp - s["old"][at].double())
        above, below = (A > 0) & (rho > high), (A < 0) & (rho < low)
        off = above | below
        bound = torch.where(above, high, low).double()
        surrogate = torch.where(off, bound, rho) * A
        d = s["ref"][at].double() - lp if s["ref"] is not None else torch.zeros_like(lp)
        kl = torch.expm1(d) - d
        stats += torch.stack(((w * (s["kl"] * kl - surrogate)).sum(), -(w * surrogate).sum(), (w * kl).sum(),
                              (w * off).sum()))
        logp[at] = lp
        if grad is not None:
            dlp = w * tau * (torch.where(off, 0.0, -rho * A) - s["kl"] * torch.expm1(d))
            p = torch.exp(z - lse[:, None]) * -dlp[:, None]
            p[torch.arange(len(at), device=dev), y] += dlp
            grad[at] = p
    return {"stats": stats, "logp": logp} | ({} if grad is None else {"dlogits": grad})


def exact_norm(s):
    total = sum(float((x.double() ** 2).sum()) for x in s["grad"].split(1 << 28))
    return {"norm_and_factor": torch.tensor([math.sqrt(total), min(1.0, 1.0 / (math.sqrt(total) + 1e-6))],
                                            dtype=torch.float64)}


def exact_adamw(s):
    wide = {k: [] for k in kept(s)}
    length, step = s["grad"].numel(), 1 << 26
    starts = torch.tensor(s["starts"], device=s["grad"].device)
    scale, b1, b2 = float(s["scale"]), s["beta1"], s["beta2"]
    for a in range(0, length, step):
        part = slice(a, min(a + step, length))
        g = s["grad"][part].double() * scale
        if s["bits"] == 32:
            m, v = s["m"][part].double(), s["v"][part].double()
        else:
            blocks = slice(a // BLOCK, (part.stop + BLOCK - 1) // BLOCK)
            m = s["m"][part].double() * s["m_scale"][blocks].double().repeat_interleave(BLOCK)
            v = (s["r"][part].double() * s["r_scale"][blocks].double().repeat_interleave(BLOCK)) ** 2
        m += (g - m) * (1 - b1)
        v += (g * g - v) * (1 - b2)
        hat = m / (1 - b1 ** s["t"]) / (torch.sqrt(v / (1 - b2 ** s["t"])) + s["eps"])
        w = s["weight"][part].double()
        wide["weight"].append(w - s["lr"] * (hat + s["decay"] * w))
        if s["bits"] == 32:
            wide["m"].append(m)
            wide["v"].append(v)
            continue
        index = torch.arange(part.start, part.stop, device=g.device)
        index = index - starts[torch.searchsorted(starts, index, right=True) - 1]
        for name, x, k, least in (("m", m, 0, 0.0), ("r", torch.sqrt(v), 1, 2.0 ** -9)):
            u = ((index * (DITHER_M, DITHER_R)[k] + s["dither"][k]) % 2 ** 32 // 2 ** 16 + 0.5) / 65536
            peak = x.abs().view(-1, BLOCK).amax(1)
            peak = torch.where(peak < TINY, 0.0, peak)
            each = peak.repeat_interleave(BLOCK)
            y = torch.where(each > 0, x.abs() / each * E4M3_MAX, 0.0)
            gap = torch.exp2(torch.floor(torch.log2(y.clamp(min=2.0 ** -6))) - 3)   # between neighbours near y
            y = torch.floor(y / gap + u) * gap
            y = torch.where((x != 0) & (each > 0), y.clamp(least, E4M3_MAX), 0.0)
            wide[name].append(torch.sign(x) * y)
            wide[name + "_scale"].append(peak / E4M3_MAX)
    return {k: torch.cat(v) for k, v in wide.items()}
