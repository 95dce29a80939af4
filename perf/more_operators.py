"""Operators around a 16-bit key/value cache, as cases that can be timed and checked.

Four operators:

    rope     rotary positions on queries and keys, alone or with the gradient:
             pair p of a head's first `rot` dims is turned by position * theta_p,
             (x, y) -> m (x cos - y sin, x sin + y cos); pairs are (p, p + rot / 2)
             or, interleaved, (2p, 2p + 1); theta_p = base^(-2p / rot), scaled for
             long contexts ("linear", "ntk", "yarn")
    shared   attention of a few query rows per sequence over the keys of a prefix
             that the whole batch shares and then over keys of their own
    weigh    attention of a few query rows per sequence over their cache, which also
             adds to a score per cached token the attention weight that it got from
             the rows of its kv head
    evict    a cache is cut to `keep` tokens per kv head: the `recent` last ones and,
             of the others, those with the largest scores (of equal ones the earlier),
             in their order

The plain forms below are elementary torch operations in 32 bits (angles in 64).
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one decoded token of each running sequence gets its position: latency
        dict(name="rope token", op="rope", dtype="bf16", B=32, Hq=32, Hkv=8, N=1, D=512, rot=512, interleaved=False,
             scaling="none", factor=1.0, far=16000, packed=False, grad=False),
        # a training step's queries and keys, forward and gradient
        dict(name="rope train", op="rope", dtype="bf16", B=1, Hq=32, Hkv=8, N=8192, D=512, rot=512, interleaved=False,
             scaling="none", factor=1.0, far=0, packed=False, grad=True),
        # packed prompt chunks behind long contexts, interleaved pairs on a part of the head, frequencies by parts
        dict(name="rope packed part", op="rope", dtype="fp16", B=6, Hq=16, Hkv=4, N=4000, D=320, rot=128,
             interleaved=True, scaling="yarn", factor=16.0, far=120000, packed=True, grad=False),
        # a few sequences behind a short common prompt: latency
        dict(name="shared few", op="shared", dtype="bf16", B=4, Hkv=8, G=4, Nq=1, D=512, Np=2000, lo=1, hi=90,
             causal=False),
        # a batch behind one system prompt with documents
        dict(name="shared batch", op="shared", dtype="bf16", B=32, Hkv=8, G=4, Nq=1, D=512, Np=16384, lo=20, hi=1000,
             causal=False),
        # drafted tokens of a large batch, ragged
        dict(name="shared draft", op="shared", dtype="fp16", B=64, Hkv=4, G=4, Nq=4, D=320, Np=8000, lo=4, hi=300,
             causal=True),
        # a few samples over one very long context
        dict(name="shared long", op="shared", dtype="bf16", B=16, Hkv=8, G=4, Nq=1, D=512, Np=131000, lo=0, hi=500,
             causal=False),
        # one sequence, a short context: latency
        dict(name="weigh one", op="weigh", dtype="bf16", B=1, Hkv=8, G=4, Nq=1, D=512, N=2048, lo=2000, hi=2000,
             causal=False),
        # the decode benchmark's workload
        dict(name="weigh batch", op="weigh", dtype="bf16", B=8, Hkv=8, G=4, Nq=1, D=512, N=16384, lo=16384, hi=16384,
             causal=False),
        # four drafted tokens per sequence, ragged contexts
        dict(name="weigh draft", op="weigh", dtype="fp16", B=16, Hkv=4, G=4, Nq=4, D=320, N=8000, lo=1, hi=8000,
             causal=True),
        # small ragged caches, some short enough to stay whole
        dict(name="evict short", op="evict", dtype="fp16", B=7, Hkv=2, D=320, N=900, lo=100, hi=900, keep=512,
             recent=100),
        # the decode benchmark's cache cut to half
        dict(name="evict batch", op="evict", dtype="bf16", B=8, Hkv=8, D=512, N=16384, lo=16384, hi=16384, keep=8192,
             recent=1024),
    ]


def log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "shared", "shared", "weigh", "evict"])
    c = dict(op=op, dtype=rng.choice(["bf16", "fp16"]), Hkv=rng.choice([1, 2, 3, 4, 8, 16]))
    H, G = c["Hkv"], rng.choice([1, 2, 4, 4, 7, 8, 16])
    if op == "rope":
        D = 32 * rng.choice([2, 3, 4, 6, 10, 16, 16, 20, 32])
        grad = rng.random() < 0.4
        B = log_int(rng, 1, 64)
        most = 8192 * 40 * 512 // (B * H * (G + 1) * D * (1 if grad else 2))
        N = max(1, min(log_int(rng, 1, 16000), most))
        c.update(B=B, Hq=H * G, N=N, D=D, rot=rng.choice([D, D, max(16, D // 4 // 16 * 16), D // 2 // 16 * 16]),
                 interleaved=rng.random() < 0.5, scaling=rng.choice(["none", "linear", "ntk", "yarn"]),
                 factor=rng.choice([2.0, 8.0, 40.0]), far=rng.choice([0, log_int(rng, 10, 1000000)]),
                 packed=rng.random() < 0.4, grad=grad)
        return c
    D = 64 * rng.choice([1, 2, 3, 4, 5, 6, 8, 8, 8, 10, 12, 13, 16])
    c["D"] = D
    if op == "shared":
        B, Nq = log_int(rng, 2, 128), rng.choice([1, 1, 1, 2, 3, 4])
        rows = B * G * Nq
        cells = 131000 * 8 * 512  # cached values of the prefix; with many rows fewer
        Np = min(log_int(rng, 1, 131000), max(1, min(cells, cells * 64 // rows) // (H * D)))
        hi = min(log_int(rng, 1, 2000), max(1, 32 * 1000 * 8 * 512 // (B * H * D)))
        c.update(B=B, G=G, Nq=Nq, Np=Np, hi=hi, lo=rng.choice([hi, rng.randint(0, hi)]), causal=rng.random() < 0.5)
        return c
    B = log_int(rng, 1, 64)
    N = max(1, min(log_int(rng, 2, 60000), 8 * 8 * 16384 * 512 // (B * H * D)))
    hi = rng.choice([N, rng.randint(1, N)])
    c.update(B=B, N=N, hi=hi, lo=rng.choice([hi, rng.randint(0, hi)]))
    if op == "weigh":
        c.update(G=G, Nq=rng.choice([1, 1, 1, 2, 3, 4]), causal=rng.random() < 0.5)
    else:
        keep = rng.randint(1, hi)
        c.update(keep=keep, recent=rng.choice([0, rng.randint(0, keep)]))
    return c


def some(case, lo, hi, salt):
    """B lengths in [lo, hi] that the case alone fixes, `hi` among them."""
    r = random.Random("%s %d %d %d" % (salt, case["B"], lo, hi))
    n = [r.randint(lo, hi) for _ in range(case["B"])]
    n[r.randrange(case["B"])] = hi
    return n


def tokens_of(case):
    """New tokens of each sequence of a rotary case."""
    return some(case, (case["N"] + 3) // 4, case["N"], "new") if case["packed"] else [case["N"]] * case["B"]


def work(case):
    B, D = case["B"], case["D"]
    if case["op"] == "rope":
        v = sum(tokens_of(case)) * (case["Hq"] + case["Hkv"]) * D  # read and written once per direction
        ways = 2 if case["grad"] else 1
        return {"bytes": 4 * v * ways, "flops": 3 * v * case["rot"] / D * ways}
    H = case["Hkv"]
    n = some(case, case["lo"], case["hi"], "context")
    if case["op"] == "evict":
        kept = sum(min(x, case["keep"]) for x in n) * H
        return {"bytes": 4 * sum(n) * H + kept * (2 * 2 * 2 * D + 4 + 4), "flops": sum(n) * H}
    R = case["G"] * case["Nq"]
    io = B * H * R * (2 * D * 2 + 4)
    if case["op"] == "shared":
        return {"bytes": 4 * H * D * (case["Np"] + sum(n)) + io, "flops": 4 * H * R * D * (B * case["Np"] + sum(n))}
    return {"bytes": 4 * H * D * sum(n) + io + 8 * H * sum(n), "flops": 4 * H * R * D * sum(n)}


# ------------------------------------------------------------- frequencies
BASE, ORIGINAL = 10000.0, 4096


def frequencies(case):
    """Radians per position of each pair, in 64 bits, and the factor on the result."""
    rot, s, how = case["rot"], case["factor"], case["scaling"]
    p = torch.arange(rot // 2, dtype=torch.float64)
    base = BASE * s ** (rot / (rot - 2)) if how == "ntk" else BASE
    theta = base ** (-2 * p / rot)
    if how == "linear":
        return theta / s, 1.0
    if how == "yarn":  # pairs that turn 32 times within the original length stay, those below one turn are stretched
        keep = ((ORIGINAL * theta / (2 * math.pi) - 1) / (32 - 1)).clamp(0, 1)
        return theta * keep + theta / s * (1 - keep), 0.1 * math.log(s) + 1
    return theta, 1.0


# ------------------------------------------------------------------ states
def prepare(case, seed):
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    g = torch.Generator(dev).manual_seed(seed)
    dt, B, D, H = DTYPES[case["dtype"]], case["B"], case["D"], case["Hkv"]

    def randn(*shape):
        return torch.randn(shape, generator=g, device=dev)

    # keys: some channels are much larger than others, as behind a norm; values: plain
    channel = torch.exp(0.4 * randn(H, 1, D))
    channel[..., :: max(1, D // 8)] *= 3

    def rows(b, h, n, scale=1.0):
        """A projection's output [b, n, h, D], seen as [b, h, n, D]."""
        out = torch.empty((b, n, h, D), dtype=dt, device=dev)
        for i in range(b):
            out[i] = (randn(h, n, D) * scale).transpose(0, 1)
        return out.transpose(1, 2)

    def cache(b, n, scale=1.0):
        out = torch.empty((b, H, n, D), dtype=dt, device=dev)
        for i in range(b):
            for h in range(H):
                out[i, h] = randn(n, D) * (scale if isinstance(scale, float) else scale[h])
        return out

    st = dict(case=case, dtype=dt)
    if case["op"] == "rope":
        n, Hq, far = tokens_of(case), case["Hq"], case["far"]
        start = torch.randint(0, far + 1, (B,), generator=g, device=dev, dtype=torch.int32)
        st["theta"], st["m"] = frequencies(case)
        st["theta"] = st["theta"].to(dev)
        if own:
            import head_dim_flash_gb300 as ffpa

            st["plan"] = ffpa.rope_plan(case["rot"], base=BASE, interleaved=case["interleaved"],
                                        scaling=case["scaling"], factor=case["factor"], original_len=ORIGINAL,
                                        device=dev)
        st["start"] = start
        names = ("q", "k", "gq", "gk") if case["grad"] else ("q", "k")
        for name in names:
            h = Hq if name[-1] == "q" else H
            if case["packed"]:
                st[name] = randn(sum(n), h, D).to(dt)
            else:
                st[name] = rows(B, h, case["N"])
        if case["packed"]:
            cu = [0]
            for x in n:
                cu.append(cu[-1] + x)
            st["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
            b = torch.repeat_interleave(torch.arange(B, device=dev), torch.tensor(n, device=dev))
            st["pos"] = torch.arange(cu[-1], device=dev) - st["cu"].long()[b] + start.long()[b]  # [T]
            st["most"] = max(n)
        else:
            st["pos"] = start.long()[:, None] + torch.arange(case["N"], device=dev)  # [B, N]
        return st
    n = some(case, case["lo"], case["hi"], "context")
    st["lens"] = torch.tensor(n, dtype=torch.int32, device=dev)
    if case["op"] in ("shared", "weigh"):
        st["q"] = rows(B, H * case["G"], case["Nq"], 1.2)
    if case["op"] == "shared":
        st["kp"], st["vp"] = cache(1, case["Np"], channel), cache(1, case["Np"])
        st["k"], st["v"] = cache(B, max(1, case["hi"]), channel), cache(B, max(1, case["hi"]))
        return st
    st["k"], st["v"] = cache(B, case["N"], channel), cache(B, case["N"])
    # scores of earlier steps: a few tokens got much of the weight
    st["weights"] = torch.exp(2 * randn(B, H, case["N"])) * 0.01
    if case["op"] == "weigh":
        st["weights_out"] = torch.zeros_like(st["weights"])
    else:
        most = case["keep"]
        st["weights"][..., ::5] = st["weights"][..., :1]  # ties
        st["k_out"], st["v_out"] = (torch.zeros((B, H, most, D), dtype=dt, device=dev) for _ in range(2))
        st["weights_out"] = torch.zeros((B, H, most), device=dev)
        st["lens_out"] = torch.zeros_like(st["lens"])
    return st


# --------------------------------------------------------------------- run
def run(st):
    op = st["case"]["op"]
    return (run_own if own else {"rope": plain_rope, "shared": plain_shared, "weigh": plain_weigh,
                                 "evict": plain_evict}[op])(st)


def run_own(st):
    import head_dim_flash_gb300 as ffpa

    case, op = st["case"], st["case"]["op"]
    if op == "rope":
        q, k = st["q"], st["k"]
        if case["grad"]:
            q, k = q.detach().requires_grad_(), k.detach().requires_grad_()
        if case["packed"]:
            yq, yk = ffpa.varlen_rope(q, k, st["plan"], st["cu"], start=st["start"])
        else:
            yq, yk = ffpa.rope(q, k, st["plan"], start=st["start"])
        if not case["grad"]:
            return {"q": yq, "k": yk}
        dq, dk = torch.autograd.grad((yq, yk), (q, k), (st["gq"], st["gk"]))
        return {"q": yq.detach(), "k": yk.detach(), "dq": dq, "dk": dk}
    if op == "shared":
        o, lse = ffpa.decode_fwd_shared(st["q"], st["kp"], st["vp"], st["k"], st["v"], st["lens"],
                                        causal=case["causal"])
        return {"o": o, "lse": lse}
    if op == "weigh":
        o, lse, w = ffpa.decode_fwd_weights(st["q"], st["k"], st["v"], st["weights"], st["lens"],
                                            causal=case["causal"], weights_out=st["weights_out"])
        return {"o": o, "lse": lse, "weights": w}
    k, v, w, lens, kept = ffpa.kv_evict(st["k"], st["v"], st["weights"], st["lens"], case["keep"],
                                        recent=case["recent"], k_out=st["k_out"], v_out=st["v_out"],
                                        weights_out=st["weights_out"], lens_out=st["lens_out"])
    return {"k": k, "v": v, "weights": w, "lens": lens, "kept": kept}


def turn(x, st, sign):
    """x [B, H, N, D] or [T, H, D], each pair turned by its position."""
    case = st["case"]
    rot = case["rot"]
    angle = st["pos"].double()[..., None] * st["theta"]
    c, s = (torch.cos(angle) * st["m"]).float(), (torch.sin(angle) * st["m"]).float() * sign
    c, s = (t.unsqueeze(1) for t in (c, s))  # over the heads
    y = x.float()
    head, tail = y[..., :rot], y[..., rot:]
    if case["interleaved"]:
        a, b = head[..., 0::2], head[..., 1::2]
        head = torch.stack((a * c - b * s, a * s + b * c), -1).flatten(-2)
    else:
        a, b = head[..., :rot // 2], head[..., rot // 2:]
        head = torch.cat((a * c - b * s, a * s + b * c), -1)
    return torch.cat((head, tail), -1).to(x.dtype)


def plain_rope(st):
    out = {"q": turn(st["q"], st, 1), "k": turn(st["k"], st, 1)}
    if st["case"]["grad"]:
        out.update(dq=turn(st["gq"], st, -1), dk=turn(st["gk"], st, -1))
    return out


def ends(st, R, before=0):
    """First key that a row [B, R] does not see, of `before` shared keys and its sequence's own."""
    Nq = st["case"]["Nq"]
    n = st["lens"].long().unsqueeze(1) + before
    i = torch.arange(Nq, device=n.device).repeat(R // Nq)
    return n - Nq + 1 + i if st["case"]["causal"] else n.expand(-1, R)


def plain_shared(st):
    case, q = st["case"], st["q"]
    B, Hq, Nq, D = q.shape
    H, Np, Ns, R = case["Hkv"], case["Np"], st["k"].shape[2], Hq // case["Hkv"] * Nq
    end = ends(st, R, Np)[:, None, :, None]  # [B, 1, R, 1]
    rows = q.float().reshape(B, H, R, D) * (1.0 / math.sqrt(D))
    flat = rows.transpose(0, 1).reshape(H, B * R, D)
    dev = q.device
    s = (flat @ st["kp"][0].float().transpose(1, 2)).view(H, B, R, Np).transpose(0, 1)
    s = torch.where(torch.arange(Np, device=dev) < end, s, -math.inf)
    t = rows @ st["k"].float().transpose(2, 3)
    t = torch.where(torch.arange(Np, Np + Ns, device=dev) < end, t, -math.inf)
    m = torch.maximum(s.amax(-1, keepdim=True), t.amax(-1, keepdim=True))
    shift = torch.where(m == -math.inf, 0.0, m)
    s, t = torch.exp(s - shift), torch.exp(t - shift)
    total = s.sum(-1, keepdim=True) + t.sum(-1, keepdim=True)
    seen = torch.arange(Ns, device=dev) < st["lens"].unsqueeze(1)
    v = torch.where(seen[:, None, :, None], st["v"].float(), 0.0)
    o = (s.transpose(0, 1).reshape(H, B * R, Np) @ st["vp"][0].float()).view(H, B, R, D).transpose(0, 1) + t @ v
    o = o / torch.where(total == 0, 1.0, total)
    return {"o": o.reshape(B, Hq, Nq, D).to(q.dtype), "lse": (m + torch.log(total)).reshape(B, Hq, Nq)}


def plain_weigh(st):
    case, q = st["case"], st["q"]
    B, Hq, Nq, D = q.shape
    H, N, R = case["Hkv"], case["N"], Hq // case["Hkv"] * Nq
    pos = torch.arange(N, device=q.device)
    s = q.float().reshape(B, H, R, D) @ st["k"].float().transpose(2, 3) * (1.0 / math.sqrt(D))
    s = torch.where(pos < ends(st, R)[:, None, :, None], s, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total == 0, 1.0, total)
    seen = pos < st["lens"].unsqueeze(1)
    o = p @ torch.where(seen[:, None, :, None], st["v"].float(), 0.0)
    w = torch.where(seen[:, None], st["weights"] + p.sum(2), st["weights_out"])
    return {"o": o.reshape(B, Hq, Nq, D).to(q.dtype), "lse": (m + torch.log(total)).reshape(B, Hq, Nq), "weights": w}


def plain_evict(st):
    case, w, lens = st["case"], st["weights"], st["lens"].long()
    B, H, N = w.shape
    keep, recent, D = case["keep"], case["recent"], case["D"]
    pos = torch.arange(N, device=w.device)
    n = lens[:, None, None]
    whole = n <= keep
    late = (pos >= n - recent) | whole  # stay whatever their scores
    rank = torch.where(late, math.inf, w)
    rank = torch.where(pos < n, rank, -math.inf)  # behind the last token
    order = torch.argsort(rank, dim=-1, descending=True, stable=True)[..., :keep]
    stays = torch.zeros_like(w, dtype=torch.bool).scatter_(-1, order, True) & (pos < n)
    kept = torch.argsort((~stays).int(), dim=-1, stable=True)[..., :keep]
    count = torch.clamp(lens, max=keep)
    if kept.shape[-1] < keep:
        kept = torch.nn.functional.pad(kept, (0, keep - kept.shape[-1]))
    there = torch.arange(keep, device=w.device) < count[:, None, None]
    there = there.expand(B, H, keep)
    index = kept[..., None].expand(-1, -1, -1, D)
    for x, y in (("k", "k_out"), ("v", "v_out")):
        st[y].copy_(torch.where(there[..., None], torch.gather(st[x], 2, index), st[y]))
    st["weights_out"].copy_(torch.where(there, torch.gather(w, 2, kept), st["weights_out"]))
    st["lens_out"].copy_(count)
    return {"k": st["k_out"], "v": st["v_out"], "weights": st["weights_out"], "lens": st["lens_out"],
            "kept": torch.where(there, kept, -1).int()}


# ------------------------------------------------------- the definition, in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    dev = st["q"].device if "q" in st else st["k"].device
    n = some(case, case["lo"], case["hi"], "context") if case["op"] != "rope" else None
    H, D, B = case["Hkv"], case["D"], case["B"]
    if case["op"] == "rope":
        rot = case["rot"]
        first = torch.arange(rot // 2, device=dev) * (2 if case["interleaved"] else 1)
        other = first + (1 if case["interleaved"] else rot // 2)

        def turned(x, sign):
            y = x.double()
            out = y.clone()
            z = torch.polar(torch.full((), st["m"], dtype=torch.float64, device=dev),
                            sign * st["pos"].double()[..., None] * st["theta"])  # complex, [.., rot / 2]
            for h in range(y.shape[1]):
                w = torch.complex(y[:, h][..., first], y[:, h][..., other]) * z
                out[:, h, ..., first], out[:, h, ..., other] = w.real, w.imag
            return out

        out = {"q": turned(st["q"], 1), "k": turned(st["k"], 1)}
        if case["grad"]:
            out.update(dq=turned(st["gq"], -1), dk=turned(st["gk"], -1))
        return out
    if case["op"] == "evict":
        w = st["weights"].cpu()
        out = {x: st[x + "_out"].double() for x in ("k", "v", "weights")}
        lens = torch.tensor([min(x, case["keep"]) for x in n], dtype=torch.int32, device=dev)
        kept = torch.full((B, H, case["keep"]), -1, dtype=torch.int32)
        for b in range(B):
            for h in range(H):
                stay = list(range(n[b]))
                if n[b] > case["keep"]:
                    early = n[b] - case["recent"]
                    score = w[b, h].tolist()
                    best = sorted(range(early), key=lambda j: (-score[j], j))[:case["keep"] - case["recent"]]
                    stay = sorted(best) + stay[early:]
                j = torch.tensor(stay, dtype=torch.long)
                kept[b, h, :len(stay)] = j.int()
                j = j.to(dev)
                out["k"][b, h, :len(stay)] = st["k"][b, h, j].double()
                out["v"][b, h, :len(stay)] = st["v"][b, h, j].double()
                out["weights"][b, h, :len(stay)] = st["weights"][b, h, j].double()
        out.update(lens=lens, kept=kept.to(dev))
        return out
    G, Nq = case["G"], case["Nq"]
    Np = case["Np"] if case["op"] == "shared" else 0
    o = torch.zeros(B, H * G, Nq, D, dtype=torch.float64, device=dev)
    lse = torch.full((B, H * G, Nq), -math.inf, dtype=torch.float64, device=dev)
    total = st["weights_out"].double() if case["op"] == "weigh" else None
    for h in range(H):
        q = st["q"][:, h * G:(h + 1) * G].double() / math.sqrt(D)  # [B, G, Nq, D]
        if Np:
            kp, vp = st["kp"][0, h].double(), st["vp"][0, h].double()
            common = (q.reshape(-1, D) @ kp.T).view(B, G, Nq, Np)
        for b in range(B):
            k, v = st["k"][b, h, :n[b]].double(), st["v"][b, h, :n[b]].double()
            s = q[b] @ k.T
            if Np:
                s = torch.cat((common[b], s), -1)
            if case["causal"]:
                for i in range(Nq):
                    s[:, i, max(0, Np + n[b] - Nq + 1 + i):] = -math.inf
            z = torch.logsumexp(s, -1) if s.shape[-1] else torch.full((G, Nq), -math.inf, device=dev).double()
            lse[b, h * G:(h + 1) * G] = z
            p = torch.where(torch.isinf(z)[..., None], 0.0, torch.exp(s - z[..., None]))
            out = p[..., Np:] @ v
            if Np:
                out = out + (p[..., :Np].reshape(-1, Np) @ vp).view(G, Nq, D)
            o[b, h * G:(h + 1) * G] = out
            if total is not None:
                total[b, h, :n[b]] = st["weights"][b, h, :n[b]].double() + p.sum((0, 1))
    out = {"o": o, "lse": lse}
    if total is not None:
        out["weights"] = total
    return out
