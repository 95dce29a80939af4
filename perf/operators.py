"""The 4-bit key/value cache operators, as cases that can be timed and checked.

A cache holds keys and values as e2m1 codes in groups of 16 along the head dim,
one unsigned e5m3 scale byte per group (4.5 bits a value), in pages of
``page`` tokens:

    cache [pages, 2 (keys, values), Hkv, page / 16, D / 64, 576 bytes]

576 bytes hold 16 tokens x 64 head dims: 512 bytes of codes, 64 scale bytes.
With s a token's place among the 16 and x a head dim's among the 64:

    keys    code   byte ((s % 8) * 4 + x / 16) * 16 + (s / 8) * 8 + (x % 16) / 2
            scale  byte 512 + (s % 8) * 8 + (x / 16) * 2 + s / 8
    values  code   byte ((x / 8) * 4 + (s % 8) / 2) * 16 + (s / 8) * 8 + (s % 2) * 4 + (x % 8) / 2
            scale  byte 512 + (x / 16) * 16 + ((s % 8) / 2) * 4 + (s / 8) * 2 + s % 2

(even head dims in the low nibble). A group's scale is its largest magnitude
over 6, rounded to nearest even to five exponent bits and three bits of
mantissa (magnitudes above 61440 count as 61440); a code is the value over
the scale, rounded to nearest even in e2m1 and saturating.

Three operators:

    write   new tokens are quantised into a paged cache and read back
    read    the cached tokens of each sequence are read back to 16 bits
    decode  attention of a few query rows per sequence over the 4-bit cache

The plain forms below are elementary torch operations in 32 bits.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one decoded token of each running sequence enters the cache
        dict(name="write token", op="write", dtype="bf16", B=32, Hkv=8, D=512, page=64, lo=100, hi=16000, new_lo=1,
             new_hi=1, packed=False),
        # a ragged batch of drafted tokens, odd sizes, the smallest pages
        dict(name="write draft", op="write", dtype="fp16", B=7, Hkv=2, D=320, page=16, lo=0, hi=900, new_lo=0,
             new_hi=5, packed=False),
        # two long prompts in a padded batch, at the start of their sequences
        dict(name="write prompt", op="write", dtype="bf16", B=2, Hkv=8, D=512, page=64, lo=0, hi=0, new_lo=5000,
             new_hi=8192, packed=False),
        # packed prompt chunks behind what their sequences have cached
        dict(name="write packed chunks", op="write", dtype="fp16", B=6, Hkv=4, D=640, page=32, lo=0, hi=5000,
             new_lo=512, new_hi=6144, packed=True),
        # a short context of small heads, read back for a dense kernel
        dict(name="read short", op="read", dtype="fp16", B=3, Hkv=4, D=64, page=16, lo=300, hi=777, packed=False),
        # the cached prefixes of a packed batch, for chunked prefill
        dict(name="read packed prefixes", op="read", dtype="bf16", B=6, Hkv=8, D=512, page=64, lo=512, hi=6144,
             packed=True),
        # one sequence, a short context: latency
        dict(name="decode one", op="decode", dtype="bf16", B=1, Hkv=8, G=4, Nq=1, D=512, page=64, lo=2000, hi=2000,
             idle=0, causal=False),
        # the decode benchmark's workload
        dict(name="decode batch", op="decode", dtype="bf16", B=8, Hkv=8, G=4, Nq=1, D=512, page=64, lo=16384,
             hi=16384, idle=0, causal=False),
        # one very long context
        dict(name="decode long", op="decode", dtype="fp16", B=1, Hkv=8, G=4, Nq=1, D=512, page=128, lo=131000,
             hi=131000, idle=0, causal=False),
        # four drafted tokens per sequence, ragged contexts, idle batch slots
        dict(name="decode draft", op="decode", dtype="fp16", B=16, Hkv=4, G=4, Nq=4, D=320, page=16, lo=1, hi=8000,
             idle=2, causal=True),
        # many query heads on one kv head of the largest head dim
        dict(name="decode shared head", op="decode", dtype="bf16", B=4, Hkv=1, G=16, Nq=2, D=1024, page=64, lo=4000,
             hi=6000, idle=0, causal=True),
        # a large batch of short contexts, one query head per kv head
        dict(name="decode many short", op="decode", dtype="fp16", B=64, Hkv=16, G=1, Nq=1, D=128, page=16, lo=20,
             hi=1000, idle=5, causal=False),
    ]


def log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "read", "decode", "decode"])
    c = dict(op=op, dtype=rng.choice(["bf16", "fp16"]), Hkv=rng.choice([1, 2, 3, 4, 8, 16]),
             D=64 * rng.choice([1, 2, 3, 4, 5, 6, 8, 8, 8, 10, 12, 13, 16]), page=rng.choice([16, 32, 48, 64, 128, 256]))
    budget = 8 * 8 * 16384 * 512 if op == "decode" else 6 * 8 * 3000 * 512
    B = log_int(rng, 1, 64)
    hi = log_int(rng, 2, 60000)
    if op != "decode":
        hi = min(hi, 12000)
    hi = max(1, min(hi, budget // (B * c["Hkv"] * c["D"])))
    lo = rng.choice([hi, rng.randint(0, hi)])
    c.update(B=B, lo=lo, hi=hi)
    if op == "write":
        new = max(1, min(log_int(rng, 1, 8000), budget // (B * c["Hkv"] * c["D"])))
        c.update(new_hi=new, new_lo=rng.choice([new, rng.randint(0, new)]), packed=rng.random() < 0.4)
    elif op == "read":
        c.update(packed=rng.random() < 0.5)
    else:
        c.update(G=rng.choice([1, 2, 3, 4, 4, 8, 8, 16]), Nq=rng.choice([1, 1, 1, 2, 3, 4]), causal=rng.random() < 0.5,
                 idle=rng.choice([0, 0, 1]))
    return c


def some(case, lo, hi, salt):
    """B lengths in [lo, hi] that the case alone fixes, `hi` among them."""
    r = random.Random("%s %d %d %d" % (salt, case["B"], lo, hi))
    n = [r.randint(lo, hi) for _ in range(case["B"])]
    n[r.randrange(case["B"])] = hi
    return n


def lengths(case):
    n = some(case, case["lo"], case["hi"], "context")
    for i in range(min(case.get("idle", 0), case["B"] - 1)):  # idle batch slots hold no sequence
        n[(case["B"] // 2 + 3 * i) % case["B"]] = 0
    return n


def work(case):
    B, H, D, n = case["B"], case["Hkv"], case["D"], lengths(case)
    if case["op"] == "write":
        new = sum(some(case, case["new_lo"], case["new_hi"], "new"))
        v = 2 * new * H * D  # values: read in 16 bits, stored in 4.5, read, written in 16 bits
        return {"bytes": v * (2 + 9 / 16 + 9 / 16 + 2), "flops": 3 * v}
    if case["op"] == "read":
        v = 2 * sum(n) * H * D
        return {"bytes": v * (9 / 16 + 2), "flops": v}
    R = case["G"] * case["Nq"]
    v = 2 * sum(n) * H * D
    return {"bytes": v * 9 / 16 + B * H * R * (2 * D * 2 + 4) + 4 * sum(-(-x // case["page"]) for x in n),
            "flops": 2 * R * v}


# ------------------------------------------------- the cache, in torch operations
def scales(amax):
    """Group magnitudes -> (scale codes, the scales they stand for), in 64 bits: a magnitude that is six times a
    border between two scales has to be seen on it."""
    v = amax.double().clamp(max=61440.0)
    v = v / torch.full_like(v, 6.0)  # by a tensor: a division, not a product with a rounded 1/6
    m = torch.frexp(v)[0]  # in [1/2, 1): v / m is a power of two, without pow()
    unit = torch.where(v < 2.0 ** -14, 2.0 ** -17, v / torch.where(m > 0, m, 1.0) / 16)
    s = torch.round(v / unit) * unit  # half to even; a carry gives the next power of two
    bits = s.to(torch.float16).view(torch.int16)  # exact: three bits of mantissa, and a sixteen-bit float's exponents
    return (bits >> 7).to(torch.uint8), s


def quantise(x):
    """x [..., D] -> codes [..., D/2] (even head dims in the low nibbles) and scale codes [..., D/16]."""
    g = x.float().reshape(*x.shape[:-1], -1, 16)
    code, s = scales(g.abs().amax(-1))
    s = s.unsqueeze(-1)
    a = torch.where(s > 0, g.abs().double() / torch.where(s > 0, s, 1.0), 0.0).clamp(max=6.0)
    m = torch.where(a < 2, torch.round(2 * a), torch.where(a < 4, torch.round(a) + 2, torch.round(a / 2) + 4))
    n = (m.to(torch.uint8) | ((g < 0).to(torch.uint8) << 3)).reshape(*x.shape[:-1], -1, 2)
    return n[..., 0] | (n[..., 1] << 4), code


def tiles(cache, kv):
    """Views of a cache's code and scale bytes with a token's place in front:
    codes [pages, strip, s / 8, (s / 2) % 4, s % 2, Hkv, D / 64, ...], scales alike (s: the token's place in 16)."""
    P, _, H, S, C, _ = cache.shape
    code, scale = cache[:, kv, ..., :512], cache[:, kv, ..., 512:]
    if kv == 0:  # [s % 8 as (4, 2), x / 16, s / 8, (x % 16) / 2]
        code = code.view(P, H, S, C, 4, 2, 4, 2, 8).permute(0, 2, 7, 4, 5, 1, 3, 6, 8)
        scale = scale.view(P, H, S, C, 4, 2, 4, 2).permute(0, 2, 7, 4, 5, 1, 3, 6)
    else:        # [x / 8, (s % 8) / 2, s / 8, s % 2, (x % 8) / 2]
        code = code.view(P, H, S, C, 8, 4, 2, 2, 4).permute(0, 2, 6, 5, 7, 1, 3, 4, 8)
        scale = scale.view(P, H, S, C, 4, 4, 2, 2).permute(0, 2, 6, 5, 7, 1, 3, 4)
    return code, scale


def place(cache, table, b, pos):
    """Where token `pos` of sequence `b` is: (page, strip, s / 8, (s / 2) % 4, s % 2)."""
    page = cache.shape[3] * 16
    p = table[b, pos // page].long()
    s = pos % page
    return p, s // 16, (s // 8) % 2, (s // 2) % 4, s % 2


def put(cache, kv, at, x):
    """Quantises x [tokens, Hkv, D] into the cells `at`."""
    code, scale = tiles(cache, kv)
    q, s = quantise(x)
    T, H, D = x.shape
    code[at] = q.view(T, H, D // 64, 4, 8) if kv == 0 else q.view(T, H, D // 64, 8, 4)
    scale[at] = s.view(T, H, D // 64, 4)


def get(cache, kv, at):
    """The cells `at`, [tokens..., Hkv, D] in 32 bits."""
    code, scale = tiles(cache, kv)
    q, s = code[at], scale[at]
    s = (s.to(torch.int16) << 7).view(torch.float16).float()
    lead = q.shape[:-3]
    q = q.reshape(*lead, q.shape[-3], 32)
    table = torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), device=q.device)
    v = torch.stack([table[(q & 15).int()], table[(q >> 4).int()]], -1)
    v = v.reshape(*lead, q.shape[-2], 4, 16) * s.unsqueeze(-1)
    return v.reshape(*lead, -1)


# ------------------------------------------------------------------ states
def prepare(case, seed):
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    g = torch.Generator(dev).manual_seed(seed)
    host = random.Random(seed)
    dt, B, H, D, page = DTYPES[case["dtype"]], case["B"], case["Hkv"], case["D"], case["page"]
    n = lengths(case)
    new = some(case, case["new_lo"], case["new_hi"], "new") if case["op"] == "write" else [0] * B
    blocks = [-(-(x + y) // page) for x, y in zip(n, new)]
    pages = sum(blocks) + 2  # a pool has pages to spare
    order = list(range(pages))
    host.shuffle(order)
    width, used = max(1, max(blocks)), 0
    table = torch.full((B, width), -1, dtype=torch.int32)
    for b, k in enumerate(blocks):
        table[b, :k] = torch.tensor(order[used:used + k], dtype=torch.int32)
        used += k
    # keys: some channels are much larger than others, as behind a norm and a rotation; values: plain
    channel = torch.exp(0.4 * torch.randn(2, H, D, generator=g, device=dev))
    channel[0, :, :: max(1, D // 8)] *= 3

    def tokens(kv, count):
        return torch.randn(count, H, D, generator=g, device=dev) * channel[kv]

    cache = torch.zeros(pages, 2, H, page // 16, D // 64, 576, dtype=torch.uint8, device=dev)
    some_pages = max(1, (1 << 25) // (page * H * D))
    for p in range(0, pages, some_pages):  # every page holds what an earlier prompt left
        k = min(some_pages, pages - p)
        i = torch.arange(k * page, device=dev)
        at = place(cache, torch.arange(p, p + k, device=dev).unsqueeze(0), 0, i)
        for kv in (0, 1):
            put(cache, kv, at, tokens(kv, k * page).to(dt))
    st = dict(case=case, cache=cache, table=table.to(dev), dtype=dt,
              lens=torch.tensor(n, dtype=torch.int32, device=dev))
    if case["op"] == "decode":
        R = (B, H * case["G"], case["Nq"], D)
        st["q"] = (1.2 * torch.randn(R, generator=g, device=dev)).to(dt)
        return st
    count = new if case["op"] == "write" else n
    st["most"], st["total"] = max(count), sum(count)
    st["count"] = torch.tensor(count, dtype=torch.int32, device=dev)
    cu = [0]
    for x in count:
        cu.append(cu[-1] + x)
    st["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
    st["token_b"] = torch.repeat_interleave(torch.arange(B, device=dev), st["count"].long())
    st["token_i"] = torch.arange(cu[-1], device=dev) - st["cu"].long()[st["token_b"]]
    shape = (cu[-1], H, D) if case["packed"] else (B, H, st["most"], D)
    st["k_out"], st["v_out"] = (torch.zeros(shape, dtype=dt, device=dev) for _ in range(2))
    if case["op"] == "write":
        if case["packed"]:
            st["k"], st["v"] = (tokens(kv, cu[-1]).to(dt) for kv in (0, 1))
        else:  # a projection's output [B, N, H, D], seen as [B, H, N, D]
            st["k"], st["v"] = (tokens(kv, B * st["most"]).to(dt).view(B, st["most"], H, D).transpose(1, 2)
                                for kv in (0, 1))
    return st


# --------------------------------------------------------------------- run
def run(st):
    op, packed = st["case"]["op"], st["case"].get("packed")
    cache, table = st["cache"], st["table"]
    if own:
        import head_dim_flash_gb300 as ffpa

        if op == "decode":
            o, lse = ffpa.decode_fwd_kv4(st["q"], cache, table, st["lens"], causal=st["case"]["causal"])
            return {"o": o, "lse": lse}
        if packed:
            start = None
            if op == "write":
                start = st["lens"]
                ffpa.varlen_kv4_write(cache, table, st["k"], st["v"], st["cu"], st["most"], start=start)
            k, v = ffpa.varlen_kv4_read(cache, table, st["cu"], st["most"], k_out=st["k_out"], v_out=st["v_out"],
                                        start=start)
        else:
            start = None
            if op == "write":
                start = st["lens"]
                ffpa.kv4_write(cache, table, st["k"], st["v"], start=start, count=st["count"])
            k, v = ffpa.kv4_read(cache, table, st["count"], k_out=st["k_out"], v_out=st["v_out"], start=start)
        return {"k": k, "v": v}
    if op == "decode":
        return plain_decode(st)
    b, i = st["token_b"], st["token_i"]
    pos = i + st["lens"].long()[b] if op == "write" else i
    at = place(cache, table, b, pos)
    if op == "write":
        for kv, x in ((0, st["k"]), (1, st["v"])):
            put(cache, kv, at, x if packed else x[b, :, i])
    for kv, x in ((0, st["k_out"]), (1, st["v_out"])):
        y = get(cache, kv, at).to(st["dtype"])
        if packed:
            x.copy_(y)
        else:
            x[b, :, i] = y
    return {"k": st["k_out"], "v": st["v_out"]}


def plain_decode(st):
    q, cache, table, lens = st["q"], st["cache"], st["table"], st["lens"].long()
    B, Hq, Nq, D = q.shape
    H, L = cache.shape[2], table.shape[1] * cache.shape[3] * 16
    pos = torch.arange(L, device=q.device)
    at = place(cache, table.clamp(min=0), torch.arange(B, device=q.device).unsqueeze(1), pos.unsqueeze(0))
    k = get(cache, 0, at).transpose(1, 2)  # [B, Hkv, L, D]
    s = q.float().view(B, H, -1, D) @ k.transpose(2, 3) * (1.0 / math.sqrt(D))
    del k
    i = torch.arange(Nq, device=q.device).repeat(Hq // H)
    end = lens.unsqueeze(1).expand(B, i.numel())  # first key that a row does not see
    if st["case"]["causal"]:
        end = end - Nq + 1 + i
    s = torch.where(pos < end[:, None, :, None], s, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
    del s
    total = p.sum(-1, keepdim=True)
    v = get(cache, 1, at).transpose(1, 2)
    v = torch.where((pos < lens.unsqueeze(1))[:, None, :, None], v, 0.0)
    o = (p @ v) / torch.where(total == 0, 1.0, total)
    lse = m + torch.log(total)
    return {"o": o.view(B, Hq, Nq, D).to(q.dtype), "lse": lse.view(B, Hq, Nq)}


# ------------------------------------------------------- the definition, in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    B, H, D, page = case["B"], case["Hkv"], case["D"], case["page"]
    n, table, dev = lengths(case), st["table"].cpu(), st["cache"].device
    levels = torch.tensor(MAGNITUDES, dtype=torch.float64, device=dev)

    def rounded(x):  # [T, Hkv, D]: what the cache holds of it
        x = x.double().reshape(x.shape[0], H, D // 16, 16)
        a = x.abs().amax(-1, keepdim=True).clamp(max=61440.0)
        unit = torch.full_like(a, 2.0 ** -17)  # grows while sixteen steps do not reach a / 6
        for _ in range(40):
            unit = torch.where(a > 6 * 16 * unit, 2 * unit, unit)
        s = torch.round(a / (6 * unit)) * unit
        best = torch.zeros_like(x)
        off = x.abs().clone()
        for j in range(1, 8):  # the nearest level; of two as near, the one with an even code
            d = (x.abs() - levels[j] * s).abs()
            take = (d < off) | ((d == off) & (j % 2 == 0))
            best, off = torch.where(take, levels[j] * s, best), torch.where(take, d, off)
        return torch.where(x < 0, -best, best).reshape(x.shape[0], H, D)

    def held(b, kv, count):  # [count, Hkv, D]: the first cells of sequence b
        j = torch.arange(count, device=dev)
        d = torch.arange(D, device=dev)
        s, x = (j % 16).unsqueeze(1), (d % 64).unsqueeze(0)
        if kv == 0:
            byte = ((s % 8) * 4 + x // 16) * 16 + (s // 8) * 8 + (x % 16) // 2
            mul = 512 + (s % 8) * 8 + (x // 16) * 2 + s // 8
        else:
            byte = ((x // 8) * 4 + (s % 8) // 2) * 16 + (s // 8) * 8 + (s % 2) * 4 + (x % 8) // 2
            mul = 512 + (x // 16) * 16 + ((s % 8) // 2) * 4 + (s // 8) * 2 + s % 2
        base = (((j % page) // 16) * (D // 64)).unsqueeze(1) * 576 + (d // 64).unsqueeze(0) * 576
        blocks = -(-count // page)
        rows = st["cache"][table[b, :blocks].long().to(dev), kv].transpose(0, 1).reshape(H, blocks, -1)
        rows = rows.reshape(H, -1)
        base = base + (j // page).unsqueeze(1) * (page // 16 * (D // 64) * 576)
        out = torch.empty(count, H, D, dtype=torch.float64, device=dev)
        for h in range(H):
            c = rows[h][base + byte].int()
            c = torch.where((d % 2 == 1).unsqueeze(0), c >> 4, c & 15)
            f = rows[h][base + mul].double()
            m = torch.where(f < 8, f * 2.0 ** -17, (8 + f % 8) * torch.exp2(torch.floor(f / 8) - 18))
            out[:, h] = levels[(c & 7).long()] * m * torch.where(c > 7, -1.0, 1.0)
        return out

    if case["op"] != "decode":
        outs = [torch.zeros(st["k_out"].shape, dtype=torch.float64, device=dev) for _ in range(2)]
        cu, count = st["cu"].tolist(), st["count"].tolist()
        for b in range(B):
            for kv in (0, 1):
                if case["op"] == "read":
                    y = held(b, kv, n[b])
                elif case["packed"]:
                    y = rounded(st["kv"[kv]][cu[b]:cu[b + 1]])
                else:
                    y = rounded(st["kv"[kv]][b, :, :count[b]].transpose(0, 1))
                if case["packed"]:
                    outs[kv][cu[b]:cu[b + 1]] = y
                else:
                    outs[kv][b, :, :count[b]] = y.transpose(0, 1)
        return {"k": outs[0], "v": outs[1]}

    Hq, Nq, G = H * case["G"], case["Nq"], case["G"]
    o = torch.zeros(B, Hq, Nq, D, dtype=torch.float64, device=dev)
    lse = torch.full((B, Hq, Nq), -math.inf, dtype=torch.float64, device=dev)
    for b in range(B):
        if n[b] == 0:
            continue
        k, v = held(b, 0, n[b]), held(b, 1, n[b])
        for i in range(Nq):
            e = n[b] - Nq + 1 + i if case["causal"] else n[b]
            if e <= 0:
                continue
            s = torch.einsum("hgd,jhd->hgj", st["q"][b, :, i].double().view(H, G, D), k[:e]) / math.sqrt(D)
            lse[b, :, i] = torch.logsumexp(s, -1).view(Hq)
            o[b, :, i] = torch.einsum("hgj,jhd->hgd", torch.softmax(s, -1), v[:e]).reshape(Hq, D)
    return {"o": o, "lse": lse}
