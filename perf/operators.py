"""The operators around a quantised projection, as they are measured.

Four kinds of case, each with the plain form of its operator (elementary torch operations in 32 or
64 bits) and the framework's call:

  rope    rotary positions on the heads of a projection's output (strided rows, several position
          axes, part of the head, both pair layouts)
  lora    low-rank adapters of many requests added to a shared projection's output
  select  the key blocks that each block of queries attends to, by the product of block means
  attend  attention over those blocks, with the log of each row's softmax denominator
"""

import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BLOCK_Q, BLOCK_K = 128, 64


# ----------------------------------------------------------------------------------- the cases

def listed():
    return [
        # one token of one request: queries and keys of 40 heads each, straight from the qkv row
        rope("rope one token", rows=1, heads=80, spare=40, D=128, rot=128, axes=1, inter=True),
        # prompts of a model with a rotated half of each head, halves layout, scaled for positions
        # far beyond the trained ones
        rope("rope long prompts", rows=8191, heads=40, spare=8, D=128, rot=64, axes=1, inter=False,
             scaled=True, far=1000000),
        # a video's tokens: time, height and width turn sections of every query and key head
        rope("rope video", rows=32760, heads=80, spare=40, D=128, rot=128, axes=3, inter=True),
        # a step that adds one token to each of 64 requests, which share 16 adapters
        lora("lora one token each", M=64, K=5120, N=15360, R=16, adapters=16, requests=64),
        # prompts of nine requests, one in five without an adapter, with padding behind the last
        lora("lora ragged prompts", M=4099, K=13824, N=5120, R=32, adapters=5, requests=9, tail=35),
        # both halves of a guided sampling step, each a whole video
        lora("lora video", M=32760, K=5120, N=13824, R=64, adapters=2, requests=2),
        # one new token against the kept block means of a long context
        select("select one token", B=1, Hq=40, Hkv=40, Lq=1, Lk=32760, D=128, T=77, first=1, last=1),
        # a whole video at 15 % density
        select("select video", B=1, Hq=40, Hkv=40, Lq=32760, Lk=32760, D=128, T=77),
        # one new token over the blocks selected from a long context
        attend("attend one token", B=1, Hq=40, Hkv=40, Lq=1, Lk=32760, D=128, T=77, causal=True),
        # short prompts, fewer keys than a tile in places
        attend("attend short prompts", dtype="f16", B=3, Hq=8, Hkv=8, Lq=200, Lk=200, D=64, T=3,
               ragged=True),
        # ragged prompts with shared key heads, each row seeing only what came before it
        attend("attend causal prompts", B=2, Hq=32, Hkv=8, Lq=4099, Lk=4099, D=128, T=16,
               causal=True, ragged=True),
        # a whole video at 15 % density
        attend("attend video", B=1, Hq=40, Hkv=40, Lq=32760, Lk=32760, D=128, T=77),
    ]


def rope(name, rows, heads, spare, D, rot, axes, inter, scaled=False, far=0, dtype="bf16"):
    return dict(name=name, kind="rope", dtype=dtype, rows=rows, heads=heads, spare=spare, D=D, rot=rot,
                axes=axes, inter=inter, scaled=scaled, far=far)


def lora(name, M, K, N, R, adapters, requests, tail=0):
    return dict(name=name, kind="lora", dtype="bf16", M=M, K=K, N=N, R=R, adapters=adapters,
                requests=requests, tail=tail)


def select(name, B, Hq, Hkv, Lq, Lk, D, T, first=0, last=0, causal=False, ragged=False, dtype="bf16"):
    return dict(name=name, kind="select", dtype=dtype, B=B, Hq=Hq, Hkv=Hkv, Lq=Lq, Lk=Lk, D=D, T=T,
                first=first, last=last, causal=causal, ragged=ragged)


def attend(name, B, Hq, Hkv, Lq, Lk, D, T, causal=False, ragged=False, dtype="bf16"):
    return dict(name=name, kind="attend", dtype=dtype, B=B, Hq=Hq, Hkv=Hkv, Lq=Lq, Lk=Lk, D=D, T=T,
                causal=causal, ragged=ragged)


def draw(rng):
    def log(lo, hi):
        return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49))))))

    kind = rng.choice(("rope", "lora", "select", "attend"))
    if kind == "rope":
        D = 2 * rng.randint(16, 64)
        rows = log(1, 32760)
        heads = log(1, max(1, min(96, 32760 * 80 * 128 // (rows * D))))
        c = rope("", rows, heads, spare=rng.randint(0, 16), D=D,
                 rot=rng.choice((D, 2 * rng.randint(1, D // 2))), axes=rng.choice((1, 1, 2, 3)),
                 inter=rng.random() < 0.5, scaled=rng.random() < 0.4, far=rng.choice((0, 1000000)),
                 dtype=rng.choice(("bf16", "bf16", "f16", "f32")))
    elif kind == "lora":
        M = log(1, 32760)
        c = lora("", M, K=128 * log(2, 60), N=16 * log(16, 600), R=8 * log(1, 12),
                 adapters=rng.randint(1, 8), requests=log(1, min(M, 64)), tail=rng.choice((0, 0, 3)))
        c["tail"] = min(c["tail"], M - c["requests"])
    else:
        D = rng.choice((64, 128, 128))
        Hkv = rng.choice((1, 2, 4, 8))
        Hq = Hkv * rng.choice((1, 1, 2, 4))
        Lk = log(1, 32760)
        Lq = rng.choice((1, Lk, log(1, Lk)))
        nk = -(-Lk // BLOCK_K)
        B = rng.randint(1, 4)
        T = rng.randint(1, max(1, min(nk, round(0.25 * nk) + 3)))
        while B > 1 and B * Hq * Lq > 40 * 32760:
            B -= 1
        T = max(1, min(T, 40 * 32760 * 77 // (B * Hq * Lq)))
        causal, ragged = rng.random() < 0.4, rng.random() < 0.5
        dtype = rng.choice(("bf16", "bf16", "f16"))
        if kind == "select":
            c = select("", B, Hq, Hkv, Lq, Lk, D, T, first=rng.randint(0, 1), last=rng.randint(0, 2),
                       causal=causal, ragged=ragged, dtype=dtype)
        else:
            c = attend("", B, Hq, Hkv, Lq, Lk, D, T, causal=causal, ragged=ragged, dtype=dtype)
    del c["name"]
    return c


def lengths(case):
    """(query, key) lengths of the sequences of a batch: the first is full, others shorter where ragged."""
    rng = random.Random(f"{case['B']}/{case['Lq']}/{case['Lk']}")
    kl = [case["Lk"] if b == 0 or not case["ragged"] else rng.randint(1, case["Lk"]) for b in range(case["B"])]
    return [min(case["Lq"], n) for n in kl], kl


def visible(case):
    """For each sequence and query block: its rows, and how many keys its last row sees."""
    got = []
    for ql, kl in zip(*lengths(case)):
        for i in range(-(-case["Lq"] // BLOCK_Q)):
            rows = max(0, min(ql - i * BLOCK_Q, BLOCK_Q))
            last = i * BLOCK_Q + rows + kl - ql if case["causal"] else kl
            got.append((rows, max(0, min(last, kl)) if rows else 0))
    return got


def requests(case):
    """First row of each request (and the end of the last), and each request's adapter (-1: none)."""
    rng = random.Random(f"{case['M']}/{case['requests']}")
    rows = case["M"] - case["tail"]
    cuts = sorted(rng.sample(range(1, rows), case["requests"] - 1)) if case["requests"] > 1 else []
    ids = [-1 if case["requests"] > 4 and i % 5 == 4 else (7 * i) % case["adapters"] for i in range(case["requests"])]
    return [0, *cuts, rows], ids


# ---------------------------------------------------------------------------------- the inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return {"case": case, **{"rope": inputs_rope, "lora": inputs_lora, "select": inputs_select,
                             "attend": inputs_attend}[case["kind"]](case, seed, g)}


def randn(g, *shape, by=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=g, device="cuda") * by).to(dtype)


def inputs_rope(case, seed, g):
    n, axes = case["rot"] // 2, min(case["axes"], case["rot"] // 2)
    sizes = [n - (axes - 1) * (n // axes)] + [n // axes] * (axes - 1)
    inv = torch.cat([10000.0 ** (-torch.arange(s, dtype=torch.float64) / s) for s in sizes])
    scale = 1.0
    if case["scaled"]:  # low frequencies interpolated 32-fold, high ones kept, a ramp between
        d, f = case["rot"], 32.0
        lo, hi = (d * math.log(4096 / (beta * 2 * math.pi)) / (2 * math.log(10000.0)) for beta in (32, 1))
        ramp = ((torch.arange(n, dtype=torch.float64) - math.floor(lo)) / max(math.ceil(hi) - math.floor(lo), 0.001)).clamp(0, 1)
        inv = inv / f * ramp + inv * (1 - ramp)
        scale = 0.1 * math.log(f) + 1.0
    pos = torch.arange(case["rows"], device="cuda")
    if axes > 1:  # a token's frame, row and column
        pos = torch.stack([pos // 1560, pos // 52 % 30, pos % 52][:axes], 1)
    pos = pos + torch.randint(0, 1 + case["far"], (1,), generator=g, device="cuda")
    return {"qkv": randn(g, case["rows"], (case["heads"] + case["spare"]) * case["D"], by=2.0, dtype=DT[case["dtype"]]),
            "positions": pos.contiguous(), "inv_freq": inv.cuda(), "scale": scale,
            "pair_axis": torch.cat([torch.full((s,), a, dtype=torch.int32) for a, s in enumerate(sizes)]).cuda()}


def inputs_lora(case, seed, g):
    M, K, N, R, n = (case[k] for k in ("M", "K", "N", "R", "adapters"))
    starts, ids = requests(case)
    return {"x": randn(g, M, K), "y": randn(g, M, N, by=1.5), "out": torch.zeros((M, N), dtype=torch.bfloat16, device="cuda"),
            "a": randn(g, n, R, K, by=1 / math.sqrt(K)), "b": randn(g, n, N, R, by=0.5 / math.sqrt(R)),
            "scale": torch.rand(n, generator=g, device="cuda") + 0.5,
            "starts": torch.tensor(starts, dtype=torch.int32, device="cuda"),
            "ids": torch.tensor(ids, dtype=torch.int32, device="cuda")}


def inputs_qk(case, g):
    dtype, D = DT[case["dtype"]], case["D"]
    ql, kl = lengths(case)
    return {"q": randn(g, case["B"], case["Lq"], case["Hq"], D, by=1.5, dtype=dtype),
            "k": randn(g, case["B"], case["Lk"], case["Hkv"], D, dtype=dtype),
            "q_len": torch.tensor(ql, dtype=torch.int32, device="cuda") if case["ragged"] else None,
            "k_len": torch.tensor(kl, dtype=torch.int32, device="cuda") if case["ragged"] else None}


def inputs_select(case, seed, g):
    s = inputs_qk(case, g)
    if case["Lq"] == 1:  # a program that adds tokens keeps the means of the blocks before them
        s["means"] = randn(g, case["B"], case["Hkv"], -(-case["Lk"] // BLOCK_K), case["D"], by=0.125, dtype=torch.float32)
    return s


def inputs_attend(case, seed, g):
    s = inputs_qk(case, g)
    B, Hq, nk = case["B"], case["Hq"], -(-case["Lk"] // BLOCK_K)
    s["v"] = randn(g, *s["k"].shape, dtype=s["k"].dtype)
    s["out"] = torch.zeros_like(s["q"])
    s["lse"] = torch.zeros((B, Hq, case["Lq"]), dtype=torch.float32, device="cuda")
    seen = torch.tensor([-(-n // BLOCK_K) for _, n in visible(case)], device="cuda").view(B, 1, -1, 1)
    j = torch.arange(nk, device="cuda")
    score = torch.rand(B, Hq, seen.shape[2], nk, generator=g, device="cuda")
    score = torch.where(j == seen - 1, 2.0, torch.where(j < seen, score, -1.0))  # the newest block always
    top = score.topk(case["T"], dim=-1)
    chosen = torch.where(top.values >= 0, top.indices, nk).sort(-1).values
    s["blocks"] = torch.where(chosen < nk, chosen, -1).int()
    return s


# ------------------------------------------------------------------------------------ one pass

def run(s):
    kind = s["case"]["kind"]
    if own:
        return run_own(s, kind)
    return {"rope": plain_rope, "lora": plain_lora, "select": plain_select, "attend": plain_attend}[kind](s)


def run_own(s, kind):
    import bit_quantized_linear_hadamard_b200 as qs

    c = s["case"]
    if kind == "rope":
        x = s["qkv"][:, : c["heads"] * c["D"]].view(c["rows"], c["heads"], c["D"])
        return qs.rope(x, s["positions"], s["inv_freq"], pair_axis=s["pair_axis"], interleaved=c["inter"], scale=s["scale"])
    if kind == "lora":
        return qs.lora_add(s["y"], s["x"], s["a"], s["b"], s["starts"], s["ids"], scale=s["scale"], out=s["out"])
    if kind == "select":
        means = s["means"] if "means" in s else qs.block_means(s["k"], lens=s["k_len"])
        blocks = qs.block_select(s["q"], means, c["T"], c["Lk"], first=c["first"], last=c["last"], causal=c["causal"],
                                 q_len=s["q_len"], k_len=s["k_len"])
        return means, blocks
    return qs.block_attention(s["q"], s["k"], s["v"], s["blocks"], causal=c["causal"], q_len=s["q_len"], k_len=s["k_len"],
                              out=s["out"], lse=s["lse"])


def plain_rope(s):
    c = s["case"]
    rows, heads, D, rot = c["rows"], c["heads"], c["D"], c["rot"]
    x = s["qkv"][:, : heads * D].view(rows, heads, D).float()
    angle = s["positions"].view(rows, -1)[:, s["pair_axis"].long()].double() * s["inv_freq"]
    cos = (angle.cos() * s["scale"]).float()[:, None, :]
    sin = (angle.sin() * s["scale"]).float()[:, None, :]
    if c["inter"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = x[..., : rot // 2], x[..., rot // 2 : rot]
        turned = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((turned, x[..., rot:]), -1).to(s["qkv"].dtype)


def plain_lora(s):
    M, (n, R, K) = s["x"].shape[0], s["a"].shape
    row = torch.arange(M, device="cuda")
    request = torch.searchsorted(s["starts"], row, right=True) - 1
    inside = (request >= 0) & (request < len(s["ids"]))
    adapter = torch.where(inside, s["ids"][request.clamp(0, len(s["ids"]) - 1)], -1)
    t = (s["x"].float() @ s["a"].float().view(n * R, K).T).view(M, n, R)
    t = t * (adapter[:, None] == torch.arange(n, device="cuda"))[:, :, None] * s["scale"][None, :, None]
    y = s["y"].float() + t.view(M, n * R) @ s["b"].float().transpose(1, 2).reshape(n * R, -1)
    return torch.where(inside[:, None], y.to(s["y"].dtype), s["out"])


def block_mean(x, length, size):
    """Means of the valid rows of each block of x [B, L, H, D]: [B, H, blocks, D] in 32 bits, from 64-bit sums."""
    B, L, H, D = x.shape
    n = -(-L // size)
    row = torch.arange(n * size, device="cuda")
    valid = row < (length.view(B, 1) if length is not None else torch.full((B, 1), L, device="cuda"))
    full = torch.nn.functional.pad(x, (0, 0, 0, 0, 0, n * size - L)).double()
    total = torch.where(valid[:, :, None, None], full, 0.0).view(B, n, size, H, D).sum(2)
    count = valid.view(B, n, size).sum(2).clamp(min=1)
    return (total / count[:, :, None, None]).float().transpose(1, 2).contiguous()


def lens(s):
    c = s["case"]
    full = torch.ones(c["B"], dtype=torch.int32, device="cuda")
    return (s["q_len"], s["k_len"]) if s["q_len"] is not None else (full * c["Lq"], full * c["Lk"])


def plain_select(s):
    c = s["case"]
    means = s["means"] if "means" in s else block_mean(s["k"], s["k_len"], BLOCK_K)
    qm = block_mean(s["q"], s["q_len"], BLOCK_Q)
    group, nk = c["Hq"] // c["Hkv"], means.shape[2]
    score = torch.matmul(qm.double(), means.double().repeat_interleave(group, 1).transpose(2, 3))
    ql, kl = (t.view(-1, 1) for t in lens(s))
    start = torch.arange(qm.shape[2], device="cuda") * BLOCK_Q
    end = torch.minimum(start + BLOCK_Q, ql)
    keys = (end + kl - ql if c["causal"] else kl + 0 * end).clamp(min=0).minimum(kl)
    n = torch.where(start < ql, (keys + BLOCK_K - 1) // BLOCK_K, 0)[:, None, :, None]
    j = torch.arange(nk, device="cuda")
    always = (j < c["first"]) | (j >= n - c["last"])
    score = torch.where(always, math.inf, score)
    rank = torch.where(j < n, score, -math.inf).sort(dim=-1, descending=True, stable=True).indices[..., : c["T"]]
    chosen = torch.where(rank < n, rank, nk).sort(-1).values
    return means, torch.where(chosen < nk, chosen, -1).int()


def plain_attend(s):
    c = s["case"]
    B, Lq, Hq, D = s["q"].shape
    Lk, group = c["Lk"], c["Hq"] // c["Hkv"]
    nq, nk, T = -(-Lq // BLOCK_Q), -(-Lk // BLOCK_K), c["T"]
    ql, kl = (t.view(B, 1, 1, 1, 1) for t in lens(s))
    q = torch.nn.functional.pad(s["q"], (0, 0, 0, 0, 0, nq * BLOCK_Q - Lq)).float().view(B, nq, BLOCK_Q, Hq, D).permute(0, 3, 1, 2, 4)
    key = (s["blocks"].long()[..., None] * BLOCK_K + torch.arange(BLOCK_K, device="cuda")).view(B, Hq, nq, 1, T * BLOCK_K)
    row = torch.arange(nq * BLOCK_Q, device="cuda").view(1, 1, nq, BLOCK_Q, 1)
    seen = (key >= 0) & (key < kl) & (row < ql)
    if c["causal"]:
        seen = seen & (key <= row + kl - ql)
    b = torch.arange(B, device="cuda").view(B, 1, 1, 1)
    h = torch.arange(Hq, device="cuda").view(1, Hq, 1, 1) // group
    at = key.clamp(0, Lk - 1)[:, :, :, 0]
    score = torch.matmul(q, s["k"][b, at, h].float().transpose(-1, -2)) * (1 / math.sqrt(D))
    score.masked_fill_(~seen, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = score.sub_(torch.where(top > -math.inf, top, 0.0)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, s["v"][b, at, h].float()) / torch.where(total > 0, total, 1.0)
    lse = (total.log() + top).reshape(B, Hq, nq * BLOCK_Q)[:, :, :Lq]
    o = o.permute(0, 2, 3, 1, 4).reshape(B, nq * BLOCK_Q, Hq, D)[:, :Lq]
    valid = torch.arange(Lq, device="cuda") < ql.view(B, 1)
    return torch.where(valid[:, :, None, None], o.to(s["q"].dtype), s["out"]), torch.where(valid[:, None], lse, s["lse"])


# --------------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": exact_rope, "lora": exact_lora, "select": exact_select, "attend": exact_attend}[case["kind"]](case, s)


def exact_rope(case, s):
    """Each pair as a complex number times scale * exp(i angle)."""
    rows, heads, D, n = case["rows"], case["heads"], case["D"], case["rot"] // 2
    out = s["qkv"][:, : heads * D].double().reshape(rows, heads, D)
    for i in range(n):
        lo, hi = (2 * i, 2 * i + 1) if case["inter"] else (i, i + n)
        p = s["positions"] if s["positions"].dim() == 1 else s["positions"][:, int(s["pair_axis"][i])]
        turn = torch.polar(torch.full((rows, 1), float(s["scale"]), dtype=torch.float64, device="cuda"),
                           (p.double() * s["inv_freq"][i])[:, None])
        z = torch.complex(out[:, :, lo].clone(), out[:, :, hi].clone()) * turn
        out[:, :, lo], out[:, :, hi] = z.real, z.imag
    return out


def exact_lora(case, s):
    starts, ids = requests(case)
    out = s["out"].double()
    for lo, hi, i in zip(starts, starts[1:], ids):
        out[lo:hi] = s["y"][lo:hi].double()
        if i >= 0:
            delta = (s["x"][lo:hi].double() @ s["a"][i].double().T) @ s["b"][i].double().T
            out[lo:hi] += delta * s["scale"][i].double()
    return out


def exact_select(case, s):
    if "means" in s:
        return s["means"].double(), None
    _, kl = lengths(case)
    B, L, H, D = s["k"].shape
    out = torch.zeros(B, H, -(-L // BLOCK_K), D, dtype=torch.float64, device="cuda")
    for b, n in enumerate(kl):
        for j in range(-(-n // BLOCK_K)):
            out[b, :, j] = s["k"][b, j * BLOCK_K : min(n, (j + 1) * BLOCK_K)].double().mean(0)
    return out, None


def exact_attend(case, s):
    B, Lq, Hq, D = s["q"].shape
    Lk, nk = case["Lk"], -(-case["Lk"] // BLOCK_K)
    out, lse = s["out"].double(), s["lse"].double()
    step = max(1, min(64, (1 << 28) // (case["T"] * BLOCK_K * BLOCK_Q)))  # query blocks at a time
    for b, (ql, kl) in enumerate(zip(*lengths(case))):
        for h in range(Hq):
            g = h // (Hq // case["Hkv"])
            fill = (0, 0, 0, nk * BLOCK_K - Lk)
            k = torch.nn.functional.pad(s["k"][b, :, g].double(), fill).view(nk, BLOCK_K, D)
            v = torch.nn.functional.pad(s["v"][b, :, g].double(), fill).view(nk, BLOCK_K, D)
            for i0 in range(0, -(-ql // BLOCK_Q), step):
                lists = s["blocks"][b, h, i0 : min(i0 + step, -(-ql // BLOCK_Q))].long()
                n = lists.shape[0]
                lo, hi = i0 * BLOCK_Q, min((i0 + n) * BLOCK_Q, ql)
                q = torch.zeros(n * BLOCK_Q, D, dtype=torch.float64, device="cuda")
                q[: hi - lo] = s["q"][b, lo:hi, h].double()
                w = torch.einsum("nrd,ntkd->nrtk", q.view(n, BLOCK_Q, D), k[lists.clamp(min=0)]) / math.sqrt(D)
                key = lists[:, :, None] * BLOCK_K + torch.arange(BLOCK_K, device="cuda")
                off = (lists < 0)[:, None, :, None] | (key >= kl)[:, None]
                if case["causal"]:
                    row = torch.arange(lo, lo + n * BLOCK_Q, device="cuda").view(n, BLOCK_Q, 1, 1)
                    off = off | (key[:, None] > row + (kl - ql))
                w = w.masked_fill(off, -math.inf).flatten(2)
                z = torch.logsumexp(w, -1, keepdim=True)
                p = torch.where(z > -math.inf, (w - z).exp(), 0.0)
                o = torch.matmul(p, v[lists.clamp(min=0)].flatten(1, 2))
                out[b, lo:hi, h] = o.reshape(-1, D)[: hi - lo]
                lse[b, h, lo:hi] = z.reshape(-1)[: hi - lo]
    return out, lse


# --------------------------------------------------------------------------------- the floor

def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    if case["kind"] == "rope":
        n = case["rows"] * case["heads"] * case["D"]
        return {"bytes": 2 * n * size + 8 * case["rows"] * case["axes"],
                "flops": 3 * case["rows"] * case["heads"] * case["rot"]}
    if case["kind"] == "lora":
        starts, ids = requests(case)
        inside, turned = starts[-1], sum(hi - lo for lo, hi, i in zip(starts, starts[1:], ids) if i >= 0)
        weights = len({i for i in ids if i >= 0}) * case["R"] * (case["K"] + case["N"])
        return {"bytes": 2 * (turned * case["K"] + 2 * inside * case["N"] + weights),
                "flops": 2 * turned * case["R"] * (case["K"] + case["N"])}
    B, Hq, Hkv, D, T = (case[k] for k in ("B", "Hq", "Hkv", "D", "T"))
    ql, kl = lengths(case)
    blocks = [(rows, min(T, -(-n // BLOCK_K)), n) for rows, n in visible(case)]
    lists = 4 * Hq * T * len(blocks)
    if case["kind"] == "select":
        nk = -(-case["Lk"] // BLOCK_K)
        keys = 0 if case["Lq"] == 1 else sum(kl) * Hkv * D
        return {"bytes": size * (sum(ql) * Hq * D + keys) + 4 * B * Hkv * nk * D + lists,
                "flops": sum(ql) * Hq * D + keys + 2 * D * Hq * sum(-(-n // BLOCK_K) for _, _, n in blocks)}
    keys = min(sum(kl) * Hkv, Hq * sum(min(n * BLOCK_K, most) for _, n, most in blocks))
    pairs = Hq * sum(rows * min(n * BLOCK_K, most) for rows, n, most in blocks)
    return {"bytes": size * D * (2 * sum(ql) * Hq + 2 * keys) + 4 * sum(ql) * Hq + lists, "flops": 4 * D * pairs}
