"""Cases of the serving operators that stand around the adapter delta: the 4-bit base projection, the paged KV cache
(append, attention of new tokens over it, page moves).  With ``own`` false every operator runs in its plain form,
elementary torch operations in fp32; with ``own`` true through this package's kernels."""
import math

import torch

own = False

# Element e (0..7) of a 32-bit word of packed 4-bit codes sits in nibble NIBBLE[e].
NIBBLE = (0, 4, 1, 5, 2, 6, 3, 7)


def listed():
    return [
        # one token through a square 4-bit projection: a single user's decode step, where the call's latency counts
        w4("w4 one token", m=1, n=4096, k=4096, group=128, zeros=False, scales="bf16"),
        # one decode step of a 16-request batch through the widest projection of the 70B-shape layer
        w4("w4 batch wide", m=16, n=28672, k=8192, group=128, zeros=False, scales="bf16"),
        # small groups with zero points and fp32 scales, odd token count, ragged output and input widths
        w4("w4 ragged zeros", m=5, n=1288, k=4128, group=32, zeros=True, scales="f32"),
        # the decode tokens of a full batch through a square projection of the 70B-shape layer
        w4("w4 batch 64", m=64, n=8192, k=8192, group=64, zeros=True, scales="bf16"),
        # one request's decode token over a short context: latency
        attn("attn one token", seqs=1, q=1, kv=200, heads=32, kv_heads=8, dim=128, page=16),
        # a ragged decode batch at the 70B layer's heads over contexts of up to 8192 tokens
        attn("attn decode batch", seqs=64, q=1, kv=8192, heads=64, kv_heads=8, dim=128, page=64),
        # a ragged batch of short chunks, one kv head per query head, a sliding window, pages that end inside tiles
        attn("attn windowed chunks", seqs=7, q=333, kv=1500, heads=12, kv_heads=12, dim=64, page=24, window=257),
        # a long prompt's chunk of 4096 tokens over the 12288 that are cached already
        attn("attn long chunk", seqs=1, q=4096, kv=16384, heads=64, kv_heads=8, dim=128, page=64),
        # one decode step of a full batch written into the cache
        append("append decode", seqs=256, q=1, kv=2000, kv_heads=8, dim=128, page=64),
        # a prefill batch written into the cache, odd pages
        append("append chunks", seqs=9, q=2048, kv=5000, kv_heads=8, dim=128, page=24),
        # sequences forked: each one's last, partly filled page copied
        pages("pages fork", pages=12, move=5, page_kib=32, table=40),
        # a fragmented pool compacted: a quarter of its 256 KiB pages moved, every page table rewritten
        pages("pages compact", pages=8192, move=2048, page_kib=256, table=300000),
    ]


def w4(name, **kw):
    return {"name": name, "op": "w4", **kw}


def attn(name, window=0, causal=True, **kw):
    return {"name": name, "op": "attn", "window": window, "causal": causal, **kw}


def append(name, **kw):
    return {"name": name, "op": "append", **kw}


def pages(name, **kw):
    return {"name": name, "op": "pages", **kw}


def draw(rng):
    """One more case of the listed ranges."""
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    largest = {}
    for c in listed():
        w = work(c)
        largest[c["op"]] = max(largest.get(c["op"], 0.0), cost(w))
    op = rng.choice(("w4", "w4", "attn", "attn", "attn", "append", "pages"))
    while True:
        if op == "w4":
            group = rng.choice((32, 64, 128))
            c = {"op": op, "m": log(1, 64), "n": 8 * log(64, 3584), "k": group * max(1, log(512, 14336) // group), "group": group,
                 "zeros": rng.random() < 0.5, "scales": rng.choice(("bf16", "f32"))}
        elif op == "attn":
            kv_heads, group = rng.choice((1, 2, 4, 8)), rng.choice((1, 3, 4, 8, 16))
            kv = log(32, 16384)
            q = 1 if rng.random() < 0.4 else min(kv, log(2, 4096))
            c = {"op": op, "seqs": log(1, 64), "q": q, "kv": kv, "heads": kv_heads * group, "kv_heads": kv_heads, "dim": rng.choice((64, 80, 128, 128, 256)),
                 "page": rng.choice((8, 16, 24, 64, 128)), "window": rng.choice((0, 0, 0, log(16, 4096))), "causal": rng.random() < 0.85}
            # the plain form holds every score at once
            if c["seqs"] * c["heads"] * q * kv > 64 * 4096 * 16384 or c["seqs"] * kv_heads * kv * c["dim"] > 64 * 8 * 8192 * 128:
                continue
        elif op == "append":
            kv = log(32, 16384)
            c = {"op": op, "seqs": log(1, 256), "q": 1 if rng.random() < 0.4 else min(kv, log(2, 2048)), "kv": kv, "kv_heads": rng.choice((1, 2, 4, 8)),
                 "dim": rng.choice((64, 80, 128, 256)), "page": rng.choice((8, 16, 24, 64, 128))}
            if c["seqs"] * kv * c["kv_heads"] * c["dim"] > 64 * 8 * 8192 * 128:
                continue
        else:
            n = log(8, 8192)
            c = {"op": op, "pages": n, "move": max(1, int(n * rng.uniform(0.02, 0.45))), "page_kib": rng.choice((16, 32, 48, 64, 256)), "table": log(32, 300000)}
        if cost(work(c)) <= largest[op]:
            return c


def cost(w):
    return max(w["bytes"] / 5e12, w["flops"] / 1e15)


# ---------------------------------------------------------------- lengths and layouts
def lengths(case):
    """(new tokens, cached plus new tokens) of each sequence: the case's own for one sequence, ragged for more, the first ones full."""
    got = []
    for i in range(case["seqs"]):
        part = 1.0 - 0.75 * ((i * 0.6180339887498949) % 1.0)
        kv = max(1, int(case["kv"] * part))
        got.append((min(kv, max(1, int(case["q"] * part))) if case["q"] > 1 else 1, kv))
    return got


def paged(case, gen, slack=1.25):
    """A page table over a shuffled pool and its page count; entries behind a sequence's last page are -1."""
    lens = lengths(case)
    need = [-(-kv // case["page"]) for _, kv in lens]
    total = max(sum(need) + 1, int(sum(need) * slack))
    ids = torch.randperm(total, generator=gen, device="cuda").int()
    table = torch.full((len(need), max(need)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, c in enumerate(need):
        table[i, :c] = ids[at: at + c]
        at += c
    return table, total


def tokens_of(case):
    """(sequence, position) of each new token, in the batch's packed order."""
    seq, pos = [], []
    for i, (q, kv) in enumerate(lengths(case)):
        seq.append(torch.full((q,), i, dtype=torch.int32))
        pos.append(torch.arange(kv - q, kv, dtype=torch.int32))
    return torch.cat(seq), torch.cat(pos)


def pairs_of(case):
    """Attended (query, key) pairs of one query head."""
    n, w = 0, case["window"]
    for q, kv in lengths(case):
        if not case["causal"]:
            if not w:
                n += q * kv
            else:
                n += sum(kv - max(0, p - w + 1) for p in range(kv - q, kv))
        elif not w:
            n += q * (kv - q) + q * (q + 1) // 2
        else:
            n += sum(min(p + 1, w) for p in range(kv - q, kv))
    return n


def keys_read(case):
    """Cached tokens that some new token of their sequence attends to."""
    w = case["window"]
    return sum(min(kv, q + w - 1) if w else kv for q, kv in lengths(case))


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=gen, device="cuda") * std).bfloat16()

    op = case["op"]
    s = {"case": case}
    if op == "w4":
        m, n, k, group = case["m"], case["n"], case["k"], case["group"]
        dtype = torch.bfloat16 if case["scales"] == "bf16" else torch.float32
        s["x"] = normal(m, k)
        s["codes"] = torch.randint(0, 256, (-(-n // 16), -(-k // 128), 64, 16), generator=gen, device="cuda", dtype=torch.uint8)
        s["scales"] = ((0.5 + torch.rand((k // group, n), generator=gen, device="cuda")) / (4.6 * math.sqrt(k))).to(dtype)
        s["zeros"] = (8 + 2 * torch.randn((k // group, n), generator=gen, device="cuda")).round().clamp(0, 15).to(dtype) if case["zeros"] else None
        s["y"] = torch.empty((m, n), dtype=torch.bfloat16, device="cuda")
    elif op in ("attn", "append"):
        h, d, p = case["kv_heads"], case["dim"], case["page"]
        s["table"], total = paged(case, gen)
        s["cache"] = normal(total, 2, h, p, d)
        seq, pos = tokens_of(case)
        s["seq"], s["pos"] = seq.cuda(), pos.cuda()
        t = seq.numel()
        if op == "append":
            s["k"], s["v"] = normal(t, h, d), normal(t, h, d)
        else:
            s["q"] = normal(t, case["heads"], d, std=1.5)
            s["kv_len"] = torch.tensor([kv for _, kv in lengths(case)], dtype=torch.int32, device="cuda")
            s["out"] = torch.empty((t, case["heads"], d), dtype=torch.bfloat16, device="cuda")
            s["lse"] = torch.empty((t, case["heads"]), dtype=torch.float32, device="cuda")
    else:
        n, mv = case["pages"], case["move"]
        s["store"] = normal(n, case["page_kib"] * 512)
        order = torch.randperm(n, generator=gen, device="cuda").int()
        s["src"], s["dst"] = order[:mv].contiguous(), order[mv: 2 * mv].contiguous()
        remap = torch.arange(n, dtype=torch.int32, device="cuda")
        remap[s["src"].long()] = s["dst"]
        s["remap"] = remap
        s["table"] = torch.randint(-1, n, (case["table"],), generator=gen, device="cuda", dtype=torch.int32)
        s["new_table"] = torch.empty_like(s["table"])
    if own:
        handles(case, s)
    return s


def handles(case, s):
    """What a serving program keeps between calls: descriptors, and the attention's plan of the batch with its workspace."""
    from segmented_gather_gemm_segments_amd import binding as B
    if case["op"] == "w4":
        s["w"] = B.W4Weights(case["n"], case["k"], case["group"], s["codes"], s["scales"], s["zeros"])
    elif case["op"] in ("attn", "append"):
        s["view"] = B.KvView(s["cache"][:, 0], s["cache"][:, 1], s["table"])
        if case["op"] == "attn":
            lens = lengths(case)
            starts = [0]
            for q, _ in lens:
                starts.append(starts[-1] + q)
            s["plan"] = B.lora_kv_attn_plan(starts, list(range(len(lens))), [kv for _, kv in lens], case["heads"], case["kv_heads"], case["dim"],
                                            causal=case["causal"], window=case["window"]).to("cuda")


# ---------------------------------------------------------------- one pass
def run(s):
    case = s["case"]
    if own:
        from segmented_gather_gemm_segments_amd import binding as B
        if case["op"] == "w4":
            B.lora_base_w4(s["x"], s["w"], s["y"])
            return s["y"]
        if case["op"] == "attn":
            B.lora_kv_attn(s["view"], s["plan"], s["q"], s["out"], lse=s["lse"])
            return {"out": s["out"], "lse": s["lse"]}
        if case["op"] == "append":
            B.lora_kv_append(s["view"], s["k"], s["v"], s["seq"], s["pos"])
            return s["cache"]
        B.lora_pages_copy(s["store"], s["src"], s["dst"])
        B.lora_page_table_remap(s["remap"], s["table"], s["new_table"])
        return {"store": s["store"], "table": s["new_table"]}
    return {"w4": plain_w4, "attn": plain_attn, "append": plain_append, "pages": plain_pages}[case["op"]](s)


def plain_w4(s):
    """y = x W^T with W = (code - zero) * scale, one scale (and zero point, else 8) per row and group."""
    case = s["case"]
    n, k = case["n"], case["k"]
    c = s["codes"]
    rows, cols = c.shape[:2]
    c = c.view(rows, cols, 4, 16, 4, 4, 1)  # row tile, column tile, 8-run, row, 32-run, byte
    c = torch.cat((c & 15, c >> 4), dim=-1).view(rows, cols, 4, 16, 4, 8)[..., list(NIBBLE)]
    c = c.permute(0, 3, 1, 4, 2, 5).reshape(rows * 16, cols * 128)[:n, :k].float()
    w = c.view(n, k // case["group"], case["group"])
    w = w - (8.0 if s["zeros"] is None else s["zeros"].float().t().unsqueeze(-1))
    w = (w * s["scales"].float().t().unsqueeze(-1)).view(n, k)
    return (s["x"].float() @ w.t()).bfloat16()


def plain_attn(s):
    case, q = s["case"], s["q"]
    n, h, d = case["seqs"], case["kv_heads"], case["dim"]
    g = case["heads"] // h
    got = s["cache"][s["table"].clamp(min=0).long()]  # [n, pages, 2, h, page, d]
    got = got.permute(2, 0, 3, 1, 4, 5).reshape(2, n, h, -1, d).float()
    k, v = got[0], got[1]
    width = k.shape[2]
    first = (s["kv_len"] - torch.bincount(s["seq"], minlength=n)).long()  # position of each sequence's first new token
    off = s["pos"].long() - first[s["seq"].long()]
    most = case["q"]
    at = (s["seq"].long(), off)
    padded = torch.zeros((n, most, h, g, d), device=q.device)
    padded[at] = q.view(-1, h, g, d).float()
    padded = padded.permute(0, 2, 1, 3, 4).reshape(n, h, most * g, d)
    score = torch.matmul(padded, k.transpose(2, 3).contiguous()) / math.sqrt(d)
    where = torch.arange(width, device=q.device)
    pos = first[:, None] + torch.arange(most, device=q.device)
    keep = (where < s["kv_len"][:, None, None]).expand(n, most, width)
    if case["causal"]:
        keep = keep & (where <= pos[..., None])
    if case["window"]:
        keep = keep & (where > pos[..., None] - case["window"])
    score = score.view(n, h, most, g, width).masked_fill_(~keep[:, None, :, None, :], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    score = score.sub_(top).exp_()
    total = score.sum(-1, keepdim=True)
    out = torch.matmul(score.view(n, h, most * g, width), v).view(n, h, most, g, d) / total.clamp(min=1e-30)
    lse = (top + total.log()).squeeze(-1)
    out = out.permute(0, 2, 1, 3, 4)[at].reshape(-1, case["heads"], d)
    return {"out": out.bfloat16(), "lse": lse.permute(0, 2, 1, 3)[at].reshape(-1, case["heads"])}


def plain_append(s):
    page, slot = (s["pos"] // s["case"]["page"]).long(), (s["pos"] % s["case"]["page"]).long()
    at = s["table"][s["seq"].long(), page].long()
    s["cache"][at, 0, :, slot] = s["k"]
    s["cache"][at, 1, :, slot] = s["v"]
    return s["cache"]


def plain_pages(s):
    s["store"][s["dst"].long()] = s["store"][s["src"].long()]
    table = torch.where(s["table"] < 0, s["table"], s["remap"][s["table"].clamp(min=0).long()])
    return {"store": s["store"], "table": table}


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    op = case["op"]
    if op == "w4":
        m, n, k = case["m"], case["n"], case["k"]
        per = (2 if case["scales"] == "bf16" else 4) * (2 if case["zeros"] else 1)
        return {"bytes": n * k / 2 + n * (k // case["group"]) * per + 2 * m * k + 2 * m * n, "flops": 2.0 * m * n * k}
    if op == "attn":
        t = sum(q for q, _ in lengths(case))
        cached = 2 * keys_read(case) * case["kv_heads"] * case["dim"] * 2
        return {"bytes": cached + t * case["heads"] * (4 * case["dim"] + 4), "flops": 4.0 * pairs_of(case) * case["heads"] * case["dim"]}
    if op == "append":
        t = sum(q for q, _ in lengths(case))
        return {"bytes": t * (8 * case["kv_heads"] * case["dim"] + 8), "flops": 0}
    return {"bytes": 2 * case["move"] * (case["page_kib"] * 1024 + 4) + 8 * case["table"], "flops": 0}


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "w4":
        n, k = case["n"], case["k"]
        word = s["codes"].view(torch.int32).view(*s["codes"].shape[:2], 4, 16, 4)  # a lane's four words: row lane % 16, k 8 (lane / 16) + 32 word
        w = torch.empty((word.shape[0] * 16, word.shape[1] * 128), dtype=torch.float64, device="cuda")
        for e in range(8):
            code = ((word >> (4 * NIBBLE[e])) & 15).double()
            for run8 in range(4):
                for step in range(4):
                    w[:, 32 * step + 8 * run8 + e:: 128] = code[:, :, run8, :, step].permute(0, 2, 1).reshape(w.shape[0], -1)
        w = w[:n, :k]
        z = torch.full((k // case["group"], n), 8.0, dtype=torch.float64, device="cuda") if s["zeros"] is None else s["zeros"].double()
        for i in range(k // case["group"]):
            part = w[:, i * case["group"]: (i + 1) * case["group"]]
            part.sub_(z[i][:, None]).mul_(s["scales"][i].double()[:, None])
        return s["x"].double() @ w.t()
    if case["op"] == "attn":
        group = case["heads"] // case["kv_heads"]
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
        lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
        at = 0
        for i, (q, kv) in enumerate(lengths(case)):
            ids = s["table"][i, : -(-kv // case["page"])].long()
            pos = torch.arange(kv - q, kv, device="cuda")
            j = torch.arange(kv, device="cuda")
            bad = torch.zeros((q, kv), dtype=torch.bool, device="cuda")
            if case["causal"]:
                bad |= j[None, :] > pos[:, None]
            if case["window"]:
                bad |= j[None, :] <= pos[:, None] - case["window"]
            for h in range(case["kv_heads"]):
                k = s["cache"][ids, 0, h].reshape(-1, case["dim"])[:kv].double()
                v = s["cache"][ids, 1, h].reshape(-1, case["dim"])[:kv].double()
                for head in range(h * group, (h + 1) * group):
                    z = s["q"][at: at + q, head].double() @ k.t() * case["dim"] ** -0.5
                    z.masked_fill_(bad, -math.inf)
                    lse[at: at + q, head] = torch.logsumexp(z, 1)
                    out[at: at + q, head] = torch.softmax(z, 1) @ v
            at += q
        return {"out": out, "lse": lse}
    return None
