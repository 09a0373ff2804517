"""Cases of what a decoder does with its paged KV cache beyond bf16 rows and causal masks: a cache quantised to FP8 E4M3 as
it is written (append, rows read back, attention over it), a tree of drafted tokens (its mask, attention, the accepted path
moved into place), and attention over the pages that bounds of their keys select for each token.  With ``own`` false every
operator runs in its plain form, elementary torch operations in fp32; with ``own`` true through this package's kernels.

The 8-bit cache: a row of K or V of one position and head is x ~ 2^e c with c in E4M3 and one exponent e for the row, the
least for which its largest finite magnitude is at most 448, and -117 at least; e + 127 is stored in a byte.

The bounds of a page and head: for each of D dimensions the largest and the least of its keys, in integers of
steps 2^f, the largest rounded up and the least down; a query row in steps of its own, 2^g, rounded to nearest.  A page's score is the
largest over the query heads that share the KV head of sum_d max(q_d hi_d, q_d lo_d), whole numbers
times 2^(f + g): exact in fp32."""
import math
import random

import torch

own = False

LEAST_EXP = -117  # of an 8-bit row: its smallest code then stands for a normal bf16 number


def listed():
    return [
        # one decode step of a full batch written into an 8-bit cache
        make("append8 decode", "append8", seqs=256, q=1, kv=2000, kv_heads=8, dim=128, page=64),
        # a prefill batch written into it, odd pages
        make("append8 chunks", "append8", seqs=9, q=2048, kv=5000, kv_heads=8, dim=128, page=24),
        # a short sequence's rows handed over in bf16: latency
        make("read8 short", "read8", seqs=1, q=200, kv=200, kv_heads=8, dim=128, page=16),
        # the rows of a few long sequences handed over in bf16
        make("read8 long", "read8", seqs=5, q=16384, kv=16384, kv_heads=8, dim=128, page=64),
        # a ragged decode batch at the 70B-shape layer's heads over 8-bit contexts of up to 8192 tokens
        make("attn8 decode batch", "attn", fp8=True, seqs=64, q=1, kv=8192, heads=64, kv_heads=8, dim=128, page=64),
        # a long prompt's chunk of 2048 tokens over the 14336 that are cached already, in 8 bits
        make("attn8 long chunk", "attn", fp8=True, seqs=1, q=2048, kv=16384, heads=64, kv_heads=8, dim=128, page=64),
        # one user's drafted tree verified over a short context: latency
        make("tree one request", "tree", fp8=False, seqs=1, q=26, kv=700, heads=32, kv_heads=8, dim=128, page=16),
        # the trees of a batch verified over contexts of up to 8192 tokens, bf16 and a window that some models have
        make("tree batch", "tree", fp8=False, seqs=32, q=61, kv=8192, heads=64, kv_heads=8, dim=128, page=64, window=4096),
        # one request's accepted tokens moved to where its sequence goes on
        make("path one request", "path", fp8=False, seqs=1, q=26, kv=700, kv_heads=8, dim=128, page=16, path=5),
        # the same for a batch and every layer's worth of heads side by side
        make("path batch", "path", fp8=True, seqs=128, q=61, kv=3000, kv_heads=64, dim=128, page=24, path=8),
        # a decode step over long contexts that attends to 64 pages of up to 512
        make("blocks decode", "blocks", fp8=False, seqs=32, q=1, kv=32768, heads=64, kv_heads=8, dim=128, page=64, count=64),
        # a ragged batch of short chunks in 8 bits, odd pages, one query head per KV head
        make("blocks chunks", "blocks", fp8=True, seqs=5, q=45, kv=5000, heads=12, kv_heads=12, dim=64, page=24, count=20),
    ]


def make(name, op, **kw):
    return {"name": name, "op": op, **kw}


def draw(rng):
    """One more case of the listed ranges."""
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    largest = {}
    for c in listed():
        largest[c["op"]] = max(largest.get(c["op"], 0.0), cost(work(c)))
    op = rng.choice(("append8", "read8", "attn", "attn", "tree", "tree", "path", "blocks", "blocks"))
    while True:
        kv_heads, group = rng.choice((1, 2, 4, 8)), rng.choice((1, 3, 4, 8, 16))
        kv = log(32, 16384)
        c = {"op": op, "seqs": log(1, 64), "kv": kv, "kv_heads": kv_heads, "dim": rng.choice((64, 80, 128, 128, 256)),
             "page": rng.choice((8, 16, 24, 64, 128))}
        if op in ("append8", "read8"):
            c["seqs"] = log(1, 256) if op == "append8" else log(1, 16)
            c["q"] = 1 if op == "append8" and rng.random() < 0.4 else min(kv, log(2, 2048)) if op == "append8" else kv
        elif op == "attn":
            c.update(fp8=True, heads=kv_heads * group, q=1 if rng.random() < 0.5 else min(kv, log(2, 2048)), window=rng.choice((0, 0, log(16, 4096))))
        elif op == "tree":
            c.update(fp8=rng.random() < 0.5, heads=kv_heads * group, q=min(kv, log(2, 200)), window=rng.choice((0, 0, log(16, 4096))))
        elif op == "path":
            c.update(fp8=rng.random() < 0.5, q=min(kv, log(8, 200)), path=1)
            c["path"] = rng.randint(1, max(1, c["q"] // 4))
        else:
            c.update(fp8=rng.random() < 0.5, heads=kv_heads * group, q=1 if rng.random() < 0.5 else min(kv, log(2, 64)), count=log(4, 64))
        # the plain forms hold every row in fp32 and every score at once
        if c["seqs"] * kv_heads * kv * c["dim"] > 64 * 8 * 8192 * 128 or c["seqs"] * c.get("heads", 0) * c["q"] * kv > 64 * 4096 * 8192:
            continue
        if op == "blocks" and c["seqs"] * c["q"] * kv_heads * c["count"] * c["page"] * c["dim"] > 32 * 8 * 64 * 64 * 128:
            continue
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
        q = case["q"] if case["op"] in ("tree", "path") or case["q"] == 1 else max(1, int(case["q"] * part))
        got.append((min(kv, q), kv))
    return got


def paged(case, gen, slack=1.25):
    """A page table over a shuffled pool and its page count; entries behind a sequence's last page are -1."""
    need = [-(-kv // case["page"]) for _, kv in lengths(case)]
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


def starts_of(case):
    starts = [0]
    for q, _ in lengths(case):
        starts.append(starts[-1] + q)
    return starts


def row_bytes(dim):
    """Bytes of a page's bounds for one head: dim largest, dim least, padding to 64, then the exponent in 4 of 16."""
    return -(-2 * dim // 64) * 64 + 16


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=gen, device="cuda") * std).bfloat16()

    op, h, d, p = case["op"], case["kv_heads"], case["dim"], case["page"]
    s = {"case": case}
    s["table"], total = paged(case, gen)
    s["fp8"] = op in ("append8", "read8") or case["fp8"]
    if s["fp8"]:
        # codes as rows of a normal distribution leave them: the largest of a row between 224 and 448
        s["cache"] = torch.empty((total, 2, h, p, d), dtype=torch.float8_e4m3fn, device="cuda")
        for i in range(0, total, 1024):
            part = s["cache"][i: i + 1024]
            part.copy_((torch.randn(part.shape, generator=gen, device="cuda") * 110).clamp_(-448, 448))
        s["scales"] = torch.randint(119, 122, (total, 2, h, p), generator=gen, device="cuda", dtype=torch.uint8)
    else:
        s["cache"] = normal(total, 2, h, p, d)
    seq, pos = tokens_of(case)
    s["seq"], s["pos"] = seq.cuda(), pos.cuda()
    t = seq.numel()
    if op == "append8":
        s["k"], s["v"] = normal(t, h, d), normal(t, h, d)
    elif op == "read8":
        s["k"], s["v"] = (torch.empty((t, h, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    elif op == "path":
        # nodes of an accepted path, ascending; their rows lie behind the places that they move to
        rng = random.Random(seed)
        paths = []
        for q, _ in lengths(case):
            n = min(case["path"], q // 2)
            paths.append(sorted(rng.sample(range(n, q), n)) + [-1] * (case["path"] - n))
        s["path"] = torch.tensor(paths, dtype=torch.int32, device="cuda")
        s["base"] = torch.tensor([kv - q for q, kv in lengths(case)], dtype=torch.int32, device="cuda")
        s["rows"] = torch.arange(case["seqs"], dtype=torch.int32, device="cuda")
    else:
        s["q"] = normal(t, case["heads"], d, std=1.5)
        s["kv_len"] = torch.tensor([kv for _, kv in lengths(case)], dtype=torch.int32, device="cuda")
        s["starts"] = torch.tensor(starts_of(case), dtype=torch.int32, device="cuda")
        s["out"] = torch.empty((t, case["heads"], d), dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty((t, case["heads"]), dtype=torch.float32, device="cuda")
    if op == "tree":
        # node i hangs below one of the eight before it, or below the context
        index = s["pos"] - (s["kv_len"] - (s["starts"][1:] - s["starts"][:-1]))[s["seq"].long()]
        back = (torch.rand(t, generator=gen, device="cuda") * (index + 1).clamp(max=8)).int()
        s["parent"] = (index - 1 - back).clamp(min=-1).int()
    if op == "blocks":
        s["blocks"] = torch.empty((t, h, case["count"]), dtype=torch.int32, device="cuda")
        s["bounds"] = torch.zeros((total, h, row_bytes(d)), dtype=torch.uint8, device="cuda")
        new = torch.tensor([q for q, _ in lengths(case)], dtype=torch.int32, device="cuda")
        s["begin"], s["end"], s["rows"] = s["kv_len"] - new, s["kv_len"], torch.arange(case["seqs"], dtype=torch.int32, device="cuda")
        used = s["table"] >= 0
        ids = s["table"][used].long()
        filled = (s["begin"][:, None] - torch.arange(s["table"].shape[1], device="cuda") * p).clamp(0, p)[used]
        for i in range(0, ids.numel(), 2048):
            s["bounds"][ids[i: i + 2048]] = bounds_rows(dequantised(s, ids[i: i + 2048], 0), filled[i: i + 2048])
    if own:
        handles(case, s)
    return s


def handles(case, s):
    """What a serving program keeps between calls: descriptors, and the attention's plan of the batch with its workspace."""
    from segmented_gather_gemm_segments_amd import binding as B
    if s["fp8"]:
        s["view"] = B.KvView(s["cache"][:, 0], s["cache"][:, 1], s["table"], s["scales"][:, 0], s["scales"][:, 1])
    else:
        s["view"] = B.KvView(s["cache"][:, 0], s["cache"][:, 1], s["table"])
    lens = lengths(case)
    if case["op"] in ("attn", "tree"):
        if case["op"] == "tree":
            s["tree"] = B.Tree(s["seq"].numel(), case["q"], "cuda")
        s["plan"] = B.lora_kv_attn_plan(starts_of(case), list(range(len(lens))), [kv for _, kv in lens], case["heads"], case["kv_heads"],
                                        case["dim"], window=case.get("window", 0), tree=case["op"] == "tree").to("cuda")
    elif case["op"] == "blocks":
        s["bound"] = B.KvBounds(s["view"], s["bounds"])
        n = s["seq"].numel()
        s["plan"] = B.lora_kv_attn_plan(list(range(n + 1)), s["seq"].tolist(), [case["count"] * case["page"]] * n, case["heads"],
                                        case["kv_heads"], case["dim"], blocks=True).to("cuda")


# ---------------------------------------------------------------- one pass
def run(s):
    case = s["case"]
    if not own:
        return {"append8": plain_append8, "read8": plain_read8, "attn": plain_attn, "tree": plain_tree, "path": plain_path, "blocks": plain_blocks}[case["op"]](s)
    from segmented_gather_gemm_segments_amd import binding as B
    if case["op"] == "append8":
        B.lora_kv_append(s["view"], s["k"], s["v"], s["seq"], s["pos"])
        return {"cache": s["cache"], "scales": s["scales"]}
    if case["op"] == "read8":
        B.lora_kv_read(s["view"], s["seq"], s["pos"], s["k"], s["v"])
        return {"k": s["k"], "v": s["v"]}
    if case["op"] == "attn":
        B.lora_kv_attn(s["view"], s["plan"], s["q"], s["out"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    if case["op"] == "tree":
        B.lora_tree_mask(s["starts"], s["parent"], s["tree"], window=case.get("window", 0))
        B.lora_kv_attn_tree(s["view"], s["plan"], s["tree"], s["q"], s["out"], lse=s["lse"])
        return {"mask": s["tree"].mask, "depth": s["tree"].depth, "out": s["out"], "lse": s["lse"]}
    if case["op"] == "path":
        B.lora_kv_keep_path(s["view"], s["rows"], s["base"], s["path"])
        return {"cache": s["cache"], "scales": s["scales"]} if s["fp8"] else s["cache"]
    B.lora_kv_bounds_update(s["view"], s["bound"], s["rows"], s["begin"], s["end"], case["q"])
    B.lora_kv_block_select(s["view"], s["bound"], s["seq"], s["pos"], s["q"], s["blocks"], sink=1, recent=2)
    B.lora_kv_attn_blocks(s["view"], s["plan"], s["blocks"], s["pos"], s["q"], s["out"], lse=s["lse"])
    return {"bounds": s["bounds"], "blocks": s["blocks"], "out": s["out"], "lse": s["lse"]}


def power(e):
    """2^e in fp32, -126 <= e <= 127."""
    return ((e.int() + 127) << 23).view(torch.float32)


def quantised(x):
    """E4M3 codes and biased exponents of rows."""
    x = x.float()
    top = torch.where(x.isfinite(), x.abs(), 0).amax(-1)
    part, e = torch.frexp(top)
    e = torch.where(top > 0, (e - 9 + (part > 0.875)).clamp(min=LEAST_EXP), LEAST_EXP)
    big = 1.875 * 2.0 ** 127
    y = torch.where(x.isfinite(), x.clamp(-big, big) * power(-e)[..., None], math.nan)
    return y.to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def dequantised(s, pages, which, heads=slice(None)):
    """Rows of whole pages in fp32: K (which 0) or V (1)."""
    if not s["fp8"]:
        return s["cache"][pages, which, heads].float()
    codes = s["cache"].view(torch.uint8)[pages, which, heads].view(torch.float8_e4m3fn)
    return codes.float() * power(s["scales"][pages, which, heads].int() - 127)[..., None]


def plain_append8(s):
    page, slot = (s["pos"] // s["case"]["page"]).long(), (s["pos"] % s["case"]["page"]).long()
    at = s["table"][s["seq"].long(), page].long()
    for which, rows in ((0, s["k"]), (1, s["v"])):
        codes, e = quantised(rows)
        s["cache"].view(torch.uint8)[at, which, :, slot] = codes.view(torch.uint8)
        s["scales"][at, which, :, slot] = e
    return {"cache": s["cache"], "scales": s["scales"]}


def plain_read8(s):
    page, slot = (s["pos"] // s["case"]["page"]).long(), (s["pos"] % s["case"]["page"]).long()
    at = s["table"][s["seq"].long(), page].long()
    got = []
    for which in (0, 1):
        codes = s["cache"].view(torch.uint8)[at, which, :, slot].view(torch.float8_e4m3fn)
        got.append((codes.float() * power(s["scales"][at, which, :, slot].int() - 127)[..., None]).bfloat16())
    return {"k": got[0], "v": got[1]}


def gathered(s):
    """K and V of each sequence's pages in fp32, [n, kv_heads, positions, dim]."""
    case, ids = s["case"], s["table"].clamp(min=0).long()
    n, h, d = case["seqs"], case["kv_heads"], case["dim"]
    return [dequantised(s, ids.flatten(), w).view(n, -1, h, case["page"], d).permute(0, 2, 1, 3, 4).reshape(n, h, -1, d) for w in (0, 1)]


def plain_attn(s, keep_of=None):
    case, q = s["case"], s["q"]
    n, h, d = case["seqs"], case["kv_heads"], case["dim"]
    g = case["heads"] // h
    k, v = gathered(s)
    width = k.shape[2]
    first = (s["kv_len"] - (s["starts"][1:] - s["starts"][:-1])).long()  # position of each sequence's first new token
    at = (s["seq"].long(), s["pos"].long() - first[s["seq"].long()])
    most = case["q"]
    padded = torch.zeros((n, most, h, g, d), device=q.device)
    padded[at] = q.view(-1, h, g, d).float()
    padded = padded.permute(0, 2, 1, 3, 4).reshape(n, h, most * g, d)
    score = torch.matmul(padded, k.transpose(2, 3).contiguous()) / math.sqrt(d)
    where = torch.arange(width, device=q.device)
    if keep_of is None:
        pos = first[:, None] + torch.arange(most, device=q.device)
        keep = (where < s["kv_len"][:, None, None]) & (where <= pos[..., None])
        if case.get("window"):
            keep = keep & (where > pos[..., None] - case["window"])
    else:
        keep = keep_of(first, where)
    score = score.view(n, h, most, g, width).masked_fill_(~keep[:, None, :, None, :], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    score = score.sub_(top).exp_()
    total = score.sum(-1, keepdim=True)
    out = torch.matmul(score.view(n, h, most * g, width), v).view(n, h, most, g, d) / total.clamp(min=1e-30)
    lse = (top + total.log()).squeeze(-1)
    out = out.permute(0, 2, 1, 3, 4)[at].reshape(-1, case["heads"], d)
    return {"out": out.bfloat16(), "lse": lse.permute(0, 2, 1, 3)[at].reshape(-1, case["heads"])}


def plain_tree(s):
    """Ancestors of every node by squaring the parent relation; a window counts depths."""
    case = s["case"]
    n, most, w = case["seqs"], case["q"], case.get("window", 0)
    count = (s["starts"][1:] - s["starts"][:-1]).long()
    index = torch.arange(s["seq"].numel(), device="cuda") - s["starts"][s["seq"].long()].long()
    at = (s["seq"].long(), index)
    up = torch.zeros((n, most, most + 1), device="cuda")  # the last column: the context
    up[at[0], index, torch.where(s["parent"] < 0, most, s["parent"].long())] = 1
    reach = up[..., :most] + torch.eye(most, device="cuda")
    for _ in range(max(1, (most - 1).bit_length())):
        reach = torch.matmul(reach, reach.contiguous()).clamp_(max=1)
    depth = reach.sum(-1).long() - 1
    keep_new = reach > 0
    if w:
        keep_new = keep_new & (depth[:, None, :] > depth[..., None] - w)
    words = -(-most // 64)
    bits = torch.zeros((n, most, words * 64), dtype=torch.int64, device="cuda")
    bits[..., :most] = keep_new
    mask = (bits.view(n, most, words, 64) << torch.arange(64, device="cuda")).sum(-1)

    def keep_of(first, where):
        new = where - first[:, None]  # [n, width]: the node at each position
        context = new < 0
        inside = (new >= 0) & (new < count[:, None])
        node = keep_new.gather(2, new.clamp(0, most - 1)[:, None, :].expand(n, most, -1))
        context = context[:, None, :].expand(n, most, -1)
        if w:
            context = context & (where > (first[:, None] + depth)[..., None] - w)
        return context | (inside[:, None, :] & node)

    return {"mask": mask[at], "depth": depth[at].int(), **plain_attn(s, keep_of)}


def plain_path(s):
    page = s["case"]["page"]
    seq, i = (s["path"] >= 0).nonzero(as_tuple=True)
    src, dst = s["base"][seq].long() + s["path"][seq, i].long(), s["base"][seq].long() + i
    table = s["table"].long()
    a, b = (table[seq, src // page], src % page), (table[seq, dst // page], dst % page)
    for name in ("cache", "scales") if s["fp8"] else ("cache",):
        rows = s[name].view(torch.uint8) if s[name].dtype == torch.float8_e4m3fn else s[name]
        rows[b[0], :, :, b[1]] = rows[a[0], :, :, a[1]]
    return {"cache": s["cache"], "scales": s["scales"]} if s["fp8"] else s["cache"]


def steps(top):
    """The exponent of whole-number steps for magnitudes up to `top`, and its limits."""
    part, e = torch.frexp(top)
    return torch.where(top > 0, (e - 7 + (part > 127 / 128)).clamp(-50, 50), -50)


def bounds_rows(k, filled):
    """Bounds of pages from their keys k [pages, heads, page, dim] in fp32, the first `filled` [pages] of each."""
    n, h, p, d = k.shape
    use = (torch.arange(p, device=k.device) < filled[:, None])[:, None, :, None] & k.isfinite()
    hi = torch.where(use, k, -math.inf).amax(2)
    lo = torch.where(use, k, math.inf).amin(2)
    none = hi < lo
    hi, lo = torch.where(none, 0, hi), torch.where(none, 0, lo)
    e = steps(torch.maximum(hi.abs(), lo.abs()).amax(-1))
    unit = power(-e)[..., None]
    rows = torch.zeros((n, h, row_bytes(d)), dtype=torch.uint8, device=k.device)
    rows[..., :d] = (hi * unit).ceil().clamp(-127, 127).to(torch.int8).view(torch.uint8)
    rows[..., d: 2 * d] = (lo * unit).floor().clamp(-127, 127).to(torch.int8).view(torch.uint8)
    rows[..., -16:-12] = e.int().contiguous().view(torch.uint8).view(n, h, 4)
    return rows


def query_steps(q):
    """Whole numbers of query rows in steps of 2^g, and g."""
    q = q.float()
    q = torch.where(q.isfinite(), q, 0)
    g = steps(q.abs().amax(-1))
    return (q * power(-g)[..., None]).round().clamp(-127, 127), g


def plain_blocks(s):
    case = s["case"]
    n, h, d, p, count = case["seqs"], case["kv_heads"], case["dim"], case["page"], case["count"]
    t, grp = s["seq"].numel(), case["heads"] // h
    # the bounds of every page that the new tokens reached
    first, width = s["begin"].long() // p, s["table"].shape[1]
    at = torch.arange(width, device="cuda")
    touched = (at >= first[:, None]) & (at * p < s["end"][:, None])
    seq, page = touched.nonzero(as_tuple=True)
    ids = s["table"][seq, page].long()
    s["bounds"][ids] = bounds_rows(dequantised(s, ids, 0), (s["end"][seq].long() - page * p).clamp(max=p))
    # scores: the sum of max(q hi, q lo) is that of the positive part times hi and the negative part times lo
    rows = s["bounds"][s["table"].clamp(min=0).long()]  # [n, pages, heads, bytes]
    limit = rows[..., : 2 * d].contiguous().view(torch.int8)
    e = rows[..., -16:-12].contiguous().view(torch.int32).squeeze(-1)
    q, g = query_steps(s["q"].view(t, h, grp, d))
    q = torch.cat((q.clamp(min=0), q.clamp(max=0)), -1)
    score = torch.empty((t, h, width), device="cuda")
    most = case["q"]
    padded = torch.zeros((n, most, h, grp, 2 * d), device="cuda")
    index = (torch.arange(t, device="cuda") - s["starts"][s["seq"].long()].long())
    padded[s["seq"].long(), index] = q
    padded = padded.permute(0, 2, 1, 3, 4).reshape(n * h, most * grp, 2 * d)
    dots = torch.matmul(padded, limit.float().permute(0, 2, 3, 1).reshape(n * h, 2 * d, width).contiguous())
    dots = dots.view(n, h, most, grp, width).permute(0, 2, 1, 3, 4)[s["seq"].long(), index]  # [t, h, grp, pages]
    score = (dots * power(g)[..., None]).amax(2) * power(e.permute(0, 2, 1)[s["seq"].long()])
    # the first page, the last two, and the best of the others; ties go to the lowest
    own_n = (s["pos"].long() // p + 1)[:, None, None]
    forced = (at < 1) | (at >= own_n - 2)
    score = torch.where(forced, math.inf, score)
    score = torch.where(at < own_n, score, -math.inf).expand(t, h, width)
    best = score.sort(dim=-1, descending=True, stable=True).indices[..., :count]
    best = torch.where(torch.arange(best.shape[-1], device="cuda") < own_n, best, 1 << 30).sort(-1).values
    blocks = torch.full((t, h, count), -1, dtype=torch.int32, device="cuda")
    blocks[..., : best.shape[-1]] = torch.where(best < 1 << 30, best, -1)
    # attention over them
    ids = s["table"][s["seq"].long()[:, None, None], blocks.clamp(min=0).long()].long()
    head = torch.arange(h, device="cuda")[None, :, None].expand_as(ids)
    k, v = (dequantised(s, ids, w, head).view(t, h, count * p, d) for w in (0, 1))
    pos = (blocks[..., None].long() * p + torch.arange(p, device="cuda")).view(t, h, count * p)
    keep = (blocks >= 0)[..., None].expand(t, h, count, p).reshape(t, h, count * p) & (pos <= s["pos"].long()[:, None, None])
    z = torch.matmul(s["q"].view(t, h, grp, d).float(), k.transpose(2, 3).contiguous()) / math.sqrt(d)
    z = z.masked_fill_(~keep[:, :, None, :], -math.inf)
    top = z.amax(-1, keepdim=True)
    z = z.sub_(top).exp_()
    total = z.sum(-1, keepdim=True)
    out = (torch.matmul(z, v) / total).view(t, case["heads"], d)
    return {"bounds": s["bounds"], "blocks": blocks, "out": out.bfloat16(), "lse": (top + total.log()).view(t, case["heads"])}


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    op, h, d = case["op"], case["kv_heads"], case["dim"]
    lens = lengths(case)
    t = sum(q for q, _ in lens)
    row = d + 1 if op in ("append8", "read8") or case["fp8"] else 2 * d  # bytes of a cached row of one head
    if op in ("append8", "read8"):
        return {"bytes": t * (2 * h * (2 * d + row) + 8), "flops": 0}
    if op == "path":
        moved = sum(min(case["path"], q // 2) for q, _ in lens)
        return {"bytes": 4 * moved * h * row, "flops": 0}
    outside = t * case["heads"] * (4 * d + 4)
    if op == "blocks":
        p, count = case["page"], case["count"]
        rows = sum(min(kv, q * count * p) for q, kv in lens) * h  # a selected page is read once, however many tokens select it
        pairs = sum(min(kv - q + i + 1, count * p) for q, kv in lens for i in range(q))
        scored = sum(-(-kv // p) for _, kv in lens) * h * row_bytes(d)
        marks = sum(-(-(kv - q + i + 1) // p) for q, kv in lens for i in range(q))
        return {"bytes": 2 * rows * row + scored + outside + 4 * t * h * count, "flops": 4.0 * pairs * case["heads"] * d + 4.0 * marks * case["heads"] * d}
    w = case.get("window", 0)
    kept = sum(min(kv, q + w - 1) if w else kv for q, kv in lens)
    if op == "tree":
        pairs = sum(q * (min(kv - q, w) if w else kv - q) + 4 * q for q, kv in lens)
        outside += 8 * t * (-(-case["q"] // 64)) + 8 * t
    else:
        pairs = sum(min(kv - q + i + 1, w) if w else kv - q + i + 1 for q, kv in lens for i in range(q))
    return {"bytes": 2 * kept * h * row + outside, "flops": 4.0 * pairs * case["heads"] * d}


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op, h, d, p = case["op"], case["kv_heads"], case["dim"], case["page"]
    lens = lengths(case)

    def rows64(which, i, head, count):
        """The first `count` rows of one head of sequence i."""
        ids = s["table"][i, : -(-count // p)].long()
        got = s["cache"].view(torch.uint8)[ids, which, head].view(torch.float8_e4m3fn).double() if s["fp8"] else s["cache"][ids, which, head].double()
        if s["fp8"]:
            got = got * torch.exp2(s["scales"][ids, which, head].double() - 127)[..., None]
        return got.reshape(-1, d)[:count]

    if op == "append8":
        cache, scales = s["cache"].double(), s["scales"].clone()
        at = s["table"][s["seq"].long(), s["pos"].long() // p].long()
        slot = s["pos"].long() % p
        for which, new in ((0, s["k"]), (1, s["v"])):
            new = new.double()
            top = new.abs().amax(-1)
            e = torch.full(top.shape, float(LEAST_EXP), dtype=torch.float64, device="cuda")
            e = torch.where(top > 0, torch.ceil(torch.log2(top.clamp(min=1e-300) / 448)), e)
            # the logarithm may be a hair off at a power of two: the least exponent that holds the row
            e = torch.where(top * torch.exp2(-(e - 1)) <= 448, e - 1, e)
            e = torch.where(top * torch.exp2(-e) > 448, e + 1, e).clamp(min=LEAST_EXP)
            cache[at, which, :, slot] = new * torch.exp2(-e)[..., None]
            scales[at, which, :, slot] = (e + 127).to(torch.uint8)
        return {"cache": cache, "scales": scales}
    if op == "read8":
        got = [torch.cat([torch.stack([rows64(w, i, j, kv)[kv - q:] for j in range(h)], 1) for i, (q, kv) in enumerate(lens)]) for w in (0, 1)]
        return {"k": got[0], "v": got[1]}
    if op == "path":
        cache = s["cache"].double()
        scales = s["scales"].clone() if s["fp8"] else None
        path, base, table = s["path"].tolist(), s["base"].tolist(), s["table"].tolist()
        for i in range(case["seqs"]):
            for j, node in enumerate(path[i]):
                if node < 0:
                    break
                a, b = base[i] + node, base[i] + j
                for store in (cache, scales) if s["fp8"] else (cache,):
                    store[table[i][b // p], :, :, b % p] = store[table[i][a // p], :, :, a % p]
        return {"cache": cache, "scales": scales} if s["fp8"] else cache
    if op == "blocks":
        return exact_blocks(case, s, lens, rows64)

    group, w = case["heads"] // h, case.get("window", 0)
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    if sum(q * kv for q, kv in lens) * case["heads"] * d > 3e12:
        return None
    words = -(-case["q"] // 64)
    masks, depths, at = [], [], 0
    parent = s["parent"].tolist() if op == "tree" else None
    for i, (q, kv) in enumerate(lens):
        j = torch.arange(kv, device="cuda")
        pos = torch.arange(kv - q, kv, device="cuda")
        if op == "attn":
            bad = j[None, :] > pos[:, None]
            if w:
                bad |= j[None, :] <= pos[:, None] - w
        else:
            bad = torch.ones((q, kv), dtype=torch.bool)
            chains = []
            for node in range(q):
                up = parent[at + node]
                chains.append((chains[up] if up >= 0 else []) + [node])
                line = chains[node]
                seen = line[-w:] if w else line
                depths.append(len(line) - 1)
                for word in range(words):
                    v = sum(1 << (x - 64 * word) for x in seen if x // 64 == word)
                    masks.append(v - (1 << 64) if v >> 63 else v)
                low = max(0, kv - q + len(line) - 1 - w + 1) if w else 0
                bad[node, low: kv - q] = False
                bad[node, [kv - q + x for x in seen]] = False
            bad = bad.cuda()
        for head_kv in range(h):
            k, v = rows64(0, i, head_kv, kv), rows64(1, i, head_kv, kv)
            for head in range(head_kv * group, (head_kv + 1) * group):
                z = s["q"][at: at + q, head].double() @ k.t() * d ** -0.5
                z.masked_fill_(bad, -math.inf)
                lse[at: at + q, head] = torch.logsumexp(z, 1)
                out[at: at + q, head] = torch.softmax(z, 1) @ v
        at += q
    if op == "attn":
        return {"out": out, "lse": lse}
    return {"mask": torch.tensor(masks, dtype=torch.int64, device="cuda").view(-1, words),
            "depth": torch.tensor(depths, dtype=torch.int32, device="cuda"), "out": out, "lse": lse}


def exact_blocks(case, s, lens, rows64):
    """Bounds, scores and lists of one sequence and head after the other, all of it whole numbers times powers of two."""
    h, d, p, count = case["kv_heads"], case["dim"], case["page"], case["count"]
    group = case["heads"] // h
    bounds = s["bounds"].clone()
    blocks = torch.full(s["blocks"].shape, -1, dtype=torch.int32, device="cuda")
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device="cuda")

    def unit(top):
        e = torch.full(top.shape, -50.0, dtype=torch.float64, device="cuda")
        some = top > 0
        e[some] = torch.floor(torch.log2(top[some])) - 6
        e[some & (top * torch.exp2(-e) > 127)] += 1
        return e.clamp(-50, 50)

    at = 0
    for i, (q, kv) in enumerate(lens):
        pages = -(-kv // p)
        ids = s["table"][i, :pages].long()
        for head in range(h):
            k, v = rows64(0, i, head, kv), rows64(1, i, head, kv)
            for page in range((kv - q) // p, pages):
                part = k[page * p: min(kv, (page + 1) * p)]
                hi, lo = part.amax(0), part.amin(0)
                e = unit(torch.maximum(hi.abs().max(), lo.abs().max())[None])
                both = torch.cat((torch.ceil(hi * torch.exp2(-e)), torch.floor(lo * torch.exp2(-e)))).clamp(-127, 127)
                bounds[ids[page], head, : 2 * d] = both.to(torch.int8).view(torch.uint8)
                bounds[ids[page], head, -16:-12] = e.to(torch.int32).view(torch.uint8)
            limit = bounds[ids, head, : 2 * d].view(torch.int8).double()
            e = bounds[ids, head, -16:-12].contiguous().view(torch.int32).double().flatten()
            x = s["q"][at: at + q, head * group: (head + 1) * group].double()
            g = unit(x.abs().amax(-1).flatten()).view(q, group)
            x = torch.round(x * torch.exp2(-g)[..., None]).clamp(-127, 127)
            total = torch.maximum(x[..., None, :] * limit[:, :d], x[..., None, :] * limit[:, d:]).sum(-1) if q * group * pages * d < 3e8 else \
                x.clamp(min=0) @ limit[:, :d].t() + x.clamp(max=0) @ limit[:, d:].t()
            total = (total * torch.exp2(g)[..., None]).amax(1) * torch.exp2(e)  # [q, pages]
            for t in range(q):
                pos = kv - q + t
                n = pos // p + 1
                part = total[t, :n].clone()
                part[:1] = math.inf
                part[max(0, n - 2):] = math.inf
                pick = torch.sort(part, descending=True, stable=True).indices[:count].sort().values
                blocks[at + t, head, : pick.numel()] = pick.int()
                cols = (pick[:, None] * p + torch.arange(p, device="cuda")).flatten()
                cols = cols[cols <= pos]
                z = s["q"][at + t, head * group: (head + 1) * group].double() @ k[cols].t() * d ** -0.5
                lse[at + t, head * group: (head + 1) * group] = torch.logsumexp(z, 1)
                out[at + t, head * group: (head + 1) * group] = torch.softmax(z, 1) @ v[cols]
        at += q
    return {"bounds": bounds, "blocks": blocks, "out": out, "lse": lse}
