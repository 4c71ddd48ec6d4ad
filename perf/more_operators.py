"""Measured cases of the operators for several continuations of one prompt: the decode
of a batch that shares prefixes, the selection over beams and vocabulary, and the
forking and reserving of cache pages.

``run`` computes each operator in its plain form (elementary torch operations) or,
with ``own``, through the package's entry points.  ``exact`` gives the same outputs
from the definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

LATENT, ROPE, ROW, PAGE = 512, 64, 576, 1536
SCALE = 1.0 / math.sqrt(192.0)
KV_SCALE = 6.0 / 448.0          # N(0, 1) values reach E4M3's 448 at 6 deviations
E4M3 = torch.float8_e4m3fn
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4, "e4m3": 1}


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def listed():
    return [
        # two answers to one short prompt, 16 heads: the smallest step, latency only
        {"name": "shared tiny bf16", "op": "shared", "type": "bf16", "groups": 1, "reqs": 2,
         "n_q": 1, "heads": 16, "prefix_lo": 1500, "prefix_hi": 1500, "own_lo": 1, "own_hi": 90,
         "alone": 0, "lens_seed": 0},
        # eight answers to a document of 20k tokens: neither bytes nor products dominate
        {"name": "shared answers bf16", "op": "shared", "type": "bf16", "groups": 1, "reqs": 8,
         "n_q": 1, "heads": 64, "prefix_lo": 20011, "prefix_hi": 20011, "own_lo": 100,
         "own_hi": 2000, "alone": 0, "lens_seed": 1},
        # a serving batch of 64 under one long system prompt
        {"name": "shared system prompt bf16", "op": "shared", "type": "bf16", "groups": 1,
         "reqs": 64, "n_q": 1, "heads": 64, "prefix_lo": 32768, "prefix_hi": 32768,
         "own_lo": 300, "own_hi": 4000, "alone": 0, "lens_seed": 2},
        # a 4-draft verification over the FP8 cache: four prompts and requests of their own
        {"name": "shared verify e4m3", "op": "shared", "type": "e4m3", "groups": 4, "reqs": 48,
         "n_q": 4, "heads": 64, "prefix_lo": 3000, "prefix_hi": 12000, "own_lo": 64,
         "own_hi": 3000, "alone": 4, "lens_seed": 3},
        # one prompt's four beams over a small vocabulary: latency only
        {"name": "beams tiny fp32", "op": "beams", "type": "fp32", "batch": 1, "beams": 4,
         "vocab": 32000, "first": False, "ended": False},
        # a batch of beam searches over a large vocabulary, some beams at their end
        {"name": "beams batch bf16", "op": "beams", "type": "bf16", "batch": 32, "beams": 4,
         "vocab": 150001, "first": False, "ended": True},
        # wide beams
        {"name": "beams wide fp16", "op": "beams", "type": "fp16", "batch": 4, "beams": 32,
         "vocab": 100257, "first": False, "ended": False},
        # four beams of a short prompt move to their parents: latency only
        {"name": "fork tiny", "op": "fork", "prompts": 1, "rows": 4, "pages_lo": 2, "pages_hi": 2,
         "pool": 64, "lens_seed": 5},
        # 128 searches of eight beams over histories of up to 500k tokens
        {"name": "fork long", "op": "fork", "prompts": 128, "rows": 1024, "pages_lo": 40,
         "pages_hi": 330, "pool": 65536, "lens_seed": 6},
        # two continuations of one prompt part: one page copied
        {"name": "reserve tiny bf16", "op": "reserve", "type": "bf16", "prompts": 1, "rows": 2,
         "pages_lo": 1, "pages_hi": 1, "layers": 1, "new": 1, "pool": 8, "lens_seed": 7},
        # eight prompts part into 64 continuations, four layers of an FP8 cache
        {"name": "reserve layers e4m3", "op": "reserve", "type": "e4m3", "prompts": 8, "rows": 64,
         "pages_lo": 1, "pages_hi": 4, "layers": 4, "new": 200, "pool": 192, "lens_seed": 8},
    ]


def draw(rng):
    def log(lo, hi):
        return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))

    op = rng.choice(["shared", "shared", "beams", "fork", "reserve"])
    seed = rng.randrange(1 << 20)
    if op == "shared":
        n_q = rng.choice([1, 1, 1, 2, 3, 4, 8])
        heads = rng.choice([8, 16, 32, 48, 64, 64, 64, 80, 128])
        reqs = log(1, 64)
        groups = rng.randint(1, max(1, reqs // 2))
        most = min(2000000 // reqs, 140000000 // (reqs * n_q * heads))
        prefix = log(min(100, most // 2), max(101, most * 3 // 4))
        tail = log(n_q, max(n_q + 1, min(6000, most // 4)))
        return {"op": op, "type": rng.choice(["bf16", "bf16", "e4m3"]), "groups": groups,
                "reqs": reqs, "n_q": n_q, "heads": heads, "prefix_lo": max(1, prefix // 2),
                "prefix_hi": prefix,
                "own_lo": rng.choice([n_q, max(n_q, tail // 3)]), "own_hi": tail,
                "alone": rng.choice([0, 0, min(3, reqs - groups)]), "lens_seed": seed}
    if op == "beams":
        beams = log(1, 64)
        vocab = log(100, 200000)
        return {"op": op, "type": rng.choice(["bf16", "bf16", "fp16", "fp32"]), "beams": beams,
                "batch": log(1, max(1, min(64, 19000000 // (beams * vocab)))), "vocab": vocab,
                "first": rng.random() < 0.25, "ended": rng.random() < 0.4}
    if op == "fork":
        prompts = log(1, 128)
        rows = prompts * rng.randint(1, 8)
        hi = log(1, 330)
        return {"op": op, "prompts": prompts, "rows": rows, "pages_lo": max(1, hi // 3),
                "pages_hi": hi, "pool": prompts * hi + 3 * rows + log(20, 20000), "lens_seed": seed}
    prompts = log(1, 8)
    rows = prompts * rng.randint(1, 8)
    hi = rng.randint(1, 4)
    new = rng.choice([1, 1, 4, log(1, 1500)])
    return {"op": op, "type": rng.choice(["bf16", "e4m3"]), "prompts": prompts, "rows": rows,
            "pages_lo": 1, "pages_hi": hi, "layers": rng.choice([1, 2, 3]), "new": new,
            "pool": prompts * hi + 3 * rows + log(2, 16), "lens_seed": seed}


def shared_plan(case):
    """Group starts, tokens that a group shares, history lengths, as numpy arrays."""
    rng = np.random.default_rng(case["lens_seed"])
    grouped = case["reqs"] - case["alone"]
    cuts = np.sort(rng.choice(np.arange(1, grouped), case["groups"] - 1, replace=False)) \
        if case["groups"] > 1 else np.zeros(0, dtype=np.int64)
    # requests of no group come last, each a group of its own that shares nothing
    starts = np.concatenate([[0], cuts, np.arange(grouped, case["reqs"] + 1)]).astype(np.int64)
    G = len(starts) - 1
    prefix = rng.integers(case["prefix_lo"], case["prefix_hi"] + 1, G)
    prefix[case["groups"]:] = 0
    group = np.repeat(np.arange(G), np.diff(starts))
    lens = prefix[group] + rng.integers(case["own_lo"], case["own_hi"] + 1, case["reqs"])
    return starts, prefix, group, lens


def page_plan(case):
    """Histories of prompts that parted earlier (fork) or not yet (reserve): the prompt of
    each row, its parent, the tokens of each row."""
    rng = np.random.default_rng(case["lens_seed"])
    each = case["rows"] // case["prompts"]
    prompt = np.repeat(np.arange(case["prompts"]), each)
    if case["op"] == "reserve":
        pages = rng.integers(case["pages_lo"], case["pages_hi"] + 1, case["prompts"])
        lens = pages * PAGE - rng.integers(0, PAGE, case["prompts"])
        return prompt, prompt, lens
    pages = rng.integers(case["pages_lo"], case["pages_hi"] + 1, case["prompts"])
    lens = np.repeat(pages * PAGE - rng.integers(0, PAGE, case["prompts"]), each)
    parent = prompt * each + rng.integers(0, each, case["rows"])
    parent[rng.random(case["rows"]) < 0.02] = -1        # a search that has ended
    return prompt, parent, lens


def work(case):
    op = case["op"]
    if op == "shared":
        starts, prefix, _, lens = shared_plan(case)
        members = np.diff(starts)
        rows = case["n_q"] * case["heads"]
        tokens = int(lens.sum() - ((members - 1) * prefix).sum())
        total = case["reqs"] * rows
        return {"bytes": tokens * ROW * BYTES[case["type"]] + total * (2 * ROW + 4 * LATENT + 4),
                "flops": 2 * (ROW + LATENT) * rows * int(lens.sum())}
    if op == "beams":
        n = case["batch"] * case["beams"]
        return {"bytes": n * case["vocab"] * BYTES[case["type"]] + 16 * n,
                "flops": 4 * n * case["vocab"]}
    prompt, parent, lens = page_plan(case)
    if op == "fork":
        pages = int((-(-lens // PAGE))[parent[parent >= 0]].sum())
        return {"bytes": 8 * pages + 8 * min(case["pool"], pages) + 12 * case["rows"],
                "flops": 2 * pages}
    each = case["rows"] // case["prompts"]
    copied = int((lens % PAGE).sum()) * (each - 1)
    return {"bytes": 2 * case["layers"] * copied * ROW * BYTES[case["type"]]
            + 4 * case["pool"] + 24 * case["rows"], "flops": 0}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    mix = np.random.default_rng(seed)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.empty(*shape, dtype=dtype, device=dev).normal_(generator=g)

    def slab(pool):
        s = normal(pool, PAGE * ROW)
        return (s.float() / KV_SCALE).clamp(-448, 448).to(E4M3) if case["type"] == "e4m3" else s

    def ints(a):
        return torch.as_tensor(np.ascontiguousarray(a), dtype=torch.int32, device=dev)

    op = case["op"]
    s = {"case": case, "op": op}
    if op == "beams":
        n, V = case["batch"] * case["beams"], case["vocab"]
        # a next-token distribution: a few likely tokens over a broad tail
        x = normal(n, V, dtype=torch.float32)
        s["logits"] = (2.0 * x + 0.25 * x.abs().pow(3)).to(TYPES[case["type"]])
        score = normal(case["batch"], case["beams"], dtype=torch.float32) - 20.0
        if case["first"]:
            # before the first token the beams are one: the others count nothing
            score[:, 0], score[:, 1:] = 0.0, -math.inf
        s["scores"] = score.sort(1, descending=True).values
        s["ended"], s["end"] = None, -1
        if case["ended"]:
            s["ended"] = torch.rand(score.shape, generator=g, device=dev) < 0.3
            s["end"] = V // 3
        return s
    if op == "shared":
        starts, prefix, group, lens = shared_plan(case)
        whole = prefix // PAGE                       # pages that a group's members share
        need = -(-lens // PAGE)
        pool = int(whole.sum() + (need - whole[group]).sum()) + 2
        ids = mix.permutation(pool)
        table = np.zeros((case["reqs"], int(max(1, need.max()))), dtype=np.int64)
        at = 0
        common = []
        for n in whole:
            common.append(ids[at:at + n])
            at += n
        for r in range(case["reqs"]):
            n = whole[group[r]]
            table[r, :n] = common[group[r]]
            table[r, n:need[r]] = ids[at:at + need[r] - n]
            at += need[r] - n
        s["slab"] = slab(pool)
        # the prefix's last rows lie in a page of each member: copies of the first one's
        part = prefix % PAGE
        mine = table[np.arange(case["reqs"]), whole[group]]
        theirs = mine[starts[:-1]][group]
        rows = s["slab"].view(torch.uint8) if case["type"] == "e4m3" else s["slab"]
        rows = rows.view(pool, PAGE, ROW)
        same = torch.arange(PAGE, device=dev)[None, :, None] < \
            torch.as_tensor(part[group], device=dev)[:, None, None]
        mine, theirs = torch.as_tensor(mine, device=dev), torch.as_tensor(theirs, device=dev)
        rows[mine] = torch.where(same, rows[theirs], rows[mine])
        T = case["reqs"] * case["n_q"]
        s["qn"], s["qr"] = normal(T, case["heads"], LATENT), normal(T, case["heads"], ROPE)
        s["gate"] = normal(T, case["heads"], LATENT)
        s["table"], s["lens"] = ints(table), ints(lens)
        s["starts"], s["prefix"] = ints(starts), ints(prefix)
        s["top"] = int(lens.max())
        if own:
            import paged_latent_attention_gb300 as plmla
            s["workspace"] = plmla.allocate_shared_workspace(
                case["reqs"], case["n_q"], case["heads"], fp8=case["type"] == "e4m3")
        return s
    prompt, parent, lens = page_plan(case)
    pool, rows = case["pool"], case["rows"]
    need = -(-lens // PAGE)
    ids = mix.permutation(pool)
    cols = int(need.max()) + 2
    at = 0
    if op == "reserve":
        table = np.zeros((case["prompts"], cols), dtype=np.int64)
        for r in range(case["prompts"]):
            table[r, :need[r]] = ids[at:at + need[r]]
            at += need[r]
        s["slabs"] = [slab(pool) for _ in range(case["layers"])]
    else:
        # beams of a prompt share all pages but the last
        table = np.zeros((rows, cols), dtype=np.int64)
        for r in range(rows):
            if r == 0 or prompt[r] != prompt[r - 1]:
                common = ids[at:at + need[r] - 1]
                at += need[r] - 1
            table[r, :need[r] - 1] = common
            table[r, need[r] - 1] = ids[at]
            at += 1
    inside = np.arange(cols)[None] < need[:, None]
    counts = np.bincount(table[inside], minlength=pool)
    # some of the remaining pages belong to others
    rest = ids[at:]
    spare = 2 * rows if op == "reserve" else len(rest) // 2
    counts[rest[:max(0, len(rest) - spare)]] = 1
    s["counts"] = ints(counts)
    s["table"], s["lens"], s["parents"] = ints(table), ints(lens), ints(parent)
    s["out_table"] = torch.zeros(rows, cols, dtype=torch.int32, device=dev)
    s["out_lens"] = torch.zeros(rows, dtype=torch.int32, device=dev)
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def run(state):
    op = state["op"]
    if own:
        return {"shared": own_shared, "beams": own_beams, "fork": own_fork,
                "reserve": own_reserve}[op](state)
    return {"shared": plain_shared, "beams": plain_beams, "fork": plain_fork,
            "reserve": plain_reserve}[op](state)


def own_shared(s):
    import paged_latent_attention_gb300 as plmla
    c = s["case"]
    args = (s["qn"], s["qr"], s["gate"], s["slab"], s["table"], s["lens"], s["starts"],
            s["prefix"])
    if c["type"] == "e4m3":
        return plmla.mla_decode_shared_fp8(*args, kv_scale=KV_SCALE, n_q=c["n_q"],
                                           workspace=s["workspace"])
    return plmla.mla_decode_shared(*args, n_q=c["n_q"], workspace=s["workspace"])


def own_beams(s):
    import paged_latent_attention_gb300 as plmla
    return plmla.mla_beam_select(s["logits"], s["scores"], ended=s["ended"], end_token=s["end"])


def own_fork(s):
    import paged_latent_attention_gb300 as plmla
    # out_table's rows give up the pages of the pass before
    plmla.mla_pages_fork(s["table"], s["lens"], s["parents"], s["counts"], s["out_table"],
                         s["out_lens"])
    return s["out_table"], s["out_lens"], s["counts"]


def own_reserve(s):
    import paged_latent_attention_gb300 as plmla
    new = s["case"]["new"]
    plmla.mla_pages_fork(s["table"], s["lens"], s["parents"], s["counts"], s["out_table"],
                         s["out_lens"])
    plmla.mla_pages_reserve(s["slabs"], s["out_table"], s["out_lens"], new, s["counts"])
    s["out_lens"] += new
    return s["out_table"], s["out_lens"], s["counts"], s["slabs"]


def plain_shared(s):
    c, R, top = s["case"], s["lens"].shape[0], s["top"]
    if c["type"] == "e4m3":
        k = s["slab"].view(torch.uint8)[s["table"].long()].view(E4M3).float() * KV_SCALE
    else:
        k = s["slab"][s["table"].long()].float()
    k = k.view(R, -1, ROW)[:, :top]
    q = torch.cat([s["qn"], s["qr"]], -1).float().view(R, c["n_q"] * c["heads"], ROW)
    score = torch.bmm(q, k.transpose(1, 2)) * SCALE
    behind = c["n_q"] - 1 - torch.arange(c["n_q"], device=k.device).repeat_interleave(c["heads"])
    seen = torch.arange(top, device=k.device)[None, None] < \
        (s["lens"].long()[:, None] - behind[None])[:, :, None]
    score = score.masked_fill_(~seen, -math.inf)
    high = score.amax(2, keepdim=True)
    high = torch.where(high == -math.inf, 0.0, high)
    weight = torch.exp(score.sub_(high))
    total = weight.sum(2, keepdim=True)
    out = torch.bmm(weight, k[:, :, :LATENT]) / torch.where(total > 0.0, total, 1.0)
    lse = (torch.log(total) + high).view(-1, c["heads"])
    out = out.view(-1, c["heads"], LATENT) / (1.0 + torch.exp(-s["gate"].float()))
    return out.to(torch.bfloat16), lse


def plain_beams(s):
    B, K = s["scores"].shape
    # in 64 bits: candidates of different beams are compared
    x = s["logits"].double().view(B, K, -1)
    V = x.shape[2]
    high = x.amax(2, keepdim=True)
    lse = torch.log(torch.exp(x - high).sum(2, keepdim=True)) + high
    cand = s["scores"].double()[:, :, None] + (x - lse)
    if s["ended"] is not None:
        stay = torch.where(torch.arange(V, device=x.device) == s["end"],
                           s["scores"].double()[:, :, None], -math.inf)
        cand = torch.where(s["ended"][:, :, None], stay, cand)
    best = cand.view(B, K * V).sort(dim=1, descending=True, stable=True)
    i = best.indices[:, :K]
    first = K * torch.arange(B, device=x.device)[:, None]
    return (i % V).int(), (first + i // V).int(), best.values[:, :K].float()


def held(table, lens):
    """Which entries of a table's rows hold a page."""
    return torch.arange(table.shape[1], device=table.device)[None] < \
        ((lens.long() + PAGE - 1) // PAGE)[:, None]


def plain_fork(s):
    out, counts = s["out_table"], s["counts"]
    counts.scatter_add_(0, out.long().view(-1), -held(out, s["out_lens"]).int().view(-1))
    parent = s["parents"].long()
    lens = torch.where(parent >= 0, s["lens"][parent.clamp(min=0)], 0)
    rows = s["table"][parent.clamp(min=0)]
    keep = held(rows, lens)
    out.copy_(torch.where(keep, rows, out))
    counts.scatter_add_(0, rows.long().view(-1), keep.int().view(-1))
    s["out_lens"].copy_(lens)
    return out, s["out_lens"], counts


def plain_reserve(s):
    plain_fork(s)
    new, table, counts = s["case"]["new"], s["out_table"], s["counts"]
    lens = s["out_lens"].long()
    R, cols = table.shape
    have, want = (lens + PAGE - 1) // PAGE, (lens + new + PAGE - 1) // PAGE
    at = (lens // PAGE)[:, None]
    last = table.long().gather(1, at)[:, 0]
    part = lens % PAGE > 0
    # earlier rows that part from the same page leave one holder less each
    same = (last[:, None] == last[None]) & part[:, None] & part[None]
    order = torch.arange(R, device=lens.device)
    earlier = (same & (order[None] < order[:, None])).sum(1)
    copied = part & (counts[last] - earlier > 1)
    need = want - have + copied
    # pages without a holder, lowest first
    free = (counts > 0).int().sort(stable=True).indices
    first = need.cumsum(0) - need
    fresh = free[first.clamp(max=counts.shape[0] - 1)]
    counts.scatter_add_(0, last, -copied.int())
    # the copy's page, then those of the new tokens
    page = torch.where(copied, fresh, last)
    table.scatter_(1, at, torch.where(part, page, table.long().gather(1, at)[:, 0])[:, None].int())
    c = torch.arange(cols, device=lens.device)[None]
    grown = (c >= have[:, None]) & (c < want[:, None])
    nth = (first + copied)[:, None] + c - have[:, None]
    table.copy_(torch.where(grown, free[nth.clamp(0, counts.shape[0] - 1)].int(), table))
    counts.scatter_add_(0, page, copied.int())
    counts.scatter_add_(0, table.long().view(-1), grown.int().view(-1))
    inside = torch.arange(PAGE, device=lens.device)[None, :] < \
        torch.where(copied, lens % PAGE, 0)[:, None]
    dst = torch.where(inside, page[:, None] * PAGE + torch.arange(PAGE, device=lens.device), -1)
    src = torch.where(inside, last[:, None] * PAGE + torch.arange(PAGE, device=lens.device), -1)
    [copy_rows(x, src.view(-1), dst.view(-1)) for x in s["slabs"]]
    s["out_lens"] += new
    return table, s["out_lens"], counts, s["slabs"]


def copy_rows(slab, src, dst):
    """Rows src to rows dst; a pair of -1 repeats the pair with the highest dst (where every
    pair is -1, row 0 goes onto itself)."""
    x, last = rows_of(slab), dst.argmax()
    src, dst = torch.where(dst < 0, src[last], src), torch.where(dst < 0, dst[last], dst)
    x.index_copy_(0, dst.clamp(min=0), x[src.clamp(min=0)])


def rows_of(slab):
    return (slab.view(torch.uint8) if slab.dtype == E4M3 else slab).view(-1, ROW)


# --------------------------------------------------------------------------
# 64 bits
# --------------------------------------------------------------------------

def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "shared":
        T, H, n_q = s["qn"].shape[0], case["heads"], case["n_q"]
        out = torch.zeros(T, H, LATENT, dtype=torch.float64, device="cuda")
        lse = torch.full((T, H), -math.inf, dtype=torch.float64, device="cuda")
        table, lens = s["table"].cpu().numpy(), s["lens"].cpu().numpy()
        rows = rows_of(s["slab"])
        for r in range(case["reqs"]):
            t = np.arange(lens[r])
            at = torch.as_tensor(table[r, t // PAGE].astype(np.int64) * PAGE + t % PAGE,
                                 device="cuda")
            x = rows[at]
            x = (x.view(E4M3) if case["type"] == "e4m3" else x).double()
            x = x * KV_SCALE if case["type"] == "e4m3" else x
            for j in range(n_q):
                seen = int(lens[r]) - (n_q - 1 - j)
                if seen <= 0:
                    continue
                i = r * n_q + j
                a = SCALE * (s["qn"][i].double() @ x[:seen, :LATENT].T
                             + s["qr"][i].double() @ x[:seen, LATENT:].T)
                lse[i] = torch.logsumexp(a, 1)
                y = torch.exp(a - lse[i][:, None]) @ x[:seen, :LATENT]
                out[i] = y * torch.sigmoid(s["gate"][i].double())
        return out, lse
    if op == "beams":
        B, K, V = case["batch"], case["beams"], case["vocab"]
        score = s["scores"].double()
        tokens, parents = np.zeros((B, K), np.int32), np.zeros((B, K), np.int32)
        values = np.zeros((B, K))
        for b in range(B):
            lp = torch.log_softmax(s["logits"][b * K:(b + 1) * K].double(), 1)
            cand = score[b][:, None] + lp
            if s["ended"] is not None:
                for k in range(K):
                    if bool(s["ended"][b, k]):
                        cand[k] = -math.inf
                        cand[k, s["end"]] = score[b, k]
            flat = cand.reshape(-1)
            least = flat.topk(K).values[-1]
            above = (flat > least).nonzero()[:, 0].cpu().numpy()
            tied = (flat == least).nonzero()[:K, 0].cpu().numpy()
            v = flat.cpu().numpy()
            above = above[np.argsort(-v[above], kind="stable")]
            pick = np.concatenate([above, tied])[:K]
            tokens[b], parents[b], values[b] = pick % V, b * K + pick // V, v[pick]
        return torch.as_tensor(tokens), torch.as_tensor(parents), torch.as_tensor(values)
    table, lens = s["table"].cpu().numpy(), s["lens"].cpu().numpy()
    out, counts = s["out_table"].cpu().numpy(), s["counts"].cpu().numpy()
    parents = s["parents"].cpu().numpy()
    new_lens = np.zeros(case["rows"], np.int32)
    for r, p in enumerate(parents):
        if p >= 0:
            new_lens[r] = lens[p]
            for c in range(-(-int(lens[p]) // PAGE)):
                out[r, c] = table[p, c]
                counts[table[p, c]] += 1
    if op == "fork":
        return torch.as_tensor(out), torch.as_tensor(new_lens), torch.as_tensor(counts)
    slabs = [x.clone() for x in s["slabs"]]
    free = [p for p in range(case["pool"]) if counts[p] == 0]
    for r in range(case["rows"]):
        n = int(new_lens[r])
        full, part = n // PAGE, n % PAGE
        if part and counts[out[r, full]] > 1:
            old, page = int(out[r, full]), free.pop(0)
            counts[old] -= 1
            counts[page] += 1
            out[r, full] = page
            for x in slabs:
                y = rows_of(x)
                y[page * PAGE:page * PAGE + part] = y[old * PAGE:old * PAGE + part]
        for c in range(-(-n // PAGE), -(-(n + case["new"]) // PAGE)):
            out[r, c] = free.pop(0)
            counts[out[r, c]] += 1
        new_lens[r] = n + case["new"]
    return torch.as_tensor(out), torch.as_tensor(new_lens), torch.as_tensor(counts), slabs
