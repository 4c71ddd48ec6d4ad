"""Measured cases of the cache-budget operators: rotary positions, the rotating KV
append, accumulated attention mass, eviction selection and page compaction.

``run`` computes each operator in its plain form (elementary torch operations in
fp32, rounded once at the end) or, with ``own``, through the package's entry
points.  ``exact`` gives the same outputs from the definitions in 64 bits.
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
        # the smallest step: two requests' queries of 16 heads, latency only
        {"name": "rope queries tiny", "op": "rope", "tokens": 2, "heads": 16, "dim": 64,
         "head_dim": 192, "type": "bf16", "layout": "half", "inverse": False, "base": 10000.0,
         "factor": 1.0, "original": 0, "far": 2000},
        # the gradient of a long chunk's queries back through a scaled rotation
        {"name": "rope back fp32", "op": "rope", "tokens": 8192, "heads": 64, "dim": 64,
         "head_dim": 64, "type": "fp32", "layout": "interleaved", "inverse": True,
         "base": 50000.0, "factor": 32.0, "original": 4096, "far": 1000000},
        # the step before a 4-draft verification: 128 requests, FP8 cache
        {"name": "append rope verify e4m3", "op": "append", "reqs": 128, "new": 4, "heads": 64,
         "type": "e4m3", "layout": "half", "lo": 1000, "hi": 4600, "lens_seed": 3,
         "base": 10000.0, "factor": 1.0, "original": 0, "shift": 0},
        # chunks of new tokens of four evicted histories (positions beyond the rows)
        {"name": "append rope chunk bf16", "op": "append", "reqs": 4, "new": 2047, "heads": 64,
         "type": "bf16", "layout": "interleaved", "lo": 4000, "hi": 20000, "lens_seed": 5,
         "base": 50000.0, "factor": 32.0, "original": 4096, "shift": 700001},
        # the smallest decode step's mass (two requests, 16 heads)
        {"name": "mass tiny bf16", "op": "mass", "reqs": 2, "n_q": 1, "heads": 16, "type": "bf16",
         "lo": 1000, "hi": 2000, "lens_seed": 0, "decay": 1.0},
        # a steady serving batch: 64 requests of 8k to 32k tokens
        {"name": "mass steady bf16", "op": "mass", "reqs": 64, "n_q": 1, "heads": 64,
         "type": "bf16", "lo": 8192, "hi": 32768, "lens_seed": 1, "decay": 1.0},
        # a 4-draft verification over the FP8 cache
        {"name": "mass verify e4m3", "op": "mass", "reqs": 32, "n_q": 4, "heads": 64,
         "type": "e4m3", "lo": 4096, "hi": 65536, "lens_seed": 3, "decay": 0.96875},
        # the observation window at the end of two long prompts: 32 queries each
        {"name": "mass window bf16", "op": "mass", "reqs": 2, "n_q": 32, "heads": 64,
         "type": "bf16", "lo": 60001, "hi": 131072, "lens_seed": 7, "decay": 0.0},
        # two short histories cut to 512 tokens, latency only
        {"name": "select tiny", "op": "select", "reqs": 2, "lo": 1000, "hi": 2000, "lens_seed": 0,
         "keep": 512, "sink": 4, "recent": 64},
        # million-token histories cut to an eighth
        {"name": "select long", "op": "select", "reqs": 4, "lo": 1000000, "hi": 1000000,
         "lens_seed": 4, "keep": 131072, "sink": 4, "recent": 1024},
        # four layers of an FP8 cache cut to 4k tokens a request
        {"name": "compact layers e4m3", "op": "compact", "reqs": 8, "layers": 4, "type": "e4m3",
         "lo": 9000, "hi": 40000, "lens_seed": 8, "keep": 4096},
        # a batch of long histories cut to 16k tokens a request
        {"name": "compact batch bf16", "op": "compact", "reqs": 32, "layers": 1, "type": "bf16",
         "lo": 20000, "hi": 60000, "lens_seed": 2, "keep": 16384},
    ]


def draw(rng):
    def log(lo, hi):
        return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))

    op = rng.choice(["rope", "append", "mass", "mass", "select", "compact"])
    scaled = rng.random() < 0.5
    turn = {"base": rng.choice([10000.0, 50000.0, 1000000.0]),
            "factor": rng.uniform(2.0, 40.0) if scaled else 1.0,
            "original": rng.choice([4096, 8192, 32768]) if scaled else 0,
            "layout": rng.choice(["half", "interleaved"])}
    seed = rng.randrange(1 << 20)
    if op == "rope":
        dim = rng.choice([16, 32, 64, 64, 64, 128, 20])
        heads = log(1, 128)
        return {"op": op, "tokens": log(1, max(1, 33554432 // (heads * dim))), "heads": heads,
                "dim": dim, "head_dim": dim + rng.choice([0, 128, 128, 6]),
                "type": rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                "inverse": rng.random() < 0.4, "far": log(100, 4000000), **turn}
    if op == "append":
        new = log(1, 2048)
        reqs = log(1, max(1, min(128, 8192 // new)))
        lo = new + log(1, 3000)
        return {"op": op, "reqs": reqs, "new": new, "heads": log(1, 128),
                "type": rng.choice(["bf16", "e4m3"]), "lo": lo, "hi": lo + log(1, 3000),
                "lens_seed": seed, "shift": rng.choice([0, log(1, 900000)]), **turn}
    if op == "mass":
        n_q = rng.choice([1, 1, 1, 2, 3, 4, 4, 8, 17, 32])
        heads = rng.choice([16, 32, 48, 64, 64, 64, 112, 128])
        tokens = min(1200000, 250000000 // (n_q * heads))
        reqs = log(1, 64)
        hi = log(30, max(31, tokens // reqs))
        return {"op": op, "reqs": reqs, "n_q": n_q, "heads": heads,
                "type": rng.choice(["bf16", "bf16", "e4m3"]),
                "lo": 0 if rng.random() < 0.3 else max(1, hi // 4), "hi": hi, "lens_seed": seed,
                "decay": rng.choice([0.0, 1.0, 0.875])}
    if op == "select":
        reqs = log(1, 64)
        hi = log(60, 4000000 // reqs)
        keep = log(30, hi)
        sink, recent = rng.randint(0, min(keep // 4, 64)), rng.randint(0, keep // 2)
        return {"op": op, "reqs": reqs, "lo": rng.choice([0, hi // 3]), "hi": hi,
                "lens_seed": seed, "keep": keep, "sink": sink, "recent": recent}
    reqs, layers = log(1, 32), rng.choice([1, 1, 2, 4])
    hi = log(100, 1200000 // (reqs * layers))
    return {"op": op, "reqs": reqs, "layers": layers, "type": rng.choice(["bf16", "e4m3"]),
            "lo": max(1, hi // 3), "hi": hi, "lens_seed": seed,
            "keep": log(1, max(1, min(hi, 500000 // (reqs * layers))))}


def lengths(case):
    rng = np.random.default_rng(case["lens_seed"])
    return rng.integers(case["lo"], case["hi"] + 1, case["reqs"]).astype(np.int64)


def work(case):
    op = case["op"]
    if op == "rope":
        n = case["tokens"] * case["heads"] * case["dim"]
        return {"bytes": 2 * n * BYTES[case["type"]] + 4 * case["tokens"], "flops": 3 * n}
    L = lengths(case)
    if op == "append":
        rows = case["reqs"] * case["new"]
        q = rows * case["heads"] * ROPE
        return {"bytes": rows * ROW * (2 + BYTES[case["type"]]) + 4 * q + 4 * rows,
                "flops": 3 * (q + rows * ROPE)}
    if op == "mass":
        rows = case["n_q"] * case["heads"]
        tokens = int(L.sum())
        rw = 4 if case["decay"] == 0.0 else 8
        return {"bytes": tokens * (ROW * BYTES[case["type"]] + rw)
                + case["reqs"] * rows * (2 * ROW + 4),
                "flops": 2 * ROW * rows * tokens}
    kept = int(np.minimum(L, case["keep"]).sum())
    if op == "select":
        return {"bytes": 4 * int(L.sum()) + 4 * kept, "flops": int(L.sum())}
    return {"bytes": kept * (2 * case["layers"] * ROW * BYTES[case["type"]] + 12), "flops": 0}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def rope_freqs(case, dim):
    """Radians per position of each pair, with the by-parts scaling of long contexts."""
    f = case["base"] ** (-2.0 * torch.arange(dim // 2, dtype=torch.float64) / dim)
    if case["factor"] != 1.0:
        turns = case["original"] * f / (2.0 * math.pi)
        g = ((turns - 1.0) / 31.0).clamp(0.0, 1.0)
        f = (1.0 - g) * f / case["factor"] + g * f
    return f


def rope_handle(case, dim):
    import paged_latent_attention_gb300 as plmla
    if case["factor"] == 1.0:
        return plmla.rope_table(dim, base=case["base"])
    return plmla.rope_table(dim, base=case["base"], scaling="by_parts", factor=case["factor"],
                            original_len=case["original"], low=1.0, high=32.0, magnitude=1.0)


def pages_of(case, L, spare=2):
    """A page table that scatters the histories' pages over the pool."""
    need = -(-L // PAGE)
    pool = int(need.sum()) + spare
    perm = np.random.default_rng(case["lens_seed"] + 1).permutation(pool).astype(np.int32)
    table = np.zeros((len(L), max(1, int(need.max()))), dtype=np.int32)
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = perm[at:at + n]
        at += n
    return table, pool


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.empty(*shape, dtype=dtype, device=dev).normal_(generator=g)

    def slab(pool):
        s = normal(pool, PAGE * ROW)
        return (s.float() / KV_SCALE).clamp(-448, 448).to(E4M3) if case["type"] == "e4m3" else s

    def ints(a):
        return torch.as_tensor(np.ascontiguousarray(a), dtype=torch.int32, device=dev)

    op = case["op"]
    s = {"case": case, "op": op}
    if op == "rope":
        full = normal(case["tokens"], case["heads"], case["head_dim"], dtype=TYPES[case["type"]])
        s["x"] = full[..., case["head_dim"] - case["dim"]:]
        s["positions"] = torch.randint(0, case["far"], (case["tokens"],), generator=g, device=dev,
                                       dtype=torch.int32)
        s["freqs"] = rope_freqs(case, case["dim"]).to(dev)
        if own:
            s["table"] = rope_handle(case, case["dim"])
        return s
    L = lengths(case)
    if op == "append":
        table, pool = pages_of(case, L)
        rows = case["reqs"] * case["new"]
        s["latent"], s["rope"] = normal(rows, LATENT), normal(rows, ROPE)
        s["q"] = normal(rows, case["heads"], 192)[..., 128:]
        s["slab"] = torch.zeros(pool, PAGE * ROW, device=dev,
                                dtype=torch.uint8 if case["type"] == "e4m3" else torch.bfloat16)
        s["slab"] = s["slab"].view(E4M3) if case["type"] == "e4m3" else s["slab"]
        s["page_table"], s["lens"] = ints(table), ints(L)
        at = L[:, None] - case["new"] + np.arange(case["new"])[None] + case["shift"]
        s["positions"] = ints(at.reshape(-1))
        s["freqs"] = rope_freqs(case, ROPE).to(dev)
        if own:
            s["table"] = rope_handle(case, ROPE)
        return s
    R, top = case["reqs"], max(1, int(L.max()))
    s["lens"], s["top"] = ints(L), top
    if op == "select":
        # weights as they accumulate: a few heavy tokens over a long light tail
        s["mass"] = torch.empty(R, top, device=dev).exponential_(generator=g).pow_(3.0)
        s["kept"] = torch.full((R, case["keep"]), -1, dtype=torch.int32, device=dev)
        s["kept_lens"] = torch.zeros(R, dtype=torch.int32, device=dev)
        return s
    s["mass"] = torch.rand(R, top, generator=g, device=dev)
    if op == "mass":
        table, pool = pages_of(case, L)
        rows = case["n_q"] * case["heads"]
        s["page_table"], s["slab"] = ints(table), slab(pool)
        s["mass"] *= rows / top     # of the size of one step's weights
        s["qn"] = normal(R * case["n_q"], case["heads"], LATENT)
        s["qr"] = normal(R * case["n_q"], case["heads"], ROPE)
        # the log-sum-exps that the decode of this step returned
        s["lse"] = torch.zeros(R * case["n_q"], case["heads"], device=dev)
        score, seen = plain_scores(s)
        score = torch.where(seen, score, -math.inf)
        s["lse"] = torch.logsumexp(score, 1).reshape(-1, case["heads"]).contiguous()
        if own and case["type"] == "e4m3":
            import paged_latent_attention_gb300 as plmla
            s["workspace"] = plmla.allocate_mass_workspace(R, case["n_q"], case["heads"])
        return s
    # compact: source pages first, the fresh pages behind them
    table, pool = pages_of(case, L, 0)
    n = np.minimum(L, case["keep"])
    s["fresh"], fresh = pool, -(-n // PAGE)
    out = np.zeros((R, int(fresh.max())), dtype=np.int32)
    perm = pool + np.random.default_rng(case["lens_seed"] + 2).permutation(int(fresh.sum()))
    at = 0
    for r, k in enumerate(fresh):
        out[r, :k] = perm[at:at + k]
        at += k
    s["page_table"], s["out_table"], s["kept_lens"] = ints(table), ints(out), ints(n)
    s["slabs"] = [slab(pool + int(fresh.sum())) for _ in range(case["layers"])]
    weight = torch.rand(R, top, generator=g, device=dev)
    weight = torch.where(torch.arange(top, device=dev)[None] < s["lens"][:, None], weight, -1.0)
    best = weight.topk(min(case["keep"], top), 1).indices
    inside = torch.arange(best.shape[1], device=dev)[None] < s["kept_lens"][:, None]
    best = torch.where(inside, best, 1 << 30).sort(1).values
    s["kept"] = torch.where(inside, best, 0).to(torch.int32)
    s["mass_out"] = torch.zeros(R, best.shape[1], device=dev)
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def run(state):
    op = state["op"]
    if own:
        return {"rope": own_rope, "append": own_append, "mass": own_mass, "select": own_select,
                "compact": own_compact}[op](state)
    return {"rope": plain_rope, "append": plain_append, "mass": plain_mass,
            "select": plain_select, "compact": plain_compact}[op](state)


def own_rope(s):
    import paged_latent_attention_gb300 as plmla
    return plmla.mla_rope(s["x"], s["positions"], s["table"], layout=s["case"]["layout"],
                          inverse=s["case"]["inverse"])


def own_append(s):
    import paged_latent_attention_gb300 as plmla
    c = s["case"]
    args = (s["latent"], s["rope"], s["slab"], s["page_table"], s["lens"], c["new"], s["table"])
    more = {"positions": s["positions"], "layout": c["layout"], "q_rope": s["q"]}
    if c["type"] == "e4m3":
        q = plmla.mla_kv_append_rope_fp8(*args, kv_scale=KV_SCALE, **more)
    else:
        q = plmla.mla_kv_append_rope(*args, **more)
    return q, s["slab"]


def own_mass(s):
    import paged_latent_attention_gb300 as plmla
    c = s["case"]
    args = (s["qn"], s["qr"], s["lse"], s["slab"], s["page_table"], s["lens"], s["mass"])
    if c["type"] == "e4m3":
        return plmla.mla_attention_mass_fp8(*args, kv_scale=KV_SCALE, n_q=c["n_q"],
                                            decay=c["decay"], workspace=s["workspace"])
    return plmla.mla_attention_mass(*args, n_q=c["n_q"], decay=c["decay"])


def own_select(s):
    import paged_latent_attention_gb300 as plmla
    c = s["case"]
    return plmla.mla_evict_select(s["mass"], s["lens"], c["keep"], sink=c["sink"],
                                  recent=c["recent"], kept=s["kept"], kept_lens=s["kept_lens"])


def own_compact(s):
    import paged_latent_attention_gb300 as plmla
    plmla.mla_kv_compact(s["slabs"], s["page_table"], s["lens"], s["out_table"], s["kept"],
                         s["kept_lens"], mass=s["mass"], mass_out=s["mass_out"])
    return [x[s["fresh"]:] for x in s["slabs"]], s["mass_out"]


def rotate(x, angle, layout):
    """x [T, H, D] in fp32 rotated by angle [T, D / 2] (64 bits)."""
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    if layout == "half":
        a, b = x.float().chunk(2, -1)
        return torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    a, b = x[..., 0::2].float(), x[..., 1::2].float()
    return torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)


def plain_rope(s):
    c = s["case"]
    angle = s["positions"].double()[:, None] * s["freqs"][None]
    return rotate(s["x"], -angle if c["inverse"] else angle, c["layout"]).to(s["x"].dtype)


def plain_append(s):
    c = s["case"]
    angle = s["positions"].double()[:, None] * s["freqs"][None]
    rope = rotate(s["rope"][:, None], angle, c["layout"])[:, 0]
    rows = torch.cat([s["latent"].float(), rope], 1)
    at = s["lens"][:, None].long() - c["new"] + torch.arange(c["new"], device=rows.device)[None]
    page = s["page_table"].long().gather(1, at // PAGE).reshape(-1)
    if c["type"] == "e4m3":
        codes = (rows / KV_SCALE).clamp(-448.0, 448.0).to(E4M3).view(torch.uint8)
        s["slab"].view(torch.uint8).view(-1, PAGE, ROW)[page, (at % PAGE).reshape(-1)] = codes
    else:
        s["slab"].view(-1, PAGE, ROW)[page, (at % PAGE).reshape(-1)] = rows.to(torch.bfloat16)
    return rotate(s["q"], angle, c["layout"]).to(torch.bfloat16), s["slab"]


def plain_scores(s):
    """Scaled scores [R, tokens, rows] in fp32 and which of them are visible."""
    c, top, R = s["case"], s["top"], s["lens"].shape[0]
    if c["type"] == "e4m3":
        k = s["slab"].view(torch.uint8)[s["page_table"].long()].view(E4M3).float() * KV_SCALE
    else:
        k = s["slab"][s["page_table"].long()].float()
    k = k.view(R, -1, ROW)[:, :top]
    q = torch.cat([s["qn"], s["qr"]], -1).float().view(R, c["n_q"] * c["heads"], ROW)
    score = torch.bmm(k, q.transpose(1, 2)) * SCALE
    behind = c["n_q"] - 1 - torch.arange(c["n_q"], device=k.device).repeat_interleave(c["heads"])
    seen = torch.arange(top, device=k.device)[None, :, None] < \
        s["lens"].long()[:, None, None] - behind[None, None]
    return score, seen


def plain_mass(s):
    c, top, R = s["case"], s["top"], s["lens"].shape[0]
    score, seen = plain_scores(s)
    weight = torch.where(seen, torch.exp(score - s["lse"].view(R, 1, -1)), 0.0).sum(2)
    new = weight if c["decay"] == 0.0 else c["decay"] * s["mass"] + weight
    inside = torch.arange(top, device=new.device)[None] < s["lens"][:, None]
    s["mass"].copy_(torch.where(inside, new, s["mass"]))
    return s["mass"]


def plain_select(s):
    c, top = s["case"], s["top"]
    t = torch.arange(top, device=s["mass"].device)[None]
    L = s["lens"].long()[:, None]
    rank = torch.where((t < c["sink"]) | (t >= L - c["recent"]), math.inf, s["mass"])
    order = torch.where(t < L, rank, -math.inf).sort(dim=1, descending=True, stable=True).indices
    n = L.clamp(max=c["keep"])
    i = torch.arange(min(c["keep"], top), device=t.device)[None]
    best = torch.where(i < n, order[:, :c["keep"]], top).sort(1).values
    s["kept"][:, :i.shape[1]] = torch.where(i < n, best, s["kept"][:, :i.shape[1]].long()).int()
    s["kept_lens"].copy_(n[:, 0])
    return s["kept"], s["kept_lens"]


def plain_compact(s):
    kept, n = s["kept"].long(), s["kept_lens"][:, None]
    i = torch.arange(kept.shape[1], device=kept.device)[None].expand_as(kept)
    inside = i < n
    src = s["page_table"].long().gather(1, kept // PAGE) * PAGE + kept % PAGE
    dst = s["out_table"].long().gather(1, i // PAGE) * PAGE + i % PAGE
    # rows past a request's count copy its row 0 onto itself (every request has one)
    src = torch.where(inside, src, src[:, :1]).reshape(-1)
    dst = torch.where(inside, dst, dst[:, :1]).reshape(-1)
    [rows_of(x).index_copy_(0, dst, rows_of(x)[src]) for x in s["slabs"]]
    s["mass_out"].copy_(torch.where(inside, s["mass"].gather(1, kept), s["mass_out"]))
    return [x[s["fresh"]:] for x in s["slabs"]], s["mass_out"]


def rows_of(slab):
    return (slab.view(torch.uint8) if slab.dtype == E4M3 else slab).view(-1, ROW)


# --------------------------------------------------------------------------
# 64 bits
# --------------------------------------------------------------------------

def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "select":
        mass, kept = s["mass"].cpu().double().numpy(), s["kept"].cpu().numpy()
        L = lengths(case)
        for r, n in enumerate(L):
            lo, hi = min(case["sink"], n), max(min(case["sink"], n), n - case["recent"])
            rest = max(0, min(case["keep"], n) - lo - (n - hi))
            best = lo + np.argsort(-mass[r, lo:hi], kind="stable")[:rest]
            mine = np.concatenate([np.arange(lo), np.sort(best), np.arange(hi, n)])
            kept[r, :len(mine)] = mine
        return (torch.as_tensor(kept),
                torch.as_tensor(np.minimum(L, case["keep"]).astype(np.int32)))
    if op in ("rope", "append"):
        def turn(x, back):
            z = torch.polar(torch.ones_like(s["freqs"])[None],
                            s["positions"].double()[:, None] * s["freqs"][None])
            z = (z.conj() if back else z)[:, None]
            x = x.double()
            if case["layout"] == "half":
                y = torch.complex(x[..., :x.shape[-1] // 2], x[..., x.shape[-1] // 2:]) * z
                return torch.cat([y.real, y.imag], -1)
            y = torch.view_as_complex(x.reshape(*x.shape[:-1], -1, 2).contiguous()) * z
            return torch.view_as_real(y).flatten(-2)

        if op == "rope":
            return turn(s["x"], case["inverse"])
        rope = turn(s["rope"][:, None], False)[:, 0]
        pool = torch.zeros(s["slab"].shape, dtype=torch.float64, device=rope.device)
        pool = pool.view(-1, PAGE, ROW)
        table, new = s["page_table"].cpu().numpy(), case["new"]
        unit = KV_SCALE if case["type"] == "e4m3" else 1.0
        for r, n in enumerate(lengths(case)):
            p = np.arange(n - new, n)
            pages = torch.as_tensor(table[r, p // PAGE].astype(np.int64), device=rope.device)
            at = torch.as_tensor(p % PAGE, device=rope.device)
            mine = slice(r * new, (r + 1) * new)
            pool[pages, at, :LATENT] = s["latent"][mine].double() / unit
            pool[pages, at, LATENT:] = rope[mine] / unit
        if case["type"] == "e4m3":
            pool.clamp_(-448.0, 448.0)
        return turn(s["q"], False), pool.view(s["slab"].shape)
    if op == "mass":
        out = s["mass"].double()
        table = s["page_table"].long()
        for r, n in enumerate(lengths(case)):
            n = int(n)
            k = s["slab"][table[r, :-(-n // PAGE)]] if case["type"] == "bf16" else \
                s["slab"].view(torch.uint8)[table[r, :-(-n // PAGE)]].view(E4M3)
            k = k.reshape(-1, ROW)[:n].double() * (KV_SCALE if case["type"] == "e4m3" else 1.0)
            total = torch.zeros(n, dtype=torch.float64, device=k.device)
            for j in range(case["n_q"]):
                at, seen = r * case["n_q"] + j, max(0, n - (case["n_q"] - 1 - j))
                q = torch.cat([s["qn"][at], s["qr"][at]], -1).double()
                p = torch.exp(SCALE * (k[:seen] @ q.T) - s["lse"][at].double()[None])
                total[:seen] += p.sum(1)
            if case["decay"] == 0.0:
                out[r, :n] = total
            else:
                out[r, :n] = case["decay"] * out[r, :n] + total
        return out
    outs = [x[s["fresh"]:].clone() for x in s["slabs"]]
    mass = torch.zeros_like(s["mass_out"])
    kept, n = s["kept"].cpu().numpy(), s["kept_lens"].cpu().numpy()
    src, dst = s["page_table"].cpu().numpy(), s["out_table"].cpu().numpy()
    for r in range(case["reqs"]):
        k, i = kept[r, :n[r]].astype(np.int64), np.arange(n[r])
        take = torch.as_tensor(src[r, k // PAGE].astype(np.int64) * PAGE + k % PAGE)
        put = torch.as_tensor((dst[r, i // PAGE].astype(np.int64) - s["fresh"]) * PAGE + i % PAGE)
        for x, y in zip(s["slabs"], outs):
            rows_of(y)[put.to(y.device)] = rows_of(x)[take.to(x.device)]
        mass[r, :n[r]] = s["mass"][r, torch.as_tensor(k).to(mass.device)]
    return outs, mass
