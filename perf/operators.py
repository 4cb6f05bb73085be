"""Cases, plain forms and exact values of the operators that follow a decode or
verification step: the verification of drafted tokens, the accumulation of the
attention weight of cache entries, and the eviction of entries by that weight.

Sizes: the batch sizes, context lengths, Top-k and candidate counts of this
repository's workloads (B = 64, L up to 2^20, k = 512, six candidates, a ragged
batch of 48, 4096-row pages) and generic vocabulary sizes, odd ones among them.
"""
import math

import torch

own = False

HEADS, DIM, CODE_B, SCALE_B, IDX_CODE_B, IDX_SCALE_B = 16, 512, 256, 16, 64, 4
SM_SCALE = 1.0 / math.sqrt(DIM)
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one interactive request, four drafts: the latency of one call
        {"name": "verify_b1_n5_v32000", "op": "verify", "B": 1, "n_lo": 5, "n_hi": 5, "V": 32000, "p": "f32", "q": "f32"},
        # the verification workload's batch (64 sequences, six candidates) over a large vocabulary
        {"name": "verify_b64_n6_v131072", "op": "verify", "B": 64, "n_lo": 6, "n_hi": 6, "V": 131072, "p": "f32", "q": "f32"},
        # a ragged batch (0 to 9 candidates), an odd vocabulary, half-width draft probabilities
        {"name": "verify_b48_ragged_v100003", "op": "verify", "B": 48, "n_lo": 0, "n_hi": 9, "V": 100003, "p": "f32", "q": "bf16"},
        # drafts without probabilities (greedy or looked up), half-width target, a large batch
        {"name": "verify_b256_n4_v50001_nodraft", "op": "verify", "B": 256, "n_lo": 4, "n_hi": 4, "V": 50001, "p": "f16", "q": "none"},
        # one request's layer: the latency of one call
        {"name": "weights_b1_k512", "op": "weights", "B": 1, "m": 1, "k": 512, "lo": 8192, "hi": 8192, "page": 0},
        # the decode batch: one query a sequence, Top-512 of 131072 entries
        {"name": "weights_b64_k512", "op": "weights", "B": 64, "m": 1, "k": 512, "lo": 131072, "hi": 131072, "page": 0},
        # the verification batch: six candidates a sequence, the accepted ones count, paged caches
        {"name": "weights_b64_m6_paged", "op": "weights", "B": 64, "m": 6, "k": 512, "lo": 4096, "hi": 65536, "page": 4096},
        # a ragged batch with long candidate lists and the widest selection (2048), short sequences that leave slots empty
        {"name": "weights_b48_m16_k2048", "op": "weights", "B": 48, "m": 16, "k": 2048, "lo": 1000, "hi": 100001, "page": 0},
        # one short request cut to half
        {"name": "evict_b1_l8192", "op": "evict", "B": 1, "lo": 8192, "hi": 8192, "keep": 0.5, "idx": True, "page": 0},
        # a ragged batch in pages, cut to a quarter
        {"name": "evict_b48_ragged_paged", "op": "evict", "B": 48, "lo": 600, "hi": 65536, "keep": 0.25, "idx": True, "page": 512},
        # main KV without an indexer cache (a layer that shares another's indexer), light trimming, odd lengths
        {"name": "evict_b16_l100001_main", "op": "evict", "B": 16, "lo": 100001, "hi": 100001, "keep": 0.9, "idx": False, "page": 0},
        # million-entry sequences cut to half
        {"name": "evict_b4_l1m", "op": "evict", "B": 4, "lo": 1048576, "hi": 1048576, "keep": 0.5, "idx": True, "page": 0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["verify", "weights", "evict"])
    if op == "verify":
        B = _log(rng, 1, 256)
        V = _log(rng, 1000, min(131072, 64 * 131072 // B))
        n_hi = rng.randint(1, max(1, min(16, 64 * 6 * 131072 // (B * V))))
        return {"op": op, "B": B, "n_lo": rng.randint(0, n_hi), "n_hi": n_hi, "V": V,
                "p": rng.choice(["f32", "bf16", "f16"]), "q": rng.choice(["f32", "bf16", "f16", "none"])}
    if op == "weights":
        B = _log(rng, 1, 64)
        m = _log(rng, 1, 16)
        k = min(_log(rng, 64, 2048), 48 * 16 * 2048 // (B * m))
        hi = _log(rng, 600, 131072)
        return {"op": op, "B": B, "m": m, "k": k, "lo": rng.randint(max(1, hi // 8), hi), "hi": hi,
                "page": rng.choice([0, 0, 512, 4096])}
    B = _log(rng, 1, 64)
    hi = _log(rng, 1000, min(1048576, 4 * 1048576 // B))
    return {"op": op, "B": B, "lo": rng.randint(max(1, hi // 8), hi), "hi": hi, "keep": round(rng.uniform(0.1, 0.95), 3),
            "idx": rng.random() < 0.7, "page": rng.choice([0, 0, 512, 4096])}


def _lengths(c):
    """Sequence lengths from lo to hi, evenly spaced on a log scale."""
    B, lo, hi = c["B"], c["lo"], c["hi"]
    return [hi if B == 1 else int(round(lo * (hi / lo) ** (b / (B - 1)))) for b in range(B)]


def _counts(c):
    """Candidates of each sequence (the first is the last known token)."""
    lo, hi = c["n_lo"], c["n_hi"]
    return [lo + (7 * b) % (hi - lo + 1) for b in range(c["B"])]


def _keeps(c):
    return [max(1, int(n * c["keep"])) for n in _lengths(c)]


def _accepted(c):
    """Accepted drafts of each sequence of a weights case (m candidates each)."""
    return [(5 * b + 2) % c["m"] if c["m"] > 1 else 0 for b in range(c["B"])]


FIRST, LAST = 4, 64  # entries that an eviction always keeps: a few first ones, the recent ones


def work(c):
    if c["op"] == "verify":
        # the stop row of every sequence: the target's, and the draft's where a draft was rejected
        # (drafts near the target's distribution: about 0.7 of them are accepted)
        size = {"f32": 4, "bf16": 2, "f16": 2, "none": 0}
        b = f = 0.0
        for n in _counts(c):
            if n:
                rejected = 1.0 - 0.7 ** (n - 1)
                b += c["V"] * (size[c["p"]] + size[c["q"]] * rejected) + 20 * n + 16
                f += 4 * c["V"]
        return {"bytes": max(b, 16.0), "flops": max(f, 1.0)}
    if c["op"] == "weights":
        b = f = 0.0
        for n, a in zip(_lengths(c), _accepted(c)):
            k = min(c["k"], n)
            b += (a + 1) * (k * (CODE_B + SCALE_B + 8) + HEADS * DIM * 2 + HEADS * 4) + 4 * c["m"] * c["k"]
            f += (a + 1) * k * HEADS * (2 * DIM + 2)
        return {"bytes": b, "flops": f}
    row = CODE_B + SCALE_B + 4 + (IDX_CODE_B + IDX_SCALE_B if c["idx"] else 0)
    b = sum(4 * L + n * (2 * row - 4 + 4) for L, n in zip(_lengths(c), _keeps(c)))
    return {"bytes": b, "flops": sum(_lengths(c))}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _layout(c, lens, page, g):
    """Where sequences lie: (row offsets or None, page table or None, cache rows)."""
    if not page:
        off, rows = [], 0
        for n in lens:
            off.append(rows)
            rows += (n + 7) // 8 * 8
        return torch.tensor(off, dtype=torch.int64, device="cuda"), None, max(rows, 8)
    need = [(n + page - 1) // page for n in lens]
    total = max(1, sum(need))
    perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros((len(lens), max(1, max(need))), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return None, table, total * page


def _bytes(shape, g):
    return torch.randint(0, 256, shape, dtype=torch.uint8, device="cuda", generator=g)


def _scales(shape, g):
    return torch.randint(125, 128, shape, dtype=torch.uint8, device="cuda", generator=g)


def prepare(c, seed):
    g = _gen(seed)
    if c["op"] == "verify":
        return _prepare_verify(c, g)
    if c["op"] == "weights":
        return _prepare_weights(c, g)
    return _prepare_evict(c, g)


def _prepare_verify(c, g):
    B, V, n = c["B"], c["V"], _counts(c)
    Q = max(1, sum(n))
    off = [0]
    for x in n:
        off.append(off[-1] + x)
    # a model's logits, and a draft model's that follow them
    z = torch.randn((Q, V), device="cuda", generator=g) * 2.5
    p = torch.softmax(z, dim=1)
    qd = torch.softmax(z + 0.5 * torch.randn((Q, V), device="cuda", generator=g), dim=1)
    s = {"c": c, "target": p.to(TYPES[c["p"]]), "draft": None, "q_off": _i32(off), "max_n": max(n),
         "u": torch.rand(Q, device="cuda", generator=g), "r": torch.rand(B, device="cuda", generator=g)}
    # candidate i+1 is drawn from row i of the draft (without one: the draft's likeliest token)
    if c["q"] == "none":
        drawn = qd.argmax(dim=1)
    else:
        s["draft"] = qd.to(TYPES[c["q"]])
        drawn = torch.multinomial(qd, 1, generator=g)[:, 0]
    s["tokens"] = torch.cat([drawn[:1], drawn[:-1]]).to(torch.int32)
    s["n_accept"] = torch.zeros(B, dtype=torch.int32, device="cuda")
    s["next"] = torch.zeros(B, dtype=torch.int32, device="cuda")
    s["out"] = torch.zeros((B, max(1, max(n))), dtype=torch.int32, device="cuda")
    if own:
        from long_context_decode_csa2_b200 import csa2 as C

        s["ws"] = C.workspace(C.csa2_verify_drafts_workspace_bytes(B, V))
    return s


def _prepare_weights(c, g):
    B, m, k, lens = c["B"], c["m"], c["k"], _lengths(c)
    off, pages, rows = _layout(c, lens, c["page"], g)
    Q = B * m
    # candidates of a sequence select mostly the same entries
    vis = torch.tensor(lens, dtype=torch.float64, device="cuda")[:, None, None]
    shared = torch.rand((B, 1, k), device="cuda", generator=g, dtype=torch.float64)
    each = torch.rand((B, m, k), device="cuda", generator=g, dtype=torch.float64)
    jit = torch.where(torch.rand((B, 1, k), device="cuda", generator=g) < 0.75, shared, each)
    j = torch.arange(k, dtype=torch.float64, device="cuda")
    spread = torch.floor((j + jit.clamp(max=0.999999)) * vis / k)
    ids = torch.where(vis >= k, spread, torch.where(j < vis, j.expand(B, m, k), -1.0)).to(torch.int32).reshape(Q, k)
    s = {"c": c, "q": (torch.randn((Q, HEADS, DIM), device="cuda", generator=g) * 0.5).to(torch.bfloat16),
         "codes": _bytes((rows, CODE_B), g), "scales": _scales((rows, SCALE_B), g), "off": off, "pages": pages,
         "seq_len": _i32(lens), "topk": ids.contiguous(), "q_off": _i32([b * m for b in range(B + 1)]),
         "n_accept": _i32(_accepted(c)), "acc": torch.rand(rows, device="cuda", generator=g) * 0.1,
         "weights": torch.zeros((Q, k), device="cuda")}
    # the attention's own log-sum-exp: the selected entries, and a window that takes a quarter of the mass
    x = _logits(s)
    s["lse"] = (torch.logsumexp(x.double(), dim=2) + math.log(4.0 / 3.0)).float().contiguous()
    if own:
        from long_context_decode_csa2_b200 import csa2 as C

        s["cache"] = C.cache(s["codes"], s["scales"])
        s["where"] = off if pages is None else C.PageTable(pages, c["page"])
        s["ws"] = C.workspace(C.csa2_attn_weights_workspace_bytes(B, Q, k))
    return s


def _prepare_evict(c, g):
    lens, keeps, page = _lengths(c), _keeps(c), c["page"]
    off, pages, rows = _layout(c, lens, page, g)
    doff, dpages, drows = _layout(c, keeps, page, g)
    # accumulated weights: most entries were never selected and stand at zero, a few carry the mass
    w = torch.rand(rows, device="cuda", generator=g)
    acc = torch.where(torch.rand(rows, device="cuda", generator=g) < 0.6, 0.0, w * w * w)
    z = lambda *shape: torch.zeros(shape, dtype=torch.uint8, device="cuda")  # noqa: E731
    s = {"c": c, "off": off, "pages": pages, "doff": doff, "dpages": dpages, "acc": acc, "seq_len": _i32(lens),
         "keep": _i32(keeps), "max_len": max(lens), "max_keep": max(keeps),
         "main": (_bytes((rows, CODE_B), g), _scales((rows, SCALE_B), g)), "dmain": (z(drows, CODE_B), z(drows, SCALE_B)),
         "idx": None, "didx": None, "dacc": torch.zeros(drows, device="cuda"),
         "kept": torch.zeros((c["B"], max(keeps)), dtype=torch.int32, device="cuda"),
         "len_out": torch.zeros(c["B"], dtype=torch.int32, device="cuda")}
    if c["idx"]:
        s["idx"] = (_bytes((rows, IDX_CODE_B), g), _scales((rows, IDX_SCALE_B), g))
        s["didx"] = (z(drows, IDX_CODE_B), z(drows, IDX_SCALE_B))
    if own:
        from long_context_decode_csa2_b200 import csa2 as C

        for name in ("main", "dmain", "idx", "didx"):
            s["c_" + name] = None if s[name] is None else C.cache(*s[name])
        s["src"] = off if pages is None else C.PageTable(pages, page)
        s["dst"] = doff if dpages is None else C.PageTable(dpages, page)
        s["ws"] = C.workspace(C.csa2_cache_evict_workspace_bytes(c["B"], max(lens)))
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    op = s["c"]["op"]
    if own:
        from long_context_decode_csa2_b200 import csa2 as C

        if op == "verify":
            C.csa2_verify_drafts(s["target"], s["tokens"], s["q_off"], s["u"], s["r"], s["n_accept"], s["next"], s["ws"],
                                 draft=s["draft"], out_tokens=s["out"])
            return {"n_accept": s["n_accept"], "next": s["next"], "out": s["out"]}
        if op == "weights":
            C.csa2_attn_weights(s["q"], s["cache"], s["where"], s["seq_len"], s["topk"], s["lse"], SM_SCALE, s["acc"],
                                s["ws"], q_off=s["q_off"], n_accept=s["n_accept"], weights=s["weights"])
            return {"acc": s["acc"], "weights": s["weights"]}
        C.csa2_cache_evict(s["c_main"], s["c_idx"], s["acc"], s["src"], s["seq_len"], s["keep"], s["max_len"],
                           s["max_keep"], s["c_dmain"], s["c_didx"], s["dacc"], s["dst"], s["kept"], s["len_out"], s["ws"],
                           first=FIRST, last=LAST)
        return _evict_outputs(s)
    return {"verify": _plain_verify, "weights": _plain_weights, "evict": _plain_evict}[op](s)


def _plain_verify(s):
    """accept candidate i+1 iff u_i q_i(x) < p_i(x); the first row that is not passed gives the next token from
    max(p - q, 0) (or from p behind the last candidate), by the running sum of its weights against r."""
    p, q, off, V = s["target"], s["draft"], s["q_off"].long(), s["target"].shape[1]
    B, M = off.numel() - 1, max(1, s["max_n"])
    n = off[1:] - off[:-1]
    i = torch.arange(M, device=p.device)
    row = (off[:-1, None] + i).clamp(max=p.shape[0] - 1)
    tok = s["tokens"].long()[(row + 1).clamp(max=p.shape[0] - 1)]
    px = p[row, tok].double()
    qx = q[row, tok].double() if q is not None else torch.ones_like(px)
    ok = (i < n[:, None] - 1) & (s["u"][row].double() * qx < px)
    a = ok.long().cumprod(1).sum(1)
    stop = row.gather(1, a[:, None].clamp(max=M - 1))[:, 0]
    rejected = a < n - 1
    w = p[stop].double()
    if q is not None:
        less = (w - q[stop].double()).clamp(min=0)
    else:
        j = torch.arange(V, device=p.device)
        drafted = tok.gather(1, a[:, None].clamp(max=M - 1))
        less = torch.where(j == drafted, (w - 1.0).clamp(min=0), w)
    less = torch.where(less.sum(1, keepdim=True) > 0, less, w)
    w = torch.where(rejected[:, None], less, w)
    run_ = w.cumsum(1)
    nxt = (run_ <= s["r"].double()[:, None] * run_[:, -1:]).sum(1)
    lastw = (w > 0).long().mul(torch.arange(1, V + 1, device=p.device)).amax(1) - 1
    nxt = torch.where(n > 0, torch.minimum(nxt, lastw), -1)
    a = torch.where(n > 0, a, 0)
    out = torch.where(i < a[:, None], tok, torch.where((i == a[:, None]) & (n[:, None] > 0), nxt[:, None], -1))
    return {"n_accept": a.int(), "next": nxt.int(), "out": out.int()}


def _rows(off, pages, page, pos):
    """Cache rows of positions pos [B, ...] (contiguous offsets, or a page table)."""
    flat = pos.reshape(pos.shape[0], -1).long()
    if pages is None:
        r = off[:, None] + flat
    else:
        r = pages.long().gather(1, flat // page) * page + flat % page
    return r.reshape(pos.shape)


def _logits(s):
    """Scaled logits of every candidate's selected entries (-inf where a slot is empty)."""
    c = s["c"]
    ids = s["topk"]
    rows = _rows(s["off"], s["pages"], c["page"], ids.clamp(min=0).view(c["B"], -1)).reshape(ids.shape)
    table = torch.tensor(E2M1, device=ids.device)
    out = torch.empty((ids.shape[0], HEADS, ids.shape[1]), device=ids.device)
    step = max(1, (1 << 19) // ids.shape[1])  # a gigabyte of dequantised rows at a time
    for i in range(0, ids.shape[0], step):
        r = rows[i:i + step]
        code = s["codes"][r].int()
        val = table[torch.stack([code & 15, code >> 4], dim=-1)].view(*r.shape, SCALE_B, 32)
        key = (val * torch.exp2(s["scales"][r].float() - 127.0)[..., None]).view(*r.shape, DIM)
        out[i:i + step] = torch.matmul(s["q"][i:i + step].float(), key.transpose(1, 2))
    return torch.where(ids[:, None, :] >= 0, out * SM_SCALE, -math.inf)


def _plain_weights(s):
    """weight of entry j under candidate i: sum over heads of exp(logit - lse); the accepted candidates' weights are added
    to their entries."""
    c = s["c"]
    rank = torch.arange(c["m"], device=s["q"].device)
    counts = (rank[None, :] <= s["n_accept"][:, None]).reshape(-1, 1)
    w = torch.exp(_logits(s) - s["lse"][:, :, None]).sum(1)
    w = torch.where(counts, w, 0.0)
    rows = _rows(s["off"], s["pages"], c["page"], s["topk"].clamp(min=0).view(c["B"], -1))
    s["acc"].index_add_(0, rows.reshape(-1), w.reshape(-1))
    return {"acc": s["acc"], "weights": w}


def _evict_outputs(s):
    out = {"kept": s["kept"], "len": s["len_out"], "acc": s["dacc"], "codes": s["dmain"][0], "scales": s["dmain"][1]}
    if s["didx"] is not None:
        out["idx_codes"], out["idx_scales"] = s["didx"]
    return out


def _plain_evict(s):
    """keeps the first FIRST and last LAST entries and, up to keep[b] in all, the best others by (weight desc, position asc)."""
    c, L, keep = s["c"], s["seq_len"].long()[:, None], s["keep"].long()[:, None]
    pos = torch.arange(s["max_len"], device=L.device).expand(c["B"], -1)
    rows = _rows(s["off"], s["pages"], c["page"], torch.minimum(pos, L - 1))
    n = torch.minimum(keep, L)
    last = torch.minimum(n, torch.full_like(n, LAST))
    first = torch.minimum(n - last, torch.full_like(n, FIRST))
    bits = s["acc"][rows].view(torch.int32).long()  # weights are not negative: their bits rise with them
    bits = torch.where((pos < first) | (pos >= L - last), 1 << 40, bits)
    bits = torch.where(pos < L, bits, -1)
    order = torch.sort(bits, dim=1, descending=True, stable=True).indices
    chosen = torch.zeros(pos.shape[0], pos.shape[1] + 1, dtype=torch.bool, device=L.device)
    chosen.scatter_(1, torch.where(pos < n, order, pos.shape[1]), True)
    chosen = chosen[:, :-1]
    at = torch.where(chosen, chosen.long().cumsum(1) - 1, s["max_keep"])
    kept = torch.full((pos.shape[0], s["max_keep"] + 1), -1, dtype=torch.long, device=L.device)
    kept.scatter_(1, at, pos.expand_as(at))
    kept = kept[:, :-1].contiguous()
    s["kept"].copy_(kept)
    s["len_out"].copy_(n[:, 0])
    # slots past a sequence's last kept entry repeat that entry
    j = torch.minimum(torch.arange(s["max_keep"], device=L.device)[None, :], n - 1)
    src = _rows(s["off"], s["pages"], c["page"], kept.gather(1, j)).reshape(-1)
    dst = _rows(s["doff"], s["dpages"], c["page"], j).reshape(-1)
    s["dacc"][dst] = s["acc"][src]
    for a, b in ((s["main"], s["dmain"]), (s["idx"], s["didx"])):
        if a is not None:
            b[0][dst] = a[0][src]
            b[1][dst] = a[1][src]
    return _evict_outputs(s)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "verify":
        return None  # whole numbers only
    if c["op"] == "weights":
        return _exact_weights(s)
    return _exact_evict(s)


def _place(s, off, pages, b, pos):
    page = s["c"]["page"]
    return int(off[b]) + pos if pages is None else pages[b].long()[pos // page] * page + pos % page


def _exact_weights(s):
    """One candidate after the other, every value in 64 bits."""
    acc = s["acc"].double()
    w = torch.zeros(s["topk"].shape, dtype=torch.float64, device=acc.device)
    q_off, n_acc = s["q_off"].tolist(), s["n_accept"].tolist()
    for b in range(len(n_acc)):
        for i in range(q_off[b], q_off[b] + n_acc[b] + 1):
            slot = (s["topk"][i] >= 0).nonzero()[:, 0]
            row = _place(s, s["off"], s["pages"], b, s["topk"][i][slot].long())
            byte = s["codes"][row].long()
            code = torch.empty((len(row), DIM), dtype=torch.int64, device=acc.device)
            code[:, 0::2], code[:, 1::2] = byte % 16, byte // 16
            mag = code % 8
            e, f = mag // 2, mag % 2
            val = torch.where(e == 0, f * 0.5, torch.exp2(e.double() - 1) * (1 + f * 0.5))
            val = torch.where(code >= 8, -val, val) * torch.exp2(s["scales"][row].double() - 127).repeat_interleave(32, dim=1)
            x = (s["q"][i].double() @ val.T) * SM_SCALE - s["lse"][i].double()[:, None]
            w[i, slot] = x.exp().sum(0)
            acc.index_add_(0, row, w[i, slot])
    return {"acc": acc, "weights": w}


def _exact_evict(s):
    """One sequence after the other; the rows themselves are copies."""
    c, dev = s["c"], s["acc"].device
    dacc = torch.zeros(s["dacc"].shape, dtype=torch.float64, device=dev)
    for b, (L, n) in enumerate(zip(_lengths(c), _keeps(c))):
        n = min(n, L)
        last = min(LAST, n)
        first = min(FIRST, n - last)
        a = s["acc"][_place(s, s["off"], s["pages"], b, torch.arange(L, device=dev))].double()
        mid = a[first:L - last]
        best = torch.sort(-mid, stable=True).indices[:n - first - last] + first
        pos = torch.cat([torch.arange(first, device=dev), best.sort().values, torch.arange(L - last, L, device=dev)])
        dacc[_place(s, s["doff"], s["dpages"], b, torch.arange(n, device=dev))] = a[pos]
    return {"acc": dacc, "kept": None, "len": None, "codes": None, "scales": None}
