"""Dense attention over the paged FP4 main KV, and the pages' own operations: what is measured.

Cases come in four kinds:
  decode   one query token per sequence (16 heads sharing one K and one V) over all of its entries
  prefill  chunks of query tokens over their sequence's entries: causal at ratio 1 or 2, or, with
           `cross`, every entry for every query (a decoder's queries over an encoder's states)
  beam     one step of a beam search: every surviving hypothesis is forked into a free row of the
           page table (full pages shared, the partly filled last page copied), then the old rows are freed
  compact  live pages moved into the holes below them, page table and reference counts rewritten

An entry is 256 channels (K, then V): 128 bytes of E2M1 codes, channel 2j in the low nibble of byte j,
and 16 E4M3 scales, one per 16 channels.
"""
import math
import random

import torch

own = False

H, D = 16, 128
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------

def listed():
    return [
        # one user at a 4K context: latency only
        {"name": "decode 1 x 4095", "kind": "decode", "seqs": 1, "lo": 4095, "hi": 4095, "page": 64, "f32": False},
        # a serving batch of ragged sequences
        {"name": "decode 64 ragged", "kind": "decode", "seqs": 64, "lo": 509, "hi": 32768, "page": 64, "f32": False},
        # eight long sequences: the cache streamed once per token
        {"name": "decode 8 x 262144", "kind": "decode", "seqs": 8, "lo": 262144, "hi": 262144, "page": 64, "f32": False},
        # a 1M context whose fp32 partial result is merged with other shards' by log-sum-exp
        {"name": "decode 1 x 1048573 fp32", "kind": "decode", "seqs": 1, "lo": 1048573, "hi": 1048573, "page": 64,
         "f32": True},
        # eight sequences checking a draft of five tokens
        {"name": "draft 8 x 5 over 65536", "kind": "prefill", "seqs": 8, "qlo": 5, "qhi": 5, "lo": 65536, "hi": 65536,
         "ratio": 1, "cross": False, "page": 64, "f32": False},
        # the last 4096 tokens of a 32K prompt at ratio 2
        {"name": "prefill 4096 of 32768", "kind": "prefill", "seqs": 1, "qlo": 4096, "qhi": 4096, "lo": 16384,
         "hi": 16384, "ratio": 2, "cross": False, "page": 64, "f32": False},
        # ragged whole prompts, odd lengths, small pages, fp32 results
        {"name": "prefill ragged prompts", "kind": "prefill", "seqs": 6, "qlo": 37, "qhi": 2001, "lo": 37, "hi": 2001,
         "ratio": 1, "cross": False, "page": 16, "f32": True},
        # decoder tokens over their encoder's states
        {"name": "cross 8 x 257", "kind": "prefill", "seqs": 8, "qlo": 129, "qhi": 257, "lo": 4099, "hi": 16384,
         "ratio": 2, "cross": True, "page": 64, "f32": False},
        # a beam search of four hypotheses for four requests, one cache
        {"name": "beam 4 x 4", "kind": "beam", "groups": 4, "width": 4, "lo": 200, "hi": 1001, "caches": 1, "page": 64},
        # the same over a full server: the encoder's three caches
        {"name": "beam 32 x 8, 3 caches", "kind": "beam", "groups": 32, "width": 8, "lo": 1500, "hi": 8191, "caches": 3,
         "page": 64},
        # a small pool after a few requests left
        {"name": "compact 255 pages", "kind": "compact", "pages": 255, "seqs": 7, "live": 0.6, "caches": 1, "page": 64},
        # a large pool, two thirds in use
        {"name": "compact 12000 pages", "kind": "compact", "pages": 12000, "seqs": 64, "live": 0.66, "caches": 1,
         "page": 64},
    ]


def _log(rng, lo, hi):
    return int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))


def draw(rng):
    kind = rng.choice(["decode", "decode", "prefill", "prefill", "prefill", "beam", "compact"])
    page = rng.choice([8, 16, 32, 64, 64, 128, 256])
    if kind == "decode":
        seqs = _log(rng, 1, 96)
        hi = _log(rng, 1, min(1 << 20, (1 << 21) // seqs))
        return {"kind": kind, "seqs": seqs, "lo": _log(rng, max(1, hi // 50), hi), "hi": hi, "page": page,
                "f32": rng.random() < 0.3}
    if kind == "prefill":
        cross = rng.random() < 0.3
        seqs = _log(rng, 1, 12)
        qhi = _log(rng, 1, max(1, 4096 // seqs))
        hi = _log(rng, 1, min(65536, max(1, (1 << 24) // (qhi * seqs))))
        return {"kind": kind, "seqs": seqs, "qlo": _log(rng, max(1, qhi // 20), qhi), "qhi": qhi,
                "lo": _log(rng, max(1, hi // 20), hi), "hi": hi, "ratio": rng.choice([1, 2]), "cross": cross,
                "page": page, "f32": rng.random() < 0.3}
    if kind == "beam":
        return {"kind": kind, "groups": _log(rng, 1, 32), "width": _log(rng, 1, 8), "lo": _log(rng, 1, 500),
                "hi": _log(rng, 500, 8191), "caches": rng.choice([1, 1, 2, 3]), "page": page}
    return {"kind": kind, "pages": _log(rng, 8, 12000), "seqs": _log(rng, 1, 64),
            "live": rng.uniform(0.05, 1.0), "caches": rng.choice([1, 1, 2]), "page": rng.choice([8, 16, 32, 64])}


def _spread(case, n, lo, hi, what):
    """n lengths in [lo, hi], log-uniform, from the case alone (the last one is hi)."""
    rng = random.Random("%s %d %d %d %s" % (case["kind"], n, lo, hi, what))
    return [_log(rng, lo, hi) if hi > lo else hi for _ in range(n - 1)] + [hi]


def _lens(case):
    """(entries of each sequence, query tokens of each sequence, first query position)."""
    n = case["seqs"]
    lens = [min(case["hi"], max(case["lo"], v)) for v in _spread(case, n, case["lo"], case["hi"], "entries")]
    if case["kind"] == "decode":
        return lens, [1] * n, [0] * n
    qs = [min(case["qhi"], max(case["qlo"], v)) for v in _spread(case, n, case["qlo"], case["qhi"], "queries")]
    # the chunk is the sequence's last tokens; where it is longer than what the cache holds it starts at 0
    start = [max(0, L * case["ratio"] - q) for L, q in zip(lens, qs)]
    return lens, qs, start


def _visible(case):
    """Entries seen by each query token, per sequence: lists of (first count, step numerator) folded to sums."""
    lens, qs, start = _lens(case)
    if case["kind"] == "decode":
        return sum(lens)
    if case["cross"]:
        return sum(L * q for L, q in zip(lens, qs))
    return sum(min(L, (s + i + 1) // case["ratio"]) for L, q, s in zip(lens, qs, start) for i in range(q))


def _beam(case):
    """Per group: entries, shared full pages, private pages of each row."""
    lens = _spread(case, case["groups"], case["lo"], case["hi"], "beam")
    lens = [min(case["hi"], max(case["lo"], v)) for v in lens]
    shared = [max(0, L // case["page"] - 1) for L in lens]
    private = [-(-L // case["page"]) - f for L, f in zip(lens, shared)]
    return lens, shared, private


def _page_bytes(page):
    return page * (128 + 16 + 128) + page // 8 * 128


def work(case):
    if case["kind"] in ("decode", "prefill"):
        lens, qs, _ = _lens(case)
        rows, seen = sum(qs) * H, _visible(case)
        out = 4 if case["f32"] else 2
        return {"bytes": sum(lens) * 144 + rows * (D * 2 + D * out + 4), "flops": 4 * H * D * seen}
    if case["kind"] == "beam":
        lens, shared, private = _beam(case)
        per_row = [f + p for f, p in zip(shared, private)]
        tails = sum(case["width"] for L in lens if L % case["page"])
        table = sum(case["width"] * n for n in per_row)
        # each tail page read and written; the parents' entries read, the children's written, the old rows' cleared;
        # the reference counts of all of them read and written
        return {"bytes": tails * case["caches"] * 2 * _page_bytes(case["page"]) + table * 4 * 3 + table * 4 * 4,
                "flops": 0}
    n = max(1, int(case["pages"] * case["live"]))
    moved = int(n * (1 - n / case["pages"]))
    return {"bytes": moved * case["caches"] * 2 * _page_bytes(case["page"]) + 4 * 4 * case["pages"], "flops": 0}


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------

def _gen(seed, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(int(seed) * 7919 + 12345)
    return g


def _quantised(n, g):
    """n entries of normal rows with a gain per channel, quantised: codes [n, 128] and scales [n, 16] (bytes)."""
    codes = torch.empty((n, 128), dtype=torch.uint8, device="cuda")
    scales = torch.empty((n, 16), dtype=torch.uint8, device="cuda")
    gain = torch.rand(256, generator=g, device="cuda") * 1.5 + 0.5
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    for o in range(0, n, 1 << 17):
        m = min(1 << 17, n - o)
        x = torch.randn((m, 16, 16), generator=g, device="cuda") * gain.view(16, 16)
        s = (x.abs().amax(2) / 6.0).to(torch.float8_e4m3fn)
        y = x / s.float().clamp_min(2.0 ** -9)[:, :, None]
        c = torch.bucketize(y.abs(), edges, out_int32=True) + (y < 0).int() * 8
        c = c.view(m, 128, 2)
        codes[o:o + m] = (c[:, :, 0] + 16 * c[:, :, 1]).to(torch.uint8)
        scales[o:o + m] = s.view(torch.uint8)
    return codes, scales


def _int(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _prepare_attention(case, seed):
    g = _gen(seed)
    lens, qs, start = _lens(case)
    need = [-(-L // case["page"]) for L in lens]
    n_pages = sum(need) + 1
    perm = torch.randperm(n_pages, generator=g, device="cuda").int()
    table = torch.full((len(lens), max(need)), -1, dtype=torch.int32, device="cuda")
    o = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[o:o + n]
        o += n
    codes, scales = _quantised(n_pages * case["page"], g)
    T = sum(qs)
    cu = [0]
    for q in qs:
        cu.append(cu[-1] + q)
    return {"case": case, "codes": codes, "scales": scales, "table": table, "lens": _int(lens), "max_len": max(lens),
            "q": torch.randn((T, H, D), generator=g, device="cuda").to(torch.bfloat16), "cu_q": _int(cu),
            "q_max": max(qs), "q_start": _int(start), "dtype": torch.float32 if case["f32"] else torch.bfloat16}


def _planes(case, n_pages, g):
    """The arrays of each cache: codes, scales, indexer K and pooled indexer K."""
    n, r = n_pages * case["page"], lambda *s: torch.randint(0, 256, s, generator=g, device="cuda", dtype=torch.uint8)
    return [[r(n, 128), r(n, 16), r(n, 128).view(torch.int16), r(n // 8, 128).view(torch.int16)]
            for _ in range(case["caches"])]


def _prepare_beam(case, seed):
    g = _gen(seed)
    lens, shared, private = _beam(case)
    W, G = case["width"], case["groups"]
    used = sum(f + W * p for f, p in zip(shared, private))
    n_pages = int(used * 1.4) + G * W + 1
    perm = torch.randperm(n_pages, generator=g, device="cuda").int()
    S = G * W
    table = torch.full((2 * S, max(f + p for f, p in zip(shared, private))), -1, dtype=torch.int32, device="cuda")
    refs = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    o = 0
    for i, (f, p) in enumerate(zip(shared, private)):
        table[i * W:(i + 1) * W, :f] = perm[o:o + f]
        refs[perm[o:o + f].long()] = W
        o += f
        table[i * W:(i + 1) * W, f:f + p] = perm[o:o + W * p].view(W, p)
        refs[perm[o:o + W * p].long()] = 1
        o += W * p
    seq = torch.zeros(2 * S, dtype=torch.int32, device="cuda")
    seq[:S] = _int(lens).repeat_interleave(W)
    pick = torch.randint(0, W, (G, W), generator=g, device="cuda", dtype=torch.int32)
    parents = (pick + _int(list(range(0, S, W)))[:, None]).view(-1).contiguous()
    rows = torch.arange(2 * S, dtype=torch.int32, device="cuda")
    return {"case": case, "planes": _planes(case, n_pages, g), "table": table, "refs": refs, "lens": seq,
            "parents": parents, "children": rows[S:].contiguous(), "old": rows[:S].contiguous(), "n_pages": n_pages}


def _prepare_compact(case, seed):
    g = _gen(seed)
    P, S = case["pages"], case["seqs"]
    n = max(1, int(P * case["live"]))
    perm = torch.randperm(P, generator=g, device="cuda").int()[:n]
    per = -(-n // S)
    flat = torch.full((S * per,), -1, dtype=torch.int32, device="cuda")
    flat[:n] = perm
    table = torch.full((S, per + 2), -1, dtype=torch.int32, device="cuda")
    table[:, :per] = flat.view(S, per)
    refs = torch.zeros(P, dtype=torch.int32, device="cuda")
    refs[perm.long()] = 1
    return {"case": case, "planes": _planes(case, P, g), "table": table, "refs": refs, "n_pages": P}


def prepare(case, seed):
    if case["kind"] == "beam":
        return _prepare_beam(case, seed)
    if case["kind"] == "compact":
        return _prepare_compact(case, seed)
    return _prepare_attention(case, seed)


# ---------------------------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------------------------

def _handles(s):
    """What a program that serves keeps: the caches' handles, a workspace, a descriptor."""
    import fp4_kv_cache_nvfp4_b200 as csa2
    if "handles" not in s:
        c = s["case"]
        if "planes" in s:
            table = torch.empty_like(s["table"])  # the pages' operations rewrite it in place
            caches = [csa2.KVCache.from_tensors(p[0], p[1], table, c["page"], idx_k=p[2], pooled=p[3])
                      for p in s["planes"]]
            n_req = s["children"].numel() if c["kind"] == "beam" else 1
            size = csa2.kv_pages_workspace_bytes(s["n_pages"], n_req)
            s["handles"] = caches, table, torch.empty(size, dtype=torch.uint8, device="cuda")
        else:
            cache = csa2.KVCache.from_tensors(s["codes"], s["scales"], s["table"], c["page"])
            desc = csa2.default_desc(csa2.FULL, c.get("ratio", 1))
            size = csa2.dense_attn_workspace_bytes(desc, s["lens"].numel(), c["kind"] == "prefill")
            s["handles"] = cache, desc, torch.empty(size, dtype=torch.uint8, device="cuda")
    return csa2, s["handles"]


def _own_attention(s):
    csa2, (cache, desc, ws) = _handles(s)
    q = s["q"]
    out = torch.empty(q.shape, dtype=s["dtype"], device="cuda")
    lse = torch.empty(q.shape[:2], dtype=torch.float32, device="cuda")
    if s["case"]["kind"] == "decode":
        csa2.dense_attn_decode(desc, cache, q, s["lens"], out, lse, s["max_len"], ws)
    else:
        csa2.dense_attn_prefill(desc, cache, q, s["cu_q"], s["lens"], out, lse, s["max_len"], ws,
                                q_start=None if s["case"]["cross"] else s["q_start"])
    return {"out": out, "lse": lse}


def _own_beam(s):
    csa2, (caches, table, ws) = _handles(s)
    table.copy_(s["table"])
    refs, lens = s["refs"].clone(), s["lens"].clone()
    csa2.kv_pages_fork(caches, refs, lens, s["parents"], s["children"], ws)
    csa2.kv_pages_free(caches[0], refs, lens, s["old"])
    return {"table": table, "refs": refs, "lens": lens, "planes": s["planes"]}


def _own_compact(s):
    csa2, (caches, table, ws) = _handles(s)
    table.copy_(s["table"])
    refs = s["refs"].clone()
    moved = torch.empty_like(refs)
    live = torch.empty(1, dtype=torch.int32, device="cuda")
    csa2.kv_pages_compact(caches, refs, moved, live, ws)
    return {"table": table, "refs": refs, "map": moved, "live": live, "planes": s["planes"]}


# ---------------------------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------------------------

def _entries(s):
    """K and V of every sequence's entries, fp32 [seqs, longest, 128] each (rows behind a sequence's last are another's)."""
    page, L = s["case"]["page"], s["max_len"]
    pos = torch.arange(L, device="cuda")
    slots = s["table"][:, pos // page].clamp_min(0).long() * page + pos % page
    nibble = torch.tensor(E2M1, device="cuda")
    byte = torch.arange(256, device="cuda")
    pairs = torch.stack([nibble[byte % 16], nibble[byte // 16]], 1)
    x = pairs[s["codes"][slots].int()].view(*slots.shape, 16, 16)
    x = x * s["scales"][slots].view(torch.float8_e4m3fn).float()[..., None]
    x = x.view(*slots.shape, 256)
    return x[..., :D], x[..., D:]


def _plain_attention(s):
    case, lens = s["case"], s["lens"].long()
    B, T, tq = lens.numel(), s["q"].shape[0], s["q_max"]
    K, V = _entries(s)
    cu = s["cu_q"].long()
    i = torch.arange(tq, device="cuda")
    real = i[None] < (cu[1:] - cu[:-1])[:, None]                       # [B, tq]
    row = (cu[:-1, None] + i[None]).clamp_max(T - 1)
    q = s["q"].float()[row]                                            # [B, tq, 16, 128]
    if case["kind"] == "decode" or case["cross"]:
        seen = lens[:, None].expand(B, tq)
    else:
        seen = torch.minimum((s["q_start"].long()[:, None] + i[None] + 1) // case["ratio"], lens[:, None])
    logits = (q.reshape(B, tq * H, D) @ K.transpose(1, 2)) * (1.0 / math.sqrt(D))
    logits = logits.view(B, tq, H, -1)
    hidden = torch.arange(s["max_len"], device="cuda")[None, None] >= seen[:, :, None]
    logits.masked_fill_(hidden[:, :, None, :], -math.inf)
    m = logits.amax(3)
    m0 = torch.where(m == -math.inf, 0.0, m)
    p = logits.sub_(m0[..., None]).exp_()
    l = p.sum(3)
    V = V * (torch.arange(s["max_len"], device="cuda")[None] < lens[:, None])[..., None]
    o = (p.view(B, tq * H, -1) @ V).view(B, tq, H, D) / torch.where(l == 0, 1.0, l)[..., None]
    lse = m0 + torch.log(l)
    return {"out": o[real].to(s["dtype"]), "lse": lse[real]}


def _plain_beam(s):
    page = s["case"]["page"]
    table, refs, lens = s["table"].clone(), s["refs"].clone(), s["lens"].clone()
    parents, children = s["parents"].long(), s["children"].long()
    L = lens[parents].long()
    rows = table[parents]
    part = L % page > 0
    free = torch.nonzero(refs == 0).view(-1)
    new = free[:int(part.sum())]
    tail = rows[part, (L // page)[part]].long()
    for planes in s["planes"]:
        for p in planes:
            v = p.view(s["n_pages"], -1)
            v[new] = v[tail]
    rows[part, (L // page)[part]] = new.int()
    table[children] = rows
    refs.index_add_(0, rows[rows >= 0].long(), torch.ones_like(rows[rows >= 0]))
    lens[children] = lens[parents]
    old = table[s["old"].long()]
    refs.index_add_(0, old[old >= 0].long(), -torch.ones_like(old[old >= 0]))
    table[s["old"].long()] = -1
    lens[s["old"].long()] = 0
    return {"table": table, "refs": refs, "lens": lens, "planes": s["planes"]}


def _plain_compact(s):
    refs = s["refs"]
    used = refs > 0
    live = used.sum()
    below = torch.arange(s["n_pages"], device="cuda") < live
    holes, high = torch.nonzero(below & ~used).view(-1), torch.nonzero(~below & used).view(-1)
    moved = torch.where(used, torch.arange(s["n_pages"], device="cuda"), -1)
    moved[high] = holes
    for planes in s["planes"]:
        for p in planes:
            v = p.view(s["n_pages"], -1)
            v[holes] = v[high]
    new = torch.zeros_like(refs)
    new[moved[used]] = refs[used]
    table = torch.where(s["table"] >= 0, moved[s["table"].clamp_min(0).long()], -1).int()
    return {"table": table, "refs": new, "map": moved.int(), "live": live.int().view(1), "planes": s["planes"]}


def run(state):
    kind = state["case"]["kind"]
    if own:
        return _own_beam(state) if kind == "beam" else _own_compact(state) if kind == "compact" else _own_attention(state)
    return _plain_beam(state) if kind == "beam" else _plain_compact(state) if kind == "compact" else _plain_attention(state)


# ---------------------------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------------------------

def exact(case, seed):
    """out = sum_j softmax_j(q . k_j / sqrt(128)) v_j and the logarithm of the softmax's sum, one sequence and one
    block of queries at a time."""
    if case["kind"] in ("beam", "compact"):
        return None
    s = _prepare_attention(case, seed)
    lens, qs, start = _lens(case)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    values = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
    t = 0
    for b, (L, n) in enumerate(zip(lens, qs)):
        pages = s["table"][b, :-(-L // case["page"])].long()
        byte = s["codes"].view(-1, case["page"], 128)[pages].reshape(-1, 128)[:L]
        kv = torch.empty((L, 256), dtype=torch.float64, device="cuda")
        kv[:, 0::2] = values[(byte & 15).int()]
        kv[:, 1::2] = values[(byte >> 4).int()]
        sc = s["scales"].view(-1, case["page"], 16)[pages].reshape(-1, 16)[:L].view(torch.float8_e4m3fn).double()
        kv *= sc.repeat_interleave(16, 1)
        step = max(1, (1 << 25) // (16 * L))
        for o in range(0, n, step):
            m = min(step, n - o)
            x = torch.einsum("thd,ld->thl", s["q"][t + o:t + o + m].double(), kv[:, :128]) / 128 ** 0.5
            if case["kind"] == "prefill" and not case["cross"]:
                last = torch.arange(L, device="cuda") * case["ratio"] + case["ratio"] - 1  # an entry's last token
                at = start[b] + o + torch.arange(m, device="cuda")
                x = x.masked_fill((last[None] > at[:, None])[:, None], -math.inf)
            z = torch.logsumexp(x, 2)
            lse[t + o:t + o + m] = z
            w = torch.exp(x - torch.where(torch.isinf(z), 0.0, z)[..., None])
            out[t + o:t + o + m] = torch.einsum("thl,ld->thd", w, kv[:, 128:])
        t += n
    return {"out": out, "lse": lse}
