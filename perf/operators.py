"""Cases, plain forms and exact values of the 8-bit paged KV cache operators.

Four operators make up one serving step over a cache held in 8 bits (e4m3
codes, one power-of-two scale for each page of 16 tokens and KV head):

  tables   block table, lengths, indptr, positions and slot map of a step,
           from the rows' lengths and token counts and a pool of free pages
  append   rotate K, quantise K and V, write them into their pages
  decode   attention of one query per row over the cache
  prefill  causal attention of a chunk of queries per row over the cache

``own`` false: elementary torch operations; ``own`` true: the library's calls.
"""
import math
import random

import torch

own = False

D = 128           # head_dim
PAGE = 16         # tokens per page
THETA = 1e6       # RoPE base
E_MIN = -64       # smallest scale exponent
F8 = torch.float8_e4m3fn
DEV = "cuda"


# ------------------------------------------------------------------ cases ----

def listed():
    return [
        # one decode step of a serving batch: every row gets one token, a few rows a new page
        {"name": "tables decode step", "op": "tables", "B": 64, "new_lo": 1, "new_hi": 1, "len_lo": 100, "len_hi": 8000},
        # admission of many prompts at once, some of them continuing an earlier chunk
        {"name": "tables admission", "op": "tables", "B": 1024, "new_lo": 1, "new_hi": 1024, "len_lo": 0, "len_hi": 2000},
        # one token per row: the decode step's append
        {"name": "append decode step", "op": "append", "B": 64, "Hkv": 8, "new_lo": 1, "new_hi": 1, "len_lo": 100, "len_hi": 900},
        # the chunk of the chunked prefill workload: 4 x 512 tokens on whole pages
        {"name": "append chunk", "op": "append", "B": 4, "Hkv": 8, "new_lo": 512, "new_hi": 512, "len_lo": 1536, "len_hi": 1536},
        # ragged chunks that start and end inside pages
        {"name": "append ragged", "op": "append", "B": 24, "Hkv": 8, "new_lo": 1, "new_hi": 1300, "len_lo": 5, "len_hi": 700},
        # a single request: latency
        {"name": "decode one row", "op": "decode", "B": 1, "Hq": 32, "Hkv": 8, "len_lo": 777, "len_hi": 777},
        # the decode throughput workload
        {"name": "decode 64 x 4096", "op": "decode", "B": 64, "Hq": 32, "Hkv": 8, "len_lo": 4096, "len_hi": 4096},
        # rows of very different lengths, eight query heads to a KV head
        {"name": "decode ragged", "op": "decode", "B": 20, "Hq": 64, "Hkv": 8, "len_lo": 90, "len_hi": 9001},
        # two long contexts, two query heads to a KV head
        {"name": "decode long", "op": "decode", "B": 2, "Hq": 16, "Hkv": 8, "len_lo": 100001, "len_hi": 131071},
        # the chunked prefill workload: 4 x (1536 prefix + 512 chunk)
        {"name": "prefill chunk", "op": "prefill", "B": 4, "Sq": 512, "Hq": 32, "Hkv": 8, "pre_lo": 1536, "pre_hi": 1536},
        # the long prefill workload
        {"name": "prefill 8192", "op": "prefill", "B": 1, "Sq": 8192, "Hq": 32, "Hkv": 8, "pre_lo": 0, "pre_hi": 0},
        # short chunks behind prefixes of different lengths, one query head to a KV head
        {"name": "prefill short", "op": "prefill", "B": 3, "Sq": 33, "Hq": 8, "Hkv": 8, "pre_lo": 100, "pre_hi": 700},
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["tables", "append", "decode", "decode", "prefill", "prefill"])
    if op == "tables":
        B = _log(rng, 1, 1024)
        hi = 1 if rng.random() < 0.3 else _log(rng, 2, 1024)
        return {"op": op, "B": B, "new_lo": 1, "new_hi": hi, "len_lo": 0, "len_hi": _log(rng, 1, 8000)}
    if op == "append":
        B = _log(rng, 1, 64)
        hi = 1 if rng.random() < 0.3 else _log(rng, 2, max(2, min(2048, 24000 // B)))
        return {"op": op, "B": B, "Hkv": rng.choice([1, 2, 4, 8]), "new_lo": 1, "new_hi": hi,
                "len_lo": 0, "len_hi": _log(rng, 1, 900)}
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 4, 8])
    if op == "decode":
        B = _log(rng, 1, 64)
        hi = _log(rng, 64, 262144 // B)
        return {"op": op, "B": B, "Hq": Hq, "Hkv": Hkv, "len_lo": _log(rng, 1, hi), "len_hi": hi}
    B = _log(rng, 1, 8)
    Sq = _log(rng, 64, 2048 // B)
    hi = _log(rng, 200, 8192 // B)
    return {"op": op, "B": B, "Sq": Sq, "Hq": min(Hq, 32), "Hkv": Hkv, "pre_lo": min(200, hi), "pre_hi": hi}


def _spread(n, lo, hi, salt):
    """n whole numbers of [lo, hi], the same for a case whatever the seed."""
    r = random.Random(1000003 * n + 8191 * lo + hi + salt)
    return [r.randint(lo, hi) for _ in range(n)]


def _rows(case):
    """(tokens in the cache before the step, tokens of the step) of each row."""
    if case["op"] in ("tables", "append"):
        return (_spread(case["B"], case["len_lo"], case["len_hi"], 1), _spread(case["B"], case["new_lo"], case["new_hi"], 2))
    if case["op"] == "decode":
        return [n - 1 for n in _spread(case["B"], case["len_lo"], case["len_hi"], 3)], [1] * case["B"]
    return _spread(case["B"], case["pre_lo"], case["pre_hi"], 4), [case["Sq"]] * case["B"]


def _pages(n):
    return (n + PAGE - 1) // PAGE


def work(case):
    before, new = _rows(case)
    B, tokens = len(before), sum(new)
    after = [a + b for a, b in zip(before, new)]
    fresh = sum(_pages(x) - _pages(y) for x, y in zip(after, before))
    if case["op"] == "tables":
        return {"bytes": 4 * (3 * B + B + 1) + 8 * fresh + 8 * tokens, "flops": 0}
    if case["op"] == "append":
        touched = sum(_pages(x) - y // PAGE for x, y in zip(after, before))
        return {"bytes": case["Hkv"] * (tokens * D * (2 * 2 + 2 * 1) + touched * 8) + 8 * tokens, "flops": 0}
    Hq, Hkv = case["Hq"], case["Hkv"]
    cache = Hkv * (2 * D * sum(after) + 8 * sum(_pages(n) for n in after)) + 4 * sum(_pages(n) for n in after)
    if case["op"] == "decode":
        return {"bytes": cache + B * Hq * (4 * D + 4), "flops": 4 * D * Hq * sum(after)}
    pairs = sum(n * p + n * (n + 1) // 2 for p, n in zip(before, new))
    return {"bytes": cache + tokens * Hq * (4 * D + 4), "flops": 4 * D * Hq * pairs}


# ----------------------------------------------------------------- inputs ----

def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _cache(g, num_pages, Hkv):
    """Codes and scales of a cache in use: about N(0, 1) values, scales 2^-7 .. 2^-5."""
    shape = (num_pages, Hkv, PAGE, D)
    e = torch.randint(-7, -4, (num_pages, Hkv), generator=g, device=DEV, dtype=torch.int32)
    scale = torch.ldexp(torch.ones_like(e, dtype=torch.float32), e)
    x = torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)
    x = x / scale[:, :, None, None].to(torch.bfloat16)
    x = torch.where(x.abs() < 31 / 2048, torch.zeros_like(x), x).clamp_(-448, 448)
    return x.to(F8), scale


def _table(before, after, perm, W, known):
    """Block table [B, W] of the pages that `known` tokens of each row take out of `perm`, and how many pages that are."""
    need = [_pages(n) for n in known]
    j = torch.arange(W, device=DEV)[None]
    start = torch.tensor([0] + need, device=DEV).cumsum(0)[:-1, None]
    live = j < torch.tensor(need, device=DEV)[:, None]
    at = (start + j).clamp(max=perm.numel() - 1)
    return torch.where(live, perm[at], torch.full_like(at, -1).to(torch.int32)).contiguous(), sum(need)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    before, new = _rows(case)
    after = [a + b for a, b in zip(before, new)]
    B, W = len(before), max(_pages(n) for n in after) + 2
    num_pages = sum(_pages(n) for n in after) + 7
    perm = torch.randperm(num_pages, generator=g, device=DEV).to(torch.int32)
    s = {"op": case["op"], "B": B, "W": W, "num_pages": num_pages, "tokens": sum(new)}
    n_new = torch.tensor(new, device=DEV)
    indptr = torch.zeros(B + 1, dtype=torch.int64, device=DEV)
    indptr[1:] = n_new.cumsum(0)
    s["qo_indptr"] = indptr.to(torch.int32)
    if case["op"] == "tables":
        s["block_table"], held = _table(before, after, perm, W, before)
        s["pool"] = perm[held:].contiguous()
        s["taken"] = _i32([0])
        s["kv_lens"], s["n_new"] = _i32(before), _i32(new)
        s["out"] = {"block_table": s["block_table"].clone(), "kv_lens": torch.empty_like(s["kv_lens"]),
                    "taken": torch.empty_like(s["taken"]), "qo_indptr": torch.empty_like(s["qo_indptr"]),
                    "position_ids": torch.empty(s["tokens"], dtype=torch.int32, device=DEV),
                    "slot_map": torch.empty(s["tokens"], dtype=torch.int32, device=DEV)}
        Hq = Hkv = 8
    else:
        s["block_table"], _ = _table(before, after, perm, W, after)
        s["kv_lens"] = _i32(after)
        Hkv = case["Hkv"]
        Hq = case.get("Hq", Hkv)
        s["k_cache"], s["k_scale"] = _cache(g, num_pages, Hkv)
        s["v_cache"], s["v_scale"] = _cache(g, num_pages, Hkv)
    if case["op"] in ("append", "decode", "prefill"):
        i = torch.arange(s["tokens"], device=DEV)
        row = torch.repeat_interleave(torch.arange(B, device=DEV), n_new)
        pos = torch.tensor(before, device=DEV)[row] + i - indptr[row]
        s["position_ids"] = pos.to(torch.int32)
        if case["op"] == "append":
            s["slot_map"] = (s["block_table"].long()[row, pos // PAGE] * PAGE + pos % PAGE).to(torch.int32)
            size = torch.rand((1, Hkv, 1), generator=g, device=DEV) + 0.5
            s["k_new"] = (torch.randn((s["tokens"], Hkv, D), generator=g, device=DEV) * size).to(torch.bfloat16)
            s["v_new"] = (torch.randn((s["tokens"], Hkv, D), generator=g, device=DEV) * size).to(torch.bfloat16)
        else:
            Sq = s["Sq"] = case.get("Sq", 1)
            s["position_ids"] = s["position_ids"].view(B, Sq)
            s["q"] = torch.randn((B, Hq, Sq, D), generator=g, device=DEV).to(torch.bfloat16)
            s["out"] = torch.empty_like(s["q"])
            s["lse"] = torch.empty((B, Hq, Sq), dtype=torch.float32, device=DEV)
    if own:
        from deterministic_paged_kv_gb300 import binding
        s["plan"] = binding.plan(B, s.get("Sq", 1), Hq, Hkv, D, PAGE, num_pages, W)
        s["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
        if case["op"] == "decode":
            n = binding.decode_q8_scratch_bytes(s["plan"])
            s["scratch"] = torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)
    return s


# ------------------------------------------------------------ plain forms ----

def _angles(pos):
    """cos and sin of the rotation of positions [...], in 64 bits: [..., D / 2]."""
    rate = torch.pow(torch.tensor(THETA, dtype=torch.float64, device=DEV),
                     -torch.arange(0, D, 2, device=DEV, dtype=torch.float64) / D)
    a = pos.to(torch.float64)[..., None] * rate
    return torch.cos(a), torch.sin(a)


def _rotate(x, pos):
    """Rotate-half RoPE of x [..., D] at positions that broadcast to [...]."""
    c, s = _angles(pos)
    c, s = c.to(x.dtype), s.to(x.dtype)
    lo, hi = x[..., : D // 2], x[..., D // 2:]
    return torch.cat([lo * c - hi * s, hi * c + lo * s], -1)


def _tables(s):
    n_new, lens, B, W = s["n_new"].long(), s["kv_lens"].long(), s["B"], s["W"]
    after = lens + n_new
    indptr = torch.zeros(B + 1, dtype=torch.int64, device=DEV)
    indptr[1:] = n_new.cumsum(0)
    have, need = (lens + PAGE - 1) // PAGE, (after + PAGE - 1) // PAGE
    end = (need - have).cumsum(0)
    first = s["taken"].long() + end - (need - have)
    j = torch.arange(W, device=DEV)[None]
    fresh = (j >= have[:, None]) & (j < need[:, None])
    at = (first[:, None] + j - have[:, None]).clamp(0, s["pool"].numel() - 1)
    table = torch.where(fresh, s["pool"][at], s["block_table"])
    i = torch.arange(s["tokens"], device=DEV)
    row = torch.searchsorted(indptr[1:], i, right=True)
    pos = lens[row] + i - indptr[row]
    slot = table.long()[row, pos // PAGE] * PAGE + pos % PAGE
    i32 = torch.int32
    return {"block_table": table, "kv_lens": after.to(i32), "taken": s["taken"] + end[-1:].to(i32),
            "qo_indptr": indptr.to(i32), "position_ids": pos.to(i32), "slot_map": slot.to(i32)}


def _code(v):
    """e4m3 values of v (64 bits), with 4 significant bits or zero."""
    return torch.where(v.abs() < 31 / 2048, torch.zeros_like(v), v).to(torch.float32).to(F8)


def _append_one(x, y, cache, scale, page, off, first):
    """x [T, Hkv, D] as given, y what is stored (64 bits), into cache and scale, in place."""
    amax = x.float().abs().amax(-1)
    e_tok = torch.where(amax > 0, torch.frexp(amax)[1] - 8, E_MIN).clamp(min=E_MIN)
    e_old = torch.frexp(scale)[1] - 1
    at = page[:, None].expand(-1, x.shape[1])
    # pages that start in this step forget what their scale was
    start = torch.where((off == 0)[:, None], torch.full_like(e_old[page], E_MIN), e_old[page])
    e_new = e_old.scatter_reduce(0, at, start, "amin").scatter_reduce(0, at, e_tok.to(e_old.dtype), "amax")
    # tokens that were there before the step take the new scale
    p = page[first]
    old = cache.view(torch.uint8)[p].view(F8).to(torch.float64)
    moved = _code(torch.ldexp(old, (e_old[p] - e_new[p])[:, :, None, None]))
    stay = torch.arange(PAGE, device=DEV)[None] < off[first][:, None]
    held = torch.where(stay[:, None, :, None], moved.view(torch.uint8), cache.view(torch.uint8)[p])
    cache.view(torch.uint8)[p] = held
    cache.view(torch.uint8)[page, :, off] = _code(torch.ldexp(y, -e_new[page][..., None])).view(torch.uint8)
    scale.copy_(torch.ldexp(torch.ones_like(scale), e_new))


def _append(s):
    page, off = s["slot_map"].long() // PAGE, s["slot_map"].long() % PAGE
    first = s["qo_indptr"][:-1].long()
    k = _rotate(s["k_new"].to(torch.float64), s["position_ids"][:, None])
    _append_one(s["k_new"], k, s["k_cache"], s["k_scale"], page, off, first)
    _append_one(s["v_new"], s["v_new"].to(torch.float64), s["v_cache"], s["v_scale"], page, off, first)
    return {n: s[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale")}


def _gather(cache, scale, table):
    """Values [B, Hkv, W * 16, D] (32 bits) of the rows' pages in order."""
    B, W = table.shape
    t = table.long().clamp(min=0)
    x = cache.view(torch.uint8)[t].view(F8).to(torch.float32) * scale[t][..., None, None]
    return x.permute(0, 2, 1, 3, 4).reshape(B, cache.shape[1], W * PAGE, D)


def _attention(s):
    q, B, Sq = s["q"], s["B"], s["Sq"]
    Hq, Hkv = q.shape[1], s["k_cache"].shape[1]
    k = _gather(s["k_cache"], s["k_scale"], s["block_table"])
    v = _gather(s["v_cache"], s["v_scale"], s["block_table"])
    T = k.shape[2]
    r = _rotate(q.float(), s["position_ids"][:, None]).view(B, Hkv, Hq // Hkv * Sq, D)
    x = torch.matmul(r, k.transpose(2, 3)).mul_(1 / math.sqrt(D)).view(B, Hkv, Hq // Hkv, Sq, T)
    t = torch.arange(T, device=DEV)
    seen = (t <= s["position_ids"].long()[..., None]) & (t < s["kv_lens"].long()[:, None, None])
    x.masked_fill_(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    x = x.sub_(m).exp_()
    l = x.sum(-1, keepdim=True)
    out = torch.matmul(x.view(B, Hkv, -1, T), v).view(B, Hkv, Hq // Hkv, Sq, D) / l
    return out.view(B, Hq, Sq, D).to(torch.bfloat16), (m + l.log()).view(B, Hq, Sq)


# -------------------------------------------------------------------- run ----

def _run_own(s):
    from deterministic_paged_kv_gb300 import binding
    if s["op"] == "tables":
        o = s["out"]
        binding.tables_extend(s["plan"], s["n_new"], s["kv_lens"], s["pool"], s["taken"], o["block_table"], o["kv_lens"],
                              o["taken"], o["qo_indptr"], o["position_ids"], o["slot_map"], status=s["status"])
        return o
    if s["op"] == "append":
        binding.kv_append_q8(s["plan"], s["k_new"], s["v_new"], s["slot_map"], s["position_ids"], s["k_cache"],
                             s["v_cache"], s["k_scale"], s["v_scale"], status=s["status"])
        return {n: s[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale")}
    a = (s["plan"], s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["block_table"], s["kv_lens"],
         s["position_ids"], s["out"], s["lse"])
    if s["op"] == "decode":
        binding.attn_decode_q8(*a, s["scratch"], status=s["status"])
    else:
        binding.attn_prefill_q8(*a, status=s["status"])
    return s["out"], s["lse"]


def run(state):
    if own:
        return _run_own(state)
    if state["op"] == "tables":
        return _tables(state)
    return _append(state) if state["op"] == "append" else _attention(state)


# ------------------------------------------------------------------ exact ----

def _exact_append(s, before, new):
    """Row by row and page by page, on values: a page's scale is the largest that one of its tokens asks for."""
    f64 = torch.float64
    got = {}
    half = D // 2
    w = THETA ** (-torch.arange(half, dtype=f64, device=DEV) * 2 / D)
    ang = s["position_ids"].to(f64)[:, None] * w
    z = torch.polar(torch.ones_like(ang), ang)[:, None]
    x = s["k_new"].to(f64)
    z = torch.complex(x[..., :half], x[..., half:]) * z
    stored = {"k": torch.cat([z.real, z.imag], -1), "v": s["v_new"].to(f64)}
    for n in ("k", "v"):
        val = s[n + "_cache"].to(f64)
        exp = torch.round(torch.log2(s[n + "_scale"].to(f64)))
        amax = s[n + "_new"].to(f64).abs().amax(-1)
        # a largest value of exactly 2^k may come out of log2 a hair below k; the next one below it is 2^-8 away
        ask = torch.floor(torch.log2(amax.clamp(min=2.0 ** (E_MIN + 7))) + 1e-9) - 7

        def rounded(v):
            """To 4 significant bits, half to even; zero below 2^-6."""
            step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -40))) - 3)
            r = torch.round(v / step) * step
            return torch.where(r.abs() < 2.0 ** -6, torch.zeros_like(r), r)

        table, i = s["block_table"].tolist(), 0
        for b, (t0, cnt) in enumerate(zip(before, new)):
            t = t0
            while t < t0 + cnt:
                pg, o = table[b][t // PAGE], t % PAGE
                m = min(PAGE - o, t0 + cnt - t)
                e = ask[i:i + m].amax(0)
                if o:
                    e = torch.maximum(e, exp[pg])
                    val[pg, :, :o] = rounded(val[pg, :, :o] * torch.exp2(exp[pg] - e)[:, None, None])
                val[pg, :, o:o + m] = rounded(stored[n][i:i + m] / torch.exp2(e)[None, :, None]).transpose(0, 1)
                exp[pg] = e
                t, i = t + m, i + m
        got[n + "_cache"], got[n + "_scale"] = val, torch.round(torch.exp2(exp + 64)) / 2.0 ** 64
    return got


def _exact_attention(s):
    """One row and KV head after the other, blocks of queries, rotation as a product of complex numbers."""
    f64 = torch.float64
    half = D // 2
    B, Hq, Sq, _ = s["q"].shape
    Hkv = s["k_cache"].shape[1]
    G = Hq // Hkv
    out = torch.empty((B, Hq, Sq, D), dtype=f64, device=DEV)
    lse = torch.empty((B, Hq, Sq), dtype=f64, device=DEV)
    w = THETA ** (-torch.arange(half, dtype=f64, device=DEV) * 2 / D)
    for b, n in enumerate(s["kv_lens"].tolist()):
        pg = s["block_table"][b, :_pages(n)].long()
        pos = s["position_ids"][b].to(f64)
        turn = torch.polar(torch.ones((Sq, half), dtype=f64, device=DEV), pos[:, None] * w)
        for h in range(Hkv):
            k = (s["k_cache"].view(torch.uint8)[pg, h].view(F8).to(f64) * s["k_scale"][pg, h].to(f64)[:, None, None]).reshape(-1, D)[:n]
            v = (s["v_cache"].view(torch.uint8)[pg, h].view(F8).to(f64) * s["v_scale"][pg, h].to(f64)[:, None, None]).reshape(-1, D)[:n]
            for g in range(h * G, h * G + G):
                x = s["q"][b, g].to(f64)
                z = torch.complex(x[:, :half], x[:, half:]) * turn
                x = torch.cat([z.real, z.imag], -1)
                for q0 in range(0, Sq, 2048):
                    last = int(pos[min(Sq, q0 + 2048) - 1]) + 1
                    sc = x[q0:q0 + 2048] @ k[:last].T / D ** 0.5
                    hide = torch.arange(sc.shape[1], device=DEV)[None] > pos[q0:q0 + 2048, None]
                    sc = sc.masked_fill(hide, -math.inf)
                    ls = torch.logsumexp(sc, -1)
                    lse[b, g, q0:q0 + 2048] = ls
                    out[b, g, q0:q0 + 2048] = torch.exp(sc - ls[:, None]) @ v[:last]
    return out, lse


def exact(case, seed):
    if case["op"] == "tables":
        return None
    s = prepare(case, seed)
    return _exact_append(s, *_rows(case)) if case["op"] == "append" else _exact_attention(s)
