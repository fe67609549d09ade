"""Cases, plain forms and exact values of the speculative step's operators.

A speculative step drafts a tree of T tokens behind every row of the BF16 page
cache, has the model judge all of them in one pass, and keeps one path.  Four
operators make it up, beside the append and the table calls there are:

  tree     attention of the T nodes of a row's tree: every node sees the row's
           prefix, its ancestors and itself
  verify   the walk down the tree: which nodes the target's distribution
           accepts, the token behind them, and the tokens' log-probabilities
  compact  K and V of the accepted nodes moved to the slots that follow the prefix
  trim     the dropped tokens leave the rows' lengths, and the pages that they
           leave empty go back to the pool of free ones

A tree is ``parents`` [B, T]: node n's parent is a node before it, -1 for a
root, -2 where a row has no such node.  Node n lies in slot prefix + n, at
position prefix + depth.  Node 0 is the token that the last step ended with.

``own`` false: elementary torch operations; ``own`` true: the library's calls.
"""
import math
import random

import torch

own = False

D = 128           # head_dim
PAGE = 16         # tokens per page
THETA = 1e6       # RoPE base
DEV = "cuda"
UNUSED = -2


# ------------------------------------------------------------------ cases ----

def listed():
    return [
        # a single request with a small tree: latency
        {"name": "tree one row", "op": "tree", "B": 1, "T": 8, "Hq": 32, "Hkv": 8, "len_lo": 777, "len_hi": 777, "shape": "tree"},
        # the decode throughput batch, each row with a tree of 8
        {"name": "tree 64 x 4096", "op": "tree", "B": 64, "T": 8, "Hq": 32, "Hkv": 8, "len_lo": 4096, "len_hi": 4096, "shape": "tree"},
        # rows of very different lengths, eight query heads to a KV head, chains of an odd length
        {"name": "tree ragged", "op": "tree", "B": 20, "T": 13, "Hq": 64, "Hkv": 8, "len_lo": 90, "len_hi": 9001, "shape": "chain"},
        # the largest trees behind the chunked prefill workload's rows
        {"name": "tree wide", "op": "tree", "B": 8, "T": 64, "Hq": 32, "Hkv": 8, "len_lo": 2048, "len_hi": 2048, "shape": "tree"},
        # two long contexts, two query heads to a KV head
        {"name": "tree long", "op": "tree", "B": 2, "T": 32, "Hq": 16, "Hkv": 8, "len_lo": 100001, "len_hi": 131071, "shape": "tree"},
        # a single request, drafts without probabilities (looked up in its own text): latency
        {"name": "verify one row", "op": "verify", "B": 1, "T": 8, "V": 32000, "dtype": "bf16", "probs": False, "shape": "chain"},
        # the throughput batch, drafts of a small model with its probabilities
        {"name": "verify 64 x 8", "op": "verify", "B": 64, "T": 8, "V": 131072, "dtype": "bf16", "probs": True, "shape": "tree"},
        # an odd vocabulary and 32-bit logits
        {"name": "verify odd", "op": "verify", "B": 20, "T": 13, "V": 100003, "dtype": "f32", "probs": False, "shape": "tree"},
        # the throughput batch's accepted nodes
        {"name": "compact 64 x 8", "op": "compact", "B": 64, "T": 8, "Hkv": 8, "len_lo": 100, "len_hi": 900},
        # many rows with the largest trees
        {"name": "compact 256 x 64", "op": "compact", "B": 256, "T": 64, "Hkv": 8, "len_lo": 5, "len_hi": 700},
        # the step's rejected tokens
        {"name": "trim step", "op": "trim", "B": 64, "drop_lo": 0, "drop_hi": 64, "len_lo": 100, "len_hi": 8000},
        # a thousand finished requests give all their pages back
        {"name": "trim all", "op": "trim", "B": 1024, "drop_lo": 10 ** 9, "drop_hi": 10 ** 9, "len_lo": 1, "len_hi": 8000},
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "verify", "verify", "compact", "trim"])
    if op == "trim":
        hi = _log(rng, 1, 8000)
        return {"op": op, "B": _log(rng, 1, 1024), "drop_lo": 0, "drop_hi": _log(rng, 1, hi), "len_lo": _log(rng, 1, hi), "len_hi": hi}
    shape = rng.choice(["tree", "chain"])
    if op == "verify":
        return {"op": op, "B": _log(rng, 1, 64), "T": _log(rng, 1, 8 if shape == "chain" else 16), "V": _log(rng, 1000, 65000),
                "dtype": rng.choice(["bf16", "f32"]), "probs": rng.random() < 0.5, "shape": shape}
    T = _log(rng, 1, 64)
    Hkv = rng.choice([1, 2, 4, 8])
    if op == "compact":
        return {"op": op, "B": _log(rng, 1, 256), "T": T, "Hkv": Hkv, "len_lo": 5, "len_hi": _log(rng, 5, 700)}
    Hq = Hkv * rng.choice([1, 2, 4, 8])
    B = _log(rng, 1, min(64, max(1, 16384 // (T * Hq))))
    hi = _log(rng, 300, 131072 // B)
    return {"op": op, "B": B, "T": T, "Hq": Hq, "Hkv": Hkv, "len_lo": _log(rng, 300, hi), "len_hi": hi, "shape": shape}


def _spread(n, lo, hi, salt):
    """n whole numbers of [lo, hi], the same for a case whatever the seed."""
    r = random.Random(1000003 * n + 8191 * lo + hi + salt)
    return [r.randint(lo, hi) for _ in range(n)]


def _pages(n):
    return (n + PAGE - 1) // PAGE


def _lens(case):
    """Tokens of each row before the drafted ones (trim: before the drop)."""
    return _spread(case["B"], case["len_lo"], case["len_hi"], 1)


def _drops(case):
    return [min(n, d) for n, d in zip(_lens(case), _spread(case["B"], case["drop_lo"], case["drop_hi"], 2))]


def _used(case):
    """Nodes of each row's tree: chains are whole, trees fill three quarters of the places or more."""
    B, T = case["B"], case["T"]
    return [T] * B if case.get("shape") != "tree" else _spread(B, max(1, T - T // 4), T, 3)


def _kept(case):
    """Accepted nodes of each row: one to an eighth of the tree and one."""
    return _spread(case["B"], 1, max(1, case["T"] // 8 + 1), 4)


def _walked(case):
    """Nodes of a row whose distribution a walk looks at, on average over the inputs below."""
    return min(case["T"], 2.5 if case["probs"] else 2)


def work(case):
    op, B = case["op"], case["B"]
    if op == "trim":
        lens, drops = _lens(case), _drops(case)
        freed = sum(_pages(n) - _pages(n - d) for n, d in zip(lens, drops))
        return {"bytes": 4 * (3 * B + 2) + 12 * freed, "flops": 0}
    T = case["T"]
    if op == "compact":
        kept = sum(_kept(case)) - B  # the first node stays where it is
        return {"bytes": kept * case["Hkv"] * D * 2 * 2 * 2 + 4 * (2 * B + kept), "flops": 0}
    if op == "verify":
        V, size = case["V"], 2 if case["dtype"] == "bf16" else 4
        # the walked nodes' logits, the random numbers of the last draw, and one node's draft probabilities
        rows = _walked(case) * V * size + V * 4 + (V * 4 if case["probs"] else 0)
        return {"bytes": int(B * (rows + T * 28 + 16)), "flops": int(B * 4 * _walked(case) * V)}
    Hq, Hkv, lens = case["Hq"], case["Hkv"], _lens(case)
    nodes = sum(_used(case))
    after = [n + T for n in lens]
    cache = Hkv * 2 * 2 * D * (sum(lens) + nodes) + 4 * sum(_pages(n) for n in after)
    return {"bytes": cache + B * T * (Hq * (4 * D + 4) + 4) + 4 * B,
            "flops": 4 * D * Hq * sum(u * n for u, n in zip(_used(case), lens))}


# ----------------------------------------------------------------- inputs ----

def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _parents(case, seed):
    """A tree for every row: a chain, or nodes that hang on one of the later half of those before them."""
    r = random.Random(seed * 7919 + 13)
    rows = []
    for used in _used(case):
        row = [-1]
        for n in range(1, used):
            row.append(n - 1 if case.get("shape") == "chain" else r.randint(max(0, n // 2 - 2), n - 1))
        rows.append(row + [UNUSED] * (case["T"] - used))
    return rows


def _table(need, perm, W):
    """Block table [B, W] of need[b] pages for each row, in order out of `perm`."""
    j = torch.arange(W, device=DEV)[None]
    start = torch.tensor([0] + need, device=DEV).cumsum(0)[:-1, None]
    live = j < torch.tensor(need, device=DEV)[:, None]
    at = (start + j).clamp(max=perm.numel() - 1)
    return torch.where(live, perm[at], torch.full_like(at, -1).to(torch.int32)).contiguous()


def _prepare_verify(case, seed, g, s):
    B, T, V = case["B"], case["T"], case["V"]
    rows = _parents(case, seed)
    s["parents"] = _i32(rows)
    # a wide bulk of tokens, and four that stand out by more or less
    logits = torch.randn((B * T, V), generator=g, device=DEV).mul_(2)
    tops = torch.randint(0, V, (B * T, 4), generator=g, device=DEV)
    lift = torch.rand((B * T, 4), generator=g, device=DEV) * 7 + (math.log(V) - 1)
    logits.scatter_(1, tops, lift + 2)
    # the draft model's view of the same, and tokens drawn from it
    q = torch.randn((B * T, V), generator=g, device=DEV).mul_(0.7).add_(logits).softmax(-1)
    rank, most = [], 1
    for row in rows:
        seen = {}
        rank.append([])
        for p in row:
            rank[-1].append(seen.get(p, 0))
            seen[p] = seen.get(p, 0) + 1
            most = max(most, seen[p] if p >= 0 else 1)
    drawn = torch.multinomial(q, most, replacement=True, generator=g).view(B, T, most)
    at = s["parents"].long().clamp(min=0)
    k = torch.tensor(rank, device=DEV).clamp(max=most - 1)
    s["draft_tokens"] = drawn[torch.arange(B, device=DEV)[:, None], at, k].to(torch.int32)
    s["draft_probs"] = q.view(B, T, V) if case["probs"] else None
    s["logits"] = logits.to(torch.bfloat16 if case["dtype"] == "bf16" else torch.float32).view(B, T, V)
    s["coins"] = torch.rand((B, T), generator=g, device=DEV)
    s["race"] = torch.rand((B, V), generator=g, device=DEV).neg_().log1p_().neg_().clamp_(min=2.0 ** -40)
    # most rows at 1, some colder, one in eight greedy
    s["temperature"] = torch.tensor([(1.0, 1.0, 0.8, 1.0, 0.6, 1.0, 1.0, 0.0)[b % 8] for b in range(B)], device=DEV)
    i32 = {"dtype": torch.int32, "device": DEV}
    s["out"] = {"n_accepted": torch.empty(B, **i32), "n_drop": torch.empty(B, **i32), "path": torch.empty((B, T), **i32),
                "tokens": torch.empty((B, T), **i32), "logprobs": torch.empty((B, T), device=DEV)}


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    op, B = case["op"], case["B"]
    s = {"op": op, "B": B, "T": case.get("T", 1)}
    Hq = Hkv = case.get("Hkv", 8)
    W = num_pages = 1
    if op == "verify":
        _prepare_verify(case, int(seed), g, s)
    else:
        lens = _lens(case)
        after = [n + (0 if op == "trim" else case["T"]) for n in lens]
        need = [_pages(n) for n in after]
        W, num_pages = max(need) + 2, sum(need) + 7
        perm = torch.randperm(num_pages, generator=g, device=DEV).to(torch.int32)
        s["block_table"] = _table(need, perm, W)
        s["kv_lens"] = _i32(after)
    if op == "trim":
        s["n_drop"] = _i32(_drops(case))
        s["pool"] = perm.clone()  # all handed out but the last seven
        s["taken"] = _i32([sum(need)])
        s["out"] = {"block_table": torch.empty_like(s["block_table"]), "kv_lens": torch.empty_like(s["kv_lens"]),
                    "taken": torch.empty_like(s["taken"]), "pool": s["pool"]}
    if op in ("tree", "compact"):
        shape = (num_pages, PAGE, Hkv, D)
        s["k_cache"] = torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)
        s["v_cache"] = torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)
    if op == "compact":
        r = random.Random(int(seed) * 104729 + 7)
        s["n_keep"] = _i32(_kept(case))
        path = [[0] + sorted(r.sample(range(1, case["T"]), n - 1)) for n in _kept(case)]
        s["path"] = _i32([p + [-1] * (case["T"] - len(p)) for p in path])
    if op == "tree":
        Hq = case["Hq"]
        s["parents"] = _i32(_parents(case, int(seed)))
        s["q"] = torch.randn((B, Hq, case["T"], D), generator=g, device=DEV, dtype=torch.bfloat16)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((B, Hq, case["T"]), device=DEV)
    if own:
        from deterministic_paged_kv_gb300 import binding
        s["plan"] = binding.plan(B, s["T"], Hq, Hkv, D, PAGE, num_pages, W)
        s["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
        if op == "tree":
            s["scratch"] = torch.empty(max(binding.tree_scratch_bytes(s["plan"]), 16), dtype=torch.uint8, device=DEV)
    return s


# ------------------------------------------------------------ plain forms ----

def _rotate(x, pos):
    """Rotate-half RoPE of x [..., D] at positions that broadcast to [...]; the angles in 64 bits."""
    rate = torch.pow(torch.tensor(THETA, dtype=torch.float64, device=DEV),
                     -torch.arange(0, D, 2, device=DEV, dtype=torch.float64) / D)
    a = pos.to(torch.float64)[..., None] * rate
    c, s = torch.cos(a).to(x.dtype), torch.sin(a).to(x.dtype)
    lo, hi = x[..., : D // 2], x[..., D // 2:]
    return torch.cat([lo * c - hi * s, hi * c + lo * s], -1)


def _family(parents):
    """sees [B, T, T]: is m node n or one of its ancestors; depth [B, T] (0 of a root)."""
    p = parents.long()
    B, T = p.shape
    n = torch.arange(T, device=DEV)
    up = p.clamp(min=0)
    at = torch.where(p == UNUSED, torch.full_like(p, -1), n.expand(B, T))
    sees = torch.zeros((B, T, T), dtype=torch.bool, device=DEV)
    depth = torch.full((B, T), -1, dtype=torch.int64, device=DEV)
    for _ in range(T):  # one step towards the root for all nodes at once
        live = at >= 0
        sees |= (n == at[..., None]) & live[..., None]
        depth += live
        at = torch.where(live, torch.where(p.gather(1, at.clamp(min=0)) >= 0, up.gather(1, at.clamp(min=0)), -1), at)
    return sees, depth.clamp(min=0)


def _tree(s):
    q, B, T = s["q"], s["B"], s["T"]
    Hq, Hkv = q.shape[1], s["k_cache"].shape[2]
    sees, depth = _family(s["parents"])
    prefix = s["kv_lens"].long() - T
    N = s["block_table"].shape[1] * PAGE
    t = torch.arange(N, device=DEV)
    node = t[None] - prefix[:, None]                      # [B, N]: which node the slot holds
    inside = (node >= 0) & (node < T)
    pos = torch.where(inside, prefix[:, None] + depth.gather(1, node.clamp(0, T - 1)), t[None])
    table = s["block_table"].long().clamp(min=0)
    k = _rotate(s["k_cache"][table].view(B, N, Hkv, D).float(), pos[..., None]).transpose(1, 2)
    v = s["v_cache"][table].view(B, N, Hkv, D).float().transpose(1, 2)
    r = _rotate(q.float(), (prefix[:, None] + depth)[:, None]).reshape(B, Hkv, Hq // Hkv * T, D)
    x = torch.matmul(r, k.transpose(2, 3)).mul_(1 / math.sqrt(D)).view(B, Hkv, Hq // Hkv, T, N)
    real = s["parents"] != UNUSED
    seen = torch.where(inside[:, None], sees.gather(2, node.clamp(0, T - 1)[:, None].expand(B, T, N)), node[:, None] < 0)
    seen = seen & real[..., None]
    x.masked_fill_(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True).clamp(min=-1e30)
    x = x.sub_(m).exp_()
    l = x.sum(-1, keepdim=True)
    out = torch.matmul(x.view(B, Hkv, -1, N), v).view(B, Hkv, Hq // Hkv, T, D) / l.clamp(min=1e-30)
    return out.view(B, Hq, T, D).to(torch.bfloat16), (m + l.log()).view(B, Hq, T)


def _verify(s):
    """Nodes in order: a node whose parent the walk stands on is tried, and the walk stands on it or tries on."""
    f64 = torch.float64
    B, T, V = s["logits"].shape
    b = torch.arange(B, device=DEV)
    temp = s["temperature"].to(f64)
    greedy = temp == 0
    scale = torch.where(greedy, torch.ones_like(temp), temp)[:, None]
    par, tok, q = s["parents"].long(), s["draft_tokens"].long(), s["draft_probs"]
    at = torch.zeros(B, dtype=torch.int64, device=DEV)
    n_acc = torch.ones(B, dtype=torch.int64, device=DEV)
    path = torch.full((B, T), -1, dtype=torch.int64, device=DEV)
    path[:, 0] = 0
    tokens = torch.full((B, T), -1, dtype=torch.int64, device=DEV)
    logprobs = torch.zeros((B, T), dtype=f64, device=DEV)

    def look(at):
        x = s["logits"][b, at].to(f64) / scale
        return torch.log_softmax(x, -1), x.argmax(-1)

    logp, best = look(at)
    left = logp.exp()                                    # what is left of p, not normalised
    for n in range(1, T):
        tries = par[:, n] == at
        x = tok[:, n]
        lx = left.gather(1, x[:, None])[:, 0]
        draft = torch.ones((), dtype=f64, device=DEV) if q is None else q[b, at].to(f64).gather(1, x[:, None])[:, 0]
        mass = left.sum(-1)
        yes = tries & torch.where(greedy, x == best, s["coins"][:, n].to(f64) * draft * mass < lx)
        no = tries & ~yes
        # the rejected token's share leaves: all of it where the draft has no probabilities, else mass * q
        if q is None:
            gone = left.scatter(1, x[:, None], 0.0)
        else:
            gone = (left - mass[:, None] * q[b, at].to(f64)).clamp(min=0)
        left = torch.where(no[:, None], gone, left)
        tokens[b, n_acc - 1] = torch.where(yes, x, tokens[b, n_acc - 1])
        logprobs[b, n_acc - 1] = torch.where(yes, logp.gather(1, x[:, None])[:, 0], logprobs[b, n_acc - 1])
        path[b, n_acc.clamp(max=T - 1)] = torch.where(yes, torch.full_like(at, n), path[b, n_acc.clamp(max=T - 1)])
        n_acc = n_acc + yes
        at = torch.where(yes, torch.full_like(at, n), at)
        there, most = look(at)
        logp = torch.where(yes[:, None], there, logp)
        best = torch.where(yes, most, best)
        left = torch.where(yes[:, None], there.exp(), left)
    left = torch.where(left.sum(-1, keepdim=True) > 0, left, logp.exp())
    last = torch.where(greedy, best, (left / s["race"].to(f64)).argmax(-1))
    tokens[b, n_acc - 1] = last
    logprobs[b, n_acc - 1] = logp.gather(1, last[:, None])[:, 0]
    i32 = torch.int32
    return {"n_accepted": n_acc.to(i32), "n_drop": (T - n_acc).to(i32), "path": path.to(i32), "tokens": tokens.to(i32),
            "logprobs": logprobs.float()}


def _compact(s):
    B, T = s["B"], s["T"]
    prefix = s["kv_lens"].long()[:, None] - T
    i = torch.arange(T, device=DEV)[None].expand(B, T)
    keep = i < s["n_keep"][:, None]
    rows = torch.arange(B, device=DEV)[:, None].expand(B, T)[keep]

    def slots(t):
        return s["block_table"].long()[rows, t // PAGE] * PAGE + t % PAGE

    src, dst = slots((prefix + s["path"].long())[keep]), slots((prefix + i)[keep])
    for n in ("k_cache", "v_cache"):
        flat = s[n].view(-1, *s[n].shape[2:])
        flat[dst] = flat[src]
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _trim(s):
    o, lens = s["out"], s["kv_lens"].long()
    after = lens - s["n_drop"].long()
    have, left = (lens + PAGE - 1) // PAGE, (after + PAGE - 1) // PAGE
    j = torch.arange(s["block_table"].shape[1], device=DEV)[None]
    free = (j >= left[:, None]) & (j < have[:, None])
    ids = s["block_table"][free]                           # row after row, page after page
    taken = s["taken"] - free.sum().to(torch.int32)
    at = taken.long() + torch.arange(ids.numel(), device=DEV)
    s["pool"][at] = ids
    table = torch.where(free, torch.full_like(s["block_table"], -1), s["block_table"])
    return {"block_table": table, "kv_lens": after.to(torch.int32), "taken": taken, "pool": s["pool"]}


# -------------------------------------------------------------------- run ----

def _run_own(s):
    from deterministic_paged_kv_gb300 import binding
    op = s["op"]
    if op == "tree":
        binding.attn_tree(s["plan"], s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["kv_lens"], s["parents"],
                          s["out"], s["lse"], s["scratch"], status=s["status"])
        return s["out"], s["lse"]
    o = s.get("out")
    if op == "verify":
        binding.verify_tree(s["plan"], s["logits"], s["draft_tokens"], s["parents"], s["coins"], s["race"],
                            s["temperature"], o["n_accepted"], o["n_drop"], o["path"], o["tokens"], o["logprobs"],
                            draft_probs=s["draft_probs"], status=s["status"])
        return o
    if op == "compact":
        binding.kv_compact(s["plan"], s["path"], s["n_keep"], s["block_table"], s["kv_lens"], s["k_cache"], s["v_cache"],
                           status=s["status"])
        return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    # the call writes the table in place: a pass begins with the table as the step left it
    o["block_table"].copy_(s["block_table"])
    binding.tables_trim(s["plan"], s["n_drop"], s["kv_lens"], s["pool"], s["taken"], o["block_table"], o["kv_lens"],
                        o["taken"], status=s["status"])
    return o


def run(state):
    if own:
        return _run_own(state)
    return {"tree": _tree, "verify": _verify, "compact": _compact, "trim": _trim}[state["op"]](state)


# ------------------------------------------------------------------ exact ----

def _exact_tree(s):
    """One row and KV head after the other; each node's keys by its way to the root; rotation as a product of complex numbers."""
    f64, half = torch.float64, D // 2
    q = s["q"]
    B, Hq, T, _ = q.shape
    Hkv = s["k_cache"].shape[2]
    G = Hq // Hkv
    out = torch.zeros((B, Hq, T, D), dtype=f64, device=DEV)
    lse = torch.full((B, Hq, T), -math.inf, dtype=f64, device=DEV)
    w = THETA ** (-torch.arange(half, dtype=f64, device=DEV) * 2 / D)

    def turn(x, pos):
        z = torch.complex(x[..., :half], x[..., half:]) * torch.polar(torch.ones((), dtype=f64, device=DEV).expand(pos.shape + (half,)), pos[..., None] * w)
        return torch.cat([z.real, z.imag], -1)

    for b, (n, row) in enumerate(zip(s["kv_lens"].tolist(), s["parents"].tolist())):
        pre = n - T
        ways = []
        for m, p in enumerate(row):
            ways.append([] if p == UNUSED else ([m] if p < 0 else ways[p] + [m]))
        hide = torch.ones((T, T), dtype=torch.bool)
        for m, way in enumerate(ways):
            hide[m, way] = False
        hide = torch.cat([torch.zeros((T, pre), dtype=torch.bool), hide], 1).to(DEV)
        deep = torch.tensor([max(len(x) - 1, 0) for x in ways], dtype=f64, device=DEV) + pre
        pos = torch.cat([torch.arange(pre, dtype=f64, device=DEV), deep])
        some = torch.tensor([bool(x) for x in ways], device=DEV)
        pg = s["block_table"][b, :_pages(n)].long()
        for h in range(Hkv):
            k = turn(s["k_cache"][pg, :, h].reshape(-1, D)[:n].to(f64), pos)
            v = s["v_cache"][pg, :, h].reshape(-1, D)[:n].to(f64)
            x = turn(q[b, h * G:h * G + G].to(f64), deep[None])
            sc = (x @ k.T / D ** 0.5).masked_fill(hide[None], -math.inf)[:, some]
            ls = torch.logsumexp(sc, -1)
            lse[b, h * G:h * G + G, some] = ls
            out[b, h * G:h * G + G, some] = torch.exp(sc - ls[..., None]) @ v
    return out, lse


def _exact_verify(s):
    """Row after row, down the tree by lists of children; the residual distribution is normalised after every rejection."""
    f64 = torch.float64
    B, T, V = s["logits"].shape
    res = torch.zeros((B, T), dtype=f64, device=DEV)
    coins, toks, pars = s["coins"].tolist(), s["draft_tokens"].tolist(), s["parents"].tolist()
    for b, temp in enumerate(s["temperature"].tolist()):
        kids = [[c for c in range(T) if pars[b][c] == n] for n in range(T)]
        n, i = 0, 0
        while True:
            x = s["logits"][b, n].to(f64)
            if temp > 0:
                x = x / temp
            logp = x - torch.logsumexp(x, 0)
            dist, took = logp.exp(), None
            for c in kids[n]:
                t = toks[b][c]
                if temp == 0:
                    good = int((x == x.max()).nonzero()[0]) == t
                else:
                    d = 1.0 if s["draft_probs"] is None else float(s["draft_probs"][b, n, t])
                    good = coins[b][c] * d < float(dist[t])
                if good:
                    took = c
                    break
                if temp > 0:
                    if s["draft_probs"] is None:
                        dist = dist.clone()
                        dist[t] = 0
                    else:
                        dist = torch.relu(dist - s["draft_probs"][b, n].to(f64))
                    if float(dist.sum()) == 0:
                        break
                    dist = dist / dist.sum()
            if took is None:
                if float(dist.sum()) == 0:
                    dist = logp.exp()
                t = int((x == x.max()).nonzero()[0]) if temp == 0 else int((dist / s["race"][b].to(f64)).argmax())
                res[b, i] = logp[t]
                break
            res[b, i] = logp[toks[b][took]]
            n, i = took, i + 1
    return {"n_accepted": None, "n_drop": None, "path": None, "tokens": None, "logprobs": res}


def exact(case, seed):
    if case["op"] in ("compact", "trim"):
        return None
    s = prepare(case, seed)
    return _exact_tree(s) if case["op"] == "tree" else _exact_verify(s)
