"""Plain 64-bit statements of the speculative step's operators (CPU, loops) and seeded
inputs for their tests."""
import math

import numpy as np
import torch

from q8_ref import rotate

PAGE, D, UNUSED = 16, 128, -2


# ------------------------------------------------------------------ trees ----

def tree(rng, T, shape):
    """Parents of a tree of T places: 'chain', 'star' (one root, all others its children), 'tree',
    'forest' (several roots, unused places between the nodes), 'none' (no node)."""
    if shape == "chain":
        return list(range(-1, T - 1))
    if shape == "star":
        return [-1] + [0] * (T - 1)
    if shape == "none":
        return [UNUSED] * T
    if shape == "tree":
        return [-1] + [int(rng.randint(max(0, n // 2 - 2), n)) for n in range(1, T)]
    row = []
    for n in range(T):
        real = [m for m in range(n) if row[m] != UNUSED]
        c = rng.randint(0, 5)
        row.append(UNUSED if c == 0 else -1 if c == 1 or not real else int(real[rng.randint(0, len(real))]))
    return row


def ways(parents):
    """The nodes that each node sees, itself last; [] where there is none."""
    out = []
    for n, p in enumerate(parents):
        out.append([] if p == UNUSED else [n] if p < 0 else out[p] + [n])
    return out


# -------------------------------------------------------------- attention ----

def case(seed, lens, T, Hq, Hkv, shapes, extra_w=1):
    """lens: tokens before the tree; -T (the tree's size, negative) a row of kv_len 0."""
    rng = np.random.RandomState(seed)
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    kv = [0 if n == -T else n + T for n in lens]
    need = [-(-n // PAGE) for n in kv]
    NP = sum(need) + 3
    W = max(need) + extra_w
    perm = rng.permutation(NP)
    bt = np.full((B, W), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        bt[b, :n] = perm[at:at + n]
        at += n
    par = np.array([tree(rng, T, shapes[b % len(shapes)]) for b in range(B)], np.int32).reshape(B, T)
    r = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16)  # noqa: E731
    return {"q": r(B, Hq, T, D), "k_cache": r(NP, PAGE, Hkv, D), "v_cache": r(NP, PAGE, Hkv, D),
            "block_table": torch.from_numpy(bt), "kv_lens": torch.tensor(kv, dtype=torch.int32),
            "parents": torch.from_numpy(par)}


def attention(c):
    """float64 out [B, Hq, T, D] and lse [B, Hq, T] (an empty query: 0 and -inf), and for each query what
    its error bounds need: 'pairs' max over its keys of sum |q pair| |k pair|, 'abs' max of sum |q| + sum |k|,
    'av' sum p |v|."""
    q = c["q"].double().numpy()
    B, Hq, T, _ = q.shape
    kc, vc = c["k_cache"].double().numpy(), c["v_cache"].double().numpy()
    G = Hq // kc.shape[2]
    out, lse = np.zeros(q.shape), np.full((B, Hq, T), -np.inf)
    pairs, ab, av = np.zeros((B, Hq, T)), np.zeros((B, Hq, T)), np.zeros(q.shape)
    plen = lambda x: np.sqrt(x[..., :64] ** 2 + x[..., 64:] ** 2)  # noqa: E731
    for b in range(B):
        kv = int(c["kv_lens"][b])
        if kv == 0:
            continue
        pre, way = kv - T, ways(c["parents"][b].tolist())
        pos = np.array(list(range(pre)) + [pre + max(len(w) - 1, 0) for w in way])
        pg = c["block_table"][b, :-(-kv // PAGE)].numpy()
        for h in range(kc.shape[2]):
            raw = kc[pg, :, h].reshape(-1, D)[:kv]
            k, v = rotate(raw, pos), vc[pg, :, h].reshape(-1, D)[:kv]
            for hq in range(h * G, h * G + G):
                for n, w in enumerate(way):
                    if not w:
                        continue
                    keys = list(range(pre)) + [pre + m for m in w]
                    s = k[keys] @ rotate(q[b, hq, n], pos[pre + n]) / math.sqrt(D)
                    m = s.max()
                    p = np.exp(s - m)
                    l = p.sum()
                    lse[b, hq, n] = m + math.log(l)
                    out[b, hq, n] = p @ v[keys] / l
                    av[b, hq, n] = p @ np.abs(v[keys]) / l
                    pairs[b, hq, n] = (plen(raw[keys]) @ plen(q[b, hq, n])).max()
                    ab[b, hq, n] = np.abs(raw[keys]).sum(-1).max() + np.abs(q[b, hq, n]).sum()
    return out, lse, {"pairs": pairs, "abs": ab, "av": av}


def bounds(ref):
    """How far out and lse may be.  A score: its two rotated operands are rounded to FP16 (2^-11 each of
    an element, or 2^-25 where that is more; over a rotation pair 2^-10 of the lengths' product in all),
    and their angles, stepped in FP32 from an exact one, are good to 2^-14; sums are FP32.  Weights are rounded to
    BF16 (2^-8), and so is out; a score's error moves a weight by as much, up and down.  FP32's share is below 2^-16."""
    out, lse, x = ref
    s = (x["pairs"] * (2.0 ** -10 + 2.0 ** -14) + x["abs"] * 2.0 ** -25) / math.sqrt(D) * 1.01
    e_lse = s + 2.0 ** -16 * (1 + np.abs(np.where(np.isfinite(lse), lse, 0)))
    e_out = (2 * s + 2.0 ** -8 + 2.0 ** -16)[..., None] * x["av"]
    return e_out + 2.0 ** -8 * (np.abs(out) + e_out), e_lse


# ----------------------------------------------------------- verification ----

def verify(c, b):
    """Row b's walk.  Returns n_accepted, path, tokens, logprobs and whether some choice was so near a
    border (2^-14 of what is compared) that FP32 may make it the other way."""
    T, V = c["logits"].shape[1:]
    par, tok = c["parents"][b].tolist(), c["draft_tokens"][b].tolist()
    temp, coins = float(c["temperature"][b]), c["coins"][b].double().tolist()
    race = c["race"][b].double().numpy()
    path, out, logs, near, eps = [0], [], [], False, 2.0 ** -14
    n = 0
    while True:
        x = c["logits"][b, n].double().numpy()
        x = x / temp if temp else x
        logp = x - x.max() - math.log(np.exp(x - x.max()).sum())
        p = np.exp(logp)
        q = c["draft_probs"][b, n].double().numpy() if c["draft_probs"] is not None else None
        r, took, size = p.copy(), None, p.copy()
        for m in [m for m in range(T) if par[m] == n]:
            t = tok[m]
            if temp == 0:
                yes = int(x.argmax()) == t
            else:
                lhs = coins[m] * (1.0 if q is None else q[t]) * r.sum()
                near |= abs(lhs - r[t]) <= eps * (lhs + size[t])
                yes = lhs < r[t]
            if yes:
                took = m
                break
            if temp == 0:
                continue
            if q is None:
                r[t] = size[t] = 0.0
            else:
                size = size + r.sum() * q
                r = np.maximum(r - r.sum() * q, 0)
        if took is not None:
            out.append(tok[took])
            logs.append(logp[tok[took]])
            path.append(took)
            n = took
            continue
        if temp == 0:
            t = int(x.argmax())
        else:
            if r.sum() <= eps * eps:  # next to nothing left: the choice between r and p is at a border
                near = near or r.sum() > 0
            if not r.sum() > 0:
                r, size = p, p
            key = r / race
            t = int(key.argmax())
            hi = (r + eps * size) / race
            hi[t] = -1
            near |= bool(hi.max() >= key[t] - eps * size[t] / race[t]) if V > 1 else False
        out.append(t)
        logs.append(logp[t])
        return len(path), path, out, logs, near


def verify_case(seed, B, T, V, dtype, probs, shapes, temps=(1.0, 0.7, 0.0, 1.3)):
    """Peaked distributions, drafts drawn from a neighbouring one."""
    rng = np.random.RandomState(seed)
    g = torch.Generator().manual_seed(seed)
    par = np.array([tree(rng, T, shapes[b % len(shapes)]) for b in range(B)], np.int32).reshape(B, T)
    x = torch.randn((B, T, V), generator=g) * 2
    top = torch.randint(0, V, (B, T, 3), generator=g)
    x.scatter_(2, top, torch.rand((B, T, 3), generator=g) * 5 + math.log(V) + 1)
    q = (x + torch.randn((B, T, V), generator=g) * 0.7).softmax(-1)
    at = torch.from_numpy(np.maximum(par, 0)).long()
    rows = q.view(B * T, V)[(torch.arange(B)[:, None] * T + at).reshape(-1)]
    tokens = torch.multinomial(rows, 1, generator=g).view(B, T).to(torch.int32)
    return {"logits": x.to(dtype), "draft_probs": q if probs else None, "draft_tokens": tokens,
            "parents": torch.from_numpy(par), "coins": torch.rand((B, T), generator=g),
            "race": (-torch.log1p(-torch.rand((B, V), generator=g))).clamp(min=2.0 ** -40),
            "temperature": torch.tensor([temps[b % len(temps)] for b in range(B)])}


# ------------------------------------------------------------------ pages ----

def compact(c, T, path, n_keep):
    """(k_cache, v_cache) after the moves, token by token."""
    k, v = c["k_cache"].clone(), c["v_cache"].clone()
    for b in range(len(n_keep)):
        pre = int(c["kv_lens"][b]) - T
        for i in range(int(n_keep[b])):
            s, d = pre + int(path[b][i]), pre + i
            ps, pd = int(c["block_table"][b, s // PAGE]), int(c["block_table"][b, d // PAGE])
            for x in (k, v):
                x[pd, d % PAGE] = x[ps, s % PAGE].clone()
    return k, v


def trim(n_drop, kv_lens, pool, taken, block_table, num_pages):
    """Row after row.  Returns the outputs and the set of refusals ('kvlen', 'pool', 'oob')."""
    bt, pool, said = np.array(block_table), np.array(pool), set()
    B, W = bt.shape
    pages = lambda t: -(-t // PAGE)  # noqa: E731
    room = taken if 0 <= taken <= len(pool) else 0
    if not 0 <= taken <= len(pool):
        said.add("pool")
    kv, freed, run = [int(x) for x in kv_lens], [], 0
    for b in range(B):
        d = int(n_drop[b])
        if kv[b] < 0 or kv[b] > W * PAGE or d < 0 or d > kv[b]:
            said.add("kvlen")
            continue
        lo, hi = pages(kv[b] - d), pages(kv[b])
        run += hi - lo
        if hi > lo and run > room:
            said.add("pool")
            continue
        for j in range(lo, hi):
            if not 0 <= bt[b, j] < num_pages:
                said.add("oob")
            freed.append(int(bt[b, j]))
            bt[b, j] = -1
        kv[b] -= d
    if freed:
        pool[taken - len(freed):taken] = freed
    return {"block_table": bt, "kv_lens": kv, "pool": pool, "taken": taken - len(freed)}, said
