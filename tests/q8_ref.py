"""Plain 64-bit statements of the 8-bit cache operators (CPU, loops) and seeded
inputs for their tests."""
import math

import numpy as np
import torch

PAGE, D = 16, 128
F8 = torch.float8_e4m3fn
E_MIN = -64
_W = 1e6 ** (-np.arange(0, D, 2) / D)  # radians per position of each rotation pair


def rotate(x, pos):
    """Rotate-half RoPE of x [..., 128] (float64) at integer positions [...]."""
    z = (x[..., :64] + 1j * x[..., 64:]) * np.exp(1j * np.asarray(pos, np.float64)[..., None] * _W)
    return np.concatenate([z.real, z.imag], -1)


def tables(n_new, kv_lens, pool, taken, block_table, cap, num_pages):
    """Row after row.  Returns the outputs and the set of refusals ('kvlen', 'pool', 'oob')."""
    bt = np.array(block_table)
    B, W = bt.shape
    said = set()
    n = [int(x) for x in n_new]
    avail = len(pool) - taken
    if not 0 <= taken <= len(pool):
        said.add("pool")
        avail = 0
    pages = lambda t: -(-t // PAGE)  # noqa: E731
    for b in range(B):
        if kv_lens[b] < 0 or n[b] < 0 or kv_lens[b] + n[b] > W * PAGE:
            said.add("kvlen")
            n[b] = 0
    run = 0
    for b in range(B):
        run += n[b]
        if run > cap and n[b] > 0:
            said.add("pool")
            n[b] = 0
    run = 0
    for b in range(B):
        need = pages(kv_lens[b] + n[b]) - pages(kv_lens[b]) if n[b] else 0
        run += need
        if need and run > avail:
            said.add("pool")
            n[b] = 0
    indptr, pos, slot, kv = [0], [], [], []
    for b in range(B):
        for i in range(n[b]):
            p = int(kv_lens[b]) + i
            if p % PAGE == 0:
                bt[b, p // PAGE] = pool[taken]
                taken += 1
            pg = int(bt[b, p // PAGE])
            ok = 0 <= pg < num_pages
            if not ok:
                said.add("oob")
            pos.append(p)
            slot.append(pg * PAGE + p % PAGE if ok else -1)
        indptr.append(indptr[-1] + n[b])
        kv.append(int(kv_lens[b]) + n[b])
    pad = [-1] * (cap - len(pos))
    return {"block_table": bt, "kv_lens": kv, "taken": taken, "qo_indptr": indptr, "position_ids": pos + pad,
            "slot_map": slot + pad}, said


def round4(v):
    """To 4 significant bits, half to even; 0 below 2^-6."""
    m, e = np.frexp(v)
    r = np.ldexp(np.round(m * 16) / 16, e)  # np.round: half to even
    return np.where(np.abs(r) < 2.0 ** -6, 0.0, r)


class Cache:
    """An 8-bit cache of one tensor, written token by token, on values: code values
    [num_pages, Hkv, 16, 128] (float64), exponents [num_pages, Hkv], and beside them the
    values before rounding (``near`` where a code may fall on either side of a border)."""

    def __init__(self, codes, scale):
        self.code = codes.to(torch.float32).double().numpy().copy()
        self.exp = np.round(np.log2(np.abs(scale.double().numpy()))).astype(int)
        self.y = None

    def append(self, x, y, slots):
        """x [n, Hkv, 128]: the inputs; y: what is stored; slots in order."""
        self.near = np.zeros(self.code.shape, bool)
        for i, s in enumerate(slots):
            if s < 0:
                continue
            pg, o = s // PAGE, s % PAGE
            for h in range(x.shape[1]):
                amax = np.abs(x[i, h]).max()
                e = max(math.frexp(amax)[1] - 8, E_MIN) if amax > 0 else E_MIN
                if o > 0 and self.exp[pg, h] > e:
                    e = self.exp[pg, h]
                if o > 0 and e > self.exp[pg, h]:
                    old = self.code[pg, h, :o]
                    self.code[pg, h, :o] = round4(np.ldexp(old, self.exp[pg, h] - e))
                self.exp[pg, h] = e
                v = np.ldexp(y[i, h], -e)
                self.code[pg, h, o] = round4(v)
                # FP32 products of the rotation: within 2^-18 of the largest input
                d = np.ldexp(amax, -e) * 2.0 ** -18
                self.near[pg, h, o] = round4(v - d) != round4(v + d)


def attention(q, k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, position_ids):
    """float64 [B, Hq, Sq, 128] out, [B, Hq, Sq] lse, and what error bounds need of each
    query: 'sabs' max over keys of sum r_i |k_i| (r: length of q's rotation pair), 'qk' max
    over keys of amax|q| sum |k_i|, 'av' sum p |v|, 'pv' p_max max |v|."""
    q = q.double().numpy()
    B, Hq, Sq, _ = q.shape
    Hkv = k_cache.shape[1]
    kc, vc = k_cache.to(torch.float32).double().numpy(), v_cache.to(torch.float32).double().numpy()
    ks, vs = k_scale.double().numpy(), v_scale.double().numpy()
    out, lse = np.zeros(q.shape), np.full((B, Hq, Sq), -np.inf)
    b_s, b_q = np.zeros((B, Hq, Sq)), np.zeros((B, Hq, Sq))
    b_av, b_pv = np.zeros(q.shape), np.zeros((B, Hq, Sq))
    for b in range(B):
        n = int(kv_lens[b])
        pg = np.asarray(block_table[b][:-(-n // PAGE)], np.int64)
        pos = np.asarray(position_ids[b])
        for h in range(Hkv):
            k = (kc[pg, h] * ks[pg, h][:, None, None]).reshape(-1, D)[:n]
            v = (vc[pg, h] * vs[pg, h][:, None, None]).reshape(-1, D)[:n]
            for g in range(h * (Hq // Hkv), (h + 1) * (Hq // Hkv)):
                r = rotate(q[b, g], pos)
                pair = np.sqrt(q[b, g][:, :64] ** 2 + q[b, g][:, 64:] ** 2)
                pair = np.concatenate([pair, pair], -1)
                for s in range(Sq):
                    nv = min(n, int(pos[s]) + 1)
                    if nv <= 0:
                        continue
                    x = k[:nv] @ r[s] / math.sqrt(D)
                    m = x.max()
                    p = np.exp(x - m)
                    l = p.sum()
                    out[b, g, s] = p @ v[:nv] / l
                    lse[b, g, s] = m + math.log(l)
                    b_s[b, g, s] = (np.abs(k[:nv]) @ pair[s]).max() / math.sqrt(D)
                    b_q[b, g, s] = np.abs(q[b, g, s]).max() * np.abs(k[:nv]).sum(1).max() / math.sqrt(D)
                    b_av[b, g, s] = p @ np.abs(v[:nv]) / l
                    b_pv[b, g, s] = np.abs(v[:nv]).max() / l
    return out, lse, {"sabs": b_s, "qk": b_q, "av": b_av, "pv": b_pv}


def close(got, ref, q_rel, q_abs, p_rel, p_abs):
    """Asserts out and lse against attention()'s answer.  A score is off by at most
    d = q_rel sabs + q_abs qk (what q's operand rounding costs, relative to the element and to
    the largest one); a softmax weight by 2 d and, rounded for the product with V, by p_rel of
    itself and p_abs of the largest weight; bf16 rounds the result by 2^-8 at most."""
    out, lse = got[0].double().cpu().numpy(), got[1].double().cpu().numpy()
    ro, rl, b = ref
    fin = np.isfinite(rl)
    assert np.array_equal(np.isneginf(lse), ~fin) and not np.isnan(lse).any()
    d = q_rel * b["sabs"] + q_abs * b["qk"]
    # the sum of the weights and the logarithm add FP32 roundings
    el = np.abs(lse[fin] - rl[fin])
    tl = (d + 2.0 ** -20 * (1 + np.abs(np.where(fin, rl, 0))))[fin]
    assert (el <= tl).all(), "lse off by %.3g, %.2f of what may be" % (el.max(), (el / tl).max())
    to = 2.0 ** -8 * np.abs(ro) + (2 * d[..., None] + p_rel) * b["av"] + p_abs * b["pv"][..., None] + 1e-30
    eo = np.abs(out - ro)
    assert (eo <= to).all(), "out off by %.3g, %.2f of what may be" % (eo.max(), (eo / to).max())
    return float((el / tl).max()) if el.size else 0.0, float((eo / to).max())


def case(seed, kv_lens, Hq, Hkv, Sq=1, pos=None, W=None, size=1.0, extra=3):
    """A cache in use and queries (CPU tensors).  Slots past a row's last token and pages
    of no row hold NaN codes, pages of no row NaN scales.  pos: [B, Sq], default trailing."""
    g = torch.Generator().manual_seed(seed)
    B = len(kv_lens)
    need = [-(-n // PAGE) for n in kv_lens]
    NP = sum(need) + extra
    W = W or max(need + [1])
    perm = torch.randperm(NP, generator=g).to(torch.int32)
    bt = torch.full((B, W), -1, dtype=torch.int32)
    e = torch.randint(-8, -3, (2, NP, Hkv), generator=g)
    scale = torch.ldexp(torch.ones(2, NP, Hkv), e)
    x = torch.randn((2, NP, Hkv, PAGE, D), generator=g) * size / scale[..., None, None]
    codes = x.clamp(-448, 448).to(F8).view(torch.uint8)
    at = 0
    for b, n in enumerate(kv_lens):
        bt[b, :need[b]] = perm[at:at + need[b]]
        at += need[b]
        if n % PAGE:
            codes[:, bt[b, need[b] - 1].long(), :, n % PAGE:] = 0x7F
    free = perm[at:].long()
    codes[:, free] = 0x7F
    scale[:, free] = float("nan")
    if pos is None:
        pos = [[max(n - Sq, 0) + s for s in range(Sq)] for n in kv_lens]
    return {"q": (torch.randn((B, Hq, Sq, D), generator=g) * size).to(torch.bfloat16),
            "k_cache": codes[0].view(F8), "v_cache": codes[1].view(F8), "k_scale": scale[0].contiguous(),
            "v_scale": scale[1].contiguous(), "block_table": bt, "kv_lens": torch.tensor(kv_lens, dtype=torch.int32),
            "position_ids": torch.tensor(pos, dtype=torch.int32).view(B, Sq)}


NAMES = ("q", "k_cache", "v_cache", "k_scale", "v_scale", "block_table", "kv_lens", "position_ids")
