"""GPU tests of rk_paged_tables_extend and rk_paged_kv_append_q8 against plain
statements in 64 bits: exact tables, exact scales and codes (K's codes up to
rounding borders that FP32 products cannot tell apart), independence of how
calls cut the tokens, and the refusals."""
import numpy as np
import pytest
import torch

import q8_ref as ref
from deterministic_paged_kv_gb300 import binding

pytestmark = pytest.mark.gpu

i32 = torch.int32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from deterministic_paged_kv_gb300 import build
    build.build()
    binding.load()


def _t(x):
    return torch.tensor(np.asarray(x), dtype=i32, device="cuda")


# ----------------------------------------------------------------- tables ----

def _tables_case(B, lens, new, seed, W=None, spare=5):
    r = np.random.RandomState(seed)
    lens = r.randint(lens[0], lens[1] + 1, B)
    new = r.randint(new[0], new[1] + 1, B)
    pages = -(-lens // 16)
    W = W or int(max(-(-(lens + new) // 16), default=1)) + 1
    need = int((-(-(lens + new) // 16) - pages).sum())
    NP = int(pages.sum()) + need + spare
    perm = r.permutation(NP)
    bt = np.full((B, W), -1)
    at = 0
    for b in range(B):
        bt[b, :pages[b]] = perm[at:at + pages[b]]
        at += pages[b]
    return lens, new, bt, perm[at:], NP


def _extend(lens, new, bt, pool, NP, cap, taken=0, inplace=False, offset=0, stream=None):
    B, W = bt.shape
    p = binding.plan(B, 1, 8, 8, 128, 16, NP, W)
    kv, tk, table = _t(lens), _t([taken]), _t(bt).view(B, W)
    o = {"kv_lens": kv if inplace else torch.full((B,), -9, dtype=i32, device="cuda"),
         "taken": tk if inplace else torch.full((1,), -9, dtype=i32, device="cuda"),
         "qo_indptr": torch.full((B + 1,), -9, dtype=i32, device="cuda"),
         "position_ids": torch.full((cap + offset + 2,), -9, dtype=i32, device="cuda"),
         "slot_map": torch.full((cap + offset + 2,), -9, dtype=i32, device="cuda"), "block_table": table}
    st = torch.zeros(1, dtype=i32, device="cuda")
    pos, slot = o["position_ids"][offset:offset + cap], o["slot_map"][offset:offset + cap]
    binding.tables_extend(p, _t(new), kv, _t(pool), tk, table, o["kv_lens"], o["taken"], o["qo_indptr"], pos, slot,
                          status=st, stream=stream)
    torch.cuda.synchronize()
    assert int(o["position_ids"][offset + cap:].max()) == -9 and int(o["slot_map"][offset + cap:].max()) == -9
    o["position_ids"], o["slot_map"] = pos, slot
    return {k: v.cpu().numpy() for k, v in o.items()}, int(st.item())


BITS = {"kvlen": 2, "pool": 64, "oob": 1}


def _same(got, want):
    for k, v in want[0].items():
        assert np.array_equal(got[0][k], np.asarray(v).reshape(got[0][k].shape)), k
    assert got[1] == sum(BITS[x] for x in want[1])


@pytest.mark.parametrize("B,lens,new,more", [
    (1, (0, 0), (1, 1), 0), (1, (0, 0), (16, 16), 3), (3, (0, 40), (0, 20), 1), (64, (1, 200), (1, 1), 0),
    (7, (15, 17), (1, 2), 5), (33, (0, 100), (0, 300), 130), (1025, (0, 50), (0, 30), 0), (300, (0, 5), (0, 1), 7),
    (2500, (0, 40), (0, 6), 1), (4, (5, 9), (0, 0), 4),
])
@pytest.mark.parametrize("inplace", [False, True])
def test_tables_extend(B, lens, new, more, inplace):
    lens, new, bt, pool, NP = _tables_case(B, lens, new, seed=B)
    cap = int(new.sum()) + more
    want = ref.tables(new, lens, pool, 0, bt, cap, NP)
    _same(_extend(lens, new, bt, pool, NP, cap, inplace=inplace), want)


@pytest.mark.parametrize("offset", [1, 2, 3])
def test_tables_extend_unaligned_and_offset_in_the_pool(offset):
    lens, new, bt, pool, NP = _tables_case(9, (0, 60), (0, 50), seed=5)
    pool = np.concatenate([[-7, -7, -7], pool])
    cap = int(new.sum()) + 3
    _same(_extend(lens, new, bt, pool, NP, cap, taken=3, offset=offset), ref.tables(new, lens, pool, 3, bt, cap, NP))


def test_tables_extend_refuses_rows_and_leaves_them():
    lens, new, bt, pool, NP = _tables_case(12, (1, 60), (1, 50), seed=8, W=8)
    lens, new = lens.copy(), new.copy()
    lens[1], new[2], new[3] = -1, -4, 8 * 16 - lens[3] + 1       # negative, negative, past W * 16
    cap = int(np.maximum(new, 0).sum()) + 40
    want = ref.tables(new, lens, pool, 0, bt, cap, NP)
    assert want[1] == {"kvlen"}
    _same(_extend(lens, new, bt, pool, NP, cap), want)
    new[2] = 3
    for short in (0, 1, 2, 5):                                    # the pool runs out
        want = ref.tables(new, lens, pool[:short], 0, bt, cap, NP)
        _same(_extend(lens, new, bt, pool[:short], NP, cap), want)
    for c in (0, 1, 30, 90):                                      # the token arrays run out
        _same(_extend(lens, new, bt, pool, NP, c), ref.tables(new, lens, pool, 0, bt, c, NP))
    c = 90                                                        # both
    _same(_extend(lens, new, bt, pool[:3], NP, c), ref.tables(new, lens, pool[:3], 0, bt, c, NP))
    for taken in (-1, len(pool) + 1):
        _same(_extend(lens, new, bt, pool, NP, cap, taken=taken), ref.tables(new, lens, pool, taken, bt, cap, NP))


def test_tables_extend_page_ids_out_of_range():
    lens, new, bt, pool, NP = _tables_case(4, (3, 20), (20, 40), seed=9)
    pool, bt = pool.copy(), bt.copy()
    pool[1], bt[3, lens[3] // 16] = NP, -5
    cap = int(new.sum())
    lens[3] += 1 if lens[3] % 16 == 0 else 0
    want = ref.tables(new, lens, pool, 0, bt, cap, NP)
    assert "oob" in want[1]
    _same(_extend(lens, new, bt, pool, NP, cap), want)


def test_tables_extend_no_rows():
    p = binding.plan(0, 1, 8, 8, 128, 16, 4, 2)
    e = torch.empty(0, dtype=i32, device="cuda")
    out, tk, pos, slot = _t([5]), _t([0]), _t([7] * 6), _t([7] * 6)
    binding.tables_extend(p, e, e, _t([1, 2]), _t([1]), e.view(0, 2), e, tk, out, pos, slot)
    assert out.tolist() == [0] and tk.tolist() == [1] and pos.tolist() == [-1] * 6 and slot.tolist() == [-1] * 6


def test_tables_extend_captured_steps_advance():
    """A captured step, replayed: lengths, tables and pool go on in place."""
    lens, _, bt, pool, NP = _tables_case(5, (0, 30), (20, 20), seed=4)
    B, W = bt.shape
    p = binding.plan(B, 1, 8, 8, 128, 16, NP, W)
    kv, tk, table, n = _t(lens), _t([0]), _t(bt), _t([1] * B)
    ip, pos, slot, pl = _t([0] * (B + 1)), _t([0] * B), _t([0] * B), _t(pool)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        binding.tables_extend(p, n, kv, pl, tk, table, kv, tk, ip, pos, slot)
    t = 0
    for _ in range(20):
        g.replay()
        want, _ = ref.tables([1] * B, lens, pool, t, bt, B, NP)
        lens, t, bt = np.array(want["kv_lens"]), want["taken"], want["block_table"]
        assert kv.tolist() == list(lens) and tk.tolist() == [t] and slot.tolist() == want["slot_map"]
        assert np.array_equal(table.cpu().numpy(), bt)


# ----------------------------------------------------------------- append ----

def _append_case(seed, runs, Hkv, size=1.0, NP=None):
    """runs: (first position, tokens) of each row, one row to a set of pages of its own."""
    g = torch.Generator().manual_seed(seed)
    NP = NP or sum(-(-(a + n) // 16) for a, n in runs) + 2
    perm = torch.randperm(NP, generator=g).tolist()
    slots, pos, at = [], [], 0
    for a, n in runs:
        pages = perm[at:at + -(-(a + n) // 16)]
        at += len(pages)
        slots += [pages[t // 16] * 16 + t % 16 for t in range(a, a + n)]
        pos += list(range(a, a + n))
    e = torch.randint(-9, -4, (2, NP, Hkv), generator=g)
    scale = torch.ldexp(torch.ones(2, NP, Hkv), e)
    x = torch.randn((2, NP, Hkv, 16, 128), generator=g) * 0.5 / scale[..., None, None]
    codes = torch.where(x.abs() < 31 / 2048, 0 * x, x).clamp(-448, 448).to(ref.F8)
    # token sizes from tiny to large, so that scales grow inside pages, and a few zeros
    mag = torch.exp2(torch.randint(-12, 3, (2, len(slots), Hkv, 1), generator=g).float()) * size
    new = (torch.randn((2, len(slots), Hkv, 128), generator=g) * mag).to(torch.bfloat16)
    new[:, ::11] = 0
    return {"codes": codes, "scale": scale, "new": new, "slots": slots, "pos": pos, "NP": NP, "Hkv": Hkv}


def _dev(c):
    return [c["codes"][0].cuda(), c["codes"][1].cuda(), c["scale"][0].cuda().contiguous(), c["scale"][1].cuda().contiguous()]


def _append(c, cache, lo=0, hi=None, status=None, new=None, slots=None, pos=None):
    p = binding.plan(1, 1, c["Hkv"], c["Hkv"], 128, 16, c["NP"], 1)
    hi = len(c["slots"]) if hi is None else hi
    n = (c["new"] if new is None else new)[:, lo:hi].cuda()
    binding.kv_append_q8(p, n[0].contiguous(), n[1].contiguous(), _t((slots or c["slots"])[lo:hi]),
                         _t((pos or c["pos"])[lo:hi]), *cache, status=status)


def _bits(cache):
    return [x.cpu().view(torch.uint8) if x.dtype == ref.F8 else x.cpu().view(i32) for x in cache]


RUNS = [
    [(0, 1)], [(15, 1)], [(5, 11)], [(0, 16)], [(3, 40)],
    [(a, 1) for a in (0, 1, 7, 15, 16, 17, 31, 33, 100, 4095)],                 # a decode step
    [(1536, 64), (7, 45), (0, 33), (31, 2), (16, 16), (12, 3), (9, 1), (0, 70)],  # ragged chunks
    [(13, 35)] * 4 + [(2, 1)] * 17 + [(6, 26)] * 3,
]


@pytest.mark.parametrize("runs", RUNS, ids=range(len(RUNS)))
@pytest.mark.parametrize("Hkv", [1, 3, 8])
def test_append_q8(runs, Hkv):
    c = _append_case(len(runs) * 10 + Hkv, runs, Hkv)
    cache = _dev(c)
    st = torch.zeros(1, dtype=i32, device="cuda")
    _append(c, cache, status=st)
    assert int(st.item()) == 0
    x = c["new"].double().numpy()
    for t, y in ((0, ref.rotate(x[0], np.asarray(c["pos"])[:, None])), (1, x[1])):
        r = ref.Cache(c["codes"][t], c["scale"][t])
        r.append(x[t], y, c["slots"])
        assert np.array_equal(cache[2 + t].cpu().double().numpy(), np.ldexp(1.0, r.exp)), "scales"
        got = cache[t].cpu().to(torch.float32).double().numpy()
        differ = got != r.code
        if t:
            assert not differ.any()
        else:
            assert not (differ & ~r.near).any()
            # next to a border: one step, and less than a step of the smallest code around zero
            assert (np.abs(got - r.code)[differ] <= np.maximum(2.0 ** -3 * np.abs(r.code[differ]), 2.0 ** -6)).all()


def test_append_q8_does_not_depend_on_the_cut():
    """One call, one call per token and calls cut anywhere leave the same bits."""
    c = _append_case(77, [(3, 61), (16, 16), (0, 7), (30, 35)], 4)
    n = len(c["slots"])
    whole = _dev(c)
    _append(c, whole)
    rng = np.random.RandomState(3)
    for cuts in (list(range(n + 1)), [0] + sorted(rng.choice(np.arange(1, n), 9, replace=False).tolist()) + [n]):
        parts = _dev(c)
        for lo, hi in zip(cuts, cuts[1:]):
            _append(c, parts, lo, hi)
        assert all(torch.equal(a, b) for a, b in zip(_bits(whole), _bits(parts)))


def test_append_q8_skips_and_refuses_tokens():
    c = _append_case(5, [(0, 40), (4, 9), (0, 20)], 2)
    want = _dev(c)
    keep = [i for i in range(69) if i not in (45, 46, 47, 48)]
    st = torch.zeros(1, dtype=i32, device="cuda")
    # tokens 45 .. 48 (the end of the second row) dropped: skipped, out of range, negative position
    sub = {**c, "new": c["new"][:, keep], "slots": [c["slots"][i] for i in keep], "pos": [c["pos"][i] for i in keep]}
    _append(sub, want)
    slots, pos = list(c["slots"]), list(c["pos"])
    slots[45], slots[46], slots[47] = -1, c["NP"] * 16, -2
    pos[48] = -3
    got = _dev(c)
    _append(c, got, slots=slots, pos=pos, status=st)
    assert int(st.item()) == binding.STATUS_PAGE_OOB | binding.STATUS_POSITION
    assert all(torch.equal(a, b) for a, b in zip(_bits(want), _bits(got)))


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan"), 2.0 ** 64])
def test_append_q8_values_out_of_range(value):
    """The token's codes of that tensor become NaN; the rest is as if it were a token of zeros."""
    c = _append_case(6, [(2, 20), (0, 3)], 3)
    new = c["new"].clone()
    new[0, 5, 1, 17] = value
    new[1, 21, 2, 90] = value
    zero = c["new"].clone()
    zero[0, 5, 1] = 0
    zero[1, 21, 2] = 0
    got, want = _dev(c), _dev(c)
    st = torch.zeros(1, dtype=i32, device="cuda")
    _append(c, got, new=new, status=st)
    _append(c, want, new=zero)
    assert int(st.item()) == binding.STATUS_RANGE
    g, w = _bits(got), _bits(want)
    s = c["slots"][5]
    w[0][s // 16, 1, s % 16] = 0x7F
    s = c["slots"][21]
    w[1][s // 16, 2, s % 16] = 0x7F
    assert all(torch.equal(a, b) for a, b in zip(g, w))


def test_append_q8_largest_and_smallest_inputs():
    c = _append_case(7, [(0, 4)], 1)
    new = torch.zeros((2, 4, 1, 128), dtype=torch.bfloat16)
    top = torch.tensor([0x5F7F], dtype=torch.int16).view(torch.bfloat16)[0]  # the largest below 2^64
    new[:, 0] = 2.0 ** -120
    new[:, 1, 0, 64] = 2.0 ** -70
    new[:, 2, 0, 3] = -2.0 ** -58
    for k, n in enumerate((1, 2, 3)):
        cache = _dev(c)
        _append(c, cache, 0, n, new=new)
        e = (-64, -64, -64)[k]
        assert float(cache[3][c["slots"][0] // 16, 0]) == 2.0 ** e
        v = cache[1][c["slots"][0] // 16, 0].cpu().float()
        assert float(v[0].abs().max()) == 0.0                      # 2^-120: below 2^-70
        if n > 1:
            assert float(v[1, 64]) == 2.0 ** -6                    # 2^-70: the smallest that stays
        if n > 2:
            assert float(v[2, 3]) == -2.0 ** 6
    new[:, 3] = top
    cache = _dev(c)
    st = torch.zeros(1, dtype=i32, device="cuda")
    _append(c, cache, new=new, status=st)
    assert int(st.item()) == 0 and float(cache[3][c["slots"][0] // 16, 0]) == 2.0 ** 56
    v = cache[1][c["slots"][0] // 16, 0].cpu().float()
    assert float(v[3].max()) == 256.0 and float(v[:3].abs().max()) == 0.0
    assert torch.isfinite(cache[0].cpu().float()[c["slots"][0] // 16, 0, :4]).all()


@pytest.mark.parametrize("scale", [0.0, float("nan"), float("inf"), -2.0 ** -6, 3.0 * 2.0 ** -8, 2.0 ** -65, 2.0 ** 58])
def test_append_q8_refuses_scales_it_did_not_write(scale):
    c = _append_case(8, [(5, 4), (0, 4), (7, 30)], 2)
    page = c["slots"][0] // 16
    c["scale"][1, page, 1] = scale
    got, want = _dev(c), _dev(c)
    st = torch.zeros(1, dtype=i32, device="cuda")
    _append(c, got, status=st)
    assert int(st.item()) == binding.STATUS_SCALE
    before = _bits(_dev(c))
    c["scale"][1, page, 1] = 2.0 ** -6
    want = _dev(c)
    _append(c, want)
    for a, b, z in zip(_bits(got), _bits(want), before):
        b[page, 1] = z[page, 1]           # that page of that head is as it was
        assert torch.equal(a, b)


def test_append_q8_whole_pages_forget_their_scale():
    """A token at slot 0 starts the page anew, whatever its scale holds."""
    c = _append_case(9, [(0, 20)], 2)
    a = _dev(c)
    _append(c, a)
    c["scale"].fill_(float("nan"))
    b = _dev(c)
    _append(c, b)
    for s in {s // 16 for s in c["slots"]}:
        assert torch.equal(a[2][s], b[2][s]) and torch.equal(a[3][s], b[3][s])
    assert all(torch.equal(x, y) for x, y in zip(_bits(a)[:2], _bits(b)[:2]))
