"""GPU tests of attention over the 8-bit cache (rk_paged_attn_decode_q8,
rk_paged_attn_prefill_q8) against a plain statement in 64 bits, of what may not
change a result, of the refusals, and of the four operators as one serving loop."""
import numpy as np
import pytest
import torch

import q8_ref as ref
from deterministic_paged_kv_gb300 import binding

pytestmark = pytest.mark.gpu

i32 = torch.int32
# Operand roundings (relative to the element, to the largest element; see q8_ref.close).
# e4m3 keeps 4 bits: a part leaves 2^-4 of what it stands for.  Decode: q as four parts
# (2^-16, with the FP32 rotation, sums and exponent: 2^-14), weights as three (2^-12);
# a part is exact to 2^-10, of at least 2^7 for the largest q (two parts at 2^-8: 2^-25) and
# 2^8 for the largest weight of a split of 512: 512 2^-18.
DECODE = dict(q_rel=2.0 ** -14, q_abs=2.0 ** -24, p_rel=2.0 ** -11, p_abs=2.0 ** -9)
# Prefill: q in FP16 (2^-11, with the FP32 rotation and exponent 2^-16 more), weights in FP16
# (2^-11, with their sums 2^-10; their least step, 2^-25 of weights of which the largest is at least
# 2^7, for each of up to 2^13 keys: 2^-19).
PREFILL = dict(q_rel=2.0 ** -11 + 2.0 ** -16, q_abs=2.0 ** -24, p_rel=2.0 ** -10, p_abs=2.0 ** -19)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from deterministic_paged_kv_gb300 import build
    build.build()
    binding.load()


def _plan(c, W=None):
    B, Hq, Sq, D = c["q"].shape
    return binding.plan(B, Sq, Hq, c["k_cache"].shape[1], D, 16, c["k_cache"].shape[0], W or c["block_table"].shape[1])


def _run(c, split=0, status=None, plan=None, stream=None, mode=None, d=None):
    mode = mode or ("decode" if c["q"].shape[2] == 1 else "prefill")
    d = d or [c[n].cuda() for n in ref.NAMES]
    p = plan or _plan(c)
    out = torch.full(c["q"].shape, 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(c["q"].shape[:3], 7.0, device="cuda")
    if mode == "decode":
        n = binding.decode_q8_scratch_bytes(p, split)
        scratch = torch.full((n // 4,), float("nan"), device="cuda") if n else None
        binding.attn_decode_q8(p, *d, out, lse, scratch, split_tokens=split, status=status, stream=stream)
    else:
        binding.attn_prefill_q8(p, *d, out, lse, status=status, stream=stream)
    torch.cuda.synchronize()
    return out, lse


def _check(c, got, tol):
    return ref.close(got, ref.attention(*[c[n] for n in ref.NAMES]), **tol)


def _equal(a, b):
    return all(torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8)) for x, y in zip(a, b))


LENS = [1, 15, 16, 17, 127, 128, 129, 200, 511, 512, 513, 700, 1024, 1100, 0]


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 8), (4, 2), (32, 8), (8, 1), (24, 3)])
@pytest.mark.parametrize("split", [0, 16, 144, 1 << 20])
def test_decode_q8(Hq, Hkv, split):
    c = ref.case(Hq + 100 * Hkv, LENS, Hq, Hkv)
    st = torch.zeros(1, dtype=i32, device="cuda")
    _check(c, _run(c, split, st), DECODE)
    assert int(st.item()) == 0


def test_decode_q8_positions():
    """The query at kv_len, at kv_len - 1 and inside the row: keys past it are not seen."""
    lens = [40, 40, 40, 600, 600, 600, 600]
    pos = [[40], [39], [7], [600], [0], [512], [130]]
    c = ref.case(3, lens, 16, 4, pos=pos)
    for split in (0, 32):
        _check(c, _run(c, split), DECODE)


@pytest.mark.parametrize("size", [1e-6, 0.02, 6.0, 1e6])
def test_decode_q8_sizes_of_values(size):
    """Flat and one-hot softmaxes (scores from 1e-12 to 1e14)."""
    c = ref.case(4, [513, 33, 1], 8, 2, size=1.0)
    c["q"] = (c["q"].float() * size).to(torch.bfloat16)
    _check(c, _run(c), DECODE)


def test_decode_q8_long_row():
    c = ref.case(5, [40000, 3], 4, 1)
    _check(c, _run(c), DECODE)


@pytest.mark.parametrize("scales", ["apart", "any"])
def test_decode_q8_scales(scales):
    """Page scales 2^-40 .. 2^20 side by side, and scales that are no powers of two."""
    c = ref.case(6, [300, 77, 1000], 8, 2)
    g = torch.Generator().manual_seed(1)
    for n in ("k_scale", "v_scale"):
        if scales == "any":
            c[n] = c[n] * (1 + torch.rand(c[n].shape, generator=g))
        elif n == "v_scale":
            c[n] = torch.exp2(torch.randint(-40, 21, c[n].shape, generator=g).float()).nan_to_num()
    tol = dict(DECODE)
    if scales == "apart":  # weights are rounded with their page's scale in them: the largest product counts
        tol["p_rel"] = 2.0 ** -10
    _check(c, _run(c), tol)


PRE = [(1, 40, [40]), (2, 33, [33, 100]), (3, 128, [128, 700, 130]), (2, 200, [1000, 200]), (1, 2, [2]), (2, 129, [300, 129])]


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 2), (8, 2), (8, 1)])
@pytest.mark.parametrize("B,Sq,lens", PRE)
def test_prefill_q8(Hq, Hkv, B, Sq, lens):
    c = ref.case(Sq + Hq, lens, Hq, Hkv, Sq=Sq)
    st = torch.zeros(1, dtype=i32, device="cuda")
    _check(c, _run(c, status=st), PREFILL)
    assert int(st.item()) == 0


def test_prefill_q8_single_queries_and_odd_positions():
    """Sq = 1; positions past the last key; rows whose queries see nothing or little."""
    c = ref.case(11, [30, 1, 0, 513], 8, 2, Sq=1)
    _check(c, _run(c, mode="prefill"), PREFILL)
    pos = [[50 + s for s in range(40)], [s for s in range(40)], [s for s in range(40)]]
    c = ref.case(12, [90, 300, 0], 4, 2, Sq=40, pos=pos)
    _check(c, _run(c), PREFILL)


@pytest.mark.parametrize("size", [1e-6, 0.02, 6.0, 1e6])
def test_prefill_q8_sizes_of_values(size):
    c = ref.case(13, [300, 70], 4, 2, Sq=70)
    c["q"] = (c["q"].float() * size).to(torch.bfloat16)
    _check(c, _run(c), PREFILL)


def test_prefill_q8_scales():
    c = ref.case(14, [300, 77], 8, 2, Sq=60)
    g = torch.Generator().manual_seed(1)
    for n in ("k_scale", "v_scale"):
        c[n] = c[n] * (1 + torch.rand(c[n].shape, generator=g))
    _check(c, _run(c), PREFILL)


# ---------------------------------------------- what changes no result ----

def _rows(c, rows, W=None, shift=0):
    """The rows of a case as a batch of their own, the table wider, the pages moved."""
    o = dict(c)
    for n in ("q", "kv_lens", "position_ids"):
        o[n] = c[n][rows].contiguous()
    bt = c["block_table"][rows]
    W = W or bt.shape[1]
    t = torch.full((len(rows), W), -1, dtype=i32)
    w = min(W, bt.shape[1])
    t[:, :w] = bt[:, :w]
    NP = c["k_cache"].shape[0]
    t = torch.where(t >= 0, (t + shift) % NP, t).to(i32)
    o["block_table"] = t.contiguous()
    for n in ("k_cache", "v_cache"):
        o[n] = c[n].view(torch.uint8).roll(shift, 0).view(ref.F8)
    for n in ("k_scale", "v_scale"):
        o[n] = c[n].roll(shift, 0)
    return o


@pytest.mark.parametrize("mode", ["decode", "prefill"])
def test_q8_does_not_depend_on_batch_width_or_pages(mode):
    if mode == "decode":
        c = ref.case(21, [700, 33, 1300, 512, 1, 900] * 9, 8, 2)
        rows = [2, 0, 40, 5]
    else:
        c = ref.case(22, [700, 300, 1000, 130], 8, 2, Sq=130)
        rows = [2, 0]
    whole = _run(c)
    for pick, W, shift in ((rows, None, 0), (rows, 200, 5), ([rows[1]], 90, 11)):
        part = _run(_rows(c, pick, W, shift))
        assert _equal(part, [x[pick] for x in whole])


@pytest.mark.parametrize("mode", ["decode", "prefill"])
def test_q8_graph_stream_and_repeats(mode):
    c = ref.case(23, [700, 33, 1300], 8, 2, Sq=1 if mode == "decode" else 30)
    d = [c[n].cuda() for n in ref.NAMES]
    p = _plan(c)
    want = _run(c)
    assert _equal(want, _run(c, d=d, plan=p))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    assert _equal(want, _run(c, d=d, plan=p, stream=s))
    out, lse = torch.zeros_like(d[0]), torch.zeros(c["q"].shape[:3], device="cuda")
    scratch = torch.empty(max(binding.decode_q8_scratch_bytes(p), 16), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        if mode == "decode":
            binding.attn_decode_q8(p, *d, out, lse, scratch)
        else:
            binding.attn_prefill_q8(p, *d, out, lse)
    for _ in range(3):
        out.fill_(3)
        g.replay()
    torch.cuda.synchronize()
    assert _equal(want, (out, lse))
    c2 = ref.case(24, [100, 1000, 40], 8, 2, Sq=c["q"].shape[2], W=c["block_table"].shape[1])
    # new contents of the same buffers
    if c2["k_cache"].shape[0] <= c["k_cache"].shape[0]:
        for t, n in zip(d, ref.NAMES):
            src = c2[n].cuda()
            if n in ("k_cache", "v_cache"):
                t.view(torch.uint8)[:src.shape[0]] = src.view(torch.uint8)
            elif n in ("k_scale", "v_scale"):
                t[:src.shape[0]] = src
            else:
                t.copy_(src)
        g.replay()
        torch.cuda.synchronize()
        assert _equal(_run(c2), (out, lse))


# ----------------------------------------------------------------- refusals ----

def _failed(got, want, bad_rows, c, heads=None):
    """Rows (or query heads) that fail are 0 / NaN, the others bit for bit as before."""
    out, lse = got
    for b in range(out.shape[0]):
        for h in range(out.shape[1]):
            if b in bad_rows and (heads is None or h in heads):
                assert (out[b, h] == 0).all() and torch.isnan(lse[b, h]).all(), (b, h)
            elif b not in bad_rows or (heads is not None and h // (out.shape[1] // c["k_cache"].shape[1]) not in
                                       {x // (out.shape[1] // c["k_cache"].shape[1]) for x in heads}):
                assert torch.equal(out[b, h], want[0][b, h]) and torch.equal(lse[b, h], want[1][b, h]), (b, h)


@pytest.mark.parametrize("mode", ["decode", "prefill"])
def test_q8_status(mode):
    Sq = 1 if mode == "decode" else 20
    def make():
        return ref.case(31, [600, 70, 130], 8, 2, Sq=Sq)
    want = _run(make())
    st = torch.zeros(1, dtype=i32, device="cuda")

    def expect(c, bit, rows, heads=None):
        st.zero_()
        got = _run(c, status=st)
        assert int(st.item()) == bit
        _failed(got, want, rows, c, heads)

    for v in (-1, 600 + 16 * 40):
        c = make()
        c["kv_lens"][0] = v
        expect(c, binding.STATUS_KVLEN, {0})
    for v in (-1, 10 ** 6):
        c = make()
        c["block_table"][1, 2] = v
        expect(c, binding.STATUS_PAGE_OOB, {1})
    c = make()
    c["position_ids"][2, 0] = -4
    st.zero_()
    got = _run(c, status=st)
    assert int(st.item()) == binding.STATUS_POSITION
    # the query fails, others of its row may (they share its tile) or are as before
    assert (got[0][2, :, 0] == 0).all() and torch.isnan(got[1][2, :, 0]).all()
    same = (got[0][2] == want[0][2]).all(-1) & (got[1][2] == want[1][2])
    assert (same | ((got[0][2] == 0).all(-1) & torch.isnan(got[1][2]))).all()
    assert _equal([x[:2] for x in got], [x[:2] for x in want])
    for n in ("k_scale", "v_scale"):
        for v in (0.0, -1.0, float("nan"), float("inf"), 1e-40):
            c = make()
            c[n][c["block_table"][0, 3].long(), 1] = v
            expect(c, binding.STATUS_SCALE, {0}, {4, 5, 6, 7})
    for n in ("k_cache", "v_cache"):
        c = make()
        c[n].view(torch.uint8)[c["block_table"][0, 3].long(), 1, 6, 99] = 0x7F
        expect(c, binding.STATUS_RANGE, {0}, {4, 5, 6, 7})
    for v in (float("nan"), float("inf"), 2.0 ** 64):
        c = make()
        c["q"][1, 2, 0, 5] = v
        st.zero_()
        got = _run(c, status=st)
        assert int(st.item()) == binding.STATUS_RANGE
        assert torch.isnan(got[1][1, 2, 0]) and (got[0][1, 2, 0] == 0).all()
        assert _equal([x[[0, 2]] for x in got], [x[[0, 2]] for x in want])
        assert _equal([x[1, 4:] for x in got], [x[1, 4:] for x in want])


def test_q8_empty_rows_need_nothing_of_the_query():
    for Sq in (1, 3):
        c = ref.case(33, [0, 40], 4, 2, Sq=Sq, pos=[list(range(Sq)), [40 - Sq + s for s in range(Sq)]])
        c["q"][0] = float("nan")
        st = torch.zeros(1, dtype=i32, device="cuda")
        out, lse = _run(c, status=st)
        assert int(st.item()) == 0 and (out[0] == 0).all() and torch.isneginf(lse[0]).all()


# -------------------------------------------------- as they are used together ----

def test_q8_serving_loop():
    """Admit prompts, prefill them in chunks, decode: tables, append and attention
    from lengths on the device, each step against 64 bits on the cache as it is."""
    g = torch.Generator().manual_seed(41)
    B, Hq, Hkv, W, NP = 3, 8, 2, 20, 60
    pool = torch.randperm(NP, generator=g).to(i32).cuda()
    taken = torch.zeros(1, dtype=i32, device="cuda")
    table = torch.full((B, W), -1, dtype=i32, device="cuda")
    lens = torch.zeros(B, dtype=i32, device="cuda")
    kc = torch.full((NP, Hkv, 16, 128), 0x7F, dtype=torch.uint8, device="cuda").view(ref.F8)
    vc = kc.clone()
    ks = torch.full((NP, Hkv), float("nan"), device="cuda")
    vs = ks.clone()
    st = torch.zeros(1, dtype=i32, device="cuda")
    seen = [[], [], []]
    for n in (100, 37, 1, 1, 1):
        p = binding.plan(B, n, Hq, Hkv, 128, 16, NP, W)
        ip = torch.empty(B + 1, dtype=i32, device="cuda")
        pos = torch.empty(B * n, dtype=i32, device="cuda")
        slot = torch.empty(B * n, dtype=i32, device="cuda")
        binding.tables_extend(p, torch.full((B,), n, dtype=i32, device="cuda"), lens, pool, taken, table, lens, taken, ip,
                              pos, slot, status=st)
        k = torch.randn((B * n, Hkv, 128), generator=g).to(torch.bfloat16)
        v = torch.randn((B * n, Hkv, 128), generator=g).to(torch.bfloat16)
        q = torch.randn((B, Hq, n, 128), generator=g).to(torch.bfloat16)
        binding.kv_append_q8(p, k.cuda(), v.cuda(), slot, pos, kc, vc, ks, vs, status=st)
        c = {"q": q, "k_cache": kc, "v_cache": vc, "k_scale": ks, "v_scale": vs, "block_table": table, "kv_lens": lens,
             "position_ids": pos.view(B, n)}
        got = _run(c, status=st)
        host = {x: y.cpu() for x, y in c.items()}
        assert host["kv_lens"].tolist() == [len(s) + n for s in seen] if n == 100 else True
        _check(host, got, DECODE if n == 1 else PREFILL)
        # the cache stands for the tokens: within e4m3's half step (2^-4) of the rotated k and of v
        for b in range(B):
            for i in range(n):
                s = int(slot[b * n + i])
                val = host["v_cache"].to(torch.float32)[s // 16, :, s % 16] * host["v_scale"][s // 16][:, None]
                ref_v = v[b * n + i].float()
                assert ((val - ref_v).abs() <= 2.0 ** -4 * ref_v.abs() + 2.0 ** -6 * host["v_scale"][s // 16][:, None]).all()
                val = host["k_cache"].to(torch.float32)[s // 16, :, s % 16] * host["k_scale"][s // 16][:, None]
                ref_k = torch.from_numpy(ref.rotate(k[b * n + i].double().numpy(), int(pos[b * n + i]))).float()
                assert ((val - ref_k).abs() <= 2.0 ** -4 * ref_k.abs() * 1.001 + 2.0 ** -6 * host["k_scale"][s // 16][:, None]).all()
            seen[b] += [0] * n
    assert int(st.item()) == 0 and lens.tolist() == [140] * B and int(taken) == 27
