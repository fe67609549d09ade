"""GPU tests of the 8-bit attention calls at the ends of their ranges: scores up to the
largest that FP32 holds, queries and scales so small that their product vanishes, and pages
whose scales lie far apart."""
import math

import numpy as np
import pytest
import torch

import q8_ref as ref
import test_gpu_q8_attention as att
import test_gpu_q8_tables_append as tab
from deterministic_paged_kv_gb300 import binding

pytestmark = pytest.mark.gpu

i32 = torch.int32
TOL = {"decode": att.DECODE, "prefill": att.PREFILL}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from deterministic_paged_kv_gb300 import build
    build.build()
    binding.load()


# ------------------------------------------------------------- large scores ----

# (size of q, of K): |scores| of some 1e8 to 1e36; FP32 ends at 3e38
SIZES = [(1e7, 1.0), (1e8, 1.0), (1e9, 1.0), (2.0 ** 40, 1.0), (2.0 ** 57, 1.0), (2.0 ** 57, 2.0 ** 57), (1.0, 2.0 ** 40)]


@pytest.mark.parametrize("mode", ["decode", "prefill"])
@pytest.mark.parametrize("q_size,k_size", SIZES)
def test_q8_large_scores(mode, q_size, k_size):
    """No row fails and none has a value that is not finite."""
    c = ref.case(101, [300, 70, 513], 4, 2, Sq=1 if mode == "decode" else 70)
    c["q"] = (c["q"].double() * q_size).to(torch.bfloat16)
    c["k_scale"] = c["k_scale"] * k_size
    st = torch.zeros(1, dtype=i32, device="cuda")
    got = att._run(c, status=st, mode=mode)
    assert int(st.item()) == 0
    att._check(c, got, TOL[mode])


@pytest.mark.parametrize("mode", ["decode", "prefill"])
@pytest.mark.parametrize("q_size,k_size", SIZES)
def test_q8_large_scores_choose_one_key(mode, q_size, k_size):
    """Every query has a key along itself, whose score is more than a thousand above the others': the
    weights are one and zeros, so out is that key's value, exactly (a code over a power of two is a
    bf16 number), zeros included."""
    Sq = 1 if mode == "decode" else 40
    G, Hkv, n = 4, 2, 300
    c = ref.case(103, [n], G * Hkv, Hkv, Sq=Sq)
    pos = c["position_ids"][0].tolist()
    ks, vs = 2.0 ** -6, 2.0 ** -5
    c["k_scale"], c["v_scale"] = torch.full_like(c["k_scale"], ks), torch.full_like(c["v_scale"], vs)
    g = torch.Generator().manual_seed(7)
    v = (torch.randn((n, Hkv, 128), generator=g) / vs).to(ref.F8).float()
    v[:, :, ::3] = 0
    k = torch.randn((n, Hkv, 128), generator=g).double() * 0.1
    t = torch.randperm(n - Sq, generator=g)[:G * Sq].view(G, Sq)  # visible to every query
    for h in range(Hkv):
        for i in range(G):
            k[t[i], h] = torch.from_numpy(ref.rotate(c["q"][0, h * G + i].double().numpy(), pos))
    kc = (k / ks).float().clamp(-448, 448).to(ref.F8)
    page, off = c["block_table"][0].long()[torch.arange(n) // 16], torch.arange(n) % 16
    c["k_cache"].view(torch.uint8)[page, :, off] = kc.view(torch.uint8)
    c["v_cache"].view(torch.uint8)[page, :, off] = v.to(ref.F8).view(torch.uint8)
    # the second largest score of each query is far below the first, at a size of 1 already
    for h in range(Hkv):
        x = torch.from_numpy(np.concatenate([ref.rotate(c["q"][0, h * G + i].double().numpy(), pos) for i in range(G)]))
        s = (x @ (kc[:, h].double() * ks).T / math.sqrt(128)).topk(2).values
        assert float((s[:, 0] - s[:, 1]).min()) > 1
    c["q"] = (c["q"].double() * q_size).to(torch.bfloat16)
    c["k_scale"] = c["k_scale"] * k_size
    st = torch.zeros(1, dtype=i32, device="cuda")
    out, lse = att._run(c, status=st, mode=mode)
    assert int(st.item()) == 0 and torch.isfinite(lse).all()
    want = torch.stack([(v[t[i], h] * vs) for h in range(Hkv) for i in range(G)])[None].to(torch.bfloat16)
    assert torch.equal(out.cpu(), want)


# ------------------------------------------- products that vanish in 32 bits ----

@pytest.mark.parametrize("mode", ["decode", "prefill"])
@pytest.mark.parametrize("k_exp", [-60, -83, -100, -126])
@pytest.mark.parametrize("q_size", [0.0, 2.0 ** -70, 2.0 ** -57])
def test_q8_scores_that_vanish(mode, k_exp, q_size):
    """A query of (next to) nothing against small scales of K: equal scores, so the values' mean."""
    c = ref.case(105, [300, 70, 16], 4, 2, Sq=1 if mode == "decode" else 30)
    c["q"] = (c["q"].double() * q_size).to(torch.bfloat16)
    c["k_scale"].fill_(2.0 ** k_exp)
    st = torch.zeros(1, dtype=i32, device="cuda")
    got = att._run(c, status=st, mode=mode)
    assert int(st.item()) == 0
    att._check(c, got, TOL[mode])


# ------------------------------------------------- weights far below the largest ----

# What a weight is off by: of itself, and of the largest product of a weight and its page's scale of V.
# Decode: three e4m3 parts of 4 bits, each 32 times finer than the one before: 2^-12, and where a
# part is below e4m3's normal numbers 2^-8 of its 2^-10 steps, on weights scaled to 2^8: 2^-26.
# (An exponential and the FP32 sums: 2^-16 of it.)  Prefill: FP16, 2^-11 and steps of 2^-24 on
# weights of which the largest is at least 2^7: 2^-32.
SMALL = {"decode": (2.0 ** -12 + 2.0 ** -16, 2.0 ** -26), "prefill": (2.0 ** -11 + 2.0 ** -16, 2.0 ** -32)}


def _small_weights_bound(c, b, h, g, s, mode):
    """Answer and bound of one query in 64 bits, from each weight's error and each token's code."""
    rel, part = SMALL[mode]
    G = c["q"].shape[1] // c["k_cache"].shape[1]
    n = min(int(c["kv_lens"][b]), int(c["position_ids"][b, s]) + 1)
    pg = c["block_table"][b, :-(-n // 16)].long()
    kc, vc = (c[i].to(torch.float32).double()[pg, h].reshape(-1, 128)[:n] for i in ("k_cache", "v_cache"))
    ks, vs = (c[i].double()[pg, h].repeat_interleave(16)[:n] for i in ("k_scale", "v_scale"))
    q = c["q"][b, h * G + g, s].double().numpy()
    r = torch.from_numpy(ref.rotate(q, int(c["position_ids"][b, s])))
    k = kc * ks[:, None]
    x = k @ r / math.sqrt(128)
    p = torch.exp(x - x.max())
    p = p / p.sum()
    pair = torch.from_numpy(np.tile(np.hypot(q[:64], q[64:]), 2))
    t = TOL[mode]
    d = (t["q_rel"] * (k.abs() @ pair).max() + t["q_abs"] * np.abs(q).max() * k.abs().sum(1).max()) / math.sqrt(128)
    w = p * vs
    out = w @ vc
    off = (2 * d + rel) * (w @ vc.abs()) + part * w.max() * vc.abs().sum(0)
    return out, 2.0 ** -8 * out.abs() + off + 1e-30


def _small_weights_check(c, mode):
    st = torch.zeros(1, dtype=i32, device="cuda")
    out = att._run(c, status=st, mode=mode)[0].double().cpu()
    assert int(st.item()) == 0
    B, Hq, Sq, _ = c["q"].shape
    Hkv = c["k_cache"].shape[1]
    worst = 0.0
    for b in range(B):
        for hq in range(Hq):
            for s in {0, Sq // 2, Sq - 1}:
                want, off = _small_weights_bound(c, b, hq // (Hq // Hkv), hq % (Hq // Hkv), s, mode)
                worst = max(worst, float(((out[b, hq, s] - want).abs() / off).max()))
    assert worst <= 1, "off by %.2f of what may be" % worst


@pytest.mark.parametrize("mode", ["decode", "prefill"])
@pytest.mark.parametrize("Hq,Hkv", [(8, 8), (8, 4), (8, 2), (8, 1)])
@pytest.mark.parametrize("ratio", [8, 11, 15])
def test_q8_a_page_of_large_values(mode, Hq, Hkv, ratio):
    """One page of V has an outlier in one dim, and with it a scale 2^ratio of the others': what the
    other pages give in the other dims keeps its bits."""
    c = ref.case(111, [200, 47, 600], Hq, Hkv, Sq=1 if mode == "decode" else 20)
    c["v_scale"] = torch.full_like(c["v_scale"], 2.0 ** -7)
    for b in range(3):
        pg = c["block_table"][b, 1].long()
        c["v_scale"][pg] = 2.0 ** (ratio - 7)
        codes = torch.zeros((Hkv, 16, 128))
        codes[:, :, 5] = 240.0
        c["v_cache"].view(torch.uint8)[pg] = codes.to(ref.F8).view(torch.uint8)
    _small_weights_check(c, mode)


@pytest.mark.parametrize("mode", ["decode", "prefill"])
@pytest.mark.parametrize("Hq,Hkv", [(8, 8), (8, 4), (8, 2), (8, 1)])
@pytest.mark.parametrize("lead", [4.0, 7.0, 10.0])
def test_q8_a_key_that_takes_nearly_all(mode, Hq, Hkv, lead):
    """A row's first key, whose value is zero, scores `lead` above the rest for every query: the
    others' weights, down to e^-lead of it, are all of the result."""
    Sq = 1 if mode == "decode" else 20
    c = ref.case(113, [200, 47, 600], Hq, Hkv, Sq=Sq)
    # (one query for all heads, and small keys, so that one key leads all of a head's queries)
    c["q"] = c["q"][:, :1, :1].expand(-1, Hq, Sq, -1).contiguous()
    c["k_scale"] = torch.full_like(c["k_scale"], 2.0 ** -9)
    for b in range(3):
        pg = c["block_table"][b, 0].long()
        # at the middle query's position; its neighbours' rotations differ by a few steps
        r = ref.rotate(c["q"][b, 0, 0].double().numpy(), int(c["position_ids"][b, Sq // 2]))
        key = torch.from_numpy(r * (lead * math.sqrt(128) / (r @ r))).float() * 2.0 ** 9
        c["k_scale"][pg] = 2.0 ** -7
        codes = c["k_cache"].view(torch.uint8)
        codes[pg, :, 0] = (key / 4).clamp(-448, 448).to(ref.F8).view(torch.uint8)
        c["v_cache"].view(torch.uint8)[pg, :, 0] = 0
    _small_weights_check(c, mode)


# ------------------------------------------------------------- append's scales ----

@pytest.mark.parametrize("e,taken", [(-65, False), (-64, True), (56, True), (57, False)])
def test_append_q8_scales_that_it_writes(e, taken):
    """A started page's scale is one that the append itself writes, 2^-64 to 2^56 (inputs below
    2^64), or the run is refused and the page stays."""
    c = tab._append_case(8, [(5, 4)], 2)
    page = c["slots"][0] // 16
    c["scale"][:, page] = 2.0 ** e
    got = tab._dev(c)
    st = torch.zeros(1, dtype=i32, device="cuda")
    tab._append(c, got, status=st)
    assert int(st.item()) == (0 if taken else binding.STATUS_SCALE)
    same = all(torch.equal(a, b) for a, b in zip(tab._bits(got), tab._bits(tab._dev(c))))
    assert same == (not taken)


# -------------------------------------------------- V scales that lie far apart ----

def _apart(mode, gap, low_page, n=200, Hq=8, Hkv=2):
    """Rows of equal scores (q = 0), the first's KV head 1 with one page of V (None: no page) at 2^-gap of the others."""
    c = ref.case(121, [n, 70], Hq, Hkv, Sq=1 if mode == "decode" else 20)
    c["q"].zero_()
    top = 20 if gap <= 100 else 60
    c["v_scale"].fill_(2.0 ** top)
    if low_page is not None:
        c["v_scale"][c["block_table"][0, low_page].long(), 1] = 2.0 ** (top - gap)
    return c


@pytest.mark.parametrize("mode", ["decode", "prefill"])
@pytest.mark.parametrize("low_page", [0, 5, 11])
@pytest.mark.parametrize("gap", [30, 79])
def test_q8_v_scales_apart(mode, low_page, gap):
    """Up to 2^80 apart every key is in the sum of the weights: equal ones here."""
    c = _apart(mode, gap, low_page)
    st = torch.zeros(1, dtype=i32, device="cuda")
    got = att._run(c, 1 << 20, status=st, mode=mode)
    assert int(st.item()) == 0
    att._check(c, got, TOL[mode])


@pytest.mark.parametrize("mode", ["decode", "prefill"])
@pytest.mark.parametrize("low_page", [0, 5, 11])
@pytest.mark.parametrize("gap", [82, 135, 150, 180])
def test_q8_v_scales_too_far_apart(mode, low_page, gap):
    """Further apart, where 32 bits lose the smaller ones' weights, that head fails; the rest does not."""
    c = _apart(mode, gap, low_page)
    want = att._run(_apart(mode, gap, None), 1 << 20, mode=mode)
    st = torch.zeros(1, dtype=i32, device="cuda")
    out, lse = att._run(c, 1 << 20, status=st, mode=mode)
    assert int(st.item()) == binding.STATUS_RANGE
    s = c["q"].shape[2] - 1  # sees every page
    assert (out[0, 4:, s] == 0).all() and torch.isnan(lse[0, 4:, s]).all()
    assert torch.equal(out[0, :4], want[0][0, :4]) and torch.equal(lse[0, :4], want[1][0, :4])
    assert att._equal((out[1], lse[1]), (want[0][1], want[1][1]))


def test_decode_q8_v_scales_apart_in_other_splits():
    """Splits are joined by their own sums, so what lies in different ones may be any distance apart
    (as long as each sum is in FP32: 128 weights of up to 2^8 over scales of 2^-120 are not)."""
    for gap in (150, 180):
        c = _apart("decode", gap, 3, n=300)
        c["v_scale"][c["block_table"][0].long(), 1] = 2.0 ** (60 - gap)
        c["v_scale"][c["block_table"][0, 8:16].long(), 1] = 2.0 ** 60
        st = torch.zeros(1, dtype=i32, device="cuda")
        out, lse = att._run(c, 128, status=st)
        if gap == 180:
            assert int(st.item()) == binding.STATUS_RANGE
            assert (out[0, 4:] == 0).all() and torch.isnan(lse[0, 4:]).all() and torch.isfinite(lse[0, :4]).all()
        else:
            assert int(st.item()) == 0
            att._check(c, (out, lse), att.DECODE)


@pytest.mark.parametrize("mode,split", [("decode", 0), ("decode", 1 << 20), ("prefill", 0)])
def test_q8_v_scales_apart_in_other_steps(mode, split):
    """Pages far apart that are read in different steps or tiles; a split of its own is no reason to fail,
    and a row behind one that fails starts afresh."""
    for low_page, high_page in ((1, 50), (70, 2)):
        c = ref.case(123, [1200, 40, 300], 16, 2, Sq=1 if mode == "decode" else 20)
        c["v_scale"].fill_(2.0 ** -6)
        pages = c["block_table"][0].long()
        c["v_scale"][pages[low_page], 0] = 2.0 ** -50
        c["v_scale"][pages[high_page], 0] = 2.0 ** 40
        st = torch.zeros(1, dtype=i32, device="cuda")
        out, lse = att._run(c, split, status=st, mode=mode)
        apart = mode == "decode" and split == 0  # pages 0 .. 31 are the first split, 32 .. 63 the next
        assert int(st.item()) == (0 if apart else binding.STATUS_RANGE)
        c["v_scale"][pages[low_page], 0] = c["v_scale"][pages[high_page], 0] = 2.0 ** -6
        want = att._run(c, split, mode=mode)
        assert torch.equal(out[0, 8:], want[0][0, 8:]) and torch.equal(lse[0, 8:], want[1][0, 8:])
        assert att._equal((out[1:], lse[1:]), (want[0][1:], want[1][1:]))
        if not apart:
            assert (out[0, :8, -1] == 0).all() and torch.isnan(lse[0, :8, -1]).all()


# ------------------------------------------------------------------- neighbours ----

def test_prefill_q8_bits_do_not_depend_on_the_neighbours():
    """A query beside queries with scores of any size (of its own row and KV head, in its tile) has
    the bits that it has beside others, and in a chunk of its own."""
    c = ref.case(141, [500, 300], 8, 2, Sq=64)
    want = att._run(c)
    big = {n: t.clone() for n, t in c.items()}
    hit = [(b, h, s) for b in (0, 1) for h in (1, 6) for s in (3, 17, 40)]
    for i, (b, h, s) in enumerate(hit):
        big["q"][b, h, s] = (c["q"][b, h, s].double() * (1e7, 1e9, 2.0 ** 40)[i % 3]).to(torch.bfloat16)
    st = torch.zeros(1, dtype=i32, device="cuda")
    out, lse = att._run(big, status=st)
    assert int(st.item()) == 0
    keep = torch.ones(c["q"].shape[:3], dtype=torch.bool)
    for b, h, s in hit:
        keep[b, h, s] = False
    keep = keep.cuda()
    assert torch.equal(out[keep], want[0][keep]) and torch.equal(lse[keep], want[1][keep])
    for lo, hi in ((0, 5), (5, 37), (37, 64)):
        part = dict(big, q=big["q"][:, :, lo:hi].contiguous(), position_ids=big["position_ids"][:, lo:hi].contiguous())
        o, l = att._run(part, mode="prefill")
        assert torch.equal(o, out[:, :, lo:hi]) and torch.equal(l, lse[:, :, lo:hi])
