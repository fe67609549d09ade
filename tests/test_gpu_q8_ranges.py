"""GPU tests of the 8-bit attention calls at the ends of their ranges: scores up to the
largest that FP32 holds, queries and scales so small that their product vanishes, and pages
whose scales lie far apart."""
import math

import numpy as np
import pytest
import torch

import q8_ref as ref
import test_gpu_q8_attention as att
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
