"""GPU tests of rk_paged_attn_tree over batches of short rows, of which a CTA has many items of one or two tiles:
what it says of queries out of range is said of them alone."""
import numpy as np
import pytest
import torch

import tree_ref as ref
from deterministic_paged_kv_gb300 import binding

pytestmark = pytest.mark.gpu

i32 = torch.int32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from deterministic_paged_kv_gb300 import build
    build.build()
    binding.load()


def _call(c, d, p, scratch, status):
    out = torch.full(c["q"].shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full(c["q"].shape[:3], 7.0, device="cuda")
    binding.attn_tree(p, d["q"], d["k_cache"], d["v_cache"], d["block_table"], d["kv_lens"], d["parents"], out, lse,
                      scratch, status=status)
    return out, lse


# up to 32, 64 and 128 queries a KV head, and two blocks of queries; prefixes of no, one and two tiles
@pytest.mark.parametrize("B,T,Hq,Hkv,hi", [(900, 4, 8, 4, 0), (700, 8, 16, 4, 15), (700, 20, 8, 4, 60), (500, 30, 16, 4, 140),
                                          (400, 40, 16, 4, 140), (1200, 1, 4, 4, 140)])
def test_bad_queries_of_many_short_rows_fail_alone(B, T, Hq, Hkv, hi):
    r = np.random.RandomState(B + T)
    c = ref.case(B + T, r.randint(0, hi + 1, B).tolist(), T, Hq, Hkv, ["tree", "chain"])
    d = {k: v.cuda() for k, v in c.items()}
    NP, _, _, _ = c["k_cache"].shape
    p = binding.plan(B, T, Hq, Hkv, 128, 16, NP, c["block_table"].shape[1])
    n = binding.tree_scratch_bytes(p)
    scratch = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
    st = torch.zeros(1, dtype=i32, device="cuda")
    good = _call(c, d, p, scratch, st)
    assert int(st.item()) == 0 and torch.isfinite(good[1]).all()
    for seed, share in ((0, 0.002), (1, 0.03), (2, 0.3)):
        g = torch.Generator().manual_seed(seed)
        hit = torch.rand((B, Hq, T), generator=g) < share
        hit[B // 2, Hq - 1, T - 1] = True
        junk = torch.tensor([float("nan"), 32768.0, -float("inf"), -40000.0])[torch.randint(0, 4, (B, Hq, T), generator=g)]
        q = c["q"].clone()
        q[..., 77] = torch.where(hit, junk.to(torch.bfloat16), q[..., 77])
        d["q"] = q.cuda()
        hd = hit.cuda()
        for _ in range(8):
            st.zero_()
            out, lse = _call(c, d, p, scratch, st)
            assert int(st.item()) == binding.STATUS_RANGE
            assert torch.equal(torch.isnan(lse), hd) and (out[hd] == 0).all()
            assert torch.equal(out[~hd].view(torch.int16), good[0][~hd].view(torch.int16))
            assert torch.equal(lse[~hd].view(i32), good[1][~hd].view(i32))
