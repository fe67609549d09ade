"""GPU tests of rk_paged_attn_tree on rows of many parts that a single missing, doubled or foreign key fails: with scores
of 0 the lse is ln of the number of keys, and values that mark their tile and their place in it count them."""
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


def _marks(c):
    """V of the rows' keys: one of the first 64 dims says the key's tile of 128, one of the others its place."""
    NP, _, Hkv, _ = c["v_cache"].shape
    v = torch.zeros((NP, 16, Hkv, 128), dtype=torch.bfloat16)
    for b in range(len(c["kv_lens"])):
        t = np.arange(int(c["kv_lens"][b]))
        pg = c["block_table"][b].numpy()[t // 16]
        v[pg, t % 16, :, t // 128 % 64] = 1.0
        v[pg, t % 16, :, 64 + t * 5 % 64] = 1.0
    return v


def _counts(c):
    """Keys that each node sees, and how many of them have each mark."""
    B, T = c["parents"].shape
    n, marks = np.zeros((B, T)), np.zeros((B, T, 128))
    for b in range(B):
        kv = int(c["kv_lens"][b])
        for i, way in enumerate(ref.ways(c["parents"][b].tolist())):
            t = np.concatenate([np.arange(kv - T), kv - T + np.array(way, int)])
            n[b, i] = len(t)
            marks[b, i] = np.bincount(t // 128 % 64, minlength=128) + np.bincount(64 + t * 5 % 64, minlength=128)
    return n, marks


@pytest.mark.parametrize("zero", ["q", "k_cache"])
@pytest.mark.parametrize("T,Hq,Hkv", [(4, 2, 2), (12, 8, 2), (20, 16, 4), (40, 4, 1)])
@pytest.mark.parametrize("lens", [[1023, 1024, 1025, 2049, 512, 513], [33000, 16385, 7], [70001, 1024]])
def test_every_key_counts_once(lens, T, Hq, Hkv, zero):
    c = ref.case(len(lens) + T, lens, T, Hq, Hkv, ["tree", "chain"])
    c["v_cache"] = _marks(c)
    c[zero].zero_()
    d = {k: v.cuda() for k, v in c.items()}
    p = binding.plan(len(lens), T, Hq, Hkv, 128, 16, c["k_cache"].shape[0], c["block_table"].shape[1])
    out, lse = torch.full_like(d["q"], float("nan")), torch.full(c["q"].shape[:3], 7.0, device="cuda")
    scratch = torch.full((max(binding.tree_scratch_bytes(p), 16),), 255, dtype=torch.uint8, device="cuda")
    binding.attn_tree(p, d["q"], d["k_cache"], d["v_cache"], d["block_table"], d["kv_lens"], d["parents"], out, lse, scratch)
    n, marks = _counts(c)
    # Every weight is 1 and every sum of a part exact.  In log2: a part's lse has 2^-20 (log2f to a last bit of 10), so the
    # merge's weights 2^-20 ln 2, their ex2 2^-22, sums of up to 16 of them 2^-20; log2f of those 2^-21, the sum of it
    # and the maximum (17) 2^-20: 4.2e-6 in all, 2.9e-6 in ln, and its rounding 5e-7: below 2^-18.  A key more or less
    # is 1 / n, 1.4e-5 at least.
    assert 2.0 ** -18 < 0.5 / n.max()
    assert np.abs(lse.cpu().double().numpy() - np.log(n)[:, None]).max() <= 2.0 ** -18
    # out is rounded once to BF16 (2^-8), and has FP32's share of 2^-18 as above; a tile is at least a tenth of
    # the keys that have its mark (70001 keys are 547 tiles, nine to a mark)
    want = (marks / n[..., None])[:, None]
    assert (np.abs(out.cpu().double().numpy() - want) <= want * (2.0 ** -8 + 2.0 ** -16)).all()


@pytest.mark.parametrize("n,T,Hq", [(1500, 8, 1), (16400, 16, 1), (70001, 8, 1), (33000, 40, 1), (2100, 24, 8)])
def test_a_key_that_a_node_looks_for_is_found_anywhere(n, T, Hq):
    """Every node's query is turned so that one key of the prefix, another for each node, has a score of 36 where the
    others have less than 17: lse and out are that key's, and a key turned to another position, or of another part, would
    change them by much more than their bounds."""
    from q8_ref import rotate
    c = ref.case(n, [n], T, Hq, 1, ["tree"])
    r = np.random.RandomState(n)
    ends = [0, 15, 16, 127, 128, 511, 512, 1023, 1024, 1151, n // 16 * 16 - 1, n - 1, n // 16 * 16]
    at = np.array([ends[i] if i < len(ends) else r.randint(0, n) for i in r.permutation(max(T, len(ends)))[:T]])
    at[np.asarray(at) >= n] = n - 1
    pos = np.array([n + len(w) - 1 for w in ref.ways(c["parents"][0].tolist())])
    bt = c["block_table"][0].numpy()
    for t in set(at.tolist()):
        k = r.randn(128)
        c["k_cache"][bt[t // 16], t % 16, 0] = torch.from_numpy(k * np.sqrt(128 * 3.2 / (k @ k))).to(torch.bfloat16)
    k = c["k_cache"].double().numpy()[bt[at // 16], at % 16, 0]
    for h in range(Hq):
        c["q"][0, h] = torch.from_numpy(rotate(k, at - pos)).to(torch.bfloat16)
    d = {x: y.cuda() for x, y in c.items()}
    p = binding.plan(1, T, Hq, 1, 128, 16, c["k_cache"].shape[0], len(bt))
    out, lse = torch.empty_like(d["q"]), torch.empty(c["q"].shape[:3], device="cuda")
    scratch = torch.empty(max(binding.tree_scratch_bytes(p), 16), dtype=torch.uint8, device="cuda")
    binding.attn_tree(p, d["q"], d["k_cache"], d["v_cache"], d["block_table"], d["kv_lens"], d["parents"], out, lse, scratch)
    want = ref.attention(c)
    v = c["v_cache"].double().numpy()[bt[at // 16], at % 16, 0]
    e_out, e_lse = ref.bounds(want)
    # the case is what it says: the key has all but a hundredth of the weight, and the bounds are small beside it
    assert np.abs(want[0][0] - v).max() < 0.05 and want[1].min() > 30 and e_lse.max() < 0.2 and (e_out[0] <= 0.15 * np.abs(v) + 0.02).all()
    assert (np.abs(lse.cpu().double().numpy() - want[1]) <= e_lse).all()
    assert (np.abs(out.cpu().double().numpy() - want[0]) <= e_out).all()
