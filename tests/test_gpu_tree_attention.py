"""GPU tests of rk_paged_attn_tree against its formula in 64 bits: lengths, trees, head groups, what
lies in slots that nothing sees, failed rows and queries, and that a row's bits are its own."""
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


def _plan(c, **kw):
    B, Hq, T, D = c["q"].shape
    NP, P, Hkv, _ = c["k_cache"].shape
    return binding.plan(B, T, Hq, Hkv, D, P, NP, c["block_table"].shape[1], **kw)


def _run(c, status=None, plan=None, stream=None):
    d = {k: v.cuda() for k, v in c.items()}
    p = plan or _plan(c)
    out = torch.full(c["q"].shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full(c["q"].shape[:3], 7.0, device="cuda")
    n = binding.tree_scratch_bytes(p)
    scratch = torch.full((n,), 255, dtype=torch.uint8, device="cuda") if n else None
    binding.attn_tree(p, d["q"], d["k_cache"], d["v_cache"], d["block_table"], d["kv_lens"], d["parents"], out, lse,
                      scratch, status=status, stream=stream)
    torch.cuda.synchronize()
    return out.cpu(), lse.cpu()


def _bits(x):
    return x.view(torch.int16) if x.dtype == torch.bfloat16 else x.view(torch.int32)


def _equal(a, b):
    return all(torch.equal(_bits(x), _bits(y)) for x, y in zip(a, b))


def _near(got, want, mask=None):
    """Every element within the derived bounds; mask [B, T]: the queries that are compared."""
    e_out, e_lse = ref.bounds(want)
    o, l = got[0].double().numpy(), got[1].double().numpy()
    sel = np.ones(l.shape, bool) if mask is None else np.broadcast_to(np.asarray(mask)[:, None], l.shape)
    fin = np.isfinite(want[1])
    assert (np.isneginf(l) == np.isneginf(want[1]))[sel].all() and np.isfinite(l[fin & sel]).all()
    d = np.abs(l - want[1])[fin & sel] - e_lse[fin & sel]
    assert d.size == 0 or d.max() <= 0, "lse off by %g more than its bound" % d.max()
    d = (np.abs(o - want[0]) - e_out)[sel]
    assert d.size == 0 or d.max() <= 0, "out off by %g more than its bound" % d.max()


CASES = [
    # lens before the tree, T, Hq, Hkv, shapes
    ([0], 1, 1, 1, ["chain"]), ([0, 5], 3, 8, 8, ["tree"]), ([1, 15, 16, 17], 8, 8, 2, ["tree", "chain"]),
    ([120, 127, 128, 129, 255, 256], 5, 32, 8, ["tree", "star", "chain"]),
    ([-8, 100, -8, 0], 8, 8, 1, ["forest", "tree"]), ([33, 700, 1], 13, 16, 2, ["forest", "none", "chain"]),
    ([777], 64, 8, 1, ["tree"]), ([50, 1000], 64, 4, 4, ["chain", "star"]), ([511, 512, 513, 1023, 1025], 7, 4, 2, ["tree"]),
    ([300, 4], 33, 16, 2, ["forest"]), ([2047, 2049, 3000], 17, 32, 8, ["tree"]), ([64] * 40, 2, 8, 8, ["chain", "star"]),
    ([95, 96, 97, 111, 112, 113], 16, 8, 4, ["tree", "forest"]), ([200, 1], 63, 8, 1, ["tree", "forest"]),
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_tree_attention_matches_its_formula(i):
    lens, T, Hq, Hkv, shapes = CASES[i]
    c = ref.case(100 + i, lens, T, Hq, Hkv, shapes)
    st = torch.zeros(1, dtype=i32, device="cuda")
    got = _run(c, st)
    assert int(st.item()) == 0
    _near(got, ref.attention(c))
    empty = (c["parents"] == ref.UNUSED) | (c["kv_lens"] == 0)[:, None]
    assert (got[0].permute(0, 2, 1, 3)[empty] == 0).all() and torch.isneginf(got[1].permute(0, 2, 1)[empty]).all()


@pytest.mark.parametrize("lens,T,Hq,Hkv", [([20000, 33000], 6, 8, 2), ([70001], 40, 2, 1), ([16383, 16384, 16400], 2, 2, 2)])
def test_tree_attention_long_rows(lens, T, Hq, Hkv):
    c = ref.case(7, lens, T, Hq, Hkv, ["tree"])
    _near(_run(c), ref.attention(c))


def test_a_chain_is_a_causal_chunk():
    """A chain's queries see what rk_paged_attn_prefill shows them."""
    c = ref.case(3, [100, 700, 0, 129], 24, 16, 4, ["chain"])
    got = _run(c)
    d = {k: v.cuda() for k, v in c.items()}
    pos = (c["kv_lens"][:, None] - 24 + torch.arange(24, dtype=i32)).to(i32).cuda()
    out, lse = torch.empty_like(d["q"]), torch.empty(c["q"].shape[:3], device="cuda")
    binding.attn_prefill(_plan(c), d["q"], d["k_cache"], d["v_cache"], d["block_table"], d["kv_lens"], pos, out, lse)
    want = ref.attention(c)
    _near((out.cpu(), lse.cpu()), want)
    _near(got, want)


@pytest.mark.parametrize("theta,scale", [(1e4, 1.0), (1e6, 4.0), (5e5, 0.5)])
def test_tree_attention_other_rope_constants(theta, scale, monkeypatch):
    import q8_ref
    c = ref.case(5, [90, 300], 9, 8, 2, ["tree"])
    got = _run(c, plan=_plan(c, rope_theta=theta, rope_scale=scale))
    monkeypatch.setattr(q8_ref, "_W", theta ** (-np.arange(0, 128, 2) / 128) / scale)
    _near(got, ref.attention(c))


def test_rows_are_bitwise_their_own():
    """Alone, among others, in another order, in a wider table, on other pages: the same bits."""
    lens = [0, 40, 700, 1100, 128, 3000, 17, 515]
    c = ref.case(11, lens, 12, 16, 2, ["tree", "forest", "chain"])
    whole = _run(c)
    assert _equal(whole, _run(c))
    for b in (0, 2, 5, 7):
        one = {k: v[b:b + 1].contiguous() if k in ("q", "block_table", "kv_lens", "parents") else v for k, v in c.items()}
        assert _equal([x[b:b + 1].contiguous() for x in whole], _run(one))
    order = torch.tensor([5, 1, 7, 0, 3, 2, 6, 4])
    mixed = {k: v[order].contiguous() if k in ("q", "block_table", "kv_lens", "parents") else v for k, v in c.items()}
    assert _equal([x[order].contiguous() for x in whole], _run(mixed))
    wide = dict(c)
    wide["block_table"] = torch.cat([c["block_table"], torch.full((8, 5000), -1, dtype=i32)], 1).contiguous()
    assert _equal(whole, _run(wide))
    move = torch.randperm(c["k_cache"].shape[0], generator=torch.Generator().manual_seed(1))
    back = torch.argsort(move)
    moved = dict(c)
    moved["k_cache"], moved["v_cache"] = c["k_cache"][back].contiguous(), c["v_cache"][back].contiguous()
    bt = c["block_table"].long()
    moved["block_table"] = torch.where(bt >= 0, move[bt.clamp(min=0)], bt).to(i32)
    assert _equal(whole, _run(moved))


@pytest.mark.parametrize("junk", [float("nan"), float("inf"), -float("inf"), 3.0e38])
def test_slots_that_nothing_sees_may_hold_anything(junk):
    lens, T = [5, 100, 131, 640], 11
    c = ref.case(13, lens, T, 8, 2, ["forest", "tree"])
    want = _run(c)
    d = dict(c)
    d["k_cache"], d["v_cache"] = c["k_cache"].clone(), c["v_cache"].clone()
    used = torch.zeros(c["k_cache"].shape[:2], dtype=torch.bool)
    for b, n in enumerate(lens):
        for t in range(n + T):
            if t < n or int(c["parents"][b, t - n]) != ref.UNUSED:
                used[int(c["block_table"][b, t // 16]), t % 16] = True
    d["k_cache"][~used] = junk
    d["v_cache"][~used] = junk
    st = torch.zeros(1, dtype=i32, device="cuda")
    assert _equal(want, _run(d, st)) and int(st.item()) == 0


@pytest.mark.parametrize("what,junk", [("k", float("nan")), ("k", 40000.0), ("v", float("inf")), ("v", float("nan")), ("k", -float("inf"))])
@pytest.mark.parametrize("n", [0, 3, 9])
def test_a_bad_node_fails_the_queries_that_see_it_and_no_other(what, junk, n):
    lens, T, row = [30, 250, 128], 10, 1
    c = ref.case(17, lens, T, 8, 4, ["tree"])
    want = _run(c)
    t, h = lens[row] + n, 2
    d = dict(c)
    d[what + "_cache"] = c[what + "_cache"].clone()
    d[what + "_cache"][int(c["block_table"][row, t // 16]), t % 16, h, 77] = junk
    st = torch.zeros(1, dtype=i32, device="cuda")
    got = _run(d, st)
    sees = torch.tensor([n in w for w in ref.ways(c["parents"][row].tolist())])
    hit = torch.zeros(want[1].shape, dtype=torch.bool)
    hit[row, 2 * h:2 * h + 2] = sees
    assert int(st.item()) == binding.STATUS_RANGE
    assert torch.isnan(got[1][hit]).all() and (got[0][hit] == 0).all()
    assert _equal([x[~hit] for x in want], [x[~hit] for x in got])


@pytest.mark.parametrize("junk", [float("nan"), 32768.0, float("inf")])
def test_a_bad_query_fails_alone_and_a_bad_prefix_key_its_head(junk):
    lens, T = [30, 250, 1300], 6
    c = ref.case(19, lens, T, 8, 4, ["tree"])
    want = _run(c)
    d = dict(c)
    d["q"] = c["q"].clone()
    d["q"][1, 5, 2, 127] = junk
    st = torch.zeros(1, dtype=i32, device="cuda")
    got = _run(d, st)
    hit = torch.zeros(want[1].shape, dtype=torch.bool)
    hit[1, 5, 2] = True
    assert int(st.item()) == binding.STATUS_RANGE
    assert torch.isnan(got[1][hit]).all() and (got[0][hit] == 0).all()
    assert _equal([x[~hit] for x in want], [x[~hit] for x in got])
    d = dict(c)
    d["k_cache"] = c["k_cache"].clone()
    d["k_cache"][int(c["block_table"][2, 777 // 16]), 777 % 16, 3, 5] = junk
    st.zero_()
    got = _run(d, st)
    hit[:] = False
    hit[2, 6:8] = True
    assert int(st.item()) == binding.STATUS_RANGE
    assert torch.isnan(got[1][hit]).all() and (got[0][hit] == 0).all()
    assert _equal([x[~hit] for x in want], [x[~hit] for x in got])


@pytest.mark.parametrize("what", ["page", "page_node", "kv_neg", "kv_short", "kv_wide", "parent_self", "parent_later", "parent_low",
                                  "parent_unused"])
def test_bad_metadata_fails_its_row_alone(what):
    lens, T, row = [30, 250, 700], 7, 1
    c = ref.case(23, lens, T, 8, 2, ["tree"])
    want = _run(c)
    d = {k: v.clone() for k, v in c.items()}
    bit = binding.STATUS_TREE
    if what == "page":
        d["block_table"][row, 3], bit = c["k_cache"].shape[0], binding.STATUS_PAGE_OOB
    elif what == "page_node":
        d["block_table"][row, (lens[row] + T - 1) // 16], bit = -1, binding.STATUS_PAGE_OOB
    elif what.startswith("kv"):
        d["kv_lens"][row], bit = {"kv_neg": -3, "kv_short": T - 1, "kv_wide": 16 * c["block_table"].shape[1] + 1}[what], binding.STATUS_KVLEN
    elif what == "parent_unused":
        d["parents"][row, 1], d["parents"][row, 2] = ref.UNUSED, 1
    else:
        d["parents"][row, 4] = {"parent_self": 4, "parent_later": 6, "parent_low": -3}[what]
    st = torch.zeros(1, dtype=i32, device="cuda")
    got = _run(d, st)
    assert int(st.item()) == bit
    assert torch.isnan(got[1][row]).all() and (got[0][row] == 0).all()
    others = [0, 2]
    assert _equal([x[others].contiguous() for x in want], [x[others].contiguous() for x in got])


def test_large_scores_and_tied_ones():
    """Scores to some thousands, and rows whose keys are all one key."""
    c = ref.case(29, [40, 300], 9, 8, 2, ["tree"])
    c["q"] = (c["q"].float() * 40).to(torch.bfloat16)
    c["k_cache"] = (c["k_cache"].float() * 30).to(torch.bfloat16)
    _near(_run(c), ref.attention(c))
    c["q"].zero_()
    got, want = _run(c), ref.attention(c)
    _near(got, want)
    d = {k: v.clone() for k, v in c.items()}
    d["k_cache"].zero_()
    assert np.allclose(_run(d)[1].numpy(), want[1], atol=1e-5)  # ln of the number of keys, whatever they are


def test_captured_step_replays_with_new_contents():
    a, b = (ref.case(s, lens, 6, 8, 2, ["tree", "forest"]) for s, lens in ((31, [100, 900, 2, 50]), (32, [700, 3, 260, 140])))
    W, NP = 80, max(x["k_cache"].shape[0] for x in (a, b))
    for x in (a, b):
        x["block_table"] = torch.cat([x["block_table"], torch.full((4, W - x["block_table"].shape[1]), -1, dtype=i32)], 1)
        for n in ("k_cache", "v_cache"):
            x[n] = torch.cat([x[n], torch.zeros((NP - x[n].shape[0],) + x[n].shape[1:], dtype=torch.bfloat16)])
    want = [_run(x) for x in (a, b)]
    dev = {k: v.cuda() for k, v in a.items()}
    p = _plan(a)
    out, lse = torch.empty_like(dev["q"]), torch.empty(a["q"].shape[:3], device="cuda")
    scratch = torch.empty(max(binding.tree_scratch_bytes(p), 16), dtype=torch.uint8, device="cuda")
    args = [dev[k] for k in ("q", "k_cache", "v_cache", "block_table", "kv_lens", "parents")]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        binding.attn_tree(p, *args, out, lse, scratch)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        binding.attn_tree(p, *args, out, lse, scratch)
    for i in (0, 1, 0):
        for k in dev:
            dev[k].copy_((a, b)[i][k])
        g.replay()
        torch.cuda.synchronize()
        assert _equal(want[i], (out.cpu(), lse.cpu()))


def test_tree_attention_on_another_stream():
    c = ref.case(37, [100, 800], 5, 8, 2, ["tree"])
    want = _run(c)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    assert _equal(want, _run(c, stream=s)) and _equal(want, _run(c, stream=s.cuda_stream))


def test_no_rows_and_rows_without_pages():
    p = binding.plan(0, 4, 8, 2, 128, 16, 5, 3)
    e = lambda *s, dt=torch.bfloat16: torch.empty(s, dtype=dt, device="cuda")  # noqa: E731
    cache = torch.zeros((5, 16, 2, 128), dtype=torch.bfloat16, device="cuda")
    binding.attn_tree(p, e(0, 8, 4, 128), cache, cache, e(0, 3, dt=i32), e(0, dt=i32), e(0, 4, dt=i32), e(0, 8, 4, 128),
                      e(0, 8, 4, dt=torch.float32))
    p = binding.plan(2, 4, 8, 2, 128, 16, 0, 0)
    out, lse = e(2, 8, 4, 128), e(2, 8, 4, dt=torch.float32)
    none = e(0, 16, 2, 128)
    n = binding.tree_scratch_bytes(p)
    binding.attn_tree(p, e(2, 8, 4, 128), none, none, e(2, 0, dt=i32), torch.zeros(2, dtype=i32, device="cuda"),
                      torch.tensor([[-1, 0, 1, 2]] * 2, dtype=i32, device="cuda"), out, lse, e(n, dt=torch.uint8) if n else None)
    assert (out == 0).all() and torch.isneginf(lse).all()


def test_offsets_past_32_bits():
    """Pages whose bytes start past 2^32 and whose elements start past 2^31."""
    Hkv, T = 8, 5
    NP = (1 << 31) // (16 * Hkv * 128) + 40
    c = ref.case(41, [37, 150], T, 16, Hkv, ["tree"])
    want = _run(c)
    small = c["k_cache"].shape[0]
    kc = torch.empty((NP, 16, Hkv, 128), dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    kc[-small:], vc[-small:] = c["k_cache"].cuda(), c["v_cache"].cuda()
    bt = torch.where(c["block_table"] >= 0, c["block_table"] + (NP - small), c["block_table"]).cuda()
    p = binding.plan(2, T, 16, Hkv, 128, 16, NP, bt.shape[1])
    out, lse = torch.empty(c["q"].shape, dtype=torch.bfloat16, device="cuda"), torch.empty(c["q"].shape[:3], device="cuda")
    n = binding.tree_scratch_bytes(p)
    binding.attn_tree(p, c["q"].cuda(), kc, vc, bt, c["kv_lens"].cuda(), c["parents"].cuda(), out, lse,
                      torch.empty(n, dtype=torch.uint8, device="cuda") if n else None)
    assert _equal(want, (out.cpu(), lse.cpu()))


@pytest.mark.parametrize("T,Hq,Hkv", [(5, 8, 2), (60, 8, 2), (40, 8, 1)])
def test_tree_attention_timeout_exit(T, Hq, Hkv):
    """A wait that nothing ends gives up: rows are written as failed, and a call after it is as before it."""
    c = ref.case(43, [300, -T, 2500, 40], T, Hq, Hkv, ["tree", "forest"])
    want = _run(c)
    p = _plan(c)
    p.wait_limit_ns, p.timeout_drill = 1, 1  # 1 us is the least limit that a launch takes
    st = torch.zeros(1, dtype=i32, device="cuda")
    out, lse = _run(c, st, plan=p)
    assert int(st.item()) & binding.STATUS_TIMEOUT
    assert (out == 0).all() and torch.isnan(lse[[0, 2, 3]]).all() and (torch.isnan(lse[1]) | torch.isneginf(lse[1])).all()
    st.zero_()
    assert _equal(want, _run(c, st)) and int(st.item()) == 0


@pytest.mark.parametrize("B,T,Hq,Hkv,hi", [(3000, 3, 4, 2, 40), (400, 20, 8, 1, 300), (1500, 1, 2, 2, 600)])
def test_many_rows_are_those_of_small_batches(B, T, Hq, Hkv, hi):
    r = np.random.RandomState(B)
    lens = [-T if x < 0.1 else int(n) for x, n in zip(r.rand(B), r.randint(0, hi + 1, B))]
    c = ref.case(B, lens, T, Hq, Hkv, ["tree", "forest", "chain"])
    st = torch.zeros(1, dtype=i32, device="cuda")
    whole = _run(c, st)
    assert int(st.item()) == 0
    for lo in range(0, B, max(1, B // 7)):
        part = {k: v[lo:lo + 9].contiguous() if k in ("q", "block_table", "kv_lens", "parents") else v for k, v in c.items()}
        assert _equal([x[lo:lo + 9].contiguous() for x in whole], _run(part))
    few = {k: v[-20:].contiguous() if k in ("q", "block_table", "kv_lens", "parents") else v for k, v in c.items()}
    _near([x[-20:] for x in whole], ref.attention(few))


def test_two_calls_at_once_and_two_graphs_with_one_scratch():
    """Calls on two streams with no order between them, each with its own scratch; two captured graphs that
    share a scratch and are replayed one after the other."""
    cases = [ref.case(61, [900, 30, 1500], 6, 8, 2, ["tree"]), ref.case(62, [2500, 1100], 20, 8, 4, ["tree", "star"])]
    want = [_run(c) for c in cases]
    plans = [_plan(c) for c in cases]
    need = [binding.tree_scratch_bytes(p) for p in plans]
    assert min(need) > 0
    dev = [{k: v.cuda() for k, v in c.items()} for c in cases]
    outs = [(torch.empty_like(d["q"]), torch.empty(d["q"].shape[:3], device="cuda")) for d in dev]

    def call(i, scratch):
        d = dev[i]
        binding.attn_tree(plans[i], d["q"], d["k_cache"], d["v_cache"], d["block_table"], d["kv_lens"], d["parents"], *outs[i], scratch)

    own = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in need]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(10):
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                call(i, own[i])
    torch.cuda.synchronize()
    for i in (0, 1):
        assert _equal(want[i], [x.cpu() for x in outs[i]])
    shared = torch.empty(max(need), dtype=torch.uint8, device="cuda")
    graphs = []
    for i in (0, 1):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(i, shared[:need[i]])
        graphs.append(g)
    for o in outs:
        o[0].zero_()
    for i in (0, 1, 1, 0, 1, 0):
        graphs[i].replay()
    torch.cuda.synchronize()
    for i in (0, 1):
        assert _equal(want[i], [x.cpu() for x in outs[i]])


@pytest.mark.parametrize("lens,T,Hq,Hkv", [([40, 1200], 3, 160, 160), ([70, 300, 9], 20, 640, 80), ([5], 64, 512, 64)])
def test_more_heads_than_a_grid_has_blocks(lens, T, Hq, Hkv):
    c = ref.case(67, lens, T, Hq, Hkv, ["tree", "chain"])
    _near(_run(c), ref.attention(c))
