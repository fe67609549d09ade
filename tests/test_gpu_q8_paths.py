"""GPU tests of the 8-bit cache operators where their paths part: the kernels' timeout
exit, steps large enough for the second form of a launch, caches past 32-bit offsets,
pages shared by rows, K's codes at any position, a captured serving step, and two
captured graphs in flight."""
import numpy as np
import pytest
import torch

import q8_ref as ref
import test_gpu_q8_attention as att
import test_gpu_q8_tables_append as tab
from deterministic_paged_kv_gb300 import binding

pytestmark = pytest.mark.gpu

i32 = torch.int32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from deterministic_paged_kv_gb300 import build
    build.build()
    binding.load()


# ------------------------------------------------------------- timeout exit ----

@pytest.mark.parametrize("mode,split,heads", [("decode", 0, (32, 8)), ("decode", 1 << 20, (8, 1)), ("decode", 0, (8, 2)),
                                              ("prefill", 0, (8, 2))])
def test_q8_timeout_exit(mode, split, heads):
    """A wait that nothing ends gives up: rows are written as failed, and a call after it is as before it."""
    c = ref.case(51, [300, 77, 2500], *heads, Sq=1 if mode == "decode" else 70)
    want = att._run(c, split)
    p = att._plan(c)
    p.wait_limit_ns, p.timeout_drill = 1, 1  # 1 us is the least limit that a launch takes
    st = torch.zeros(1, dtype=i32, device="cuda")
    out, lse = att._run(c, split, status=st, plan=p)
    assert int(st.item()) & binding.STATUS_TIMEOUT
    assert (out == 0).all() and torch.isnan(lse).all()
    st.zero_()
    assert att._equal(want, att._run(c, split, status=st)) and int(st.item()) == 0


# ------------------------------------------------------------------- tables ----

@pytest.mark.parametrize("B,lens,new,cap", [
    (1, (0, 0), (9000, 9000), 9000), (300, (0, 500), (0, 60), 20000), (2000, (1, 40), (1, 9), 18001),
    (40, (100, 100), (400, 400), 16003), (5, (3, 90), (0, 0), 4097)])
@pytest.mark.parametrize("inplace", [False, True])
def test_tables_extend_large_steps(B, lens, new, cap, inplace):
    """Steps of more than 4096 tokens' room, some longer than the room or the pool."""
    lens, new, bt, pool, NP = tab._tables_case(B, lens, new, 7 * B + inplace)
    offset = 0 if inplace else 3
    got = tab._extend(lens, new, bt, pool, NP, cap, inplace=inplace, offset=offset)
    tab._same(got, ref.tables(new, lens, pool, 0, bt, cap, NP))
    # a pool that ends too early, a bad row, a bad page id
    if B > 1:
        lens, new, bt, pool = lens.copy(), new.copy(), bt.copy(), pool.copy()
        lens[B // 2], new[B // 3] = -1, -5
        pool[len(pool) // 4:len(pool) // 4 + 1] = NP
        few = pool[:max(1, len(pool) // 2)]
        got = tab._extend(lens, new, bt, few, NP, cap, taken=min(1, len(few)), inplace=inplace)
        tab._same(got, ref.tables(new, lens, few, min(1, len(few)), bt, cap, NP))


# ------------------------------------------------------------------- append ----

@pytest.mark.parametrize("Hkv", [2, 8])
def test_append_q8_many_tokens(Hkv):
    """Enough tokens for four warps to a window, against a call per token (a warp each) and 64 bits."""
    r = np.random.RandomState(5)
    runs = [(int(r.randint(0, 40)), int(n)) for n in r.randint(1, 90, 30)] + [(0, 16), (0, 128), (15, 17)]
    c = tab._append_case(90 + Hkv, runs, Hkv)
    n = len(c["slots"])
    assert n * Hkv >= 152 * 16
    whole = tab._dev(c)
    tab._append(c, whole)
    parts = tab._dev(c)
    for lo in range(0, n, 7):
        tab._append(c, parts, lo, min(n, lo + 7))
    assert all(torch.equal(a, b) for a, b in zip(tab._bits(whole), tab._bits(parts)))
    v = ref.Cache(c["codes"][1], c["scale"][1])
    v.append(c["new"][1].double().numpy(), c["new"][1].double().numpy(), c["slots"])
    assert np.array_equal(whole[3].cpu().double().numpy(), np.ldexp(1.0, v.exp))
    assert np.array_equal(whole[1].cpu().to(torch.float32).double().numpy(), v.code)


def test_append_q8_k_codes_are_those_of_the_real_number():
    """A token to a page at positions up to 131071.  The angle of the 64-bit statement is off by at
    most 2^17 2^-52 (its product and the rate's own rounding), the kernel's result by less, so only
    codes within 2^-34 of the pair's length of a border may differ; some one in 2^30 are."""
    n, Hkv = 700, 8
    g = torch.Generator().manual_seed(3)
    x = torch.randn((n, Hkv, 128), generator=g).to(torch.bfloat16)
    pos = torch.randint(0, 131072, (n,), generator=g, dtype=i32)
    pos[:3] = torch.tensor([0, 1, 131071], dtype=i32)
    kc = torch.zeros((n, Hkv, 16, 128), dtype=torch.uint8, device="cuda").view(ref.F8)
    vc = kc.clone()
    ks, vs = torch.ones((n, Hkv), device="cuda"), torch.ones((n, Hkv), device="cuda")
    p = binding.plan(1, 1, Hkv, Hkv, 128, 16, n, 1)
    slots = (torch.arange(n, dtype=i32) * 16).cuda()
    binding.kv_append_q8(p, x.cuda(), x.cuda(), slots, pos.cuda(), kc, vc, ks, vs)
    xd = x.double().numpy()
    y = ref.rotate(xd, pos.numpy()[:, None])
    e = np.maximum(np.frexp(np.abs(xd).max(-1))[1] - 8, ref.E_MIN)[..., None]
    length = np.sqrt(xd[..., :64] ** 2 + xd[..., 64:] ** 2)
    d = np.ldexp(np.concatenate([length, length], -1), -e) * 2.0 ** -34
    y = np.ldexp(y, -e)
    got = kc[:, :, 0].cpu().to(torch.float32).double().numpy()
    assert ((got == ref.round4(y - d)) | (got == ref.round4(y + d))).all()
    # at position 0 the values are the bf16 inputs (8 bits, one in 16 of them half-way between two
    # codes) and stay what they are; elsewhere hardly any value is next to a border
    assert np.array_equal(got[0], ref.round4(y[0]))
    assert (ref.round4(y - d) != ref.round4(y + d))[1:].sum() <= 3


# ---------------------------------------------------------------- attention ----

def test_decode_q8_does_not_depend_on_the_merge():
    """A table so wide that long rows' merge runs (quarters of a row), and one of few splits."""
    c = ref.case(61, [5000, 33, 1300], 8, 2)
    want = att._run(c)
    att._check(c, want, att.DECODE)
    rows = [0, 1, 2]
    assert att._equal(want, att._run(att._rows(c, rows, 2500)))
    for split in (16, 48):  # more than 32 splits either way: five thousand keys in each
        assert att._equal(att._run(c, split), att._run(att._rows(c, rows, 700), split))


def test_decode_q8_largest_split():
    c = ref.case(67, [700, 0, 33, 1], 8, 2)
    want = att._run(c, 1 << 20)
    st = torch.zeros(1, dtype=i32, device="cuda")
    assert att._equal(want, att._run(c, 2 ** 31 - 16, status=st)) and int(st.item()) == 0


@pytest.mark.parametrize("mode", ["decode", "prefill"])
def test_q8_rows_share_pages(mode):
    c = ref.case(63, [600, 64, 350], 8, 2, Sq=1 if mode == "decode" else 40)
    want = att._run(c)
    d = att._rows(c, [0, 0, 2, 0])  # the same pages and queries in several rows
    got = att._run(d)
    assert att._equal(got, [x[[0, 0, 2, 0]] for x in want])


@pytest.mark.parametrize("mode", ["append", "decode", "prefill"])
def test_q8_cache_past_32_bit_offsets(mode):
    """Pages at the end of a cache of 4.9 GB give what the same pages give at its start."""
    Hq, Hkv, NP = 16, 8, 300000
    c = ref.case(65, [300, 45], Hq, Hkv, Sq=1 if mode == "decode" else 33)
    n, at = c["k_cache"].shape[0], NP - c["k_cache"].shape[0]
    assert at * Hkv * 2048 > 2 ** 32
    big = []
    for name in ("k_cache", "v_cache"):
        t = torch.empty((NP, Hkv, 16, 128), dtype=torch.uint8, device="cuda")
        t[at:] = c[name].view(torch.uint8).cuda()
        big.append(t.view(ref.F8))
    for name in ("k_scale", "v_scale"):
        t = torch.empty((NP, Hkv), device="cuda")
        t[at:] = c[name].cuda()
        big.append(t)
    if mode == "append":
        g = torch.Generator().manual_seed(1)
        x = torch.randn((2, 40, Hkv, 128), generator=g).to(torch.bfloat16).cuda()
        page = c["block_table"][0, :3].tolist()
        slots = [page[t // 16] * 16 + t % 16 for t in range(4, 44)]
        small = [c[k].cuda() for k in ("k_cache", "v_cache", "k_scale", "v_scale")]
        for cache, first, pages in ((small, 0, n), (big, at, NP)):
            p = binding.plan(1, 1, Hkv, Hkv, 128, 16, pages, 1)
            binding.kv_append_q8(p, x[0], x[1], tab._t([s + first * 16 for s in slots]), tab._t(range(4, 44)), *cache)
        for s, b in zip(small, big):
            assert torch.equal(s.view(torch.uint8), b[at:].view(torch.uint8))
        return
    want = att._run(c)
    o = dict(c)
    o["block_table"] = torch.where(c["block_table"] >= 0, c["block_table"] + at, c["block_table"]).to(i32)
    d = [o["q"].cuda(), *big, *[o[k].cuda() for k in ("block_table", "kv_lens", "position_ids")]]
    p = binding.plan(2, c["q"].shape[2], Hq, Hkv, 128, 16, NP, c["block_table"].shape[1])
    assert att._equal(want, att._run(o, plan=p, d=d))


@pytest.mark.parametrize("split", [0, 16, 128, 1 << 20])
@pytest.mark.parametrize("Hq,Hkv", [(8, 8), (32, 8), (16, 2), (3, 3)])
def test_decode_q8_nan_codes(split, Hq, Hkv):
    """A NaN code in one dim of one token fails that KV head's queries of that row in all dims, and nothing else."""
    G = Hq // Hkv
    lens = [900, 40, 17, 300, 1, 513] * 8
    c = ref.case(81, lens, Hq, Hkv)
    want = att._run(c, split)
    r = np.random.RandomState(split % 1000 + Hq)
    hit = set()
    for n in ("k_cache", "v_cache"):
        for b in r.permutation(len(lens))[:12]:
            h, t = int(r.randint(Hkv)), int(r.choice([0, lens[b] - 1, r.randint(lens[b])]))
            c[n].view(torch.uint8)[c["block_table"][b, t // 16].long(), h, t % 16, r.randint(128)] = r.choice([0x7F, 0xFF])
            hit.add((int(b), h))
    st = torch.zeros(1, dtype=i32, device="cuda")
    out, lse = att._run(c, split, status=st)
    assert int(st.item()) == binding.STATUS_RANGE
    for b in range(len(lens)):
        for h in range(Hkv):
            x, y = out[b, h * G:(h + 1) * G], lse[b, h * G:(h + 1) * G]
            if (b, h) in hit:
                assert (x == 0).all() and torch.isnan(y).all(), (b, h)
            else:
                assert torch.equal(x, want[0][b, h * G:(h + 1) * G]) and torch.equal(y, want[1][b, h * G:(h + 1) * G]), (b, h)


# ----------------------------------------------------------- captured graphs ----

class _Server:
    """Rows that decode: a step is tables, append and attention, all on the device."""

    def __init__(self, seed, B=6, Hq=8, Hkv=2, W=30, NP=200, lens=(3, 90, 15, 16, 200, 31)):
        g = torch.Generator().manual_seed(seed)
        self.p = binding.plan(B, 1, Hq, Hkv, 128, 16, NP, W)
        c = ref.case(seed, list(lens), Hq, Hkv, W=W, extra=NP - sum(-(-n // 16) for n in lens))
        self.cache = [c[n].cuda() for n in ("k_cache", "v_cache", "k_scale", "v_scale")]
        self.table, self.lens = c["block_table"].cuda(), c["kv_lens"].cuda()
        used = set(c["block_table"][c["block_table"] >= 0].tolist())
        self.pool = torch.tensor([x for x in torch.randperm(NP, generator=g).tolist() if x not in used], dtype=i32).cuda()
        self.taken, self.one = torch.zeros(1, dtype=i32, device="cuda"), torch.ones(B, dtype=i32, device="cuda")
        self.ip = torch.empty(B + 1, dtype=i32, device="cuda")
        self.pos, self.slot = torch.empty(B, dtype=i32, device="cuda"), torch.empty(B, dtype=i32, device="cuda")
        new = torch.randn((2, B, Hkv, 128), generator=g).to(torch.bfloat16).cuda()
        self.k, self.v = new[0], new[1]
        self.q = torch.randn((B, Hq, 1, 128), generator=g).to(torch.bfloat16).cuda()
        self.out, self.lse = torch.zeros_like(self.q), torch.zeros((B, Hq, 1), device="cuda")
        self.status = torch.zeros(1, dtype=i32, device="cuda")
        self.scratch = torch.empty(binding.decode_q8_scratch_bytes(self.p, 16), dtype=torch.uint8, device="cuda")

    def step(self, stream=None):
        binding.tables_extend(self.p, self.one, self.lens, self.pool, self.taken, self.table, self.lens, self.taken, self.ip,
                              self.pos, self.slot, status=self.status, stream=stream)
        binding.kv_append_q8(self.p, self.k, self.v, self.slot, self.pos, *self.cache, status=self.status, stream=stream)
        binding.attn_decode_q8(self.p, self.q, *self.cache, self.table, self.lens, self.pos.view(-1, 1), self.out, self.lse,
                               self.scratch, split_tokens=16, status=self.status, stream=stream)

    def state(self):
        torch.cuda.synchronize()
        return [x.clone().view(torch.uint8) for x in (self.out, self.lse, self.lens, self.taken, self.table, *self.cache)]


def test_q8_captured_steps_on_two_streams():
    """Two servers' steps, each captured once and replayed on its own stream at the same time, end
    where eager steps end (a step leaves the caches, lengths and tables of the next)."""
    steps = 25
    eager = [_Server(s) for s in (71, 72)]
    for e in eager:
        for _ in range(steps):
            e.step()
    ours = [_Server(s) for s in (71, 72)]
    streams, graphs = [torch.cuda.Stream(), torch.cuda.Stream()], []
    torch.cuda.synchronize()
    for o, s in zip(ours, streams):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            o.step()
        graphs.append(graph)
    for _ in range(steps):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    for e, o in zip(eager, ours):
        assert int(e.status.item()) == 0 and int(o.status.item()) == 0
        assert all(torch.equal(a, b) for a, b in zip(e.state(), o.state()))


def test_q8_calls_take_the_streams_order():
    """A call on a side stream waits for what that stream waits for, and on nothing else's order."""
    c = ref.case(75, [700, 33], 8, 2)
    want = att._run(c)
    d = [c[n].cuda() for n in ref.NAMES]
    keep = d[0].clone()
    p = att._plan(c)
    out, lse = torch.zeros_like(d[0]), torch.zeros(c["q"].shape[:3], device="cuda")
    n = binding.decode_q8_scratch_bytes(p)
    scratch = torch.empty(max(16, n), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    d[0].zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(2000000)
        d[0].copy_(keep)
    binding.attn_decode_q8(p, *d, out, lse, scratch, stream=side)
    side.synchronize()
    assert att._equal(want, (out, lse))
