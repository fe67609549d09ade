"""GPU tests of serving steps over the 8-bit cache whose rows get different numbers of tokens:
the tables in both their forms, captured and replayed, and what the append and the attention
calls make of them."""
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


@pytest.mark.parametrize("cap", [300, 4096, 4097, 20000])
def test_tables_extend_captured_ragged_steps(cap):
    """One launch (up to 4096 tokens' room) and two: a captured step of ragged rows, replayed with
    new counts, goes on in place from the step before."""
    r = np.random.RandomState(cap)
    B, W, steps = 30, 40, 6
    counts = r.randint(0, 10 if cap == 300 else 60, (steps, B))
    lens = r.randint(0, 60, B)
    NP = 900
    perm = r.permutation(NP)
    bt, at = np.full((B, W), -1), 0
    for b in range(B):
        n = -(-lens[b] // 16)
        bt[b, :n] = perm[at:at + n]
        at += n
    pool = perm[at:]
    p = binding.plan(B, 1, 8, 8, 128, 16, NP, W)
    kv, tk, table, n, pl = tab._t(lens), tab._t([0]), tab._t(bt), tab._t([0] * B), tab._t(pool)
    ip, pos, slot = tab._t([0] * (B + 1)), tab._t([0] * cap), tab._t([0] * cap)
    st = torch.zeros(1, dtype=i32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        binding.tables_extend(p, n, kv, pl, tk, table, kv, tk, ip, pos, slot, status=st)
    t = 0
    for k in range(steps):
        n.copy_(tab._t(counts[k]))
        pos.fill_(7)
        slot.fill_(7)
        g.replay()
        want, said = ref.tables(counts[k], lens, pool, t, bt, cap, NP)
        assert said == set()
        lens, t, bt = np.array(want["kv_lens"]), want["taken"], want["block_table"]
        assert kv.tolist() == list(lens) and tk.tolist() == [t] and ip.tolist() == want["qo_indptr"]
        assert pos.tolist() == want["position_ids"] and slot.tolist() == want["slot_map"]
        assert np.array_equal(table.cpu().numpy(), bt)
    assert int(st.item()) == 0


@pytest.mark.parametrize("room", [400, 5000])
@pytest.mark.parametrize("captured", [False, True])
def test_q8_ragged_steps(room, captured):
    """Admission, chunks and single tokens in one step: tables, append and attention (each row's
    queries padded to the longest, behind its last token), against 64 bits on the cache as it is and
    against the tokens themselves."""
    g = torch.Generator().manual_seed(room)
    Hq, Hkv, W, NP, Sq = 8, 2, 30, 140, 90
    steps = [(90, 3, 0, 37, 16), (1, 61, 70, 1, 16), (17, 1, 1, 0, 90), (1, 1, 1, 1, 1)]
    B = 5
    p = binding.plan(B, Sq, Hq, Hkv, 128, 16, NP, W)
    pool = torch.randperm(NP, generator=g).to(i32).cuda()
    taken, lens = torch.zeros(1, dtype=i32, device="cuda"), torch.zeros(B, dtype=i32, device="cuda")
    table = torch.full((B, W), -1, dtype=i32, device="cuda")
    cache = [torch.full((NP, Hkv, 16, 128), 0x7F, dtype=torch.uint8, device="cuda").view(ref.F8) for _ in range(2)]
    cache += [torch.full((NP, Hkv), float("nan"), device="cuda") for _ in range(2)]
    n_new, ip = torch.zeros(B, dtype=i32, device="cuda"), torch.zeros(B + 1, dtype=i32, device="cuda")
    pos, slot = (torch.zeros(room, dtype=i32, device="cuda") for _ in range(2))
    new = torch.zeros((2, room, Hkv, 128), dtype=torch.bfloat16, device="cuda")
    qpos = torch.zeros((B, Sq), dtype=i32, device="cuda")
    q = torch.zeros((B, Hq, Sq, 128), dtype=torch.bfloat16, device="cuda")
    out, lse = torch.zeros_like(q), torch.zeros((B, Hq, Sq), device="cuda")
    st = torch.zeros(1, dtype=i32, device="cuda")
    ahead = torch.arange(Sq, dtype=i32, device="cuda")

    def step(stream=None):
        torch.add(lens[:, None], ahead, out=qpos)  # a row's queries start behind its tokens so far
        binding.tables_extend(p, n_new, lens, pool, taken, table, lens, taken, ip, pos, slot, status=st, stream=stream)
        binding.kv_append_q8(p, new[0], new[1], slot, pos, *cache, status=st, stream=stream)
        binding.attn_prefill_q8(p, q, *cache, table, lens, qpos, out, lse, status=st, stream=stream)

    graph = torch.cuda.CUDAGraph()
    if captured:
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(graph, stream=s):
            step()
    tokens = [[] for _ in range(B)]
    for counts in steps:
        n_new.copy_(torch.tensor(counts, dtype=i32))
        new.copy_(torch.randn(new.shape, generator=g).to(torch.bfloat16))
        q.copy_(torch.randn(q.shape, generator=g).to(torch.bfloat16))
        graph.replay() if captured else step()
        torch.cuda.synchronize()
        at = 0
        for b, n in enumerate(counts):
            tokens[b] += [new[:, at + i].cpu() for i in range(n)]
            at += n
        assert lens.tolist() == [len(x) for x in tokens] and (slot[at:] == -1).all()
        c = {k: v.cpu() for k, v in zip(ref.NAMES, (q, *cache, table, lens, qpos))}
        for b, n in enumerate(counts):
            if n == 0:
                continue
            one = {k: (v[b:b + 1] if k in ("block_table", "kv_lens") else v) for k, v in c.items()}
            one["q"], one["position_ids"] = c["q"][b:b + 1, :, :n], c["position_ids"][b:b + 1, :n]
            att._check(one, (out[b:b + 1, :, :n], lse[b:b + 1, :, :n]), att.PREFILL)
        for b in range(B):  # every code within half a step of its token (e4m3: 2^-4 of it)
            for t, x in enumerate(tokens[b]):
                pg = int(c["block_table"][b, t // 16])
                k = ref.rotate(x[0].double().numpy(), t)
                for i, y in ((0, torch.from_numpy(k)), (1, x[1].double())):
                    sc = c[("k_scale", "v_scale")[i]][pg][:, None].double()
                    val = c[("k_cache", "v_cache")[i]].to(torch.float32)[pg, :, t % 16].double() * sc
                    assert ((val - y).abs() <= 2.0 ** -4 * y.abs() * (1 + 2.0 ** -30) + 2.0 ** -6 * sc).all()
    assert int(st.item()) == 0


@pytest.mark.parametrize("theta,scale", [(1e4, 1.0), (5e5, 8.0), (1e6, 0.5)])
def test_q8_rope_constants(theta, scale):
    """Append, decode and prefill rotate by the plan's constants, not by the usual ones."""
    g = torch.Generator().manual_seed(9)
    n, Hq, Hkv = 150, 4, 2
    w = theta ** (-np.arange(0, 128, 2) / 128) / scale
    turn = lambda x, pos: np.concatenate([(z := (x[..., :64] + 1j * x[..., 64:]) * np.exp(1j * np.asarray(pos, np.float64)[..., None] * w)).real,  # noqa: E731
                                          z.imag], -1)
    k, v = (torch.randn((n, Hkv, 128), generator=g).to(torch.bfloat16) for _ in range(2))
    q = torch.randn((1, Hq, n, 128), generator=g).to(torch.bfloat16)
    table = torch.randperm(12, generator=g).to(i32)[:10].view(1, 10).cuda()
    pos = torch.arange(n, dtype=i32).cuda()
    cache = [torch.zeros((12, Hkv, 16, 128), dtype=torch.uint8, device="cuda").view(ref.F8) for _ in range(2)]
    cache += [torch.ones((12, Hkv), device="cuda") for _ in range(2)]
    slot = (table[0, pos.long() // 16] * 16 + pos % 16).to(i32)
    kv = tab._t([n])
    st = torch.zeros(1, dtype=i32, device="cuda")
    plan = lambda Sq: binding.plan(1, Sq, Hq, Hkv, 128, 16, 12, 10, rope_theta=theta, rope_scale=scale)  # noqa: E731
    binding.kv_append_q8(plan(1), k.cuda(), v.cuda(), slot, pos, *cache, status=st)
    out, lse = torch.empty_like(q).cuda(), torch.empty((1, Hq, n), device="cuda")
    binding.attn_prefill_q8(plan(n), q.cuda(), *cache, table, kv, pos.view(1, n), out, lse, status=st)
    one, one_l = torch.empty((1, Hq, 1, 128), dtype=torch.bfloat16, device="cuda"), torch.empty((1, Hq, 1), device="cuda")
    binding.attn_decode_q8(plan(1), q[:, :, -1:].contiguous().cuda(), *cache, table, kv, pos[-1:].view(1, 1), one, one_l, status=st)
    assert int(st.item()) == 0
    pg = table[0].long().cpu()
    kc, vc = ((c.cpu().float()[pg] * s.cpu()[pg][..., None, None]).double().transpose(1, 2).reshape(-1, Hkv, 128)[:n].numpy()
              for c, s in ((cache[0], cache[2]), (cache[1], cache[3])))
    y = turn(k.double().numpy(), np.arange(n)[:, None])
    sc = cache[2].cpu()[pg].double().numpy().repeat(16, 0)[:n, :, None]
    assert (np.abs(kc - y) <= 2.0 ** -4 * np.abs(y) * (1 + 2.0 ** -30) + 2.0 ** -6 * sc).all()
    for h in range(Hq):
        r = turn(q[0, h].double().numpy(), np.arange(n))
        x = r @ kc[:, h // 2].T / np.sqrt(128)
        x[np.triu_indices(n, 1)] = -np.inf
        p = np.exp(x - x.max(-1, keepdims=True))
        want = p @ vc[:, h // 2] / p.sum(-1, keepdims=True)
        pair = np.tile(np.hypot(q[0, h, :, :64].double().numpy(), q[0, h, :, 64:].double().numpy()), 2)
        d = 2.0 ** -11 * 1.1 * (pair @ np.abs(kc[:, h // 2]).T / np.sqrt(128)).max(-1)[:, None]
        bound = 2.0 ** -8 * np.abs(want) + (2 * d + 2.0 ** -10) * np.abs(vc).max() + 1e-30
        assert (np.abs(out[0, h].double().cpu().numpy() - want) <= bound).all()
        assert (np.abs(one[0, h, 0].double().cpu().numpy() - want[-1]) <= bound[-1]).all()


@pytest.mark.parametrize("mode", ["decode", "prefill"])
@pytest.mark.parametrize("NP,W", [(0, 0), (0, 3), (5, 0)])
def test_q8_attention_without_pages_or_table(mode, NP, W):
    """No pool, no table: empty rows are empty, rows that claim tokens fail."""
    Sq = 1 if mode == "decode" else 3
    p = binding.plan(2, Sq, 4, 2, 128, 16, NP, W)
    q = torch.randn((2, 4, Sq, 128), device="cuda").to(torch.bfloat16)
    cache = [torch.zeros((NP, 2, 16, 128), dtype=torch.uint8, device="cuda").view(ref.F8) for _ in range(2)]
    cache += [torch.ones((NP, 2), device="cuda") for _ in range(2)]
    st = torch.zeros(1, dtype=i32, device="cuda")
    out, lse = torch.full_like(q, 3), torch.full((2, 4, Sq), 3.0, device="cuda")
    f = binding.attn_decode_q8 if mode == "decode" else binding.attn_prefill_q8
    f(p, q, *cache, torch.full((2, W), -1, dtype=i32, device="cuda"), tab._t([0, 5]), torch.zeros((2, Sq), dtype=i32, device="cuda"),
      out, lse, status=st)
    assert int(st.item()) == (binding.STATUS_PAGE_OOB if W else binding.STATUS_KVLEN)
    assert (out == 0).all() and torch.isneginf(lse[0]).all() and torch.isnan(lse[1]).all()
