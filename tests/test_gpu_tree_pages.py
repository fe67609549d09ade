"""GPU tests of rk_paged_kv_compact and rk_paged_tables_trim, and of a speculative step from the tables to
the trimmed tables, captured and replayed."""
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


def _dev(x):
    return torch.as_tensor(np.array(x), dtype=i32).cuda()


# ---------------------------------------------------------------- compact ----

def _paths(seed, B, T, keep):
    r = np.random.RandomState(seed)
    n = [int(r.randint(0, min(T, keep) + 1)) for _ in range(B)]
    rows = [sorted(r.choice(T, k, replace=False).tolist()) + [-9] * (T - k) for k in n]
    return np.array(rows, np.int32).reshape(B, T), np.array(n, np.int32)


def _compact(c, T, path, n_keep, status=None):
    k, v = c["k_cache"].cuda(), c["v_cache"].cuda()
    p = binding.plan(len(n_keep), T, k.shape[2], k.shape[2], 128, 16, k.shape[0], c["block_table"].shape[1])
    binding.kv_compact(p, _dev(path), _dev(n_keep), c["block_table"].cuda(), c["kv_lens"].cuda(), k, v, status=status)
    return k.cpu(), v.cpu()


def _same(a, b):
    return all(torch.equal(x.view(torch.int16), y.view(torch.int16)) for x, y in zip(a, b))


@pytest.mark.parametrize("lens,T,Hkv,keep", [([0], 1, 1, 1), ([3, 15, 16, 100], 8, 8, 8), ([0, 1, 17, 31, 250] * 8, 64, 2, 64),
                                             ([40, 41, 42], 64, 16, 64), ([5, 700], 33, 1, 7), ([9] * 200, 5, 4, 5), ([77, 3], 16, 24, 16)])
def test_compact_moves_the_path(lens, T, Hkv, keep):
    c = ref.case(len(lens) + T, lens, T, Hkv, Hkv, ["tree"])
    # bit patterns of every kind: NaN, infinities, -0
    for n in ("k_cache", "v_cache"):
        c[n] = torch.randint(-32768, 32768, c[n].shape, dtype=torch.int16, generator=torch.Generator().manual_seed(T)).view(torch.bfloat16)
    path, n = _paths(T, len(lens), T, keep)
    st = torch.zeros(1, dtype=i32, device="cuda")
    assert _same(_compact(c, T, path, n, st), ref.compact(c, T, path, n)) and int(st.item()) == 0


@pytest.mark.parametrize("what", ["same", "down", "neg", "past", "n_neg", "n_big", "kv", "kv_wide", "page", "page_to"])
def test_compact_leaves_bad_rows_alone(what):
    lens, T, row = [30, 44, 60], 9, 1
    c = ref.case(3, lens, T, 2, 2, ["tree"])
    path = np.array([[0, 2, 5, 8, -1, -1, -1, -1, -1]] * 3, np.int32)
    n = np.array([4, 4, 3], np.int32)
    good = np.array([4, 0, 3], np.int32)
    want = ref.compact(c, T, path, good)
    bit = binding.STATUS_TREE
    if what in ("same", "down", "neg", "past"):
        path[row, 2] = {"same": 2, "down": 1, "neg": -1, "past": T}[what]
    elif what.startswith("n_"):
        n[row] = -1 if what == "n_neg" else T + 1
    elif what.startswith("kv"):
        c["kv_lens"][row], bit = T - 1 if what == "kv" else 16 * c["block_table"].shape[1] + 1, binding.STATUS_KVLEN
    else:
        c["block_table"][row, (lens[row] + (8 if what == "page" else 0)) // 16] = -1 if what == "page" else c["k_cache"].shape[0]
        bit = binding.STATUS_PAGE_OOB
    st = torch.zeros(1, dtype=i32, device="cuda")
    assert _same(_compact(c, T, path, n, st), want) and int(st.item()) == bit


# ------------------------------------------------------------------- trim ----

def _tables(seed, B, len_hi, extra=2):
    r = np.random.RandomState(seed)
    lens = r.randint(0, len_hi + 1, B)
    need = -(-lens // 16)
    NP = int(need.sum()) + 9
    W = int(need.max()) + extra
    perm = r.permutation(NP).astype(np.int32)
    bt = np.full((B, W), -1, np.int32)
    at = 0
    for b in range(B):
        bt[b, :need[b]] = perm[at:at + need[b]]
        at += need[b]
    return lens.astype(np.int32), bt, r.permutation(NP).astype(np.int32), at, NP, r


def _trim(drop, lens, pool, taken, bt, NP, inplace):
    st = torch.zeros(1, dtype=i32, device="cuda")
    d = [_dev(x) for x in (drop, lens, pool, [taken], bt)]
    lo, to = (d[1], d[3]) if inplace else (torch.empty_like(d[1]), torch.empty_like(d[3]))
    p = binding.plan(len(lens), 1, 8, 8, 128, 16, NP, bt.shape[1])
    binding.tables_trim(p, d[0], d[1], d[2], d[3], d[4], lo, to, status=st)
    return {"block_table": d[4].cpu().numpy(), "kv_lens": lo.tolist(), "pool": d[2].cpu().numpy(), "taken": int(to.item())}, int(st.item())


def _agree(got, want):
    bits = {"kvlen": binding.STATUS_KVLEN, "pool": binding.STATUS_POOL, "oob": binding.STATUS_PAGE_OOB}
    for k in want[0]:
        assert np.array_equal(np.asarray(got[0][k]), np.asarray(want[0][k])), k
    assert got[1] == sum(bits[s] for s in want[1])


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("B,len_hi,drop_hi", [(1, 0, 0), (1, 5, 5), (1, 5000, 5000), (3, 40, 8), (64, 8000, 64), (100, 300, 300), (1024, 2000, 2000),
                                             (1025, 90, 20), (3000, 40, 40), (16384, 33, 33)])
def test_trim_against_rows_one_by_one(B, len_hi, drop_hi, inplace):
    lens, bt, pool, taken, NP, r = _tables(B + len_hi, B, len_hi)
    drop = np.minimum(lens, r.randint(0, drop_hi + 1, B)).astype(np.int32)
    _agree(_trim(drop, lens, pool, taken, bt, NP, inplace), ref.trim(drop, lens, pool, taken, bt, NP))
    _agree(_trim(lens, lens, pool, taken, bt, NP, inplace), ref.trim(lens, lens, pool, taken, bt, NP))  # all of it
    # refusals of every kind at once, and a pool that has handed out less than comes back
    if B >= 3:
        lens, drop, bt = lens.copy(), drop.copy(), bt.copy()
        lens[0], drop[B // 2], drop[B - 1] = -4, -1, lens[B - 1] + 1
        for few in (taken, taken // 3, 0, -1, NP + 1):
            _agree(_trim(drop, lens, pool, few, bt, NP, inplace), ref.trim(drop, lens, pool, few, bt, NP))
        lens[1] = 16 * bt.shape[1] + 1
        _agree(_trim(drop, lens, pool, taken, bt, NP, inplace), ref.trim(drop, lens, pool, taken, bt, NP))


def test_trim_of_a_freed_row_says_so():
    lens, bt, pool, taken, NP, _ = _tables(5, 4, 100)
    lens[:] = [40, 50, 60, 70]
    bt[:, :5] = np.arange(20).reshape(4, 5) % NP
    bt[2] = -1
    bt[3, 2] = NP
    got, want = _trim(lens, lens, pool, 20, bt, NP, False), ref.trim(lens, lens, pool, 20, bt, NP)
    _agree(got, want)
    assert got[1] == binding.STATUS_PAGE_OOB


def test_trim_without_rows_or_pages():
    p = binding.plan(0, 1, 8, 8, 128, 16, 4, 3)
    e = torch.empty(0, dtype=i32, device="cuda")
    taken, out = _dev([2]), _dev([9])
    binding.tables_trim(p, e, e, _dev([0, 1, 2, 3]), taken, e.view(0, 3), e, out)
    assert int(out.item()) == 2


def test_extend_then_trim_leaves_the_tables_as_they_were():
    lens, bt, pool, taken, NP, r = _tables(8, 50, 400, extra=6)
    held = set(bt[bt >= 0].tolist())
    pool = np.array([x for x in range(NP) if x in held] + [x for x in r.permutation(NP) if x not in held], np.int32)
    new = np.minimum(r.randint(0, 3, 50), 1).astype(np.int32)
    p = binding.plan(50, 1, 8, 8, 128, 16, NP, bt.shape[1])
    d = [_dev(x) for x in (new, lens, pool, [taken], bt)]
    ind, pos, slot = (torch.empty(n, dtype=i32, device="cuda") for n in (51, 64, 64))
    st = torch.zeros(1, dtype=i32, device="cuda")
    binding.tables_extend(p, *d, d[1], d[3], ind, pos, slot, status=st)
    ok = int(st.item()) == 0
    done = (d[1].cpu().numpy() - lens).astype(np.int32)
    assert done.sum() > 0
    binding.tables_trim(p, _dev(done), d[1], d[2], d[3], d[4], d[1], d[3], status=st if ok else None)
    assert np.array_equal(d[1].cpu().numpy(), lens) and np.array_equal(d[4].cpu().numpy(), bt)
    assert np.array_equal(d[2].cpu().numpy(), pool) and int(d[3].item()) == taken


# ------------------------------------------------------------ a whole step ----

def _chain_bits(emb, seqs, table, kv, cap):
    """What one token after the other leaves in the rows' slots."""
    return [torch.stack([emb[t] for t in s[:kv]]) for s in seqs]


@pytest.mark.parametrize("T,shape", [(7, "tree"), (16, "tree"), (5, "chain"), (1, "chain")])
def test_a_speculative_step_captured_and_replayed(T, shape):
    """Tables, append, attention, verification, compaction, trimmed tables in one graph, replayed with new
    drafts: the rows' tokens, lengths, pages and cache bits are those of one token after the other, and each
    step's attention is the formula's."""
    B, Hq, Hkv, V, steps, W = 6, 8, 2, 40, 9, 14
    NP = B * W + 5
    r, g = np.random.RandomState(T), torch.Generator().manual_seed(T)
    emb_k, emb_v = (torch.randn((V, Hkv, 128), generator=g).to(torch.bfloat16) for _ in range(2))
    target = torch.randn((V, V), generator=g) * 4  # the target's logits behind a token
    dek, dev_, dtarget = emb_k.cuda(), emb_v.cuda(), target.cuda()
    p = binding.plan(B, T, Hq, Hkv, 128, 16, NP, W)
    z = lambda *s, dt=i32: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
    kc, vc = z(NP, 16, Hkv, 128, dt=torch.bfloat16), z(NP, 16, Hkv, 128, dt=torch.bfloat16)
    pool, taken, bt, lens = _dev(r.permutation(NP)), z(1), torch.full((B, W), -1, dtype=i32, device="cuda"), z(B)
    first = pool.cpu().numpy().copy()
    new, ind, pos, slot, st = torch.full((B,), T, dtype=i32, device="cuda"), z(B + 1), z(B * T), z(B * T), z(1)
    tok, par = z(B, T), z(B, T)
    coins, race, temp = z(B, T, dt=torch.float32), z(B, V, dt=torch.float32), torch.ones(B, device="cuda")
    q, out, lse = z(B, Hq, T, 128, dt=torch.bfloat16), z(B, Hq, T, 128, dt=torch.bfloat16), z(B, Hq, T, dt=torch.float32)
    n_acc, n_drop, path, toks, logp = z(B), z(B), z(B, T), z(B, T), z(B, T, dt=torch.float32)
    after = z(B)
    scratch = z(max(binding.tree_scratch_bytes(p), 16), dt=torch.uint8)

    def step():
        binding.tables_extend(p, new, lens, pool, taken, bt, lens, taken, ind, pos, slot, status=st)
        after.copy_(lens)
        k_new, v_new = dek[tok.long()], dev_[tok.long()]
        binding.kv_append(p, T, k_new, v_new, bt, lens, kc, vc, status=st)
        binding.attn_tree(p, q, kc, vc, bt, lens, par, out, lse, scratch, status=st)
        logits = dtarget[tok.long()]
        binding.verify_tree(p, logits, tok, par, coins, race, temp, n_acc, n_drop, path, toks, logp, status=st)
        binding.kv_compact(p, path, n_acc, bt, lens, kc, vc, status=st)
        binding.tables_trim(p, n_drop, lens, pool, taken, bt, lens, taken, status=st)

    state = [kc, vc, pool, taken, bt, lens]
    saved = [x.clone() for x in state]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    par.copy_(_dev([ref.tree(r, T, shape) for _ in range(B)]))
    race.fill_(1.0)
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for x, y in zip(state, saved):
        x.copy_(y)
    st.zero_()
    last = r.randint(0, V, B)
    seqs = [[] for _ in range(B)]
    moved = 0
    for _ in range(steps):
        parents = [ref.tree(r, T, shape) for _ in range(B)]
        drafts = np.array([[last[b]] + r.randint(0, V, T - 1).tolist() for b in range(B)]).reshape(B, T)
        for b in range(B):  # likely drafts, so that paths are long
            for n in range(1, T):
                best = target[drafts[b, parents[b][n]]].topk(3).indices.tolist()
                drafts[b, n] = best[r.randint(0, 3)]
        c = {"logits": target[torch.as_tensor(drafts)], "draft_probs": None, "draft_tokens": torch.as_tensor(drafts),
             "parents": torch.as_tensor(np.array(parents)), "coins": torch.rand((B, T), generator=g),
             "race": (-torch.log1p(-torch.rand((B, V), generator=g))).clamp(min=2.0 ** -40), "temperature": torch.ones(B)}
        tok.copy_(_dev(drafts))
        par.copy_(_dev(parents))
        coins.copy_(c["coins"])
        race.copy_(c["race"])
        q.copy_(torch.randn(q.shape, generator=g).to(torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        # the step's attention, on the cache as the nodes were in it
        full = {"q": q.cpu(), "kv_lens": after.cpu(), "parents": par.cpu(),
                "block_table": torch.arange(B * W, dtype=i32).view(B, W)}
        kh, vh = (torch.zeros((B * W * 16, Hkv, 128), dtype=torch.bfloat16) for _ in range(2))
        for b in range(B):
            ids = torch.as_tensor(seqs[b] + drafts[b].tolist())
            kh[b * W * 16:b * W * 16 + len(ids)], vh[b * W * 16:b * W * 16 + len(ids)] = emb_k[ids], emb_v[ids]
        full["k_cache"], full["v_cache"] = kh.view(B * W, 16, Hkv, 128), vh.view(B * W, 16, Hkv, 128)
        want = ref.attention(full)
        e_out, e_lse = ref.bounds(want)
        assert (np.abs(out.cpu().double().numpy() - want[0]) <= e_out).all()
        assert (np.abs(lse.cpu().double().numpy() - want[1]) <= e_lse).all()
        for b in range(B):
            n, way, said, _, near = ref.verify(c, b)
            if not near:
                assert path[b, :n].tolist() == way and toks[b, :n].tolist() == said and int(n_acc[b]) == n
            n = int(n_acc[b])
            moved += any(m != i for i, m in enumerate(path[b, :n].tolist()))
            seqs[b] += [int(drafts[b, m]) for m in path[b, :n].tolist()]
            last[b] = int(toks[b, n - 1])
        assert lens.tolist() == [len(s) for s in seqs]
    assert moved > 0 or shape == "chain"
    # the cache holds what one token after the other would have left; pages are the rows' or the pool's
    held, table = [], bt.cpu()
    for b, s in enumerate(seqs):
        n = -(-len(s) // 16)
        assert (table[b, n:] == -1).all()
        held += table[b, :n].tolist()
        pg = table[b, :n].long()
        ids = torch.as_tensor(s)
        for cache, emb in ((kc, emb_k), (vc, emb_v)):
            got = cache.cpu()[pg].reshape(-1, Hkv, 128)[:len(s)]
            assert torch.equal(got.view(torch.int16), emb[ids].view(torch.int16))
    assert int(taken.item()) == len(held)
    assert sorted(held + pool.cpu().tolist()[len(held):]) == sorted(first.tolist())
