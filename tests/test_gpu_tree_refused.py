"""GPU tests of rk_paged_tree_rows, and of a captured speculative step in which some rows get no nodes: they
run out of pages or of table, or are idle.  Such rows keep their tokens, pages and bits."""
import numpy as np
import pytest
import torch

import tree_ref as ref
from deterministic_paged_kv_gb300 import binding

pytestmark = pytest.mark.gpu

i32 = torch.int32
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from deterministic_paged_kv_gb300 import build
    build.build()
    binding.load()


def _dev(x):
    return torch.as_tensor(np.array(x), dtype=i32).cuda()


def _rows(T, counts, lens, parents, inplace=False):
    B = len(counts)
    p = binding.plan(B, T, 8, 2, 128, 16, 4, 3)
    d = [_dev(np.concatenate([[0], np.cumsum(counts)])), _dev(lens), _dev(parents).view(B, T)]
    out, par = torch.full((B,), 99, dtype=i32, device="cuda"), d[2] if inplace else torch.full((B, T), 99, dtype=i32, device="cuda")
    st = torch.zeros(1, dtype=i32, device="cuda")
    binding.tree_rows(p, *d, out, par, status=st)
    assert d[1].tolist() == list(lens)
    return out.tolist(), par.cpu().numpy(), int(st.item())


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("B,T", [(1, 1), (1, 64), (7, 5), (300, 13), (5000, 64)])
def test_rows_without_their_tokens_have_no_tree(B, T, inplace):
    r = np.random.RandomState(B + T)
    counts = np.where(r.rand(B) < 0.6, T, 0)
    lens, parents = r.randint(0, 5000, B), r.randint(-2, T, (B, T))
    got = _rows(T, counts, lens, parents, inplace)
    assert got[0] == np.where(counts == T, lens, 0).tolist() and got[2] == 0
    assert np.array_equal(got[1], np.where((counts == T)[:, None], parents, ref.UNUSED))
    if T > 1:  # another number of tokens is no tree, and is reported
        counts[B // 2] = T - 1
        got = _rows(T, counts, lens, parents, inplace)
        assert got[0] == np.where(counts == T, lens, 0).tolist() and got[2] == binding.STATUS_TREE
        assert np.array_equal(got[1], np.where((counts == T)[:, None], parents, ref.UNUSED))


class Step:
    """A captured step of rows with given lengths, tables and counts of new tokens."""

    def __init__(self, T, W, lens, new, tables, pool, taken, NP, seed):
        self.T, self.B, self.W, V, Hq, Hkv = T, len(lens), W, 50, 8, 2
        self.V = V
        B = self.B
        g = torch.Generator().manual_seed(seed)
        z = lambda *s, dt=i32: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
        self.kc, self.vc = (torch.randn((NP, 16, Hkv, 128), generator=g).to(BF).cuda() for _ in range(2))
        self.emb = [torch.randn((V, Hkv, 128), generator=g).to(BF).cuda() for _ in range(2)]
        self.target = (torch.randn((V, V), generator=g) * 4).cuda()
        self.p = binding.plan(B, T, Hq, Hkv, 128, 16, NP, W)
        self.pool, self.taken, self.bt, self.lens = _dev(pool), _dev([taken]), _dev(tables), _dev(lens)
        self.new = _dev(new)
        self.ind, self.pos, self.slot = z(B + 1), z(B * T), z(B * T)
        self.tok, self.par, self.tree_par, self.tree_lens = z(B, T), z(B, T), z(B, T), z(B)
        self.coins, self.race, self.temp = z(B, T, dt=torch.float32), torch.ones((B, V), device="cuda"), torch.ones(B, device="cuda")
        self.q, self.out, self.lse = z(B, Hq, T, 128, dt=BF), z(B, Hq, T, 128, dt=BF), z(B, Hq, T, dt=torch.float32)
        self.n_acc, self.n_drop, self.path, self.toks, self.logp = z(B), z(B), z(B, T), z(B, T), z(B, T, dt=torch.float32)
        self.scratch = z(max(binding.tree_scratch_bytes(self.p), 16), dt=torch.uint8)
        self.st, self.st2 = z(1), z(1)
        held = [x.clone() for x in self.state()]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            self.once()
        torch.cuda.current_stream().wait_stream(side)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.once()
        for x, y in zip(self.state(), held):
            x.copy_(y)

    def state(self):
        return [self.kc, self.vc, self.pool, self.taken, self.bt, self.lens]

    def once(self):
        s, tok = self, self.tok.long()
        binding.tables_extend(s.p, s.new, s.lens, s.pool, s.taken, s.bt, s.lens, s.taken, s.ind, s.pos, s.slot, status=s.st)
        binding.tree_rows(s.p, s.ind, s.lens, s.par, s.tree_lens, s.tree_par, status=s.st2)
        binding.kv_append(s.p, s.T, s.emb[0][tok], s.emb[1][tok], s.bt, s.tree_lens, s.kc, s.vc)
        binding.attn_tree(s.p, s.q, s.kc, s.vc, s.bt, s.tree_lens, s.tree_par, s.out, s.lse, s.scratch, status=s.st2)
        binding.verify_tree(s.p, s.target[tok], s.tok, s.tree_par, s.coins, s.race, s.temp, s.n_acc, s.n_drop, s.path, s.toks,
                            s.logp, status=s.st2)
        binding.kv_compact(s.p, s.path, s.n_acc, s.bt, s.tree_lens, s.kc, s.vc, status=s.st2)
        binding.tables_trim(s.p, s.n_drop, s.lens, s.pool, s.taken, s.bt, s.lens, s.taken, status=s.st2)

    def replay(self, drafts, parents, coins, race, q):
        self.tok.copy_(drafts)
        self.par.copy_(parents)
        self.coins.copy_(coins)
        self.race.copy_(race)
        self.q.copy_(q)
        self.st.zero_()
        self.st2.zero_()
        self.graph.replay()
        torch.cuda.synchronize()
        return int(self.st.item()), int(self.st2.item())

    def tokens(self, b):
        """Bits of row b's tokens, its length and its table."""
        n = int(self.lens[b])
        pg = self.bt[b, :-(-n // 16)].long()
        return n, self.bt[b].tolist(), [c[pg].reshape(-1, *c.shape[2:])[:n].view(torch.int16).cpu() for c in (self.kc, self.vc)]


@pytest.mark.parametrize("T", [1, 5, 20])
def test_rows_that_get_no_nodes_keep_what_they_have(T):
    W, steps = 8, 4
    full = 16 * W
    # two rows that go on; one at the end of its table; idle ones with many tokens, few and none; one for which no page is left
    lens = [30, 3, full - T + 1, 40, 1, 0, 48]
    new = [T, T, T, 0, 0, 0, T]
    goes = [0, 1]
    need = [-(-n // 16) for n in lens]
    NP = 64
    ids = np.random.RandomState(T).permutation(NP)
    tables, at = np.full((len(lens), W), -1, np.int32), 0
    for b, n in enumerate(need):
        tables[b, :n] = ids[at:at + n]
        at += n
    s = Step(T, W, lens, new, tables, ids, at, NP, seed=T)
    alone = Step(T, W, [lens[b] for b in goes], [new[b] for b in goes], tables[goes], ids, at, NP, seed=T)
    kept = {b: s.tokens(b) for b in range(len(lens)) if b not in goes}
    r, g = np.random.RandomState(T), torch.Generator().manual_seed(T)
    for _ in range(steps):
        B = len(lens)
        now = s.lens.tolist()
        wants = sum(-(-(now[b] + T) // 16) - -(-now[b] // 16) for b in goes)
        # rows are served in order: as many pages are left as the first two rows need
        held = set(s.bt[s.bt >= 0].tolist())
        free = [x for x in ids.tolist() if x not in held][:wants]
        for x in (s, alone):
            x.taken.fill_(NP - wants)
            x.pool[NP - wants:] = _dev(free)
        drafts = torch.as_tensor(r.randint(0, s.V, (B, T))).to(i32)
        parents = torch.as_tensor(np.array([ref.tree(r, T, "tree") for _ in range(B)]).reshape(B, T)).to(i32)
        coins, race = torch.rand((B, T), generator=g) * 0.2, (-torch.log1p(-torch.rand((B, s.V), generator=g))).clamp(min=2.0 ** -40)
        q = torch.randn(s.q.shape, generator=g).to(BF)
        st, st2 = s.replay(drafts, parents, coins, race, q)
        want = alone.replay(drafts[goes], parents[goes], coins[goes], race[goes], q[goes])
        assert want == (0, 0) and st2 == 0
        assert st & binding.STATUS_KVLEN  # the row at the end of its table
        assert st & binding.STATUS_POOL   # the row without a page
        # rows without nodes: nothing accepted, nothing dropped, nothing moved
        for b, was in kept.items():
            assert int(s.n_acc[b]) == 0 and int(s.n_drop[b]) == 0 and (s.path[b] == -1).all() and (s.toks[b] == -1).all()
            assert (s.out[b] == 0).all() and torch.isneginf(s.lse[b]).all()
            n, table, bits = s.tokens(b)
            assert n == was[0] and table == was[1] and all(torch.equal(x, y) for x, y in zip(bits, was[2]))
        # the others: bit for bit as without them
        for i, b in enumerate(goes):
            assert int(s.n_acc[b]) >= 1
            for x, y in ((s.out, alone.out), (s.lse, alone.lse), (s.n_acc, alone.n_acc), (s.path, alone.path), (s.toks, alone.toks),
                         (s.logp, alone.logp)):
                assert torch.equal(x[b:b + 1].contiguous().view(torch.int16), y[i:i + 1].contiguous().view(torch.int16))
            mine, theirs = s.tokens(b), alone.tokens(i)
            assert mine[0] == theirs[0] and mine[1] == theirs[1] and all(torch.equal(x, y) for x, y in zip(mine[2], theirs[2]))
        assert int(s.taken.item()) == int(alone.taken.item()) and torch.equal(s.pool, alone.pool)
