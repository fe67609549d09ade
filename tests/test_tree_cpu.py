"""The speculative step's calls on the host (no GPU): what they refuse, scratch sizes, the binding's checks, and
pins of the 64-bit statements that the GPU tests compare with."""
import ctypes
import math

import numpy as np
import pytest
import torch

import tree_ref as ref


@pytest.fixture(scope="module")
def rk():
    from deterministic_paged_kv_gb300 import binding, build
    build.build()
    binding.load()
    return binding


def _code(rk, rc, name):
    assert rk.ERRORS.get(rc) == name and rk.last_error()


A = 1 << 20  # an aligned address that no call here reads


def _tree(rk, p, ptrs=None, scratch=A, nbytes=1 << 62):
    a = [A] * 8 if ptrs is None else ptrs
    return rk.load().rk_paged_attn_tree(ctypes.byref(p) if p else None, *a, scratch, nbytes, None, None)


def test_tree_attention_refusals(rk):
    p = rk.plan(2, 8, 8, 2, 128, 16, 10, 4)
    _code(rk, _tree(rk, None), "RK_E_ARG")
    _code(rk, _tree(rk, rk.plan(2, 65, 8, 2, 128, 16, 10, 4)), "RK_E_UNSUPPORTED")
    for i in range(8):
        a = [A] * 8
        a[i] = None
        _code(rk, _tree(rk, p, a), "RK_E_ARG")
    for i, off in ((0, 8), (1, 8), (2, 2), (3, 2), (4, 1), (5, 2), (6, 8), (7, 2)):
        a = [A] * 8
        a[i] = A + off
        _code(rk, _tree(rk, p, a), "RK_E_ARG")
    assert _tree(rk, rk.plan(0, 8, 8, 2, 128, 16, 10, 4), [None] * 8, None, 0) == rk.RK_OK
    need = rk.tree_scratch_bytes(rk.plan(2, 8, 8, 2, 128, 16, 10, 4000))
    if need:
        q = rk.plan(2, 8, 8, 2, 128, 16, 10, 4000)
        _code(rk, _tree(rk, q, None, None, 0), "RK_E_ARG")
        _code(rk, _tree(rk, q, None, A + 8, need), "RK_E_ARG")
        _code(rk, _tree(rk, q, None, A, need - 1), "RK_E_ARG")
    with pytest.raises(rk.RkError):
        rk.tree_scratch_bytes(rk.plan(2, 65, 8, 2, 128, 16, 10, 4))


def test_other_refusals(rk):
    lib = rk.load()
    p = rk.plan(2, 8, 8, 2, 128, 16, 10, 4)
    big = rk.plan(2, 65, 8, 2, 128, 16, 10, 4)

    def verify(plan=p, kind=0, V=100, a=None, logits=A):
        return lib.rk_paged_verify_tree(ctypes.byref(plan), logits, kind, V, *(a or [A] * 11), None, None)
    _code(rk, verify(big), "RK_E_UNSUPPORTED")
    _code(rk, verify(kind=2), "RK_E_ARG")
    _code(rk, verify(V=0), "RK_E_ARG")
    _code(rk, verify(logits=None), "RK_E_ARG")
    _code(rk, verify(logits=A + 1), "RK_E_ARG")
    _code(rk, verify(kind=1, logits=A + 2), "RK_E_ARG")
    for i in range(1, 11):
        for bad in (None, A + 2):
            a = [A] * 11
            a[i] = bad
            _code(rk, verify(a=a), "RK_E_ARG")

    def compact(plan=p, a=None):
        return lib.rk_paged_kv_compact(ctypes.byref(plan), *(a or [A] * 6), None, None)
    _code(rk, compact(big), "RK_E_UNSUPPORTED")
    _code(rk, compact(rk.plan(2, 8, 8, 2, 128, 16, 0, 4)), "RK_E_KVLEN")
    _code(rk, compact(rk.plan(2, 8, 8, 2, 128, 16, 4, 0)), "RK_E_KVLEN")
    assert compact(rk.plan(0, 8, 8, 2, 128, 16, 10, 4), [None] * 6) == rk.RK_OK
    for i in range(6):
        for bad in (None, A + (8 if i > 3 else 2)):
            a = [A] * 6
            a[i] = bad
            _code(rk, compact(a=a), "RK_E_ARG")

    def trim(plan=p, n_pool=5, a=None):
        a = a or [A] * 7
        return lib.rk_paged_tables_trim(ctypes.byref(plan), a[0], a[1], a[2], n_pool, *a[3:], None, None)
    _code(rk, trim(n_pool=-1), "RK_E_ARG")
    _code(rk, trim(rk.plan(16385, 1, 8, 2, 128, 16, 10, 4)), "RK_E_UNSUPPORTED")
    for i in range(7):
        for bad in (None, A + 2):
            a = [A] * 7
            a[i] = bad
            _code(rk, trim(a=a), "RK_E_ARG")


@pytest.mark.parametrize("what", ["q", "k_cache", "v_cache", "block_table", "kv_lens", "parents", "out", "lse"])
def test_binding_checks_types_and_shapes(rk, what):
    p = rk.plan(2, 3, 8, 2, 128, 16, 10, 4)
    t = {"q": torch.zeros(2, 8, 3, 128, dtype=torch.bfloat16), "k_cache": torch.zeros(10, 16, 2, 128, dtype=torch.bfloat16),
         "v_cache": torch.zeros(10, 16, 2, 128, dtype=torch.bfloat16), "block_table": torch.zeros(2, 4, dtype=torch.int32),
         "kv_lens": torch.zeros(2, dtype=torch.int32), "parents": torch.zeros(2, 3, dtype=torch.int32),
         "out": torch.zeros(2, 8, 3, 128, dtype=torch.bfloat16), "lse": torch.zeros(2, 8, 3)}
    call = lambda: rk.attn_tree(p, *[t[k] for k in t])  # noqa: E731
    with pytest.raises(ValueError, match="CUDA"):
        call()
    # a wrong one is named before the tensors' device is asked, when it comes first
    good = t[what]
    t[what] = good.to(torch.float64)
    with pytest.raises((TypeError, ValueError)):
        call()
    t[what] = good[..., :-1] if good.dim() > 1 else good[:-1]
    with pytest.raises(ValueError):
        call()


# ---------------------------------------------------- the 64-bit statements ----

def test_ways_and_trees():
    assert ref.ways([-1, 0, 0, 2, ref.UNUSED, -1, 5]) == [[0], [0, 1], [0, 2], [0, 2, 3], [], [5], [5, 6]]
    r = np.random.RandomState(0)
    for shape in ("chain", "star", "tree", "forest", "none"):
        for T in (1, 2, 9, 64):
            row = ref.tree(r, T, shape)
            assert len(row) == T and all(-2 <= p < n for n, p in enumerate(row))
            assert all(p < 0 or row[p] != ref.UNUSED for p in row)


def test_attention_statement_is_dense_causal_attention_for_a_chain():
    import oracle
    oracle.build()
    c = ref.case(1, [21, 0, 40], 5, 4, 2, ["chain"])
    out, lse, _ = ref.attention(c)
    pos = (c["kv_lens"][:, None] - 5 + torch.arange(5, dtype=torch.int32)).to(torch.int32)
    ro, rl = oracle.attention(c["q"], c["k_cache"], c["v_cache"], c["block_table"], c["kv_lens"], pos)
    assert np.abs(out - ro).max() < 1e-9 and np.abs(lse - rl).max() < 1e-9


def test_attention_statement_of_a_path_is_that_path_as_a_chain():
    """A node's result is that of its ancestors laid out one after the other."""
    c = ref.case(2, [19], 8, 2, 1, ["tree"])
    out, lse, _ = ref.attention(c)
    for n, way in enumerate(ref.ways(c["parents"][0].tolist())):
        T = len(way)
        one = {k: v.clone() for k, v in c.items()}
        path = np.array([way + [-1] * (8 - T)])
        one["k_cache"], one["v_cache"] = ref.compact(c, 8, path, [T])
        one["kv_lens"] = torch.tensor([19 + T], dtype=torch.int32)
        one["q"] = c["q"][:, :, way].contiguous()
        one["parents"] = torch.tensor([list(range(-1, T - 1))], dtype=torch.int32)
        o, l, _ = ref.attention(one)
        assert np.abs(o[:, :, -1] - out[:, :, n]).max() < 1e-12 and np.abs(l[:, :, -1] - lse[:, :, n]).max() < 1e-12


def test_verification_statement_has_the_targets_distribution():
    """Over drafts, coins and draws the first token is distributed as p says (chi squared, 6 deviations)."""
    V, T, N = 5, 3, 6000
    g = torch.Generator().manual_seed(3)
    x = torch.randn((1, T, V), generator=g)
    q = torch.randn((1, T, V), generator=g).softmax(-1)
    p = x[0, 0].double().softmax(-1).numpy()
    par = torch.tensor([[-1, 0, 0]])
    tok = torch.multinomial(q[0, 0], N * T, replacement=True, generator=g).view(N, 1, T)
    coins, race = torch.rand((N, 1, T), generator=g), -torch.log1p(-torch.rand((N, 1, V), generator=g))
    for probs in (q, None):
        n = np.zeros(V)
        for i in range(N):
            c = {"logits": x, "draft_probs": probs, "parents": par, "draft_tokens": tok[i] if probs is not None else torch.tensor([[0, 2, 4]]),
                 "coins": coins[i], "race": race[i], "temperature": torch.ones(1)}
            n[ref.verify(c, 0)[2][0]] += 1
        assert ((n - N * p) ** 2 / (N * p)).sum() < V - 1 + 6 * math.sqrt(2 * (V - 1))


def test_trim_statement():
    bt = [[3, 4, 5, -1], [6, 7, -1, -1]]
    got, said = ref.trim([17, 20], [40, 20], [3, 4, 5, 6, 7, 0, 1, 2], 5, bt, 8)
    assert not said and got["kv_lens"] == [23, 0] and got["taken"] == 2
    assert got["block_table"].tolist() == [[3, 4, -1, -1], [-1, -1, -1, -1]] and got["pool"].tolist() == [3, 4, 5, 6, 7, 0, 1, 2]


def test_policy_names_the_speculative_step(rk):
    pol = dict(kv.split("=", 1) for kv in rk.policy().split(";"))
    assert pol["split_kv"] == "disabled"  # of the calls that it was said of before
    assert "512_before_1024_with_up_to_64" in pol["tree"] and "1024_tokens" in pol["tree"] and "ordered_fp32_merge" in pol["tree"]
    assert "64_fixed_parts" in pol["verify"]
    # the parts that the scratch size tells: of 512 tokens before token 1024 with up to 64 queries a head, else of 1024
    for T, heads, want in ((64, 1, {512: 0, 528: 2, 1024: 2, 1040: 3, 2048: 3, 2064: 4}), (33, 2, {1024: 0, 1040: 2, 2048: 2, 2064: 3})):
        for tokens, parts in want.items():
            p = rk.plan(1, T, heads, 1, 128, 16, 1, tokens // 16)
            assert rk.tree_scratch_bytes(p) == parts * T * heads * (128 + 1) * 4, (T, tokens)
