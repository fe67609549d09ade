"""GPU tests of rk_paged_verify_tree against the walk in 64 bits, of what it refuses, and of the
distribution that its tokens have."""
import math

import numpy as np
import pytest
import torch

import tree_ref as ref
from deterministic_paged_kv_gb300 import binding

pytestmark = pytest.mark.gpu

i32 = torch.int32
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from deterministic_paged_kv_gb300 import build
    build.build()
    binding.load()


def _run(c, status=None, stream=None):
    B, T, V = c["logits"].shape
    d = {k: None if v is None else v.cuda() for k, v in c.items()}
    p = binding.plan(B, T, 1, 1, 128, 16, 1, 1)
    o = {"n_accepted": torch.full((B,), 99, dtype=i32, device="cuda"), "n_drop": torch.full((B,), 99, dtype=i32, device="cuda"),
         "path": torch.full((B, T), 99, dtype=i32, device="cuda"), "tokens": torch.full((B, T), 99, dtype=i32, device="cuda"),
         "logprobs": torch.full((B, T), 99.0, device="cuda")}
    binding.verify_tree(p, d["logits"], d["draft_tokens"], d["parents"], d["coins"], d["race"], d["temperature"],
                        o["n_accepted"], o["n_drop"], o["path"], o["tokens"], o["logprobs"], draft_probs=d["draft_probs"],
                        status=status, stream=stream)
    torch.cuda.synchronize()
    return {k: v.cpu() for k, v in o.items()}


def _check(c, got, skip=()):
    """Against 64 bits; rows whose choices are next to a border are left out, and are few."""
    B, T, _ = c["logits"].shape
    left = 0
    for b in range(B):
        if b in skip:
            continue
        n, path, toks, logs, near = ref.verify(c, b)
        if near:
            left += 1
            continue
        assert int(got["n_accepted"][b]) == n and int(got["n_drop"][b]) == T - n
        assert got["path"][b].tolist() == path + [-1] * (T - n)
        assert got["tokens"][b].tolist() == toks + [-1] * (T - n)
        l = got["logprobs"][b].double().numpy()
        # the exponent's argument and ln Z are FP32 (2^-21 of them at most), Z's sum good to 2^-17
        assert (np.abs(l[:n] - logs) <= 2.0 ** -16 + np.abs(logs) * 2.0 ** -21).all() and (l[n:] == 0).all()
    assert left <= 1 + B // 16


@pytest.mark.parametrize("probs", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,T,V,shapes", [
    (40, 1, 50, ["chain"]), (40, 8, 1000, ["chain"]), (40, 16, 4099, ["tree"]), (24, 64, 257, ["tree", "star"]), (9, 5, 32001, ["chain", "star"]),
    (30, 12, 1, ["star"]), (30, 12, 7, ["tree"]), (3, 9, 131072, ["tree"]), (4, 3, 262147, ["chain"]), (16, 20, 8192, ["star"])])
def test_verify_matches_the_walk(B, T, V, dtype, probs, shapes):
    c = ref.verify_case(1000 + B + T, B, T, V, dtype, probs, shapes)
    st = torch.zeros(1, dtype=i32, device="cuda")
    got = _run(c, st)
    assert int(st.item()) == 0
    _check(c, got)


@pytest.mark.parametrize("probs", [False, True])
def test_rows_do_not_depend_on_the_batch(probs):
    c = ref.verify_case(5, 33, 7, 5003, BF, probs, ["tree", "chain", "star"])
    whole = _run(c)
    order = torch.randperm(33, generator=torch.Generator().manual_seed(2))
    mixed = _run({k: None if v is None else v[order].contiguous() for k, v in c.items()})
    for k in whole:
        assert torch.equal(whole[k][order].view(i32), mixed[k].view(i32))
    for b in (0, 7, 32):
        one = _run({k: None if v is None else v[b:b + 1].contiguous() for k, v in c.items()})
        for k in whole:
            assert torch.equal(whole[k][b:b + 1].view(i32), one[k].view(i32))


def test_masked_tokens_are_never_drawn_and_masks_may_be_lowest_values():
    for low in (-math.inf, -3.3895e38):
        for probs in (False, True):
            c = ref.verify_case(9, 16, 6, 300, BF, probs, ["tree"])
            c["logits"][:, :, 100:] = low
            c["logits"][3, 0, :] = low
            c["logits"][3, 0, 42] = -3.3895e38  # a row with a single token, of the type's lowest value
            if low == -math.inf:
                got = _run(c)
                _check(c, got)
                assert int(got["tokens"][3, 0]) == 42
            else:
                _check(c, _run(c), skip=(3,))
            assert (got["tokens"][:3] < 100).all()


def test_all_logits_equal_to_the_lowest_value_are_uniform():
    c = ref.verify_case(11, 8, 4, 64, BF, False, ["chain"], temps=(1.0,))
    c["logits"][:] = -3.3895e38
    got = _run(c)
    _check(c, got)
    assert np.allclose(got["logprobs"][:, 0].numpy(), -math.log(64), atol=1e-6)


@pytest.mark.parametrize("what", ["nan", "inf", "empty", "temp_nan", "temp_neg", "temp_inf", "temp_tiny", "parent", "token", "token_neg", "unused",
                                  "q_nan", "q_inf"])
def test_bad_rows_keep_nothing_and_leave_the_others(what):
    c = ref.verify_case(13, 9, 6, 500, F32, what.startswith("q"), ["star"], temps=(1.0,))
    c["coins"][4] = 0.9999
    c["draft_tokens"][4] = 7
    c["logits"][4, :, 7] = -9.0
    want = _run(c)
    bit = binding.STATUS_RANGE
    if what in ("nan", "inf"):
        c["logits"][4, 0, 333] = math.nan if what == "nan" else math.inf
    elif what == "empty":
        c["logits"][4, 0] = -math.inf
    elif what.startswith("temp"):
        c["temperature"][4] = {"temp_nan": math.nan, "temp_neg": -1.0, "temp_inf": math.inf, "temp_tiny": 1e-30}[what]
    elif what.startswith("q"):
        c["draft_probs"][4, 0, 99] = math.nan if what == "q_nan" else math.inf
    else:
        bit = binding.STATUS_TREE
        if what == "parent":
            c["parents"][4, 3] = 3
        elif what == "unused":
            c["parents"][4, 3], c["parents"][4, 4] = ref.UNUSED, 3
        else:
            c["draft_tokens"][4, 5] = 500 if what == "token" else -1
    st = torch.zeros(1, dtype=i32, device="cuda")
    got = _run(c, st)
    assert int(st.item()) == bit
    assert int(got["n_accepted"][4]) == 0 and int(got["n_drop"][4]) == 6
    assert (got["path"][4] == -1).all() and (got["tokens"][4] == -1).all() and torch.isnan(got["logprobs"][4]).all()
    rest = [b for b in range(9) if b != 4]
    for k in want:
        assert torch.equal(want[k][rest].view(i32), got[k][rest].view(i32))


def test_what_the_walk_does_not_reach_may_be_anything():
    c = ref.verify_case(17, 12, 8, 700, F32, True, ["chain"])
    want = _run(c)
    for b in range(12):
        for n in range(8):
            if n not in want["path"][b].tolist():
                c["logits"][b, n] = math.nan
                c["draft_probs"][b, n] = math.nan
    c["draft_tokens"][:, 0] = -77
    got = _run(c)
    for k in want:
        assert torch.equal(want[k].view(i32), got[k].view(i32))


def test_rows_without_a_root_and_unused_nodes():
    c = ref.verify_case(19, 6, 5, 200, BF, False, ["chain", "none"])
    c["parents"][2, 3:] = ref.UNUSED
    c["draft_tokens"][2, 3:] = -5
    st = torch.zeros(1, dtype=i32, device="cuda")
    got = _run(c, st)
    assert int(st.item()) == 0
    _check(c, got, skip=(1, 3, 5))
    for b in (1, 3, 5):
        assert int(got["n_accepted"][b]) == 0 and int(got["n_drop"][b]) == 0
        assert (got["path"][b] == -1).all() and (got["tokens"][b] == -1).all() and (got["logprobs"][b] == 0).all()


def test_certain_drafts():
    """p one token: its draft is accepted; another's is not; nothing left of r: the token is p's."""
    V, T = 90, 4
    c = ref.verify_case(23, 3, T, V, F32, False, ["star"], temps=(1.0,))
    c["logits"][:] = -200.0
    c["logits"][:, :, 5] = 0.0
    c["draft_tokens"][0] = 5
    c["draft_tokens"][1] = 6
    c["coins"][:] = 1.0 - 2.0 ** -24
    c["logits"][2] = -math.inf
    c["logits"][2, :, 8] = 3.0
    c["draft_tokens"][2] = 8
    got = _run(c)
    assert got["tokens"][0].tolist() == [5, 5, -1, -1] and got["path"][0].tolist() == [0, 1, -1, -1]
    assert got["tokens"][1].tolist() == [5, -1, -1, -1]
    assert got["tokens"][2].tolist() == [8, 8, -1, -1]
    c["coins"][2] = 1.0  # past the range of a uniform draw: refused, and r is empty
    got = _run(c)
    assert got["tokens"][2].tolist() == [8, -1, -1, -1]


def test_race_of_zero_and_ties_go_to_the_lowest_token():
    c = ref.verify_case(29, 2, 1, 64, F32, False, ["chain"], temps=(1.0,))
    c["logits"][:] = 0.0
    c["race"][:] = 1.0
    assert _run(c)["tokens"][:, 0].tolist() == [0, 0]
    c["race"][0, 40:] = 0.5
    c["race"][1, 33] = 0.0
    assert _run(c)["tokens"][:, 0].tolist() == [40, 33]
    c["temperature"][:] = 0.0
    c["logits"][0, 0, 9:12] = 1.0
    assert _run(c)["tokens"][:, 0].tolist() == [9, 0]


@pytest.mark.parametrize("probs,shape", [(False, "chain"), (True, "chain"), (True, "star"), (False, "star")])
def test_the_first_token_is_distributed_as_the_target_says(probs, shape):
    """8192 rows of the same p and q with drafts of their own draws: counts of the step's first token
    against p, by the sum of (count - n p)^2 / (n p): mean V - 1, variance 2 (V - 1) and a little more."""
    B, T, V = 8192, 4, 12
    g = torch.Generator().manual_seed(31)
    x = torch.randn((1, T, V), generator=g) * 1.5
    q = (x + torch.randn((1, T, V), generator=g)).softmax(-1)
    par = torch.tensor([ref.tree(None, T, shape)], dtype=i32)
    # drafts without probabilities: fixed tokens, which must not move the distribution either
    draws = torch.multinomial(q[0, 0], B * T, replacement=True, generator=g).view(B, T).to(i32)
    draws = draws if probs else torch.arange(3, 3 + T, dtype=i32).expand(B, T)
    c = {"logits": x.expand(B, T, V).contiguous(), "draft_probs": q.expand(B, T, V).contiguous() if probs else None,
         "draft_tokens": draws.contiguous(), "parents": par.expand(B, T).contiguous(), "coins": torch.rand((B, T), generator=g),
         "race": (-torch.log1p(-torch.rand((B, V), generator=g))).clamp(min=2.0 ** -40), "temperature": torch.ones(B)}
    first = _run(c)["tokens"][:, 0].long()
    p = x[0, 0].double().softmax(-1).numpy()
    n = np.bincount(first.numpy(), minlength=V)
    chi = ((n - B * p) ** 2 / (B * p)).sum()
    assert chi < V - 1 + 6 * math.sqrt(2 * (V - 1))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("off", [1, 2, 3, 5])
def test_logits_at_any_element(dtype, off):
    c = ref.verify_case(37, 7, 5, 1003, dtype, True, ["tree"])
    want = _run(c)
    d = dict(c)
    for k in ("logits", "draft_probs", "race"):
        flat = torch.empty(c[k].numel() + off, dtype=c[k].dtype, device="cuda")
        flat[off:] = c[k].cuda().view(-1)
        d[k] = flat[off:].view(c[k].shape)
    got = _run(d)
    for k in want:
        assert torch.equal(want[k].view(i32), got[k].view(i32))


def test_captured_and_on_another_stream():
    c = ref.verify_case(41, 10, 6, 2000, BF, True, ["tree"])
    want = _run(c)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = _run(c, stream=s)
    assert all(torch.equal(want[k].view(i32), got[k].view(i32)) for k in want)


@pytest.mark.parametrize("probs", [False, True])
@pytest.mark.parametrize("low", [-math.inf, -3.3895e38, -1.0e4])
@pytest.mark.parametrize("V", [300, 40000])
def test_draws_of_zero_choose_no_token_that_weighs_nothing(V, low, probs):
    """Masked tokens with a draw of 0 in the race: the results of a race in which their draws are 1."""
    c = ref.verify_case(47, 8, 5, V, BF, probs, ["tree", "star"])
    c["logits"][:, :, V // 3:] = low
    c["race"][:, V // 3:] = 1.0
    want = _run(c)
    _check(c, want)
    c["race"][:, V // 3:] = 0.0
    got = _run(c)
    assert all(torch.equal(want[k].view(i32), got[k].view(i32)) for k in want)
    assert (got["tokens"] < V // 3).all()


def test_a_race_without_numbers_is_refused_where_it_is_read():
    c = ref.verify_case(53, 3, 3, 500, F32, False, ["chain"], temps=(1.0, 1.0, 0.0))
    want = _run(c)
    c["race"][0] = math.nan
    c["race"][2] = math.nan   # greedy: not read
    st = torch.zeros(1, dtype=i32, device="cuda")
    got = _run(c, status=st)
    assert int(st.item()) == binding.STATUS_RANGE
    assert int(got["n_accepted"][0]) == 0 and got["tokens"][0].tolist() == [-1] * 3 and got["logprobs"][0].isnan().all()
    assert all(torch.equal(want[k][1:].view(i32), got[k][1:].view(i32)) for k in want)


def test_two_captured_calls_at_once():
    """Two graphs replayed on two streams with no order between them, over and over."""
    cases = [ref.verify_case(59 + i, 24, 6, V, BF, probs, ["tree", "chain"]) for i, (V, probs) in enumerate(((50000, True), (3001, False)))]
    want = [_run(c) for c in cases]
    streams, graphs, outs, keep = [], [], [], []
    for c in cases:
        B, T, V = c["logits"].shape
        d = {k: None if v is None else v.cuda() for k, v in c.items()}
        o = {k: torch.zeros_like(v, device="cuda") for k, v in want[0].items()}
        p = binding.plan(B, T, 1, 1, 128, 16, 1, 1)
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            binding.verify_tree(p, d["logits"], d["draft_tokens"], d["parents"], d["coins"], d["race"], d["temperature"],
                                o["n_accepted"], o["n_drop"], o["path"], o["tokens"], o["logprobs"], draft_probs=d["draft_probs"])
        streams.append(torch.cuda.Stream())
        graphs.append(g)
        outs.append(o)
        keep.append(d)
    torch.cuda.synchronize()
    for _ in range(10):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert all(torch.equal(w[k].view(i32), o[k].cpu().view(i32)) for k in w)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_hundred_and_more_rows_and_the_smallest_vocabularies(dtype):
    """Every number of CTAs to a row, and vocabularies that fill no chunk."""
    for B, T, V in ((305, 3, 70), (160, 4, 5000), (80, 2, 17), (2, 3, 1), (5, 4, 2), (40, 3, 7), (30, 2, 9)):
        c = ref.verify_case(61 + B, B, T, V, dtype, B % 2 == 0, ["tree", "chain"]) if V >= 3 else None
        if c is None:
            g = torch.Generator().manual_seed(V)
            c = {"logits": torch.randn((B, T, V), generator=g).to(dtype), "draft_probs": None,
                 "draft_tokens": torch.randint(0, V, (B, T), generator=g, dtype=torch.int64).to(i32),
                 "parents": torch.arange(-1, T - 1, dtype=i32).expand(B, T).contiguous(), "coins": torch.rand((B, T), generator=g),
                 "race": torch.rand((B, V), generator=g) + 0.1, "temperature": torch.ones(B)}
        _check(c, _run(c))


def test_verify_offsets_past_32_bits():
    """The last row of a batch whose logits and probabilities pass 2^31 elements: the bits of the row alone."""
    B, T, V = 36, 64, 1000003
    assert B * T * V > 2 ** 31
    c = ref.verify_case(71, 1, T, 2003, BF, True, ["tree"], temps=(1.0,))
    small = c["logits"].shape[2]
    lg = torch.zeros((B, T, V), dtype=BF, device="cuda")
    lg[-1] = -40.0
    lg[-1, :, -small:] = c["logits"][0].cuda()
    q = torch.zeros((B, T, V), device="cuda")
    q[-1, :, -small:] = c["draft_probs"][0].cuda()
    par = torch.full((B, T), -2, dtype=i32)
    par[-1] = c["parents"][0]
    tok = torch.zeros((B, T), dtype=i32)
    tok[-1] = c["draft_tokens"][0] + (V - small)
    race = torch.ones((B, V), device="cuda")
    race[-1, -small:] = c["race"][0].cuda()
    coins, temp = torch.zeros((B, T)), torch.ones(B)
    coins[-1] = c["coins"][0]

    def go(rows):
        n = len(range(B)[rows])
        p = binding.plan(n, T, 1, 1, 128, 16, 1, 1)
        o = [torch.full(s, 99, dtype=i32, device="cuda") for s in ((n,), (n,), (n, T), (n, T))] + [torch.full((n, T), 9.0, device="cuda")]
        binding.verify_tree(p, lg[rows], tok[rows].cuda(), par[rows].cuda(), coins[rows].cuda(), race[rows], temp[rows].cuda(), *o,
                            draft_probs=q[rows])
        return [x.cpu() for x in o]

    every, alone = go(slice(0, B)), go(slice(B - 1, B))
    assert int(alone[0][0]) >= 1 and (every[0][:-1] == 0).all()
    assert (alone[3][0, :int(alone[0][0])] >= V - small).all()
    assert all(torch.equal(x[-1:].view(i32), y.view(i32)) for x, y in zip(every, alone))
