"""GPU tests of rk_paged_verify_tree: the last token by each of its ways (the race run along with the sum, a sweep of
its own, the largest logit), which all have to find the token itself and not only its place."""
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


def _run(c):
    B, T, V = c["logits"].shape
    d = {k: None if v is None else v.cuda() for k, v in c.items()}
    p = binding.plan(B, T, 1, 1, 128, 16, 1, 1)
    z = lambda *s: torch.full(s, 99, dtype=i32, device="cuda")  # noqa: E731
    o = [z(B), z(B), z(B, T), z(B, T), torch.full((B, T), 99.0, device="cuda")]
    st = torch.zeros(1, dtype=i32, device="cuda")
    binding.verify_tree(p, d["logits"], d["draft_tokens"], d["parents"], d["coins"], d["race"], d["temperature"], *o,
                        draft_probs=d["draft_probs"], status=st)
    assert int(st.item()) == 0
    return [x.cpu() for x in o]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [1, 5, 8, 9, 1000, 4099, 40000])
def test_the_last_token_of_every_way(V, dtype):
    """A child of probability 0 is refused and leaves p as it is, so the race without children, the one behind a
    refused child and, with draft probabilities that are 0 but there, the one over the residual draw the same token: the one
    that 64 bits say.  Temperatures whose factor is no power of two."""
    B, T = 96, 2
    g = torch.Generator().manual_seed(V)
    x = (torch.randn((B, T, V + 1), generator=g) * 3).to(dtype)
    x[:, :, V] = -math.inf  # the child's token
    temp = torch.rand(B, generator=g) + 0.3
    temp[::8] = 0.0
    race = (-torch.log1p(-torch.rand((B, V + 1), generator=g))).clamp(min=2.0 ** -40)
    c = {"logits": x, "draft_probs": None, "draft_tokens": torch.full((B, T), V, dtype=i32), "coins": torch.rand((B, T), generator=g),
         "race": race, "temperature": temp, "parents": torch.tensor([[-1, ref.UNUSED]] * B, dtype=i32)}
    key = x[:, 0].double() / torch.where(temp > 0, temp, torch.ones(())).double()[:, None]
    key = torch.where((temp > 0)[:, None], key - race.double().log(), key)
    best = key.max(-1)
    two = key.topk(2, -1).values
    # keys are FP32: a token within 2^-16 of the largest may be the one that is chosen (greedy: equal ones, the lowest)
    sure = ((two[:, 0] - two[:, 1] > 2.0 ** -16) | (temp == 0)).numpy()
    first = np.array([int((key[b] == best.values[b]).nonzero()[0]) for b in range(B)])
    assert sure.mean() > 0.9
    runs = [_run(c)]
    c["parents"] = torch.tensor([[-1, 0]] * B, dtype=i32)
    runs.append(_run(c))
    q = torch.zeros((B, T, V + 1))
    q[:, :, V] = 1.0
    c["draft_probs"] = q
    runs.append(_run(c))
    for n, drop, path, tok, logp in runs:
        assert (n == 1).all() and (path[:, 0] == 0).all()
        assert np.array_equal(tok[:, 0].numpy()[sure], first[sure])
        assert ((tok[:, 0] >= 0) & (tok[:, 0] < V)).all() and torch.isfinite(logp[:, 0]).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [1, 7, 8, 9, 15, 16, 17, 23, 24, 25, 40, 1003, 16392, 40000])
def test_arrays_that_begin_and_end_anywhere_among_others(V, dtype):
    """Logits, probabilities and draws cut out of larger arrays of NaN, at every element of 16 bytes: the bits of
    arrays of their own."""
    B, T = 5, 3
    c = ref.verify_case(400 + V, B, T, V, dtype, True, ["tree", "chain"]) if V >= 3 else {
        "logits": torch.zeros((B, T, V), dtype=dtype), "draft_probs": torch.ones((B, T, V)), "draft_tokens": torch.zeros((B, T), dtype=i32),
        "parents": torch.tensor([[-1, 0, 1]] * B, dtype=i32), "coins": torch.rand((B, T), generator=torch.Generator().manual_seed(1)),
        "race": torch.ones((B, V)), "temperature": torch.ones(B)}
    for probs in (True, False):
        if not probs:
            c = dict(c, draft_probs=None)
        want = _run(c)
        for off in range(1, 8):
            d = dict(c)
            for k in ("logits", "draft_probs", "race"):
                if d[k] is None:
                    continue
                n = d[k].numel()
                flat = torch.full((n + 16,), math.nan, dtype=d[k].dtype, device="cuda")
                flat[off:off + n] = d[k].cuda().view(-1)
                d[k] = flat[off:off + n].view(d[k].shape)
            assert all(torch.equal(x.view(i32), y.view(i32)) for x, y in zip(want, _run(d)))


def test_a_captured_call_replayed_with_new_inputs():
    """One captured call; every input changes in place between its replays and the outputs are spoilt before each."""
    B, T, V = 12, 6, 3001
    cases = [ref.verify_case(500 + i, B, T, V, BF, True, shapes, temps=temps)
             for i, (shapes, temps) in enumerate(((["tree"], (1.0, 0.7)), (["chain", "star"], (0.0, 1.3)), (["forest", "none"], (1.0, 0.0))))]
    for c in cases:  # (a walk begins at node 0: a forest's first node may be unused)
        c["draft_tokens"] = c["draft_tokens"].clamp(0, V - 1)
    want = [_run(c) for c in cases]
    d = {k: v.cuda() for k, v in cases[0].items()}
    p = binding.plan(B, T, 1, 1, 128, 16, 1, 1)
    o = [torch.zeros(x.shape, dtype=x.dtype, device="cuda") for x in want[0]]
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        binding.verify_tree(p, d["logits"], d["draft_tokens"], d["parents"], d["coins"], d["race"], d["temperature"], *o,
                            draft_probs=d["draft_probs"])
    for i in (0, 1, 2, 1, 0):
        for k in d:
            d[k].copy_(cases[i][k])
        for x in o:
            x.fill_(-99)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x.view(i32), y.cpu().view(i32)) for x, y in zip(want[i], o))


@pytest.mark.parametrize("temp", [math.nan, -1.0, math.inf, 1e-30])
def test_a_row_without_a_root_drops_nothing_whatever_its_temperature(temp):
    """An idle row's temperature may be anything: its tokens are not nodes, and none is dropped."""
    c = ref.verify_case(600, 4, 5, 100, F32, False, ["chain", "none"])
    want = _run(c)
    c["temperature"][1::2] = temp
    got = _run(c)  # (no status)
    assert all(torch.equal(x.view(i32), y.view(i32)) for x, y in zip(want, got))
    assert got[0][1::2].tolist() == [0, 0] and got[1][1::2].tolist() == [0, 0]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("which", ["logits", "draft_probs", "race"])
@pytest.mark.parametrize("V", [1000, 4096, 33000])
def test_one_array_alone_off_its_alignment(V, which, dtype):
    """Rows of whole chunks of which one array does not start at 16 bytes, with children refused and accepted."""
    c = ref.verify_case(700 + V, 20, 5, V, dtype, True, ["tree", "star"])
    c["coins"][::3] = 0.999
    want = _run(c)
    n = c[which].numel()
    flat = torch.full((n + 8,), math.nan, dtype=c[which].dtype, device="cuda")
    flat[1:n + 1] = c[which].cuda().view(-1)
    got = _run(dict(c, **{which: flat[1:n + 1].view(c[which].shape)}))
    assert all(torch.equal(x.view(i32), y.view(i32)) for x, y in zip(want, got))
