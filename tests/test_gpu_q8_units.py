"""GPU tests of the 8-bit attention calls where a CTA has several pieces of work, one after
the other: prefill units behind units of another row, length or verdict, and decode batches of
more rows than the item list has entries."""
import numpy as np
import pytest
import torch

import q8_ref as ref
import test_gpu_q8_attention as att
from deterministic_paged_kv_gb300 import binding

pytestmark = pytest.mark.gpu

i32 = torch.int32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from deterministic_paged_kv_gb300 import build
    build.build()
    binding.load()


def _head(c, row, h):
    """One row and KV head of a case, as a case."""
    G = c["q"].shape[1] // c["k_cache"].shape[1]
    o = att._rows(c, [row])
    o["q"] = o["q"][:, h * G:(h + 1) * G].contiguous()
    for n in ("k_cache", "v_cache", "k_scale", "v_scale"):
        o[n] = o[n].view(torch.uint8)[:, h:h + 1].contiguous().view(ref.F8) if "cache" in n else o[n][:, h:h + 1].contiguous()
    return o


def _spoil(c, r):
    """Makes some rows fail (a page id, a length) and returns them with the status they give."""
    B = c["q"].shape[0]
    bad = [int(x) for x in r.permutation(B)[:max(2, B // 10)]]
    for i, b in enumerate(bad):
        if i % 2 or c["kv_lens"][b] == 0:
            c["kv_lens"][b] = -1 - i
        else:
            c["block_table"][b, 0] = c["k_cache"].shape[0] + i
    return set(bad), sum({binding.STATUS_KVLEN if c["kv_lens"][b] < 0 else binding.STATUS_PAGE_OOB for b in bad})


@pytest.mark.parametrize("B,Sq,Hq,Hkv,lo,hi", [
    (60, 33, 8, 8, 1, 700),     # one q-tile of two: 480 units
    (8, 600, 32, 8, 600, 1100),  # 19 q-tiles: 640 units, those of the odd tile first
    (40, 130, 8, 4, 130, 400),  # 480 units of one or two KV tiles more or less
    (70, 40, 64, 8, 40, 300),   # 16 queries to a q-tile: three of them
])
def test_prefill_q8_units_after_one_another(B, Sq, Hq, Hkv, lo, hi):
    """Three units to a CTA or more, full and empty, good and failing: each row as when it runs
    alone (a unit to a CTA), and as in 64 bits."""
    r = np.random.RandomState(B + Sq)
    lens = [int(x) for x in r.randint(lo, hi + 1, B)]
    lens[B // 2] = lens[B // 3] = 0
    lens[1] = 128 * (hi // 128)
    c = ref.case(B * Sq, lens, Hq, Hkv, Sq=Sq)
    bad, bits = _spoil(c, r)
    st = torch.zeros(1, dtype=i32, device="cuda")
    out, lse = att._run(c, status=st, mode="prefill")
    assert int(st.item()) == bits
    for b in range(B):
        if b in bad:
            assert (out[b] == 0).all() and torch.isnan(lse[b]).all(), b
            continue
        one = att._run(att._rows(c, [b]), mode="prefill")
        assert att._equal([out[b:b + 1], lse[b:b + 1]], one), b
    G = Hq // Hkv
    good = [b for b in range(B) if b not in bad]
    for b, h in ((good[0], 0), (good[-1], Hkv - 1), (good[len(good) // 2], Hkv // 2)):
        att._check(_head(c, b, h), (out[b:b + 1, h * G:(h + 1) * G], lse[b:b + 1, h * G:(h + 1) * G]), att.PREFILL)


@pytest.mark.parametrize("B,Hq,Hkv,split", [(700, 8, 2, 0), (2100, 4, 1, 0), (2100, 4, 2, 16), (1500, 6, 3, 1 << 20)])
def test_decode_q8_large_batches(B, Hq, Hkv, split):
    """More rows than the threads that count their steps (640), than the list's entries (1024) and
    than twice those: each row as in a batch of fifty, and as in 64 bits."""
    r = np.random.RandomState(B + Hkv)
    lens = [int(x) for x in r.choice([0, 1, 15, 16, 17, 40, 100, 130, 300, 700], B, p=[.05, .1, .1, .1, .1, .2, .2, .1, .04, .01])]
    c = ref.case(B, lens, Hq, Hkv)
    bad, bits = _spoil(c, r)
    st = torch.zeros(1, dtype=i32, device="cuda")
    out, lse = att._run(c, split, status=st)
    assert int(st.item()) == bits
    gone = torch.tensor(sorted(bad))
    assert (out[gone] == 0).all() and torch.isnan(lse[gone]).all()
    good = [b for b in range(B) if b not in bad]
    d = [c[n].cuda() for n in ref.NAMES]
    for at in range(0, len(good), 50):
        rows = torch.tensor(good[at:at + 50], device="cuda")
        part = [t if n in ("k_cache", "v_cache", "k_scale", "v_scale") else t[rows].contiguous() for t, n in zip(d, ref.NAMES)]
        few = dict(c, q=part[0], block_table=part[5])
        assert att._equal([out[rows], lse[rows]], att._run(few, split, d=part)), at
    pick = good[::max(1, len(good) // 40)]
    att._check(att._rows(c, pick), (out[pick], lse[pick]), att.DECODE)


def test_decode_q8_many_rows_in_a_wide_table():
    """A table that holds long rows, with more rows and heads than the merge takes in quarters (512) and
    with fewer: the bits of a table as wide as the longest row."""
    lens = [33, 700, 1, 0, 513, 5000] + [40] * 60
    c = ref.case(131, lens, 16, 2)
    want = att._run(c)
    rows = list(range(len(lens)))
    assert len(rows) * 16 > 512
    assert att._equal(want, att._run(att._rows(c, rows, 1300)))
    few = [5, 1, 0]
    assert att._equal([x[few] for x in want], att._run(att._rows(c, few, 1300)))
    att._check(att._rows(c, few), [x[few] for x in want], att.DECODE)
