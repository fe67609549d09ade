"""rk_paged_tree_rows on the host (no GPU): what it refuses, and the binding's checks."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def rk():
    from deterministic_paged_kv_gb300 import binding, build
    build.build()
    binding.load()
    return binding


A = 1 << 20  # an aligned address that no call here reads


def test_refusals(rk):
    def call(plan, a):
        return rk.ERRORS.get(rk.load().rk_paged_tree_rows(ctypes.byref(plan) if plan else None, *a, None))
    p = rk.plan(2, 8, 8, 2, 128, 16, 10, 4)
    good = [A, A + 64, A + 128, A + 512, A + 1024, A + 2048]  # the last one the status word
    assert call(None, good) == "RK_E_ARG"
    assert call(rk.plan(2, 65, 8, 2, 128, 16, 10, 4), good) == "RK_E_UNSUPPORTED"
    for i in range(6):
        for bad in ((None, good[i] + 2) if i < 5 else (good[i] + 2,)):
            a = list(good)
            a[i] = bad
            assert call(p, a) == "RK_E_ARG" and rk.last_error()
    a = list(good)
    a[3] = a[1]  # the lengths that the trim needs
    assert call(p, a) == "RK_E_ARG" and "kv_lens" in rk.last_error()
    assert rk.load().rk_paged_tree_rows(ctypes.byref(rk.plan(0, 8, 8, 2, 128, 16, 10, 4)), *[None] * 6, None) == rk.RK_OK


def test_binding_checks(rk):
    p = rk.plan(2, 3, 8, 2, 128, 16, 10, 4)
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    t = [i(3), i(2), i(2, 3), i(2), i(2, 3)]
    with pytest.raises(ValueError, match="CUDA"):
        rk.tree_rows(p, *t)
    with pytest.raises(TypeError, match="qo_indptr"):
        rk.tree_rows(p, t[0].long(), *t[1:])
    with pytest.raises(ValueError, match="shape"):
        rk.tree_rows(p, i(2), *t[1:])
