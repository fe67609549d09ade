"""Sizes near the ends of 32 and 64 bits in the host side of the 8-bit cache calls (no GPU)."""
import pytest


@pytest.fixture(scope="module")
def rk():
    from deterministic_paged_kv_gb300 import binding, build
    build.build()
    binding.load()
    return binding


@pytest.mark.parametrize("B,Hq,Hkv,W,split", [
    (1 << 27, 8, 8, 1 << 24, 16), (1 << 27, 8, 1, 1 << 25, 16), (2 ** 31 - 1, 1, 1, 1 << 25, 0), (1 << 20, 8, 8, 1 << 20, 0)])
def test_decode_q8_scratch_bytes_of_a_plan_that_the_call_refuses(rk, B, Hq, Hkv, W, split):
    """A size of scratch is the call's own need, or the call's refusal; never a product that passed 64 bits."""
    p = rk.plan(B, 1, Hq, Hkv, 128, 16, 10, W)
    with pytest.raises(rk.RkError) as e:
        rk.decode_q8_scratch_bytes(p, split)
    assert e.value.name == "RK_E_UNSUPPORTED"


def test_decode_q8_scratch_bytes_of_the_largest_tables(rk):
    for B, Hq, Hkv, W in ((1, 8, 1, 1 << 24), (64, 64, 8, 1 << 20), (1, 64, 8, 1 << 25)):
        p = rk.plan(B, 1, Hq, Hkv, 128, 16, 10, W)
        cap = W * 16
        splits = 32 + -(-(cap - 16384) // 1024)
        assert rk.decode_q8_scratch_bytes(p) == B * Hq * splits * 129 * 4
        assert rk.decode_q8_scratch_bytes(p, 4096) == B * Hq * -(-cap // 4096) * 129 * 4
