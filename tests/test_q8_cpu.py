"""Host-side refusals of the 8-bit cache calls (no GPU: every check comes before
the device is touched) and pins of the plain statements that the GPU tests use."""
import ctypes

import numpy as np
import pytest
import torch

import q8_ref as ref


@pytest.fixture(scope="module")
def rk():
    from deterministic_paged_kv_gb300 import binding, build
    build.build()
    binding.load()
    return binding


A = 1 << 20  # a device address that is never followed


def _plan(rk, B=2, Sq=1, Hq=8, Hkv=2, NP=10, W=40):
    return rk.plan(B, Sq, Hq, Hkv, 128, 16, NP, W)


def _code(rk, rc):
    return {v: k for k, v in rk.CODES.items()}.get(rc, "RK_OK")


def test_tables_extend_refuses(rk):
    f = rk.load().rk_paged_tables_extend

    def call(p, change=None, n_pool=4, cap=8):
        ptr = dict(zip(["n_new", "kv", "pool", "taken", "bt", "kvo", "tko", "ip", "pos", "slot"], [A] * 10))
        ptr.update(change or {})
        return _code(rk, f(ctypes.byref(p) if p is not None else None, ptr["n_new"], ptr["kv"], ptr["pool"], n_pool,
                           ptr["taken"], ptr["bt"], ptr["kvo"], ptr["tko"], ptr["ip"], ptr["pos"], ptr["slot"], cap, None, None))

    assert call(None) == "RK_E_ARG"
    assert call(rk.Plan()) == "RK_E_ARG"
    p = _plan(rk)
    for n in ("n_new", "kv", "pool", "taken", "bt", "kvo", "tko", "ip", "pos", "slot"):
        assert call(p, {n: None}) == "RK_E_ARG", n
        assert call(p, {n: A + 2}) == "RK_E_ARG", n
    assert call(p, n_pool=-1) == "RK_E_ARG" and call(p, cap=-1) == "RK_E_ARG"
    assert call(_plan(rk, B=16385)) == "RK_E_UNSUPPORTED"


def test_append_q8_refuses(rk):
    f = rk.load().rk_paged_kv_append_q8

    def call(p, n=3, at=None, value=None):
        ptr = [A] * 8
        if at is not None:
            ptr[at] = value
        return _code(rk, f(ctypes.byref(p) if p is not None else None, n, *ptr, None, None))

    p = _plan(rk)
    assert call(None) == "RK_E_ARG" and call(rk.Plan()) == "RK_E_ARG"
    assert call(p, n=-1) == "RK_E_ARG" and call(p, n=0) == "RK_OK"
    assert call(_plan(rk, NP=0)) == "RK_E_KVLEN"
    for i in range(8):
        assert call(p, at=i, value=None) == "RK_E_ARG", i
        assert call(p, at=i, value=A + 2) == "RK_E_ARG", i
    for i in (0, 1, 4, 5):
        assert call(p, at=i, value=A + 8) == "RK_E_ARG", i


def test_attention_q8_refuses(rk):
    lib = rk.load()

    def decode(p, split=0, at=None, value=None, scratch=A, nbytes=1 << 40):
        ptr = [A] * 10
        if at is not None:
            ptr[at] = value
        return _code(rk, lib.rk_paged_attn_decode_q8(ctypes.byref(p) if p is not None else None, split, *ptr, scratch, nbytes,
                                                     None, None))

    def prefill(p, at=None, value=None):
        ptr = [A] * 10
        if at is not None:
            ptr[at] = value
        return _code(rk, lib.rk_paged_attn_prefill_q8(ctypes.byref(p) if p is not None else None, *ptr, None, None))

    p = _plan(rk)
    for f in (decode, prefill):
        assert f(None) == "RK_E_ARG" and f(rk.Plan()) == "RK_E_ARG"
        for i in range(10):
            assert f(p, at=i, value=None) == "RK_E_ARG", i
            assert f(p, at=i, value=A + 2) == "RK_E_ARG", i
        assert f(_plan(rk, B=0)) in ("RK_OK",)
    assert decode(_plan(rk, Sq=2)) != "RK_OK"
    n = rk.decode_q8_scratch_bytes(p)
    assert n == 2 * 8 * 2 * 129 * 4 and rk.decode_q8_scratch_bytes(p, 640) == 0  # 640 tokens, a split at 512
    assert rk.decode_q8_scratch_bytes(_plan(rk, W=32)) == 0 and rk.decode_q8_scratch_bytes(_plan(rk, W=33)) == 2 * 8 * 2 * 129 * 4
    assert rk.decode_q8_scratch_bytes(_plan(rk, W=65)) == 2 * 8 * 3 * 129 * 4       # 512, 1024
    assert rk.decode_q8_scratch_bytes(_plan(rk, W=1025)) == 2 * 8 * 33 * 129 * 4    # 32 below 16384, one from there
    assert rk.decode_q8_scratch_bytes(_plan(rk, W=1089)) == 2 * 8 * 34 * 129 * 4
    assert rk.decode_q8_scratch_bytes(p, 16) == 2 * 8 * 40 * 129 * 4
    for split in (-16, 8, 17):
        assert decode(p, split=split) == "RK_E_ARG"
    assert decode(p, scratch=None) == "RK_E_ARG" and decode(p, scratch=A + 8) == "RK_E_ARG"
    assert decode(p, nbytes=n - 1) == "RK_E_ARG"


def test_scratch_bytes_refuses(rk):
    p = _plan(rk)
    for split in (-16, 8, 17):
        with pytest.raises(rk.RkError) as e:
            rk.decode_q8_scratch_bytes(p, split)
        assert e.value.name == "RK_E_ARG"
    with pytest.raises(rk.RkError):
        rk.decode_q8_scratch_bytes(rk.Plan())


def test_binding_refuses_tensors(rk):
    p = _plan(rk)
    i32 = torch.int32
    ok = dict(k_new=torch.zeros((3, 2, 128), dtype=torch.bfloat16), v_new=torch.zeros((3, 2, 128), dtype=torch.bfloat16),
              slot_map=torch.zeros(3, dtype=i32), position_ids=torch.zeros(3, dtype=i32),
              k_cache=torch.zeros((10, 2, 16, 128), dtype=torch.uint8).view(ref.F8),
              v_cache=torch.zeros((10, 2, 16, 128), dtype=torch.uint8).view(ref.F8), k_scale=torch.ones(10, 2),
              v_scale=torch.ones(10, 2))
    with pytest.raises(ValueError, match="CUDA tensor"):
        rk.kv_append_q8(p, **ok)
    entries = [(t, t.dtype, t.shape, n) for n, t in ok.items()]
    for name, bad, err in (("k_new", ok["k_new"].float(), TypeError), ("v_new", ok["v_new"][:2], ValueError),
                           ("k_cache", ok["k_cache"].view(torch.uint8), TypeError), ("v_cache", ok["v_cache"][:9], ValueError),
                           ("k_scale", ok["k_scale"].double(), TypeError), ("position_ids", ok["position_ids"][:2], ValueError),
                           ("slot_map", ok["slot_map"].long(), TypeError)):
        with pytest.raises(err, match=name):
            rk._pointers([(bad, dt, sh, n) for t, dt, sh, n in entries if n == name])
    with pytest.raises(ValueError):
        rk.tables_extend(p, *[torch.zeros(3, dtype=i32)] * 10)


def test_pin_round4_is_e4m3_without_subnormals():
    """Every e4m3 value is a fixed point, and values between round as the type does."""
    codes = torch.arange(256, dtype=torch.uint8).view(ref.F8).float().double().numpy()
    codes = codes[np.isfinite(codes)]
    normal = codes[np.abs(codes) >= 2.0 ** -6]
    assert np.array_equal(ref.round4(normal), normal)
    x = np.random.RandomState(0).uniform(2.0 ** -6, 440, 20000)
    want = torch.from_numpy(x).float().to(ref.F8).float().double().numpy()
    assert np.array_equal(ref.round4(x.astype(np.float32).astype(np.float64)), want)
    assert ref.round4(np.array([31 / 2048, np.nextafter(31 / 2048, 0)])).tolist() == [2.0 ** -6, 0.0]


def test_pin_cache_composes():
    """Rounding, then moving to a larger scale, is rounding at the larger scale."""
    x = np.random.RandomState(1).standard_normal(5000) * 2.0 ** np.random.RandomState(2).randint(-12, 8, 5000)
    for by in range(0, 14):
        assert np.array_equal(ref.round4(np.ldexp(ref.round4(x), -by)), ref.round4(np.ldexp(x, -by)))


def test_pin_attention_closed_forms():
    c = ref.case(1, [1, 33], 4, 2)
    out, lse, _ = ref.attention(*[c[n] for n in ref.NAMES])
    pg = int(c["block_table"][0, 0])
    v = c["v_cache"].to(torch.float32)[pg, 1, 0] * c["v_scale"][pg, 1]
    assert np.allclose(out[0, 2, 0], v.double().numpy(), rtol=1e-12)          # one key: its value
    c["q"].zero_()
    out, lse, _ = ref.attention(*[c[n] for n in ref.NAMES])
    assert np.allclose(lse[1], np.log(33), rtol=1e-12)                        # equal scores
    x = np.random.RandomState(3).standard_normal((2, 128))
    for a, b in ((5, 9), (100, 104)):                                         # scores depend on the distance
        s = ref.rotate(x[0], a) @ ref.rotate(x[1], b)
        assert np.isclose(s, ref.rotate(x[0], 0) @ ref.rotate(x[1], 4), rtol=1e-9)


def test_pin_tables():
    got, said = ref.tables([2, 0, 17], [15, 3, 0], [7, 4, 9, 2], 1, [[5, -1, -1], [1, -1, -1], [-1, -1, -1]], 20, 10)
    assert said == set() and got["taken"] == 4 and got["qo_indptr"] == [0, 2, 2, 19] and got["kv_lens"] == [17, 3, 17]
    assert got["block_table"].tolist() == [[5, 4, -1], [1, -1, -1], [9, 2, -1]]
    assert got["slot_map"] == [95, 64] + list(range(144, 160)) + [32, -1] and got["position_ids"][:3] == [15, 16, 0]
