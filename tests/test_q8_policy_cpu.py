"""The library's policy text says how the 8-bit cache calls reduce (no GPU)."""


def test_policy_names_the_8_bit_calls():
    from deterministic_paged_kv_gb300 import binding, build
    build.build()
    binding.load()
    pol = dict(kv.split("=", 1) for kv in binding.policy().split(";"))
    assert pol["split_kv"] == "disabled"  # of the BF16 calls, as before
    assert "e4m3" in pol["q8_cache"] and "scale_per_page_and_kv_head" in pol["q8_cache"]
    # the splits that the scratch size tells: 512 tokens below token 16384, 1024 from there
    assert "512" in pol["q8_decode"] and "1024_from_16384" in pol["q8_decode"] and "ordered_fp32_merge" in pol["q8_decode"]
    one = binding.decode_q8_scratch_bytes(binding.plan(1, 1, 1, 1, 128, 16, 1, 64)) // 2
    for tokens, splits in ((16384, 32), (16400, 33), (17408, 33), (17424, 34)):
        assert binding.decode_q8_scratch_bytes(binding.plan(1, 1, 1, 1, 128, 16, 1, tokens // 16)) == splits * one
    assert "fp16" in pol["q8_prefill"] and "split_kv_disabled" in pol["q8_prefill"]
