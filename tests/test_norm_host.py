"""The refusal of the RMS norm's token counts names the counts that it takes (CPU)."""
import ternary_quantized_moe_amd as tq


def test_token_counts_in_the_refusal():
    L = tq.lib()
    for T in (-1, 1 << 31):
        assert L.moe_rms_norm(0x100000, None, T, 256, 0x300000, 1e-6, None, 0x500000, None, None, None) == -3
        assert f"token count {T} outside [0, 2^31)" in L.moe_last_error().decode()
