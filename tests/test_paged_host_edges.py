"""Host-side checks of the paged 4-bit cache at its limits (no GPU: no refused call gets that far)."""
import pytest

from test_paged_host import ATT, HEADS, kv, lib  # noqa: F401


@pytest.mark.parametrize("heads", [1 << 24, 1 << 30, 65536 + 2])
def test_attention_refuses_rows_beyond_32_bits(lib, heads):
    """2^24 heads of 128 are 2^31 values a row, which the kernels count in 32 bits."""
    a = {**ATT, "kv": kv(lib, hd=128), "H": heads, "ld_q": heads * 128, "n": 1}
    assert lib.status("rz_attention_paged_q4", *a.values()) == 2 and "n_heads" in lib.last_error()
    assert lib.load().rz_attention_paged_q4_workspace_bytes(heads, 2, 128) == 0 and "n_heads" in lib.last_error()


def test_heads_refuses_as_many(lib):
    a = {**HEADS, "kv": kv(lib), "H": 65537, "ld_q": 1 << 30, "ld_qo": 1 << 30}
    assert lib.status("rz_qk_norm_rope", *a.values()) == 2 and "n_heads" in lib.last_error()
