"""Part counts and workspace sizes of the decode over the 8-bit cache at the limits of their arguments (no GPU needed)."""
import pytest

from mla_decode_attention_03_gb300 import build, ops


@pytest.fixture(scope="module")
def lib():
    build.build()
    return ops.load_library()


@pytest.mark.parametrize("s_q,h_q", [(1 << 25, 128), (1 << 30, 4), (262141, 1), (0x7fffffff, 1)])
def test_more_rows_than_a_decode_takes(lib, s_q, h_q):
    assert lib.mla_num_parts_kv8(s_q, h_q, 1, 0) == -2
    assert lib.mla_workspace_bytes_kv8(1, s_q, h_q, 1, 4) == 0


def test_the_most_rows_that_a_decode_takes(lib):
    slots = 5 * 262140 * (512 + 1) * 4  # split-KV slots of output and lse
    assert lib.mla_workspace_bytes_kv8(1, 65535, 4, 1, 4) >= slots
