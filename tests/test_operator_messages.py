"""What a refusal says is true of the operation that refused (no GPU needed): each limit below is
asked of the entry point, and has to stand in the status's text."""
import pytest

import moe_expert_routing_sort_gb300 as mrs
from moe_expert_routing_sort_gb300 import _build

BASE = 0x7F0000000000


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return mrs.load()


def test_row_lengths(lib):
    def quantize(cols):  # (the misaligned codes are looked at behind the length)
        return lib.moe_fp8_quantize(BASE, 0, 1, cols, cols, BASE + 4, BASE, None)

    def swiglu(cols):
        return lib.moe_swiglu(BASE, 0, 2 * cols, 1, cols, None, BASE + 4, None, None, None)

    for call in (quantize, swiglu):
        assert [call(c) for c in (0, 12, 16392)] == [-18] * 3 and [call(c) for c in (8, 16384)] == [-8] * 2
    text = mrs.strerror(-18)
    assert "of 8 in [8, 16384]" in text and "of 32 in [32, 32768]" in text and "[8, 65536]" in text
    assert "16, up to 65536" in text


def test_parts_and_eps(lib):
    def norm(parts=1, eps=0.0):
        return lib.moe_rms_norm(BASE, 0, 64, parts, None, 64, 1, 64, BASE, 0, eps, BASE + 4, None, None,
                                None, None, None)

    assert norm() == -8 and norm(parts=32) == -8 and norm(eps=1.0) == -8
    assert norm(parts=33) == -4 and "a token's rows) must be in [1, 32]" in mrs.strerror(-4)
    assert norm(eps=1.5) == -11 and "eps in [0, 1]" in mrs.strerror(-11)


def test_alignment_and_sizes(lib):
    assert lib.moe_fp8_quantize(BASE + 8, 0, 1, 64, 64, BASE, BASE, None) == -8
    assert lib.moe_fp8_quantize(BASE, 0, 1, 64, 64, BASE + 0x1004, BASE, None) == -8
    assert "16-byte aligned" in mrs.strerror(-8) and "8-bit codes 8-byte" in mrs.strerror(-8)
    assert lib.moe_fp8_quantize(BASE, 0, 1 << 31, 64, 64, BASE, BASE, None) == -7
    assert "a number of rows or a row stride" in mrs.strerror(-7)
