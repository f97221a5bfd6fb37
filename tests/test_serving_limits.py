"""Refusals of the serving calls at the limits of their arguments (CPU: the pointers are never
dereferenced, and nothing is launched)."""
import pytest

from compressed_kv_cache_gva_b200 import _build, gva

FAKE = 1 << 20


@pytest.fixture(scope="module")
def L():
    _build.build()
    return gva.lib()


def verify(L, n_rows, tokens=FAKE, out=2 * FAKE):
    return L.gva_verify_draft(3, 10, n_rows, tokens, FAKE, 0, FAKE, 10, None, 0, FAKE, FAKE, out, FAKE, None, None, None, None)


@pytest.mark.parametrize("n_rows", [2 ** 31 - 1, 2 ** 31 - 1024])
def test_verification_rows_that_a_block_would_count_past_31_bits(L, n_rows):
    assert verify(L, n_rows) == 1 and "n_rows" in L.gva_last_error().decode()


@pytest.mark.parametrize("shift", [0, 4, -4, 4 * 99, -4 * 99])
def test_verified_tokens_over_the_fed_ones(L, shift):
    assert verify(L, 100, out=FAKE + shift) == 1 and "overlap" in L.gva_last_error().decode()

