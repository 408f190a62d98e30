"""Sizes next to the limits of the model operators' index arithmetic are refused before a pointer is looked at (on a
machine without a GPU)."""
import pytest

from tests.test_model_ops_refusals import CAPACITY, INVALID, L, embedding, embedding_grad  # noqa: F401

MOST = (1 << 31) - 1 - 4096


@pytest.mark.parametrize("cols", [MOST + 1, (1 << 31) - 8, (1 << 31) - 1])
def test_rows_whose_last_run_leaves_32_bits(L, cols):
    """The lookup counts the columns of a row's last run of up to 1024 in 32 bits, also those past the row."""
    assert embedding(L, vocab=1, cols=cols, ldw=cols, ldo=cols, w=None) == CAPACITY
    assert embedding_grad(L, vocab=1, cols=cols, lddy=cols, lddw=cols, dy=None) == CAPACITY


def test_the_widest_row_is_looked_at(L):
    assert embedding(L, vocab=1, cols=MOST, ldw=MOST, ldo=MOST, w=None) == INVALID
    assert embedding_grad(L, vocab=1, cols=MOST, lddy=MOST, lddw=MOST, dy=None) == INVALID
