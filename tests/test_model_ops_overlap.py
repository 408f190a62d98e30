"""Which memory the model operators take as overlapping (on a machine without a GPU): with the environment check made to
fail, a call that gets past the overlap check returns that status instead."""
import ctypes

import pytest

from tests.test_model_ops_refusals import (ENV, OVERLAP, A, B, C, D, E, L, embedding, embedding_grad, layer_norm,  # noqa: F401
                                           layer_norm_grad, xent, xent_grad)

P = ctypes.c_void_p


@pytest.fixture(autouse=True)
def no_device(monkeypatch):
    monkeypatch.setenv("REPRO_FORCE_ENV_FAIL", "1")


def at(p, elements, size=2):
    return P(p.value + elements * size)


# matrices of 8 columns in rows of 16 and more: column slices of one buffer
SIDE_BY_SIDE = [
    (layer_norm, dict(ldx=16, ldy=16, y=at(A, 8))),
    (layer_norm, dict(ldx=24, ldy=24, y=at(A, 16))),
    (layer_norm, dict(ldx=24, ldy=24, x=at(A, 8), y=A)),
    (layer_norm, dict(ldx=16, ldy=16, y=at(A, 16 + 8))),                # from the next row on
    (layer_norm, dict(rows=1, ldx=8, ldy=8, y=at(A, 8))),
    (layer_norm_grad, dict(ldx=16, lddx=16, dx=at(B, 8))),
    (layer_norm_grad, dict(lddy=16, lddx=16, dx=at(A, 8))),
    (embedding, dict(ldw=16, ldo=16, out=at(A, 8))),
    (embedding, dict(n=1, ldw=16, ldo=8, out=at(A, 8))),                # one row has no stride of its own
    (embedding_grad, dict(lddy=32, lddw=32, dw=at(A, 24))),
    (xent_grad, dict(ldh=16, lddh=16, dh=at(B, 8))),
    (xent_grad, dict(ldw=16, lddw=16, dw=at(C, 8))),
    (xent_grad, dict(lddh=16, lddw=16, dw=at(P(0x60000000), 8))),       # dh next to dweight
]


@pytest.mark.parametrize("call,change", SIDE_BY_SIDE)
def test_column_slices_of_one_buffer_do_not_overlap(L, call, change):
    assert call(L, **change) == ENV


SHARED = [
    (layer_norm, dict(ldx=16, ldy=16, y=at(A, 7))), (layer_norm, dict(ldx=16, ldy=16, y=at(A, 9))),
    (layer_norm, dict(ldx=16, ldy=16, y=at(A, 16))), (layer_norm, dict(ldx=16, ldy=16, x=at(A, 8), y=at(A, 15))),
    (layer_norm, dict(ldx=16, ldy=24, y=at(A, 8))),                     # strides of their own
    (layer_norm_grad, dict(ldx=15, lddx=15, dx=at(B, 8))),
    (embedding, dict(n=1, ldw=16, ldo=8, out=at(A, 12))),
    (embedding, dict(n=1, cols=8, ldw=8, ldo=8, out=at(A, 8))),
    (embedding_grad, dict(lddy=32, lddw=32, dw=at(A, 32))),
    (xent_grad, dict(ldh=16, lddh=16, dh=at(B, 1))),
]


@pytest.mark.parametrize("call,change", SHARED)
def test_shared_elements(L, call, change):
    assert call(L, **change) == OVERLAP


# the same of vectors: tokens and labels (B, C, D below), weights, statistics; one element in common
VECTORS = [
    (embedding, dict(out=at(B, 3, 8))), (embedding_grad, dict(dw=at(B, 3, 8))),
    (layer_norm, dict(ldx=32, mean=at(A, 26))), (xent, dict(ldw=16, loss=at(B, 10))), (xent, dict(ldw=16, loss=at(B, 6))),
    (layer_norm, dict(y=at(B, 7))), (layer_norm, dict(y=at(C, 7))), (layer_norm, dict(mean=at(A, 30))),
    (layer_norm, dict(mean=at(B, 6))), (layer_norm, dict(rstd=at(C, 6))), (layer_norm, dict(rstd=A)),
    (layer_norm_grad, dict(dx=at(C, 7))), (layer_norm_grad, dict(dx=at(D, 3, 4))), (layer_norm_grad, dict(dx=E)),
    (layer_norm_grad, dict(dw=at(A, 31))), (layer_norm_grad, dict(dw=C)), (layer_norm_grad, dict(db=at(B, 31))),
    (layer_norm_grad, dict(db=at(D, 3, 4))), (layer_norm_grad, dict(dw=E)),
    (xent, dict(loss=A)), (xent, dict(loss=at(B, 78))), (xent, dict(lse=at(C, 3, 8))), (xent, dict(lse=A)),
    (xent_grad, dict(dh=at(A, 3, 4))), (xent_grad, dict(dh=D)), (xent_grad, dict(dw=E)), (xent_grad, dict(dw=at(D, 3, 8))),
]


@pytest.mark.parametrize("call,change", VECTORS)
def test_vectors_in_an_output(L, call, change):
    assert call(L, **change) == OVERLAP


@pytest.mark.parametrize("call,change", [
    (embedding, dict(out=at(B, 4, 8))), (layer_norm, dict(y=A)), (layer_norm, dict(y=at(B, 8))), (layer_norm, dict(mean=at(A, 32))),
    (layer_norm, dict(w=None, b=None)), (layer_norm_grad, dict(dx=A)), (layer_norm_grad, dict(dw=None, db=None)),
    (layer_norm_grad, dict(dx=at(D, 4, 4))), (xent, dict(loss=at(C, 4, 8))), (xent_grad, dict(dh=at(E, 4, 4))),
    # between two rows of a matrix, of another type
    (layer_norm, dict(ldx=32, mean=at(A, 8), rstd=at(A, 32 + 24))), (xent, dict(ldw=16, loss=at(B, 8)))])
def test_vectors_beside_an_output(L, call, change):
    assert call(L, **change) == ENV
