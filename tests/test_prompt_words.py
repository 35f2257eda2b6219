"""The bound of the prompts' precision tests sees a word or a product that is left out."""
import numpy as np
import pytest

from tests.prompt_words import BOUND, bf16_product, f16_product

D = 128


def _operands():
    rng = np.random.default_rng(3)
    q = rng.standard_normal((200, D))
    q = (q / np.linalg.norm(q, axis=1, keepdims=True)).astype(np.float32)
    return q, (0.3 * rng.standard_normal((D, D))).astype(np.float32)


def _error(got, a, b):
    want = a.astype(np.float64) @ b.astype(np.float64)
    return np.linalg.norm(got - want) / np.linalg.norm(want)


def test_whole_operands_are_well_within_the_bound():
    q, S = _operands()
    assert _error(bf16_product(q, S, 3, 3), q, S) < BOUND / 4
    assert _error(f16_product(q, S), q, S) < BOUND / 4


@pytest.mark.parametrize("words", [(2, 3), (3, 2), (2, 2)])
def test_two_bf16_words_are_not(words):
    q, S = _operands()
    assert _error(bf16_product(q, S, *words), q, S) > 2 * BOUND


@pytest.mark.parametrize("lost", [(0, 2), (1, 1), (2, 0), (0, 1), (1, 0)])
def test_a_bf16_product_left_out_is_seen(lost):
    q, S = _operands()
    assert _error(bf16_product(q, S, 3, 3, [lost]), q, S) > 2 * BOUND


@pytest.mark.parametrize("lost", [(0, 1), (1, 0)])
def test_an_f16_product_left_out_is_seen(lost):
    q, S = _operands()
    assert _error(f16_product(q, S, [lost]), q, S) > 2 * BOUND


def test_a_bf16_row_beside_a_state_of_two_words_is_seen():
    # bf16 queries are one word; the state still needs three
    q, S = _operands()
    q = (q.view(np.uint32) & np.uint32(0xFFFF0000)).view(np.float32)
    assert _error(bf16_product(q, S, 1, 3), q, S) < BOUND / 4
    assert _error(bf16_product(q, S, 1, 2), q, S) > 2 * BOUND
