"""Pins of the oracle of chunks over the cache, key weights and eviction: closed forms and worked examples."""
import math

import numpy as np
import pytest

from oracle import kv_cache as okv


def test_masks_worked():
    m = okv.chunk_mask(5, 2, 1)
    assert m.astype(int).tolist() == [[1, 1, 1, 1, 0], [1, 1, 1, 1, 1]]
    m = okv.chunk_mask(6, 3, 2, window=2, sinks=1)
    assert m.astype(int).tolist() == [[1, 0, 1, 1, 0, 0], [1, 0, 0, 1, 1, 0], [1, 0, 0, 0, 1, 1]]
    m = okv.chunk_mask(4, 3, 4, prefix=3)
    assert m.astype(int).tolist() == [[1, 1, 1, 0], [1, 1, 1, 0], [1, 1, 1, 1]]
    assert okv.chunk_mask(3, 3, 0).all()
    assert not okv.chunk_mask(4, 2, 2).any()                  # no window, no sinks: queries without keys


def test_window_of_one_is_the_value():
    rng = np.random.default_rng(1)
    q, k, v = (rng.standard_normal((6, 8)) for _ in range(3))
    out, lse, _ = okv.attend_rows(q[3:], k, v, okv.chunk_mask(6, 3, 2, window=1), 0.5)
    assert np.allclose(out, v[3:], rtol=0, atol=1e-15)
    assert np.allclose(lse, 0.5 * np.sum(q[3:] * k[3:], -1), rtol=0, atol=1e-14)


def test_rows_are_the_causal_attention_of_a_whole():
    torch = pytest.importorskip("torch")
    rng = np.random.default_rng(2)
    q, k, v = (torch.from_numpy(rng.standard_normal((1, 1, 40, 16))) for _ in range(3))
    ref = torch.nn.functional.scaled_dot_product_attention(q, k, v, is_causal=True)[0, 0].numpy()
    for m in (1, 7, 40):
        out, _, _ = okv.attend_rows(q[0, 0, 40 - m:].numpy(), k[0, 0].numpy(), v[0, 0].numpy(),
                                    okv.chunk_mask(40, m, 1), 0.25)
        assert np.allclose(out, ref[40 - m:], rtol=0, atol=1e-13)


def test_weights_sum_to_the_queries():
    rng = np.random.default_rng(3)
    q, k, v = rng.standard_normal((5, 8)), rng.standard_normal((30, 8)), rng.standard_normal((30, 8))
    mask = okv.chunk_mask(30, 5, 1)
    out, lse, _ = okv.attend_rows(q, k, v, mask, 0.3)
    w = okv.weigh(q, lse, k, mask, 0.3)
    assert abs(w.sum() - 5) < 1e-12 and (w >= 0).all()
    one = okv.weigh(q[-1:], lse[-1:], k, mask[-1:], 0.3)
    assert np.allclose(one @ v, out[-1], rtol=0, atol=1e-13)
    assert not okv.weigh(q, np.full(5, -math.inf), k, mask, 0.3).any()


def test_evict_worked():
    w = [5.0, 1.0, 3.0, 3.0, 0.0, 3.0, 2.0, 0.0]
    assert okv.evict(w, 4, 0, 0).tolist() == [0, 2, 3, 5]
    assert okv.evict(w, 3, 0, 0).tolist() == [0, 2, 3]              # equal weights: the first
    assert okv.evict(w, 4, 2, 0).tolist() == [0, 2, 6, 7]
    assert okv.evict(w, 4, 1, 2).tolist() == [0, 1, 2, 7]
    assert okv.evict(w, 4, 4, 0).tolist() == [4, 5, 6, 7]
    assert okv.evict(w, 8, 1, 1).tolist() == list(range(8))
    assert okv.evict(w, 9, 1, 1).tolist() == list(range(8))
    assert okv.evict([math.nan, math.inf, -1.0, None, 0.0, -0.0], 4, 0, 0).tolist() == [0, 1, 4, 5]
    assert okv.evict([None, -math.inf, None, -1.0], 3, 0, 0).tolist() == [0, 1, 3]
