"""Pins of the FP64 expert definitions (no GPU): closed forms, library
functions, the input generator's own layout, brute force."""

import numpy as np
import pytest
import torch

import oracle as O
from moe_decode_layer_logits_gb300.inputs import draw_bf16, expert_sorted_map


def test_softmax_renormalised_is_the_topk_route():
    lg = np.random.default_rng(0).standard_normal((20, 64)).astype(np.float32)
    ids, w = O.group_topk_route(lg, 6, 2.5, scores="softmax", renormalize=True)
    rids, _, rw = O.topk_route(lg, 6, 2.5)
    assert np.array_equal(ids, rids) and np.allclose(w, rw, rtol=1e-14, atol=0)


def test_scores_are_the_library_functions():
    lg = np.random.default_rng(1).standard_normal((9, 32)).astype(np.float32) * 3
    z = torch.from_numpy(lg).double()
    for scores, fn in [("sigmoid", torch.sigmoid), ("softmax", lambda v: torch.softmax(v, 1))]:
        ids, w = O.group_topk_route(lg, 5, 1.0, scores=scores, renormalize=False)
        want = fn(z).sort(dim=1, descending=True, stable=True)
        assert np.array_equal(ids, want.indices[:, :5].numpy())
        assert np.allclose(w, want.values[:, :5].numpy(), rtol=1e-13, atol=0)


def test_bias_moves_the_choice_and_not_the_weights():
    lg = np.array([[0.0, 1.0, 2.0, 3.0]], np.float32)
    bias = np.array([10.0, 0.0, 0.0, -10.0], np.float32)
    ids, w = O.group_topk_route(lg, 2, 1.0, bias=bias, renormalize=False)
    assert ids.tolist() == [[0, 2]]
    assert np.allclose(w, [[0.5, 1 / (1 + np.exp(-2.0))]], rtol=1e-15)


def test_groups_by_their_two_best_or_their_best():
    # group 0 holds the best expert, group 1 the best pair
    lg = np.array([[5.0, -9.0, 3.0, 2.9]], np.float32)
    b = np.zeros(4, np.float32)
    assert O.group_topk_route(lg, 1, 1.0, bias=b, n_group=2, topk_group=1, group_top=1)[0].tolist() == [[0]]
    assert O.group_topk_route(lg, 1, 1.0, bias=b, n_group=2, topk_group=1, group_top=2)[0].tolist() == [[2]]


def test_ties_and_masked_rows():
    lg = np.zeros((1, 8), np.float32)
    ids, w = O.group_topk_route(lg, 3, 3.0, n_group=4, topk_group=2)
    assert ids.tolist() == [[0, 1, 2]] and np.allclose(w, 1.0)
    none = np.full((1, 8), -np.inf, np.float32)
    for scores in ("sigmoid", "softmax"):
        ids, w = O.group_topk_route(none, 3, 3.0, scores=scores)
        assert ids.tolist() == [[0, 1, 2]] and np.all(w == 0)


@pytest.mark.parametrize("block", [0, 1, 16])
def test_map_is_the_input_generators_layout(block):
    emap, rows, experts = expert_sorted_map(np.random.default_rng(3), 23, 40, 5, block)
    row_map, row_token, offsets, counts = O.expert_map(experts, 40, max(block, 1))
    assert np.array_equal(row_map, emap) and offsets[-1] == rows
    assert np.array_equal(row_token[row_map], np.repeat(np.arange(23), 5).reshape(23, 5))
    assert counts.sum() == 23 * 5 and (row_token >= 0).sum() == 23 * 5


def test_products_against_torch_and_planted_mistakes():
    rng = np.random.default_rng(4)
    E, N, K, T, k = 4, 16, 24, 7, 2
    x, w = draw_bf16(rng, (T, K), 1.0), draw_bf16(rng, (E, N, K), 0.3)
    ids = np.argsort(rng.random((T, E)), axis=1)[:, :k]
    row_map, row_token, offsets, counts = O.expert_map(ids, E)
    xd, wd = torch.from_numpy(O.bf16_bits_to_f64(x)), torch.from_numpy(O.bf16_bits_to_f64(w))
    got = O.expert_linear(x, w, offsets, counts, row_token, act="swiglu")
    plain = O.expert_linear(x, w, offsets, counts, row_token)
    for t in range(T):
        for j in range(k):
            y = wd[ids[t, j]] @ xd[t]
            want = torch.nn.functional.silu(y[: N // 2]) * y[N // 2:]
            assert np.allclose(plain[row_map[t, j]][0], y.numpy(), rtol=1e-12, atol=1e-14)
            assert np.allclose(got[row_map[t, j]][0], want.numpy(), rtol=1e-12, atol=1e-14)
            swapped = torch.nn.functional.silu(y[N // 2:]) * y[: N // 2]  # up taken for gate
            assert not np.allclose(got[row_map[t, j]][0], swapped.numpy(), rtol=1e-3)


def test_adapter_is_the_merged_weight():
    rng = np.random.default_rng(5)
    T, N, K, R, L = 6, 24, 32, 8, 3
    x, w = draw_bf16(rng, (T, K), 1.0), draw_bf16(rng, (N, K), 0.2)
    a, b = draw_bf16(rng, (L, R, K), 0.2), draw_bf16(rng, (L, N, R), 0.2)
    scale = np.array([0.5, 2.0, 1.0], np.float32)
    ids = np.array([0, 2, -1, 1, 1, 3])
    y, _ = O.adapter_linear(x, w, a, b, ids, scale)
    f = O.bf16_bits_to_f64
    for t, i in enumerate(ids):
        merged = f(w) + (scale[i] * f(b)[i] @ f(a)[i] if 0 <= i < L else 0)
        assert np.allclose(y[t], merged @ f(x)[t], rtol=1e-12, atol=1e-13)
