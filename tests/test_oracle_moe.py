"""Pins of the oracle of the operators around the experts and of the adapters: values worked out by
hand, and agreement with torch's float64 operations."""
import numpy as np
import torch

from oracle import moe_oracle as o

NEG = -np.inf


def test_route_by_hand():
    l = np.log(np.array([[1.0, 2.0, 4.0, 1.0]]))
    e, w = o.route(l, 2)
    assert e.tolist() == [[2, 1]] and np.allclose(w, [[2 / 3, 1 / 3]], atol=1e-15)
    e, w = o.route(l, 2, renormalize=False, scale=2.0)
    assert np.allclose(w, [[1.0, 0.5]], atol=1e-15)
    e, w = o.route(l, 2, bias=np.array([0.9, 0, 0, 0]))            # the bias chooses, the weights leave it out
    assert e.tolist() == [[0, 2]] and np.allclose(w, [[0.2, 0.8]], atol=1e-15)
    e, w = o.route(l, 3, sigmoid=True, renormalize=False)          # sigmoid(log v) = v / (1 + v)
    assert e.tolist() == [[2, 1, 0]] and np.allclose(w, [[0.8, 2 / 3, 0.5]], atol=1e-15)


def test_route_groups_ties_and_masks_by_hand():
    l = np.array([[3.0, 0.0, 2.0, 2.0, 2.5, 0.0]])
    assert o.route(l, 2, groups=3, topk_groups=1)[0].tolist() == [[0, 1]]
    assert o.route(l, 2, groups=3, topk_groups=2)[0].tolist() == [[0, 4]]
    zero = np.zeros(6)
    s = 1 / (1 + np.exp(-l[0]))                                    # pairs: 1.45, 1.76, 1.42
    assert s[2] + s[3] > s[0] + s[1] > s[4] + s[5]
    assert o.route(l, 2, bias=zero, sigmoid=True, groups=3, topk_groups=1, best=2)[0].tolist() == [[2, 3]]
    assert o.route(np.zeros((1, 5)), 3)[0].tolist() == [[0, 1, 2]]
    e, w = o.route(np.array([[NEG, 1.0, NEG, NEG]]), 2)
    assert e.tolist() == [[1, -1]] and w.tolist() == [[1.0, 0.0]]
    e, w = o.route(np.full((1, 4), NEG), 2)
    assert e.tolist() == [[-1, -1]] and w.tolist() == [[0.0, 0.0]]
    e, w = o.route(np.array([[0.0, np.nan, 1.0]]), 2)
    assert e.tolist() == [[0, 1]] and np.isnan(w).all()


def test_route_agrees_with_torch():
    g = torch.Generator().manual_seed(0)
    l = torch.randn(40, 33, generator=g, dtype=torch.float64)
    w, e = torch.softmax(l, 1).topk(5, 1)
    got = o.route(l.numpy(), 5, renormalize=False)
    assert np.array_equal(got[0], e.numpy()) and np.allclose(got[1], w.numpy(), atol=1e-14)
    b = torch.randn(33, generator=g, dtype=torch.float64)
    e = (torch.sigmoid(l) + b).topk(5, 1).indices
    w = torch.sigmoid(l).gather(1, e)
    got = o.route(l.numpy(), 5, bias=b.numpy(), sigmoid=True)
    assert np.array_equal(got[0], e.numpy()) and np.allclose(got[1], (w / w.sum(1, keepdim=True)).numpy(), atol=1e-14)


def test_group_rows_by_hand():
    ids = np.array([[2, 0], [0, 5], [2, -1]])
    rows, offsets, position = o.group_rows(ids, 3)
    assert offsets.tolist() == [0, 2, 2, 4] and rows.tolist() == [0, 1, 0, 2, 1, 2]
    assert position.tolist() == [[2, 0], [1, -1], [3, -1]]


def test_combine_and_lora_by_hand():
    y = np.array([[1.0, 2.0], [3.0, 4.0]])
    out, A = o.combine(y, np.array([[1, 0], [-1, 0]]), np.array([[2.0, -1.0], [9.0, 1.0]]), np.ones((2, 2)))
    assert out.tolist() == [[6.0, 7.0], [2.0, 3.0]] and A.tolist() == [[8.0, 11.0], [2.0, 3.0]]
    x, a, b = np.array([[1.0, 2.0], [1.0, 1.0]]), np.array([[[3.0, 4.0]]]), np.array([[[2.0], [-1.0], [0.0]]])
    y, At, Ab, Am = o.lora(x, a, b, np.array([0.5]), np.array([0, -1]), np.ones((2, 3)))
    assert y.tolist() == [[12.0, -4.5, 1.0], [1.0, 1.0, 1.0]]      # t = 11
    assert Ab[0].tolist() == [11.0, 5.5, 0.0] and Am[0].tolist() == [11.0, 5.5, 0.0] and (At[1] == 0).all()
