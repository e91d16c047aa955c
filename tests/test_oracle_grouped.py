"""The 64-bit forms of the grouped operators against worked values and independent identities (CPU)."""
import numpy as np

import synth
from oracle import benq, grouped as og


def test_group_rows_worked():
    order, offsets = og.group_rows(np.array([2, 0, -1, 2, 0, 7]), 3)
    assert order.tolist() == [1, 4, 0, 3, -1, -1] and offsets.tolist() == [0, 2, 2, 4]


def test_route_worked():
    ninf = -np.inf
    l = np.array([[0.0, np.log(3.0), 0.0, ninf], [ninf, ninf, 1.0, ninf], [ninf] * 4], dtype=np.float64)
    e, w = og.route(l, 2, True)
    assert e.tolist() == [[1, 0], [2, -1], [-1, -1]]
    assert np.allclose(w, [[0.75, 0.25], [1, 0], [0, 0]])
    _, w = og.route(l, 2, False)
    assert np.allclose(w, [[0.6, 0.2], [1, 0], [0, 0]])


def test_grouped_linear_is_the_single_layer_per_row():
    G, N, K = 3, 5, 8
    ws = [synth.benq_weights(N, K, seed=s) for s in range(G)]
    codes, lut = np.stack([w.codes for w in ws]), np.stack([w.lut for w in ws])
    x = synth.activations(4, K, seed=9)
    xr = [3, 0, 2, 2, 1]
    y, _ = og.grouped_linear(codes, lut, x, [0, 2, 2, 5], xr, K)
    for i, g in enumerate([0, 0, 2, 2, 2]):
        assert np.allclose(y[i], benq.linear(ws[g].codes, ws[g].lut, x[xr[i]], K)[0], rtol=1e-14, atol=0)


def test_combine_and_lora_worked():
    out, _ = og.combine(np.array([[1.0, 2.0], [np.nan, np.nan]]), np.array([[4, -1]]), np.array([[0.5, 9.0]]),
                        np.array([[1.0, 1.0]]))
    assert out.tolist() == [[1.5, 2.0]]
    one = synth.f32_to_bf16_bits(np.array([1.0], dtype=np.float32))[0]
    two = synth.f32_to_bf16_bits(np.array([2.0], dtype=np.float32))[0]
    A, B = np.full((1, 2, 3), one), np.full((1, 1, 2), two)
    out, mag = og.lora(A, B, np.array([[10.0], [20.0]]), np.full((2, 3), one), [0, -1], [0.5])
    assert out.tolist() == [[16.0], [20.0]] and mag.tolist() == [[6.0], [0.0]]
