"""Hand-worked pins of the oracle of the serving operators (no GPU)."""

import math

import numpy as np

from oracle import serve as O


def test_e4m3_table_is_the_format():
    import torch
    t = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, O.E4M3)


def test_group_by_hand():
    # max 6 -> scale 1; the borders .25, .75, ... go to the even code
    x = np.array([6, 5, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, -6, -5, -3.5, -2.5, -1.75, -1.25, -0.75, -0.25])
    code, sb = O.quantise(x[None])
    assert O.E4M3[sb[0, 0]] == 1.0
    want = np.array([6, 4, 4, 2, 2, 1, 1, 0])
    assert np.array_equal(O.values(code, sb)[0], np.concatenate([want, -want]))
    assert np.array_equal(code[0, :8], [7, 6, 6, 4, 4, 2, 2, 0])


def test_scale_rounds_to_nearest_even_and_saturates():
    x = np.zeros((4, 16))
    x[0, 3] = 6 * 1.0625          # half way between 1 and 1.125: even mantissa 1
    x[1, 3] = 6 * 1.1875          # half way between 1.125 and 1.25: 1.25
    x[2, 3] = 1e6                 # saturates: 448 * 6
    x[3, 3] = 6 * 2.0 ** -10      # half way between 0 and the smallest scale: 0
    v = O.held(x)
    assert list(v[:, 3]) == [6.0, 6 * 1.25, 2688.0, 0.0]


def test_held_values_are_exact_in_16_bits():
    import torch
    prod = np.multiply.outer(O.E2M1, O.E4M3).ravel()
    for t in (torch.float16, torch.bfloat16):
        assert np.array_equal(torch.from_numpy(prod).to(t).double().numpy(), prod)


def test_rotation_by_hand():
    x = np.array([[1.0, 2.0] * 8])
    f = np.array([math.pi / 2] * 8)
    y = O.norm_rope(x, None, 0.0, f, [1], 16, True)       # a quarter turn of (1, 2)
    assert np.allclose(y, np.array([[-2.0, 1.0] * 8]))
    y = O.norm_rope(x, None, 0.0, f, [1], 16, False)      # pairs (1, 1) and (2, 2)
    assert np.allclose(y[0, :8], [-1, -2] * 4) and np.allclose(y[0, 8:], [1, 2] * 4)
    y = O.norm_rope(x, np.full(16, 2.0), 0.0, f, [0], 16, False)
    assert np.allclose(y, x / math.sqrt(2.5) * 2)


def test_attention_by_hand():
    k = np.zeros((3, 64))
    k[1, 0] = 8 * math.log(3)     # weights 1 : 3 with q = e_0
    q = np.zeros((2, 64))
    q[:, 0] = 1.0
    v = np.array([[1.0] * 64, [5.0] * 64, [100.0] * 64])
    out, lse, _ = O.attention(q, k, v, np.array([0, 4, -1]), np.array([4, -1]))
    assert np.allclose(out[0], 4.0) and math.isclose(lse[0], math.log(4))
    assert np.all(out[1] == 0) and lse[1] == -np.inf
