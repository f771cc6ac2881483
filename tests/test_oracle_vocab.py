"""Pins for the oracle's vocabulary projection and token log probabilities (CPU only)."""
import numpy as np
import torch

from oracle import vocab as O


def test_e4m3_values_and_rounding_agree_with_torch():
    codes = torch.arange(256, dtype=torch.uint8)
    np.testing.assert_array_equal(O.e4m3_values(), codes.view(torch.float8_e4m3fn).double().numpy())
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.standard_normal(4000) * 10.0 ** rng.uniform(-4, 2.6, 4000), O.e4m3_values()[:127],
                        (O.e4m3_values()[:126] + O.e4m3_values()[1:127]) / 2])  # values and every tie
    x = np.clip(x, -448, 448).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(O.e4m3_round(x.astype(np.float64)), want)


def test_quant_hand_worked_block():
    x = np.zeros((2, 130))
    x[0, 0], x[0, 1], x[1, 129] = 2.0, -1.0, np.inf
    scaled, scale = O.quant(x, 1)
    assert scaled[0, 0] == 448 and scaled[0, 1] == -224 and np.isnan(scaled[1, 129])
    assert scale[0, 0] == 2 / 448 and scale[1, 1] == 2.0 ** -100 / 448
    both, s2 = O.quant(x, 128)
    assert s2.shape == (1, 2) and s2[0, 0] == 2 / 448 and both[1, 0] == 0


def test_matmul_of_scaled_identity():
    one = 0x38  # e4m3 code of 1.0
    a = np.zeros((3, 200), np.uint8)
    w = np.zeros((200, 200), np.uint8)
    a[0, 5], a[1, 150], a[2, 199] = one, one, one
    np.fill_diagonal(w, one)
    sa = np.arange(6, dtype=float).reshape(3, 2) + 1
    sw = np.array([[1.0, 10.0], [100.0, 1000.0]])
    y, mag = O.matmul(a, sa, w, sw)
    want = np.zeros((3, 200))
    want[0, 5], want[1, 150], want[2, 199] = 1 * 1, 4 * 1000, 6 * 1000
    np.testing.assert_array_equal(y, want)
    np.testing.assert_array_equal(mag, want)


def test_logprobs_closed_forms():
    # a uniform row, a two-candidate row at T = 2, a row with nothing left
    z = np.zeros((3, 8))
    z[1] = [np.log(9.0) * 2, 0, -np.inf, np.nan, 0, 0, 0, 0]
    z[2] = -np.inf
    mask = np.array([[0xFF], [0b111], [0xFF]])
    o = O.token_logprobs(z, [3, 1, 0], [0.0, 2.0, 1.0], 3, mask)
    np.testing.assert_allclose(o["logprob"], [-np.log(8), np.log(0.1), -np.inf])
    np.testing.assert_allclose(o["entropy"], [np.log(8), -0.9 * np.log(0.9) - 0.1 * np.log(0.1), 0], rtol=1e-12)
    np.testing.assert_array_equal(o["rank"], [3, 1, -1])
    np.testing.assert_array_equal(o["top_id"], [[0, 1, 2], [0, 1, -1], [-1, -1, -1]])
    np.testing.assert_allclose(o["row_stat"][1], [np.log(9.0) * 2, 10 / 9])


def test_gradient_is_the_difference_quotient_of_the_loss():
    rng = np.random.default_rng(3)
    N, V, top = 6, 17, 3
    z = rng.standard_normal((N, V)) * 2
    z[1, 4] = -np.inf
    mask = rng.integers(0, 2 ** 17, (N, 1)) | 1
    mask[2] = 0
    tok = np.array([0, 4, 3, -1, 0, 16])
    T = np.array([1.0, 0.5, 1.0, 2.0, 0.0, 0.7])
    tid = O.token_logprobs(z, tok, T, top, mask)["top_id"]
    g = [rng.standard_normal(N), rng.standard_normal(N), rng.standard_normal((N, top))]
    d = O.token_logprobs_grad(z, tok, T, tid, *g, mask)
    h = 1e-6
    for v in range(V):
        e = np.zeros(V)
        e[v] = h
        num = (O.loss(z + e, tok, T, tid, *g, mask) - O.loss(z - e, tok, T, tid, *g, mask)) / (2 * h)
        np.testing.assert_allclose(d[:, v], num, atol=1e-8)
    assert (d[2] == 0).all()
    np.testing.assert_allclose(d.sum(1), 0, atol=1e-12)
