"""The decoder-layer oracle against hand-worked values and plain identities (CPU)."""
import numpy as np

from oracle import layer


def test_e4m3_values_and_codes():
    assert layer.e4m3_value([0, 1, 8, 0x38, 0x7E, 0xB8]).tolist() == [0.0, 2.0 ** -9, 2.0 ** -6, 1.0, 448.0, -1.0]
    assert np.isnan(layer.e4m3_value([0x7F, 0xFF])).all()
    every = np.array([c for c in range(256) if c & 127 != 127], np.uint8)
    assert np.array_equal(layer.e4m3_code(layer.e4m3_value(every)), every)
    # ties to the even code: 17 lies between 16 (0x58) and 18 (0x59), 19 between 18 and 20 (0x5A)
    assert layer.e4m3_code([17.0, 19.0, 1e9, -np.inf, 2.0 ** -10, 1.5 * 2.0 ** -9]).tolist() == [0x58, 0x5A, 0x7E, 0xFE, 0, 2]
    assert layer.e4m3_code([np.nan])[0] & 127 == 127


def test_rotation_is_one_and_keeps_products_of_equal_distance():
    rng = np.random.default_rng(1)
    f = 100.0 ** (-np.arange(8) / 8)
    for inter in (False, True):
        x, z = rng.normal(size=(2, 1, 3, 24))
        r = lambda a, p: layer.rotate(a, [p], f, inter)  # noqa: E731
        assert np.allclose(np.linalg.norm(r(x, 977)), np.linalg.norm(x))
        assert np.allclose((r(x, 40) * r(z, 47)).sum(-1), (r(x, 0) * r(z, 7)).sum(-1))
        assert np.array_equal(r(x, 5)[..., 16:], x[..., 16:])
    one = layer.rotate(np.array([[[1.0, 0.0]]]), [1], [np.pi / 2], False)
    assert np.allclose(one, [[[0.0, 1.0]]])


def test_attend_by_hand():
    k = np.array([[[0.0]], [[1.0]], [[5.0]]])
    v = np.array([[[1.0]], [[3.0]], [[100.0]]])
    y, spread, size, reach = layer.attend(np.array([[[np.log(3.0)]], [[2.0]]]), k, v, np.array([[1, 1, 0], [0, 0, 0]], bool), 1.0)
    assert np.allclose(y[:, 0, 0], [0.25 * 1 + 0.75 * 3, 0.0]) and np.allclose(spread[0], 0.75) and np.allclose(size[0], 2.5)
    assert np.allclose(reach[:, 0], [np.log(3.0), 0.0])


def test_w4_format_positions():
    codes = np.zeros((16, 128), np.int64)
    codes[3, 32 * 2 + 8 * 1 + 5] = 9     # tile 0, chunk 2, word 1, element 5: bit 4*2 + 16
    buf = layer.w4_pack(codes, np.full((1, 16), 0.5), np.full((1, 16), 2.0)).view(np.uint32)
    at = (2 * 16 + 3) * 4 + 1
    assert buf[at] == 9 << 24 and np.count_nonzero(buf[:16 * 128 // 8]) == 1
    assert buf[16 * 128 // 8] == 0x3800 | (0x4000 << 16) and buf.size == 16 * 128 // 8 + 16
    w = layer.w4_matrix(codes, np.full((1, 16), 0.5), np.full((1, 16), 2.0))
    assert w[3, 77] == 3.5 and w[0, 0] == -1.0
