"""The definitions that the 4-bit matrices and dropout are tested against."""
import numpy as np

import mx4_ref as ref


def test_philox_known_answers():
    # the published answers of the generator for a counter and a key of zeros
    assert ref.philox([0] * 4, [0] * 2, 7) == [0x5f6fb709, 0x0d893f64, 0x4f121f81, 0x4f730a48]
    assert ref.philox([0] * 4, [0] * 2, 10) == [0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8]


def test_random16_is_philox():
    seed, step = 0x123456789abcdef0, 0xfedcba9876543210
    bits = ref.random16(3, 19, seed, step)
    for r in range(3):
        for c in range(19):
            w = ref.philox([c // 8, r, step & 0xffffffff, step >> 32],
                           [seed & 0xffffffff, seed >> 32])
            assert bits[r, c] == (w[c % 8 // 2] >> (16 * (c % 2))) & 0xffff
    assert np.array_equal(ref.random16(1, 5, seed, step, 2, 11), bits[2:3, 11:16])


def test_quantize_of_every_representable_value():
    rng = np.random.default_rng(0)
    codes, scales = ref.random_mx4(rng, 7, 70)
    # a block whose largest element is 4 or 6 keeps its scale
    codes[:, ::16] = 0x67
    values = ref.dequantize(codes, scales, 70)
    again, s = ref.quantize(values)
    assert np.array_equal(ref.dequantize(again, s, 70), values) and np.array_equal(s, scales)


def test_quantize_by_hand():
    w = np.zeros((1, 33))
    w[0, :12] = [7.9, 5, 5.01, 3.5, 2.5, 1.75, 0.25, 0.26, -0.75, -1.25, 6, 0]
    w[0, 32] = 2.0 ** -130
    codes, scales = ref.quantize(w)
    v = ref.dequantize(codes, scales, 33)
    assert v[0, :12].tolist() == [6, 4, 6, 4, 2, 2, 0, 0.5, -1, -1, 6, 0]
    assert scales.tolist() == [[127, 0]] and v[0, 32] == 0  # an eighth of the least scale
    w[0, 3] = np.inf
    codes, scales = ref.quantize(w)
    assert scales[0, 0] == 255 and np.isnan(ref.dequantize(codes, scales, 33)[0, :32]).all()
