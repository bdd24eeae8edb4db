"""The oracle of the cache of e4m3 codes against hand-worked cases."""
import math

import numpy as np
import torch

from oracle import cache8 as o8


def test_codes_agree_with_torch_and_saturate():
    x = torch.cat([torch.linspace(-500, 500, 4001), torch.logspace(-12, 3, 2000, base=2)])
    want = x.clamp(-448, 448).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(o8.code(x.double().numpy()), want)
    assert np.array_equal(o8.code([np.inf, -np.inf, 1e9]), [448, -448, 448]) and np.isnan(o8.code(np.nan))


def test_scales():
    assert o8.scale_for(448.0) == 1 and o8.scale_for(448.0001) == 2 and o8.scale_for(224.0) == 0.5
    assert o8.scale_for(0.0) == 2.0 ** -60 and o8.scale_for(1e38) == 2.0 ** 60
    assert np.array_equal(o8.as_read([0, -1, np.nan, 1e30, 3.0]), [2.0 ** -60] * 3 + [2.0 ** 60, 3])


def test_rotation():
    x = np.array([[[1.0, 2, 3, 4, 5]]])
    f = [math.pi / 2, math.pi]
    # position 1: the first pair by a quarter, the second by half a turn
    assert np.allclose(o8.rotate(x, [1], f, False), [[[-3, -2 * 1, 1, -4, 5]]])
    assert np.allclose(o8.rotate(x, [1], f, True), [[[-2, 1, -3, -4, 5]]])
    assert np.allclose(o8.rotate(x, [-1], f, True), [[[2, -1, -3, -4, 5]]])
    far = o8.rotate(x, [1 << 30], [0.1, 0.0], True)
    a = math.fmod((1 << 30) * 0.1, 2 * math.pi)
    assert np.allclose(far[0, 0, :2], [math.cos(a) - 2 * math.sin(a), 2 * math.cos(a) + math.sin(a)], atol=1e-6)


def test_append_begins_keeps_and_grows_a_block():
    codes, scales = np.zeros((2, 16, 1, 1)), np.ones((2, 1, 1))
    table = [[1]]
    c, s = o8.append(np.full((2, 1, 1), 100.0), [0, 2], codes, scales, table, [2])
    assert s[1] == 0.25 and np.array_equal(c[1, :2, 0, 0], [384, 384])       # 400 lies between 384 and 416: even
    c, s = o8.append(np.full((1, 1, 1), 3.0), [0, 1], c, s, table, [3])
    assert s[1] == 0.25 and c[1, 2] == 12
    c, s = o8.append(np.full((1, 1, 1), 1000.0), [0, 1], c, s, table, [4])
    assert s[1] == 4 and np.array_equal(c[1, :4, 0, 0], [24, 24, 0.75, 256])  # 250 to 256
    assert np.all(c[0] == 0) and s[0] == 1


def test_accept_takes_the_largest_scale():
    codes, scales = np.zeros((1, 2, 16, 1, 1)), np.array([1.0, 4.0]).reshape(1, 2, 1, 1)
    codes[0, 0, :, 0, 0] = np.arange(16) * 16
    codes[0, 1, :, 0, 0] = 32 + np.arange(16) % 8 * 4
    c, s, lens = o8.accept([[0, 3]], [0, 4], codes, scales, [[0, 1]], [18])
    # base 14: node 0 stays in place 14, node 3 (place 17, page 1) goes to place 15
    assert lens == [16] and np.array_equal(s[0, :, 0, 0], [4, 4])
    assert np.array_equal(c[0, 0, 13:, 0, 0], [52, 56, 36])
    assert np.array_equal(c[0, 0, :5, 0, 0], [0, 4, 8, 12, 16]) and np.array_equal(c[0, 1], codes[0, 1])
