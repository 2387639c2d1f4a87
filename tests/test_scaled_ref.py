"""The tests' plain block-scaled formats against the formats' own tables and torch's E4M3."""
import numpy as np
import torch

from . import scaled_ref as S


def test_e4m3_values_and_rounding():
    codes = np.arange(127, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(S.decode(S.M8, codes), want)
    v = np.random.default_rng(0).standard_normal(4096) * np.exp2(np.random.default_rng(1).integers(-12, 9, 4096))
    v = np.clip(v, -448, 448).astype(np.float32)
    got = S.decode(S.M8, S.encode(S.M8, v.astype(np.float64)))
    assert np.array_equal(got, torch.from_numpy(v).to(torch.float8_e4m3fn).double().numpy())


def test_e2m1_ties_to_even():
    v = np.array([.25, .75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, -.25, -5.0])
    assert S.decode(S.NV, S.encode(S.NV, v)).tolist() == [0, 1, 1, 2, 2, 4, 4, 6, 0, -4]


def test_power_of_two_scales():
    for fmt, top in ((S.M8, 448.0), (S.M4, 6.0)):
        for a in (top, np.nextafter(np.float32(top), np.float32(1e9)), 1.0, 2.0 ** -126, 0.0, 3e38):
            x = np.zeros((1, 32), np.float32)
            x[0, 5] = a
            e = int(S.quantise(fmt, x)[1][0, 0]) - 127
            if a == 0:
                assert e == -127
            else:
                assert np.float64(np.float32(a)) <= top * 2.0 ** e and (e == -127 or np.float64(np.float32(a)) > top * 2.0 ** (e - 1))


def test_tiles_are_a_permutation():
    for fmt, n in ((S.NV, 192), (S.M8, 160), (S.M4, 128)):
        i = S.scale_index(fmt, n, np.arange(300))
        assert len(np.unique(i)) == i.size and i.max() < 3 * S.col_tiles(fmt, n) * 512
    # groups never share a row of the tiles
    off = [0, 0, 1, 128, 129, 400, 400]
    r = S.scale_rows(off, 513)
    assert len(np.unique(r)) == 513 and r.max() < (513 // 128 + len(off)) * 128


def test_four_bit_packing():
    c = np.arange(16, dtype=np.uint8)[None]
    assert S.pack(S.NV, c)[0, 0] == 0x10 and np.array_equal(S.unpack(S.NV, S.pack(S.NV, c)), c)
