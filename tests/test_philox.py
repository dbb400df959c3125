"""The tests' generator against the known answers that its authors publish with
it, and its statistics."""
import numpy as np

from philox import border, philox, words


def test_known_answers():
    f = 0xFFFFFFFF
    for counter, key, want in (
            ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
            ((f, f, f, f), (f, f), (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
            ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0), (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))):
        assert tuple(int(v) for v in philox(counter, key)) == want


def test_layout():
    w = words(3, 10, 5 + (7 << 32), 11 + (13 << 32))
    for m, n in ((0, 0), (2, 9), (1, 4), (2, 3)):
        assert int(w[m, n]) == int(philox((n // 4, m, 11, 13), (5, 7))[n % 4])


def test_share_and_borders():
    w = words(64, 4096, 1234, 0)
    for p in (0.1, 0.5):
        got = float(np.mean(w < border(p)))
        assert abs(got - p) <= 6 * (p * (1 - p) / w.size) ** 0.5
    assert border(0.0) == 0 and border(1.0) == 2 ** 32 and border(0.5) == 2 ** 31
