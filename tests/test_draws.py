"""The tests' own draws of dropout: Philox4x32-10 against the answers published with its definition."""
import numpy as np
import pytest

import draws64 as D


@pytest.mark.parametrize("counter,key,want", [
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0), (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
])
def test_known_answers(counter, key, want):
    assert tuple(int(v) for v in D.philox(counter, key)) == want


@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 0.999, 1.0])
def test_share_kept(p):
    """2^18 draws: the share kept is within five deviations of 1 - p as taken."""
    k = D.keep(256, 1024, p, seed=-5, step=3, site=2)
    q = 1 - D.cut_of(p) / 65536
    assert abs(float(k.double().mean()) - q) <= 5 * np.sqrt(q * (1 - q) / 2 ** 18)


def test_columns_do_not_depend_on_the_width():
    a, b = D.keep(5, 64, 0.3, 7, 1, 0), D.keep(5, 61, 0.3, 7, 1, 0)
    assert (a[:, :61] == b).all()
    assert (a[2:] == D.keep(3, 64, 0.3, 7, 1, 0, row0=2)).all()
    assert (a != D.keep(5, 64, 0.3, 7, 2, 0)).any() and (a != D.keep(5, 64, 0.3, 7, 1, 1)).any() and (a != D.keep(5, 64, 0.3, 8, 1, 0)).any()
