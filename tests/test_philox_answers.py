"""The published known answers of Philox 4x32-10 with every bit of counter and key in use (CPU only)."""
import pytest

from tests.test_gpu_ragged_more import words_at


@pytest.mark.parametrize("counter,key,want", [
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
])
def test_known_answers(counter, key, want):
    c0, c1, c2, c3 = counter
    words = words_at(c0 | c1 << 32, key[0] | key[1] << 32, c2 | c3 << 32)
    assert tuple(int(words[2 * i]) | int(words[2 * i + 1]) << 16 for i in range(4)) == want
