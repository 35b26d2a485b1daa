"""A table of angles that are no numbers is refused on the host."""

from integer_only_dnn_amd import ie
from tests.test_abi_attention import NULL, OK, UNSUPPORTED, by, freqs


def table(f, rot=64, positions=1000, at=None):
    """Without a place for it, so that a good call ends at that."""
    return ie.lib().ie_rope_table(by(f), rot, positions, at, None)


def test_angles_past_float64():
    assert table(freqs()) == NULL
    # frequencies of up to 10^(307 * 255 / 256) and of 10^306, times 1000; without positions or pairs there are no angles
    for f in (freqs(base=1e-307), freqs(factor=1e-306), freqs(base=1e-307, trained=100.0), freqs(base=5e-324)):
        assert ie.lib().ie_rope_table(by(f), 512, 1000, 1 << 20, None) == UNSUPPORTED
    assert ie.lib().ie_rope_table(by(freqs(base=1e-307)), 512, 0, 1 << 20, None) == OK
    assert ie.lib().ie_rope_table(by(freqs(factor=1e-306)), 0, 1000, 1 << 20, None) == OK
