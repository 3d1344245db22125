"""Host side of the paged serving operators (no GPU): pins of the oracle, what the C
entries refuse and accept without touching a device."""

import numpy as np

from oracle import serve_oracle as S


def test_slots_oracle_gives_unserved_requests_no_length():
    # request 1 wants two pages of one; request 2 none; request 3 is out of range
    got = S.slots([0, 0, 3, -2], [4, 5, 1, 3], np.zeros((4, 2), int), [0, 0, 1, 0],
                  np.array([4, 5]), 2, 4, 20)
    assert got["errors"] == {"blocks", "len"} and got["held"] == [1, 0, 1, 0]
    assert got["seq_lens"] == [4, -1, 4, -1]
