"""Row counts beyond the launch grid are refused on the host before anything is
enqueued, by the write + attend call before its write."""

import pytest

from tests.test_host_e2m1 import UNSUPPORTED, attend

ROWS = 65535 * 16


@pytest.mark.parametrize("write", [False, True])
@pytest.mark.parametrize("hq, mq", [(ROWS // 4 + 1, 5), (ROWS // 4 + 1, 4), (ROWS // 3 + 1, 3), (ROWS + 1, 1),
                                    (2 ** 31 - 1, 4), (2 ** 31 - 1, 1000)])
def test_too_many_rows_a_request(write, hq, mq):
    assert attend(write, hq=hq, hkv=1, mq=mq, tokens=mq, seqs=1, width=100, ms=1600) == UNSUPPORTED
