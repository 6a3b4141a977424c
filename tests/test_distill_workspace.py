"""The workspace of idx_distill for a batch and length serves every smaller one (no GPU: sizes and refusals alone)."""
import pytest

from test_abi import FAKE, call, fx  # noqa: F401


def test_the_size_grows_with_rows_and_length(fx):
    rows = list(range(1, 40)) + [63, 64, 65, 100, 127, 128, 255, 256, 341, 342, 511, 512, 513, 700, 1022, 1023, 1024, 1025, 2047,
                                 2048, 4096, 65535]
    lengths = [0, 1, 4095, 4096, 4097, 8192, 8193, 40000, 1 << 20, 1 << 24, 1 << 30]
    size = [[fx.workspace_size(fx.IDX_OP_DISTILL, nq, n, 1) for n in lengths] for nq in rows]
    for i in range(len(rows)):
        for j in range(len(lengths)):
            assert size[i][j] >= 16
            assert j == 0 or size[i][j] >= size[i][j - 1], (rows[i], lengths[j])
            assert i == 0 or size[i][j] >= size[i - 1][j], (rows[i], lengths[j])
    assert size[-1][-1] <= 1 << 15


@pytest.mark.parametrize("nq,n", [(4, 100000), (1024, 100000), (5, 10)])
def test_less_is_refused(fx, nq, n):
    ws = fx.workspace_size(fx.IDX_OP_DISTILL, nq, n, 1)
    got, msg = call(fx, "idx_distill", FAKE, n, FAKE, nq, n, FAKE, FAKE, 64, 64, 1.0, FAKE, FAKE, FAKE, FAKE, ws - 1, None)
    assert got == fx.IDX_EWORKSPACE and "idx_distill" in msg
