"""kvc_i4_tree_commit refuses outputs that lie where it still reads: the queries and the row statistics (CPU)."""
import pytest

from test_tree_args import A, INVALID, UNSUPPORTED, commit, lib  # noqa: F401

Q, LSE = A + (1 << 16), A + (1 << 17)


@pytest.mark.parametrize("out", ["ko", "vo"])
@pytest.mark.parametrize("over", [Q, LSE])
def test_outputs_over_what_is_read(lib, out, over):  # noqa: F811
    assert commit(lib, q=Q, lse=LSE, **{out: over}) == INVALID
    assert commit(lib, q=Q, lse=LSE) not in (INVALID, UNSUPPORTED)
    # without queries neither is read
    assert commit(lib, q=None, lse=LSE, **{out: LSE}) not in (INVALID, UNSUPPORTED)
