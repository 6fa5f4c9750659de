"""An append without tokens (no GPU): what an empty tensor's null pointer must not refuse."""
import pytest

from tests.test_kv8_host import FAKE, append, cache, lib  # noqa: F401


@pytest.mark.parametrize("over", [
    dict(), dict(cu=FAKE), dict(table=FAKE), dict(table=FAKE, rows=1),  # positions: an empty tensor
    dict(table=FAKE, rows=1, cu=FAKE), dict(table=FAKE, rows=1, pos=FAKE)])
def test_no_tokens_need_no_positions(lib, over):  # noqa: F811
    assert append(lib, cache(), T=0, k=None, v=None, **over) == 0
    # with tokens, the cache's rows have to be in the table
    if over.get("rows") and not over.get("pos"):
        assert append(lib, cache(), T=1, **over) == 1
