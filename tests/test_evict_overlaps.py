"""What pa_evict writes must not lie in what it reads: refused before anything
is enqueued (no GPU)."""

import pytest

from test_cache4_host import APART, FAKE, INVALID, WEIGHTS, evict_call, lib, weights  # noqa: F401 (lib: fixture)

# weights: 3 rows of 4 heads of 160 tokens from WEIGHTS on
SIZE = 3 * 4 * 160 * 4


@pytest.mark.parametrize("change", [
    dict(kept=WEIGHTS), dict(kept=WEIGHTS + SIZE - 4), dict(kept=WEIGHTS - 4), dict(new_lens=WEIGHTS + 64),
    dict(new_lens=WEIGHTS + SIZE - 4), dict(new_w=FAKE + (1 << 20)), dict(new_w=FAKE + (1 << 20) - SIZE + 4),
    dict(new_w=FAKE + 2048 - 64), dict(new_w=FAKE + 4096), dict(dst=FAKE + (1 << 24), new_w=FAKE + (1 << 24) + 64),
], ids=str)
def test_outputs_in_inputs_are_refused(lib, change):  # noqa: F811
    # lengths of their own: FAKE lies below the other buffers
    a = dict(APART, lens=FAKE + 512)
    a.update(change)
    assert evict_call(lib, dict(a, w=weights(weights=WEIGHTS))) == INVALID
