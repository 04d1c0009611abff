"""paged_tree_attention with windows where a sequence has more tokens than keys, and around the lengths from which no row
is kept from a key, against the float64 oracle."""
import pytest

from test_gpu_tree_attention import BF, HF, check, make, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("page", [16, 5])
@pytest.mark.parametrize("window", [1, 15, 16, 17, 20, 31, 33, 39, 40, 41, 55, 56, 57, 1000, 2 ** 30, 2 ** 31 - 1, 2 ** 31, 2 ** 40])
def test_more_tokens_than_keys(window, page, tree):
    """Keys of the first page alone: token i of a chain of 40 has the keys above i - window of 16 (or 15)."""
    n = 16 // page * page
    c = make(4, 2, 64, [n, 3, n, 0], [40, 17, 2, 5], page, BF, seed=window % 1000, tree=tree)
    c["table"] = c["table"][:, :n // page].contiguous()
    check(c, *run(c, window=window), window=window)
    c["max_nodes"] = 40
    check(c, *run(c, window=window, max_len=n + 3), window=window)


@pytest.mark.parametrize("G", [1, 8])
@pytest.mark.parametrize("window", [60, 64, 65, 66, 100, 130, 163, 164, 165])
def test_tokens_past_the_bound_of_the_lengths(window, G):
    """max_len cuts the keys, not the tokens: rows behind it see what the window leaves of the keys before."""
    c = make(2 * G, 2, 128, [164, 90], [100, 70], 16, HF, seed=window, tree=False)
    full = c["lengths"].clone()
    out, lse = run(c, window=window, max_len=64)
    c["lengths"] = full.clamp(max=64)
    check(c, out, lse, window=window)
