"""paged_tree_attention on more than 64 sequences (their tiles are dealt from 64 at a time), and blocks of rows whose
keys lie in more than 16 workgroups' stretches, against the float64 oracle."""
import random

import pytest

from test_gpu_tree_attention import BF, HF, check, make, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tree", [True, False])
@pytest.mark.parametrize("kind", ["same", "e4m3"])
@pytest.mark.parametrize("window", [0, 50])
@pytest.mark.parametrize("B", [63, 64, 65, 128, 129, 130, 300])
def test_many_sequences(B, window, kind, tree):
    """Lengths and numbers of tokens mixed, sequences without tokens or keys among them."""
    r = random.Random(B + window)
    nodes = [r.choice([0, 1, 2, 5, 9, r.randrange(0, 21)]) for _ in range(B)]
    lengths = [r.choice([m, m + r.randrange(0, 40), m + r.randrange(0, 300)]) for m in nodes]
    c = make(4, 2, 64, lengths, nodes, 16, BF if B % 2 else HF, kind, B, tree)
    check(c, *run(c, window=window), window=window)


@pytest.mark.parametrize("first", [0, 1, 63, 64, 100, 199])
def test_one_sequence_with_tokens_among_many(first):
    """All but one of 200 have nothing to do, some of them with keys."""
    nodes, lengths = [0] * 200, [7 * (b % 3) for b in range(200)]
    nodes[first], lengths[first] = 11, 1500
    c = make(8, 2, 64, lengths, nodes, 16, BF, seed=first)
    check(c, *run(c))


@pytest.mark.parametrize("B", [100, 300])
def test_many_long_sequences(B):
    """More tiles than workgroups: stretches of whole blocks and of parts, of sequences past the 64th too."""
    r = random.Random(B)
    nodes = [r.choice([1, 3, 17, 40]) if b % 7 else 0 for b in range(B)]
    lengths = [m + r.randrange(0, 900) for m in nodes]
    c = make(2, 1, 64, lengths, nodes, 32, HF, seed=B)
    check(c, *run(c))


@pytest.mark.parametrize("D", [64, 80, 128, 256])
@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("kind", ["same", "e4m3"])
@pytest.mark.parametrize("m", [3, 9, 24])
def test_many_parts(m, kind, dt, D):
    """12, 36 and 96 rows of two heads over 5000 keys: about 160 steps of 64 keys in 80 stretches (of 128 keys: 86 in 40)."""
    tree = (m + D // 16) % 2 == 0
    c = make(8, 2, D, [5000], [m], 16 if D != 80 else 7, dt, kind, m + D, tree)
    check(c, *run(c))
    check(c, *run(c, window=3900), window=3900)
    # holes over most of the keys: stretches of which no row sees a key
    c["table"][0, 30:c["table"].shape[1] - 20] = -1
    check(c, *run(c))


@pytest.mark.parametrize("m", [2, 20])
def test_many_parts_without_any_key(m):
    """A table of holes: every part is empty, and so is the result."""
    c = make(8, 2, 64, [5000], [m], 16, BF, seed=m)
    c["table"][:] = -1
    out, lse = run(c)
    check(c, out, lse)
    assert (out[:m] == 0).all()


@pytest.mark.parametrize("window", [0, 200])
def test_a_long_chain(window):
    """Blocks of rows of one sequence whose keys end, and with a window begin, elsewhere from block to block."""
    c = make(4, 1, 64, [1500], [600], 16, BF, seed=window, tree=False)
    check(c, *run(c, window=window), window=window)
