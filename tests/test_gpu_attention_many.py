"""More than 64 sequences, whose units are found through LDS, in every type and
head width; more (row, query head)s than are joined by a workgroup each; packed
rows of many sequences that are joined by tiles.
"""
import random

import pytest
import torch

from test_gpu_attention import BF16, E4M3, Batch, decode, mep, prefill  # noqa: F401  (mep: the fixture)

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

TYPES = [BF16, E4M3]


def some_lengths(n, seed, long):
    rnd = random.Random(seed)
    lengths = [rnd.choice([0, 1, rnd.randint(1, 40), rnd.randint(1, 200)]) for _ in range(n)]
    lengths[rnd.randrange(n)] = long
    return rnd, lengths


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("head", [64, 128, 256])
@pytest.mark.parametrize("n,heads,hq", [(65, 2, 6), (200, 1, 3)])
def test_decode(mep, n, heads, hq, head, dtype):  # noqa: F811
    _, lengths = some_lengths(n, n + head, 5000)
    decode(mep, Batch(mep, lengths, heads, head, 32, dtype, seed=n), hq, (n, head, dtype))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("head", [64, 128, 256])
@pytest.mark.parametrize("n,heads,hq", [(60, 4, 72), (130, 2, 32)])
def test_decode_joined_by_waves(mep, n, heads, hq, head, dtype):  # noqa: F811
    """n * hq of 4320 and 4160: the joining launch takes a wave for each, and more than one in turn."""
    assert n * hq > 4096
    _, lengths = some_lengths(n, n + head, 3000)
    lengths[3] = 900
    decode(mep, Batch(mep, lengths, heads, head, 64, dtype, seed=n), hq, (n, hq, head, dtype))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("head", [64, 128, 256])
@pytest.mark.parametrize("n,heads,hq", [(65, 1, 4), (200, 2, 2)])
def test_prefill(mep, n, heads, hq, head, dtype):  # noqa: F811
    """At most 4096 (row, query head)s: joined one by one."""
    rnd, lengths = some_lengths(n, n * head, 3000)
    rows = [min(m, rnd.choice([0, 1, 5, 20])) for m in lengths]
    assert (sum(rows) + 2) * hq <= 4096
    prefill(mep, Batch(mep, lengths, heads, head, 32, dtype, seed=n), rows, hq, (n, head, dtype))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("head", [64, 128, 256])
@pytest.mark.parametrize("n,heads,hq", [(65, 1, 8), (150, 2, 10)])
def test_prefill_joined_by_tiles(mep, n, heads, hq, head, dtype):  # noqa: F811
    rnd, lengths = some_lengths(n, n * head, 3000)
    long = lengths.index(3000)
    rows = [min(m, rnd.choice([0, 1, 5, 20])) for m in lengths]
    rows[long], rows[(long + 1) % n], lengths[(long + 1) % n] = 500, 70, 1500
    assert sum(rows) * hq > 4096
    prefill(mep, Batch(mep, lengths, heads, head, 32, dtype, seed=n), rows, hq, (n, head, dtype))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("head", [64, 128, 256])
def test_decode_rows_by_starts(mep, head, dtype):  # noqa: F811
    rnd, lengths = some_lengths(90, head, 3000)
    starts = [1]
    for _ in lengths:
        starts.append(starts[-1] + rnd.choice([0, 1, 1, 1, 3]))
    decode(mep, Batch(mep, lengths, 2, head, 32, dtype, seed=head), 4, (head, dtype), starts=starts)
