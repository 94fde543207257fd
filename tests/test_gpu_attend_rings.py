"""GPU: spec_attend in bf16 where few tiles pass through a short ring: items of 64 rows with more than 64 columns
(two slots), texts of a few tiles whose last one a mask cuts, tiles that arrive late (pages copied slot by slot).
The result is float64's, and the same bits call after call."""
import pytest
import torch

from attend_ref import Batch, check

pytestmark = pytest.mark.gpu

BF = torch.bfloat16

# rows, kv, Hq, Hkv, D, page, window, sinks, shared, order
CASES = {
    "two tiles, prefix": ([3, 1, 5, 2, 0, 8, 8, 2, 5, 5, 8, 8, 5, 0, 2, 3, 0, 1, 1, 3, 0, 1, 8, 8],
                          [533, 1, 71, 2, 211, 53, 8, 3, 65, 5, 6, 40, 3, 1, 671, 2, 43, 0, 0, 2, 0, 1, 8, 49],
                          24, 3, 112, 3, 0, 0, 33, "slot"),
    "two tiles, window": ([5, 3, 1, 2, 8, 0, 2, 1, 2, 2, 1, 1, 5, 0, 1, 8, 1, 3, 8, 1, 5, 0, 0],
                          [3, 1, 1, 47, 29, 0, 503, 300, 2, 2, 558, 5, 183, 103, 0, 52, 1, 31, 600, 321, 6, 0, 21],
                          48, 3, 112, 3, 530, 27, 13, "slot"),
    "prompts and rounds": ([5, 0, 3, 8, 138, 3, 2, 0, 1, 0, 2, 112, 2, 0, 2, 148, 0, 0, 0, 147, 5, 3, 5, 3, 0, 8, 39, 5, 3,
                            1, 129, 2],
                           [3, 0, 4, 8, 139, 3, 460, 0, 11, 657, 11, 110, 390, 37, 2, 167, 0, 184, 0, 148, 5, 2, 32, 30,
                            0, 8, 287, 5, 16, 4, 128, 2],
                           3, 3, 128, 1, 418, 4, 0, "head"),
    "three tiles cut in two": ([2, 8, 8, 1, 8, 0, 0, 0, 3, 1, 1, 2, 1, 3, 5, 3, 3, 1, 0, 5, 8, 1, 8, 1, 3, 1, 5, 5, 1, 8, 1,
                                0, 2, 1, 1, 2],
                               [1, 168, 9, 51, 8, 0, 0, 23, 2, 30, 1, 3, 45, 181, 5, 3, 415, 0, 0, 6, 7, 169, 8, 2, 3, 1,
                                5, 5, 0, 6, 36, 18, 1, 31, 0, 1],
                               32, 2, 128, 3, 0, 0, 151, "head"),
    "pages of 16": ([9, 10, 8, 9, 10, 12], [390, 140, 523, 266, 129, 1030], 8, 2, 128, 16, 0, 0, 0, "slot"),
    "pages of 16, window": ([9, 10, 8, 9, 10, 12], [390, 140, 523, 266, 129, 1030], 8, 2, 80, 16, 200, 4, 0, "head"),
    "pages of one": ([9, 10, 8, 9, 10, 12], [390, 140, 523, 266, 129, 1030], 8, 2, 96, 1, 0, 0, 0, "slot"),
}


def repeat(b, kernel, times):
    a = b.place().attention()
    assert a.plan() == kernel
    first = None
    for k in range(times):
        a.workspace.fill_(0xFF * (k % 2))
        a.out.out.fill_(7.0)
        a.run()
        torch.cuda.synchronize()
        got = a.out.out.view(torch.int16).clone(), a.out.lse.clone()
        if first is None:
            first = got
            check(b, a.out)
        assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1]), k


@pytest.mark.parametrize("name", list(CASES))
def test_rings_of_two(name):
    rows, kv, Hq, Hkv, D, page, W, S, L, order = CASES[name]
    repeat(Batch(rows, kv, Hq, Hkv, D, BF, page, W, S, L, seed=len(name), order=order), "spec_attend_round_kernel", 40)


@pytest.mark.parametrize("D,page,window", [(128, 3, 0), (64, 1, 0), (128, 16, 200)])
def test_items_of_one_accumulator_before_items_of_two(D, page, window):
    """Items of up to 128 rows, whose tiles the second accumulator's threads do not use, each followed by an item
    of more rows over a text of less than a tile."""
    rows = [30, 60] * 60
    kv = [x for i in range(60) for x in (300 + 7 * (i % 40), 60 + i % 50)]
    repeat(Batch(rows, kv, 16, 4, D, BF, page, window, 2 if window else 0, 0, seed=D), "spec_attend_pair_kernel", 20)
