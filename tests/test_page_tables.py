"""PageTables.release: pages go back to the ring once each, as many as the request holds on the device.
AttentionBlock takes tables of its own cache's form only."""
from __future__ import annotations

from types import SimpleNamespace as Some

import pytest
import torch

import moe_expert_layer_07_gb300 as moe

I32 = torch.int32


def _tables(lengths, table, ring, free_range, page=16):
    """Tables that hold this, on the CPU (release is torch's own operations)."""
    t = moe.PageTables.__new__(moe.PageTables)
    t.page = page
    t.lengths, t.table = torch.tensor(lengths, dtype=I32), torch.tensor(table, dtype=I32)
    t.free_pages, t.free_range = torch.tensor(ring, dtype=I32), torch.tensor(free_range, dtype=torch.int64)
    t.status = torch.zeros(1, dtype=I32)
    return t


def _free(t):
    a, b = t.free_range.tolist()
    return [int(t.free_pages[i % t.free_pages.shape[0]]) for i in range(a, b)]


@pytest.mark.parametrize("length", [None, 33, 40, 0, 16, 64, 1000])
def test_pages_are_those_that_the_device_holds(length):
    t = _tables([33, 20], [[4, 0, 2, 7], [5, 1, 9, 9]], [3, 6, 8, 0, 0, 0, 0, 0, 0], [0, 3])
    t.release(0, length)
    assert _free(t) == [3, 6, 8, 4, 0, 2] and t.lengths.tolist() == [0, 20]
    assert int(t.status) == (0 if length in (None, 33, 40) else moe.DEV_BAD_INDEX)
    assert t.free_pages[6:].tolist() == [0, 0, 0]
    t.release(1, 20)
    assert _free(t) == [3, 6, 8, 4, 0, 2, 5, 1] and t.lengths.tolist() == [0, 0]


def test_a_second_release_gives_nothing():
    t = _tables([33], [[4, 0, 2, 7]], [0] * 5, [0, 0])
    t.release(0, 33)
    t.release(0)
    assert _free(t) == [4, 0, 2] and int(t.status) == 0
    t.release(0, 33)
    assert _free(t) == [4, 0, 2] and int(t.status) == moe.DEV_BAD_INDEX


def test_around_the_ring_and_with_more_columns_than_pages():
    t = _tables([64], [[2, 0, 3, 1, -1, -1, -1]], [9, 9, 9, 9], [7, 7])
    t.release(0)
    assert _free(t) == [2, 0, 3, 1] and t.free_range.tolist() == [7, 11]
    t = _tables([0], [[]], [], [0, 0])
    t.release(0)
    assert t.free_range.tolist() == [0, 0]


@pytest.mark.parametrize("request_", [-1, 2, 100])
def test_a_request_that_is_none(request_):
    t = _tables([33, 20], [[4, 0, 2, 7], [5, 1, 9, 9]], [3, 6, 8, 0, 0, 0, 0, 0, 0], [0, 3])
    with pytest.raises(IndexError):
        t.release(request_, 20)
    assert t.lengths.tolist() == [33, 20] and t.free_range.tolist() == [0, 3]


@pytest.mark.parametrize("page,requests,columns", [(32, 2, 4), (16, 3, 4), (16, 2, 5)])
def test_a_block_refuses_tables_of_another_form(page, requests, columns):
    """Before anything is computed or written: slots of other pages would be other tokens' places."""
    block = moe.AttentionBlock.__new__(moe.AttentionBlock)
    block.max_rows, block.cache = 8, Some(page=16)
    block.plan = Some(d=Some(requests=2, max_pages=4), of_rows=lambda rows: pytest.fail("went on"))
    block._plans = {}
    tables = _tables([1] * requests, [[0] * columns] * requests, [1], [0, 1], page=page)
    tables.slots = torch.zeros(8, dtype=I32)
    with pytest.raises(ValueError):
        block.forward(None, torch.zeros(1, 4), None, tables)
