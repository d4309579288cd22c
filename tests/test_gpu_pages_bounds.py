"""mk_assign_pages at the ends of its 32-bit range: as many tokens, blocks taken and blocks given back as an int32 counts."""
import ctypes
import gc

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import persistent_megakernel_decode_sm_gb300 as mk  # noqa: E402

TOP = 2 ** 31 - 1


@pytest.fixture(autouse=True)
def nothing_left_behind():
    """These take up to 40 GB: back to the device before the next test."""
    yield
    gc.collect()
    torch.cuda.empty_cache()


def words(*values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def assign(ring, ends, table, lens, new, block, slots, status):
    a = mk.mk_pages_args(batch=len(lens), block_size=block, max_blocks=table.shape[1], n_blocks=len(ring), max_tokens=len(slots),
                         ring=ring.data_ptr(), ends=ends.data_ptr(), ends_out=ends.data_ptr(), table=table.data_ptr(), lens=lens.data_ptr(),
                         new_lens=new.data_ptr(), slots=slots.data_ptr(), status=status.data_ptr())
    assert mk.lib.mk_assign_pages(ctypes.addressof(a), torch.cuda.current_stream().cuda_stream) == mk.MK_OK


def filled(first, last, slots):
    """slots hold first .. last - 1, and -1 behind."""
    n = last - first
    assert torch.equal(slots[:n], torch.arange(first, last, dtype=torch.int32, device="cuda")) and bool((slots[n:] == -1).all())


@pytest.mark.parametrize("block,requests,behind", [(TOP, [TOP], 0), (TOP, [TOP - 1], 1), (TOP, [TOP - 126], 126), (2 ** 30 - 1, [2 ** 30 - 1, 2 ** 30 - 1], 1),
                                                   (2 ** 30 - 1, [2 ** 30 - 1, 2 ** 30 - 3], 0)])
def test_the_last_tokens(block, requests, behind):
    batch, status = len(requests), words(0)
    slots = torch.full((sum(requests) + behind,), -9, dtype=torch.int32, device="cuda")
    ends, table = words(0, batch, 0), torch.full((batch, 1), -7, dtype=torch.int32, device="cuda")
    assign(torch.arange(batch, dtype=torch.int32, device="cuda"), ends, table, torch.zeros_like(table[:, 0]), words(*requests), block, slots, status)
    assert status.item() == 0 and ends.tolist() == [0, 0, 0] and table[:, 0].tolist() == list(range(batch))
    filled(0, sum(requests), slots)   # (request b's block is b, so its slots follow on those before)


def test_as_many_blocks_as_there_can_be():
    front, status = 5, words(0)
    ring, table = torch.arange(TOP, dtype=torch.int32, device="cuda"), torch.full((1, TOP), -7, dtype=torch.int32, device="cuda")
    ends, slots = words(front, TOP, 0), torch.full((TOP,), -9, dtype=torch.int32, device="cuda")
    assign(ring, ends, table, words(0), words(TOP), 1, slots, status)
    assert status.item() == 0 and ends.tolist() == [front, 0, 0]
    for got in (slots, table[0]):
        filled(front, TOP, got[:TOP - front])
        assert got[TOP - front:].tolist() == list(range(front))
    ring.fill_(-7)
    assign(ring, ends, table, words(TOP), words(0), 1, slots[:1], status)
    assert status.item() == 0 and ends.tolist() == [front, TOP, 0] and slots[0].item() == -1
    filled(0, TOP, ring)
