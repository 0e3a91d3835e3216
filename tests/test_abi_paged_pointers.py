"""What the paged operators' C entry points refuse by their pointers alone, before any launch (no GPU): addresses
that a kernel could not load from, and outputs that lie on inputs which other parts of the kernel still read."""
import pytest

import block_sparse_streaming_b200 as bss
from test_abi_paged import INVALID, _bwd, _decode, _plan

CTX, NEW, FREE, TABLE = 1 << 20, 1 << 21, 1 << 22, 1 << 23  # _plan's inputs: 4 requests, 9 free pages, 4 rows of 8


@pytest.fixture(scope="module")
def L():
    bss.build()
    return bss.lib()


def refused(L, call, **over):
    count = L.loza_launch_count()
    return call(L, **over) == INVALID and L.loza_launch_count() == count


@pytest.mark.parametrize("over", [
    dict(lens=CTX), dict(lens=NEW), dict(cu=CTX), dict(cu=NEW), dict(counts=CTX), dict(pos=NEW), dict(slots=CTX),
    dict(lens=CTX + 12), dict(lens=CTX - 12), dict(cu=NEW - 16), dict(counts=NEW - 8), dict(slots=CTX - 32 * 8 + 16),
    dict(lens=FREE), dict(pos=FREE + 32), dict(cu=FREE + 32), dict(slots=FREE - 240),
    dict(lens=TABLE), dict(cu=TABLE + 4 * 4 * 7), dict(pos=TABLE - 16), dict(slots=TABLE + 96), dict(counts=TABLE + 124),
    dict(table=CTX), dict(table=NEW - 4), dict(table=FREE + 32), dict(table=FREE - 4 * 31),
    dict(table=CTX - 4 * 12, stride=10), dict(lens=(1 << 24) + 16), dict(counts=1 << 26), dict(slots=(1 << 26) + 112),
    dict(cu=1 << 28), dict(lens=1 << 28), dict(pos=1 << 27)])
def test_plan_refuses_outputs_on_its_inputs_and_on_each_other(L, over):
    assert refused(L, _plan, **over)


@pytest.mark.parametrize("over", [
    dict(lens=CTX + 16), dict(lens=CTX - 16), dict(cu=NEW - 20), dict(pos=FREE + 48), dict(slots=CTX - 256),
    dict(lens=TABLE + 32, stride=16), dict(ctx=TABLE + 32, stride=16), dict(ctx=NEW), dict(lens=TABLE + 128),
    dict(table=0, cols=0, stride=0, lens=1 << 25), dict(capacity=0, pos=0, slots=0), dict(n_free=0, lens=FREE),
    dict(free=TABLE, n_free=0), dict(capacity=0, pos=CTX, slots=CTX)])
def test_plan_takes_neighbours(L, over):
    """Outputs right beside the inputs, in the gaps between the table's rows, and on memory of no length are not
    refused. (Without a GPU the launch itself fails; on one these addresses are not memory, so nothing is called.)"""
    import torch
    if torch.cuda.is_available():
        pytest.skip("would launch")
    assert _plan(L, **over) == -4


@pytest.mark.parametrize("over", [dict(ctx=CTX + 2), dict(new=NEW + 1), dict(free=FREE + 2), dict(table=TABLE + 2),
                                  dict(cu=(1 << 24) + 2), dict(lens=(1 << 25) + 1), dict(counts=(1 << 28) + 2)])
def test_plan_refuses_misaligned_pointers(L, over):
    assert refused(L, _plan, **over)


@pytest.mark.parametrize("over", [dict(bt=(1 << 21) + 2), dict(lens=(1 << 22) + 1), dict(lse=(1 << 24) + 2)])
def test_decode_refuses_misaligned_pointers(L, over):
    assert refused(L, _decode, **over)


@pytest.mark.parametrize("over", [dict(dkw=1 << 30), dict(dkw=(1 << 30) + 4 * 127), dict(dkw=(1 << 30) - 4 * 127)])
def test_backward_refuses_one_place_for_both_weights_gradients(L, over):
    assert refused(L, _bwd, **over)
