"""Paged operators at the bounds of what they may touch: tables without pages, numbers on
the device that wrap 32 bits, memory around the workspace and the outputs."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def csa():
    import long_context_compressed_gated_b200 as m
    m.lib()
    return m


def guarded(nbytes, fill=0xA5):
    """(a workspace of nbytes with a clear status word, the allocation around it, its place)"""
    whole = torch.full((nbytes + 2 * 65536,), fill, dtype=torch.uint8, device="cuda")
    ws = whole[65536:65536 + nbytes]
    ws.zero_()
    return ws, whole


def untouched(whole, nbytes, fill=0xA5):
    return bool((whole[:65536] == fill).all()) and bool((whole[65536 + nbytes:] == fill).all())


@pytest.mark.parametrize("nodes", [0, 1])
def test_tree_attention_with_tables_without_pages(csa, nodes):
    """[B, 0] tables: nothing happens without a node, a node is reported; either way nothing
    outside the workspace is written."""
    B, H, Hk, d, page = 64, 64, 8, 64, 16
    need = csa.lib().csa_tree_attn_workspace_bytes(B, B, H, Hk, d, page, 0)
    ws, whole = guarded(need)
    q = torch.zeros(B, H, d, dtype=BF, device="cuda")
    pages = torch.zeros(2, Hk, page, d, dtype=BF, device="cuda")
    table = torch.zeros(B, 0, dtype=torch.int32, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    start = torch.arange(B + 1, dtype=torch.int32, device="cuda") * nodes
    mask = torch.ones(B, dtype=torch.int64, device="cuda")
    O = torch.full((B, H, d), 7.0, dtype=BF, device="cuda")
    csa.csa_tree_attn(q, pages, pages.clone(), table, lens, start, mask, 1 / math.sqrt(d), O=O, workspace=ws)
    assert csa.csa_check_status(ws) == (-8 if nodes else 0)
    assert untouched(whole, need)
    if not nodes:
        assert (O == 7).all()


@pytest.mark.parametrize("r0,r1", [(2 ** 31 - 1, -2 ** 31), (2 ** 31 - 3, -2 ** 31 + 20), (5, -2 ** 31), (-2 ** 31, 2 ** 31 - 1),
                                   (2 ** 31 - 1, 2 ** 31 - 1), (-1, 0), (11, 11)])
def test_row_numbers_that_wrap_are_reported(csa, r0, r1):
    """q_start whose difference in 32 bits looks like a few nodes: reported, and the rows of the
    call, none of which it names, are left."""
    B, R, H, d, page = 1, 10, 8, 64, 16
    q = torch.randn(R, H, d, device="cuda").to(BF)
    pages = torch.randn(6, 2, page, d, device="cuda").to(BF)
    table = torch.arange(6, dtype=torch.int32, device="cuda").view(B, 6)
    lens = torch.tensor([40], dtype=torch.int32, device="cuda")
    mask, pos = (torch.ones(R, dtype=torch.int64, device="cuda") for _ in range(2))
    start = torch.tensor([r0, r1], dtype=torch.int32, device="cuda")
    O = torch.full((R, H, d), 7.0, dtype=BF, device="cuda")
    for W in (-1, 4):
        _, _, ws = csa.csa_tree_attn(q, pages, pages.clone(), table, lens, start, mask, 0.1, W=W, pos=pos, O=O)
        assert csa.csa_check_status(ws) == -8 and (O == 7).all()
