"""Paged operators at the bounds of what they may touch: tables without pages, numbers on
the device that wrap 32 bits, memory around the workspace and the outputs."""
import math

import pytest
import torch

from tests.test_gpu_tree import call, check, make

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


@pytest.mark.parametrize("L,n,real,page", [(62, 8, 2, 64), (62, 8, 0, 64), (0, 9, 1, 16), (15, 64, 17, 16), (127, 33, 1, 128),
                                           (250, 12, 3, 16), (255, 40, 1, 256)])
@pytest.mark.parametrize("garbage", [-1, 2 ** 31 - 1])
def test_pages_behind_the_last_seen_draft_are_not_used(csa, L, n, real, page, garbage):
    """Padding nodes (mask 0) whose rows would lie in pages that were never taken."""
    x = make([L, 30], [n, 2], 8, 2, 64, page, seed=L)
    x["mask"][real:n] = 0
    x["table"][0, -(-(L + real) // page):] = garbage
    O, lse, ws = call(csa, x)
    assert csa.csa_check_status(ws) == 0 and check(x, O, lse).all()


@pytest.mark.parametrize("W", [-1, 0, 40])
@pytest.mark.parametrize("d,page,seed", [(64, 16, 1), (128, 16, 2), (128, 64, 3), (64, 128, 4), (128, 256, 5)])
def test_pages_that_no_node_sees_are_not_used(csa, W, d, page, seed):
    """Any masks: a page number is used only if some node sees a row of it."""
    g = torch.Generator().manual_seed(seed)
    lens, nodes = [700, 0, 129, 5, 260], [64, 40, 17, 33, 1]
    x = make(lens, nodes, 8, 2, d, page, seed=seed)
    r = 0
    for b, (L, n) in enumerate(zip(lens, nodes)):
        keep = torch.randint(0, n, (2,), generator=g).tolist()   # two drafts at most are seen
        lo = L if W >= 0 else 0
        seen = set()
        for i in range(n):
            m = sum(1 << j for j in keep) if i % 3 == 0 else 0
            x["mask"][r + i] = m - (1 << 64) if m >> 63 else m
            seen |= {L + j for j in keep if m >> j & 1}
            if W >= 0:
                lo = min(lo, max(0, int(x["pos"][r + i]) - W + 1))
        seen |= set(range(lo, L))
        for p in range(-(-(L + n) // page)):
            if not any(s in seen for s in range(p * page, (p + 1) * page)):
                x["table"][b, p] = -1 - p
        r += n
    O, lse, ws = call(csa, x, W=W)
    assert csa.csa_check_status(ws) == 0 and check(x, O, lse, W=W).all()
