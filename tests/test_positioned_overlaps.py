"""Outputs of the positioned operators that share memory with what their kernels still read
are refused on the host, without a GPU; neighbours are not."""
import pytest

from tests.test_positioned_abi import A, APP, BWD, FWD, INV, P, TREE, lib  # noqa: F401


def at(p, offset):
    return P(p.value + offset)


# FWD: T = 10, H = 4, Hk = 1, d = 64, bf16.  yq 5120 bytes, yk 1280; weights 256, positions 80
@pytest.mark.parametrize("change", [
    dict(yq=A[2]), dict(yk=A[3]), dict(yq=A[4]), dict(yk=A[4]), dict(yq=A[3]), dict(yk=A[2]),
    dict(yq=at(A[2], -5104)), dict(yk=at(A[4], 64)), dict(wq=at(A[5], 5104)), dict(pos=at(A[6], 1264))])
def test_norm_rope(lib, change):  # noqa: F811
    assert lib.csa_qk_norm_rope(*dict(FWD, **change).values()) == INV


# BWD: fp32 rows: dq 10240 bytes, dk 2560
@pytest.mark.parametrize("change", [
    dict(dq=A[2]), dict(dk=A[3]), dict(dq=A[4]), dict(dq=A[9]), dict(dk=A[10]), dict(dq=A[10]), dict(dwk=A[9]),
    dict(dwq=at(A[10], 240)), dict(dwk=at(A[8], 2544)), dict(wk=at(A[7], 10224))])
def test_norm_rope_backward(lib, change):  # noqa: F811
    assert lib.csa_qk_norm_rope_backward(*dict(BWD, **change).values()) == INV


# APP: 12 pages of 2 x 16 x 64: 49152 bytes each; T = 10, B x max_pages = 12
@pytest.mark.parametrize("change", [
    dict(pos=A[7]), dict(slot=A[8]), dict(seq=at(A[7], 49136)), dict(wk=at(A[8], 1024)), dict(table=A[8]),
    dict(table=at(A[7], -32))])
def test_paged_append(lib, change):  # noqa: F811
    assert lib.csa_paged_append(*dict(APP, **change).values()) == INV


# TREE: R = 10, H = 8, d = 64: O 10240 bytes in bf16, lse 320; caches 49152 bytes
@pytest.mark.parametrize("change", [
    dict(O=A[1]), dict(O=at(A[2], 49136)), dict(lse=A[1]), dict(lse=A[0]), dict(lse=A[8]), dict(lse=at(A[8], 10224)),
    dict(O=A[3]), dict(O=A[4]), dict(lse=A[5]), dict(lse=A[6]), dict(O=at(A[6], 64)), dict(W=8, lse=A[7]),
    dict(ot=1, lse=at(A[8], 20464)), dict(O=at(A[5], 0))])
def test_tree_attn(lib, change):  # noqa: F811
    assert lib.csa_tree_attn(*dict(TREE, **change).values()) == INV
