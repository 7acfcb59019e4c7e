"""Workspace sizes of the norm + rotation's backward pass and of the tree attention, on the
host: they cover what a call of the same shape writes, and answer for any shape."""
import pytest


@pytest.fixture(scope="module")
def lib():
    import long_context_compressed_gated_b200 as csa
    from long_context_compressed_gated_b200 import build
    build.build()
    return csa.lib()


HEADER, RECORDS = 256, 32   # bytes: the status word's block; what every thread block of the attention records


@pytest.mark.parametrize("B,R,H,Hk,d", [(1, 1, 1, 1, 64), (64, 64, 64, 8, 64), (3, 10, 8, 2, 128), (65536, 1, 1024, 1, 64)])
def test_tree_attention_without_pages(lib, B, R, H, Hk, d):
    """Tables without an entry: the call still launches, and a block writes its record."""
    assert lib.csa_tree_attn_workspace_bytes(B, R, H, Hk, d, 16, 0) >= HEADER + RECORDS


def test_tree_attention_sizes_grow_with_the_tables(lib):
    need = [lib.csa_tree_attn_workspace_bytes(64, 64, 64, 8, 64, 16, m) for m in (0, 1, 2, 100, 10000)]
    assert need == sorted(need)


@pytest.mark.parametrize("d", [-(2 ** 31), -64, -1, 0, 1, 4, 7, 8, 32, 96, 1024, 1032, 2048, 2 ** 31 - 1])
def test_head_dims_that_are_refused_have_a_size(lib, d):
    """The binding asks for the size before the call refuses the head dim."""
    assert lib.csa_qk_norm_rope_backward_workspace_bytes(10, 4, 1, d) == HEADER
    assert lib.csa_tree_attn_workspace_bytes(3, 10, 8, 2, d, 16, 4) == HEADER


@pytest.mark.parametrize("T,H,Hk", [(10, 0, 0), (10, -1, -5), (-1, 4, 1), (0, 4, 1), (2 ** 40, 4096, 4096)])
def test_norm_rope_backward_sizes_of_any_shape(lib, T, H, Hk):
    assert HEADER <= lib.csa_qk_norm_rope_backward_workspace_bytes(T, H, Hk, 64) < 1 << 20
