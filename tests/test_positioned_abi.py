"""Refusals of the norm + rotation, the paged append and the tree attention on the
host, without a GPU: nothing is enqueued, the pointers are never followed."""
import ctypes

import pytest
import torch

P = ctypes.c_void_p
A = [P(0x1000000 * (i + 1)) for i in range(16)]   # 16-byte aligned, far apart
ODD = P(0x1008)
INV, MIS, SHAPE, WS = -1, -2, -3, -5


@pytest.fixture(scope="module")
def lib():
    import long_context_compressed_gated_b200 as csa
    from long_context_compressed_gated_b200 import build
    build.build()
    return csa.lib()


def freq(n=32, bad=None):
    f = [1.0 / (i + 1) for i in range(n)]
    if bad is not None:
        f[n - 1] = bad
    return (ctypes.c_double * n)(*f)


FWD = dict(q=A[0], qs=4 * 64, k=A[1], ks=64, wq=A[2], wk=A[3], eps=1e-6, pos=A[4], t0=0, f=freq(), start=0, rot=64,
           style=0, T=10, H=4, Hk=1, d=64, xt=0, yq=A[5], yk=A[6], yt=0, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(T=-1), INV), (dict(H=-1), INV), (dict(Hk=5000), INV), (dict(xt=2), INV), (dict(yt=-1), INV),
    (dict(d=96), SHAPE), (dict(qs=4 * 64 - 8), INV), (dict(qs=4 * 64 + 4), INV), (dict(ks=63), INV),
    (dict(style=2), INV), (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV), (dict(rot=8), SHAPE),
    (dict(rot=24), SHAPE), (dict(rot=-16), SHAPE), (dict(rot=80), SHAPE), (dict(start=8), SHAPE),
    (dict(start=4, rot=16), SHAPE), (dict(start=-8, rot=16), SHAPE), (dict(f=None), INV),
    (dict(f=freq(bad=float("inf"))), INV), (dict(q=None), INV), (dict(k=ODD), MIS), (dict(wq=ODD), MIS),
    (dict(pos=ODD), MIS), (dict(yq=None), INV), (dict(yk=ODD), MIS),
    (dict(yq=P(A[0].value + 512)), INV),            # overlaps q without being q
    (dict(yq=A[0], yt=1), INV),                     # in place needs one type
    (dict(q=A[0], qs=8 * 64, yq=A[0]), INV),        # and a dense input
    (dict(yk=A[0]), INV), (dict(yk=A[5]), INV),     # the other side's input, the other output
    (dict(T=0), 0), (dict(H=0, Hk=0), 0), (dict(T=0, q=None, yq=None), 0)])
def test_norm_rope_refuses(lib, change, code):
    a = dict(FWD, **change)
    assert lib.csa_qk_norm_rope(*a.values()) == code


BWD = dict(q=A[0], qs=4 * 64, k=A[1], ks=64, wq=A[2], wk=A[3], eps=1e-6, pos=A[4], t0=0, f=freq(), start=0, rot=64,
           style=1, dyq=A[5], dyk=A[6], T=10, H=4, Hk=1, d=64, xt=1, yt=0, dq=A[7], dqs=4 * 64, dk=A[8], dks=64,
           dwq=A[9], dwk=A[10], ws=A[11], wsb=1 << 20, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(T=-1), INV), (dict(d=32), SHAPE), (dict(xt=3), INV), (dict(dyq=None), INV), (dict(dk=ODD), MIS),
    (dict(dqs=100), INV), (dict(dqs=4 * 64 + 2), INV), (dict(dwq=None), INV), (dict(wq=None), INV),
    (dict(wk=None, dwk=None, H=0, wq=None), INV),   # dwq without queries
    (dict(dwk=ODD), MIS), (dict(ws=None), WS), (dict(wsb=256), WS), (dict(ws=ODD), MIS),
    (dict(dq=A[0]), INV), (dict(dq=A[5]), INV), (dict(dk=P(A[5].value + 64)), INV), (dict(rot=64, f=None), INV)])
def test_norm_rope_backward_refuses(lib, change, code):
    a = dict(BWD, **change)
    assert lib.csa_qk_norm_rope_backward(*a.values()) == code


def test_norm_rope_backward_workspace(lib):
    need = lib.csa_qk_norm_rope_backward_workspace_bytes
    assert need(0, 64, 1, 128) == 256
    assert need(1, 1, 0, 64) == 256 + 256
    assert need(1 << 30, 64, 1, 128) == need(1 << 20, 64, 1, 128) < 1 << 20   # bounded by the GPU's size


APP = dict(k=A[0], ks=2 * 64, v=A[1], vs=2 * 64, wk=A[2], eps=1e-6, pos=A[3], slot=A[4], seq=A[5], f=freq(), start=0,
           rot=64, style=0, table=A[6], T=10, Hk=2, d=64, B=3, max_pages=4, n_pages=12, page=16, Kp=A[7], Vp=A[8],
           ws=A[9], wsb=256, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(T=-1), INV), (dict(Hk=0), INV), (dict(B=-1), INV), (dict(max_pages=-1), INV), (dict(n_pages=-1), INV),
    (dict(d=80), SHAPE), (dict(page=8), SHAPE), (dict(page=48), SHAPE), (dict(page=512), SHAPE), (dict(page=0), SHAPE),
    (dict(ks=64), INV), (dict(vs=2 * 64 + 4), INV), (dict(k=None), INV), (dict(v=ODD), MIS), (dict(pos=None), INV),
    (dict(seq=None), INV), (dict(slot=ODD), MIS), (dict(wk=ODD), MIS), (dict(table=None), INV), (dict(Kp=None), INV),
    (dict(Vp=ODD), MIS), (dict(ws=None), WS), (dict(wsb=0), WS), (dict(rot=72), SHAPE), (dict(style=7), INV),
    (dict(Vp=A[7]), INV), (dict(k=P(A[7].value + 256)), INV),       # caches apart, tokens outside them
    (dict(T=0), 0)])
def test_paged_append_refuses(lib, change, code):
    a = dict(APP, **change)
    assert lib.csa_paged_append(*a.values()) == code


TREE = dict(q=A[0], Kp=A[1], Vp=A[2], table=A[3], lens=A[4], start=A[5], mask=A[6], pos=A[7], R=10, B=3, H=8, Hk=2,
            d=64, page=16, n_pages=12, max_pages=4, W=-1, scale=0.1, O=A[8], ot=0, lse=A[9], ws=A[10], wsb=1 << 30,
            stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(R=-1), INV), (dict(R=1 << 31), INV), (dict(B=-1), INV), (dict(H=0), INV), (dict(Hk=0), INV),
    (dict(n_pages=-1), INV), (dict(max_pages=-1), INV), (dict(W=-2), INV), (dict(scale=0.0), INV),
    (dict(scale=float("inf")), INV), (dict(scale=float("nan")), INV), (dict(ot=2), INV), (dict(d=256), SHAPE),
    (dict(page=24), SHAPE), (dict(H=2048), SHAPE), (dict(Hk=3), SHAPE), (dict(max_pages=1 << 27), SHAPE), (dict(B=65537), SHAPE),
    (dict(ws=None), WS), (dict(wsb=16), WS), (dict(ws=ODD), MIS), (dict(q=None), INV), (dict(Kp=None), INV),
    (dict(Vp=ODD), MIS), (dict(table=None), INV), (dict(lens=None), INV), (dict(start=ODD), MIS), (dict(mask=None), INV),
    (dict(W=4, pos=None), INV), (dict(O=None), INV), (dict(lse=ODD), MIS), (dict(R=0), 0), (dict(B=0), 0),
    (dict(scale=3e38), INV), (dict(O=A[0]), INV), (dict(O=P(0x1000000 + 10224)), INV),
    (dict(ot=1, q=P(0x9000000 + 20464)), INV)])
def test_tree_attn_refuses(lib, change, code):
    a = dict(TREE, **change)
    assert lib.csa_tree_attn(*a.values()) == code


def test_binding_refuses_host_tensors():
    import long_context_compressed_gated_b200 as csa
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        csa.csa_qk_norm_rope(q, None, csa.rope_inv_freq(64))
    with pytest.raises(ValueError):
        csa.csa_qk_norm_rope(None, None, csa.rope_inv_freq(64))
    with pytest.raises(TypeError):
        csa.csa_paged_append(q, q, q, q, q, q, q, None)
    from long_context_compressed_gated_b200.speculative import tree_verify_step
    with pytest.raises(TypeError):
        tree_verify_step(q[0], 2, 1, q, q, q, q, q, q, q, q, q, None, 1.0)
