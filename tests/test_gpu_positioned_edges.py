"""Edges of the norm + rotation, the paged append and the tree attention: refused head
dims, values that are not finite, groups that take many heads, sums over long calls."""
import math

import pytest
import torch

from tests import positioned_ref as ref
from tests.test_gpu_tree import call, make

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def csa():
    import long_context_compressed_gated_b200 as m
    m.lib()
    return m


@pytest.mark.parametrize("d", [4, 96, 2048])
def test_backward_refuses_head_dims_without_a_workspace(csa, d):
    x = torch.zeros(3, 2, d, device="cuda")
    with pytest.raises(csa.CsaError):
        csa.csa_qk_norm_rope_backward(x, None, x, None, None)


# ---------------------------------------------------------------- values that are not finite


def spoiled(T, heads, d, dtype, seed):
    """Rows with an infinity or a NaN at every channel in turn."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, heads, d, generator=g).to(dtype)
    for t in range(T):
        for h in range(heads):
            x[t, h, (t * heads + h) % d] = (math.inf, -math.inf, math.nan)[(t + h) % 3]
    return x


def same_kind(got, want):
    """NaN, +inf, -inf and finite in the same places."""
    got, want = got.cpu().double(), want.double()
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got.isposinf(), want.isposinf()) and torch.equal(got.isneginf(), want.isneginf())
    return want.isfinite()


ROTATIONS = [(64, 0, 0), (64, 0, 1), (64, 16, 0), (64, 16, 1), (128, 48, 0), (128, 48, 1), (128, 128, 1), (128, 128, 0)]


@pytest.mark.parametrize("d,rot,style", ROTATIONS)
@pytest.mark.parametrize("normed", [False, True])
@pytest.mark.parametrize("dtype,out", [(BF, BF), (F32, F32), (BF, F32)])
def test_norm_rope_keeps_infinities_where_they_are(csa, d, rot, style, normed, dtype, out):
    """An infinity or a NaN reaches the channels that the formula takes it to (its pair, and with
    a norm its row's sum of squares), no other; channels outside the rotation keep n."""
    T, H, start = 24, 6, d - rot
    x = spoiled(T, H, d, dtype, d + rot + style)
    f = csa.rope_inv_freq(rot) if rot else None
    w = torch.linspace(0.5, 1.5, d) if normed else None
    y, _ = csa.csa_qk_norm_rope(x.cuda(), None, f, wq=None if w is None else w.cuda(), eps=1e-6, t0=3, rot_start=start,
                                rot_style=style, out_dtype=out)
    ang = ref.angles(range(3, 3 + T), f if rot else [])
    want = ref.norm_rope(x, w, 1e-6, ang, start, style)
    ok = same_kind(y, want)
    xf = torch.where(x.isfinite(), x.double(), torch.zeros((), dtype=torch.float64))
    bound = ref.norm_rope_bound(xf, w, 1e-6, ang, start, style, out)
    err = (y.cpu().double() - want).abs()
    assert (err[ok] <= bound[ok]).all()
    if not normed:   # the untouched channels are the input's
        a, b = y.cpu()[..., :start], x[..., :start].to(out)
        assert torch.equal(a.nan_to_num(9, 8, 7), b.nan_to_num(9, 8, 7))


@pytest.mark.parametrize("d,rot,style", ROTATIONS)
def test_backward_keeps_infinities_where_they_are(csa, d, rot, style):
    """Without a norm the gradient is the rotation's transpose of dy."""
    T, H, start = 24, 6, d - rot
    dy = spoiled(T, H, d, F32, d + rot + style)
    x = torch.randn(T, H, d)
    f = csa.rope_inv_freq(rot) if rot else None
    dq, *_ = csa.csa_qk_norm_rope_backward(x.cuda(), None, dy.cuda(), None, f, t0=3, rot_start=start, rot_style=style)
    want = ref.rotate(dy.double(), -ref.angles(range(3, 3 + T), f if rot else []), start, style)
    same_kind(dq, want)
    a, b = dq.cpu()[..., :start], dy[..., :start]
    assert torch.equal(a.nan_to_num(9, 8, 7), b.nan_to_num(9, 8, 7))


@pytest.mark.parametrize("d,rot,style", ROTATIONS)
def test_append_keeps_infinities_where_they_are(csa, d, rot, style):
    T, Hk, start, page = 32, 6, d - rot, 16
    x = spoiled(T, Hk, d, BF, d + rot + style)
    f = csa.rope_inv_freq(rot) if rot else None
    Kp, Vp = (torch.zeros(2, Hk, page, d, dtype=BF, device="cuda") for _ in range(2))
    table = torch.tensor([[1, 0]], dtype=torch.int32)
    pos = torch.arange(3, 3 + T)
    csa.csa_paged_append(x.cuda(), x.cuda(), Kp, Vp, table.cuda(), torch.zeros(T, dtype=torch.int32, device="cuda"),
                         pos.cuda(), f, slot=(pos - 3).cuda(), rot_start=start, rot_style=style)
    k = ref.paged_rows(Kp.cpu(), table, 0, T)
    want = ref.rotate(x.double(), ref.angles(pos, f if rot else []), start, style)
    same_kind(k, want)
    a, b = k[..., :start], x[..., :start]
    assert torch.equal(a.nan_to_num(9, 8, 7), b.nan_to_num(9, 8, 7))
    assert torch.equal(ref.paged_rows(Vp.cpu(), table, 0, T).view(torch.int16), x.view(torch.int16))


@pytest.mark.parametrize("lens,nodes,H,Hk,d,page", [
    ([700], [1], 64, 1, 128, 64),                  # shared by several thread blocks, one row tile
    ([20000, 3], [2, 2], 4, 1, 64, 64),            # many parts of few rows
    ([3000, 800], [12, 30], 64, 1, 128, 64),       # two row tiles
    ([40, 0, 90], [3, 2, 5], 8, 2, 64, 16)])       # within one block
@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_queries_that_are_not_finite_show(csa, lens, nodes, H, Hk, d, page, out, value):
    """NaN where such a query sees something, the empty result where it does not, and not a bit
    changed anywhere else."""
    x = make(lens, nodes, H, Hk, d, page, seed=50)
    O, lse, _ = call(csa, x, out=out)
    x["q"][0, H // 2, 5] = value
    mid = (x["q"].shape[0] - 1) // 2
    x["q"][mid, H - 1] = value
    last = x["q"].shape[0] - 1
    x["q"][last, 0, d - 1] = value
    P, lp, ws = call(csa, x, out=out)
    assert csa.csa_check_status(ws) == 0
    bad = torch.zeros(lse.shape, dtype=torch.bool, device="cuda")
    bad[0, H // 2] = bad[mid, H - 1] = bad[last, 0] = True
    bad &= lse != -math.inf
    assert P[bad].isnan().all() and lp[bad].isnan().all()
    assert torch.equal(P[~bad], O[~bad]) and torch.equal(lp[~bad], lse[~bad])


def test_verification_step_wants_slots(csa):
    """Two children of one node share a position: without slots they would share a cache row."""
    from long_context_compressed_gated_b200.speculative import tree_verify_step
    x = make([20], [3], 4, 2, 64, 16, seed=51)
    c = {k: v.cuda() for k, v in x.items()}
    c["pos"].copy_(torch.tensor([20, 21, 21]))
    keep = c["Kp"].clone(), c["Vp"].clone()
    good = dict(qkv=torch.randn(3, 8 * 64, device="cuda").to(BF), H=4, Hk=2, Kpages=c["Kp"], Vpages=c["Vp"],
                block_table=c["table"], seq_lens=c["lens"], q_start=c["start"], mask=c["mask"],
                seq=torch.zeros(3, dtype=torch.int32, device="cuda"), pos=c["pos"], inv_freq=csa.rope_inv_freq(64), scale=0.1)
    with pytest.raises(ValueError):
        tree_verify_step(slot=None, **good)
    assert torch.equal(c["Kp"].view(torch.int16), keep[0].view(torch.int16))
    tree_verify_step(slot=torch.tensor([20, 21, 22]).cuda(), **good)
    rows = ref.paged_rows(c["Vp"].cpu(), x["table"], 0, 23)[20:]
    assert torch.equal(rows, good["qkv"].cpu().view(3, 8, 64)[:, 6:])


def test_sides_without_heads(csa):
    """A side of no heads: no rows, and a weight whose gradient is the empty sum."""
    f, w = csa.rope_inv_freq(64), torch.ones(64, device="cuda")
    x, dy = (torch.randn(5, 2, 64, device="cuda") for _ in range(2))
    none = x[:, :0].contiguous()
    y = csa.csa_qk_norm_rope(x, none, f, wq=w, wk=w)
    assert y[1].shape == (5, 0, 64)
    want = csa.csa_qk_norm_rope_backward(x, None, dy, None, f, wq=w)
    for given in (None, torch.full((64,), 3.0, device="cuda")):
        got = csa.csa_qk_norm_rope_backward(x, none, dy, none, f, wq=w, wk=w, dwk=given)
        assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2]) and got[1].shape == (5, 0, 64)
        assert (got[3] == 0).all() and (given is None or got[3] is given)
