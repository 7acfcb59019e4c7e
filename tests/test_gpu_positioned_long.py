"""Calls long enough that a group of lanes takes many heads of a token, and many tokens: the
loops that short calls never enter a second time, and the sums of the weight gradients, against
64-bit forms (evaluated on the GPU; positions stay below 2^17, so pos * f in 64 bits is good to
2^-36 of a radian)."""
import pytest
import torch

from tests import positioned_ref as ref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-6


@pytest.fixture(scope="module")
def csa():
    import long_context_compressed_gated_b200 as m
    m.lib()
    return m


def angles(pos, f):
    return pos.double().view(-1, 1, 1) * f.to(pos.device)


def packed(T, H, Hk, d, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, (H + 2 * Hk) * d, generator=g, device="cuda").to(dtype)
    w = [1 + 0.3 * torch.randn(d, generator=g, device="cuda") for _ in range(2)]
    return x[:, :H * d].view(T, H, d), x[:, H * d:(H + Hk) * d].view(T, Hk, d), x[:, (H + Hk) * d:].view(T, Hk, d), *w


# heads a group takes (148 SMs): 16 + 16 + 5 and 3; 8 + 8 + 1 and 8 + 2; 8 .. 5 left; 4 .. 1 left; ...
FORWARD = [(7300, 37, 3, 128, BF, BF, 0), (7300, 17, 10, 128, BF, F32, 1), (1000, 37, 1, 128, BF, BF, 1),
           (400, 37, 5, 128, F32, F32, 0), (7300, 21, 9, 64, F32, BF, 1), (14000, 16, 7, 64, BF, BF, 0),
           (7111, 6, 11, 128, F32, F32, 1)]


@pytest.mark.parametrize("T,H,Hk,d,dtype,out,style", FORWARD)
@pytest.mark.parametrize("normed", [True, False])
def test_forward_of_long_calls(csa, T, H, Hk, d, dtype, out, style, normed):
    q, k, _, wq, wk = packed(T, H, Hk, d, dtype, T + H)
    f = csa.rope_inv_freq(48)
    w = dict(wq=wq, wk=wk) if normed else {}
    y = csa.csa_qk_norm_rope(q, k, f, eps=EPS, t0=5, rot_start=d - 48, rot_style=style, out_dtype=out, **w)
    ang = angles(torch.arange(5, 5 + T, device="cuda"), f)
    for x, got, wt in ((q, y[0], wq), (k, y[1], wk)):
        wt = wt if normed else None
        err = (got.double() - ref.norm_rope(x, wt, EPS, ang, d - 48, style)).abs()
        assert (err <= ref.norm_rope_bound(x, wt, EPS, ang, d - 48, style, out)).all(), err.max()


@pytest.mark.parametrize("T,H,Hk,d,dtype,out,style", FORWARD)
def test_in_place_and_alone_give_the_same_bits(csa, T, H, Hk, d, dtype, out, style):
    q, k, _, wq, wk = packed(T, H, Hk, d, dtype, T + H)
    f, kw = csa.rope_inv_freq(48), dict(rot_start=d - 48, rot_style=style)
    both = csa.csa_qk_norm_rope(q, k, f, wq=wq, wk=wk, **kw)
    assert torch.equal(csa.csa_qk_norm_rope(q, None, f, wq=wq, **kw)[0], both[0])
    assert torch.equal(csa.csa_qk_norm_rope(None, k, f, wk=wk, **kw)[1], both[1])
    a, b = q.contiguous(), k.contiguous()
    csa.csa_qk_norm_rope(a, b, f, wq=wq, wk=wk, yq=a, yk=b, **kw)
    assert torch.equal(a, both[0]) and torch.equal(b, both[1])


@pytest.mark.parametrize("T,Hk,d,page,rot,style", [(7300, 13, 128, 32, 128, 0), (7300, 8, 64, 16, 48, 1), (7300, 3, 128, 64, 64, 1),
                                                   (900, 21, 128, 16, 64, 0), (400, 29, 64, 256, 64, 1), (9000, 1, 128, 64, 64, 1)])
@pytest.mark.parametrize("normed", [True, False])
def test_append_of_long_calls(csa, T, Hk, d, page, rot, style, normed):
    B = 3
    g = torch.Generator(device="cuda").manual_seed(T + Hk)
    _, k, v, _, wk = packed(T, 2, Hk, d, BF, T + Hk)
    per = -(-T // B)
    max_pages = -(-per // page) + 1
    table = torch.randperm(B * max_pages, generator=g, device="cuda").to(torch.int32).view(B, max_pages)
    order = torch.randperm(T, generator=g, device="cuda")
    seq, slot = (order % B).to(torch.int32), order // B
    skipped = torch.rand(T, generator=g, device="cuda") < 0.02
    pos = slot + 1000 * seq + 17
    f = csa.rope_inv_freq(rot)
    Kp, Vp = (torch.full((B * max_pages, Hk, page, d), 7.0, dtype=BF, device="cuda") for _ in range(2))
    ws = csa.csa_paged_append(k, v, Kp, Vp, table, seq, pos, f, slot=torch.where(skipped, -1, slot),
                              wk=wk if normed else None, eps=EPS, rot_start=d - rot, rot_style=style)
    assert csa.csa_check_status(ws) == 0
    pg, row = table[seq.long(), slot // page].long(), slot % page
    wt, ang, live = wk if normed else None, angles(pos, f), ~skipped
    err = (Kp[pg, :, row].double() - ref.norm_rope(k, wt, EPS, ang, d - rot, style)).abs()
    assert (err <= ref.norm_rope_bound(k, wt, EPS, ang, d - rot, style, BF))[live].all()
    assert torch.equal(Vp[pg, :, row][live], v[live])
    Kp[pg[live], :, row[live]] = 7.0
    Vp[pg[live], :, row[live]] = 7.0
    assert (Kp == 7).all() and (Vp == 7).all()   # the skipped rows and all others as they were


@pytest.mark.parametrize("T,H,Hk,d,dtype,out,style", [
    (20011, 9, 2, 64, F32, F32, 0), (20011, 17, 1, 128, BF, BF, 1), (20011, 3, 3, 64, BF, F32, 1), (9001, 37, 5, 128, F32, BF, 0),
    (60000, 1, 1, 64, BF, BF, 0)])
def test_backward_of_long_calls(csa, T, H, Hk, d, dtype, out, style):
    """dx: as for short calls (g 8u, r 9u, sums 13u, products 6u: under 64u of its terms).
    dw: a thread adds its rows one by one, then a block its groups, then 32 warps the blocks' rows,
    then those.  With at least 4 blocks an SM shared by the sides in proportion to their work (to
    whole blocks: at most twice a side's even share), that is a chain of
      c = 2 T (H + Hk) / (4 SMs groups) + 16 + groups + 5 SMs / 32 + 32
    additions, so |error| <= (c + 20) u sum |terms|, 20u for a term itself."""
    q, k, _, wq, wk = packed(T, H, Hk, d, dtype, T + H)
    g = torch.Generator(device="cuda").manual_seed(T)
    dy = [torch.randn(T, n, d, generator=g, device="cuda").to(out) for n in (H, Hk)]
    f = csa.rope_inv_freq(48)
    got = csa.csa_qk_norm_rope_backward(q, k, *dy, f, wq=wq, wk=wk, eps=EPS, t0=5, rot_start=d - 48, rot_style=style)
    ang = angles(torch.arange(5, 5 + T, device="cuda"), f)
    sms, groups = torch.cuda.get_device_properties(0).multi_processor_count, 128 // (d // 8)
    chain = 2 * T * (H + Hk) / (4 * sms * groups) + 16 + groups + 5 * sms / 32 + 32
    for i, (x, wt) in enumerate(((q, wq), (k, wk))):
        x, wt = x.double(), wt.double()
        G = ref.rotate(dy[i].double(), -ang, d - 48, style)
        size = ref.norm_rope_bound(dy[i].double(), None, EPS, ang, d - 48, style, F32) / (20.2 * ref.U)  # |dy| of the pair
        r = (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
        xh = x * r
        dx = r * (G * wt - xh * (G * wt * xh).mean(-1, keepdim=True))
        M = r * (size * wt.abs() + xh.abs() * (size * wt.abs() * xh.abs()).mean(-1, keepdim=True))
        err = (got[i].double() - dx).abs()
        assert (err <= ref.half(dtype) * dx.abs() + 64 * ref.U * M + 1e-30).all(), err.max()
        dw, terms = (G * xh).sum((0, 1)), (size * xh.abs()).sum((0, 1))
        bound = (chain + 20) * ref.U * terms
        assert ((got[2 + i].double() - dw).abs() <= bound).all()
        # what the bound tells apart: no sum, half of the tokens, one token twice
        assert (dw.abs() > bound).any() and ((G * xh)[:T // 2].sum((0, 1)).abs() > bound).any()
        assert ((G * xh)[-1].sum(0).abs() > bound).any()
