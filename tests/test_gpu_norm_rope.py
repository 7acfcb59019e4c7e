"""csa_qk_norm_rope and its backward against the 64-bit form: types, head layouts,
packed and dense rows, partial and shifted rotations, far positions, in place,
no norm, captured calls."""
import math

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


def make(T, H, Hk, d, dtype, packed, seed=0, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(T, (H + 2 * Hk) * d, generator=g) * spread).to(dtype)
    q, k = x[:, :H * d].view(T, H, d), x[:, H * d:(H + Hk) * d].view(T, Hk, d)
    w = [1 + 0.3 * torch.randn(d, generator=g) for _ in range(2)]
    dev = x.cuda()
    qd, kd = dev[:, :H * d].view(T, H, d), dev[:, H * d:(H + Hk) * d].view(T, Hk, d)
    if not packed:
        qd, kd = qd.contiguous(), kd.contiguous()
    return q, k, w[0], w[1], qd, kd


CASES = [
    # T, H, Hk, d, rot, start, style, dtype, out, packed, t0
    (1, 1, 1, 64, 64, 0, 0, BF, BF, False, 0),
    (1, 64, 1, 128, 64, 64, 1, BF, BF, True, 1048575),
    (5, 64, 1, 128, 128, 0, 0, BF, BF, True, 77),
    (33, 28, 4, 128, 48, 8, 0, BF, F32, True, 1000000),
    (7, 17, 3, 64, 48, 16, 0, F32, F32, True, 12345),
    (257, 8, 2, 64, 16, 0, 1, F32, BF, False, 0),
    (19, 40, 8, 128, 112, 16, 1, F32, F32, False, 999),
    (3, 130, 5, 64, 32, 32, 0, BF, BF, True, 5),
    (1031, 4, 4, 128, 128, 0, 1, BF, BF, True, 0),
    (6, 16, 2, 64, 0, 0, 0, BF, BF, False, 3),
]


@pytest.mark.parametrize("T,H,Hk,d,rot,start,style,dtype,out,packed,t0", CASES)
@pytest.mark.parametrize("normed", [True, False])
def test_forward(csa, T, H, Hk, d, rot, start, style, dtype, out, packed, t0, normed):
    q, k, wq, wk, qd, kd = make(T, H, Hk, d, dtype, packed, seed=T)
    f = csa.rope_inv_freq(rot) if rot else None
    w = dict(wq=wq.cuda(), wk=wk.cuda()) if normed else {}
    yq, yk = csa.csa_qk_norm_rope(qd, kd, f, eps=EPS, t0=t0, rot_start=start, rot_style=style, out_dtype=out, **w)
    ang = ref.angles(range(t0, t0 + T), f if rot else [])
    for x, y, wt in ((q, yq, wq), (k, yk, wk)):
        wt = wt if normed else None
        assert y.dtype == out and y.shape == x.shape and y.is_contiguous()
        want = ref.norm_rope(x, wt, EPS, ang, start, style)
        err = (y.cpu().double() - want).abs()
        assert (err <= ref.norm_rope_bound(x, wt, EPS, ang, start, style, out)).all(), err.max()


def test_positions_far_negative_and_repeated(csa):
    pos = [0, 1, -1, 1048575, -(2 ** 40) - 3, 2 ** 40 + 12345, 2 ** 40 + 12345, 7, -(2 ** 62)]
    T, H, d = len(pos), 3, 128
    q, k, wq, wk, qd, kd = make(T, H, 1, d, F32, False, seed=3)
    f = csa.rope_inv_freq(d, base=500000.0)
    f[0], f[1] = 7.5, -0.3  # above a turn a position, and backwards
    for style in (0, 1):
        yq, yk = csa.csa_qk_norm_rope(qd, kd, f, wq=wq.cuda(), pos=torch.tensor(pos).cuda(), rot_style=style, eps=EPS)
        # F is rounded to 2^-65 of a turn and |pos| <= 2^62: up to 2^-3 turns there; 2^-24 turns at 2^41
        near = [i for i, p in enumerate(pos) if abs(p) < 2 ** 41]
        ang = ref.angles(pos, f)
        extra = 2 * math.pi * 2.0 ** -24
        for x, y, w in ((q, yq, wq), (k, yk, None)):
            want = ref.norm_rope(x, w, EPS, ang, 0, style)
            bound = ref.norm_rope_bound(x, w, EPS, ang, 0, style, F32) + extra * 2 * ref.norm(x, w, EPS).abs().amax(-1, keepdim=True)
            assert ((y.cpu().double() - want).abs() <= bound)[near].all()
        assert torch.isfinite(yq).all()


def test_one_side_in_place_and_empty(csa):
    q, k, wq, wk, qd, kd = make(9, 12, 2, 64, BF, False, seed=4)
    f = csa.rope_inv_freq(64)
    both = csa.csa_qk_norm_rope(qd, kd, f, wq=wq.cuda(), wk=wk.cuda())
    only, none = csa.csa_qk_norm_rope(qd, None, f, wq=wq.cuda())
    assert none is None and torch.equal(only, both[0])
    none, only = csa.csa_qk_norm_rope(None, kd, f, wk=wk.cuda())
    assert none is None and torch.equal(only, both[1])
    a, b = qd.clone(), kd.clone()
    r = csa.csa_qk_norm_rope(a, b, f, wq=wq.cuda(), wk=wk.cuda(), yq=a, yk=b)
    assert r[0] is a and torch.equal(a, both[0]) and torch.equal(b, both[1])
    e, _ = csa.csa_qk_norm_rope(qd[:0], None, f, wq=wq.cuda())
    assert e.shape == (0, 12, 64)


@pytest.mark.parametrize("T,H,Hk,d,rot,start,style,dtype,out,packed,t0", CASES)
@pytest.mark.parametrize("normed", [True, False])
def test_backward(csa, T, H, Hk, d, rot, start, style, dtype, out, packed, t0, normed):
    q, k, wq, wk, qd, kd = make(T, H, Hk, d, dtype, packed, seed=T + 1)
    f = csa.rope_inv_freq(rot) if rot else None
    g = torch.Generator().manual_seed(T + 2)
    dy = [torch.randn(T, n, d, generator=g).to(out) for n in (H, Hk)]
    w = dict(wq=wq.cuda(), wk=wk.cuda()) if normed else {}
    if packed:  # gradients straight into a packed gradient
        dqkv = torch.zeros(T, (H + 2 * Hk) * d, dtype=dtype, device="cuda")
        w.update(dq=dqkv[:, :H * d].view(T, H, d), dk=dqkv[:, H * d:(H + Hk) * d].view(T, Hk, d))
    got = csa.csa_qk_norm_rope_backward(qd, kd, dy[0].cuda(), dy[1].cuda(), f, eps=EPS, t0=t0, rot_start=start,
                                        rot_style=style, **w)
    if packed:
        assert (dqkv[:, (H + Hk) * d:] == 0).all()
    ang = ref.angles(range(t0, t0 + T), f if rot else [])
    for i, (x, wt) in enumerate(((q, wq), (k, wk))):
        # the formula by automatic differentiation of the 64-bit forward
        xd = x.double().requires_grad_()
        wd = wt.double().requires_grad_() if normed else None
        y = ref.norm_rope(xd, wd, EPS, ang, start, style)
        y.backward(dy[i].double())
        # bounds, u = 2^-24: g 8u; r 9u (r^3 27u); the two row sums 13u; products 6u: under 64u of
        # r |g w| + |x| r^3 mean |g w x|, with |g| <= the sum of the pair's |dy|
        one = torch.ones(d)
        G = ref.norm_rope_bound(dy[i].double(), None, EPS, ang, start, style, F32) / (20.2 * ref.U)
        if normed:
            r = (x.double().square().mean(-1, keepdim=True) + EPS).rsqrt()
            wabs = wt.double().abs()
            M = r * G * wabs + x.double().abs() * r ** 3 * (G * wabs * x.double().abs()).mean(-1, keepdim=True)
        else:
            M = G
        dx = got[i]
        assert dx.dtype == dtype
        err = (dx.cpu().double() - xd.grad).abs()
        assert (err <= ref.half(dtype) * xd.grad.abs() + 64 * ref.U * M + 1e-30).all(), err.max()
        if normed:
            # a term is good to 20u; the sum's longest chain is under rows + 64 additions
            rows = T * (H, Hk)[i]
            err = (got[2 + i].cpu().double() - wd.grad).abs()
            assert (err <= (rows + 84) * ref.U * (G * x.double().abs() * r).sum((0, 1)) + 1e-30).all(), err.max()
        else:
            assert got[2 + i] is None


@pytest.mark.parametrize("H,Hk,d,dtype,out", [(9, 2, 64, F32, F32), (17, 1, 128, BF, BF), (3, 3, 64, BF, F32)])
def test_backward_of_long_calls(csa, H, Hk, d, dtype, out):
    """More rows than the GPU's blocks take at once: each side with the other and alone, against
    short calls.  dx is the same row by row; dw adds up in another order: both are within
    rows * u of the sum of its terms' sizes, bounded by Cauchy-Schwarz per channel."""
    T, cut = 20011, 1009
    q, k, wq, wk, qd, kd = make(T, H, Hk, d, dtype, False, seed=12)
    g = torch.Generator().manual_seed(13)
    dq, dk = (torch.randn(T, n, d, generator=g).to(out).cuda() for n in (H, Hk))
    f, w = csa.rope_inv_freq(32), dict(wq=wq.cuda(), wk=wk.cuda())
    both = csa.csa_qk_norm_rope_backward(qd, kd, dq, dk, f, **w)
    alone = [csa.csa_qk_norm_rope_backward(qd, None, dq, None, f, wq=w["wq"]),
             csa.csa_qk_norm_rope_backward(None, kd, None, dk, f, wk=w["wk"])]
    parts = [csa.csa_qk_norm_rope_backward(qd[t:t + cut], kd[t:t + cut], dq[t:t + cut], dk[t:t + cut], f, t0=t, **w)
             for t in range(0, T, cut)]
    for i, (x, dy, n) in enumerate(((q, dq, H), (k, dk, Hk))):
        assert torch.equal(both[i], alone[i][i]) and torch.equal(both[i], torch.cat([p[i] for p in parts]))
        want = sum(p[2 + i].double() for p in parts)
        xh = x.double() * (x.double().square().mean(-1, keepdim=True) + EPS).rsqrt()
        e = dy.cpu().double().square().sum((0, 1))   # a channel of g mixes its own and its partner's dy
        size = ((e + e.max()) * xh.square().sum((0, 1))).sqrt().cuda()
        for dw in (both[2 + i], alone[i][2 + i]):
            assert ((dw.double() - want).abs() <= 2 * (T * n + 84) * ref.U * size).all()


def test_gradient_against_differences(csa):
    """Directional differences of the fp32 kernel itself.  h = 2^-7: the truncation
    is h^2/6 of the third derivative (the norm's, of order |v|^3 |y| / |x|^2 a row), the
    rounding 40u |y| / 2h a value, summed over n values at random signs."""
    T, H, d = 6, 5, 64
    q, _, wq, _, qd, _ = make(T, H, 1, d, F32, False, seed=9)
    g = torch.Generator().manual_seed(10)
    dy = torch.randn(T, H, d, generator=g).cuda()
    v, vw = torch.randn(T, H, d, generator=g).cuda(), torch.randn(d, generator=g).cuda()
    f, h, w = csa.rope_inv_freq(64), 2.0 ** -7, wq.cuda()
    dq, _, dwq, _, _ = csa.csa_qk_norm_rope_backward(qd, None, dy, None, f, wq=w, t0=100)
    loss = lambda x, w: (csa.csa_qk_norm_rope(x, None, f, wq=w, t0=100)[0].double() * dy.double()).sum()
    n = T * H * d
    for along, diff in (((dq.double() * v.double()).sum(), loss(qd + h * v, w) - loss(qd - h * v, w)),
                        ((dwq.double() * vw.double()).sum(), loss(qd, w + h * vw) - loss(qd, w - h * vw))):
        # rounding: 40u * ~1 / 2h * sqrt(n) * 4 deviations; truncation: h^2 * sqrt(n) * 4
        assert abs(float(along - diff / (2 * h))) <= 4 * math.sqrt(n) * (40 * ref.U / (2 * h) + h * h)


def test_repeats_bit_for_bit_and_replays(csa):
    q, k, wq, wk, qd, kd = make(700, 16, 4, 128, BF, True, seed=11)
    w = dict(wq=wq.cuda(), wk=wk.cuda())
    f = csa.rope_inv_freq(128)
    pos = torch.arange(700, device="cuda")
    dy = torch.randn(700, 16, 128, device="cuda").bfloat16(), torch.randn(700, 4, 128, device="cuda").bfloat16()
    first = csa.csa_qk_norm_rope_backward(qd, kd, *dy, f, pos=pos, **w)
    ws = first[4]
    yf = csa.csa_qk_norm_rope(qd, kd, f, pos=pos, **w)
    outs = [torch.empty_like(t) for t in first[:4]] + [torch.empty_like(t) for t in yf]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream), torch.cuda.graph(graph, stream=stream):
        csa.csa_qk_norm_rope(qd, kd, f, pos=pos, yq=outs[4], yk=outs[5], **w)
        csa.csa_qk_norm_rope_backward(qd, kd, *dy, f, pos=pos, dq=outs[0], dk=outs[1], dwq=outs[2], dwk=outs[3],
                                      workspace=ws, **w)
    for _ in range(2):
        for o in outs:
            o.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for o, e in zip(outs, list(first[:4]) + list(yf)):
            assert torch.equal(o, e)
    # a replay follows new positions
    pos += 5
    graph.replay()
    again = csa.csa_qk_norm_rope(qd, kd, f, pos=pos, **w)
    assert torch.equal(outs[4], again[0]) and not torch.equal(again[0], yf[0])


def test_zero_rows_and_empty_batch(csa):
    f = csa.rope_inv_freq(64)
    x = torch.zeros(3, 2, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    y, _ = csa.csa_qk_norm_rope(x, None, f, wq=w)
    assert (y == 0).all()
    dwq = torch.full((64,), float("nan"), device="cuda")
    e = x[:0]
    r = csa.csa_qk_norm_rope_backward(e, None, e, None, f, wq=w, dwq=dwq)
    assert (r[2] == 0).all()
