"""csa_paged_append against the 64-bit form: page sizes, key heads, ragged and
padding rows, drafted rows whose slot is not their position, untouched rows, bad
numbers reported and skipped, captured calls."""
import pytest
import torch

from tests import positioned_ref as ref

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
EPS = 1e-6


@pytest.fixture(scope="module")
def csa():
    import long_context_compressed_gated_b200 as m
    m.lib()
    return m


def cache(n_pages, Hk, page, d, B, max_pages, seed):
    g = torch.Generator().manual_seed(seed)
    Kp, Vp = (torch.randn(n_pages, Hk, page, d, generator=g).to(BF) for _ in range(2))
    table = torch.randperm(n_pages, generator=g)[:B * max_pages].view(B, max_pages).to(torch.int32)
    return Kp, Vp, table


@pytest.mark.parametrize("page,Hk,d,rot,start,style,normed,T", [
    (16, 1, 128, 64, 64, 1, True, 1), (16, 5, 64, 48, 16, 0, True, 130), (64, 8, 128, 128, 0, 0, True, 77),
    (128, 1, 128, 64, 64, 1, False, 513), (256, 2, 64, 0, 0, 0, True, 40), (32, 4, 64, 64, 0, 1, False, 31)])
def test_append(csa, page, Hk, d, rot, start, style, normed, T):
    B, max_pages = 3, 6
    Kp, Vp, table = cache(B * max_pages + 2, Hk, page, d, B, max_pages, T)
    g = torch.Generator().manual_seed(T + 1)
    qkv = torch.randn(T, (3 + 2 * Hk) * d, generator=g).to(BF)
    seq = torch.randint(0, B, (T,), generator=g).to(torch.int32)
    room = B * max_pages * page
    slot = torch.randperm(max_pages * page, generator=g).repeat(B)[:T] if T > max_pages * page else \
        torch.randperm(max_pages * page, generator=g)[:T]
    slot = slot.clone()
    if T > 20:
        slot[3], slot[17] = -1, -5   # padding rows
    seen = set()
    for t in range(T):               # (sequence, slot) pairs are distinct
        while int(slot[t]) >= 0 and (int(seq[t]), int(slot[t])) in seen:
            slot[t] = (slot[t] + 1) % (max_pages * page)
        seen.add((int(seq[t]), int(slot[t])))
    assert len(seen) <= room
    pos = slot + torch.randint(-3, 100000, (T,), generator=g)
    w = 1 + 0.3 * torch.randn(d, generator=g)
    f = csa.rope_inv_freq(rot) if rot else None
    x = qkv.cuda()
    k, v = x[:, 3 * d:(3 + Hk) * d].view(T, Hk, d), x[:, (3 + Hk) * d:].view(T, Hk, d)
    Kg, Vg = Kp.cuda(), Vp.cuda()
    ws = csa.csa_paged_append(k, v, Kg, Vg, table.cuda(), seq.cuda(), pos.cuda(), f, slot=slot.cuda(),
                              wk=w.cuda() if normed else None, eps=EPS, rot_start=start, rot_style=style)
    assert csa.csa_check_status(ws) == 0
    kc = k.cpu()
    ang = ref.angles(pos, f if rot else [])
    wt = w if normed else None
    want = ref.norm_rope(kc, wt, EPS, ang, start, style)
    bound = ref.norm_rope_bound(kc, wt, EPS, ang, start, style, BF)
    Kw, Vw, E = Kp.double(), Vp.clone(), torch.zeros(Kp.shape, dtype=torch.float64)
    for t in range(T):
        s = int(slot[t])
        if s >= 0:
            p, o = int(table[int(seq[t]), s // page]), s % page
            Kw[p, :, o], Vw[p, :, o], E[p, :, o] = want[t], v[t].cpu(), bound[t]
    assert torch.equal(Vg.cpu(), Vw)
    assert ((Kg.cpu().double() - Kw).abs() <= E).all()   # bound 0 where nothing was written


def test_slot_defaults_to_position_and_matches_the_rotation(csa):
    T, Hk, d = 50, 2, 128
    Kp, Vp, table = cache(8, Hk, 16, d, 2, 4, 5)
    x = torch.randn(T, Hk, d).to(BF).cuda()
    f = csa.rope_inv_freq(64)
    pos = torch.cat([torch.arange(30), torch.arange(20)]).cuda()
    seq = torch.tensor([0] * 30 + [1] * 20, dtype=torch.int32).cuda()
    Kg, Vg = Kp.cuda(), Vp.cuda()
    csa.csa_paged_append(x, x, Kg, Vg, table.cuda(), seq, pos, f, rot_start=64, rot_style=1)
    _, y = csa.csa_qk_norm_rope(None, x, f, pos=pos, rot_start=64, rot_style=1)
    for b, n in ((0, 30), (1, 20)):   # the same bits as the rotation alone
        assert torch.equal(ref.paged_rows(Kg.cpu(), table, b, n), y.cpu()[seq.cpu() == b])
        assert torch.equal(ref.paged_rows(Vg.cpu(), table, b, n), x.cpu()[seq.cpu() == b])


@pytest.mark.parametrize("what", ["seq", "seq_negative", "slot", "page", "page_negative"])
def test_bad_numbers_are_reported_and_skipped(csa, what):
    T, Hk, d = 4, 1, 64
    Kp, Vp, table = cache(6, Hk, 16, d, 2, 2, 6)
    seq, pos = torch.tensor([0, 0, 1, 1], dtype=torch.int32), torch.tensor([3, 17, 4, 18])
    if what == "seq":
        seq[1] = 2
    elif what == "seq_negative":
        seq[1] = -1
    elif what == "slot":
        pos[1] = 2 ** 33
    else:
        table[0, 1] = 6 if what == "page" else -1
    x = torch.randn(T, Hk, d).to(BF).cuda()
    Kg, Vg = Kp.cuda(), Vp.cuda()
    ws = csa.csa_paged_append(x, x, Kg, Vg, table.cuda(), seq.cuda(), pos.cuda(), None)
    assert csa.csa_check_status(ws) == -8 and csa.csa_check_status(ws) == 0
    Kw = Kp.clone()
    for t in (0, 2, 3):
        Kw[int(table[int(seq[t]), int(pos[t]) // 16]), :, int(pos[t]) % 16] = x[t].cpu()
    assert torch.equal(Kg.cpu(), Kw)


def test_empty_and_replayed(csa):
    Hk, d = 1, 128
    Kp, Vp, table = cache(4, Hk, 32, d, 1, 4, 7)
    Kg, Vg, tg = Kp.cuda(), Vp.cuda(), table.cuda()
    x = torch.randn(1, Hk, d).to(BF).cuda()
    seq = torch.zeros(1, dtype=torch.int32, device="cuda")
    pos = torch.zeros(1, dtype=torch.int64, device="cuda")
    f = csa.rope_inv_freq(128)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    csa.csa_paged_append(x[:0], x[:0], Kg, Vg, tg, seq[:0], pos[:0], f, workspace=ws)
    assert torch.equal(Kg.cpu(), Kp)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        csa.csa_paged_append(x, x, Kg, Vg, tg, seq, pos, f, workspace=ws)
    for p in (0, 31, 32, 100):   # one captured call serves every later position
        pos.fill_(p)
        x.normal_()
        graph.replay()
        _, y = csa.csa_qk_norm_rope(None, x, f, pos=pos)
        pg = int(table[0, p // 32])
        assert torch.equal(Kg[pg, 0, p % 32], y[0, 0]) and torch.equal(Vg[pg, 0, p % 32], x[0, 0])
