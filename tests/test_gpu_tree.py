"""csa_tree_attn against the 64-bit form: lengths around the tiles, ragged batches,
trees of 1 to 64 nodes, head groups of any size, pages that end inside a tile,
windows, rows that see nothing, rows outside every sequence, garbage where nothing
is visible, bad numbers, captured calls; and the verification step as a whole."""
import math

import pytest
import torch

from tests import positioned_ref as ref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def csa():
    import long_context_compressed_gated_b200 as m
    m.lib()
    return m


def tree(n, g):
    m = []
    for i in range(n):
        p = int(torch.randint(-1, i, (1,), generator=g)) if i else -1
        m.append((m[p] if p >= 0 else 0) | 1 << i)
    return m


def signed(m):
    return m - (1 << 64) if m >> 63 else m


def make(lens, nodes, H, Hk, d, page, seed=0, garbage=math.nan, lead=0, tail=0, spread=1.0):
    """A batch whose cache holds `garbage` wherever no sequence has a row, and whose
    tables hold -1 where they need no page."""
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    need = [-(-(L + n) // page) for L, n in zip(lens, nodes)]
    total = sum(need) + 2
    Kp, Vp = (torch.full((total, Hk, page, d), garbage).to(BF) for _ in range(2))
    table = torch.full((B, max(need + [0]) + 1), -1, dtype=torch.int32)
    order = torch.randperm(total, generator=g)
    at = 0
    for b in range(B):
        table[b, :need[b]] = order[at:at + need[b]].to(torch.int32)
        at += need[b]
        S = lens[b] + nodes[b]
        s = torch.arange(S)
        Kp[table[b].long()[s // page], :, s % page] = (torch.randn(S, Hk, d, generator=g) * spread).to(BF)
        Vp[table[b].long()[s // page], :, s % page] = torch.randn(S, Hk, d, generator=g).to(BF)
    start = [lead]
    for n in nodes:
        start.append(start[-1] + n)
    R = start[-1] + tail
    mask, pos = [0] * lead, [0] * lead
    for b in range(B):
        m = tree(nodes[b], g)
        mask += m
        pos += [lens[b] + bin(x).count("1") - 1 for x in m]
    mask += [0] * tail
    pos += [0] * tail
    q = torch.randn(R, H, d, generator=g).to(BF)
    return dict(q=q, Kp=Kp, Vp=Vp, table=table, lens=torch.tensor(lens, dtype=torch.int32),
                start=torch.tensor(start, dtype=torch.int32), mask=torch.tensor([signed(m) for m in mask], dtype=torch.int64),
                pos=torch.tensor(pos, dtype=torch.int64))


def call(csa, x, W=-1, out=BF, **kw):
    c = {k: v.cuda() for k, v in x.items()}
    scale = kw.pop("scale", 1 / math.sqrt(x["q"].shape[2]))
    return csa.csa_tree_attn(c["q"], c["Kp"], c["Vp"], c["table"], c["lens"], c["start"], c["mask"], scale, W=W,
                             pos=c["pos"], out_dtype=out, **kw)


def check(x, O, lse, W=-1, scale=None):
    """Against the 64-bit form.  u = 2^-24, Z the largest scale * sum |q||k| of a row's keys:
      a logit is a d-term fp32 sum, scaled: (d + 4) u Z; its exponential (2 ulp, argument rounded,
      its maximum subtracted) 4u + 2u Z; merged shares and the final division a few u: each weight
      is good to e = (d + 16) u max(Z, 1), and its bf16 rounding for the product with V adds
      half(bf16).  O: (half(bf16) + 2e) sum p|v|, plus its own rounding; lse: e plus n u of the sum
      of n weights, plus 4u of its value."""
    d = x["q"].shape[2]
    scale = 1 / math.sqrt(d) if scale is None else scale
    want, wl, A = ref.tree_attention(x["q"], x["Kp"], x["Vp"], x["table"], x["lens"], x["start"], x["mask"], scale, W,
                                     x["pos"])
    inside = ~want.isnan().any(-1).any(-1)
    Kmax = x["Kp"].double().nan_to_num(0, 0, 0).abs().amax((0, 1, 2))
    Z = scale * (x["q"].double().abs() * Kmax).sum(-1, keepdim=True).clamp(min=1)
    e = (d + 16) * ref.U * Z
    O, lse = O.cpu(), lse.cpu()
    bound = (ref.half(BF) + 2 * e) * 1.01 * A + ref.half(O.dtype) * want.abs() + 1e-30
    err = (O.double() - want).abs()
    assert (err <= bound)[inside].all(), (err - bound)[inside].max()
    n = int((x["lens"] + (x["start"][1:] - x["start"][:-1])).max()) if len(x["lens"]) else 0
    empty = wl == -math.inf
    assert torch.equal(lse[inside] == -math.inf, empty[inside])
    el = (lse.double() - wl).abs()
    ok = el <= e[..., 0] + n * ref.U + 4 * ref.U * wl.abs()
    assert (ok | empty)[inside].all(), el[inside & ~empty.any(-1)].max()
    return inside


SHAPES = [
    # lens, nodes, H, Hk, d, page
    ([0], [1], 1, 1, 64, 16),
    ([1], [1], 64, 1, 128, 64),
    ([0, 5, 16, 31], [3, 1, 16, 2], 8, 2, 64, 16),
    ([127, 128, 126, 129], [1, 1, 2, 1], 64, 1, 128, 64),
    ([255, 700, 256, 1], [1, 1, 1, 1], 32, 8, 128, 128),
    ([300, 17, 1000], [64, 33, 5], 28, 4, 128, 32),
    ([1500, 64], [64, 64], 64, 1, 128, 64),
    ([90, 0, 411], [7, 0, 12], 40, 8, 64, 16),
    ([2049], [9], 16, 16, 64, 256),
    ([640, 130], [16, 3], 128, 1, 64, 32),
    ([513, 1025], [31, 63], 5, 1, 128, 16),
    ([7000], [1], 4, 2, 128, 64),
]


@pytest.mark.parametrize("lens,nodes,H,Hk,d,page", SHAPES)
@pytest.mark.parametrize("out", [BF, F32])
def test_against_the_formula(csa, lens, nodes, H, Hk, d, page, out):
    x = make(lens, nodes, H, Hk, d, page, seed=sum(lens) + H)
    O, lse, ws = call(csa, x, out=out)
    assert csa.csa_check_status(ws) == 0
    assert O.dtype == out and check(x, O, lse).all()


@pytest.mark.parametrize("W", [0, 1, 5, 64, 130, 300, 100000])
@pytest.mark.parametrize("lens,nodes,H,Hk,d,page", [([700, 3, 0, 129], [9, 4, 2, 1], 64, 1, 128, 32),
                                                     ([1100, 257], [30, 40], 12, 4, 64, 16)])
def test_window(csa, W, lens, nodes, H, Hk, d, page):
    x = make(lens, nodes, H, Hk, d, page, seed=W)
    for b in range(len(lens)):   # pages wholly below every row's window are freed, rows below it garbage
        lo = max(0, lens[b] - W + 1)
        s = torch.arange(min(lo, lens[b]))
        pg = x["table"][b].long()[s // page]
        x["Kp"][pg, :, s % page] = math.nan
        x["Vp"][pg, :, s % page] = math.inf
        x["table"][b, :min(lo, lens[b]) // page] = -1
    O, lse, ws = call(csa, x, W=W)
    assert csa.csa_check_status(ws) == 0
    check(x, O, lse, W=W)


@pytest.mark.parametrize("W", [0, 3, 2**31 - 1])
def test_window_at_any_position(csa, W):
    x = make([300, 40], [5, 3], 8, 2, 64, 16, seed=30)
    x["pos"][:] = torch.tensor([2**63 - 1, -2**63, 2**62, W, 299 + W, 2**63 - 1, -1, 40 + W])
    O, lse, ws = call(csa, x, W=W)
    assert csa.csa_check_status(ws) == 0 and check(x, O, lse, W=W).all()


def test_rows_that_see_nothing(csa):
    x = make([0, 40, 0], [4, 3, 70 - 6], 16, 2, 64, 16, seed=5)
    x["mask"][1] = 0            # no key at all
    x["mask"][2] = -16          # only nodes that are not there
    x["mask"][5] = 0            # committed rows only
    x["mask"][7:] = 0
    O, lse, _ = call(csa, x, out=F32)
    check(x, O, lse)
    assert (O[1] == 0).all() and (O[2] == 0).all() and (lse[1] == -math.inf).all() and (O[7:] == 0).all()
    O, lse, _ = call(csa, x, W=0)   # and a window that hides every committed row
    check(x, O, lse, W=0)
    assert (O[5] == 0).all()


def test_rows_outside_the_sequences_are_left(csa):
    x = make([100, 20], [5, 2], 8, 1, 64, 16, seed=6, lead=3, tail=4)
    O = torch.full(x["q"].shape, 7.0, dtype=BF, device="cuda")
    lse = torch.full(x["q"].shape[:2], 7.0, device="cuda")
    call(csa, x, O=O, lse=lse)
    inside = check(x, O, lse)
    assert inside.tolist() == [False] * 3 + [True] * 7 + [False] * 4
    assert (O.cpu()[~inside] == 7).all() and (lse.cpu()[~inside] == 7).all()


def test_peaked_and_large_logits(csa):
    x = make([900, 333], [8, 20], 16, 4, 128, 64, seed=7, spread=8.0)
    O, lse, _ = call(csa, x)
    check(x, O, lse)
    x = make([900, 333], [8, 20], 16, 4, 64, 64, seed=8)
    x["Kp"][x["table"][0, 0]] *= 30      # the first page's logits dwarf the rest, then the last page's those
    x["Kp"][x["table"][0, 14]] *= 60
    O, lse, _ = call(csa, x)
    check(x, O, lse)


def test_hidden_drafts_with_equal_pages_and_shared_prefix(csa):
    """Two sequences share their prefix pages; the answer is that of separate copies."""
    x = make([256, 256], [6, 6], 8, 2, 128, 64, seed=9)
    for t in ("Kp", "Vp"):
        x[t][x["table"][1, :4].long()] = x[t][x["table"][0, :4].long()]
    O, lse, _ = call(csa, x)
    x["table"][1, :4] = x["table"][0, :4]
    O2, lse2, _ = call(csa, x)
    assert torch.equal(O, O2) and torch.equal(lse, lse2)
    check(x, O2, lse2)


@pytest.mark.parametrize("what", ["page", "page_negative", "long", "negative", "nodes", "backwards", "beyond"])
def test_bad_numbers_are_reported(csa, what):
    lens, nodes = [100, 200, 50], [3, 4, 2]
    x = make(lens, nodes, 8, 2, 64, 16, seed=10)
    good, glse, _ = call(csa, x)
    good = good.cpu()
    if what == "page":
        x["table"][1, 3] = x["Kp"].shape[0]
    elif what == "page_negative":
        x["table"][1, 3] = -7
    elif what == "long":
        x["lens"][1] = 16 * x["table"].shape[1] - 3
    elif what == "negative":
        x["lens"][1] = -1
    elif what == "nodes":
        y = make([100, 200, 50], [3, 65, 2], 8, 2, 64, 16, seed=10)
        O, lse, ws = call(csa, y)
        assert csa.csa_check_status(ws) == -8
        return
    elif what == "backwards":
        x["start"][2] = 1
    else:
        x["start"][3] = 10
    O, lse, ws = call(csa, x)
    assert csa.csa_check_status(ws) == -8 and csa.csa_check_status(ws) == 0
    if what not in ("backwards", "beyond"):   # the other sequences' rows stand
        O = O.cpu()
        assert torch.equal(O[:3], good[:3]) and torch.equal(O[7:], good[7:])


def test_repeats_and_captured_calls_follow_new_lengths(csa):
    x = make([4000, 900, 77], [1, 1, 1], 64, 1, 128, 64, seed=11)
    c = {k: v.cuda() for k, v in x.items()}
    O, lse, ws = call(csa, x)
    out = torch.empty_like(O)
    l2 = torch.empty_like(lse)
    run = lambda: csa.csa_tree_attn(c["q"], c["Kp"], c["Vp"], c["table"], c["lens"], c["start"], c["mask"],
                                    1 / math.sqrt(128), pos=c["pos"], O=out, lse=l2, workspace=ws)
    for _ in range(3):
        out.fill_(math.nan)
        run()
        assert torch.equal(out, O) and torch.equal(l2, lse)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        run()
    for lens in ([4000, 900, 77], [1, 900, 0], [127, 128, 64], [3999, 0, 70]):
        x["lens"] = torch.tensor(lens, dtype=torch.int32)
        c["lens"].copy_(x["lens"])
        graph.replay()
        check(x, out, l2)
    assert csa.csa_check_status(ws) == 0


def test_many_items_a_share(csa):
    """Shares of several items whose last row tiles are filled in part, back to back."""
    x = make([2052, 1930], [47, 53], 32, 8, 128, 64, seed=17)
    first = None
    for _ in range(6):
        O, lse, _ = call(csa, x)
        first = O if first is None else first
        assert torch.equal(O, first)
    check(x, O, lse)


@pytest.mark.parametrize("H,Hk,d,page", [(64, 1, 128, 128), (28, 4, 64, 32)])
def test_short_sequences_back_to_back(csa, H, Hk, d, page):
    """Items of one or two key tiles, whose products finish before the outputs of the
    item before are written: the roles of a CTA may drift apart as far as they can."""
    g = torch.Generator().manual_seed(18)
    lens = torch.randint(0, 150, (90,), generator=g).tolist()
    nodes = torch.randint(1, 9, (90,), generator=g).tolist()
    x = make(lens, nodes, H, Hk, d, page, seed=19)
    c = {k: v.cuda() for k, v in x.items()}
    O, lse, ws = call(csa, x)
    check(x, O, lse)
    for _ in range(40):
        again, _, _ = csa.csa_tree_attn(c["q"], c["Kp"], c["Vp"], c["table"], c["lens"], c["start"], c["mask"],
                                        1 / math.sqrt(d), pos=c["pos"], workspace=ws)
    assert torch.equal(again, O) and csa.csa_check_status(ws) == 0


def test_empty_calls(csa):
    x = make([10], [2], 4, 1, 64, 16)
    x["start"] = torch.zeros(2, dtype=torch.int32)   # rows, but no nodes
    O = torch.full(x["q"].shape, 3.0, dtype=BF, device="cuda")
    call(csa, x, O=O)
    assert (O == 3).all()
    x = make([], [], 4, 1, 64, 16)
    O, lse, _ = call(csa, x)
    assert O.shape == (0, 4, 64)


@pytest.mark.parametrize("W", [-1, 40])
def test_many_sequences(csa, W):
    g = torch.Generator().manual_seed(12)
    lens = torch.randint(0, 300, (200,), generator=g).tolist()
    nodes = torch.randint(0, 4, (200,), generator=g).tolist()
    x = make(lens, nodes, 8, 2, 64, 16, seed=13)
    O, lse, ws = call(csa, x, W=W)
    assert csa.csa_check_status(ws) == 0 and check(x, O, lse, W=W).all()


@pytest.mark.parametrize("d,page", [(64, 16), (128, 16), (128, 256)])
def test_long_tables(csa, d, page):
    """More pages than are read ahead at once, from the middle of a run on (window)."""
    x = make([9000, 4100], [3, 5], 8, 2, d, page, seed=20)
    for W in (-1, 3333):
        O, lse, ws = call(csa, x, W=W)
        assert csa.csa_check_status(ws) == 0 and check(x, O, lse, W=W).all()


def test_two_streams_at_once(csa):
    """Calls that overlap on the GPU, each with its own workspace."""
    xs = [make([3000, 50, 777], [9, 4, 1], 16, 2, 128, 64, seed=s) for s in (21, 22)]
    cs = [{k: v.cuda() for k, v in x.items()} for x in xs]
    want = [call(csa, x)[:2] for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = []
    for _ in range(20):
        got = []
        for c, st in zip(cs, streams):
            with torch.cuda.stream(st):
                got.append(csa.csa_tree_attn(c["q"], c["Kp"], c["Vp"], c["table"], c["lens"], c["start"], c["mask"],
                                             1 / math.sqrt(128), pos=c["pos"])[:2])
    torch.cuda.synchronize()
    for (O, l), (wO, wl) in zip(got, want):
        assert torch.equal(O, wO) and torch.equal(l, wl)


def test_partials_combine_with_compressed_entries(csa):
    """The window branch over the paged cache plus the selected compressed entries,
    merged by csa_attn_combine, is the one joint softmax of csa_sparse_attn."""
    T, H, d, W, k, m, page, n = 600, 16, 128, 128, 32, 4, 64, 7
    g = torch.Generator().manual_seed(14)
    K, V, Z = (torch.randn(T, d, generator=g).to(BF).cuda() for _ in range(3))
    Kc, Vc = csa.csa_compress(K, V, Z, torch.zeros(m, d, device="cuda"), m)
    Q = torch.randn(n, H, d, generator=g).to(BF).cuda()
    idx = torch.stack([torch.randperm((T - n) // m, generator=g)[:k] for _ in range(n)]).to(torch.int32).cuda()
    scale = 1 / math.sqrt(d)
    want, wl, _ = csa.csa_sparse_attn(Q, Kc, Vc, idx, K, V, W, scale, t0=T - n, out_dtype=F32)
    a, la, _ = csa.csa_sparse_attn(Q, Kc, Vc, idx, K, V, 0, scale, t0=T - n, out_dtype=F32)
    pages = -(-T // page)
    Kp, Vp = (torch.zeros(pages * page, d, dtype=BF, device="cuda") for _ in range(2))
    Kp[:T], Vp[:T] = K, V
    shape = (pages, 1, page, d)
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    b, lb, _ = csa.csa_tree_attn(Q, Kp.view(shape), Vp.view(shape), table,
                                 torch.tensor([T - n], dtype=torch.int32).cuda(),
                                 torch.tensor([0, n], dtype=torch.int32).cuda(),
                                 torch.tensor([(2 << i) - 1 for i in range(n)]).cuda(), scale, W=W,
                                 pos=torch.arange(T - n, T).cuda(), out_dtype=F32)
    O, lse = csa.csa_attn_combine(torch.stack([a, b]), torch.stack([la, lb]), out_dtype=F32)
    # two paths of bf16 weights apart: twice half(bf16) of sum p|v| <= max|v| (about 4)
    assert (O - want).abs().max() <= 2 * ref.half(BF) * 4
    assert (lse - wl).abs().max() <= 1e-4


@pytest.mark.parametrize("H,Hk,d,page,W", [(64, 1, 128, 64, -1), (12, 3, 64, 16, 200)])
def test_verification_step(csa, H, Hk, d, page, W):
    """Norm + rotation, append and attention together, against the 64-bit forms."""
    from long_context_compressed_gated_b200.speculative import tree_verify_step
    lens, nodes = [500, 0, 63], [6, 1, 17]
    x = make(lens, nodes, H, Hk, d, page, seed=15, tail=2)
    R = x["q"].shape[0]
    g = torch.Generator().manual_seed(16)
    qkv = torch.randn(R, (H + 2 * Hk) * d, generator=g).to(BF)
    wq, wk = (1 + 0.2 * torch.randn(d, generator=g) for _ in range(2))
    seq = torch.tensor([b for b in range(3) for _ in range(nodes[b])] + [0, 0], dtype=torch.int32)
    slot = torch.tensor([lens[b] + i for b in range(3) for i in range(nodes[b])] + [-1, -1])
    f = csa.rope_inv_freq(64)
    c = {k: v.cuda() for k, v in x.items()}
    start = d - 64
    lse = torch.zeros(R, H, device="cuda")
    need = csa.lib().csa_tree_attn_workspace_bytes(3, R, H, Hk, d, page, x["table"].shape[1])
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    scale = 1 / math.sqrt(d)
    O = tree_verify_step(qkv.cuda(), H, Hk, c["Kp"], c["Vp"], c["table"], c["lens"], c["start"], c["mask"],
                         seq.cuda(), slot.cuda(), c["pos"], f, scale, wq=wq.cuda(), wk=wk.cuda(), rot_start=start,
                         rot_style=1, W=W, lse=lse, workspace=ws)
    assert csa.csa_check_status(ws) == 0
    a = qkv.view(R, H + 2 * Hk, d)
    ang = ref.angles(x["pos"], f)
    q = ref.norm_rope(a[:, :H], wq, 1e-6, ang, start, 1)
    k = ref.norm_rope(a[:, H:H + Hk], wk, 1e-6, ang, start, 1)
    kb = ref.norm_rope_bound(a[:, H:H + Hk], wk, 1e-6, ang, start, 1, BF)
    for t in range(R - 2):
        p, o = int(x["table"][int(seq[t]), int(slot[t]) // page]), int(slot[t]) % page
        assert ((c["Kp"][p, :, o].cpu().double() - k[t]).abs() <= kb[t]).all()
        x["Kp"][p, :, o], x["Vp"][p, :, o] = c["Kp"][p, :, o].cpu(), a[t, H + Hk:]
    assert torch.equal(c["Vp"].cpu().nan_to_num(9), x["Vp"].nan_to_num(9))
    # the attention's queries are the kernel's own bf16 ones, which the first assertion pins
    yq, _ = csa.csa_qk_norm_rope(qkv.cuda().view(R, H + 2 * Hk, d)[:, :H], None, f, wq=wq.cuda(), pos=c["pos"],
                                 rot_start=start, rot_style=1)
    qb = ref.norm_rope_bound(a[:, :H], wq, 1e-6, ang, start, 1, BF)
    assert ((yq.cpu().double() - q).abs() <= qb).all()
    x["q"] = yq.cpu()
    check(x, O, lse, W=W)


@pytest.mark.parametrize("out", [BF, F32])
def test_verification_step_is_its_three_calls(csa, out):
    """Rows of a wider projection, eager and captured, bit for bit as the three functions."""
    from long_context_compressed_gated_b200.speculative import tree_verify_step
    H, Hk, d, page, lens, nodes = 12, 3, 64, 16, [200, 31], [5, 9]
    x = make(lens, nodes, H, Hk, d, page, seed=40)
    c = {k: v.cuda() for k, v in x.items()}
    R, width = x["q"].shape[0], (H + 2 * Hk) * d
    g = torch.Generator().manual_seed(41)
    qkv = torch.randn(R, width + 64, generator=g).to(BF).cuda()[:, :width]
    seq = torch.tensor([b for b in range(2) for _ in range(nodes[b])], dtype=torch.int32).cuda()
    slot = torch.tensor([lens[b] + i for b in range(2) for i in range(nodes[b])]).cuda()
    f, w = csa.rope_inv_freq(32), torch.ones(d, device="cuda")
    v = qkv.view(R, H + 2 * Hk, d)
    Kp, Vp = c["Kp"].clone(), c["Vp"].clone()
    q, _ = csa.csa_qk_norm_rope(v[:, :H], None, f, wq=w, pos=c["pos"], eps=1e-5)
    csa.csa_paged_append(v[:, H:H + Hk], v[:, H + Hk:], Kp, Vp, c["table"], seq, c["pos"], f, slot=slot, wk=w, eps=1e-5)
    want, wl, _ = csa.csa_tree_attn(q, Kp, Vp, c["table"], c["lens"], c["start"], c["mask"], 0.2, W=150, pos=c["pos"],
                                    out_dtype=out)
    lse, ws = torch.empty(R, H, device="cuda"), torch.zeros(1 << 22, dtype=torch.uint8, device="cuda")

    def step(O=None, **kw):
        return tree_verify_step(qkv, H, Hk, c["Kp"], c["Vp"], c["table"], c["lens"], c["start"], c["mask"], seq, slot,
                                c["pos"], f, 0.2, wq=w, wk=w, eps=1e-5, W=150, O=O, out_dtype=out, **kw)

    def same(O):
        bits = lambda t: t.view(torch.int16)
        return torch.equal(O, want) and torch.equal(bits(c["Kp"]), bits(Kp)) and torch.equal(bits(c["Vp"]), bits(Vp))

    assert same(step(lse=lse)) and torch.equal(lse, wl)
    O = torch.empty_like(want)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(O=O, workspace=ws)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step(O=O, workspace=ws)
    torch.cuda.synchronize()
    O.zero_(), c["Kp"].copy_(x["Kp"]), c["Vp"].copy_(x["Vp"])
    graph.replay()
    torch.cuda.synchronize()
    assert same(O) and csa.csa_check_status(ws) == 0
    none = [t[:0] for t in (qkv, c["mask"], seq, slot, c["pos"])]
    e = tree_verify_step(none[0], H, Hk, c["Kp"], c["Vp"], c["table"], c["lens"], c["start"] * 0, none[1], none[2],
                         none[3], none[4], f, 0.2)
    assert e.shape == (0, H, d)


def test_verification_step_refuses(csa):
    from long_context_compressed_gated_b200.speculative import tree_verify_step
    x = make([20], [2], 4, 2, 64, 16, seed=42)
    c = {k: v.cuda() for k, v in x.items()}
    seq, slot = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.tensor([20, 21]).cuda()
    good = dict(qkv=torch.zeros(2, 8 * 64, dtype=BF, device="cuda"), H=4, Hk=2, Kpages=c["Kp"], Vpages=c["Vp"],
                block_table=c["table"], seq_lens=c["lens"], q_start=c["start"], mask=c["mask"], seq=seq, slot=slot,
                pos=c["pos"], inv_freq=csa.rope_inv_freq(64), scale=0.1)
    tree_verify_step(**good)
    for change, error in ((dict(H=5), ValueError), (dict(Hk=1), ValueError), (dict(qkv=good["qkv"].float()), TypeError),
                          (dict(qkv=good["qkv"].cpu()), TypeError), (dict(qkv=good["qkv"][0]), ValueError),
                          (dict(qkv=good["qkv"].t().contiguous().t()), ValueError), (dict(pos=None), ValueError),
                          (dict(slot=slot[:1]), ValueError), (dict(seq=slot), TypeError),
                          (dict(mask=c["mask"].cpu()), TypeError), (dict(out_dtype=torch.float16), TypeError),
                          (dict(O=torch.zeros(2, 4, 32, dtype=BF, device="cuda")), ValueError),
                          (dict(lse=torch.zeros(2, 4, dtype=BF, device="cuda")), TypeError),
                          (dict(workspace=torch.zeros(256, dtype=torch.uint8, device="cuda")), csa.CsaError),
                          (dict(scale=0.0), csa.CsaError), (dict(wq=torch.zeros(32, device="cuda")), ValueError)):
        with pytest.raises(error):
            tree_verify_step(**dict(good, **change))
