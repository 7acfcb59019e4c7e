"""The positioned, paged serving and training operators around the attention of this library: what is timed and
compared, in plain torch form and through the library's own entry points.

  norm_rope       per-head RMS norm of queries and keys with the position rotation (csa_qk_norm_rope)
  norm_rope_grad  its backward pass (csa_qk_norm_rope_backward)
  append          keys (normed and rotated on the way) and values into a paged cache (csa_paged_append)
  tree            attention of a tree of drafted tokens, or of one token, over that cache (csa_tree_attn)
  step            one verification step: norm + rotation, append, attention (tree_verify_step)

A case is a dict of plain values; `run` computes it in its plain form, or through the library where `own` is set.
"""
import math
import random

import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32
TYPES = {"bf16": BF16, "f32": F32}
EPS = 1e-6


def listed():
    return [
        # one decode step's queries and keys of 16 sequences at the end of a 1M-token context: latency alone
        dict(name="norm_rope_decode_B16", op="norm_rope", T=16, H=64, Hk=1, d=128, rot=64, start=64, style=1,
             dtype="bf16", out="bf16", packed=True, far=1048575),
        # a prefill of 32768 tokens, queries and keys views of one packed projection
        dict(name="norm_rope_prefill_T32768", op="norm_rope", T=32768, H=64, Hk=1, d=128, rot=64, start=64, style=1,
             dtype="bf16", out="bf16", packed=True, far=0),
        # a small model's training batch in fp32, every channel rotated, an odd number of tokens
        dict(name="norm_rope_f32_T4099", op="norm_rope", T=4099, H=16, Hk=4, d=64, rot=64, start=0, style=0,
             dtype="f32", out="f32", packed=False, far=262144),
        # the gradients of one 16384-token chunk
        dict(name="norm_rope_grad_T16384", op="norm_rope_grad", T=16384, H=64, Hk=1, d=128, rot=64, start=64, style=1,
             dtype="bf16", out="bf16", packed=True, far=0),
        # the gradients of a short, ragged batch with shared key heads
        dict(name="norm_rope_grad_T1537", op="norm_rope_grad", T=1537, H=8, Hk=2, d=64, rot=48, start=0, style=0,
             dtype="f32", out="bf16", packed=False, far=4096),
        # one token of each of 16 sequences enters its cache
        dict(name="append_decode_B16", op="append", B=16, new=1, base=32768, H=64, Hk=1, d=128, page=64, rot=64,
             start=64, style=1, norm=True, pick=1),
        # chunks of a prefill of grouped-query heads, ragged over 5 sequences, some rows padding
        dict(name="append_chunks_B5", op="append", B=5, new=8192, base=3000, H=64, Hk=8, d=128, page=32, rot=128,
             start=0, style=0, norm=True, pick=2),
        # one short sequence, one token: latency alone
        dict(name="tree_one_token_L700", op="tree", B=1, nodes=1, longest=700, shortest=700, H=64, Hk=1, d=128,
             page=64, window=-1, pick=3),
        # ordinary decode of 16 long sequences, one token each: the cache's bytes
        dict(name="tree_decode_B16_L131072", op="tree", B=16, nodes=1, longest=131072, shortest=65536, H=64, Hk=1,
             d=128, page=64, window=-1, pick=4),
        # drafted trees of up to 16 tokens of 64 heads on one shared key head: tensor work
        dict(name="tree_draft16_B16_L32768", op="tree", B=16, nodes=16, longest=32768, shortest=16384, H=64, Hk=1,
             d=128, page=64, window=-1, pick=5),
        # grouped-query heads of 64 channels, ragged lengths and trees, small pages, a sliding window
        dict(name="tree_gqa_window_B24", op="tree", B=24, nodes=33, longest=8000, shortest=1, H=32, Hk=8, d=64,
             page=16, window=4096, pick=6),
        # a whole verification step of 8 sequences, 8 drafted tokens each
        dict(name="step_draft8_B8_L8192", op="step", B=8, nodes=8, longest=8192, shortest=1024, H=64, Hk=1, d=128,
             page=64, window=-1, rot=64, start=64, style=1, pick=7),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def _rotation(rng, d):
    rot = rng.choice([16, 32, 48, 64, d // 2, d])
    return dict(rot=rot, start=rng.choice([0, d - rot]), style=rng.randrange(2))


def draw(rng):
    op = rng.choice(["norm_rope", "norm_rope", "norm_rope_grad", "append", "tree", "tree", "tree", "step"])
    d = rng.choice([64, 128])
    if op in ("norm_rope", "norm_rope_grad"):
        H, Hk = rng.choice([(4, 1), (8, 2), (16, 1), (16, 4), (28, 4), (32, 8), (40, 8), (64, 1), (64, 8), (128, 1)])
        most = (32768 if op == "norm_rope" else 16384) * 65 * 128 // ((H + Hk) * d)
        dtype, out = rng.choice([("bf16", "bf16"), ("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16"), ("bf16", "f32")])
        most = min(most if dtype == out == "bf16" else most // 2, 65536)
        return dict(op=op, T=_spread(rng, 1, most), H=H, Hk=Hk, d=d, dtype=dtype, out=out, packed=rng.random() < 0.5,
                    far=rng.choice([0, 1000, 131072, 1048000]), **_rotation(rng, d))
    H, Hk = rng.choice([(4, 4), (8, 1), (16, 2), (16, 1), (28, 4), (32, 8), (32, 4), (40, 8), (64, 1), (64, 8), (128, 1)])
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        B = _spread(rng, 1, 32)
        return dict(op=op, B=B, new=_spread(rng, 1, min(8192, 5 * 8192 * 8 * 128 // (B * Hk * d))),
                    base=rng.randrange(0, 4096), H=H, Hk=Hk, d=d, page=page, norm=rng.random() < 0.7,
                    pick=rng.randrange(1 << 30), **_rotation(rng, d))
    B, nodes = _spread(rng, 1, 32), rng.choice([1, 1, 2, 5, 8, 16, 27, 48, 64])
    # at most the work of the largest listed cases: 16 sequences of 16 nodes x 64 heads over 24576 keys, or their bytes
    longest = min(131072, 16 * 16 * 64 * 24576 * 128 // (B * nodes * H * d), 16 * 98304 * 128 // (B * Hk * d))
    longest = _spread(rng, 64, max(64, longest // (4 if op == "step" else 1)))
    case = dict(op=op, B=B, nodes=nodes, longest=longest, shortest=rng.choice([1, max(1, longest // 2), longest]), H=H,
                Hk=Hk, d=d, page=page, window=rng.choice([-1, -1, 128, 1024, 4096]), pick=rng.randrange(1 << 30))
    if op == "step":
        case.update(_rotation(rng, d))
    return case


# ---------------------------------------------------------------- shapes that a case fixes without its seed


def _sequences(case):
    """Committed lengths, tree sizes and parents (-1: the last committed token) of a case's sequences."""
    r = random.Random(case["pick"])
    lens, trees = [], []
    for _ in range(case["B"]):
        lens.append(r.randint(case["shortest"], case["longest"]))
        n = case["nodes"] if case["nodes"] <= 2 else r.randint((case["nodes"] + 1) // 2, case["nodes"])
        trees.append([r.randint(max(-1, i - 6), i - 1) for i in range(n)])
    lens[0] = case["longest"]
    return lens, trees


def _appends(case):
    """Per sequence (first position, number of new tokens), and the padding rows behind each sequence's."""
    r = random.Random(case["pick"])
    return [(r.randint(0, case["base"]), case["new"] if case["new"] < 4 else r.randint(case["new"] // 2, case["new"]),
             0 if case["new"] < 4 else r.randint(0, 3)) for _ in range(case["B"])]


def _masks(parents):
    m = []
    for i, p in enumerate(parents):
        m.append((m[p] if p >= 0 else 0) | 1 << i)
    return m


def _depths(parents):
    dep = []
    for p in parents:
        dep.append(dep[p] + 1 if p >= 0 else 0)
    return dep


def work(case):
    d, H, Hk = case["d"], case["H"], case["Hk"]
    if case["op"] in ("norm_rope", "norm_rope_grad"):
        i, o = (2 if case[k] == "bf16" else 4 for k in ("dtype", "out"))
        n = case["T"] * (H + Hk) * d
        grad = case["op"] == "norm_rope_grad"
        return {"bytes": n * (2 * i + o if grad else i + o) + case["T"] * 8, "flops": n * (16 if grad else 8)}
    if case["op"] == "append":
        rows = sum(n for _, n, _ in _appends(case))
        return {"bytes": rows * (Hk * d * 8 + 20), "flops": rows * Hk * d * 8}
    lens, trees = _sequences(case)
    W = case["window"]
    nbytes = flops = 0
    for L, parents in zip(lens, trees):
        dep, mask = _depths(parents), _masks(parents)
        lo = max(0, L + min(dep) - W + 1) if W >= 0 else 0
        seen = sum(L - min(L, max(0, L + e - W + 1) if W >= 0 else 0) + bin(m).count("1") for e, m in zip(dep, mask))
        nbytes += (L - min(L, lo) + len(parents)) * Hk * d * 4 + len(parents) * (H * (d * 4 + 4) + 16)
        flops += 4 * H * d * seen
        if case["op"] == "step":
            nbytes += len(parents) * (H + 4 * Hk) * d * 2
    return {"bytes": nbytes, "flops": flops}


# ---------------------------------------------------------------- inputs


def _maker(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * int(seed) + 17)

    def normal(*shape, dtype=F32, std=1.0, mean=0.0):
        x = torch.randn(shape, generator=g, device="cuda", dtype=F32)
        return x.mul_(std).add_(mean).to(dtype)

    return g, normal


def _inv_freq(rot):
    return 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)


def _cache(case, lens, g, normal):
    """A paged cache whose sequences hold `lens` tokens each, in pages taken at random; -1 where a table has none."""
    page, B = case["page"], case["B"]
    need = [-(-n // page) for n in lens]
    order = torch.randperm(sum(need) + 3, generator=g, device="cuda")
    table = torch.full((B, max(need) + 1), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n].to(torch.int32)
        at += n
    shape = (sum(need) + 3, case["Hk"], page, case["d"])
    return normal(*shape, dtype=BF16), normal(*shape, dtype=BF16), table


def _workspace(s, name, *sizes):
    """The workspace that a program of the library keeps from call to call."""
    if own:
        import long_context_compressed_gated_b200 as csa
        need = getattr(csa.lib(), name + "_workspace_bytes")(*sizes) if name else 256
        s["ws"] = torch.zeros(need, dtype=torch.uint8, device="cuda")


def prepare(case, seed):
    g, normal = _maker(seed)
    s = {"case": case}
    d, H, Hk = case["d"], case["H"], case["Hk"]
    if "rot" in case:
        s["inv_freq"] = _inv_freq(case["rot"])
        s["wq"], s["wk"] = normal(d, std=0.2, mean=1.0), normal(d, std=0.2, mean=1.0)
    if case["op"] in ("norm_rope", "norm_rope_grad"):
        T, dt, ot = case["T"], TYPES[case["dtype"]], TYPES[case["out"]]
        if case["packed"]:  # one projection's output: queries, keys and values side by side
            x = normal(T, (H + 2 * Hk) * d, dtype=dt)
            s["q"], s["k"] = x[:, :H * d].view(T, H, d), x[:, H * d:(H + Hk) * d].view(T, Hk, d)
        else:
            s["q"], s["k"] = normal(T, H, d, dtype=dt), normal(T, Hk, d, dtype=dt)
        s["pos"] = torch.arange(T, device="cuda") + case["far"]
        if case["op"] == "norm_rope_grad":
            s["dyq"], s["dyk"] = normal(T, H, d, dtype=ot), normal(T, Hk, d, dtype=ot)
            _workspace(s, "csa_qk_norm_rope_backward", T, H, Hk, d)
        return s
    if case["op"] == "append":
        new = _appends(case)
        rows = sum(n + pad for _, n, pad in new)
        x = normal(rows, (H + 2 * Hk) * d, dtype=BF16)
        s["k"], s["v"] = x[:, H * d:(H + Hk) * d].view(rows, Hk, d), x[:, (H + Hk) * d:].view(rows, Hk, d)
        s["Kp"], s["Vp"], s["table"] = _cache(case, [p + n for p, n, _ in new], g, normal)
        pos, seq = [], []
        for b, (p, n, pad) in enumerate(new):
            pos.append(torch.arange(p, p + n))
            pos.append(torch.full((pad,), -1))
            seq.append(torch.full((n + pad,), b))
        s["pos"], s["seq"] = torch.cat(pos).cuda(), torch.cat(seq).to(torch.int32).cuda()
        _workspace(s, None)
        return s
    lens, trees = _sequences(case)
    R = sum(map(len, trees))
    s["lens"], s["trees"] = lens, trees
    s["Kp"], s["Vp"], s["table"] = _cache(case, [n + len(t) for n, t in zip(lens, trees)], g, normal)
    start = [0]
    for t in trees:
        start.append(start[-1] + len(t))
    s["seq_lens"] = torch.tensor(lens, dtype=torch.int32).cuda()
    s["q_start"] = torch.tensor(start, dtype=torch.int32).cuda()
    s["mask"] = torch.tensor([m - (1 << 64) if m >> 63 else m for t in trees for m in _masks(t)]).cuda()
    s["pos"] = torch.tensor([n + e for n, t in zip(lens, trees) for e in _depths(t)]).cuda()
    if case["op"] == "step":
        s["qkv"] = normal(R, (H + 2 * Hk) * d, dtype=BF16)
        s["slot"] = torch.tensor([n + i for n, t in zip(lens, trees) for i in range(len(t))]).cuda()
        s["seq"] = torch.tensor([b for b, t in enumerate(trees) for _ in t], dtype=torch.int32).cuda()
    else:
        s["q"] = normal(R, H, d, dtype=BF16)
    _workspace(s, "csa_tree_attn", case["B"], R, H, Hk, d, case["page"], s["table"].shape[1])
    return s


# ---------------------------------------------------------------- the plain forms (32 bits, rounded once)


def _angles(pos, inv_freq):
    """cos and sin of every position's angles [T, 1, rot/2], the angles in 64 bits."""
    a = pos.double()[:, None, None] * inv_freq.to(pos.device)
    return a.cos(), a.sin()


def _turn(x, cos, sin, start, rot, style):
    """Rotate channels start .. start + rot of x: pairs (i, i + rot/2) for style 0, (2i, 2i + 1) for style 1."""
    y = x.clone()
    r = x[..., start:start + rot]
    if style == 0:
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        y[..., start:start + rot // 2] = a * cos - b * sin
        y[..., start + rot // 2:start + rot] = b * cos + a * sin
    else:
        a, b = r[..., 0::2], r[..., 1::2]
        y[..., start:start + rot:2] = a * cos - b * sin
        y[..., start + 1:start + rot:2] = b * cos + a * sin
    return y


def _norm_rope(x, w, pos, s):
    c = s["case"]
    f = x.float()
    if w is not None:
        f = f * torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS) * w
    cos, sin = _angles(pos, s["inv_freq"])
    return _turn(f, cos.float(), sin.float(), c["start"], c["rot"], c["style"])


def _norm_rope_grad(x, w, dy, pos, s):
    c = s["case"]
    f, cos_sin = x.float(), _angles(pos, s["inv_freq"])
    g = _turn(dy.float(), cos_sin[0].float(), -cos_sin[1].float(), c["start"], c["rot"], c["style"])
    r = torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS)
    xh = f * r
    gw = g * w
    dx = r * (gw - xh * (gw * xh).mean(-1, keepdim=True))
    return dx.to(x.dtype), (g * xh).sum((0, 1))


def _store(Kp, Vp, table, seq, slot, k, v):
    page = Kp.shape[2]
    live = slot >= 0
    at = slot.clamp(min=0)
    p = table[seq.long(), at // page].long()[live]
    Kp[p, :, (at % page)[live]] = k[live]
    Vp[p, :, (at % page)[live]] = v[live]


def _tree(q, s):
    c = s["case"]
    H, Hk, d, W = c["H"], c["Hk"], c["d"], c["window"]
    G, scale = H // Hk, 1.0 / math.sqrt(c["d"])
    O = torch.empty_like(q)
    lse = torch.empty(q.shape[:2], dtype=F32, device=q.device)
    r0 = 0
    for b, (L, parents) in enumerate(zip(s["lens"], s["trees"])):
        n = len(parents)
        S = L + n
        pages = s["table"][b, :-(-S // c["page"])].long()
        K = s["Kp"][pages].transpose(0, 1).reshape(Hk, -1, d)[:, :S].float()
        V = s["Vp"][pages].transpose(0, 1).reshape(Hk, -1, d)[:, :S].float()
        x = q[r0:r0 + n].view(n, Hk, G, d).transpose(0, 1).reshape(Hk, n * G, d).float()
        z = torch.matmul(x, K.transpose(1, 2)).mul_(scale).view(Hk, n, G, S)
        key = torch.arange(S, device=q.device)
        bits = s["mask"][r0:r0 + n, None] >> (key[L:] - L) & 1
        if W >= 0:
            hide = key[:L] <= s["pos"][r0:r0 + n, None] - W
            z[..., :L].masked_fill_(hide[:, None], -math.inf)
        z[..., L:].masked_fill_((bits == 0)[:, None], -math.inf)
        m = z.amax(-1, keepdim=True)
        p = z.sub_(m).exp_()
        l = p.sum(-1, keepdim=True)
        o = torch.matmul(p.view(Hk, n * G, S), V).view(Hk, n, G, d) / l
        O[r0:r0 + n] = o.transpose(0, 1).reshape(n, H, d).to(q.dtype)
        lse[r0:r0 + n] = (m + l.log())[..., 0].transpose(0, 1).reshape(n, H)
        r0 += n
    return O, lse


def _plain(s):
    c = s["case"]
    if c["op"] == "norm_rope":
        ot = TYPES[c["out"]]
        return _norm_rope(s["q"], s["wq"], s["pos"], s).to(ot), _norm_rope(s["k"], s["wk"], s["pos"], s).to(ot)
    if c["op"] == "norm_rope_grad":
        dq, dwq = _norm_rope_grad(s["q"], s["wq"], s["dyq"], s["pos"], s)
        dk, dwk = _norm_rope_grad(s["k"], s["wk"], s["dyk"], s["pos"], s)
        return dq, dk, dwq, dwk
    if c["op"] == "append":
        k = _norm_rope(s["k"], s["wk"] if c["norm"] else None, s["pos"], s).to(BF16)
        _store(s["Kp"], s["Vp"], s["table"], s["seq"], s["pos"], k, s["v"])
        return s["Kp"], s["Vp"]
    if c["op"] == "tree":
        return _tree(s["q"], s)
    H, Hk, d = c["H"], c["Hk"], c["d"]
    x = s["qkv"].view(-1, H + 2 * Hk, d)
    q = _norm_rope(x[:, :H], s["wq"], s["pos"], s).to(BF16)
    k = _norm_rope(x[:, H:H + Hk], s["wk"], s["pos"], s).to(BF16)
    _store(s["Kp"], s["Vp"], s["table"], s["seq"], s["slot"], k, x[:, H + Hk:])
    return _tree(q, s)[0], s["Kp"], s["Vp"]


def run(s):
    if not own:
        return _plain(s)
    import long_context_compressed_gated_b200 as csa
    c = s["case"]
    rope = dict(rot_start=c.get("start", 0), rot_style=c.get("style", 0), eps=EPS)
    if c["op"] == "norm_rope":
        return csa.csa_qk_norm_rope(s["q"], s["k"], s["inv_freq"], wq=s["wq"], wk=s["wk"], pos=s["pos"],
                                    out_dtype=TYPES[c["out"]], **rope)
    if c["op"] == "norm_rope_grad":
        return csa.csa_qk_norm_rope_backward(s["q"], s["k"], s["dyq"], s["dyk"], s["inv_freq"], wq=s["wq"],
                                             wk=s["wk"], pos=s["pos"], workspace=s["ws"], **rope)[:4]
    if c["op"] == "append":
        csa.csa_paged_append(s["k"], s["v"], s["Kp"], s["Vp"], s["table"], s["seq"], s["pos"], s["inv_freq"],
                             wk=s["wk"] if c["norm"] else None, workspace=s["ws"], **rope)
        return s["Kp"], s["Vp"]
    scale = 1.0 / math.sqrt(c["d"])
    if c["op"] == "tree":
        return csa.csa_tree_attn(s["q"], s["Kp"], s["Vp"], s["table"], s["seq_lens"], s["q_start"], s["mask"], scale,
                                 W=c["window"], pos=s["pos"], workspace=s["ws"])[:2]
    from long_context_compressed_gated_b200.speculative import tree_verify_step
    O = tree_verify_step(s["qkv"], c["H"], c["Hk"], s["Kp"], s["Vp"], s["table"], s["seq_lens"], s["q_start"],
                         s["mask"], s["seq"], s["slot"], s["pos"], s["inv_freq"], scale, wq=s["wq"], wk=s["wk"],
                         W=c["window"], workspace=s["ws"], **rope)
    return O, s["Kp"], s["Vp"]


# ---------------------------------------------------------------- the definitions in 64 bits


def _exact_rotation(pos, s):
    """Per token the d x d matrix of its rotation (the identity on channels that do not turn)."""
    c = s["case"]
    d, rot, start = c["d"], c["rot"], c["start"]
    ang = pos.double()[:, None] * s["inv_freq"].cuda()[None]
    i = torch.arange(rot // 2, device="cuda")
    a, b = (start + i, start + i + rot // 2) if c["style"] == 0 else (start + 2 * i, start + 2 * i + 1)
    M = torch.eye(d, dtype=torch.float64, device="cuda").repeat(len(pos), 1, 1)
    M[:, a, a], M[:, b, b] = torch.cos(ang), torch.cos(ang)
    M[:, a, b], M[:, b, a] = -torch.sin(ang), torch.sin(ang)
    return M


def _exact_norm_rope(x, w, pos, s):
    out = []
    for t in range(0, x.shape[0], 2048):
        f = x[t:t + 2048].double()
        if w is not None:
            f = f / (f.square().sum(-1, keepdim=True) / f.shape[-1] + EPS).sqrt() * w.double()
        out.append(torch.einsum("tij,thj->thi", _exact_rotation(pos[t:t + 2048], s), f))
    return torch.cat(out)


def _exact_grad(x, w, dy, pos, s):
    dxs, dw = [], 0
    for t in range(0, x.shape[0], 2048):
        f, W = x[t:t + 2048].double(), w.double()
        ms = f.square().sum(-1, keepdim=True) / f.shape[-1] + EPS
        g = torch.einsum("tij,thi->thj", _exact_rotation(pos[t:t + 2048], s), dy[t:t + 2048].double())
        dw = dw + torch.einsum("thi,thi->i", g, f / ms.sqrt())
        along = (g * W * f).sum(-1, keepdim=True)
        dxs.append(g * W / ms.sqrt() - f * along / (f.shape[-1] * ms ** 1.5))
    return torch.cat(dxs), dw


def _exact_store(s, k, v, seq, slot):
    """The two caches after the tokens' rows, one by one where the tables put them."""
    page = s["Kp"].shape[2]
    table = s["table"].cpu()
    Kp, Vp = s["Kp"].double(), s["Vp"].double()
    rows = [(t, int(table[b, p // page]), p % page) for t, (b, p) in enumerate(zip(seq.tolist(), slot.tolist())) if p >= 0]
    t, p, o = (torch.tensor(x, device="cuda") for x in zip(*rows))
    Kp.permute(0, 2, 1, 3)[p, o] = k[t].double()
    Vp.permute(0, 2, 1, 3)[p, o] = v[t].double()
    return Kp, Vp


def _exact_tree(q, Kp, Vp, s):
    c = s["case"]
    H, Hk, d, page, W = c["H"], c["Hk"], c["d"], c["page"], c["window"]
    O, lse = [], []
    r = 0
    for b, (L, parents) in enumerate(zip(s["lens"], s["trees"])):
        S = L + len(parents)
        where = torch.arange(S, device="cuda")
        p, o = s["table"][b].long()[where // page], where % page
        K, V = Kp[p, :, o].double(), Vp[p, :, o].double()  # [S, Hk, d]
        for mask, depth in zip(_masks(parents), _depths(parents)):
            lo = max(0, L + depth - W + 1) if W >= 0 else 0
            mine = torch.tensor([L + j for j in range(len(parents)) if mask >> j & 1], device="cuda")
            at = torch.cat([torch.arange(min(lo, L), L, device="cuda"), mine])
            x = q[r].double().view(Hk, H // Hk, d)
            logit = torch.einsum("hgd,khd->hgk", x, K[at]) / math.sqrt(d)
            total = torch.logsumexp(logit, -1)
            O.append(torch.einsum("hgk,khd->hgd", (logit - total[..., None]).exp(), V[at]).reshape(H, d))
            lse.append(total.reshape(H))
            r += 1
    return torch.stack(O), torch.stack(lse)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm_rope":
        return _exact_norm_rope(s["q"], s["wq"], s["pos"], s), _exact_norm_rope(s["k"], s["wk"], s["pos"], s)
    if case["op"] == "norm_rope_grad":
        (dq, dwq), (dk, dwk) = (_exact_grad(s[x], s["w" + x], s["dy" + x], s["pos"], s) for x in "qk")
        return dq, dk, dwq, dwk
    if case["op"] == "append":
        k = _exact_norm_rope(s["k"], s["wk"] if case["norm"] else None, s["pos"], s)
        return _exact_store(s, k, s["v"], s["seq"], s["pos"])
    if case["op"] == "tree":
        return _exact_tree(s["q"], s["Kp"], s["Vp"], s)
    H, Hk = case["H"], case["Hk"]
    x = s["qkv"].view(-1, H + 2 * Hk, case["d"])
    q = _exact_norm_rope(x[:, :H], s["wq"], s["pos"], s).to(BF16)  # the queries and the cache are held in bf16
    k = _exact_norm_rope(x[:, H:H + Hk], s["wk"], s["pos"], s)
    Kp, Vp = _exact_store(s, k, x[:, H + Hk:], s["seq"], s["slot"])
    return _exact_tree(q, Kp.to(BF16), Vp.to(BF16), s)[0], Kp, Vp
