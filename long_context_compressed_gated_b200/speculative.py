"""One verification step of drafted tokens over a paged raw K/V cache, the serving
loop's call between two projections: queries normed and positioned, keys and
values into the cache, attention of every drafted token over its sequence and its
ancestors (with one token a sequence: an ordinary decode step).

Only argument plumbing happens here: every step runs in libcsa.  The arguments are
checked once and the three calls made with addresses into the packed projection
(a step of 8 sequences spends 35 us on the host so, 49 through the three functions
of the binding)."""
import torch

from . import (_ODTYPE, ROPE_HALVES, _check, _dense, _device, _freq, _given, _paged, _ptr, _scratch, _stream, _vector,
               lib)


def tree_verify_step(qkv, H, Hk, Kpages, Vpages, block_table, seq_lens, q_start, mask, seq, slot, pos, inv_freq, scale,
                     wq=None, wk=None, eps=1e-6, rot_start=0, rot_style=ROPE_HALVES, W=-1, O=None, lse=None,
                     workspace=None, out_dtype=torch.bfloat16):
    """qkv [R, (H + 2 Hk) * d] bf16: the projections' output for the R drafted rows,
    queries, keys and values side by side.  seq [R] int32, slot and pos [R] int64:
    a row's sequence, its cache row (seq_lens[b] + its node number; negative:
    padding) and its position (seq_lens[b] + its depth).  The caches are updated in
    place; a later step commits the accepted rows by moving seq_lens (a chain's
    first rows stay where they are; rows of another branch are appended again to
    their final slots).  workspace: csa_tree_attn_workspace_bytes(), its status word
    zeroed; pass one to read the status, which both kernels report to (without one a
    number outside its table goes unseen).  Returns O [R, H, d]; lse [R, H] f32
    receives the log-sum-exps when given.  An argument that only the attention
    refuses raises after the rows have been appended: repeating the step is safe."""
    dev = _device(qkv, "qkv")
    n_pages, cached, page, d = _paged(Kpages, Vpages, dev)
    if qkv.dtype != torch.bfloat16:
        raise TypeError("qkv must be %s, got %s" % (torch.bfloat16, qkv.dtype))
    if cached != Hk or qkv.dim() != 2 or qkv.shape[1] != (H + 2 * Hk) * d or qkv.stride(1) != 1:
        raise ValueError("qkv must be [R, %d] with dense rows, the cache's key heads %d" % ((H + 2 * Hk) * d, Hk))
    R, row = qkv.shape[0], qkv.stride(0) if qkv.shape[0] > 1 else qkv.shape[1]
    B, max_pages = _dense(block_table, torch.int32, 2, "block_table", dev)
    if pos is None or slot is None:  # (siblings share a position: it cannot stand in for their rows)
        raise ValueError("pos and slot must be given")
    pp, slots = _vector(pos, R, torch.int64, "pos", dev), _vector(slot, R, torch.int64, "slot", dev)
    seqs, masks = _vector(seq, R, torch.int32, "seq", dev), _vector(mask, R, torch.int64, "mask", dev)
    lens = _vector(seq_lens, B, torch.int32, "seq_lens", dev)
    starts = _vector(q_start, B + 1, torch.int32, "q_start", dev)
    wqp, wkp = _vector(wq, d, torch.float32, "wq", dev), _vector(wk, d, torch.float32, "wk", dev)
    fp, rot = _freq(inv_freq)
    if out_dtype not in _ODTYPE:
        raise TypeError("out_dtype must be torch.bfloat16 or torch.float32")
    q = qkv.new_empty((R, H, d))
    O = qkv.new_empty((R, H, d), dtype=out_dtype) if O is None else _given(O, out_dtype, (R, H, d), "O", dev)
    if lse is not None:
        _given(lse, torch.float32, (R, H), "lse", dev)
    L = lib()
    ws = _scratch(workspace, dev, lambda: L.csa_tree_attn_workspace_bytes(B, R, H, Hk, d, page, max_pages))
    at, qp, wp, stream = qkv.data_ptr(), q.data_ptr(), ws.data_ptr(), _stream(dev)
    k, v = (at + 2 * H * d, at + 2 * (H + Hk) * d) if R else (None, None)
    Kp, Vp, table, bf16 = Kpages.data_ptr(), Vpages.data_ptr(), block_table.data_ptr(), _ODTYPE[torch.bfloat16]
    _check(L.csa_qk_norm_rope(at, row, None, 0, wqp, None, eps, pp, 0, fp, rot_start, rot, rot_style, R, H, 0, d, bf16,
                              qp, None, bf16, stream), "csa_qk_norm_rope")
    _check(L.csa_paged_append(k, row, v, row, wkp, eps, pp, slots, seqs, fp, rot_start, rot, rot_style, table, R, Hk,
                              d, B, max_pages, n_pages, page, Kp, Vp, wp, ws.numel(), stream), "csa_paged_append")
    _check(L.csa_tree_attn(qp, Kp, Vp, table, lens, starts, masks, pp, R, B, H, Hk, d, page, n_pages, max_pages, W,
                           scale, O.data_ptr(), _ODTYPE[out_dtype], _ptr(lse), wp, ws.numel(), stream),
           "csa_tree_attn")
    return O
