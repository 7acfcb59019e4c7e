"""One verification step of drafted tokens over a paged raw K/V cache, the serving
loop's call between two projections: queries normed and positioned, keys and
values into the cache, attention of every drafted token over its sequence and its
ancestors (with one token a sequence: an ordinary decode step).

Only argument plumbing happens here: every step runs in libcsa."""
import torch

from . import ROPE_HALVES, csa_paged_append, csa_qk_norm_rope, csa_tree_attn, lib


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
    zeroed; pass one to read the status, which both kernels report to.  Returns
    O [R, H, d]; lse [R, H] f32 receives the log-sum-exps when given."""
    d = Kpages.shape[3]
    q, k, v = qkv.view(qkv.shape[0], H + 2 * Hk, d).split((H, Hk, Hk), 1)
    if workspace is None:
        B, max_pages = block_table.shape
        n = lib().csa_tree_attn_workspace_bytes(B, q.shape[0], H, Hk, d, Kpages.shape[2], max_pages)
        workspace = torch.empty(n, dtype=torch.uint8, device=qkv.device)
        workspace[:4].zero_()
    rope = dict(eps=eps, rot_start=rot_start, rot_style=rot_style)
    q, _ = csa_qk_norm_rope(q, None, inv_freq, wq=wq, pos=pos, **rope)
    csa_paged_append(k, v, Kpages, Vpages, block_table, seq, pos, inv_freq, slot=slot, wk=wk, workspace=workspace,
                     **rope)
    return csa_tree_attn(q, Kpages, Vpages, block_table, seq_lens, q_start, mask, scale, W=W, pos=pos, O=O, lse=lse,
                         want_lse=lse is not None, workspace=workspace, out_dtype=out_dtype)[0]
