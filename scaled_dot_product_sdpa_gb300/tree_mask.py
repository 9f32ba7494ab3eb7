"""Masks of drafted token trees, as attn_decode_tree takes them."""
from __future__ import annotations

import torch


def attn_tree_mask(parents) -> tuple[torch.Tensor, torch.Tensor]:
    """The mask and the depths of drafted tokens whose parents are given: parents[..., t] < t is the token that t follows, -1
    for one that follows the older tokens directly.  A token sees itself and all that it follows.  Returns int32 words
    [..., T, (T + 31) // 32] (bit j % 32 of word j // 32 of row t: whether t sees j) and int32 depths [..., T] (0 without a parent):
    a token's rotary position is that of the first new token plus its depth.  On the device of `parents` (a tensor, or
    nested lists: the CPU).  The check of the parents reads one result back, and the rest is a loop over T in Python: on a GPU it waits for that and
    cannot be captured.  A tree of fixed shape needs it once; one that is chosen anew each step gets its masks outside the captured part."""
    parents = torch.as_tensor(parents)
    if parents.dim() < 1 or parents.shape[-1] < 1 or parents.dtype.is_floating_point or parents.dtype == torch.bool:
        raise ValueError("gbattn: parents must be whole numbers [..., T], T > 0")
    T = parents.shape[-1]
    p = parents.long()
    if bool(((p < -1) | (p >= torch.arange(T, device=p.device))).any()):
        raise ValueError("gbattn: a token's parent must be an earlier token, or -1")
    seen = torch.zeros(*p.shape, T, dtype=torch.bool, device=p.device)
    for t in range(T):  # a token sees what its parent sees, and itself
        up = p[..., t].clamp(min=0)[..., None, None].expand(*p.shape[:-1], 1, T)
        seen[..., t, :] = torch.gather(seen, -2, up)[..., 0, :] & (p[..., t] >= 0)[..., None]
        seen[..., t, t] = True
    depths = (seen.sum(-1) - 1).to(torch.int32)
    bits = torch.nn.functional.pad(seen.long(), (0, -T % 32)).unflatten(-1, (-1, 32))
    words = (bits << torch.arange(32, device=p.device)).sum(-1)
    return torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32), depths
