"""How far a sum over many rows may be off, by the number of additions that one term goes through."""
import torch

from tests import feature_ref as ref


def weight_grad_roundings(rows: int) -> int:
    """Roundings of a term of the norm's weight gradient: its two products; the rows of one thread (the
    rows in at least min(rows, 1024) parts); six doublings over a wave, three over its workgroup; 32 slices of
    at most 32 parts, and the slices."""
    return 2 + -(-rows // 1024) + 6 + 3 + 32 + 31


def weight_grad_bound(terms_abs_sum: torch.Tensor, rows: int) -> torch.Tensor:
    return terms_abs_sum * weight_grad_roundings(rows) * ref.U32 * (1 + 2.0 ** -10)
