"""MXFP4 weights (OCP microscaling: e2m1 codes, one e8m0 scale for 32 neighbours
of a row) by their definition, on the CPU."""
import torch

VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def quantise(w):
    """codes [.., C/2] (the even column's in the low half) and scale bytes [.., C/32] of the nearest values."""
    *lead, C = w.shape
    v = w.double().view(*lead, C // 32, 32)
    top = torch.frexp(v.abs().amax(-1, keepdim=True).clamp_min(1e-30)).exponent - 3
    u = torch.ldexp(v, -top)
    near = (u.abs()[..., None] - torch.tensor(VALUES, dtype=torch.float64)).abs().argmin(-1)
    code = (near + 8 * (u < 0)).to(torch.uint8).view(*lead, C // 2, 2)
    return code[..., 0] | code[..., 1] << 4, (top[..., 0] + 127).to(torch.uint8)


def values(codes, sf):
    """float64 values."""
    table = torch.tensor(VALUES + tuple(-v for v in VALUES), dtype=torch.float64)
    v = torch.stack([table[(codes & 15).long()], table[(codes >> 4).long()]], -1).flatten(-2)
    scale = torch.ldexp(torch.ones_like(sf, dtype=torch.float64), sf.int() - 127)
    return v * torch.where(sf == 255, torch.full_like(scale, float("nan")), scale).repeat_interleave(32, -1)
