"""Window attention's fp32 scores as the kernels make them, in 64 bits but for the
operands: each in two tf32 parts, three products of four."""
import torch


def tf32(x):
    """The nearest number of 11 significant bits, as float64."""
    m, e = torch.frexp(x)
    return torch.ldexp(torch.floor(m.abs() * 2048 + 0.5) / 2048 * m.sign(), e)


def parts(x):
    x = x.double()
    hi = tf32(x)
    return hi, tf32(x - hi)


def scores(q, k, lost=None):
    """q [T, Hq, d], k [T, Hk, d] fp32 -> [Hq, T, T]; ``lost``: "lo hi" or "hi lo", a product left out."""
    k = k.repeat_interleave(q.shape[1] // k.shape[1], 1)
    (qh, ql), (kh, kl) = parts(q), parts(k)
    s = torch.einsum("ihd,jhd->hij", qh, kh)
    if lost != "lo hi":
        s = s + torch.einsum("ihd,jhd->hij", ql, kh)
    if lost != "hi lo":
        s = s + torch.einsum("ihd,jhd->hij", qh, kl)
    return s


def bound(q, k, scale):
    """How far a score, and so a weight relative to itself, may be off. With parts of 11 bits
    an operand keeps 22 bits, and the product of the small parts is left out: 3 x 2^-22 |q_c k_c|
    at most for a channel; the sums' roundings of 2^-24 a step come on top. Channels' errors
    are independent, so that a quarter of the sum of their bounds is not reached: 2^-22 |q| |k|
    scale, and 1e-6 for what else is rounded."""
    return 1e-6 + 2.0 ** -22 * float(q.double().norm(dim=-1).max() * k.double().norm(dim=-1).max()) * scale


CASES = [(1.5, 128, None), (8.0, 128, None), (8.0, 64, None), (40.0, 128, 0.25), (40.0, 128, 1.0), (40.0, 64, 1.0)]  # sharp, d, scale
