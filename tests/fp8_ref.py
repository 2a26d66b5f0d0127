"""The 8-bit operators' definition in 64 bits, and how far one rounding can be off (tests only)."""
import torch

TOP = 448.0
TINY = TOP * 2.0 ** -126
E4M3 = torch.float8_e4m3fn


def half_step(q: torch.Tensor) -> torch.Tensor:
    """Half the distance of neighbouring e4m3 numbers around |q|: 2^(exponent - 4), and 2^-10
    below the smallest normal number 2^-6."""
    return torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 4)


def group_amax(x: torch.Tensor, block: int) -> torch.Tensor:
    rows, cols = x.shape
    g, r = -(-cols // 128), -(-rows // block)
    p = torch.zeros(r * block, g * 128, dtype=torch.float64, device=x.device)
    p[:rows, :cols] = x.abs()
    return p.view(r, block, g, 128).amax(dim=(1, 3)).clamp(min=TINY)


def spread(s: torch.Tensor, rows: int, cols: int, block: int) -> torch.Tensor:
    """One value per group [row blocks, groups] as one per element."""
    return s.repeat_interleave(128, 1)[:, :cols].repeat_interleave(block, 0)[:rows]


def values(codes: torch.Tensor, scales: torch.Tensor, block: int) -> torch.Tensor:
    """What codes and scales (group-major for block 1) stand for."""
    s = scales.double().t() if block == 1 else scales.double()
    return codes.double() * spread(s, codes.shape[0], codes.shape[1], block)


def check_quantised(codes, scales, x64, block, err=None, rel=2.0 ** -21):
    """codes, scales are a quantisation of x64, whose fp32 computation may be off by ``err`` (absolute,
    per element) and ``rel`` (relative; the two quotients and the product of a plain quantisation
    are three fp32 roundings, 3 * 2^-24 < 2^-21)."""
    rows, cols = x64.shape
    err = torch.zeros_like(x64) if err is None else err
    a = group_amax(x64, block)
    a_err = torch.zeros_like(a) + group_amax(err, block) * (group_amax(err, block) > TINY)
    s = scales.double().t() if block == 1 else scales.double()
    assert s.shape == a.shape
    assert torch.all((s - a / TOP).abs() <= a / TOP * rel + a_err / TOP), float(((s - a / TOP).abs() / (a / TOP)).max())
    sp = spread(s, rows, cols, block)
    # the value is half a step off at most, the step taken where the computed value may lie
    q = x64.abs() / sp * (1 + rel) + err / sp
    tol = half_step(q) * sp + err + x64.abs() * rel
    # the largest magnitude itself may be clamped from just above 448
    bad = (values(codes, scales, block) - x64).abs() > tol
    assert not bool(bad.any()), (int(bad.sum()), torch.nonzero(bad)[:4].tolist())


def silu64(x):
    return x / (1 + torch.exp(-x))


def product(a, sa, b, sb):
    """(A B^T, sum of the magnitudes of its terms) in 64 bits."""
    va, vb = values(a, sa, 1), values(b, sb, 128)
    return va @ vb.t(), va.abs() @ vb.abs().t()


def product_error(terms: torch.Tensor, k: int) -> torch.Tensor:
    """Bound of an fp32 product's error from the sum of its terms' magnitudes: a group's 128
    products are exact in fp32 and summed by at most 128 additions that may truncate (2^-23 each),
    the scales' product and its multiplication round once each, and each of the ceil(k / 128)
    groups is added with one rounding (2^-24 each)."""
    return terms * ((2 * 128 + 2 + -(-k // 128)) * 2.0 ** -24)
