"""Plain 64-bit forms of the 16/32-bit operators, for the tests: the checkpoint's definition,
the activations and their slopes, and the bounds their rounding steps give."""
import math

import torch

FMAX = {0: 448.0, 1: 57344.0}
F8 = {0: torch.float8_e4m3fn, 1: torch.float8_e5m2}
HALF_CODE = {0: 2.0 ** -4, 1: 2.0 ** -3}    # a code's rounding, relative
TINY_CODE = {0: 2.0 ** -10, 1: 2.0 ** -17}  # half the least subnormal code
U = 2.0 ** -24                              # half a step of fp32, relative


def half(dtype):
    """Half a step of a type, relative to the value."""
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    """Half the least subnormal of a type."""
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


def blocks(v):
    """[rows, cols] -> [rows, blocks, 32], zeros after the last column."""
    rows, cols = v.shape
    out = torch.zeros(rows, (cols + 31) // 32 * 32, dtype=v.dtype, device=v.device)
    out[:, :cols] = v
    return out.view(rows, -1, 32)


def scale_bytes(v, fmt):
    """The scale byte of each block: the least b >= 0 with max|v| <= FMAX 2^(b - 127); 255 if not finite."""
    b = blocks(v.double())
    top = b.abs().amax(2)
    bad = ~torch.isfinite(b).all(2)
    byte = torch.zeros_like(top)
    for k in range(256):  # by trying: the least one that fits
        byte += ((top > FMAX[fmt] * 2.0 ** (k - 127)) & ~bad).double()
    byte[bad] = 255
    return byte.to(torch.uint8)


def decode(codes, scales, fmt):
    """fp64 values of a checkpoint."""
    cols = codes.shape[1]
    v = codes.view(F8[fmt]).double()
    s = torch.exp2(scales[:, : (cols + 31) // 32].double() - 127)
    s[scales[:, : (cols + 31) // 32] == 255] = math.nan
    return v * s.repeat_interleave(32, dim=1)[:, :cols]


def act(z, name):
    if name == "gelu":  # z (1 + tanh(w)) / 2 = z sigmoid(2w): the sum would cancel for w below -18 even in 64 bits
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    return {"none": z, "relu": z.clamp_min(0), "silu": z * torch.sigmoid(z)}[name]


def slope(z, name):
    if name == "gelu":
        k = 2 * math.sqrt(2 / math.pi)
        w = k * (z + 0.044715 * z ** 3)
        s = torch.sigmoid(w)
        return s + z * s * torch.sigmoid(-w) * k * (1 + 3 * 0.044715 * z * z)
    s = torch.sigmoid(z)
    return {"none": torch.ones_like(z), "relu": (z > 0).double(), "silu": s * (1 + z * (1 - s))}[name]


def assert_within(got, want, tol, what):
    """Elementwise |got - want| <= tol; says where and by how much it is not."""
    err = (got.double() - want).abs()
    bad = ~(err <= tol)
    if bad.any():
        i = int(torch.argmax(torch.where(torch.isnan(err), torch.full_like(err, math.inf), err - tol)))
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside; at {i}: got {got.reshape(-1)[i].item()}, "
                             f"want {want.reshape(-1)[i].item()}, tolerance {torch.as_tensor(tol).expand_as(err).reshape(-1)[i].item()}")
