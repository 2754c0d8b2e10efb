"""64-bit references of the batched products and the 8-bit checkpoints.

The matrices come from the CPU oracle's decoder; products and activations are
torch float64 on the device the inputs are on."""
import math

import numpy as np
import torch

from oracle import oracle_decode, oracle_mad_codebook
from trellis_coded_weight_tcq_b200 import tcq


def random_matrix(rng, L, k, T, rows, cols, code, scaled, device, small_scales=False):
    """(arguments of tcq.gemm up to cols, W in float64 on the device)."""
    nb = rows * (cols // T)
    W = tcq.tcq_words_per_block(k, T)
    bits = rng.integers(0, 2**32, size=(nb, W), dtype=np.uint64).astype(np.uint32)
    used = T * k - 32 * (W - 1)
    if used < 32:
        bits[:, -1] &= np.uint32(((1 << used) - 1) << (32 - used))
    start = rng.integers(0, 2**32, size=nb, dtype=np.uint64).astype(np.uint32)
    if code == "mad":
        table, book = oracle_mad_codebook(L).astype(np.float32), tcq.MAD
    else:
        table = rng.standard_normal(1 << L).astype(np.float16 if code == "f16" else np.float32)
        book = torch.from_numpy(table).to(device)
    values = oracle_decode(bits, start, table, L, k, T).reshape(rows, cols)
    scale = None
    if scaled:
        scale = rng.lognormal(-4.0, 0.5, nb).astype(np.float32)
        if small_scales:
            scale *= np.float32(2.0**-60)
        values = values * np.repeat(scale.astype(np.float64).reshape(rows, -1), T, axis=1)
        scale = torch.from_numpy(scale).to(device)
    args = (torch.from_numpy(bits.view(np.int32)).to(device), torch.from_numpy(start.view(np.int32)).to(device),
            scale, book, L, k, T, rows, cols)
    return args, torch.from_numpy(values).to(device)


def weight_half_step(n, dtype, exact):
    """Half a step of the weights' rounding: to bfloat16 (2^-8) for more than 256 tokens of
    that type, else to binary16 (2^-11), 0 where binary16 holds them."""
    if dtype == torch.bfloat16 and n > 256:
        return 2.0**-8
    return 0.0 if exact else 2.0**-11


def product_bound(a, b, half):
    """Bound of |computed - exact| for a @ b.T summed by the tensor cores.

    A 16-deep MMA adds its products and the running sum in fp32 with a few roundings
    or truncations: 2^-22 of the sum of magnitudes per MMA is allowed.  ``half``: the
    weights were rounded, each term off by at most this half step, independently: 8
    standard deviations' worth by Hoeffding's bound (a chance of 3e-14 per element), and
    binary16 subnormals by 2^-25 of an operand's unit (the operands are scaled to below 1
    and 2^15).  A scaled row of ``a`` is within 2^-39 of its largest."""
    mags = a.abs() @ b.abs().T
    bound = (a.shape[1] / 16 + 2) * 2.0**-22 * mags
    if half:
        bound = bound + 8 * half * ((a * a) @ (b * b).T).sqrt()
        bound = bound + 2.0**-24 * a.abs().sum(1, keepdim=True) * b.abs().amax(1)[None, :]
    return bound + 2.0**-39 * a.abs().amax(1, keepdim=True) * b.abs().sum(1)[None, :]


def act(z, name):
    if name == "relu":
        return torch.relu(z)
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z / math.sqrt(2)))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z**3)))
    return z


def act_slope(z, name):
    if name == "none":
        return torch.ones_like(z)
    z = z.detach().clone().requires_grad_()
    return torch.autograd.grad(act(z, name).sum(), z)[0]


def act_error(z):
    """fp32 evaluation of an activation or its slope at z, relative to 1 + |z|: the
    exponential is within (2 + 1.2 |t|) units in the last place and |t| <= 2 |z| (1 +
    z^2 / 20) there; below e^-20 its error no longer counts.  Some ten more roundings."""
    t = (2 * z.abs() * (1 + z * z / 20)).clamp_max(20)
    return (16 + 2 * t) * 2.0**-23


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def quantised(x, fmt):
    """(codes as integers or values, exponent bytes, values) of numpy float64 rows [n, cols]."""
    n, cols = x.shape
    groups = -(-cols // 32)
    padded = np.zeros((n, groups * 32))
    padded[:, :cols] = x
    padded = padded.reshape(n, groups, 32)
    most = 127.0 if fmt == "int8" else 448.0
    finite = np.isfinite(padded).all(2)
    amax = np.abs(np.where(finite[:, :, None], padded, 0)).max(2)
    byte = np.zeros((n, groups), dtype=np.int64)
    for b in range(255):  # the least byte whose scale holds the group
        byte[amax > most * 2.0**(b - 127)] = b + 1
    scale = np.exp2(byte.astype(np.float64) - 127)
    y = np.where(finite[:, :, None], padded / scale[:, :, None], 0)
    if fmt == "int8":
        codes = np.rint(y)
    else:
        step = np.exp2(np.floor(np.log2(np.maximum(np.abs(y), 2.0**-6))) - 3)
        codes = np.rint(y / step) * step
    values = codes * scale[:, :, None]
    values[~finite] = np.nan
    byte[~finite] = 255
    return (codes.reshape(n, -1)[:, :cols], byte.astype(np.uint8), values.reshape(n, -1)[:, :cols])


def packed_values(packed):
    """float64 values of a Packed8, from its bytes."""
    codes = packed.codes.view(torch.int8)
    if packed.format == "int8":
        v = codes.double()
    else:
        b = codes.view(torch.uint8).long()
        power, frac = (b >> 3) & 15, (b & 7).double()
        v = (1 - 2 * (b >> 7)) * torch.where(power > 0, (1 + frac / 8) * torch.exp2(power.double() - 7), frac / 512)
    s = torch.where(packed.scales == 255, torch.full_like(packed.scales, 0).double() * math.nan,
                    torch.exp2(packed.scales.double() - 127))
    return v * s.repeat_interleave(32, 1)[:, :codes.shape[1]]
