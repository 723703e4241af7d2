"""Tolerances and inputs shared by the tests of the norm, the e4m3 blocks and the grouped products."""
import numpy as np
import torch

from oracle import nf4
from quantized_lora_fine_b200 import synth

U_BF16, U_F32 = 2.0 ** -8, 2.0 ** -24     # largest relative rounding error, half a step


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().double().numpy()


def normal(shape, seed, std=1.0, index=0) -> torch.Tensor:
    return synth.normal_bf16(shape, std, seed, synth.STREAM_X, index)


def outliers(shape, seed) -> torch.Tensor:
    """Normal rows with some channels 20 times larger, as activations have."""
    x = normal(shape, seed).float()
    x[:, ::61] *= 20
    return x.to(torch.bfloat16)


def assert_product(got, A, B, name, bf16_out=True):
    """got against A @ B in fp64. Products of the operands are exact in fp32; a sum of K of them in
    fp32, in any order and even if each addition is truncated instead of rounded (2^-23), is off by at
    most K 2^-23 sum|a b|, the scales' product and the multiply-add of each block included; then one
    rounding to bf16."""
    ref = A @ B
    mag = np.abs(A) @ np.abs(B)
    tol = (A.shape[1] + 8) * 2.0 ** -23 * mag
    if bf16_out:
        tol = tol * (1 + U_BF16) + U_BF16 * np.abs(ref) + 2.0 ** -134
    else:
        tol = tol + 2.0 ** -149
    got = np.asarray(got, np.float64)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (f"{name}: {int(bad.sum())} of {bad.size} off, first at {np.argwhere(bad)[0].tolist()}: "
                           f"{got[bad][0]} for {ref[bad][0]} +- {tol[bad][0]}")


def offsets_of(sizes, first=0) -> list:
    return [first + sum(sizes[:e]) for e in range(len(sizes) + 1)]


def bf16_bits(t: torch.Tensor) -> np.ndarray:
    return synth.bf16_bits(t)


def bf16_round(x: np.ndarray) -> np.ndarray:
    return nf4.f32_from_bf16_bits(nf4.bf16_bits_from_f64(x)).astype(np.float64)
