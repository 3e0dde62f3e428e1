"""The bars of the orthogonalised update, derived on the CPU.

The update is returned in bf16 (half a step: 2^-8 of a value, 0.17% RMS over
values spread evenly in an octave).  Before it, each step's products take fp16
operands: X's upper part, P and Q = bP + cPP, each rounded at 2^-11, while X
itself is carried in two fp16 parts.  The emulation below makes exactly these
roundings (products in float64) on small matrices of every kind the GPU tests
use.  It stays below 0.4% RMS and 3.5% of the RMS at the worst element (8 x 8 and 24 x 2056);
the bars are twice those.  Rounding X itself at each step instead (no second
part) shows 1.5 to 5% RMS on gradients of falling singular values, which the bars
reject, and so does a dropped term of the polynomial.
"""
import math

import pytest
import torch

from tests import ops_ref as ref

RMS_BAR = 8e-3
MAX_BAR = 0.07


def gradients(kind, E, M, N, seed=0):
    """Stacks of gradient-like fp32 matrices."""
    g = torch.Generator()
    g.manual_seed(1000 * M + N + seed)
    if kind == "random":
        return torch.randn((E, M, N), generator=g) * 1e-3
    if kind == "rank8":
        return torch.randn((E, M, 8), generator=g) @ torch.randn((E, 8, N), generator=g) * 1e-3
    k = min(M, N)
    if kind == "low_rank":
        k = min(k, 16)
        s = torch.exp(-0.5 * torch.arange(float(k)))
        return (torch.randn((E, M, k), generator=g) * s) @ torch.randn((E, k, N), generator=g) \
            + 0.01 * torch.randn((E, M, N), generator=g)
    u = torch.linalg.qr(torch.randn((E, M, k), generator=g))[0]
    v = torch.linalg.qr(torch.randn((E, N, k), generator=g))[0]
    return (u * torch.logspace(0, -6, k)) @ v.transpose(1, 2)


def fp16(x):
    assert x.abs().max() < 65504
    return x.to(torch.float16).double()


def emulate(g, steps=5, eps=1e-7, carry=True, c=ref.NS[2]):
    a, b, _ = ref.NS
    m, n = g.shape
    S = 2.0 ** math.ceil(math.log2(math.sqrt(m * n)))
    SP = 2.0 ** 13
    x = g.double() * (S / (g.double().norm() + eps))
    if m > n:
        x = x.T
    for _ in range(steps):
        hi = fp16(x)
        lo = fp16(x - hi) if carry else 0
        p = fp16(hi @ hi.T * (SP / S / S))
        q = fp16(b * p + c * (p @ p) / SP)
        x = a * (hi + lo) + q @ hi / SP
    x = (x / S).to(torch.bfloat16).double()
    return x.T if m > n else x


def errors(y, want):
    rms = want.square().mean().sqrt()
    err = (y - want).abs()
    return float(err.square().mean().sqrt() / rms), float(err.max() / rms)


KINDS = ["random", "low_rank", "rank8", "decay"]
SHAPES = [(8, 8), (24, 2056), (64, 64), (128, 256), (256, 128), (264, 264), (520, 72), (8, 1024), (16, 40), (512, 768)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M,N", SHAPES)
def test_emulated_roundings_stay_below_half_the_bars(kind, M, N):
    for g in gradients(kind, 2, M, N):
        rms, top = errors(emulate(g), ref.orthogonalize(g[None])[0])
        assert rms <= RMS_BAR / 2 and top <= MAX_BAR / 2, (rms, top)


@pytest.mark.parametrize("kind", ["low_rank", "rank8", "decay"])
def test_the_bars_reject_a_single_fp16_part(kind):
    g = gradients(kind, 1, 128, 256)[0]
    assert errors(emulate(g, carry=False), ref.orthogonalize(g[None])[0])[0] > RMS_BAR


def test_the_bars_reject_a_wrong_polynomial():
    g = gradients("random", 1, 128, 256)[0]
    want = ref.orthogonalize(g[None])[0]
    assert errors(emulate(g, c=1.02 * ref.NS[2]), want)[0] > RMS_BAR
    assert errors(emulate(g, steps=4), want)[0] > RMS_BAR


def test_float64_reference_is_the_polynomial_of_the_singular_values():
    """X = U s V^T goes to U p(p(...p(s))) V^T: the same by a singular value decomposition."""
    g = gradients("random", 1, 40, 64)[0].double()
    u, s, vt = torch.linalg.svd(g / (g.norm() + 1e-7), full_matrices=False)
    a, b, c = ref.NS
    for _ in range(5):
        s = a * s + b * s ** 3 + c * s ** 5
    assert torch.allclose((u * s) @ vt, ref.orthogonalize(g[None])[0], atol=1e-12)


def test_two_parts_hold_sixteen_bits():
    g = torch.Generator()
    g.manual_seed(0)
    v = torch.randn(100000, generator=g)
    hi = v.to(torch.bfloat16)
    lo = (v - hi.float()).to(torch.bfloat16)
    assert ((hi.double() + lo.double() - v.double()).abs() <= ref.TWO_PARTS * v.double().abs()).all()
