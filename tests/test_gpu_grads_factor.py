"""The factor of clipping where it is awkward: quotients far below 1, and a
product that rounds once."""

from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU-only machines
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from dense_fp32_matrix_02_gb300 import gemm as G  # noqa: E402
from dense_fp32_matrix_02_gb300 import grads as C  # noqa: E402

DEV = torch.device("cuda:0")
F32 = torch.float32


def bound_of(max_norm):
    """The bound as the call takes it, in fp32."""
    return float(torch.tensor(max_norm, dtype=F32))


@pytest.mark.parametrize("power", [-40, 0, 30, 125])
@pytest.mark.parametrize("max_norm", [1.3, 0.7, 1e-3, 1e-20, 3e-38, 1e-44])
def test_factors_far_below_one(max_norm, power):
    """n = 5·2^power exactly, from 3 and 4 of it: each element is within half a
    step of fp32 of g·max_norm/n (2^-16 of that for the quotient and the
    product before the rounding), with 2^-150 where what the factor's second
    part adds is below the smallest number."""
    t = torch.zeros(70, device=DEV)
    t[3], t[50] = 3.0 * 2.0 ** power, -4.0 * 2.0 ** power
    norm = 5.0 * 2.0 ** power
    before = t.clone()
    n = C.clip_([t], max_norm)
    assert float(n) == (norm if norm < 2.0 ** 128 else math.inf)
    want = before.double() * min(1.0, bound_of(max_norm) / norm)
    half = torch.clamp(want.abs() * 2.0 ** -24, min=2.0 ** -150)
    tol = half * (1 + 2.0 ** -16) + 2.0 ** -150
    assert bool(((t.double() - want).abs() <= tol).all())
    assert G.device_status() == 0


@pytest.mark.parametrize("max_norm", [1.0, 1.3, 0.9999, 1e-25])
def test_norms_beyond_fp32(max_norm):
    """More of the largest numbers, whose norm only a double holds."""
    for n in (4096, 1 << 20):
        t = torch.full((n,), 1.5 * 2.0 ** 126, device=DEV)
        norm = 1.5 * 2.0 ** 126 * math.sqrt(n)  # (both are powers of 4)
        assert float(C.clip_([t], max_norm)) == math.inf
        want = 1.5 * 2.0 ** 126 * (bound_of(max_norm) / norm)
        tol = max(want * 2.0 ** -24, 2.0 ** -150) * (1 + 2.0 ** -16)
        assert bool(((t.double() - want).abs() <= tol + 2.0 ** -150).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, F32],
                         ids=["bf16", "f16", "f32"])
def test_one_rounding(dtype):
    """Each element is within half a step of its type of the exact product,
    with what the way by fp32 adds to a 16-bit result (2^-24 of it).  The
    squares of small integers and their sum are exact, and the norm in
    float64 is off by 2^-53."""
    u = torch.finfo(dtype).eps / 2
    for scale in (1.0, 2.0 ** -7, 2.0 ** 6):
        t = torch.zeros(64, dtype=dtype, device=DEV)
        t[::8] = torch.tensor([1.0, 2.0, 3.0, 5.0, 5.0, 6.0, 10.0, 7.0],
                              device=DEV).to(dtype) * scale
        norm = math.sqrt(249.0) * scale
        for max_norm in torch.linspace(0.03, 0.99, 97).tolist():
            out = torch.empty_like(t)
            C.clip_([t], max_norm * scale, out=[out])
            want = t.double() * (bound_of(max_norm * scale) / norm)
            step = torch.exp2(torch.floor(torch.log2(want.abs())))
            # (below the type's smallest normal number steps shrink no more:
            # binary16's 0.03 * 2^-7 / 15.8 = 1.5e-5 lies below 6.1e-5)
            step = step.clamp_min(torch.finfo(dtype).smallest_normal)
            half = torch.where(want == 0, torch.zeros_like(want), step * u)
            tol = half * (1 + 2.0 ** -16)
            if dtype != F32:
                tol += want.abs() * 2.0 ** -24
            err = (out.double() - want).abs()
            assert bool((err <= tol).all()), max_norm


def test_zeros_keep_their_sign():
    for dtype in (torch.bfloat16, torch.float16, F32):
        for max_norm in (0.0, 1e-25, 0.3, 0.7, 0.9):
            t = torch.tensor([0.0, -0.0, 1.0, -1.0] * 5, device=DEV).to(dtype)
            C.clip_([t], max_norm)
            assert t.signbit().tolist() == [False, True, False, True] * 5
