"""The global norm and clipping on the GPU against float64.

Tolerances: squares are summed in fp32, at most 32 in a run and three more
additions, then in float64, so the norm is off by at most half of
35 · 2^-24 relative, and by its own rounding: 20 · 2^-24.  A clipped element
has the factor's error, that of its product and one rounding to its type
(half a step, or half the smallest step).
"""

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
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
NORM_TOL = 20 * 2.0 ** -24
SMALLEST = {BF16: 2.0 ** -133, F16: 2.0 ** -24, F32: 2.0 ** -149}


def tensor(rows, cols, dtype, seed, scale=1.0, pad=0, skew=0):
    """Rows cols + pad apart, `skew` elements into the storage; NaN around."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    store = torch.full((skew + rows * (cols + pad),), math.nan, dtype=dtype,
                       device=DEV)
    view = store[skew:].view(rows, cols + pad)[:, :cols]
    view.copy_(torch.randn(rows, cols, generator=gen, device=DEV) * scale)
    return view


def norm_of(ts):
    return math.sqrt(sum(float((t.double() ** 2).sum()) for t in ts))


def check_clipped(before, after, max_norm, norm):
    factor = min(1.0, max_norm / norm) if norm > 0 else 1.0
    for b, a in zip(before, after):
        want = b.double() * factor
        u = torch.finfo(b.dtype).eps / 2
        tol = want.abs() * (u + 2 * NORM_TOL) + SMALLEST[b.dtype] / 2
        if factor == 1.0:
            assert torch.equal(a, b)
        bad = ~((a.double() - want).abs() <= tol)
        assert not bool(bad.any()), (bad.nonzero()[0].tolist(), a.shape)


def check(ts, max_norm):
    before = [t.clone() for t in ts]
    want = norm_of(ts)
    got = C.global_norm(ts)
    assert got.shape == (1,) and got.dtype == F32
    assert abs(float(got) - want) <= NORM_TOL * want
    # apart, then in place
    out = [torch.full_like(t, 7.0) for t in before]
    n2 = C.clip_(ts, max_norm, out=out)
    assert torch.equal(n2, got)
    for t, b in zip(ts, before):
        assert torch.equal(t, b)
    check_clipped(before, out, max_norm, want)
    n3 = C.clip_(ts, max_norm)
    assert torch.equal(n3, got)
    for t, o in zip(ts, out):
        assert torch.equal(t, o)
    torch.cuda.synchronize()
    assert G.device_status() == 0


@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=["bf16", "f16", "f32"])
@pytest.mark.parametrize("n", [1, 2, 3, 7, 8, 9, 255, 256, 257, 2047, 2048,
                               2049, 8191, 32768, 100003, 4_000_037])
def test_one_vector(n, dtype):
    check([tensor(1, n, dtype, n)[0]], 0.5 * math.sqrt(n))


@pytest.mark.parametrize("skew", [0, 1, 2, 3, 4, 5, 8])
@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=["bf16", "f16", "f32"])
def test_offsets_and_rows(dtype, skew):
    """Rows of every width around a group's, apart by even and odd numbers,
    from any element on; what lies between the rows stays as it was."""
    ts = [tensor(r, c, dtype, r + c, 1.0, pad, skew)
          for r in (1, 2, 33) for c in (1, 3, 4, 7, 8, 9, 31, 64, 300)
          for pad in (0, 1, 3, 8)]
    check(ts, 3.0)
    for t in ts:
        if t.stride(0) > t.shape[1] and t.shape[0] > 1:
            gap = t.as_strided((t.shape[0] - 1, t.stride(0) - t.shape[1]),
                               (t.stride(0), 1),
                               t.storage_offset() + t.shape[1])
            assert bool(gap.isnan().all())


@pytest.mark.parametrize("count", [0, 1, 31, 32, 33, 519, 520, 521, 1100])
def test_numbers_of_gradients(count):
    """Lists of one launch and of several, empty gradients among them."""
    if count == 0:
        with pytest.raises(ValueError, match="no gradients"):
            C.clip_([], 1.0)
        return
    kinds = (BF16, F16, F32)
    ts = [tensor(1, 1 + (i * 37) % 500, kinds[i % 3], i)[0]
          for i in range(count)]
    ts.insert(count // 2, torch.empty(0, device=DEV))
    ts.append(torch.empty(0, 5, device=DEV, dtype=BF16))
    check(ts, 2.0)


def test_contiguous_beside_rows():
    """A gradient whose rows are apart, clipped into one whose are not."""
    a, b = tensor(37, 53, BF16, 1, pad=11), tensor(37, 53, BF16, 1)
    for src, dst in ((a, torch.zeros_like(b)),
                     (b, tensor(37, 53, BF16, 5, pad=3))):
        C.clip_([src], 1.0, out=[dst])
        check_clipped([src], [dst], 1.0, norm_of([src]))
    with pytest.raises(ValueError, match="contiguous"):
        C.global_norm([tensor(8, 8, BF16, 1).t()[:, 1:]])
    flat = torch.zeros(100, dtype=BF16, device=DEV)  # pieces of one buffer
    src = [tensor(3, 7, BF16, 2), tensor(5, 4, BF16, 3)]
    C.clip_(src, 1.0, out=[flat[1:22], flat[22:42]])
    check_clipped(src, [flat[1:22].view(3, 7), flat[22:42].view(5, 4)], 1.0,
                  norm_of(src))
    assert float(flat[0]) == 0.0 and bool((flat[42:] == 0).all())
    with pytest.raises(ValueError, match="shapes"):  # rows of another width
        C.clip_([tensor(6, 4, BF16, 1, pad=1)], 1.0, out=[flat[:24]])
    x = tensor(4, 6, F32, 3).view(2, 2, 6)  # any shape, contiguous
    check([x, tensor(1, 1, F32, 2).reshape(())], 1.0)


def test_not_clipped_to_the_bit():
    """A norm within the bound: out is a copy, NaN payloads, zeros of either
    sign and subnormals included; a bound of infinity, a norm of zero."""
    bits = torch.arange(-2000, 2000, dtype=torch.int32, device=DEV)
    t = bits.view(F32)[2000:]  # subnormals
    for max_norm in (1.0, math.inf):
        out = [torch.ones_like(t)]
        C.clip_([t], max_norm, out=out)
        assert torch.equal(out[0].view(torch.int32), t.view(torch.int32))
    z = torch.tensor([0.0, -0.0] * 4, device=DEV)
    for max_norm in (0.0, 1.0):
        out = [torch.ones_like(z)]
        assert float(C.clip_([z], max_norm, out=out)) == 0.0
        assert torch.equal(out[0].view(torch.int32), z.view(torch.int32))


def test_bound_of_zero():
    t = tensor(3, 100, F16, 1)
    C.clip_([t], 0.0)
    assert bool((t == 0).all())


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("at", [0, 5000, 9999])
def test_norms_that_are_not_finite(bad, at):
    a, b = tensor(1, 10000, BF16, 1)[0], tensor(1, 777, F32, 2)[0]
    a[at] = bad
    keep = [a.clone(), b.clone()]
    n = float(C.clip_([a, b], 0.1))
    assert math.isnan(n) if math.isnan(bad) else n == math.inf
    for t, k in zip((a, b), keep):
        assert torch.equal(t.nan_to_num(9.0), k.nan_to_num(9.0))


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("power", [-126, -100, -70, -64, -50, 50, 63, 64, 100,
                                   120])
def test_squares_out_of_range(power, dtype):
    """Squares that overflow or vanish in fp32, where the norm does not."""
    ts = [tensor(1, n, dtype, n, 2.0 ** power)[0] for n in (1, 9, 3001)]
    want = norm_of(ts)
    assert abs(float(C.global_norm(ts)) - want) <= NORM_TOL * want
    small = tensor(1, 5000, dtype, 3, 2.0 ** -120)[0]  # beside others
    both = [small, *ts]
    want = norm_of(both)
    before = [t.clone() for t in both]
    assert abs(float(C.clip_(both, want / 4)) - want) <= NORM_TOL * want
    check_clipped(before, both, want / 4, want)


def test_norm_beyond_fp32():
    """A norm that only a double holds is written as infinity and clips."""
    t = torch.full((4096,), 2.0 ** 127, device=DEV)
    n = C.clip_([t], 1.0)
    assert float(n) == math.inf
    want = 1.0 / 64
    assert bool(((t - want).abs() <= want * 2 * NORM_TOL).all())


def test_same_bits_again_and_graph():
    """The same call gives the same bits; captured, it works on what the
    tensors hold when it is replayed; two graphs share a workspace."""
    ts = [tensor(1, 70001, BF16, 4)[0], tensor(200, 301, F32, 5, pad=3)]
    out = [torch.empty_like(t) for t in ts]
    ws = torch.empty(C.workspace_size(2), dtype=torch.uint8, device=DEV)
    eager = C.clip_(ts, 3.0, out=out, workspace=ws)
    keep = [o.clone() for o in out]
    assert torch.equal(C.clip_(ts, 3.0, out=out), eager)
    graphs, norms = [], []
    for bound in (3.0, 1.0):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            norms.append(C.clip_(ts, bound, out=out, workspace=ws))
        graphs.append(g)
    for order in ((0, 1, 0), (1, 0, 0)):
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(norms[0], eager)
        for o, k in zip(out, keep):
            assert torch.equal(o, k)
    for t in ts:
        t.mul_(2.0)
    graphs[0].replay()
    assert abs(float(norms[0]) - 2 * float(eager)) <= 4e-6 * float(eager)


def test_many_gradients_in_a_graph():
    """A captured launch holds its list of gradients, a long one too."""
    ts = [tensor(1, 1 + (i * 37) % 500, F32, i)[0] for i in range(600)]
    out = [torch.empty_like(t) for t in ts]
    C.clip_(ts, 3.0, out=out)
    keep = [o.clone() for o in out]
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        C.clip_(ts, 3.0, out=out)
    for o in out:
        o.fill_(math.nan)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, k) for o, k in zip(out, keep))


def test_streams():
    ts = [tensor(1, 3_000_001, F32, 6)[0]]
    want = C.global_norm(ts)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = C.global_norm(ts, stream=s)
    with torch.cuda.stream(s):
        got2 = C.global_norm(ts)
    s.synchronize()
    assert torch.equal(got, want) and torch.equal(got2, want)


def test_large():
    """More elements than 2^31, rows of which start past 2^32 bytes."""
    n = 2 ** 31 + 4099
    t = torch.full((n,), 0.5, dtype=BF16, device=DEV)
    t[-1] = 3.0
    want = math.sqrt((n - 1) / 4 + 9)
    got = C.clip_([t], want / 2)
    assert abs(float(got) - want) <= NORM_TOL * want
    assert float(t[0]) == 0.25 and float(t[-2]) == 0.25
    assert float(t[-1]) == 1.5
    assert bool((t[:-1] == 0.25).all())


def test_refusals():
    a = tensor(4, 8, BF16, 1)
    with pytest.raises(TypeError):
        C.global_norm([a.double()])
    with pytest.raises(TypeError, match="types"):
        C.clip_([a], 1.0, out=[a.float()])
    with pytest.raises(ValueError, match="shapes"):
        C.clip_([a], 1.0, out=[a[:2]])
    with pytest.raises(ValueError, match="tensor for each"):
        C.clip_([a], 1.0, out=[])
    with pytest.raises(ValueError, match="CUDA"):
        C.global_norm([a.cpu()])
    for bad in (-1.0, math.nan):
        with pytest.raises(G.GemmError):
            C.clip_([a], bad)
    ws = torch.empty(64, dtype=torch.uint8, device=DEV)
    with pytest.raises(G.GemmError):
        C.clip_([a], 1.0, workspace=ws)
    # a gradient that is listed twice: in the norm twice, never clipped
    twice = math.sqrt(2) * norm_of([a])
    assert abs(float(C.global_norm([a, a])) - twice) <= NORM_TOL * twice
    keep = a.clone()
    with pytest.raises(G.GemmError):
        C.clip_([a, a], 1.0)
    with pytest.raises(G.GemmError):
        C.clip_([a, a.clone()], 1.0, out=[keep, keep])
    assert torch.equal(a, keep)


def test_columns_of_one_matrix():
    """Gradients side by side in one matrix, each with its own columns."""
    m = tensor(50, 96, BF16, 1)
    parts = [m[:, :32], m[:, 32:41], m[:, 41:]]
    before = [t.clone() for t in parts]
    want = norm_of(parts)
    assert abs(float(C.clip_(parts, want / 3)) - want) <= NORM_TOL * want
    check_clipped(before, parts, want / 3, want)


def test_checked_build_runs_clean():
    """The checked build, in a process of its own: no index leaves its
    buffer."""
    import os
    import subprocess
    import sys

    from dense_fp32_matrix_02_gb300 import build
    path = build.build(checked=True)
    here = os.path.dirname(os.path.abspath(__file__))
    r = subprocess.run(
        [sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-k",
         "not checked and not large", os.path.join(here, "test_gpu_grads.py")],
        env=dict(os.environ, GEMM_F32_LIBRARY=path), cwd=here,
        capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
