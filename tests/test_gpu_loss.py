"""The vocabulary losses on the GPU against the definitions in float64.

Tolerances are derived in tests/vocab_reference.py from the kernels'
arithmetic.  Sizes sit around the tiles' and blocks' edges (64, 128, 256 and
one beside), down to one token, one vocabulary entry and a width of one.
"""

from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU-only machines
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import vocab_reference as ref  # noqa: E402
from dense_fp32_matrix_02_gb300 import gemm as G  # noqa: E402
from dense_fp32_matrix_02_gb300 import loss as L  # noqa: E402

DEV = torch.device("cuda:0")
BF16, F16 = torch.bfloat16, torch.float16


def matrix(rows, cols, dtype, seed, scale=1.0, pad=0, skew=0):
    """A random rows × cols matrix whose rows are cols + pad apart, starting
    `skew` elements into its storage; the padding holds NaN."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    store = torch.full((skew + rows * (cols + pad),), math.nan, dtype=dtype,
                       device=DEV)
    view = store[skew:].view(rows, cols + pad)[:, :cols]
    view.copy_(torch.randn(rows, cols, generator=gen, device=DEV) * scale)
    return view


def ce_case(T, V, D, dtype, seed=0, ignored=0.0, pad=0, skew=0):
    x = matrix(T, D, dtype, seed, 1.0, pad, skew)
    w = matrix(V, D, dtype, seed + 1, 2.0 / math.sqrt(D), pad, skew)
    gen = torch.Generator(device=DEV).manual_seed(seed + 2)
    y = torch.randint(0, V, (T,), generator=gen, device=DEV)
    if ignored:
        out = torch.rand(T, generator=gen, device=DEV) < ignored
        y = torch.where(out, torch.where(y % 2 == 0, -100, V + y), y)
        x[out] = math.nan  # rows that are not learnt from are not read
    g = torch.rand(T, generator=gen, device=DEV) + 0.1
    return x, w, y, g


def kd_case(T, V, D, top, dtype, seed=0, pad=0, skew=0):
    """Repeated ids, ids outside the vocabulary, logits of -inf, rows where
    nothing counts (their rows of x hold NaN)."""
    x, w, _, g = ce_case(T, V, D, dtype, seed, 0.0, pad, skew)
    gen = torch.Generator(device=DEV).manual_seed(seed + 3)
    ids = torch.randint(0, V, (T, top), generator=gen, device=DEV)
    u = 3.0 * torch.randn(T, top, generator=gen, device=DEV)
    r = torch.rand(T, top, generator=gen, device=DEV)
    ids = torch.where(r < 0.1, -1, torch.where(r > 0.95, V + ids, ids))
    u = torch.where((r > 0.1) & (r < 0.2), -math.inf, u)
    if T > 2:
        ids[1] = -1
        u[2] = -math.inf
    counts = ((ids >= 0) & (ids < V) & (u > -math.inf)).any(1)
    x[~counts] = math.nan
    return x, w, u, ids, g


def check(got, want, names):
    for name in names:
        a, b, tol = got[name].double(), want[name], want[name + "_tol"]
        bad = ~((a - b).abs() <= tol)
        assert not bool(bad.any()), (
            f"{name}: {int(bad.sum())} of {bad.numel()} outside tolerance; "
            f"first at {bad.nonzero()[0].tolist()}: got "
            f"{float(a[bad][0])!r}, want {float(b[bad][0])!r}, tol "
            f"{float(tol[bad][0])!r}")
    torch.cuda.synchronize()
    assert G.device_status() == 0


def run_ce(x, w, y, g, **kw):
    loss, lse = L.cross_entropy(x, w, y, **kw)
    dx, dw = L.cross_entropy_grad(x, w, y, lse, g, **kw)
    return {"loss": loss, "lse": lse, "dx": dx, "dw": dw}


def run_kd(x, w, u, ids, g, tau, **kw):
    loss, lse = L.distill(x, w, u, ids, tau, **kw)
    dx, dw = L.distill_grad(x, w, u, ids, lse, g, tau, **kw)
    return {"loss": loss, "lse": lse, "dx": dx, "dw": dw}


def want_ce(x, w, y, g):
    return ref.loss_and_grads(
        x, w, *ref.cross_entropy_targets(y, w.shape[0]), 1.0, g)


def want_kd(x, w, u, ids, g, tau):
    return ref.loss_and_grads(
        x, w, *ref.distill_targets(u, ids, tau, w.shape[0]), tau, g)


ALL = ("loss", "lse", "dx", "dw")
SIZES = [(1, 1, 1), (1, 1000, 64), (2, 5, 7), (63, 255, 63), (64, 256, 64),
         (65, 257, 65), (127, 511, 128), (128, 512, 200), (129, 513, 72),
         (255, 1000, 520), (257, 129, 264), (300, 4099, 96), (513, 70, 136),
         (1030, 300, 33), (3, 20011, 1000), (2100, 3001, 160)]


@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("T,V,D", SIZES)
def test_cross_entropy_sizes(T, V, D, dtype):
    x, w, y, g = ce_case(T, V, D, dtype, seed=T + V)
    check(run_ce(x, w, y, g), want_ce(x, w, y, g), ALL)


@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("ignored", [0.02, 0.5, 0.97])
@pytest.mark.parametrize("T,V,D", [(70, 300, 40), (600, 1031, 136)])
def test_ignored_tokens(T, V, D, ignored, dtype):
    x, w, y, g = ce_case(T, V, D, dtype, seed=5, ignored=ignored)
    g[(y < 0) | (y >= V)] = math.nan
    check(run_ce(x, w, y, g), want_ce(x, w, y, torch.nan_to_num(g)), ALL)


@pytest.mark.parametrize("T", [1, 64, 300])
def test_no_token_learnt_from(T):
    x, w, _, g = ce_case(T, 300, 72, BF16)
    x.fill_(math.nan)
    y = torch.full((T,), -100, device=DEV)
    got = run_ce(x, w, y, g)
    for name in ALL:
        assert bool((got[name] == 0).all()), name
    ids = torch.full((T, 3), -1, device=DEV)
    got = run_kd(x, w, torch.zeros(T, 3, device=DEV), ids, g, 2.0)
    for name in ALL:
        assert bool((got[name] == 0).all()), name


def test_no_tokens():
    x = torch.empty(0, 40, dtype=BF16, device=DEV)
    w = matrix(100, 40, BF16, 1)
    y = torch.empty(0, dtype=torch.int64, device=DEV)
    g = torch.empty(0, device=DEV)
    got = run_ce(x, w, y, g)
    assert got["loss"].shape == (0,) and got["dx"].shape == (0, 40)
    assert bool((got["dw"] == 0).all())


@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("T,V,D,top,tau", [
    (1, 300, 64, 1, 1.0), (5, 33, 17, 40, 0.5), (129, 1031, 136, 5, 2.0),
    (300, 700, 96, 64, 1.5), (64, 256, 64, 256, 4.0), (700, 513, 72, 31, 1.0),
    (2, 9001, 520, 128, 3.0)])
def test_distillation(T, V, D, top, tau, dtype):
    x, w, u, ids, g = kd_case(T, V, D, top, dtype, seed=top)
    check(run_kd(x, w, u, ids, g, tau), want_kd(x, w, u, ids, g, tau), ALL)


def test_distillation_of_one_entry_is_cross_entropy():
    x, w, y, g = ce_case(200, 777, 88, BF16, ignored=0.2)
    a = run_ce(x, w, y, g)
    b = run_kd(x, w, torch.full((200, 1), -3.0, device=DEV), y[:, None], g,
               1.0)
    for name in ALL:
        assert torch.equal(a[name], b[name]), name


@pytest.mark.parametrize("pad,skew", [(0, 1), (3, 0), (8, 0), (8, 4),
                                      (5, 3), (24, 8)])
@pytest.mark.parametrize("D", [64, 77])
def test_strides_and_alignment(D, pad, skew):
    x, w, y, g = ce_case(140, 333, D, BF16, pad=pad, skew=skew, ignored=0.1)
    check(run_ce(x, w, y, g), want_ce(x, w, y, g), ALL)
    x, w, u, ids, g = kd_case(140, 333, D, 9, F16, pad=pad, skew=skew)
    wide = torch.full((140, 13), 7.0, device=DEV)
    wide[:, :9] = u
    wide_ids = torch.full((140, 12), 3, device=DEV)
    wide_ids[:, :9] = ids
    got = run_kd(x, w, wide[:, :9], wide_ids[:, :9], g, 2.0)
    check(got, want_kd(x, w, u, ids, g, 2.0), ALL)


@pytest.mark.parametrize("pad,skew", [(0, 0), (3, 1), (8, 8)])
def test_outputs_given(pad, skew):
    x, w, y, g = ce_case(130, 270, 72, BF16, ignored=0.3)
    dx = matrix(130, 72, BF16, 1, 1.0, pad, skew).fill_(math.nan)
    dw = matrix(270, 72, BF16, 1, 1.0, pad, skew).fill_(math.nan)
    beside = dw.as_strided((270, 72 + pad), (72 + pad, 1))
    _, lse = L.cross_entropy(x, w, y)
    a, b = L.cross_entropy_grad(x, w, y, lse, g, dx=dx, dw=dw)
    assert a is dx and b is dw
    want = want_ce(x, w, y, g)
    check({"dx": dx, "dw": dw}, want, ("dx", "dw"))
    if pad:  # nothing is written beside the rows
        assert bool(beside[:, 72:].isnan().all())


def test_one_gradient_for_every_token():
    x, w, y, _ = ce_case(190, 400, 56, F16)
    g = torch.tensor(0.25, device=DEV).expand(190)
    check(run_ce(x, w, y, g), want_ce(x, w, y, g), ALL)


@pytest.mark.parametrize("size", [1e-6, 1.0, 3e3])
@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "f16"])
def test_gradient_magnitudes(size, dtype):
    """Upstream gradients from a mean over many tokens up to a scaled
    loss; 0 for some."""
    x, w, y, g = ce_case(150, 600, 72, dtype)
    x.mul_(0.25)
    g = g * size
    g[::7] = 0
    check(run_ce(x, w, y, g), want_ce(x, w, y, g), ALL)


@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "f16"])
def test_large_logits(dtype):
    """Logits of some thousands: without the running maximum the
    exponentials overflow."""
    x, w, y, g = ce_case(80, 500, 64, dtype)
    x.mul_(200.0)
    got, want = run_ce(x, w, y, g), want_ce(x, w, y, g)
    assert float(want["lse"].max()) > 400
    check(got, want, ("loss", "lse"))


def test_nan_spreads_only_as_it_should():
    """A NaN in a token's row reaches that token's loss and row of dx, and
    every row of dw; an Inf in a target's row of w its logits."""
    x, w, y, g = ce_case(150, 300, 64, BF16)
    x[70, 3] = math.nan
    got = run_ce(x, w, y, g)
    nan = got["loss"].isnan()
    assert bool(nan[70]) and int(nan.sum()) == 1
    rows = got["dx"].isnan().any(1)
    assert bool(rows[70]) and int(rows.sum()) == 1
    x[70, 3] = 1.0
    u = torch.zeros(150, 2, device=DEV)
    u[9, 1] = math.nan
    got = run_kd(x, w, u, torch.stack([y, (y + 1) % 300], 1), g, 1.0)
    nan = got["loss"].isnan()
    assert bool(nan[9]) and int(nan.sum()) == 1


@pytest.mark.parametrize("op", ["ce", "kd"])
def test_same_call_same_bits(op):
    if op == "ce":
        args = ce_case(700, 2500, 264, BF16, ignored=0.3)
        runs = [run_ce(*args) for _ in range(3)]
    else:
        args = kd_case(700, 2500, 264, 20, BF16)
        runs = [run_kd(*args, 2.0) for _ in range(3)]
    for r in runs[1:]:
        for name in ALL:
            assert torch.equal(r[name], runs[0][name]), name


def test_workspace_of_any_content():
    x, w, y, g = ce_case(300, 900, 72, F16, ignored=0.2)
    want = want_ce(x, w, y, g)
    for fill in (0, 255, 127):
        ws = torch.full((L.workspace_size(300, 900, 72, grad=True),), fill,
                        dtype=torch.uint8, device=DEV)
        need = L.workspace_size(300, 900, 72)
        loss, lse = L.cross_entropy(x, w, y, workspace=ws[:need])
        dx, dw = L.cross_entropy_grad(x, w, y, lse, g, workspace=ws)
        check({"loss": loss, "lse": lse, "dx": dx, "dw": dw}, want, ALL)


def test_other_stream():
    x, w, y, g = ce_case(300, 900, 72, BF16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = run_ce(x, w, y, g, stream=side)
    side.synchronize()
    check(a, want_ce(x, w, y, g), ALL)
    with torch.cuda.stream(side):
        b = run_ce(x, w, y, g)
    side.synchronize()
    for name in ALL:
        assert torch.equal(a[name], b[name]), name


def test_graph_capture():
    x, w, y, g = ce_case(260, 700, 72, BF16, ignored=0.2)
    run_ce(x, w, y, g)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run_ce(x, w, y, g)
    for seed in (3, 4):  # other inputs, another number of learnt tokens
        x2, w2, y2, g2 = ce_case(260, 700, 72, BF16, seed, 0.3 * (seed - 3))
        for a, b in ((x, x2), (w, w2), (y, y2), (g, g2)):
            a.copy_(b)
        graph.replay()
        check(got, want_ce(x, w, y, g), ALL)


@pytest.mark.parametrize("op", ["ce", "kd"])
def test_gradient_against_differences(op):
    """The kernels' gradients along a direction against a central difference
    of the float64 loss; the tolerance is the gradients' own, summed along
    the direction, and the difference's h² term."""
    T, V, D, tau = 40, 150, 24, 2.0 if op == "kd" else 1.0
    if op == "ce":
        x, w, y, g = ce_case(T, V, D, F16, ignored=0.0)
        targets = ref.cross_entropy_targets(y, V)
        got, want = run_ce(x, w, y, g), want_ce(x, w, y, g)
    else:
        x, w, u, ids, g = kd_case(T, V, D, 6, F16)
        x = torch.nan_to_num(x)
        targets = ref.distill_targets(u, ids, tau, V)
        got, want = run_kd(x, w, u, ids, g, tau), want_kd(x, w, u, ids, g,
                                                          tau)

    def total(xd, wd):
        z = xd @ wd.t() / tau
        ids, lq = targets
        q = lq.exp()
        at = z.gather(1, ids.clamp(0, V - 1))
        lse = torch.logsumexp(z, 1, keepdim=True)
        terms = torch.where(q > 0, q * (lq - (at - lse)), 0.0).sum(1)
        return float((g.double() * tau * tau * terms).sum())

    gen = torch.Generator(device=DEV).manual_seed(9)
    xd, wd, h = x.double(), w.double(), 1e-4
    for name, base in (("dx", xd), ("dw", wd)):
        way = torch.randn(base.shape, generator=gen, device=DEV,
                          dtype=torch.float64)
        if name == "dx":
            diff = total(xd + h * way, wd) - total(xd - h * way, wd)
        else:
            diff = total(xd, wd + h * way) - total(xd, wd - h * way)
        along = float((got[name].double() * way).sum())
        tol = float((want[name + "_tol"] * way.abs()).sum()) + 1e-4
        assert abs(along - diff / (2 * h)) <= tol, (name, along, diff)


def test_offsets_past_32_bits():
    """W of more than 2^31 elements: the last rows count as the first do."""
    V, D = 270_000, 8192
    w = torch.zeros(V, D, dtype=BF16, device=DEV)
    x = matrix(3, D, BF16, 1)
    hot = [0, 131_071, 262_143, 262_144, 269_999]
    rows = matrix(len(hot), D, BF16, 2, 4.0 / math.sqrt(D))
    w[hot] = rows
    y = torch.tensor([269_999, 262_144, 5], device=DEV)
    g = torch.tensor([0.5, 1.0, 2.0], device=DEV)
    got = run_ce(x, w, y, g)
    X, R = x.double(), rows.double()
    z = X @ R.t()
    total = torch.exp(z).sum(1) + (V - len(hot))
    lse = torch.log(total)
    at = torch.stack([z[0, 4], z[1, 3], torch.zeros_like(z[2, 0])])
    d = (1e-5 * math.sqrt(D) * (X.abs() @ R.abs().t())).amax(1)
    tol = d + 2e-5 + 1e-6 * lse
    assert bool(((got["lse"].double() - lse).abs() <= tol).all())
    assert bool(((got["loss"].double() - (lse - at)).abs()
                 <= d + tol + 1e-6 * at.abs() + 2e-5).all())
    # dw of a few rows, far apart
    p = torch.exp(z) / total[:, None]
    Q = torch.zeros_like(p)
    Q[0, 4] = Q[1, 3] = 1.0
    gd = g.double()[:, None]
    P = gd * (p - Q)
    dP = 2.0 ** -8 * P.abs() + gd * p * (d + tol + 2e-5)[:, None]
    want = P.t() @ X
    lim = (dP.t() @ X.abs() + 2e-5 * (P.abs().t() @ X.abs())
           + 2.0 ** -8 * want.abs())
    assert bool(((got["dw"][hot].double() - want).abs() <= lim).all())
    cold = torch.tensor([7, 262_150, 269_998], device=DEV)
    base = gd / total[:, None]
    want = (base * X).sum(0)
    lim = ((2.0 ** -8 * base + base * (d + tol + 2e-5)[:, None])
           * X.abs()).sum(0) + 2.0 ** -8 * want.abs() + 2e-5 * (
               base * X.abs()).sum(0)
    assert bool(((got["dw"][cold].double() - want).abs() <= lim).all())
    assert G.device_status() == 0


@pytest.mark.parametrize("op", ["ce", "kd"])
def test_pieces_of_the_vocabulary(op):
    """More logits than one piece of G holds: several launches, a shorter
    last piece, dX added up over them, some tokens ignored."""
    T, V, D = 8200, 20011, 72
    if op == "ce":
        x, w, y, g = ce_case(T, V, D, BF16, ignored=0.1)
        got, want = run_ce(x, w, y, g), want_ce(x, w, y, g)
    else:
        x, w, u, ids, g = kd_case(T, V, D, 7, F16)
        got = run_kd(x, w, u, ids, g, 2.0)
        want = want_kd(x, w, u, ids, g, 2.0)
    check(got, want, ALL)


@pytest.mark.parametrize("T,V", [(8200, 7000), (2100, 6500), (1500, 20011)])
def test_entries_stay_inside_the_vocabulary(T, V):
    """Whole tiles whose second half lies past an odd number of blocks of 128
    columns: no entry there."""
    x, w, u, ids, g = kd_case(T, V, 72, 7, F16)
    check(run_kd(x, w, u, ids, g, 2.0), want_kd(x, w, u, ids, g, 2.0), ALL)


@pytest.mark.parametrize("T,V,D", [(9000, 600, 40), (5000, 260, 520),
                                   (20, 12000, 72), (600, 9000, 264),
                                   (257, 40000, 64)])
def test_cuts_of_the_gradients(T, V, D):
    """Deep sums over tokens (dW in slots) and over the vocabulary (dX in
    many slots), with one and several rows of tiles."""
    x, w, y, g = ce_case(T, V, D, BF16, ignored=0.05)
    check(run_ce(x, w, y, g), want_ce(x, w, y, g), ALL)


def test_close_ids_of_one_token():
    """All entries of a token in a few neighbouring columns, and at the ends
    of the vocabulary."""
    T, V, D, top = 300, 1111, 72, 40
    x, w, _, g = ce_case(T, V, D, BF16)
    at = torch.arange(top, device=DEV)
    first = torch.randint(0, V - top, (T, 1), device=DEV)
    first[:100] = V - top
    first[100:200] = 0
    ids = first + at.flip(0)
    u = torch.randn(T, top, device=DEV)
    check(run_kd(x, w, u, ids, g, 1.0), want_kd(x, w, u, ids, g, 1.0), ALL)


def test_negative_gradients():
    x, w, u, ids, g = kd_case(200, 700, 72, 9, F16)
    g = torch.where(torch.arange(200, device=DEV) % 2 == 0, g, -g)
    check(run_kd(x, w, u, ids, g, 2.0), want_kd(x, w, u, ids, g, 2.0), ALL)
    x, w, y, g = ce_case(200, 700, 72, BF16, ignored=0.2)
    check(run_ce(x, w, y, -g), want_ce(x, w, y, -g), ALL)


def test_masked_columns():
    """Rows of w that put whole stretches of the vocabulary at -inf."""
    T, V, D = 100, 900, 64
    x, w, y, g = ce_case(T, V, D, BF16)
    x[:, 0] = 1.0
    y = y % 200
    w[300:700] = 0
    w[300:700, 0] = -math.inf
    loss, lse = L.cross_entropy(x, w, y)
    live = torch.cat([w[:300], w[700:]])
    want = want_ce(x, live, y, None)
    check({"loss": loss, "lse": lse}, want, ("loss", "lse"))


def test_a_wait_that_runs_out_is_reported():
    x, w, y, g = ce_case(300, 600, 72, BF16)
    run_ce(x, w, y, g)
    torch.cuda.synchronize()
    old = G.set_wait_timeout_ns(20_000_000)
    G.set_debug_flags(G.DEBUG_STALL_PRODUCER)
    try:
        run_ce(x, w, y, g)
        torch.cuda.synchronize()
        assert G.device_status() == 4
    finally:
        G.set_debug_flags(0)
        G.set_wait_timeout_ns(old)
    assert G.device_status() == 0
    check(run_ce(x, w, y, g), want_ce(x, w, y, g), ALL)


def test_two_streams():
    cases = [ce_case(300, 5000, 136, BF16, seed) for seed in (1, 2)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        got = []
        for case, s in zip(cases, streams):
            with torch.cuda.stream(s):
                got.append(run_ce(*case))
    torch.cuda.synchronize()
    for g, case in zip(got, cases):
        check(g, want_ce(*case), ALL)


def test_example_learns():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(__file__), "..", "examples",
                        "train_head.py")
    spec = importlib.util.spec_from_file_location("train_head", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    history = module.train(steps=6, tokens=512, vocab=1500, width=128)
    first, last = history[0], history[-1]
    assert abs(first[0] - math.log(1500)) < 1e-3  # a matrix of zeros
    assert last[0] < first[0] and last[1] < first[1]
    assert G.device_status() == 0


def test_checked_build_runs_clean():
    """The checked build, in a process of its own: no index leaves its
    buffer, and every result is in its tolerance."""
    import os
    import subprocess
    import sys

    from dense_fp32_matrix_02_gb300 import build
    path = build.build(checked=True)
    here = os.path.dirname(os.path.abspath(__file__))
    which = ("sizes or tokens or distillation or strides or inside or pieces"
             " or cuts or close")
    r = subprocess.run(
        [sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-k", which,
         os.path.join(here, "test_gpu_loss.py")],
        env=dict(os.environ, GEMM_F32_LIBRARY=path), cwd=here,
        capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
