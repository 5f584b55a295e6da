"""Products with a quantized weight that carry per-row adapters, and tiles that are split along the
inner size, pinned bit for bit.

Scales are powers of two, zero-points, rows and factors small integers, so that every product, every
low-rank part and every partial sum is a multiple of 2^-7 far below 2^24 of them: exact in fp32 in
any order.  The 64-bit formula is then the one right answer, and binary16 results are its rounding.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_experts import WIDTHS, _ints, _quantized, _route, _want  # noqa: E402


@pytest.fixture(scope="module")
def hq():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a ROCm device")
    import bit_weight_quantization_amd as m
    m.load_library()
    return m


def _adapters(M, N, K, r, n, none, seed):
    """X, A, B, ids, scales of small integers; v = A x stays below 2 K and u = B^T dy below 2 N."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    ids = torch.randint(0, n, (M,), device="cuda", generator=gen, dtype=torch.int32)
    off = torch.rand(M, device="cuda", generator=gen) < none
    ids[off] = torch.where(torch.rand(M, device="cuda", generator=gen)[off] < 0.5, -1, n).to(torch.int32)
    scales = 2.0 ** torch.randint(-1, 2, (n,), device="cuda", generator=gen).float()
    return dict(X=_ints((M, K), seed), A=_ints((n, r, K), seed + 1, 1), B=_ints((n, N, r), seed + 2, 1),
                ids=ids, scales=scales)


def _low(x, A, B, ids, scales):
    """s_a (x A_a^T) B_a^T per row, 64 bits."""
    y = torch.zeros((x.shape[0], B.shape[1]), device="cuda", dtype=torch.float64)
    for a in range(A.shape[0]):
        m = torch.nonzero(ids == a)[:, 0]
        if len(m):
            v = x[m].double() @ A[a].double().t().contiguous()
            y[m] = float(scales[a]) * (v @ B[a].double().t().contiguous())
    return y


def _factor_gradients(x, d, A, B, ids, scales):
    dA, dB = torch.zeros_like(A, dtype=torch.float64), torch.zeros_like(B, dtype=torch.float64)
    for a in range(A.shape[0]):
        m = torch.nonzero(ids == a)[:, 0]
        if len(m):
            xa, da, s = x[m].double(), d[m].double(), float(scales[a])
            dA[a] = s * ((da @ B[a].double()).t().contiguous() @ xa)
            dB[a] = s * (da.t().contiguous() @ (xa @ A[a].double().t().contiguous()))
    return dA, dB


# rows, N, K, rank, adapters, none.  One and two rows (one launch with the low-rank part inside), ranks
# on both sides of 64; 3 to 64 rows (the product, then the adapters): K that is and is not a multiple
# of 256, split sums; more rows (tiles): one adapter or many in 128 rows, an adapter a row, K in
# several units of 512 that end inside one, ragged N, N of one column, tiles fewer than an XCD's
SHAPES = [(1, 130, 384, 8, 1, 0.0), (1, 257, 2048, 136, 3, 0.0), (2, 515, 640, 64, 2, 0.5), (2, 33, 128, 256, 2, 0.0),
          (3, 100, 640, 16, 2, 0.2), (20, 700, 2048, 24, 4, 0.1), (33, 515, 1280, 16, 3, 0.1), (64, 260, 512, 72, 9, 0.3),
          (65, 300, 128, 8, 1, 0.0), (100, 257, 640, 16, 90, 0.1), (129, 1, 1152, 64, 2, 0.2), (200, 515, 2048, 32, 3, 0.1),
          (400, 1000, 1152, 24, 5, 1.0), (700, 770, 640, 128, 300, 0.1), (1030, 260, 1152, 16, 4, 0.0)]


@pytest.mark.parametrize("nbits,g", WIDTHS)
def test_a_projection_with_adapters_is_exact_on_exact_inputs(hq, nbits, g):
    for M, N, K, r, n, none in SHAPES:
        q, W = _quantized(hq, N, K, nbits, g, seed=N + K)
        t = _adapters(M, N, K, r, n, none, seed=M)
        dY = _ints((M, N), seed=M + 9, lim=1)
        want = t["X"].double() @ W.t().contiguous() + _low(t["X"], t["A"], t["B"], t["ids"], t["scales"])
        assert torch.equal(hq.matmul_adapters(t["X"], q, t["A"], t["B"], t["ids"], t["scales"], out_f32=True).double(),
                           want), (M, N, K)
        assert torch.equal(hq.matmul_adapters(t["X"], q, t["A"], t["B"], t["ids"], t["scales"]), want.half()), (M, N, K)
        want = dY.double() @ W + _low(dY, t["B"].transpose(1, 2), t["A"].transpose(1, 2), t["ids"], t["scales"])
        dA, dB = _factor_gradients(t["X"], dY, t["A"], t["B"], t["ids"], t["scales"])
        for f32 in (True, False):
            gX, gA, gB = hq.matmul_adapters_backward(dY, t["X"], q, t["A"], t["B"], t["ids"], t["scales"], out_f32=f32)
            assert torch.equal(gX.double(), want) if f32 else torch.equal(gX, want.half()), (M, N, K)
            assert torch.equal(gA.double(), dA) and torch.equal(gB.double(), dB), (M, N, K)


# tokens, topk, experts, N, K, dropped: means of 49 to 64 rows (64-row tiles) and above, K in several
# units of 512, a weight of few groups, N below a tile; the gradient's N in several units, K ragged
TILES = [(110, 1, 2, 300, 1152, 0.0), (128, 2, 4, 257, 640, 0.2), (130, 1, 1, 2, 128, 0.0), (260, 1, 2, 2100, 640, 0.1),
         (150, 2, 3, 515, 2048, 0.1), (1100, 1, 1, 1030, 1152, 0.0), (2100, 1, 2, 130, 640, 0.5)]


@pytest.mark.parametrize("nbits,g", WIDTHS)
def test_tiles_of_experts_that_are_split_are_exact(hq, nbits, g):
    for tokens, topk, E, N, K, dropped in TILES:
        r, _, _ = _route(hq, tokens, topk, E, dropped, tokens + N)
        offsets = r.offsets.cpu().numpy()
        q, W = _quantized(hq, E * N, K, nbits, g, seed=N + K)
        X, dY = _ints((tokens, K), seed=tokens), _ints((r.rows, N), seed=tokens + 1, lim=1)
        Xs = hq.expert_gather(X, r)
        want = _want(Xs, W, offsets, N, False)
        for f32 in (True, False):
            got = hq.matmul_experts(X, q, r, out_f32=f32)
            assert torch.equal(got.double(), want) if f32 else torch.equal(got, want.half()), (tokens, N, K)
            got = hq.matmul_experts(Xs, q, r, sorted_rows=True, out_f32=f32)
            assert torch.equal(got.double(), want) if f32 else torch.equal(got, want.half()), (tokens, N, K)
            got = hq.matmul_experts_backward(dY, q, r, out_f32=f32)
            back = _want(dY, W, offsets, N, True)
            assert torch.equal(got.double(), back) if f32 else torch.equal(got, back.half()), (tokens, N, K)


@pytest.mark.parametrize("M", [2, 30, 300])
def test_rows_and_weights_of_any_alignment_within_the_call(hq, M):
    """Scales and zero-points two bytes off 16 take other kernels and give the same exact result."""
    N, K, g = 260, 512, 64
    q, W = _quantized(hq, N, K, 4, g, seed=5)
    t = _adapters(M, N, K, 16, 3, 0.2, seed=M)
    dY = _ints((M, N), seed=M, lim=1)

    def odd(x):
        held = torch.empty(x.numel() + 1, dtype=x.dtype, device="cuda")
        held[1:] = x.flatten()
        return held[1:].view(x.shape)
    q2 = hq.QuantizedWeight(packed=q.packed, scale=odd(q.scale), zero=odd(q.zero), rows=N, cols=K, nbits=4, group_size=g)
    rest = (t["A"], t["B"], t["ids"], t["scales"])
    for a, b in zip((hq.matmul_adapters(t["X"], q, *rest), *hq.matmul_adapters_backward(dY, t["X"], q, *rest)),
                    (hq.matmul_adapters(t["X"], q2, *rest), *hq.matmul_adapters_backward(odd(dY), t["X"], q2, *rest))):
        assert torch.equal(a, b)


@pytest.mark.parametrize("M", [1, 2, 30, 300])
def test_what_a_row_does_not_use_reaches_no_result(hq, M):
    """Adapters of no row hold NaN and infinities, rows of no adapter keep the product alone; a row that
    holds NaN spoils itself and its adapter's gradients only."""
    N, K = 260, 640
    q, W = _quantized(hq, N, K, 4, 64, seed=6)
    t = _adapters(M, N, K, 16, 4, 0.0, seed=M)
    t["ids"] = torch.arange(M, device="cuda", dtype=torch.int32) % 2 * 2 - 1  # -1, 1, -1, ...
    dY = _ints((M, N), seed=M, lim=1)
    rest = (t["A"], t["B"], t["ids"], t["scales"])
    clean = (hq.matmul_adapters(t["X"], q, *rest), *hq.matmul_adapters_backward(dY, t["X"], q, *rest))
    A, B, s = t["A"].clone(), t["B"].clone(), t["scales"].clone()
    for a in (0, 2, 3):
        A[a], B[a], s[a] = float("nan"), float("inf"), float("nan")
    got = (hq.matmul_adapters(t["X"], q, A, B, t["ids"], s),
           *hq.matmul_adapters_backward(dY, t["X"], q, A, B, t["ids"], s))
    assert all(torch.equal(a, b) for a, b in zip(got, clean))
    X, dYb = t["X"].clone(), dY.clone()
    X[0], dYb[0] = float("nan"), float("nan")  # a row of no adapter
    got = (hq.matmul_adapters(X, q, *rest), *hq.matmul_adapters_backward(dYb, X, q, *rest))
    for a, b in zip(got[:2], clean[:2]):
        assert bool(a[0].isnan().all()) and torch.equal(a[1:], b[1:])
    assert torch.equal(got[2], clean[2]) and torch.equal(got[3], clean[3])


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("M", [2, 5, 64, 65, 300])
def test_an_adapter_that_holds_nan_spoils_its_own_rows_only(hq, M, dtype):
    """Other requests' rows, and rows of no adapter, keep their results when one adapter in use (its
    rows between theirs, in the same tiles) holds NaN and infinities."""
    N, K = 260, 640
    t = _adapters(M, N, K, 16, 4, 0.0, seed=M)
    t["ids"] = torch.arange(M, device="cuda", dtype=torch.int32) % 4 - 1  # -1, 0, 1, 2, -1, ...
    t = {k: v.to(dtype) if v.dtype == torch.float16 else v for k, v in t.items()}
    dY = _ints((M, N), seed=M, lim=1).to(dtype)
    bad = dict(t, A=t["A"].clone(), B=t["B"].clone())
    bad["A"][0, 3, 5], bad["A"][0, 4, :] = float("inf"), float("nan")
    bad["B"][0, 7, 2], bad["B"][0, 11, :] = float("nan"), float("-inf")
    keep, other = t["ids"] != 0, torch.arange(4, device="cuda") != 0
    calls = [lambda u: (hq.adapters(**u), *hq.adapters_backward(dY, **u))]
    if dtype == torch.float16:
        for nbits in (4, 3):
            q, _ = _quantized(hq, N, K, nbits, 64, seed=8)
            calls.append(lambda u, q=q: (hq.matmul_adapters(u["X"], q, u["A"], u["B"], u["ids"], u["scales"]),
                                         *hq.matmul_adapters_backward(dY, u["X"], q, u["A"], u["B"], u["ids"], u["scales"])))
    for call in calls:
        clean, got = call(t), call(bad)
        for a, b in zip(got[:2], clean[:2]):
            assert torch.equal(a[keep], b[keep])
        for a, b in zip(got[2:], clean[2:]):
            assert torch.equal(a[other], b[other])
        assert not bool(got[0][~keep].isfinite().all(1).any())


def test_one_workspace_serves_call_after_call(hq):
    """A workspace that the caller keeps, with what earlier calls of other sizes left in it."""
    held = torch.full((1 << 28,), 255, dtype=torch.uint8, device="cuda")  # NaN in every type
    for M, N, K in ((1, 130, 640), (30, 260, 2048), (300, 515, 1152), (65, 130, 640), (1100, 260, 640), (20, 260, 512)):
        q, W = _quantized(hq, N, K, 4, 64, seed=7)
        t = _adapters(M, N, K, 16, 3, 0.2, seed=M)
        dY = _ints((M, N), seed=M, lim=1)
        rest = (t["A"], t["B"], t["ids"], t["scales"])
        want = (hq.matmul_adapters(t["X"], q, *rest), *hq.matmul_adapters_backward(dY, t["X"], q, *rest))
        got = (hq.matmul_adapters(t["X"], q, *rest, workspace=held),
               *hq.matmul_adapters_backward(dY, t["X"], q, *rest, workspace=held))
        assert all(torch.equal(a, b) for a, b in zip(got, want))
