"""Sizes at both ends: tensors of more than 2^31 elements, where a 32-bit offset would read or
write another row, and products over nothing.

Small integers and scales that are powers of two make every sum exact, so results are compared for
equality with 64-bit formulas on the rows behind the 2^31st element.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hq():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a ROCm device")
    import bit_weight_quantization_amd as m
    m.load_library()
    yield m
    torch.cuda.empty_cache()


def _ints(shape, seed, dtype=torch.float16, lim=1):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-lim, lim + 1, shape, device="cuda", generator=gen, dtype=torch.int8).to(dtype)


def _weight(hq, rows, K, seed):
    """A 4-bit weight of groups of 64 (two codes a byte, the even one below)."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    packed = torch.randint(0, 256, (rows * K // 2,), device="cuda", generator=gen, dtype=torch.uint8)
    s = 2.0 ** -torch.randint(3, 6, (rows, K // 64), device="cuda", generator=gen).half()
    z = torch.randint(0, 16, (rows, K // 64), device="cuda", generator=gen).half()
    return hq.QuantizedWeight(packed=packed, scale=s, zero=z, rows=rows, cols=K, nbits=4, group_size=64)


def _rows64(q, a, b):
    p = q.packed.view(q.rows, -1)[a:b]
    codes = torch.stack([p & 15, p >> 4], 2).view(b - a, q.cols).double()
    z = q.zero[a:b].double().repeat_interleave(64, 1)
    return q.scale[a:b].double().repeat_interleave(64, 1) * (codes - z)


def _probes(rows, width):
    """Rows at the start, around the 2^31st element and at the end."""
    mid = 2 ** 31 // width
    assert 200 < mid < rows - 200
    return torch.cat([torch.arange(50), torch.arange(mid - 100, mid + 100), torch.arange(rows - 100, rows)]).cuda()


@pytest.mark.parametrize("topk", [1, 2])
def test_rows_and_results_of_more_than_2_to_31_elements(hq, topk):
    E, N, K, T = 3, 16640, 64, 140000 // topk
    q = _weight(hq, E * N, K, 1)
    gen = torch.Generator(device="cuda").manual_seed(2)
    r = hq.expert_sort(torch.randint(0, E, (T, topk), device="cuda", generator=gen, dtype=torch.int32), E)
    X = _ints((T, K), 3)
    Y = hq.matmul_experts(X, q, r, out_f32=False)
    at = _probes(r.rows, N)
    expert = torch.searchsorted(r.offsets[1:].contiguous(), at.int(), right=True)
    W = [_rows64(q, e * N, (e + 1) * N) for e in range(E)]
    rows = X[(r.order[at] // topk).long()].double()
    for e in range(E):
        m = expert == e
        assert torch.equal(Y[at[m]].double(), rows[m] @ W[e].t().contiguous())
    back = hq.expert_combine(Y, r)  # gathered and combined behind 2^31 elements
    tokens = torch.arange(T - 60, T, device="cuda")
    want = sum(Y[r.position[tokens * topk + j].long()].float() for j in range(topk)).half()
    assert torch.equal(back[tokens], want)
    assert torch.equal(hq.expert_gather(back, r)[at], back[(r.order[at] // topk).long()])
    dX = hq.matmul_experts_backward(Y.clamp_(-1, 1).round_(), q, r, out_f32=True)
    for e in range(E):
        m = expert == e
        assert torch.equal(dX[at[m]].double(), Y[at[m]].double() @ W[e])


def test_inner_sizes_whose_rows_pass_2_to_31_elements(hq):
    E, N, K, M = 2, 40, 262144, 9000
    q = _weight(hq, E * N, K, 4)
    ids = (torch.arange(M, device="cuda", dtype=torch.int32) % E)
    r = hq.expert_sort(ids, E)
    X = _ints((M, K), 5)
    W = [_rows64(q, e * N, (e + 1) * N) for e in range(E)]
    at = _probes(M, K)
    Y = hq.matmul_experts(X, q, r, sorted_rows=True, out_f32=True)
    dY = _ints((M, N), 6)
    dX = hq.matmul_experts_backward(dY, q, r, out_f32=False)
    for e in range(E):
        rows = at[(at >= int(r.offsets[e])) & (at < int(r.offsets[e + 1]))]
        assert torch.equal(Y[rows].double(), X[rows].double() @ W[e].t().contiguous())
        assert torch.equal(dX[rows].double(), dY[rows].double() @ W[e])
    one = hq.QuantizedWeight(packed=q.packed[:N * K // 2], scale=q.scale[:N], zero=q.zero[:N], rows=N, cols=K,
                             nbits=4, group_size=64)
    assert torch.equal(hq.matmul_backward(dY, one)[at].double(), dY[at].double() @ W[0])


@pytest.mark.parametrize("M", [3, 8, 100, 600, 3000])
def test_experts_behind_the_2_to_31st_byte_of_codes(hq, M):
    E, N, K = 20, 16384, 16384
    q = _weight(hq, E * N, K, 7)
    assert q.packed.numel() > 2 ** 31 and E * N * K > 2 ** 32
    r = hq.expert_sort(torch.full((M,), E - 1, device="cuda", dtype=torch.int32), E)
    X, dY = _ints((M, K), 8), _ints((M, N), 9)
    W = _rows64(q, (E - 1) * N, E * N)
    some = torch.arange(min(M, 8), device="cuda") * (M // min(M, 8))
    Y, dX = hq.matmul_experts(X, q, r, out_f32=True), hq.matmul_experts_backward(dY, q, r, out_f32=True)
    assert torch.equal(Y[some].double(), X[some].double() @ W.t().contiguous())
    assert torch.equal(dX[some].double(), dY[some].double() @ W)


@pytest.mark.parametrize("M", [20, 100])
def test_adapters_behind_the_2_to_31st_element(hq, M):
    n, r, N, K = 600, 256, 16384, 16384
    t = dict(X=_ints((M, K), 1), A=_ints((n, r, K), 2), B=_ints((n, N, r), 3), ids=torch.full((M,), n - 1, device="cuda", dtype=torch.int32),
             scales=torch.full((n,), 0.5, device="cuda"))
    dY = _ints((M, N), 4)
    A, B = t["A"][n - 1].double(), t["B"][n - 1].double()
    v, u = t["X"].double() @ A.t().contiguous(), dY.double() @ B
    assert torch.equal(hq.adapters(**t, out_f32=True).double(), 0.5 * (v @ B.t().contiguous()))
    dX, dA, dB = hq.adapters_backward(dY, **t, out_f32=True)
    assert torch.equal(dX.double(), 0.5 * (u @ A))
    assert torch.equal(dA[n - 1].double(), 0.5 * (u.t().contiguous() @ t["X"].double()))
    assert torch.equal(dB[n - 1].double(), 0.5 * (dY.double().t().contiguous() @ v))
    assert not bool(dA[0].any()) and not bool(dB[n - 2].any())


def test_adapters_of_rows_of_more_than_2_to_31_elements(hq):
    M, N, K, r = 140000, 16384, 16640, 8
    ids = torch.arange(M, device="cuda", dtype=torch.int32) % 4 - 1
    t = dict(X=_ints((M, K), 1, torch.bfloat16), A=_ints((3, r, K), 2, torch.bfloat16),
             B=_ints((3, N, r), 3, torch.bfloat16), ids=ids, scales=torch.ones(3, device="cuda"))
    dY = _ints((M, N), 4, torch.bfloat16)
    Y = hq.adapters(**t, base=dY, out_f32=True)
    dX, dA, dB = hq.adapters_backward(dY, **t, base=t["X"], out_f32=True)
    at = torch.cat([_probes(M, N), _probes(M, K)])
    for a in range(3):
        A, B = t["A"][a].double(), t["B"][a].double()
        m = at[ids[at] == a]
        v, u = t["X"][m].double() @ A.t().contiguous(), dY[m].double() @ B
        assert torch.equal(Y[m].double(), dY[m].double() + v @ B.t().contiguous())
        assert torch.equal(dX[m].double(), t["X"][m].double() + u @ A)
        rows = torch.nonzero(ids == a)[:, 0]
        x, d = t["X"][rows].double(), dY[rows].double()
        # u and v up to about 2^12 in 24 bits, sums of 35000 products of integers: below 2^24 * 2^4
        # in magnitude, so fp32 sums may round: 40000 of them, half a unit of the magnitude each
        for got, want, mag in ((dA[a], (d @ B).t().contiguous() @ x, (d @ B).abs().t().contiguous() @ x.abs()),
                               (dB[a], d.t().contiguous() @ (x @ A.t().contiguous()),
                                d.abs().t().contiguous() @ (x @ A.t().contiguous()).abs())):
            assert bool(((got.double() - want).abs() <= (3 * len(rows) + 8) * 2.0 ** -24 * mag).all())
    none = at[ids[at] < 0]
    assert torch.equal(Y[none], dY[none].float()) and torch.equal(dX[none], t["X"][none].float())


@pytest.mark.parametrize("nbits", [3, 4])
@pytest.mark.parametrize("rows", [2, 40, 400])
def test_products_over_nothing_are_zeros(hq, nbits, rows):
    """K = 0 (no inner size) and, for the gradient, N = 0."""
    empty = dict(packed=torch.empty(0, dtype=torch.uint8, device="cuda"), nbits=nbits, group_size=64)
    half = dict(dtype=torch.float16, device="cuda")
    r = hq.expert_sort(torch.arange(rows, device="cuda", dtype=torch.int32) % 3, 2)
    q = hq.QuantizedWeight(scale=torch.empty((60, 0), **half), zero=torch.empty((60, 0), **half), rows=60, cols=0, **empty)
    for out_f32 in (False, True):
        dt = torch.float32 if out_f32 else torch.float16
        y = torch.full((rows, 30), float("nan"), dtype=dt, device="cuda")
        assert hq.matmul_experts(torch.empty((rows, 0), **half), q, r, out_f32=out_f32, out=y) is y
        assert not bool(y.ne(0).any())
        q0 = hq.QuantizedWeight(scale=torch.empty((0, 2), **half), zero=torch.empty((0, 2), **half), rows=0, cols=128, **empty)
        x = torch.full((rows, 128), float("nan"), dtype=dt, device="cuda")
        assert not bool(hq.matmul_experts_backward(torch.empty((rows, 0), **half), q0, r, out_f32=out_f32, out=x).ne(0).any())
        x.fill_(float("nan"))
        assert not bool(hq.matmul_backward(torch.empty((rows, 0), **half), q0, out_f32=out_f32, out=x).ne(0).any())
