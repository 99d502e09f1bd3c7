"""Arguments the language-model calls refuse or have to read with care."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sg():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import fp32_sgemm_gb300 as m
    m.build()
    m.load_library()
    return m


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32], ids=["bf16", "f16", "f32"])
def test_broadcast_rows_are_refused(sg, dtype):
    # All rows one and the same memory, of one column (row stride 0, which is
    # not below a row's length by itself) and of more.
    T, G = 40, 3
    ends = torch.tensor([10, 10, T], dtype=torch.int32, device="cuda")
    target = torch.zeros(T, dtype=torch.int64, device="cuda")
    row = torch.zeros(T, device="cuda")
    for n in (1, 8):
        def full(*shape):
            return torch.ones(*shape, dtype=dtype, device="cuda")
        rows, w, tall = full(1, n).expand(T, n), full(G, n, 5), full(1, 1, n).expand(G, 7, n)
        with pytest.raises(ValueError):
            sg.grouped_gemm(rows, w, ends)
        with pytest.raises(ValueError):
            sg.grouped_gemm(full(T, 7), tall, ends)
        with pytest.raises(ValueError):
            sg.grouped_gemm(full(T, n), full(G, 1, n).expand(G, 7, n), ends, trans_w=True)
        with pytest.raises(ValueError):
            sg.grouped_gemm(full(T, 4), full(G, 4, n), ends, out=rows)
        with pytest.raises(ValueError):
            sg.grouped_gemm_weight_grad(rows, full(T, 6), ends)
        with pytest.raises(ValueError):
            sg.grouped_gemm_weight_grad(full(T, 6), rows, ends)
        with pytest.raises(ValueError):
            sg.grouped_gemm_weight_grad(full(T, 7), full(T, n), ends, out=tall)
        with pytest.raises(ValueError):
            sg.linear_cross_entropy(rows, full(9, n), target)
        with pytest.raises(ValueError):
            sg.linear_cross_entropy(full(T, n), full(1, n).expand(9, n), target)
        with pytest.raises(ValueError):
            sg.linear_cross_entropy_grad(rows, full(9, n), target, row, row)
    q = torch.zeros(6, 32, dtype=torch.uint8, device="cuda")
    x, scales = full(T, 64), full(1, 1).expand(6, 1)
    with pytest.raises(ValueError):
        sg.w4_gemm(x, q, scales)
    with pytest.raises(ValueError):
        sg.w4_gemm(x, q, full(6, 1), torch.zeros(1, 1, dtype=torch.uint8, device="cuda").expand(6, 1))
    with pytest.raises(ValueError):
        sg.w4_gemm(x, q[:1], full(1, 1), out=full(1, 1).expand(T, 1))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_one_column_with_a_pitch(sg, dtype):
    # One column of a wider matrix: its rows lie a pitch apart.
    T = 40
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randint(-3, 4, (T, 9), generator=g, device="cuda").to(dtype)[:, 4:5]
    w = torch.randint(-3, 4, (2, 1, 6), generator=g, device="cuda").to(dtype)
    ends = torch.tensor([15, T], dtype=torch.int32, device="cuda")
    want = torch.cat((x[:15].double() @ w[0].double(), x[15:].double() @ w[1].double()))
    assert torch.equal(sg.grouped_gemm(x, w, ends).double(), want)


def test_broadcast_rows_of_an_fp32_product_are_refused(sg):
    full = torch.ones(40, 40, device="cuda")
    for rows in (torch.ones(1, 40, device="cuda").expand(40, 40), full.as_strided((40, 40), (8, 1))):
        with pytest.raises(ValueError):
            sg.sgemm(rows, full)
        with pytest.raises(ValueError):
            sg.sgemm(full, rows)
        with pytest.raises(ValueError):
            sg.sgemm(full, full, rows)
    assert (sg.sgemm(torch.ones(1, 40, device="cuda"), full) == 40).all()


def test_a_flag_without_a_truth_value_raises_its_own_error(sg):
    x, w = torch.ones(8, 16, device="cuda"), torch.ones(1, 16, 16, device="cuda")
    ends = torch.tensor([8], dtype=torch.int32, device="cuda")
    two = torch.ones(2)
    with pytest.raises(RuntimeError, match="ambiguous"):
        sg.grouped_gemm(x, w, ends, trans_w=two)
    with pytest.raises(RuntimeError, match="ambiguous"):
        sg.grouped_gemm_weight_grad(x, x, ends, trans_w=two)


def test_what_does_not_fit_raises_torchs_own_error(sg):
    # 1024 gradients of 65536 x 65536: nothing is launched.
    x = torch.zeros(8, 65536, dtype=torch.bfloat16, device="cuda")
    ends = torch.full((1024,), 8, dtype=torch.int32, device="cuda")
    with pytest.raises(torch.OutOfMemoryError):
        sg.grouped_gemm_weight_grad(x, x, ends)
    # (An operand that fits, and the three planes of it that do not.)
    free = torch.cuda.mem_get_info()[0]
    rows = int(free * 0.55) // (4 * 65537)
    w = torch.empty(rows, 65537, device="cuda")
    target = torch.zeros(8, dtype=torch.int64, device="cuda")
    with pytest.raises(torch.OutOfMemoryError):
        sg.linear_cross_entropy(torch.zeros(8, 65537, device="cuda"), w, target)
    del w
    torch.cuda.empty_cache()
