"""Calls without a handle of their own on several streams, from several threads
and in graphs: none may use another's workspace."""
import threading

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


def _work(sg, seed, dtype, rows):
    """A closure over inputs of its own: every operator that takes a
    workspace."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rand(*shape):
        return (torch.randn(*shape, generator=g, device="cuda") * shape[-1] ** -0.5).to(dtype)
    x, head, w, dy = rand(rows, 520), rand(3001, 520), rand(3, 520, 260), rand(rows, 260)
    xo, wo = rand(rows, 521)[:, :517], rand(3, 517, 131)          # (copied: TMA cannot address them)
    ends = torch.tensor([rows // 3, rows // 2, rows], dtype=torch.int32, device="cuda")
    target = torch.randint(0, 3001, (rows,), generator=g, device="cuda")
    dloss = torch.full((rows,), 1.0 / rows, device="cuda")
    q = torch.randint(0, 256, (64, 32768), generator=g, device="cuda", dtype=torch.uint8)
    scales, x4 = rand(64, 512), rand(9, 65536)                    # (x beside the weights: K is cut)

    def run(**kw):
        loss, lse = sg.linear_cross_entropy(x, head, target, **kw)
        return [loss, lse, *sg.linear_cross_entropy_grad(x, head, target, lse, dloss, **kw),
                sg.grouped_gemm(x, w, ends, **kw), sg.grouped_gemm(xo, wo, ends, **kw),
                sg.grouped_gemm_weight_grad(x, dy, ends, **kw), sg.w4_gemm(x4, q, scales, **kw)]
    return run


def _same(a, b):
    return all(torch.equal(u, v) for u, v in zip(a, b))


@pytest.mark.parametrize("given", [False, True], ids=["current", "given"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_streams_side_by_side(sg, dtype, given):
    work = [_work(sg, i, dtype, rows) for i, rows in enumerate((300, 300, 100))]
    want = [w() for w in work]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in work]
    # All streams start together, behind a pause.
    for s in streams:
        with torch.cuda.stream(s):
            torch.cuda._sleep(20_000_000)
    got = [[] for _ in work]
    for _ in range(12):
        for i, (w, s) in enumerate(zip(work, streams)):
            if given:
                got[i].append(w(stream=s))
            else:
                with torch.cuda.stream(s):
                    got[i].append(w())
    torch.cuda.synchronize()
    for i in range(len(work)):
        assert all(_same(want[i], g) for g in got[i]), f"stream {i}"
    assert sg.default_handle().device_error() == 0


def test_threads_with_streams_of_their_own(sg):
    work = [_work(sg, i, torch.bfloat16, rows) for i, rows in enumerate((300, 40, 200, 300))]
    want = [w() for w in work]
    torch.cuda.synchronize()
    wrong, started = [], threading.Barrier(len(work))

    def go(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                started.wait(60)
                for _ in range(10):
                    got = work[i]()
                    torch.cuda.current_stream().synchronize()
                    if not _same(want[i], got):
                        wrong.append(i)
        except Exception as e:                                    # reported by the assertion below
            wrong.append(e)
    threads = [threading.Thread(target=go, args=(i,)) for i in range(len(work))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


@pytest.mark.parametrize("own", [False, True], ids=["default", "handle"])
def test_a_graph_beside_other_calls(sg, own):
    # The captured calls' workspace stays theirs: larger calls later, memory
    # taken and filled in between, replays beside calls on another stream.
    h = sg.Handle() if own else None
    small, large = _work(sg, 1, torch.bfloat16, 60), _work(sg, 2, torch.bfloat16, 900)
    want_small, want_large = small(handle=h), large(handle=h)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = small(handle=h)
    assert _same(large(handle=h), want_large)
    other = torch.cuda.Stream()
    for _ in range(4):
        for o in out:
            o.zero_()
        junk = [torch.full((1 << 22,), float("nan"), device="cuda") for _ in range(8)]
        other.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(other):
            beside = [large() for _ in range(3)]
        graph.replay()
        torch.cuda.synchronize()
        assert _same(out, want_small) and all(_same(b, want_large) for b in beside)
        del junk
    if own:
        h.close()
