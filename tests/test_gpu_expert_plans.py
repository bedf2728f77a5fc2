"""Plans of the expert-layer operators: the scratch that captured graphs keep, use on
other streams, and calls without a plan."""
import threading

import pytest
import torch

import dense_gemm_epilogues_gb300 as G
from expert_helpers import DT, check, offsets_of, q4_weights, random_q4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    G.load_library()


def _gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def _layer(E=4, counts=(30, 70, 0, 50), K=192, N=256, seed=3):
    gen = _gen(seed)
    off, R = offsets_of(counts), sum(counts)
    x = torch.randn((R, K), device="cuda", generator=gen).bfloat16()
    dy = torch.randn((R, N), device="cuda", generator=gen).bfloat16()
    w = torch.randn((E, K, N), device="cuda", generator=gen).bfloat16()
    return off, x, dy, w, random_q4(N, K, 64, DT["bf16"], True, gen, E)


def _calls(off, x, dy, w, q4, **kw):
    """One call of each operator; kw: plan of bf16 operands, if any."""
    q, s, z = q4
    return [lambda: G.grouped_matmul(x, w, off, **kw), lambda: G.grouped_weight_grad(x, dy, off, **kw),
            lambda: G.q4_matmul(x, q, s, 64, zeros=z, offsets=off, **kw), lambda: G.orthogonalize(w, **kw)]


def _grow(plan, seed):
    """Calls on the plan that need more scratch than _layer's, with values of their own."""
    gen = _gen(seed)
    x = torch.randn((300, 1024), device="cuda", generator=gen).bfloat16()
    q, s, z = random_q4(2048, 1024, 64, DT["bf16"], True, gen)
    G.q4_matmul(x, q, s, 64, zeros=z, plan=plan)
    G.orthogonalize(torch.randn((1200, 2048), device="cuda", generator=gen).bfloat16(), plan=plan)


def _odd_layer():
    """Operands that TMA cannot address: every operator needs scratch."""
    return _layer(K=190, N=251)


def _layer_of(kind):
    return {"even": _layer, "odd": _odd_layer}[kind]()


@pytest.mark.parametrize("kind", ["even", "odd"])
def test_graphs_survive_a_larger_call_on_their_plan(kind):
    """The scratch of captured calls stays when the plan grows: replays after larger calls on
    the plan, and on another one that would be given what it freed, agree with eager calls."""
    a = _layer_of(kind)
    plan, other = G.Plan(G.GEMM_BF16, G.GEMM_F32), G.Plan(G.GEMM_BF16, G.GEMM_F32)
    want = [c() for c in _calls(*a, plan=plan)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [c() for c in _calls(*a, plan=plan)]
    for turn in range(3):
        _grow(plan, 10 + turn)
        for c in _calls(*_layer(seed=20 + turn), plan=other):
            c()
        for t in got:
            t.zero_()
        graph.replay()
        for u, v in zip(got, want):
            assert torch.equal(u, v)
    for u, v in zip([c() for c in _calls(*a, plan=plan)], want):
        assert torch.equal(u, v)
    assert plan.device_status() == 0 and other.device_status() == 0


@pytest.mark.parametrize("kind", ["even", "odd"])
def test_a_plan_first_used_inside_a_capture(kind):
    """Its scratch is ordinary memory: eager calls before the first replay may use it, and it
    may grow within the capture."""
    a = _layer_of(kind)
    _grow(G.Plan(G.GEMM_BF16, G.GEMM_F32), 1)
    want = [c() for c in _calls(*a, plan=G.Plan(G.GEMM_BF16, G.GEMM_F32))]
    torch.cuda.synchronize()
    plan, graph = G.Plan(G.GEMM_BF16, G.GEMM_F32), torch.cuda.CUDAGraph()
    big = torch.randn((700, 900), device="cuda", generator=_gen(2)).bfloat16()
    with torch.cuda.graph(graph):
        got = [c() for c in _calls(*a, plan=plan)]
        up = G.orthogonalize(big, plan=plan)
    for u, v in zip([c() for c in _calls(*a, plan=plan)], want):
        assert torch.equal(u, v)
    for _ in range(2):
        graph.replay()
        for u, v in zip(got, want):
            assert torch.equal(u, v)
        assert torch.equal(up, G.orthogonalize(big, plan=plan))
        _grow(plan, 3)
    assert plan.device_status() == 0


def test_a_kept_plan_follows_its_stream():
    """Inputs that are written behind queued work on a side stream, with a kept plan (no call
    in between waits for the device)."""
    off, x, dy, w, q4 = _layer()
    plan = G.Plan(G.GEMM_BF16, G.GEMM_F32)
    want = [c() for c in _calls(off, x, dy, w, q4, plan=plan)]
    x2, dy2, w2 = torch.zeros_like(x), torch.zeros_like(dy), torch.zeros_like(w)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(500_000_000)
        for to, src in ((x2, x), (dy2, dy), (w2, w)):
            to.copy_(src)
        got, done = [c() for c in _calls(off, x2, dy2, w2, q4, plan=plan)], torch.cuda.Event()
        done.record()
    assert not done.query()
    side.synchronize()
    for u, v in zip(got, want):
        assert torch.equal(u, v)
    assert plan.device_status() == 0


def test_calls_without_a_plan_do_not_wait_for_the_device():
    """Work queued ahead on the stream is still running when such a call returns."""
    for call in _calls(*_layer()):
        want = call()
        torch.cuda.synchronize()
        torch.cuda._sleep(1_000_000_000)
        got, done = call(), torch.cuda.Event()
        done.record()
        assert not done.query()
        torch.cuda.synchronize()
        assert torch.equal(got, want)


def test_calls_without_a_plan_report_their_errors():
    off, x, dy, w, q4 = _layer()
    assert G.default_plan_status() == 0
    bad = torch.tensor([0, 30, 20, 100, 150], dtype=torch.int32, device="cuda")
    for call in _calls(bad, x, dy, w, q4)[:3]:
        call()
        assert G.default_plan_status() == G.GEMM_ERR_INVALID_ARG
        assert G.default_plan_status() == 0
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        G.grouped_matmul(x, w, bad)
    assert G.default_plan_status() == G.GEMM_ERR_INVALID_ARG


def test_calls_without_a_plan_on_several_streams_and_threads():
    """Every stream and thread has scratch of its own: calls that run together agree with
    calls one after the other."""
    layers = [_layer(seed=s) for s in range(4)]
    want = [[c() for c in _calls(*a)] for a in layers]
    torch.cuda.synchronize()
    got = [None] * 4

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(20):
                got[i] = [c() for c in _calls(*layers[i])]
        s.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for a, b in zip(want, got):
        for u, v in zip(a, b):
            assert torch.equal(u, v)
    assert G.default_plan_status() == 0


def test_calls_without_a_plan_inside_a_capture():
    """The first such call of a stream, too: its plan is made during the capture."""
    a = _layer()
    want = [c() for c in _calls(*a)]
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        got = [c() for c in _calls(*a)]
    for _ in range(2):
        graph.replay()
        for u, v in zip(got, want):
            assert torch.equal(u, v)
    with torch.cuda.stream(side):
        again = [c() for c in _calls(*a)]
    torch.cuda.synchronize()
    for u, v in zip(again, want):
        assert torch.equal(u, v)
    assert G.default_plan_status() == 0


def test_calls_without_a_plan_keep_one():
    from dense_gemm_epilogues_gb300 import expert
    a = _layer()
    for c in _calls(*a):
        c()
    made = len(expert._DEFAULTS)
    for c in _calls(*a):
        c()
    G.grouped_weight_grad(a[1], a[2], a[0], out_dtype=DT["f32"])
    assert len(expert._DEFAULTS) == made


def test_4_bit_products_without_memory_for_decoded_weights():
    """1024 experts that share 8192 x 20480 weights would decode into 343 GB: more than the
    device has, so the product decodes inside."""
    gen, E, N, K, R = _gen(5), 1024, 8192, 20480, 34 * 1024
    assert 2 * E * N * K > torch.cuda.get_device_properties(0).total_memory
    q, s, _ = random_q4(N, K, 128, DT["bf16"], False, gen)
    x = torch.zeros((R, K), device="cuda", dtype=DT["bf16"])
    x[:40] = torch.randn((40, K), device="cuda", generator=gen).bfloat16()
    off = torch.full((E + 1,), 40, dtype=torch.int32, device="cuda")
    off[:6] = 0
    plan = G.Plan(G.GEMM_BF16, G.GEMM_F32)
    y = G.q4_matmul(x, q.expand(E, -1, -1), s.expand(E, -1, -1), 128, offsets=off, out_dtype=DT["f32"], plan=plan)
    assert plan.device_status() == 0
    w = q4_weights(q[:500], s[:500], None, K, 128)
    v = x[:40].double()
    check(y[:40, :500], v @ w.mT, v.abs() @ w.abs().mT, K, "f32")
    for c in _calls(*_layer(), plan=plan):   # the plan is as good as before
        c()
    assert plan.device_status() == 0


def test_a_plan_in_threads_that_use_cuda_for_the_first_time():
    """A plan and memory that the main thread made: the call is the new thread's first."""
    a = _layer()
    plan, b = G.Plan(G.GEMM_BF16, G.GEMM_F32), a[3][0]
    big = torch.randn((4096, 4096), device="cuda", generator=_gen(1)).bfloat16()

    def diagonal():
        d = torch.empty((4096, 4096), device="cuda")
        G.gemm_run_diag(plan.handle, G.GEMM_SIDE_LEFT, G.GEMM_OP_T, 4096, 4096, 1.0, big.data_ptr(), big.data_ptr(), 4096,
                        0.0, None, 0, d.data_ptr(), 4096)
        return d

    calls = _calls(*a, plan=plan) + [lambda: G.matmul(a[1], b, plan=plan), diagonal]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    for call, out in zip(calls, want):
        got = []
        t = threading.Thread(target=lambda: got.append(call()))
        t.start()
        t.join()
        torch.cuda.synchronize()
        assert len(got) == 1 and torch.equal(got[0], out)
    assert plan.device_status() == 0


def test_threads_that_end_leave_their_plans_to_others():
    from dense_gemm_epilogues_gb300 import expert
    a = _layer()
    want = [c() for c in _calls(*a)]
    got = []

    def work():
        got.append([c() for c in _calls(*a)])

    def one():
        t = threading.Thread(target=work)
        t.start()
        t.join()

    one()
    made = len(expert._DEFAULTS)
    for _ in range(5):
        one()
    assert len(expert._DEFAULTS) == made and len(got) == 6
    for out in got:
        for u, v in zip(out, want):
            assert torch.equal(u, v)
