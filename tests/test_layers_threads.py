"""Operators around the products called by several host threads at once, each with its own
stream and plan: the same bits as alone."""
import threading

import pytest
import torch

import dense_gemm_epilogues_gb300 as G

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    G.load_library()


def _run_together(works):
    errors = []

    def guard(work):
        try:
            work()
        except Exception as e:   # (a thread's exception would only be printed)
            errors.append(e)

    threads = [threading.Thread(target=guard, args=(w,)) for w in works]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors[0]


# Numbers of experts that share a kernel and differ in its shared memory (up to 48 KB and beyond).
# The C entry point is called in a row, so that the threads are in it together most of the time.
@pytest.mark.parametrize("experts", [(512, 384), (1024, 600, 513), (360, 512, 1024, 64)], ids=str)
def test_routings_of_several_numbers_of_experts(experts):
    gen = torch.Generator("cuda").manual_seed(1)
    logits = [torch.randn((20, e), device="cuda", generator=gen) for e in experts]
    want = [G.route(z, 4) for z in logits]
    got = [G.route(z, 4) for z in logits]
    plans = [G.Plan(G.GEMM_F32, G.GEMM_F32) for _ in experts]
    streams = [torch.cuda.Stream() for _ in experts]
    torch.cuda.synchronize()
    start = threading.Barrier(len(experts))

    def work(i):
        r, z = got[i], logits[i]
        c = G.gemm_routing_t(*(t.data_ptr() for t in r[:7]), 4, 1)
        call, args = G.load_library().gemm_route, (plans[i].handle, 20, experts[i], z.data_ptr(), experts[i], None, c, streams[i].cuda_stream)
        start.wait()
        for turn in range(60):
            status = {call(*args) for _ in range(500)}
            assert status == {0}, (experts[i], turn, status)
            streams[i].synchronize()

    _run_together([lambda i=i: work(i) for i in range(len(experts))])
    for a, b in zip(got, want):
        assert all(torch.equal(u, v) for u, v in zip(a[:7], b[:7]))
    assert all(p.device_status() == 0 for p in plans)


def test_all_operators():
    """A layer's calls without plans in four threads."""
    def data(i):
        gen = torch.Generator("cuda").manual_seed(i)
        rand = lambda *s: torch.randn(s, device="cuda", generator=gen).bfloat16()   # noqa: E731
        return rand(70 + 50 * i, 131), rand(131, 260), rand(70 + 50 * i, 260), torch.randn((70 + 50 * i, 100 * (i + 1)), device="cuda", generator=gen)

    sets = [data(i) for i in range(4)]

    def step(x, w, dy, z):
        y, pre = G.linear(x, w, activation="gelu", save_pre=True)
        dx, dw, db = G.linear_grad(dy, x, w, activation="gelu", pre=pre)
        r = G.route(z, 3)
        rows = G.dispatch(x, r)
        out = G.combine(rows, r, residual=x)
        d, dweights = G.combine_grad(x, rows, r)
        dz = G.route_grad(z, r, dweights=dweights, dloss=0.1)
        return [y, dx, dw, db, out, d, dweights, dz, G.clip_grad_norm([dw, db], 0.5), r.loss]

    want = [step(*s) for s in sets]
    torch.cuda.synchronize()
    got = [None] * 4

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                got[i] = step(*sets[i])
            torch.cuda.current_stream().synchronize()

    _run_together([lambda i=i: work(i) for i in range(4)])
    for a, b in zip(got, want):
        assert all(torch.equal(u, v) for u, v in zip(a, b))
    assert G.default_plan_status() == 0
