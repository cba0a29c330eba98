"""``PagedAttnStep`` with ``StepIO`` on the GPU: bound outputs, late inputs,
captured steps, and timing events inside a capture."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU machines
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import prefill_csa_compress_gb300 as csa  # noqa: E402
from prefill_csa_compress_gb300.pipeline import PagedAttnStep, StepChain, StepIO  # noqa: E402

from test_gpu_paged import DEV, _bf, _i32  # noqa: E402

HQ, HK, DIM, CTX = 8, 2, 128, 300
INPUTS = ["q", "k", "v", "row_req", "row_pos", "kv_len"]


def _tensors(rng, n, pools):
    cos, sin = torch.empty((512, DIM // 2), device=DEV), torch.empty((512, DIM // 2), device=DEV)
    csa.csa_rope_table(cos=cos, sin=sin)
    return dict(q=_bf(rng, n, HQ, DIM), k=_bf(rng, n, HK, DIM), v=_bf(rng, n, HK, DIM), row_req=_i32([0] * n),
                row_pos=_i32(np.arange(CTX, CTX + n)), kv_len=_i32([CTX + n]), k_pool=pools[0].clone(),
                v_pool=pools[1].clone(), kv_table=_i32([[1, 4, 0]]), rope_cos=cos, rope_sin=sin,
                q_gamma=_bf(rng, DIM), k_gamma=_bf(rng, DIM), sink=torch.zeros(HQ, device=DEV))


def _pools(rng):
    return [_bf(rng, 5, 128, HK, DIM) for _ in range(2)]


def _plain(t):
    """out and lse of the step on its own tensors, its caches left as they were."""
    t = {**t, "k_pool": t["k_pool"].clone(), "v_pool": t["v_pool"].clone()}
    step = PagedAttnStep(t)
    step.run()
    torch.cuda.synchronize()
    assert int(step.status.item()) == 0
    return step.out.clone(), step.lse.clone()


def _host(io, step):
    nb = step.out.numel() * 2
    at = io._span(step.out)
    out = io.host_out[:nb].view(torch.bfloat16).view(step.out.shape)
    return out, io.host_out[at:at + step.lse.numel() * 4].view(torch.float32).view(step.lse.shape)


@pytest.mark.parametrize("late", [(), ("q",), ("q", "k", "v")])
@pytest.mark.parametrize("chained", [False, True])
@pytest.mark.parametrize("ran_before", [False, True])
def test_step_io_round_trip(late, chained, ran_before):
    """New host inputs, one captured step, host outputs: those of the step run
    alone on the same inputs, over and over."""
    rng = np.random.default_rng(3)
    n = 5
    t = _tensors(rng, n, _pools(rng))
    step = PagedAttnStep(t)
    whole = StepChain([step]) if chained else step
    if ran_before:
        whole.run()
    io = StepIO(t, INPUTS, late=late).bind_outputs(whole)
    whole.run()  # (eagerly, on the tensors that are bound now)
    graph = io.capture(whole)
    for i in range(4):
        new = {"q": _bf(rng, n, HQ, DIM), "k": _bf(rng, n, HK, DIM), "v": _bf(rng, n, HK, DIM),
               "row_req": _i32([0] * n), "row_pos": _i32(np.arange(CTX - i, CTX - i + n)),
               "kv_len": _i32([CTX - i + n])}
        for k, x in new.items():
            io.host_input(k, x).copy_(x)
        want = _plain({**t, **new})
        step.out.fill_(7)
        step.lse.fill_(7)
        io.host_out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(step.out, want[0]) and torch.equal(step.lse, want[1])
        out, lse = _host(io, step)
        assert torch.equal(out, want[0].cpu()) and torch.equal(lse, want[1].cpu())
    assert int(step.status.item()) == 0


@pytest.mark.parametrize("kernel", ["norm_rope", "kv_append", "paged_attn", "paged_merge"])
@pytest.mark.parametrize("chained", [False, True])
def test_timed_capture(kernel, chained):
    """A step captured while one of its kernels is timed, alone and as a chain's
    last layer: the capture ends well, and the events can be read."""
    rng = np.random.default_rng(4)
    t = _tensors(rng, 3, _pools(rng))
    want = _plain(t)
    step = PagedAttnStep(t)
    whole = StepChain([PagedAttnStep({**t, "k_pool": t["k_pool"].clone(), "v_pool": t["v_pool"].clone()}), step]) \
        if chained else step
    whole.run()
    torch.cuda.synchronize()
    csa.prof_enable(kernel, 8)
    try:
        whole.capture()
        whole.replay()
        torch.cuda.synchronize()
        ms, launches = csa.prof_read(kernel)
        assert launches == (2 if chained else 1) and ms > 0
    finally:
        whole.drop_graph()
        csa.prof_disable()
    assert torch.equal(step.out, want[0]) and torch.equal(step.lse, want[1])


def _csa():
    from prefill_csa_compress_gb300.pipeline import CsaStep
    from workloads import make_workload, spec_for

    spec = spec_for("tiny_decode", seed=5)
    t = make_workload(spec).to(DEV)
    return t, lambda: CsaStep(t, spec.ratio, spec.topk), ["q", "row_req", "row_pos", "kv_len"]


def _paged():
    rng = np.random.default_rng(5)
    t = _tensors(rng, 4, _pools(rng))
    return t, lambda: PagedAttnStep(t), INPUTS


@pytest.mark.parametrize("kind", [_csa, _paged])
@pytest.mark.parametrize("late", [(), ("q",)])
@pytest.mark.parametrize("chained", [False, True])
def test_eager_run_after_a_capture(kind, late, chained):
    """A step whose graph waits for late inputs still runs by itself, and its
    graph still replays afterwards."""
    t, make, inputs = kind()
    step = make()
    whole = StepChain([step]) if chained else step
    io = StepIO(t, inputs, late=late).bind_outputs(whole)
    whole.run()
    torch.cuda.synchronize()
    want = step.out.clone(), step.lse.clone()
    graph = io.capture(whole)
    for run in (whole.run, graph.replay, whole.run):
        step.out.fill_(7)
        run()
        torch.cuda.synchronize()
        assert torch.equal(step.out, want[0]) and torch.equal(step.lse, want[1])
    assert int(step.status.item()) == 0
