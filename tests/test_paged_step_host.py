"""``PagedAttnStep`` and ``StepIO`` on the host (no GPU): which tensors the
step's calls get, and in what order they are made.  The calls themselves are
stood in for by recorders."""

import pytest
import torch

from prefill_csa_compress_gb300 import pipeline as PL

NAMES = ("csa_qk_norm_rope", "csa_kv_append", "csa_paged_attn")


class _HostTorch:
    """torch without pinned memory, which needs a GPU."""

    def __getattr__(self, name):
        return getattr(torch, name)

    @staticmethod
    def empty(*a, pin_memory=False, **k):
        return torch.empty(*a, **k)


@pytest.fixture
def log(monkeypatch):
    """(name, arguments, stream) of every call made, in order."""
    made = []

    def recorder(name):
        def call(*, stream=None, prepare=False, **kw):
            ws = "workspace" if name == "csa_paged_attn" else None
            if prepare:
                return lambda stream=None: made.append((name, kw, stream)) or ws
            made.append((name, kw, stream))
            return ws

        return call

    for n in NAMES:
        monkeypatch.setattr(PL.P, n, recorder(n))
    monkeypatch.setattr(PL.B, "prof_join", lambda stream=None: made.append(("prof_join", {}, stream)))
    monkeypatch.setattr(PL, "torch", _HostTorch())
    return made


def tensors(n=3, hq=4, hk=2, dim=64):
    i32, bf16 = dict(dtype=torch.int32), dict(dtype=torch.bfloat16)
    return dict(q=torch.zeros(n, hq, dim, **bf16), k=torch.zeros(n, hk, dim, **bf16),
                v=torch.zeros(n, hk, dim, **bf16), row_req=torch.zeros(n, **i32),
                row_pos=torch.arange(n, **i32), kv_len=torch.tensor([n], **i32),
                k_pool=torch.zeros(1, 128, hk, dim, **bf16), v_pool=torch.zeros(1, 128, hk, dim, **bf16),
                kv_table=torch.zeros(1, 1, **i32), rope_cos=torch.ones(n, dim // 2),
                rope_sin=torch.zeros(n, dim // 2), sink=torch.zeros(hq))


INPUTS = ["q", "k", "v", "row_req", "row_pos", "kv_len"]


def check_tensors(log, t, step):
    calls = {name: kw for name, kw, _ in log if name in NAMES}
    assert list(calls) == list(NAMES) and len([e for e in log if e[0] in NAMES]) == 3
    norm, append, attn = (calls[n] for n in NAMES)
    assert norm["q"] is t["q"] and append["k"] is t["k"] and append["v"] is t["v"]
    assert norm["q_out"] is attn["q"]
    for kw in (norm, append, attn):
        assert kw["row_pos"] is t["row_pos"] and kw["row_req"] is t["row_req"]
        assert kw["status"] is step.status
    assert attn["kv_len"] is t["kv_len"] and attn["out"] is step.out and attn["lse"] is step.lse
    for name in ("k_pool", "v_pool"):
        assert append[name] is t[name] and attn[name] is t[name]


@pytest.mark.parametrize("chained", [False, True])
@pytest.mark.parametrize("ran_before", [False, True])
@pytest.mark.parametrize("prepared", [False, True])
def test_step_takes_what_step_io_binds(log, chained, ran_before, prepared):
    """Inputs and outputs that StepIO puts in the place of a step's own, after
    the step was built and run: its calls get those."""
    t = tensors()
    step = PL.PagedAttnStep(t)
    whole = PL.StepChain([step]) if chained else step
    if ran_before:
        whole.run()
    own = step.out, step.lse
    io = PL.StepIO(t, INPUTS).bind_outputs(whole)
    assert step.out is not own[0] and step.lse is not own[1]
    assert step.out.data_ptr() == io.dev_out.data_ptr()
    if prepared:
        whole.prepare()
    log.clear()
    whole.run()
    check_tensors(log, t, step)
    assert t["q"].data_ptr() == io.dev_in.data_ptr()


def test_unprepared_step_runs_on_its_stream(log):
    """The stream reaches every call (the attention takes its workspace on
    it), and the next run is given the workspace back."""
    step = PL.PagedAttnStep(tensors(), window=7, causal=False, rope_layout="half", eps=1e-5)
    step.run("s")
    step.run("s")
    calls = [e for e in log if e[0] in NAMES]
    assert [e[0] for e in calls] == list(NAMES) * 2 and all(e[2] == "s" for e in calls)
    assert calls[2][1]["workspace"] is None and calls[5][1]["workspace"] == "workspace"
    assert calls[2][1]["window"] == 7 and calls[2][1]["causal"] is False
    for _, kw, _ in calls[:2]:
        assert kw["rope_layout"] == "half" and kw["eps"] == 1e-5


@pytest.mark.parametrize("prepared", [False, True])
def test_late_inputs_are_waited_for(log, prepared):
    """What StepIO sets to wait for late inputs is called once a run, on the
    run's stream, before anything reads an input."""
    step = PL.PagedAttnStep(tensors())
    if prepared:
        step.prepare()
    step.before_attention = lambda stream: log.append(("wait", {}, stream))
    for stream in (None, "s"):
        log.clear()
        step.run(stream)
        assert [e[0] for e in log if e[0] != "prof_join"] == ["wait", *NAMES] and log[0][2] == stream


@pytest.mark.parametrize("prepared", [False, True])
def test_timing_events_are_joined(log, prepared):
    """A run ends by joining the timing side stream, as a capture needs."""
    step = PL.PagedAttnStep(tensors())
    if prepared:
        step.prepare()
    step.run("s")
    assert [e[0] for e in log] == [*NAMES, "prof_join"] and log[-1][2] == "s"


def test_mode_reaches_the_attention(log):
    """The kernel that a caller asks for, where the choice by averages would go
    wrong (a chunk beside single tokens, a lone chunk in a table of many)."""
    for mode in (PL.B.CSA_MODE_AUTO, PL.B.CSA_MODE_DECODE, PL.B.CSA_MODE_PREFILL):
        log.clear()
        PL.PagedAttnStep(tensors(), mode=mode).run()
        assert [kw["mode"] for name, kw, _ in log if name == "csa_paged_attn"] == [mode]
    assert PL.PagedAttnStep(tensors()).mode == PL.B.CSA_MODE_AUTO
