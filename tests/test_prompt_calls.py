"""What the bindings of the prompt calls do around the library: which stream a
workspace belongs to, sizes past the library's 32 bits, a prefill that fails.
The library and the tensors' addresses are stand-ins, so nothing is launched."""
import contextlib
from types import SimpleNamespace

import pytest
import torch

from hybrid_model_ssm_replay_b200 import rssm, stage


@pytest.fixture
def calls(monkeypatch):
    """Stand-ins for the library (every call answers OK and is recorded) and
    for the checks that need a device."""
    done = []

    class Lib:
        def __getattr__(self, name):
            def call(*args):
                done.append((name, args))
                return 4096 if name.endswith("_bytes") else 0
            return call
    monkeypatch.setattr(rssm, "lib", Lib)
    monkeypatch.setattr(stage, "_lib", Lib)
    monkeypatch.setattr(rssm, "_device", lambda t, name: 0)
    monkeypatch.setattr(rssm, "_arg", lambda t, *a: None if t is None else 0x1000)
    monkeypatch.setattr(rssm, "_stream", lambda stream=None: None)
    return done


def layer(**kw):
    base = dict(batch=1, nheads=2, head_dim=64, d_state=128, ngroups=1)
    base.update(kw)
    return SimpleNamespace(desc=rssm.make_desc(**base), struct=rssm.StateStruct(),
                           pos=SimpleNamespace(get_device=lambda: 0, device="cuda:0"))


@pytest.mark.parametrize("stream", [None, SimpleNamespace(cuda_stream=7)], ids=["current", "side"])
def test_workspace_belongs_to_the_stream_that_uses_it(calls, monkeypatch, stream):
    """Memory freed on one stream may still be at work there: a call on another
    stream may only take memory of its own stream."""
    current, taken = [None], []

    @contextlib.contextmanager
    def on(s):
        current.append(s)
        yield
        current.pop()

    def empty(n, **kw):
        taken.append(current[-1])
        return SimpleNamespace(numel=lambda: n, record_stream=lambda s: None)
    monkeypatch.setattr(torch.cuda, "stream", on)
    x = torch.zeros(4, 2, 64)
    monkeypatch.setattr(torch, "empty", empty)
    rssm.rssm_prefill_scan(layer(), x, 4, x, x, x, x, x, x, x, stream=stream)
    assert taken == [stream] and current == [None]
    assert [name for name, _ in calls] == ["rssm_prefill_scan_workspace_bytes", "rssm_prefill_scan"]


@pytest.mark.parametrize("n", [1 << 31, (1 << 32) + 3])
def test_sizes_past_32_bits_are_refused(calls, n):
    """Not taken modulo 2^32: 2^32 + 3 rows are not three rows."""
    t = lambda *s, dtype=torch.bfloat16: torch.empty(s, dtype=dtype, device="meta")
    d = layer(head_dim=1, nheads=1, d_state=16).desc
    w = t(1)
    for call in (lambda: stage.rssm_stage_add_norm(t(n, 1), t(n, 1), w, 1e-5, t(n, 1)),
                 lambda: stage.rssm_stage_add_norm(t(1, n), None, w, 1e-5, t(1, n)),
                 lambda: stage.rssm_stage_gate_norm_prompt(d, t(n, 1), t(n, 35), w, 1e-5, t(n, 1)),
                 lambda: stage.rssm_stage_conv_prompt(d, w, t(n, 35), w, w, w, w, w, w, w, w),
                 lambda: rssm.rssm_prefill_scan(layer(), w, 1, t(n, 2, 64), w, w, w, w, w, w)):
        with pytest.raises(ValueError, match="rows|wide"):
            call()
    assert not calls


def test_any_bound_on_the_lengths_is_taken(calls):
    """A bound past 32 bits still bounds every length."""
    x = torch.zeros(4, 2, 64)
    rssm.rssm_prefill_scan(layer(), x, (1 << 32) + 1, x, x, x, x, x, x, x, workspace=x)
    (name, args), = calls
    assert name == "rssm_prefill_scan" and args[2:4] == (4, (1 << 31) - 1)


class Stop(Exception):
    pass


def bare_stage(monkeypatch, t):
    """A stage after t decoded tokens whose prefill flushes and then fails, as
    one without memory for its buffers does; returns it, the flushes it makes
    and the residual streams that its first norm gets."""
    s, flushes, streams = stage.HybridStage.__new__(stage.HybridStage), [], []
    s.shape, s.scheme, s.t, s.t0 = stage.StageShape(2, 64, 4, 16, 16, 1, n_ssm=1, n_attn=0), "replay", t, 0
    s.blocks, s.attn, s.ssm = [{"A": None, "norm": torch.ones(64)}], [], [{"state": None}]

    def norm(u, *args):
        streams.append(u)
        raise Stop
    monkeypatch.setattr(rssm, "rssm_flush", lambda st, A, force=False: flushes.append(force))
    monkeypatch.setattr(stage, "rssm_stage_add_norm", norm)
    return s, flushes, streams


def test_intervals_count_from_the_prefills_flush(monkeypatch):
    """A prefill folds what is buffered first. Where it fails after that,
    decoding goes on, and its intervals count from the empty buffer."""
    s, flushes, _ = bare_stage(monkeypatch, 5)
    with pytest.raises(Stop):
        s.prefill(torch.zeros(2, 3, 64, dtype=torch.bfloat16))
    assert flushes == [True] and s.t == s.t0 == 5


@pytest.mark.parametrize("layout", ["transposed", "columns first", "every second column", "strided rows"])
def test_prefill_takes_any_strides(monkeypatch, layout):
    """The kernels need dense rows: prefill makes them of any tensor, and
    leaves the caller's as it is."""
    s, _, streams = bare_stage(monkeypatch, 0)
    g = torch.Generator().manual_seed(1)
    rn = lambda *size: torch.randn(*size, generator=g).to(torch.bfloat16)
    u = {"transposed": lambda: rn(3, 2, 64).transpose(0, 1), "columns first": lambda: rn(64, 2, 3).permute(1, 2, 0),
         "every second column": lambda: rn(2, 3, 128)[..., ::2], "strided rows": lambda: rn(2, 3, 128)[..., :64]}[layout]()
    with pytest.raises(Stop):
        s.prefill(u)
    (got,) = streams
    assert got.is_contiguous() and torch.equal(got.view(2, 3, 64), u) and got.data_ptr() != u.data_ptr()
