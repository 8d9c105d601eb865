"""The prompt calls (rssm_prefill_scan, rssm_stage_conv_prompt,
rssm_stage_gate_norm_prompt, rssm_stage_add_norm) reject bad arguments on the
host, before any CUDA call."""
import ctypes as ct

import pytest
import torch

from hybrid_model_ssm_replay_b200 import rssm, stage

OK, INVALID, SHAPE, UNSUPPORTED, CAPACITY = 0, 1, 2, 3, 4
P = ct.c_void_p(0x1000)    # never touched: the calls below fail, or have nothing to do
ODD = ct.c_void_p(0x1008)  # not 16-byte aligned


@pytest.fixture(scope="module")
def L():
    from hybrid_model_ssm_replay_b200 import build
    build.build()
    return stage._lib()


def cfg(**kw):
    base = dict(batch=2, nheads=64, head_dim=64, d_state=128, ngroups=8)
    base.update(kw)
    return rssm.make_desc(**base)


def scan(L, d, st, total=4, longest=4, cu=P, x=P, ws=None, size=0, y=P):
    return L.rssm_prefill_scan(ct.byref(d), ct.byref(st) if st else None, total, longest, cu, x, P, P, P, P, P, y, ws,
                               size, None)


def test_scan_rejects_bad_arguments(L):
    st = rssm.StateStruct(*([0x1000] * 7))
    d = cfg()
    assert scan(L, d, None) == INVALID
    assert scan(L, d, st, total=-1) == INVALID
    assert scan(L, d, st, longest=-1) == INVALID
    assert scan(L, d, st, cu=None) == INVALID
    assert scan(L, d, st, x=None) == INVALID
    assert scan(L, d, st, x=ODD) == INVALID
    assert scan(L, d, st, y=ODD) == INVALID
    assert scan(L, cfg(d_state=100), st) == SHAPE
    assert scan(L, cfg(update_dtype=rssm.RSSM_BF16), st) == UNSUPPORTED
    assert scan(L, cfg(update_dtype=rssm.RSSM_F32, out_copy=rssm.RSSM_OUTCOPY_FP4), st) == UNSUPPORTED
    bad = rssm.StateStruct(*([0x1000] * 7))
    bad.pos = None
    assert scan(L, d, bad) == INVALID
    assert scan(L, d, st, total=0, x=None) == OK  # nothing to do


def test_scan_workspace(L):
    """A long prompt of few requests needs a workspace, a full batch none;
    one that is missing or too small is refused."""
    st = rssm.StateStruct(*([0x1000] * 7))
    ws = rssm.rssm_prefill_scan_workspace_bytes
    d = cfg(batch=1)
    assert ws(cfg(batch=256), 256 * 512, 512) == 0
    assert ws(d, 0, 0) == 0 and ws(cfg(d_state=100), 1 << 14, 1 << 14) == 0
    assert ws(d, 77, 77) == 0
    need = ws(d, 1 << 14, 1 << 14)
    assert need > 0
    assert scan(L, d, st, 1 << 14, 1 << 14) == INVALID
    assert scan(L, d, st, 1 << 14, 1 << 14, ws=P, size=need - 1) == CAPACITY
    assert scan(L, d, st, 1 << 14, 1 << 14, ws=ODD, size=need) == INVALID


def conv(L, d, total=4, cu=P, zx=P, state=P, w=P):
    return L.rssm_stage_conv_prompt(ct.byref(d), total, cu, zx, state, w, P, P, P, P, P, P, None, None)


def test_conv_prompt_rejects_bad_arguments(L):
    d = cfg()
    assert L.rssm_stage_conv_prompt(None, 4, P, P, P, P, P, P, P, P, P, P, None, None) == INVALID
    assert conv(L, d, total=-1) == INVALID
    assert conv(L, d, cu=None) == INVALID
    assert conv(L, d, zx=None) == INVALID
    assert conv(L, d, state=None) == INVALID
    assert conv(L, d, w=ODD) == INVALID
    assert conv(L, cfg(in_dtype=rssm.RSSM_F32)) == UNSUPPORTED
    assert conv(L, cfg(nheads=63)) == SHAPE
    assert conv(L, d, total=0, zx=None) == OK


def test_gate_norm_prompt_rejects_bad_arguments(L):
    def call(d, rows=4, y=P, w=P, eps=1e-5):
        return L.rssm_stage_gate_norm_prompt(ct.byref(d), rows, y, P, w, ct.c_float(eps), P, None)
    d = cfg()
    assert call(d, rows=-1) == INVALID
    assert call(d, y=None) == INVALID
    assert call(d, w=ODD) == INVALID
    assert call(d, eps=0.0) == INVALID and call(d, eps=float("nan")) == INVALID
    assert call(cfg(in_dtype=rssm.RSSM_F32)) == UNSUPPORTED
    assert call(d, rows=0) == OK


def test_add_norm_rejects_bad_arguments(L):
    def call(rows=4, dim=64, t=1, u=P, v=P, pw=None, g=None, scale=1.0, w=P, eps=1e-5, uo=P, out=P):
        return L.rssm_stage_add_norm(rows, dim, t, u, v, pw, g, ct.c_float(scale), w, ct.c_float(eps), uo, out, None)
    assert call(rows=-1) == INVALID
    assert call(dim=0) == SHAPE and call(dim=16385) == SHAPE
    assert call(t=2) == INVALID
    assert call(u=None) == INVALID
    assert call(uo=None) == INVALID            # v is added, nowhere to keep the sum
    assert call(w=None) == INVALID and call(out=None) == INVALID  # a norm needs both
    assert call(scale=float("inf")) == INVALID and call(scale=float("nan")) == INVALID
    assert call(eps=-1.0) == INVALID
    assert call(pw=ODD) == INVALID and call(u=ODD) == INVALID
    assert call(rows=0) == OK


def test_bindings_refuse_cpu_tensors_and_wrong_types():
    t = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        stage.rssm_stage_add_norm(t, t.bfloat16(), t[0], 1e-5, t.bfloat16())
    with pytest.raises(ValueError):
        rssm._arg(t, torch.float32, (4, 8), "t", 0)


def test_stage_prefill_needs_the_replay_scheme():
    """Checked before anything runs: an object without state is enough."""
    s = stage.HybridStage.__new__(stage.HybridStage)
    s.shape = stage.StageShape(2, 64, 4, 16, 16, 1, ctx=8)
    s.scheme = "conventional"
    with pytest.raises(ValueError, match="replay"):
        s.prefill(torch.zeros(2, 3, 64, dtype=torch.bfloat16))
    s.scheme = "replay"
    with pytest.raises(ValueError, match="bf16"):
        s.prefill(torch.zeros(2, 3, 64))
    with pytest.raises(ValueError, match="cache"):
        s.prefill(torch.zeros(2, 9, 64, dtype=torch.bfloat16))


def test_sizes_past_32_bit_counters_are_refused(L):
    """Row numbers go 128 past a call's last row, a CTA's dt values are one int."""
    st = rssm.StateStruct(*([0x1000] * 7))
    assert scan(L, cfg(), st, total=0x7fffff01) == INVALID
    assert rssm.rssm_prefill_scan_workspace_bytes(cfg(batch=1), 0x7fffff01, 0x7fffffff) == 0
    assert conv(L, cfg(), total=0x7fffff01) == INVALID
    assert conv(L, cfg(nheads=1 << 24, head_dim=1, d_state=1, ngroups=1)) == SHAPE
