"""Packed prompts through a Mamba-2 block (rssm_prefill_scan,
rssm_stage_conv_prompt, rssm_stage_gate_norm_prompt, rssm_stage_add_norm),
one by one against 64-bit references and together as HybridStage.prefill.

Tolerances. Scan: the framework's bound, max |d| <= 1e-4 rms, and 1e-5 in the
2-norm: a factor that goes to the tensor cores as bf16 parts is within 2^-18
of itself (3.8e-6) at worst, and the fp32 sums behind an output (up to a few
hundred terms, each addition within 2^-24 of its partial sum) add less than
as much again in the 2-norm. bf16 results: half a spacing, 2^-8 of the value,
plus 1e-5 for the fp32 arithmetic before the rounding. Values that are copied
(the conv state) are equal."""
import math

import numpy as np
import pytest
import torch

from hybrid_model_ssm_replay_b200 import rssm
from hybrid_model_ssm_replay_b200.inputs import LayerShape, make_inputs
from hybrid_model_ssm_replay_b200.stage import (HybridStage, StageShape, make_weights, rssm_stage_add_norm,
                                                rssm_stage_conv, rssm_stage_conv_prompt, rssm_stage_gate_norm,
                                                rssm_stage_gate_norm_prompt)

from gpu_helpers import assert_close, desc_for, oracle_map, to_np

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from hybrid_model_ssm_replay_b200 import build
    build.build()


def bounds(lens, first=0):
    return torch.tensor([first] + lens).cumsum(0).to(torch.int32).cuda()


def near(got, ref, what, rel=1e-5):
    assert_close(got, ref, what)
    d, n = np.linalg.norm(np.asarray(got) - ref), np.linalg.norm(ref)
    assert d <= rel * n, f"{what}: 2-norm {d / n:.2e}"


# ------------------------------------------------------------------- scan

class Packed:
    """Random prompts back to back, `first` unused rows before and 3 behind."""

    def __init__(self, shape, lens, seed, dtype=BF, first=0, dt=None):
        self.shape, self.lens, self.first, self.dtype = shape, lens, first, dtype
        T = first + sum(lens) + 3
        inp = make_inputs(LayerShape(1, shape.nheads, shape.head_dim, shape.d_state, shape.ngroups), T, seed, dtype,
                          device="cuda")
        self.x, self.B, self.C, self.dt = (inp[k][:, 0].contiguous() for k in ("x", "B", "C", "dt"))
        if dt is not None:
            self.dt.copy_(dt(self.dt))
        self.A, self.D, self.T = inp["A"], inp["D"], T
        g = torch.Generator(device="cuda").manual_seed(seed + 1)
        self.ckpt = torch.randn(len(lens), shape.nheads, shape.head_dim, shape.d_state, generator=g, device="cuda") * 0.1
        self.cu = bounds(lens, first)
        self.y = torch.full((T, shape.nheads, shape.head_dim), float("nan"), device="cuda")

    def state(self):
        st = rssm.RssmState(desc_for(self.shape, self.dtype))
        st.ckpt.copy_(self.ckpt)
        return st

    def run(self, st=None, longest=None, **kw):
        st = st or self.state()
        rssm.rssm_prefill_scan(st, self.cu, max(self.lens) if longest is None else longest, self.x, self.B, self.C,
                               self.dt, self.A, self.D, self.y, **kw)
        return st

    def check(self, st, requests=None):
        """Outputs and end states against the oracle; rows of no request untouched."""
        requests = range(len(self.lens)) if requests is None else requests
        at = self.cu.cpu().tolist()
        live = [b for b in requests if self.lens[b]]
        jobs = []
        for b in live:
            r = slice(at[b], at[b + 1])
            jobs.append(("conv", dict(ckpt=to_np(self.ckpt[b]), x=to_np(self.x[r]), B=to_np(self.B[r]), C=to_np(self.C[r]),
                                      dt=to_np(self.dt[r]), A=to_np(self.A), D=to_np(self.D)), [self.lens[b] - 1]))
        for b, (y_ref, snaps) in zip(live, oracle_map(jobs) if jobs else []):
            near(to_np(self.y[at[b]:at[b + 1]]), y_ref, f"outputs of request {b} ({self.lens[b]} tokens)")
            near(to_np(st.ckpt[b]), snaps[self.lens[b] - 1], f"end state of request {b} ({self.lens[b]} tokens)")
        for b in requests:
            if not self.lens[b]:
                assert torch.equal(st.ckpt[b], self.ckpt[b]), f"request {b} without tokens"
        assert self.y[:at[0]].isnan().all() and self.y[at[-1]:].isnan().all()


SHAPES = [LayerShape(5, 4, 64, 128, 2), LayerShape(5, 3, 128, 128, 3), LayerShape(5, 4, 32, 64, 1),
          LayerShape(5, 4, 40, 64, 2), LayerShape(5, 2, 17, 16, 1), LayerShape(5, 6, 80, 128, 2),
          LayerShape(5, 2, 256, 64, 2), LayerShape(5, 2, 8, 32, 1)]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"H{s.nheads}P{s.head_dim}N{s.d_state}G{s.ngroups}")
def test_scan_ragged_prompts_match_recurrence(shape, dtype):
    """Lengths 1, 0, past one block of tokens, and 2; unused rows around; then
    decoding goes on from the state the scan left."""
    p = Packed(shape, [1, 0, 150, 37, 2], 7, dtype, first=2)
    st = p.run()
    assert rssm.rssm_get_error(st) == 0
    p.check(st)
    assert st.pos.cpu().tolist() == [0] * 5 and st.flush_count.cpu().tolist() == [0] * 5
    nxt = make_inputs(shape, 3, 8, dtype, device="cuda")
    h = st.ckpt.clone()
    y, yc = (torch.empty(5, shape.nheads, shape.head_dim, device="cuda") for _ in range(2))
    for t in range(3):
        args = [nxt[k][t] for k in ("x", "B", "C", "dt")] + [p.A, p.D]
        rssm.rssm_decode_step(st, *args, y)
        rssm.rssm_conv_step(st.desc, h, *args, yc)
        assert_close(to_np(y), to_np(yc), f"decoded token {t}")


@pytest.mark.parametrize("T", [1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 385])
def test_scan_block_edges(T):
    """Prompts around the edges of the blocks of tokens the kernels work in."""
    p = Packed(LayerShape(3, 2, 64, 128, 1), [T, max(0, T - 1), T], 11 + T)
    st = p.run()
    assert rssm.rssm_get_error(st) == 0
    p.check(st)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("lens", [[1500], [0, 1111, 3], [700, 0, 900]], ids=["one", "with-short", "two"])
def test_scan_long_prompts_in_segments(lens, dtype):
    """Few heads and long prompts: the call cuts them into segments."""
    shape = LayerShape(len(lens), 2, 64, 128, 1)
    p = Packed(shape, lens, 21, dtype, first=5)
    assert rssm.rssm_prefill_scan_workspace_bytes(desc_for(shape, dtype), p.T, max(lens)) > 0
    st = p.run()
    assert rssm.rssm_get_error(st) == 0
    p.check(st)
    y = p.y.clone()
    ws = torch.full((rssm.rssm_prefill_scan_workspace_bytes(desc_for(shape, dtype), p.T, max(lens)),), 255,
                    dtype=torch.uint8, device="cuda")  # NaN all over: nothing of it is read before it is written
    st2 = p.run(workspace=ws)
    at = p.cu.cpu().tolist()
    assert torch.equal(p.y[at[0]:at[-1]], y[at[0]:at[-1]]) and torch.equal(st2.ckpt, st.ckpt)


def test_scan_full_size_sampled():
    """The small layer's heads (64 x 64 x 128, 8 groups), 512-token prompts."""
    p = Packed(LayerShape(16, 64, 64, 128, 8), [512] * 15 + [77], 31)
    st = p.run()
    assert rssm.rssm_get_error(st) == 0
    p.check(st, [0, 9, 15])


def test_scan_decay_extremes():
    """Steps that forget everything (decays that underflow), steps of zero and
    of a millionth, mixed in one prompt."""
    def dt(d):
        pick = torch.arange(d.shape[0], device="cuda")[:, None] % 5
        return torch.where(pick == 1, 300.0, torch.where(pick == 3, 0.0, torch.where(pick == 4, 1e-6, d)))
    p = Packed(LayerShape(2, 4, 64, 128, 2), [200, 131], 41, dt=dt)
    st = p.run()
    assert rssm.rssm_get_error(st) == 0
    p.check(st)
    q = Packed(LayerShape(1, 2, 64, 128, 1), [300], 42, dt=lambda d: d * 1e-4)  # hardly any decay
    st = q.run()
    q.check(st)


@pytest.mark.parametrize("what", ["x", "B", "C", "dt"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_scan_bad_values_stay_behind(what, value, dtype):
    """A NaN or infinity of one token changes no output before it, and nothing
    of another request or (of x) another column."""
    shape = LayerShape(2, 2, 64, 128, 1)
    p = Packed(shape, [300, 40], 51, dtype)
    clean = p.run()
    y0, h0 = p.y.clone(), clean.ckpt.clone()
    t = 170
    getattr(p, what)[t].view(-1)[0 if what == "dt" else 5] = value
    st = p.run()
    assert rssm.rssm_get_error(st) == 0
    assert torch.equal(p.y[:t], y0[:t]) and torch.equal(p.y[300:340], y0[300:340])
    assert torch.equal(st.ckpt[1], h0[1])
    if what == "dt":
        return
    assert not p.y[t:300].isfinite().all()
    if what == "x":
        keep = torch.ones(2, 64, dtype=torch.bool)
        keep[0, 5] = False
        near(to_np(p.y[:300][:, keep]), to_np(y0[:300][:, keep]), "the other columns")
        near(to_np(st.ckpt[0][keep]), to_np(h0[0][keep]), "the other rows of the state")


@pytest.mark.parametrize("shape", [LayerShape(2, 2, 64, 128, 1), LayerShape(2, 2, 40, 64, 1)], ids=["P64N128", "P40N64"])
@pytest.mark.parametrize("lens", [[300, 40], [1300, 40]], ids=["whole", "segments"])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_scan_rows_of_others_do_not_matter(shape, lens, dtype):
    """NaN in every row of the next request and of no request, and in the
    columns of the other head, changes nothing of a request."""
    p = Packed(shape, lens, 55, dtype, first=3)
    st0 = p.run()
    y0, n = p.y.clone(), lens[0]
    rows = torch.ones(p.T, dtype=torch.bool, device="cuda")
    rows[3:3 + n] = False
    for k in ("x", "B", "C", "dt"):
        getattr(p, k)[rows] = float("nan")
    p.x[:, 1] = float("nan")  # the second head
    st = p.run()
    assert rssm.rssm_get_error(st) == 0
    assert torch.equal(p.y[3:3 + n, 0], y0[3:3 + n, 0]) and torch.equal(st.ckpt[0, 0], st0.ckpt[0, 0])


def test_scan_loose_bound_on_the_lengths():
    """max_seqlen only bounds the lengths: any larger one gives the same."""
    p = Packed(LayerShape(3, 2, 64, 128, 1), [200, 5, 129], 56)
    p.run()
    y, n = p.y.clone(), sum(p.lens)
    for longest in (201, 1 << 20, (1 << 31) - 1):
        p.y.fill_(float("nan"))
        st = p.run(longest=longest)
        assert rssm.rssm_get_error(st) == 0
        near(to_np(p.y[:n]), to_np(y[:n]), f"max_seqlen {longest}")


def test_scan_device_errors_leave_the_request():
    shape = LayerShape(3, 2, 64, 128, 1)
    p = Packed(shape, [20, 30, 25], 61)
    st = p.state()
    st.pos[1] = 4
    p.run(st)
    assert rssm.rssm_get_error(st) == 1  # RSSM_DEVERR_POS_RANGE
    assert torch.equal(st.ckpt[1], p.ckpt[1]) and p.y[20:50].isnan().all()
    assert st.pos.cpu().tolist() == [0, 4, 0]
    at = p.cu.cpu().tolist()
    assert p.y[at[0]:at[1]].isfinite().all() and p.y[at[2]:at[3]].isfinite().all()
    for cu, longest, left in (([0, 20, 50, 79], 30, [2]),    # past the rows
                              ([0, 20, 10, 40], 30, [1]),    # going back
                              ([-1, 20, 50, 75], 30, [0]),   # before the rows
                              ([0, 20, 50, 75], 24, [1, 2])):  # longer than said
        p.cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        p.y.fill_(float("nan"))
        st = p.state()
        p.run(st, longest)
        assert rssm.rssm_get_error(st) == 5, cu  # RSSM_DEVERR_SEQ_RANGE
        for b in left:
            assert torch.equal(st.ckpt[b], p.ckpt[b]), (cu, b)
    # the same in segments
    p = Packed(LayerShape(2, 2, 64, 128, 1), [900, 40], 62)
    p.cu = torch.tensor([0, 900, 960], dtype=torch.int32, device="cuda")
    st = p.run(longest=900)
    assert rssm.rssm_get_error(st) == 5 and torch.equal(st.ckpt[1], p.ckpt[1])


def test_scan_no_tokens():
    p = Packed(LayerShape(3, 2, 64, 128, 1), [0, 0, 0], 63)
    st = p.run(longest=0)
    assert rssm.rssm_get_error(st) == 0 and torch.equal(st.ckpt, p.ckpt) and p.y.isnan().all()
    rssm.rssm_prefill_scan(st, p.cu, 0, p.x[:0], p.B[:0], p.C[:0], p.dt[:0], p.A, p.D, p.y[:0])
    assert torch.equal(st.ckpt, p.ckpt)


def test_scan_refuses_bad_tensors():
    p = Packed(LayerShape(2, 2, 64, 128, 1), [9, 9], 64)
    st = p.state()
    def call(**kw):
        a = dict(cu=p.cu, x=p.x, B=p.B, C=p.C, dt=p.dt, A=p.A, D=p.D, y=p.y)
        a.update(kw)
        rssm.rssm_prefill_scan(st, a["cu"], 9, a["x"], a["B"], a["C"], a["dt"], a["A"], a["D"], a["y"])
    for bad in (dict(x=p.x.float()), dict(cu=p.cu.long())):
        with pytest.raises(TypeError):
            call(**bad)
    for bad in (dict(x=p.x.transpose(1, 2)), dict(B=p.B[:-1]), dict(y=p.y[:, :1]), dict(cu=p.cu[:2]), dict(dt=p.dt.cpu()),
                dict(y=torch.empty(p.y.numel() + 1, device="cuda")[1:].view(p.y.shape))):
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises(rssm.RssmError):
        rssm.rssm_prefill_scan(rssm.RssmState(desc_for(p.shape, update_dtype=rssm.RSSM_BF16)), p.cu, 9, p.x, p.B, p.C,
                               p.dt, p.A, p.D, p.y)


@pytest.mark.parametrize("lens", [[130, 64], [1400, 100]], ids=["whole", "segments"])
def test_scan_repeats_on_streams_and_in_graphs(lens):
    """Bit-identical on a repeat, on two other streams at once, and captured
    and replayed."""
    p = Packed(LayerShape(2, 2, 64, 128, 1), lens, 71)
    ref = p.run()
    y = p.y.clone()
    n = sum(lens)
    sides = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    states, ys = [p.state() for _ in sides], [torch.zeros_like(p.y) for _ in sides]
    torch.cuda.synchronize()
    for s, st, out in zip(sides, states, ys):
        rssm.rssm_prefill_scan(st, p.cu, max(lens), p.x, p.B, p.C, p.dt, p.A, p.D, out, stream=s)
    torch.cuda.synchronize()
    for st, out in zip(states, ys):
        assert torch.equal(out[:n], y[:n]) and torch.equal(st.ckpt, ref.ckpt)
    graph = torch.cuda.CUDAGraph()
    st = p.state()
    with torch.cuda.graph(graph):
        p.run(st)
    for _ in range(2):
        st.ckpt.copy_(p.ckpt)
        p.y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(p.y[:n], y[:n]) and torch.equal(st.ckpt, ref.ckpt)


# ------------------------------------------------------------------- conv

def check_bf16(got, ref, what, slack=0.0):
    """Half a bf16 spacing and 1e-5 of the value, and an absolute `slack` for a
    value whose fp32 terms may cancel."""
    got, ref = to_np(got).ravel(), np.asarray(ref, np.float64).ravel()
    bad = np.abs(got - ref) > (2.0 ** -8 + 1e-5) * np.abs(ref) + 1e-30 + np.ravel(slack)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} beyond half a bf16 spacing"


def conv_inputs(shape, lens, seed, first=0):
    g = torch.Generator().manual_seed(seed)
    H, P, N, G = shape.nheads, shape.head_dim, shape.d_state, shape.ngroups
    chans, T = H * P + 2 * G * N, first + sum(lens) + 2
    rn = lambda *s: torch.randn(*s, generator=g)
    c = dict(zx=(rn(T, H * P + chans + H) * 2).to(BF), state=rn(len(lens), 3, chans).to(BF), w=rn(chans, 4), b=rn(chans),
             dtb=rn(H) * 8)
    c = {k: v.cuda() for k, v in c.items()}
    c.update(x=torch.full((T, H, P), 7.0, dtype=BF, device="cuda"), B=torch.full((T, G, N), 7.0, dtype=BF, device="cuda"),
             C=torch.full((T, G, N), 7.0, dtype=BF, device="cuda"), dt=torch.full((T, H), 7.0, device="cuda"),
             cu=bounds(lens, first), desc=rssm.make_desc(len(lens), H, P, N, G))
    return c


def conv_run(c, err=None):
    rssm_stage_conv_prompt(c["desc"], c["cu"], c["zx"], c["state"], c["w"], c["b"], c["dtb"], c["x"], c["B"], c["C"],
                           c["dt"], err=err)


CONV_SHAPES = [LayerShape(1, 4, 32, 64, 2), LayerShape(1, 3, 5, 16, 1), LayerShape(1, 8, 64, 128, 1),
               LayerShape(1, 7, 24, 16, 7), LayerShape(1, 64, 64, 128, 8)]


@pytest.mark.parametrize("shape", CONV_SHAPES, ids=lambda s: f"H{s.nheads}P{s.head_dim}N{s.d_state}G{s.ngroups}")
@pytest.mark.parametrize("lens", [[1, 2, 3, 0, 4, 5, 0], [15, 1, 1, 16, 17, 31, 64, 2, 90], [200], [1] * 40],
                         ids=["short", "mixed", "one", "ones"])
def test_conv_prompt_matches_single_tokens_and_reference(shape, lens):
    """Every token's results and the state are those of rssm_stage_conv token
    by token, bit for bit, and those of the formula; other rows are untouched."""
    c = conv_inputs(shape, lens, 3, first=1)
    state0 = c["state"].clone()
    conv_run(c)
    torch.cuda.synchronize()
    H, P, N, G = shape.nheads, shape.head_dim, shape.d_state, shape.ngroups
    at, din, gn = c["cu"].cpu().tolist(), H * P, G * N
    one = rssm.make_desc(1, H, P, N, G)
    for b, n in enumerate(lens):
        st = state0[b:b + 1].clone()
        ref = torch.cat([state0[b], c["zx"][at[b]:at[b + 1], din:2 * din + 2 * gn]])
        for t in range(at[b], at[b + 1]):
            row = [torch.empty(1, H, P, dtype=BF, device="cuda"), torch.empty(1, G, N, dtype=BF, device="cuda"),
                   torch.empty(1, G, N, dtype=BF, device="cuda"), torch.empty(1, H, device="cuda")]
            if n <= 64 or t < at[b] + 5 or t >= at[b + 1] - 5:
                src = c["zx"][t:t + 1]
                k = t - at[b]
                rssm_stage_conv(one, src, ref[k:k + 3].unsqueeze(0).clone(), c["w"], c["b"], c["dtb"], *row)
                for got, want, name in zip((c["x"], c["B"], c["C"], c["dt"]), row, "x B C dt".split()):
                    assert torch.equal(got[t], want[0]), f"{name} of request {b}, token {k}"
        assert torch.equal(c["state"][b], ref[-3:]), f"state of request {b}"
        if n:
            r, w = to_np(ref), to_np(c["w"])
            o = to_np(c["b"]) + sum(w[:, k] * r[k:k + n] for k in range(4))
            act = o / (1 + np.exp(-o))
            # the five terms of o are added by four fp32 fma, each off by at most
            # 2^-24 of a partial sum <= m = sum |terms|, and silu's slope is at most
            # 1.1: 4.4 x 2^-24 m where the terms cancel, whatever is left of o
            m = 5 * 2.0 ** -24 * (np.abs(to_np(c["b"])) + sum(np.abs(w[:, k] * r[k:k + n]) for k in range(4)))
            rows = slice(at[b], at[b + 1])
            check_bf16(c["x"][rows], act[:, :din], "x", m[:, :din])
            check_bf16(c["B"][rows], act[:, din:din + gn], "B", m[:, din:din + gn])
            check_bf16(c["C"][rows], act[:, din + gn:], "C", m[:, din + gn:])
            v = to_np(c["zx"][rows, 2 * din + 2 * gn:]) + to_np(c["dtb"])
            sp = np.where(v > 20, v, np.log1p(np.exp(np.minimum(v, 700))))
            assert np.max(np.abs(to_np(c["dt"][rows]) - sp) / sp) < 1e-5
    for name in ("x", "B", "C", "dt"):
        assert (c[name][:at[0]] == 7).all() and (c[name][at[-1]:] == 7).all(), name


def test_conv_prompt_many_tokens_matches_in_one_and_in_parts():
    """A prompt in one call and cut in two calls give the same bits."""
    shape = LayerShape(1, 8, 64, 128, 1)
    c = conv_inputs(shape, [1000], 5)
    d = {k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in c.items()}
    conv_run(c)
    for lo, hi in ((0, 389), (389, 1000)):
        d["cu"] = torch.tensor([lo, hi], dtype=torch.int32, device="cuda")
        conv_run(d)
    for k in ("x", "B", "C", "dt", "state"):
        assert torch.equal(c[k], d[k]), k


def test_conv_prompt_bad_bounds():
    shape = LayerShape(1, 4, 32, 64, 2)
    for cu, left in (([0, 5, 3, 9], 1), ([0, 5, 9, 40], 2), ([-2, 5, 9, 12], 0)):
        c = conv_inputs(shape, [5, 4, 3], 6)
        old = c["state"].clone()
        c["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        conv_run(c, err)
        assert int(err) == 5, cu
        assert torch.equal(c["state"][left], old[left]), cu


# ------------------------------------------------------------------ norms

@pytest.mark.parametrize("rows", [0, 1, 3, 130])
@pytest.mark.parametrize("shape", [LayerShape(1, 4, 32, 64, 2), LayerShape(1, 3, 5, 16, 1), LayerShape(1, 64, 64, 128, 8),
                                   LayerShape(1, 64, 64, 128, 1), LayerShape(1, 6, 11, 16, 2), LayerShape(1, 128, 128, 16, 1),
                                   LayerShape(1, 24, 64, 128, 4), LayerShape(1, 9, 8, 16, 3)],
                         ids=lambda s: f"H{s.nheads}P{s.head_dim}G{s.ngroups}")
def test_gate_norm_prompt_matches_reference(shape, rows):
    g = torch.Generator().manual_seed(4)
    H, P, N, G = shape.nheads, shape.head_dim, shape.d_state, shape.ngroups
    din = H * P
    y = torch.randn(rows, H, P, generator=g).cuda()
    zx = (torch.randn(rows, 2 * din + 2 * G * N + H, generator=g) * 2).to(BF).cuda()
    w = (1 + 0.1 * torch.randn(din, generator=g)).cuda()
    if rows > 2:
        y[1] = 0     # nothing but eps under the root
        y[2] *= 1e15  # squares far from one
        zx[0, :din] = -90.0  # a gate that underflows
    out = torch.empty(rows, din, dtype=BF, device="cuda")
    rssm_stage_gate_norm_prompt(rssm.make_desc(1, H, P, N, G), y, zx, w, 1e-5, out)
    z = to_np(zx)[:, :din]
    v = (to_np(y).reshape(rows, din) * (z / (1 + np.exp(-z)))).reshape(rows, G, din // G)
    ref = (v / np.sqrt(np.mean(v * v, -1, keepdims=True) + 1e-5)).reshape(rows, din) * to_np(w)
    check_bf16(out, ref, "gated norm")


def test_gate_norm_prompt_matches_single_token_form():
    """Many rows of the small layer: within a bf16 spacing of rssm_stage_gate_norm."""
    rows, H, P, N, G = 300, 64, 64, 128, 8
    g = torch.Generator(device="cuda").manual_seed(6)
    y = torch.randn(rows, H * P, generator=g, device="cuda")
    zx = torch.randn(rows, 2 * H * P + 2 * G * N + H, generator=g, device="cuda").to(BF)
    w = torch.randn(H * P, generator=g, device="cuda")
    a, b = (torch.empty(rows, H * P, dtype=BF, device="cuda") for _ in range(2))
    rssm_stage_gate_norm_prompt(rssm.make_desc(1, H, P, N, G), y, zx, w, 1e-5, a)
    rssm_stage_gate_norm(rssm.make_desc(rows, H, P, N, G), y, zx, w, 1e-5, b)
    d = (a.double() - b.double()).abs()
    assert (d <= 2.0 ** -7 * b.double().abs()).all()
    assert (d > 0).double().mean() < 0.01  # only sums that differ near a border


@pytest.mark.parametrize("stream", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("post,gate", [(0, 0), (1, 0), (0, 1), (1, 1)])
@pytest.mark.parametrize("rows,dim", [(1, 1), (3, 7), (5, 64), (130, 2048), (4, 2561), (3, 8192), (2, 16384), (300, 1000),
                                      (2, 4104), (7, 12)])
def test_add_norm_matches_reference(rows, dim, stream, post, gate):
    g = torch.Generator().manual_seed(dim)
    rn = lambda *s: torch.randn(*s, generator=g)
    u, v = (rn(rows, dim) * 3).to(stream).cuda(), rn(rows, dim).to(BF).cuda()
    pw, gw, w = (1 + 0.1 * rn(dim)).cuda(), rn(dim).cuda(), (1 + 0.1 * rn(dim)).cuda()
    u0, n, eps = u.clone(), torch.empty(rows, dim, dtype=BF, device="cuda"), 1e-5
    uo = torch.empty_like(u)
    kw = dict(post_w=pw if post else None, gate=gw if gate else None, scale=0.37)
    rssm_stage_add_norm(u, v, w, eps, n, u_out=uo, **kw)
    assert torch.equal(u, u0)
    r = to_np(v)
    if post:
        r = r / np.sqrt(np.mean(r * r, -1, keepdims=True) + eps) * to_np(pw)
    if gate:
        r = r * to_np(gw)
    r = 0.37 * r  # (0.37 to fp32: 2^-25 of it)
    s = to_np(u) + r
    half = 2.0 ** -8 if stream == BF else 2.0 ** -24
    size = np.abs(to_np(u)) + np.abs(r)  # of the terms: they may cancel
    assert (np.abs(to_np(uo) - s) <= half * np.abs(s) + 2e-6 * size).all()
    k = to_np(uo)
    check_bf16(n, k / np.sqrt(np.mean(k * k, -1, keepdims=True) + eps) * to_np(w), "norm before")
    # in place, and the sum alone, are the same
    n2 = torch.empty_like(n)
    rssm_stage_add_norm(u, v, w, eps, n2, **kw)
    assert torch.equal(u, uo) and torch.equal(n, n2)
    u.copy_(u0)
    rssm_stage_add_norm(u, v, None, eps, None, **kw)
    assert torch.equal(u, uo)
    # the norm alone
    rssm_stage_add_norm(uo, None, w, eps, n2)
    assert torch.equal(n, n2)


@pytest.mark.parametrize("stream", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,dim", [(20011, 1), (20011, 12), (9001, 257), (5003, 2561), (1500, 4089), (1501, 4090),
                                      (700, 5001), (800, 8185), (300, 8186)])
def test_add_norm_many_odd_rows(rows, dim, stream):
    """Rows that start at every place of a 16-byte piece, more of them than
    run at once, in place, with what lies behind the last one left alone."""
    g = torch.Generator(device="cuda").manual_seed(dim)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")
    guard = lambda t: torch.cat([t.flatten(), torch.full((64,), 7.0, dtype=t.dtype, device="cuda")])
    ub, vb = guard((3 * rn(rows, dim)).to(stream)), rn(rows, dim).to(BF)
    u, pw, gw, w = ub[:-64].view(rows, dim), 1 + 0.1 * rn(dim), rn(dim), 1 + 0.1 * rn(dim)
    nb, eps, u0 = guard(torch.zeros_like(vb)), 1e-5, u.double()
    v, n = vb, nb[:-64].view(rows, dim)
    rssm_stage_add_norm(u, v, w, eps, n, post_w=pw, gate=gw, scale=0.37)
    assert (ub[-64:] == 7).all() and (nb[-64:] == 7).all()
    r = v.double()
    r = 0.37 * r / (r.square().mean(-1, keepdim=True) + eps).sqrt() * pw.double() * gw.double()
    half = 2.0 ** -8 if stream == BF else 2.0 ** -24
    assert ((u.double() - u0 - r).abs() <= half * (u0 + r).abs() + 2e-6 * (u0.abs() + r.abs())).all()
    k = u.double()
    check_bf16(n, to_np(k / (k.square().mean(-1, keepdim=True) + eps).sqrt() * w.double()), "norm before")


def test_add_norm_special_rows():
    """A row of zeros, one of huge values, and one with a NaN that stays in it."""
    u = torch.randn(4, 512, device="cuda").to(BF)
    v, w, n = torch.zeros_like(u), torch.ones(512, device="cuda"), torch.empty_like(u)
    u[1], u[2] = 0, 1e16
    u[3, 9] = float("nan")
    rssm_stage_add_norm(u, v, w, 1e-5, n)
    assert (n[1] == 0).all() and (n[2] == 1).all() and n[3].isnan().all() and n[0].isfinite().all()


# --------------------------------------------------------------- together

STAGE = StageShape(batch=3, d_model=64, nheads=4, head_dim=32, d_state=64, ngroups=2, interval=16, n_ssm=2, n_attn=1,
                   attn_heads=2, kv_heads=1, attn_head_dim=32, ctx=24)


def stream_close(got, ref, what):
    """The residual stream in aggregate, as in the stage's own tests: an
    element may round to the neighbouring bf16 and carry that on."""
    scale = math.sqrt(float(np.mean(ref * ref)))
    d = got - ref
    assert math.sqrt(float(np.mean(d * d))) <= 0.01 * scale, f"{what}: rms"
    assert float(np.max(np.abs(d))) <= 0.05 * scale, f"{what}: max"


@pytest.mark.parametrize("before,T,after", [(0, 20, 20), (5, 1, 3), (18, 24, 17), (0, 7, 30)])
def test_stage_prefill_matches_steps(before, T, after):
    """Tokens decoded, then a prompt, then tokens decoded: the same as all of
    them one by one, through conv, scan, norms and the attention cache."""
    w = make_weights(STAGE, 11)
    one, many = HybridStage(STAGE, w, seed=5), HybridStage(STAGE, w, seed=5)
    g = torch.Generator().manual_seed(9)
    u = torch.randn(before + T + after, STAGE.batch, STAGE.d_model, generator=g).to(BF).cuda()
    ref = [to_np(one.step(u[t])) for t in range(len(u))]
    for t in range(before):
        stream_close(to_np(many.step(u[t])), ref[t], f"token {t}")
    got = many.prefill(u[before:before + T].transpose(0, 1))
    for t in range(T):
        stream_close(to_np(got[:, t]), ref[before + t], f"prompt token {t}")
    for t in range(before + T, len(u)):
        stream_close(to_np(many.step(u[t])), ref[t], f"token {t} after the prompt")
    for a, b in zip(one.ssm, many.ssm):
        assert rssm.rssm_get_error(b["state"]) == 0
    assert many.t == one.t


# ------------------------------------------------- far offsets, other streams

def test_rows_past_32_bits():
    """The last of 600000 rows (more than 2^31 elements before them) come out
    as in a call of their own, for every call."""
    H, P, N, G, n, T = 64, 64, 128, 8, 300, 600000
    g = torch.Generator(device="cuda").manual_seed(91)
    lens = [T - n, n]
    cu, cu1 = bounds(lens), bounds([n])
    desc, one = rssm.make_desc(2, H, P, N, G), rssm.make_desc(1, H, P, N, G)
    din, gn = H * P, G * N
    rn = lambda *s, t=BF: torch.randn(*s, generator=g, device="cuda", dtype=t)
    zx = torch.zeros(T, 2 * din + 2 * gn + H, dtype=BF, device="cuda")
    zx[-2 * n:] = rn(2 * n, zx.shape[1])
    w, b, dtb, nw = rn(din + 2 * gn, 4, t=F32), rn(din + 2 * gn, t=F32), rn(H, t=F32) - 3, rn(din, t=F32)
    state = rn(2, 3, din + 2 * gn)
    keep = state.clone()

    def outs(rows):
        return (torch.zeros(rows, H, P, dtype=BF, device="cuda"), torch.zeros(rows, G, N, dtype=BF, device="cuda"),
                torch.zeros(rows, G, N, dtype=BF, device="cuda"), torch.zeros(rows, H, device="cuda"))
    full, last = outs(T), outs(n)
    rssm_stage_conv_prompt(desc, cu, zx, state, w, b, dtb, *full)
    st1 = keep[1:].clone()
    rssm_stage_conv_prompt(one, cu1, zx[-n:], st1, w, b, dtb, *last)
    for a, c in zip(full, last):
        assert torch.equal(a[-n:], c)
    assert torch.equal(state[1:], st1)
    A, D = -torch.rand(H, generator=g, device="cuda") - 0.5, rn(H, t=F32)
    y, y1 = torch.zeros(T, H, P, device="cuda"), torch.zeros(n, H, P, device="cuda")
    s2, s1 = rssm.RssmState(desc), rssm.RssmState(one)
    rssm.rssm_prefill_scan(s2, cu, lens[0], *full, A, D, y)
    rssm.rssm_prefill_scan(s1, cu1, n, *last, A, D, y1)
    assert rssm.rssm_get_error(s2) == 0 and rssm.rssm_get_error(s1) == 0
    near(to_np(y[-n:]), to_np(y1), "scan")  # (the long prompt's call may cut in segments)
    near(to_np(s2.ckpt[1]), to_np(s1.ckpt[0]), "scan's state")
    del full
    out, out1 = torch.zeros(T, din, dtype=BF, device="cuda"), torch.zeros(n, din, dtype=BF, device="cuda")
    rssm_stage_gate_norm_prompt(desc, y, zx, nw, 1e-5, out)
    rssm_stage_gate_norm_prompt(one, y[-n:], zx[-n:], nw, 1e-5, out1)
    assert torch.equal(out[-n:], out1)
    u, u1 = zx.new_zeros(T, din), zx.new_zeros(n, din)
    n1, n2 = torch.zeros_like(out), torch.zeros_like(out1)
    rssm_stage_add_norm(u, out, nw, 1e-5, n1, post_w=nw)
    rssm_stage_add_norm(u1, out1, nw, 1e-5, n2, post_w=nw)
    assert torch.equal(n1[-n:], n2) and torch.equal(u[-n:], u1)


def test_scan_beside_other_tensor_memory_kernels():
    """The scan on one stream, the tcgen05 prefill and the refresh on others,
    all holding tensor memory on the same SMs: each result as alone."""
    shape = LayerShape(64, 8, 64, 128, 2)
    p = Packed(shape, [200] * 64, 95)
    inp = make_inputs(shape, 200, 96, BF, device="cuda")
    ref = p.run()
    y0 = p.y.clone()
    a = rssm.RssmState(desc_for(shape))
    rssm.rssm_prefill(a, inp["x"], inp["B"], inp["dt"], inp["A"])
    fd = desc_for(shape, update_dtype=rssm.RSSM_BF16, out_copy=rssm.RSSM_OUTCOPY_FP4, seed=3)

    def refreshed(stream=None):
        f = rssm.RssmState(fd)
        f.ckpt.copy_(inp["ckpt"].to(BF))
        torch.cuda.synchronize()
        for _ in range(4):
            rssm.rssm_lowprec_refresh(f, inp["A"], force=True, stream=stream)
        return f
    f0 = refreshed()
    s = [torch.cuda.Stream() for _ in range(3)]
    b, st = rssm.RssmState(desc_for(shape)), p.state()
    f1 = rssm.RssmState(fd)
    f1.ckpt.copy_(inp["ckpt"].to(BF))
    p.y.zero_()
    torch.cuda.synchronize()
    for _ in range(4):
        rssm.rssm_lowprec_refresh(f1, inp["A"], force=True, stream=s[2])
    rssm.rssm_prefill_scan(st, p.cu, 200, p.x, p.B, p.C, p.dt, p.A, p.D, p.y, stream=s[0])
    rssm.rssm_prefill(b, inp["x"], inp["B"], inp["dt"], inp["A"], stream=s[1])
    torch.cuda.synchronize()
    assert torch.equal(p.y[:12800], y0[:12800]) and torch.equal(st.ckpt, ref.ckpt)
    assert torch.equal(b.ckpt, a.ckpt) and torch.equal(f1.ckpt, f0.ckpt)
    for q in (st, b, f0, f1):
        assert rssm.rssm_get_error(q) == 0
