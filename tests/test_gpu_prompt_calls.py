"""The prompt calls as programs make them: memory that another stream still
works on, two host threads, the most heads that a call takes. Results are
compared bit for bit with those of the calls alone, or with the formula; the
residual stream of a stage in aggregate, as in its own tests."""
import ctypes as ct
import threading

import pytest
import torch

from hybrid_model_ssm_replay_b200 import rssm, stage
from hybrid_model_ssm_replay_b200.inputs import LayerShape, make_inputs
from hybrid_model_ssm_replay_b200.stage import HybridStage, StageShape, make_weights, rssm_stage_conv_prompt

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from hybrid_model_ssm_replay_b200 import build
    build.build()


class Prompt:
    """One long prompt of two heads, which the scan cuts into segments."""

    def __init__(self, T, seed):
        inp = make_inputs(LayerShape(1, 2, 64, 128, 1), T, seed, BF, device="cuda")
        self.args = [inp[k][:, 0].contiguous() for k in ("x", "B", "C", "dt")] + [inp["A"], inp["D"]]
        self.desc = rssm.make_desc(1, 2, 64, 128, 1)
        self.need = rssm.rssm_prefill_scan_workspace_bytes(self.desc, T, T)
        self.cu, self.T = torch.tensor([0, T], dtype=torch.int32, device="cuda"), T

    def fresh(self):
        return rssm.RssmState(self.desc), torch.zeros(self.T, 2, 64, device="cuda")

    def run(self, st, y, **kw):
        rssm.rssm_prefill_scan(st, self.cu, self.T, *self.args, y, **kw)


def test_scan_workspace_is_not_what_another_stream_still_uses():
    """A block freed on the current stream, with work on it still queued, is
    not taken by a scan on a side stream that nothing makes wait."""
    p, side = Prompt(6000, 3), torch.cuda.Stream()
    assert p.need > 0
    st0, y0 = p.fresh()
    p.run(st0, y0)
    st, y = p.fresh()
    held, copy = (torch.empty(p.need, dtype=torch.uint8, device="cuda") for _ in range(2))
    held.fill_(1)
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)  # about 50 ms
    copy.copy_(held)
    del held
    p.run(st, y, stream=side)
    torch.cuda.synchronize()
    assert (copy == 1).all()
    assert torch.equal(y, y0) and torch.equal(st.ckpt, st0.ckpt)


def test_scans_on_two_streams_back_to_back():
    """A segmented scan on the current stream and at once others on side
    streams and on the current one again, their inputs ready long before."""
    ps, sides = [Prompt(T, 5 + T) for T in (20000, 20000, 12000)], [torch.cuda.Stream() for _ in range(2)]
    alone, out = [p.fresh() for p in ps], [p.fresh() for p in ps]
    for p, (st, y) in zip(ps, alone):
        p.run(st, y)
    torch.cuda.synchronize()
    for _ in range(20):
        for st, y in out:
            st.ckpt.zero_()
            y.zero_()
        torch.cuda.synchronize()
        for p, (st, y), s in zip(ps, out, [None] + sides):
            p.run(st, y, stream=s)
        torch.cuda.synchronize()
        for (st, y), (st0, y0) in zip(out, alone):
            assert rssm.rssm_get_error(st) == 0
            assert torch.equal(y, y0) and torch.equal(st.ckpt, st0.ckpt)


def test_scans_of_two_shapes_from_two_threads():
    """Two host threads call the same kernel with heads of 256 x 64 and 128 x
    128, whose shared memory differs: no launch is refused."""
    L, calls = rssm.lib(), []
    for P, N in ((256, 64), (128, 128)):
        inp = make_inputs(LayerShape(1, 1, P, N, 1), 1, 9, torch.float32, device="cuda")
        st = rssm.RssmState(rssm.make_desc(1, 1, P, N, 1, in_dtype=rssm.RSSM_F32))
        y, cu = torch.zeros(1, 1, P, device="cuda"), torch.tensor([0, 1], dtype=torch.int32, device="cuda")
        s = torch.cuda.Stream()
        keep = [cu] + [inp[k][:, 0].contiguous() for k in ("x", "B", "C", "dt")] + [inp["A"], inp["D"], y]
        args = (ct.byref(st.desc), ct.byref(st.struct), 1, 1, *[ct.c_void_p(t.data_ptr()) for t in keep], None, 0,
                ct.c_void_p(s.cuda_stream))
        calls.append((args, keep, st, s))
    torch.cuda.synchronize()
    start, refused = threading.Barrier(2), []

    def go(args):
        start.wait()
        refused.extend(r for r in (L.rssm_prefill_scan(*args) for _ in range(20000)) if r)
    threads = [threading.Thread(target=go, args=(c[0],)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not refused, f"{len(refused)} launches refused: {set(refused)}"
    for _, _, st, _ in calls:
        assert rssm.rssm_get_error(st) == 0


def test_conv_of_the_most_heads_the_call_takes():
    """256 tokens of 2^23 heads: 2^31 values of dt by one CTA, all of them written."""
    T, N, heads = 256, 4, 1 << 23
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    g = torch.Generator(device="cuda").manual_seed(17)
    chans = heads + 2 * N
    zx = torch.randn(T, heads + chans + heads, generator=g, device="cuda", dtype=BF)
    state = torch.zeros(1, 3, chans, dtype=BF, device="cuda")
    w, b = torch.randn(chans, 4, generator=g, device="cuda"), torch.randn(chans, generator=g, device="cuda")
    dtb = torch.randn(heads, generator=g, device="cuda")
    x, dt = torch.zeros(T, heads, 1, dtype=BF, device="cuda"), torch.full((T, heads), -1.0, device="cuda")
    B, C = (torch.zeros(T, 1, N, dtype=BF, device="cuda") for _ in range(2))
    cu, err = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([0, T], [0]))
    rssm_stage_conv_prompt(rssm.make_desc(1, heads, 1, N, 1), cu, zx, state, w, b, dtb, x, B, C, dt, err=err)
    assert int(err) == 0
    assert torch.equal(state[0], zx[-3:, heads:heads + chans])
    # softplus of an fp32 sum: its rounding, 2^-24 of v, and a few spacings of log1p and exp
    for t in (0, 1, 100, T - 1):
        v = zx[t, heads + chans:].double() + dtb.double()
        ref = torch.where(v > 20, v, torch.log1p(torch.exp(v)))
        assert ((dt[t].double() - ref).abs() <= 1e-6 * (ref + v.abs())).all(), t
    assert (dt >= 0).all()


STAGE = StageShape(batch=3, d_model=64, nheads=4, head_dim=32, d_state=64, ngroups=2, interval=16, n_ssm=2, n_attn=1,
                   attn_heads=2, kv_heads=1, attn_head_dim=32, ctx=24)


def test_stage_decodes_on_after_a_prefill_that_failed(monkeypatch):
    """A prefill that stops right after its flush (no memory for its buffers),
    after five decoded tokens: the next forty are those of a stage that never
    tried, over two ends of intervals."""
    w = make_weights(STAGE, 11)
    ref, st = HybridStage(STAGE, w, seed=5), HybridStage(STAGE, w, seed=5)
    g = torch.Generator().manual_seed(9)
    u = torch.randn(45, STAGE.batch, STAGE.d_model, generator=g).to(BF).cuda()

    def stop(*args, **kw):
        raise MemoryError
    for t in range(45):
        if t == 5:
            with monkeypatch.context() as m:
                m.setattr(stage, "rssm_stage_add_norm", stop)
                with pytest.raises(MemoryError):
                    st.prefill(u[:3].transpose(0, 1))
        a, b = ref.step(u[t]).double(), st.step(u[t]).double()
        d, scale = (a - b).abs(), a.square().mean().sqrt()
        assert d.square().mean().sqrt() <= 0.01 * scale and d.max() <= 0.05 * scale, t
    for layer in st.ssm:
        assert rssm.rssm_get_error(layer["state"]) == 0


@pytest.mark.parametrize("P,N", [(64, 128), (64, 64), (40, 32)])
@pytest.mark.parametrize("T,scale", [(1, 1.0), (16, 10.0), (256, 10.0), (300, 1.0)])
def test_scan_from_a_full_state(T, scale, P, N):
    """Outputs that are mostly those of a full checkpoint, in fp32 accuracy.
    Tolerance: the state's bf16 parts leave 2^-27 of a term, and a sum takes 3
    N / 16 <= 24 steps of fp32, each off by at most 2^-23 of its partial sum:
    2^-23 sqrt(24) = 5.8e-7 where they are independent, and as much again (in
    all 1e-6, in the 2-norm) for the decays and the tokens' own products. The
    largest by the framework's bound, 1e-4 of the rms."""
    b, H, G = 16, 4, 2
    g = torch.Generator(device="cuda").manual_seed(T)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x, B, C = rn(b * T, H, P).to(BF), rn(b * T, G, N).to(BF), rn(b * T, G, N).to(BF)
    dt = torch.nn.functional.softplus(rn(b * T, H) - 3)
    A, D, ckpt = -16 ** torch.rand(H, generator=g, device="cuda"), rn(H), scale * rn(b, H, P, N)
    st, y = rssm.RssmState(rssm.make_desc(b, H, P, N, G)), torch.empty(b * T, H, P, device="cuda")
    st.ckpt.copy_(ckpt)
    cu = torch.arange(b + 1, dtype=torch.int32, device="cuda") * T
    rssm.rssm_prefill_scan(st, cu, T, x, B, C, dt, A, D, y)
    assert rssm.rssm_get_error(st) == 0
    h, ref = ckpt.double(), []
    X, Bd, Cd, d = (v.double().view(b, T, *v.shape[1:]) for v in (x, B, C, dt))
    Bd, Cd = Bd.repeat_interleave(H // G, 2), Cd.repeat_interleave(H // G, 2)
    for t in range(T):
        h = torch.exp(d[:, t] * A.double())[..., None, None] * h + (d[:, t, :, None] * X[:, t])[..., None] * Bd[:, t, :, None]
        ref.append((h * Cd[:, t, :, None]).sum(-1) + D.double()[:, None] * X[:, t])
    for got, want, what in ((y.double().view(b, T, H, P), torch.stack(ref, 1), "outputs"), (st.ckpt.double(), h, "state")):
        e = got - want
        assert e.norm() <= 1e-6 * want.norm(), f"{what}: {float(e.norm() / want.norm()):.2e}"
        assert e.abs().max() <= 1e-4 * want.square().mean().sqrt(), what
