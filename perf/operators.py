"""Prompt operators of a Mamba-2 mixer block, as they are measured.

Four operators run a packed batch of prompts (the tokens of all requests back
to back, their bounds in cu_seqlens) through a mixer block between its two
projections and on to the next block:
  conv  causal conv1d of width 4 with SiLU on the x, B, C channels of the
        input projection, dt = softplus(raw + bias), and the conv state;
  scan  the selective state space scan with its outputs, from and into the
        fp32 checkpoint that decoding continues from;
  gate  the gated RMS norm per group before the output projection;
  add   the norm after the block, its gate and scale, the residual add and
        the next block's norm before.
"""
import math
import random

import torch

own = False

EPS = 1e-5
CHUNK = 64  # tokens per block of the plain form's products


# ------------------------------------------------------------------- cases

SMALL = dict(H=64, P=64, N=128, G=8)    # the benchmark's small layer
LARGE = dict(H=128, P=64, N=128, G=8)   # the benchmark's large layer


def listed():
    return [
        # one short prompt by itself: what a user waits for before the first token
        dict(name="scan one prompt 77", op="scan", batch=1, longest=77, ragged=False, lens=0, dtype="bf16", **SMALL),
        # an arriving batch of prompts of mixed lengths, odd ones among them
        dict(name="scan 16 mixed prompts", op="scan", batch=16, longest=1501, ragged=True, lens=3, dtype="bf16", **SMALL),
        # the benchmark's prefill: 512-token prompts at batch 256
        dict(name="scan 256 x 512", op="scan", batch=256, longest=512, ragged=False, lens=0, dtype="bf16", **SMALL),
        # a long document alone on the large layer: few rows, a long axis
        dict(name="scan one prompt 16384", op="scan", batch=1, longest=16384, ragged=False, lens=0, dtype="bf16", **LARGE),
        # fp32 inputs, a head_dim and a state size off the usual ones
        dict(name="scan fp32 odd head", op="scan", batch=4, longest=300, ragged=True, lens=5, dtype="fp32", H=8, P=40, N=64, G=2),
        # the conv of the mixed batch, and of the benchmark's prefill
        dict(name="conv 16 mixed prompts", op="conv", batch=16, longest=1501, ragged=True, lens=3, **SMALL),
        dict(name="conv 256 x 512", op="conv", batch=256, longest=512, ragged=False, lens=0, **SMALL),
        # the gated norm of one prompt, and of the benchmark's prefill
        dict(name="gate 301 rows", op="gate", rows=301, **SMALL),
        dict(name="gate 131072 rows", op="gate", rows=131072, **SMALL),
        # between two blocks: a decode batch (no post norm), the prefill with every
        # option, and an fp32 residual stream of an odd width
        dict(name="add 256 rows", op="add", rows=256, dim=2048, stream="bf16", post=False, gate=False, scale=1.0),
        dict(name="add 131072 rows", op="add", rows=131072, dim=2048, stream="bf16", post=True, gate=True, scale=0.5),
        dict(name="add fp32 odd width", op="add", rows=5003, dim=2561, stream="fp32", post=True, gate=False, scale=1.0),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["scan", "scan", "conv", "gate", "add"])
    H, G = rng.choice([(8, 2), (24, 1), (64, 8), (64, 1), (128, 8)])
    if op == "add":
        dim = _log_int(rng, 256, 8192)
        return dict(op=op, rows=_log_int(rng, 1, 200000000 // dim), dim=dim if rng.random() < 0.3 else dim // 8 * 8,
                    stream=rng.choice(["bf16", "bf16", "fp32"]), post=rng.random() < 0.5, gate=rng.random() < 0.5,
                    scale=rng.choice([1.0, 0.22]))
    if op == "gate":
        P = rng.choice([32, 64, 128])
        return dict(op=op, rows=_log_int(rng, 1, 400000000 // (H * P)), H=H, P=P, N=128, G=G)
    fp32 = op == "scan" and rng.random() < 0.2
    if fp32:
        H, G, P, N = 8, 2, rng.choice([16, 17, 40, 64]), rng.choice([16, 32, 64, 128])
    else:
        P, N = rng.choice([(64, 128), (64, 128), (64, 64), (32, 128), (48, 64), (128, 128)])
    # up to 32768 tokens of 64 heads of 64 (counted padded to the longest prompt)
    tokens = 32768 * 64 * 64 // (H * P) if not fp32 else 4096
    batch = _log_int(rng, 1, 64)
    longest = _log_int(rng, 1, max(1, min(16384, tokens // batch)))
    case = dict(op=op, batch=batch, longest=longest, ragged=rng.random() < 0.7, lens=rng.randrange(1000), H=H, P=P, N=N, G=G)
    return dict(case, dtype="fp32" if fp32 else "bf16") if op == "scan" else case


def _lengths(case):
    """The prompts' lengths: all alike, or spread over 1 .. longest by their logarithm."""
    if not case["ragged"]:
        return [case["longest"]] * case["batch"]
    r = random.Random(case["lens"])
    lens = [_log_int(r, 1, case["longest"]) for _ in range(case["batch"])]
    lens[r.randrange(case["batch"])] = case["longest"]
    return lens


def work(case):
    op = case["op"]
    if op == "add":
        n, el = case["rows"] * case["dim"], 4 if case["stream"] == "fp32" else 2
        return dict(bytes=n * (2 * el + 4) + case["dim"] * 4 * (1 + case["post"] + case["gate"]), flops=10 * n)
    H, P, N, G = case["H"], case["P"], case["N"], case["G"]
    if op == "gate":
        return dict(bytes=case["rows"] * H * P * 8 + 4 * H * P, flops=10 * case["rows"] * H * P)
    T, chans = sum(_lengths(case)), H * P + 2 * G * N
    if op == "conv":
        return dict(bytes=T * (4 * chans + 6 * H) + case["batch"] * 12 * chans + 20 * chans, flops=T * chans * 13)
    el = 4 if case["dtype"] == "fp32" else 2
    # the recurrence as it is defined: decay, rank-1 update and output, 5 operations per state element
    return dict(bytes=T * (chans * el + 4 * H * P + 4 * H) + 8 * case["batch"] * H * P * N, flops=5 * T * H * P * N)


# ------------------------------------------------------------------ inputs

def _desc(case, batch):
    """The framework's description of the layer, which its calls take."""
    if not own:
        return None
    from hybrid_model_ssm_replay_b200 import rssm
    return rssm.make_desc(batch, case["H"], case["P"], case["N"], case["G"], in_dtype=rssm.RSSM_F32 if case.get("dtype") == "fp32" else rssm.RSSM_BF16)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]

    def rn(*size, std=1.0, dtype=torch.float32):
        return (torch.randn(size, generator=g, device="cuda") * std).to(dtype)

    if op == "add":
        d, t = case["dim"], torch.float32 if case["stream"] == "fp32" else torch.bfloat16
        s = dict(u=rn(case["rows"], d, std=2.0, dtype=t), v=rn(case["rows"], d, dtype=torch.bfloat16),
                 post_w=1 + rn(d, std=0.1) if case["post"] else None,
                 gate=rn(d, std=0.5) if case["gate"] else None, pre_w=1 + rn(d, std=0.1))
        s.update(u_out=torch.zeros_like(s["u"]), out=torch.zeros_like(s["v"]), scale=case["scale"])
        return dict(s, op=op)
    H, P, N, G = case["H"], case["P"], case["N"], case["G"]
    din, gn = H * P, G * N
    if op == "gate":
        rows = case["rows"]
        return dict(op=op, H=H, P=P, N=N, G=G, y=rn(rows, H, P), w=1 + rn(din, std=0.1), desc=_desc(case, 1),
                    zx=rn(rows, 2 * din + 2 * gn + H, std=1.5, dtype=torch.bfloat16),
                    out=torch.zeros(rows, din, dtype=torch.bfloat16, device="cuda"))
    lens = _lengths(case)
    T, batch, chans = sum(lens), case["batch"], din + 2 * gn
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    s = dict(op=op, H=H, P=P, N=N, G=G, lens=lens, longest=max(lens), cu=cu, batch=batch, desc=_desc(case, batch))
    if op == "conv":
        s.update(zx=rn(T, 2 * din + 2 * gn + H, std=1.5, dtype=torch.bfloat16), w=rn(chans, 4, std=0.5),
                 b=rn(chans, std=0.1), dt_bias=rn(H, std=0.5) - 3.0, state=rn(batch, 3, chans, dtype=torch.bfloat16),
                 x=torch.zeros(T, H, P, dtype=torch.bfloat16, device="cuda"),
                 B=torch.zeros(T, G, N, dtype=torch.bfloat16, device="cuda"),
                 C=torch.zeros(T, G, N, dtype=torch.bfloat16, device="cuda"), dt=torch.zeros(T, H, device="cuda"))
        return s
    # the distributions of the framework's decode inputs (A, D, dt, checkpoint)
    t = torch.float32 if case["dtype"] == "fp32" else torch.bfloat16
    s.update(x=rn(T, H, P, dtype=t), B=rn(T, G, N, dtype=t), C=rn(T, G, N, dtype=t),
             dt=torch.nn.functional.softplus(rn(T, H) - 3.0),
             A=-torch.exp(torch.rand(H, generator=g, device="cuda") * math.log(16.0)), D=rn(H),
             ckpt=rn(batch, H, P, N, std=0.1), y=torch.zeros(T, H, P, device="cuda"))
    if own:  # the layer's state, which a user's program keeps from the prompt to the last decoded token
        from hybrid_model_ssm_replay_b200 import rssm
        s["layer"] = rssm.RssmState(s["desc"])
        s["layer"].ckpt.copy_(s.pop("ckpt"))
    return s


# --------------------------------------------------------------------- run

def run(s):
    return {"scan": _scan, "conv": _conv, "gate": _gate, "add": _add}[s["op"]](s)


def _places(s):
    """Row of the packed tokens for place i of prompt b, [batch][longest], and where there is one."""
    start = s["cu"][:-1].long()[:, None]
    i = torch.arange(s["longest"], device="cuda")[None, :]
    there = start + i < s["cu"][1:].long()[:, None]
    return torch.where(there, start + i, torch.zeros_like(i)), there


def _scan(s):
    if own:
        from hybrid_model_ssm_replay_b200 import rssm
        rssm.rssm_prefill_scan(s["layer"], s["cu"], s["longest"], s["x"], s["B"], s["C"], s["dt"], s["A"], s["D"], s["y"])
        return [s["y"], s["layer"].ckpt]
    # blocks of CHUNK tokens: products within a block, the state between blocks by their decays
    H, P, N, G, b, Q = s["H"], s["P"], s["N"], s["G"], s["batch"], CHUNK
    rows, there = _places(s)
    nc = -(-s["longest"] // Q)
    fill = nc * Q - s["longest"]
    rows = torch.nn.functional.pad(rows, (0, fill))
    there = torch.nn.functional.pad(there, (0, fill))

    def blocks(v, *tail):  # packed tokens -> [batch][block][token] + tail, zeros where there is none
        v = v.float()[rows] * there.view(b, nc * Q, *([1] * (v.dim() - 1)))
        return v.view(b, nc, Q, *tail)

    x, B, C, dt = blocks(s["x"], G, H // G, P), blocks(s["B"], G, N), blocks(s["C"], G, N), blocks(s["dt"], G, H // G)
    a = (dt.double() * s["A"].double().view(G, H // G)).cumsum(2)              # log decay within the block
    seen = torch.ones(Q, Q, dtype=torch.bool, device="cuda").tril()
    diff = a.permute(0, 1, 3, 4, 2)
    diff = diff[..., :, None] - diff[..., None, :]
    decay = torch.exp(diff.masked_fill_(~seen, -math.inf)).float()              # [b][nc][G][hpg][t][s]
    del diff
    cb = torch.einsum("bctgn,bcsgn->bcgts", C, B)
    m = decay.mul_(cb[:, :, :, None])
    dx = dt[..., None] * x
    y = torch.einsum("bcghts,bcsghp->bctghp", m, dx)
    del m, decay
    last = a[:, :, -1]
    rest = torch.exp(last[:, :, None] - a).float()
    own_state = torch.einsum("bcsghp,bcsgn->bcghpn", rest[..., None] * dx, B)   # what each block adds
    h0 = s["ckpt"].view(b, 1, G, H // G, P, N)
    states = torch.cat([h0, own_state], 1)
    del own_state
    total = torch.cat([torch.zeros_like(last[:, :1]), last], 1).cumsum(1)       # [b][nc + 1][G][hpg]
    gap = total[:, :, None] - total[:, None, :]                                 # from block j's end to block i's
    order = torch.ones(nc + 1, nc + 1, dtype=torch.bool, device="cuda").tril()[None, :, :, None, None]
    carry = torch.exp(gap.masked_fill(~order, -math.inf)).float()
    states = torch.einsum("bijgh,bjghpn->bighpn", carry, states)
    y = y + torch.einsum("bctgn,bcghpn->bctghp", C, states[:, :-1]) * torch.exp(a).float()[..., None]
    y = y + s["D"].view(G, H // G, 1) * x
    s["y"][rows[there]] = y.reshape(b, nc * Q, H, P)[there]
    s["ckpt"].copy_(states[:, -1].reshape(b, H, P, N))
    return [s["y"], s["ckpt"]]


def _conv(s):
    if own:
        from hybrid_model_ssm_replay_b200 import stage
        stage.rssm_stage_conv_prompt(s["desc"], s["cu"], s["zx"], s["state"], s["w"], s["b"], s["dt_bias"], s["x"], s["B"], s["C"], s["dt"])
        return [s["x"], s["B"], s["C"], s["dt"], s["state"]]
    din, gn, H, T = s["H"] * s["P"], s["G"] * s["N"], s["H"], s["zx"].shape[0]
    raw = s["zx"][:, din:2 * din + 2 * gn]
    rows, there = _places(s)
    prompt = torch.zeros(T, dtype=torch.long, device="cuda")
    prompt[rows[there]] = torch.arange(s["batch"], device="cuda")[:, None].expand_as(rows)[there]
    place = torch.arange(T, device="cuda") - s["cu"].long()[prompt]             # within its prompt

    def back(k):  # the input k tokens earlier: of the prompt, or of the state before it
        t = torch.arange(T, device="cuda") - k
        old = s["state"][prompt, (3 + place - k).clamp(max=2)]
        return torch.where((place >= k)[:, None], raw[t.clamp(min=0)], old).float()

    o = s["b"] + s["w"][:, 3] * raw.float() + s["w"][:, 2] * back(1) + s["w"][:, 1] * back(2) + s["w"][:, 0] * back(3)
    act = (o / (1 + torch.exp(-o))).to(torch.bfloat16)
    v = s["zx"][:, 2 * din + 2 * gn:].float() + s["dt_bias"]
    s["x"].copy_(act[:, :din].view_as(s["x"]))
    s["B"].copy_(act[:, din:din + gn].view_as(s["B"]))
    s["C"].copy_(act[:, din + gn:].view_as(s["C"]))
    s["dt"].copy_(torch.where(v > 20, v, torch.log1p(torch.exp(v))))
    n = (s["cu"][1:] - s["cu"][:-1]).long()[:, None]
    at = n - 3 + torch.arange(3, device="cuda")[None, :]                        # the last three inputs
    new = raw[(s["cu"][:-1].long()[:, None] + at).clamp(0, T - 1)]
    old = torch.gather(s["state"], 1, (at + 3).clamp(0, 2)[..., None].expand(-1, -1, raw.shape[1]))
    s["state"].copy_(torch.where((at >= 0)[..., None], new, old))
    return [s["x"], s["B"], s["C"], s["dt"], s["state"]]


def _gate(s):
    if own:
        from hybrid_model_ssm_replay_b200 import stage
        stage.rssm_stage_gate_norm_prompt(s["desc"], s["y"], s["zx"], s["w"], EPS, s["out"])
        return s["out"]
    din = s["H"] * s["P"]
    z = s["zx"][:, :din].float()
    v = (s["y"].view(-1, din) * (z / (1 + torch.exp(-z)))).view(-1, s["G"], din // s["G"])
    v = v / torch.sqrt((v * v).mean(-1, keepdim=True) + EPS)
    s["out"].copy_(v.view(-1, din) * s["w"])
    return s["out"]


def _add(s):
    if own:
        from hybrid_model_ssm_replay_b200 import stage
        stage.rssm_stage_add_norm(s["u"], s["v"], s["pre_w"], EPS, s["out"], post_w=s["post_w"], gate=s["gate"], scale=s["scale"], u_out=s["u_out"])
        return [s["u_out"], s["out"]]
    v = s["v"].float()
    if s["post_w"] is not None:
        v = v / torch.sqrt((v * v).mean(-1, keepdim=True) + EPS) * s["post_w"]
    if s["gate"] is not None:
        v = v * s["gate"]
    s["u_out"].copy_(s["u"].float() + s["scale"] * v)
    u = s["u_out"].float()  # the stream as it is kept
    s["out"].copy_(u / torch.sqrt((u * u).mean(-1, keepdim=True) + EPS) * s["pre_w"])
    return [s["u_out"], s["out"]]


# ------------------------------------------------------------------- exact

def exact(case, seed):
    s = prepare(case, seed)
    d = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() and v.numel() < 1 << 31 else v for k, v in s.items() if k not in ("y", "out", "layer") or case["op"] == "gate"}
    if case["op"] == "add":
        v = d["v"]
        if d["post_w"] is not None:
            v = v * torch.rsqrt(v.square().mean(1, keepdim=True) + EPS) * d["post_w"]
        u = d["u"] + d["scale"] * (v if d["gate"] is None else v * d["gate"])
        kept = u.to(s["u"].dtype).double()  # the norm is of the stream as it is kept
        return [u, kept * torch.rsqrt(kept.square().mean(1, keepdim=True) + EPS) * d["pre_w"]]
    H, P, N, G = case["H"], case["P"], case["N"], case["G"]
    din, gn = H * P, G * N
    if case["op"] == "gate":
        v = d["y"].view(-1, din) * torch.nn.functional.silu(s["zx"][:, :din].double())
        v = v.view(-1, G, din // G)
        return (v * torch.rsqrt(v.square().mean(2, keepdim=True) + EPS)).view(-1, din) * d["w"]
    cu = [0]
    for n in s["lens"]:
        cu.append(cu[-1] + n)
    if case["op"] == "conv":
        acts, states = [], []
        for b, n in enumerate(s["lens"]):  # one prompt at a time, its state before it
            run_in = torch.cat([s["state"][b], s["zx"][cu[b]:cu[b + 1], din:2 * din + 2 * gn]]).double()
            o = torch.nn.functional.conv1d(run_in.T[None], d["w"][:, None, :], d["b"], groups=run_in.shape[1])[0].T
            acts.append(torch.nn.functional.silu(o))
            states.append(run_in[-3:])
        act = torch.cat(acts)
        dt = torch.nn.functional.softplus(s["zx"][:, 2 * din + 2 * gn:].double() + d["dt_bias"])
        return [act[:, :din].reshape(-1, H, P), act[:, din:din + gn].reshape(-1, G, N), act[:, din + gn:].reshape(-1, G, N), dt, torch.stack(states)]
    # the recurrence, token by token, for all prompts at once (a prompt that has ended keeps its state)
    if case["batch"] * H * P * N * case["longest"] > 1 << 38:
        return None
    h = d["ckpt"].view(case["batch"], G, H // G, P, N).clone()
    y = torch.zeros(cu[-1], H, P, dtype=torch.float64, device="cuda")
    lens, start = torch.tensor(s["lens"], device="cuda"), torch.tensor(cu[:-1], device="cuda")
    for t in range(s["longest"]):
        if case["ragged"]:
            live = (lens > t).nonzero()[:, 0]
            hl, at = h[live], start[live] + t
        else:
            live, hl, at = None, h, start + t
        dt = d["dt"][at].view(-1, G, H // G, 1, 1)
        x = d["x"][at].view(-1, G, H // G, P, 1)
        hl.mul_(torch.exp(dt * d["A"].view(G, H // G, 1, 1)))
        hl.addcmul_(dt * x, d["B"][at].view(-1, G, 1, 1, N))
        out = torch.matmul(hl, d["C"][at].view(-1, G, 1, N, 1))[..., 0] + d["D"].view(G, H // G, 1) * x[..., 0]
        y[at] = out.reshape(-1, H, P)
        if live is not None:
            h[live] = hl
    return [y, h.view(case["batch"], H, P, N)]
