"""A synthetic hybrid SSM/attention decode stage around librssm.

The ReplaySSM article (devotd.net "nvidia-replayssm-hybrid-model-ssm-
decoding-state-buffer", s2 "Reduce state transfers at large batch sizes")
reports the SSM-kernel speed-up diluted by the rest of each decode step: a
decode-stage gain smaller than the kernel gain, and none at batch 1. This
module builds such a stage with random weights so the dilution can be
measured: n_ssm Mamba-2 mixer blocks and n_attn attention blocks, one decode
token per request per step.

Mamba-2 mixer block (Dao and Gu, "Transformers are SSMs", ICML 2024), per
request, u the residual stream [d_model]:
    zxbcdt = W_in^T rmsnorm(u)                      (GEMM, bf16, cuBLAS via torch)
    x, B, C, dt = conv1d+SiLU, softplus             (rssm_stage_conv)
    y = SSM step                                    (rssm_decode_step [+ rssm_flush], or rssm_conv_step)
    v = gated RMS norm(y, z)                        (rssm_stage_gate_norm)
    u += W_out^T v                                  (GEMM)
Attention block (the stand-in for a hybrid model's attention layers):
    q, k, v = W_qkv^T rmsnorm(u); k, v overwrite the oldest slot of a KV
    cache of ctx tokens; o = softmax(q K^T / sqrt(d)) V (torch SDPA, GQA);
    u += W_o^T o.
The projections and the attention are library calls; the SSM step and the
block's element-wise glue run in librssm's kernels. scheme="replay" uses the
replay decode (flush every interval tokens); scheme="conventional" the
per-token read + write kernel on the same inputs and weights.

HybridStage.prefill runs a prompt through the same blocks at once (replay
scheme): the prompt forms of the block's steps, rssm_stage_conv_prompt,
rssm_prefill_scan, rssm_stage_gate_norm_prompt and rssm_stage_add_norm, between
the same GEMMs, and attention over the cache with the prompt's own tokens.
"""
import ctypes as ct
import math
from dataclasses import dataclass

import torch

from . import rssm


@dataclass(frozen=True)
class StageShape:
    batch: int
    d_model: int
    nheads: int          # SSM heads H
    head_dim: int        # P
    d_state: int         # N
    ngroups: int         # G
    interval: int = 16
    n_ssm: int = 4       # Mamba-2 blocks per stage
    n_attn: int = 1      # attention blocks per stage
    attn_heads: int = 16
    kv_heads: int = 4
    attn_head_dim: int = 128
    ctx: int = 1024      # KV-cache length each attention block attends over
    eps: float = 1e-5

    @property
    def d_inner(self):
        return self.nheads * self.head_dim

    @property
    def d_proj(self):
        return 2 * self.d_inner + 2 * self.ngroups * self.d_state + self.nheads


def _lib():
    L = rssm.lib()
    if not hasattr(L, "_stage_sigs"):
        vp, D = ct.c_void_p, ct.POINTER(rssm.Desc)
        L.rssm_stage_conv.argtypes = [D, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
        L.rssm_stage_conv.restype = ct.c_int
        L.rssm_stage_gate_norm.argtypes = [D, vp, vp, vp, ct.c_float, vp, vp]
        L.rssm_stage_gate_norm.restype = ct.c_int
        i32, f32 = ct.c_int32, ct.c_float
        L.rssm_stage_conv_prompt.argtypes = [D, i32] + [vp] * 12
        L.rssm_stage_conv_prompt.restype = ct.c_int
        L.rssm_stage_gate_norm_prompt.argtypes = [D, i32, vp, vp, vp, f32, vp, vp]
        L.rssm_stage_gate_norm_prompt.restype = ct.c_int
        L.rssm_stage_add_norm.argtypes = [i32, i32, i32, vp, vp, vp, vp, f32, vp, f32, vp, vp, vp]
        L.rssm_stage_add_norm.restype = ct.c_int
        L._stage_sigs = True
    return L


def rssm_stage_conv(desc, zxbcdt, conv_state, conv_w, conv_b, dt_bias, x, B, C, dt, stream=None):
    p = rssm._ptr
    rssm._check(_lib().rssm_stage_conv(ct.byref(desc), p(zxbcdt, torch.bfloat16, "zxbcdt"),
                                       p(conv_state, torch.bfloat16, "conv_state"),
                                       p(conv_w, torch.float32, "conv_w"), p(conv_b, torch.float32, "conv_b"),
                                       p(dt_bias, torch.float32, "dt_bias"), p(x, torch.bfloat16, "x"),
                                       p(B, torch.bfloat16, "B"), p(C, torch.bfloat16, "C"),
                                       p(dt, torch.float32, "dt"), rssm._stream(stream)), "rssm_stage_conv")


def rssm_stage_gate_norm(desc, y, zxbcdt, norm_w, eps, out, stream=None):
    p = rssm._ptr
    rssm._check(_lib().rssm_stage_gate_norm(ct.byref(desc), p(y, torch.float32, "y"),
                                            p(zxbcdt, torch.bfloat16, "zxbcdt"),
                                            p(norm_w, torch.float32, "norm_w"), float(eps),
                                            p(out, torch.bfloat16, "out"), rssm._stream(stream)),
                "rssm_stage_gate_norm")


def rssm_stage_conv_prompt(desc, cu_seqlens, zxbcdt, conv_state, conv_w, conv_b, dt_bias, x, B, C, dt, err=None,
                           stream=None):
    """rssm_stage_conv for every token of packed prompts; conv_state is read
    and updated. err: the state's error word (RssmState.err), or None."""
    a, bf, f32, dev = rssm._arg, torch.bfloat16, torch.float32, rssm._device(zxbcdt, "zxbcdt")
    H, P, N, G = desc.nheads, desc.head_dim, desc.d_state, desc.ngroups
    total, chans = rssm._rows(zxbcdt, "zxbcdt"), H * P + 2 * G * N
    rssm._check(_lib().rssm_stage_conv_prompt(
        ct.byref(desc), total, a(cu_seqlens, torch.int32, (desc.batch + 1,), "cu_seqlens", dev),
        a(zxbcdt, bf, (total, H * P + chans + H), "zxbcdt", dev),
        a(conv_state, bf, (desc.batch, 3, chans), "conv_state", dev), a(conv_w, f32, (chans, 4), "conv_w", dev),
        a(conv_b, f32, (chans,), "conv_b", dev), a(dt_bias, f32, (H,), "dt_bias", dev),
        a(x, bf, (total, H, P), "x", dev), a(B, bf, (total, G, N), "B", dev), a(C, bf, (total, G, N), "C", dev),
        a(dt, f32, (total, H), "dt", dev), a(err, torch.int32, (1,), "err", dev), rssm._stream(stream)),
        "rssm_stage_conv_prompt")


def rssm_stage_gate_norm_prompt(desc, y, zxbcdt, norm_w, eps, out, stream=None):
    """rssm_stage_gate_norm for every row of packed prompts (desc's batch is
    not used); y [rows][d_inner] or [rows][H][P]."""
    a, bf, f32, dev = rssm._arg, torch.bfloat16, torch.float32, rssm._device(zxbcdt, "zxbcdt")
    H, P = desc.nheads, desc.head_dim
    rows, din = rssm._rows(zxbcdt, "zxbcdt"), H * P
    rssm._check(_lib().rssm_stage_gate_norm_prompt(
        ct.byref(desc), rows, a(y, f32, (rows, din) if y.dim() == 2 else (rows, H, P), "y", dev),
        a(zxbcdt, bf, (rows, 2 * din + 2 * desc.ngroups * desc.d_state + H), "zxbcdt", dev),
        a(norm_w, f32, (din,), "norm_w", dev), float(eps), a(out, bf, (rows, din), "out", dev), rssm._stream(stream)),
        "rssm_stage_gate_norm_prompt")
    return out


def rssm_stage_add_norm(u, v, pre_w, eps, out, post_w=None, gate=None, scale=1.0, u_out=None, stream=None):
    """u_out = u + scale * gate * norm(v, post_w); out = norm(u_out, pre_w).
    u_out None: u itself is updated. v None: the norm of u alone (u_out then
    receives a copy, if it is given). pre_w and out None: no norm."""
    a, bf, f32, dev = rssm._arg, torch.bfloat16, torch.float32, rssm._device(u, "u")
    if u.dim() != 2:
        raise ValueError(f"u has shape {tuple(u.shape)}, expected rows of one width")
    shape, wide, rows = u.shape, u.shape[1:], rssm._rows(u, "u")
    if shape[1] > rssm.I32_MAX:
        raise ValueError(f"u is {shape[1]} wide, more than a call takes")
    t = f32 if u.dtype == f32 else bf
    up = a(u, t, shape, "u", dev)
    uo = (None if v is None else up) if u_out is None else a(u_out, t, shape, "u_out", dev)
    rssm._check(_lib().rssm_stage_add_norm(
        rows, shape[1], rssm.RSSM_F32 if t == f32 else rssm.RSSM_BF16, up, a(v, bf, shape, "v", dev),
        a(post_w, f32, wide, "post_w", dev), a(gate, f32, wide, "gate", dev), float(scale),
        a(pre_w, f32, wide, "pre_w", dev), float(eps), uo, a(out, bf, shape, "out", dev), rssm._stream(stream)),
        "rssm_stage_add_norm")
    return out


def rmsnorm(u, w, eps):
    """Pre-norm of a block (fp32 arithmetic, bf16 result)."""
    uf = u.float()
    return (uf * torch.rsqrt(uf.pow(2).mean(-1, keepdim=True) + eps) * w).to(torch.bfloat16)


def make_weights(shape: StageShape, seed: int, device="cuda"):
    """Random weights of the stage (seeded; scaled so activations stay O(1))."""
    g = torch.Generator(device="cpu").manual_seed(seed)

    def rn(*size, std=1.0):
        return (torch.randn(*size, generator=g) * std)

    s = shape
    chans = s.d_inner + 2 * s.ngroups * s.d_state
    blocks = []
    for _ in range(s.n_ssm):
        blocks.append({
            "norm": (1.0 + 0.1 * rn(s.d_model)).float(),
            "w_in": rn(s.d_model, s.d_proj, std=1.0 / math.sqrt(s.d_model)).to(torch.bfloat16),
            "conv_w": rn(chans, 4, std=0.5).float(),
            "conv_b": rn(chans, std=0.1).float(),
            "dt_bias": (torch.rand(s.nheads, generator=g) * 2.0 - 4.0).float(),
            "A": (-torch.exp(torch.rand(s.nheads, generator=g) * math.log(16.0))).float(),
            "D": rn(s.nheads).float(),
            "gnorm": (1.0 + 0.1 * rn(s.d_inner)).float(),
            "w_out": rn(s.d_inner, s.d_model, std=1.0 / math.sqrt(s.d_inner)).to(torch.bfloat16),
        })
    attn = []
    qkv = (s.attn_heads + 2 * s.kv_heads) * s.attn_head_dim
    for _ in range(s.n_attn):
        attn.append({
            "norm": (1.0 + 0.1 * rn(s.d_model)).float(),
            "w_qkv": rn(s.d_model, qkv, std=1.0 / math.sqrt(s.d_model)).to(torch.bfloat16),
            "w_o": rn(s.attn_heads * s.attn_head_dim, s.d_model,
                      std=1.0 / math.sqrt(s.attn_heads * s.attn_head_dim)).to(torch.bfloat16),
        })
    mv = lambda d: {k: v.to(device) for k, v in d.items()}
    return [mv(b) for b in blocks], [mv(a) for a in attn]


class HybridStage:
    """n_ssm Mamba-2 blocks then n_attn attention blocks, one decode token per
    request per step(); scheme "replay" or "conventional" for the SSM step."""

    def __init__(self, shape: StageShape, weights, scheme="replay", seed=0, device="cuda"):
        assert scheme in ("replay", "conventional")
        s = self.shape = shape
        self.scheme = scheme
        self.blocks, self.attn = weights
        self.desc = rssm.make_desc(s.batch, s.nheads, s.head_dim, s.d_state, s.ngroups, interval=s.interval)
        g = torch.Generator(device="cpu").manual_seed(seed + 1)
        chans = s.d_inner + 2 * s.ngroups * s.d_state
        self.ssm = []
        for _ in range(s.n_ssm):
            ck = (torch.randn(s.batch, s.nheads, s.head_dim, s.d_state, generator=g) * 0.1).to(device)
            if scheme == "replay":
                st = rssm.RssmState(self.desc, device)
                st.ckpt.copy_(ck)
            else:
                st = ck
            self.ssm.append({"state": st,
                             "conv": torch.zeros(s.batch, 3, chans, dtype=torch.bfloat16, device=device)})
        self.kv = []
        for _ in range(s.n_attn):
            kc = (torch.randn(s.batch, s.kv_heads, s.ctx, s.attn_head_dim, generator=g)).to(torch.bfloat16)
            vc = (torch.randn(s.batch, s.kv_heads, s.ctx, s.attn_head_dim, generator=g)).to(torch.bfloat16)
            self.kv.append({"k": kc.to(device), "v": vc.to(device)})
        self.t = 0
        self.t0 = 0  # the token from which the replay intervals count
        B_, din, gn = s.batch, s.d_inner, s.ngroups * s.d_state
        self.zx = torch.empty(B_, s.d_proj, dtype=torch.bfloat16, device=device)
        self.x = torch.empty(B_, s.nheads, s.head_dim, dtype=torch.bfloat16, device=device)
        self.Bv = torch.empty(B_, s.ngroups, s.d_state, dtype=torch.bfloat16, device=device)
        self.Cv = torch.empty_like(self.Bv)
        self.dt = torch.empty(B_, s.nheads, dtype=torch.float32, device=device)
        self.y = torch.empty(B_, s.nheads, s.head_dim, dtype=torch.float32, device=device)
        self.v = torch.empty(B_, din, dtype=torch.bfloat16, device=device)

    def ssm_block(self, i, u):
        s, b = self.shape, self.blocks[i]
        st = self.ssm[i]
        torch.matmul(rmsnorm(u, b["norm"], s.eps), b["w_in"], out=self.zx)
        rssm_stage_conv(self.desc, self.zx, st["conv"], b["conv_w"], b["conv_b"], b["dt_bias"],
                        self.x, self.Bv, self.Cv, self.dt)
        if self.scheme == "replay":
            rssm.rssm_decode_step(st["state"], self.x, self.Bv, self.Cv, self.dt, b["A"], b["D"], self.y)
            if (self.t + 1 - self.t0) % s.interval == 0:
                rssm.rssm_flush(st["state"], b["A"])
        else:
            rssm.rssm_conv_step(self.desc, st["state"], self.x, self.Bv, self.Cv, self.dt, b["A"], b["D"], self.y)
        rssm_stage_gate_norm(self.desc, self.y, self.zx, b["gnorm"], s.eps, self.v)
        return u + torch.matmul(self.v, b["w_out"])

    def attn_block(self, i, u):
        s, a, kv = self.shape, self.attn[i], self.kv[i]
        hq, hk, hd = s.attn_heads, s.kv_heads, s.attn_head_dim
        qkv = torch.matmul(rmsnorm(u, a["norm"], s.eps), a["w_qkv"])
        q = qkv[:, :hq * hd].view(s.batch, hq, 1, hd)
        k = qkv[:, hq * hd:(hq + hk) * hd].view(s.batch, hk, hd)
        v = qkv[:, (hq + hk) * hd:].view(s.batch, hk, hd)
        slot = self.t % s.ctx
        kv["k"][:, :, slot].copy_(k)
        kv["v"][:, :, slot].copy_(v)
        o = torch.nn.functional.scaled_dot_product_attention(q, kv["k"], kv["v"], enable_gqa=True)
        return u + torch.matmul(o.reshape(s.batch, hq * hd), a["w_o"])

    def step(self, u):
        """One decode token per request: u [batch][d_model] bf16 -> same."""
        for i in range(self.shape.n_ssm):
            u = self.ssm_block(i, u)
        for i in range(self.shape.n_attn):
            u = self.attn_block(i, u)
        self.t += 1
        return u

    def prefill(self, u):
        """T prompt tokens per request at once: u [batch][T][d_model] bf16 ->
        the residual stream after the stage, of every token. The same tokens
        through step(), one by one, give the same up to rounding; step() goes
        on from here. Replay scheme; T at most ctx when there is attention."""
        s = self.shape
        if self.scheme != "replay":
            raise ValueError("prefill needs the replay scheme (a checkpoint to scan into)")
        if u.dim() != 3 or u.shape[0] != s.batch or u.shape[2] != s.d_model or u.dtype != torch.bfloat16:
            raise ValueError(f"u must be bf16 [{s.batch}][T][{s.d_model}]")
        T = int(u.shape[1])
        if s.n_attn and T > s.ctx:
            raise ValueError(f"a prompt of {T} tokens does not fit the attention cache of {s.ctx}")
        if T == 0:
            return u.clone()
        if (self.t - self.t0) % s.interval:  # decoded tokens still in the buffers
            for b, st in zip(self.blocks, self.ssm):
                rssm.rssm_flush(st["state"], b["A"], force=True)
            self.t0 = self.t  # the buffers are empty, whatever comes of the prompt
        rows, dev = s.batch * T, u.device
        u = u.reshape(rows, s.d_model).clone(memory_format=torch.contiguous_format)
        cu = torch.arange(s.batch + 1, dtype=torch.int32, device=dev) * T
        kw = dict(dtype=torch.bfloat16, device=dev)
        n = torch.empty(rows, s.d_model, **kw)
        zx = torch.empty(rows, s.d_proj, **kw)
        x = torch.empty(rows, s.nheads, s.head_dim, **kw)
        Bv = torch.empty(rows, s.ngroups, s.d_state, **kw)
        Cv = torch.empty_like(Bv)
        dt = torch.empty(rows, s.nheads, device=dev)
        y = torch.empty(rows, s.nheads, s.head_dim, device=dev)
        v = torch.empty(rows, s.d_inner, **kw)
        norms = [b["norm"] for b in self.blocks] + [a["norm"] for a in self.attn] + [None]
        if norms[0] is not None:
            rssm_stage_add_norm(u, None, norms[0], s.eps, n)
        for i, b in enumerate(self.blocks):
            st = self.ssm[i]
            torch.matmul(n, b["w_in"], out=zx)
            rssm_stage_conv_prompt(self.desc, cu, zx, st["conv"], b["conv_w"], b["conv_b"], b["dt_bias"], x, Bv, Cv,
                                   dt, err=st["state"].err)
            rssm.rssm_prefill_scan(st["state"], cu, T, x, Bv, Cv, dt, b["A"], b["D"], y)
            rssm_stage_gate_norm_prompt(self.desc, y, zx, b["gnorm"], s.eps, v)
            nxt = norms[i + 1]
            rssm_stage_add_norm(u, torch.matmul(v, b["w_out"]), nxt, s.eps, None if nxt is None else n)
        for i in range(s.n_attn):
            nxt = norms[s.n_ssm + i + 1]
            rssm_stage_add_norm(u, self._attn_prompt(i, n, T), nxt, s.eps, None if nxt is None else n)
        self.t += T
        self.t0 = self.t
        return u.view(s.batch, T, s.d_model)

    def _attn_prompt(self, i, n, T):
        """An attention block's output for T tokens per request: token j sees
        the prompt's tokens up to itself and the cache slots that none of
        them has overwritten."""
        s, a, kv = self.shape, self.attn[i], self.kv[i]
        hq, hk, hd = s.attn_heads, s.kv_heads, s.attn_head_dim
        qkv = torch.matmul(n, a["w_qkv"]).view(s.batch, T, hq + 2 * hk, hd).transpose(1, 2)
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        j = torch.arange(T, device=n.device)
        age = (torch.arange(s.ctx, device=n.device) - self.t) % s.ctx  # the token that overwrites the slot
        seen = torch.cat([age[None, :] > j[:, None], j[None, :] <= j[:, None]], 1)
        o = torch.nn.functional.scaled_dot_product_attention(
            q, torch.cat([kv["k"], k], 2), torch.cat([kv["v"], v], 2), attn_mask=seen, enable_gqa=True)
        slots = (self.t + j) % s.ctx
        kv["k"][:, :, slots] = k
        kv["v"][:, :, slots] = v
        return torch.matmul(o.transpose(1, 2).reshape(s.batch * T, hq * hd), a["w_o"])
