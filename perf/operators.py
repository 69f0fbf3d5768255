"""Cases of the gated delta rule and of the q/k norm with rotation.

Each case names an operator, its sizes and its element type:

* ``prefill``: the chunked gated delta rule over a prompt, from a carried
  state: outputs and the state after the last token;
* ``train``: forward and backward of the same (gradients of q, k, v, the log
  decay, the write strength and, with a carried state, of that state);
* ``decode``: one token per sequence, the state updated in place, in a pool
  of states addressed by slot where the case says so;
* ``rope``: the per-head norm of queries and keys with the position rotation,
  from token-major projection rows to head-major rows; with ``train`` its
  backward too (gradients of the rows and of the norm's weights).
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
CHUNK = 64          # rows of a chunk in the plain form


def _delta(name, op, dtype, B, H, Hk, N, D, M, carry=False, **more):
    return dict(name=name, op=op, dtype=dtype, B=B, H=H, Hk=Hk, N=N, D=D, M=M, carry=carry, **more)


def _rope(name, dtype, B, H, Hk, N, D, R, norm, train):
    return dict(name=name, op="rope", dtype=dtype, B=B, H=H, Hk=Hk, N=N, D=D, R=R, norm=norm,
                train=train)


def listed():
    return [
        # one sequence being answered: a token's step, where latency counts
        _delta("decode_b1_h16_d64", "decode", "bf16", 1, 16, 16, 1, 64, 64, slots=0),
        # a full serving batch at the sizes the decode step is benchmarked at
        _delta("decode_b512_h16_d64", "decode", "bf16", 512, 16, 16, 1, 64, 64, slots=0),
        # a batch out of a larger pool of states, some of its rows idle, shared key heads
        _delta("decode_b61_h8_d128_slots", "decode", "f16", 61, 8, 4, 1, 128, 128, slots=96),
        # the smallest workload, fp32
        _delta("prefill_f32_h2_n64_d16", "prefill", "f32", 1, 2, 2, 64, 16, 16),
        # the main training shape as a batch of prompts
        _delta("prefill_bf16_b8h16_n4096_d64", "prefill", "bf16", 8, 16, 16, 4096, 64, 64),
        # prompts of an odd length that continue a conversation, two value heads to a key head
        _delta("prefill_bf16_b4h8_n8229_d128_m64", "prefill", "bf16", 4, 8, 4, 8229, 128, 64,
               carry=True),
        # few heads over a long document
        _delta("prefill_bf16_b2h8_n32768_d128", "prefill", "bf16", 2, 8, 8, 32768, 128, 128),
        # a training step at a short context
        _delta("train_bf16_b4h8_n1024_d64", "train", "bf16", 4, 8, 8, 1024, 64, 64),
        # a training step at the main shape
        _delta("train_bf16_b8h16_n4096_d64", "train", "bf16", 8, 16, 16, 4096, 64, 64),
        # full precision, an odd length, shared key heads, a carried state with its gradient
        _delta("train_f32_b2h4_n509_d64", "train", "f32", 2, 4, 2, 509, 64, 64, carry=True),
        # the norm and rotation of a serving batch's new tokens
        _rope("rope_f16_b61_n1_h16_d64", "f16", 61, 16, 4, 1, 64, 64, "rms", False),
        # the norm and rotation of a training step, a quarter of the features turned
        _rope("rope_train_bf16_b8h16_n4096_d64", "bf16", 8, 16, 16, 4096, 64, 16, "rms", True),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "train", "train", "decode", "rope"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f16", "f32"])
    group = rng.choice([1, 1, 2, 4])
    Hk = rng.randint(1, 8)
    H = Hk * group
    D, M = rng.choice([16, 40, 64, 64, 96, 128]), rng.choice([16, 64, 64, 72, 128])
    if op == "decode":
        B = _log(rng, 1, 512)
        slots = 0 if rng.random() < 0.5 else B + rng.randint(0, B)
        return {k: v for k, v in _delta("", op, dtype, B, H, Hk, 1, D, M, slots=slots).items()
                if k != "name"}
    if op == "rope":
        N = 1 if rng.random() < 0.3 else _log(rng, 2, 8229)
        B = _log(rng, 1, max(1, min(64, 33_000 // N)))
        R = rng.choice([0, 2 * rng.randint(1, D // 2), D])
        return {k: v for k, v in _rope("", dtype, B, H, Hk, N, D, R, rng.choice(["rms", "l2"]),
                                       rng.random() < 0.5).items() if k != "name"}
    # at most the products of the largest listed case of the operator, fewer for fp32 and fp16
    most = (8.5e9 if op == "prefill" else 2.1e9) if dtype == "bf16" else 2.7e8
    rows = max(1, min(524_288, int(most / (D * M))) // H)
    N = _log(rng, 1, min(32768 if op == "prefill" else 8229, rows))
    B = _log(rng, 1, max(1, min(8, rows // N)))
    return {k: v for k, v in _delta("", op, dtype, B, H, Hk, N, D, M,
                                    carry=rng.random() < 0.5).items() if k != "name"}


def _gates(c, gen, dev):
    """Log decays of heads whose memory spans a few tokens to a few thousand,
    with tokens that are padding (no decay, nothing written) and tokens that
    start a new document (the state is cleared)."""
    B, H, N = c["B"], c["H"], c["N"]
    rate = torch.exp(torch.rand((1, H, 1), generator=gen, device=dev) * 6.0 - 7.0)
    step = torch.nn.functional.softplus(torch.randn((B, H, N), generator=gen, device=dev) + 1.0)
    g = -rate * step
    beta = torch.sigmoid(torch.randn((B, H, N), generator=gen, device=dev) * 1.5)
    kind = torch.rand((B, 1, N), generator=gen, device=dev)
    pad = kind < 0.02
    new = (kind > 0.9995) & (torch.arange(N, device=dev) > 0)
    g = torch.where(new, torch.full_like(g, -math.inf), torch.where(pad, torch.zeros_like(g), g))
    return g, torch.where(pad, torch.zeros_like(beta), beta)


def _unit(x):
    return x / x.square().sum(-1, keepdim=True).add(1e-6).sqrt()


def prepare(case, seed):
    c, dt = case, DTYPES[case["dtype"]]
    dev = torch.device("cuda", 0)
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    rnd = lambda *shape: torch.randn(shape, generator=gen, device=dev)  # noqa: E731
    B, H, Hk, N, D = c["B"], c["H"], c["Hk"], c["N"], c["D"]
    st = {"case": c}
    if c["op"] == "rope":
        # one projection's rows: queries, keys and values side by side
        proj = (rnd(B, N, (H + 2 * Hk) * D) * 1.5).to(dt)
        st["xq"] = proj[..., :H * D].view(B, N, H, D).transpose(1, 2)
        st["xk"] = proj[..., H * D:(H + Hk) * D].view(B, N, Hk, D).transpose(1, 2)
        st["wq"] = (1.0 + 0.2 * rnd(D)).to(dt)
        st["wk"] = (1.0 + 0.2 * rnd(D)).to(dt)
        half = c["R"] // 2
        first = torch.randint(0, 4096, (B, 1, 1), generator=gen, device=dev)
        pos = (first + torch.arange(N, device=dev)[None, :, None]).float()
        freq = torch.exp(-math.log(10000.0) * torch.arange(half, device=dev) / max(half, 1))
        st["cos"], st["sin"] = torch.cos(pos * freq), torch.sin(pos * freq)
        if c["train"]:
            st["gq"], st["gk"] = rnd(B, H, N, D).to(dt), rnd(B, Hk, N, D).to(dt)
        return st
    M = c["M"]
    # rows as the norm leaves them, the keys of a head with a common part
    q = _unit(rnd(B, Hk, N, D)).to(dt)
    k = _unit(rnd(B, Hk, N, D) + 0.5 * rnd(1, Hk, 1, D)).to(dt)
    v = rnd(B, H, N, M).to(dt)
    g, beta = _gates(c, gen, dev)
    st["scale"] = D ** -0.5
    if c["op"] == "decode":
        P = c["slots"] or B
        st.update(q=q[:, :, 0].contiguous(), k=k[:, :, 0].contiguous(),
                  v=v[:, :, 0].contiguous(), g=g[:, :, 0].contiguous(),
                  beta=beta[:, :, 0].contiguous(), state=rnd(P, H, D, M) * 0.3, slots=None)
        if c["slots"]:
            slots = torch.randperm(P, generator=gen, device=dev)[:B].to(torch.int32)
            idle = torch.rand((B,), generator=gen, device=dev) < 0.1
            st["slots"] = torch.where(idle, torch.full_like(slots, -1), slots)
        return st
    st.update(q=q, k=k, v=v, g=g, beta=beta, state=rnd(B, H, D, M) * 0.3 if c["carry"] else None)
    if c["op"] == "train":
        st["go"] = rnd(B, H, N, M).to(dt)
        st["gs"] = rnd(B, H, D, M) * 0.1 if c["carry"] else None
    return st


# ------------------------------------------------------------ plain forms
def _chunked(q, k, v, g, beta, s, scale):
    """The gated delta rule in 32 bits, a chunk of rows at a time: the rows of
    a chunk are joined by a triangular solve, the chunks by the state."""
    B, H, N, M = v.shape
    D, C = q.shape[-1], CHUNK
    group = H // q.shape[1]
    n = -(-N // C)
    rows = lambda x: torch.nn.functional.pad(x, (0, 0, 0, n * C - N)).view(B, -1, n, C, x.shape[-1])  # noqa: E731
    q, k = (rows(x).repeat_interleave(group, 1) for x in (q, k))
    v = rows(v)
    # a decay of e^-120 is none at all in 32 bits, and sums of it stay finite
    G = rows(g.clamp_min(-120.0)[..., None])[..., 0].cumsum(-1)
    b = rows(beta[..., None])
    low = torch.ones((C, C), device=q.device, dtype=torch.bool).tril()
    gam = torch.exp(torch.where(low, G[..., :, None] - G[..., None, :], -math.inf))
    A = (b * gam * (k @ k.mT)).tril(-1)
    P = scale * gam * (q @ k.mT)
    eye = torch.eye(C, device=q.device).expand_as(A)
    T = torch.linalg.solve_triangular(eye + A, eye, upper=False, unitriangular=True)
    e = torch.exp(G)[..., None]
    last = torch.exp(G[..., -1:] - G)[..., None]
    TV, W, Q, E = T @ (b * v), T @ (b * e * k), scale * e * q, e[..., -1:, :]
    kl = (k * last).mT
    if s is None:
        s = torch.zeros((B, H, D, M), device=q.device)
    outs = []
    for tv, w, p, qq, kk, ee in zip(*(x.unbind(2) for x in (TV, W, P, Q, kl, E))):
        u = tv - w @ s
        outs.append(qq @ s + p @ u)
        s = ee * s + kk @ u
    return torch.stack(outs, 2).reshape(B, H, n * C, M)[:, :, :N], s


def _rotate(x, cos, sin):
    half = cos.shape[-1]
    a, b, rest = x[..., :half], x[..., half:2 * half], x[..., 2 * half:]
    return torch.cat((a * cos - b * sin, b * cos + a * sin, rest), -1)


def _norm_rotate(x, w, cos, sin, norm):
    x, w = x.float(), w.float()
    ss = x.square().mean(-1, keepdim=True) if norm == "rms" else x.square().sum(-1, keepdim=True)
    return _rotate(x * torch.rsqrt(ss + 1e-6) * w, cos[:, None], sin[:, None])


def _norm_rotate_back(x, w, cos, sin, norm, gy):
    x, w = x.float(), w.float()
    c = 1.0 / x.shape[-1] if norm == "rms" else 1.0
    r = torch.rsqrt(c * x.square().sum(-1, keepdim=True) + 1e-6)
    d = _rotate(gy.float(), cos[:, None], -sin[:, None])
    t = d * w
    return r * (t - c * r * r * x * (x * t).sum(-1, keepdim=True)), (d * x * r).sum((0, 1, 2))


def _run_plain(st):
    c, dt = st["case"], DTYPES[st["case"]["dtype"]]
    f = lambda x: None if x is None else x.float()  # noqa: E731
    if c["op"] == "rope":
        got = {}
        for x, w, gy in (("xq", "wq", "gq"), ("xk", "wk", "gk")):
            got[x[1]] = _norm_rotate(st[x], st[w], st["cos"], st["sin"], c["norm"]).to(dt).contiguous()
            if c["train"]:
                dx, dw = _norm_rotate_back(st[x], st[w], st["cos"], st["sin"], c["norm"], st[gy])
                got["d" + x], got["d" + w] = dx.to(dt).contiguous(), dw.to(dt)
        return got
    if c["op"] == "decode":
        H, Hk, P = c["H"], c["Hk"], st["state"].shape[0]
        state = st["state"]
        at = torch.arange(c["B"], device=state.device) if st["slots"] is None else st["slots"].long()
        on = (at >= 0)[:, None, None]
        s = state[at.clamp_min(0)]
        q, k = (x.float().repeat_interleave(H // Hk, 1) for x in (st["q"], st["k"]))
        s = s * torch.exp(st["g"])[..., None, None]
        u = st["beta"][..., None] * (st["v"].float() - (s * k[..., None]).sum(-2))
        s = s + k[..., None] * u[..., None, :]
        out = st["scale"] * (s * q[..., None]).sum(-2)
        if st["slots"] is None:
            state.copy_(s)
        else:
            # idle rows write to a place of their own past the pool
            pool = torch.cat((state, state[:1]))
            pool[torch.where(at >= 0, at, torch.full_like(at, P))] = s
            state.copy_(pool[:P])
        return {"out": torch.where(on, out, torch.zeros_like(out)).to(dt), "state": state}
    args = [f(st[x]) for x in ("q", "k", "v", "g", "beta", "state")]
    if c["op"] == "prefill":
        out, s = _chunked(*args, st["scale"])
        return {"out": out.to(dt), "state": s}
    with torch.enable_grad():
        args = [x if x is None else x.detach().requires_grad_(True) for x in args]
        out, s = _chunked(*args, st["scale"])
        wrt = [x for x in args if x is not None]
        if c["carry"]:
            d = torch.autograd.grad((out, s), wrt, (st["go"].float(), st["gs"]))
        else:
            d = torch.autograd.grad(out, wrt, st["go"].float())
    got = {"out": out.detach().to(dt), "dq": d[0].to(dt), "dk": d[1].to(dt), "dv": d[2].to(dt),
           "dg": d[3], "dbeta": d[4]}
    if c["carry"]:
        got.update(state=s.detach(), dstate=d[5])
    return got


# ------------------------------------------------ the framework's kernels
def _run_own(st):
    import prefix_sum_outer_gb300 as cp

    c = st["case"]
    if c["op"] == "rope":
        kw = dict(cos=st["cos"], sin=st["sin"], norm=c["norm"], eps=1e-6)
        q, k = cp.causal_product_qk_rope(st["xq"], st["xk"], st["wq"], st["wk"], **kw)
        got = {"q": q, "k": k}
        if c["train"]:
            got["dxq"], got["dxk"], got["dwq"], got["dwk"] = cp.causal_product_qk_rope_bwd(
                st["xq"], st["xk"], st["wq"], st["wk"], st["gq"], st["gk"], **kw)
        return got
    if c["op"] == "decode":
        out = cp.causal_product_decode_delta(st["q"], st["k"], st["v"], st["g"], st["beta"],
                                             st["state"], scale=st["scale"], slots=st["slots"])
        return {"out": out, "state": st["state"]}
    args = [st[x] for x in ("q", "k", "v", "g", "beta")]
    if c["op"] == "prefill":
        out, s = cp.causal_product_fwd_delta(*args, state_in=st["state"], return_state=True,
                                             scale=st["scale"])
        return {"out": out, "state": s}
    if not c["carry"]:
        out, ckpt = cp.causal_product_fwd_delta(*args, scale=st["scale"], save=True)
        d = cp.causal_product_bwd_delta(*args, st["go"], ckpt, scale=st["scale"])
        return dict(zip(("dq", "dk", "dv", "dg", "dbeta"), d), out=out)
    out, s, ckpt = cp.causal_product_fwd_delta(*args, state_in=st["state"], return_state=True,
                                               scale=st["scale"], save=True)
    d = cp.causal_product_bwd_delta(*args, st["go"], ckpt, scale=st["scale"],
                                    grad_state_out=st["gs"], return_state_grad=True)
    return dict(zip(("dq", "dk", "dv", "dg", "dbeta", "dstate"), d), out=out, state=s)


def run(state):
    return _run_own(state) if own else _run_plain(state)


def work(case):
    c, e = case, SIZE[case["dtype"]]
    B, H, Hk, N, D = c["B"], c["H"], c["Hk"], c["N"], c["D"]
    if c["op"] == "rope":
        rows = B * N * (H + Hk) * D
        turns = B * N * c["R"] * 4 + 2 * D * e
        # x in, y out; training: x, dy in, dx out besides, and the weights' gradients
        return {"bytes": rows * e * (5 if c["train"] else 2) + turns + (2 * D * e if c["train"] else 0),
                "flops": rows * (18 if c["train"] else 7)}
    M = c["M"]
    qk, vo, gates, s = 2 * B * Hk * N * D * e, B * H * N * M * e, 8 * B * H * N, 4 * B * H * D * M
    if c["op"] == "decode":
        return {"bytes": 2 * s + qk + 2 * vo + gates + (4 * B if c["slots"] else 0),
                "flops": 6 * B * H * D * M}
    if c["op"] == "prefill":
        return {"bytes": qk + 2 * vo + gates + s * (2 if c["carry"] else 1),
                "flops": 6 * B * H * N * D * M}
    # q, k, v, the gates and the output's gradient in; the output and five gradients out
    return {"bytes": 2 * qk + 4 * vo + 2 * gates + (4 * s if c["carry"] else 0),
            "flops": 18 * B * H * N * D * M}


# --------------------------------------------------------- 64 bits
def _exact_rope(c, st):
    got = {}
    cos, sin = st["cos"].double()[:, None], st["sin"].double()[:, None]
    R, D = c["R"], c["D"]
    # the rotation as a complex product
    turn = torch.complex(cos, sin)
    for x, w, gy in (("xq", "wq", "gq"), ("xk", "wk", "gk")):
        X, W = st[x].double(), st[w].double()
        n = X.norm(dim=-1, keepdim=True)
        size = (n * n / D + 1e-6).sqrt() if c["norm"] == "rms" else (n * n + 1e-6).sqrt()

        def turned(y, by):
            z = torch.complex(y[..., :R // 2], y[..., R // 2:R]) * by
            return torch.cat((z.real, z.imag, y[..., R:]), -1)

        got[x[1]] = turned(X / size * W, turn)
        if c["train"]:
            d = turned(st[gy].double(), turn.conj())
            hat = X / size
            share = D if c["norm"] == "rms" else 1
            t = d * W
            got["d" + x] = (t - hat * ((hat * t).sum(-1, keepdim=True) / share)) / size
            got["d" + w] = (d * hat).sum((0, 1, 2))
    return got


def _exact_delta(c, st):
    """The recurrence, a token at a time, and its reverse."""
    decode = c["op"] == "decode"
    if decode:
        st = dict(st, **{n: st[n][:, :, None] for n in ("q", "k", "v", "g", "beta")})
    B, H, N, D, M = c["B"], c["H"], c["N"], c["D"], c["M"]
    group, scale = H // c["Hk"], st["scale"]
    per = lambda x: x.double().repeat_interleave(H // x.shape[1], 1).transpose(0, 2).transpose(1, 2).contiguous()  # noqa: E731
    q, k, v = per(st["q"]), per(st["k"]), per(st["v"])            # [N, B, H, .]
    a, b = (per(st[n][..., None]) for n in ("g", "beta"))
    a = torch.exp(a)
    first = st["state"]
    if decode:
        at = torch.arange(B, device=q.device) if st["slots"] is None else st["slots"].long()
        s = first.double()[at.clamp_min(0)]
    else:
        s = torch.zeros((B, H, D, M), device=q.device, dtype=torch.float64) if first is None else first.double()

    def step(s, t):
        s = s * a[t][..., None]
        u = b[t] * (v[t] - torch.einsum("bhd,bhdm->bhm", k[t], s))
        return s + k[t][..., None] * u[..., None, :], u

    train = c["op"] == "train"
    every = max(1, math.isqrt(N))
    kept, out = [], torch.empty((N, B, H, M), device=q.device, dtype=torch.float64)
    for t in range(N):
        if train and t % every == 0:
            kept.append(s)
        s, _ = step(s, t)
        out[t] = scale * torch.einsum("bhd,bhdm->bhm", q[t], s)
    back = lambda x: x.permute(1, 2, 0, 3)  # noqa: E731
    if decode:
        pool, on = first.double().clone(), at >= 0
        pool[at[on]] = s[on]
        return {"out": torch.where(on[:, None, None], out[0], torch.zeros_like(out[0])), "state": pool}
    got = {"out": back(out)}
    if not train:
        return dict(got, state=s)
    go = per(st["go"])
    ds = st["gs"].double() if c["carry"] else torch.zeros_like(s)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    da, db = torch.empty_like(a), torch.empty_like(b)
    for n in reversed(range(len(kept))):
        lo, hi = n * every, min(N, (n + 1) * every)
        states = [kept[n]]
        for t in range(lo, hi):
            states.append(step(states[-1], t)[0])
        for t in reversed(range(lo, hi)):
            old, new = states[t - lo] * a[t][..., None], states.pop()
            dq[t] = scale * torch.einsum("bhdm,bhm->bhd", new, go[t])
            ds = ds + scale * q[t][..., None] * go[t][..., None, :]
            miss = v[t] - torch.einsum("bhd,bhdm->bhm", k[t], old)
            du = torch.einsum("bhd,bhdm->bhm", k[t], ds)
            dv[t] = b[t] * du
            db[t] = (du * miss).sum(-1, keepdim=True)
            dk[t] = torch.einsum("bhdm,bhm->bhd", ds, b[t] * miss) - torch.einsum("bhdm,bhm->bhd", old, dv[t])
            ds = ds - k[t][..., None] * dv[t][..., None, :]
            da[t] = (ds * old).sum((-1, -2))[..., None]
            ds = ds * a[t][..., None]
    heads = lambda x: back(x).reshape(B, c["Hk"], group, N, D).sum(2)  # noqa: E731
    got.update(dq=heads(dq), dk=heads(dk), dv=back(dv), dg=back(da)[..., 0], dbeta=back(db)[..., 0])
    if c["carry"]:
        got.update(state=s, dstate=ds)
    return got


def exact(case, seed):
    st = prepare(case, seed)
    with torch.no_grad():
        return _exact_rope(case, st) if case["op"] == "rope" else _exact_delta(case, st)
