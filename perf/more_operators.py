"""Cases of linear attention with a decay for each head and of the layer norm.

Each case names an operator, its sizes and its element type:

* ``prefill``: the chunked product over a prompt, the state decaying by a
  constant factor per token, from a carried state and over sequences of
  different lengths where the case says so: outputs and the state after each
  sequence's last token;
* ``train``: forward and backward of the same (gradients of q, k, v and, with
  a carried state, of that state);
* ``decode``: one token per sequence, the state updated in place, in a pool of
  states addressed by slot where the case says so;
* ``norm``: layer norm of rows; ``H`` > 0 means the rows of H heads, head-major
  in and token-major out, with weights of their own for each head, ``H`` = 0
  rows of a model's width; with ``train`` its backward too (gradients of the
  rows, the weight and the bias).
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
CHUNK = 256         # rows of a chunk in the plain form
EPS = 1e-5


def _decay(name, op, dtype, B, H, Hk, N, D, M, carry=False, ragged=False, **more):
    return dict(name=name, op=op, dtype=dtype, B=B, H=H, Hk=Hk, N=N, D=D, M=M, carry=carry,
                ragged=ragged, **more)


def _norm(name, dtype, B, H, N, C, train):
    return dict(name=name, op="norm", dtype=dtype, B=B, H=H, N=N, C=C, train=train)


def listed():
    return [
        # one sequence being answered: a token's step, where latency counts
        _decay("decode_b1_h16_d64", "decode", "bf16", 1, 16, 16, 1, 64, 64, slots=0),
        # a full serving batch at the sizes the decode step is benchmarked at
        _decay("decode_b512_h16_d64", "decode", "bf16", 512, 16, 16, 1, 64, 64, slots=0),
        # a batch out of a larger pool of states, some of its rows idle, shared key heads
        _decay("decode_b61_h8_d128_slots", "decode", "f16", 61, 8, 4, 1, 128, 128, slots=96),
        # the smallest workload, fp32
        _decay("prefill_f32_h2_n64_d16", "prefill", "f32", 1, 2, 2, 64, 16, 16),
        # the main training shape as a batch of prompts
        _decay("prefill_bf16_b8h16_n4096_d64", "prefill", "bf16", 8, 16, 16, 4096, 64, 64),
        # prompts of different lengths that continue a conversation, two value heads to a key head
        _decay("prefill_bf16_b4h8_n8229_d128_m64", "prefill", "bf16", 4, 8, 4, 8229, 128, 64,
               carry=True, ragged=True),
        # few heads over a long document
        _decay("prefill_bf16_b2h8_n32768_d128", "prefill", "bf16", 2, 8, 8, 32768, 128, 128),
        # a training step at the main shape
        _decay("train_bf16_b8h16_n4096_d64", "train", "bf16", 8, 16, 16, 4096, 64, 64),
        # full precision, an odd length, shared key heads, a carried state with its gradient
        _decay("train_f32_b2h4_n509_d64", "train", "f32", 2, 4, 2, 509, 64, 64, carry=True),
        # the norm of a serving batch's new tokens, head by head
        _norm("norm_f16_b61_n1_h16_c64", "f16", 61, 16, 1, 64, False),
        # the norm of a training step's heads
        _norm("norm_train_bf16_b8h16_n4096_c64", "bf16", 8, 16, 4096, 64, True),
        # the norm at a layer's input, 16 heads of 64 wide
        _norm("norm_train_bf16_b8_n4096_c1024", "bf16", 8, 0, 4096, 1024, True),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "train", "train", "decode", "norm", "norm"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f16", "f32"])
    if op == "norm":
        H = rng.choice([0, 0, rng.randint(1, 16)])
        C = rng.choice([16, 40, 64, 64, 96, 128, 200]) if H else _log(rng, 16, 12288)
        rows = 33_554_432 // (C * max(H, 1)) // (2 if dtype == "f32" else 1)
        N = 1 if rng.random() < 0.2 else _log(rng, 2, max(2, min(8229, rows)))
        B = _log(rng, 1, max(1, min(64, rows // N)))
        return {k: v for k, v in _norm("", dtype, B, H, N, C, rng.random() < 0.6).items()
                if k != "name"}
    group = rng.choice([1, 1, 2, 4])
    Hk = rng.randint(1, 8)
    H = Hk * group
    D, M = rng.choice([16, 40, 64, 64, 96, 128]), rng.choice([16, 64, 64, 72, 128])
    if dtype != "bf16" and rng.random() < 0.2:
        D, M = rng.choice([7, 33, 65]), rng.choice([5, 33, 66])
    if op == "decode":
        B = _log(rng, 1, 512)
        slots = 0 if rng.random() < 0.5 else B + rng.randint(0, B)
        return {k: v for k, v in _decay("", op, dtype, B, H, Hk, 1, D, M, slots=slots).items()
                if k != "name"}
    # at most the products of the largest listed case of the operator, fewer for fp32 and fp16
    most = (8.5e9 if op == "prefill" else 2.1e9) if dtype == "bf16" else 5.4e8
    rows = max(1, min(524_288, int(most / (D * M))) // H)
    N = _log(rng, 1, min(32768 if op == "prefill" else 8229, rows))
    B = _log(rng, 1, max(1, min(8, rows // N)))
    return {k: v for k, v in _decay("", op, dtype, B, H, Hk, N, D, M, carry=rng.random() < 0.5,
                                    ragged=B > 1 and rng.random() < 0.4).items() if k != "name"}


def _unit(x):
    return x / x.square().sum(-1, keepdim=True).add(1e-6).sqrt()


def prepare(case, seed):
    c, dt = case, DTYPES[case["dtype"]]
    dev = torch.device("cuda", 0)
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    rnd = lambda *shape: torch.randn(shape, generator=gen, device=dev)  # noqa: E731
    B, H, N = c["B"], c["H"], c["N"]
    st = {"case": c}
    if c["op"] == "norm":
        C = c["C"]
        lead = (B, H, N) if H else (B, N)
        wide = (H, C) if H else (C,)
        # rows with a mean of their own, as a residual stream's or a state's read-out
        st["x"] = (rnd(*lead, C) * 1.5 + rnd(*lead, 1)).to(dt)
        st["w"], st["b"] = (1.0 + 0.2 * rnd(*wide)).to(dt), (0.2 * rnd(*wide)).to(dt)
        if c["train"]:
            st["gy"] = rnd(*((B, N, H, C) if H else (B, N, C))).to(dt)
        return st
    Hk, D, M = c["Hk"], c["D"], c["M"]
    # heads whose memory spans a few tokens to a few thousand
    st["g"] = -torch.exp(torch.rand((H,), generator=gen, device=dev) * 8.0 - 8.5)
    st["scale"] = D ** -0.5
    st["lengths"] = None
    q = rnd(B, Hk, N, D).to(dt)
    k = _unit(rnd(B, Hk, N, D) + 0.5 * rnd(1, Hk, 1, D)).to(dt)
    v = rnd(B, H, N, M).to(dt)
    if c["op"] == "decode":
        P = c["slots"] or B
        st.update(q=q[:, :, 0].contiguous(), k=k[:, :, 0].contiguous(), v=v[:, :, 0].contiguous(),
                  state=rnd(P, H, D, M) * 0.3, slots=None)
        if c["slots"]:
            slots = torch.randperm(P, generator=gen, device=dev)[:B].to(torch.int32)
            idle = torch.rand((B,), generator=gen, device=dev) < 0.1
            st["slots"] = torch.where(idle, torch.full_like(slots, -1), slots)
        return st
    st.update(q=q, k=k, v=v, state=rnd(B, H, D, M) * 0.3 if c["carry"] else None)
    if c["ragged"]:
        # a batch padded to its longest sequence
        n = torch.randint(N // 2, N + 1, (B,), generator=gen, device=dev)
        n[0] = N
        st["lengths"] = n.to(torch.int32)
    if c["op"] == "train":
        st["go"] = rnd(B, H, N, M).to(dt)
        st["gs"] = rnd(B, H, D, M) * 0.1 if c["carry"] else None
    return st


# ------------------------------------------------------------ plain forms
def _chunked(q, k, v, g, s, lengths, scale):
    """The product in 32 bits: the rows of a chunk by their decayed scores, the
    chunks by sums of k v^T that decay from chunk to chunk (factors in 64)."""
    B, H, N, M = v.shape
    D, C = q.shape[-1], min(CHUNK, N)
    dev, n = q.device, -(-N // C)
    at = torch.arange(N, device=dev)
    ends = torch.full((B,), N, device=dev) if lengths is None else lengths.long()
    live = (at < ends[:, None])[:, None, :, None]
    q, k = (x.repeat_interleave(H // q.shape[1], 1) for x in (q, k))
    zero = torch.zeros((), device=dev)
    k, v = torch.where(live, k, zero), torch.where(live, v, zero)
    rows = lambda x: torch.nn.functional.pad(x, (0, 0, 0, n * C - N)).view(B, H, n, C, x.shape[-1])  # noqa: E731
    q, k, v = rows(q), rows(k), rows(v)
    powers = lambda e: torch.where(e >= 0, torch.exp(g.double().view(-1, *[1] * e.dim()) * e), 0.0)  # noqa: E731
    r = torch.arange(C, device=dev)
    P = (q @ k.mT) * powers(r[:, None] - r).float()[:, None]
    # what a chunk adds, and the state before each: with every earlier chunk's decay
    added = (k * powers(C - 1 - r).float()[:, None, :, None]).mT @ v
    c = torch.arange(n, device=dev)
    before = powers(C * (c[:, None] - 1 - c)).float() @ added.flatten(3)
    if s is not None:
        before = before + powers(C * c).float()[:, :, None] * s.flatten(2)[:, :, None]
    before = before.view(B, H, n, D, M)
    out = P @ v + powers(r + 1).float()[:, None, :, None] * (q @ before)
    out = scale * torch.where(live, out.view(B, H, n * C, M)[:, :, :N], zero)
    # the state after each sequence's own last row
    left = torch.nn.functional.pad(ends[:, None] - 1 - at, (0, n * C - N), value=-1)
    weight = powers(left).float().transpose(0, 1).reshape(B, H, n, C, 1)
    end = ((k * weight).mT @ v).sum(2)
    if s is not None:
        end = end + powers(ends).float().transpose(0, 1)[..., None, None] * s
    return out, end


def _plain_norm(st):
    c, dt = st["case"], DTYPES[st["case"]["dtype"]]
    x, w, b = st["x"].float(), st["w"].float(), st["b"].float()
    turn = (lambda t: t.transpose(1, 2)) if c["H"] else (lambda t: t)
    wide = lambda t: t[:, None] if c["H"] else t  # noqa: E731
    d = x - x.mean(-1, keepdim=True)
    rstd = torch.rsqrt(d.square().mean(-1, keepdim=True) + EPS)
    xh = d * rstd
    got = {"y": turn(xh * wide(w) + wide(b)).to(dt).contiguous()}
    if c["train"]:
        gy = turn(st["gy"].float())
        t = gy * wide(w)
        dx = rstd * (t - t.mean(-1, keepdim=True) - xh * (t * xh).mean(-1, keepdim=True))
        over = (0, 2) if c["H"] else (0, 1)
        got.update(dx=dx.to(dt).contiguous(), dw=(gy * xh).sum(over).to(dt), db=gy.sum(over).to(dt))
    return got


def _run_plain(st):
    c, dt = st["case"], DTYPES[st["case"]["dtype"]]
    f = lambda x: None if x is None else x.float()  # noqa: E731
    if c["op"] == "norm":
        return _plain_norm(st)
    if c["op"] == "decode":
        H, Hk, P = c["H"], c["Hk"], st["state"].shape[0]
        state = st["state"]
        at = torch.arange(c["B"], device=state.device) if st["slots"] is None else st["slots"].long()
        on = (at >= 0)[:, None, None]
        q, k = (x.float().repeat_interleave(H // Hk, 1) for x in (st["q"], st["k"]))
        s = (state[at.clamp_min(0)] * torch.exp(st["g"])[:, None, None]
             + k[..., None] * st["v"].float()[..., None, :])
        out = st["scale"] * (s * q[..., None]).sum(-2)
        if st["slots"] is None:
            state.copy_(s)
        else:
            # idle rows write to a place of their own past the pool
            pool = torch.cat((state, state[:1]))
            pool[torch.where(at >= 0, at, torch.full_like(at, P))] = s
            state.copy_(pool[:P])
        return {"out": torch.where(on, out, torch.zeros_like(out)).to(dt), "state": state}
    args = [f(st[x]) for x in ("q", "k", "v")]
    s, more = st["state"], (st["lengths"], st["scale"])
    if c["op"] == "prefill":
        out, s = _chunked(*args, st["g"], s, *more)
        return {"out": out.to(dt), "state": s}
    with torch.enable_grad():
        args = [x.detach().requires_grad_(True) for x in args]
        s = s if s is None else s.detach().requires_grad_(True)
        out, end = _chunked(*args, st["g"], s, *more)
        if c["carry"]:
            d = torch.autograd.grad((out, end), (*args, s), (st["go"].float(), st["gs"]))
        else:
            d = torch.autograd.grad(out, args, st["go"].float())
    got = {"out": out.detach().to(dt), "dq": d[0].to(dt), "dk": d[1].to(dt), "dv": d[2].to(dt)}
    if c["carry"]:
        got.update(state=end.detach(), dstate=d[3])
    return got


# ------------------------------------------------ the framework's kernels
def _run_own(st):
    import prefix_sum_outer_gb300 as cp

    c = st["case"]
    if c["op"] == "norm":
        kw = dict(eps=EPS, token_major=c["H"] > 0)
        got = {"y": cp.causal_product_layer_norm(st["x"], st["w"], st["b"], **kw)}
        if c["train"]:
            got["dx"], got["dw"], got["db"] = cp.causal_product_layer_norm_bwd(
                st["x"], st["w"], st["b"], st["gy"], **kw)
        return got
    args = [st[x] for x in ("q", "k", "v", "g")]
    if c["op"] == "decode":
        out = cp.causal_product_decode_decay(*args, st["state"], scale=st["scale"],
                                             slots=st["slots"])
        return {"out": out, "state": st["state"]}
    kw = dict(state_in=st["state"], scale=st["scale"], lengths=st["lengths"])
    if c["op"] == "prefill":
        out, s = cp.causal_product_fwd_decay(*args, return_state=True, **kw)
        return {"out": out, "state": s}
    if not c["carry"]:
        out = cp.causal_product_fwd_decay(*args, **kw)
        d = cp.causal_product_bwd_decay(*args, st["go"], **kw)
        return dict(zip(("dq", "dk", "dv"), d), out=out)
    out, s = cp.causal_product_fwd_decay(*args, return_state=True, **kw)
    d = cp.causal_product_bwd_decay(*args, st["go"], grad_state_out=st["gs"],
                                    return_state_grad=True, **kw)
    return dict(zip(("dq", "dk", "dv", "dstate"), d), out=out, state=s)


def run(state):
    return _run_own(state) if own else _run_plain(state)


def work(case):
    c, e = case, SIZE[case["dtype"]]
    B, H, N = c["B"], c["H"], c["N"]
    if c["op"] == "norm":
        n, w = B * max(H, 1) * N * c["C"], max(H, 1) * c["C"]
        if c["train"]:
            return {"bytes": e * (4 * n + 4 * w), "flops": 20 * n}
        return {"bytes": e * (2 * n + 2 * w), "flops": 8 * n}
    Hk, D, M = c["Hk"], c["D"], c["M"]
    qk, vo, state = 2 * B * Hk * N * D * e, 2 * B * H * N * M * e, 4 * B * H * D * M
    if c["op"] == "decode":
        return {"bytes": qk + vo + 2 * state, "flops": 5 * B * H * D * M}
    if c["op"] == "prefill":
        return {"bytes": qk + vo + state * (2 if c["carry"] else 1), "flops": 4 * B * H * N * D * M}
    # q, k, v, grad_out in once; out, dq, dk, dv out once
    return {"bytes": 2 * (qk + vo) + (4 * state if c["carry"] else 0),
            "flops": 14 * B * H * N * D * M}


# ------------------------------------------------------------- in 64 bits
def _walk64(a, b, c, lam, s, n):
    """sum_{j<=i} lam^(i-j) (a_i . b_j) c_j + lam^(i+1) s^T a_i and the state
    after the last row, block by block from the recurrence's own sums."""
    T = 64
    outs = []
    for i in range(0, n, T):
        x, y, z = a[:, :, i:i + T], b[:, :, i:i + T], c[:, :, i:i + T]
        t = torch.arange(x.shape[2], device=x.device, dtype=torch.float64)
        gap = t[:, None] - t
        mask = torch.where(gap >= 0, lam[:, None, None] ** gap.clamp_min(0), 0.0)
        up = (lam[:, None] ** (t + 1))[..., None]
        down = (lam[:, None] ** (x.shape[2] - 1 - t))[..., None]
        outs.append((mask * (x @ y.mT)) @ z + up * (x @ s))
        s = lam[:, None, None] ** x.shape[2] * s + (down * y).mT @ z
    return torch.cat(outs, 2) if outs else c[:, :, :0], s


def _sequence64(q, k, v, lam, s, scale, n, go, gs):
    """One sequence's results, its rows past n zero."""
    N, group = q.shape[2], v.shape[1] // q.shape[1]
    many = lambda x: x[:, :, :n].repeat_interleave(group, 1)  # noqa: E731
    back = lambda x: x.flip(2)  # noqa: E731
    full = lambda x: torch.nn.functional.pad(x, (0, 0, 0, N - n))  # noqa: E731
    few = lambda x: full(x.unflatten(1, (-1, group)).sum(2))  # noqa: E731
    q, k, v = many(q), many(k), v[:, :, :n]
    out, end = _walk64(q, k, v, lam, s, n)
    got = {"out": full(scale * out), "state": end}
    if go is not None:
        go = scale * go[:, :, :n]
        # the gradient of the state after the last row, as the one after row n is
        # lam times nearer: the walk from the end multiplies by lam once too often
        one = 1.0 / lam[:, None, None]
        dq, _ = _walk64(go, v, k, lam, s.mT, n)
        dv, ds = _walk64(back(k), back(q), back(go), lam, gs * one, n)
        dk, _ = _walk64(back(v), back(go), back(q), lam, (gs * one).mT, n)
        got.update(dq=few(dq), dk=few(back(dk)), dv=full(back(dv)),
                   dstate=ds * lam[:, None, None])
    return got


def exact(case, seed):
    c, st = case, prepare(case, seed)
    d = lambda x: None if x is None else x.double()  # noqa: E731
    if c["op"] == "norm":
        x, w, b = d(st["x"]), d(st["w"]), d(st["b"])
        if c["H"]:
            x = x.transpose(1, 2)
        mu = x.mean(-1, keepdim=True)
        sd = torch.sqrt(((x - mu) ** 2).sum(-1, keepdim=True) / c["C"] + EPS)
        xh = (x - mu) / sd
        got = {"y": xh * w + b}
        if c["train"]:
            gy = d(st["gy"])
            t = gy * w
            dx = (c["C"] * t - t.sum(-1, keepdim=True) - xh * (t * xh).sum(-1, keepdim=True)) / (c["C"] * sd)
            got.update(dx=(dx.transpose(1, 2) if c["H"] else dx).contiguous(),
                       dw=(gy * xh).sum((0, 1)), db=gy.sum((0, 1)))
        return got
    B, H, Hk = c["B"], c["H"], c["Hk"]
    lam = torch.exp(d(st["g"]))
    if c["op"] == "decode":
        at = range(B) if st["slots"] is None else st["slots"].tolist()
        idx = torch.tensor([max(a, 0) for a in at], device=lam.device)
        on = torch.tensor([a >= 0 for a in at], device=lam.device)
        q, k = (d(st[x]).repeat_interleave(H // Hk, 1) for x in ("q", "k"))
        s = lam[:, None, None] * d(st["state"])[idx] + torch.einsum("bhd,bhm->bhdm", k, d(st["v"]))
        out = st["scale"] * torch.einsum("bhdm,bhd->bhm", s, q)
        state = d(st["state"])
        state[idx[on]] = s[on]
        return {"out": torch.where(on[:, None, None], out, 0.0), "state": state}
    if 80.0 * c["N"] * B * H * c["D"] * c["M"] > 2e13:
        return None
    ends = [c["N"]] * B if st["lengths"] is None else st["lengths"].tolist()
    parts = []
    # sequences of one length go together
    groups = [slice(0, B)] if len(set(ends)) == 1 else [slice(i, i + 1) for i in range(B)]
    for at in groups:
        s = torch.zeros((at.stop - at.start, H, c["D"], c["M"]), device=lam.device,
                        dtype=torch.float64) if st["state"] is None else d(st["state"][at])
        go = d(st["go"][at]) if c["op"] == "train" else None
        gs = (d(st["gs"][at]) if c["carry"] else torch.zeros_like(s)) if go is not None else None
        parts.append(_sequence64(*(d(st[x][at]) for x in ("q", "k", "v")), lam, s, st["scale"],
                                 ends[at.start], go, gs))
    got = {x: torch.cat([p[x] for p in parts]) for x in parts[0]}
    if c["op"] == "train" and not c["carry"]:
        got.pop("state"), got.pop("dstate")
    return got
