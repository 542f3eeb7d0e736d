"""Cases, plain forms and exact values of the gated delta rule and of the state-pool operators.

Operators
  forward   wkv_recurrence_02_b200.ops.delta_forward over many tokens (prefill, training)
  decode    delta_forward over one token (or a few), the states updated in their pool slots
  backward  ops.delta_backward, the gradients of forward
  copy      ops.state_copy: copy, fork and free slots of a state pool
  compact   ops.state_compact: move the live slots of a pool to its front

With `own` false, run() computes each in its plain form: elementary torch operations in 32
bits, rounded once at the end.  With `own` true it makes the framework's calls.

Gated delta rule, per sequence and value head (state S: 64 x 64, row = key channel):
  S' = exp(g_t) S,  u_t = beta_t (v_t - k_t S'),  S = S' + k_t^T u_t,  o_t = scale q_t S
"""
import math

import torch

own = False

N = 64        # head size
C = 64        # tokens per chunk of the plain form
SCALE = N ** -0.5
_T = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------------------ the cases

def listed():
    return [
        # training / prefill of a 1.6B-class model's layer: batch 8, context 4096, 32 heads
        dict(name="forward_b8_t4096_h32", op="forward", type="bf16", lens="8x4096", packed=False, hk=32, h=32,
             state=True, slots=False),
        # one long context of a 7B-class layer, every key head shared by two value heads
        dict(name="forward_b1_t4096_h64", op="forward", type="bf16", lens="1x4096", packed=False, hk=32, h=64,
             state=True, slots=False),
        # a serving step's packed prompts of uneven length (one token, an empty one, odd ones),
        # states taken from and returned to pool slots
        dict(name="forward_packed", op="forward", type="bf16",
             lens="1 517 2048 63 0 129 1000 64 333 1535 65 7 901", packed=True, hk=16, h=16, state=True,
             slots=True),
        # fp32 inputs, the small full-precision workload
        dict(name="forward_fp32_t256_h4", op="forward", type="fp32", lens="1x256", packed=False, hk=4, h=4, state=False,
             slots=False),
        # one decoded token for each of 256 sequences of a 7B-class layer
        dict(name="decode_b256_h64", op="decode", type="bf16", lens="256x1", packed=False, hk=64, h=64, state=True,
             slots=True),
        # one decoded token of a single sequence: launch and latency
        dict(name="decode_b1_h32", op="decode", type="bf16", lens="1x1", packed=False, hk=32, h=32, state=True,
             slots=True),
        # a training step's gradients at the 1.6B-class layer, no carried state
        dict(name="backward_b8_t4096_h32", op="backward", type="bf16", lens="8x4096", packed=False, hk=32, h=32,
             state=False, slots=False),
        # packed documents of odd lengths with shared key heads and carried states
        dict(name="backward_packed", op="backward", type="bf16", lens="700 1 321 64 1023", packed=True, hk=8, h=16,
             state=True, slots=False),
        # eight samples forked from each of eight prompts over 12 layers, two finished ones freed
        dict(name="copy_fork_l12_h32", op="copy", layers=12, slots=96, heads=32, prompts=8, samples=8, freed=2),
        # one sequence's state of one layer: launch and latency
        dict(name="copy_one_h4", op="copy", layers=1, slots=16, heads=4, prompts=1, samples=1, freed=0),
        # a decode batch of 256 states of a 7B-class layer after about half of it has finished
        dict(name="compact_p256_h64", op="compact", layers=1, slots=256, heads=64, live=0.5),
        # a small odd pool over four layers, few sequences finished
        dict(name="compact_p33_h5", op="compact", layers=4, slots=33, heads=5, live=0.8),
    ]


def _lens(case):
    """Tokens of each sequence: "8x4096" is eight of 4096, "3 0 5" three of those lengths."""
    if "x" in case["lens"]:
        n, t = case["lens"].split("x")
        return [int(t)] * int(n)
    return [int(t) for t in case["lens"].split()]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["forward", "forward", "forward", "decode", "decode", "backward", "backward", "copy", "compact"])
    if op in ("forward", "backward"):
        kind = rng.choice(["bf16", "bf16", "bf16", "fp32"])
        most = 1 << 19 if kind == "bf16" else 1 << 14  # tokens x heads
        hk = _log(rng, 1, 32)
        h = hk * rng.choice([1, 1, 1, 2, 3])
        h = min(h, 64 // hk * hk)
        packed = rng.random() < 0.5
        n = _log(rng, 1, 12)
        if packed:
            t = _log(rng, 2, max(2, min(4096, most // (h * n))))
            lens = [max(0, int(t * rng.uniform(0.0, 1.0))) for _ in range(n)]
            lens[rng.randrange(n)] = t
            lens = " ".join(map(str, lens))
        else:
            lens = "%dx%d" % (n, _log(rng, 2, max(2, min(8192, most // (h * n)))))
        state = rng.random() < 0.6
        return dict(op=op, type=kind, lens=lens, packed=packed, hk=hk, h=h, state=state,
                    slots=state and op == "forward" and rng.random() < 0.5)
    if op == "decode":
        hk = _log(rng, 1, 64)
        h = hk * rng.choice([1, 1, 2, 4])
        h = min(h, 64 // hk * hk)
        t = rng.choice([1, 1, 1, 1, 2, 3, 4])
        return dict(op=op, type=rng.choice(["bf16", "bf16", "fp32"]), lens="%dx%d" % (_log(rng, 1, 256), t), packed=False, hk=hk,
                    h=h, state=True, slots=True)
    layers, heads = _log(rng, 1, 12), _log(rng, 1, 32)
    if op == "copy":
        prompts, samples = _log(rng, 1, 8), _log(rng, 1, 8)
        freed = rng.randrange(0, 4)
        return dict(op=op, layers=layers, heads=heads, prompts=prompts, samples=samples, freed=freed,
                    slots=prompts * (samples + 1) + freed + rng.randrange(0, 9))
    return dict(op=op, layers=layers, heads=heads, slots=_log(rng, 2, 96), live=round(rng.uniform(0.1, 0.95), 3))


def work(case):
    op = case["op"]
    if op in ("copy", "compact"):
        slot = case["layers"] * case["heads"] * N * N * 4
        if op == "copy":  # each source read once, each destination written once
            moved = case["prompts"] * (1 + case["samples"]) + case["freed"]
        else:  # the live slots that do not stay in place, read and written
            moved = 2 * case["live"] * case["slots"]
        return {"bytes": int(moved * slot), "flops": 0}
    tok, seqs = sum(_lens(case)), len(_lens(case))
    h, hk, e = case["h"], case["hk"], 2 if case["type"] == "bf16" else 4
    states = seqs * h * N * N * 4
    qkv = tok * e * (2 * hk * N + h * N + 2 * h)  # q, k, v, g, beta
    if op == "backward":  # those and do read, their gradients written; the states' gradients
        return {"bytes": 2 * qkv + tok * e * h * N + (3 * states if case["state"] else 0), "flops": tok * h * 16 * N * N}
    return {"bytes": qkv + tok * e * h * N + states * (2 if case["state"] else 1), "flops": tok * h * 6 * N * N}


# ----------------------------------------------------------------------------- the inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    if case["op"] in ("copy", "compact"):
        p = case["slots"]
        st = {"case": case, "pool": randn(case["layers"], p, case["heads"], N, N)}
        order = torch.randperm(p, generator=gen, device="cuda")
        if case["op"] == "copy":
            np_, ns, nf = case["prompts"], case["samples"], case["freed"]
            src = torch.cat([order[:np_].repeat_interleave(ns), order.new_full((nf,), -1)])
            st["src"], st["dst"] = src.int(), order[np_: np_ + np_ * ns + nf].int()
        else:
            live = torch.zeros(p, dtype=torch.bool, device="cuda")
            live[order[: max(1, round(case["live"] * p))]] = True
            st["live"] = live
        return st
    lens, dt = _lens(case), _T[case["type"]]
    b, t = (1, sum(lens)) if case["packed"] else (len(lens), lens[0])
    h, hk = case["h"], case["hk"]
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    st = {"case": case}
    # queries and keys of unit length, decays exp(-exp(omega)) as the recurrence's, gates a sigmoid
    st["q"] = unit(randn(b, t, hk, N)).to(dt)
    st["k"] = unit(randn(b, t, hk, N)).to(dt)
    st["v"] = randn(b, t, h, N).to(dt)
    omega = torch.rand(h, generator=gen, device="cuda") * 5.5 - 6.0
    st["g"] = (-torch.exp(omega + 0.3 * randn(b, t, h))).to(dt)
    st["beta"] = torch.sigmoid(randn(b, t, h)).to(dt)
    if case["packed"]:
        off = [0]
        for n in lens:
            off.append(off[-1] + n)
        st["offsets"] = torch.tensor(off, dtype=torch.int32, device="cuda")
    if case["state"]:
        extra = 3 if case["slots"] else 0  # slots of other sequences
        st["s0"] = 0.1 * randn(len(lens) + extra, h, N, N)
        if case["slots"]:
            st["slots"] = torch.randperm(len(lens) + extra, generator=gen, device="cuda")[: len(lens)].int()
    if case["op"] == "backward":
        st["do"] = randn(b, t, h, N).to(dt)
        if case["state"]:
            st["dsT"] = 0.1 * randn(len(lens), h, N, N)
    return st


# ------------------------------------------------------------------- layout of the sequences

def _index(case):
    """(sequences, longest) token index of each padded place, and which places hold a token."""
    lens = _lens(case)
    longest = max(max(lens), 1)
    at = torch.arange(longest, device="cuda").expand(len(lens), longest)
    n = torch.tensor(lens, device="cuda")[:, None]
    start = torch.cumsum(n, 0) - n
    return torch.where(at < n, start + at, 0), at < n


def _to_rows(x, idx, valid, heads, dt):
    """[B, T, heads', ...] -> [sequence, head, place, ...], zero where there is no token."""
    y = x.reshape(-1, *x.shape[2:])[idx].to(dt)  # [S, L, heads', ...]
    y = y * valid.reshape(*valid.shape, *([1] * (y.dim() - 2)))
    if y.shape[2] != heads:
        y = y.repeat_interleave(heads // y.shape[2], dim=2)
    return y.transpose(1, 2)


def _from_rows(y, idx, valid, like, dt):
    """The inverse of _to_rows; heads that share one are summed."""
    y = y.transpose(1, 2)[valid]  # [tokens, heads, ...]
    hs = like.shape[2]
    if y.shape[1] != hs:
        y = y.reshape(y.shape[0], hs, y.shape[1] // hs, *y.shape[2:]).sum(2)
    out = torch.zeros(like.shape, device=y.device, dtype=y.dtype).reshape(-1, *like.shape[2:])
    out[idx[valid]] = y
    return out.reshape(like.shape).to(dt)


def _initial(st, dt):
    case = st["case"]
    if not case["state"]:
        return torch.zeros(len(_lens(case)), case["h"], N, N, device="cuda", dtype=dt)
    s = st["s0"][st["slots"].long()] if "slots" in st else st["s0"]
    return s.to(dt)


# --------------------------------------------------------------------------- plain forms

def _chunks(st):
    case = st["case"]
    idx, valid = _index(case)
    pad = -idx.shape[1] % C
    f = torch.float32

    def cut(x):
        y = _to_rows(x, idx, valid, case["h"], f)
        y = torch.nn.functional.pad(y, [0, 0] * (y.dim() - 3) + [0, pad])
        return y.reshape(*y.shape[:2], -1, C, *y.shape[3:])

    x = {n: cut(st[n]) for n in ("q", "k", "v", "g", "beta") + (("do",) if "do" in st else ())}
    q, k, v, g, b = (x[n] for n in ("q", "k", "v", "g", "beta"))
    gc = torch.cumsum(g, -1)
    low = torch.ones(C, C, device="cuda", dtype=torch.bool).tril()
    ratio = torch.exp((gc[..., :, None] - gc[..., None, :]).masked_fill(~low, -math.inf))
    kk = k @ k.transpose(-1, -2)
    strict = ratio * low.tril(-1)
    lmat = b[..., None] * strict * kk
    inv = torch.eye(C, device="cuda").expand(lmat.shape).clone()  # (I + lmat)^-1 by rows
    for i in range(1, C):
        inv[..., i, :i] = -(lmat[..., i, None, :i] @ inv[..., :i, :i])[..., 0, :]
    x.update(idx=idx, valid=valid, inv=inv, strict=strict, kk=kk, eg=torch.exp(gc), tail=torch.exp(gc[..., -1:] - gc),
             qk=q @ k.transpose(-1, -2), ratio=ratio, cut=cut)
    x["p"] = SCALE * ratio * x["qk"]
    return x


def _walk(x, s):
    """States entering the chunks, u of every chunk, and the last state."""
    k, v, b, eg, tail = x["k"], x["v"], x["beta"], x["eg"], x["tail"]
    u0 = x["inv"] @ (b[..., None] * v)
    wk = x["inv"] @ ((b * eg)[..., None] * k)
    states, us = [], []
    for c in range(k.shape[2]):
        states.append(s)
        u = u0[:, :, c] - wk[:, :, c] @ s
        us.append(u)
        s = eg[:, :, c, -1, None, None] * s + (tail[:, :, c, :, None] * k[:, :, c]).transpose(-1, -2) @ u
    return torch.stack(states, 2), torch.stack(us, 2), s, wk


def _plain_forward(st):
    case, dt = st["case"], _T[st["case"]["type"]]
    x = _chunks(st)
    s0, u, s, _ = _walk(x, _initial(st, torch.float32))
    o = SCALE * x["eg"][..., None] * (x["q"] @ s0) + x["p"] @ u
    o = o.reshape(*o.shape[:2], -1, N)[:, :, : x["idx"].shape[1]]
    o = _from_rows(o, x["idx"], x["valid"], st["v"], dt)
    if case["slots"]:
        st["s0"][st["slots"].long()] = s
        s = st["s0"]
    return {"o": o, "sT": s}


def _plain_decode(st):
    """A few tokens: the recurrence itself."""
    case, dt, f = st["case"], _T[st["case"]["type"]], torch.float32
    idx, valid = _index(case)
    q, k, v, g, b = (_to_rows(st[n], idx, valid, case["h"], f) for n in ("q", "k", "v", "g", "beta"))
    s, os = _initial(st, f), []
    for t in range(k.shape[2]):
        s = torch.exp(g[:, :, t])[..., None, None] * s
        kt = k[:, :, t]
        u = b[:, :, t, None] * (v[:, :, t] - (kt[..., None] * s).sum(-2))
        s = s + kt[..., None] * u[..., None, :]
        os.append(SCALE * (q[:, :, t, :, None] * s).sum(-2))
    o = _from_rows(torch.stack(os, 2), idx, valid, st["v"], dt)
    st["s0"][st["slots"].long()] = s
    return {"o": o, "sT": st["s0"]}


def _plain_backward(st):
    case, dt = st["case"], _T[st["case"]["type"]]
    x = _chunks(st)
    s0, u, s1, wk = _walk(x, _initial(st, torch.float32))
    q, k, v, b, do, eg, tail, inv, p = (x[n] for n in ("q", "k", "v", "beta", "do", "eg", "tail", "inv", "p"))
    t_ = lambda m: m.transpose(-1, -2)  # noqa: E731
    ds = st["dsT"] if "dsT" in st else torch.zeros_like(s1)
    du0 = t_(p) @ do
    x0 = SCALE * t_(q) @ (eg[..., None] * do)
    kd = tail[..., None] * k
    dus, dss = [], []
    for c in reversed(range(k.shape[2])):
        dss.append(ds)
        du = du0[:, :, c] + kd[:, :, c] @ ds
        dus.append(du)
        ds = eg[:, :, c, -1, None, None] * ds + x0[:, :, c] - t_(wk[:, :, c]) @ du
    du, d1 = torch.stack(dus[::-1], 2), torch.stack(dss[::-1], 2)
    dw = t_(inv) @ du
    dv = b[..., None] * dw
    w0 = eg[..., None] * (k @ s0)
    a1 = x["ratio"] * SCALE * (do @ t_(u))
    dl = -(dw @ t_(u)) * x["strict"]
    a2 = b[..., None] * dl
    qs, uk, ks = SCALE * eg[..., None] * (do @ t_(s0)), tail[..., None] * (u @ t_(d1)), -(b * eg)[..., None] * (dw @ t_(s0))
    dq = qs + a1 @ k
    dk = uk + ks + t_(a1) @ q + (a2 + t_(a2)) @ k
    db = (dw * (v - w0)).sum(-1) + (dl * x["kk"]).sum(-1)
    e1, e2 = a1 * x["qk"], a2 * x["kk"]
    end = (k * uk).sum(-1)
    dg = (q * qs).sum(-1) + (k * ks).sum(-1) - end + (e1 + e2).sum(-1) - (e1 + e2).sum(-2)
    dg[..., -1] += end.sum(-1) + eg[..., -1] * (d1 * s0).sum((-1, -2))
    dg = torch.flip(torch.cumsum(torch.flip(dg, [-1]), -1), [-1])
    n = x["idx"].shape[1]
    back = lambda y, like: _from_rows(y.reshape(*y.shape[:2], -1, *y.shape[4:])[:, :, :n], x["idx"], x["valid"], like, dt)  # noqa: E731
    out = {"dq": back(dq, st["q"]), "dk": back(dk, st["k"]), "dv": back(dv, st["v"]), "dg": back(dg, st["g"]),
           "dbeta": back(db, st["beta"])}
    if case["state"]:
        out["ds0"] = ds
    return out


def _plain_copy(st):
    pool, src, dst = st["pool"], st["src"].long(), st["dst"].long()
    keep = (src >= 0).to(pool.dtype).reshape(1, -1, 1, 1, 1)
    pool[:, dst] = pool[:, src.clamp(min=0)] * keep
    return {"pool": pool}


def _plain_compact(st):
    pool, live = st["pool"], st["live"]
    at = torch.cumsum(live, 0) - 1
    new = torch.where(live, at, -1).int()
    order = torch.nonzero(live)[:, 0]
    pool[:, : order.numel()] = pool[:, order]
    return {"pool": pool, "new_index": new, "count": live.sum().reshape(1).int()}


# ----------------------------------------------------------------------- the framework's calls

def _own(st):
    from wkv_recurrence_02_b200 import ops

    case = st["case"]
    if case["op"] == "copy":
        ops.state_copy(st["pool"], st["src"], st["dst"], slot_dim=1)
        return {"pool": st["pool"]}
    if case["op"] == "compact":
        new, count = ops.state_compact(st["pool"], st["live"], slot_dim=1)
        return {"pool": st["pool"], "new_index": new, "count": count}
    x = [st[n] for n in ("q", "k", "v", "g", "beta")]
    if case["op"] == "backward":
        return ops.delta_backward(*x, st["do"], s0=st.get("s0"), dsT=st.get("dsT"), offsets=st.get("offsets"),
                                  want_ds0=case["state"])
    o, sT = ops.delta_forward(*x, s0=st.get("s0"), offsets=st.get("offsets"), slots=st.get("slots"),
                              sT=st["s0"] if case["slots"] else None)
    return {"o": o, "sT": sT}


def run(state):
    if own:
        return _own(state)
    return {"forward": _plain_forward, "decode": _plain_decode, "backward": _plain_backward, "copy": _plain_copy,
            "compact": _plain_compact}[state["case"]["op"]](state)


# -------------------------------------------------------------------------------- exact values

def exact(case, seed):
    """The recurrence and its adjoint token by token in 64 bits.  None for the pool operators,
    whose outputs are copies."""
    if case["op"] in ("copy", "compact") or sum(_lens(case)) == 0:
        return None
    st = prepare(case, seed)
    idx, valid = _index(case)
    f = torch.float64
    q, k, v, g, b = (_to_rows(st[n], idx, valid, case["h"], f) for n in ("q", "k", "v", "g", "beta"))
    a, s, steps = torch.exp(g)[..., None, None], _initial(st, f), k.shape[2]

    def step(s, t):
        kt, sp = k[:, :, t], a[:, :, t] * s
        u = b[:, :, t, None] * (v[:, :, t] - (kt[:, :, None] @ sp)[:, :, 0])
        return sp, u, sp + kt[..., None] * u[:, :, None]

    if case["op"] != "backward":
        o = torch.empty_like(v)
        for t in range(steps):
            s = step(s, t)[2]
            o[:, :, t] = SCALE * (q[:, :, t, None] @ s)[:, :, 0]
        if case["slots"]:
            pool = st["s0"].to(f)
            pool[st["slots"].long()] = s
            s = pool
        return {"o": _from_rows(o, idx, valid, st["v"], f), "sT": s}
    do = _to_rows(st["do"], idx, valid, case["h"], f)
    marks = []
    for t in range(steps):  # a state every 64 tokens; the ones between are formed again
        if t % 64 == 0:
            marks.append(s)
        s = step(s, t)[2]
    ds = st["dsT"].to(f) if "dsT" in st else torch.zeros_like(s)
    dq, dk, dv, dg, db = (torch.empty_like(y) for y in (q, k, v, g, b))
    for m in reversed(range(len(marks))):
        run_, s = [], marks[m]
        for t in range(64 * m, min(64 * m + 64, steps)):
            sp, u, s1 = step(s, t)
            run_.append((t, s, sp, u, s1))
            s = s1
        for t, s_prev, sp, u, s1 in reversed(run_):
            dot, kt = do[:, :, t], k[:, :, t]
            ds = ds + SCALE * q[:, :, t, :, None] * dot[:, :, None]
            dq[:, :, t] = SCALE * (s1 @ dot[..., None])[..., 0]
            du = (kt[:, :, None] @ ds)[:, :, 0]
            r = v[:, :, t] - (kt[:, :, None] @ sp)[:, :, 0]
            bu = b[:, :, t, None] * du
            db[:, :, t] = (du * r).sum(-1)
            dv[:, :, t] = bu
            dk[:, :, t] = (ds @ u[..., None])[..., 0] - (sp @ bu[..., None])[..., 0]
            dsp = ds - kt[..., None] * bu[:, :, None]
            dg[:, :, t] = (dsp * sp).sum((-1, -2))
            ds = a[:, :, t] * dsp
    out = {n: _from_rows(y, idx, valid, st[w], f)
           for n, y, w in (("dq", dq, "q"), ("dk", dk, "k"), ("dv", dv, "v"), ("dg", dg, "g"), ("dbeta", db, "beta"))}
    if case["state"]:
        out["ds0"] = ds
    return out
