"""Gated delta rule and state-pool operators in plain 64-bit torch on the CPU (test reference).

The recurrence is written token by token from its definition; gradients come from autograd
through it.  Errors are 2-norms of the difference over the 2-norm of the reference.
"""
import torch


def forward(q, k, v, g, beta, scale, s0=None, spans=None):
    """q, k [B,T,Hk,N], v [B,T,H,N], g, beta [B,T,H] in any type -> o, sT in float64.
    spans: [(first, length)] of packed sequences (B = 1)."""
    f = torch.float64
    q, k, v, g, beta = (x.to(f) for x in (q, k, v, g, beta))
    B, T, H, N = v.shape
    G = H // q.shape[2]
    q, k = q.repeat_interleave(G, 2), k.repeat_interleave(G, 2)
    packed = spans is not None
    if not packed:
        spans = [(0, T)] * B
    o = torch.zeros(B, T, H, N, dtype=f)
    outs, states = [], []
    for i, (first, n) in enumerate(spans):
        s = torch.zeros(H, N, N, dtype=f) if s0 is None else s0[i].to(f)
        for t in range(first, first + n):
            r = 0 if packed else i
            sp = torch.exp(g[r, t])[:, None, None] * s
            u = beta[r, t][:, None] * (v[r, t] - torch.einsum("hi,hij->hj", k[r, t], sp))
            s = sp + k[r, t][:, :, None] * u[:, None, :]
            outs.append((r, t, scale * torch.einsum("hi,hij->hj", q[r, t], s)))
        states.append(s)
    if outs:
        idx = torch.tensor([(r, t) for r, t, _ in outs])
        o = o.index_put((idx[:, 0], idx[:, 1]), torch.stack([x for _, _, x in outs]))
    return o, torch.stack(states) if states else torch.zeros(0, H, N, N, dtype=f)


def backward(q, k, v, g, beta, do, scale, s0=None, dsT=None, spans=None):
    """Gradients of sum(o * do) + sum(sT * dsT), float64."""
    f = torch.float64
    x = [t.detach().to(f).clone().requires_grad_() for t in (q, k, v, g, beta)]
    n = len(spans) if spans is not None else q.shape[0]
    s = (torch.zeros(n, v.shape[2], 64, 64) if s0 is None else s0).detach().to(f).clone().requires_grad_()
    o, sT = forward(*x, scale, s, spans)
    loss = (o * do.to(f)).sum()
    if dsT is not None:
        loss = loss + (sT * dsT.to(f)).sum()
    grads = torch.autograd.grad(loss, x + [s], allow_unused=True)
    return {name: torch.zeros_like(t) if d is None else d
            for name, t, d in zip(("dq", "dk", "dv", "dg", "dbeta", "ds0"), x + [s], grads)}


def inputs(B, T, Hk, H, dtype, seed, nseq=None, state=True, N=64):
    """Seeded inputs on the CPU: unit queries and keys, decays exp(-exp(omega)), sigmoid gates."""
    gen = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    x = {"q": unit(rn(B, T, Hk, N)), "k": unit(rn(B, T, Hk, N)), "v": rn(B, T, H, N),
         "g": -torch.exp(torch.rand(H, generator=gen) * 5.5 - 6 + 0.3 * rn(B, T, H)),
         "beta": torch.sigmoid(rn(B, T, H)), "do": rn(B, T, H, N)}
    x = {n: t.to(dtype) for n, t in x.items()}
    n = B if nseq is None else nseq
    x["s0"] = 0.1 * rn(n, H, N, N) if state else None
    x["dsT"] = 0.1 * rn(n, H, N, N) if state else None
    return x


def rel(got, ref):
    got, ref = got.detach().to("cpu", torch.float64), ref.detach().to(torch.float64)
    assert got.shape == ref.shape, (got.shape, ref.shape)
    assert torch.isfinite(got).all(), "non-finite values in the result"
    den = float(ref.norm())
    off = float((got - ref).norm())
    return off / den if den else off


def spans_of(lens, first=0):
    out = []
    for n in lens:
        out.append((first, n))
        first += n
    return out


def copied(pool, src, dst, slot_dim=0):
    """state_copy: all sources as they were, pairs in order, out-of-range pairs left out."""
    old = pool.clone().movedim(slot_dim, 0)
    new = pool.clone()
    view = new.movedim(slot_dim, 0)
    P = old.shape[0]
    for s, d in zip(src, dst):
        if d < 0 or d >= P or s >= P:
            continue
        view[d] = 0 if s < 0 else old[s]
    return new


def compacted(pool, live, slot_dim=0):
    new = pool.clone()
    view, old = new.movedim(slot_dim, 0), pool.movedim(slot_dim, 0)
    index, n = [], 0
    for i, x in enumerate(live):
        index.append(n if x else -1)
        if x:
            view[n] = old[i]
            n += 1
    return new, index, n
