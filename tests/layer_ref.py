"""Plain 64-bit references of the operators around the recurrence, written from
their definitions (token by token, differentiable), and the rounding units that
the tests' bounds count."""
import torch

# half a step of a rounding, relative to the value
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
U = 2.0 ** -24  # one fp32 rounding
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def spans(batch, seq_len, lens):
    """[(batch row, first token, end)] of the sequences: equal rows, or packed."""
    if lens is None:
        return [(b, 0, seq_len) for b in range(batch)]
    out, t = [], 0
    for n in lens:
        out.append((0, t, t + n))
        t += n
    return out


def offsets(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32)


def conv_ref(x, weight, bias, state, act, seqs):
    """x [B, T, C], state [N, W-1, C]: (out, final state)."""
    W = weight.shape[1]
    out, fin = [], []
    for n, (b, t0, t1) in enumerate(seqs):
        rows = torch.cat([state[n], x[b, t0:t1]])
        z = sum(rows[j: j + t1 - t0] * weight[:, j] for j in range(W))
        if bias is not None:
            z = z + bias
        out.append(z * torch.sigmoid(z) if act == "silu" else z)
        fin.append(rows[len(rows) - (W - 1):])
    return torch.cat(out).reshape(x.shape), torch.stack(fin)


def qk_ref(x, w, table, pos, kind, eps, inter):
    """x [..., H, d]."""
    d = x.shape[-1]
    ss = (x * x).sum(-1, keepdim=True)
    y = x / torch.sqrt((ss if kind == "l2" else ss / d) + eps)
    if w is not None:
        y = y * w
    if table is None:
        return y
    half = table.shape[1] // 2
    i = torch.arange(half)
    a, b = (2 * i, 2 * i + 1) if inter else (i, i + half)
    row = table[pos.long()].unsqueeze(-2)
    cos, sin = row[..., :half], row[..., half:]
    out = y.clone()
    out[..., a] = y[..., a] * cos - y[..., b] * sin
    out[..., b] = y[..., b] * cos + y[..., a] * sin
    return out


def ssm_ref(x, dt, A, B, C, D, state, seqs, raw=False):
    """x [B, T, H, P], dt [B, T, H], B, C [B, T, G, N], state [n, H, P, N]:
    (y, final state), token by token.  raw: x already holds dt x."""
    per = x.shape[2] // B.shape[2]
    Bh, Ch = (v.repeat_interleave(per, 2) for v in (B, C))
    out, fin = [], []
    for n, (b, t0, t1) in enumerate(seqs):
        S = state[n]
        for t in range(t0, t1):
            u = x[b, t] if raw else dt[b, t, :, None] * x[b, t]
            S = torch.exp(dt[b, t] * A)[:, None, None] * S + u[..., None] * Bh[b, t][:, None]
            y = (S * Ch[b, t][:, None]).sum(-1)
            out.append(y if D is None else y + D[:, None] * x[b, t])
        fin.append(S)
    y = torch.stack(out).reshape(x.shape) if out else torch.zeros_like(x)
    return y, torch.stack(fin)


def within(got, ref, bound, what):
    """Every element of got within bound of ref (all in 64 bits)."""
    got, ref = got.detach().double().cpu(), ref.detach()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    if not got.numel():
        return
    assert torch.isfinite(got).all(), f"{what}: values that are not finite"
    off = (got - ref).abs()
    worst = (off / bound.clamp_min(1e-300)).max()
    assert (off <= bound).all(), f"{what}: {float(worst):.2f} times the bound"


def rel(got, ref):
    """2-norm of the difference over the reference's."""
    got, ref = got.detach().double().cpu(), ref.detach()
    n = ref.norm()
    return float((got - ref).norm() / n) if n > 0 else float((got - ref).norm())
