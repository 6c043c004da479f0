"""Plain f64 forms of the block operators, for the GPU tests, and the bounds
that their outputs are held to.

Bounds (u = 2^-8, half a bf16 step relative to the value)
* means: the f64 sum is exact for the inputs used, so the f32 result is the
  correctly rounded quotient up to one f64 rounding: compared bit for bit;
* attention: with A = sum_k p_k |v_k| over a row's keys (p normalised),
    |o - ref| <= u A + u |ref| + 2 ds A + 2^-18 A,
  P rounded to bf16 (u A), the output rounded (u |ref|), scores off by at most
  ds = (D + 2) 2^-23 sum_d |q_d k_d| / sqrt(D) (f32 accumulation, each step
  off by at most one unit of the last place, since the tensor cores need not
  round), and 2^-18 A for ex2 (2^-22 relative), the f32 sums and quotients;
* lse: |lse - ref| <= ds + 2^-20 (1 + |lse|).
"""
import torch

BLOCK, GROUP = 128, 256


def blocks_of(n):
    return -(-n // BLOCK)


def means64(x, size):
    """f64 [heads][ceil(n / size)][dim]."""
    return torch.stack([p.double().sum(1) / p.shape[1] for p in torch.split(x, size, dim=1)], 1)


def select64(q, means, keep, forced=()):
    """int32 [heads][groups][keep], one row at a time by a stable sort on the host."""
    qm = means64(q, GROUP).float().double()
    s = (qm[:, :, None, :] * means.double()[:, None]).sum(-1).cpu()
    s[:, :, list(forced)] = float("inf")
    h, g, n = s.shape
    out = torch.full((h, g, keep), -1, dtype=torch.int32)
    for i in range(h):
        for j in range(g):
            row = s[i, j].tolist()
            best = sorted(range(n), key=lambda b: (-row[b], b))[:keep]
            out[i, j, :len(best)] = torch.tensor(sorted(best), dtype=torch.int32)
    return out


def rows_of(lists, seg_len, n_blocks):
    """Key rows of one list (python ints), block by block; entries outside 0..n_blocks-1 are empty."""
    bps = blocks_of(seg_len)
    rows = []
    for b in lists:
        if 0 <= b < n_blocks:
            s, o = b // bps * seg_len, b % bps * BLOCK
            rows += range(s + o, s + min(seg_len, o + BLOCK))
    return rows


def attend64(q, k, v, rows):
    """q [heads][n][D]; k, v [heads][.][D]; rows(head, group): key rows.
    f64 out [n][heads][D], lse [n][heads] and the bounds on their errors."""
    h, n, d = q.shape
    new = lambda *s: torch.zeros(*s, dtype=torch.float64, device=q.device)  # noqa: E731
    out, lse, bo, bl = new(n, h, d), new(n, h), new(n, h, d), new(n, h)
    lse.fill_(-float("inf"))
    u = 2.0 ** -8
    for i in range(h):
        for g in range(-(-n // GROUP)):
            at = torch.tensor(rows(i, g), dtype=torch.long, device=q.device)
            a, e = g * GROUP, min(n, (g + 1) * GROUP)
            if at.numel() == 0:
                continue
            qg, kk, vv = q[i, a:e].double(), k[i][at].double(), v[i][at].double()
            s = qg @ kk.T / d ** 0.5
            ds = ((d + 2) * 2.0 ** -23 * (qg.abs() @ kk.abs().T) / d ** 0.5).amax(1, keepdim=True)
            p = torch.softmax(s, 1)
            o, mag = p @ vv, p @ vv.abs()
            out[a:e, i], lse[a:e, i] = o, torch.logsumexp(s, 1)
            bo[a:e, i] = (u + 2 * ds + 2.0 ** -18) * mag + u * o.abs()
            bl[a:e, i] = ds[:, 0] + 2.0 ** -20 * (1 + lse[a:e, i].abs())
    return out, lse, bo, bl


def check_attention(out, lse, ref, what=""):
    o, e, bo, bl = ref
    got = out.double()
    assert torch.isfinite(got).all(), f"{what}: non-finite output"
    over = ((got - o).abs() - bo).max().item()
    assert over <= 0, f"{what}: output off its bound by {over:.3g}"
    if lse is not None:
        empty = torch.isinf(e)
        assert torch.equal(lse[empty].double(), e[empty]), f"{what}: lse of empty rows"
        over = ((lse.double() - e)[~empty].abs() - bl[~empty]).max().item() if (~empty).any() else 0
        assert over <= 0, f"{what}: lse off its bound by {over:.3g}"
