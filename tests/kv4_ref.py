"""The 4-bit store, its attention and rotary positions with several axes in 64
bits, by their definitions (CPU tensors), and the error bounds of the tests."""
import math

import torch

GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
GRID = torch.cat((GRID, -GRID))
D, ROWS, PAGE = 128, 16, 1152
BF16, F32 = 2.0 ** -8, 2.0 ** -24   # half a step, relative


# ------------------------------------------------------------- the store
def quantise(x, ts):
    """Codes [.., 128] and scale bytes [.., 8] of fp32 rows: the stated rounding
    (the quotients in fp32, each to the nearest number, ties to even)."""
    b = x.float().unflatten(-1, (8, 16))
    amax = b.abs().amax(-1)
    bad = ~torch.isfinite(b).all(-1)
    scale = (amax / torch.tensor(6.0 * ts, dtype=torch.float32)).clamp(max=448)
    scale = torch.where(bad, 0.0, scale).to(torch.float8_e4m3fn)
    S = scale.float() * torch.tensor(ts, dtype=torch.float32)
    live = (S > 0) & ~bad
    q = torch.where(live[..., None], b / torch.where(live, S, 1.0)[..., None], 0.0)
    code = nearest_code(q.double())
    code = torch.where(live[..., None], code, 0).flatten(-2).to(torch.uint8)
    byte = scale.view(torch.uint8).clone()
    byte[~live] = 0
    byte[bad] = 0x7F
    return code, byte


def nearest_code(q):
    """E2M1 code nearest q (64 bits), ties to the even code, at most 6 in magnitude."""
    d = (q.abs().clamp(max=6)[..., None] - GRID[:8]).abs()  # clamped: a huge q is as far from all
    best = d.amin(-1, keepdim=True)
    tied = d == best
    even = tied & (torch.arange(8) % 2 == 0)
    pick = torch.where(even.any(-1), even.int().argmax(-1), tied.int().argmax(-1))
    return pick + 8 * torch.signbit(q).int()


def pack(code, byte):
    """Pages [B, H, ceil(n / 16), 1152] of codes [B, H, n, 128] and scale bytes."""
    B, H, n, _ = code.shape
    g = -(-n // 16)
    c = torch.zeros(B, H, g * 16, D, dtype=torch.uint8)
    s = torch.zeros(B, H, g * 16, 8, dtype=torch.uint8)
    c[:, :, :n], s[:, :, :n] = code, byte
    b = (c[..., 0::2] | (c[..., 1::2] << 4)).view(B, H, g, 16, 4, 16).transpose(3, 4)
    return torch.cat((b.reshape(B, H, g, 1024), s.view(B, H, g, 128)), -1).contiguous()


def values(pages, ts):
    """Rows [.., 16 * pages, 128] of pages in 64 bits."""
    lead = pages.shape[:-2]
    b = pages[..., :1024].reshape(*lead, -1, 4, 16, 16).transpose(-3, -2).reshape(*lead, -1, 64)
    code = torch.stack((b & 15, b >> 4), -1).flatten(-2)
    s = pages[..., 1024:].reshape(*lead, -1, 8).view(torch.float8_e4m3fn).double()
    return GRID[code.long()] * s.repeat_interleave(16, -1) * ts


# ------------------------------------------------------------- positions
def angles(positions, pair_axis, theta, d):
    """[NB, T, d/2] of positions [axes, NB, T] (any real type)."""
    axis = torch.tensor(pair_axis[:d // 2])
    freq = theta ** (-2.0 * torch.arange(d // 2, dtype=torch.float64) / d) * (axis >= 0)
    return (positions.double()[axis.clamp(min=0)] * freq[:, None, None]).permute(1, 2, 0)


def rotate(x, a):
    x1, x2 = x.double().chunk(2, -1)
    c, s = torch.cos(a), torch.sin(a)
    return torch.cat((x1 * c - x2 * s, x1 * s + x2 * c), -1)


# ------------------------------------------------------------- attention
def visible(cfg, sel, n_sel, qpos):
    """Key positions that the query at qpos attends to."""
    C, G = cfg.chunk_size, cfg.groups_per_chunk
    j = qpos // C
    chunks = set(range(min(cfg.n_sink, j + 1))) | set(range(max(0, j - cfg.n_local), j + 1))
    at = [t for c in sorted(chunks) for t in range(c * C, min((c + 1) * C, qpos + 1))]
    at += [t for g in sel[:n_sel].tolist() for t in range(16 * g, 16 * g + 16)]
    return torch.tensor(at)


def attend(cfg, q, k, v, sel, n_sel):
    """Output [B, q_len, Hq, D] in 64 bits and a bound of the kernels' error.
    k, v: [B, Hkv, >= q_begin + q_len, D] 64-bit values; sel [B, Hu, nQC, kg].

    The bound: a weight w_i = exp(s_i) is rounded to bf16 or fp16 (half a step,
    2^-8 at most) and its score is off by ds = (D + 8) 2^-24 sum|q k| / sqrt(D)
    (a sum of D products in fp32) plus 2^-20 for the exponential, so numerator
    and denominator are each off by at most r = 2^-8 + ds + 2^-20 relative to
    sum w |v| and sum w; with the sums over n keys in fp32 (n 2^-24) and the
    output's own rounding. Besides, fp16 has no step below 2^-24: a weight below 2^-14
    is off by up to 2^-25 absolutely. Weights are relative to a maximum that was a score
    of the row when it was taken, so that score's own weight is 1 and sum w >= 1; n
    weights so rounded move the numerator by n 2^-25 max|v| and the denominator by
    n 2^-25, the output by n 2^-25 (max|v| + |o|) (weights rounded against an earlier,
    smaller maximum shrink with it)."""
    B, T, Hq, _ = q.shape
    Hu = sel.shape[1]
    out = torch.zeros(B, T, Hq, D, dtype=torch.float64)
    tol = torch.zeros_like(out)
    C = cfg.chunk_size
    j0 = cfg.q_begin // C
    for b in range(B):
        for t in range(T):
            qpos = cfg.q_begin + t
            for h in range(Hq):
                u, kh = h // (Hq // Hu), h // (Hq // cfg.n_kv_heads)
                at = visible(cfg, sel[b, u, qpos // C - j0], int(n_sel[b, u, qpos // C - j0]), qpos)
                kk, vv, x = k[b, kh, at], v[b, kh, at], q[b, t, h].double()
                w = torch.softmax(kk @ x / math.sqrt(D), 0)
                ds = (D + 8) * F32 * float((kk.abs() @ x.abs()).max()) / math.sqrt(D)
                out[b, t, h] = w @ vv
                r = BF16 + ds + 2.0 ** -20 + len(at) * F32
                tol[b, t, h] = 2 * r * (w @ vv.abs()) + BF16 * out[b, t, h].abs() * (1 + 2 * r) + (
                    len(at) * 2.0 ** -25 * (vv.abs().amax(0) + out[b, t, h].abs()) * (1 + 2 * r))
    return out, tol


def lists(cfg, heads, seed=0, count=None):
    """Random valid selection lists [B, heads, nQC, kg] and counts of a span."""
    g = torch.Generator().manual_seed(seed)
    C, G = cfg.chunk_size, cfg.groups_per_chunk
    j0 = cfg.q_begin // C
    sel = torch.full((cfg.batch, heads, cfg.n_qchunks, cfg.top_k_groups), -1, dtype=torch.int32)
    n = torch.zeros(cfg.batch, heads, cfg.n_qchunks, dtype=torch.int32)
    for b in range(cfg.batch):
        for h in range(heads):
            for i in range(cfg.n_qchunks):
                j = j0 + i
                open_ = [c * G + e for c in range(cfg.n_sink, max(0, j - cfg.n_local))
                         for e in range(G)]
                m = min(len(open_), cfg.top_k_groups)
                if count is not None:
                    m = min(m, count)
                pick = torch.randperm(len(open_), generator=g)[:m].sort().values
                n[b, h, i] = m
                sel[b, h, i, :m] = torch.tensor([open_[int(e)] for e in pick], dtype=torch.int32)
    return sel, n
