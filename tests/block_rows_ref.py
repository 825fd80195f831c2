"""The norm, its gradient and the block-scaled 8-bit float products in 64 bits
(numpy), with the errors that 32-bit arithmetic may add to them."""

import numpy as np
import torch

U = 2.0 ** -24  # half a step of binary32, relative
BLOCK, LARGEST, TINY = 128, 448.0, 2.0 ** -100
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
# half a step of each type: relative, and absolute where it is subnormal
HALF = {"bf16": (2.0 ** -8, 2.0 ** -134), "fp16": (2.0 ** -11, 2.0 ** -25), "fp32": (2.0 ** -24, 2.0 ** -150)}


def blocks(width):
    return (width + BLOCK - 1) // BLOCK


def scale_at(width):
    return (width + 31) // 32 * 32


def row_bytes(width):
    return (scale_at(width) + 4 * blocks(width) + 127) // 128 * 128


def e4m3(v):
    """Values rounded half-even to e4m3 (magnitudes below 464)."""
    v = np.asarray(v, np.float64)
    e = np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -6)))
    step = 2.0 ** (e - 3)
    got = np.rint(v / step) * step
    assert not (np.abs(got) > LARGEST).any()
    return got


def spread(per_block, width):
    """A value a block -> a value a column."""
    return np.repeat(per_block, BLOCK, axis=-1)[..., :width]


def block_max(y):
    rows, width = y.shape
    padded = np.zeros((rows, blocks(width) * BLOCK))
    padded[:, :width] = np.abs(y)
    return padded.reshape(rows, -1, BLOCK).max(axis=2)


def check_rows(codes, scales, y, err):
    """codes and scales of 8-bit rows against y, of which each value may be off by err."""
    top = block_max(y)
    off = block_max(err * np.ones_like(y))  # the largest magnitude is off by at most the largest error
    d = np.maximum(top, TINY)
    assert (np.abs(scales * LARGEST - d) <= off + 2 * U * d).all()
    factor = spread(LARGEST / d, y.shape[1])
    t = y * factor
    # the value, the factor (two roundings and the largest magnitude's error) and the product
    slack = err * factor + np.abs(t) * (spread(off / d, y.shape[1]) * 1.01 + 4 * U)
    low, high = e4m3(np.clip(t - slack, -LARGEST, LARGEST)), e4m3(np.clip(t + slack, -LARGEST, LARGEST))
    assert ((codes >= low) & (codes <= high)).all()


def unpack(buf, rows, width):
    """(codes, scales) of a uint8 tensor of e4m3 rows, as float64."""
    m = buf.view(rows, row_bytes(width))
    at = scale_at(width)
    codes = m[:, :width].contiguous().view(torch.float8_e4m3fn).float().cpu().double().numpy()
    scales = m[:, at:at + 4 * blocks(width)].contiguous().view(torch.float32).cpu().double().numpy()
    return codes, scales


def padding(buf, rows, width):
    """The bytes of e4m3 rows that hold neither codes nor scales."""
    m = buf.view(rows, row_bytes(width)).cpu().numpy()
    at = scale_at(width)
    return np.concatenate([m[:, width:at], m[:, at + 4 * blocks(width):]], axis=1)


def near(got, want, kind, err):
    """got (of a type) against want, which is off by err before the rounding to the type."""
    rel, sub = HALF[kind]
    return (np.abs(got - want) <= (np.abs(want) + err) * rel + sub + err).all()


# ---- the norm --------------------------------------------------------------------

# A row's sum of squares is a chain of at most 32 multiply-adds a lane, 6 additions
# over the lanes and 16 over the waves, all of one sign; rstd takes half of its error,
# and the division, the addition, the root and the reciprocal a rounding each.
RSTD = 31 * U
NORM = RSTD + 2 * U


def norm(s, weight, eps):
    """(y, rstd) of the rows s as they are kept."""
    rstd = 1.0 / np.sqrt((s * s).mean(axis=1, keepdims=True) + eps)
    return s * rstd * weight, rstd[:, 0]


def norm_backward(g, s, weight, rstd, skip=None):
    """(dx, error of dx, dw, error of dw)."""
    h = s.shape[1]
    xh, gw = s * rstd[:, None], g * weight
    dot = (gw * xh).mean(axis=1, keepdims=True)
    dx = rstd[:, None] * (gw - xh * dot)
    # a lane's chain, the lanes and the waves of the mean, its product's and factors' roundings: 60 at most
    off = 60 * U * np.abs(gw * xh).mean(axis=1, keepdims=True)
    err = rstd[:, None] * (4 * U * (np.abs(gw) + np.abs(xh * dot)) + np.abs(xh) * off)
    if skip is not None:
        dx = dx + skip
        err = err + U * np.abs(dx)
    # a column's sum: a rounding for each row and for each part, and two in its terms
    dw_err = (s.shape[0] + 8) * U * np.abs(g * xh).sum(axis=0)
    return dx, err + 2 * U * np.abs(dx), (g * xh).sum(axis=0), dw_err


def matmul(a, b):
    """a @ b in 64 bits, on the GPU where there is one (the host takes minutes over the largest cases)."""
    if torch.cuda.is_available():
        return (torch.from_numpy(np.ascontiguousarray(a)).cuda() @ torch.from_numpy(np.ascontiguousarray(b)).cuda()).cpu().numpy()
    return a @ b


# ---- the products ----------------------------------------------------------------


def owners(counts, rows):
    """Expert of each row, -1 for none."""
    got = np.full(rows, -1)
    at = 0
    for g, c in enumerate(counts):
        c = max(int(c), 0)
        got[min(at, rows):min(at + c, rows)] = g
        at += c
    return got


def product(a, ts, w, ws, own, n):
    """(y, its error): a [rows, k] and w [groups, parts * n, k] code values, ts [rows, kb], ws [groups, parts * nb, kb]."""
    rows, k = a.shape
    wide = w.shape[1]
    y, err = np.zeros((rows, wide)), np.zeros((rows, wide))
    full = a * spread(ts, k)
    for g in np.unique(own[own >= 0]):
        at = own == g
        per_row = np.concatenate([np.repeat(p, BLOCK, axis=0)[:n] for p in np.split(ws[g], wide // n)])
        wf = w[g] * spread(per_row, k)
        y[at] = matmul(full[at], wf.T)
        # 128 terms a block, a multiply-add for each block, the scales' product and parts of k added at the end
        err[at] = (128 + blocks(k) + 8) * U * matmul(np.abs(full[at]), np.abs(wf).T)
    return y, err


def cut(a, ts, w, ws, own, n):
    """What the 8-bit matrix instruction may lose: of each eight consecutive products whatever lies below 2^-13 of
    the largest, seven times at most (the largest keeps all of its 8 bits)."""
    rows, k = a.shape
    wide = w.shape[1]
    lost = np.zeros((rows, wide))

    def eights(v):
        return np.abs(v).reshape(*v.shape[:-1], k // 8, 8).max(axis=-1)

    full = eights(a * spread(ts, k))  # a block's scale is the same for its sixteen eights
    for g in np.unique(own[own >= 0]):
        at = own == g
        per_row = np.concatenate([np.repeat(p, BLOCK, axis=0)[:n] for p in np.split(ws[g], wide // n)])
        lost[at] = 7 * 2.0 ** -13 * matmul(full[at], eights(w[g] * spread(per_row, k)).T)
    return lost


def gated(y, err, n):
    """(act, its error) of gate and up columns."""
    g, u, eg, eu = y[:, :n], y[:, n:], err[:, :n], err[:, n:]
    with np.errstate(over="ignore"):
        silu = g / (1.0 + np.exp(-g))
    act = silu * u
    # the slope of g / (1 + e^-g) is at most 1.1; e^-g to 2 units, and four operations
    return act, 1.1 * eg * (np.abs(u) + eu) + np.abs(silu) * eu + 8 * U * np.abs(act)
