"""The microscaled 4-bit linear layers in 64 bits on the CPU, straight from include/mq.h, and the
bounds of what a kernel's results may be off."""
import numpy as np
import torch

BLOCK, PIECE, E_MIN, E_MAX = 32, 256, 2, 252
GRID = np.array([0, .5, 1, 1.5, 2, 3, 4, 6])


def philox(counter, key):
    """Philox4x32-10 of counters [n][4] (uint64 arrays holding 32-bit words) under one key."""
    c, k = [counter[:, i].astype(np.uint64) for i in range(4)], [int(key[0]), int(key[1])]
    low = np.uint64(0xFFFFFFFF)
    for _ in range(10):
        p0, p1 = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(p1 >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), p1 & low,
             (p0 >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), p0 & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.stack(c, 1)


def draws(blocks, d, seed):
    """The 16-bit draws [blocks][32] of blocks 0.. in direction d."""
    n = np.arange(4 * blocks, dtype=np.uint64)
    z = np.zeros_like(n)
    words = philox(np.stack([n & np.uint64(0xFFFFFFFF), n >> np.uint64(32), z + np.uint64(d), z], 1),
                   (seed & 0xFFFFFFFF, seed >> 32 & 0xFFFFFFFF))
    return np.stack([words & np.uint64(0xFFFF), words >> np.uint64(16)], 2).reshape(blocks, 32).astype(np.int64)


def scale_exponent(amax):
    """e of blocks with these largest magnitudes (64 bits; 255 where not finite)."""
    finite = np.isfinite(amax)
    mant, power = np.frexp(np.where(finite, amax, 1.0))  # amax = mant * 2^power, mant in [.5, 1)
    e = power - 3 + (mant > 0.75) + 127                 # 6 = .75 * 2^3
    return np.where(finite, np.clip(np.where(amax == 0, E_MIN, e), E_MIN, E_MAX), 255)


def quantize(x, sr_seed=None, d=0):
    """x [rows][cols] (values in float64) -> (codes [rows][padded cols] 0..15, e [rows][padded blocks]);
    padded to whole pieces."""
    x = np.asarray(x, dtype=np.float64)
    rows, cols = x.shape
    width = -(-cols // PIECE) * PIECE
    p = np.zeros((rows, width))
    p[:, :cols] = x
    sign = np.signbit(p)
    b = p.reshape(rows, -1, BLOCK)
    with np.errstate(invalid="ignore"):
        e = scale_exponent(np.abs(b).max(2, initial=0.0))
    a = np.abs(np.where((e == 255)[..., None], 0.0, b)) * np.exp2(127.0 - np.where(e == 255, 127, e))[..., None]
    if sr_seed is None:
        edge = (GRID[1:] + GRID[:-1]) / 2
        up, down = np.searchsorted(edge, a, side="right"), np.searchsorted(edge, a, side="left")
        code = np.where(up % 2 == 0, up, down)
    else:
        a = np.minimum(a, 6.0)
        lo = np.minimum(np.searchsorted(GRID, a, side="right") - 1, 6)
        frac = (a - GRID[lo]) / (GRID[lo + 1] - GRID[lo])
        per_row = -(-cols // BLOCK)
        u = np.zeros((rows, width // BLOCK, BLOCK), dtype=np.int64)
        u[:, :per_row] = draws(rows * per_row, d, sr_seed).reshape(rows, per_row, BLOCK)
        code = lo + (u < frac * 65536)
    code = np.where((e == 255)[..., None], 0, code + 8 * sign.reshape(b.shape))
    return code.reshape(rows, width), e


def packed(code, e):
    """Codes and scale bytes as they are held: [pieces][rows][128], [pieces][rows][8]."""
    rows, width = code.shape
    c = code.reshape(rows, width // PIECE, PIECE // 2, 2)
    codes = (c[..., 0] + 16 * c[..., 1]).astype(np.uint8).transpose(1, 0, 2)
    return (torch.from_numpy(np.ascontiguousarray(codes)),
            torch.from_numpy(np.ascontiguousarray(e.astype(np.uint8).reshape(rows, -1, 8).transpose(1, 0, 2))))


def values(code, e, cols):
    """The values [rows][cols] that codes and scale bytes stand for (NaN where e is 255)."""
    v = GRID[code & 7] * np.where(code & 8, -1.0, 1.0)
    s = np.where(e == 255, np.nan, np.exp2(np.where(e == 255, 0, e) - 127.0))
    return (v.reshape(*e.shape, BLOCK) * s[..., None]).reshape(code.shape)[:, :cols]


def rounded(x, sr_seed=None, d=0):
    return values(*quantize(x, sr_seed, d), np.shape(x)[1])


def product(a, b):
    """a b^T in 64 bits, and the bound of an fp32 sum of its K exact terms in any order: each of
    its K additions is off by at most one unit of 2^-23 of what it makes (2^-24 if it rounds to
    nearest), and no partial sum exceeds the sum of the magnitudes."""
    return a @ b.T, a.shape[1] * 2.0 ** -23 * (np.abs(a) @ np.abs(b).T)


def half_step(dtype, v):
    """What rounding v once to dtype may change: half a step, of normal or subnormal numbers."""
    f = torch.finfo(dtype)
    return np.maximum(np.abs(v) * f.eps / 2, f.smallest_normal * f.eps / 2)


def sigmoid(g):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-g))


def gradients(dh, g, u):
    """dg and du of h = silu(g) u."""
    s = sigmoid(g)
    return dh * u * s * (1 + g * (1 - s)), dh * g * s


# A gradient computed in fp32 may be off by this much of |dh u| (dg) or |dh g s| (du): s carries the
# exponential's argument, rounded twice (|g| 2^-23 of it at most: |g| s (1-s) < 0.28, and as much
# again in g (1 - s)), and under 24 operations of 2^-23 each.
LOOSE = 32 * 2.0 ** -23


def unsure(v, off):
    """How much each quantized value of v [rows][cols] may change if v is off by up to `off`: a code
    step (at the next scale up) where v lies that near a border, or where its block's largest
    magnitude lies that near a border of scales (then every element of the block)."""
    rows, cols = v.shape
    width = -(-cols // BLOCK) * BLOCK
    pad = lambda x: np.pad(x, ((0, 0), (0, width - cols))).reshape(rows, -1, BLOCK)
    b, o = np.abs(pad(v)), pad(off)
    low, high = scale_exponent((b - o).clip(0).max(2)), scale_exponent((b + o).max(2))
    step = np.exp2(high - 127.0)[..., None]
    edge = (GRID[1:] + GRID[:-1]) / 2
    near = (np.abs(b[..., None] / step[..., None] - edge) <= (o / step)[..., None]).any(3)
    return (np.where((low != high)[..., None] | near, 2 * step, 0.0)).reshape(rows, -1)[:, :cols]
