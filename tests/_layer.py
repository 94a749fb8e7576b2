"""A layer's operators in plain form, in 64 bits: what zero_layer_norm,
zero_dropout and their backward passes are tested against. numpy only."""
import numpy as np

MASK = 0xFFFFFFFF


def philox(c, k):
    """Philox4x32-10 (Salmon et al., 2011): counters [n, 4], key (two words) -> words [n, 4]."""
    c = [np.asarray(c)[:, i].astype(np.uint64) for i in range(4)]
    k = [int(k[0]), int(k[1])]
    m = np.uint64(MASK)
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & m, (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), a & m]
        k = [(k[0] + 0x9E3779B9) & MASK, (k[1] + 0xBB67AE85) & MASK]
    return np.stack(c, 1).astype(np.uint32)


def kept(n, p, seed, offset=0, first=0):
    """Which of the elements [first, first + n) dropout keeps."""
    b0 = first // 4
    blocks = np.arange(b0, (first + n + 3) // 4, dtype=np.uint64)
    c = np.zeros((blocks.size, 4), np.uint64)
    c[:, 0], c[:, 1] = blocks & np.uint64(MASK), blocks >> np.uint64(32)
    c[:, 2], c[:, 3] = offset & MASK, offset >> 32 & MASK
    words = philox(c, (seed & MASK, seed >> 32 & MASK)).reshape(-1)[first - 4 * b0:][:n]
    return words.astype(np.uint64) >= np.uint64(round(p * 2 ** 32))


def norm(x, w, b, eps):
    """y, mean, rstd."""
    mean = x.mean(1, keepdims=True)
    rstd = 1 / np.sqrt(((x - mean) ** 2).mean(1, keepdims=True) + eps)
    y = (x - mean) * rstd * w + (0 if b is None else b)
    return y, mean[:, 0], rstd[:, 0]


def norm_grad(dy, x, w, mean, rstd, dresidual=None):
    """dx, dw, db."""
    xhat = (x - mean[:, None]) * rstd[:, None]
    v = dy * w
    dx = rstd[:, None] * (v - v.mean(1, keepdims=True) - xhat * (v * xhat).mean(1, keepdims=True))
    return dx + (0 if dresidual is None else dresidual), (dy * xhat).sum(0), dy.sum(0)
