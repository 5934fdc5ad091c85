"""fp64 oracle of the ends of a training step (numpy; test infrastructure): the balance of the routing, the softmax cross
entropy over a vocabulary, orthogonalised matrices, and their gradients.  Written from the formulas that include/moe.h
states, one row or matrix at a time."""
import numpy as np

NS = (3.4445, -4.7750, 2.0315)


def softmax(z):
    e = np.exp(z - z.max(-1, keepdims=True))
    return e / e.sum(-1, keepdims=True)


def logsumexp(z):
    m = z.max(-1, keepdims=True)
    return (m + np.log(np.exp(z - m).sum(-1, keepdims=True)))[..., 0]


# ----------------------------------------------------------------- balance
def _rows(T, B, b, mask):
    t = np.arange(b * (T // B), (b + 1) * (T // B))
    return t if mask is None else t[np.asarray(mask)[t] != 0]


def balance_fwd(logits, topk_idx, B, mask=None):
    """(counts [B, E], mean_p [B, E], loss [B], zloss [B])"""
    T, E = logits.shape
    k = topk_idx.shape[1]
    counts, mean_p = np.zeros((B, E), np.int64), np.zeros((B, E))
    loss, zloss = np.zeros(B), np.zeros(B)
    for b in range(B):
        t = _rows(T, B, b, mask)
        if len(t) == 0:
            continue
        z = logits[t].astype(np.float64)
        counts[b] = np.bincount(topk_idx[t].reshape(-1), minlength=E)
        mean_p[b] = softmax(z).mean(0)
        loss[b] = E / (k * len(t)) * (counts[b] * mean_p[b]).sum()
        zloss[b] = (logsumexp(z) ** 2).mean()
    return counts, mean_p, loss, zloss


def balance_bwd(logits, topk_idx, B, dloss, dzloss, dlogits_in=None, mask=None):
    T, E = logits.shape
    k = topk_idx.shape[1]
    out = np.zeros((T, E)) if dlogits_in is None else dlogits_in.astype(np.float64)
    for b in range(B):
        t = _rows(T, B, b, mask)
        n = len(t)
        if n == 0:
            continue
        z = logits[t].astype(np.float64)
        p = softmax(z)
        a = dloss[b] * E * np.bincount(topk_idx[t].reshape(-1), minlength=E) / (k * n * n)
        out[t] += p * (a - (p * a).sum(1, keepdims=True)) + 2 * dzloss[b] / n * logsumexp(z)[:, None] * p
    return out


# ----------------------------------------------------------- cross entropy
def xent_fwd(x, W, target):
    """(loss [T], lse [T]); target below 0: none."""
    z = x @ W.T
    lse = logsumexp(z)
    use = target >= 0
    t = np.arange(len(target))
    d = z - z[t, np.where(use, target, 0)][:, None]
    return np.where(use, logsumexp(d), 0.0), lse


def xent_grad(x, W, target, dloss, dlse=None):
    """D [T, V]: the gradient of dloss . loss + dlse . lse for the logits."""
    T = len(target)
    use = target >= 0
    g = np.where(use, dloss, 0.0)
    h = np.zeros(T) if dlse is None else dlse
    z = x @ W.T
    p = softmax(z)
    D = (g + h)[:, None] * p
    t = np.arange(T)[use]
    # 1 - p of the target as the sum of the others
    others = p.copy()
    others[t, target[use]] = 0.0
    D[t, target[use]] = h[use] * p[t, target[use]] - g[use] * others[t].sum(1)
    return D


# --------------------------------------------------------- orthogonalised
def orthogonalize(G, steps, eps=1e-7):
    X = G.astype(np.float64) / (np.sqrt((G.astype(np.float64) ** 2).sum()) + eps)
    a, b, c = NS
    for _ in range(steps):
        if X.shape[0] <= X.shape[1]:
            A = X @ X.T
            X = a * X + (b * A + c * A @ A) @ X
        else:
            A = X.T @ X
            X = a * X + X @ (b * A + c * A @ A)
    return X


def orthogonalize_spread(G, steps, unit=2.0 ** -11, eps=1e-7):
    """Bound on the Frobenius norm of what comes of rounding X, A and the polynomial B to relative `unit` after each
    product, relative to the result's norm.  A step f of singular values changes a perturbation of X by at most
    L = max(|f'|, f(s)/s) over [0, 1.3]; what rounding adds is unit |X|_F, and unit (|B|_F + |b| |A|_F + 2 |c| |A|_2 |A|_F)
    |X|_2 through B X.  sqrt(3) of each is left out: a rounding is spread evenly below its largest value."""
    a, b, c = NS
    s = np.linspace(0.0, 1.3, 2601)
    L = max(np.abs(a + 3 * b * s ** 2 + 5 * c * s ** 4).max(), np.abs(a + b * s ** 2 + c * s ** 4).max())
    X = G.astype(np.float64) / (np.sqrt((G.astype(np.float64) ** 2).sum()) + eps)
    if X.shape[0] > X.shape[1]:
        X = X.T
    u = unit / np.sqrt(3.0)
    err = u * np.linalg.norm(X)
    for _ in range(steps):
        A = X @ X.T
        B = b * A + c * A @ A
        n2, nA = np.linalg.norm(X, 2), np.linalg.norm(A)
        add = u * (np.linalg.norm(B) + abs(b) * nA + 2 * abs(c) * np.linalg.norm(A, 2) * nA) * n2
        X = a * X + B @ X
        err = L * err + add + u * np.linalg.norm(X)
    return err / np.linalg.norm(X)


def orthogonalize_rounded(G, steps, eps=1e-7):
    """The same with the library's roundings: X times 2^10 to fp16, with what that leaves times 2^9 in e4m3 beside it for
    the first term of all steps but the last; A times 2^12 and the polynomial (plus 2.5 I in the last two steps) times
    2^11 to fp16 after each product; the result to bf16 (sums in fp64, where the library's are fp32)."""
    def f16(v):
        return v.astype(np.float16).astype(np.float64)

    def e4m3(v):
        step = 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(np.abs(v), 1e-300))), -6) - 3)
        return np.clip(np.rint(v / step) * step, -448, 448)

    def bf16(v):
        u = v.astype(np.float32).view(np.uint32).astype(np.uint64)
        return ((u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32).astype(np.float64)

    def parts(v):
        hi = f16(v)
        return hi, e4m3((v - hi) * 512) / 512

    G = G.astype(np.float64)
    norm = np.sqrt((G ** 2).sum())
    up = 2.0 ** (10 - np.frexp(norm)[1])
    a, b, c = NS
    (X, lo), r = parts(G * up), 1.0 / (norm + eps) / up
    wide = X.shape[0] <= X.shape[1]
    for i in range(steps):
        s = 2.5 if i >= steps - 2 else 0.0
        A = f16((X @ X.T if wide else X.T @ X) * r * r * 4096)
        B = f16(b * 2048 / 4096 * A + c * 2048 / 4096 ** 2 * (A @ A) + s * 2048 * np.eye(len(A)))
        Y = (a - s) * r * (X + (lo if i < steps - 1 else 0)) + r / 2048 * (B @ X if wide else X @ B)
        if i == steps - 1:
            return bf16(Y)
        (X, lo), r = parts(Y * 1024), 1.0 / 1024
