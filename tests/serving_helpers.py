"""Plain 64-bit forms of the serving operators (prompt attention, the 4-bit cache), in NumPy, written
from their definitions; they import nothing of the library."""
import numpy as np


def to_bf16(x):
    """float64/32 -> the nearest bfloat16's value (ties to even), by integer arithmetic on float32."""
    u = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    u = (u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000
    return u.astype(np.uint32).view(np.float32).reshape(np.shape(x))


def softmax_rows(x):
    """Softmax over the last axis; a row of -inf gives zeros."""
    m = x.max(-1, keepdims=True, initial=-np.inf)
    e = np.exp(x - np.where(np.isinf(m), 0.0, m))
    l = e.sum(-1, keepdims=True)
    return e / np.where(l == 0, 1.0, l)


def prompt_attention(q, k, v, cu_q, cu_kv, n_weight):
    """q [rows, H, d], k, v [rows, H_kv, d] float64 -> o, weight [B, H_kv, n_weight]."""
    H, d, Hk = q.shape[1], q.shape[2], k.shape[1]
    B = len(cu_q) - 1
    o, w = np.zeros(q.shape), np.zeros((B, Hk, n_weight))
    for b in range(B):
        qs, ks = slice(cu_q[b], cu_q[b + 1]), slice(cu_kv[b], cu_kv[b + 1])
        n_q, n_kv = cu_q[b + 1] - cu_q[b], cu_kv[b + 1] - cu_kv[b]
        hidden = np.arange(n_kv)[None, :] > np.arange(n_q)[:, None] + (n_kv - n_q)
        for h in range(H):
            g = h // (H // Hk)
            x = q[qs, h] @ k[ks, g].T / np.sqrt(d)
            x[hidden] = -np.inf
            p = softmax_rows(x) if n_kv else np.zeros((n_q, 0))
            o[qs, h] = p @ v[ks, g]
            w[b, g, :min(n_kv, n_weight)] += p.sum(0)[:n_weight]
    return o, w


def quantize4(x):
    """x [..., d] float32 -> codes [..., d] int, scales [..., d/32] (bfloat16 values)."""
    x = np.asarray(x, np.float32)
    g = np.where(np.isfinite(x), x, np.float32(0)).reshape(x.shape[:-1] + (x.shape[-1] // 32, 32))
    s = to_bf16(np.abs(g).max(-1) / np.float32(7))
    s = np.where(s == 0, np.float32(1), s).astype(np.float32)
    code = np.clip(np.rint(g / s[..., None]), -7, 7).astype(np.int64)
    return code.reshape(x.shape), s


def _nibble_of_channel(d, run):
    c = np.arange(d)
    return (((c % 32) // run) * (d // 32) + c // 32) * run + c % run


def pack4(code, run):
    """codes [..., d] -> bytes; run: channels kept together (8 for K, 4 for V)."""
    d = code.shape[-1]
    nib = np.zeros(code.shape, np.uint8)
    nib[..., _nibble_of_channel(d, run)] = (code + 8).astype(np.uint8)
    return nib[..., 0::2] | (nib[..., 1::2] << 4)


def unpack4(byts, run):
    d = byts.shape[-1] * 2
    nib = np.zeros(byts.shape[:-1] + (d,), np.int64)
    nib[..., 0::2], nib[..., 1::2] = byts & 15, byts >> 4
    return nib[..., _nibble_of_channel(d, run)] - 8


def values4(byts, scale, run):
    return unpack4(byts, run).astype(np.float64) * np.repeat(np.asarray(scale, np.float64), 32, axis=-1)


def kv4_attention(q, k, v, n):
    """q [H, d], k, v [H_kv, rows, d] float64 -> o [H, d], weight increment [H_kv, rows]."""
    H, d = q.shape
    Hk = k.shape[0]
    o, w = np.zeros((H, d)), np.zeros(k.shape[:2])
    if n:
        for h in range(H):
            g = h // (H // Hk)
            p = softmax_rows(q[h] @ k[g, :n].T / np.sqrt(d))
            o[h] = p @ v[g, :n]
            w[g, :n] += p
    return o, w


def evict_sources(weight, pos, n, seen, keep, recent):
    """The row each of the rows 0 .. min(n, keep)-1 takes its contents from."""
    if n <= keep:
        return list(range(n))
    def rank(j):
        if recent > 0 and pos[j] >= seen - recent:
            return (0, 0.0, j)
        return (2, 0.0, j) if np.isnan(weight[j]) else (1, -float(weight[j]), j)
    kept = set(sorted(range(n), key=rank)[:keep])
    behind = iter(sorted(j for j in kept if j >= keep))
    return [r if r in kept else next(behind) for r in range(keep)]
