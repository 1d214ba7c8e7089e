"""CPU oracle of the paged key/value cache and of the attention over it, numpy,
float64 wherever the definition does not name a 32-bit step.

TEST INFRASTRUCTURE ONLY, like the rest of ``oracle/``.

A batch: cu_q [B + 1] starts of each sequence's new rows, kv_len [B] positions
(new ones included), pages [B, max_pages] page table.  Row i of a sequence's n
new rows stands at position kv_len - n + i; position p lies in page
pages[b, p // page_size], slot p % page_size.

Function      Definition followed
------------  ---------------------------------------------------------------
places        (row, sequence, position, page, slot) of every row that has one
quantise      s = RN32(127 / max(max|x|, 1e-5)), code = clamp(rint(RN32(x s)),
              -128, 127), step = RN32(1 / s); a row holding an infinity or NaN:
              zero codes, NaN step
dequantise    RN32(code step)
attention     softmax(q k^T scale) v over the positions a row sees, query head
              h reading key/value head h // group; no position seen: zeros
"""
import numpy as np


def places(cu_q, kv_len, pages, page_size):
    for b in range(len(kv_len)):
        n = int(cu_q[b + 1]) - int(cu_q[b])
        for i in range(n):
            p = int(kv_len[b]) - n + i
            if p >= 0:
                yield int(cu_q[b]) + i, b, p, int(pages[b][p // page_size]), p % page_size


def quantise(x):
    """float32 rows [..., d] (values of bf16) -> (int8 codes, float32 steps [...])."""
    x = np.asarray(x, np.float32)
    ok = np.isfinite(x).all(-1)
    h = np.where(ok[..., None], x, np.float32(0))
    s = np.float32(127) / np.maximum(np.abs(h).max(-1), np.float32(1e-5))
    code = np.clip(np.rint(h * s[..., None]), -128, 127).astype(np.int8)
    return code, np.where(ok, np.float32(1) / s, np.float32(np.nan)).astype(np.float32)


def dequantise(code, step):
    return code.astype(np.float32) * np.asarray(step, np.float32)[..., None]


def attention(q, ks, vs, cu_q, kv_len, scale, causal, out):
    """q [T, H, d]; ks[b], vs[b]: that sequence's positions [kv_len[b], H_kv, d];
    out [T, H, d] holds the rows' earlier contents.  Returns float64 (out, absv,
    mag, seen): absv = sum_j p_j |v_j| of every element, mag [T, H] the largest
    scale * sum_i |q_i k_ji| of a seen position, seen [T, H] their number."""
    q = np.asarray(q, np.float64)
    res = np.array(out, np.float64)
    mag = np.zeros(q.shape[:2])
    seen = np.zeros(q.shape[:2], np.int64)
    absv = np.zeros_like(res)
    for b in range(len(kv_len)):
        n, L = int(cu_q[b + 1]) - int(cu_q[b]), int(kv_len[b])
        k, v = np.asarray(ks[b], np.float64), np.asarray(vs[b], np.float64)
        for i in range(n):
            r = int(cu_q[b]) + i
            end = max(0, min(L, L - n + i + 1)) if causal else L
            for h in range(q.shape[1]):
                g = h // (q.shape[1] // k.shape[1])
                if end == 0:
                    res[r, h] = 0.0
                    continue
                s = (k[:end, g] @ q[r, h]) * float(scale)
                p = np.exp(s - s.max())
                p /= p.sum()
                res[r, h] = p @ v[:end, g]
                absv[r, h] = p @ np.abs(v[:end, g])
                mag[r, h] = float(scale) * (np.abs(k[:end, g]) @ np.abs(q[r, h])).max()
                seen[r, h] = end
    return res, absv, mag, seen
