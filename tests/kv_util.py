"""Batches over a paged cache for the tests: seeded contents, guarded device
buffers, and the same contents as numpy arrays for the oracle."""
import numpy as np
import torch

import oracle.kvcache as OK
import ternary_weight_bitlinear_b200 as B
from gpu_util import bf16_dev, bf16_host, f32_of_bf16
from ternary_weight_bitlinear_b200 import workloads as WL


def bf16_values(rng, shape, std=1.0):
    """Normal values rounded to bf16, as float32."""
    x = torch.from_numpy((rng.standard_normal(shape) * std).astype(np.float32)).to(torch.bfloat16)
    return x.float().numpy()


def bits(x):
    """bf16 bits of float32 values that are bf16 values."""
    return (np.ascontiguousarray(x, np.float32).view(np.uint32) >> 16).astype(np.uint16)


class Paged:
    """A cache of `num_pages` pages holding random rows everywhere (every slot of
    every page, so that a wrong page or slot shows), and a batch over it with
    `new` rows and `lens` positions per sequence.  `spare` extra pages belong to
    no sequence; `pad` rows at the end belong to none."""

    def __init__(self, guard, new, lens, page, kv_heads, d, fmt, seed, pad=0, spare=2, order="slots", poison=True):
        rng = np.random.default_rng(seed)
        self.rng, self.guard = rng, guard
        self.new, self.lens, self.page, self.Hkv, self.d, self.i8 = list(new), list(lens), page, kv_heads, d, fmt == "int8"
        B_ = len(self.new)
        per = [-(-x // page) for x in self.lens]
        num = max(1, sum(per) + spare)
        perm = rng.permutation(num)
        cols = max(per + [1]) + 1
        # entries past a sequence's positions are no pages at all: they must not be used
        self.pages = np.full((B_, cols), 0x7FFFFFF0, np.int32)
        at = 0
        for b, c in enumerate(per):
            self.pages[b, :c] = perm[at:at + c]
            at += c
        self.cu = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        self.T = int(self.cu[-1]) + pad
        shape = (num, page, kv_heads, d)
        k, v = bf16_values(rng, shape), bf16_values(rng, shape)
        if self.i8:
            (self.kc, self.ks), (self.vc, self.vs) = OK.quantise(k), OK.quantise(v)
        else:
            self.kc, self.vc, self.ks, self.vs = k, v, None, None
        if poison:
            self._poison()
        self.order = order
        self.upload()

    def _poison(self):
        """NaN in every slot that no sequence's position has (steps, for an int8 cache)."""
        live = np.zeros(self.kc.shape[:2], bool)
        for b, L in enumerate(self.lens):
            p = np.arange(L)
            live[self.pages[b][p // self.page], p % self.page] = True
        if self.i8:
            self.ks[~live] = np.nan
            self.vs[~live] = np.nan
        else:
            self.kc[~live] = np.nan
            self.vc[~live] = np.nan

    def upload(self):
        g = self.guard

        def pages_dev(x):
            t = torch.from_numpy(x).cuda() if self.i8 else bf16_dev(bits(x))
            if self.order == "heads":   # stored [page, head, slot, d], seen as [page, slot, head, d]
                return g.copy(t.transpose(1, 2).contiguous()).transpose(1, 2)
            return g.copy(t)

        def steps_dev(x):
            return g.copy(torch.from_numpy(np.ascontiguousarray(x.transpose(0, 2, 1))).cuda())

        self.k_dev, self.v_dev = pages_dev(self.kc), pages_dev(self.vc)
        self.ks_dev, self.vs_dev = (steps_dev(self.ks), steps_dev(self.vs)) if self.i8 else (None, None)
        self.cache = B.make_kv_cache(self.k_dev, self.v_dev, self.ks_dev, self.vs_dev)
        self.batch = B.make_kv_batch(g.copy(torch.from_numpy(self.cu).cuda()),
                                     g.copy(torch.tensor(self.lens, dtype=torch.int32, device="cuda")),
                                     g.copy(torch.from_numpy(self.pages).cuda()))

    def sequence(self, b):
        """(k, v) float32 values [len, H_kv, d] of sequence b's positions."""
        p = np.arange(self.lens[b])
        at = self.pages[b][p // self.page], p % self.page
        if not self.i8:
            return self.kc[at], self.vc[at]
        return OK.dequantise(self.kc[at], self.ks[at]), OK.dequantise(self.vc[at], self.vs[at])

    def device_pages(self):
        """The device's pages (and steps) in the oracle's layout."""
        host = lambda t: t.cpu().numpy() if self.i8 else f32_of_bf16(bf16_host(t))  # noqa: E731
        r = [host(self.k_dev), host(self.v_dev)]
        if self.i8:
            r += [t.cpu().numpy().transpose(0, 2, 1) for t in (self.ks_dev, self.vs_dev)]
        return r


def attention_error_bound(want, absv, mag, seen, d):
    """Bound on |gpu - exact| of every output element, from the arithmetic.
    Output rounding to bf16: 2^-8 |want|.  A probability rounded to bf16 for the
    product with the values: 2^-8 each, together at most 2^-8 sum p|v|.  Scores:
    a d-term binary32 sum whose additions may truncate (2^-23 each) of terms
    summing to at most mag in magnitude, the multiplications by the scale (and an
    int8 row's step) and the subtraction of the maximum -- (d + 8) 2^-23 mag
    absolute, the same in the maximum, so a probability is off by the factor
    exp(2 (d + 8) 2^-23 mag), and so is their sum: 4 (d + 8) 2^-23 mag sum p|v|.
    exp2 and the running sums: 2^-20 + seen 2^-22."""
    rel = 2.0 ** -8 + 2.0 ** -20 + seen * 2.0 ** -22 + 4 * (d + 8) * 2.0 ** -23 * mag
    return 2.0 ** -8 * np.abs(want) + rel[..., None] * absv + 2.0 ** -126


def run_attention(p, H, causal, seed, q_std=1.0, scale=None):
    """bitlinear_attn_paged on the batch `p` against the oracle."""
    d = p.d
    scale = float(np.float32(d ** -0.5 if scale is None else scale))
    rng = np.random.default_rng(seed)
    q = bf16_values(rng, (p.T, H, d), q_std)
    out0 = bf16_values(rng, (p.T, H, d))
    qd, od = p.guard.copy(bf16_dev(bits(q))), p.guard.copy(bf16_dev(bits(out0)))
    need = B.bitlinear_attn_paged_workspace_size(p.T, H, p.Hkv, d)
    ws = p.guard.workspace(need) if need else torch.empty(16, dtype=torch.uint8, device="cuda")
    B.bitlinear_attn_paged(qd, p.cache, p.batch, scale, causal=causal, out=od, workspace=ws)
    torch.cuda.synchronize()
    got = f32_of_bf16(bf16_host(od)).astype(np.float64)
    seqs = [p.sequence(b) for b in range(len(p.lens))]
    want, absv, mag, seen = OK.attention(q, [s[0] for s in seqs], [s[1] for s in seqs], p.cu, p.lens, scale, causal, out0)
    used = int(p.cu[-1])
    assert np.array_equal(got[used:], out0[used:].astype(np.float64)), "rows of no sequence were written"
    assert np.array_equal(np.isfinite(got), np.isfinite(want)), "non-finite outputs differ"
    ok = np.isfinite(want)
    err = np.where(ok, np.abs(got - np.where(ok, want, 0)), 0)
    bound = np.where(ok, attention_error_bound(want, absv, mag, seen, d), 1)
    w = np.unravel_index(int(np.argmax(err - bound)), err.shape) if err.size else None
    assert err.size == 0 or (err <= bound).all(), "row %d head %d dim %d: error %g > bound %g (got %g, want %g)" % (
        *w, err[w], bound[w], got[w], want[w])
    assert (got[:used][seen[:used] == 0] == 0).all(), "a row that sees nothing must be zeros"
    return got, od


def padded_batch(count, most_new, most_len, seed):
    """New rows and positions of `count` sequences, most of them without rows: here and there, a run of them longer
    than anything looks at at once, and the batch's end."""
    rng = np.random.default_rng(seed)
    lens = rng.integers(1, most_len + 1, count)
    new = np.minimum(rng.integers(0, most_new + 1, count), lens)
    new[count // 4:count // 4 + 300] = 0
    new[-(count // 5):] = 0
    return [int(x) for x in new], [int(x) for x in lens]
