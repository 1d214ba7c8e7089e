"""Attention over the paged cache on the GPU against the float64 oracle, within
the bound derived in kv_util.attention_error_bound."""
import numpy as np
import pytest
import torch

import ternary_weight_bitlinear_b200 as B
from gpu_util import bf16_dev, bf16_host, f32_of_bf16
from kv_util import Paged, attention_error_bound, bf16_values, bits, padded_batch, run_attention
from ternary_weight_bitlinear_b200 import workloads as WL

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _device_status_clean():
    yield
    assert B.bitlinear_device_status() == 0


HEADS = [(20, 5, 128), (8, 8, 64), (16, 2, 128), (4, 2, 64), (8, 1, 128), (6, 2, 64), (7, 1, 128)]


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
@pytest.mark.parametrize("H,Hkv,d", HEADS)
def test_mixed_batch(H, Hkv, d, fmt, guard):
    """Decode rows, drafts, a chunk, a prompt, an empty sequence and rows without positions, in one padded batch."""
    p = Paged(guard, [1, 5, 33, 70, 0, 3, 1], [1, 140, 200, 70, 9, 2, 129], 16, Hkv, d, fmt, seed=H, pad=5)
    run_attention(p, H, True, seed=H + 1)


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
@pytest.mark.parametrize("L", [1, 2, 15, 16, 17, 127, 128, 129, 255, 257, 1000, 2048])
def test_decode_lengths(L, fmt, guard):
    p = Paged(guard, [1], [L], 64, WL.KV_HEADS, WL.HEAD_DIM, fmt, seed=L)
    got, _ = run_attention(p, WL.Q_HEADS, True, seed=L + 1)
    if L == 1 and fmt == "bf16":  # one position: its value row, exactly
        assert np.array_equal(got[0].reshape(5, 4, -1), np.repeat(p.sequence(0)[1][0][:, None], 4, 1))


@pytest.mark.parametrize("page", [16, 32, 48, 64, 96, 128, 144, 256])
@pytest.mark.parametrize("fmt", ["bf16", "int8"])
def test_page_sizes(page, fmt, guard):
    p = Paged(guard, [40, 1, 3], [300, 513, 77], page, 2, 128, fmt, seed=page, order="heads")
    run_attention(p, 8, True, seed=page)


@pytest.mark.parametrize("n,L", [(31, 31), (32, 32), (33, 33), (64, 64), (65, 65), (127, 300), (130, 131), (257, 257)])
@pytest.mark.parametrize("causal", [True, False])
def test_prompt_sizes(n, L, causal, guard):
    p = Paged(guard, [n], [L], 32, 1, 128, "bf16" if n % 2 else "int8", seed=n)
    run_attention(p, 4, causal, seed=n)


@pytest.mark.parametrize("d", [64, 128])
def test_prompts_without_grouping(d, guard):
    p = Paged(guard, [300, 129], [300, 500], 16, 1, d, "bf16", seed=d)
    run_attention(p, 1, True, seed=d)


@pytest.mark.parametrize("group", [1, 3, 12, 100, 128])
def test_group_sizes(group, guard):
    p = Paged(guard, [3, 1, 9], [140, 64, 9], 16, 1, 64, "int8" if group % 2 else "bf16", seed=group)
    run_attention(p, group, True, seed=group)


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
@pytest.mark.parametrize("H,Hkv,d", [(20, 5, 128), (8, 8, 64)])
def test_many_items_of_mixed_lengths(H, Hkv, d, fmt, guard):
    """More items than SMs: runs of one-tile sequences between long ones, so shares end anywhere and the softmax
    groups' turns at the rings differ."""
    rng = np.random.default_rng(H)
    lens = [int(rng.choice([1, 60, 128, 129, 300, 700, 2500])) for _ in range(80)]
    new = [int(min(L, rng.choice([1, 1, 1, 2, 20]))) for L in lens]
    p = Paged(guard, new, lens, 64, Hkv, d, fmt, seed=H + 5)
    run_attention(p, H, True, seed=H + 6)


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
@pytest.mark.parametrize("H,Hkv,d", [(20, 5, 128), (8, 8, 64), (16, 2, 128)])
def test_many_decode_rows_and_one_chunk(H, Hkv, d, fmt, guard):
    """Decode rows (few rows a sequence on average) with one sequence of many rows among them."""
    rng = np.random.default_rng(H + 1)
    lens = [int(rng.choice([1, 31, 32, 33, 300, 1900])) for _ in range(60)] + [333]
    new = [1] * 30 + [2, 0] * 15 + [50]
    p = Paged(guard, [min(a, b) for a, b in zip(new, lens)], lens, 16, Hkv, d, fmt, seed=H + 7, pad=3)
    run_attention(p, H, True, seed=H + 8)


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
@pytest.mark.parametrize("H,Hkv,d", [(4, 4, 64), (40, 2, 64), (100, 1, 128)])
def test_many_sequences(H, Hkv, d, fmt, guard):
    """More sequences than a CTA has threads, runs of empty ones among them and behind them: few rows a sequence and
    many (of the heads)."""
    new, lens = padded_batch(1100, 1, 70, seed=H)
    p = Paged(guard, new, lens, 16, Hkv, d, fmt, seed=H + 9, pad=3)
    run_attention(p, H, True, seed=H + 10)


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
@pytest.mark.parametrize("n,group,L", [(1, 4, 2051), (1, 12, 2051), (2, 4, 4500), (1, 4, 7001), (1, 16, 30000),
                                       (8, 4, 2051), (8, 4, 20001), (70, 4, 20001)])
def test_one_sequence_over_many_parts(n, group, L, fmt, guard):
    """One key/value head: the positions of a single item are shared out over most of the GPU, or all of it."""
    p = Paged(guard, [n], [L], 64, 1, 128 if n > 1 or group == 4 else 64, fmt, seed=L + n)
    run_attention(p, group, True, seed=L + group)


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
def test_peaked_scores(fmt, guard):
    # large queries: the softmax is close to one-hot and the running maximum moves
    p = Paged(guard, [1, 64], [700, 300], 16, 5, 128, fmt, seed=77)
    run_attention(p, 20, True, seed=78, q_std=8.0)


def test_scores_that_climb(guard):
    """Keys that grow along the sequence: the running maximum rises in every tile."""
    p = Paged(guard, [1, 40], [900, 900], 16, 1, 128, "bf16", seed=79)
    for b in range(2):
        pos = np.arange(900)
        at = p.pages[b][pos // 16], pos % 16
        p.kc[at] = f32_of_bf16(bits(np.abs(p.kc[at]) * (pos[:, None, None] / 60.0)))
    p.upload()
    d, H = 128, 4
    q = np.abs(bf16_values(np.random.default_rng(80), (p.T, H, d)))
    import oracle.kvcache as OK
    qd, od = bf16_dev(bits(q)), guard.empty((p.T, H, d), torch.bfloat16)
    B.bitlinear_attn_paged(qd, p.cache, p.batch, 0.05, out=od)
    s = [p.sequence(b) for b in range(2)]
    want, absv, mag, seen = OK.attention(q, [x[0] for x in s], [x[1] for x in s], p.cu, p.lens, np.float32(0.05), True,
                                         np.zeros_like(q))
    got = f32_of_bf16(bf16_host(od))
    assert (np.abs(got - want) <= attention_error_bound(want, absv, mag, seen, d)).all()


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
@pytest.mark.parametrize("what", ["k nan", "k inf", "v nan", "v inf"])
def test_non_finite_rows_reach_only_rows_that_see_them(what, fmt, guard):
    """A position that holds an infinity or NaN: rows before it (causal) are untouched."""
    p = Paged(guard, [60, 1], [90, 50], 16, 2, 64, fmt, seed=81)
    at = p.pages[0][57 // 16], 57 % 16  # position 57: seen by rows 27.. of the first sequence
    bad = np.nan if "nan" in what else np.inf
    if fmt == "int8":  # the cache holds such a row as zero codes with a NaN step
        (p.ks if what[0] == "k" else p.vs)[at] = np.nan
    else:
        (p.kc if what[0] == "k" else p.vc)[at][..., 11] = bad
    p.upload()
    H, d = 8, 64
    q = bf16_values(np.random.default_rng(82), (p.T, H, d))
    clean = Paged(guard, [60, 1], [90, 50], 16, 2, 64, fmt, seed=81)
    a = B.bitlinear_attn_paged(bf16_dev(bits(q)), p.cache, p.batch, d ** -0.5)
    b = B.bitlinear_attn_paged(bf16_dev(bits(q)), clean.cache, clean.batch, d ** -0.5)
    a, b = f32_of_bf16(bf16_host(a)), f32_of_bf16(bf16_host(b))
    import oracle.kvcache as OK
    s = [p.sequence(i) for i in range(2)]
    with np.errstate(invalid="ignore"):
        want, absv, mag, seen = OK.attention(q, [x[0] for x in s], [x[1] for x in s], p.cu, p.lens,
                                             np.float32(d ** -0.5), True, np.zeros_like(q))
    assert np.array_equal(np.isfinite(a), np.isfinite(want)) and np.array_equal(np.isnan(a), np.isnan(want))
    assert np.isfinite(b).all() and np.isfinite(a[:27]).all() and np.isfinite(a[60]).all()
    ok = np.isfinite(want)
    bound = attention_error_bound(np.where(ok, want, 0), np.where(ok, absv, 0), np.where(np.isfinite(mag), mag, 0), seen, d)
    assert (np.abs(a - np.where(ok, want, 0))[ok] <= bound[ok]).all()


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
@pytest.mark.parametrize("n,L", [(4, 4), (4, 40), (4, 5000), (64, 64), (64, 3000)])
@pytest.mark.parametrize("d", [64, 128])
def test_a_nan_among_the_new_rows(n, L, d, fmt, guard):
    """The last new row is NaN in keys and values: the others, which do not see it, are as without it, whichever
    kernel computes them and however the positions are shared out."""
    p = Paged(guard, [n], [L], 16, 1, d, fmt, seed=L + d)
    at = p.pages[0][(L - 1) // 16], (L - 1) % 16
    if fmt == "int8":
        p.ks[at] = p.vs[at] = np.nan
    else:
        p.kc[at] = p.vc[at] = np.nan
    p.upload()
    q = bf16_values(np.random.default_rng(n), (n, 4, d))
    scale = np.float32(d ** -0.5)
    got = f32_of_bf16(bf16_host(B.bitlinear_attn_paged(bf16_dev(bits(q)), p.cache, p.batch, float(scale))))
    assert np.isnan(got[-1]).all()
    import oracle.kvcache as OK
    k, v = (x[:-1] for x in p.sequence(0))
    want, absv, mag, seen = OK.attention(q[:-1], [k], [v], np.array([0, n - 1]), [L - 1], scale, True,
                                         np.zeros_like(q[:-1]))
    assert (np.abs(got[:-1] - want) <= attention_error_bound(want, absv, mag, seen, d)).all()


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
@pytest.mark.parametrize("n,L,d", [(3, 3, 128), (3, 700, 64), (70, 70, 128), (70, 900, 64)])
def test_a_nan_query_reaches_its_own_row_only(n, L, d, fmt, guard):
    """Rows share products: a NaN or an infinity in one head of one token stays there."""
    p = Paged(guard, [n, 2], [L, 40], 16, 2, d, fmt, seed=L + d)
    q = bf16_values(np.random.default_rng(n), (n + 2, 8, d))
    bad = q.copy()
    bad[1, 3, 7], bad[n - 1, 6, 0] = np.nan, np.inf
    a, b = (B.bitlinear_attn_paged(bf16_dev(bits(x)), p.cache, p.batch, d ** -0.5) for x in (q, bad))
    own = torch.zeros(n + 2, 8, dtype=torch.bool, device="cuda")
    own[1, 3] = own[n - 1, 6] = True
    assert torch.equal(a[~own], b[~own]) and torch.isnan(b[1, 3]).all() and not torch.isfinite(b[n - 1, 6]).any()


def test_rows_that_overlap_are_refused(guard):
    p = Paged(guard, [3], [20], 16, 1, 64, "bf16", seed=85)
    w = torch.zeros((4, 8, 64), dtype=torch.bfloat16, device="cuda")
    for q, out in ((w[:3, :4], w[:3, :4]), (w[:3, :4], w[:3, 3:7]), (w[:3, 4:], w[1:, 3:7]), (w[1:, :4], w[:3, 1:5])):
        with pytest.raises(B.BitLinearError):
            B.bitlinear_attn_paged(q, p.cache, p.batch, 0.125, out=out)
    q = torch.randn((3, 4, 64), device="cuda").to(torch.bfloat16)
    w[:3, :4] = q
    B.bitlinear_attn_paged(w[:3, :4], p.cache, p.batch, 0.125, out=w[:3, 4:])
    B.bitlinear_attn_paged(w[:3, :4], p.cache, p.batch, 0.125, out=w[1:, 4:])
    assert torch.equal(w[1:, 4:], B.bitlinear_attn_paged(q, p.cache, p.batch, 0.125))


def test_every_score_minus_infinity_is_nan(guard):
    p = Paged(guard, [1], [3], 16, 1, 64, "bf16", seed=83)
    at = p.pages[0][0], slice(0, 3)
    p.kc[at] = -np.inf
    p.upload()
    out = B.bitlinear_attn_paged(torch.ones((1, 2, 64), dtype=torch.bfloat16, device="cuda"), p.cache, p.batch, 1.0)
    assert torch.isnan(out).all()


def test_strided_rows(guard):
    """q as a slice of a fused projection, out as a slice of a wider buffer."""
    p = Paged(guard, [3, 20], [50, 20], 16, 2, 64, "bf16", seed=84)
    H, d = 4, 64
    w = torch.randn((p.T, H + 4, d), device="cuda").to(torch.bfloat16)
    wide = guard.empty((p.T, H + 2, d), torch.bfloat16, fill=0)
    a = B.bitlinear_attn_paged(w[:, 1:1 + H], p.cache, p.batch, 0.125, out=wide[:, 1:1 + H])
    b = B.bitlinear_attn_paged(w[:, 1:1 + H].contiguous(), p.cache, p.batch, 0.125)
    c = B.bitlinear_attn_paged(w[:, 1:1 + H].reshape(p.T, -1), p.cache, p.batch, 0.125)
    assert torch.equal(a, b) and torch.equal(b.reshape(p.T, -1), c)
    assert (wide[:, 0] == 0).all() and (wide[:, -1] == 0).all()


def test_repeats_are_equal(guard):
    p = Paged(guard, [1, 90, 7], [3000, 400, 1200], 64, 2, 128, "int8", seed=85)
    q = torch.randn((p.T, 8, 128), device="cuda").to(torch.bfloat16)
    first = B.bitlinear_attn_paged(q, p.cache, p.batch, 0.1)
    for _ in range(5):
        assert torch.equal(first, B.bitlinear_attn_paged(q, p.cache, p.batch, 0.1))


def test_bad_pages_are_recorded(guard):
    p = Paged(guard, [4, 2], [40, 33], 16, 2, 64, "bf16", seed=86)
    q = bf16_dev(bits(bf16_values(np.random.default_rng(1), (p.T, 4, 64))))
    ref = B.bitlinear_attn_paged(q, p.cache, p.batch, 0.125)
    for bad in (-1, p.kc.shape[0], 2 ** 31 - 1, -2 ** 31):
        p.pages[0, 1] = bad
        p.batch.held[2].copy_(torch.from_numpy(p.pages))
        out = B.bitlinear_attn_paged(q, p.cache, p.batch, 0.125)
        assert B.bitlinear_device_status() == 9
        assert torch.equal(out[4:], ref[4:])  # the other sequence is not affected


def test_arrays_that_lie_stay_inside_the_buffers(guard):
    p = Paged(guard, [4, 4], [20, 20], 16, 2, 64, "bf16", seed=87, poison=False)
    q = torch.randn((p.T, 4, 64), device="cuda").to(torch.bfloat16)
    for cu, lens in (([-5, 3, 900], [20, 20]), ([0, 4, 8], [2 ** 31 - 1, -7]), ([8, 4, 0], [20, 20]),
                     ([2 ** 31 - 1, -2 ** 31, 5], [20, 20])):
        p.batch.held[0].copy_(torch.tensor(cu, dtype=torch.int32))
        p.batch.held[1].copy_(torch.tensor(lens, dtype=torch.int32))
        out = guard.empty((p.T, 4, 64), torch.bfloat16)
        ws = guard.workspace(max(16, B.bitlinear_attn_paged_workspace_size(p.T, 4, 2, 64)))
        B.bitlinear_attn_paged(q, p.cache, p.batch, 0.125, out=out, workspace=ws)
        torch.cuda.synchronize()
    assert B.bitlinear_device_status() in (0, 9)  # whether a page was missed depends on the table


def test_graphs_that_share_a_workspace(guard):
    """Two captured calls with one workspace, replayed in turn, with lengths changed in between."""
    ps = [Paged(guard, [1, 1, 1], [900, 70, 2000], 64, 5, 128, "int8", seed=88),
          Paged(guard, [50, 3], [700, 1500], 16, 1, 128, "bf16", seed=89)]
    heads = (20, 8)
    qs = [torch.randn((p.T, H, 128), device="cuda").to(torch.bfloat16) for p, H in zip(ps, heads)]
    need = max(B.bitlinear_attn_paged_workspace_size(p.T, H, p.Hkv, 128) for p, H in zip(ps, heads))
    ws = guard.workspace(max(16, need))
    outs, graphs = [guard.empty(q.shape, torch.bfloat16) for q in qs], []
    for p, q, o in zip(ps, qs, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            B.bitlinear_attn_paged(q, p.cache, p.batch, 0.09, out=o, workspace=ws)
        graphs.append(g)
    for lens in (([900, 70, 2000], [700, 1500]), ([2, 70, 1999], [50, 1])):
        for p, l in zip(ps, lens):
            p.batch.held[1].copy_(torch.tensor(l, dtype=torch.int32))
        for o in outs:
            o.zero_()
        for _ in range(3):
            for g in graphs:
                g.replay()
        torch.cuda.synchronize()
        for p, q, o in zip(ps, qs, outs):
            assert torch.equal(o, B.bitlinear_attn_paged(q, p.cache, p.batch, 0.09))


def test_two_calls_at_once(guard):
    """Calls on two streams, each with its own workspace, beside one another."""
    ps = [Paged(guard, [1, 80], [5000, 300], 64, 5, 128, f, seed=90) for f in ("int8", "bf16")]
    qs = [torch.randn((p.T, 20, 128), device="cuda").to(torch.bfloat16) for p in ps]
    want = [B.bitlinear_attn_paged(q, p.cache, p.batch, 0.09) for p, q in zip(ps, qs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ps]
    got = [[], []]
    for _ in range(10):
        for i, (p, q, s) in enumerate(zip(ps, qs, streams)):
            got[i].append(B.bitlinear_attn_paged(q, p.cache, p.batch, 0.09, stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for outs, w in zip(got, want) for o in outs)


def test_a_decode_step_as_it_is_used(guard):
    """A prompt, then two decode steps of a batch, as a layer runs them: rotate, write the new keys and values,
    attend over the cache -- against the one-token kernel on a contiguous cache of the same rows."""
    H, Hkv, d, page, theta = WL.Q_HEADS, WL.KV_HEADS, WL.HEAD_DIM, 16, 500000.0
    rng = np.random.default_rng(91)
    prompts = [37, 5, 16]
    cols = 5
    kp = torch.zeros((16, page, Hkv, d), dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    cache = B.make_kv_cache(kp, vp)
    table = torch.from_numpy(rng.permutation(16)[:3 * cols].reshape(3, cols).astype(np.int32)).cuda()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    flat = [[torch.zeros((64, Hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)] for _ in range(3)]
    lens = [0, 0, 0]
    for new in (prompts, [1, 1, 1], [1, 1, 1]):
        T = sum(new)
        q, k, v = (bf16_dev(bits(bf16_values(rng, (T, h * d)))) for h in (H, Hkv, Hkv))
        lens = [a + b for a, b in zip(lens, new)]
        pos = i32([L - n + i for L, n in zip(lens, new) for i in range(n)])
        q, k = B.bitlinear_rope(q, pos, H, theta), B.bitlinear_rope(k, pos, Hkv, theta)
        cu = np.concatenate([[0], np.cumsum(new)])
        batch = B.make_kv_batch(i32(cu.tolist()), i32(lens), table)
        B.bitlinear_kv_write(k, v, cache, batch)
        out = B.bitlinear_attn_paged(q, cache, batch, d ** -0.5)
        for b in range(3):
            n, L = new[b], lens[b]
            flat[b][0][L - n:L] = k[cu[b]:cu[b + 1]].view(-1, Hkv, d)
            flat[b][1][L - n:L] = v[cu[b]:cu[b + 1]].view(-1, Hkv, d)
            for i in range(n):
                one = B.bitlinear_attn_decode(q[cu[b] + i], flat[b][0], flat[b][1], L - n + i + 1, H, Hkv, d ** -0.5)
                top = float(flat[b][1][:L].abs().max())
                # both are within their bounds of the exact value: 2^-8 of the output, and 2^-8 sum p|v| <= 2^-8 max|v|
                err = (out[cu[b] + i].float() - one.float()).abs()
                assert float((err - 2.0 ** -7 * one.float().abs()).max()) <= (2.0 ** -8 + 2.0 ** -12) * top
