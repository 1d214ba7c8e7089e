"""The paged key/value cache on the GPU: rows written (bit for bit the oracle's
codes, steps and copies, and nothing else of the pages touched) and read back."""
import numpy as np
import pytest
import torch

import oracle.kvcache as OK
import ternary_weight_bitlinear_b200 as B
from gpu_util import bf16_dev, bf16_host, f32_of_bf16
from kv_util import Paged, bf16_values, bits, padded_batch

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _device_status_clean():
    yield
    assert B.bitlinear_device_status() == 0


def same(a, b):
    """Equal bit for bit, any NaN being like another."""
    return np.array_equal(np.asarray(a), np.asarray(b), equal_nan=np.asarray(a).dtype.kind == "f")


def rows_of(p, seed, std=1.0, fused=False):
    """k, v rows as float32 values and as device tensors (slices of one wider tensor when `fused`)."""
    rng = np.random.default_rng(seed)
    k, v = bf16_values(rng, (p.T, p.Hkv, p.d), std), bf16_values(rng, (p.T, p.Hkv, p.d), std)
    return k, v, *upload(p, k, v, fused)


def upload(p, k, v, fused=False):
    if not fused:
        return p.guard.copy(bf16_dev(bits(k))), p.guard.copy(bf16_dev(bits(v)))
    w = torch.full((p.T, 3 + 2 * p.Hkv, p.d), float("nan"), dtype=torch.bfloat16, device="cuda")
    kd, vd = w[:, 3:3 + p.Hkv], w[:, 3 + p.Hkv:]
    kd.copy_(bf16_dev(bits(k)))
    vd.copy_(bf16_dev(bits(v)))
    return kd, vd


def expect_write(p, k, v):
    kc, vc, ks, vs = p.kc.copy(), p.vc.copy(), None if p.ks is None else p.ks.copy(), None if p.vs is None else p.vs.copy()
    for r, _, _, page, slot in OK.places(p.cu, p.lens, p.pages, p.page):
        if p.i8:
            kc[page, slot], ks[page, slot] = OK.quantise(k[r])
            vc[page, slot], vs[page, slot] = OK.quantise(v[r])
        else:
            kc[page, slot], vc[page, slot] = k[r], v[r]
    return [kc, vc] + ([ks, vs] if p.i8 else [])


CASES = [  # new rows, positions, page, heads, d
    ([1], [1], 16, 1, 64),
    ([1], [2048], 64, 5, 128),
    ([1] * 9, [1, 16, 17, 31, 32, 33, 64, 5, 48], 16, 5, 128),
    ([5, 0, 3, 1, 0], [5, 7, 130, 1, 0], 32, 3, 64),      # no rows; no rows and no positions
    ([40, 4], [3, 2], 16, 2, 128),                         # more rows than positions: the first have no place
    ([333, 1, 70], [400, 1, 70], 48, 5, 128),
    ([0, 0, 0, 2], [0, 0, 0, 300], 256, 8, 64),
    ([1] * 70, list(range(1, 71)), 16, 1, 128),             # more sequences than a warp looks at at once
]


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_write_then_read(case, fmt, guard):
    new, lens, page, heads, d = CASES[case]
    p = Paged(guard, new, lens, page, heads, d, fmt, seed=case, pad=7, order="heads" if case % 2 else "slots",
              poison=False)
    k, v, kd, vd = rows_of(p, seed=100 + case, fused=case % 3 == 0)
    B.bitlinear_kv_write(kd, vd, p.cache, p.batch)
    want = expect_write(p, k, v)
    for got, w, what in zip(p.device_pages(), want, ("k", "v", "k steps", "v steps")):
        assert same(got, w), what
    old = bf16_values(np.random.default_rng(5), (2, p.T, heads, d))
    ko, vo = guard.copy(bf16_dev(bits(old[0]))), guard.copy(bf16_dev(bits(old[1])))
    B.bitlinear_kv_read(p.cache, p.batch, k=ko, v=vo)
    for got, o, pages, steps in ((ko, old[0], want[0], want[2:3]), (vo, old[1], want[1], want[3:4])):
        ref = o.copy()
        for r, _, _, page_, slot in OK.places(p.cu, p.lens, p.pages, p.page):
            x = OK.dequantise(pages[page_, slot], steps[0][page_, slot]) if p.i8 else pages[page_, slot]
            ref[r] = torch.from_numpy(x).to(torch.bfloat16).float().numpy()
        assert same(f32_of_bf16(bf16_host(got)), ref)


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
@pytest.mark.parametrize("heads,d", [(1, 64), (2, 128)])
@pytest.mark.parametrize("count,most", [(33, 3), (1100, 2), (1025, 40)])
def test_many_sequences(count, most, heads, d, fmt, guard):
    """More sequences than are looked at at once, with runs of empty ones; the last has rows for several a group."""
    new, lens = padded_batch(count, most, 50, seed=count + d)
    p = Paged(guard, new, lens, 16, heads, d, fmt, seed=count, pad=9, poison=False)
    k, v, kd, vd = rows_of(p, seed=count + 1)
    B.bitlinear_kv_write(kd, vd, p.cache, p.batch)
    want = expect_write(p, k, v)
    for got, w, what in zip(p.device_pages(), want, ("k", "v", "k steps", "v steps")):
        assert same(got, w), what
    used = int(p.cu[-1])
    ko, vo = B.bitlinear_kv_read(p.cache, p.batch, T=p.T)
    at = np.array([(page, slot) for _, _, _, page, slot in OK.places(p.cu, p.lens, p.pages, p.page)]).T
    for got, x, steps in ((ko, want[0], want[2:3]), (vo, want[1], want[3:4])):
        x = x[at[0], at[1]]
        x = OK.dequantise(x, steps[0][at[0], at[1]]) if p.i8 else x
        got = f32_of_bf16(bf16_host(got))
        assert same(got[:used], torch.from_numpy(x).to(torch.bfloat16).float().numpy()) and not got[used:].any()


def test_codes_are_the_activation_quantisers(guard):
    p = Paged(guard, [33], [33], 16, 5, 128, "int8", seed=3)
    k, v, kd, vd = rows_of(p, seed=4, std=5.0)
    B.bitlinear_kv_write(kd, vd, p.cache, p.batch)
    q, s_x, _ = B.bitlinear_act_quant(kd.reshape(-1, 128).contiguous())
    kc, _, ks, _ = p.device_pages()
    pos = np.arange(33)
    at = p.pages[0][pos // 16], pos % 16
    assert same(kc[at].reshape(-1, 128), q.cpu().numpy())
    assert same(ks[at].reshape(-1), (np.float32(1) / s_x.cpu().numpy()).astype(np.float32))


@pytest.mark.parametrize("d", [64, 128])
def test_int8_extreme_rows(d, guard):
    """Zero rows, rows below the scale's floor, the largest and smallest finite values, ties, infinities and NaN."""
    top = 2.0 ** 127 * (2 - 2.0 ** -7)
    rows = np.zeros((9, 1, d), np.float32)
    rows[1] = 2.0 ** -133
    rows[2] = 1e-7 * np.float32(2.0 ** -3)
    rows[3, 0, ::2], rows[3, 0, 1::2] = top, -top
    rows[4, 0, 0], rows[4, 0, 1:] = 127.0, np.arange(1, d) - 32.5  # s = 1: codes are ties to even
    rows[5], rows[5, 0, d - 1] = 1.0, np.inf
    rows[6], rows[6, 0, 0] = 1.0, np.nan
    rows[7], rows[7, 0, 9] = 1.0, -np.inf
    rows[8, 0, 3] = -2.0
    rows = f32_of_bf16(bits(rows))
    p = Paged(guard, [9], [9], 16, 1, d, "int8", seed=8, poison=False)
    kd, vd = upload(p, rows, rows[::-1].copy())
    B.bitlinear_kv_write(kd, vd, p.cache, p.batch)
    want = expect_write(p, rows, rows[::-1])
    for got, w in zip(p.device_pages(), want):
        assert same(got, w)
    k, v = B.bitlinear_kv_read(p.cache, p.batch, T=p.T)
    k = f32_of_bf16(bf16_host(k))
    assert np.isnan(k[[5, 6, 7]]).all() and np.isfinite(k[[0, 1, 2, 3, 4, 8]]).all() and (k[0] == 0).all()
    assert (k[3, 0, ::2] == top).all()


def test_read_in_new_tensors_leaves_zeros_behind(guard):
    p = Paged(guard, [3, 2], [3, 20], 16, 2, 64, "bf16", seed=9, pad=4)
    k, v = B.bitlinear_kv_read(p.cache, p.batch, T=p.T)
    assert (k[5:] == 0).all() and (v[5:] == 0).all()
    assert same(f32_of_bf16(bf16_host(k))[3:5], p.sequence(1)[0][18:])


def test_page_outside_the_cache_is_recorded_and_skipped(guard):
    for fmt in ("bf16", "int8"):
        p = Paged(guard, [20, 3], [20, 3], 16, 2, 64, fmt, seed=10, poison=False)
        for bad in (-1, p.kc.shape[0], 2 ** 31 - 1, -2 ** 31):
            p.pages[0, 1] = bad
            p.batch.held[2].copy_(torch.from_numpy(p.pages))
            k, v, kd, vd = rows_of(p, seed=11)
            before = p.device_pages()
            B.bitlinear_kv_write(kd, vd, p.cache, p.batch)
            assert B.bitlinear_device_status() == 9 and B.bitlinear_device_status() == 0
            after = p.device_pages()
            touched = {(pg, s) for r, b, pos, pg, s in OK.places(p.cu, p.lens, p.pages, 16) if pg != bad}
            for x, y in zip(before[:2], after[:2]):
                moved = (x.view(np.uint8) != y.view(np.uint8)).reshape(*x.shape[:2], -1).any(-1)
                assert {(a, b) for a, b in zip(*np.nonzero(moved))} <= touched
                assert moved.any() or bad != -1  # the later calls write the same rows again
            B.bitlinear_kv_read(p.cache, p.batch, T=p.T)
            assert B.bitlinear_device_status() == 9


def test_arrays_that_lie_stay_inside_the_buffers(guard):
    """Starts outside the rows, lengths outside the table: cut, whatever is written stays in the cache."""
    p = Paged(guard, [4, 4], [20, 20], 16, 2, 64, "int8", seed=12, poison=False, spare=6)
    for cu, lens in (([-5, 3, 900], [20, 20]), ([0, 4, 8], [2 ** 31 - 1, -7]), ([8, 4, 0], [20, 20]),
                     ([2 ** 31 - 1, -2 ** 31, 5], [20, 20])):
        p.batch.held[0].copy_(torch.tensor(cu, dtype=torch.int32))
        p.batch.held[1].copy_(torch.tensor(lens, dtype=torch.int32))
        k, v, kd, vd = rows_of(p, seed=13)
        B.bitlinear_kv_write(kd, vd, p.cache, p.batch)
        B.bitlinear_kv_read(p.cache, p.batch, T=p.T)
    B.bitlinear_device_status()  # whether a page was missed depends on the table: not the point here


def test_write_on_another_stream_and_in_a_graph(guard):
    p = Paged(guard, [2, 1], [40, 17], 16, 5, 128, "int8", seed=14, poison=False)
    k, v, kd, vd = rows_of(p, seed=15)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    B.bitlinear_kv_write(kd, vd, p.cache, p.batch, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    first = p.device_pages()
    assert all(same(a, b) for a, b in zip(first, expect_write(p, k, v)))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.bitlinear_kv_write(kd, vd, p.cache, p.batch)
    # the captured call reads the lengths and rows of the moment of its replay
    p.kc, p.vc, p.ks, p.vs = first
    p.lens = [39, 9]
    p.batch.held[1].copy_(torch.tensor(p.lens, dtype=torch.int32))
    k2, v2, kd2, vd2 = rows_of(p, seed=16)
    kd.copy_(kd2)
    vd.copy_(vd2)
    g.replay()
    torch.cuda.synchronize()
    assert all(same(a, b) for a, b in zip(p.device_pages(), expect_write(p, k2, v2)))


def test_cache_past_two_gi_elements(guard):
    """Offsets beyond 31 bits: rows at the far end of a 2.2-GiB int8 cache."""
    heads, d, page = 8, 128, 256
    num = (2 ** 31 + 2 ** 27) // (heads * d * page)
    kp = torch.zeros((num, page, heads, d), dtype=torch.int8, device="cuda")
    vp = torch.zeros_like(kp)
    ks, vs = (torch.zeros((num, heads, page), device="cuda") for _ in range(2))
    cache = B.make_kv_cache(kp, vp, ks, vs)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    batch = B.make_kv_batch(i32([0, 3]), i32([300]), i32([[0, num - 1]]))
    x = bf16_values(np.random.default_rng(17), (3, heads, d))
    xd = bf16_dev(bits(x))
    B.bitlinear_kv_write(xd, -xd, cache, batch)
    code, step = OK.quantise(x)
    assert same(kp[num - 1, 41:44].cpu().numpy(), code) and same(ks[num - 1, :, 41:44].T.cpu().numpy(), step)
    assert int((kp != 0).sum()) == int((code != 0).sum())
    k, _ = B.bitlinear_kv_read(cache, batch, T=3)
    assert same(f32_of_bf16(bf16_host(k)), torch.from_numpy(OK.dequantise(code, step)).to(torch.bfloat16).float().numpy())


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
def test_rows_read_into_each_other_are_refused(fmt, guard):
    """k and v into one tensor: refused where they share elements, right where they take turns within its rows."""
    p = Paged(guard, [3, 2], [20, 2], 16, 2, 64, fmt, seed=18)
    w = guard.empty((7, 6, 64), torch.bfloat16, fill=0)
    one = w[:5, :2]
    for k, v in ((one, one), (w[:5, :2], w[:5, 1:3]), (w[:5, 2:4], w[1:6, 2:4]), (w[1:6, 1:3], w[:5, 2:4]),
                 (w[:5, 4:], w[1:6, 3:5])):
        with pytest.raises(B.BitLinearError) as e:
            B.bitlinear_kv_read(p.cache, p.batch, k=k, v=v)
        assert e.value.status == 2
    assert not w.any()
    want = [x.clone() for x in B.bitlinear_kv_read(p.cache, p.batch, T=p.T)]
    for k, v in ((w[:5, :2], w[:5, 2:4]), (w[:5, 4:], w[1:6, :2]), (w[2:, 2:4], w[:5, 4:])):
        B.bitlinear_kv_read(p.cache, p.batch, k=k, v=v)
        assert torch.equal(k, want[0]) and torch.equal(v, want[1])
