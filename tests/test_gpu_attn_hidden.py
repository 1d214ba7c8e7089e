"""Attention over the paged cache where positions that only some rows see hold
infinities and NaN among their values: every row gets the result of what it sees,
whatever the rest holds, however much of it there is and however long the cache."""
import numpy as np
import pytest
import torch

import oracle.kvcache as OK
import ternary_weight_bitlinear_b200 as B
from gpu_util import bf16_dev, bf16_host, f32_of_bf16
from kv_util import Paged, attention_error_bound, bf16_values, bits

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _device_status_clean():
    yield
    assert B.bitlinear_device_status() == 0


def spoil(p, share, seed):
    """NaN and infinities of both signs in a few dimensions of a share of each sequence's new positions, the last
    one always."""
    rng = np.random.default_rng(seed)
    for b, (n, L) in enumerate(zip(p.new, p.lens)):
        for pos in range(max(L - n, 0), L):
            if pos == L - 1 or rng.random() < share:
                at = p.pages[b][pos // p.page], pos % p.page
                dims = rng.integers(0, p.d, 3)
                p.vc[at][:, dims] = rng.choice([np.nan, np.inf, -np.inf], 3).astype(np.float32)
    p.upload()


# new rows, positions, heads of a group, head size; up to 16 rows of a head a sequence
FEW = [([4], [40], 4, 64), ([16], [300], 1, 128), ([5], [37], 3, 64), ([2, 2], [33, 1500], 8, 128), ([8], [8], 2, 64),
       ([4, 0, 3], [5000, 3, 64], 4, 128), ([2], [2], 7, 128), ([2], [100], 4, 128), ([8], [20], 1, 64)]
# more
MANY = [([64], [64], 4, 64), ([200], [333], 1, 128), ([70], [900], 12, 64), ([33], [33], 7, 128), ([300, 5], [300, 2000], 4, 128),
        ([20, 0, 90], [3, 9, 1500], 2, 64), ([130], [130], 1, 64), ([1, 70], [5000, 3000], 16, 128), ([2], [700], 100, 64)]


@pytest.mark.parametrize("share", [0.1, 1.0])
@pytest.mark.parametrize("new,lens,group,d", FEW + MANY)
def test_non_finite_values_among_the_new_rows(new, lens, group, d, share, guard):
    p = Paged(guard, new, lens, 16, 2, d, "bf16", seed=sum(lens) + d)
    spoil(p, share, seed=group)
    H = 2 * group
    q = bf16_values(np.random.default_rng(d), (p.T, H, d))
    out = guard.empty((p.T, H, d), torch.bfloat16, fill=0)
    scale = np.float32(d ** -0.5)
    ws = guard.workspace(max(16, B.bitlinear_attn_paged_workspace_size(p.T, H, 2, d)))
    B.bitlinear_attn_paged(bf16_dev(bits(q)), p.cache, p.batch, float(scale), out=out, workspace=ws)
    got = f32_of_bf16(bf16_host(out))
    s = [p.sequence(b) for b in range(len(new))]
    with np.errstate(invalid="ignore"):
        want, absv, mag, seen = OK.attention(q, [x[0] for x in s], [x[1] for x in s], p.cu, p.lens, scale, True,
                                             np.zeros_like(q))
    ok = np.isfinite(want)
    assert ok[:, :, 0].any() and not ok.all()
    assert np.array_equal(got[~ok], want[~ok].astype(np.float32), equal_nan=True)
    bound = attention_error_bound(np.where(ok, want, 0), np.where(ok, absv, 0), mag, seen, d)
    assert (np.abs(got - np.where(ok, want, 0))[ok] <= bound[ok]).all()


LONG = [(2, 8, 2 ** 21, 128), (16, 8, 2 ** 18, 64), (16, 8, 2 ** 18, 128)]


@pytest.mark.parametrize("n,group,L,d", LONG)
def test_a_hidden_nan_costs_no_wait_its_limit(n, group, L, d):
    """160 long sequences over the same few pages, the last position NaN among its values: the rows before it are
    computed as without it, and all of them.  (Computing such a row again over a part of the positions while the
    rest of its block waits takes seconds here.)"""
    S, page = 160, 256
    rng = np.random.default_rng(L)
    k, v = (bf16_dev(bits(bf16_values(rng, (17, page, 1, d)))) for _ in range(2))
    cols = L // page
    table = torch.arange(cols, dtype=torch.int32, device="cuda") % 16
    table[-1] = 16
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    batch = B.make_kv_batch(i32([n * b for b in range(S + 1)]), i32([L] * S), table.repeat(S, 1))
    q = bf16_dev(bits(bf16_values(rng, (S * n, group, d))))
    cache = B.make_kv_cache(k, v)
    clean = B.bitlinear_attn_paged(q, cache, batch, d ** -0.5).float().view(S, n, group, d)
    assert torch.isfinite(clean).all()
    v[16, page - 1, 0, 5] = float("nan")
    got = B.bitlinear_attn_paged(q, cache, batch, d ** -0.5).float().view(S, n, group, d)
    assert B.bitlinear_device_status() == 0
    assert torch.isnan(got[:, -1, :, 5]).all() and torch.isfinite(got[:, -1, :, 6]).all()
    # the same terms, those of 16 positions in another order: both results are bf16 roundings (2^-8 of the value each)
    # of sums that differ by at most 2 * 17 * 2^-23 of the largest value
    a, b = got[:, :-1], clean[:, :-1]
    assert ((a - b).abs() <= 2.0 ** -7 * b.abs() + 2.0 ** -17 * float(v[:16].float().abs().max())).all()
