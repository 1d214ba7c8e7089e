"""Attention over the paged cache on batches so large that the work, in units of
position tiles, passes 2^22: from there on shares are cut in 64-bit arithmetic."""
import numpy as np
import pytest
import torch

import ternary_weight_bitlinear_b200 as B

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _device_status_clean():
    yield
    assert B.bitlinear_device_status() == 0


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def check(got, q, k, v, see, scale):
    """Rows got, q [r, H, d] against float64 over k, v [L, H_kv, d]; see [r] positions of each row.  The bound is
    kv_util.attention_error_bound's."""
    r, H, d = q.shape
    G = H // k.shape[1]
    q = q.double().view(r, -1, G, d)
    k, v = k.double(), v.double()
    s = torch.einsum("rhgd,lhd->rhgl", q, k) * scale
    hidden = torch.arange(k.shape[0], device="cuda")[None, :] >= see[:, None]
    p = torch.softmax(s.masked_fill(hidden[:, None, None], -torch.inf), -1)
    want = torch.einsum("rhgl,lhd->rhgd", p, v)
    absv = torch.einsum("rhgl,lhd->rhgd", p, v.abs())
    mag = scale * q.abs().sum(-1) * k.abs().amax()  # at least the largest sum |q_i k_i|
    rel = 2.0 ** -8 + 2.0 ** -20 + see[:, None, None] * 2.0 ** -22 + 4 * (d + 8) * 2.0 ** -23 * mag
    err = (got.double().view_as(want) - want).abs()
    assert (err <= 2.0 ** -8 * want.abs() + rel[..., None] * absv).all()


def test_many_heads_and_sequences():
    """700 sequences of 33 to 96 positions (two or three chunks of 32, and four units an item beside them), 1024 heads:
    4.6 Mi units of the few-rows kernel, most shares ending inside an item."""
    rng = np.random.default_rng(1)
    S, H, d, page, pages = 700, 1024, 64, 16, 10
    k, v = (torch.randn((pages, page, H, d), device="cuda").to(torch.bfloat16) for _ in range(2))
    lens = rng.integers(33, 97, S)
    assert H * int((4 + (lens + 31) // 32).sum()) > 2 ** 22
    table = torch.from_numpy(rng.integers(0, pages, (S, 6)).astype(np.int32)).cuda()
    q = torch.randn((S, H, d), device="cuda").to(torch.bfloat16)
    batch = B.make_kv_batch(i32(list(range(S + 1))), i32(lens.tolist()), table)
    out = B.bitlinear_attn_paged(q, B.make_kv_cache(k, v), batch, d ** -0.5)
    for b in range(S):
        n = int(lens[b])
        at = table[b].long()
        check(out[b:b + 1], q[b:b + 1], k[at].flatten(0, 1)[:n], v[at].flatten(0, 1)[:n], i32([n]), d ** -0.5)


def test_a_very_long_prompt():
    """66,000 new tokens, 32 heads over 4: items of 32 tokens, one unit and two a tile of 128 positions each, so
    4.3 Mi units of the many-rows kernel.  One token of every item is checked."""
    rng = np.random.default_rng(2)
    n, H, Hkv, d, page = 66000, 32, 4, 64, 64
    pages = -(-n // page)
    k, v = (torch.randn((pages, page, Hkv, d), device="cuda").to(torch.bfloat16) for _ in range(2))
    ends = np.minimum(np.arange(32, n + 32, 32), n)
    assert Hkv * int((1 + 2 * ((ends + 127) // 128)).sum()) > 2 ** 22
    q = torch.randn((n, H, d), device="cuda").to(torch.bfloat16)
    order = torch.randperm(pages, device="cuda").to(torch.int32)
    batch = B.make_kv_batch(i32([0, n]), i32([n]), order[None])
    out = B.bitlinear_attn_paged(q, B.make_kv_cache(k, v), batch, d ** -0.5)
    ks, vs = (x[order.long()].flatten(0, 1)[:n] for x in (k, v))
    rows = torch.from_numpy(np.minimum(np.arange(0, n, 32) + rng.integers(0, 32, len(ends)), n - 1)).cuda()
    for r in rows.split(32):
        check(out[r], q[r], ks[:int(r.max()) + 1], vs[:int(r.max()) + 1], r + 1, d ** -0.5)
