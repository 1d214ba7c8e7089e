"""Argument checks of the paged-cache entry points, without a GPU: a refused
call returns its status before any device is looked at."""
import ctypes

import pytest
import torch

B = pytest.importorskip("ternary_weight_bitlinear_b200")

A = 0x10000  # 16-byte aligned, never dereferenced by host checks
NULL, SHAPE, ALIGN, DTYPE, WORKSPACE, DEVICE = 1, 2, 3, 4, 5, 8


def cache(**kw):
    f = dict(k=A, v=A, k_step=None, v_step=None, num_pages=8, page_size=16, kv_heads=5, head_dim=128,
             stride_page=16 * 640, stride_slot=640, stride_head=128, format=0)
    f.update(kw)
    return B.bitlinear.KvCache(**f)


def batch(**kw):
    f = dict(cu_q=A, kv_len=A, pages=A, batch=2, max_pages=4)
    f.update(kw)
    return B.bitlinear.KvBatch(**f)


BAD = [
    (dict(format=2), {}, DTYPE),
    (dict(format=-1), {}, DTYPE),
    (dict(head_dim=96), {}, SHAPE),
    (dict(head_dim=256), {}, SHAPE),
    (dict(num_pages=0), {}, SHAPE),
    (dict(num_pages=2 ** 31), {}, SHAPE),
    (dict(page_size=0), {}, SHAPE),
    (dict(page_size=24), {}, SHAPE),
    (dict(page_size=2 ** 21), {}, SHAPE),
    (dict(kv_heads=0), {}, SHAPE),
    (dict(kv_heads=65536), {}, SHAPE),
    (dict(stride_head=0), {}, SHAPE),
    (dict(stride_page=-640), {}, SHAPE),
    (dict(stride_slot=2 ** 40), {}, SHAPE),
    (dict(stride_slot=644), {}, ALIGN),
    (dict(k=None), {}, NULL),
    (dict(v=A + 2), {}, ALIGN),
    (dict(format=1), {}, NULL),                                     # int8 without steps
    (dict(format=1, k_step=A, v_step=A + 4), {}, ALIGN),
    (dict(format=1, k_step=A, v_step=A, stride_head=136), {}, ALIGN),  # 16 bytes are 16 codes
    ({}, dict(batch=-1), SHAPE),
    ({}, dict(batch=2 ** 31), SHAPE),
    ({}, dict(batch=2 ** 31 - 1), SHAPE),
    ({}, dict(max_pages=-1), SHAPE),
    ({}, dict(max_pages=2 ** 26 + 1), SHAPE),
    ({}, dict(cu_q=None), NULL),
    ({}, dict(kv_len=None), NULL),
    ({}, dict(pages=None), NULL),
]


def write(c, b, k=A, ks=640, v=A, vs=640, T=3, fn="bitlinear_kv_write"):
    return getattr(B.lib(), fn)(ctypes.byref(c), ctypes.byref(b), k, ks, v, vs, T, None)


def attend(c, b, q=A, qs=2560, T=3, heads=20, scale=0.1, causal=1, out=0x4000000, os=2560, ws=A, wsb=1 << 40):
    return B.lib().bitlinear_attn_paged(ctypes.byref(c), ctypes.byref(b), q, qs, T, heads, scale, causal, out, os, ws,
                                        wsb, None)


@pytest.mark.parametrize("c,b,status", BAD)
def test_cache_and_batch_are_checked(c, b, status):
    assert write(cache(**c), batch(**b)) == status
    assert write(cache(**c), batch(**b), fn="bitlinear_kv_read") == status
    if c.get("kv_heads") is None:
        assert attend(cache(**c), batch(**b)) == status


@pytest.mark.parametrize("fn", ["bitlinear_kv_write", "bitlinear_kv_read"])
def test_rows_are_checked(fn):
    c, b = cache(), batch()
    assert write(c, b, T=-1, fn=fn) == SHAPE
    assert write(c, b, T=2 ** 31, fn=fn) == SHAPE
    assert write(c, b, T=(2 ** 31 - 1024) // 5 + 1, fn=fn) == SHAPE  # more (row, head) pairs than 32 bits hold
    assert write(c, b, ks=632, fn=fn) == SHAPE          # rows that overlap
    assert write(c, b, vs=644, fn=fn) == ALIGN
    assert write(c, b, k=None, fn=fn) == NULL
    assert write(c, b, v=A + 8, fn=fn) == ALIGN
    assert write(c, b, T=0, k=None, v=None, fn=fn) == 0   # nothing to do
    assert write(c, batch(batch=0, cu_q=None, kv_len=None, pages=None), fn=fn) == 0
    assert getattr(B.lib(), fn)(None, ctypes.byref(b), A, 640, A, 640, 3, None) == NULL
    assert getattr(B.lib(), fn)(ctypes.byref(c), None, A, 640, A, 640, 3, None) == NULL


def test_attention_is_checked():
    c, b = cache(), batch()
    assert attend(c, b, T=-1) == SHAPE
    assert attend(c, b, heads=18) == SHAPE               # not a multiple of the key/value heads
    assert attend(c, b, heads=5 * 129, qs=5 * 129 * 128, os=5 * 129 * 128) == SHAPE
    assert attend(c, b, heads=0) == SHAPE
    assert attend(c, b, T=2 ** 27) == SHAPE              # T * heads past INT32_MAX
    for scale in (0.0, -1.0, float("inf"), float("nan"), 3e38):
        assert attend(c, b, scale=scale) == SHAPE
    assert attend(c, b, qs=2552) == SHAPE
    assert attend(c, b, os=2564) == ALIGN
    assert attend(c, b, q=None) == NULL
    assert attend(c, b, out=A + 2) == ALIGN
    for out in (A, A + 2 * 2560 * 2, A - 2 * 2544):      # q's rows, one of them, the end of one
        assert attend(c, b, out=out) == SHAPE
    assert attend(c, b, qs=5120, os=5120, out=A + 2 * 2552) == SHAPE
    assert attend(c, b, qs=2560, os=5120, out=A + 2 * 5120) == SHAPE
    for out in (A + 3 * 2 * 2560, A - 3 * 2 * 2560):     # behind it, before it
        assert attend(c, b, out=out, ws=None) in (WORKSPACE, DEVICE)
    for out in (A + 2 * 2560, A - 2 * 2560, A + 2 * 7680):  # in turns within rows of 5120
        assert attend(c, b, qs=5120, os=5120, out=out, ws=None) in (WORKSPACE, DEVICE)
    assert attend(c, b, T=0, q=None, out=None, ws=None, wsb=0) == 0
    n = ctypes.c_size_t()
    assert B.lib().bitlinear_attn_paged_workspace_size(3, 20, 5, 128, None) == NULL
    assert B.lib().bitlinear_attn_paged_workspace_size(3, 20, 5, 80, ctypes.byref(n)) == SHAPE
    assert B.lib().bitlinear_attn_paged_workspace_size(-1, 20, 5, 128, ctypes.byref(n)) == SHAPE
    assert B.lib().bitlinear_attn_paged_workspace_size(3, 20, 0, 128, ctypes.byref(n)) == SHAPE


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device path")
def test_no_device_is_reported():
    assert write(cache(), batch()) == DEVICE
    assert write(cache(), batch(), fn="bitlinear_kv_read") == DEVICE
    assert attend(cache(), batch()) == DEVICE


def test_binding_refuses_other_tensors():
    x = torch.zeros((4, 16, 5, 128), dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        B.make_kv_cache(x, x)  # not on a GPU
    with pytest.raises(TypeError):
        B.make_kv_batch(*(torch.zeros(s, dtype=torch.int32) for s in (3, 2, (2, 4))))
    with pytest.raises(TypeError):
        B.bitlinear_kv_write(x[0], x[0], cache(), batch())
    with pytest.raises(TypeError):
        B.bitlinear_attn_paged(x[0], cache(), batch(), 0.1)
    with pytest.raises(TypeError):
        B.bitlinear_kv_read(cache(), batch())
    assert B.status_string(9) and "unknown" not in B.status_string(9)


@pytest.mark.gpu
def test_binding_refuses_mismatched_tensors():
    dev = "cuda"
    x = torch.zeros((4, 16, 5, 128), dtype=torch.bfloat16, device=dev)
    i8, steps = x.to(torch.int8), torch.zeros((4, 5, 16), device=dev)
    for args in ((x, x[:2]), (x, x.float()), (x, i8), (x, x.transpose(1, 2)), (x[..., ::2], x[..., ::2]), (x, x, steps, steps),
                 (i8, i8), (i8, i8, steps, steps[:2]), (i8, i8, steps, steps.transpose(1, 2)), (x[0], x[0])):
        with pytest.raises(TypeError):
            B.make_kv_cache(*args)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device=dev)  # noqa: E731
    for args in ((i32(3), i32(3), i32(2, 4)), (i32(2), i32(2), i32(2, 4)), (i32(3), i32(2), i32(2, 4).t()),
                 (i32(3).long(), i32(2), i32(2, 4))):
        with pytest.raises(TypeError):
            B.make_kv_batch(*args)
    c, b = B.make_kv_cache(x, x.clone()), B.make_kv_batch(i32(3), i32(2), i32(2, 4))
    r = torch.zeros((6, 5, 128), dtype=torch.bfloat16, device=dev)
    for k, v in ((r, r[:5]), (r[:, :4], r[:, :4]), (r.float(), r), (r.transpose(0, 1), r), (r[..., ::2], r)):
        with pytest.raises(TypeError):
            B.bitlinear_kv_write(k, v, c, b)
    q = torch.zeros((6, 20, 128), dtype=torch.bfloat16, device=dev)
    with pytest.raises(TypeError):
        B.bitlinear_attn_paged(q, c, b, 0.1, out=q[:5].clone())
    with pytest.raises(B.BitLinearError):
        B.bitlinear_attn_paged(q[:, :18], c, b, 0.1, out=q[:, :18].clone())
    need = B.bitlinear_attn_paged_workspace_size(6, 20, 5, 128)
    if need > 16:
        with pytest.raises(B.BitLinearError):
            B.bitlinear_attn_paged(q, c, b, 0.1, workspace=torch.empty(16, dtype=torch.uint8, device=dev))
