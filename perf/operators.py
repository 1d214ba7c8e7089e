"""The paged key/value cache and the attention that reads it, in plain form and through the library.

Three operators share one description of a batch -- cu_q (where each sequence's new rows start), kv_len
(positions of each sequence, its new ones included) and a page table:

  write      the new rows' keys and values into the pages: as they are (bf16), or quantised per row (int8);
  read       those rows back out of the pages, as bf16;
  attention  of the new rows over all positions of their sequence in the pages.

Row i of the n new rows of a sequence with L positions stands at position L - n + i.

int8 rows (head_dim values of one key/value head of one token): a = max |x|, s = RN32(127 / max(a, 1e-5)),
code = clamp(rint(RN32(x s)), -128, 127), step = RN32(1 / s); a code stands for RN32(code step).
"""
import math

import torch

own = False

SCALE_FLOOR = 1e-5

# (query heads, key/value heads, head dimension): the decoder's own, and the groupings that the tests run
HEADS = [(20, 5, 128), (8, 8, 64), (16, 2, 128), (4, 2, 64), (8, 1, 128)]


def _case(name, op, heads, batch, new, past, page, fmt, causal=True, pad=0, even=False):
    H, Hkv, d = heads
    c = {"op": op, "heads": H, "kv_heads": Hkv, "dim": d, "batch": batch, "new": new, "past": past, "page": page,
         "format": fmt, "causal": causal, "pad": pad, "even": even}
    return c if name is None else dict(c, name=name)


def listed():
    D = HEADS[0]
    return [
        # one decode step of a batch: a token of each sequence appended, and what the cache now holds for it
        _case("append_64_int8", "write", D, 64, 1, 1900, 64, "int8"),
        # prompts entering a quantised cache, ragged
        _case("prompts_write_int8", "write", D, 8, 2048, 0, 64, "int8"),
        # long prompts entering an unquantised cache from slices of one fused projection, 64-wide heads
        _case("prompts_write_bf16", "write", HEADS[1], 6, 7001, 500, 16, "bf16"),
        # a short sequence read back (odd length, pages of 16)
        _case("read_short_bf16", "read", D, 1, 333, 0, 16, "bf16", even=True),
        # sequences taken out of a quantised cache (moved elsewhere, or shared as a prefix)
        _case("read_long_int8", "read", D, 4, 16000, 0, 128, "int8"),
        # one user's decode step at the model's longest context: latency
        _case("decode_1_bf16", "attention", D, 1, 1, 2047, 64, "bf16", even=True),
        # a serving batch's decode step over a quantised cache, lengths mixed
        _case("decode_64_int8", "attention", D, 64, 1, 6000, 64, "int8"),
        # one token over a very long document
        _case("decode_long_bf16", "attention", HEADS[4], 2, 1, 150000, 128, "bf16"),
        # a few drafted tokens of each sequence checked in one pass, 64-wide heads without grouping
        _case("drafts_16x5_bf16", "attention", HEADS[1], 16, 5, 1800, 16, "bf16"),
        # chunks of long prompts beside short ones, over a quantised cache, the batch padded
        _case("chunks_6_int8", "attention", D, 6, 600, 9000, 64, "int8", pad=37),
        # one whole prompt
        _case("prompt_8192_bf16", "attention", D, 1, 8192, 0, 64, "bf16", even=True),
        # documents embedded: every position sees every other, odd lengths
        _case("documents_bf16", "attention", HEADS[2], 5, 1777, 0, 32, "bf16", causal=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    heads = rng.choice(HEADS)
    page = rng.choice([16, 32, 48, 64, 128, 256])
    fmt = rng.choice(["bf16", "int8"])
    op = rng.choice(["write", "read", "attention", "attention", "attention"])
    causal = True
    pad = rng.choice([0, 0, rng.randint(1, 100)])
    if op != "attention":
        batch = _log_int(rng, 1, 64)
        new = _log_int(rng, 1, 40000 / batch)
        return _case(None, op, heads, batch, new, rng.randint(0, 500), page, fmt, pad=pad)
    kind = rng.choice(["decode", "drafts", "chunks", "prompt"])
    if kind == "decode":
        batch = _log_int(rng, 1, 64)
        new, past = 1, _log_int(rng, 1, 300000 / batch)
    elif kind == "drafts":
        batch = _log_int(rng, 1, 32)
        new, past = rng.randint(2, 16), _log_int(rng, 1, 100000 / batch)
    elif kind == "chunks":
        batch = rng.randint(1, 8)
        new, past = _log_int(rng, 17, 4096 / batch), _log_int(rng, 1, 40000 / batch)
    else:
        batch = rng.randint(1, 4)
        new, past = _log_int(rng, 64, 8192 / batch), 0
        causal = rng.random() < 0.75
    return _case(None, op, heads, batch, new, past, page, fmt, causal=causal, pad=pad, even=rng.random() < 0.3)


def _lengths(case):
    """New rows and positions of each sequence: the case's own where even, else spread over a quarter to the whole of them."""
    B, even = case["batch"], case["even"]
    part = [1.0 if even else 1.0 - 0.75 * ((0.618034 * b) % 1.0) for b in range(B)]
    back = [1.0 if even else 1.0 - 0.75 * ((0.754878 * b) % 1.0) for b in range(B)]
    n = [max(1, round(case["new"] * p)) for p in part]
    return n, [a + round(case["past"] * p) for a, p in zip(n, back)]


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _rows(g, *shape):
    """Rows as projections give them: normal, each head's rows of their own size, a few wide channels."""
    x = _randn(g, *shape)
    size = torch.exp(0.4 * _randn(g, *shape[:-1], 1))
    wide = 1.0 + 3.0 * (torch.rand(shape[-1], generator=g, device="cuda") < 0.04)
    return (x * size * wide).to(torch.bfloat16)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    B, P, H, Hkv, d = case["batch"], case["page"], case["heads"], case["kv_heads"], case["dim"]
    n, L = _lengths(case)
    per = [-(-x // P) for x in L]
    cols, total, T = max(per), sum(per), sum(n) + case["pad"]
    num_pages = total + 3
    order = torch.randperm(num_pages, generator=g, device="cuda")[:total].to(torch.int32)
    first = torch.tensor([sum(per[:b]) for b in range(B)], device="cuda")
    col = torch.arange(cols, device="cuda")
    live = col[None, :] < torch.tensor(per, device="cuda")[:, None]
    pages = torch.where(live, order[(first[:, None] + col[None, :]).clamp(max=total - 1)], -1).to(torch.int32)
    cu = [sum(n[:b]) for b in range(B + 1)]
    s = {"case": case, "cu_q": torch.tensor(cu, dtype=torch.int32, device="cuda"),
         "kv_len": torch.tensor(L, dtype=torch.int32, device="cuda"), "pages": pages.contiguous(),
         "longest_new": max(n), "longest": max(L), "k_step": None, "v_step": None}
    shape = (num_pages, P, Hkv, d)
    if case["format"] == "int8":
        s["k_pages"], s["k_step"] = _quantise(_rows(g, *shape))
        s["v_pages"], s["v_step"] = _quantise(_rows(g, *shape))
        s["k_step"], s["v_step"] = (x.transpose(1, 2).contiguous() for x in (s["k_step"], s["v_step"]))
    else:
        s["k_pages"], s["v_pages"] = _rows(g, *shape), _rows(g, *shape)
    if case["op"] == "write":
        fused = _rows(g, T, H + 2 * Hkv, d)  # q | k | v of one fused projection: k and v are slices of it
        s["k"], s["v"] = fused[:, H:H + Hkv], fused[:, H + Hkv:]
    if case["op"] == "attention":
        s["q"] = _rows(g, T, H, d)
        s["scale"] = d ** -0.5
        s["out"] = _randn(g, T, H, d).to(torch.bfloat16)
    if case["op"] == "read" or case["op"] == "write" and case["format"] == "int8":
        s["k_out"], s["v_out"] = (_randn(g, T, Hkv, d).to(torch.bfloat16) for _ in range(2))
    return s


# ---- the plain form ------------------------------------------------------------------------------------------------------------
def _quantise(x):
    """bf16 rows [..., d] -> (int8 codes, fp32 steps [...])."""
    x = x.float()
    s = 127.0 / x.abs().amax(-1, keepdim=True).clamp(min=SCALE_FLOOR)
    return (x * s).round().clamp(-128, 127).to(torch.int8), (1.0 / s)[..., 0]


def _where(state, T, P):
    """Of each of T rows: its page and its place there, and whether any sequence has it."""
    row = torch.arange(T, device="cuda", dtype=torch.int32)
    cu = state["cu_q"]
    live = row < cu[-1]
    b = (torch.searchsorted(cu, row, right=True) - 1).clamp(max=cu.numel() - 2)
    pos = (state["kv_len"][b] - (cu[b + 1] - row)).clamp(min=0)
    return state["pages"][b, (pos // P).long()].long(), (pos % P).long(), live


def _plain_write(state):
    P = state["case"]["page"]
    page, slot, live = _where(state, state["k"].shape[0], P)
    # rows that no sequence has go where the last one that some sequence has goes, with its values
    keep = torch.minimum(torch.arange(live.numel(), device="cuda"), state["cu_q"][-1].long() - 1)
    page, slot = page[keep], slot[keep]
    k, v = state["k"][keep], state["v"][keep]
    if state["k_step"] is None:
        state["k_pages"][page, slot] = k
        state["v_pages"][page, slot] = v
        return
    (k, ks), (v, vs) = _quantise(k), _quantise(v)
    state["k_pages"][page, slot] = k
    state["v_pages"][page, slot] = v
    state["k_step"][page, :, slot] = ks
    state["v_step"][page, :, slot] = vs


def _values(pages, step, page, slot):
    x = pages[page, slot].float()
    return x if step is None else x * step[page, :, slot][..., None]


def _plain_read(state):
    page, slot, live = _where(state, state["k_out"].shape[0], state["case"]["page"])
    page, m = page.clamp(min=0), live[:, None, None]
    k = _values(state["k_pages"], state["k_step"], page, slot).to(torch.bfloat16)
    v = _values(state["v_pages"], state["v_step"], page, slot).to(torch.bfloat16)
    return torch.where(m, k, state["k_out"]), torch.where(m, v, state["v_out"])


def _plain_attention(state):
    c, q, cu, kv_len = state["case"], state["q"], state["cu_q"], state["kv_len"]
    B, H, Hkv, d, P = c["batch"], c["heads"], c["kv_heads"], c["dim"], c["page"]
    T, G, Q, L = q.shape[0], c["heads"] // c["kv_heads"], state["longest_new"], state["longest"]
    i, j = torch.arange(Q, device="cuda"), torch.arange(L, device="cuda")
    n = cu[1:] - cu[:-1]
    rows = torch.where(i[None, :] < n[:, None], cu[:-1, None] + i[None, :], T).long()  # [B, Q]; T: none
    qp = q[rows.clamp(max=T - 1)].float().view(B, Q, Hkv, G, d).permute(0, 2, 3, 1, 4)
    page = state["pages"].clamp(min=0)[:, j // P].long()
    slot = (j % P)[None, :].expand(B, L)
    inside = j[None, :] < kv_len[:, None]
    # [B, Hkv, 1, L, d]; positions that a sequence does not have count as zeros
    k = torch.where(inside[..., None, None], _values(state["k_pages"], state["k_step"], page, slot), 0.0)
    v = torch.where(inside[..., None, None], _values(state["v_pages"], state["v_step"], page, slot), 0.0)
    k, v = k.transpose(1, 2).unsqueeze(2), v.transpose(1, 2).unsqueeze(2)
    s = torch.matmul(qp.reshape(B, Hkv, 1, G * Q, d), k.transpose(-1, -2)).view(B, Hkv, G, Q, L)
    s *= state["scale"]
    see = inside[:, None, :].expand(B, Q, L)
    if c["causal"]:
        see = see & (j[None, None, :] <= (kv_len - n)[:, None, None] + i[None, :, None])
    s.masked_fill_(~see[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    s.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = s.sum(-1, keepdim=True)
    o = torch.matmul(s.view(B, Hkv, 1, G * Q, L), v).view(B, Hkv, G, Q, d)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 3, 1, 2, 4).reshape(B * Q, H, d)
    out = torch.cat([state["out"], state["out"][:1]])
    out[rows.reshape(-1)] = o.to(torch.bfloat16)
    return out[:T]


# ---- one pass ------------------------------------------------------------------------------------------------------------------
def _own_run(state):
    import ternary_weight_bitlinear_b200 as B
    op = state["case"]["op"]
    cache = B.make_kv_cache(state["k_pages"], state["v_pages"], state["k_step"], state["v_step"])
    batch = B.make_kv_batch(state["cu_q"], state["kv_len"], state["pages"])
    if op == "attention":
        return B.bitlinear_attn_paged(state["q"], cache, batch, state["scale"], causal=state["case"]["causal"],
                                      out=state["out"])
    if op == "write":
        B.bitlinear_kv_write(state["k"], state["v"], cache, batch)
        if state["k_step"] is None:
            return state["k_pages"], state["v_pages"]
    return B.bitlinear_kv_read(cache, batch, k=state["k_out"], v=state["v_out"])


def run(state):
    if own:
        return _own_run(state)
    op = state["case"]["op"]
    if op == "attention":
        return _plain_attention(state)
    if op == "write":
        _plain_write(state)
        if state["k_step"] is None:
            return state["k_pages"], state["v_pages"]
    # an int8 cache is returned as the values that it stands for: the rows just written, read back
    return _plain_read(state)


def work(case):
    n, L = _lengths(case)
    H, Hkv, d, T = case["heads"], case["kv_heads"], case["dim"], sum(n)
    row = Hkv * (d * 2 if case["format"] == "bf16" else d + 4)  # one position's keys (or values) in the cache
    table = 4 * sum(-(-x // case["page"]) for x in L) + 8 * len(n)
    plain = 2 * T * Hkv * d * 2  # the rows' keys and values, bf16
    if case["op"] == "read":
        return {"bytes": 2 * T * row + plain + table, "flops": 2 * T * Hkv * d if case["format"] == "int8" else 0}
    if case["op"] == "write":
        back = (2 * T * row + plain, 2 * T * Hkv * d) if case["format"] == "int8" else (0, 0)
        return {"bytes": plain + 2 * T * row + back[0] + table,
                "flops": (6 * T * Hkv * d if case["format"] == "int8" else 0) + back[1]}
    if case["causal"]:
        pairs = sum(a * (x - a) + a * (a + 1) // 2 for a, x in zip(n, L))
    else:
        pairs = sum(a * x for a, x in zip(n, L))
    return {"bytes": 2 * sum(L) * row + 2 * T * H * d * 2 + table, "flops": 4 * d * H * pairs}


# ---- the definitions in 64 bits --------------------------------------------------------------------------------------------------
def _held64(x):
    """What an int8 cache holds of bf16 rows, in 64 bits (the scale, its reciprocal and each product are 32-bit numbers by definition)."""
    r32 = lambda t: t.float().double()  # noqa: E731
    x = x.double()
    s = r32(127.0 / torch.clamp(x.abs().amax(-1, keepdim=True), min=float(torch.tensor(SCALE_FLOOR))))
    return torch.clamp(torch.round(r32(x * s)), -128, 127), r32(1.0 / s)


def exact(case, seed):
    st = prepare(case, seed)
    n, L = _lengths(case)
    P, G = case["page"], case["heads"] // case["kv_heads"]
    k64, v64 = st["k_pages"].double(), st["v_pages"].double()
    if st["k_step"] is not None:
        k64 *= st["k_step"].double().transpose(1, 2)[..., None]
        v64 *= st["v_step"].double().transpose(1, 2)[..., None]
    at, out = 0, None
    if case["op"] == "attention":
        out = st["out"].double()
    elif "k_out" in st:
        out = [st["k_out"].double(), st["v_out"].double()]
    for b in range(case["batch"]):
        mine = st["pages"][b, :-(-L[b] // P)].long()
        new = slice(at, at + n[b])
        at += n[b]
        if case["op"] == "write":
            pos = torch.arange(L[b] - n[b], L[b], device="cuda")
            for pages, rows in ((k64, st["k"][new]), (v64, st["v"][new])):
                if st["k_step"] is None:
                    pages[mine[pos // P], pos % P] = rows.double()
                else:
                    code, step = _held64(rows)
                    pages[mine[pos // P], pos % P] = code * step
        k, v = (x[mine].flatten(0, 1)[:L[b]] for x in (k64, v64))
        if case["op"] == "attention":
            i = torch.arange(n[b], device="cuda")[:, None]
            hidden = torch.arange(L[b], device="cuda")[None, :] > L[b] - n[b] + i
            for h in range(case["heads"]):
                s = (st["q"][new, h].double() @ k[:, h // G].T) * st["scale"]
                if case["causal"]:
                    s.masked_fill_(hidden, -math.inf)
                out[new, h] = torch.softmax(s, -1) @ v[:, h // G]
        elif out is not None:
            out[0][new], out[1][new] = k[L[b] - n[b]:], v[L[b] - n[b]:]
    if out is None:
        return k64, v64
    return tuple(out) if isinstance(out, list) else out
