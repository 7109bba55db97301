"""Operators of a ragged serving step over the paged latent cache, case by case.

Three operators, as a serving loop calls them one after the other:

- ``tables``: block tables, positions and slot maps built on the GPU from the
  requests' lengths (``mla_batch_tables``);
- ``chunk``: every request's new tokens attend to its paged latent rows and
  causally to each other (``mla_chunk_attention``);
- ``window``: the same with a sliding window and a few first rows that stay
  visible (``mla_window_attention``); with one new token per request this is
  the windowed decode.

``run`` computes a case in plain torch operations, or with ``own`` through the
package.  Attention with heads h, latent rows c_u and rotary keys r_u:

    s_u = scale (q_lat . c_u + q_rope . r_u),   visible(u) only
    lse = log2 sum_u exp(s_u),   o_lat = sum_u softmax(s)_u c_u

Token j of a request's n new tokens stands at position p = seq_len - n + j and
sees the rows u <= p, with a window only those with u > p - window or
u < n_sinks.
"""

import math
import random

import numpy as np
import torch

own = False

PAGE = 64
WIDE = dict(H=128, d_c=512, d_r=64, nope=128)    # the 128-head shape of the bench workload
TINY = dict(H=4, d_c=64, d_r=16, nope=32)        # the fp32 shape


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step's bookkeeping of the bench workload: 64 requests, one new token each
        dict(name="tables decode b64", op="tables", batch=64, ctx_lo=1024, ctx_hi=8192, new_lo=1, new_hi=1, pad=0, lens=1),
        # continuous batching: requests without new tokens, decodes and prompts mixed, padded token arrays
        dict(name="tables mixed b509", op="tables", batch=509, ctx_lo=0, ctx_hi=16384, new_lo=0, new_hi=300, pad=777, lens=2),
        # the smallest attention call: one token of a short request
        dict(name="chunk one token", op="chunk", dtype="bf16", batch=1, ctx_lo=100, ctx_hi=100, new_lo=1, new_hi=1, pad=0,
             window=0, sinks=0, lens=3),
        # the tiny fp32 shape, ragged, a request without new tokens likely
        dict(name="chunk tiny fp32", op="chunk", dtype="f32", batch=7, ctx_lo=0, ctx_hi=400, new_lo=0, new_hi=40, pad=5,
             window=0, sinks=0, lens=4),
        # one request's single token over a long cache: the split over the long axis
        dict(name="chunk decode 100k", op="chunk", dtype="bf16", batch=1, ctx_lo=100000, ctx_hi=100000, new_lo=1, new_hi=1,
             pad=0, window=0, sinks=0, lens=5),
        # chunked prefill of the repository's workload: 8 requests, 64 new tokens, 1k to 4k cached
        dict(name="chunk prefill b8 c64", op="chunk", dtype="bf16", batch=8, ctx_lo=1024, ctx_hi=4096, new_lo=64, new_hi=64,
             pad=0, window=0, sinks=0, lens=6),
        # decodes and odd chunks in one ragged batch with padded rows behind
        dict(name="chunk ragged b23", op="chunk", dtype="bf16", batch=23, ctx_lo=0, ctx_hi=3000, new_lo=0, new_hi=130, pad=19,
             window=0, sinks=0, lens=7),
        # a long prompt's last chunk: the largest
        dict(name="chunk prefill 16k c1024", op="chunk", dtype="bf16", batch=1, ctx_lo=15360, ctx_hi=15360, new_lo=1024,
             new_hi=1024, pad=0, window=0, sinks=0, lens=8),
        # windowed decode: 64 long requests, one token each
        dict(name="window decode b64", op="window", dtype="bf16", batch=64, ctx_lo=4096, ctx_hi=16384, new_lo=1, new_hi=1,
             pad=0, window=2048, sinks=4, lens=9),
        # windowed prefill: ragged chunks, window and sinks off the page grid
        dict(name="window prefill b6", op="window", dtype="bf16", batch=6, ctx_lo=500, ctx_hi=6000, new_lo=100, new_hi=400,
             pad=0, window=1000, sinks=70, lens=10),
        # the tiny fp32 shape with a window shorter than a page
        dict(name="window tiny fp32", op="window", dtype="f32", batch=9, ctx_lo=0, ctx_hi=700, new_lo=1, new_hi=30, pad=3,
             window=33, sinks=5, lens=11),
    ]


def _log(rng, lo, hi):
    """An integer of [lo, hi], spread over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    while True:
        op = rng.choice(["tables", "chunk", "chunk", "window", "window"])
        lens = rng.randrange(1 << 20)
        if op == "tables":
            new_hi = _log(rng, 1, 300)
            return dict(op=op, batch=_log(rng, 1, 600), ctx_lo=0, ctx_hi=_log(rng, 64, 16384), new_lo=rng.choice([0, 1]),
                        new_hi=new_hi, pad=rng.choice([0, rng.randrange(1, 800)]), lens=lens)
        dtype = "f32" if rng.random() < 0.2 else "bf16"
        wide = dtype == "bf16"
        c = dict(op=op, dtype=dtype, batch=_log(rng, 1, 64 if wide else 12), ctx_lo=rng.choice([0, 1, 500]),
                 ctx_hi=_log(rng, 500, 100000 if wide else 700), new_lo=rng.choice([0, 1]),
                 new_hi=rng.choice([1, _log(rng, 2, 500 if wide else 40)]), pad=rng.choice([0, rng.randrange(1, 40)]),
                 window=0, sinks=0, lens=lens)
        if op == "window":
            c.update(window=_log(rng, 1, 4096 if wide else 300), sinks=rng.choice([0, rng.randrange(1, 9), rng.randrange(1, 150)]))
        # no dearer than the largest listed case, neither in work nor in the plain form's padded scores
        cached, new = _lens(c)
        padded = c["batch"] * max(new) * max(a + b for a, b in zip(cached, new))
        pages = sum((a + b + PAGE - 1) // PAGE for a, b in zip(cached, new))
        if sum(new) > 0 and padded <= 1024 * 16384 and pages <= 12000 and c["batch"] * max(a + b for a, b in zip(cached, new)) <= 800000:
            return c


def _lens(case):
    """(cached, new) lengths of every request: a matter of the case, not of the seed."""
    r = random.Random(case["lens"])
    cached = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["batch"])]
    new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["batch"])]
    if sum(new) == 0:
        new[-1] = 1
    return cached, new


def _shape(case):
    return WIDE if case.get("dtype", "bf16") == "bf16" else TINY


def _visible(case, p):
    """Rows that a token at position p sees."""
    w, s = case["window"], case["sinks"]
    return p + 1 if w == 0 or p + 1 <= w + s else w + s


def work(case):
    cached, new = _lens(case)
    B, n = case["batch"], sum(new)
    pages = [((c + k + PAGE - 1) // PAGE, (c + PAGE - 1) // PAGE) for c, k in zip(cached, new)]
    if case["op"] == "tables":
        taken = sum(a - b for a, b in pages)
        # read: both lengths, the free ids taken, one table entry of each request that goes on in an open page
        opened = sum(1 for c, k in zip(cached, new) if k > 0 and c % PAGE)
        read = 4 * (2 * B + taken + opened + 1)
        # written: the new table entries, prefix, lengths, and 16 bytes a token slot
        return {"bytes": read + 4 * (taken + 2 * B + 2) + 16 * (n + case["pad"]), "flops": 0}
    s = _shape(case)
    H, row, e = s["H"], s["d_c"] + s["d_r"], 2 if case["dtype"] == "bf16" else 4
    seen = sum(_visible(case, c + j) for c, k in zip(cached, new) for j in range(k))
    rows = 0        # distinct cached rows that any token of a request sees
    for c, k in zip(cached, new):
        if k:
            first = max(0, c - case["window"] + 1) if case["window"] else 0
            rows += c + k - first + min(case["sinks"], first)
    return {"bytes": n * H * (row + s["d_c"]) * e + 4 * n * H + rows * row * e + 4 * rows // PAGE + 8 * B,
            "flops": 2 * H * (row + s["d_c"]) * seen}


# ------------------------------------------------------------------ state

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    cached, new = _lens(case)
    B, n = case["batch"], sum(new)
    n_tok = n + case["pad"]
    blocks = sum((c + k + PAGE - 1) // PAGE for c, k in zip(cached, new)) + 3
    width = max((c + k + PAGE - 1) // PAGE for c, k in zip(cached, new)) + 1
    ids = torch.randperm(blocks, device="cuda", generator=g).int()     # physical pages in no order
    have = torch.tensor([(c + PAGE - 1) // PAGE for c in cached])
    need = torch.tensor([(c + k + PAGE - 1) // PAGE for c, k in zip(cached, new)])
    at = torch.arange(width).expand(B, width)
    held = (at < (have if case["op"] == "tables" else need)[:, None]).cuda()
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    n_held = int(held.sum())
    table[held] = ids[:n_held]
    st = dict(case=case, cached=torch.tensor(cached, dtype=torch.int32, device="cuda"),
              new=torch.tensor(new, dtype=torch.int32, device="cuda"), table=table, n_tok=n_tok, blocks=blocks)
    i32 = dict(dtype=torch.int32, device="cuda")
    if case["op"] == "tables":
        lead = 5                                   # ids before the cursor were handed out in earlier steps
        free = torch.cat([torch.zeros(lead, **i32), ids[n_held:]])
        st.update(free=free, head=torch.full((1,), lead, **i32), head_out=torch.zeros(1, **i32),
                  cu_q=torch.zeros(B + 1, **i32), seq_lens=torch.zeros(B, **i32), seq_idx=torch.zeros(n_tok, **i32),
                  pos=torch.zeros(n_tok, **i32), slots=torch.zeros(n_tok, dtype=torch.int64, device="cuda"))
        return st
    s = _shape(case)
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    cu = [0]
    for k in new:
        cu.append(cu[-1] + k)
    # latent rows of unit variance; queries as the projections of unit-variance
    # hidden states give them (scores of about unit variance after the scale)
    pool = torch.randn(blocks, PAGE, s["d_c"] + s["d_r"], device="cuda", generator=g).to(dt)
    q_lat = 0.5 * torch.randn(n_tok, s["H"], s["d_c"], device="cuda", generator=g)
    q_rope = torch.randn(n_tok, s["H"], s["d_r"], device="cuda", generator=g)
    q = torch.cat([q_lat, q_rope], -1).to(dt) if dt == torch.bfloat16 else (q_lat, q_rope)
    st.update(pool=pool, q=q, cu_q=torch.tensor(cu, **i32),
              seq_lens=torch.tensor([c + k for c, k in zip(cached, new)], **i32),
              o_lat=torch.zeros(n_tok, s["H"], s["d_c"], dtype=dt, device="cuda"),
              lse=torch.zeros(n_tok, s["H"], device="cuda"))
    return st


# ------------------------------------------------------------------ one pass

def run(state):
    if own:
        return _run_own(state)
    return _plain_tables(state) if state["case"]["op"] == "tables" else _plain_attention(state)


def _run_own(state):
    import mla_latent_kv_39_b200 as mla
    case = state["case"]
    if "handle" not in state:      # what a program makes once: configuration, cache view, workspace
        s = _shape(case)
        cfg = mla.Config(hidden=256, n_heads=s["H"], d_c=s["d_c"], d_r=s["d_r"], qk_nope=s["nope"], v_head=s["nope"], q_lora=0,
                         dtype=case.get("dtype", "bf16"))
        if case["op"] == "tables":
            state["handle"] = (mla, cfg, None, None)
        else:
            ws = torch.empty(mla.mla_chunk_workspace_size(cfg, state["n_tok"]), dtype=torch.uint8, device="cuda")
            state["handle"] = (mla, cfg, mla.Cache(state["pool"], state["table"]), ws)
    mla, cfg, cache, ws = state["handle"]
    if case["op"] == "tables":
        mla.mla_batch_tables(cfg, state["cached"], state["new"], state["free"], state["head"], state["blocks"], state["table"],
                             state["cu_q"], state["seq_lens"], state["seq_idx"], state["pos"], state["slots"],
                             state["head_out"])
        return {k: state[k] for k in ("table", "cu_q", "seq_lens", "seq_idx", "pos", "slots", "head_out")}
    if case["op"] == "chunk":
        mla.mla_chunk_attention(cfg, state["q"], state["cu_q"], cache, state["seq_lens"], state["o_lat"], ws, state["lse"])
    else:
        mla.mla_window_attention(cfg, state["q"], state["cu_q"], cache, state["seq_lens"], case["window"], case["sinks"],
                                 state["o_lat"], ws, state["lse"])
    return {"o_lat": state["o_lat"], "lse": state["lse"]}


def _plain_tables(st):
    cached, new, table, free, head = (st[k] for k in ("cached", "new", "table", "free", "head"))
    B, n_tok = cached.numel(), st["n_tok"]
    have = (cached + PAGE - 1) // PAGE
    need = (cached + new + PAGE - 1) // PAGE
    zero = torch.zeros(1, dtype=torch.int64, device="cuda")
    first = torch.cat([zero, torch.cumsum(need - have, 0)]) + head       # cursor at each request's first new page
    at = torch.arange(table.shape[1], device="cuda")
    fresh = (at >= have[:, None]) & (at < need[:, None])
    take = (first[:-1, None] + at - have[:, None]).clamp(0, free.numel() - 1)
    table = torch.where(fresh, free[take], table)
    cu = torch.cat([zero, torch.cumsum(new, 0)])
    t = torch.arange(n_tok, device="cuda")
    b = torch.searchsorted(cu, t, right=True) - 1
    real = b < B
    b = b.clamp(max=B - 1)
    pos = cached[b] + t - cu[b]
    page = (pos // PAGE).clamp(0, table.shape[1] - 1)
    slots = table[b, page].long() * PAGE + pos % PAGE
    return {"table": table, "cu_q": cu.int(), "seq_lens": cached + new, "seq_idx": torch.where(real, b, -1).int(),
            "pos": torch.where(real, pos, 0).int(), "slots": torch.where(real, slots, -1), "head_out": first[-1:].int()}


def _plain_attention(st):
    case = st["case"]
    s = _shape(case)
    H, d_c, d_r = s["H"], s["d_c"], s["d_r"]
    scale = 1.0 / math.sqrt(s["nope"] + d_r)
    cu, lens = st["cu_q"].long(), st["seq_lens"].long()
    B, n_tok = lens.numel(), st["n_tok"]
    q = st["q"] if isinstance(st["q"], torch.Tensor) else torch.cat(st["q"], -1)
    new = cu[1:] - cu[:-1]
    # rows [B, L, d_c + d_r] of every request (pages past its own are never visible)
    rows = st["pool"][st["table"].clamp(min=0).long()].reshape(B, -1, d_c + d_r).float()
    L = rows.shape[1]
    # queries [B, N, H, d_c + d_r], padded to the longest chunk
    _, fresh = _lens(case)
    N = max(fresh)
    j = torch.arange(N, device="cuda")
    real = j < new[:, None]
    qp = q[(cu[:-1, None] + j).clamp(max=n_tok - 1)].float()
    p = (lens - new)[:, None] + j
    u = torch.arange(L, device="cuda")
    see = u <= p[..., None]
    if case["window"]:
        see = see & ((u > p[..., None] - case["window"]) | (u < case["sinks"]))
    scores = torch.matmul(qp.reshape(B, N * H, -1), rows.transpose(1, 2)).view(B, N, H, L).mul_(scale)
    scores.masked_fill_(~see[:, :, None, :], -math.inf)
    top = scores.amax(-1, keepdim=True)
    w = scores.sub_(top).exp_()
    z = w.sum(-1, keepdim=True)
    o = torch.matmul(w.view(B, N * H, L), rows[..., :d_c]).view(B, N, H, d_c) / z
    lse = (top / math.log(2) + torch.log2(z)).squeeze(-1)
    n = int(sum(fresh))
    out, out_lse = torch.zeros_like(st["o_lat"]), torch.zeros_like(st["lse"])
    out[:n] = o[real].to(out.dtype)
    out_lse[:n] = lse[real]
    return {"o_lat": out, "lse": out_lse}


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    cached, new = _lens(case)
    if case["op"] == "tables":
        return None
    s = _shape(case)
    H, d_c = s["H"], s["d_c"]
    q = st["q"] if isinstance(st["q"], torch.Tensor) else torch.cat(st["q"], -1)
    out = torch.zeros(st["n_tok"], H, d_c, dtype=torch.float64, device="cuda")
    lse = torch.zeros(st["n_tok"], H, dtype=torch.float64, device="cuda")
    scale = (s["nope"] + s["d_r"]) ** -0.5
    t = 0
    for b, (c, k) in enumerate(zip(cached, new)):
        kv = st["pool"][st["table"][b, : (c + k + PAGE - 1) // PAGE].long()].double().flatten(0, 1)[: c + k]
        for lo in range(0, k, 16):
            m = min(16, k - lo)
            x = torch.einsum("jhd,ud->jhu", q[t + lo:t + lo + m].double(), kv) * scale
            hidden = np.zeros((m, c + k), dtype=bool)
            for i in range(m):
                p = c + lo + i
                hidden[i, p + 1:] = True
                if case["window"] and p - case["window"] + 1 > case["sinks"]:
                    hidden[i, case["sinks"]:p - case["window"] + 1] = True
            x = x.masked_fill(torch.from_numpy(hidden).cuda()[:, None, :], -math.inf)
            lse[t + lo:t + lo + m] = torch.logsumexp(x, -1) / math.log(2)
            out[t + lo:t + lo + m] = torch.einsum("jhu,ud->jhd", torch.softmax(x, -1), kv[:, :d_c])
        t += k
    return {"o_lat": out, "lse": lse}
