"""Shared by the tests of ragged steps: seeded batches over a poisoned paged
pool, the definition of the attention in 64 bits, and how far a kernel may be
from it."""

from __future__ import annotations

import math

import torch

from mla_latent_kv_39_b200 import Cache, Config, abi

V3 = dict(hidden=256, n_heads=128, d_c=512, d_r=64, qk_nope=128, v_head=128, q_lora=0)
TINY = dict(hidden=256, n_heads=4, d_c=64, d_r=16, qk_nope=32, v_head=32, q_lora=0, dtype="f32")


class Ragged:
    """A batch: ``cached`` rows and ``new`` tokens per sequence.  Every pool row
    that holds no row of a sequence is NaN, so are the padding queries."""

    def __init__(self, cfg: Config, cached, new, pad=0, seed=0, spread=1.0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        self.cfg, self.cached, self.new, self.pad = cfg, list(cached), list(new), pad
        bs, row, H = cfg.block_size, cfg.d_c + cfg.d_r, cfg.n_heads
        self.lens = [c + n for c, n in zip(cached, new)]
        self.n = sum(new)
        self.n_tok = self.n + pad
        pages = [(x + bs - 1) // bs for x in self.lens]
        blocks, width = sum(pages) + 2, max(pages) + 1
        ids = torch.randperm(blocks, device=device, generator=g).int()
        self.table = torch.full((len(new), width), -1, dtype=torch.int32, device=device)
        self.pool64 = []           # the sequences' rows as the cache holds them
        full = torch.full((blocks, bs, row), math.nan, device=device)
        scales = torch.ones(blocks, bs, device=device)
        at = 0
        for b, (x, n) in enumerate(zip(self.lens, pages)):
            self.table[b, :n] = ids[at:at + n]
            rows = spread * torch.randn(x, row, device=device, generator=g)
            if cfg.fp8_cache:
                sc = 2.0 ** torch.randint(-4, -1, (x, 1), device=device, generator=g).float()
                codes = (rows / sc).clamp(-448, 448).to(torch.float8_e4m3fn)
                self.pool64.append(codes.double() * sc.double())
                rows = codes.float()
                buf = torch.ones(n * bs, device=device)
                buf[:x] = sc[:, 0]
                scales[ids[at:at + n].long()] = buf.view(n, bs)
            else:
                rows = rows.to(cfg.torch_dtype)
                self.pool64.append(rows.double())
            buf = torch.full((n * bs, row), math.nan, device=device)
            buf[:x] = rows.float()
            full[ids[at:at + n].long()] = buf.view(n, bs, row)
            at += n
        self.pool = full.to(torch.float8_e4m3fn).view(torch.uint8) if cfg.fp8_cache else full.to(cfg.torch_dtype)
        self.row_scale = scales if cfg.fp8_cache else None
        q_lat = 0.5 * torch.randn(self.n_tok, H, cfg.d_c, device=device, generator=g)
        q_rope = torch.randn(self.n_tok, H, cfg.d_r, device=device, generator=g)
        q_lat[self.n:] = math.nan
        q_rope[self.n:] = math.nan
        q = torch.cat([q_lat, q_rope], -1)
        if cfg.dtype == "bf16" and not cfg.fp8_cache:
            hi = q.bfloat16()
            self.q, self.q64 = hi, hi.double()
            if cfg.split_query:
                lo = (q - hi.float()).bfloat16()
                self.q, self.q64 = torch.cat([hi, lo]), hi.double() + lo.double()
        else:
            self.q, self.q64 = (q_lat.contiguous(), q_rope.contiguous()), q.double()
        cu = [0]
        for k in new:
            cu.append(cu[-1] + k)
        self.cu = cu
        self.cu_q = torch.tensor(cu, dtype=torch.int32, device=device)
        self.seq_lens = torch.tensor(self.lens, dtype=torch.int32, device=device)
        self.o_lat = torch.full((self.n_tok, H, cfg.d_c), 7.0, dtype=cfg.torch_dtype, device=device)
        self.lse = torch.full((self.n_tok, H), 7.0, device=device)
        self.ws = torch.full((abi.mla_chunk_workspace_size(cfg, self.n_tok),), 0xFF, dtype=torch.uint8, device=device)
        self.cache = Cache(self.pool, self.table, self.row_scale)

    def run(self, window=0, sinks=0, max_workers=0, stream=None):
        if window:
            abi.mla_window_attention(self.cfg, self.q, self.cu_q, self.cache, self.seq_lens, window, sinks, self.o_lat,
                                     self.ws, self.lse, max_workers, stream)
        else:
            abi.mla_chunk_attention(self.cfg, self.q, self.cu_q, self.cache, self.seq_lens, self.o_lat, self.ws, self.lse,
                                    max_workers, stream)

    def expect(self, window=0, sinks=0):
        """(o_lat, lse, bound of |o_lat error|, bound of |lse error|) in 64 bits, from the definition."""
        cfg = self.cfg
        H, d_c = cfg.n_heads, cfg.d_c
        scale = 1.0 / math.sqrt(cfg.qk_nope + cfg.d_r)
        dev = self.o_lat.device
        o = torch.zeros(self.n, H, d_c, dtype=torch.float64, device=dev)
        lse = torch.full((self.n, H), -math.inf, dtype=torch.float64, device=dev)
        eo, el = torch.zeros_like(o), torch.zeros_like(lse)
        # what a score may be off: the fp32 sum of its 576 products.  A CUDA-core
        # lane adds them one by one in four chains, a tensor core 16 at a step; at
        # most row / 4 + 2 additions follow one another, each with a step of 2^-23
        # relative to the sum of magnitudes.  exp2 and the sums of the softmax add
        # 2^-19 (2^-22 an exponential, up to 8 rescalings).
        chain = ((cfg.d_c + cfg.d_r) / 4 + 2) * 2.0 ** -23
        half = 2.0 ** -8 if cfg.dtype == "bf16" else 0.0        # half a bf16 step
        for b, n in enumerate(self.new):
            rows = self.pool64[b]
            L = rows.shape[0]
            u = torch.arange(L, device=dev)
            for j in range(n):
                t, p = self.cu[b] + j, L - n + j
                see = u <= p
                if window:
                    see &= (u > p - window) | (u < sinks)
                kv = rows[see]
                s = (self.q64[t] @ kv.T) * scale
                ds = chain * ((self.q64[t].abs() @ kv.abs().T) * scale).amax(-1) + 2.0 ** -19
                w = torch.softmax(s, -1)
                o[t] = w @ kv[:, :d_c]
                lse[t] = torch.logsumexp(s, -1) / math.log(2)
                mag = w @ kv[:, :d_c].abs()
                # P rounded once (tensor cores), the output rounded once, the scores' error in the weights
                eo[t] = half * (mag + o[t].abs()) * (1 + half) + (torch.expm1(2 * ds)[:, None] + 2.0 ** -18) * mag
                el[t] = ds / math.log(2) + 2.0 ** -20 * (1 + lse[t].abs())
        return o, lse, eo, el

    def check(self, window=0, sinks=0, skip=()):
        torch.cuda.synchronize()
        o, lse, eo, el = self.expect(window, sinks)
        got, got_lse = self.o_lat[:self.n].double(), self.lse[:self.n].double()
        keep = torch.ones(self.n, dtype=torch.bool, device=got.device)
        for b in skip:
            keep[self.cu[b]:self.cu[b + 1]] = False
        bad = ~((got - o).abs() <= eo) & keep[:, None, None]
        assert not bad.any(), ("o_lat", bad.any(-1).any(-1).nonzero().flatten().tolist()[:20],
                               float(((got - o).abs() / eo)[keep].nan_to_num(math.inf).max()))
        bad = ~((got_lse - lse).abs() <= el) & keep[:, None]
        assert not bad.any(), ("lse", bad.any(-1).nonzero().flatten().tolist()[:20])
        # the padding rows are as they were
        assert (self.o_lat[self.n:] == 7).all() and (self.lse[self.n:] == 7).all()
