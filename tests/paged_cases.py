"""Seeded paged caches for the tests: ragged lengths, shuffled pages, stale
contents in every slot that holds no position."""
import numpy as np
import torch

from oracle import paged as OP


class Case:
    """A cache of sequences with `ctx` cached positions before `new` new
    rows each; `extra` rows belong to nobody.  `window` > 0 gives pages only
    to positions some new row sees (the others' table entries are -1)."""

    def __init__(self, ctx, new, *, g=4, ps=16, fp8=False, window=0, rope=False, seed=0, extra=0, w_scale=1.0,
                 v_scale=1.0, stale="nan", sinks=None, theta=10000.0):
        r = np.random.default_rng(seed)
        self.ctx, self.new = np.array(ctx, np.int32), np.array(new, np.int32)
        self.B, self.g, self.ps, self.fp8, self.window, self.rope, self.theta = len(ctx), g, ps, fp8, window, rope, theta
        self.cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.rows, self.T = int(self.cu[-1]), int(self.cu[-1]) + extra
        self.wq = (1 + 0.1 * r.standard_normal(128)).astype(np.float32) * np.float32(w_scale)
        self.wk = (1 + 0.1 * r.standard_normal(128)).astype(np.float32) * np.float32(w_scale)
        self.sinks = r.standard_normal(8 * g).astype(np.float32) if sinks is None else np.asarray(sinks, np.float32)
        bf = lambda *s: torch.from_numpy(r.standard_normal(s).astype(np.float32)).bfloat16()  # noqa: E731
        self.q, self.k = bf(self.T, 8 * g, 128), bf(self.T, g, 128)
        self.v = (bf(self.T, g, 128).float() * v_scale).bfloat16()
        first = [max(0, c - window + 1) // ps if window else 0 for c in ctx]
        last = [(c + n - 1) // ps if c + n else -1 for c, n in zip(ctx, new)]
        width = max(max(last) + 1, 1) + 2
        self.P = sum(max(0, y - x + 1) for x, y in zip(first, last)) + 3
        order = r.permutation(self.P)
        self.table = np.full((self.B, width), -1, np.int32)
        at = 0
        for b in range(self.B):
            for i in range(first[b], last[b] + 1):
                self.table[b, i] = order[at]
                at += 1
        # contents: what earlier calls would have left at cached positions,
        # stale bits (NaN, or the largest numbers) everywhere else
        shape = (self.P, g, ps, 128)
        held = np.zeros((self.P, ps), bool)
        for b in range(self.B):
            for p in range(first[b] * ps, ctx[b]):
                held[self.table[b, p // ps], p % ps] = True
        held = torch.from_numpy(held)[:, None, :, None]
        kk = OP.norm_rope(r.standard_normal(shape), self.wk, 0, False)
        vv = torch.from_numpy((r.standard_normal(shape) * v_scale).astype(np.float32)).bfloat16()
        bad = float("nan") if stale == "nan" else 448.0 if fp8 else 65504.0
        if fp8:
            kc, ke = OP.quantise(kk)
            vc, ve = OP.quantise(vv.double().numpy())
            self.k_pages = torch.where(held, torch.from_numpy(kc).float(), torch.tensor(bad)).to(torch.float8_e4m3fn)
            self.v_pages = torch.where(held, torch.from_numpy(vc).float(), torch.tensor(bad)).to(torch.float8_e4m3fn)
            top = 255 if stale == "nan" else 167
            sc = [torch.where(held[..., 0], torch.from_numpy(e + 127), torch.tensor(top)).to(torch.uint8) for e in (ke, ve)]
            self.k_scales, self.v_scales = (x.contiguous().view(torch.float8_e8m0fnu) for x in sc)
        else:
            self.k_pages = torch.where(held, torch.from_numpy(kk).half(), torch.tensor(bad).half())
            self.v_pages = torch.where(held, vv, torch.tensor(bad).bfloat16())
            self.k_scales = self.v_scales = None

    def to(self, dev):
        """Every tensor of the calls, on dev."""
        c = lambda x: None if x is None else (torch.from_numpy(x) if isinstance(x, np.ndarray) else x).to(dev).contiguous()  # noqa: E731
        return {n: c(getattr(self, n)) for n in ("q", "k", "v", "wq", "wk", "sinks", "k_pages", "v_pages", "k_scales",
                                                 "v_scales", "table", "ctx", "cu")}

    def slots(self):
        """(page, slot) of every new row; page -1 where it is not kept."""
        b, pos = OP.rows_of(self.ctx, self.cu)
        return self.table[b, pos // self.ps], pos % self.ps


def values(pages, scales):
    """float64 values that pages stand for."""
    x = pages.cpu().double().numpy()
    return x if scales is None else x * np.exp2(scales.cpu().view(torch.uint8).double().numpy() - 127.0)[..., None]
