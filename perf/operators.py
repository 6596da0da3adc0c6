"""The paged key/value cache of a serving step, measured: append, read back, attention of new tokens.

Three operators, each in a plain form (elementary torch operations) and through the package's entry points:

* append: the new tokens' keys are normalised per head (weight-form RMSNorm), rotated on sliding layers, and
  written with their values into the pages that a page table names; 16-bit pages (K FP16, V BF16) or 8-bit
  pages (E4M3 with one power-of-two scale per token and head);
* read: a run of cached positions of each sequence, out of the pages into packed rows (K FP16, V BF16);
* attn: causal sink attention of a ragged batch of new tokens (one per sequence, a few drafted ones, or a
  prompt's chunk) over their pages, the new tokens' own keys included.

Sequence b has `cache_len[b]` cached positions before its new rows cu_new[b] .. cu_new[b + 1] - 1.
"""
import math
import random

import torch

own = False

HD = 128          # head dimension
GROUP = 8         # query heads per key/value head
THETA, EPS = 10000.0, 1e-6
E_MIN, E_MAX = -24, 40


def _case(name, op, b, heads, fp8, page, window, rope, ctx, new, lens):
    c = {"op": op, "b": b, "heads": heads, "fp8": fp8, "page": page, "window": window, "rope": rope,
         "ctx_lo": ctx[0], "ctx_hi": ctx[1], "new_lo": new[0], "new_hi": new[1], "lens": lens}
    return dict(c, name=name) if name else c


def listed():
    return [
        # a decode step's new rows of a sliding layer, 128 sequences anywhere in long documents
        _case("append_step_16", "append", 128, 4, False, 64, 513, True, (513, 262143), (1, 1), 1),
        # four prompts' chunks written at once into an 8-bit cache on a full layer
        _case("append_prompts_8", "append", 4, 4, True, 32, 0, False, (0, 9000), (2500, 8191), 2),
        # one shared prefix moved out of 16-bit pages (to another worker, or a contiguous cache)
        _case("read_prefix_16", "read", 1, 4, False, 128, 0, False, (0, 0), (4096, 4096), 3),
        # many sequences' whole 8-bit caches read back at once
        _case("read_all_8", "read", 24, 4, True, 16, 0, False, (0, 0), (1, 8191), 4),
        # the smallest step: one sequence, one token, a short conversation
        _case("decode_one_16", "attn", 1, 4, False, 16, 0, False, (300, 300), (1, 1), 5),
        # the benchmark's sliding decode step: 128 sequences, window 513, far positions
        _case("decode_sliding_16", "attn", 128, 4, False, 64, 513, True, (513, 262143), (1, 1), 6),
        # the benchmark's full decode step at ragged lengths, on an 8-bit cache
        _case("decode_full_8", "attn", 64, 4, True, 64, 0, False, (1, 4095), (1, 1), 7),
        # two very long conversations, one token each: the long axis has to be split
        _case("decode_long_16", "attn", 2, 4, False, 128, 0, False, (100003, 131071), (1, 1), 8),
        # drafted tokens under verification, on a slice of two heads (head-split serving)
        _case("draft_16", "attn", 16, 2, False, 32, 0, False, (700, 16383), (2, 6), 9),
        # a 2,048-token chunk of a long prompt on a full layer
        _case("chunk_long_16", "attn", 1, 4, False, 64, 0, False, (30001, 30001), (2048, 2048), 10),
        # prompts' chunks over an 8-bit cache on a full layer
        _case("chunk_full_8", "attn", 4, 4, True, 16, 0, False, (100, 8191), (257, 512), 11),
        # a step that mixes decoding sequences with short prompts on a sliding layer, 8-bit cache
        _case("mixed_sliding_8", "attn", 24, 4, True, 32, 513, True, (0, 40000), (1, 384), 12),
    ]


def draw(rng):
    def logu(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    while True:
        op = rng.choice(("append", "read", "attn", "attn", "attn"))
        sliding = op != "read" and rng.random() < 0.4
        window = rng.choice((513, 513, logu(16, 2048))) if sliding else 0
        kind = rng.choice(("one", "few", "chunk"))
        new_hi = {"one": 1, "few": rng.randint(2, 16), "chunk": logu(17, 2048)}[kind]
        new_lo = new_hi if kind == "one" else rng.randint(1, new_hi)
        ctx_hi = logu(1, 200000 if sliding else 100000)
        ctx_lo = rng.randint(0, ctx_hi)
        if op == "read":
            ctx_lo = ctx_hi = 0
            new_hi = logu(1, 30000)
            new_lo = rng.randint(1, new_hi)
        c = _case(None, op, logu(1, 128), rng.choice((4, 4, 4, 2, 1)), rng.random() < 0.5,
                  rng.choice((16, 32, 64, 128)), window, sliding, (ctx_lo, ctx_hi), (new_lo, new_hi),
                  rng.randrange(1 << 20))
        if op == "attn":
            span = (min(c["window"] - 1, ctx_hi) if c["window"] else ctx_hi) + new_hi
            w = work(c)
            # the padded score and key arrays of the plain form, and the largest listed case's work
            if (c["b"] * c["heads"] * GROUP * new_hi * span <= 1.2e9 and c["b"] * c["heads"] * span <= 2.2e6 and w["flops"] <= 1e12 and w["bytes"] <= 5e8):
                return c
        elif work(c)["bytes"] <= 2.5e8 and c["b"] * c["heads"] * (min(ctx_hi, c["window"] or ctx_hi) + new_hi) <= 2.2e6:
            return c


def _lens(c):
    """(cached positions, new rows) of each sequence."""
    r = random.Random(c["lens"])
    ctx = [r.randint(c["ctx_lo"], c["ctx_hi"]) for _ in range(c["b"])]
    new = [r.randint(c["new_lo"], c["new_hi"]) for _ in range(c["b"])]
    return ctx, new


def _first(c, ctx):
    """First position of a sequence that any of its new rows sees."""
    return max(0, ctx - c["window"] + 1) if c["window"] else 0


def work(case):
    c = case
    ctx, new = _lens(c)
    T, g = sum(new), c["heads"]
    kv = g * 2 * ((HD + 1) if c["fp8"] else HD * 2)          # a position's keys and values in the cache
    if c["op"] == "append":
        return {"bytes": T * (g * HD * 4 + kv), "flops": T * g * HD * 8}
    if c["op"] == "read":
        return {"bytes": T * (g * HD * 4 + kv), "flops": T * g * HD * 2}
    seen = pairs = 0
    for L, n in zip(ctx, new):
        seen += L + n - _first(c, L)
        w = c["window"] or L + n
        full = max(0, min(n, w - L))                         # rows that see every earlier position
        pairs += full * L + full * (full + 1) // 2 + (n - full) * w
    return {"bytes": T * g * GROUP * HD * 4 + seen * kv, "flops": 4 * HD * g * GROUP * pairs}


def _pow2(e):
    """2^e in FP32 from its bits (a power function may be off by a last place)."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _quantise(x):
    """E4M3 values of rows [..., 128] and their scales 2^e: the smallest e in [E_MIN, E_MAX] with max|x| <= 448 x 2^e."""
    m, e = torch.frexp(x.abs().amax(-1))
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(E_MIN, E_MAX)
    codes = (x * _pow2(-e)[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return codes, (e + 127).to(torch.uint8)


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    ctx, new = _lens(c)
    b, g, ps = c["b"], c["heads"], c["page"]
    T = sum(new)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)
    # pages of the positions that are kept; the others' table entries are -1
    first = [(_first(c, x) if c["op"] != "read" else x) // ps for x in ctx]
    last = [(x + n - 1) // ps for x, n in zip(ctx, new)]
    width = max(last) + 1 + 3
    table = torch.full((b, width), -1, dtype=torch.int32)
    count = sum(y - x + 1 for x, y in zip(first, last))
    P = count + 5
    order = torch.randperm(P, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    at = 0
    for i in range(b):
        n = last[i] - first[i] + 1
        table[i, first[i]:last[i] + 1] = order[at:at + n]
        at += n
    w = 1 + 0.1 * normal(2, HD)
    k_rows = normal(P, g, ps, HD)
    k_rows = k_rows * torch.rsqrt(k_rows.square().mean(-1, keepdim=True) + EPS) * w[1]
    v_rows = normal(P, g, ps, HD).bfloat16()
    s = {"case": c, "T": T, "max_new": max(new), "max_end": max(x + n for x, n in zip(ctx, new)),
         "span": max(x + n - _first(c, x) for x, n in zip(ctx, new)),
         "k_scales": None, "v_scales": None, "table": table.to(dev),
         "len": torch.tensor(ctx, dtype=torch.int32, device=dev),
         "cu": torch.tensor([sum(new[:i]) for i in range(b + 1)], dtype=torch.int32, device=dev),
         "q_norm_w": w[0].contiguous(), "k_norm_w": w[1].contiguous(), "sinks": normal(g * GROUP)}
    if c["fp8"]:
        s["k_pages"], ks = _quantise(k_rows)
        s["v_pages"], vs = _quantise(v_rows.float())
        s["k_scales"], s["v_scales"] = ks.view(torch.float8_e8m0fnu), vs.view(torch.float8_e8m0fnu)
    else:
        s["k_pages"], s["v_pages"] = k_rows.half(), v_rows
    if c["op"] == "append":
        s["k"], s["v"] = normal(T, g, HD).bfloat16(), normal(T, g, HD).bfloat16()
    if c["op"] == "attn":
        s["q"] = normal(T, g * GROUP, HD).bfloat16()
    return s


def _rows(s):
    """Sequence, position and row within the sequence of each of the T packed rows."""
    t = torch.arange(s["T"], device=s["cu"].device)
    b = torch.searchsorted(s["cu"], t, right=True) - 1
    i = t - s["cu"][b]
    return b, s["len"][b] + i, i


def _norm_rope(x, w, pos, rope):
    x = x.float()
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w
    if not rope:
        return y
    f = THETA ** (-torch.arange(HD // 2, device=x.device, dtype=torch.float64) / (HD // 2))
    a = pos.double()[:, None, None] * f
    cos, sin = a.cos().float(), a.sin().float()
    lo, hi = y[..., :HD // 2], y[..., HD // 2:]
    return torch.cat((lo * cos - hi * sin, hi * cos + lo * sin), -1)


def _take(pages, scales, page, slot):
    """Rows [..., heads, 128] of the pages as FP32 values."""
    if scales is None:
        return pages[page, :, slot].float()
    x = pages.view(torch.uint8)[page, :, slot].view(torch.float8_e4m3fn).float()
    return x * _pow2(scales.view(torch.uint8)[page, :, slot].int() - 127)[..., None]


def _append(s):
    b, pos, _ = _rows(s)
    ps = s["case"]["page"]
    page, slot = s["table"][b, pos // ps].long(), pos % ps
    k = _norm_rope(s["k"], s["k_norm_w"], pos, s["case"]["rope"])
    if s["k_scales"] is None:
        s["k_pages"][page, :, slot] = k.clamp(-65504, 65504).half()
        s["v_pages"][page, :, slot] = s["v"]
        return
    for x, pages, scales in ((k, "k_pages", "k_scales"), (s["v"].float(), "v_pages", "v_scales")):
        codes, e = _quantise(x)
        s[pages].view(torch.uint8)[page, :, slot] = codes.view(torch.uint8)
        s[scales].view(torch.uint8)[page, :, slot] = e


def _read(s):
    b, pos, _ = _rows(s)
    ps = s["case"]["page"]
    page, slot = s["table"][b, pos // ps].long(), pos % ps
    return (_take(s["k_pages"], s["k_scales"], page, slot).half(),
            _take(s["v_pages"], s["v_scales"], page, slot).bfloat16())


def _attn(s):
    c = s["case"]
    B, g, ps, N = c["b"], c["heads"], c["page"], s["max_new"]
    b, pos, i = _rows(s)
    q = _norm_rope(s["q"], s["q_norm_w"], pos, c["rope"]) * HD ** -0.5
    # queries padded to [B, heads, N x 8, 128]; keys and values of the span that any of them sees
    qp = torch.zeros(B, N, g, GROUP, HD, device=q.device)
    qp[b, i] = q.view(-1, g, GROUP, HD)
    qp = qp.permute(0, 2, 1, 3, 4).reshape(B, g, N * GROUP, HD)
    lo = (s["len"] - c["window"] + 1).clamp(min=0) if c["window"] else torch.zeros_like(s["len"])
    idx = lo[:, None] + torch.arange(s["span"], device=q.device)
    page = s["table"].gather(1, (idx // ps).clamp(max=s["table"].shape[1] - 1)).clamp(min=0).long()
    k = _take(s["k_pages"], s["k_scales"], page, idx % ps)                     # [B, S, heads, 128]
    v = _take(s["v_pages"], s["v_scales"], page, idx % ps)
    at = s["len"][:, None] + torch.arange(N, device=q.device)                  # positions of the queries
    seen = idx[:, None, :] <= at[:, :, None]
    if c["window"]:
        seen &= idx[:, None, :] > at[:, :, None] - c["window"]
    z = torch.matmul(qp, k.permute(0, 2, 3, 1)).view(B, g, N, GROUP, -1)
    z.masked_fill_(~seen[:, None, :, None, :], float("-inf"))
    sink = s["sinks"].view(1, g, 1, GROUP)
    m = torch.maximum(z.amax(-1), sink)
    z.sub_(m[..., None]).exp_()
    l = z.sum(-1) + (sink - m).exp()
    o = torch.matmul(z.view(B, g, N * GROUP, -1), v.permute(0, 2, 1, 3)).view(B, g, N, GROUP, HD) / l[..., None]
    return o.permute(0, 2, 1, 3, 4)[b, i].reshape(s["T"], -1).bfloat16()


def run(state):
    s = state
    c = s["case"]
    if own:
        import full_gqa_learned_b200 as fa
        kw = {"k_scales": s["k_scales"], "v_scales": s["v_scales"]}
    if c["op"] == "append":
        if own:
            fa.paged_append(s["k"], s["v"], s["k_norm_w"], s["k_pages"], s["v_pages"], s["table"], s["len"], s["cu"],
                            use_rope=c["rope"], rope_theta=THETA, eps=EPS, **kw)
        else:
            _append(s)
        return {n: s[n] for n in ("k_pages", "v_pages", "k_scales", "v_scales") if s[n] is not None}
    if c["op"] == "read":
        k, v = (fa.paged_read(s["k_pages"], s["v_pages"], s["table"], s["len"], s["cu"], s["T"], **kw)
                if own else _read(s))
        return {"k": k, "v": v}
    if own:
        out, _ = fa.attn_paged(s["q"], s["q_norm_w"], s["sinks"], s["k_pages"], s["v_pages"], s["table"], s["len"],
                               s["cu"], max_new=s["max_new"], window=c["window"], use_rope=c["rope"],
                               rope_theta=THETA, eps=EPS, want_lse=False, **kw)
        return {"out": out}
    return {"out": _attn(s)}


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    ctx, new = _lens(c)
    g, ps = c["heads"], c["page"]
    table, d = s["table"].tolist(), torch.float64
    dev = s["cu"].device
    freq = torch.tensor([THETA ** (-2.0 * f / HD) for f in range(HD // 2)], dtype=d, device=dev)

    def prologue(x, w, p0):
        """Weight-form RMSNorm, then the rotation by position of rows [n, heads, 128] at positions p0 ..: complex form."""
        x = x.to(d)
        y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * w.to(d)
        if c["rope"]:
            ang = torch.arange(p0, p0 + x.shape[0], dtype=d, device=dev)[:, None] * freq
            z = torch.complex(y[..., :64].contiguous(), y[..., 64:].contiguous()) * torch.polar(torch.ones_like(ang), ang)[:, None]
            y = torch.cat((z.real, z.imag), -1)
        return y

    def flat(name):
        x = s[name].double()
        return x * s[name[0] + "_scales"].double()[..., None] if c["fp8"] else x

    def two_to(e):
        return ((e.long() + 1023) << 52).view(d)

    def places(i, p0, p1):
        """Page and slot of positions p0 .. p1 - 1 of sequence i."""
        p = torch.arange(p0, p1)
        return torch.tensor(table[i])[p // ps].long().to(dev), (p % ps).to(dev)

    if c["op"] == "append":
        out = {n: s[n].double() for n in ("k_pages", "v_pages", "k_scales", "v_scales") if s[n] is not None}
        t = 0
        for i, (L, n) in enumerate(zip(ctx, new)):
            page, slot = places(i, L, L + n)
            for name, x in (("k", prologue(s["k"][t:t + n], s["k_norm_w"], L)), ("v", s["v"][t:t + n].to(d))):
                if not c["fp8"]:
                    out[name + "_pages"][page, :, slot] = x.half().double() if name == "k" else x
                    continue
                m, x2 = torch.frexp(x.abs().amax(-1) / 448)      # m in [1/2, 1): the quotient is a power of two at 1/2
                e = (x2 - (m == 0.5).int()).clamp(E_MIN, E_MAX)
                sc = two_to(e)
                r = x / sc[..., None]
                # E4M3: 3 mantissa bits, smallest exponent -6, ties to even
                step = two_to(torch.frexp(r.abs().clamp(min=2.0 ** -6))[1] - 4)
                out[name + "_pages"][page, :, slot] = (torch.round(r / step) * step).clamp(-448, 448)
                out[name + "_scales"][page, :, slot] = sc
            t += n
        return out
    kf, vf = flat("k_pages"), flat("v_pages")
    if c["op"] == "read":
        rows = [places(i, L, L + n) for i, (L, n) in enumerate(zip(ctx, new))]
        return {"k": torch.cat([kf[p, :, o] for p, o in rows]), "v": torch.cat([vf[p, :, o] for p, o in rows])}
    outs, t = [], 0
    for i, (L, n) in enumerate(zip(ctx, new)):
        p0 = _first(c, L)
        page, slot = places(i, p0, L + n)
        K, V = kf[page, :, slot], vf[page, :, slot]
        q = prologue(s["q"][t:t + n], s["q_norm_w"], L)
        o = torch.empty(n, g * GROUP, HD, dtype=d, device=dev)
        j = torch.arange(p0, L + n, device=dev)
        p = torch.arange(L, L + n, device=dev)[:, None]
        hide = (j > p) | (j <= p - c["window"]) if c["window"] else j > p
        for h in range(g * GROUP):
            z = (q[:, h] @ K[:, h // GROUP].T / math.sqrt(HD)).masked_fill(hide, -math.inf)
            z = torch.cat((z, s["sinks"][h].to(d).expand(n, 1)), 1)
            o[:, h] = torch.softmax(z, 1)[:, :-1] @ V[:, h // GROUP]
        outs.append(o.reshape(n, -1))
        t += n
    return {"out": torch.cat(outs)}
