"""The paged operators at the sizes where a kernel's rule takes another form
(GPU): tokens a warp of append (2,048, 4,096, 16,384 tokens) and read (65,536,
too), plans of more than 1,024 groups, shares whose boundaries move by more than
a chunk, and small keys through the chunk kernel.  Tolerances are
test_paged.py's."""
import numpy as np
import pytest
import torch

from tests.paged_cases import Case
from tests.test_paged import append, attend, check_append, check_attend, fa  # noqa: F401

pytestmark = pytest.mark.gpu


def ragged(T, seed, most):
    """Rows of sequences that sum to T: many short ones, some empty, one long;
    no part of an eight or thirty-two token run is theirs alone."""
    r = np.random.default_rng(seed)
    n = []
    while sum(n) < T - T // 4:
        n.append(int(r.integers(0, most)) if r.random() < 0.8 else 0)
    n.insert(len(n) // 2, T // 4)
    n[-1] -= max(0, sum(n) - T)
    n += [0, T - sum(n), 0]
    assert sum(n) == T and min(n) >= 0
    return n


class Pool:
    """Pages with random contents for sequences of n[b] rows at start[b]."""

    def __init__(self, n, start, g, ps, fp8, seed):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        r = np.random.default_rng(seed)
        last = [(s + k - 1) // ps if k else -1 for s, k in zip(start, n)]
        P = sum(last) + len(last) + 1
        order = r.permutation(P)
        table, at = np.full((len(n), max(last) + 2), -1, np.int32), 0
        for b, z in enumerate(last):
            table[b, :z + 1] = order[at:at + z + 1]
            at += z + 1
        i32 = dict(dtype=torch.int32, device="cuda")
        self.table, self.start = torch.from_numpy(table).cuda(), torch.tensor(start, **i32)
        self.cu = torch.tensor(np.concatenate([[0], np.cumsum(n)]), **i32)
        self.ps, self.T, self.n, self.fp8 = ps, sum(n), n, fp8
        x = [torch.randn(P, g, ps, 128, generator=gen, device="cuda") for _ in range(2)]
        if fp8:
            self.kp, self.vp = (y.clamp(-448, 448).to(torch.float8_e4m3fn) for y in x)
            self.ks, self.vs = (torch.randint(115, 132, (P, g, ps), generator=gen, device="cuda", dtype=torch.uint8)
                                .view(torch.float8_e8m0fnu) for _ in range(2))
        else:
            self.kp, self.vp, self.ks, self.vs = x[0].half(), x[1].bfloat16(), None, None

    def places(self):
        b = torch.repeat_interleave(torch.arange(len(self.n), device="cuda"), torch.tensor(self.n, device="cuda"))
        pos = self.start[b] + torch.arange(self.T, device="cuda") - self.cu[b]
        return self.table[b, pos // self.ps].long(), (pos % self.ps).long()

    def pools(self):
        return [x for x in (self.kp, self.vp, self.ks, self.vs) if x is not None]

    def scales(self):
        return dict(k_scales=self.ks, v_scales=self.vs)


SIZES = [2047, 2048, 4095, 4096, 16383, 16384]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("g", [1, 2, 4])
@pytest.mark.parametrize("T", SIZES + [65535, 65536, 65543])
def test_read(fa, T, g, fp8):  # noqa: F811
    n = ragged(T, T + g, 24)
    c = Pool(n, [i % 37 for i in range(len(n))], g, 16, fp8, T)
    k = torch.full((T + 3, g, 128), 9.0, dtype=torch.float16, device="cuda")
    v = torch.full((T + 3, g, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    fa.paged_read(c.kp, c.vp, c.table, c.start, c.cu, T + 3, k=k, v=v, **c.scales())
    assert fa.device_status(fa.paged_read.last_workspace) == 0
    page, slot = c.places()
    for got, pages, sc, dt in ((k, c.kp, c.ks, torch.float16), (v, c.vp, c.vs, torch.bfloat16)):
        if fp8:
            x = pages.view(torch.uint8)[page, :, slot].view(torch.float8_e4m3fn).float()
            e = sc.view(torch.uint8)[page, :, slot].int()
            want = (x * (e << 23).view(torch.float32)[..., None]).to(dt)
        else:
            want = pages[page, :, slot]
        assert torch.equal(got[:T], want) and (got[T:] == 9).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("g", [1, 2, 4])
@pytest.mark.parametrize("T", SIZES + [20001])
def test_append(fa, T, g, fp8):  # noqa: F811
    """The pools after one long call are those after calls of under 2,048
    tokens each (which test_paged.py compares with the oracle), bit for bit."""
    n = ragged(T, T + g, 24)
    gen = torch.Generator(device="cuda").manual_seed(T)
    k, v = (torch.randn(T + 3, g, 128, generator=gen, device="cuda").bfloat16() for _ in range(2))
    w = 1 + 0.1 * torch.randn(128, generator=gen, device="cuda")
    start = [(i * 7) % 41 for i in range(len(n))]
    a, b = Pool(n, start, g, 16, fp8, T), Pool(n, start, g, 16, fp8, T)
    fa.paged_append(k, v, w, a.kp, a.vp, a.table, a.start, a.cu, **a.scales())
    assert fa.device_status(fa.paged_append.last_workspace) == 0
    cu = a.cu.tolist()
    for s, rows in enumerate(n):
        for x in range(0, rows, 2000):                    # a long sequence in parts
            m = min(2000, rows - x)
            i32 = dict(dtype=torch.int32, device="cuda")
            fa.paged_append(k[cu[s] + x:cu[s] + x + m], v[cu[s] + x:cu[s] + x + m], w, b.kp, b.vp, b.table[s:s + 1],
                            torch.tensor([start[s] + x], **i32), torch.tensor([0, m], **i32), **b.scales())
    for x, y in zip(a.pools(), b.pools()):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


@pytest.mark.parametrize("fp8", [False, True])
def test_append_against_the_oracle(fa, fp8):  # noqa: F811
    c = Case([5] * 40, [int(x) for x in np.random.default_rng(51).integers(0, 110, 40)], g=1, fp8=fp8, rope=True, seed=52)
    assert c.rows >= 2048                                 # two tokens a warp (at least four rows of one head)
    t = c.to("cuda")
    assert append(fa, c, t) == 0
    check_append(c, t)


def sources(fa, c, t, fp8):
    """The chunk kernel's calls: in the usual workspace (8-bit pages: expanded
    first), and on chip."""
    yield {}
    if fp8:
        need = fa.paged_workspace_bytes(c.B, c.T, int(max(c.new.max(), 9)), c.table.shape[1], c.ps, kv_heads=c.g, window=c.window)
        yield {"workspace": torch.empty(need, dtype=torch.uint8, device="cuda")}


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("window", [0, 33])
def test_more_than_1024_groups(fa, window, fp8):  # noqa: F811
    r = np.random.default_rng(53)
    ctx, new = r.integers(0, 200, 2200).tolist(), r.integers(0, 2, 2200).tolist()
    ctx[1500], new[1500] = 3000, 200
    c = Case(ctx, new, g=1, ps=16, fp8=fp8, window=window, rope=window > 0, seed=54)
    assert sum((x + 31) // 32 for x in new) > 1024
    t = c.to("cuda")
    assert append(fa, c, t) == 0
    for kw in sources(fa, c, t, fp8):
        st, out, lse = attend(fa, c, t, **kw)
        assert st == 0
        check_attend(c, t, out, lse, chunk=True)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("ctx", [2300, 4700])
def test_share_boundaries_move_by_chunks(fa, ctx, fp8):  # noqa: F811
    """Two pairs a CTA or more, of 18 (37) chunks: a boundary within 2 (4)
    chunks of a pair's end moves there."""
    B = 80
    r = np.random.default_rng(55)
    c = Case([ctx + int(x) for x in r.integers(-60, 60, B)], [int(x) for x in r.integers(1, 3, B)], ps=128, fp8=fp8, seed=56)
    pairs, chunks = 4 * B, 4 * sum((x + 127) // 128 for x in c.ctx)
    assert pairs >= 2 * 148 and chunks // (16 * 148) >= (2 if ctx < 4000 else 4)
    t = c.to("cuda")
    assert append(fa, c, t) == 0
    for kw in sources(fa, c, t, fp8):
        st, out, lse = attend(fa, c, t, max_new=9, **kw)
        assert st == 0
        check_attend(c, t, out, lse, chunk=True)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("w_scale,v_scale", [(4.0, 1.0), (1e-3, 1.0), (1.0, 1e4), (1.0, 1e-4)])
def test_large_and_small_rows_in_chunks(fa, w_scale, v_scale, fp8):  # noqa: F811
    """With w_scale 1e-3 the 8-bit keys' scales are below 2^-15: the chunk
    kernel rounds those keys to FP16's subnormals, by at most 2^-25 an element,
    which moves a logit by less than 2^-25 x 128 x 4e-3 / sqrt(128): nothing
    beside the 2e-5 of every logit."""
    c = Case([200, 70, 513], [12, 33, 2], ps=16, fp8=fp8, seed=57, w_scale=w_scale, v_scale=v_scale)
    t = c.to("cuda")
    assert append(fa, c, t) == 0
    check_append(c, t)
    if fp8 and w_scale == 1e-3:
        page, slot = c.slots()
        assert (t["k_scales"].cpu().view(torch.uint8)[page, :, slot] < 127 - 15).any()
    for kw in sources(fa, c, t, fp8):
        st, out, lse = attend(fa, c, t, **kw)
        assert st == 0
        check_attend(c, t, out, lse, chunk=True)
