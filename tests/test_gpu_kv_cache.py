"""GPU tests of the paged cache: block tables, cache writes, and attention of drafted tokens.

Whole numbers and copies are compared exactly.  Attention's tolerance per element, with u = eps / 2
of the type: e (1 + u) + u |want|, e = u sum|terms| (probabilities rounded for the second product) +
2^-13 sum|terms| (fp32 scores, below 2^5 here, and sums); the result before its own rounding is at
most |want| + e.  2^-25 for float16 subnormals.
"""
import numpy as np
import pytest
import torch

import tensor_core_gemm_multistage_gb300 as gsr
from oracle import llm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    gsr.build()
    yield


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


# ---------------------------------------------------------------------------- block tables

def run_tables(kv, new, free, head, table, page, max_tokens):
    out = {"table": i32(table), "kv_out": i32([-9] * len(kv)), "head_out": i32([-9]), "q_starts": i32([-9] * (len(kv) + 1)),
           "positions": i32([-9] * max_tokens), "slots": i32([-9] * max_tokens), "counts": i32([-9] * 3)}
    gsr.kv_block_tables(i32(kv), i32(new), i32(free), i32([head]), out["table"], page, out["kv_out"], out["head_out"],
                        out["q_starts"], out["positions"], out["slots"], out["counts"])
    want = llm.block_tables(kv, new, free, head, table, page, max_tokens)
    for k, w in want.items():
        assert np.array_equal(out[k].cpu().numpy(), w), k


def tables_case(B, page, ctx, new, seed, short=0, width=1):
    r = np.random.default_rng(seed)
    kv, nw = [int(x) for x in r.integers(0, ctx + 1, B)], [int(x) for x in r.integers(0, new + 1, B)]
    W = max(1, max(-(-(a + n) // page) for a, n in zip(kv, nw)) // width)
    pool = r.permutation(sum(-(-(a + n) // page) for a, n in zip(kv, nw)) + 10)
    table, at = np.full((B, W), -1), 0
    for b in range(B):
        n = min(-(-kv[b] // page), W)
        table[b, :n] = pool[at:at + n]
        at += n
    free = [int(x) for x in pool[at:]]
    return kv, nw, free[:max(1, len(free) // short)] if short else free, table.tolist(), page, sum(nw)


@pytest.mark.parametrize("B,page,ctx,new", [(1, 16, 0, 1), (1, 8, 7, 1), (3, 16, 40, 5), (64, 16, 200, 1), (33, 7, 90, 30),
                                            (700, 32, 100, 9), (8192, 16, 60, 3), (5, 128, 4000, 3000)])
def test_block_tables(B, page, ctx, new):
    kv, nw, free, table, page, total = tables_case(B, page, ctx, new, B + page)
    run_tables(kv, nw, free, 0, table, page, total + 3)
    run_tables(kv, nw, free, 2, table, page, max(total - 2, 0))     # a head inside the list, a map too short


def test_block_tables_run_out_of_pages_and_width():
    kv, nw, free, table, page, total = tables_case(40, 8, 60, 50, 3, short=3)
    run_tables(kv, nw, free, 1, table, page, total)
    kv, nw, free, table, page, total = tables_case(40, 8, 60, 50, 4, width=2)
    kv = [min(a, len(table[0]) * page) for a in kv]
    run_tables(kv, nw, free, 0, table, page, total + 1)
    run_tables([5, 3], [0, 0], [1], 5, [[0], [1]], 8, 2)            # a head behind the list, nothing new
    run_tables([-4, 3], [2, -1], [1, 2], -3, [[9], [8]], 8, 4)      # negative lengths count as 0


# ---------------------------------------------------------------------------- cache writes

@pytest.mark.parametrize("N,H,D,page,dtype", [(1, 1, 64, 16, F16), (5, 2, 128, 8, BF16), (777, 3, 128, 24, F16), (4000, 8, 64, 64, BF16),
                                              (9, 1, 8, 1, F16), (31, 5, 40, 10, F16)])
@pytest.mark.parametrize("layout", ["pages", "heads_first", "one_buffer"])
def test_append(N, H, D, page, dtype, layout):
    g = torch.Generator().manual_seed(N)
    pages = N // page + 3
    if layout == "one_buffer":            # keys and values of a page side by side
        both = torch.zeros(pages, 2, page, H, D, dtype=dtype, device=DEV)
        kc, vc = both[:, 0], both[:, 1]
    elif layout == "heads_first":
        kc, vc = (torch.zeros(pages, H, page, D, dtype=dtype, device=DEV).transpose(1, 2) for _ in range(2))
    else:
        kc, vc = (torch.zeros(pages, page, H, D, dtype=dtype, device=DEV) for _ in range(2))
    if layout == "one_buffer":
        with pytest.raises(gsr.GsrError):
            gsr.kv_cache_append(kc[:1, 0], kc[:1, 0], i32([0]), kc, kc)
    qkv = torch.randn(N, 3 * H, D, generator=g).to(dtype).to(DEV)
    k, v = qkv[:, H:2 * H], qkv[:, 2 * H:]
    slots = torch.randperm(pages * page, generator=g)[:N].to(torch.int32)
    slots[N // 2] = -1
    if N > 3:
        slots[0] = pages * page          # behind the cache: skipped
    kc.fill_(3.0)
    vc.fill_(4.0)
    gsr.kv_cache_append(k, v, slots.to(DEV), kc, vc)
    for cache, new, old in ((kc, k, 3.0), (vc, v, 4.0)):
        want = torch.full((pages * page, H, D), old, dtype=dtype)
        ok = (slots >= 0) & (slots < pages * page)
        want[slots[ok].long()] = new.cpu()[ok]
        assert torch.equal(cache.cpu().reshape(pages * page, H, D), want)


# ---------------------------------------------------------------------------- drafted tokens

class Tree:
    def __init__(self, kv, T, Hq, Hkv, D, page, dtype=F16, cap=0.0, alibi=False, parents="random", seed=0, scale=0.0,
                 layout="pages", extra_rows=0):
        r, g = np.random.default_rng(seed + 5), torch.Generator().manual_seed(seed)
        self.kv, self.T, self.page = kv, T, page
        B = len(kv)
        need = [-(-n // page) for n in kv]
        pool = sum(need) + 3
        order = [int(x) for x in r.permutation(pool)]
        self.table = np.full((B, max(need + [1]) + 1), -1)
        at = 0
        for b in range(B):
            self.table[b, :need[b]] = order[at:at + need[b]]
            at += need[b]
        self.starts = np.concatenate([[0], np.cumsum(T)])
        N = int(self.starts[-1]) + extra_rows
        shape = (pool, page, Hkv, D) if layout == "pages" else (pool, Hkv, page, D)
        self.kc, self.vc = (torch.randn(shape, generator=g).to(dtype).to(DEV) for _ in range(2))
        if layout != "pages":
            self.kc, self.vc = self.kc.transpose(1, 2), self.vc.transpose(1, 2)
        self.q = (torch.randn(N, Hq, D, generator=g) * 1.5).to(dtype).to(DEV)
        self.parents = None
        if parents == "random":
            self.parents = [int(r.integers(-1, t)) if t else -1 for n in T for t in range(n)] + [-1] * extra_rows
        elif parents == "flat":
            self.parents = [-1] * N
        self.slopes = (2.0 ** -torch.linspace(1, 8, Hq)).to(DEV) if alibi else None
        self.cap, self.scale, self.max_nodes, self.N = cap, scale, max(T + [1]), N
        self.u, self.tiny = torch.finfo(dtype).eps / 2, 2.0 ** -25 if dtype == F16 else 0.0

    def run(self, stream=None, workspace=None):
        self.o = torch.full_like(self.q, 7.0)
        self.args = (self.q, self.kc, self.vc, i32(self.table), i32(self.kv), i32(self.starts),
                     None if self.parents is None else i32(self.parents), self.o, self.max_nodes)
        self.kw = dict(softmax_scale=self.scale, softcap=self.cap, alibi_slopes=self.slopes)
        gsr.tree_attention_fwd(*self.args, **self.kw, stream=stream, workspace=workspace)
        status, code = gsr.device_status(stream)
        assert status == gsr.Status.OK, hex(code)
        return self

    def check(self, rows=None):
        """`rows`: the rows that are compared (the others may hold NaN)."""
        want, terms = llm.tree_attention(self.q, self.kc, self.vc, self.table, self.kv, self.starts, self.parents, self.scale,
                                         self.cap, None if self.slopes is None else self.slopes.cpu().numpy(), self.max_nodes)
        got = llm.f64(self.o)
        if rows is not None:
            got, want, terms = got[rows], want[rows], terms[rows]
        real = ~np.isnan(want)
        assert np.all(got[~real] == 7.0), "rows of no request were written"
        got, want, terms = got[real], want[real], terms[real]
        assert not np.isnan(got).any()
        tol = (self.u + 2.0 ** -13) * terms * (1 + self.u) + self.u * np.abs(want) + self.tiny
        assert np.all(np.abs(got - want) <= tol), (np.abs(got - want).max(), (np.abs(got - want) / np.maximum(tol, 1e-30)).max())
        return self


TREES = {
    "one_token": dict(kv=[1], T=[1], Hq=1, Hkv=1, D=64, page=8),
    "one_token_no_group": dict(kv=[300], T=[1], Hq=4, Hkv=4, D=128, page=16, dtype=BF16),
    "decode_batch": dict(kv=[1, 128, 129, 1000, 57, 640], T=[1] * 6, Hq=16, Hkv=4, D=128, page=16, dtype=BF16),
    "decode_long": dict(kv=[9000, 20], T=[1, 1], Hq=8, Hkv=1, D=64, page=64),
    "decode_many": dict(kv=list(range(1, 300, 3)), T=[1] * 100, Hq=8, Hkv=2, D=64, page=16),
    "trees": dict(kv=[200, 77, 513], T=[7, 20, 64], Hq=8, Hkv=2, D=128, page=32),
    "trees_only": dict(kv=[5, 64, 1], T=[5, 64, 1], Hq=4, Hkv=1, D=64, page=8, dtype=BF16),
    "trees_cap_alibi": dict(kv=[300, 41], T=[30, 9], Hq=6, Hkv=2, D=64, page=16, cap=3.0, alibi=True),
    "trees_alibi": dict(kv=[150, 260], T=[40, 3], Hq=4, Hkv=2, D=128, page=16, alibi=True, dtype=BF16),
    "chain": dict(kv=[257, 130], T=[33, 2], Hq=5, Hkv=1, D=128, page=128, parents="chain"),
    "chain_alibi_cap": dict(kv=[257, 130], T=[33, 2], Hq=4, Hkv=1, D=64, page=24, parents="chain", alibi=True, cap=5.0),
    "flat": dict(kv=[140], T=[64], Hq=8, Hkv=1, D=64, page=16, parents="flat"),
    "large_group": dict(kv=[333], T=[3], Hq=96, Hkv=1, D=64, page=16),
    "odd_group": dict(kv=[333, 90], T=[50, 26], Hq=21, Hkv=3, D=128, page=40),
    "large_page": dict(kv=[700, 300], T=[2, 10], Hq=8, Hkv=2, D=64, page=256),
    "odd_large_page": dict(kv=[700, 300], T=[2, 10], Hq=8, Hkv=2, D=64, page=136),
    "some_without_rows": dict(kv=[100, 0, 50, 8], T=[3, 0, 0, 1], Hq=4, Hkv=2, D=64, page=16),
    "heads_first": dict(kv=[220, 31], T=[4, 1], Hq=4, Hkv=2, D=128, page=16, layout="heads"),
    "negative_scale": dict(kv=[220, 31], T=[4, 1], Hq=4, Hkv=2, D=128, page=16, scale=-0.1),
    "rows_behind": dict(kv=[220, 31], T=[4, 1], Hq=4, Hkv=2, D=128, page=16, extra_rows=5),
}


@pytest.mark.parametrize("name", TREES)
def test_tree_attention(name):
    Tree(**TREES[name]).run().check()


def _random_trees(n, seed):
    r = np.random.default_rng(seed)
    out = []
    for _ in range(n):
        B = int(r.integers(1, 9))
        T = [int(x) for x in r.integers(0, int(r.choice([2, 9, 65])), B)]
        out.append(dict(kv=[t + int(x) for t, x in zip(T, r.integers(0, int(r.choice([50, 900])), B))], T=T,
                        Hkv=int(r.choice([1, 2, 3])), D=int(r.choice([64, 128])), page=int(r.choice([8, 16, 32, 48, 64])),
                        dtype=[F16, BF16][int(r.integers(2))], cap=float(r.choice([0.0, 2.0])), alibi=bool(r.integers(2)),
                        parents=str(r.choice(["random", "chain", "flat"])), seed=int(r.integers(100))))
        out[-1]["Hq"] = out[-1]["Hkv"] * int(r.choice([1, 3, 8]))
    return out


@pytest.mark.parametrize("c", _random_trees(14, 11))
def test_random_trees(c):
    Tree(**c).run().check()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_rows_nothing_sees_have_no_influence(bad):
    t = Tree(kv=[100, 131, 40], T=[5, 12, 1], Hq=8, Hkv=2, D=64, page=16)
    clean = t.run().check().o.clone()
    used = {(int(t.table[b][j // 16]), j % 16) for b, n in enumerate(t.kv) for j in range(n)}
    for pg in range(t.kc.shape[0]):
        for row in range(16):
            if (pg, row) not in used:
                t.kc[pg, row] = bad
                t.vc[pg, row] = bad
    assert torch.equal(t.run().o, clean)
    # a sibling no other node sees: only its own row changes
    t.parents[5 + 11] = t.parents[5 + 10] = -1
    t.run().check()
    j = t.kv[1] - 1
    t.kc[int(t.table[1][j // 16]), j % 16] = bad
    t.vc[int(t.table[1][j // 16]), j % 16] = bad
    t.run().check([n for n in range(t.N) if n != 5 + 11])
    if bad != bad:
        assert torch.isnan(t.o[5 + 11]).all()


def test_pages_outside_the_pool_hold_nothing():
    t = Tree(kv=[300, 90], T=[6, 1], Hq=4, Hkv=2, D=64, page=16)
    t.table[0][2], t.table[0][9], t.table[1][0] = -1, 10 ** 6, -(2 ** 31)
    t.run().check()
    t.table[1][:] = -1                    # a request whose every page is missing: O = 0
    t.run().check()
    assert torch.all(t.o[6] == 0)


def test_lengths_the_table_cannot_hold_are_cut():
    t = Tree(kv=[60, 30], T=[2, 1], Hq=2, Hkv=1, D=64, page=16)
    t.table = t.table[:, :2].copy()       # 32 of 60 tokens
    t.run().check()


def test_nodes_behind_the_limit_are_left():
    t = Tree(kv=[60, 30], T=[6, 3], Hq=2, Hkv=1, D=64, page=16, parents="chain")
    t.max_nodes = 4
    t.run().check()


def test_repeatable_and_on_two_streams_at_once():
    ts = [Tree(kv=[5000, 300, 77], T=[1, 8, 30], Hq=8, Hkv=2, D=128, page=16, seed=1),
          Tree(kv=[900] * 9, T=[2] * 9, Hq=16, Hkv=4, D=64, page=32, dtype=BF16, seed=2)]
    first = [t.run().o.clone() for t in ts]
    streams = [torch.cuda.Stream(DEV), torch.cuda.Stream(DEV)]
    torch.cuda.synchronize()
    for _ in range(4):
        for t, s in zip(ts, streams):
            gsr.tree_attention_fwd(*t.args, **t.kw, stream=s)
    for s in streams:
        assert gsr.device_status(s)[0] == gsr.Status.OK
    assert all(torch.equal(t.o, f) for t, f in zip(ts, first))


@pytest.mark.parametrize("T", [1, 40])
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right(T):
    t = Tree(kv=[900, 200], T=[T, T], Hq=8, Hkv=2, D=64, page=16).run()
    gsr.set_wait_timeout_ns(50_000_000)
    gsr.set_test_flags(1)                          # the first query tile is never copied
    try:
        gsr.tree_attention_fwd(*t.args, **t.kw)
        status, code = gsr.device_status()
    finally:
        gsr.set_test_flags(0)
        gsr.set_wait_timeout_ns(1_000_000_000)
    assert status == gsr.Status.ERR_DEVICE_TIMEOUT and code & 0xF00 == 0x700
    t.run().check()


@pytest.mark.parametrize("kv,T,Hq,Hkv", [([1 + 7 * i % 128 for i in range(1500)], [1] * 1500, 16, 8),
                                         ([40 + 11 * i % 90 for i in range(600)], [1 + 5 * i % 39 for i in range(600)], 16, 2)])
def test_many_short_items_of_one_cta(kv, T, Hq, Hkv):
    """Items of one or two key tiles follow one another on every CTA: one item's rows are read before the next one's
    products overwrite them, so all runs give the same bits."""
    t = Tree(kv=kv, T=T, Hq=Hq, Hkv=Hkv, D=64, page=16, dtype=BF16).run().check()
    want = t.o.clone()
    for _ in range(50):
        for _ in range(10):
            t.o.fill_(7.0)
            gsr.tree_attention_fwd(*t.args, **t.kw)
        assert gsr.device_status()[0] == gsr.Status.OK and torch.equal(t.o, want)


def test_workspaces():
    t = Tree(kv=[3000, 77], T=[1, 9], Hq=8, Hkv=2, D=128, page=16).run().check()
    want = t.o.clone()
    size = gsr.tree_attention_workspace(2, t.N, 8, 2, 128, t.kc.shape[0], 16, t.table.shape[1], t.max_nodes)
    own = torch.full((size + 64,), 255, dtype=torch.uint8, device=DEV)
    assert torch.equal(t.run(workspace=own[:size]).o, want) and torch.all(own[size:] == 255)
    s = torch.cuda.Stream(DEV)
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(2):
        t.o.fill_(7.0)
        torch.cuda.synchronize()
        gsr.tree_attention_fwd(*t.args, **t.kw, stream=s)
        assert gsr.device_status(s)[0] == gsr.Status.OK and torch.equal(t.o, want)
        gsr.release_stream(s)
    with pytest.raises(gsr.GsrError):
        t.run(workspace=own[:size - 16])


def test_a_cache_past_32_bits():
    """The last pages of a cache of more than 2^31 elements: written and read as in a small one."""
    t = Tree(kv=[150, 61], T=[3, 1], Hq=8, Hkv=8, D=128, page=16, dtype=BF16).run().check()
    want, pool = t.o.clone(), t.kc.shape[0]
    pages = 2 ** 31 // (16 * 8 * 128) + pool
    kc, vc = (torch.empty(pages, 16, 8, 128, dtype=BF16, device=DEV) for _ in range(2))
    k, v = (x.reshape(-1, 8, 128) for x in (t.kc, t.vc))
    first = pages - pool
    gsr.kv_cache_append(k, v, torch.arange(first * 16, pages * 16, dtype=torch.int32, device=DEV), kc, vc)
    assert torch.equal(kc[first:], t.kc) and torch.equal(vc[first:], t.vc)
    t.kc, t.vc = kc, vc
    t.table[t.table >= 0] += first
    assert torch.equal(t.run().o, want)


def test_rows_of_no_request():
    t = Tree(kv=[40, 9], T=[0, 0], Hq=4, Hkv=2, D=64, page=16, extra_rows=6).run()
    assert torch.all(t.o == 7.0)


# ---------------------------------------------------------------------------- infinities and NaN that some nodes see

def check_natural(t):
    """The formula in fp64 with infinities and NaN taking their course among the keys that a node sees."""
    q, kc, vc, got = (llm.f64(x) for x in (t.q, t.kc, t.vc, t.o))
    N, Hq, D = q.shape
    Hkv, pages, slopes = kc.shape[2], kc.shape[0], None if t.slopes is None else t.slopes.cpu().double().numpy()
    for b, kv in enumerate(t.kv):
        s, T = int(t.starts[b]), t.T[b]
        ctx = kv - T
        for u in range(T):
            chain = [u]
            while True:
                up = chain[-1] - 1 if t.parents is None else t.parents[s + chain[-1]]
                if up < 0 or up >= chain[-1]:
                    break
                chain.append(up)
            keys = [(j, j) for j in range(ctx)] + [(ctx + c, ctx + d) for d, c in enumerate(reversed(chain))]
            pg, off, at = np.array([(int(t.table[b][j // t.page]), j % t.page, where) for j, where in keys]).T
            for h in range(Hq):
                k, v = kc[pg, off, h * Hkv // Hq], vc[pg, off, h * Hkv // Hq]
                with np.errstate(invalid="ignore"):
                    x = k @ q[s + u, h] * (t.scale or D ** -0.5)
                    if t.cap:
                        x = t.cap * np.tanh(x / t.cap)
                    if slopes is not None:
                        x = x - slopes[h] * (ctx + len(chain) - 1 - at)
                    p = np.exp(x - x.max())
                    p /= p.sum()
                clean = np.where(np.isfinite(v), v, 0.0)
                want, terms = p @ clean, p @ np.abs(clean)
                plus, minus = ((np.isnan(v) | (v == i)).any(0) for i in (np.inf, -np.inf))
                bad, y = plus | minus | ~np.isfinite(want), got[s + u, h]
                assert np.array_equal(bad, ~np.isfinite(y)), (b, u, h)
                if slopes is None and np.isfinite(want).all():       # with a bias a weight may be 0
                    assert np.all(y[plus & ~minus] == np.inf) and np.all(y[minus & ~plus] == -np.inf)
                assert np.isnan(y[plus & minus]).all()
                tol = (t.u + 2.0 ** -13) * terms * (1 + t.u) + t.u * np.abs(want) + t.tiny
                assert np.all((np.abs(y - want) <= tol)[~bad])


@pytest.mark.parametrize("what", ["V", "K", "nodes"])
@pytest.mark.parametrize("name", ["trees", "trees_only", "trees_cap_alibi", "trees_alibi", "chain", "chain_alibi_cap", "flat", "large_group",
                                  "odd_group", "odd_large_page", "decode_batch", "heads_first"])
def test_infinite_and_nan_values_reach_the_nodes_that_see_them(name, what):
    t = Tree(**TREES[name])
    r, values = np.random.default_rng(4), [float("inf"), float("nan"), -float("inf")]
    for i in range(12):
        b = int(r.integers(len(t.kv)))
        low = t.kv[b] - t.T[b] if what == "nodes" else 0         # a key of the request, or one of its nodes
        j = int(r.integers(low, t.kv[b]))
        at = int(t.table[b][j // t.page]), j % t.page, int(r.integers(t.kc.shape[2]))
        if what == "K" and i < 2:
            t.kc[at + (int(r.integers(t.kc.shape[3])),)] = float("nan")
        elif what == "nodes" and i == 0:
            t.vc[at] = float("nan")
        elif what != "K":
            t.vc[at + (int(r.integers(t.kc.shape[3])),)] = values[i % 3]
    t.run()
    check_natural(t)


@pytest.mark.parametrize("Hq,Hkv,T", [(16, 2, 40), (21, 3, 26), (4, 2, 9)])
def test_infinite_values_among_the_nodes_give_the_same_every_time(Hq, Hkv, T):
    # two query tiles a request, each with its softmax group, and one: whoever cleans a tile first, all rows know
    t = Tree(kv=[90 + 7 * i % 60 for i in range(100)], T=[T] * 100, Hq=Hq, Hkv=Hkv, D=64, page=40)
    for b in range(100):
        j = t.kv[b] - 1 - b % T
        t.vc[int(t.table[b][j // 40]), j % 40, :, b % 64] = float("inf" if b % 2 else "nan")
    want = t.run().o.clone()
    check_natural(t)
    for _ in range(50):
        for _ in range(6):
            t.o.fill_(7.0)
            gsr.tree_attention_fwd(*t.args, **t.kw)
        assert gsr.device_status()[0] == gsr.Status.OK and torch.equal(t.o.nan_to_num(5.0), want.nan_to_num(5.0))


@pytest.mark.parametrize("T", [1, 40])
def test_an_infinite_value_takes_no_longer(T):
    # long contexts: no wait of 0.02 s runs out, and all other columns keep their bits
    t = Tree(kv=[30000, 20000, 30000], T=[T, T, 1], Hq=16, Hkv=2, D=128, page=64, parents="flat")
    clean = t.run().o.clone()
    t.vc[int(t.table[0][3]), 5, :, 7] = float("inf")              # a key that request 0's nodes all see
    j = t.kv[1] - 1                                              # request 1's last node: itself alone
    t.vc[int(t.table[1][j // 64]), j % 64, :, 9] = float("nan")
    gsr.set_wait_timeout_ns(20_000_000)
    try:
        t.run()
    finally:
        gsr.set_wait_timeout_ns(1_000_000_000)
    assert torch.all(t.o[:T, :, 7] == float("inf")) and torch.all(t.o[2 * T - 1, :, 9].isnan())
    t.o[:T, :, 7], t.o[2 * T - 1, :, 9] = clean[:T, :, 7], clean[2 * T - 1, :, 9]
    assert torch.equal(t.o, clean)


# ---------------------------------------------------------------------------- the path together

@pytest.mark.parametrize("captured", [False, True])
def test_serving_steps_equal_the_whole_sequence(captured):
    """Prompts, then steps of drafted chains: block tables, cache writes and attention of each step on
    the device alone, against masked attention over the whole sequence."""
    B, Hq, Hkv, D, page, W, pool = 3, 8, 2, 64, 16, 12, 40
    g = torch.Generator().manual_seed(21)
    total = [100, 61, 140]
    S = max(total)
    q = torch.randn(B, S, Hq, D, generator=g).to(F16).to(DEV)
    k, v = (torch.randn(B, S, Hkv, D, generator=g).to(F16).to(DEV) for _ in range(2))
    bounds = i32([[0, n] for n in total])
    whole = torch.empty_like(q).transpose(1, 2).contiguous()
    gsr.masked_attention_fwd(q.transpose(1, 2), k.transpose(1, 2), v.transpose(1, 2), whole, causal=True, doc_bounds=bounds)
    kc, vc = (torch.full((pool, page, Hkv, D), float("nan"), dtype=F16, device=DEV) for _ in range(2))
    free = torch.randperm(pool, generator=g).to(torch.int32).to(DEV)
    lens, head, table = [i32([0] * B), i32([0] * B)], [i32([0]), i32([0])], torch.full((B, W), -1, dtype=torch.int32, device=DEV)
    N = 40
    starts, pos, slots, counts, new = i32([0] * (B + 1)), i32([0] * N), i32([0] * N), i32([0] * 3), i32([0] * B)
    tok = dict(q=torch.empty(N, Hq, D, dtype=F16, device=DEV), k=torch.empty(N, Hkv, D, dtype=F16, device=DEV),
               v=torch.empty(N, Hkv, D, dtype=F16, device=DEV), o=torch.empty(N, Hq, D, dtype=F16, device=DEV))

    def step(a):
        gsr.kv_block_tables(lens[a], new, free, head[a], table, page, lens[1 - a], head[1 - a], starts, pos, slots, counts)
        req = torch.searchsorted(starts[1:].contiguous(), torch.arange(N, device=DEV, dtype=torch.int32), right=True).clamp(max=B - 1)
        at = pos.clamp(min=0).long()
        for name, src in (("q", q), ("k", k), ("v", v)):
            tok[name].copy_(src[req, at])
        gsr.kv_cache_append(tok["k"], tok["v"], slots, kc, vc)
        gsr.tree_attention_fwd(tok["q"], kc, vc, table, lens[1 - a], starts, None, tok["o"], 64)

    graphs = []
    if captured:
        side = torch.cuda.Stream(DEV)
        with torch.cuda.stream(side):
            step(0)                       # nothing new: the stream's error word and the kernels
        side.synchronize()
        for a in range(2):
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1], stream=side):
                step(a)
    done, a = [0] * B, 0
    plan = [[13, 1, 20], [13, 9, 10]] + [[1, 1, 1], [5, 2, 0], [7, 3, 9]] * 14
    for news in plan:
        news = [min(n, t - d) for n, t, d in zip(news, total, done)]
        new.copy_(i32(news))
        tok["o"].fill_(7.0)
        torch.cuda.synchronize()
        graphs[a].replay() if captured else step(a)
        assert counts.tolist()[0] == sum(news) and counts.tolist()[2] == 0
        n = 0
        for b in range(B):
            for d in range(news[b]):
                want = whole[b, :, done[b] + d].float()
                # both sides round P and O: twice the bound of one, with |V| below 6
                assert torch.all((tok["o"][n].float() - want).abs() <= 4 * 2.0 ** -11 * 2.0 + 2.0 ** -10 * want.abs())
                n += 1
            done[b] += news[b]
        assert torch.all(tok["o"][n:] == 7.0)
        a = 1 - a
    assert done == total
