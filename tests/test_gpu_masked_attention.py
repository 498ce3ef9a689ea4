"""GPU parity of masked_attention_fwd and _bwd against the fp64 oracle.

Tolerances, from the arithmetic: with u = eps / 2 of the operands' type, a probability (or dS) is
rounded once to that type before the matrix product, and the result once at the end, so per element
    |got - want| <= e (1 + u) + u |want|,   e = u sum|terms| + small,
where the sum runs over the rounded factor's terms (the result before its own rounding is off by at
most e, so it is at most |want| + e, and its rounding adds u times that).  `small` covers fp32: a score is a sum of D
products in fp32 (D 2^-24 relative to sum|q k| at worst, scores here below 2^5 in absolute terms)
and a probability's relative error equals its score's absolute one: 2^-13 of the sum of |terms| is
above all of it, as is 2^-13 of the terms of dS's own two parts.  In float16 a result below 2^-14
is subnormal: its rounding is 2^-25 absolute.  So are P and dS there, after the powers of two they are
scaled by: 2^12, and for dS at least 2^14 over 2 max|dO_i| max|V_j|, each error entering once per term.  lse is fp32 throughout: 2^-14 absolute for scores
below 2^5 and distance biases below 2^9 (2^-24 relative, a few roundings).
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


def make(B, H, n, D, dtype, g, order="bhsd", scale=1.0):
    x = (torch.randn(B, H, n, D, generator=g) * scale).to(dtype).to(DEV)
    if order == "bshd":
        return x.transpose(1, 2).contiguous().transpose(1, 2)
    if order == "hbsd":
        return x.transpose(0, 1).contiguous().transpose(0, 1)
    return x


class Case:
    def __init__(self, B, Hq, Hkv, Sq, Skv, D, dtype=F16, causal=False, docs=None, prefix=None, cap=0.0, alibi=False,
                 scale=0.0, order="bhsd", seed=0, grad=1.0):
        g = torch.Generator().manual_seed(seed * 1000 + Sq + 7 * Skv + D)
        self.q, self.k, self.v = (make(B, h, n, D, dtype, g, order, s) for h, n, s in
                                  ((Hq, Sq, 1.5), (Hkv, Skv, 1.0), (Hkv, Skv, 1.0)))
        self.do = make(B, Hq, Sq, D, dtype, g, order, grad)
        self.docs, self.prefix, self.causal, self.cap, self.scale = docs, prefix, causal, cap, scale
        self.slopes = (2.0 ** -torch.linspace(1, 8, Hq)).to(DEV) if alibi else None
        self.see = llm.visible(B, Sq, Skv, causal, docs, prefix)
        self.kw = dict(softmax_scale=scale, causal=causal, softcap=cap, alibi_slopes=self.slopes,
                       doc_bounds=None if docs is None else torch.tensor(docs, dtype=torch.int32, device=DEV),
                       prefix_lens=None if prefix is None else torch.tensor(prefix, dtype=torch.int32, device=DEV))
        self.u = torch.finfo(dtype).eps / 2
        self.tiny = 2.0 ** -25 if dtype == F16 else 0.0
        self.host = dict(scale=float(np.float32(scale)), cap=float(np.float32(cap)),
                         slopes=None if self.slopes is None else self.slopes.cpu().numpy())

    def tol(self, want, terms, wide):
        return (self.u * terms + 2.0 ** -13 * wide) * (1 + self.u) + self.u * np.abs(want) + self.tiny

    def forward(self):
        self.o = torch.full_like(self.q, float("nan"))
        self.lse = torch.full(self.q.shape[:3], float("nan"), device=DEV)
        gsr.masked_attention_fwd(self.q, self.k, self.v, self.o, self.lse, **self.kw)
        status, code = gsr.device_status()
        assert status == gsr.Status.OK, hex(code)
        return self

    def backward(self):
        self.grads = [torch.full_like(t, float("nan")) for t in (self.q, self.k, self.v)]
        gsr.masked_attention_bwd(self.do, self.q, self.k, self.v, self.o, self.lse, *self.grads, **self.kw)
        status, code = gsr.device_status()
        assert status == gsr.Status.OK, hex(code)
        return self

    def check_forward(self, rows=slice(None)):
        """`rows`: the query rows that are compared (the others may hold NaN)."""
        want, lse, terms = (t[:, :, rows] for t in llm.masked_attention(self.q, self.k, self.v, self.see, **self.host))
        got = llm.f64(self.o)[:, :, rows]
        assert not np.isnan(got).any(), "unwritten or NaN outputs"
        assert np.all(np.abs(got - want) <= self.tol(want, terms, terms)), np.abs(got - want).max()
        gl = llm.f64(self.lse)[:, :, rows]
        fin = np.isfinite(lse)
        assert np.array_equal(np.isneginf(gl), ~fin) and not np.isnan(gl).any()
        assert np.all(np.abs(gl[fin] - lse[fin]) <= 2.0 ** -14), np.abs(gl[fin] - lse[fin]).max()
        return self

    def check_backward(self, rows=slice(None)):
        want, terms, wide, plain = llm.masked_attention_bwd(self.do, self.q, self.k, self.v, self.o, self.lse, self.see, **self.host)
        norm = lambda t: np.sqrt((np.nan_to_num(llm.f64(t), nan=0.0, posinf=0.0, neginf=0.0) ** 2).sum(-1)).max()
        low = [self.tiny * 2 * norm(self.do) * norm(self.v) * 2.0 ** -14] * 2 + [self.tiny * 2.0 ** -12]
        for name, t, w, a, b, c, x in zip(("dQ", "dK", "dV"), self.grads, want, terms, wide, plain, low):
            got, w, a, b, c = (y[:, :, rows] for y in (llm.f64(t), w, a, b, c))
            assert not np.isnan(got).any(), name
            tol = self.tol(w, a, b) + x * c
            assert np.all(np.abs(got - w) <= tol), (name, np.abs(got - w).max(), (np.abs(got - w) / tol).max())
        return self

    def check(self):
        return self.forward().check_forward().backward().check_backward()


CASES = {
    "one_key": dict(B=1, Hq=1, Hkv=1, Sq=1, Skv=1, D=64),
    "one_query": dict(B=2, Hq=8, Hkv=2, Sq=1, Skv=515, D=128, causal=True, dtype=BF16),
    "tile": dict(B=1, Hq=2, Hkv=2, Sq=128, Skv=128, D=128),
    "full_odd": dict(B=2, Hq=3, Hkv=1, Sq=333, Skv=200, D=64, order="bshd"),
    "causal_odd": dict(B=1, Hq=4, Hkv=2, Sq=385, Skv=385, D=128, causal=True, dtype=BF16),
    "causal_more_keys": dict(B=1, Hq=2, Hkv=1, Sq=100, Skv=333, D=64, causal=True, order="hbsd"),
    "causal_more_queries": dict(B=1, Hq=2, Hkv=2, Sq=400, Skv=130, D=128, causal=True),
    "docs": dict(B=2, Hq=4, Hkv=2, Sq=500, Skv=500, D=64, docs=[[0, 3, 200, 200, 500], [0, 100, 257, 300, 411]], causal=True),
    "docs_two_way": dict(B=1, Hq=2, Hkv=1, Sq=700, Skv=700, D=128, docs=[[0, 127, 128, 129, 390, 700]], dtype=BF16),
    "docs_padding_in_front": dict(B=1, Hq=2, Hkv=1, Sq=300, Skv=300, D=64, docs=[[140, 150, 290]]),
    "docs_none_left": dict(B=2, Hq=2, Hkv=1, Sq=150, Skv=150, D=64, docs=[[0, 0, 0], [0, 0, 150]]),
    "padded_batch": dict(B=4, Hq=2, Hkv=2, Sq=260, Skv=260, D=128, docs=[[0, 260], [0, 1], [0, 129], [0, 0]], dtype=BF16),
    "prefix": dict(B=3, Hq=4, Hkv=4, Sq=270, Skv=270, D=64, causal=True, prefix=[0, 131, 400]),
    "prefix_more_queries": dict(B=1, Hq=1, Hkv=1, Sq=300, Skv=140, D=64, causal=True, prefix=[37]),
    "prefix_docs": dict(B=1, Hq=4, Hkv=1, Sq=520, Skv=520, D=128, causal=True, docs=[[0, 130, 400, 515]], prefix=[[20, 200, 500]]),
    "cap": dict(B=1, Hq=4, Hkv=2, Sq=300, Skv=300, D=128, cap=2.0, causal=True),
    "cap_saturated": dict(B=1, Hq=2, Hkv=2, Sq=200, Skv=200, D=64, cap=0.5, scale=2.0, dtype=BF16),
    "alibi": dict(B=1, Hq=8, Hkv=2, Sq=400, Skv=400, D=64, alibi=True, causal=True, dtype=BF16),
    "alibi_two_way": dict(B=1, Hq=4, Hkv=4, Sq=200, Skv=330, D=128, alibi=True),
    "all": dict(B=2, Hq=6, Hkv=2, Sq=390, Skv=390, D=128, cap=3.0, alibi=True, causal=True, order="bshd", dtype=BF16,
                docs=[[0, 200, 380], [5, 6, 390]], prefix=[[50, 10], [1, 300]]),
    "negative_scale": dict(B=1, Hq=2, Hkv=1, Sq=200, Skv=200, D=64, scale=-0.2, causal=True),
    "peaked": dict(B=1, Hq=2, Hkv=2, Sq=257, Skv=257, D=64, scale=0.4),
    "many_items": dict(B=2, Hq=48, Hkv=24, Sq=520, Skv=520, D=64, causal=True),
    "one_kv_head": dict(B=1, Hq=32, Hkv=1, Sq=520, Skv=520, D=128, causal=True, dtype=BF16),
    "one_kv_head_docs": dict(B=1, Hq=24, Hkv=1, Sq=700, Skv=700, D=64, docs=[[3, 40, 600, 690]]),
    "few_kv_heads": dict(B=1, Hq=16, Hkv=2, Sq=1000, Skv=700, D=64, causal=True, cap=4.0),
    "few_queries": dict(B=1, Hq=4, Hkv=2, Sq=3, Skv=5000, D=128, causal=True, dtype=BF16),
    "few_queries_two_way": dict(B=2, Hq=2, Hkv=1, Sq=130, Skv=2600, D=64, cap=3.0),
    "few_heads": dict(B=1, Hq=2, Hkv=1, Sq=1500, Skv=1500, D=128, causal=True, alibi=True, prefix=[300]),
    "few_heads_docs": dict(B=1, Hq=2, Hkv=2, Sq=2000, Skv=2000, D=64, causal=True, docs=[[3, 900, 901, 1990]], dtype=BF16),
    "far_keys_capped": dict(B=1, Hq=2, Hkv=2, Sq=21, Skv=16808, D=64, causal=True, cap=2.0, alibi=True, seed=42),
    "small_gradients": dict(B=1, Hq=2, Hkv=1, Sq=600, Skv=600, D=128, grad=2.0 ** -11),
    "large_gradients": dict(B=1, Hq=2, Hkv=1, Sq=300, Skv=300, D=64, grad=2.0 ** 7, causal=True),
}


@pytest.mark.parametrize("name", CASES)
def test_parity(name):
    Case(**CASES[name]).check()


def _random_cases(n, seed):
    r = np.random.default_rng(seed)
    out = []
    for _ in range(n):
        B, Hkv, g = int(r.integers(1, 3)), int(r.integers(1, 4)), int(r.choice([1, 2, 5]))
        S = int(r.integers(1, 600))
        c = dict(B=B, Hq=Hkv * g, Hkv=Hkv, Sq=S, Skv=S, D=int(r.choice([64, 128])), seed=int(r.integers(1000)),
                 dtype=[F16, BF16][int(r.integers(2))], order=str(r.choice(["bhsd", "bshd", "hbsd"])),
                 cap=float(r.choice([0.0, 0.0, 4.0])), alibi=bool(r.integers(2)))
        kind = r.integers(4)
        if kind == 0:
            c["Skv"], c["causal"] = int(r.integers(1, 700)), bool(r.integers(2))
        elif kind == 1:
            c["causal"], c["prefix"] = True, [int(x) for x in r.integers(0, S + 2, B)]
        else:
            n_docs = int(r.integers(1, 6))
            c["docs"] = [sorted(int(x) for x in r.integers(0, S + 1, n_docs + 1)) for _ in range(B)]
            c["causal"] = bool(r.integers(2))
            if c["causal"] and kind == 3:
                c["prefix"] = [[int(x) for x in r.integers(0, S, n_docs)] for _ in range(B)]
        out.append(c)
    return out


@pytest.mark.parametrize("c", _random_cases(14, 77))
def test_random_cases(c):
    Case(**c).check()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("D", [64, 128])
def test_masked_positions_have_no_influence(bad, D):
    # padding, and a whole document: whatever they hold, the others' results are what they were
    docs = [[0, 70, 200, 290]]
    c = Case(1, 4, 2, 300, 300, D, docs=docs, causal=True)
    for rows in (slice(290, 300), slice(70, 200)):
        for t in (c.q, c.k, c.v, c.do):
            t[:, :, rows] = bad
    keep = np.r_[0:70, 200:300]
    c.forward().check_forward(keep).backward().check_backward(keep)
    assert torch.all(c.o[:, :, 290:] == 0) and torch.all(c.lse[:, :, 290:] == -float("inf"))
    assert all(torch.all(t[:, :, 290:] == 0) for t in c.grads)


@pytest.mark.parametrize("D", [64, 128])
def test_later_keys_have_no_influence(D):
    # causal: a NaN from position 200 on reaches no earlier query, inside the same tile either
    c = Case(1, 2, 1, 260, 260, D, causal=True)
    clean = Case(1, 2, 1, 260, 260, D, causal=True).forward()
    for t in (c.k, c.v):
        t[:, :, 200:] = float("nan")
    c.forward().check_forward(slice(0, 200))
    assert torch.all((c.lse[:, :, :200] - clean.lse[:, :, :200]).abs() <= 2.0 ** -13)
    assert torch.isnan(c.o[:, :, 200:]).all()


def test_padding_rows_of_the_gradient():
    # rows without keys may hold anything in dO and in the given O
    c = Case(2, 4, 2, 200, 200, 64, docs=[[0, 150], [0, 200]])
    c.forward()
    c.do[0, :, 150:] = float("nan")
    c.o[0, :, 150:] = float("inf")
    c.backward()
    c.o[0, :, 150:] = 0
    c.do[0, :, 150:] = 0
    c.check_backward()


def test_fused_projection_views():
    # Q, K, V and their gradients as the parts of one buffer; O in (batch, row, head) order
    B, S, Hq, Hkv, D = 2, 150, 4, 2, 64
    g = torch.Generator().manual_seed(9)
    qkv = torch.randn(B, S, Hq + 2 * Hkv, D, generator=g).to(F16).to(DEV)
    dqkv = torch.full_like(qkv, float("nan"))
    part = lambda t: [x.transpose(1, 2) for x in t.split([Hq, Hkv, Hkv], 2)]
    c = Case(B, Hq, Hkv, S, S, D, causal=True)
    (c.q, c.k, c.v), grads = part(qkv), part(dqkv)
    c.do = torch.randn(B, S, Hq, D, generator=g).to(F16).to(DEV).transpose(1, 2)
    c.o, c.lse = torch.empty_like(c.do), torch.empty(B, Hq, S, device=DEV)
    gsr.masked_attention_fwd(c.q, c.k, c.v, c.o, c.lse, **c.kw)
    gsr.masked_attention_bwd(c.do, c.q, c.k, c.v, c.o, c.lse, *grads, **c.kw)
    c.grads = grads
    c.check_forward().check_backward()
    with pytest.raises(gsr.GsrError) as e:      # in place of an input
        gsr.masked_attention_fwd(c.q, c.k, c.v, c.q, c.lse, **c.kw)
    assert e.value.status == gsr.Status.ERR_ALIAS


def test_rows_behind_the_output_view_are_left():
    # O is a view of a wider buffer: what lies between its rows stays
    buf = torch.full((1, 100, 3, 64), 7.0, dtype=F16, device=DEV)
    c = Case(1, 2, 1, 100, 100, 64)
    c.o, c.lse = buf[:, :, :2].transpose(1, 2), torch.empty(1, 2, 100, device=DEV)
    gsr.masked_attention_fwd(c.q, c.k, c.v, c.o, c.lse, **c.kw)
    c.check_forward()
    assert torch.all(buf[:, :, 2] == 7.0)


def test_no_keys_and_no_queries():
    q = torch.randn(1, 2, 5, 64, device=DEV, dtype=F16)
    none = torch.empty(1, 1, 0, 64, device=DEV, dtype=F16)
    o, lse = torch.full_like(q, float("nan")), torch.zeros(1, 2, 5, device=DEV)
    gsr.masked_attention_fwd(q, none, none, o, lse)
    assert torch.all(o == 0) and torch.all(lse == -float("inf"))
    dq = torch.full_like(q, float("nan"))
    gsr.masked_attention_bwd(q, q, none, none, o, lse, dq, none.clone(), none.clone())
    assert torch.all(dq == 0)
    k = torch.randn(1, 1, 9, 64, device=DEV, dtype=F16)
    noq = torch.empty(1, 2, 0, 64, device=DEV, dtype=F16)
    dk, dv = torch.full_like(k, float("nan")), torch.full_like(k, float("nan"))
    gsr.masked_attention_bwd(noq, noq, k, k, noq, torch.empty(1, 2, 0, device=DEV), noq.clone(), dk, dv)
    assert torch.all(dk == 0) and torch.all(dv == 0)
    gsr.masked_attention_fwd(noq, k, k, noq.clone())


def test_one_query_equals_the_last_row():
    c = Case(2, 4, 2, 300, 300, 64, causal=True, cap=3.0, alibi=True).forward()
    o1, l1 = torch.empty_like(c.q[:, :, -1:]).contiguous(), torch.empty(2, 4, 1, device=DEV)
    gsr.masked_attention_fwd(c.q[:, :, -1:], c.k, c.v, o1, l1, **c.kw)
    _, _, terms = llm.masked_attention(c.q, c.k, c.v, c.see, **c.host)       # each within the bound of check_forward
    tol = 2 * c.tol(llm.f64(o1), terms[:, :, -1:], terms[:, :, -1:])
    assert np.all(np.abs(llm.f64(o1) - llm.f64(c.o[:, :, -1:])) <= tol)
    assert torch.all((l1 - c.lse[:, :, -1:]).abs() <= 2.0 ** -13)


def test_repeatable_and_on_two_streams_at_once():
    cases = [Case(2, 8, 2, 700, 700, 128, causal=True, seed=1), Case(1, 6, 3, 555, 555, 64, dtype=BF16, cap=5.0, seed=2)]
    for c in cases:
        c.forward().backward()
    first = [[t.clone() for t in (c.o, c.lse, *c.grads)] for c in cases]
    streams = [torch.cuda.Stream(DEV), torch.cuda.Stream(DEV)]
    torch.cuda.synchronize()
    for _ in range(3):
        for c, s in zip(cases, streams):
            gsr.masked_attention_fwd(c.q, c.k, c.v, c.o, c.lse, stream=s, **c.kw)
            gsr.masked_attention_bwd(c.do, c.q, c.k, c.v, c.o, c.lse, *c.grads, stream=s, **c.kw)
    for s in streams:
        assert gsr.device_status(s)[0] == gsr.Status.OK
    for c, want in zip(cases, first):
        for a, b in zip((c.o, c.lse, *c.grads), want):
            assert torch.equal(a, b)


def test_two_captured_graphs_replayed_at_once():
    cases = [Case(1, 8, 2, 512, 512, 128, causal=True, seed=3), Case(1, 4, 4, 640, 640, 128, docs=[[0, 300, 640]], seed=4)]
    graphs, first = [], []
    side = torch.cuda.Stream(DEV)
    for c in cases:
        c.forward().backward()
        first.append([t.clone() for t in (c.o, *c.grads)])
        with torch.cuda.stream(side):
            gsr.masked_attention_fwd(c.q, c.k, c.v, c.o, c.lse, **c.kw)    # the stream's error word
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            gsr.masked_attention_fwd(c.q, c.k, c.v, c.o, c.lse, **c.kw)
            gsr.masked_attention_bwd(c.do, c.q, c.k, c.v, c.o, c.lse, *c.grads, **c.kw)
        graphs.append(graph)
    for c in cases:
        for t in (c.o, c.lse, *c.grads):
            t.fill_(float("nan"))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(DEV), torch.cuda.Stream(DEV)]
    for graph, s in zip(graphs, streams):
        with torch.cuda.stream(s):
            for _ in range(3):
                graph.replay()
    torch.cuda.synchronize()
    for c, want in zip(cases, first):
        assert all(torch.equal(a, b) for a, b in zip((c.o, *c.grads), want))


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_padding_values_do_not_reach_the_gradients_scale(dtype):
    # large finite values where nothing looks: not a bit of the result changes
    c = Case(1, 4, 2, 300, 300, 64, dtype=dtype, docs=[[10, 100, 290]], causal=True)
    pads = (slice(0, 10), slice(290, 300))
    for value in (0.0, 60000.0):
        for rows in pads:
            for t in (c.q, c.k, c.v, c.do):
                t[:, :, rows] = value
        c.forward().check_forward().backward().check_backward()
        got = [t.clone() for t in (c.o, *c.grads)]
        if value:
            assert all(torch.equal(a, b) for a, b in zip(got, first))
        first = got


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("backward", [False, True])
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right(D, backward):
    c = Case(1, 2, 1, 700, 700, D, causal=True).forward()
    gsr.set_wait_timeout_ns(50_000_000)
    gsr.set_test_flags(1)                          # each kernel's first copy is never made
    try:
        if backward:
            gsr.masked_attention_bwd(c.do, c.q, c.k, c.v, c.o, c.lse, *(torch.empty_like(t) for t in (c.q, c.k, c.v)), **c.kw)
        else:
            gsr.masked_attention_fwd(c.q, c.k, c.v, torch.empty_like(c.o), None, **c.kw)
        status, code = gsr.device_status()
    finally:
        gsr.set_test_flags(0)
        gsr.set_wait_timeout_ns(1_000_000_000)
    assert status == gsr.Status.ERR_DEVICE_TIMEOUT and code & 0xF00 in ((0x500, 0x600) if backward else (0x400,))
    c.check()


def test_workspaces():
    """The caller's, the library's of two streams, one that grows, one released: the same gradients."""
    c = Case(1, 8, 2, 500, 500, 64, causal=True).forward().backward()
    want = [t.clone() for t in c.grads]

    def run(**kw):
        for t in c.grads:
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        gsr.masked_attention_bwd(c.do, c.q, c.k, c.v, c.o, c.lse, *c.grads, **c.kw, **kw)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(c.grads, want))

    size = gsr.masked_attention_bwd_workspace(1, 8, 2, 500, 500, 64)
    own = torch.full((max(size, 2 ** 24) + 64,), 255, dtype=torch.uint8, device=DEV)     # NaN everywhere
    run(workspace=own[:size])
    s = torch.cuda.Stream(DEV)
    run(workspace=own[:2 ** 24], stream=s)
    assert torch.all(own[2 ** 24:] == 255)
    run(stream=s)
    big = Case(2, 8, 2, 900, 900, 128).forward()
    gsr.masked_attention_bwd(big.do, big.q, big.k, big.v, big.o, big.lse, *(torch.empty_like(t) for t in (big.q, big.k, big.v)),
                             stream=s)
    run(stream=s)
    gsr.release_stream(s)
    run(stream=s)
    with pytest.raises(gsr.GsrError):
        run(workspace=own[:size - 256])


def test_a_capture_needs_a_workspace_of_its_own():
    # through the C interface NULL is refused, since the library's may be freed under the graph; the
    # capture goes on
    from tensor_core_gemm_multistage_gb300 import llm as L
    c = Case(1, 4, 2, 300, 300, 64, causal=True).forward().backward()
    want = [t.clone() for t in c.grads]
    d, qs, ks, dev = L._attention_desc(c.q, c.k, 0.0, True, 0.0, None, None, None)
    q, k = (lambda t: L._operand(t, "t", qs, t.dtype, dev)), (lambda t: L._operand(t, "t", ks, t.dtype, dev))
    side = torch.cuda.Stream(DEV)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        gsr.masked_attention_bwd(c.do, c.q, c.k, c.v, c.o, c.lse, *c.grads, **c.kw)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        s = gsr.lib().masked_attention_bwd(d, q(c.do), q(c.q), k(c.k), k(c.v), q(c.o), c.lse.data_ptr(), q(c.grads[0]),
                                           k(c.grads[1]), k(c.grads[2]), None, 0, side.cuda_stream)
        gsr.masked_attention_bwd(c.do, c.q, c.k, c.v, c.o, c.lse, *c.grads, **c.kw)
    assert s == gsr.Status.ERR_INVALID_ARG
    for t in c.grads:
        t.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(c.grads, want))


@pytest.mark.parametrize("handle", [False, True])
def test_a_captured_stream_that_is_not_the_current_one(handle):
    # the workspace comes from the graph's memory where the given stream is captured
    c = Case(1, 4, 2, 300, 300, 64, causal=True).forward().backward()
    want = [t.clone() for t in c.grads]
    side, other = torch.cuda.Stream(DEV), torch.cuda.Stream(DEV)
    given = side.cuda_stream if handle else side
    torch.cuda.synchronize()
    gsr.masked_attention_bwd(c.do, c.q, c.k, c.v, c.o, c.lse, *c.grads, stream=given, **c.kw)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        with torch.cuda.stream(other):
            gsr.masked_attention_bwd(c.do, c.q, c.k, c.v, c.o, c.lse, *c.grads, stream=given, **c.kw)
    big = Case(2, 8, 2, 900, 900, 128).forward()              # the library's workspace of the stream grows meanwhile
    gsr.masked_attention_bwd(big.do, big.q, big.k, big.v, big.o, big.lse, *(torch.empty_like(t) for t in (big.q, big.k, big.v)), stream=given)
    for _ in range(2):
        for t in c.grads:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(c.grads, want))


def test_threads_on_one_stream():
    """Two threads' backward calls on one stream share its workspace: each call's launches stay together."""
    import threading
    cases = [Case(1, 4, 2, 600, 600, 64, causal=True, seed=5), Case(1, 4, 4, 333, 333, 128, seed=6, dtype=BF16)]
    for c in cases:
        c.forward().backward()
    want = [[t.clone() for t in c.grads] for c in cases]
    wrong = []

    def loop(c, w):
        try:
            for _ in range(20):
                grads = [torch.full_like(t, float("nan")) for t in c.grads]
                gsr.masked_attention_bwd(c.do, c.q, c.k, c.v, c.o, c.lse, *grads, **c.kw)
                wrong.extend(not torch.equal(a, b) for a, b in zip(grads, w))
        except Exception as e:
            wrong.append(e)

    threads = [threading.Thread(target=loop, args=a) for a in zip(cases, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(wrong) == 120 and not any(wrong), wrong


def test_threads_on_the_per_thread_stream():
    """One handle, a stream of each thread's: calls that run at the same time have workspaces of their own."""
    import threading
    per_thread = 2                        # cudaStreamPerThread
    cases = [Case(1, 8, 2, 600, 600, 64, causal=True, seed=5), Case(1, 4, 4, 633, 633, 128, seed=6, dtype=BF16)]
    for c in cases:
        c.forward().backward()
    want = [[t.clone() for t in c.grads] for c in cases]
    outs = [[[torch.full_like(t, float("nan")) for t in c.grads] for _ in range(40)] for c in cases]
    torch.cuda.synchronize()
    status, together = [], threading.Barrier(2)

    def loop(c, grads):
        try:
            together.wait()
            for g in grads:
                gsr.masked_attention_bwd(c.do, c.q, c.k, c.v, c.o, c.lse, *g, stream=per_thread, **c.kw)
            status.append(gsr.device_status(per_thread)[0])
            gsr.release_stream(per_thread)
        except Exception as e:
            status.append(e)

    threads = [threading.Thread(target=loop, args=a) for a in zip(cases, outs)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert status == [gsr.Status.OK] * 2, status
    for w, grads in zip(want, outs):
        for g in grads:
            assert all(torch.equal(a, b) for a, b in zip(g, w))


def test_offsets_past_32_bits():
    """A batch row 2^31 elements behind the first, all operands the parts of one buffer: the results of
    dense copies."""
    B, H, S, D, parts = 2, 2, 260, 64, 8
    pitch = parts * H * D
    step = (2 ** 31 // pitch + 1) * pitch
    buf = torch.empty(step + S * pitch, dtype=F16, device=DEV)
    view = lambda i: buf.as_strided((B, H, S, D), (step, D, pitch, 1), i * H * D)
    c = Case(B, H, H, S, S, D, causal=True).forward().backward()
    q, k, v, do, o, dq, dk, dv = (view(i) for i in range(parts))
    for to, t in ((q, c.q), (k, c.k), (v, c.v), (do, c.do)):
        to.copy_(t)
    lse = torch.empty_like(c.lse)
    gsr.masked_attention_fwd(q, k, v, o, lse, **c.kw)
    gsr.masked_attention_bwd(do, q, k, v, o, lse, dq, dk, dv, **c.kw)
    assert torch.equal(lse, c.lse)
    for a, b in zip((o, dq, dk, dv), (c.o, *c.grads)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype,scale", [(F16, 0.3), (BF16, 0.3)])
def test_capped_scores_large_and_small(dtype, scale):
    # rows whose scores stay far below the cap next to rows far beyond it, in one tile
    c = Case(1, 2, 1, 300, 300, 64, cap=4.0, scale=scale, dtype=dtype, causal=True)
    c.q[:, :, ::3] *= 0.01
    c.q[:, :, 1::7] *= 8
    c.check()


@pytest.mark.parametrize("D,dtype", [(64, BF16), (128, F16)])
def test_many_backward_calls_finish_alike(D, dtype):
    # hundreds of launches next to one another: every wait ends, and no result depends on who was first
    c = Case(4, 16, 8, 1024, 1024, D, dtype=dtype, causal=True).forward().backward()
    want = [t.clone() for t in c.grads]
    for _ in range(10):
        for _ in range(60):
            gsr.masked_attention_bwd(c.do, c.q, c.k, c.v, c.o, c.lse, *c.grads, **c.kw)
        status, code = gsr.device_status()
        assert status == gsr.Status.OK, hex(code)
        assert all(torch.equal(a, b) for a, b in zip(c.grads, want))


@pytest.mark.parametrize("D", [64, 128])
def test_nan_everywhere_is_not_slow(D):
    # rows that are NaN by themselves are not computed key by key: no wait of 0.1 s runs out
    S = 32768
    q, k, v, do = (torch.full((1, 1, S, D), float("nan"), dtype=BF16, device=DEV) for _ in range(4))
    o, lse = torch.zeros_like(q), torch.zeros(1, 1, S, device=DEV)
    grads = [torch.zeros_like(q) for _ in range(3)]
    gsr.set_wait_timeout_ns(100_000_000)
    try:
        gsr.masked_attention_fwd(q, k, v, o, lse, causal=True)
        gsr.masked_attention_bwd(do, q, k, v, o, lse, *grads, causal=True)
        status, code = gsr.device_status()
    finally:
        gsr.set_wait_timeout_ns(1_000_000_000)
    assert status == gsr.Status.OK, hex(code)
    assert all(torch.isnan(t).all() for t in (o, lse, *grads))


@pytest.mark.parametrize("D", [64, 128])
def test_keys_in_parts(D):
    """Few queries over many keys: with the library's workspace, the caller's, in a graph; NaN among keys that
    nothing sees, and in one that all see."""
    c = Case(1, 4, 2, 5, 6000, D, causal=True, cap=2.0).forward().check_forward()
    want = c.o.clone()
    size = gsr.masked_attention_fwd_workspace(1, 4, 2, 5, 6000, D)
    own = torch.full((size + 64,), 255, dtype=torch.uint8, device=DEV)
    c.o.fill_(float("nan"))
    gsr.masked_attention_fwd(c.q, c.k, c.v, c.o, c.lse, workspace=own[:size], **c.kw)
    assert torch.equal(c.o, want) and torch.all(own[size:] == 255)
    with pytest.raises(gsr.GsrError):
        gsr.masked_attention_fwd(c.q, c.k, c.v, c.o, c.lse, workspace=own[:size // 64], **c.kw)
    side = torch.cuda.Stream(DEV)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        gsr.masked_attention_fwd(c.q, c.k, c.v, c.o, c.lse, **c.kw)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        gsr.masked_attention_fwd(c.q, c.k, c.v, c.o, c.lse, **c.kw)
    c.o.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(c.o, want)
    c.k[:, :, 5997:] = float("nan")               # the last three queries alone see it
    c.v[:, :, 5997:] = float("nan")
    c.forward().check_forward(slice(0, 2))
    assert torch.isnan(c.o[:, :, 2:]).all()
    c.k[:, :, 100] = float("nan")
    c.forward()
    assert torch.isnan(c.o).all()


# ---------------------------------------------------------------------------- infinities and NaN that some rows see

def natural(c):
    """O and lse of the formula in fp64, infinities and NaN taking their course among the pairs that a row sees:
    (O with what is not finite left out of V, whether each element meets +inf or NaN, -inf or NaN, sum of |terms|, lse)."""
    B, Hq, Sq, D = c.q.shape
    g, Skv, see = Hq // c.k.shape[1], c.k.shape[2], torch.tensor(c.see, device=DEV)[:, None]
    k, v = (t.double().repeat_interleave(g, 1) for t in (c.k, c.v))
    x = c.q.double() @ k.transpose(-1, -2) * (c.scale or D ** -0.5)
    if c.cap:
        x = c.cap * torch.tanh(x / c.cap)
    if c.slopes is not None:
        dist = torch.arange(Sq, device=DEV)[:, None] + Skv - Sq - torch.arange(Skv, device=DEV)
        x = x - c.slopes.double()[None, :, None, None] * dist.abs()
    x = torch.where(see, x, -torch.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top == -torch.inf, 0.0, top))
    l = p.sum(-1, keepdim=True)
    w = torch.where(see, p / torch.where(l == 0, 1.0, l), 0.0)
    clean = torch.where(v.isfinite(), v, 0.0)
    seen = see.double()
    plus, minus = ((seen @ ((v == s) | v.isnan()).double()) > 0 for s in (torch.inf, -torch.inf))
    return w @ clean, plus, minus, w @ clean.abs(), torch.where(top == -torch.inf, 0.0, top)[..., 0] + l[..., 0].log()


def check_natural(c):
    o, plus, minus, terms, lse = (t.cpu() for t in natural(c))
    got, gl = c.o.double().cpu(), c.lse.double().cpu()
    special = plus | minus | ~o.isfinite()
    assert torch.equal(special, ~got.isfinite())
    ok = ~special
    tol = torch.from_numpy(c.tol(o.numpy(), terms.numpy(), terms.numpy()))
    assert torch.all(((got - o).abs() <= tol)[ok])
    if c.slopes is None:                     # with a bias a weight may be 0, and 0 inf is NaN
        assert torch.all(got[plus & ~minus & o.isfinite()] == torch.inf)
        assert torch.all(got[minus & ~plus & o.isfinite()] == -torch.inf)
    assert torch.all(got[plus & minus].isnan())
    assert torch.equal(gl.isnan(), lse.isnan()) and torch.equal(gl.isneginf(), lse.isneginf())
    fin = lse.isfinite()
    assert torch.all((gl - lse)[fin].abs() <= 2.0 ** -14)


SPECIAL = {
    "causal": dict(B=1, Hq=4, Hkv=2, Sq=700, Skv=700, D=128, causal=True),
    "causal_short": dict(B=2, Hq=2, Hkv=1, Sq=100, Skv=300, D=64, causal=True, dtype=BF16),
    "two_way": dict(B=1, Hq=2, Hkv=2, Sq=300, Skv=515, D=64),
    "docs": dict(B=2, Hq=4, Hkv=2, Sq=500, Skv=500, D=64, docs=[[0, 3, 200, 200, 480], [7, 100, 257, 300, 411]], causal=True),
    "docs_two_way": dict(B=1, Hq=2, Hkv=1, Sq=700, Skv=700, D=128, docs=[[10, 127, 128, 129, 390, 690]], dtype=BF16),
    "prefix": dict(B=3, Hq=2, Hkv=2, Sq=400, Skv=400, D=64, causal=True, prefix=[0, 131, 300]),
    "alibi": dict(B=1, Hq=4, Hkv=2, Sq=640, Skv=640, D=128, causal=True, alibi=True, dtype=BF16),
    "cap": dict(B=1, Hq=2, Hkv=1, Sq=400, Skv=400, D=128, causal=True, cap=3.0),
    "all": dict(B=2, Hq=6, Hkv=2, Sq=390, Skv=390, D=64, cap=3.0, alibi=True, causal=True, order="bshd", dtype=BF16,
                docs=[[0, 200, 380], [5, 6, 390]], prefix=[[50, 10], [1, 300]]),
    "parts": dict(B=1, Hq=2, Hkv=1, Sq=5, Skv=6000, D=128, causal=True),
    "parts_capped": dict(B=1, Hq=2, Hkv=1, Sq=300, Skv=4000, D=64, causal=True, cap=2.0, alibi=True, dtype=BF16),
}


def spoil(t, n, values, seed):
    """Puts `n` of the values at random places."""
    r = np.random.default_rng(seed)
    for i in range(n):
        t[tuple(int(r.integers(0, k)) for k in t.shape)] = values[i % len(values)]


@pytest.mark.parametrize("name", SPECIAL)
def test_infinite_and_nan_values_reach_the_rows_that_see_them(name):
    # elements of V, and one whole row of it: the columns of the rows that see them and nothing else
    c = Case(**SPECIAL[name])
    spoil(c.v, 12, [float("inf"), float("nan"), -float("inf")], 3)
    c.v[0, 0, c.v.shape[2] // 2] = float("nan")
    c.forward()
    check_natural(c)


@pytest.mark.parametrize("name", SPECIAL)
def test_infinite_and_nan_queries_and_keys(name):
    c = Case(**SPECIAL[name])
    spoil(c.q, 3, [float("inf"), float("nan")], 5)
    spoil(c.k, 3, [float("nan"), -float("inf")], 6)
    c.forward()
    check_natural(c)


@pytest.mark.parametrize("D,dtype", [(128, F16), (64, BF16)])
def test_an_infinite_value_takes_no_longer(D, dtype):
    """One infinity in V, and V of NaN behind the last document, in rows of 32768 tokens: no wait of 0.02 s runs out,
    and all other results keep their bits."""
    S = 32768
    g = torch.Generator(device=DEV).manual_seed(D)
    q = torch.randn(1, 4, S, D, generator=g, device=DEV).to(dtype)
    k, v = (torch.randn(1, 1, S, D, generator=g, device=DEV).to(dtype) for _ in range(2))
    bounds = torch.tensor([[0, S - 100]], dtype=torch.int32, device=DEV)

    def run(**kw):
        o, lse = torch.empty_like(q), torch.empty(1, 4, S, device=DEV)
        gsr.masked_attention_fwd(q, k, v, o, lse, **kw)
        status, code = gsr.device_status()
        assert status == gsr.Status.OK, hex(code)
        return o, lse

    cases = (dict(causal=True), dict(doc_bounds=bounds))
    clean = [run(**kw) for kw in cases]
    v[0, 0, 200, 5] = float("inf")
    v[0, 0, S - 100:] = float("nan")
    gsr.set_wait_timeout_ns(20_000_000)
    try:
        got = [run(**kw) for kw in cases]
    finally:
        gsr.set_wait_timeout_ns(1_000_000_000)
    for (o, lse), (o0, lse0) in zip(got, clean):
        assert torch.equal(lse, lse0)
        o0[:, :, S - 100:] = o[:, :, S - 100:]
        first = 200 if o is got[0][0] else 0
        assert torch.all(o[:, :, first:S - 100, 5] == float("inf"))
        o0[:, :, first:, 5] = o[:, :, first:, 5]
        assert torch.equal(o.nan_to_num(7.0), o0.nan_to_num(7.0))
    assert got[0][0][:, :, S - 100:].isnan().all() and torch.all(got[1][0][:, :, S - 100:] == 0)


def test_infinities_in_every_item():
    # far more items on each CTA than its list of items to run again holds
    g = torch.Generator(device=DEV).manual_seed(1)
    q = torch.randn(24, 64, 1024, 64, generator=g, device=DEV).half()
    k, v = (torch.randn(24, 2, 1024, 64, generator=g, device=DEV).half() for _ in range(2))
    o, clean, lse, lse0 = torch.empty_like(q), torch.empty_like(q), *(torch.empty(24, 64, 1024, device=DEV) for _ in range(2))
    gsr.masked_attention_fwd(q, k, v, clean, lse0, causal=True)
    v[..., 3] = float("inf")
    for _ in range(3):
        gsr.masked_attention_fwd(q, k, v, o, lse, causal=True)
        status, code = gsr.device_status()
        assert status == gsr.Status.OK, hex(code)
        clean[..., 3] = float("inf")
        assert torch.equal(o, clean) and torch.equal(lse, lse0)


def check_natural_backward(c):
    """The gradients' formulas in fp64 with the given lse and O, infinities and NaN taking their course among the pairs
    that see each other; rows whose lse is -inf add nothing of their own.  Tolerances as in check_backward."""
    B, Hq, Sq, D = c.q.shape
    Hkv, Skv = c.k.shape[1:3]
    g, see = Hq // Hkv, torch.tensor(c.see, device=DEV)[:, None]
    q, do, o, lse = (t.double() for t in (c.q, c.do, c.o, c.lse))
    k, v = (t.double().repeat_interleave(g, 1) for t in (c.k, c.v))
    clean = lambda t: torch.where(t.isfinite(), t, 0.0)
    scale = c.scale or D ** -0.5
    x = q @ k.transpose(-1, -2) * scale
    t = torch.zeros_like(x)
    if c.cap:
        t = torch.tanh(x / c.cap)
        x = c.cap * t
    if c.slopes is not None:
        dist = torch.arange(Sq, device=DEV)[:, None] + Skv - Sq - torch.arange(Skv, device=DEV)
        x = x - c.slopes.double()[None, :, None, None] * dist.abs()
    none = (lse == -torch.inf)[..., None] | ~see
    P = torch.where(none, 0.0, torch.exp(x - lse[..., None]))
    dP, delta = do @ v.transpose(-1, -2), (do * o).sum(-1, keepdim=True)
    dS = torch.where(none, 0.0, P * (dP - delta) * (1 - t * t))
    aS = clean(P * (clean(do).abs() @ clean(v).abs().transpose(-1, -2) + clean(do * o).abs().sum(-1, keepdim=True)))
    fold = lambda a: a.reshape(B, Hkv, g, Skv, D).sum(2)
    T, seen = (lambda a: a.transpose(-1, -2)), see.expand(B, Hq, Sq, Skv).double()
    meets = lambda a, y: (a @ (~y.isfinite()).double()) > 0          # a pair that sees something not finite
    want = (scale * dS @ clean(k), scale * fold(T(dS) @ clean(q)), fold(T(P) @ clean(do)))
    special = (meets(seen, k), fold(meets(T(seen), q).double()) > 0, fold(meets(T(seen), do).double()) > 0)
    mags = [(scale * a @ clean(k).abs(), scale * fold(T(a) @ clean(q).abs())) for a in (clean(dS).abs(), aS, seen)]
    last = fold(T(clean(P)) @ clean(do).abs())
    norm = lambda y: clean(y).norm(dim=-1).max().item()
    low = [c.tiny * 2 * norm(do) * norm(v) * 2.0 ** -14] * 2 + [c.tiny * 2.0 ** -12]
    for i, (got, w, sp) in enumerate(zip(c.grads, want, special)):
        got, bad = got.double(), sp | ~w.isfinite()
        assert torch.equal(bad, ~got.isfinite()), ("dQ dK dV".split()[i], (bad != ~got.isfinite()).sum().item())
        a, b, plain = (m[i] for m in mags) if i < 2 else (last, last, fold(T(seen) @ clean(do).abs()))
        w = clean(w)
        tol = (c.u * a + 2.0 ** -13 * b) * (1 + c.u) + c.u * w.abs() + c.tiny + low[i] * plain
        assert torch.all(((got - w).abs() <= tol) | bad), ("dQ dK dV".split()[i], ((got - w).abs() / tol)[~bad].max().item())


@pytest.mark.parametrize("what", ["dO", "Q", "K", "V", "all"])
@pytest.mark.parametrize("name", SPECIAL)
def test_gradients_with_infinite_and_nan_values(name, what):
    c = Case(**SPECIAL[name])
    nan, inf = float("nan"), float("inf")
    if what in ("Q", "all"):
        spoil(c.q, 3, [inf, nan], 5)
    if what in ("K", "all"):
        spoil(c.k, 3, [nan, -inf], 6)
    if what in ("V", "all"):
        spoil(c.v, 3, [inf, nan], 7)
    c.forward()
    if what in ("dO", "all"):
        spoil(c.do, 4, [inf, nan, -inf], 8)
        c.do[0, 0, c.do.shape[2] // 3] = nan
    c.backward()
    check_natural_backward(c)


@pytest.mark.parametrize("D,dtype", [(128, F16), (64, BF16)])
def test_an_infinite_gradient_takes_no_longer(D, dtype):
    """One infinity in dO, 8 heads over 1 of 32768 tokens: no wait of 0.02 s runs out, and what it does not reach keeps its
    bits.  Then dO of NaN behind the last document: it reaches nothing."""
    S, i = 32768, 20001
    g = torch.Generator(device=DEV).manual_seed(D)
    q, do = (torch.randn(1, 8, S, D, generator=g, device=DEV).to(dtype) for _ in range(2))
    k, v = (torch.randn(1, 1, S, D, generator=g, device=DEV).to(dtype) for _ in range(2))
    o, lse = torch.empty_like(q), torch.empty(1, 8, S, device=DEV)

    def run(**kw):
        grads = [torch.full_like(t, 7.0) for t in (q, k, v)]
        gsr.masked_attention_bwd(do, q, k, v, o, lse, *grads, **kw)
        status, code = gsr.device_status()
        assert status == gsr.Status.OK, hex(code)
        return grads

    gsr.masked_attention_fwd(q, k, v, o, lse, causal=True)
    clean, old = run(causal=True), do[0, 3, i, 7].item()
    do[0, 3, i, 7] = float("inf")
    gsr.set_wait_timeout_ns(20_000_000)
    try:
        dq, dk, dv = run(causal=True)
        assert not dq[0, 3, i].isfinite().any() and not dk[:, :, :i + 1].isfinite().any()
        assert torch.all(dv[0, 0, :i + 1, 7] == float("inf"))
        dq[0, 3, i], dk[:, :, :i + 1], dv[0, 0, :i + 1, 7] = clean[0][0, 3, i], clean[1][:, :, :i + 1], clean[2][0, 0, :i + 1, 7]
        assert all(torch.equal(a, b) for a, b in zip((dq, dk, dv), clean))
        do[0, 3, i, 7] = old
        kw = dict(doc_bounds=torch.tensor([[0, S - 100]], dtype=torch.int32, device=DEV))
        gsr.masked_attention_fwd(q, k, v, o, lse, **kw)
        clean = run(**kw)
        for t in (do, q, k, v):
            t[:, :, S - 100:] = float("nan")
        assert all(torch.equal(a, b) for a, b in zip(run(**kw), clean))
    finally:
        gsr.set_wait_timeout_ns(1_000_000_000)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_small_gradients_beside_large_ones(D, causal, dtype):
    """Two documents and two groups of heads, with dO of sizes 2^16 apart: each document's results of each group are within
    the bound that its own dO gives."""
    edges = [0, 500, 1100]
    c = Case(1, 4, 2, 1100, 1100, D, dtype=dtype, causal=causal, docs=[edges])
    for heads, rows, size in ((slice(0, 2), slice(0, 500), 2.0 ** 10), (slice(2, 4), slice(0, 500), 2.0 ** -5),
                              (slice(0, 2), slice(500, 1100), 2.0 ** -6), (slice(2, 4), slice(500, 1100), 2.0 ** 10)):
        c.do[:, heads, rows] *= size
    c.forward().backward()
    want, terms, wide, plain = llm.masked_attention_bwd(c.do, c.q, c.k, c.v, c.o, c.lse, c.see, **c.host)
    norm = lambda t: np.sqrt((llm.f64(t) ** 2).sum(-1)).max()
    for s, e in zip(edges, edges[1:]):
        for kv in range(2):
            heads = slice(2 * kv, 2 * kv + 2)
            low = [c.tiny * 2 * norm(c.do[:, heads, s:e]) * norm(c.v[:, kv]) * 2.0 ** -14] * 2 + [c.tiny * 2.0 ** -12]
            for name, t, w, a, b, p, x in zip(("dQ", "dK", "dV"), c.grads, want, terms, wide, plain, low):
                got, w, a, b, p = (y[:, heads if name == "dQ" else slice(kv, kv + 1), s:e] for y in (llm.f64(t), w, a, b, p))
                tol = c.tol(w, a, b) + x * p
                assert np.all(np.abs(got - w) <= tol), (name, s, kv, (np.abs(got - w) / tol).max())


@pytest.mark.parametrize("S", [1, 150])
@pytest.mark.parametrize("order", ["bhsd", "sbhd"])
def test_parts_of_one_buffer(order, S):
    # Q, K, V and O as head ranges of one buffer, their gradients as those of another
    B, Hq, Hkv, D = 3, 4, 2, 64
    g = torch.Generator().manual_seed(9)
    ranges = [Hq, Hkv, Hkv, Hq]

    def parts():
        H = sum(ranges)
        x = torch.randn(*((B, H, S, D) if order == "bhsd" else (S, B, H, D)), generator=g).to(F16).to(DEV)
        if order == "sbhd":
            x = x.permute(1, 2, 0, 3)
        return x.split(ranges, 1)

    c = Case(B, Hq, Hkv, S, S, D, causal=True)
    c.q, c.k, c.v, c.o = parts()
    c.lse = torch.empty(B, Hq, S, device=DEV)
    *c.grads, c.do = parts()
    gsr.masked_attention_fwd(c.q, c.k, c.v, c.o, c.lse, **c.kw)
    c.check_forward()
    gsr.masked_attention_bwd(c.do, c.q, c.k, c.v, c.o, c.lse, *c.grads, **c.kw)
    c.check_backward()


def test_a_captured_call_follows_infinities_that_come_and_go():
    c = Case(1, 8, 2, 700, 700, 64, causal=True, docs=[[0, 300, 690]])
    side = torch.cuda.Stream(DEV)
    c.forward().backward()
    clean = [t.clone() for t in (c.o, c.lse, *c.grads)]
    v, do = c.v.clone(), c.do.clone()

    def both():
        gsr.masked_attention_fwd(c.q, c.k, c.v, c.o, c.lse, **c.kw)
        gsr.masked_attention_bwd(c.do, c.q, c.k, c.v, c.o, c.lse, *c.grads, **c.kw)

    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        both()
    first = None
    for k in range(12):
        c.v.copy_(v)
        c.do.copy_(do)
        if k % 2:
            spoil(c.v, 6, [float("inf"), float("nan")], 2)
            spoil(c.do, 6, [float("inf"), -float("inf")], 3)
            c.v[:, :, 690:] = float("nan")
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (c.o, c.lse, *c.grads)]
        if not k % 2:
            assert all(torch.equal(a, b) for a, b in zip(got, clean))
        elif first is None:
            first = got
            check_natural(c)
            check_natural_backward(c)
        else:
            assert all(torch.equal(a.nan_to_num(5.0), b.nan_to_num(5.0)) and torch.equal(a.isnan(), b.isnan()) for a, b in zip(got, first))
    assert gsr.device_status(side)[0] == gsr.Status.OK
