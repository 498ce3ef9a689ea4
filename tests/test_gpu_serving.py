"""GPU tests of head norms with rotation and their gradient, rotated cache writes, the cache of 4 bits with attention
over it, and drafted tokens' verification, against the fp64 oracle.

Tolerances per element, with u = eps / 2 of the type and 2^-25 for float16 subnormals:
  rows            u |y| + 2^-18 |terms|: fp32 sums of at most 128 squares (a tree of 16 + 3 additions, relative 2^-19.7 with
                  rsqrt's 2 ulp halved by the root), four more roundings; terms are the two products of a rotation;
  gradients       u |dx| + 2^-17 |terms|: the same for two sums and six more roundings;
  weights'        2^-16 |terms|: sums of a lane's rows in turn (fewer than 200 here), then two trees, plus the rows' own error;
  4 bits          codes equal to fp32's where no norm is in the way; else |value - y| <= s / 2 + 15 u s + u |m| + 2^-17 |terms|:
                  half a step, and what rounding the scale and the minimum moves at a code's end;
  attention       (u + 2^-13) sum p (s |C - 8| + |m + 8 s|) (1 + u) + u |want|: p s is rounded once, scores (below 2^5) and
                  sums are fp32's, as in the 16-bit cache's tests.
Whole numbers are compared exactly.
"""
import numpy as np
import pytest
import torch

import tensor_core_gemm_multistage_gb300 as gsr
from oracle import llm, serving

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    gsr.build()
    yield


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def unit(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    return 2.0 ** -25 if dtype == F16 else 0.0


def near(got, want, terms, dtype, fp32):
    got = llm.f64(got)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    ok = ~np.isnan(want)
    err, tol = np.abs(got - want)[ok], (unit(dtype) * np.abs(want) + fp32 * terms + tiny(dtype))[ok]
    assert np.all(err <= tol), (err.max(), (err / np.maximum(tol, 1e-30)).max())


# ---------------------------------------------------------------------------- norms and rotation

class Rope:
    def __init__(self, B, Hq, Hkv, S, D, R, dtype=F16, interleaved=False, weights="both", positions=None, layout="fused", seed=0, scale=1.0):
        g = torch.Generator().manual_seed(seed)
        self.B, self.S, self.D, self.R, self.dtype, self.interleaved = B, S, D, R, dtype, interleaved
        new = lambda *shape: (torch.randn(*shape, generator=g) * scale).to(dtype).to(DEV)
        if layout == "fused":               # (batch, seq, heads): queries, keys and values of a projection
            qkv = new(B, S, Hq + 2 * Hkv, D)
            self.q, self.k = qkv[:, :, :Hq].transpose(1, 2), qkv[:, :, Hq:Hq + Hkv].transpose(1, 2)
        elif layout == "seq_first":         # (seq, heads, batch)
            self.q, self.k = new(S, Hq, B, D).permute(2, 1, 0, 3), new(S, Hkv, B, D).permute(2, 1, 0, 3)
        else:
            self.q, self.k = new(B, Hq, S, D), new(B, Hkv, S, D)
        w = lambda: (1 + 0.3 * torch.randn(D, generator=g)).to(dtype).to(DEV)
        self.qw, self.kw = w() if weights in ("both", "q") else None, w() if weights in ("both", "k") else None
        self.rows = 300
        self.table = gsr.rope_table(self.rows, R, device=DEV) if R else None
        self.positions = None
        if positions == "random":
            p = torch.randint(-1, self.rows, (B, S), generator=g)
            self.positions = p.to(torch.int32).to(DEV)
        self.do = [(torch.randn(B, t.shape[1], S, D, generator=g) * 0.1).to(dtype).to(DEV) for t in (self.q, self.k)]
        self.kw_args = dict(cos_sin=self.table, positions=self.positions, q_weight=self.qw, k_weight=self.kw, interleaved=interleaved)

    def angles(self):
        """cos, sin (B, 1, S, R / 2) and padding (B, 1, S), for the oracle."""
        if self.table is None:
            return None, None, None
        pos = np.tile(np.arange(self.S), (self.B, 1)) if self.positions is None else self.positions.cpu().numpy()
        cos, sin = serving.angles(self.table, pos, self.R)
        return cos[:, None], sin[:, None], (pos < 0)[:, None]

    def check_fwd(self, outs):
        cos, sin, pad = self.angles()
        for x, w, y in ((self.q, self.qw, outs[0]), (self.k, self.kw, outs[1])):
            want, terms = serving.norm_rope(x, None if w is None else llm.f64(w), cos, sin, self.R, interleaved=self.interleaved, padding=pad)
            near(y, want, terms, self.dtype, 2.0 ** -18)

    def run_fwd(self, **kw):
        outs = [torch.full_like(t, 7.0) for t in (self.q, self.k)]
        gsr.qk_norm_rope_fwd(self.q, self.k, *outs, **self.kw_args, **kw)
        return outs

    def run_bwd(self, **kw):
        self.dw = [None if w is None else torch.full((self.D,), 7.0, device=DEV) for w in (self.qw, self.kw)]
        outs = [torch.full_like(t, 7.0) for t in (self.q, self.k)]
        gsr.qk_norm_rope_bwd(*self.do, self.q, self.k, *outs, **self.kw_args, dq_weight=self.dw[0], dk_weight=self.dw[1], **kw)
        return outs

    def check_bwd(self, outs):
        cos, sin, pad = self.angles()
        for do, x, w, dx, dw in zip(self.do, (self.q, self.k), (self.qw, self.kw), outs, self.dw):
            a, b = serving.norm_rope_bwd(do, x, None if w is None else llm.f64(w), cos, sin, self.R, interleaved=self.interleaved, padding=pad)
            near(dx, *a, self.dtype, 2.0 ** -17)
            if w is not None:
                assert np.all(np.abs(llm.f64(dw) - b[0]) <= 2.0 ** -16 * b[1])


ROPES = {
    "one_row": dict(B=1, Hq=1, Hkv=1, S=1, D=64, R=64),
    "bf16": dict(B=2, Hq=8, Hkv=2, S=37, D=128, R=128, dtype=BF16),
    "interleaved": dict(B=2, Hq=3, Hkv=1, S=41, D=64, R=64, interleaved=True),
    "interleaved_part": dict(B=1, Hq=5, Hkv=5, S=23, D=128, R=48, interleaved=True, dtype=BF16),
    "part": dict(B=2, Hq=6, Hkv=3, S=50, D=128, R=32),
    "part_of_64": dict(B=2, Hq=6, Hkv=3, S=50, D=64, R=16, dtype=BF16),
    "odd_part": dict(B=1, Hq=7, Hkv=2, S=19, D=128, R=112),
    "norm_only": dict(B=2, Hq=6, Hkv=2, S=33, D=128, R=0),
    "rotation_only": dict(B=2, Hq=6, Hkv=2, S=33, D=64, R=64, weights=None),
    "norm_of_q": dict(B=2, Hq=6, Hkv=2, S=33, D=64, R=64, weights="q", layout="plain"),
    "norm_of_k": dict(B=2, Hq=6, Hkv=2, S=33, D=128, R=64, weights="k", layout="plain", dtype=BF16),
    "positions": dict(B=3, Hq=4, Hkv=2, S=29, D=128, R=128, positions="random"),
    "positions_seq_first": dict(B=3, Hq=4, Hkv=2, S=29, D=64, R=32, positions="random", layout="seq_first", dtype=BF16),
    "many_heads": dict(B=1, Hq=67, Hkv=33, S=9, D=128, R=128),
    "long": dict(B=1, Hq=2, Hkv=1, S=299, D=64, R=64, weights="both"),
    "large": dict(B=2, Hq=4, Hkv=2, S=20, D=64, R=64, scale=300.0),
    "small": dict(B=2, Hq=4, Hkv=2, S=20, D=64, R=64, scale=1e-3),
}


@pytest.mark.parametrize("name", ROPES)
def test_norm_rope(name):
    r = Rope(**ROPES[name])
    r.check_fwd(r.run_fwd())


@pytest.mark.parametrize("name", ROPES)
def test_norm_rope_gradient(name):
    r = Rope(**ROPES[name])
    r.check_bwd(r.run_bwd())


def test_gradient_is_that_of_the_forward_call():
    """Against differences of the call itself: the change of sum(y do) along a random direction."""
    r = Rope(B=1, Hq=2, Hkv=1, S=7, D=64, R=32, dtype=F16)
    dq, dk = r.run_bwd()
    g = torch.Generator().manual_seed(3)
    for x, w, dx, dw, do, i in ((r.q, r.qw, dq, r.dw[0], r.do[0], 0), (r.k, r.kw, dk, r.dw[1], r.do[1], 1)):
        for of_weight in (False, True):
            at = w if of_weight else x
            step = (torch.randn(at.shape, generator=g) * 2.0 ** -4).to(F16).to(DEV)
            old, f = at.clone(), []
            for sign in (1, -1):
                at.copy_(old + sign * step)
                moved = (at.double() - old.double())
                f.append((r.run_fwd()[i].double() * do.double()).sum())
                f.append(((dw if of_weight else dx).double() * moved).sum())
            at.copy_(old)
            # third differences of a norm and a linear map at 2^-4, and the roundings of y: n^(1/2) u |y do|
            assert abs((f[0] - f[2]) - (f[1] - f[3])) <= 0.02 * abs(f[1] - f[3]) + 2 ** -10 * float((do.double() ** 2).sum().sqrt()) * 4


def test_padding_holds_anything():
    r = Rope(B=2, Hq=4, Hkv=2, S=30, D=64, R=64, positions="random")
    pad = r.positions < 0
    pad[0, 3] = pad[1, 29] = True
    r.positions[pad] = -5
    for t in (r.q, r.k, *r.do):
        t.transpose(1, 2)[pad] = float("nan")
    r.check_fwd(r.run_fwd())
    r.check_bwd(r.run_bwd())
    r.positions[0, 0] = r.rows                       # behind the table: seen in every element that is rotated
    q, k = r.run_fwd()
    assert torch.isnan(q[0, :, 0]).all() and torch.isnan(k[0, :, 0]).all()
    assert torch.isnan(r.run_bwd()[0][0, :, 0]).all()


def test_in_place_and_without_keys():
    for name in ("bf16", "interleaved", "positions_seq_first"):
        r = Rope(**ROPES[name])
        want, grads = r.run_fwd(), r.run_bwd()
        q = r.q.clone()
        alone = torch.empty_like(q)
        gsr.qk_norm_rope_fwd(q, None, alone, None, **r.kw_args)
        assert torch.equal(alone, want[0])
        do = [t.clone() for t in r.do]
        dw = [torch.empty_like(t) for t in r.dw]
        gsr.qk_norm_rope_bwd(do[0], do[1], r.q, r.k, do[0], do[1], **r.kw_args, dq_weight=dw[0], dk_weight=dw[1])
        assert all(torch.equal(a, b) for a, b in zip(do + dw, grads + r.dw))
        gsr.qk_norm_rope_fwd(r.q, r.k, r.q, r.k, **r.kw_args)
        assert torch.equal(r.q, want[0]) and torch.equal(r.k, want[1])


@pytest.mark.parametrize("own_workspace", [False, True])
@pytest.mark.parametrize("wanted", [False, True])
@pytest.mark.parametrize("weights", ["both", "k", "q", None])
@pytest.mark.parametrize("absent", ["k", "q"])
def test_gradient_with_an_operand_of_no_heads(absent, weights, wanted, own_workspace):
    """Its weight may be there, with its gradient (0) or without; the other operand's gradients are those of the full call."""
    r = Rope(B=2, Hq=6, Hkv=3, S=21, D=64, R=32, weights=weights, layout="plain")
    full = r.run_bwd() + r.dw
    keep, gone = (0, 1) if absent == "k" else (1, 0)
    ops = [[r.do[0], r.do[1]], [r.q, r.k], [torch.full_like(t, 7.0) for t in (r.q, r.k)]]
    for pair in ops:
        pair[gone] = None if absent == "k" else pair[gone][:, :0]
    dw = [None if t is None else torch.full_like(t, 7.0) for t in r.dw]
    if not wanted:
        dw[gone] = None
    ws = None
    if own_workspace:
        ws = torch.empty(gsr.qk_norm_rope_bwd_workspace(2, 6 if absent == "k" else 0, 0 if absent == "k" else 3, 21, 64), dtype=torch.uint8, device=DEV)
    gsr.qk_norm_rope_bwd(*ops[0], *ops[1], *ops[2], **r.kw_args, dq_weight=dw[0], dk_weight=dw[1], workspace=ws)
    assert torch.equal(ops[2][keep], full[keep])
    if dw[keep] is not None:                # the same sums, cut between CTAs by the heads that are there
        cos, sin, _ = r.angles()
        _, (want, terms) = serving.norm_rope_bwd(r.do[keep], (r.q, r.k)[keep], llm.f64((r.qw, r.kw)[keep]), cos, sin, r.R)
        assert np.all(np.abs(llm.f64(dw[keep]) - want) <= 2.0 ** -16 * terms)
    assert dw[gone] is None or torch.all(dw[gone] == 0)


def test_gradient_repeats_whatever_the_workspace_and_stream():
    r = Rope(B=3, Hq=8, Hkv=2, S=700 // 4, D=128, R=128, dtype=BF16)
    want = [t.clone() for t in r.run_bwd() + r.dw]
    n = gsr.qk_norm_rope_bwd_workspace(3, 8, 2, 175, 128)
    own = torch.full((n + 64,), 255, dtype=torch.uint8, device=DEV)
    assert all(torch.equal(a, b) for a, b in zip(r.run_bwd(workspace=own[:n]) + r.dw, want)) and torch.all(own[n:] == 255)
    s = torch.cuda.Stream(DEV)
    s.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        got = r.run_bwd() + r.dw
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    gsr.release_stream(s)


def test_weights_gradients_of_no_rows_are_zero():
    r = Rope(B=1, Hq=2, Hkv=1, S=4, D=64, R=64)
    r.q, r.k, r.do = r.q[:, :, :0], r.k[:, :, :0], [t[:, :, :0] for t in r.do]
    r.run_bwd()
    assert all(torch.all(t == 0) for t in r.dw)


def test_rows_past_32_bits():
    S, H, D = 2 ** 31 // (8 * 64) + 40, 8, 64
    q = torch.zeros(1, S, H, D, dtype=BF16, device=DEV)
    q[:, -50:] = torch.randn(1, 50, H, D).to(BF16).to(DEV)
    w, table = torch.ones(D, dtype=BF16, device=DEV), gsr.rope_table(60, D, device=DEV)
    pos = (torch.arange(S, device=DEV) % 60).to(torch.int32)[None]
    small, out = torch.empty(1, 50, H, D, dtype=BF16, device=DEV), torch.empty_like(q)
    v = lambda t: t.transpose(1, 2)
    gsr.qk_norm_rope_fwd(v(q), None, v(out), None, cos_sin=table, positions=pos, q_weight=w)
    gsr.qk_norm_rope_fwd(v(q[:, -50:]), None, v(small), None, cos_sin=table, positions=pos[:, -50:].contiguous(), q_weight=w)
    assert torch.equal(out[:, -50:], small) and torch.all(out[:, :-50] == 0)
    grad = torch.empty(D, device=DEV)
    gsr.qk_norm_rope_bwd(v(q), None, v(q), None, v(out), None, cos_sin=table, positions=pos, q_weight=w, dq_weight=grad)
    first = torch.empty(D, device=DEV)
    gsr.qk_norm_rope_bwd(v(q[:, -50:]), None, v(q[:, -50:]), None, v(small), None, cos_sin=table, positions=pos[:, -50:].contiguous(),
                         q_weight=w, dq_weight=first)
    assert torch.equal(out[:, -50:], small)
    assert torch.allclose(grad, first, rtol=1e-4, atol=1e-3)      # sums of 400 terms up to 5 in another order


# ---------------------------------------------------------------------------- cache writes

class Append:
    def __init__(self, N, Hq, H, D, page, R, dtype=F16, norm=False, interleaved=False, four=False, layout="heads", seed=0):
        g = torch.Generator().manual_seed(seed)
        self.N, self.Hq, self.H, self.D, self.R, self.page, self.dtype, self.four = N, Hq, H, D, R, page, dtype, four
        self.pages = N // page + 3
        qkv = (torch.randn(N, Hq + 2 * H, D, generator=g) * torch.exp2(torch.randn(Hq + 2 * H, D, generator=g))).to(dtype).to(DEV)
        self.q, self.k, self.v = qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:]
        w = lambda: (1 + 0.3 * torch.randn(D, generator=g)).to(dtype).to(DEV)
        self.qw, self.kw = (w(), w()) if norm else (None, None)
        self.table = gsr.rope_table(500, R, device=DEV) if R else None
        self.positions = torch.randint(500, (N,), generator=g).to(torch.int32).to(DEV) if R else None
        self.slots = torch.randperm(self.pages * page, generator=g)[:N].to(torch.int32).to(DEV)
        self.live = torch.ones(N, dtype=torch.bool)
        if N > 4:
            self.slots[1], self.slots[2] = -1, self.pages * page        # padding, and behind the cache
            self.live[1] = self.live[2] = False
            if R:
                self.positions[3] = -1
                self.live[3] = False
        if four:
            self.caches = [gsr.kv_cache4(self.pages, page, H, D, dtype, DEV) for _ in range(2)]
            if layout == "rows":
                self.caches = [gsr.Cache4(c.codes.contiguous(), c.params.contiguous()) for c in self.caches]
            for c in self.caches:
                c.codes.fill_(0x21)
                c.params.fill_(3.0)
        else:
            self.caches = [torch.full((self.pages, page, H, D), 3.0, dtype=dtype, device=DEV) for _ in range(2)]
        self.q_out = torch.full((N, Hq, D), 7.0, dtype=dtype, device=DEV) if Hq else None
        self.kwargs = dict(positions=self.positions, cos_sin=self.table, q_weight=self.qw, k_weight=self.kw, interleaved=interleaved)
        self.interleaved = interleaved

    def run(self, **kw):
        call = gsr.kv_cache4_append_rope if self.four else gsr.kv_cache_append_rope
        call(self.k, self.v, self.slots, *self.caches, Q=self.q if self.Hq else None, Q_out=self.q_out, **self.kwargs, **kw)
        return self

    def rows(self, x, w):
        cos = sin = pad = None
        if self.R:
            pos = self.positions.cpu().numpy()
            cos, sin = (a[:, None] for a in serving.angles(self.table, pos, self.R))
            pad = (pos < 0)[:, None]
        return serving.norm_rope(x, None if w is None else llm.f64(w), cos, sin, self.R, interleaved=self.interleaved, padding=pad)

    def fp32(self, x):
        """The rotated rows as fp32 gives them, each operation rounded (no norm)."""
        x = x.float().cpu()
        if not self.R:
            return x
        t = self.table.cpu()[self.positions.cpu().long().clamp(min=0)][:, None]
        c, s = t[..., :self.R // 2], t[..., self.R // 2:]
        a, b = (x[..., 0:self.R:2], x[..., 1:self.R:2]) if self.interleaved else (x[..., :self.R // 2], x[..., self.R // 2:self.R])
        y, z = a * c - b * s, b * c + a * s
        y = torch.stack([y, z], -1).flatten(-2) if self.interleaved else torch.cat([y, z], -1)
        return torch.cat([y, x[..., self.R:]], -1)

    def at(self, t):
        """The cache rows of the live tokens (tokens, heads, ..), and whether any other row has changed from `fill`."""
        slots = self.slots.cpu()[self.live].long()
        return t.cpu()[slots // self.page, slots % self.page]

    def untouched(self, t, fill):
        keep = torch.ones(self.pages * self.page, dtype=torch.bool)
        keep[self.slots.cpu()[self.live].long()] = False
        return torch.all(t.cpu().reshape(self.pages * self.page, -1)[keep] == fill)

    def check(self):
        if self.Hq:
            want, terms = self.rows(self.q, self.qw)
            near(self.q_out, want, terms, self.dtype, 2.0 ** -18)
        live = self.live.numpy()
        want, terms = (a[live] for a in self.rows(self.k, self.kw))
        if not self.four:
            near(self.at(self.caches[0]), want, terms, self.dtype, 2.0 ** -18)
            assert torch.equal(self.at(self.caches[1]), self.v.cpu()[self.live])
            assert all(self.untouched(c, 3.0) for c in self.caches)
            return self
        u = unit(self.dtype)
        for c, x, mag, exact in ((self.caches[0], want, terms, None if self.kw is not None else self.fp32(self.k)),
                                 (self.caches[1], llm.f64(self.v)[live], np.abs(llm.f64(self.v)[live]), self.v.float().cpu())):
            codes, params = self.at(c.codes), self.at(c.params)
            got, _ = serving.values4(codes.numpy(), params)
            s, m = (np.repeat(llm.f64(params)[..., i], 64, -1) for i in (0, 1))
            tol = s / 2 + 15 * u * s + u * np.abs(m) + 2.0 ** -17 * mag + tiny(self.dtype) * 16
            assert np.all(np.abs(got - x) <= tol), (np.abs(got - x) / tol).max()
            if exact is not None:
                y = exact[self.live].unflatten(-1, (-1, 64))
                low, high = y.amin(-1, keepdim=True), y.amax(-1, keepdim=True)
                sc, lo = ((high - low) * torch.tensor(1.0 / 15.0)).to(self.dtype).float(), low.to(self.dtype).float()
                code = torch.where(sc > 0, torch.round((y - lo) / torch.where(sc > 0, sc, 1.0)).clamp(0, 15), 0.0).flatten(-2).to(torch.uint8)
                assert torch.equal(params.float(), torch.cat([sc, lo], -1))
                assert torch.equal(codes, code[..., 0::2] | code[..., 1::2] << 4)
            assert self.untouched(c.codes, 0x21) and self.untouched(c.params, 3.0)
        return self


APPENDS = {
    "one": dict(N=1, Hq=0, H=1, D=64, page=16, R=64),
    "decode": dict(N=48, Hq=32, H=8, D=128, page=16, R=128, norm=True, dtype=BF16),
    "norm_only": dict(N=33, Hq=4, H=2, D=64, page=8, R=0, norm=True),
    "copy": dict(N=40, Hq=0, H=3, D=128, page=24, R=0),
    "interleaved": dict(N=77, Hq=6, H=3, D=64, page=16, R=32, interleaved=True, dtype=BF16),
    "part": dict(N=130, Hq=5, H=5, D=128, page=64, R=64),
    "odd_page": dict(N=900, Hq=0, H=2, D=64, page=7, R=64),
    "many_heads": dict(N=9, Hq=70, H=35, D=128, page=16, R=128, norm=True),
    "prompt": dict(N=3000, Hq=0, H=8, D=128, page=64, R=128),
}


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("name", APPENDS)
def test_append(name, four):
    Append(**APPENDS[name], four=four).run().check()


def test_append_by_rows_and_in_place():
    a = Append(**APPENDS["decode"], four=True, layout="rows").run().check()
    b = Append(**APPENDS["decode"], four=True)
    b.q_out = b.q
    b.run()
    assert torch.equal(b.q, a.q_out)
    for x, y in zip(a.caches, b.caches):
        assert torch.equal(x.codes, y.codes) and torch.equal(x.params, y.params)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("D", [64, 128])
def test_rows_that_are_hard_to_hold(D, dtype):
    """Constant rows, tiny and huge spans, ends of the type, infinities and NaN; each 64 values by themselves."""
    rows = []
    for x in (0.0, -3.5, 2.0 ** -24, torch.finfo(dtype).max, -torch.finfo(dtype).max):
        rows.append(torch.full((D,), x))
    top = torch.finfo(dtype).max / 4
    rows += [torch.linspace(-top, top, D), torch.linspace(1.0, 1.0 + 2.0 ** -9, D), torch.linspace(0.0, 2.0 ** -20, D),
             torch.arange(D) % 16 * 1.0, torch.arange(D) % 31 * 0.5]                    # whole codes, and halves: ties
    bad = [float("nan"), float("inf"), -float("inf")]
    for x in bad:
        r = torch.linspace(-1, 1, D)
        r[5] = x
        rows.append(r)
    N = len(rows)
    v = torch.stack(rows).to(dtype).to(DEV)[:, None].contiguous()
    kc, vc = (gsr.kv_cache4(2, 16, 1, D, dtype, DEV) for _ in range(2))
    gsr.kv_cache4_append_rope(v, v.flip(0).contiguous(), i32(list(range(N))), kc, vc)
    k, w = torch.empty_like(v), torch.empty_like(v)
    gsr.kv_cache4_read(kc, vc, i32(list(range(N))), k, w)
    assert torch.equal(k.flip(0).nan_to_num(nan=1234.0), w.nan_to_num(nan=1234.0))
    got, want, u = k.double().cpu()[:, 0], v.double().cpu()[:, 0], unit(dtype)
    for n in range(N):
        for g in range(D // 64):
            a, b = got[n, 64 * g:64 * g + 64], want[n, 64 * g:64 * g + 64]
            if not torch.isfinite(b).all():
                assert torch.isnan(a).all()
                continue
            s = (b.max() - b.min()) / 15
            # half a step, the scale's and minimum's roundings, and the value's own to the type
            tol = s / 2 + 15 * u * s + u * b.abs().max() + u * (b.abs() + s) + 16 * 2.0 ** -25
            assert torch.all((a - b).abs() <= tol), n


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("D", [64, 128])
def test_minimum_beyond_the_type(D, dtype):
    """Keys whose norm or rotation takes them past the type's end: 64 values with such a minimum are NaN, and a node that sees
    the key; past the upper end the codes still hold them."""
    N, G, top = 6, D // 64, torch.finfo(dtype).max
    k = torch.zeros(N, 1, D)
    for n, x in enumerate((1.0, -1.0, 1.0, -1.0)):
        k[n, 0, 3 if n < 2 else D - 3] = x
    k[4:] = 0.5
    table, w = torch.zeros(1, D), None
    if dtype == F16:                          # a row of one value is sqrt(D) w there
        k, w = k.to(dtype).to(DEV), torch.full((D,), 60000.0, dtype=dtype, device=DEV)
        table[:, :D // 2] = 1.0
        peak = 60000.0 * D ** 0.5
    else:                                     # float32 holds 1.0025 of bfloat16's largest value, which rounds to an infinity
        k[:4] *= top
        k, peak = k.to(dtype).to(DEV), 1.0025 * top
        table[:, :D // 2] = 1.0025
    kc, vc = (gsr.kv_cache4(1, 16, 1, D, dtype, DEV) for _ in range(2))
    v = torch.linspace(-1, 1, D).to(dtype).to(DEV).expand(N, 1, D).contiguous()
    pos, slots = i32([0] * N), i32(list(range(N)))
    gsr.kv_cache4_append_rope(k, v, slots, kc, vc, positions=pos, cos_sin=table.to(DEV), k_weight=w)
    params, codes = kc.params[0, :N, 0].double().cpu(), kc.codes[0, :N, 0].cpu()
    for n in range(4):
        lost = n % 2 == 1                     # the minimum is -peak
        for g in range(G):
            here = g == (0 if n < 2 else G - 1)
            s, m = params[n, g].tolist()
            if here and lost:
                assert np.isnan(s) and np.isnan(m), (n, g)
            else:
                assert m == 0.0 and s == pytest.approx(peak / 15 if here else 0.0, rel=2 * unit(dtype)), (n, g)
    assert torch.isfinite(params[4:]).all() and codes[0, 1] == 0xf0 and codes[2, D // 2 - 2] == 0xf0
    # attention: a request that sees row 0 alone, and one that sees row 1 as well
    table4, o = i32([[0], [0]]), torch.empty(2, 1, D, dtype=dtype, device=DEV)
    q = torch.full((2, 1, D), 2.0 ** -8 if dtype == F16 else 2.0 ** -120, dtype=dtype, device=DEV)
    gsr.tree_attention4_fwd(q, kc, vc, table4, i32([1, 2]), i32([0, 1, 2]), None, o, 1)
    assert torch.isfinite(o[0]).all() and torch.isnan(o[1]).all()


def test_read_is_what_the_codes_stand_for():
    for D, dtype in ((64, F16), (128, BF16)):
        g = torch.Generator().manual_seed(D)
        kc, vc = (gsr.kv_cache4(5, 24, 3, D, dtype, DEV) for _ in range(2))
        for c in (kc, vc):
            c.codes.copy_(torch.randint(256, c.codes.shape, generator=g).to(torch.uint8))
            c.params.copy_(torch.rand(c.params.shape, generator=g) * 3 - torch.tensor([0.0, 2.0]))
        slots = torch.randperm(120, generator=g)[:50].to(torch.int32)
        slots[3], slots[4] = -1, 120
        k, v = (torch.full((50, 3, D), 9.0, dtype=dtype, device=DEV) for _ in range(2))
        gsr.kv_cache4_read(kc, vc, slots.to(DEV), k, v)
        for c, out in ((kc, k), (vc, v)):
            code = torch.stack([c.codes & 15, c.codes >> 4], -1).flatten(-2).float().unflatten(-1, (-1, 64))
            value = (code * c.params[..., :1].float() + c.params[..., 1:].float()).flatten(-2).to(dtype).reshape(120, 3, D).cpu()
            want = torch.full((50, 3, D), 9.0, dtype=dtype)
            ok = (slots >= 0) & (slots < 120)
            want[ok] = value[slots[ok].long()]
            assert torch.equal(out.cpu(), want)


# ---------------------------------------------------------------------------- attention over 4 bits

class Tree4:
    def __init__(self, kv, T, Hq, Hkv, D, page, dtype=F16, cap=0.0, parents="random", seed=0, scale=0.0, layout="heads", extra_rows=0,
                 v_scale=1.0, k_shift=0.0, width=0):
        r, g = np.random.default_rng(seed + 5), torch.Generator().manual_seed(seed)
        self.kv, self.T, self.page, self.dtype, self.D = kv, T, page, dtype, D
        B = len(kv)
        need = [-(-n // page) for n in kv]
        pool = sum(need) + 3
        order = [int(x) for x in r.permutation(pool)]
        self.table = np.full((B, max(need + [1, width]) + 1), -1)
        at = 0
        for b in range(B):
            self.table[b, :need[b]] = order[at:at + need[b]]
            at += need[b]
        self.starts = np.concatenate([[0], np.cumsum(T)])
        self.N = N = int(self.starts[-1]) + extra_rows
        new = lambda: torch.randn(pool * page, Hkv, D, generator=g)
        k, v = (new() + k_shift).to(dtype).to(DEV), (new() * v_scale).to(dtype).to(DEV)
        self.caches = [gsr.kv_cache4(pool, page, Hkv, D, dtype, DEV) for _ in range(2)]
        if layout != "heads":
            self.caches = [gsr.Cache4(c.codes.contiguous(), c.params.contiguous()) for c in self.caches]
        gsr.kv_cache4_append_rope(k, v, torch.arange(pool * page, dtype=torch.int32, device=DEV), *self.caches)
        self.q = (torch.randn(N, Hq, D, generator=g) * 1.5).to(dtype).to(DEV)
        self.parents = None
        if parents == "random":
            self.parents = [int(r.integers(-1, t)) if t else -1 for n in T for t in range(n)] + [-1] * extra_rows
        elif parents == "flat":
            self.parents = [-1] * N
        self.cap, self.scale, self.max_nodes = cap, scale, max(T + [1])

    def workspace(self):
        return gsr.tree_attention4_workspace(len(self.kv), self.N, self.q.shape[1], self.caches[0].codes.shape[2], self.D, self.caches[0].codes.shape[0],
                                             self.page, self.table.shape[1], self.max_nodes)

    def run(self, stream=None, **kw):
        self.o = torch.full_like(self.q, 7.0)
        self.args = (self.q, *self.caches, i32(self.table), i32(self.kv), i32(self.starts),
                     None if self.parents is None else i32(self.parents), self.o, self.max_nodes)
        self.kw = dict(softmax_scale=self.scale, softcap=self.cap)
        gsr.tree_attention4_fwd(*self.args, **self.kw, stream=stream, **kw)
        return self

    def want(self):
        (k, _), (v, mag) = (serving.values4(c.codes.cpu().numpy(), c.params) for c in self.caches)
        call = lambda v: llm.tree_attention(self.q, k, v, self.table, self.kv, self.starts, self.parents, self.scale, self.cap, None, self.max_nodes)
        return call(v)[0], call(mag)[1]

    def check(self, rows=None):
        want, terms = self.want()
        got = llm.f64(self.o)
        if rows is not None:
            got, want, terms = got[rows], want[rows], terms[rows]
        real = ~np.isnan(want)
        assert np.all(got[~real] == 7.0), "rows of no request were written"
        got, want, terms = got[real], want[real], terms[real]
        assert not np.isnan(got).any()
        u = unit(self.dtype)
        tol = (u + 2.0 ** -13) * terms * (1 + u) + u * np.abs(want) + tiny(self.dtype)
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
    "trees_cap": dict(kv=[300, 41], T=[30, 9], Hq=6, Hkv=2, D=64, page=16, cap=3.0),
    "chain": dict(kv=[257, 130], T=[33, 2], Hq=5, Hkv=1, D=128, page=128, parents="chain"),
    "chain_cap": dict(kv=[257, 130], T=[33, 2], Hq=4, Hkv=1, D=64, page=24, parents="chain", cap=5.0, dtype=BF16),
    "flat": dict(kv=[140], T=[64], Hq=8, Hkv=1, D=64, page=16, parents="flat"),
    "large_group": dict(kv=[333], T=[3], Hq=96, Hkv=1, D=64, page=16),
    "odd_group": dict(kv=[333, 90], T=[50, 26], Hq=21, Hkv=3, D=128, page=40),
    "odd_large_page": dict(kv=[700, 300], T=[2, 10], Hq=8, Hkv=2, D=64, page=136),
    "some_without_rows": dict(kv=[100, 0, 50, 8], T=[3, 0, 0, 1], Hq=4, Hkv=2, D=64, page=16),
    "rows_first": dict(kv=[220, 31], T=[4, 1], Hq=4, Hkv=2, D=128, page=16, layout="rows"),
    "negative_scale": dict(kv=[220, 31], T=[4, 1], Hq=4, Hkv=2, D=128, page=16, scale=-0.1),
    "rows_behind": dict(kv=[220, 31], T=[4, 1], Hq=4, Hkv=2, D=128, page=16, extra_rows=5),
    "small_values": dict(kv=[500, 31], T=[1, 3], Hq=4, Hkv=2, D=64, page=16, v_scale=2.0 ** -12),
    "large_values": dict(kv=[500, 31], T=[1, 3], Hq=4, Hkv=2, D=128, page=16, v_scale=2.0 ** 12),
    "shifted_keys": dict(kv=[500, 31], T=[1, 3], Hq=4, Hkv=2, D=64, page=16, k_shift=0.5, dtype=BF16),
}


@pytest.mark.parametrize("even", [False, True])
@pytest.mark.parametrize("name", TREES)
def test_tree_attention4(name, even):
    """In clusters, and shared out evenly: a table that could hold much is taken for much work."""
    t = Tree4(**TREES[name], width=2 ** 21 // TREES[name]["page"] if even else 0)
    assert (t.workspace() > 0) == even
    t.run().check()


@pytest.mark.parametrize("up", [100, -100, -122])
def test_queries_of_any_size(up):
    """Queries times 2^up over keys times 2^-up: the scores, and so the answers, are those of ordinary sizes."""
    t = Tree4(kv=[300, 41], T=[9, 1], Hq=8, Hkv=2, D=128, page=16, dtype=BF16)
    t.q = (t.q.double() * 2.0 ** up).to(BF16)
    t.caches[0].params.copy_((t.caches[0].params.double() * 2.0 ** -up).to(BF16))
    t.run().check()


def _random_trees(n, seed):
    r = np.random.default_rng(seed)
    out = []
    for _ in range(n):
        B = int(r.integers(1, 9))
        T = [int(x) for x in r.integers(0, int(r.choice([2, 9, 65])), B)]
        out.append(dict(kv=[t + int(x) for t, x in zip(T, r.integers(0, int(r.choice([50, 900])), B))], T=T,
                        Hkv=int(r.choice([1, 2, 3])), D=int(r.choice([64, 128])), page=int(r.choice([8, 16, 32, 48, 64])),
                        dtype=[F16, BF16][int(r.integers(2))], cap=float(r.choice([0.0, 2.0])),
                        parents=str(r.choice(["random", "chain", "flat"])), seed=int(r.integers(100))))
        out[-1]["Hq"] = out[-1]["Hkv"] * int(r.choice([1, 3, 8]))
    return out


@pytest.mark.parametrize("even", [False, True])
@pytest.mark.parametrize("c", _random_trees(14, 12))
def test_random_trees4(c, even):
    Tree4(**c, width=2 ** 21 // c["page"] if even else 0).run().check()


def test_many_requests_shared_out_evenly():
    """More requests than a CTA has threads, some without keys or rows; and one long request among them."""
    r = np.random.default_rng(1)
    T = [int(x) for x in r.integers(0, 4, 700)]
    kv = [n + int(x) for n, x in zip(T, r.integers(0, 90, 700))]
    Tree4(kv=kv, T=T, Hq=8, Hkv=2, D=64, page=16, width=4000).run().check()          # items enough for every CTA
    t = Tree4(kv=kv, T=T, Hq=2, Hkv=1, D=64, page=16, width=4000)
    assert t.workspace() > 0
    t.run().check()
    Tree4(kv=[70000] + [5] * 30, T=[1] * 31, Hq=8, Hkv=2, D=128, page=64, dtype=BF16).run().check()


def test_workspaces():
    t = Tree4(kv=[3000, 77], T=[1, 9], Hq=8, Hkv=2, D=128, page=16, width=2 ** 17).run().check()
    want, size = t.o.clone(), t.workspace()
    assert size > 0
    own = torch.full((size + 64,), 255, dtype=torch.uint8, device=DEV)
    assert torch.equal(t.run(workspace=own[:size]).o, want) and torch.all(own[size:] == 255)
    with pytest.raises(gsr.GsrError):
        t.run(workspace=own[:size - 16])
    s = torch.cuda.Stream(DEV)
    torch.cuda.synchronize()
    for _ in range(2):
        t.o.fill_(7.0)
        torch.cuda.synchronize()
        gsr.tree_attention4_fwd(*t.args, **t.kw, stream=s)
        s.synchronize()
        assert torch.equal(t.o, want)
        gsr.release_stream(s)
    # a graph takes a workspace of its own: replays beside eager calls of the same stream's
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gsr.tree_attention4_fwd(*t.args, **t.kw)
    for _ in range(3):
        t.o.fill_(7.0)
        graph.replay()
        assert torch.equal(t.o, want)
        other = torch.empty_like(t.o)
        gsr.tree_attention4_fwd(*t.args[:7], other, t.args[8], **t.kw)
        assert torch.equal(other, want)


def test_keys_nothing_sees_have_no_influence():
    t = Tree4(kv=[100, 131, 40], T=[5, 12, 1], Hq=8, Hkv=2, D=128, page=16)
    clean = t.run().check().o.clone()
    used = {(int(t.table[b][j // 16]), j % 16) for b, n in enumerate(t.kv) for j in range(n)}
    for c in t.caches:
        for pg in range(c.codes.shape[0]):
            for row in range(16):
                if (pg, row) not in used:
                    c.params[pg, row] = float("nan")
                    c.codes[pg, row] = 255
    assert torch.equal(t.run().o, clean)
    # a sibling no other node sees: only its own row changes
    t.parents[5 + 11] = t.parents[5 + 10] = -1
    clean = t.run().check().o.clone()
    j = t.kv[1] - 1
    at = int(t.table[1][j // 16]), j % 16
    t.caches[1].params[at][:, 1] = float("nan")               # of its values, the second 64 columns
    t.run()
    others = [n for n in range(t.N) if n != 5 + 11]
    assert torch.equal(t.o[others], clean[others]) and torch.equal(t.o[16, :, :64], clean[16, :, :64]) and torch.isnan(t.o[16, :, 64:]).all()
    t.caches[0].params[at] = float("inf")
    t.run()
    assert torch.equal(t.o[others], clean[others]) and torch.isnan(t.o[16]).all()


def test_nan_in_a_seen_key():
    t = Tree4(kv=[400, 90], T=[1, 1], Hq=4, Hkv=2, D=128, page=16, dtype=BF16)
    clean = t.run().check().o.clone()
    t.caches[1].params[int(t.table[0][2]), 5, 1, 0] = float("nan")      # head 1's first 64 columns
    t.run()
    assert torch.isnan(t.o[0, 2:, :64]).all() and torch.equal(t.o[0, 2:, 64:], clean[0, 2:, 64:])
    assert torch.equal(t.o[0, :2], clean[0, :2]) and torch.equal(t.o[1], clean[1])


def test_pages_outside_the_pool_and_lengths_that_are_cut():
    t = Tree4(kv=[300, 90], T=[6, 1], Hq=4, Hkv=2, D=64, page=16)
    t.table[0][2], t.table[0][9], t.table[1][0] = -1, 10 ** 6, -(2 ** 31)
    t.run().check()
    t.table[1][:] = -1                    # a request whose every page is missing: O = 0
    t.run().check()
    assert torch.all(t.o[6] == 0)
    t = Tree4(kv=[60, 30], T=[2, 1], Hq=2, Hkv=1, D=64, page=16)
    t.table = t.table[:, :2].copy()       # 32 of 60 tokens
    t.run().check()
    t = Tree4(kv=[60, 30], T=[6, 3], Hq=2, Hkv=1, D=64, page=16, parents="chain")
    t.max_nodes = 4                       # nodes behind the limit are left
    t.run().check()


def test_repeatable_and_on_two_streams_at_once():
    ts = [Tree4(kv=[5000, 300, 77], T=[1, 8, 30], Hq=8, Hkv=2, D=128, page=16, seed=1),
          Tree4(kv=[5000, 300, 77], T=[1, 8, 30], Hq=8, Hkv=2, D=128, page=16, seed=1, width=2 ** 17),
          Tree4(kv=[900] * 9, T=[2] * 9, Hq=16, Hkv=4, D=64, page=32, dtype=BF16, seed=2)]
    first = [t.run().o.clone() for t in ts]
    streams = [torch.cuda.Stream(DEV) for _ in ts]
    torch.cuda.synchronize()
    for _ in range(4):
        for t, s in zip(ts, streams):
            gsr.tree_attention4_fwd(*t.args, **t.kw, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(t.o, f) for t, f in zip(ts, first))


@pytest.mark.parametrize("even", [False, True])
def test_rows_before_the_first_sequence(even):
    """Rows of no request in front of the first and behind the last are left as they were; the others' results stay."""
    t = Tree4(kv=[300, 77, 40], T=[5, 1, 9], Hq=8, Hkv=2, D=128, page=16, extra_rows=5, width=2 ** 17 if even else 0)
    want, N = t.run().check().o[:-5].clone(), t.N - 5
    t.q = torch.cat([t.q[N:N + 3], t.q[:N], t.q[N + 3:]])
    t.parents = [-1] * 3 + t.parents[:N] + [-1] * 2
    t.starts = t.starts + 3
    t.run()
    assert torch.equal(t.o[3:-2], want) and torch.all(t.o[:3] == 7.0) and torch.all(t.o[-2:] == 7.0)


@pytest.mark.parametrize("D", [64, 128])
def test_caches_of_views(D):
    """Keys and values side by side in one tensor, every second page of a larger one: written, read and attended alike."""
    t = Tree4(kv=[150, 61], T=[3, 20], Hq=8, Hkv=2, D=D, page=16, dtype=BF16).run().check()
    want, pool = t.o.clone(), t.caches[0].codes.shape[0]
    slots = torch.arange(pool * 16, dtype=torch.int32, device=DEV)
    k, v = (torch.empty(pool * 16, 2, D, dtype=BF16, device=DEV) for _ in range(2))
    gsr.kv_cache4_read(*t.caches, slots, k, v)
    codes = torch.zeros(2 * pool + 1, 2, 2, 16, D // 2, dtype=torch.uint8, device=DEV)
    params = torch.zeros(2 * pool + 1, 2, 2, 16, D // 64, 2, dtype=BF16, device=DEV)
    t.caches, old = [gsr.Cache4(codes[1::2, i].transpose(1, 2), params[1::2, i].transpose(1, 2)) for i in range(2)], t.caches
    for new, o in zip(t.caches, old):
        new.codes.copy_(o.codes)
        new.params.copy_(o.params)
    assert torch.equal(t.run().o, want)
    k2, v2 = torch.empty_like(k), torch.empty_like(v)
    gsr.kv_cache4_read(*t.caches, slots, k2, v2)
    assert torch.equal(k, k2) and torch.equal(v, v2)
    gsr.kv_cache4_append_rope(v, k, slots, *t.caches)
    gsr.kv_cache4_append_rope(v, k, slots, *old)
    for new, o in zip(t.caches, old):
        assert torch.equal(new.codes, o.codes) and torch.equal(new.params, o.params)
    assert not codes[::2].any() and not params[::2].any()


def test_a_cache_past_32_bits():
    t = Tree4(kv=[150, 61], T=[3, 1], Hq=8, Hkv=8, D=128, page=16, dtype=BF16).run().check()
    want, pool = t.o.clone(), t.caches[0].codes.shape[0]
    pages = 2 ** 32 // (16 * 8 * 64) + pool
    first, old = pages - pool, t.caches
    t.caches = [gsr.Cache4(torch.empty(pages, 8, 16, 64, dtype=torch.uint8, device=DEV).transpose(1, 2),
                           torch.empty(pages, 8, 16, 2, 2, dtype=BF16, device=DEV).transpose(1, 2)) for _ in range(2)]
    for c, o in zip(t.caches, old):
        c.codes[first:], c.params[first:] = o.codes, o.params
    t.table[t.table >= 0] += first
    assert torch.equal(t.run().o, want)
    slots = torch.arange(first * 16, pages * 16, dtype=torch.int32, device=DEV)
    k, v = (torch.empty(pool * 16, 8, 128, dtype=BF16, device=DEV) for _ in range(2))
    gsr.kv_cache4_read(*t.caches, slots, k, v)
    k2, v2 = torch.empty_like(k), torch.empty_like(v)
    gsr.kv_cache4_read(*old, torch.arange(pool * 16, dtype=torch.int32, device=DEV), k2, v2)
    assert torch.equal(k, k2) and torch.equal(v, v2)
    gsr.kv_cache4_append_rope(v, k, slots, *t.caches)
    gsr.kv_cache4_append_rope(v, k, torch.arange(pool * 16, dtype=torch.int32, device=DEV), *old)
    assert all(torch.equal(c.codes[first:], o.codes) and torch.equal(c.params[first:], o.params) for c, o in zip(t.caches, old))


# ---------------------------------------------------------------------------- drafted tokens

class Drafts:
    def __init__(self, T, V, probs=False, parents="chain", seed=0, sharp=3.0, max_nodes=None, pitch=0, siblings=False):
        g, r = torch.Generator().manual_seed(seed), np.random.default_rng(seed)
        self.T, self.V, B = T, V, len(T)
        self.starts = [int(x) for x in np.concatenate([[0], np.cumsum(T)])]
        N = self.starts[-1]
        self.max_nodes = max_nodes or max(T + [1])
        logits = torch.randn(N, V, generator=g) * sharp
        self.parents = None
        if parents == "tree":
            self.parents = [(-1 if t == 0 else int(r.integers(0, t)) if r.random() < 0.6 else max(0, t - 3)) for n in T for t in range(n)]
        elif parents == "flat":
            self.parents = [-1 if t == 0 else 0 for n in T for t in range(n)]
        rows = []
        for b in range(B):
            for t in range(T[b]):
                up = 0 if t == 0 else (t - 1 if self.parents is None else self.parents[self.starts[b] + t])
                rows.append(self.starts[b] + up)
        near = logits[rows] + torch.randn(N, V, generator=g) if N else logits
        buf = lambda x: torch.zeros(x.shape[0], V + pitch).copy_(torch.nn.functional.pad(x, (0, pitch))).to(DEV)[:, :V]
        self.target, self.draft = buf(torch.softmax(logits, -1)), buf(torch.softmax(near, -1)) if probs else None
        best = near.topk(min(3, V), -1).indices if N else torch.zeros(0, 1, dtype=torch.long)
        pick = torch.randint(best.shape[1], (N, 1), generator=g)
        self.tokens = best.gather(1, pick)[:, 0].to(torch.int32).tolist()
        self.ua, self.us = torch.rand(N, generator=g).to(DEV), torch.rand(B, generator=g).to(DEV)

    def run(self, stream=None):
        B = len(self.T)
        self.out = [torch.full((B, self.max_nodes), 9, dtype=torch.int32, device=DEV), i32([9] * B), i32([9] * B)]
        self.args = (self.target, i32(self.tokens), i32(self.starts), None if self.parents is None else i32(self.parents), self.ua, self.us)
        gsr.verify_drafts(*self.args, *self.out, draft_probs=self.draft, stream=stream)
        return self

    def check(self):
        paths, nexts = serving.verify(self.target.cpu(), None if self.draft is None else self.draft.cpu(), self.tokens, self.starts,
                                      self.parents, self.ua.cpu(), self.us.cpu(), self.max_nodes)
        path, counts, got = (t.tolist() for t in self.out)
        assert counts == [len(p) for p in paths]
        assert path == [p + [-1] * (self.max_nodes - len(p)) for p in paths]
        assert got == nexts
        return self


DRAFTS = {
    "one": dict(T=[1], V=10),
    "one_column": dict(T=[2, 1], V=1, probs=True),
    "chains": dict(T=[5, 1, 8, 3], V=1000, probs=True),
    "chains_sure": dict(T=[9] * 20, V=77, probs=True, sharp=8.0),
    "chains_no_probs": dict(T=[5, 4, 8, 3], V=3001),
    "trees": dict(T=[24, 1, 64, 40], V=500, parents="tree", sharp=2.0),
    "trees_flat": dict(T=[40, 64], V=12, parents="flat", sharp=0.3),
    "trees_drawn": dict(T=[24, 1, 64, 40], V=500, parents="tree", probs=True, sharp=1.0),
    "trees_drawn_flat": dict(T=[33, 64, 2], V=40, parents="flat", probs=True, sharp=0.5),
    "none_and_some": dict(T=[0, 3, 0], V=64, probs=True),
    "many": dict(T=[1 + i % 7 for i in range(300)], V=129, probs=True),
    "limit": dict(T=[9, 20], V=100, max_nodes=4, parents="tree"),
    "large_vocabulary": dict(T=[4, 3], V=151937, probs=True),
    "pitch": dict(T=[4, 6], V=4099, probs=True, pitch=13),
}


@pytest.mark.parametrize("seed", range(4))
@pytest.mark.parametrize("name", DRAFTS)
def test_verify(name, seed):
    Drafts(**DRAFTS[name], seed=seed).run().check()


def test_ends_of_the_random_numbers():
    for probs in (False, True):
        for u in (0.0, 1.0 - 2.0 ** -24):
            d = Drafts(T=[6] * 10, V=333, probs=probs, seed=5)
            d.us.fill_(u)
            d.run().check()
            d.ua.fill_(u)
            d.run().check()


def test_rows_that_leave_nothing():
    # p and q alike: nothing is left after a refusal, and the row itself is drawn from
    d = Drafts(T=[3, 2], V=50, probs=True, seed=1)
    d.draft.copy_(d.target[[0, 0, 1, 3, 3]])
    d.ua.fill_(1.0)                                   # outside [0, 1): refuses everything
    d.run().check()
    # a target row of zeros
    d.target[0] = 0.0
    d.run().check()
    assert d.out[2][0] == -1
    # one column alone
    d.target[0, 49] = 1e-30
    d.target[3] = 0.0
    d.target[3, 7] = 1.0
    d.run()
    assert d.out[2].tolist()[1] == 7


def test_what_is_no_probability_and_no_token():
    d = Drafts(T=[4, 4, 4], V=200, seed=2, parents="flat")
    d.target[0, 5], d.target[0, 6], d.target[4, 3] = float("nan"), -1.0, float("inf")
    d.tokens[1], d.tokens[2], d.tokens[6] = -1, 200, 2 ** 31 - 1
    d.run().check()
    d.parents = [-1, 3, 0, -7, -1, 0, 9, 2, -1, 2, 2, 0]      # nodes below later ones, or below none, are not reached
    d.run().check()
    d.starts = [0, 4, 8, 12]
    d.ua.fill_(float("nan"))                                # counts as 0
    d.run()
    assert d.out[1].sum() > 0


def test_verify_repeats_on_two_streams():
    ds = [Drafts(**DRAFTS["large_vocabulary"], seed=1).run().check(), Drafts(**DRAFTS["trees_drawn"], seed=2).run().check()]
    want = [[t.clone() for t in d.out] for d in ds]
    streams = [torch.cuda.Stream(DEV), torch.cuda.Stream(DEV)]
    torch.cuda.synchronize()
    for _ in range(5):
        for d, s in zip(ds, streams):
            gsr.verify_drafts(*d.args, *d.out, draft_probs=d.draft, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for d, w in zip(ds, want) for a, b in zip(d.out, w))


def test_probabilities_past_32_bits():
    d = Drafts(T=[4, 5, 3], V=700, probs=True, seed=3).run().check()
    want = [t.clone() for t in d.out]
    pitch = 2 ** 28 + 17
    for n in ("target", "draft"):
        big = torch.empty(pitch * 11 + 700, device=DEV).as_strided((12, 700), (pitch, 1))
        big.copy_(getattr(d, n))
        setattr(d, n, big)
    d.run()
    assert all(torch.equal(a, b) for a, b in zip(d.out, want))


# ---------------------------------------------------------------------------- together

def test_a_training_step_captured_beside_an_eager_one():
    """Norm and rotation, masked attention, and both gradients, in a graph that is replayed on new inputs; the same
    step runs eagerly before, between and after."""
    B, Hq, Hkv, S, D = 2, 4, 2, 96, 64
    g = torch.Generator(device=DEV).manual_seed(0)
    new = lambda *s: torch.randn(*s, generator=g, device=DEV).to(BF16)
    qkv, w, table = new(B, S, Hq + 2 * Hkv, D), new(2, D), gsr.rope_table(S, D, device=DEV)
    parts = lambda t: (t[:, :, :Hq].transpose(1, 2), t[:, :, Hq:Hq + Hkv].transpose(1, 2), t[:, :, Hq + Hkv:].transpose(1, 2))
    do = new(B, Hq, S, D)

    def step():
        q, k, v = parts(qkv)
        kw = dict(cos_sin=table, q_weight=w[0], k_weight=w[1])
        qr, kr = torch.empty(B, Hq, S, D, dtype=BF16, device=DEV), torch.empty(B, Hkv, S, D, dtype=BF16, device=DEV)
        gsr.qk_norm_rope_fwd(q, k, qr, kr, **kw)
        o, lse = torch.empty_like(do), torch.empty(B, Hq, S, device=DEV)
        gsr.masked_attention_fwd(qr, kr, v, o, lse, causal=True)
        dqr, dkr, dqkv, dw = torch.empty_like(qr), torch.empty_like(kr), torch.empty_like(qkv), torch.empty(2, D, device=DEV)
        dq, dk, dv = parts(dqkv)
        gsr.masked_attention_bwd(do, qr, kr, v, o, lse, dqr, dkr, dv, causal=True)
        gsr.qk_norm_rope_bwd(dqr, dkr, q, k, dq, dk, **kw, dq_weight=dw[0], dk_weight=dw[1])
        return [o, dqkv, dw]

    side = torch.cuda.Stream(DEV)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()                             # masked attention's first call on a stream cannot be captured
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        captured = step()
    for seed in range(3):
        qkv.copy_(new(B, S, Hq + 2 * Hkv, D))
        before = step()
        graph.replay()
        after = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(before, captured, after))
    # the gradient of the whole against fp64's
    x = qkv.double().requires_grad_()
    q, k, v = parts(x)
    W = w.double().requires_grad_()

    def rot(y, wt):
        y = y / ((y ** 2).mean(-1, keepdim=True) + 1e-6).sqrt() * wt
        c, s = table.double()[:, :D // 2], table.double()[:, D // 2:]
        a, b = y[..., :D // 2], y[..., D // 2:]
        return torch.cat([a * c - b * s, b * c + a * s], -1)

    z = rot(q, W[0]) @ rot(k, W[1]).repeat_interleave(2, 1).transpose(-1, -2) / D ** 0.5
    z = z.masked_fill(torch.ones(S, S, device=DEV).triu(1).bool(), -float("inf"))
    o = z.softmax(-1) @ v.repeat_interleave(2, 1)
    dx, dw = torch.autograd.grad(o, [x, W], do.double())
    for got, want in ((captured[0], o), (captured[1], dx), (captured[2], dw)):
        # six roundings to bf16 on the way, each 2^-9 of its terms; norms of the whole
        assert (got.double() - want).norm() <= 6 * 2.0 ** -8 * want.norm()


@pytest.mark.parametrize("captured", [False, True])
def test_serving_steps_with_drafts(captured):
    """Prompts, then steps of drafted trees: block tables, rotated writes into the cache of 4 bits, attention over it and
    verification, against the oracle; the step's lengths stay on the device, so it is captured once and replayed."""
    B, Hq, Hkv, D, page, W, V, T = 3, 8, 2, 64, 16, 8, 97, 6
    g = torch.Generator(device=DEV).manual_seed(4)
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV)
    table, weights = gsr.rope_table(200, D, device=DEV), (1 + 0.2 * rnd(2, D)).to(F16)
    kc, vc = (gsr.kv_cache4(30, page, Hkv, D, F16, DEV) for _ in range(2))
    free, blocks = torch.randperm(30, generator=g, device=DEV).to(torch.int32), torch.full((B, W), -1, dtype=torch.int32, device=DEV)
    head, lens = i32([0]), i32([0] * B)

    class Step:
        def __init__(self, N):
            self.N = N
            self.new, self.lens_out, self.head_out, self.starts = i32([0] * B), i32([0] * B), i32([0]), i32([0] * (B + 1))
            self.pos, self.slots, self.counts = i32([0] * N), i32([0] * N), i32([0] * 3)
            self.qkv = torch.zeros(N, Hq + 2 * Hkv, D, dtype=F16, device=DEV)
            self.q, self.o = torch.zeros(N, Hq, D, dtype=F16, device=DEV), torch.zeros(N, Hq, D, dtype=F16, device=DEV)
            self.parents, self.tokens = i32([-1] * N), i32([0] * N)
            self.target, self.ua, self.us = torch.zeros(N, V, device=DEV), torch.zeros(N, device=DEV), torch.zeros(B, device=DEV)
            self.path, self.kept, self.next = torch.zeros(B, T, dtype=torch.int32, device=DEV), i32([0] * B), i32([0] * B)

        def run(self, attend=True):
            gsr.kv_block_tables(lens, self.new, free, head, blocks, page, self.lens_out, self.head_out, self.starts, self.pos, self.slots, self.counts)
            k, v = self.qkv[:, Hq:Hq + Hkv], self.qkv[:, Hq + Hkv:]
            gsr.kv_cache4_append_rope(k, v, self.slots, kc, vc, positions=self.pos, cos_sin=table, Q=self.qkv[:, :Hq], Q_out=self.q,
                                      q_weight=weights[0], k_weight=weights[1])
            if attend:
                gsr.tree_attention4_fwd(self.q, kc, vc, blocks, self.lens_out, self.starts, self.parents, self.o, T)
                gsr.verify_drafts(self.target, self.tokens, self.starts, self.parents, self.ua, self.us, self.path, self.kept, self.next)

    first = Step(70)
    first.new.copy_(i32([40, 7, 19]))
    first.qkv.copy_(rnd(70, Hq + 2 * Hkv, D))
    first.run(attend=False)
    assert first.counts.tolist() == [66, 6, 0] and torch.all(first.q[66:] == 0)
    lens.copy_(first.lens_out)
    head.copy_(first.head_out)
    step = Step(B * T)
    graph = None
    for i in range(4):
        new = [[6, 4, 5], [1, 6, 6], [3, 0, 6], [6, 6, 6]][i]
        step.new.copy_(i32(new))
        step.qkv.copy_(rnd(B * T, Hq + 2 * Hkv, D))
        par = [[-1, 0, 0, 1, 1, 3][:n] for n in new]
        step.parents.copy_(i32([x for p in par for x in p] + [-1] * (B * T - sum(new))))
        step.tokens.copy_(torch.randint(V, (B * T,), generator=g, device=DEV).to(torch.int32))
        step.target.copy_(torch.softmax(4 * rnd(B * T, V), -1))
        at = torch.arange(B * T, device=DEV)
        step.target[at, step.tokens.long().roll(-1)] += 0.3        # some drafts are likely
        step.ua.copy_(torch.rand(B * T, generator=g, device=DEV))
        step.us.copy_(torch.rand(B, generator=g, device=DEV))
        if captured and graph is None:
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step.run()
        graph.replay() if captured else step.run()
        torch.cuda.synchronize()
        n, starts, kv = sum(new), step.starts.tolist(), step.lens_out.tolist()
        assert step.counts.tolist()[0] == n and step.counts.tolist()[2] == 0
        k, v = (serving.values4(c.codes.cpu().numpy(), c.params) for c in (kc, vc))
        args = (blocks.cpu().numpy(), kv, starts, step.parents.tolist(), 0.0, 0.0, None, T)
        want, terms = llm.tree_attention(step.q, k[0], v[0], *args)[0][:n], llm.tree_attention(step.q, k[0], v[1], *args)[1][:n]
        got, u = llm.f64(step.o)[:n], unit(F16)
        assert np.all(np.abs(got - want) <= (u + 2.0 ** -13) * terms * (1 + u) + u * np.abs(want) + 2.0 ** -25)
        # the rows that the step brought, where the cache holds them: half a step and the roundings that the file's head lists
        slots = step.slots[:n].long().cpu().numpy()
        cos, sin = (a[:, None] for a in serving.angles(table, step.pos[:n].cpu().numpy(), D))
        y, mag = serving.norm_rope(step.qkv[:n, Hq:Hq + Hkv], llm.f64(weights[1]), cos, sin, D)
        s, m = (np.repeat(llm.f64(kc.params)[slots // page, slots % page][..., i], 64, -1) for i in (0, 1))
        assert np.all(np.abs(k[0][slots // page, slots % page] - y) <= s / 2 + 15 * u * s + u * np.abs(m) + 2.0 ** -17 * mag + 2.0 ** -21)
        paths, nexts = serving.verify(step.target.cpu(), None, step.tokens.tolist(), starts, step.parents.tolist(), step.ua.cpu(), step.us.cpu(), T)
        assert step.kept.tolist() == [len(p) for p in paths] and step.next.tolist() == nexts
        assert step.path.tolist() == [p + [-1] * (T - len(p)) for p in paths]
        # the kept tokens stay: in earnest their rows are moved together first
        lens.add_(step.kept + 1)
        lens.copy_(torch.minimum(lens, step.lens_out))
        head.copy_(step.head_out)
        for b in range(B):                    # pages behind the kept tokens go back in this test by never being used again
            blocks[b, -(-int(lens[b]) // page):] = -1
    assert int(head) <= 30


@pytest.mark.parametrize("four", [False, True])
def test_a_branching_tree_is_its_paths(four):
    """Nodes at the positions that their depth gives them: rotated queries, cache rows and answers of every path from the root to a
    leaf are those of the same tokens written as a chain; so are the answers after the kept rows were moved together."""
    B, Hq, Hkv, D, page, W, V, T = 2, 4, 2, 64, 16, 4, 50, 7
    ctxs, parents = [21, 5], [[-1, 0, 0, 1, 1, 3, 2], [-1, 0, 1, 0, 3, 3, 5]]
    g = torch.Generator(device=DEV).manual_seed(9)
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV).to(F16)
    cs, w = gsr.rope_table(100, D, device=DEV), (1 + 0.2 * rnd(2, D).float()).to(F16)
    prompts, nodes = [rnd(n, Hq + 2 * Hkv, D) for n in ctxs], [rnd(T, Hq + 2 * Hkv, D) for _ in ctxs]
    last = rnd(B, Hq + 2 * Hkv, D)
    append, attend = (gsr.kv_cache4_append_rope, gsr.tree_attention4_fwd) if four else (gsr.kv_cache_append_rope, gsr.tree_attention_fwd)

    class Server:
        def __init__(self, seed):
            gen = torch.Generator().manual_seed(seed)
            if four:
                self.caches = [gsr.kv_cache4(20, page, Hkv, D, F16, DEV) for _ in range(2)]
                self.parts = [t for c in self.caches for t in c]
            else:
                self.caches = self.parts = [torch.zeros(20, page, Hkv, D, dtype=F16, device=DEV) for _ in range(2)]
            self.free, self.table = torch.randperm(20, generator=gen).to(torch.int32).to(DEV), torch.full((B, W), -1, dtype=torch.int32, device=DEV)
            self.lens, self.head = i32([0] * B), i32([0])

        def step(self, new, parents=None, depth=None):
            """Rows of each request; returns rotated queries, answers and the rows' slots."""
            counts = [len(x) for x in new]
            N = sum(counts) + 2                     # padding behind the last
            rows = torch.cat(new + [torch.zeros(2, Hq + 2 * Hkv, D, dtype=F16, device=DEV)])
            lens_out, head_out, q_starts, positions, slots = i32([0] * B), i32([0]), i32([0] * (B + 1)), i32([0] * N), i32([0] * N)
            gsr.kv_block_tables(self.lens, i32(counts), self.free, self.head, self.table, page, lens_out, head_out, q_starts, positions, slots,
                                i32([0] * 3))
            if depth is not None:
                request = torch.tensor([b for b in range(B) for _ in range(counts[b])] + [0, 0], device=DEV)
                index = torch.arange(N, device=DEV) - q_starts[request]
                depth = torch.tensor([x for d in depth for x in d] + [0, 0], device=DEV)
                positions = torch.where(positions < 0, positions, positions - index + depth).to(torch.int32)
            q, o = torch.full((N, Hq, D), 7.0, dtype=F16, device=DEV), torch.full((N, Hq, D), 7.0, dtype=F16, device=DEV)
            append(rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:], slots, *self.caches, positions=positions, cos_sin=cs, Q=rows[:, :Hq], Q_out=q,
                   q_weight=w[0], k_weight=w[1])
            if max(counts) <= T:
                up = None if parents is None else i32([x for p in parents for x in p] + [-1, -1])
                attend(q, *self.caches, self.table, lens_out, q_starts, up, o, T)
            self.lens_out, self.head, self.q_starts = lens_out, head_out, q_starts
            return q, o, slots

        def rows(self, slots):
            slots = slots.long()
            return [t[slots // page, slots % page] for t in self.parts]

        def tolerance(self, q, parents):
            """Of an answer, twice: both sides are within it of fp64's answer over the rows that the caches hold."""
            k, v = ((serving.values4(c.codes.cpu().numpy(), c.params) for c in self.caches) if four
                    else ((llm.f64(c), np.abs(llm.f64(c))) for c in self.caches))
            args = (self.table.cpu().numpy(), self.lens_out.tolist(), self.q_starts.tolist(), None if parents is None else [x for p in parents for x in p],
                    0.0, 0.0, None, T)
            n, u = self.q_starts.tolist()[-1], unit(F16)
            want, terms = llm.tree_attention(q, k[0], v[0], *args)[0][:n], llm.tree_attention(q, k[0], v[1], *args)[1][:n]
            return 2 * ((u + 2.0 ** -13) * terms * (1 + u) + u * np.abs(want) + 2.0 ** -25)

    depth, tree = [], Server(1)
    for p in parents:
        d = []
        for up in p:
            d.append(0 if up < 0 else d[up] + 1)
        depth.append(d)
    assert any(d != list(range(T)) for d in depth)
    tree.step(prompts)
    tree.lens.copy_(tree.lens_out)
    q, o, slots = tree.step(nodes, parents, depth)
    tol, held = tree.tolerance(q, parents), tree.rows(slots[:B * T])
    assert torch.all(q[B * T:] == 0) and torch.all(o[B * T:] == 7.0)
    paths = []
    for p in parents:
        ways = []
        for leaf in range(T):
            way = [leaf]
            while p[way[0]] >= 0:
                way.insert(0, p[way[0]])
            ways.append(way)
        paths.append(ways)
    for leaf in range(T):
        chain = Server(2 + leaf)
        chain.step(prompts)
        chain.lens.copy_(chain.lens_out)
        ways = [ways[leaf] for ways in paths]
        cq, co, cslots = chain.step([x[way] for x, way in zip(nodes, ways)])
        at = torch.tensor([b * T + n for b in range(B) for n in ways[b]], device=DEV)
        assert torch.equal(cq[:-2], q[at])
        assert all(torch.equal(a, b[at]) for a, b in zip(chain.rows(cslots[:-2]), held))
        assert np.all(np.abs(llm.f64(co[:-2]) - llm.f64(o[at])) <= tol[at.cpu().numpy()])
    # a path of each request is kept: node 0 and two or three drafts below it
    tokens, probs = i32(list(range(B * T))), torch.full((B * T, V), 0.5 / V, device=DEV)
    ways = [paths[0][5], paths[1][6]]
    for b, way in enumerate(ways):
        for up, n in zip(way, way[1:]):
            probs[b * T + up] *= 0.0
            probs[b * T + up, b * T + n] = 1.0
        probs[b * T + way[-1]] = 0.0
        probs[b * T + way[-1], V - 1] = 1.0
    path, kept, following = torch.full((B, T), 9, dtype=torch.int32, device=DEV), i32([9] * B), i32([9] * B)
    gsr.verify_drafts(probs, tokens, tree.q_starts, i32(parents).flatten(), torch.full((B * T,), 0.5, device=DEV), torch.full((B,), 0.5, device=DEV),
                      path, kept, following)
    assert [path[b, :kept[b]].tolist() for b in range(B)] == [way[1:] for way in ways] and following.tolist() == [V - 1] * B
    b, i = (path >= 0).nonzero(as_tuple=True)
    src, dst = tree.lens[b] + path[b, i], tree.lens[b] + i + 1
    row = lambda r: (tree.table[b, r // page].long(), r % page)
    for t in tree.parts:
        t[row(dst)] = t[row(src)]
    tree.lens.add_(kept + 1)
    # the next token after them, and after the same tokens as a chain
    chain = Server(20)
    chain.step(prompts)
    chain.lens.copy_(chain.lens_out)
    chain.step([x[way] for x, way in zip(nodes, ways)])
    chain.lens.copy_(chain.lens_out)
    new = [last[b:b + 1] for b in range(B)]
    (q, o, slots), (cq, co, cslots) = tree.step(new), chain.step(new)
    assert tree.lens_out.tolist() == chain.lens_out.tolist() and torch.equal(q, cq)
    assert all(torch.equal(x, y) for x, y in zip(tree.rows(slots[:B]), chain.rows(cslots[:B])))
    assert np.all(np.abs(llm.f64(o[:B]) - llm.f64(co[:B])) <= tree.tolerance(q, None))
