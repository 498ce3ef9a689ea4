"""Refusals of head norms with rotation, rotated cache writes, the cache of 4 bits and drafted tokens' verification,
without a GPU: the device addresses are fake, and every call is refused before any CUDA call."""
import pytest

import tensor_core_gemm_multistage_gb300 as gsr
from tensor_core_gemm_multistage_gb300.llm import _Tensor, _TreeDesc
from tensor_core_gemm_multistage_gb300.serving import _Cache4, _RopeDesc, _VerifyDesc

INVALID, ALIGN, ALIAS, OK = (gsr.Status.ERR_INVALID_ARG, gsr.Status.ERR_ALIGNMENT, gsr.Status.ERR_ALIAS, gsr.Status.OK)
GB = 1 << 30


@pytest.fixture(scope="module", autouse=True)
def built():
    gsr.build()
    yield


@pytest.fixture
def accepted():
    """Whether a call passes its checks: without a GPU it then fails at its first CUDA call."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("fake device addresses that pass the checks: only without a GPU")
    return lambda status: status not in (INVALID, ALIGN, ALIAS)


def dense(addr, H, S, D=64, B=2):
    return _Tensor(addr, H * S * D, S * D, D)


def rope_desc(**over):
    d = dict(batch=2, heads_q=4, heads_kv=2, seq=10, head_dim=64, rotary_dim=64, table_rows=100, dtype=0, eps=1e-6,
             q_weight=20 * GB, k_weight=21 * GB, cos_sin=22 * GB, positions=23 * GB)
    d.update(over)
    return _RopeDesc(**d)


def fwd(desc=None, **t):
    ops = dict(Q=dense(1 * GB, 4, 10), K=dense(2 * GB, 2, 10), Q_out=dense(3 * GB, 4, 10), K_out=dense(4 * GB, 2, 10))
    ops.update(t)
    return gsr.lib().qk_norm_rope_fwd(rope_desc(**(desc or {})), *ops.values(), None)


def bwd(desc=None, dqw=24 * GB, dkw=25 * GB, ws=26 * GB, ws_bytes=1 << 20, **t):
    ops = {n: dense((i + 1) * GB, 2 if "K" in n else 4, 10) for i, n in enumerate(("dQ_out", "dK_out", "Q", "K", "dQ", "dK"))}
    ops.update(t)
    return gsr.lib().qk_norm_rope_bwd(rope_desc(**(desc or {})), *ops.values(), dqw, dkw, ws, ws_bytes, None)


@pytest.mark.parametrize("desc", [
    dict(batch=-1), dict(seq=2 ** 31), dict(head_dim=96), dict(dtype=2), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
    dict(rotary_dim=8), dict(rotary_dim=24), dict(rotary_dim=80), dict(rotary_dim=0), dict(positions=None, table_rows=9),
    dict(batch=2 ** 15, seq=2 ** 15), dict(heads_kv=-1)])
def test_rope_descriptions(desc):
    assert fwd(desc) == INVALID and bwd(desc) == INVALID
    assert gsr.lib().qk_norm_rope_bwd_workspace(rope_desc(**desc)) == -1


def test_rope_operands(accepted):
    assert accepted(fwd()) and accepted(bwd())
    assert accepted(fwd(dict(positions=None))) and accepted(fwd(dict(cos_sin=None, positions=None, rotary_dim=0, table_rows=0)))
    assert accepted(fwd(dict(heads_kv=0), K=None, K_out=None))
    assert fwd(Q=None) == INVALID and fwd(K_out=None) == INVALID and fwd(Q=_Tensor(None, 1, 1, 1)) == INVALID
    assert fwd(Q=_Tensor(GB + 8, 2560, 640, 64)) == ALIGN and fwd(Q=_Tensor(GB, 2560, 644, 64)) == ALIGN
    assert fwd(Q=_Tensor(GB, 0, 640, 64)) == INVALID
    assert fwd(dict(cos_sin=22 * GB + 4)) == ALIGN and fwd(dict(q_weight=20 * GB + 2)) == ALIGN and fwd(dict(positions=23 * GB + 2)) == ALIGN
    # in place is fine, beside it is not
    assert accepted(fwd(Q_out=dense(1 * GB, 4, 10), K_out=dense(2 * GB, 2, 10)))
    assert fwd(Q_out=dense(1 * GB + 128, 4, 10)) == ALIAS and fwd(Q_out=dense(2 * GB, 4, 10)) == ALIAS
    assert fwd(Q_out=_Tensor(1 * GB, 2560, 64, 256)) == ALIAS           # Q's buffer in another order
    assert fwd(K_out=dense(3 * GB, 2, 10)) == ALIAS and fwd(Q_out=dense(22 * GB, 4, 10)) == ALIAS
    assert fwd(K_out=dense(23 * GB, 2, 10)) == ALIAS and fwd(K_out=dense(21 * GB, 2, 10)) == ALIAS
    assert fwd(dict(seq=0)) == OK and fwd(dict(batch=0)) == OK and fwd(dict(heads_q=0, heads_kv=0)) == OK
    assert gsr.lib().qk_norm_rope_fwd(None, None, None, None, None, None) == INVALID


def test_rope_gradient_operands(accepted):
    assert bwd(dqw=None) == INVALID and bwd(dict(k_weight=None)) == INVALID      # a weight and its gradient go together
    plain = dict(q_weight=None, k_weight=None)
    assert accepted(bwd(plain, dqw=None, dkw=None, Q=None, K=None, ws=None, ws_bytes=0))
    assert accepted(bwd(dQ=dense(1 * GB, 4, 10), dK=dense(4 * GB, 2, 10)))        # in place of dQ_out, of K
    assert bwd(dQ=dense(2 * GB, 4, 10)) == ALIAS and bwd(dK=dense(5 * GB, 2, 10)) == ALIAS
    assert bwd(dqw=3 * GB + 64) == ALIAS and bwd(dkw=24 * GB) == ALIAS and bwd(dkw=22 * GB) == ALIAS
    assert bwd(ws=5 * GB) == ALIAS and bwd(ws=24 * GB) == ALIAS and bwd(ws=26 * GB + 4) == ALIGN and bwd(dqw=24 * GB + 2) == ALIGN
    need = gsr.qk_norm_rope_bwd_workspace(2, 4, 2, 10, 64)
    assert need > 0 and bwd(ws_bytes=need - 1) == INVALID
    with pytest.raises(gsr.GsrError):
        gsr.qk_norm_rope_bwd_workspace(2, 4, 2, 10, 96)


def cache4(addr, H=2, page=16, D=64, apart=GB // 4):
    return _Cache4(_Tensor(addr, H * page * D // 2, page * D // 2, D // 2), _Tensor(addr + apart, H * page * D // 32, page * D // 32, D // 32))


def cache16(addr, H=2, page=16, D=64):
    return _Tensor(addr, page * H * D, D, H * D)


def append(four, desc=None, pages=10, page=16, slots=8 * GB, Q=_Tensor(1 * GB, 0, 64, 256), Q_out=_Tensor(7 * GB, 0, 64, 256),
           K=_Tensor(2 * GB, 0, 64, 384), V=_Tensor(3 * GB, 0, 64, 384), kc=None, vc=None):
    L, make = gsr.lib(), cache4 if four else cache16
    d = rope_desc(**dict(dict(batch=1), **(desc or {})))
    call = L.kv_cache4_append_rope if four else L.kv_cache_append_rope
    return call(d, Q, K, V, slots, Q_out, kc or make(4 * GB), vc or make(5 * GB), pages, page, None)


@pytest.mark.parametrize("four", [False, True])
def test_append_refusals(four, accepted):
    assert accepted(append(four)) and accepted(append(four, Q_out=_Tensor(1 * GB, 0, 64, 256)))
    assert accepted(append(four, dict(heads_q=0), Q=None, Q_out=None)) and accepted(append(four, dict(cos_sin=None, positions=None)))
    for bad in (dict(batch=2), dict(positions=None), dict(seq=-1), dict(head_dim=32), dict(rotary_dim=40)):
        assert append(four, bad) == INVALID, bad
    assert append(four, slots=None) == INVALID and append(four, page=0) == INVALID and append(four, pages=2 ** 28) == INVALID
    assert append(four, Q=None) == INVALID and append(four, K=None) == INVALID and append(four, slots=8 * GB + 1) == ALIGN
    make = cache4 if four else cache16
    assert append(four, vc=make(4 * GB)) == ALIAS and append(four, kc=make(2 * GB)) == ALIAS and append(four, kc=make(8 * GB)) == ALIAS
    assert append(four, kc=make(22 * GB)) == ALIAS and append(four, kc=make(7 * GB)) == ALIAS and append(four, kc=make(1 * GB)) == ALIAS
    assert append(four, Q_out=_Tensor(2 * GB, 0, 64, 256)) == ALIAS and append(four, Q_out=_Tensor(8 * GB, 0, 64, 256)) == ALIAS
    assert append(four, dict(seq=0)) == OK


def test_caches_of_4_bits(accepted):
    c = cache4(4 * GB)
    part = lambda codes=None, params=None: _Cache4(codes or c.codes, params or c.params)
    for bad in (_Tensor(4 * GB, 1024, 512, 0), _Tensor(4 * GB, 1024, 512, -32), _Tensor(None, 1024, 512, 32), _Tensor(4 * GB, 1024, 512, 16),
                _Tensor(4 * GB, 512, 512, 32), _Tensor(4 * GB, 512, 1024, 32), _Tensor(4 * GB, 1 << 45, 512, 32)):
        assert append(True, kc=part(codes=bad)) == INVALID, bad.stride_row
    assert append(True, kc=part(codes=_Tensor(4 * GB + 8, 1024, 512, 32))) == ALIGN
    assert append(True, kc=part(codes=_Tensor(4 * GB, 1024, 520, 32))) == ALIGN
    assert append(True, kc=part(params=_Tensor(GB * 17 // 4 + 2, 64, 32, 2))) == ALIGN
    assert append(True, kc=part(params=_Tensor(GB * 17 // 4, 65, 33, 2))) == ALIGN
    assert append(True, kc=part(params=_Tensor(GB * 17 // 4, 64, 32, 1))) in (INVALID, ALIGN)
    # codes and params of one cache, or of both, in one place
    assert append(True, kc=part(params=_Tensor(4 * GB, 64, 32, 2))) == ALIAS
    assert append(True, vc=_Cache4(cache4(5 * GB).codes, c.params)) == ALIAS
    # rows first, heads first, and both caches' pages side by side
    assert accepted(append(True, kc=part(codes=_Tensor(4 * GB, 1024, 32, 64))))
    side = lambda k: _Cache4(_Tensor(4 * GB + 1024 * k, 2048, 512, 32), _Tensor(6 * GB + 128 * k, 128, 32, 2))
    assert accepted(append(True, kc=side(0), vc=side(1)))


def read(k=None, v=None, slots=8 * GB, K=_Tensor(1 * GB, 0, 64, 128), V=_Tensor(2 * GB, 0, 64, 128), n=5, H=2, D=64, pages=10, page=16, dtype=0):
    return gsr.lib().kv_cache4_read(k or cache4(4 * GB), v or cache4(5 * GB), slots, K, V, n, H, D, pages, page, dtype, None)


def test_read_refusals(accepted):
    assert accepted(read()) and read(n=0) == OK
    assert read(n=-1) == INVALID and read(D=32) == INVALID and read(dtype=2) == INVALID and read(page=0) == INVALID
    assert read(slots=None) == INVALID and read(K=None) == INVALID and read(n=2 ** 30, H=4) == INVALID
    assert read(V=_Tensor(1 * GB, 0, 64, 128)) == ALIAS and read(K=_Tensor(4 * GB, 0, 64, 128)) == ALIAS
    assert read(K=_Tensor(GB * 21 // 4, 0, 64, 128)) == ALIAS and read(K=_Tensor(8 * GB, 0, 64, 128)) == ALIAS


def tree(desc=None, q=1 * GB, k=None, v=None, table=6 * GB, lens=7 * GB, starts=8 * GB, parents=9 * GB, o=3 * GB, ws=None, ws_bytes=0):
    d = dict(batch=2, total_q=6, heads_q=4, heads_kv=2, head_dim=64, num_pages=10, page_size=16, table_width=5,
             max_nodes=3, q_stride_row=256, q_stride_head=64, o_stride_row=256, o_stride_head=64)
    d.update(desc or {})
    return gsr.lib().tree_attention4_fwd(_TreeDesc(**d), q, k or cache4(4 * GB), v or cache4(5 * GB), table, lens, starts, parents, o, ws, ws_bytes, None)


def test_tree4_refusals(accepted):
    assert accepted(tree()) and accepted(tree(parents=None))
    for bad in (dict(batch=-1), dict(head_dim=32), dict(dtype=3), dict(max_nodes=0), dict(max_nodes=65), dict(heads_kv=3),
                dict(softcap=-2.0), dict(page_size=12), dict(total_q=2 ** 31), dict(alibi_slopes=10 * GB), dict(q_stride_row=0),
                dict(batch=2 ** 30, max_nodes=60)):
        assert tree(bad) == INVALID, bad
    assert tree(q=None) == INVALID and tree(table=None) == INVALID and tree(lens=None) == INVALID
    assert tree(q=GB + 8) == ALIGN and tree(parents=9 * GB + 1) == ALIGN
    much = dict(batch=48, total_q=48, heads_q=32, heads_kv=8, table_width=4096, max_nodes=1, q_stride_row=2048, o_stride_row=2048)
    size = gsr.tree_attention4_workspace(48, 48, 32, 8, 64, 10, 16, 4096, 1)
    assert gsr.tree_attention4_workspace(2, 6, 4, 2, 64, 10, 16, 5, 3) == 0 and size > 0
    big = lambda a: cache4(a, H=8)
    assert accepted(tree(much, k=big(4 * GB), v=big(5 * GB), ws=10 * GB, ws_bytes=size))
    assert tree(much, k=big(4 * GB), v=big(5 * GB), ws=10 * GB, ws_bytes=size - 1) == INVALID
    assert tree(much, k=big(4 * GB), v=big(5 * GB), ws=10 * GB + 8, ws_bytes=size) == ALIGN
    for at in (1, 3, 4, 5, 6, 7, 8, 9):
        assert tree(much, k=big(4 * GB), v=big(5 * GB), ws=at * GB, ws_bytes=size) == ALIAS, at
    with pytest.raises(gsr.GsrError):
        gsr.tree_attention4_workspace(2, 6, 4, 3, 64, 10, 16, 5, 3)
    assert tree(o=1 * GB) == ALIAS and tree(o=4 * GB) == ALIAS and tree(o=GB * 17 // 4) == ALIAS and tree(o=7 * GB) == ALIAS
    assert tree(dict(batch=0)) == OK and tree(dict(total_q=0)) == OK


def verify(desc=None, **over):
    d = dict(batch=2, total_q=6, vocab=100, max_nodes=4, target_stride_row=100, draft_stride_row=128)
    d.update(desc or {})
    names = ("target", "draft", "tokens", "starts", "parents", "u_accept", "u_sample", "path", "counts", "next")
    at = {n: (i + 1) * GB for i, n in enumerate(names)}
    at.update(over)
    return gsr.lib().verify_drafts(_VerifyDesc(**d), *at.values(), None)


def test_verify_refusals(accepted):
    assert accepted(verify()) and accepted(verify(draft=None)) and accepted(verify(parents=None)) and verify(dict(batch=0)) == OK
    for bad in (dict(batch=-1), dict(batch=2 ** 28), dict(vocab=0), dict(vocab=2 ** 25), dict(max_nodes=0), dict(max_nodes=65),
                dict(target_stride_row=99), dict(draft_stride_row=5), dict(total_q=-1)):
        assert verify(bad) == INVALID, bad
    for n in ("target", "tokens", "starts", "u_accept", "u_sample", "path", "counts", "next"):
        assert verify(**{n: None}) == INVALID, n
        assert verify(**{n: 30 * GB + 2}) == ALIGN, n
    for out in (8, 9, 10):
        for other in [i for i in range(1, 11) if i != out]:
            assert verify(**{("path", "counts", "next")[out - 8]: other * GB}) == ALIAS, (out, other)
    assert gsr.lib().verify_drafts(None, *[None] * 11) == INVALID


def test_binding_refusals():
    import torch
    t, i = torch.zeros(1, 2, 4, 64, dtype=torch.float16), torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        gsr.qk_norm_rope_fwd(t, t, t, t)                               # not on a GPU
    with pytest.raises(TypeError):
        gsr.qk_norm_rope_bwd(t, t, t.float(), t, t, t)
    c = gsr.kv_cache4(3, 16, 2, 64, torch.float16, device="cpu")
    with pytest.raises(ValueError):
        gsr.kv_cache_append_rope(t[0], t[0], i, t, t)
    with pytest.raises(ValueError):
        gsr.kv_cache4_append_rope(t[0], t[0], i, c, c)
    with pytest.raises(ValueError):
        gsr.kv_cache4_read(c, c, i, t[0], t[0])
    with pytest.raises(ValueError):
        gsr.tree_attention4_fwd(t[0], c, c, i, i, i, None, t[0], 1)
    with pytest.raises(ValueError):
        gsr.verify_drafts(t[0, 0].float(), i, i, None, i, i, i, i, i)
    with pytest.raises(ValueError):
        gsr.kv_cache4(1, 16, 1, 96)


def test_packed_structures():
    """Calls pack the structures as bytes: sizes, and each field's place, are those of the declared ones."""
    import ctypes
    from tensor_core_gemm_multistage_gb300 import serving
    for pack, kind in ((serving._pack_tensor, _Tensor), (serving._pack_cache4, _Cache4), (serving._pack_rope, _RopeDesc),
                       (serving._pack_tree, _TreeDesc), (serving._pack_verify, _VerifyDesc)):
        fields = [f for name, t in kind._fields_ for f in (t._fields_ if issubclass(t, ctypes.Structure) else [(name, t)])]
        made, values = pack(*range(1, len(fields) + 1)), []
        assert len(made) == ctypes.sizeof(kind)
        held = kind.from_buffer_copy(made)
        for name, t in kind._fields_:
            x = getattr(held, name)
            values += [getattr(x, n) for n, _ in t._fields_] if issubclass(t, ctypes.Structure) else [x]
        assert values == list(range(1, len(fields) + 1))


def test_tables_of_angles():
    import math
    import torch
    t = gsr.rope_table(100001, 64, device="cpu")
    assert t.shape == (100001, 64) and t.dtype is torch.float32 and torch.all(t[0, :32] == 1) and torch.all(t[0, 32:] == 0)
    for p, k in ((1, 0), (77, 3), (100000, 1), (100000, 31)):
        a = p * 10000.0 ** (-2 * k / 64)
        assert abs(float(t[p, k]) - math.cos(a)) < 2 ** -23 and abs(float(t[p, 32 + k]) - math.sin(a)) < 2 ** -23
