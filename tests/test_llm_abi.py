"""Refusals of masked attention, tree attention, block tables and cache writes, without a GPU: the
device addresses are fake, and every call is refused before any CUDA call."""
import ctypes

import pytest

import tensor_core_gemm_multistage_gb300 as gsr
from tensor_core_gemm_multistage_gb300 import llm
from tensor_core_gemm_multistage_gb300.llm import _AttentionDesc, _Tensor, _TreeDesc

INVALID, ALIGN, ALIAS, OK = (gsr.Status.ERR_INVALID_ARG, gsr.Status.ERR_ALIGNMENT, gsr.Status.ERR_ALIAS, gsr.Status.OK)
GB = 1 << 30


@pytest.fixture(scope="module", autouse=True)
def built():
    gsr.build()
    yield


def dense(addr, B, H, S, D):
    return _Tensor(addr, H * S * D, S * D, D)


def fwd(desc=None, lse=None, ws=None, ws_bytes=0, **t):
    d = dict(batch=2, heads_q=4, heads_kv=2, seq_q=100, seq_kv=100, head_dim=64, dtype=0, causal=1)
    d.update(desc or {})
    ops = dict(Q=dense(1 * GB, 2, 4, 100, 64), K=dense(2 * GB, 2, 2, 100, 64), V=dense(3 * GB, 2, 2, 100, 64),
               O=dense(4 * GB, 2, 4, 100, 64))
    ops.update(t)
    return gsr.lib().masked_attention_fwd(_AttentionDesc(**d), ops["Q"], ops["K"], ops["V"], ops["O"], lse, ws, ws_bytes, None)


def bwd(desc=None, lse=9 * GB, ws=10 * GB, ws_bytes=1 << 20, **t):
    d = dict(batch=2, heads_q=4, heads_kv=2, seq_q=100, seq_kv=100, head_dim=64, dtype=0, causal=1)
    d.update(desc or {})
    ops = {n: dense((i + 1) * GB, 2, 4 if n in ("dO", "Q", "O", "dQ") else 2, 100, 64)
           for i, n in enumerate(("dO", "Q", "K", "V", "O", "dQ", "dK", "dV"))}
    ops.update(t)
    o = ops
    return gsr.lib().masked_attention_bwd(_AttentionDesc(**d), o["dO"], o["Q"], o["K"], o["V"], o["O"], lse, o["dQ"],
                                          o["dK"], o["dV"], ws, ws_bytes, None)


@pytest.mark.parametrize("desc", [
    dict(batch=-1), dict(seq_q=2 ** 31), dict(head_dim=96), dict(dtype=2), dict(heads_kv=3), dict(heads_kv=0),
    dict(softcap=-1.0), dict(softcap=float("nan")), dict(softmax_scale=float("inf")),
    dict(doc_bounds=16 * GB, num_docs=0), dict(num_docs=2), dict(doc_bounds=16 * GB, num_docs=2, seq_q=99),
    dict(prefix_lens=16 * GB, causal=0), dict(batch=2 ** 20, heads_q=2 ** 12)])
def test_attention_descriptions(desc):
    assert fwd(desc) == INVALID and bwd(desc) == INVALID
    d = dict(batch=2, heads_q=4, heads_kv=2, seq_q=100, seq_kv=100, head_dim=64, dtype=0, causal=1)
    d.update(desc)
    assert gsr.lib().masked_attention_bwd_workspace(_AttentionDesc(**d)) == -1


def test_attention_pointers_strides_and_alignment():
    assert fwd(Q=_Tensor(None, 25600, 6400, 64)) == INVALID
    assert fwd(K=_Tensor(2 * GB + 8, 12800, 6400, 64)) == ALIGN
    assert fwd(V=_Tensor(3 * GB, 12800, 6404, 64)) == ALIGN
    assert fwd(Q=_Tensor(1 * GB, 0, 6400, 64)) == INVALID              # a broadcast
    assert fwd(Q=_Tensor(1 * GB, 25600, 6400, -64)) == INVALID
    assert fwd(O=_Tensor(4 * GB, 25600, 6400, 32)) == INVALID          # rows of O on top of each other
    assert fwd(Q=_Tensor(1 * GB, 1 << 45, 6400, 64)) == INVALID
    assert fwd(lse=9 * GB + 2) == ALIGN
    assert fwd(dict(alibi_slopes=9 * GB + 2)) == ALIGN
    assert gsr.lib().masked_attention_fwd(None, None, None, None, None, None, None, 0, None) == INVALID
    assert bwd(lse=None) == INVALID
    assert bwd(ws_bytes=llm.masked_attention_bwd_workspace(2, 4, 2, 100, 100, 64) - 1) == INVALID
    assert bwd(ws=10 * GB + 8) == ALIGN


def test_attention_aliases():
    assert fwd(O=dense(1 * GB, 2, 4, 100, 64)) == ALIAS
    assert fwd(O=dense(2 * GB - 64, 2, 4, 100, 64)) == ALIAS
    assert fwd(lse=4 * GB + 16) == ALIAS
    assert bwd(dQ=dense(2 * GB, 2, 4, 100, 64)) == ALIAS
    assert bwd(dV=dense(7 * GB, 2, 2, 100, 64)) == ALIAS               # dK and dV in one place
    assert bwd(ws=3 * GB) == ALIAS
    assert bwd(lse=10 * GB) == ALIAS
    assert bwd(lse=6 * GB) == ALIAS
    # the parts of one fused buffer lie side by side unless they overlap in its rows
    part = lambda base, col: _Tensor(base + 2 * 64 * col, 100 * 8 * 64, 64, 8 * 64)
    assert bwd(dQ=part(20 * GB, 0), dK=part(20 * GB, 3), dV=part(20 * GB, 6)) == ALIAS
    assert fwd(Q=part(20 * GB, 0), K=part(20 * GB, 4), V=part(20 * GB, 6), O=part(20 * GB, 2)) == ALIAS


def views(order, parts, B, S, D, base=20 * GB):
    """Tensors of one buffer whose dimensions lie in `order` ("b", "s", "h": the heads of all parts, or "p": the parts of
    "h" heads each); `parts` gives each part's heads."""
    size = {"b": B, "s": S, "h": max(parts) if "p" in order else sum(parts), "p": len(parts)}
    stride, at = {}, D
    for x in reversed(order):
        stride[x], at = at, at * size[x]
    step = lambda i: i * stride["p"] if "p" in order else sum(parts[:i]) * stride["h"]
    return [_Tensor(base + 2 * step(i), stride["b"], stride["h"], stride["s"]) for i in range(len(parts))]


LAYOUTS = ["bsh", "bhs", "sbh", "shb", "hbs", "hsb", "bsph", "bpsh", "bphs", "bhps", "pbhs", "sbph", "sphb", "hpsb", "bshp"]


def shared_elements(a, b, na, nb, D):
    """The definition: the elements of both, as offsets of 16-byte pieces."""
    import numpy as np
    def pieces(t, n):
        steps = [np.arange(k) * s for k, s in zip(n, (t.stride_batch, t.stride_head, t.stride_row))]
        return (t.data // 2 + steps[0][:, None, None, None] + steps[1][:, None, None] + steps[2][:, None] + np.arange(0, D, 8)).ravel()
    return np.intersect1d(pieces(a, na), pieces(b, nb)).size > 0


@pytest.fixture
def accepted():
    """Whether a call passes its checks: without a GPU it then fails at its first CUDA call.  With one it would go on and
    use the addresses, which are fake."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("fake device addresses that pass the checks: only without a GPU")
    return lambda status: status not in (INVALID, ALIGN, ALIAS)


@pytest.mark.parametrize("sizes", [(2, 100), (1, 100), (3, 1), (1, 1), (2, 7)])
@pytest.mark.parametrize("order", LAYOUTS)
def test_parts_of_one_buffer_in_any_order(order, sizes, accepted):
    """Gradients, and O beside Q, as views of one buffer: refused only where elements are shared."""
    B, S = sizes
    d = dict(batch=B, seq_q=S, seq_kv=S)
    parts = [4, 2, 2] if "p" not in order else [4, 4, 4]
    if "p" in order:
        d["heads_kv"] = 4
    kv = parts[1]
    outs = dict(zip(("dQ", "dK", "dV"), views(order, parts, B, S, 64)))
    ins = {n: dense((i + 1) * GB, B, 4 if n in ("dO", "Q", "O") else kv, S, 64) for i, n in enumerate(("dO", "Q", "K", "V", "O"))}
    assert accepted(bwd(d, **ins, **outs))
    q, o = views(order, [4, 4], B, S, 64)
    fine = dict(K=dense(2 * GB, B, kv, S, 64), V=dense(3 * GB, B, kv, S, 64))
    assert accepted(fwd(d, Q=q, O=o, **fine))
    # O moved towards Q by a piece, by a row of D, by half a part: as the definition has it
    n = (B, 4, S)
    for back in (16, 128, 2 * 64 * 2, (o.data - q.data) // 2 // 16 * 16):
        moved = _Tensor(o.data - back, o.stride_batch, o.stride_head, o.stride_row)
        assert accepted(fwd(d, Q=q, O=moved, **fine)) == (not shared_elements(q, moved, n, n, 64)), back


def test_random_views_share_as_the_definition_has_it(accepted):
    import random
    r = random.Random(5)
    seen = set()
    for _ in range(400):
        B, Hq, Hkv, S, Skv = r.randint(1, 3), r.choice([1, 2, 4]), r.choice([1, 2]), r.randint(1, 5), r.randint(1, 5)
        Hq = max(Hq, Hkv)
        order = r.sample([0, 1, 2], 3)                             # strides that grow in this order, with gaps
        stride, at = [0, 0, 0], 64
        for k in order:
            stride[k] = at + 64 * r.choice([0, 0, 1, 5])
            at = stride[k] * (max((B, Hq, max(S, Skv))[k], 1) + r.choice([0, 1]))
        t = lambda x: _Tensor(20 * GB + 128 * r.randrange(at // 64 + 2) + 16 * r.choice([0, 0, 0, 1]), *stride) if x else None
        o, k = t(1), t(1)
        d = dict(batch=B, heads_q=Hq, heads_kv=Hkv, seq_q=S, seq_kv=Skv, causal=0)
        got = accepted(fwd(d, Q=dense(1 * GB, B, Hq, S, 64), K=k, V=dense(3 * GB, B, Hkv, Skv, 64), O=o))
        want = not shared_elements(o, k, (B, Hq, S), (B, Hkv, Skv), 64)
        assert got == want, (d, stride, o.data, k.data)
        seen.add(want)
    assert len(seen) == 2


def test_empty_attention_is_a_no_op():
    assert fwd(dict(batch=0)) == OK and fwd(dict(seq_q=0)) == OK
    assert bwd(dict(batch=0)) == OK
    assert fwd(dict(seq_q=0), Q=_Tensor(), O=_Tensor()) == OK


def tree(desc=None, q=1 * GB, k=None, v=None, table=5 * GB, lens=6 * GB, starts=7 * GB, parents=8 * GB, o=4 * GB,
         ws=10 * GB, ws_bytes=1 << 34):
    d = dict(batch=2, total_q=6, heads_q=4, heads_kv=2, head_dim=64, num_pages=10, page_size=16, table_width=5,
             max_nodes=3, q_stride_row=256, q_stride_head=64, o_stride_row=256, o_stride_head=64)
    d.update(desc or {})
    cache = lambda addr: _Tensor(addr, 16 * 2 * 64, 64, 2 * 64)
    return gsr.lib().tree_attention_fwd(_TreeDesc(**d), q, k or cache(2 * GB), v or cache(3 * GB), table, lens, starts,
                                        parents, o, ws, ws_bytes, None)


def test_tree_refusals():
    for bad in (dict(batch=-1), dict(head_dim=32), dict(dtype=3), dict(max_nodes=0), dict(max_nodes=65), dict(heads_kv=3),
                dict(heads_kv=0), dict(softcap=-2.0), dict(page_size=12), dict(page_size=0), dict(page_size=4),
                dict(table_width=2 ** 30), dict(total_q=2 ** 31), dict(q_stride_row=0), dict(o_stride_row=32),
                dict(heads_q=258, heads_kv=2)):
        assert tree(bad) == INVALID, bad
    assert tree(q=None) == INVALID and tree(lens=None) == INVALID and tree(starts=None) == INVALID
    assert tree(table=None) == INVALID and tree(o=None) == INVALID
    assert tree(q=GB + 8) == ALIGN and tree(parents=8 * GB + 1) == ALIGN and tree(ws=10 * GB + 4) == ALIGN
    assert tree(dict(q_stride_head=68)) == ALIGN
    assert tree(k=_Tensor(None, 2048, 64, 128)) == INVALID
    assert tree(o=1 * GB) == ALIAS and tree(o=2 * GB + 128) == ALIAS
    assert tree(dict(batch=0)) == OK and tree(dict(total_q=0)) == OK
    assert gsr.lib().tree_attention_workspace(None) == -1


def tables(B=4, W=5, page=16, free=10, tokens=9, over=None):
    at = [(i + 1) * GB for i in range(11)]
    for i, a in (over or {}).items():
        at[i] = a
    return gsr.lib().kv_block_tables(*at, B, W, page, free, tokens, None)


def test_block_table_refusals():
    assert tables(B=-1) == INVALID and tables(page=0) == INVALID and tables(B=8193) == INVALID
    assert tables(tokens=2 ** 31) == INVALID
    for i in range(11):
        assert tables(over={i: None}) == INVALID, i
        assert tables(over={i: (i + 1) * GB + 2}) == ALIGN, i
    assert tables(over={5: 1 * GB}) == ALIAS          # kv_lens_out in place of kv_lens
    assert tables(over={6: 4 * GB}) == ALIAS          # free_head_out in place of free_head
    assert tables(over={9: 9 * GB}) == ALIAS          # slots in place of positions


def append(tokens=9, H=2, D=64, pages=10, page=16, slots=5 * GB, k=None, kc=None, vc=None):
    c = lambda a: _Tensor(a, page * H * D, D, H * D)
    return gsr.lib().kv_cache_append(k or _Tensor(1 * GB, 0, D, 3 * H * D), _Tensor(2 * GB, 0, D, 3 * H * D), slots,
                                     kc or c(3 * GB), vc or c(4 * GB), tokens, H, D, pages, page, None)


def test_append_refusals():
    assert append(tokens=-1) == INVALID and append(page=0) == INVALID and append(slots=None) == INVALID
    assert append(D=60) == ALIGN and append(slots=5 * GB + 2) == ALIGN
    assert append(pages=2 ** 28) == INVALID and append(H=2 ** 15) == INVALID
    assert append(k=_Tensor(GB + 2, 0, 64, 128)) == ALIGN and append(k=_Tensor(GB, 0, 0, 128)) == INVALID
    assert append(kc=_Tensor(4 * GB, 2048, 64, 128)) == ALIAS         # one cache for both
    assert append(kc=_Tensor(1 * GB, 2048, 64, 128)) == ALIAS
    assert append(kc=_Tensor(3 * GB, 2048, 64, 32)) == INVALID        # cache rows on top of each other
    assert append(tokens=0) == OK


@pytest.mark.parametrize("pages,page", [(10, 16), (1, 16), (5, 1)])
def test_caches_that_share_rows(pages, page, accepted):
    """k_cache and v_cache in one buffer: halves of it in any order are fine, a shift within it is not."""
    H, D = 2, 64
    cache = lambda at, *strides: _Tensor(40 * GB + 2 * at, *strides)       # page, head, row
    strides = (page * H * D, D, H * D)
    for by in (8, D, H * D, page * H * D, 3 * page * H * D + D):
        inside = by < pages * page * H * D
        got = append(pages=pages, page=page, kc=cache(0, *strides), vc=cache(by, *strides))
        assert (got == ALIAS) == inside, by
        got = append(pages=pages, page=page, kc=cache(by, *strides), vc=cache(0, *strides))
        assert (got == ALIAS) == inside, by
    for halves in (((2 * page * H * D, D, H * D), page * H * D),            # (pages, 2, rows, heads, D)
                   ((2 * page * H * D, D, 2 * H * D), H * D),               # (pages, rows, 2, heads, D)
                   ((2 * page * H * D, 2 * D, 2 * H * D), D),               # (pages, rows, heads, 2, D)
                   ((2 * page * H * D, page * D, D), page * H * D),         # (pages, 2, heads, rows, D)
                   ((page * H * D, D, H * D), pages * page * H * D)):       # (2, pages, rows, heads, D)
        assert accepted(append(pages=pages, page=page, kc=cache(0, *halves[0]), vc=cache(halves[1], *halves[0])))


def test_outputs_that_overlap_themselves():
    assert fwd(O=_Tensor(4 * GB, 25600, 64, 64)) == INVALID            # heads on rows
    assert fwd(O=_Tensor(4 * GB, 25600, 64, 128)) == INVALID           # four heads in rows of two
    assert fwd(O=_Tensor(4 * GB, 6400, 6400, 64)) == INVALID           # batches on heads
    assert bwd(dK=_Tensor(7 * GB, 12800, 6336, 64)) == INVALID         # a head's last row on the next head's first
    assert append(kc=_Tensor(3 * GB, 1024, 64, 128)) == INVALID        # pages of 16 rows every 8 rows


def test_spans_and_positions_that_are_too_large():
    assert fwd(dict(batch=2 ** 22, heads_q=1, heads_kv=1), Q=_Tensor(1 * GB, 2 ** 39 - 8, 64, 64)) == INVALID
    assert fwd(dict(batch=1, heads_q=1, heads_kv=1, seq_q=2 ** 30, seq_kv=2 ** 30)) == INVALID
    assert tree(dict(num_pages=2 ** 23), k=_Tensor(2 * GB, 2 ** 38, 64, 128)) == INVALID
    assert fwd(dict(softcap=1025.0)) == INVALID and tree(dict(softcap=1025.0)) == INVALID
    # neither pages nor heads lie a multiple of 8 rows apart
    assert tree(k=_Tensor(2 * GB, 2056, 64, 128)) == INVALID
    assert tables(B=8192, W=2 ** 19) == INVALID


def test_masks_and_lengths_in_the_way_of_outputs():
    assert fwd(dict(alibi_slopes=4 * GB)) == ALIAS and fwd(dict(prefix_lens=4 * GB + 64)) == ALIAS
    assert fwd(dict(doc_bounds=9 * GB, num_docs=3), lse=9 * GB + 16) == ALIAS
    assert bwd(dict(alibi_slopes=6 * GB)) == ALIAS and bwd(dict(prefix_lens=10 * GB)) == ALIAS
    assert tree(lens=4 * GB) == ALIAS and tree(starts=4 * GB) == ALIAS and tree(parents=4 * GB) == ALIAS
    assert tree(table=10 * GB) == ALIAS and tree(dict(alibi_slopes=10 * GB)) == ALIAS


def test_forward_workspace():
    few = dict(batch=1, heads_q=4, heads_kv=2, seq_q=100, seq_kv=20000)
    need = llm.masked_attention_fwd_workspace(1, 4, 2, 100, 20000, 64)
    assert need > 0 and llm.masked_attention_fwd_workspace(8, 32, 8, 4096, 4096, 64) == 0
    ops = dict(Q=dense(1 * GB, 1, 4, 100, 64), K=dense(2 * GB, 1, 2, 20000, 64), V=dense(3 * GB, 1, 2, 20000, 64),
               O=dense(4 * GB, 1, 4, 100, 64))
    assert fwd(few, ws=10 * GB, ws_bytes=need // 64, **ops) == INVALID
    assert fwd(few, ws=10 * GB + 8, ws_bytes=need, **ops) == ALIGN
    for at in (1, 2, 3, 4):
        assert fwd(few, ws=at * GB, ws_bytes=need, **ops) == ALIAS
    assert fwd(dict(few, alibi_slopes=10 * GB), ws=10 * GB, ws_bytes=need, **ops) == ALIAS
    assert fwd(few, ws=9 * GB, ws_bytes=need, lse=9 * GB, **ops) == ALIAS
    with pytest.raises(gsr.GsrError):
        llm.masked_attention_fwd_workspace(1, 4, 3, 100, 100, 64)


@pytest.mark.parametrize("sizes", [(1, 8, 1, 300, 300, 64), (2, 16, 2, 2000, 700, 128), (1, 32, 1, 5000, 9000, 64)])
def test_workspaces_do_not_depend_on_masks(sizes):
    d = dict(zip(("batch", "heads_q", "heads_kv", "seq_q", "seq_kv", "head_dim"), sizes))
    for of in ("fwd", "bwd"):
        c = getattr(gsr.lib(), "masked_attention_%s_workspace" % of)
        assert len({c(_AttentionDesc(**d, **e)) for e in (dict(), dict(causal=1), dict(softcap=3.0), dict(causal=1, softcap=3.0))}) == 1
        assert getattr(llm, "masked_attention_%s_workspace" % of)(*sizes) == c(_AttentionDesc(**d))


def test_binding_refusals():
    import torch
    t = torch.zeros(1, 2, 4, 64, dtype=torch.float16)
    with pytest.raises(ValueError):
        gsr.masked_attention_fwd(t, t, t, t)                           # not on a GPU
    with pytest.raises(TypeError):
        gsr.masked_attention_fwd(t.float(), t, t, t)
    with pytest.raises(ValueError):
        gsr.tree_attention_fwd(t[0], t, t, t, t, t, t, t, 1)
    with pytest.raises(ValueError):
        gsr.kv_cache_append(t[0], t[0], t, t, t)
    with pytest.raises(ValueError):
        gsr.kv_block_tables(*[torch.zeros(1, dtype=torch.int32)] * 4, t, 16, *[t] * 6)


def test_a_batch_of_none_with_documents():
    # the arrays of masks have no elements, and so no address
    none = dict(batch=0, num_docs=3, prefix_lens=None)
    assert fwd(none) == OK and bwd(none) == OK
    assert fwd(dict(none, doc_bounds=16 * GB)) == OK
    assert fwd(dict(batch=0, doc_bounds=16 * GB)) == INVALID
    assert llm.masked_attention_bwd_workspace(0, 4, 2, 100, 100, 64) >= 0
