"""Pins of the masked attention, tree attention and block table oracle (CPU)."""
import numpy as np
import pytest
import torch

from oracle import llm


def draw(B, Hq, Hkv, Sq, Skv, D, seed):
    r = np.random.default_rng(seed)
    return (r.standard_normal((B, Hq, Sq, D)), r.standard_normal((B, Hkv, Skv, D)), r.standard_normal((B, Hkv, Skv, D)),
            r.standard_normal((B, Hq, Sq, D)))


def test_visible_by_hand():
    # two documents of 3 and 2, one padding position; prefix 2 in the first, 0 in the second
    see = llm.visible(1, 6, 6, True, [[0, 3, 5]], [[2, 0]])[0].astype(int)
    assert see.tolist() == [[1, 1, 0, 0, 0, 0], [1, 1, 0, 0, 0, 0], [1, 1, 1, 0, 0, 0],
                            [0, 0, 0, 1, 0, 0], [0, 0, 0, 1, 1, 0], [0, 0, 0, 0, 0, 0]]
    assert llm.visible(1, 2, 4, True)[0].astype(int).tolist() == [[1, 1, 1, 0], [1, 1, 1, 1]]
    assert llm.visible(1, 3, 1, True)[0].astype(int).tolist() == [[0], [0], [1]]


@pytest.mark.parametrize("cap,alibi,docs", [(0.0, False, False), (1.5, True, False), (0.7, False, True), (0.0, True, True)])
def test_gradient_against_autograd_and_differences(cap, alibi, docs):
    B, Hq, Hkv, S, D = 2, 4, 2, 7, 5
    q, k, v, do = draw(B, Hq, Hkv, S, S, D, 3)
    bounds = [[0, 3, 6], [1, 5, 7]] if docs else None
    see = llm.visible(B, S, S, True, bounds, [[2, 1], [0, 2]] if docs else [[3], [0]])
    slopes = np.array([0.5, 0.25, 0.1, 0.05]) if alibi else None
    o, lse, _ = llm.masked_attention(q, k, v, see, 0.0, cap, slopes)
    (dq, dk, dv), _, _, _ = llm.masked_attention_bwd(do, q, k, v, o, lse, see, 0.0, cap, slopes)

    tq, tk, tv = (torch.tensor(t, requires_grad=True) for t in (q, k, v))
    x = tq @ tk.repeat_interleave(2, 1).transpose(-1, -2) / np.sqrt(D)
    x = cap * torch.tanh(x / cap) if cap else x
    if alibi:
        i = torch.arange(S)
        x = x - torch.tensor(slopes)[:, None, None] * (i[:, None] - i[None]).abs()
    p = torch.softmax(x.masked_fill(~torch.tensor(see)[:, None], -1e300), -1) * torch.tensor(see.any(-1))[:, None, :, None]
    to = p @ tv.repeat_interleave(2, 1)
    assert np.allclose(to.detach().numpy(), o, atol=1e-12)
    (to * torch.tensor(do)).sum().backward()
    for a, b in ((tq, dq), (tk, dk), (tv, dv)):
        assert np.allclose(a.grad.numpy(), b, atol=1e-12)

    loss = lambda *t: (llm.masked_attention(*t, see, 0.0, cap, slopes)[0] * do).sum()
    r = np.random.default_rng(4)
    for n, (t, grad) in enumerate(((q, dq), (k, dk), (v, dv))):
        step = r.standard_normal(t.shape)
        args = [q, k, v]
        args[n] = t + 1e-6 * step
        up = loss(*args)
        args[n] = t - 1e-6 * step
        assert abs((up - loss(*args)) / 2e-6 - (grad * step).sum()) < 1e-6 * max(1.0, abs((grad * step).sum()))


def test_tree_of_a_chain_is_causal_attention():
    r = np.random.default_rng(5)
    page, D, Hq, Hkv, kv, T = 8, 6, 4, 2, 21, 5
    kc, vc = r.standard_normal((6, page, Hkv, D)), r.standard_normal((6, page, Hkv, D))
    table = np.array([[4, 0, 3, 1]])
    q = r.standard_normal((T, Hq, D))
    slopes = [0.3, 0.2, 0.1, 0.0]
    o, _ = llm.tree_attention(q, kc, vc, table, [kv], [0, T], None, 0.0, 2.0, slopes)
    k = kc[table[0, :3]].reshape(-1, Hkv, D)[:kv].transpose(1, 0, 2)[None]
    v = vc[table[0, :3]].reshape(-1, Hkv, D)[:kv].transpose(1, 0, 2)[None]
    ref, _, _ = llm.masked_attention(q.transpose(1, 0, 2)[None], k, v, llm.visible(1, T, kv, True), 0.0, 2.0, slopes)
    assert np.allclose(o, ref[0].transpose(1, 0, 2), atol=1e-13)
    # siblings do not see each other: every node under -1 sees the context and itself only
    o2, _ = llm.tree_attention(q, kc, vc, table, [kv], [0, T], [-1] * T, 0.0, 2.0)
    keys = list(range(kv - T)) + [kv - 1]
    ref2, _, _ = llm.masked_attention(q[-1:].transpose(1, 0, 2)[None], k[:, :, keys], v[:, :, keys],
                                      llm.visible(1, 1, len(keys)), 0.0, 2.0)
    assert np.allclose(o2[-1], ref2[0, :, 0], atol=1e-13)


def test_block_tables_by_hand():
    table = [[7, -1, -1], [5, 6, -1], [-1, -1, -1]]
    got = llm.block_tables([3, 8, 0], [2, 0, 5], [90, 91, 92, 93], 1, table, 4, 9)
    assert got["table"].tolist() == [[7, 91, -1], [5, 6, -1], [92, 93, -1]]
    assert got["slots"].tolist() == [31, 364, 368, 369, 370, 371, 372, -1, -1]
    assert got["positions"].tolist() == [3, 4, 0, 1, 2, 3, 4, -1, -1]
    assert got["q_starts"].tolist() == [0, 2, 2, 7] and got["kv_out"].tolist() == [5, 8, 5]
    assert got["counts"].tolist() == [7, 3, 0] and got["head_out"].tolist() == [4]
    # a free list of one page, and a table too narrow
    got = llm.block_tables([0, 11], [6, 3], [9], 0, [[-1, -1, -1], [1, 2, 3]], 4, 9)
    assert got["table"].tolist() == [[9, -1, -1], [1, 2, 3]] and got["counts"].tolist() == [9, 1, 2]
    assert got["slots"].tolist() == [36, 37, 38, 39, -1, -1, 15, -1, -1]
