"""Pins of oracle/block_oracle.py on the CPU: hand values, dense attention in closed form, gradients against
differences, and planted mistakes that the checks must see."""
import math

import numpy as np
import pytest

from oracle import block_oracle as bo


def rnd(seed, *shape):
    return np.random.default_rng(seed).standard_normal(shape)


@pytest.mark.parametrize("interleaved", [True, False])
def test_rotation_keeps_norms_and_turns_by_the_difference_of_positions(interleaved):
    D = 8
    x, y = rnd(0, D), rnd(1, D)
    angle = np.arange(10)[:, None] * 0.3 ** np.arange(D // 2)
    c, s = np.cos(angle), np.sin(angle)
    turn = lambda v, p: bo.rotate(v, c[p], s[p], interleaved)  # noqa: E731
    assert np.isclose((turn(x, 7) ** 2).sum(), (x ** 2).sum())
    assert np.isclose(turn(x, 7) @ turn(y, 4), turn(x, 5) @ turn(y, 2))
    hand = turn(np.array([1.0, 0, 0, 0, 0, 0, 0, 0]), 1)
    assert np.isclose(hand[0], math.cos(1)) and np.isclose(hand[1 if interleaved else 4], math.sin(1))


def test_norm_has_unit_mean_square_and_padding_is_zero():
    x = rnd(2, 1, 3, 2, 16)
    y, _ = bo.norm_rope(x, None, None, None, 0.0, True, np.array([[-1, 0, 1]]))
    assert np.allclose((y[0, :, 1:] ** 2).mean(-1), 1) and not y[0, :, 0].any()


def test_norm_gradient_against_differences():
    B, N, H, D = 1, 2, 2, 8
    x, w, dy = rnd(3, B, N, H, D), rnd(4, D), rnd(5, B, H, N, D)
    angle = rnd(6, 4, D // 2)
    c, s, pos = np.cos(angle), np.sin(angle), np.array([[1, 3]])
    f = lambda x, w: (bo.norm_rope(x, w, c, s, 1e-3, False, pos)[0] * dy).sum()  # noqa: E731
    dx, dw, _, _ = bo.norm_rope_backward(x, w, c, s, 1e-3, False, pos, dy)
    h = 1e-6
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = h
        assert abs((f(x + e, w) - f(x - e, w)) / (2 * h) - dx[i]) < 1e-7
    for i in range(D):
        e = np.zeros(D)
        e[i] = h
        assert abs((f(x, w + e) - f(x, w - e)) / (2 * h) - dw[i]) < 1e-7


def test_selection_by_hand():
    # 5 blocks of 64 keys; scores 0, 3, 1, 3, (own)
    mean = np.zeros((1, 5, 4), np.float32)
    mean[0, :, 0] = [0, 3, 1, 3, 9]
    q = np.zeros((1, 1, 4))
    q[0, 0, 0] = 1
    pick = lambda **kw: list(bo.select_blocks(q, mean, 64, kw.pop("topk"), kw.pop("sink", 0), 1, True, [300])[0, 0])  # noqa: E731,E501
    assert pick(topk=2) == [1, 4]                   # the tie of 1 and 3 goes to the lower block
    assert pick(topk=3) == [1, 3, 4]
    assert pick(topk=3, sink=1) == [0, 1, 4]
    assert pick(topk=7) == [0, 1, 2, 3, 4, -1, -1]
    assert (bo.select_blocks(q, mean, 64, 3, 1, 1, True, [0])[0, 0] == -1).all()
    short = bo.select_blocks(np.repeat(q, 3, 1), mean, 64, 2, 1, 1, True, [1])[0]
    assert short.tolist() == [[-1, -1], [-1, -1], [0, -1]]       # left padding


def dense(q, k, v, mask, scale):
    s = np.where(mask, q @ k.T * scale, -np.inf)
    p = np.exp(s - s.max(-1, keepdims=True))
    return (p / p.sum(-1, keepdims=True)) @ v


def test_every_block_listed_is_dense_causal_attention():
    N, D = 150, 8
    q, k, v = rnd(7, 2, N, D), rnd(8, 1, N, D), rnd(9, 1, N, D)
    sel = np.tile(np.array([2, 0, 1, 1, -1, 77], np.int32), (1, N, 1))
    o, lse, _, _ = bo.attention(q, k, v, sel, 64, True, [N], 0.4)
    for h in range(2):
        assert np.allclose(o[h], dense(q[h], k[0], v[0], np.tril(np.ones((N, N), bool)), 0.4))
    # planted: one block missing must show
    bad, _, _, _ = bo.attention(q, k, v, np.where(sel == 1, -1, sel), 64, True, [N], 0.4)
    assert not np.allclose(bad[:, 70:], o[:, 70:])


def test_attention_gradient_against_differences():
    N, D, lens = 70, 4, [66]
    q, k, v, do = rnd(10, 2, N, D), rnd(11, 1, N, D), rnd(12, 1, N, D), rnd(13, 2, N, D)
    sel = np.random.default_rng(14).integers(-1, 2, (1, N, 2)).astype(np.int32)
    f = lambda q, k, v: (bo.attention(q, k, v, sel, 64, True, lens, 0.5)[0] * do).sum()  # noqa: E731
    o, lse, _, _ = bo.attention(q, k, v, sel, 64, True, lens, 0.5)
    grads, bounds = bo.attention_backward(do, q, k, v, o, lse, sel, 64, True, lens, 0.5)
    h = 1e-6
    rng = np.random.default_rng(15)
    for which, x in enumerate((q, k, v)):
        for _ in range(12):
            i = tuple(rng.integers(0, d) for d in x.shape)
            args = [q, k, v]
            e = np.zeros_like(x)
            e[i] = h
            args[which] = x + e
            up = f(*args)
            args[which] = x - e
            assert abs((up - f(*args)) / (2 * h) - grads[which][i]) < 1e-6
    assert all((b >= 0).all() for b in bounds)
    # rows behind the sequence and queries before its start have no gradient
    assert not grads[1][0, 66:].any() and not grads[2][0, 66:].any() and not grads[0][:, :4].any()


def test_bounds_see_a_wrong_scale_and_a_missing_key():
    q, k, v = rnd(16, 1, 3, 64), rnd(17, 1, 128, 64), rnd(18, 1, 128, 64)
    sel = np.tile(np.array([0, 1], np.int32), (1, 3, 1))
    o, lse, b, bl = bo.attention(q, k, v, sel, 64, False, [128], 0.125)
    for bad in (bo.attention(q, k, v, sel, 64, False, [128], 0.13), bo.attention(q, k, v, sel, 64, False, [127], 0.125)):
        assert (np.abs(bad[0] - o) > b).any() and (np.abs(bad[1] - lse) > bl).all()


def test_the_library_refuses_bad_arguments_before_any_launch():
    import ctypes

    import sparse_attention_long_svg_b200 as svg
    from sparse_attention_long_svg_b200 import build
    build.build()
    lib = svg.load_library()
    f, g, h, odd, nul = (ctypes.c_void_p(x) for x in (0x10000, 0x20000, 0x30000, 0x10002, 0))
    st = (ctypes.c_int64 * 3)(64, 64, 64)
    bad = (ctypes.c_int64 * 3)(64, 65, 64)

    vo = ctypes.c_void_p(0x50000)

    def rope(q=f, qs=st, qo=g, cos=f, sin=f, P=8, B=1, N=8, Hq=1, D=64, eps=1e-6, il=1, start=nul, ko=h, cap=8):
        return lib.svg_qk_norm_rope(q, qs, f, st, f, st, nul, nul, cos, sin, P, B, N, Hq, 1, D, eps, il, start, qo, ko,
                                    vo, cap, nul)

    assert rope(q=nul) == 1 and rope(qo=nul) == 1 and rope(qs=bad) == 1 and rope(q=odd) == 1 and rope(qo=f) == 1
    assert rope(cos=nul) == 1 and rope(P=7) == 1 and rope(B=0) == 1 and rope(N=0) == 1 and rope(cap=7) == 1
    assert rope(D=96) == 2 and rope(eps=-1.0) == 1 and rope(eps=float("nan")) == 1 and rope(il=2) == 1
    assert rope(ko=vo) == 1 and rope(ko=g) == 1 and rope(start=f, cap=0) == 1
    assert rope(ko=nul) == 1 and rope(B=1 << 20, N=1 << 12, P=1 << 12, cap=1 << 12) == 2

    def rope_back(ws=1 << 20, dq=h, dqs=st, D=64, dqo=g, dk=ctypes.c_void_p(0x60000)):
        return lib.svg_qk_norm_rope_backward(dqo, g, g, f, st, f, st, nul, nul, f, f, 8, 1, 8, 1, 1, D, 1e-6, 1, nul, 8,
                                             dq, dqs, dk, st, vo, st, nul, nul, f, ws, nul)

    assert rope_back(ws=0) == 3 and rope_back(dq=nul) == 1 and rope_back(dqs=bad) == 1 and rope_back(D=32) == 2
    assert rope_back(dq=g) == 1 and rope_back(dqo=nul) == 1 and rope_back(dk=vo) == 1 and rope_back(dk=h) == 1
    assert lib.svg_qk_norm_rope_backward_workspace_size(0, 8, 1, 1, 64) == 0

    mean = lambda k=f, B=1, Nk=100, D=64, block=64, new=0: lib.svg_block_mean(k, 2, B, Nk, D, block, nul, new, g, nul)  # noqa: E731,E501
    assert mean(k=nul) == 1 and mean(k=odd) == 1 and mean(B=3) == 1 and mean(Nk=0) == 1 and mean(new=-1) == 1
    assert mean(D=80) == 2 and mean(block=32) == 2 and mean(Nk=64 * 4096 + 1) == 2

    def select(q=f, BHq=4, Nq=70, Nk=1000, topk=4, sink=1, local=1, causal=1, ws=1 << 30, block=64):
        return lib.svg_block_select(q, g, BHq, 2, 1, Nq, Nk, 64, block, topk, sink, local, causal, nul, h, f, ws, nul)

    assert select(q=nul) == 1 and select(BHq=3) == 1 and select(topk=0) == 1 and select(sink=4) == 1
    assert select(local=0) == 1 and select(sink=-1) == 1 and select(causal=2) == 1 and select(topk=1025) == 2
    assert select(BHq=34) == 2 and select(ws=8) == 3 and select(block=100) == 2 and select(Nq=0) == 1

    def attn(q=f, o=g, BHq=4, Nq=70, Nk=1000, D=64, topk=4, block=64, causal=1, ws=1 << 30):
        return lib.svg_block_attn(q, h, h, BHq, 2, 1, Nq, Nk, D, h, topk, block, causal, 0.0, nul, o, nul, f, ws, nul)

    assert attn(q=nul) == 1 and attn(o=f) == 1 and attn(o=h) == 1 and attn(q=odd) == 1 and attn(BHq=5) == 1
    assert attn(D=256) == 2 and attn(block=16) == 2 and attn(BHq=64) == 2 and attn(topk=0) == 1 and attn(causal=3) == 1
    assert attn(Nq=1, Nk=100000, topk=64, ws=8) == 3

    def attn_back(do=f, dq=g, dk=h, ws=8, D=64):
        return lib.svg_block_attn_backward(do, f, f, f, f, f, 4, 2, 1, 70, 1000, D, f, 4, 64, 1, 0.0, nul, dq, dk,
                                           ctypes.c_void_p(0x40000), f, ws, nul)

    assert attn_back() == 3 and attn_back(do=nul) == 1 and attn_back(dq=f) == 1 and attn_back(dk=g) == 1
    assert attn_back(D=100) == 2
    assert svg.load_library().svg_last_cuda_error().decode() == ""


def test_table_angles_and_refusals_without_a_gpu():
    import sparse_attention_long_svg_b200 as svg
    cos, sin = svg.rope_table((5,), 8, device="cpu")
    assert cos.shape == (5, 4) and abs(float(sin[3, 1]) - math.sin(3 * 10000 ** -0.25)) < 1e-7
    with pytest.raises(ValueError):
        svg.rope_table((2, 2), 8, split=(3, 2), device="cpu")
    with pytest.raises(ValueError):
        svg.block_mean(__import__("torch").zeros(1, 64, 64, dtype=__import__("torch").bfloat16), 64)
