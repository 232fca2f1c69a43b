"""GPU parity of the Q/K preparation and of attention over blocks chosen for each query (blocks.py) against
oracle/block_oracle.py, whose results come with the bounds that their rounding allows.

Selections and block means are compared exactly; bf16 outputs within half a step of the result plus half a step of
every bf16 operand of the sum behind it, fp32 results within the rounding of their sums.
"""
import numpy as np
import pytest
import torch

from oracle import block_oracle as bo

pytestmark = pytest.mark.gpu

svg = pytest.importorskip("sparse_attention_long_svg_b200")

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_attention_long_svg_b200 import build
    build.build()
    svg.load_library()
    yield
    assert svg.get_error() == 0


def bf(seed, *shape, scale=1.0):
    """bf16 normal values on the device."""
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale).to(BF).cuda()


def f64(t):
    return t.detach().double().cpu().numpy()


def i32(*values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def within(got, want, bound, what=""):
    got = f64(got) if isinstance(got, torch.Tensor) else got
    off = np.abs(got - want)
    ok = (off <= bound) | ((got == want) & ~np.isfinite(want))
    assert ok.all(), (what, np.argwhere(~ok)[:4], got[~ok][:4], want[~ok][:4], np.broadcast_to(bound, off.shape)[~ok][:4])


def tokens(seed, B, Hq, Hk, Nq, Nk, D, scale=1.0):
    return (bf(seed, B * Hq, Nq, D, scale=scale), bf(seed + 1, B * Hk, Nk, D, scale=scale),
            bf(seed + 2, B * Hk, Nk, D))


# ----------------------------------------------------------------------- norm and rotation
ROPE = [  # B, N, Hq, Hk, D
    (1, 1, 1, 1, 64), (1, 1, 40, 8, 128), (3, 5, 6, 2, 128), (2, 33, 5, 5, 64), (2, 130, 4, 1, 128), (1, 257, 3, 3, 64),
]


def rope_inputs(B, N, Hq, Hk, D, seed=0):
    qkv = bf(seed, B, N, Hq + 2 * Hk, D, scale=2.0)
    w = [(1 + 0.3 * torch.randn(D, generator=torch.Generator().manual_seed(seed + i))).cuda() for i in (1, 2)]
    return qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk], qkv[:, :, Hq + Hk:], *w


def check_rows(got, x, w, cos, sin, eps, interleaved, pos, what):
    B, N, H, D = x.shape
    want, size = bo.norm_rope(f64(x), None if w is None else f64(w), None if cos is None else f64(cos),
                              None if sin is None else f64(sin), eps, interleaved, pos)
    # fp32 arithmetic: D/2 additions of squares, a handful of products
    within(got.view(B, H, N, D), want, bo.HALF_BF16 * np.abs(want) + (D / 2 + 16) * bo.HALF_F32 * size, what)


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("B,N,Hq,Hk,D", ROPE)
def test_norm_and_rotation(B, N, Hq, Hk, D, interleaved):
    q, k, v, w_q, w_k = rope_inputs(B, N, Hq, Hk, D)
    cos, sin = svg.rope_table((N + 3,), D)
    qo, ko, vo = svg.qk_norm_rope(q, k, v, w_q, w_k, cos, sin, eps=1e-5, interleaved=interleaved)
    pos = np.tile(np.arange(N), (B, 1))
    check_rows(qo, q, w_q, cos, sin, 1e-5, interleaved, pos, "q")
    check_rows(ko, k, w_k, cos, sin, 1e-5, interleaved, pos, "k")
    assert torch.equal(vo.view(B, Hk, N, D), v.transpose(1, 2))


def test_many_rows_take_chunks_of_heads_and_agree_with_few():
    """The variant for large calls (heads 8 at a time, 13 = 8 + 5) gives each row what the one for small calls gives."""
    B, N, Hq, Hk, D = 1, 6301, 13, 6, 128
    q, k, v, w_q, w_k = rope_inputs(B, N, Hq, Hk, D, seed=5)
    cos, sin = svg.rope_table((N,), D)
    assert N * (Hq + 2 * Hk) * D // 16 >= 148 * 2048 * 4          # threads of the large variant
    got = svg.qk_norm_rope(q, k, v, w_q, w_k, cos, sin)
    for a in (0, 3000, 6201):
        part = slice(a, a + 100)
        few = svg.qk_norm_rope(q[:, part], k[:, part], v[:, part], w_q, w_k, cos[part].contiguous(),
                               sin[part].contiguous())
        for x, y in zip(got, few):
            assert torch.equal(x[:, part], y)


def test_cache_rows_padding_and_no_weights():
    B, N, Hq, Hk, D, cap = 3, 4, 4, 2, 64, 20
    q, k, v, w_q, _ = rope_inputs(B, N, Hq, Hk, D, seed=7)
    cos, sin = svg.rope_table((30,), D)
    start = i32(-2, 0, 16)
    ko, vo = bf(8, B * Hk, cap, D), bf(9, B * Hk, cap, D)
    old_k, old_v = ko.clone(), vo.clone()
    qo, k2, v2 = svg.qk_norm_rope(q, k, v, w_q, None, cos, sin, interleaved=False, start=start, k_out=ko, v_out=vo)
    assert k2 is ko and v2 is vo
    pos = np.array([[-2, -1, 0, 1], [0, 1, 2, 3], [16, 17, 18, 19]])
    check_rows(qo, q, w_q, cos, sin, 1e-6, False, pos, "q")
    fresh, _, _ = svg.qk_norm_rope(k.contiguous(), None, None, None, None, cos, sin, interleaved=False, start=start)
    for b in range(B):
        for n in range(N):
            if pos[b, n] >= 0:
                for h in range(Hk):
                    assert torch.equal(ko[b * Hk + h, pos[b, n]], fresh[b * Hk + h, n])
                    assert torch.equal(vo[b * Hk + h, pos[b, n]], v[b, n, h])
                    old_k[b * Hk + h, pos[b, n]] = ko[b * Hk + h, pos[b, n]]
                    old_v[b * Hk + h, pos[b, n]] = vo[b * Hk + h, pos[b, n]]
    assert torch.equal(ko, old_k) and torch.equal(vo, old_v)      # other rows are as they were
    assert svg.get_error() == 0


def test_positions_beyond_table_or_buffer_are_recorded_and_skipped():
    q, k, v, w_q, w_k = rope_inputs(1, 3, 2, 2, 64, seed=11)
    cos, sin = svg.rope_table((10,), 64)
    ko, vo = bf(12, 2, 9, 64), bf(13, 2, 9, 64)
    keep_k, keep_v = ko.clone(), vo.clone()
    qo, _, _ = svg.qk_norm_rope(q, k, v, w_q, w_k, cos, sin, start=i32(8), k_out=ko, v_out=vo)   # rows 8, 9, 10
    assert svg.get_error_detail()[:2] == (6, "rotation range")
    assert torch.equal(ko[:, :8], keep_k[:, :8]) and torch.equal(vo[:, :8], keep_v[:, :8])
    assert torch.equal(vo[:, 8], v[0, 0]) and not qo[:, 2].any() and qo[:, 1].any()
    svg.qk_norm_rope_backward(bf(1, 2, 3, 64), ko, vo, q, k, w_q, w_k, cos, sin, start=i32(8))
    assert svg.get_error() == 6


def test_norm_of_zero_tiny_and_large_rows():
    q = torch.zeros(1, 4, 1, 64, dtype=BF, device="cuda")
    q[0, 1] = 1e-20
    q[0, 2] = 1e15
    q[0, 3, 0, 5] = 3e4
    qo, _, _ = svg.qk_norm_rope(q, eps=1e-6)
    check_rows(qo, q, None, None, None, 1e-6, True, np.arange(4)[None], "q")


def test_table_of_a_grid():
    cos, sin = svg.rope_table((2, 3, 4), 16, theta=100.0, split=(2, 3, 3))
    assert cos.shape == (24, 8)
    n = 1 * 12 + 2 * 4 + 3
    want = [1.0, 0.1, 2, 2 * 100 ** (-1 / 3), 2 * 100 ** (-2 / 3), 3, 3 * 100 ** (-1 / 3), 3 * 100 ** (-2 / 3)]
    assert np.allclose(f64(cos)[n], np.cos(want), atol=1e-7) and np.allclose(f64(sin)[n], np.sin(want), atol=1e-7)


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("B,N,Hq,Hk,D", ROPE + [(2, 700, 18, 9, 64)])
def test_norm_and_rotation_gradient(B, N, Hq, Hk, D, interleaved):
    q, k, _, w_q, w_k = rope_inputs(B, N, Hq, Hk, D, seed=20)
    cos, sin = svg.rope_table((N,), D)
    dqo, dko, dvo = bf(23, B * Hq, N, D), bf(24, B * Hk, N, D), bf(25, B * Hk, N, D)
    dqkv = torch.full((B, N, Hq + 2 * Hk, D), 7.0, dtype=BF, device="cuda")
    views = dqkv[:, :, :Hq], dqkv[:, :, Hq:Hq + Hk], dqkv[:, :, Hq + Hk:]
    dq, dk, dv, dw_q, dw_k = svg.qk_norm_rope_backward(dqo, dko, dvo, q, k, w_q, w_k, cos, sin, eps=1e-5,
                                                       interleaved=interleaved, dq=views[0], dk=views[1], dv=views[2])
    pos = np.tile(np.arange(N), (B, 1))
    for x, w, dy, dx, dw, H in ((q, w_q, dqo, dq, dw_q, Hq), (k, w_k, dko, dk, dw_k, Hk)):
        want, want_w, size, terms = bo.norm_rope_backward(f64(x), f64(w), f64(cos), f64(sin), 1e-5, interleaved, pos,
                                                          f64(dy).reshape(B, H, N, D))
        within(dx, want, bo.HALF_BF16 * np.abs(want) + (2 * D + 32) * bo.HALF_F32 * size * 2, "dx")
        # a thread sums at most B N H rows of its chunk in fp32, groups after it
        within(dw, want_w, (min(B * N, 64) * 8 + 64) * bo.HALF_F32 * terms + D * bo.HALF_F32 * terms, "dw")
    assert torch.equal(dv, dvo.view(B, Hk, N, D).transpose(1, 2))
    assert torch.equal(dqkv[:, :, :Hq], dq) and not (dqkv == 7.0).all(-1).any()
    again = svg.qk_norm_rope_backward(dqo, dko, dvo, q, k, w_q, w_k, cos, sin, eps=1e-5, interleaved=interleaved)
    for a, b in zip(again, (dq, dk, dv, dw_q, dw_k)):
        assert torch.equal(a, b)


def test_gradient_of_padding_and_cache_rows():
    B, N, H, D, cap = 2, 5, 2, 64, 12
    q, k, _, w_q, w_k = rope_inputs(B, N, H, H, D, seed=30)
    cos, sin = svg.rope_table((cap,), D)
    start = i32(-3, 6)
    dqo, dko, dvo = bf(31, B * H, N, D), bf(32, B * H, cap, D), bf(33, B * H, cap, D)
    dq, dk, dv, dw_q, dw_k = svg.qk_norm_rope_backward(dqo, dko, dvo, q, k, w_q, w_k, cos, sin, start=start)
    pos = np.array([[-3, -2, -1, 0, 1], [6, 7, 8, 9, 10]])
    rows = torch.from_numpy(np.maximum(pos, 0)).cuda()
    dy = torch.stack([dko.view(B, H, cap, D)[b][:, rows[b]] for b in range(B)])
    want, want_w, size, terms = bo.norm_rope_backward(f64(k), f64(w_k), f64(cos), f64(sin), 1e-6, True, pos, f64(dy))
    within(dk, want, bo.HALF_BF16 * np.abs(want) + 300 * bo.HALF_F32 * size, "dk")
    within(dw_k, want_w, 600 * bo.HALF_F32 * terms, "dw_k")
    assert not dq[0, :3].any() and not dk[0, :3].any() and not dv[0, :3].any()
    assert torch.equal(dv[1], dvo.view(B, H, cap, D)[1][:, 6:11].transpose(0, 1))
    assert svg.get_error() == 0


# ----------------------------------------------------------------------- block means and selection
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Nk,block", [(1, 64), (63, 64), (64, 64), (65, 64), (300, 128), (700, 64)])
def test_block_means_are_exact(Nk, block, D):
    B, Hk = 3, 2
    k = bf(40, B * Hk, Nk, D)
    lens = [Nk, Nk // 2, 0]
    per_head = [n for n in lens for _ in range(Hk)]
    mean = svg.block_mean(k, block, kv_len=i32(*lens))
    assert np.array_equal(mean.cpu().numpy(), bo.block_means(f64(k), block, per_head))
    assert torch.equal(svg.block_mean(k, block)[:Hk], mean[:Hk])


def test_block_means_of_subnormals_infinities_and_nan():
    k = bf(44, 1, 320, 64)
    bits = torch.randint(-32768, 32768, (64, 64), generator=torch.Generator().manual_seed(45), dtype=torch.int32)
    bits = torch.where((bits & 0x7F80) == 0x7F80, bits & ~0x4000, bits)
    k[0, :64] = ((bits & 0x807F) | 0x0080).to(torch.int16).view(BF).cuda()        # the smallest normal values
    k[0, 64:128] = (bits & 0x807F).to(torch.int16).view(BF).cuda()                # subnormals and zeros
    k[0, 130, 3], k[0, 130, 4] = float("inf"), -float("inf")
    k[0, 200, 7], k[0, 201, 7] = float("inf"), -float("inf")
    k[0, 260, 9], k[0, 260, 10] = float("nan"), float("nan")
    got = svg.block_mean(k, 64).cpu().numpy()
    want = bo.block_means(f64(k), 64, [320])
    assert np.array_equal(got, want, equal_nan=True), np.argwhere(~((got == want) | (np.isnan(got) & np.isnan(want))))[:5]


@pytest.mark.parametrize("new", [1, 3, 65, 1000])
def test_block_means_of_the_newest_keys(new):
    B, Hk, Nk, D = 4, 2, 520, 128
    k, lens = bf(41, B * Hk, Nk, D), [520, 64, 65, 0]
    old = torch.full((B * Hk, 9, D), 5.0, device="cuda")
    want = bo.block_means(f64(k), 64, [n for n in lens for _ in range(Hk)])
    touched = np.zeros((B, 9), bool)
    for b, n in enumerate(lens):
        if n:
            touched[b, max(0, n - new) // 64:(n - 1) // 64 + 1] = True
    got = svg.block_mean(k, 64, kv_len=i32(*lens), new=new, mean=old)
    assert got is old
    t = touched.repeat(Hk, 0)
    assert np.array_equal(got.cpu().numpy()[t], want[t]) and (got.cpu().numpy()[~t] == 5.0).all()


SELECT = [  # B, Hq, Hk, Nq, Nk, D, block, topk, sink, local, causal, lens
    (1, 1, 1, 1, 1, 64, 64, 1, 0, 1, True, None),
    (2, 10, 2, 1, 3000, 128, 64, 8, 1, 2, True, (3000, 1501)),
    (2, 4, 2, 4, 20000, 128, 64, 16, 2, 1, True, (20000, 9999)),
    (1, 2, 2, 3, 90000, 64, 64, 9, 0, 1, True, None),
    (2, 2, 1, 5, 9000, 128, 64, 40, 3, 1, True, (9000, 2)),
    (1, 4, 2, 129, 262144, 64, 64, 70, 2, 2, True, None),
    (1, 1, 1, 130, 600, 128, 64, 3, 1, 2, True, None),
    (1, 5, 1, 200, 200, 128, 64, 2, 0, 1, True, None),
    (2, 6, 2, 333, 700, 64, 64, 5, 1, 2, True, (700, 300)),
    (1, 2, 1, 70, 5000, 128, 128, 6, 0, 0, False, None),
    (1, 16, 1, 65, 33000, 64, 64, 12, 1, 1, True, None),
    (1, 3, 3, 40, 100000, 64, 64, 30, 1, 1, False, (99990,)),
]


@pytest.mark.parametrize("B,Hq,Hk,Nq,Nk,D,block,topk,sink,local,causal,lens", SELECT)
def test_selection_is_the_exact_one(B, Hq, Hk, Nq, Nk, D, block, topk, sink, local, causal, lens):
    q = bf(50, B * Hq, Nq, D)
    nblk = -(-Nk // block)
    mean = torch.randn(B * Hk, nblk, D, generator=torch.Generator().manual_seed(51)).cuda() * 0.2
    if nblk > 8:
        mean[:, 5] = mean[:, 3]                       # exact ties
        mean[:, 6] = mean[:, 4] * (1 + 2.0 ** -22)    # a gap far below the approximate scores' error
    kv = None if lens is None else i32(*lens)
    per_head = [n for n in (lens or [Nk] * B) for _ in range(Hk)]
    sel = svg.block_select(q, mean, block, topk, Nk, sink, local, causal, kv_len=kv)
    want = bo.select_blocks(f64(q), f64(mean), block, topk, sink, local, causal, per_head)
    assert np.array_equal(sel.cpu().numpy(), want), np.argwhere(sel.cpu().numpy() != want)[:5]


@pytest.mark.parametrize("Nq", [2, 70])
def test_selection_of_degenerate_scores(Nq):
    """All scores equal, queries of zero, infinite and NaN means: ties go to the lowest block, NaN counts as -inf."""
    q, Nk, D = bf(52, 4, Nq, 64), 4000, 64
    q[:, 1] = 0
    mean = torch.randn(2, 63, D, generator=torch.Generator().manual_seed(53)).cuda()
    mean[0] = mean[0, :1]
    mean[1, 7] = float("nan")
    mean[1, 9, 3] = float("inf")
    sel = svg.block_select(q, mean, 64, 6, Nk, 1, 1, True)
    want = bo.select_blocks(f64(q), f64(mean), 64, 6, 1, 1, True, [Nk, Nk])
    assert np.array_equal(sel.cpu().numpy(), want), np.argwhere(sel.cpu().numpy() != want)[:5]


@pytest.mark.parametrize("Nq", [1, 66])
def test_selection_of_flat_and_tiny_scores(Nq):
    """More near candidates than a warp has lanes, and norms whose squares underflow."""
    q, Nk, D = bf(54, 3, Nq, 64), 6400, 64
    q[2] = (q[2].double() * 1e-25).to(BF)
    mean = torch.randn(3, 100, D, generator=torch.Generator().manual_seed(55)).cuda()
    noise = torch.randn(100, D, generator=torch.Generator().manual_seed(56)).cuda()
    mean[0] = mean[0, :1] * (1 + noise * 2.0 ** -23)          # all within the approximate scores' error
    mean[1] = mean[1, :1]
    mean[1, 50:] = mean[1, 50:] * (1 + 2.0 ** -22)
    mean[2] = mean[2] * 1e-15
    sel = svg.block_select(q, mean, 64, 9, Nk, 1, 1, True)
    want = bo.select_blocks(f64(q), f64(mean), 64, 9, 1, 1, True, [Nk] * 3)
    assert np.array_equal(sel.cpu().numpy(), want), np.argwhere(sel.cpu().numpy() != want)[:5]


# ----------------------------------------------------------------------- attention
ATTN = [  # B, Hq, Hk, Nq, Nk, D, block, topk, causal, lens
    (1, 1, 1, 1, 1, 64, 64, 1, True, None),
    (2, 8, 1, 1, 500, 128, 64, 5, True, (500, 3)),
    (3, 10, 2, 2, 1000, 128, 64, 12, True, (1000, 1, 0)),
    (1, 32, 2, 1, 2000, 64, 128, 9, True, None),
    (1, 2, 2, 16, 700, 128, 64, 6, True, None),
    (1, 2, 2, 17, 700, 64, 64, 6, False, None),
    (2, 3, 1, 100, 200, 128, 64, 3, True, (200, 60)),
    (1, 5, 1, 77, 300, 64, 64, 4, True, None),
    (1, 7, 1, 40, 129, 128, 64, 3, False, None),
    (2, 2, 2, 150, 150, 128, 128, 2, True, (150, 149)),
    (1, 16, 1, 13, 257, 64, 64, 5, True, None),
]


def lists(seed, BHk, Nq, topk, nblk):
    """Lists in any order, with repeats, padding and ids outside the buffer; some rows empty."""
    g = np.random.default_rng(seed)
    sel = g.integers(-1, nblk + 1, (BHk, Nq, topk)).astype(np.int32)
    sel[g.random((BHk, Nq)) < 0.1] = -1
    sel[:, Nq // 2, 0] = 2 ** 31 - 1
    return torch.from_numpy(sel).cuda()


@pytest.mark.parametrize("B,Hq,Hk,Nq,Nk,D,block,topk,causal,lens", ATTN)
def test_attention_and_gradient(B, Hq, Hk, Nq, Nk, D, block, topk, causal, lens):
    q, k, v = tokens(60, B, Hq, Hk, Nq, Nk, D)
    sel = lists(63, B * Hk, Nq, topk, -(-Nk // block))
    kv = None if lens is None else i32(*lens)
    per_head = [n for n in (lens or [Nk] * B) for _ in range(Hk)]
    scale = 0.11
    o, lse = svg.block_attn(q, k, v, sel, block, causal, scale, kv_len=kv, want_lse=True)
    s = sel.cpu().numpy()
    want, want_l, b, bl = bo.attention(f64(q), f64(k), f64(v), s, block, causal, per_head, scale)
    within(o, want, b, "o")
    within(lse, want_l, bl, "lse")
    do = bf(64, B * Hq, Nq, D)
    got = svg.block_attn_backward(do, q, k, v, o, lse, sel, block, causal, scale, kv_len=kv)
    want, bounds = bo.attention_backward(f64(do), f64(q), f64(k), f64(v), f64(o), f64(lse), s, block, causal,
                                         per_head, scale)
    for x, y, z, n in zip(got, want, bounds, ("dq", "dk", "dv")):
        within(x, y, z, n)
    again = svg.block_attn_backward(do, q, k, v, o, lse, sel, block, causal, scale, kv_len=kv)
    assert all(torch.equal(x, y) for x, y in zip(got, again))     # sums in a fixed order
    o2, lse2 = svg.block_attn(q, k, v, sel, block, causal, scale, kv_len=kv, want_lse=True)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("G,D,causal", [(5, 128, True), (1, 64, False)])
def test_many_tiles_at_once(G, D, causal):
    """Hundreds of tiles that share the GPU, so that warps of a tile run apart: against dense attention in 64 bits, and
    twice the same."""
    Hk, N, topk = 4, 3000, 12
    Hq = Hk * G
    q, k, v = tokens(66, 1, Hq, Hk, N, N, D)
    g = torch.Generator().manual_seed(67)
    near = torch.arange(N)[None, :, None] // 64 - torch.arange(4)
    sel = torch.cat([near.expand(Hk, N, 4), torch.randint(0, 47, (Hk, N, topk - 4), generator=g)], 2).int().cuda()
    o, lse = svg.block_attn(q, k, v, sel, 64, causal, want_lse=True)
    do = bf(69, Hq, N, D)
    grads = svg.block_attn_backward(do, q, k, v, o, lse, sel, 64, causal)
    for _ in range(3):
        again = svg.block_attn(q, k, v, sel, 64, causal, want_lse=True)
        assert torch.equal(again[0], o) and torch.equal(again[1], lse)
        for x, y in zip(svg.block_attn_backward(do, q, k, v, o, lse, sel, 64, causal), grads):
            assert torch.equal(x, y)
    hit = torch.zeros(Hk, N, 48, dtype=torch.bool, device="cuda")
    hit.scatter_(2, torch.where(sel < 0, 47, sel).long(), True)
    mask = hit[:, :, :47].repeat_interleave(64, 2)[:, :, :N]
    if causal:
        mask &= torch.arange(N, device="cuda") <= torch.arange(N, device="cuda")[:, None]
    for h in range(Hq):
        kk, vv = k[h // G].double(), v[h // G].double()
        s = (q[h].double() @ kk.T * D ** -0.5).masked_fill(~mask[h // G], -float("inf"))
        p = s.softmax(-1)
        size = p @ vv.abs()
        # half a bf16 step of the result and of the weights, and their sums
        assert ((o[h].double() - p @ vv).abs() <= bo.HALF_BF16 * ((p @ vv).abs() + 1.1 * size)).all(), h
        assert ((lse[h] - s.logsumexp(-1)).abs() <= 1e-4).all()
        ds = p * (do[h].double() @ vv.T - (do[h].double() * o[h].double()).sum(-1, keepdim=True))
        want = ds @ kk * D ** -0.5
        bound = bo.HALF_BF16 * (want.abs() + 1.2 * (ds.abs() @ kk.abs()) * D ** -0.5)
        assert ((grads[0][h].double() - want).abs() <= bound + 1e-4).all(), h


def test_gradient_of_a_block_that_everyone_lists():
    """A block whose queries fill several work items: partial sums in fp32, joined in order."""
    Hq, Hk, N, D = 8, 2, 1100, 64
    q, k, v = tokens(70, 1, Hq, Hk, N, N, D)
    sel = torch.zeros(Hk, N, 3, dtype=torch.int32, device="cuda")
    sel[:, :, 1] = torch.arange(N, device="cuda") // 64
    sel[:, :, 2] = -1
    scale = D ** -0.5
    o, lse = svg.block_attn(q, k, v, sel, 64, want_lse=True)
    do = bf(73, Hq, N, D)
    got = svg.block_attn_backward(do, q, k, v, o, lse, sel, 64)
    want, bounds = bo.attention_backward(f64(do), f64(q), f64(k), f64(v), f64(o), f64(lse), sel.cpu().numpy(), 64,
                                         True, [N] * Hk, scale)
    assert N * Hq // Hk > 2 * 2048                  # more than two items' rows
    for x, y, z, n in zip(got, want, bounds, ("dq", "dk", "dv")):
        within(x, y, z, n)


@pytest.mark.parametrize("Nq", [1, 60])
def test_what_a_query_does_not_list_does_not_reach_it(Nq):
    """NaN and infinities behind the sequence and in blocks that some queries do not list."""
    Hq, Hk, Nk, D = 4, 1, 400, 128
    q, k, v = tokens(80, 2, Hq, Hk, Nq, Nk, D)
    lens = [330, 400]
    sel = torch.full((2, Nq, 2), 0, dtype=torch.int32, device="cuda")
    sel[:, ::2, 1] = 3
    kv = i32(*lens)
    clean, lse = svg.block_attn(q, k, v, sel, 64, False, kv_len=kv, want_lse=True)
    k2, v2 = k.clone(), v.clone()
    for t in (k2, v2):
        t[0, 330:] = float("nan")
        t[:, 64:192] = float("inf")
        t[1, 193] = float("nan")                    # block 3 of the second sequence
    o, lse2 = svg.block_attn(q, k2, v2, sel, 64, False, kv_len=kv, want_lse=True)
    per = o.view(2, Hq, Nq, D), clean.view(2, Hq, Nq, D)
    assert torch.equal(per[0][0], per[1][0])
    assert torch.equal(per[0][1][:, 1::2], per[1][1][:, 1::2]) and per[0][1][:, ::2].isnan().any()
    do = bf(83, 2 * Hq, Nq, D)
    g = svg.block_attn_backward(do, q, k, v, clean, lse, sel, 64, False, kv_len=kv)
    k2[1, 193], v2[1, 193] = k[1, 193], v[1, 193]
    g2 = svg.block_attn_backward(do, q, k2, v2, clean, lse, sel, 64, False, kv_len=kv)
    assert all(torch.equal(x, y) for x, y in zip(g, g2))


@pytest.mark.parametrize("D", [64, 128])
def test_weights_that_outgrow_their_reference_and_keys_of_minus_infinity(D):
    """Scores that rise by far more than the rescaling step from block to block, a key whose scores are all -inf,
    and a query with no finite score."""
    N, scale = 300, D ** -0.5
    q, k, v = tokens(85, 1, 2, 1, N, N, D)
    k[0] *= (1.0 + torch.arange(N, device="cuda") // 64 * 3)[:, None].to(BF)
    q[0, 200] = 1.0
    k[0, 70] = -float("inf")                        # -inf for that query, NaN or -inf for others
    sel = torch.arange(5, dtype=torch.int32, device="cuda").expand(1, N, 5).contiguous()
    o, lse = svg.block_attn(q, k, v, sel, 64, True, want_lse=True)
    k[0, 70] = 0
    s = (q[0, 200].float() @ k[0, :201].float().T) * scale
    s[70] = -float("inf")
    want = (s.double().softmax(0) @ v[0, :201].double())
    assert (o[0, 200].double() - want).abs().max() <= 0.04 and abs(lse[0, 200] - s.double().logsumexp(0)) <= 1e-4
    assert o[:, :70].isfinite().all()
    o, lse = svg.block_attn(q, k, v, sel, 64, True, want_lse=True)
    want, want_l, b, bl = bo.attention(f64(q), f64(k), f64(v), sel.cpu().numpy(), 64, True, [N], scale)
    within(o, want, b)
    within(lse, want_l, bl)


def test_future_keys_that_are_not_finite_stay_in_the_future():
    """Causal rows of a block whose later keys hold NaN and infinities (V and K): rows before them are clean."""
    N, D = 150, 128
    q, k, v = tokens(86, 1, 4, 2, N, N, D)
    sel = torch.arange(3, dtype=torch.int32, device="cuda").expand(2, N, 3).contiguous()
    clean, lse = svg.block_attn(q, k, v, sel, 64, True, want_lse=True)
    do = bf(87, 4, N, D)
    dq, _, _ = svg.block_attn_backward(do, q, k, v, clean, lse, sel, 64)
    k2, v2 = k.clone(), v.clone()
    v2[:, 100] = float("nan")
    k2[0, 101] = float("inf")
    v2[1, 30, 5] = float("inf")
    o, lse2 = svg.block_attn(q, k2, v2, sel, 64, True, want_lse=True)
    first = [100, 100, 30, 30]
    for h, n in enumerate(first):
        # a row computed again sums in another order: one rounding each
        off = (o[h, :n].double() - clean[h, :n].double()).abs()
        assert (off <= 2 * bo.HALF_BF16 * (clean[h, :n].double().abs() + v[h // 2].double().abs().max())).all()
        assert (lse2[h, :n] - lse[h, :n]).abs().max() <= 1e-5 * (1 + lse.abs().max())
        assert o[h, 101:].isnan().any(-1).all()
    dq2, _, _ = svg.block_attn_backward(do, q, k2, v2, clean, lse, sel, 64)
    for h, n in enumerate(first):
        a, b = dq2[h, :n].double(), dq[h, :n].double()
        assert a.isfinite().all() and (a - b).norm() <= 0.02 * b.norm()


@pytest.mark.parametrize("Nk", [130, 4000])
def test_a_token_that_is_not_finite_leaves_earlier_ones_alone(Nk):
    """Three new tokens of which the last holds NaN and infinities: one matrix tile holds all three."""
    Nq, D = 3, 64
    q, k, v = tokens(89, 2, 4, 2, Nq, Nk, D)
    sel = torch.arange(-(-Nk // 64), dtype=torch.int32, device="cuda").expand(4, Nq, -1).contiguous()
    clean, lse = svg.block_attn(q, k, v, sel, 64, True, want_lse=True)
    v[:, -1] = float("nan")
    k[0, -1] = float("inf")
    o, lse2 = svg.block_attn(q, k, v, sel, 64, True, want_lse=True)
    assert (o[:, :2].float() - clean[:, :2].float()).abs().max() <= 2 * bo.HALF_BF16 * 4
    assert (lse2[:, :2] - lse[:, :2]).abs().max() <= 1e-5 * (1 + lse.abs().max())
    assert o[:, 2].isnan().any(-1).all()


def test_gradient_without_keys():
    """Q alone (cross attention prepares K elsewhere)."""
    q, _, _, w_q, _ = rope_inputs(1, 9, 4, 1, 64, seed=130)
    cos, sin = svg.rope_table((9,), 64)
    qo, ko, vo = svg.qk_norm_rope(q, None, None, w_q, None, cos, sin)
    assert ko is None and vo is None
    dqo = bf(131, 4, 9, 64)
    dq, dk, dv, dw_q, dw_k = svg.qk_norm_rope_backward(dqo, None, None, q, None, w_q, None, cos, sin)
    assert dk is None and dv is None and dw_k is None
    pos = np.arange(9)[None]
    want, want_w, size, terms = bo.norm_rope_backward(f64(q), f64(w_q), f64(cos), f64(sin), 1e-6, True, pos,
                                                      f64(dqo).reshape(1, 4, 9, 64))
    within(dq, want, bo.HALF_BF16 * np.abs(want) + 300 * bo.HALF_F32 * size)
    within(dw_q, want_w, 600 * bo.HALF_F32 * terms)


def test_a_sequence_of_4096_blocks():
    """The longest list of blocks; its bit sets leave the gradient half a tile of tokens."""
    Hq, Nq, Nk, D = 2, 150, 262144, 128
    q, k, v = tokens(94, 1, Hq, Hq, Nq, Nk, D)
    g = np.random.default_rng(95)
    sel = torch.from_numpy(np.sort(g.integers(0, 4096, (Hq, Nq, 4)).astype(np.int32), -1)).cuda()
    sel[:, :, 3] = 4095
    o, lse = svg.block_attn(q, k, v, sel, 64, want_lse=True)
    do = bf(98, Hq, Nq, D)
    got = svg.block_attn_backward(do, q, k, v, o, lse, sel, 64)
    dk, dv = torch.zeros_like(k, dtype=torch.float64), torch.zeros_like(v, dtype=torch.float64)
    for h in range(Hq):
        for n in range(0, Nq, 7):
            keys = torch.cat([torch.arange(j * 64, (j + 1) * 64, device="cuda") for j in sel[h, n].unique()])
            keys = keys[keys <= Nk - Nq + n]
            kk, vv = k[h, keys].double(), v[h, keys].double()
            s = kk @ q[h, n].double() * D ** -0.5
            p = s.softmax(0)
            assert abs(lse[h, n] - s.logsumexp(0)) <= 1e-4
            assert ((o[h, n].double() - p @ vv).abs() <= 2.2 * bo.HALF_BF16 * (p @ vv.abs())).all()
            ds = p * (vv @ do[h, n].double() - do[h, n].double() @ o[h, n].double())
            assert ((got[0][h, n].double() - ds @ kk * D ** -0.5).abs()
                    <= 3 * bo.HALF_BF16 * (ds.abs() @ kk.abs()) * D ** -0.5 + 1e-3).all()
    # what nobody lists has no gradient
    listed = torch.zeros(Hq, 4096, dtype=torch.bool, device="cuda").scatter_(1, sel.flatten(1).long(), True)
    for x in got[1:]:
        assert not x.view(Hq, 4096, 64 * D)[~listed].any() and x.view(Hq, 4096, 64 * D)[listed].any(-1).all()


def test_a_wait_that_runs_out_is_reported_and_leaves_the_library_usable():
    """A host-set flag keeps the matrix kernels from loading K and V, so their bounded waits run out: they record it,
    free their tensor memory and return (no GPU fault)."""
    lib = svg.load_library()
    N, D = 200, 128
    q, k, v = tokens(88, 1, 4, 2, N, N, D)
    sel = torch.arange(4, dtype=torch.int32, device="cuda").expand(2, N, 4).contiguous()
    want, lse = svg.block_attn(q, k, v, sel, 64, want_lse=True)
    grads = svg.block_attn_backward(q, q, k, v, want, lse, sel, 64)
    torch.cuda.synchronize()
    assert svg.get_error() == 0
    try:
        svg.set_wait_timeout_ns(20_000_000)
        lib.svg_debug_set_fault(1)
        svg.block_attn(q, k, v, sel, 64)
        assert svg.get_error_detail()[:2] == (5, "block attention")
        svg.block_attn_backward(q, q, k, v, want, lse, sel, 64)
        assert svg.get_error_detail()[:2] == (5, "block attention")
    finally:
        lib.svg_debug_set_fault(0)
        svg.set_wait_timeout_ns(0)
    again, _ = svg.block_attn(q, k, v, sel, 64)
    assert torch.equal(again, want) and svg.get_error() == 0
    for x, y in zip(svg.block_attn_backward(q, q, k, v, want, lse, sel, 64), grads):
        assert torch.equal(x, y)


def test_offsets_beyond_32_bits():
    """The last head of a cache of more than 2^32 bytes and 2^31 elements."""
    Hk, Nk, D, Nq = 260, 65536, 128, 1
    assert Hk * Nk * D > 2 ** 31
    k = torch.zeros(Hk, Nk, D, dtype=BF, device="cuda")
    v = torch.zeros_like(k)
    k[-1, -200:], v[-1, -200:] = bf(90, 200, D), bf(91, 200, D)
    q = bf(92, Hk, Nq, D)
    mean = svg.block_mean(k, 64)
    assert np.array_equal(mean[-1, -3:].cpu().numpy(), bo.block_means(f64(k[-1:, -192:]), 64, [192])[0])
    sel = svg.block_select(q, mean, 64, 3, Nk, 0, 3)
    assert sel[-1, 0].tolist() == [1021, 1022, 1023]
    o, lse = svg.block_attn(q, k, v, sel, 64, want_lse=True)
    want, want_l, b, bl = bo.attention(f64(q[-1:]), f64(k[-1:, -192:]), f64(v[-1:, -192:]),
                                       np.array([[[0, 1, 2]]]), 64, True, [192], D ** -0.5)
    within(o[-1:], want, b)
    within(lse[-1:], want_l, bl)
    new = bf(93, Hk, 1, D).view(1, 1, Hk, D)
    svg.qk_norm_rope(new, new, new, start=i32(Nk - 1), k_out=k, v_out=v)
    assert torch.equal(v[-1, -1], new[0, 0, -1]) and torch.equal(v[-2, -1], new[0, 0, -2])


# ----------------------------------------------------------------------- together
def test_a_prompt_and_decoding_steps_through_a_cache():
    """Preparation, means, selection and attention as a generator calls them: the steps' rows are those that one call
    over the whole context gives."""
    B, Hq, Hk, D, cap, block, topk = 2, 6, 2, 64, 400, 64, 3
    total = [300, 211]
    width = Hq + 2 * Hk
    x = bf(100, B, max(total), width, D)
    w_q, w_k = rope_inputs(1, 1, 1, 1, D)[3:]
    cos, sin = svg.rope_table((cap,), D)

    def split(t):
        return t[:, :, :Hq], t[:, :, Hq:Hq + Hk], t[:, :, Hq + Hk:]

    # one call over everything, left-padded
    N = max(total)
    padded = torch.stack([torch.cat([x.new_zeros(N - n, width, D), x[b, :n]]) for b, n in enumerate(total)])
    kc, vc = (torch.zeros(B * Hk, cap, D, dtype=BF, device="cuda") for _ in range(2))
    qo, _, _ = svg.qk_norm_rope(*split(padded), w_q, w_k, cos, sin, start=i32(*(n - N for n in total)), k_out=kc,
                                v_out=vc)
    kv = i32(*total)
    whole, _, sel, mean = svg.block_attention(qo, kc, vc, block, topk, kv_len=kv)
    # the prompt without its last 5 tokens, then one token at a time
    steps = 5
    k2, v2 = torch.zeros_like(kc), torch.zeros_like(vc)
    M = N - steps
    padded_m = torch.stack([torch.cat([x.new_zeros(N - n, width, D), x[b, :n - steps]]) for b, n in enumerate(total)])
    qm, _, _ = svg.qk_norm_rope(*split(padded_m), w_q, w_k, cos, sin, start=i32(*(n - N for n in total)), k_out=k2,
                                v_out=v2)
    lens = torch.tensor(total, dtype=torch.int32, device="cuda") - steps
    means = svg.block_mean(k2, block, kv_len=lens)
    first, _, s1, _ = svg.block_attention(qm, k2, v2, block, topk, kv_len=lens)
    assert torch.equal(s1, sel[:, :M])

    def near(a, b):
        # another split of the same sums: each is within half a bf16 step of its weights and of its result
        a, b = f64(a), f64(b)
        assert np.abs(a - b).max() <= 2 * 2 * bo.HALF_BF16 * max(np.abs(b).max(), 4.0)

    near(first, whole[:, :M])
    for i in range(steps):
        tok = torch.stack([x[b, n - steps + i:n - steps + i + 1] for b, n in enumerate(total)])
        q1, _, _ = svg.qk_norm_rope(*split(tok), w_q, w_k, cos, sin, start=lens, k_out=k2, v_out=v2)
        lens = lens + 1
        o, _, s1, _ = svg.block_attention(q1, k2, v2, block, topk, kv_len=lens, mean=means, new=1)
        assert torch.equal(s1[:, 0], sel[:, M + i])
        near(o[:, 0], whole[:, M + i])
    assert torch.equal(k2, kc) and torch.equal(v2, vc) and torch.equal(means, mean)
    assert svg.get_error() == 0


def test_prepared_rows_feed_the_cluster_layer():
    """qk_norm_rope's outputs are the rows that SvgLayer reads."""
    N, H, D = 512, 2, 64
    q, k, v, w_q, w_k = rope_inputs(1, N, H, H, D, seed=110)
    cos, sin = svg.rope_table((8, 8, 8), D)
    qo, ko, vo = svg.qk_norm_rope(q, k, v, w_q, w_k, cos, sin)
    out, _ = svg.svg_attention(qo, ko, vo, qo[:, :8].float().contiguous(), ko[:, :16].float().contiguous(), 2, 1.0)
    every = torch.arange(8, dtype=torch.int32, device="cuda").expand(H, N, 8).contiguous()
    o, _ = svg.block_attn(qo, ko, vo, every, 64, causal=False)
    assert (o.float() - out.float()).norm() <= 0.01 * out.float().norm()


def all_calls(stream=None):
    """Every call once on fixed inputs; returns a function and its outputs' list."""
    B, Hq, Hk, N, D = 2, 6, 2, 150, 64
    q, k, v, w_q, w_k = rope_inputs(B, N, Hq, Hk, D, seed=120)
    cos, sin = svg.rope_table((N,), D)
    kv = i32(N, 100)
    q1 = bf(124, B * Hq, 1, D)

    def run():
        qo, ko, vo = svg.qk_norm_rope(q, k, v, w_q, w_k, cos, sin, stream=stream)
        o, lse, sel, mean = svg.block_attention(qo, ko, vo, 64, 2, 0, 1, kv_len=kv, want_lse=True, stream=stream)
        g = svg.block_attn_backward(o, qo, ko, vo, o, lse, sel, 64, kv_len=kv, stream=stream)
        h = svg.qk_norm_rope_backward(*g, q, k, w_q, w_k, cos, sin, stream=stream)
        o1, _, s1, _ = svg.block_attention(q1, ko, vo, 64, 2, 0, 1, kv_len=kv, stream=stream)
        return [qo, ko, vo, o, lse, sel, mean, *g, *h, o1, s1]

    return run


def test_another_stream_gives_the_same():
    want = all_calls()()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    run = all_calls(side)
    side.wait_stream(torch.cuda.current_stream())
    got = [run() for _ in range(3)][-1]
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_captured_and_replayed_calls_give_the_same():
    run = all_calls()
    want = run()
    torch.cuda.synchronize()
    first, second = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(first):
        a = run()
    with torch.cuda.graph(second, pool=first.pool()):
        b = run()
    for _ in range(3):
        first.replay()
        second.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(b, want))
    first.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a, want))


# ----------------------------------------------------------------------- refusals
def test_wrapper_refusals():
    q, k, v, w_q, w_k = rope_inputs(1, 4, 2, 2, 64)
    cos, sin = svg.rope_table((4,), 64)
    with pytest.raises(ValueError):
        svg.qk_norm_rope(q, k, v, w_q, w_k, cos, None)
    with pytest.raises(ValueError):
        svg.qk_norm_rope(q, k, v, w_q, w_k, cos, sin, start=i32(0))           # no buffers
    with pytest.raises(ValueError):
        svg.qk_norm_rope(q.transpose(2, 3), k, v)                             # channels not contiguous
    with pytest.raises(ValueError):
        svg.qk_norm_rope(q.float(), k, v)
    with pytest.raises(ValueError):
        svg.qk_norm_rope(q, k, v, w_q.cpu(), w_k)
    with pytest.raises(svg.SvgError):
        svg.qk_norm_rope(q, k, v, w_q, w_k, cos[:3].contiguous(), sin[:3].contiguous())   # table too short
    with pytest.raises(svg.SvgError):
        svg.qk_norm_rope(q, k, v, k_out=bf(1, 2, 3, 64), v_out=bf(1, 2, 3, 64))           # buffer too short
    with pytest.raises(ValueError):
        svg.qk_norm_rope_backward(bf(1, 2, 4, 64), None, None, q, dq=q[:, :, :1].expand(1, 4, 2, 64))
    qh, kh, vh = tokens(1, 1, 4, 2, 10, 100, 64)
    sel = torch.zeros(2, 10, 2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        svg.block_attn(qh, kh, vh, sel.long(), 64)
    with pytest.raises(ValueError):
        svg.block_attn(qh, kh, vh[:, :50], sel, 64)
    with pytest.raises(ValueError):
        svg.block_attn(qh, kh, vh, sel, 64, kv_len=i32(1, 2, 3))
    with pytest.raises(svg.SvgError):
        svg.block_attn(qh, kh, vh, sel, 32)
    with pytest.raises(svg.SvgError):
        svg.block_attn(qh, kh, vh, sel, 64, o=qh)
    with pytest.raises(svg.SvgError):
        svg.block_attn(qh[:3], kh, vh, sel, 64)
    with pytest.raises(ValueError):
        svg.block_mean(kh, 64, new=1)
    with pytest.raises(svg.SvgError):
        svg.block_select(qh, torch.zeros(2, 2, 64, device="cuda"), 64, 2, 100, 2, 1)      # sink + local > topk
    with pytest.raises(svg.SvgError):
        svg.block_select(qh, torch.zeros(2, 2, 64, device="cuda"), 64, 2, 100, 0, 0)      # causal without local
    with pytest.raises(ValueError):
        svg.block_select(qh, torch.zeros(2, 3, 64, device="cuda"), 64, 2, 100)
