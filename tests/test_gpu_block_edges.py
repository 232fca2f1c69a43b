"""GPU tests of the edges of blocks.py, against oracle/block_oracle.py or dense forms in 64 bits."""
import threading

import numpy as np
import pytest
import torch

from oracle import block_oracle as bo
from tests.test_gpu_blocks import BF, _lib, bf, check_rows, f64, i32, rope_inputs, tokens, within  # noqa: F401

pytestmark = pytest.mark.gpu

svg = pytest.importorskip("sparse_attention_long_svg_b200")


# ----------------------------------------------------------------------- selection
@pytest.mark.parametrize("Nq", [3, 70])
@pytest.mark.parametrize("nblk,topk", [(100, 9), (400, 60), (1100, 12)])
def test_selection_of_scores_beyond_fp32(Nq, nblk, topk):
    """Finite queries and means whose products overflow: the list is still the one of exact scores, and whole."""
    D, Nk = 64, nblk * 64
    q = bf(200, 8, Nq, D)
    mean = torch.randn(4, nblk, D, generator=torch.Generator().manual_seed(201)).cuda()
    q[0:2, :, 0] = 1e20                              # every score overflows, to either side
    mean[0, :, 0] *= 1e20
    q[2:4, :, 5] = 1e20                              # a few blocks do
    mean[1, :, 5] = 0
    mean[1, 3:7, 5] = torch.tensor([2e20, 1e20, -1e20, 3e20], device="cuda")
    q[4, ::2, 9] = 1e30                              # some queries, by norm alone
    q[5, 1::2, 9] = -1e30
    mean[2, :, 9] *= 1e-3
    q[6, 1, 3] = float("inf")                        # a query with an infinity, one with a NaN
    q[7, 2, 3] = float("nan")
    sel = torch.full((4, Nq, topk), -7, dtype=torch.int32, device="cuda")
    svg.block_select(q, mean, 64, topk, Nk, 1, 1, True, sel=sel)
    want = bo.select_blocks(f64(q), f64(mean), 64, topk, 1, 1, True, [Nk] * 4)
    assert np.array_equal(sel.cpu().numpy(), want), np.argwhere(sel.cpu().numpy() != want)[:5]


@pytest.mark.parametrize("B,Hq,Hk,Nq", [(1, 32, 16, 32), (1, 17, 17, 32), (4, 120, 30, 5), (3, 34, 34, 5), (1, 15, 15, 33)])
def test_selection_by_either_kernel(B, Hq, Hk, Nq):
    """Both sides of the switch between a CTA per query and a CTA per 64 queries."""
    D, Nk, lens = 64, 9000, (9000, 20, 4097, 640)[:B]
    q = bf(205, B * Hq, Nq, D)
    mean = torch.randn(B * Hk, -(-Nk // 64), D, generator=torch.Generator().manual_seed(206)).cuda()
    mean[:, 6] = mean[:, 4] * (1 + 2.0 ** -22)
    sel = svg.block_select(q, mean, 64, 12, Nk, 1, 2, True, kv_len=i32(*lens))
    want = bo.select_blocks(f64(q), f64(mean), 64, 12, 1, 2, True, [n for n in lens for _ in range(Hk)])
    assert np.array_equal(sel.cpu().numpy(), want), np.argwhere(sel.cpu().numpy() != want)[:5]


# ----------------------------------------------------------------------- norm and rotation
def test_tokens_beyond_the_table_leave_every_cache_row_alone():
    """P <= position < cap: as for padding, Q's row is zero and neither K nor V is stored; the gradient is zero."""
    B, N, H, D, cap, P = 2, 5, 3, 64, 20, 8
    q, k, v, w_q, w_k = rope_inputs(B, N, H, H, D, seed=210)
    cos, sin = svg.rope_table((P,), D)
    start = i32(5, 1)                                # positions 5 .. 9 and 1 .. 5
    ko, vo = bf(213, B * H, cap, D), bf(214, B * H, cap, D)
    old_k, old_v = ko.clone(), vo.clone()
    qo, _, _ = svg.qk_norm_rope(q, k, v, w_q, w_k, cos, sin, start=start, k_out=ko, v_out=vo)
    assert svg.get_error_detail()[:2] == (6, "rotation range")
    pos = np.array([[5, 6, 7, -1, -1], [1, 2, 3, 4, 5]])          # beyond the table: as padding
    check_rows(qo, q, w_q, cos, sin, 1e-6, True, pos, "q")
    for b in range(B):
        rows = pos[b][pos[b] >= 0].tolist()
        kept = [r for r in range(cap) if r not in rows]
        heads = slice(b * H, (b + 1) * H)
        assert torch.equal(vo[heads][:, rows], v[b, :len(rows)].transpose(0, 1))
        assert torch.equal(vo[heads][:, kept], old_v[heads][:, kept])
        assert torch.equal(ko[heads][:, kept], old_k[heads][:, kept])
        assert (ko[heads][:, rows] != old_k[heads][:, rows]).any(-1).all()
    dqo, dko, dvo = bf(215, B * H, N, D), bf(216, B * H, cap, D), bf(217, B * H, cap, D)
    dq, dk, dv, dw_q, dw_k = svg.qk_norm_rope_backward(dqo, dko, dvo, q, k, w_q, w_k, cos, sin, start=start)
    assert svg.get_error_detail()[:2] == (6, "rotation range")
    for x in (dq, dk, dv):
        assert not x[0, 3:].any() and x[0, :3].any(-1).all() and x[1].any(-1).all()
    want, want_w, size, terms = bo.norm_rope_backward(f64(q), f64(w_q), f64(cos), f64(sin), 1e-6, True, pos,
                                                      f64(dqo).reshape(B, H, N, D))
    within(dq, want, bo.HALF_BF16 * np.abs(want) + 300 * bo.HALF_F32 * size, "dq")
    within(dw_q, want_w, 600 * bo.HALF_F32 * terms, "dw_q")


def test_tokens_beyond_the_buffer_but_in_the_table():
    """cap <= position < P: Q has its row (and its gradient), K and V have none to go to."""
    N, H, D, cap = 4, 2, 64, 6
    q, k, v, w_q, w_k = rope_inputs(1, N, H, H, D, seed=220)
    cos, sin = svg.rope_table((12,), D)
    ko, vo = bf(223, H, cap, D), bf(224, H, cap, D)
    old_k, old_v = ko.clone(), vo.clone()
    qo, _, _ = svg.qk_norm_rope(q, k, v, w_q, w_k, cos, sin, start=i32(4), k_out=ko, v_out=vo)    # 4 .. 7
    assert svg.get_error_detail()[:2] == (6, "rotation range")
    pos = np.array([[4, 5, 6, 7]])
    check_rows(qo, q, w_q, cos, sin, 1e-6, True, pos, "q")
    assert torch.equal(ko[:, :4], old_k[:, :4]) and torch.equal(vo[:, :4], old_v[:, :4])
    assert torch.equal(vo[:, 4:], v[0, :2].transpose(0, 1))
    dqo, dko, dvo = bf(225, H, N, D), bf(226, H, cap, D), bf(227, H, cap, D)
    dq, dk, dv, dw_q, _ = svg.qk_norm_rope_backward(dqo, dko, dvo, q, k, w_q, w_k, cos, sin, start=i32(4))
    assert svg.get_error() == 6
    want, want_w, size, terms = bo.norm_rope_backward(f64(q), f64(w_q), f64(cos), f64(sin), 1e-6, True, pos,
                                                      f64(dqo).reshape(1, H, N, D))
    within(dq, want, bo.HALF_BF16 * np.abs(want) + 300 * bo.HALF_F32 * size, "dq")
    within(dw_q, want_w, 600 * bo.HALF_F32 * terms, "dw_q")
    assert not dk[0, 2:].any() and not dv[0, 2:].any() and dk[0, :2].any(-1).all()


def test_many_rows_of_few_heads():
    """Large calls whose chunks of 8 heads would be mostly empty: each row is what a small call gives it."""
    N, D = 55_000, 128
    q, k, v, w_q, w_k = rope_inputs(1, N, 1, 1, D, seed=228)
    cos, sin = svg.rope_table((N,), D)
    assert N * 3 * D // 16 >= 148 * 2048 * 4         # threads of a large call
    got = svg.qk_norm_rope(q, k, v, w_q, w_k, cos, sin)
    for a in (0, 30_000, 54_900):
        part = slice(a, a + 100)
        few = svg.qk_norm_rope(q[:, part], k[:, part], v[:, part], w_q, w_k, cos[part].contiguous(),
                               sin[part].contiguous())
        for x, y in zip(got, few):
            assert torch.equal(x[:, part], y)


def test_a_new_v_buffer_beside_a_longer_k_buffer_holds_nothing_else():
    N, H, D, cap = 4, 2, 64, 9
    _, k, v, _, _ = rope_inputs(1, N, H, H, D, seed=230)
    stale = [torch.full((H, cap, D), 7.0, dtype=BF, device="cuda") for _ in range(4)]
    del stale                                        # the allocator hands these out again
    ko = torch.zeros(H, cap, D, dtype=BF, device="cuda")
    _, _, vo = svg.qk_norm_rope(k, k, v, k_out=ko)
    assert torch.equal(vo[:, :N], v[0].transpose(0, 1)) and not vo[:, N:].any()


def test_a_gradient_may_replace_its_input():
    B, N, H, D = 2, 37, 3, 128
    q, k, v, w_q, w_k = rope_inputs(B, N, H, H, D, seed=235)
    cos, sin = svg.rope_table((N,), D)
    dy = [bf(238 + i, B * H, N, D) for i in range(3)]
    want = svg.qk_norm_rope_backward(*dy, q, k, w_q, w_k, cos, sin)
    got = svg.qk_norm_rope_backward(*dy, q, k, w_q, w_k, cos, sin, dq=q, dk=k, dv=v)     # slices of one buffer
    assert got[0] is q and all(torch.equal(a, b) for a, b in zip(got, want))


def test_weight_gradient_over_many_tokens():
    """Sums over 400,000 tokens with a mean, so that roundings add up: at most 256 fp32 additions to a thread's sum,
    8 to a CTA's, fp64 behind them."""
    N, H, D = 400_000, 3, 64
    g = torch.Generator(device="cuda").manual_seed(240)
    q = (torch.randn(1, N, H, D, generator=g, device="cuda") + 2.0).to(BF)
    dqo = (torch.rand(H, N, D, generator=g, device="cuda") + 0.5).to(BF)
    _, _, _, dw, _ = svg.qk_norm_rope_backward(dqo, None, None, q, eps=1e-5)
    want = torch.zeros(D, dtype=torch.float64, device="cuda")
    for a in range(0, N, 50_000):
        x = q[0, a:a + 50_000].double()
        n = x / (x.pow(2).mean(-1, keepdim=True) + 1e-5).sqrt()
        want += (n * dqo[:, a:a + 50_000].double().transpose(0, 1)).sum((0, 1))
    # a product of a value, rsqrt (2 ulp of a sum of 64 squares) and u: below 64 + 8 half steps, all terms positive
    assert ((dw.double() - want).abs() <= (256 + 32 + 72) * bo.HALF_F32 * want).all()


# ----------------------------------------------------------------------- attention
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Nq", [5, 90])
def test_rows_without_a_finite_score_have_no_gradient(Nq, D):
    """Finite Q and K whose scores are all below fp32's range: the forward call gives such a row zeros and lse = -inf,
    as without keys, so it has no part in any gradient."""
    Hq, Hk, Nk = 2, 1, 300
    q, k, v = tokens(250, 1, Hq, Hk, Nq, Nk, D)
    k[:, 64:128] = -1e20
    q[:, ::3] = 0                                    # scores of zero everywhere
    q[:, 1::3] = 1e20                                # minus infinity in block 1
    sel = torch.zeros(Hk, Nq, 2, dtype=torch.int32, device="cuda")
    sel[:, :, 1] = torch.where(torch.arange(Nq, device="cuda") % 3 == 0, 1, -1)
    sel[:, 1::3, 0] = 1
    o, lse = svg.block_attn(q, k, v, sel, 64, False, want_lse=True)
    assert not o[:, 1::3].any() and (lse[:, 1::3] == -float("inf")).all()
    assert lse[:, ::3].isfinite().all() and lse[:, 2::3].isfinite().all()
    do = bf(253, Hq, Nq, D)
    got = svg.block_attn_backward(do, q, k, v, o, lse, sel, 64, False)
    gone = sel.clone()
    gone[:, 1::3] = -1
    want, bounds = bo.attention_backward(f64(do), f64(q), f64(k), f64(v), f64(o), f64(lse), gone.cpu().numpy(), 64,
                                         False, [Nk], D ** -0.5)
    for x, y, z, n in zip(got, want, bounds, ("dq", "dk", "dv")):
        within(x, y, z, n)
    assert not got[0][:, 1::3].any()


@pytest.mark.parametrize("G,N,items", [(16, 700, 3), (4, 2200, 3)])
def test_gradient_of_key_tiles_with_three_items(G, N, items):
    """A block whose queries fill more than two work items of 4,096 rows: their sums are joined in order."""
    Hk, D = 2, 64
    Hq = Hk * G
    assert -(-N // (4096 // G)) == items
    q, k, v = tokens(260, 1, Hq, Hk, N, N, D)
    sel = torch.zeros(Hk, N, 2, dtype=torch.int32, device="cuda")
    sel[:, :, 1] = torch.arange(N, device="cuda") // 64
    o, lse = svg.block_attn(q, k, v, sel, 64, want_lse=True)
    do = bf(263, Hq, N, D)
    got = svg.block_attn_backward(do, q, k, v, o, lse, sel, 64)
    want, bounds = dense_gradient(do, q, k, v, o, lse, sel, 64, True)
    for x, y, z, n in zip(got, want, bounds, ("dq", "dk", "dv")):
        assert ((x.double() - y).abs() <= z).all(), (n, float(((x.double() - y).abs() - z).max()))


def dense_gradient(do, q, k, v, o, lse, sel, block, causal):
    """Gradients in 64 bits on the device, and their bounds (see oracle/block_oracle.py: attention_backward)."""
    Hq, N, D = q.shape
    Hk, Nk, _ = k.shape
    G, nblk, scale = Hq // Hk, -(-Nk // block), D ** -0.5
    hit = torch.zeros(Hk, N, nblk + 1, dtype=torch.bool, device="cuda")
    hit.scatter_(2, torch.where(sel < 0, nblk, sel).long(), True)
    mask = hit[:, :, :nblk].repeat_interleave(block, 2)[:, :, :Nk]
    if causal:
        mask &= torch.arange(Nk, device="cuda") <= torch.arange(Nk - N, Nk, device="cuda")[:, None]
    out = [torch.zeros_like(x, dtype=torch.float64) for x in (q, k, v, q, k, v)]
    dq, dk, dv, bq, bk, bv = out
    for h in range(Hq):
        j = h // G
        qq, kk, vv, g, y = q[h].double(), k[j].double(), v[j].double(), do[h].double(), o[h].double()
        s = qq @ kk.T * scale
        p = (s - lse[h].double()[:, None]).exp().masked_fill(~mask[j], 0)
        ds = p * (g @ vv.T - (g * y).sum(-1, keepdim=True))
        dq[h] = ds @ kk * scale
        dk[j] += ds.T @ qq * scale
        dv[j] += p.T @ g
        # scores and the exponent's argument in fp32, dP and delta too; P and dS as bf16 operands
        es = D * bo.HALF_F32 * scale * (qq.abs() @ kk.abs().T).amax(-1, keepdim=True) + 8 * bo.HALF_F32 * (
            1 + s.abs().amax(-1, keepdim=True))
        ed = D * bo.HALF_F32 * (g.abs() @ vv.abs().T + (g.abs() * y.abs()).sum(-1, keepdim=True))
        eds = (bo.HALF_BF16 * 1.01 + 2 * es) * ds.abs() + 2 * p * ed
        ep = (bo.HALF_BF16 * 1.01 + 2 * es) * p
        bq[h] = eds @ kk.abs() * scale
        bk[j] += eds.T @ qq.abs() * scale
        bv[j] += ep.T @ g.abs()
    return out[:3], [b * (1 + N * G * bo.HALF_F32) + bo.HALF_BF16 * x.abs() * 1.01 + 1e-30
                     for b, x in zip(out[3:], out[:3])]


@pytest.mark.parametrize("G,D,causal", [(5, 128, True), (1, 64, False)])
def test_all_gradients_of_many_tiles(G, D, causal):
    """dQ, dK and dV of hundreds of tiles that share the GPU, against dense attention in 64 bits."""
    Hk, N, topk = 4, 3000, 12
    Hq = Hk * G
    q, k, v = tokens(270, 1, Hq, Hk, N, N, D)
    g = torch.Generator().manual_seed(271)
    near = torch.arange(N)[None, :, None] // 64 - torch.arange(4)
    sel = torch.cat([near.expand(Hk, N, 4), torch.randint(0, 47, (Hk, N, topk - 4), generator=g)], 2).int().cuda()
    o, lse = svg.block_attn(q, k, v, sel, 64, causal, want_lse=True)
    do = bf(273, Hq, N, D)
    got = svg.block_attn_backward(do, q, k, v, o, lse, sel, 64, causal)
    want, bounds = dense_gradient(do, q, k, v, o, lse, sel, 64, causal)
    for x, y, z, n in zip(got, want, bounds, ("dq", "dk", "dv")):
        assert ((x.double() - y).abs() <= z).all(), (n, float(((x.double() - y).abs() - z).max()))


# ----------------------------------------------------------------------- calls
def test_two_threads_with_lists_of_different_lengths():
    """The kernels' shared memory grows with the number of blocks; calls from two threads do not disturb each other."""
    cases = []
    for seed, Nk in ((280, 200), (290, 262144)):
        q, k, v = tokens(seed, 1, 1, 1, 140, Nk, 64)
        nblk = -(-Nk // 64)
        sel = (torch.arange(140)[:, None] * 7 + torch.arange(3)) % nblk
        sel = sel.int().view(1, 140, 3).cuda()
        mean = svg.block_mean(k, 64)
        one = bf(seed + 5, 1, 1, 64)

        def run(q=q, k=k, v=v, sel=sel, mean=mean, one=one, Nk=Nk):
            o, lse = svg.block_attn(q, k, v, sel, 64, False, want_lse=True)
            s1 = svg.block_select(one, mean, 64, 3, Nk)
            o1, _ = svg.block_attn(one, k, v, s1, 64)
            return [o, lse, *svg.block_attn_backward(q, q, k, v, o, lse, sel, 64, False), s1, o1]

        cases.append((run, run()))
    torch.cuda.synchronize()
    failed = []

    def work(run, want):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(400):
                    got = run()
                torch.cuda.current_stream().synchronize()
                assert all(torch.equal(a, b) for a, b in zip(got, want))
        except Exception as e:  # noqa: BLE001
            failed.append(repr(e))

    threads = [threading.Thread(target=work, args=c) for c in cases * 2]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed


def test_inputs_that_require_grad_are_refused():
    """No call records a gradient, so none is lost in silence; under no_grad, and in a Function, they run."""
    q, k, v, w_q, w_k = rope_inputs(1, 6, 2, 1, 64, seed=300)
    want = svg.qk_norm_rope(q, k, v, w_q, w_k)
    par = torch.nn.Parameter(w_q)
    leaf = q.detach().clone().requires_grad_()
    for args in ((leaf, k, v, w_q, w_k), (q, k, v, par, w_k), (q, k.detach().clone().requires_grad_(), v)):
        with pytest.raises(ValueError, match="qk_norm_rope_backward"):
            svg.qk_norm_rope(*args)
    with torch.no_grad():
        got = svg.qk_norm_rope(leaf, k, v, par, w_k)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    qh, kh, vh = tokens(301, 1, 2, 1, 6, 6, 64)
    sel = torch.zeros(1, 6, 1, dtype=torch.int32, device="cuda")
    o, lse = svg.block_attn(qh, kh, vh, sel, 64, want_lse=True)
    for i in range(3):
        x = [t.clone().requires_grad_() if i == j else t for j, t in enumerate((qh, kh, vh))]
        with pytest.raises(ValueError, match="block_attn_backward"):
            svg.block_attn(*x, sel, 64)
        with pytest.raises(ValueError, match="backward"):
            svg.block_attention(*x, 64, 1, 0, 1)
    with pytest.raises(ValueError, match="detach"):
        svg.block_mean(kh.clone().requires_grad_(), 64)

    class Attend(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, v):
            o, lse = svg.block_attn(q, k, v, sel, 64, want_lse=True)
            ctx.save_for_backward(q, k, v, o, lse)
            return o

        @staticmethod
        def backward(ctx, do):
            return svg.block_attn_backward(do.contiguous(), *ctx.saved_tensors, sel, 64)

    leaves = [t.clone().requires_grad_() for t in (qh, kh, vh)]
    y = Attend.apply(*leaves)
    do = bf(305, 2, 6, 64)
    y.backward(do)
    assert torch.equal(y, o)
    # lists carry no gradient, so they may be made from such inputs; so may gradients by hand
    assert torch.equal(svg.block_select(leaves[0], svg.block_mean(kh, 64), 64, 1, 6, 0, 1), sel)
    for a, b in zip(leaves, svg.block_attn_backward(do, *leaves, o, lse, sel, 64)):
        assert torch.equal(a.grad, b)
