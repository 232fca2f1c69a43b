"""Host side of blocks.py's calls, without a GPU: refusals and workspace sizes."""
import ctypes

import pytest

import sparse_attention_long_svg_b200 as svg


@pytest.fixture(scope="module")
def lib():
    from sparse_attention_long_svg_b200 import build
    build.build()
    return svg.load_library()


def at(x):
    return ctypes.c_void_p(x)


NUL = at(0)
ROW = (ctypes.c_int64 * 3)(512, 64, 64)


def test_a_rotation_does_not_write_over_any_input(lib):
    """Outputs are other buffers than every input, not only the one of the same name; in-place gradients are open."""
    q, k, v, qo, ko, vo = (0x10000 * i for i in range(1, 7))

    def forward(qo=qo, ko=ko, vo=vo):
        return lib.svg_qk_norm_rope(at(q), ROW, at(k), ROW, at(v), ROW, NUL, NUL, NUL, NUL, 0, 1, 8, 1, 1, 64, 1e-6, 1,
                                    NUL, at(qo), at(ko), at(vo), 8, NUL)

    assert forward(qo=q) == 1 and forward(ko=k) == 1 and forward(vo=v) == 1
    assert forward(qo=k) == 1 and forward(qo=v) == 1 and forward(ko=q) == 1 and forward(ko=v) == 1
    assert forward(vo=q) == 1 and forward(vo=k) == 1

    def backward(dq=0x70000, dk=0x80000, dv=0x90000, dqs=ROW):
        return lib.svg_qk_norm_rope_backward(at(qo), at(ko), at(vo), at(q), ROW, at(k), ROW, NUL, NUL, NUL, NUL, 0, 1, 8,
                                             1, 1, 64, 1e-6, 1, NUL, 8, at(dq), dqs, at(dk), ROW, at(dv), ROW, NUL, NUL,
                                             at(0xA0000), 0, NUL)

    assert backward() == 3                            # in order but for the workspace
    assert backward(dq=qo) == 1 and backward(dk=ko) == 1 and backward(dv=vo) == 1
    assert backward(dq=ko) == 1 and backward(dq=vo) == 1 and backward(dk=qo) == 1 and backward(dk=vo) == 1
    assert backward(dv=qo) == 1 and backward(dv=ko) == 1
    assert backward(dq=k) == 1 and backward(dk=q) == 1 and backward(dv=q) == 1 and backward(dv=k) == 1
    assert backward(dq=q) == 3 and backward(dk=k) == 3  # a row's gradient may replace it
    assert backward(dq=q, dqs=(ctypes.c_int64 * 3)(512, 64, 512)) == 1


@pytest.mark.parametrize("heads,D", [(1, 64), (3, 64), (16, 64), (40, 128), (17, 128)])
@pytest.mark.parametrize("tokens", [1, 10_002, 524_160, 4_000_000])
def test_sums_of_the_weight_gradient_stay_short(lib, heads, D, tokens):
    """A thread adds at most 256 rows in fp32 before its sum goes on in fp64, whatever the number of tokens: there
    are that many partial rows."""
    size = lib.svg_qk_norm_rope_backward_workspace_size(1, tokens, heads, 0, D)
    chunks = -(-heads // 16)
    tiles = size // (4 * D * chunks)                  # (sizes are whole multiples of 256 bytes)
    groups = 128 // (D // 16)
    assert tiles * groups * 16 >= tokens


def test_refused_shapes_ask_for_no_workspace(lib):
    """A call that will be refused does not make the caller allocate first."""
    size = lib.svg_block_select_workspace_size
    assert size(8, 100, 4096, 128, 64) > 0 and size(8, 100, 4096, 128, 128) > 0
    assert size(8, 100, 4096, 128, 32) == 0 and size(8, 100, 4096, 96, 64) == 0
    assert size(8, 100, 64 * 4096 + 1, 128, 64) == 0 and size(8, 100, 1 << 20, 128, 1) == 0
    assert size(8, 4, 4096, 128, 64) == 0             # few queries need none
    for f in (lib.svg_block_attn_workspace_size, lib.svg_block_attn_backward_workspace_size):
        assert f(8, 8, 1, 4096, 128, 16, 32) == 0 and f(8, 8, 1, 64 * 4096 + 1, 128, 16, 64) == 0
        assert f(8, 3, 1, 4096, 128, 16, 64) == 0 and f(8, 8, 1, 4096, 128, 0, 64) == 0
