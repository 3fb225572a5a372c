"""Refusals of the block-scaled FP8 and mixture-of-experts calls, their layout queries, and pins of the plain
statements the GPU tests compare with (no GPU needed)."""
from __future__ import annotations

import ctypes
from fractions import Fraction

import pytest
import torch

import fp8b_ref as ref
import mixed_precision_gemm_b200 as sq
from mixed_precision_gemm_b200 import _build

P = ctypes.c_void_p
A, MIS = P(0x1000), P(0x1008)
BAD, MISALIGNED = sq.SQ_ERR_INVALID_ARG, sq.SQ_ERR_MISALIGNED


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return sq.load()


def test_layout_queries(lib):
    assert [sq.sq_k_pad_fp8b(k) for k in (8, 128, 136, 4096)] == [128, 128, 256, 4096]
    assert [sq.sq_scale_ld_fp8b(k) for k in (8, 512, 520, 4096)] == [4, 4, 8, 32]
    assert sq.sq_linear_workspace_bytes_fp8b(0, 128) == 0
    assert sq.sq_linear_workspace_bytes_fp8b(3, 136) == 768 + 256
    assert sq.sq_experts_workspace_bytes_fp8b(0, 2, 4, 128, 128) == 0
    need = sq.sq_experts_workspace_bytes_fp8b(5, 2, 4, 136, 264)
    assert need >= 20 + 40 + 10 * (256 + 16 + 384 + 16 + 272) and need % 256 == 0


@pytest.mark.parametrize("args", [
    (A, 4, 12, 16, A, A, None), (A, 4, 0, 16, A, A, None), (A, 4, 65544, 65544, A, A, None), (A, -1, 64, 64, A, A, None),
    (A, 4, 64, 60, A, A, None), (A, 4, 64, 56, A, A, None), (None, 4, 64, 64, A, A, None), (A, 4, 64, 64, None, A, None),
    (A, 4, 64, 64, A, None, None)])
def test_quant_refuses(lib, args):
    assert lib.sq_quant_fp8b(*args) == BAD
    assert lib.sq_last_error_detail()


def test_misaligned(lib):
    assert lib.sq_quant_fp8b(MIS, 4, 64, 64, A, A, None) == MISALIGNED
    assert lib.sq_gemm_fp8b(A, A, MIS, A, 4, 16, 64, A, 16, None) == MISALIGNED
    assert lib.sq_gemm_fp8b(A, A, A, A, 4, 16, 64, MIS, 16, None) == MISALIGNED
    assert lib.sq_prepare_weights_fp8b(MIS, 1, 16, 64, 64, 0, A, A, None) == MISALIGNED
    assert lib.sq_moe_dispatch(MIS, 4, 2, 8, A, A, None) == MISALIGNED
    assert lib.sq_route(MIS, 0, 4, 8, 8, None, 0, 1, 1, 1, 2, 1, 1.0, A, A, None) == MISALIGNED
    assert lib.sq_moe_combine(A, 8, 64, A, A, 4, 2, 64, MIS, 64, None) == MISALIGNED


def test_products_refuse(lib):
    assert lib.sq_gemm_fp8b(A, A, A, A, 4, 12, 64, A, 16, None) == BAD        # N
    assert lib.sq_gemm_fp8b(A, A, A, A, 4, 16, 60, A, 16, None) == BAD        # K
    assert lib.sq_gemm_fp8b(A, A, A, A, 4, 16, 64, A, 12, None) == BAD        # ldy
    assert lib.sq_gemm_fp8b(A, A, A, A, -4, 16, 64, A, 16, None) == BAD
    assert lib.sq_gemm_fp8b(None, A, A, A, 4, 16, 64, A, 16, None) == BAD
    assert lib.sq_prepare_weights_fp8b(A, -1, 16, 64, 64, 0, A, A, None) == BAD
    assert lib.sq_prepare_weights_fp8b(A, 2, 16, 64, 64, 4, A, A, None) == BAD  # stride between matrices
    need = sq.sq_linear_workspace_bytes_fp8b(8, 64)
    assert lib.sq_linear_fp8b(A, 8, 64, 64, A, A, 16, A, 16, A, need - 1, None) == BAD
    assert lib.sq_moe_gemm_fp8b(A, A, None, 8, A, A, 4, 16, 64, A, 16, None) == BAD   # offsets
    assert lib.sq_moe_gemm_fp8b(A, A, A, 8, A, A, 0, 16, 64, A, 16, None) == BAD      # E
    assert lib.sq_moe_gemm_fp8b(A, A, A, 8, A, A, 513, 16, 64, A, 16, None) == BAD
    assert lib.sq_moe_swiglu_fp8b(A, A, A, 8, A, A, 4, 12, 64, A, A, None) == BAD     # I
    assert lib.sq_moe_swiglu_fp8b(A, A, A, 8, A, A, 4, 16, 64, None, A, None) == BAD


@pytest.mark.parametrize("kw", [dict(E=0), dict(E=513), dict(k=0), dict(k=17), dict(k=9), dict(ld=7), dict(groups=3),
                                dict(groups=0), dict(groups=64, E=64), dict(groups=4, keep=5), dict(groups=4, keep=0),
                                dict(group_top=3), dict(group_top=0), dict(groups=4, keep=1, k=3), dict(T=-1)])
def test_route_refuses(lib, kw):
    a = dict(T=4, E=8, ld=None, groups=1, keep=1, group_top=1, k=2)
    a.update(kw)
    ld = a["E"] if a["ld"] is None else a["ld"]
    st = lib.sq_route(A, 0, a["T"], a["E"], ld, None, 0, a["groups"], a["keep"], a["group_top"], a["k"], 1, 1.0, A, A, None)
    assert st == BAD


def test_experts_refuse(lib):
    need = sq.sq_experts_workspace_bytes_fp8b(4, 2, 8, 64, 128)
    ok = [A, 4, 64, 64, A, A, 2, A, A, A, A, 8, 128, A, 64, A, need, None]
    for i, v in [(1, -1), (2, 60), (3, 56), (6, 0), (6, 17), (11, 0), (12, 100), (14, 56), (16, need - 1), (0, None), (4, None),
                 (5, None), (7, None), (13, None), (15, None)]:
        args = list(ok)
        args[i] = v
        assert lib.sq_experts_fp8b(*args) == BAD, i
    assert lib.sq_moe_combine(A, 8, 64, A, A, 4, 0, 64, A, 64, None) == BAD
    assert lib.sq_moe_combine(A, 8, 60, A, A, 4, 2, 64, A, 64, None) == BAD
    assert lib.sq_moe_dispatch(A, 4, 2, 8, None, A, None) == BAD
    assert lib.sq_moe_quant_fp8b(A, 4, 64, 64, None, 2, A, A, None) == BAD


def test_python_refuses_wrong_tensors():
    f = lambda *s, t=torch.bfloat16: torch.empty(*s, dtype=t)
    with pytest.raises(TypeError):
        sq.sq_quant_fp8b(f(4, 64, t=torch.float16), f(4, 128, t=torch.uint8), f(4, 4, t=torch.float32))
    with pytest.raises(ValueError):
        sq.sq_quant_fp8b(f(4, 64), f(4, 64, t=torch.uint8), f(4, 4, t=torch.float32))
    with pytest.raises(ValueError):
        sq.sq_quant_fp8b(f(4, 128)[:, ::2], f(4, 128, t=torch.uint8), f(4, 4, t=torch.float32))
    with pytest.raises(TypeError):
        sq.sq_route(f(4, 8, t=torch.float16), 2, f(4, 2, t=torch.int32), f(4, 2, t=torch.float32))
    with pytest.raises(ValueError):
        sq.sq_route(f(4, 8, t=torch.float32), 2, f(4, 2, t=torch.int32), f(4, 2, t=torch.float32), scoring="relu")
    with pytest.raises(ValueError):
        sq.sq_route(f(4, 8, t=torch.float32), 2, f(4, 3, t=torch.int32), f(4, 2, t=torch.float32))
    with pytest.raises(TypeError):
        sq.sq_moe_dispatch(f(4, 2, t=torch.int64), 8, f(9, t=torch.int32), f(4, 2, t=torch.int32))
    with pytest.raises(TypeError):
        sq.sq_prepare_weights_fp8b(f(4, 64, t=torch.float32), f(4, 128, t=torch.uint8), f(1, 4, t=torch.float32))


# ------------------------------------------------------------------ pins of the plain statements
E4M3 = sorted({Fraction(m, 8) * Fraction(2) ** (e - 7) if e == 0 else (1 + Fraction(m, 8)) * Fraction(2) ** (e - 7)
               for e in range(1, 16) for m in range(8) if not (e == 15 and m == 7)} |
              {Fraction(m, 8) * Fraction(2) ** -6 for m in range(8)})


def test_ref_encoding_is_the_nearest_value():
    assert E4M3[-1] == 448 and E4M3[1] == Fraction(1, 512)
    g = torch.Generator().manual_seed(0)
    q = torch.cat([torch.randn(300, generator=g) * 100, torch.randn(300, generator=g) * 0.01,
                   torch.tensor([0.0, 448.0, 447.9, 2.0 ** -10, 3 * 2.0 ** -10, 1.0625, 1.1875])]).clamp(-448, 448)
    got = ref.decode(ref.encode(q))
    for v, d in zip(q.tolist(), got.tolist()):
        want = min(E4M3, key=lambda c: (abs(c - Fraction(abs(v))), E4M3.index(c) % 2))
        assert Fraction(abs(d)) == want, (v, d)


def test_ref_blocks():
    """One outlier raises the step of its own block only; what a scale covers is what it is stored beside."""
    x = torch.ones(2, 300, dtype=torch.bfloat16) * 0.7
    x[1, 130] = 1000
    c, s = ref.quant_rows(x)
    assert c.shape == (2, 384) and s.shape == (2, 4) and s[0, 3] == 0 and bool((c[:, 300:] == 0).all())
    back = ref.rows64(c, s)[:, :300]
    assert bool(((back - x.double()).abs() <= 2.0 ** -4 * x.double().abs() + 2.0 ** -10 * s[1, 1].double()).all())
    assert bool((back[1, :128] == back[0, :128]).all()) and s[1, 1] == torch.tensor(1000.0) / 448
    w = torch.ones(200, 136, dtype=torch.bfloat16)
    w[150, 3] = 448
    c, s = ref.quant_weights(w)
    assert torch.allclose(s[:, :2], torch.tensor([[1 / 448, 1 / 448], [1.0, 1 / 448]]), rtol=2.0 ** -23, atol=0)
    assert bool((ref.weights64(c, s)[:, :136] - w.double()).abs().max() < 1e-6)


def test_ref_dispatch_and_route_by_hand():
    off, pos = ref.dispatch(torch.tensor([[2, 0], [0, -1], [2, 2]]), 3)
    assert off.tolist() == [0, 2, 2, 5] and pos.tolist() == [[2, 0], [1, -1], [3, 4]]
    l = torch.log(torch.tensor([[1.0, 2.0, 5.0, 2.0]]))
    ids, w = ref.route(l, 2)
    assert ids.tolist() == [[2, 1]] and torch.allclose(w, torch.tensor([[5 / 7, 2 / 7]], dtype=torch.float64))
    ids, w = ref.route(l, 2, bias=torch.tensor([1.0, 0, 0, 0]), renormalize=False)
    assert ids.tolist() == [[0, 2]] and torch.allclose(w, torch.tensor([[0.1, 0.5]], dtype=torch.float64))
    ids, _ = ref.route(l, 2, groups=2, keep_groups=1, group_top=2)
    assert ids.tolist() == [[2, 3]]


@pytest.mark.parametrize("shape", [(4, 64, 2, 136), (4, 2, 136, 64), (4, 136, 128), (4, 64, 136), (8, 64, 136), (4 * 2, 64, 136)])
def test_experts_refuse_other_layouts_of_gate_up(shape):
    """Gate and up rows interleaved, or a matrix turned: as many entries, but not the layout that is meant."""
    with pytest.raises(ValueError, match="gate_up: expected"):
        sq.SQExperts(torch.empty(shape, dtype=torch.bfloat16), torch.empty(4, 136, 64, dtype=torch.bfloat16), 2)
