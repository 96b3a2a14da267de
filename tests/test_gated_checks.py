"""What the binding of the gated block's calls refuses by itself, before the library sees it.  Runs
where no GPU is visible: a check that failed would end at the library's own."""
import os

import pytest

from tensor_transformer_mlp_03_amd import _lib as L

torch = pytest.importorskip("torch")
pytestmark = [
    pytest.mark.skipif(not os.path.exists(L.LIB_PATH), reason="libtpmlp.so not built"),
    pytest.mark.skipif(torch.cuda.device_count() > 0, reason="tensors in host memory are only passed where no GPU is visible"),
]
BF16, F32, U8 = torch.bfloat16, torch.float32, torch.uint8


def z(*shape, dtype=BF16):
    return torch.zeros(*shape, dtype=dtype)


def byte_types(*but):
    names = ("int8", "bool", "float8_e5m2", "float8_e4m3fn", "float8_e4m3fnuz", "float8_e5m2fnuz", "float8_e8m0fnu", "float4_e2m1fn_x2")
    return [getattr(torch, n) for n in names if hasattr(torch, n) and n not in but]


def as_type(t, dtype):
    """A tensor of one-byte values with another type of one byte."""
    return t.view(dtype) if dtype != torch.bool else torch.zeros(t.shape, dtype=dtype)


def fp4(X, xs):
    return L.tpmlp_fp4_fwd(X, xs, z(1088, dtype=U8), z(5, 9), stream=0)


def edge8(codes, scales):
    from tensor_transformer_mlp_03_amd.block import Edge
    Edge(64, pre="rms", w_pre=z(64)).forward_fp8(None, z(5, 64), None, codes, scales, stream=0)


def test_other_one_byte_types_are_refused():
    """A type of one byte that is not the format's would be read as if it were."""
    x, mx, w4, ws = z(5, 64, dtype=U8), z(5, 2, dtype=U8), z(9, 32, dtype=U8), z(9, 2, dtype=U8)
    for t in byte_types("float8_e4m3fn"):
        with pytest.raises(TypeError, match="X must hold one-byte values, E4M3"):
            fp4(as_type(x, t), torch.zeros(5))
        with pytest.raises(TypeError, match="codes must hold one-byte values, E4M3"):
            edge8(as_type(x, t), torch.zeros(5))
    for t in byte_types("float8_e8m0fnu"):
        with pytest.raises(TypeError, match="x_scales must hold one-byte values, E8M0"):
            fp4(x, as_type(mx, t))
        with pytest.raises(TypeError, match="scales must hold one-byte values, E8M0"):
            edge8(x, as_type(mx, t))
        with pytest.raises(TypeError, match="scales must hold one-byte values, E8M0"):
            L.tpmlp_fp4_pack(w4, as_type(ws, t), z(1088, dtype=U8))
        with pytest.raises(TypeError, match="scales must hold one-byte values, E8M0"):
            L.tpmlp_fp4_quantize(z(64, 9), w4, as_type(ws, t))
    for t in byte_types("float4_e2m1fn_x2"):
        with pytest.raises(TypeError, match="codes must hold one-byte values, E2M1"):
            L.tpmlp_fp4_pack(as_type(w4, t), ws, z(1088, dtype=U8))
        with pytest.raises(TypeError, match="codes must hold one-byte values, E2M1"):
            L.tpmlp_fp4_quantize(z(64, 9), as_type(w4, t), ws)


def test_the_formats_own_types_are_taken():
    """They pass the binding's checks and end at the library's, which refuses for want of a GPU or for the address."""
    own = lambda t, n: [t] + ([t.view(getattr(torch, n))] if hasattr(torch, n) else [])  # noqa: E731
    for x in own(z(5, 64, dtype=U8), "float8_e4m3fn"):
        for xs in (torch.zeros(5), *own(z(5, 2, dtype=U8), "float8_e8m0fnu")):
            for call in (fp4, edge8):
                with pytest.raises(L.TpmlpError):
                    call(x, xs)
    for c in own(z(9, 32, dtype=U8), "float4_e2m1fn_x2"):
        for s in own(z(9, 2, dtype=U8), "float8_e8m0fnu"):
            with pytest.raises(L.TpmlpError):
                L.tpmlp_fp4_pack(c, s, z(1088, dtype=U8), stream=0)
            with pytest.raises(L.TpmlpError):
                L.tpmlp_fp4_quantize(z(64, 9), c, s, stream=0)


def test_unknown_activations_are_named():
    """By the calls themselves, as by the objects."""
    X, A, B, P = z(5, 64), z(64, 80), z(40, 64), z(5, 80)
    for act in ("tanh", None):
        with pytest.raises(ValueError, match="no activation"):
            L.tpmlp_glu_fwd(X, A, B, z(5, 64), P, act, None)
        with pytest.raises(ValueError, match="no activation"):
            L.tpmlp_glu_bwd(X, X, A, B, P, z(5, 64), z(64, 80), z(40, 64), act, None)
        with pytest.raises(ValueError, match="no activation"):
            L.tpmlp_fp4_fwd(X, None, z(1088, dtype=U8), z(5, 9), act)


def test_first_rows_past_64_bits_are_refused():
    """They would reach the library as their low bits."""
    y, state = z(5, 64), torch.zeros(2, dtype=torch.int64)
    for first in (1 << 64, (1 << 64) + 8, -(1 << 64), -1, (1 << 32) + 1):
        with pytest.raises(ValueError, match="first_row"):
            L.tpmlp_dropout_fwd(y, None, None, z(5, 64), 0.1, state, first_row=first, stream=0)
        with pytest.raises(ValueError, match="first_row"):
            L.tpmlp_dropout_bwd(y, z(5, 64), None, 0.1, state, first_row=first, stream=0)
    with pytest.raises(L.TpmlpError, match="first_row"):  # the library counts the rows behind it
        L.tpmlp_dropout_fwd(y, None, None, z(5, 64), 0.1, state, first_row=1 << 32, stream=0)
