"""Host-side checks of activations in 8 bits and of the matrix product: what the C calls refuse before they touch a GPU, and
pins of their oracle (oracle/k2_linear.py).  No GPU is needed."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import k2_linear as L
from oracle.k2_fp8 import E4M3_VALUES


@pytest.fixture(scope="module")
def k2():
    from dense_gqa_decoder_gb300 import build
    build.build()
    from dense_gqa_decoder_gb300 import k2 as mod
    return mod


# addresses far apart that no refused call reads
X, C8, SC, R, RO, G, W, O = (0x1000000 * i for i in range(1, 9))


def quantize(k2, **kw):
    d = dict(x=X, x_dtype=k2.K2_BF16, x_stride=64, tokens=4, cols=64, codes=C8, codes_stride=64, scales=SC)
    d.update(kw)
    a = k2.RowArgs(**d)
    return k2.LIB.k2_quantize_rows(ctypes.addressof(a), None)


@pytest.mark.parametrize("kw,why", [
    (dict(x=None), "ARG"), (dict(codes=None), "ARG"), (dict(scales=None), "ARG"), (dict(x_dtype=3), "UNSUPPORTED"),
    (dict(x_dtype=9), "UNSUPPORTED"),
    (dict(tokens=-1), "SHAPE"), (dict(cols=0), "SHAPE"), (dict(cols=49153, x_stride=49153, codes_stride=49153), "SHAPE"),
    (dict(tokens=2 ** 30 + 1), "SHAPE"),
    (dict(x_stride=63), "ARG"), (dict(codes_stride=63), "ARG"), (dict(x_stride=-64), "ARG"), (dict(x_stride=2 ** 62), "ARG"),
    (dict(x=X + 1), "ARG"),
    (dict(scales=SC + 2), "ARG"), (dict(codes=X), "ARG"), (dict(codes=X + 200), "ARG"), (dict(scales=X + 64), "ARG"),
    (dict(scales=C8 + 128), "ARG"),
    (dict(residual=R), "ARG"), (dict(gain=G), "ARG"), (dict(tokens=0), None),
    (dict(tokens=0, x=None, codes=None, scales=None), None)])
def test_rows_that_are_refused(k2, kw, why):
    assert quantize(k2, **kw) == (k2.K2_OK if why is None else getattr(k2, "K2_ERR_" + why))
    if why:
        assert k2.LIB.k2_last_error(None).decode() != ""


def norm(k2, **kw):
    d = dict(x=X, x_dtype=k2.K2_F32, x_stride=64, residual=R, residual_stride=64, residual_out=RO, residual_out_stride=64,
             residual_dtype=k2.K2_BF16, gain=G, gain_dtype=k2.K2_BF16, tokens=4, cols=64, groups=2, eps=1e-6, codes=C8, codes_stride=64,
             scales=SC)
    d.update(kw)
    a = k2.RowArgs(**d)
    return k2.LIB.k2_norm_quantize(ctypes.addressof(a), None)


@pytest.mark.parametrize("kw,why", [
    (dict(x=None), "ARG"), (dict(gain=None), "ARG"), (dict(residual=None), "ARG"), (dict(residual_out=None), "ARG"),
    (dict(residual_dtype=4), "UNSUPPORTED"),
    (dict(gain_dtype=3), "UNSUPPORTED"), (dict(groups=0), "SHAPE"), (dict(groups=3), "SHAPE"), (dict(eps=0.0), "ARG"),
    (dict(eps=-1e-6), "ARG"),
    (dict(eps=float("nan")), "ARG"), (dict(eps=float("inf")), "ARG"), (dict(residual_stride=63), "ARG"),
    (dict(residual_out_stride=63), "ARG"), (dict(residual=R + 1), "ARG"),
    (dict(gain=G + 1), "ARG"), (dict(residual_out=R + 128), "ARG"), (dict(residual_out=R, residual_out_stride=128), "ARG"),
    (dict(residual_out=X), "ARG"), (dict(codes=R), "ARG"),
    (dict(codes=G), "ARG"), (dict(residual_out=G), "ARG"), (dict(scales=RO + 4), "ARG"), (dict(scales=R), "ARG"),
    (dict(residual_out=C8 + 64), "ARG"), (dict(tokens=0), None)])
def test_norms_that_are_refused(k2, kw, why):
    assert norm(k2, **kw) == (k2.K2_OK if why is None else getattr(k2, "K2_ERR_" + why))


def linear(k2, **kw):
    d = dict(w=W, w_stride=64, w_scale=G, x=X, x_stride=64, x_scale=SC, out=O, out_stride=32, tokens=4, out_features=32, in_features=64,
             dtype=k2.K2_F8, out_dtype=k2.K2_F32, activation=0)
    d.update(kw)
    a = k2.LinearArgs(**d)
    return k2.LIB.k2_linear(ctypes.addressof(a), None)


@pytest.mark.parametrize("kw,why", [
    (dict(w=None), "ARG"), (dict(x=None), "ARG"), (dict(out=None), "ARG"), (dict(w_scale=None), "ARG"), (dict(x_scale=None), "ARG"),
    (dict(dtype=0), "UNSUPPORTED"), (dict(dtype=3), "UNSUPPORTED"), (dict(dtype=1), "ARG"), (dict(out_dtype=4), "UNSUPPORTED"),
    (dict(activation=6), "ARG"), (dict(activation=-1), "ARG"), (dict(activation=5, out_features=31), "SHAPE"), (dict(tokens=-1), "SHAPE"),
    (dict(tokens=2 ** 22 + 1), "SHAPE"), (dict(out_features=0), "SHAPE"), (dict(in_features=0), "SHAPE"),
    (dict(out_features=2 ** 24 + 1), "SHAPE"), (dict(w_stride=63), "ARG"), (dict(x_stride=48), "ARG"), (dict(x_stride=72), "ARG"),
    (dict(w_stride=2 ** 50), "ARG"), (dict(out_stride=31), "ARG"), (dict(residual=R, residual_stride=31), "ARG"), (dict(w=W + 8), "ARG"),
    (dict(x=X + 4), "ARG"), (dict(out=O + 2), "ARG"), (dict(residual=R + 2, residual_stride=32), "ARG"), (dict(w_scale=G + 2), "ARG"),
    (dict(bias=G + 1), "ARG"), (dict(flags=G + 1), "ARG"), (dict(wait_limit_us=-1), "ARG"), (dict(wait_limit_us=1000001), "ARG"),
    (dict(out=X), "ARG"), (dict(out=W + 64), "ARG"), (dict(out=SC), "ARG"), (dict(out=G + 4), "ARG"), (dict(bias=O), "ARG"),
    (dict(residual=O, residual_stride=64), "ARG"), (dict(residual=O + 4, residual_stride=32), "ARG"), (dict(tokens=0), None),
    (dict(tokens=0, x=None, out=None), None)])
def test_products_that_are_refused(k2, kw, why):
    assert linear(k2, **kw) == (k2.K2_OK if why is None else getattr(k2, "K2_ERR_" + why))


def test_null_arguments_are_refused(k2):
    assert k2.LIB.k2_quantize_rows(None, None) == k2.K2_ERR_ARG
    assert k2.LIB.k2_norm_quantize(None, None) == k2.K2_ERR_ARG
    assert k2.LIB.k2_linear(None, None) == k2.K2_ERR_ARG


def test_a_cpu_tensor_is_refused_by_the_binding(k2):
    x = torch.zeros(2, 32)
    with pytest.raises(Exception):
        k2.quantize_rows(x, torch.zeros(2, 32, dtype=torch.uint8), torch.zeros(2))


# ---- pins of the oracle -------------------------------------------------------------------------------------------------

def test_codes_agree_with_torchs_conversion():
    gen = np.random.default_rng(5)
    x = (gen.standard_normal((7, 301)) * np.exp(gen.standard_normal((7, 1)) * 3)).astype(np.float32)
    codes, scale = L.encode_rows(x)
    want = torch.tensor(x / scale[:, None]).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert (codes == want).all() and (np.abs(E4M3_VALUES[codes]).max(1) == 448).all()


def test_rows_without_a_scale():
    x = np.array([[0, -0.0, 0], [1, np.nan, 2], [np.inf, 1, 2], [1e-45, 0, 0]], np.float32)
    codes, scale = L.encode_rows(x)
    assert (codes[0] == 0).all() and scale[0] == 0 and (codes[1:3] == 0x7F).all() and np.isnan(scale[1:3]).all()
    assert scale[3] == 0 and (codes[3] == 0).all()


def test_norm_and_product_agree_with_torch_in_64_bits():
    gen = torch.Generator().manual_seed(6)
    x, r, g = (torch.randn(s, generator=gen) for s in ((5, 24), (5, 24), (24,)))
    h, y = L.norm_rows(x.numpy(), r.numpy(), g.numpy(), 3, 1e-6)
    d = torch.tensor(h).double().view(5, 3, 8)
    want = torch.nn.functional.rms_norm(d, (8,), eps=float(np.float32(1e-6))).reshape(5, 24) * g.double()
    assert np.allclose(y, want.numpy(), rtol=1e-14)
    w, b = torch.randn(6, 24, generator=gen).double(), torch.randn(6, generator=gen).double()
    z = torch.nn.functional.linear(x.double(), w, b)
    f = torch.nn.functional
    for kind, fn in (("none", lambda v: v), ("relu", f.relu), ("silu", f.silu), ("gelu", f.gelu),
                     ("gelu_tanh", lambda v: f.gelu(v, approximate="tanh")), ("swiglu", lambda v: f.silu(v[:, 0::2]) * v[:, 1::2])):
        got, off = L.linear(w.numpy(), x.numpy(), bias=b.numpy(), activation=kind)
        assert np.allclose(got, fn(z).numpy(), rtol=1e-13, atol=1e-15) and (off >= 0).all() and off.max() < 1e-5 * (1 + z.abs().max()) ** 2
