"""Pins of oracle.decode: the number formats against torch's own E4M3 and hand-written E2M1 values, the
NVFP4 cache rule against oracle.activation_fake_quant, weights against oracle.dequantize, and attention
and the norm against plain torch float64 expressions."""
import numpy as np
import torch

import oracle
from oracle import decode


def test_e4m3_values_and_codes_match_torch():
    b = torch.arange(256, dtype=torch.uint8)
    ref = b.view(torch.float8_e4m3fn).double().numpy()
    got = decode.e4m3_values(b.numpy())
    assert np.array_equal(got, ref, equal_nan=True)
    fin = ~np.isnan(ref)
    assert np.array_equal(np.signbit(got[fin]), np.signbit(ref[fin]))
    x = np.random.default_rng(0).standard_normal(4000) * np.exp2(np.random.default_rng(1).integers(-12, 9, 4000))
    x = np.concatenate([x, ref[fin], (np.sort(ref[fin])[1:] + np.sort(ref[fin])[:-1]) / 2]).clip(-448, 448)
    want = torch.from_numpy(x.astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(decode.e4m3_codes(x.astype(np.float32)), want)
    assert decode.e4m3_codes([1e6, -1e6]).tolist() == [126, 254]


def test_e2m1_values():
    assert decode.e2m1_values(np.array([0x10, 0x32, 0x54, 0x76])).tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    assert decode.e2m1_values(np.array([0x98, 0xFE])).tolist() == [0, -0.5, -4, -6]


def test_weights_are_dequantize_before_its_rounding():
    r = np.random.default_rng(2)
    code = r.integers(1, 127, (1, 5, 4)).astype(np.uint8)
    fp4 = r.integers(0, 256, (1, 5, 32)).astype(np.uint8)
    ref, _ = oracle.dequantize(code, fp4, np.array([0.37]), bf16=False, norm=256.0)
    got = decode.weights(code[0], fp4[0], 0.37, 256.0)
    assert np.abs(got - ref[0]).max() <= np.abs(got).max() * 2.0 ** -23


def test_cache_rule_is_the_input_quantizers_where_the_unit_is():
    """amax = 2688 * 2^k makes amax * fp32(1/2688) and fp32(amax / 2688) the same power of two."""
    x = np.random.default_rng(3).standard_normal((40, 1, 64)).astype(np.float32).astype(np.float64)
    for amax in (2688.0 / 1024, 2688.0 / 512):
        assert decode.cache_unit([amax], True)[0] == amax / 2688.0
        codes, scales = decode.cache_codes(x, [amax], True)
        ref = oracle.activation_fake_quant(x[:, 0], np.array([amax]), np.array([0, 40]), bf16=False)
        assert np.array_equal(decode.cache_values(codes, scales, [amax], True)[:, 0], ref)


def test_e4m3_cache_holds_every_value_it_can():
    vals = decode.e4m3_values(np.arange(127))
    x = np.concatenate([vals, -vals, [0.0, 500.0]]).reshape(1, 1, 256)
    codes, _ = decode.cache_codes(x, [448.0], False)
    assert decode.cache_unit([448.0], False)[0] == 1.0
    assert np.array_equal(decode.cache_values(codes, None, [448.0], False), np.minimum(x, 448.0))
    zero, _ = decode.cache_codes(-x, [0.0], False)
    assert np.array_equal(zero & 127, np.zeros_like(zero))


def test_norm_and_attention_against_torch():
    g = torch.Generator().manual_seed(4)
    h, gamma = torch.randn(3, 160, generator=g, dtype=torch.float64), torch.rand(160, generator=g, dtype=torch.float64)
    y, s = decode.rms_norm(h.numpy(), gamma.numpy(), 1e-6, 128)
    ref = torch.nn.functional.rms_norm(h, (160,), gamma, 1e-6)
    assert np.allclose(y, ref.numpy(), rtol=1e-12, atol=0)
    assert np.allclose(s * 448, np.stack([ref[:, :128].abs().amax(1), ref[:, 128:].abs().amax(1)], 1), rtol=1e-12)
    assert np.array_equal(decode.rms_norm(np.zeros((1, 32)), np.ones(32), 0.0, 0)[0], np.zeros((1, 32)))
    q, k, v = (torch.randn(*n, generator=g, dtype=torch.float64) for n in ((16,), (9, 16), (9, 16)))
    o, mag, _ = decode.attention(q.numpy(), k.numpy(), v.numpy(), 0.3)
    p = torch.softmax(k @ q * 0.3, 0)
    assert np.allclose(o, (p @ v).numpy(), rtol=1e-12) and np.allclose(mag, (p @ v.abs()).numpy(), rtol=1e-12)
    assert np.array_equal(decode.attention(q.numpy(), k.numpy()[:0], v.numpy()[:0], 1.0)[0], np.zeros(16))
