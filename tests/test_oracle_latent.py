"""Pins of the latent oracle (CPU): the rotation against complex
multiplication, the pool forms against torch's own casts, the attention
against sums written out key by key."""
import math

import numpy as np
import torch

from oracle import latent as lo


def _table(n):
    inv = 10000.0 ** (-np.arange(0, 64, 2) / 64)
    ang = np.arange(n)[:, None] * inv
    return np.concatenate([np.cos(ang), np.sin(ang)], axis=1)


def test_rotation_is_a_complex_product():
    g = np.random.default_rng(1)
    x = g.normal(size=(5, 3, 64))
    pos = np.array([0, 1, 77, 1000, 5])
    inv = 10000.0 ** (-np.arange(0, 64, 2) / 64)
    turn = np.exp(1j * pos[:, None] * inv)[:, None, :]
    z = (x[..., 0::2] + 1j * x[..., 1::2]) * turn
    got = lo.rotate(x, _table(1001), pos, True)
    assert np.allclose(got[..., 0::2], z.real, atol=1e-12) and np.allclose(got[..., 1::2], z.imag, atol=1e-12)
    z = (x[..., :32] + 1j * x[..., 32:]) * turn
    got = lo.rotate(x, _table(1001), pos, False)
    assert np.allclose(got, np.concatenate([z.real, z.imag], axis=-1), atol=1e-12)
    assert np.allclose(lo.rotate(x, _table(1), np.zeros(5, int), True), x)
    assert np.allclose((got ** 2).sum(-1), (x ** 2).sum(-1))


def test_quantisation_matches_torchs_cast():
    g = torch.Generator().manual_seed(2)
    c = (torch.randn(40, 512, generator=g) * torch.logspace(-6, 3, 40)[:, None]).to(torch.bfloat16).float()
    c[3] = 0
    codes, s = lo.quantise(c.numpy())
    want_s = c.abs().amax(1).clamp_min(1e-4) / 448
    want = (c / want_s[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    assert np.array_equal(s, want_s.numpy()) and np.array_equal(codes, want.numpy())
    c[5, 7] = float("nan")
    codes, s = lo.quantise(c.numpy())
    assert np.isnan(s[5]) and not np.isnan(np.delete(s, 5)).any()


def test_attention_key_by_key():
    g = np.random.default_rng(3)
    q, k = g.normal(size=(2, 576)), g.normal(size=(5, 576))
    out, lse = lo.attend(q, k, 0.05)
    for i in range(2):
        w = [math.exp(0.05 * sum(float(a) * float(b) for a, b in zip(q[i], k[j]))) for j in range(5)]
        assert np.allclose(lse[i], math.log(sum(w)), rtol=1e-12)
        assert np.allclose(out[i], sum(w[j] * k[j, :512] for j in range(5)) / sum(w), rtol=1e-10, atol=1e-12)
    out, lse = lo.attend(q, k[:0], 0.05)
    assert not out.any() and np.isneginf(lse).all()
    one, l1 = lo.attend(q, k[:1], 0.05)
    assert np.allclose(one, np.broadcast_to(k[0, :512], (2, 512)))


def test_limits_cover_a_rounded_computation_and_catch_a_wrong_one():
    """The same sums with the weights rounded as a kernel rounds them stay
    inside; a key left out, a scale off by 1 % or a wrong column do not."""
    g = torch.Generator().manual_seed(4)
    q = torch.randn(4, 576, generator=g).to(torch.bfloat16).double().numpy()
    k = torch.randn(300, 576, generator=g).to(torch.bfloat16).double().numpy()
    scale = 192 ** -0.5
    out, lse = lo.attend(q, k, scale)
    for fp8, kind in ((False, torch.bfloat16), (True, torch.float16)):
        tol, ltol = lo.limits(q, k, scale, fp8)
        x = scale * (q @ k.T)
        m = x.max(1, keepdims=True) - (math.log(2 ** 7) if fp8 else 0)
        p = np.exp(x - m)
        w = torch.from_numpy(p).to(kind).double().numpy()
        got = torch.from_numpy(w @ k[:, :512] / p.sum(1, keepdims=True)).to(torch.bfloat16).double().numpy()
        assert (np.abs(got - out) <= tol).all()
        wrong, wl = lo.attend(q, np.delete(k, int(p[0].argmax()), axis=0), scale)
        assert (np.abs(wrong - out)[0] > tol[0]).any() and abs(wl[0] - lse[0]) > ltol[0]
        wrong, wl = lo.attend(q, k, 1.01 * scale)
        assert (np.abs(wl - lse) > ltol).all()
        assert (np.abs(out[[1, 0, 2, 3]] - out) > tol).any()


def test_pool_rows_as_keys():
    g = torch.Generator().manual_seed(5)
    c = torch.randn(6, 512, generator=g)
    codes, s = lo.quantise(c.numpy())
    pe = torch.randn(6, 64, generator=g).to(torch.bfloat16).double().numpy()
    k = lo.keys_of(codes, s, pe)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy() * s[:, None].astype(np.float64)
    assert np.array_equal(k[:, :512], want) and np.array_equal(k[:, 512:], pe)
