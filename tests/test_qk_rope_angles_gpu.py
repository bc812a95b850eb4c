"""The rotation's angles, position times frequency, for positions and frequencies up to the
edges of what is documented, against whole-number arithmetic."""
import math

import numpy as np
import pytest

import paged_ref as ref

pytestmark = pytest.mark.gpu


def two_pi(bits):
    """2 pi 2^bits, rounded down, by pi = 16 arctan(1/5) - 4 arctan(1/239)."""
    def arctan(x):
        term = (1 << (bits + 20)) // x
        total, n = 0, 1
        while term:
            total += term // n if n % 4 == 1 else -(term // n)
            term //= x * x
            n += 2
        return total
    return (2 * (16 * arctan(5) - 4 * arctan(239))) >> 20


TURN = two_pi(300)


def cos_sin(p, f):
    """cos and sin of p f, the angle reduced exactly (f a float32 as a fraction)."""
    m, e = float(f).as_integer_ratio()
    x = ((abs(p) * m) << 300) // e  # |p f| 2^300
    angle = math.copysign((x % TURN) / 2 ** 300, p)
    return math.cos(angle), math.sin(angle)


@pytest.mark.parametrize("rotary", [16, 64])
@pytest.mark.parametrize("interleaved", [False, True])
def test_far_positions_and_high_frequencies(rotary, interleaved):
    import torch
    import transformer_head_scaled_mha_gb300 as mha
    rng = np.random.default_rng(rotary)
    d, H = 64, 2
    edges = [0, 1, -1, 2, 1000, 2 ** 24 + 1, -(2 ** 24) - 1, 2 ** 31 - 1, -2 ** 31, 2 ** 30 + 12345]
    pos = np.concatenate([edges, rng.integers(-2 ** 31, 2 ** 31, 30)]).astype(np.int32)
    half = rotary // 2
    for freq in (np.float32(2.0) ** rng.uniform(-12, 20, half).astype(np.float32),
                 np.nextafter(np.float32(2 ** 20), np.float32(0)) - np.arange(half, dtype=np.float32),
                 -np.float32(2.0) ** rng.uniform(0, 20, half).astype(np.float32),
                 np.float32(2.0) ** np.linspace(-149, -60, half).astype(np.float32)):
        freq = np.clip(freq, -1048575.0, 1048575.0).astype(np.float32)
        x = rng.normal(size=(1, len(pos), H, d)).astype(np.float32)
        out, _ = mha.mha_qk_norm_rope_fwd(
            torch.from_numpy(x).cuda(), None, positions=torch.from_numpy(pos[None]).cuda(),
            inv_freq=torch.from_numpy(freq).cuda(), layout="bshd", interleaved=interleaved)
        got = out.double().cpu().numpy()
        cs = np.array([[cos_sin(int(p), f) for f in freq] for p in pos])[None, :, None]
        c, s = cs[..., 0], cs[..., 1]
        x = x.astype(np.float64)
        want = x.copy()
        ia = np.arange(0, rotary, 2) if interleaved else np.arange(half)
        ib = ia + 1 if interleaved else ia + half
        want[..., ia] = x[..., ia] * c - x[..., ib] * s
        want[..., ib] = x[..., ia] * s + x[..., ib] * c
        # in half steps of fp32 (2^-24): the angle in turns is off by 2^-26 (fp32) + 2^-32 + 2^-33,
        # 1.6 in radians; cos and sin by 2; a product and a fused one by 1 each; the result by 1
        tol = 7 * ref.U * ref.pair_size(x, rotary, interleaved)
        bad = np.abs(got - want) > tol
        assert not bad.any(), (np.abs(got - want) / tol).max()
